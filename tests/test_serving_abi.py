"""Refusals of the serving calls (no GPU: every call fails in a host check before any launch), their size
queries and the Python module that marshals their arguments."""

import ctypes

import numpy as np
import pytest
import torch

from mxfp4_w4a4_post_block_b200 import _lib
from mxfp4_w4a4_post_block_b200 import batq as BQ
import serving_ref as R

INVALID, SHAPE, ALIGN, WORKSPACE = (_lib.BATQ_ERR_INVALID_ARG, _lib.BATQ_ERR_SHAPE, _lib.BATQ_ERR_ALIGNMENT,
                                    _lib.BATQ_ERR_WORKSPACE)
FAKE = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def L():
    from mxfp4_w4a4_post_block_b200 import build
    build.build()
    return _lib.load()


def refused(fn, args, cases):
    """Each case is (position, value, status): args with that one argument changed."""
    for i, v, want in cases:
        a = list(args)
        a[i] = v
        assert fn(*a) == want, (i, v)


A = np.eye(8, dtype=np.float32)


def test_linear_w4a16_refusals(L):
    #       X  type S  N  ldx  A              B    fmt codes scales gs   M  type out  ldo stream
    args = [FAKE, 1, 4, 256, 256, A.ctypes.data, FAKE, 0, FAKE, FAKE, None, 128, 0, FAKE, 128, None]
    refused(L.batq_linear_w4a16, args, [
        (0, None, INVALID), (8, None, INVALID), (9, None, INVALID), (13, None, INVALID), (1, 7, INVALID),
        (12, 7, INVALID), (7, 2, INVALID), (5, None, INVALID), (6, None, INVALID), (10, FAKE, INVALID),
        (2, 0, SHAPE), (2, 17, SHAPE), (3, 250, SHAPE), (3, 0, SHAPE), (3, 131136, SHAPE), (4, 255, SHAPE),
        (11, 100, SHAPE), (11, 0, SHAPE), (14, 127, SHAPE), (0, FAKE + 2, ALIGN), (4, 260, ALIGN), (14, 130, ALIGN),
        (6, FAKE + 4, ALIGN), (8, FAKE + 8, ALIGN), (9, FAKE + 8, ALIGN), (13, FAKE + 4, ALIGN)])
    for fmt, most in ((0, 98304), (1, 49152)):
        wide = list(args)
        wide[7], wide[3], wide[4] = fmt, most + 64, most + 64
        assert L.batq_linear_w4a16(*wide) == SHAPE
        wide[3], wide[8] = most, FAKE + 8  # as far as the next refusal
        assert L.batq_linear_w4a16(*wide) == ALIGN
    nv = list(args)
    nv[7], nv[10] = 1, FAKE + 2
    assert L.batq_linear_w4a16(*nv) == ALIGN


def kv8_tail(L, args, at):
    """The refusals that the cache's writer and reader share; `at` maps names to positions."""
    p = at
    return [(p["lens"], None, INVALID), (p["table"], None, INVALID), (p["kc"], None, INVALID), (p["ks"], None, INVALID),
            (p["vc"], None, INVALID), (p["vs"], None, INVALID), (p["T"], 0, SHAPE), (p["heads"], 0, SHAPE),
            (p["heads"], 1025, SHAPE), (p["dim"], 96, SHAPE), (p["dim"], 0, SHAPE), (p["batch"], 0, SHAPE),
            (p["batch"], 65536, SHAPE), (p["max_pages"], 0, SHAPE), (p["max_pages"], 1 << 28, SHAPE),
            (p["pages"], 0, SHAPE), (p["pages"], 1 << 27, SHAPE), (p["page"], 8, SHAPE), (p["page"], 48, SHAPE),
            (p["page"], 256, SHAPE), (p["kc"], FAKE + 8, ALIGN), (p["vc"], FAKE + 8, ALIGN), (p["lens"], FAKE + 2, ALIGN),
            (p["table"], FAKE + 2, ALIGN), (p["cu"], FAKE + 1, ALIGN)]


def test_kv8_append_refusals(L):
    #       K     V  type T heads dim ldk ldv  cu   lens  table B max_pages pages page  kc    ks    vc    vs  stream
    args = [FAKE, FAKE, 1, 9, 2, 64, 128, 128, FAKE, FAKE, FAKE, 3, 4, 20, 16, FAKE, FAKE, FAKE, FAKE, None]
    at = dict(T=3, heads=4, dim=5, cu=8, lens=9, table=10, batch=11, max_pages=12, pages=13, page=14, kc=15, ks=16, vc=17,
              vs=18)
    refused(L.batq_kv8_append, args, kv8_tail(L, args, at) + [
        (0, None, INVALID), (1, None, INVALID), (2, 5, INVALID), (6, 127, SHAPE), (7, 127, SHAPE), (6, 130, ALIGN),
        (7, 130, ALIGN), (0, FAKE + 4, ALIGN), (1, FAKE + 4, ALIGN)])
    few = list(args)
    few[8], few[3] = None, 2  # one row per sequence, and fewer rows
    assert L.batq_kv8_append(*few) == SHAPE


def test_attn_kv8_refusals(L):
    #       Q    type T ldq qh heads dim cu   lens  table B max_pages pages page kc    ks    vc    vs   scale max_q ws  bytes
    args = [FAKE, 1, 9, 512, 8, 2, 64, FAKE, FAKE, FAKE, 3, 4, 20, 16, FAKE, FAKE, FAKE, FAKE, 0.125, 4, FAKE, 1 << 30,
            1, FAKE, 512, None, None]  # type out ldo lse stream
    at = dict(T=2, heads=5, dim=6, cu=7, lens=8, table=9, batch=10, max_pages=11, pages=12, page=13, kc=14, ks=15, vc=16,
              vs=17)
    cases = [c for c in kv8_tail(L, args, at)]
    refused(L.batq_attn_kv8, args, cases + [
        (0, None, INVALID), (20, None, INVALID), (23, None, INVALID), (1, 4, INVALID), (22, 4, INVALID),
        (18, float("nan"), INVALID), (18, float("inf"), INVALID), (4, 7, SHAPE), (4, 0, SHAPE), (19, 0, SHAPE),
        (3, 511, SHAPE), (24, 511, SHAPE), (3, 516, ALIGN), (24, 516, ALIGN), (0, FAKE + 2, ALIGN), (23, FAKE + 2, ALIGN),
        (20, FAKE + 8, ALIGN), (25, FAKE + 2, ALIGN), (21, 1000, WORKSPACE)])
    big = list(args)
    big[11], big[19] = 1 << 26, 1 << 20  # more work units than 32 bits count
    assert L.batq_attn_kv8(*big) == SHAPE


def test_attn_kv8_workspace_size(L):
    b = ctypes.c_size_t()
    f = L.batq_attn_kv8_workspace_size
    assert f(1, 32, 8, 128, ctypes.byref(b)) == 0 and 0 < b.value <= 64 << 20
    small = b.value
    assert f(8, 32, 8, 128, ctypes.byref(b)) == 0 and small < b.value <= 64 << 20
    assert f(1000, 32, 1, 256, ctypes.byref(b)) == 0 and b.value <= 64 << 20  # bounded, whatever the queries
    for args in ((0, 32, 8, 128), (1, 30, 8, 128), (1, 8, 0, 128), (1, 8, 8, 100), (1 << 20, 1 << 20, 1, 64)):
        assert f(*args, ctypes.byref(b)) == SHAPE
    assert f(1, 8, 8, 64, None) == INVALID


def test_gemm_mxfp4_experts_refusals(L):
    #       ac    as    wc    ws    off  E  T   M   N type out ldo stream
    args = [FAKE, FAKE, FAKE, FAKE, FAKE, 4, 30, 64, 256, 0, FAKE, 64, None]
    refused(L.batq_gemm_mxfp4_experts, args, [
        (0, None, INVALID), (1, None, INVALID), (2, None, INVALID), (3, None, INVALID), (4, None, INVALID),
        (10, None, INVALID), (9, 3, INVALID), (5, 0, SHAPE), (5, 513, SHAPE), (6, 0, SHAPE), (7, 20, SHAPE), (7, 0, SHAPE),
        (8, 32, SHAPE), (8, 100, SHAPE), (11, 63, SHAPE), (6, 1 << 29, SHAPE), (11, 66, ALIGN), (0, FAKE + 8, ALIGN),
        (1, FAKE + 8, ALIGN), (2, FAKE + 8, ALIGN), (3, FAKE + 8, ALIGN), (4, FAKE + 2, ALIGN), (10, FAKE + 8, ALIGN)])


def test_linear_experts_refusals(L):
    b = ctypes.c_size_t()
    assert L.batq_linear_experts_workspace_size(30, 256, ctypes.byref(b)) == 0
    assert b.value >= 30 * 128 + 30 * 8
    assert L.batq_linear_experts_workspace_size(30, 100, ctypes.byref(b)) == SHAPE
    assert L.batq_linear_experts_workspace_size(30, 256, None) == INVALID
    #       X  type T  N   ldx  A              B    ratios wc   ws    off  E  M  ws    bytes type out ldo stream
    args = [FAKE, 1, 30, 256, 256, A.ctypes.data, FAKE, None, FAKE, FAKE, FAKE, 4, 64, FAKE, 1 << 20, 0, FAKE, 64, None]
    refused(L.batq_linear_experts, args, [
        (13, None, INVALID), (14, 100, WORKSPACE), (13, FAKE + 8, ALIGN), (3, 100, SHAPE), (0, None, INVALID),
        (5, None, INVALID), (8, None, INVALID), (10, None, INVALID), (11, 513, SHAPE), (12, 20, SHAPE), (17, 66, ALIGN)])


def test_python_calls_refuse_cpu_tensors(L):
    x, u8, i32 = torch.zeros(2, 64), torch.zeros(4, dtype=torch.uint8), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError, match="CUDA tensor"):
        BQ.batq_linear_w4a16(x, None, None, u8, u8, 16, x)
    with pytest.raises(TypeError, match="CUDA tensor"):
        BQ.batq_kv8_append(x, x, None, i32, i32, u8, u8, u8, u8)
    with pytest.raises(TypeError, match="CUDA tensor"):
        BQ.batq_attn_kv8(x, None, i32, i32, u8, u8, u8, u8, 0.1, 1, u8, x)
    with pytest.raises(TypeError, match="CUDA tensor"):
        BQ.batq_gemm_mxfp4_experts(u8, u8, u8, u8, i32, 16, 64, x)
    with pytest.raises(TypeError, match="CUDA tensor"):
        BQ.batq_linear_experts(x, np.eye(8), None, None, u8, u8, i32, 16, u8, x)
    with pytest.raises(TypeError):
        BQ.batq_linear_w4a16(None, None, None, None, None, 16, None)
    assert BQ.batq_attn_kv8_workspace_size(1, 8, 2, 64) > 0 and BQ.batq_linear_experts_workspace_size(3, 64) > 0
    kc, ks, vc, vs = BQ.empty_kv8_cache(3, 2, 16, 64, device="cpu")
    assert kc.shape == vc.shape == (3, 2, 16, 64) and ks.shape == vs.shape == (3, 2)


# ------------------------------------------------------------------ the references themselves

def test_reference_formats():
    assert R.e4m3_value(0x7E) == 448 and R.e4m3_value(0x01) == 2.0 ** -9 and np.isnan(R.e4m3_value(0xFF))
    assert R.e8m0_value(127) == 1 and np.isnan(R.e8m0_value(255))
    v = R.e4m3_value(np.arange(127))
    mid = (v[:-1] + v[1:]) / 2
    np.testing.assert_array_equal(R.round_e4m3(mid), np.where(np.arange(126) % 2 == 0, v[:-1], v[1:]))  # ties to even
    np.testing.assert_array_equal(R.round_e4m3(v), v)
    assert R.block_exponent(448.0) == 0 and R.block_exponent(448.1) == 1 and R.block_exponent(0.0) == -127
    np.testing.assert_array_equal(R.e2m1_matrix(np.array([[0x10, 0xF7]], np.uint8)), [[0.0, 0.5, 6.0, -6.0]])


def test_reference_tile_layout_matches_the_oracle():
    from oracle import batq_oracle as O
    lin = np.random.default_rng(0).integers(0, 255, (200, 10)).astype(np.uint8)
    t = R.tile_scales(lin)
    np.testing.assert_array_equal(O.scales_from_mma_layout(t, 200, 10), lin)


def test_reference_attention_is_softmax():
    """Against torch in fp64, and its tolerance notices a token more or less."""
    rng = np.random.default_rng(0)
    page, D, G, heads = 16, 64, 2, 2
    k, v = rng.standard_normal((2, 4, heads, page, D))
    table = np.array([[2, 0, 1]], np.int32)
    q = rng.standard_normal((3, heads * G, D))
    out, lse, tol = R.attention(q, [0, 3], [41], table, page, k, v, np.ones((4, heads)), 0.125, 3)
    kk = k[table[0]].transpose(1, 0, 2, 3).reshape(heads, -1, D)[:, :41].repeat(G, 0)
    vv = v[table[0]].transpose(1, 0, 2, 3).reshape(heads, -1, D)[:, :41].repeat(G, 0)
    s = torch.einsum("nhd,hld->hnl", torch.from_numpy(q), torch.from_numpy(kk)) * 0.125
    s = s.masked_fill(torch.ones(3, 41, dtype=torch.bool).tril(38).logical_not(), float("-inf"))
    ref = torch.einsum("hnl,hld->nhd", torch.softmax(s, -1), torch.from_numpy(vv)).numpy()
    np.testing.assert_allclose(out, ref, rtol=0, atol=1e-12)
    np.testing.assert_allclose(lse.T, torch.logsumexp(s, -1).numpy(), rtol=0, atol=1e-12)
    less, _, _ = R.attention(q, [0, 3], [40], table, page, k, v, np.ones((4, heads)), 0.125, 3)
    assert (np.abs(less - out) > tol).mean() > 0.5


def test_reference_append_grows_scales():
    rng = np.random.default_rng(1)
    table = np.array([[1, 0]], np.int32)
    vals, exps = np.zeros((2, 1, 16, 4)), np.zeros((2, 1), np.int64)
    x = rng.uniform(-1, 1, (20, 1, 4))
    x[7] *= 1000
    R.append(x[:5], [0, 5], [5], table, 16, vals, exps)
    one = exps[1, 0]
    R.append(x[5:], [0, 15], [20], table, 16, vals, exps)
    assert exps[1, 0] > one
    got = (vals * np.exp2(exps)[:, :, None, None])[[1, 0]].reshape(-1, 4)[:20]
    step = np.exp2(np.array([exps[1, 0]] * 16 + [exps[0, 0]] * 4) - 9.0)[:, None]
    # half a step of 2^-3 relative, twice for codes that were rounded again, and half of the smallest step
    assert (np.abs(got - x[:, 0]) <= np.abs(x[:, 0]) * 2.0 ** -3 + step).all()


def test_attn_kv8_refuses_more_rows_than_a_grid_has(L):
    """Rows of the join's grid stay below 2^31 - 8, and are refused before anything is launched."""
    #       Q    type T          ldq qh heads dim cu   lens  table B max_pages pages page kc    ks    vc    vs   scale max_q
    args = [FAKE, 1, (1 << 31) - 1, 64, 1, 1, 64, FAKE, FAKE, FAKE, 1, 1, 20, 128, FAKE, FAKE, FAKE, FAKE, 0.125,
            (1 << 31) - 8, FAKE, 1 << 30, 1, FAKE, 64, None, None]
    assert L.batq_attn_kv8(*args) == SHAPE
    args[19], args[0] = (1 << 31) - 9, FAKE + 2  # as far as the next refusal
    assert L.batq_attn_kv8(*args) == ALIGN
