"""GPU parity of the serving operators (4-bit weight products of few tokens, 8-bit paged cache and its
attention, products grouped by expert) against their definitions in fp64."""

import numpy as np
import pytest
import torch

from mxfp4_w4a4_post_block_b200 import batq as BQ
import serving_ref as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def ok():
    assert BQ.batq_device_error() == 0


def host(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------ W4A16

def w4a16_case(S, N, M, fmt, x_dtype, tr, seed, x=None, lin=None):
    rng = np.random.default_rng(seed)
    codes, lin0 = R.random_weights(rng, M, N, fmt)
    lin = lin0 if lin is None else lin(lin0)
    x = torch.from_numpy((rng.standard_normal((S, N)) * np.exp(rng.standard_normal((S, 1)))).astype(np.float32)) if x is None else x
    x = x.to(x_dtype)
    A = (np.eye(8) + 0.1 * rng.standard_normal((8, 8))).astype(np.float32) if tr else None
    B = (np.eye(4) + 0.1 * rng.standard_normal((N // 32, 4, 4))).astype(np.float32) if tr else None
    return x, A, B, codes, lin, rng


def w4a16_run(x, A, B, codes, lin, fmt, out_dtype, gs=None):
    out = torch.full((x.shape[0], codes.shape[0]), 7.0, dtype=out_dtype, device="cuda")
    BQ.batq_linear_w4a16(x.cuda(), A, R.cuda(B) if B is not None else None, R.cuda(codes), R.cuda(R.tile_scales(lin)),
                         codes.shape[0], out, w_gs=gs,
                         w_format=BQ.BATQ_W4_MXFP4 if fmt == "mxfp4" else BQ.BATQ_W4_NVFP4)
    ok()
    return out


def w4a16_check(out, x, A, B, codes, lin, fmt, gs=1.0):
    N = x.shape[1]
    xd = x.double().numpy()
    y, cond = R.transform(xd, A, B) if A is not None else (xd, np.abs(xd))
    w = R.weights(codes, lin, fmt)
    ref = y @ w.T / gs
    # fp32 transform (12 roundings, half a step each).  y is rounded to a fixed-point number under its scale group's 2^e,
    # 2^e <= max |y|: half a step of 8^-4 2^e (bf16 out), or 8^-7 2^e, so 2^-13 or 2^-22 of the group's largest.  NVFP4's
    # 2^e is at least 2^-17 of that of a bound of the token's largest value, which lies at most 4 |A|_1 |B|_1 (here below
    # 2^5) above it: 2^-25 and 2^-34 of the largest.
    fine = out.dtype != BF
    G = 32 if fmt == "mxfp4" else 16
    top = np.repeat(np.abs(y).reshape(len(y), -1, G).max(2), G, axis=1)
    each = cond * (12 * 2.0 ** -24) + top * (2.0 ** -22 if fine else 2.0 ** -13)
    if fmt == "nvfp4":
        each = each + np.abs(y).max(1, keepdims=True) * (2.0 ** -33 if fine else 2.0 ** -24)
    # and one fp32 rounding (two half steps: the tensor core truncates) per 64 products, the digits' values adding
    # up to 2 |y| and their remainders
    tol = (each + np.abs(y) * ((N / 8 + 24) * 2.0 ** -23)) @ np.abs(w).T / gs
    tol += np.abs(ref) * (2.0 ** -8 if out.dtype == BF else 2.0 ** -23)
    err = np.abs(host(out) - ref)
    assert (err <= tol).all(), (err / np.maximum(tol, 1e-300)).max()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("S,N,M,x_dtype,out_dtype,tr", [
    (1, 64, 16, BF, F32, False), (1, 256, 128, F32, F32, True), (2, 320, 48, BF, BF, True), (3, 2112, 144, BF, F32, True),
    (4, 1024, 1040, F32, BF, False), (7, 4096, 96, BF, F32, False), (8, 512, 272, F32, F32, True),
    (13, 1088, 160, BF, F32, False), (16, 2048, 64, F32, F32, True), (16, 4160, 528, BF, BF, True),
])
def test_w4a16_shapes(S, N, M, x_dtype, out_dtype, tr, fmt):
    x, A, B, codes, lin, _ = w4a16_case(S, N, M, fmt, x_dtype, tr, S + N)
    w4a16_check(w4a16_run(x, A, B, codes, lin, fmt, out_dtype), x, A, B, codes, lin, fmt)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("S,N,tr", [(1, 32768, True), (16, 12288, True), (16, 20480, False), (9, 33024, True)])
def test_w4a16_long_rows_split_over_a_cluster(S, N, tr, fmt):
    x, A, B, codes, lin, _ = w4a16_case(S, N, 32, fmt, BF, tr, S + N)
    w4a16_check(w4a16_run(x, A, B, codes, lin, fmt, F32), x, A, B, codes, lin, fmt)


@pytest.mark.parametrize("S,N,M,x_dtype,out_dtype,tr,fmt", [
    (1, 98304, 16, BF, BF, True, "mxfp4"), (16, 98304, 32, BF, F32, False, "mxfp4"), (1, 49152, 48, F32, F32, False, "nvfp4"),
    (16, 49152, 16, BF, BF, True, "nvfp4"), (16, 28672, 4112, BF, BF, True, "mxfp4"), (9, 16384, 272, BF, F32, True, "nvfp4"),
    (5, 192, 37888, BF, BF, False, "mxfp4")])
def test_w4a16_largest_sizes(S, N, M, x_dtype, out_dtype, tr, fmt):
    """The longest rows, whose tokens go in groups; wide and flat weights; bit for bit twice."""
    x, A, B, codes, lin, _ = w4a16_case(S, N, M, fmt, x_dtype, tr, S + M)
    out = w4a16_run(x, A, B, codes, lin, fmt, out_dtype)
    w4a16_check(out, x, A, B, codes, lin, fmt)
    assert torch.equal(out, w4a16_run(x, A, B, codes, lin, fmt, out_dtype))


def test_w4a16_many_units_and_tensor_scale():
    x, A, B, codes, lin, _ = w4a16_case(2, 768, 24576, "nvfp4", BF, True, 5)
    gs = torch.tensor([37.5], device="cuda")
    w4a16_check(w4a16_run(x, A, B, codes, lin, "nvfp4", F32, gs), x, A, B, codes, lin, "nvfp4", 37.5)


def test_w4a16_equals_prepared_weights_of_the_library():
    """Weights of batq_prepare_weights: x P (W P^-T)^T is x W^T up to the weights' own rounding, and equals the
    product with the decoded codes."""
    rng = np.random.default_rng(3)
    M, N = 256, 512
    W = torch.from_numpy((rng.standard_normal((M, N)) * 0.02).astype(np.float32)).cuda()
    A = (np.eye(8) + 0.1 * rng.standard_normal((8, 8))).astype(np.float32)
    B = (np.eye(4) + 0.1 * rng.standard_normal((N // 32, 4, 4))).astype(np.float32)
    lin_codes, lin = BQ.empty_act_buffers(M, N, BQ.BATQ_SCALES_LINEAR)
    codes, scales = BQ.empty_act_buffers(M, N)
    ws = torch.empty(BQ.batq_prepare_workspace_size(N), dtype=torch.uint8, device="cuda")
    BQ.batq_prepare_weights(W, A, B, lin_codes, lin, ws, BQ.BATQ_SCALES_LINEAR)
    BQ.batq_prepare_weights(W, A, B, codes, scales, ws)
    x = torch.from_numpy(rng.standard_normal((3, N)).astype(np.float32))
    out = torch.empty(3, M, device="cuda")
    BQ.batq_linear_w4a16(x.cuda(), A, R.cuda(B), codes, scales, M, out)
    ok()
    w4a16_check(out, x, A, B, lin_codes.cpu().numpy(), lin.cpu().numpy().reshape(M, -1), "mxfp4")
    plain = host(x @ W.cpu().T.float())
    assert np.linalg.norm(host(out) - plain) < 0.2 * np.linalg.norm(plain)


@pytest.mark.parametrize("mag", [1e-38, 1e-30, 1e30])
@pytest.mark.parametrize("tr", [False, True])
def test_w4a16_magnitudes_of_tokens(mag, tr):
    """Tokens far from 1: normalisation is per token, so one does not disturb another."""
    x, A, B, codes, lin, rng = w4a16_case(4, 256, 64, "mxfp4", F32, tr, 8)
    x[1] *= mag
    x[2] = 0.0
    out = w4a16_run(x, A, B, codes, lin, "mxfp4", F32)
    assert (out[2] == 0).all()
    if mag < 1e-35:  # subnormal sums: absolute steps of 2^-149 and flushed terms
        keep = [0, 2, 3]
        assert torch.isfinite(out).all()
        w4a16_check(out[keep], x[keep], A, B, codes, lin, "mxfp4")
    else:
        w4a16_check(out, x, A, B, codes, lin, "mxfp4")


def test_w4a16_non_finite_values_stay_with_their_token_and_row():
    x, A, B, codes, lin, _ = w4a16_case(4, 256, 64, "mxfp4", BF, False, 9)
    clean = w4a16_run(x, A, B, codes, lin, "mxfp4", F32)
    x[1, 7], x[3, 200] = float("nan"), float("inf")
    lin[5, 3] = 255   # a weight row with a NaN scale
    lin[9, 2] = 0     # and one with the smallest scale
    out = w4a16_run(x, A, B, codes, lin, "mxfp4", F32)
    assert out[1].isnan().all() and not out[3].isfinite().any() and out[:, 5].isnan().all()
    same = [m for m in range(64) if m not in (5, 9)]
    assert torch.equal(out[0][same], clean[0][same]) and torch.equal(out[2][same], clean[2][same])
    w = R.weights(codes, lin, "mxfp4")
    assert abs(float(out[0, 9]) - float(x[0].double().numpy() @ w[9])) < 1e-4


def test_w4a16_strides_and_untouched_columns():
    x, A, B, codes, lin, rng = w4a16_case(5, 320, 48, "mxfp4", BF, True, 10)
    big = torch.full((5, 320 + 64), float("nan"), dtype=BF, device="cuda")
    big[:, 32:352] = x.cuda()
    out = torch.full((5, 64), 3.0, device="cuda")
    BQ.batq_linear_w4a16(big[:, 32:352], A, R.cuda(B), R.cuda(codes), R.cuda(R.tile_scales(lin)), 48, out[:, 8:56])
    ok()
    w4a16_check(out[:, 8:56], x, A, B, codes, lin, "mxfp4")
    assert (out[:, :8] == 3).all() and (out[:, 56:] == 3).all()


# ------------------------------------------------------------------ the cache

def ragged(rng, B, most_new, most_old, page, spare=3, shuffle=True):
    new = rng.integers(0, most_new + 1, B)
    new[0] = max(new[0], 1)
    lens = new + rng.integers(0, most_old + 1, B)
    need = (lens + page - 1) // page
    pages = int(need.sum()) + spare
    ids = rng.permutation(pages) if shuffle else np.arange(pages)
    table = np.full((B, int(need.max()) + 1), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return cu, lens.astype(np.int32), table, pages


def append_run(K, V, cu, lens, table, kc, ks, vc, vs):
    t = [R.cuda(a) for a in (kc, ks, vc, vs)]
    BQ.batq_kv8_append(K, V, R.cuda(cu) if cu is not None else None, R.cuda(lens), R.cuda(table), *t)
    ok()
    return [a.cpu().numpy() for a in t]


def append_check(x, cu, lens, table, page, codes, scales, got_codes, got_scales):
    vals, exps = R.e4m3_value(codes), scales.astype(np.int64) - 127
    R.append(x, cu, lens, table, page, vals, exps)
    np.testing.assert_array_equal(got_scales.astype(np.int64) - 127, exps)
    np.testing.assert_array_equal(R.e4m3_value(got_codes), vals)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page,D,heads,B,new,old", [(16, 128, 8, 9, 1, 60), (16, 64, 1, 4, 40, 20), (32, 256, 3, 5, 70, 50),
                                                    (64, 128, 2, 40, 3, 200), (128, 64, 2, 3, 300, 130)])
def test_append_exact(page, D, heads, B, new, old, dtype):
    rng = np.random.default_rng(page + D)
    cu, lens, table, pages = ragged(rng, B, new, old, page)
    T = int(cu[-1])
    kc, ks = R.cache(rng, pages, heads, page, D)
    vc, vs = R.cache(rng, pages, heads, page, D)
    # values of very different sizes, so that many scales grow and many do not
    x = torch.from_numpy((rng.standard_normal((T + 2, 2 * heads * D)) * np.exp2(rng.integers(-9, 4, (T + 2, 1)))).astype(np.float32)).to(dtype)
    K, V = x.cuda()[:, :heads * D], x.cuda()[:, heads * D:]
    g = append_run(K, V, cu, lens, table, kc, ks, vc, vs)
    xs = x.double().numpy()
    append_check(xs[:, :heads * D].reshape(-1, heads, D), cu, lens, table, page, kc, ks, g[0], g[1])
    append_check(xs[:, heads * D:].reshape(-1, heads, D), cu, lens, table, page, vc, vs, g[2], g[3])


def test_append_token_by_token_and_extremes():
    """One token a call (cu None): zeros, subnormals, the largest bf16, NaN and infinities, growing scales."""
    rng = np.random.default_rng(1)
    page, heads, D, B = 16, 2, 64, 3
    table = np.array([[5, 1], [0, 3], [2, 4]], np.int32)
    kc, ks = R.cache(rng, 6, heads, page, D)
    vc, vs = R.cache(rng, 6, heads, page, D)
    mags = [0.0, 1e-40, 1e-38, 1e-3, 1.0, 3e38, 1.0, 448.0, 449.0]
    for n, mag in enumerate(mags):
        x = (rng.uniform(-1, 1, (B, heads * D)) * mag).astype(np.float32)
        if n == 4:
            x[1, 3], x[1, 70], x[2, 5] = np.nan, np.inf, -np.inf
        xb = torch.from_numpy(x).to(BF)
        lens = np.array([n + 1, n + 15, n + 20], np.int32)
        cu = np.arange(B + 1)
        g = append_run(xb.cuda(), xb.cuda(), None, lens, table, kc, ks, vc, vs)
        xs = xb.double().numpy().reshape(B, heads, D)
        append_check(xs, cu, lens, table, page, kc, ks, g[0], g[1])
        append_check(xs, cu, lens, table, page, vc, vs, g[2], g[3])
        kc, ks, vc, vs = g


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (256, 128)])
def test_append_values_that_are_not_finite(D, page, dtype):
    """NaN and infinities of either sign among a block's rows, alone in a block, and blocks without any."""
    rng = np.random.default_rng(D)
    heads, B = 3, 2
    cu, lens = np.array([0, 2 * page + 3, 2 * page + 9], np.int32), np.array([2 * page + 3, page + 1], np.int32)
    table = np.arange(6, dtype=np.int32).reshape(B, 3)
    x = torch.from_numpy(rng.standard_normal((int(cu[-1]), heads, D)).astype(np.float32))
    x[1, 0, 3], x[page - 1, 0, D - 1], x[0, 0, 0] = float("inf"), float("-inf"), float("nan")
    x[page:2 * page, 1] = float("nan")
    x[2 * page + 4, 2, 7] = float("-inf")
    x = x.to(dtype).reshape(int(cu[-1]), heads * D)
    kc, ks = R.cache(rng, 6, heads, page, D)
    vc, vs = R.cache(rng, 6, heads, page, D)
    kc[4], vc[4] = kc[4] & 0x77, vc[4] & 0x77  # (the second sequence's older rows hold no NaN)
    kc[3], vc[3] = kc[3] & 0x77, vc[3] & 0x77
    g = append_run(x.cuda(), x.cuda(), cu, lens, table, kc, ks, vc, vs)
    xs = x.double().numpy().reshape(-1, heads, D)
    append_check(xs, cu, lens, table, page, kc, ks, g[0], g[1])
    append_check(xs, cu, lens, table, page, vc, vs, g[2], g[3])


def test_append_drops_what_has_no_place():
    """Unnamed pages, lengths behind the page table, decreasing and outside ranges, fewer tokens than rows."""
    rng = np.random.default_rng(2)
    page, heads, D = 16, 2, 64
    table = np.array([[0, 99], [-1, 1], [2, 3], [4, 5], [6, 7]], np.int32)
    cu = np.array([0, 20, 45, 65, 60, 70], np.int32)   # sequence 3's range decreases
    lens = np.array([25, 25, 40, 30, 3], np.int32)     # sequence 2 outgrows its table, 4 has fewer tokens than rows
    T = 70
    kc, ks = R.cache(rng, 8, heads, page, D)
    vc, vs = R.cache(rng, 8, heads, page, D)
    x = torch.from_numpy(rng.standard_normal((T, heads * D)).astype(np.float32))
    g = append_run(x.cuda(), x.cuda(), cu, lens, table, kc, ks, vc, vs)
    append_check(x.double().numpy().reshape(T, heads, D), cu, lens, table, page, kc, ks, g[0], g[1])
    append_check(x.double().numpy().reshape(T, heads, D), cu, lens, table, page, vc, vs, g[2], g[3])


# ------------------------------------------------------------------ attention

def attn_run(q, cu, lens, table, kc, ks, vc, vs, scale, max_q, out_dtype=BF, lse=True, heads=None):
    T, row = q.shape
    D, kv = kc.shape[3], kc.shape[1]
    out = torch.full((T, row), 7.0, dtype=out_dtype, device="cuda")
    l = torch.full((T, row // D), 7.0, device="cuda") if lse else None
    ws = torch.full((BQ.batq_attn_kv8_workspace_size(max_q, row // D, kv, D),), 255, dtype=torch.uint8, device="cuda")
    BQ.batq_attn_kv8(q.cuda(), R.cuda(cu) if cu is not None else None, R.cuda(lens), R.cuda(table), R.cuda(kc), R.cuda(ks),
                     R.cuda(vc), R.cuda(vs), scale, max_q, ws, out, lse=l)
    ok()
    return out, l


def attn_check(out, lse, q, cu, lens, table, kc, ks, vc, vs, scale, max_q):
    T = q.shape[0]
    page, D = kc.shape[2:]
    k = R.e4m3_value(kc) * R.e8m0_value(ks)[..., None, None]
    v = R.e4m3_value(vc) * R.e8m0_value(vs)[..., None, None]
    qd = q.double().numpy().reshape(T, -1, D)
    ref, rlse, tol = R.attention(qd, cu, lens, table, page, k, v, R.e8m0_value(vs), scale, max_q, 23 if q.dtype == BF else 11,
                             digits=D == 128 and table.shape[1] * page > 2048)
    got, mine = host(out).reshape(ref.shape), ~np.isnan(tol).all(2)
    assert (got[~mine] == 7).all(), "rows of no sequence were written"
    tol = tol + np.abs(ref) * (2.0 ** -8 if out.dtype == BF else 2.0 ** -22) + 2.0 ** -140
    err = np.abs(got - ref)[mine]
    assert (err <= tol[mine]).all(), (err / tol[mine]).max()
    if lse is not None:
        l = host(lse)
        assert (l[~mine] == 7).all()
        empty = mine & np.isneginf(rlse)
        assert np.isneginf(l[empty]).all() and (got[empty] == 0).all()
        m = mine & ~empty
        assert np.abs(l - rlse)[m].max(initial=0) < 2e-3 * (1 + np.abs(rlse[m]).max(initial=0))


def attn_case(seed, B, kv, G, D, page, most, q_most, q_dtype=BF, pad=0, spread=1.0, cu_given=True):
    rng = np.random.default_rng(seed)
    cu, lens, table, pages = ragged(rng, B, q_most, most, page)
    if not cu_given:
        lens = np.maximum(lens - np.diff(cu) + 1, 0).astype(np.int32)
        cu = np.arange(B + 1).astype(np.int32)
        table = np.where(np.arange(table.shape[1])[None] * page < lens[:, None], table, -1).astype(np.int32)
        need = (lens + page - 1) // page
        at = rng.permutation(pages + B)
        pages += B
        i = 0
        for b in range(B):
            table[b, :need[b]] = at[i:i + need[b]]
            i += need[b]
    kc, ks = R.cache(rng, pages, kv, page, D, spread)
    vc, vs = R.cache(rng, pages, kv, page, D, spread)
    q = torch.from_numpy(rng.standard_normal((int(cu[-1]) + pad, kv * G * D)).astype(np.float32)).to(q_dtype)
    return q, cu, lens, table, kc, ks, vc, vs


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("B,kv,G,D,most,q_most", [(1, 1, 1, 64, 5, 1), (3, 2, 1, 128, 300, 1), (5, 2, 4, 64, 700, 2),
                                                  (4, 1, 7, 128, 500, 3), (2, 3, 8, 128, 900, 8), (3, 1, 16, 256, 400, 5),
                                                  (2, 2, 3, 256, 600, 1), (7, 2, 5, 128, 40, 6)])
def test_attention_ragged(B, kv, G, D, most, q_most, page):
    c = attn_case(B * 100 + D + page, B, kv, G, D, page, most, q_most, pad=2)
    out, lse = attn_run(*c, D ** -0.5, q_most)
    attn_check(out, lse, *c, D ** -0.5, q_most)


@pytest.mark.parametrize("q_dtype,out_dtype", [(F32, F32), (BF, F32), (F32, BF)])
def test_attention_types(q_dtype, out_dtype):
    c = attn_case(7, 4, 2, 4, 128, 16, 500, 3, q_dtype=q_dtype)
    out, lse = attn_run(*c, 0.09, 3, out_dtype=out_dtype)
    attn_check(out, lse, *c, 0.09, 3)


def test_attention_one_query_without_cu():
    c = attn_case(8, 6, 2, 4, 64, 32, 300, 1, cu_given=False)
    out, lse = attn_run(c[0], None, *c[2:], 0.125, 1)
    attn_check(out, lse, *c, 0.125, 1)


@pytest.mark.parametrize("G,q_most", [(4, 1), (3, 9), (8, 40)])
def test_attention_long_sequences_are_split_and_joined(G, q_most):
    """Many key blocks of few items, so that the runs' borders cut them; row tiles beyond one."""
    rng = np.random.default_rng(9)
    B, kv, D, page = 2, 1, 64, 64
    lens = np.array([30011, 9000], np.int32)
    n = np.array([q_most, 1])
    cu = np.array([0, q_most, q_most + 1], np.int32)
    need = (lens + page - 1) // page
    pages = int(need.sum())
    ids = rng.permutation(pages).astype(np.int32)
    table = np.full((B, need.max()), -1, np.int32)
    table[0, :need[0]], table[1, :need[1]] = ids[:need[0]], ids[need[0]:]
    kc, ks = R.cache(rng, pages, kv, page, D)
    vc, vs = R.cache(rng, pages, kv, page, D)
    q = torch.from_numpy(rng.standard_normal((int(cu[-1]), G * D)).astype(np.float32)).to(BF)
    c = (q, cu, lens, table, kc, ks, vc, vs)
    out, lse = attn_run(*c, 0.125, q_most)
    attn_check(out, lse, *c, 0.125, q_most)
    again, lse2 = attn_run(*c, 0.125, q_most)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("spread", [0.0, 4.0, 12.0])
def test_attention_page_scales_far_apart(spread):
    """V pages whose scales differ by many powers of two (the accumulator changes its unit)."""
    c = attn_case(10, 3, 2, 4, 128, 16, 400, 1, spread=spread)
    out, lse = attn_run(*c, 0.01, 1)
    attn_check(out, lse, *c, 0.01, 1)


@pytest.mark.parametrize("low,high", [(0, 5), (0, 247), (27, 120), (20, 130)])
def test_attention_smallest_and_largest_page_scales(low, high):
    """V pages at the ends of the scale's range beside each other, and alone (all-zero blocks have byte 0)."""
    c = list(attn_case(20, 4, 1, 2, 64, 16, 200, 1, spread=0.0))
    rng = np.random.default_rng(20)
    c[7] = np.where(rng.random(c[7].shape) < 0.5, low, high).astype(np.uint8)
    if low == 0 and high > 100:
        c[6][c[7][:, 0] == 0] = 0
    table, lens = c[3], c[2]
    for b in range(2):  # two sequences of low pages only
        ids = table[b, :(lens[b] + 15) // 16]
        c[7][ids] = low
    out, lse = attn_run(*c, 0.05, 1, out_dtype=F32)
    attn_check(out, lse, *c, 0.05, 1)


def test_attention_sharp_and_extreme_queries():
    """Scores of hundreds (one token takes all), zero queries, tiny and huge rows."""
    c = list(attn_case(11, 5, 1, 4, 64, 32, 300, 1, spread=0.0))
    c[0][0] *= 40.0
    c[0][1] = 0.0
    c[0][2] *= 1e-30
    out, lse = attn_run(*c, 0.125, 1)
    attn_check(out, lse, *c, 0.125, 1)


def test_attention_masks_leave_rows_empty():
    """Empty sequences, fewer tokens than queries, unnamed pages, lengths behind the table, more queries than max_q_len."""
    rng = np.random.default_rng(12)
    page, kv, G, D = 16, 2, 2, 64
    kc, ks = R.cache(rng, 8, kv, page, D)
    vc, vs = R.cache(rng, 8, kv, page, D)
    table = np.array([[0, 1, 2], [3, 4, 5], [-1, 6, 99], [7, 0, 1], [2, 3, 4]], np.int32)
    lens = np.array([0, 2, 40, 70, 33], np.int32)
    cu = np.array([0, 2, 6, 7, 9, 13], np.int32)
    q = torch.from_numpy(rng.standard_normal((15, kv * G * D)).astype(np.float32)).to(BF)
    for max_q in (4, 3):
        c = (q, cu, lens, table, kc, ks, vc, vs)
        out, lse = attn_run(*c, 0.125, max_q)
        attn_check(out, lse, *c, 0.125, max_q)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64])
def test_attention_nan_does_not_pass_the_mask(page, D):
    """NaN codes behind the sequence reach nothing; a NaN token reaches the queries that see it, in V only its
    own head dims."""
    rng = np.random.default_rng(13)
    kv, G, L, n = 1, 4, 75, 4
    pages = 8
    kc, ks = R.cache(rng, pages, kv, page, D)
    vc, vs = R.cache(rng, pages, kv, page, D)
    table = np.arange(pages, dtype=np.int32)[None]
    cu, lens = np.array([0, n], np.int32), np.array([L], np.int32)
    q = torch.from_numpy(rng.standard_normal((n, kv * G * D)).astype(np.float32)).to(BF)
    clean, _ = attn_run(q, cu, lens, table, kc, ks, vc, vs, 0.1, n)
    kc2, vc2 = kc.copy(), vc.copy()
    for t in range(L, pages * page):
        kc2[t // page, 0, t % page] = 0x7F
        vc2[t // page, 0, t % page] = 0xFF
    out, _ = attn_run(q, cu, lens, table, kc2, ks, vc2, vs, 0.1, n)
    assert torch.equal(out, clean)
    t = L - 2  # seen by the last two queries
    vc2[t // page, 0, t % page, 5] = 0x7F
    vc2[t // page, 0, t % page, D - 1] = 0xFF
    out, _ = attn_run(q, cu, lens, table, kc2, ks, vc2, vs, 0.1, n)
    o = out.view(n, G, D)
    assert o[2:, :, [5, D - 1]].isnan().all()
    rest = [d for d in range(D) if d not in (5, D - 1)]
    assert torch.equal(o[:2], clean.view(n, G, D)[:2]) and torch.equal(o[2:][..., rest], clean.view(n, G, D)[2:][..., rest])
    kc2[t // page, 0, t % page, 9] = 0x7F
    out, _ = attn_run(q, cu, lens, table, kc2, ks, vc2, vs, 0.1, n)
    assert out[2:].isnan().all() and torch.equal(out[:2], clean[:2])
    vc2[0, 0, 3, 7] = 0x7F  # in a tile that every query sees whole
    out, _ = attn_run(q, cu, lens, table, kc, ks, vc2, vs, 0.1, n)
    assert out.view(n, G, D)[:, :, 7].isnan().all() and torch.equal(out.view(n, G, D)[:2, :, 8:], clean.view(n, G, D)[:2, :, 8:])


def long_table(c, page, tokens=2049):
    """The same call with a page table for more than 2048 tokens, which head dim 128 has a kernel of its own for."""
    c = list(c)
    more = -(-tokens // page) - c[3].shape[1]
    c[3] = np.concatenate([c[3], np.full((c[3].shape[0], max(more, 0)), -1, np.int32)], 1)
    return c


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("B,kv,G,most,q_most", [(1, 1, 1, 5, 1), (3, 2, 1, 300, 1), (5, 2, 4, 700, 2), (4, 1, 7, 500, 3),
                                               (2, 3, 8, 900, 8), (3, 1, 16, 400, 2), (7, 2, 5, 40, 6), (9, 1, 9, 1500, 1),
                                               (2, 2, 6, 800, 5), (2, 1, 48, 700, 3)])
def test_long_attention_ragged(B, kv, G, most, q_most, page):
    c = long_table(attn_case(B * 100 + G + page, B, kv, G, 128, page, most, q_most, pad=2), page)
    out, lse = attn_run(*c, 128 ** -0.5, q_most)
    attn_check(out, lse, *c, 128 ** -0.5, q_most)


@pytest.mark.parametrize("G,q_most", [(4, 1), (4, 3), (8, 3), (4, 8), (8, 5), (8, 6), (8, 7)])
@pytest.mark.parametrize("q_dtype,out_dtype", [(F32, F32), (BF, F32), (F32, BF)])
def test_long_attention_types(q_dtype, out_dtype, G, q_most):
    c = long_table(attn_case(7, 4, 2, G, 128, 16, 500, q_most, q_dtype=q_dtype), 16)
    out, lse = attn_run(*c, -0.09 if G == 8 else 0.09, q_most, out_dtype=out_dtype)
    attn_check(out, lse, *c, -0.09 if G == 8 else 0.09, q_most)


@pytest.mark.parametrize("G,q_most", [(4, 1), (3, 9), (8, 40)])
def test_long_attention_is_split_and_joined(G, q_most):
    """Many key blocks of few items, so that the runs' borders cut them; row tiles beyond one; bit for bit twice."""
    rng = np.random.default_rng(9)
    kv, D, page = 1, 128, 64
    lens = np.array([30011, 9000, 0], np.int32)
    cu = np.array([0, q_most, q_most + 1, q_most + 2], np.int32)
    need = (lens + page - 1) // page
    ids = rng.permutation(int(need.sum())).astype(np.int32)
    table = np.full((3, need.max()), -1, np.int32)
    table[0, :need[0]], table[1, :need[1]] = ids[:need[0]], ids[need[0]:]
    kc, ks = R.cache(rng, len(ids), kv, page, D)
    vc, vs = R.cache(rng, len(ids), kv, page, D)
    q = torch.from_numpy(rng.standard_normal((int(cu[-1]), G * D)).astype(np.float32)).to(BF)
    c = (q, cu, lens, table, kc, ks, vc, vs)
    out, lse = attn_run(*c, 0.088, q_most)
    attn_check(out, lse, *c, 0.088, q_most)
    again, lse2 = attn_run(*c, 0.088, q_most)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("G", [4, 20, 28, 36, 44])
@pytest.mark.parametrize("spread", [0.0, 4.0, 12.0])
def test_long_attention_page_scales_far_apart(spread, G):
    """K and V pages whose scales differ by many powers of two: references move, digits lose the small blocks."""
    c = long_table(attn_case(10, 3, 2, G, 128, 16, 400, 1, spread=spread), 16)
    out, lse = attn_run(*c, 0.01, 1)
    attn_check(out, lse, *c, 0.01, 1)


@pytest.mark.parametrize("low,high", [(0, 5), (0, 247), (27, 120), (20, 130)])
def test_long_attention_smallest_and_largest_page_scales(low, high):
    c = long_table(attn_case(20, 4, 1, 2, 128, 16, 200, 1, spread=0.0), 16)
    rng = np.random.default_rng(20)
    c[7] = np.where(rng.random(c[7].shape) < 0.5, low, high).astype(np.uint8)
    if low == 0 and high > 100:
        c[6][c[7][:, 0] == 0] = 0
    table, lens = c[3], c[2]
    for b in range(2):  # two sequences of low pages only
        c[7][table[b, :(lens[b] + 15) // 16]] = low
    out, lse = attn_run(*c, 0.05, 1, out_dtype=F32)
    attn_check(out, lse, *c, 0.05, 1)


@pytest.mark.parametrize("scale", [0.125, 0.0])
def test_long_attention_sharp_and_extreme_queries(scale):
    """Scores of hundreds that grow along the sequence, zero, tiny and huge queries (their rows share an item)."""
    c = long_table(attn_case(11, 5, 1, 4, 128, 32, 300, 1, spread=0.0), 32)
    c[0][0] *= 40.0
    c[0][1] = 0.0
    c[0][2, :128] *= 1e30 if scale == 0.0 else 1.0
    c[0][2, 128:256] *= 1e-30
    c[5] = np.minimum(c[5], 30).astype(np.uint8) if scale == 0.0 else c[5]
    ids = c[3][4, :(c[2][4] + 31) // 32]
    c[5][ids] = (c[5][ids].astype(np.int64) + np.arange(len(ids))[:, None] // 2).astype(np.uint8)
    out, lse = attn_run(*c, scale, 1)
    attn_check(out, lse, *c, scale, 1)


@pytest.mark.parametrize("D,tokens,G", [(64, 0, 4), (128, 0, 4), (256, 0, 20), (128, 2049, 4), (128, 2049, 20)])
@pytest.mark.parametrize("mag", [1e3, 1e6, 1e9, 1e15, 1e25])
def test_attention_scores_beyond_fp32_steps(mag, D, tokens, G):
    """Scores so large that fp32 holds them only in steps above 1: the largest takes all, of either sign, and ordinary
    rows beside them keep their softmax."""
    c = long_table(attn_case(22, 4, 1, G, D, 32, 300, 1, spread=2.0), 32, tokens)
    q = c[0].view(-1, G, D)
    q[:, 0] *= mag
    q[:, 1] = -q[:, 0]
    out, lse = attn_run(*c, 0.1, 1, out_dtype=F32)
    attn_check(out, None, *c, 0.1, 1)
    # one token's values, where the runner-up is clearly behind: 2^-20 of the score, and 40 for the weights
    k = R.e4m3_value(c[4]) * R.e8m0_value(c[5])[..., None, None]
    v = R.e4m3_value(c[6]) * R.e8m0_value(c[7])[..., None, None]
    seen = 0
    for b in range(len(c[2])):
        L = int(c[2][b])
        if c[1][b + 1] == c[1][b] or L < 2:
            continue
        ids = c[3][b, :(L + 31) // 32]
        kk, vv = (a[ids, 0].reshape(-1, D)[:L] for a in (k, v))
        for h in (0, 1):
            s = kk @ q[c[1][b], h].double().numpy() * 0.1
            order = np.sort(s)
            if order[-1] - order[-2] > 40 + np.abs(s).max() * 2.0 ** -15:
                want = vv[s.argmax()]
                got = host(out).reshape(-1, G, D)[c[1][b], h]
                # the weight's own rounding, and what e^-40 of the others may add
                assert (np.abs(got - want) <= np.abs(want) * 2.0 ** -10 + np.abs(vv).max() * 2.0 ** -19).all()
                seen += 1
    assert seen or mag < 1e6


@pytest.mark.parametrize("G", [4, 20])
def test_long_attention_rows_of_far_magnitudes_share_an_item(G):
    """A head's queries of 1e30 beside one of 1e-20 and ordinary ones: each row's softmax is its own.  (Queries of
    1e35 leave the range of fp32 scores: 128 products with keys of up to 448 sum to 5.7e39 > 3.4e38, and the
    header has NaN for those.)"""
    c = long_table(attn_case(21, 3, 1, G, 128, 32, 300, 1, spread=0.0), 32)
    q = c[0].view(-1, G, 128)
    q[:, 0] *= 1e30
    q[:, 1] *= 1e-20
    out, lse = attn_run(*c, 0.1, 1, out_dtype=F32)
    attn_check(out, None, *c, 0.1, 1)
    tiny = [c[0].clone()] + c[1:]
    tiny[0].view(-1, G, 128)[:, 1] = 0.0
    assert (attn_run(*tiny, 0.1, 1, out_dtype=F32)[0].view(-1, G, 128)[:, 1] - out.view(-1, G, 128)[:, 1]).abs().max() < 1e-6


def test_long_attention_masks_leave_rows_empty():
    rng = np.random.default_rng(12)
    page, kv, G, D = 16, 2, 2, 128
    kc, ks = R.cache(rng, 8, kv, page, D)
    vc, vs = R.cache(rng, 8, kv, page, D)
    table = np.array([[0, 1, 2], [3, 4, 5], [-1, 6, 99], [7, 0, 1], [2, 3, 4]], np.int32)
    lens = np.array([0, 2, 40, 70, 33], np.int32)
    cu = np.array([0, 2, 6, 7, 9, 13], np.int32)
    q = torch.from_numpy(rng.standard_normal((15, kv * G * D)).astype(np.float32)).to(BF)
    for max_q in (4, 3):
        c = long_table((q, cu, lens, table, kc, ks, vc, vs), page)
        out, lse = attn_run(*c, 0.125, max_q)
        attn_check(out, lse, *c, 0.125, max_q)


@pytest.mark.parametrize("G", [2, 12])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("D,tokens", [(64, 0), (128, 0), (128, 2049)])
def test_attention_nan_scales_do_not_pass_the_mask(D, tokens, page, G):
    """A NaN scale of K or V reaches the queries that see a token of its page, and no others."""
    rng = np.random.default_rng(17)
    kv, n = 1, 4
    L = 3 * page + 2  # the last page holds two tokens: queries 0 and 1 see none of them
    kc, ks = R.cache(rng, 5, kv, page, D)
    vc, vs = R.cache(rng, 5, kv, page, D)
    table = np.arange(5, dtype=np.int32)[None]
    cu, lens = np.array([0, n], np.int32), np.array([L], np.int32)
    q = torch.from_numpy(rng.standard_normal((n, kv * G * D)).astype(np.float32)).to(BF)
    c = long_table((q, cu, lens, table, kc, ks, vc, vs), page, tokens)
    clean, _ = attn_run(*c, 0.1, n)
    for which in (5, 7):
        for bad in (3, 4):  # page 4 lies behind the sequence
            d = list(c)
            d[which] = d[which].copy()
            d[which][bad] = 255
            out, _ = attn_run(*d, 0.1, n)
            assert torch.equal(out[:2], clean[:2])
            assert out[2:].isnan().all() if bad == 3 else torch.equal(out, clean)


@pytest.mark.parametrize("D,tokens,G", [(64, 0, 2), (128, 0, 2), (256, 0, 9), (128, 2049, 2), (128, 2049, 9)])
def test_attention_queries_that_are_not_finite(D, tokens, G):
    """An infinity or NaN in a query makes that query's head NaN, whatever the signs of the keys, and no other."""
    rng = np.random.default_rng(18)
    page, kv, n, L = 32, 2, 3, 200
    kc, ks = R.cache(rng, 7, kv, page, D)
    vc, vs = R.cache(rng, 7, kv, page, D)
    kc[..., 3] &= 0x7F  # keys of one sign: infinite scores of one sign
    kc[..., 3] |= 1
    cu, lens = np.array([0, n], np.int32), np.array([L], np.int32)
    q = torch.from_numpy(rng.standard_normal((n, kv * G * D)).astype(np.float32)).to(BF)
    c = long_table((q, cu, lens, np.arange(7, dtype=np.int32)[None], kc, ks, vc, vs), page, tokens)
    clean, _ = attn_run(*c, 0.1, n)
    for value in (float("-inf"), float("inf"), float("nan")):
        c[0] = q.clone()
        c[0].view(n, kv * G, D)[1, 1, 3] = value
        out, lse = attn_run(*c, 0.1, n)
        o = out.view(n, kv * G, D)
        assert o[1, 1].isnan().all() and lse[1, 1].isnan()
        o[1, 1] = clean.view(n, kv * G, D)[1, 1]
        assert torch.equal(out, clean)


@pytest.mark.parametrize("D,G", [(64, 2), (128, 2), (256, 9)])
def test_attention_scale_zero_weighs_all_tokens_alike(D, G):
    c = attn_case(19, 3, 2, G, D, 16, 100, 3)
    out, lse = attn_run(*c, 0.0, 3)
    attn_check(out, lse, *c, 0.0, 3)


@pytest.mark.parametrize("G", [2, 4, 6, 8, 10, 12])
@pytest.mark.parametrize("page", [16, 64])
def test_long_attention_nan_does_not_pass_the_mask(page, G):
    rng = np.random.default_rng(13)
    kv, L, n, D, pages = 1, 139, 4, 128, 12
    kc, ks = R.cache(rng, pages, kv, page, D)
    vc, vs = R.cache(rng, pages, kv, page, D)
    table = np.arange(pages, dtype=np.int32)[None]
    cu, lens = np.array([0, n], np.int32), np.array([L], np.int32)
    q = torch.from_numpy(rng.standard_normal((n, kv * G * D)).astype(np.float32)).to(BF)

    def run(k, v):
        return attn_run(*long_table((q, cu, lens, table, k, ks, v, vs), page), 0.1, n)[0].view(n, G, D)

    clean = run(kc, vc)
    kc2, vc2 = kc.copy(), vc.copy()
    for t in range(L, pages * page):
        kc2[t // page, 0, t % page] = 0x7F
        vc2[t // page, 0, t % page] = 0xFF
    assert torch.equal(run(kc2, vc2), clean)
    t = L - 2  # seen by the last two queries
    for d in (5, 40, D - 1):
        vc2[t // page, 0, t % page, d] = 0x7F if d == 5 else 0xFF
    o = run(kc2, vc2)
    rest = [d for d in range(D) if d not in (5, 40, D - 1)]
    assert o[2:, :, [5, 40, D - 1]].isnan().all()
    assert torch.equal(o[:2], clean[:2]) and torch.equal(o[2:][..., rest], clean[2:][..., rest])
    kc2[t // page, 0, t % page, 9] = 0x7F
    o = run(kc2, vc2)
    assert o[2:].isnan().all() and torch.equal(o[:2], clean[:2])
    vc2[0, 0, 3, 7] = 0x7F  # in a tile that every query sees whole
    o = run(kc, vc2)
    assert o[:, :, 7].isnan().all() and torch.equal(o[:2, :, 8:], clean[:2, :, 8:])


def test_attention_strided_queries_and_outputs():
    c = attn_case(14, 3, 2, 2, 64, 16, 100, 2)
    q = c[0]
    row = q.shape[1]
    big = torch.full((q.shape[0], row + 128), float("nan"), dtype=BF, device="cuda")
    big[:, 64:64 + row] = q.cuda()
    out = torch.full((q.shape[0], row + 16), 7.0, dtype=BF, device="cuda")
    ws = torch.empty(BQ.batq_attn_kv8_workspace_size(2, 4, 2, 64), dtype=torch.uint8, device="cuda")
    BQ.batq_attn_kv8(big[:, 64:64 + row], *[R.cuda(a) for a in c[1:]], 0.125, 2, ws, out[:, 8:8 + row])
    ok()
    attn_check(out[:, 8:8 + row], None, *c, 0.125, 2)
    assert (out[:, :8] == 7).all() and (out[:, 8 + row:] == 7).all()


# ------------------------------------------------------------------ experts

def experts_case(seed, counts, N, M, first=0, tail=0):
    rng = np.random.default_rng(seed)
    E, T = len(counts), first + sum(counts) + tail
    off = (first + np.concatenate([[0], np.cumsum(counts)])).astype(np.int32)
    ac, al = R.random_weights(rng, T, N, "mxfp4")
    wc, wl = zip(*(R.random_weights(rng, M, N, "mxfp4") for _ in range(E)))
    return off, ac, al, np.stack(wc), np.stack(wl)


def experts_run(off, ac, al, wc, wl, out_dtype=F32):
    E, M = wc.shape[:2]
    T, N = ac.shape[0], 2 * ac.shape[1]
    ws = np.stack([R.tile_scales(wl[e]) for e in range(E)])
    out = torch.full((T, M), 7.0, dtype=out_dtype, device="cuda")
    BQ.batq_gemm_mxfp4_experts(R.cuda(ac), R.cuda(al), R.cuda(wc), R.cuda(ws), R.cuda(off), M, N, out)
    ok()
    return out


def experts_check(out, off, ac, al, wc, wl):
    T, N = ac.shape[0], 2 * ac.shape[1]
    a = R.weights(ac, al, "mxfp4")
    got, mine = host(out), np.zeros(T, bool)
    off = np.maximum.accumulate(np.clip(off, 0, T))
    for e in range(wc.shape[0]):
        lo, hi = off[e], off[e + 1]
        if hi <= lo:
            continue
        w = R.weights(wc[e], wl[e], "mxfp4")
        ref, mag = a[lo:hi] @ w.T, np.abs(a[lo:hi]) @ np.abs(w).T
        # exact products; one fp32 step (truncated) per 64 K and their alignment inside, and the output's rounding
        tol = mag * (N / 64 + 4) * 2.0 ** -22 + np.abs(ref) * (2.0 ** -8 if out.dtype == BF else 2.0 ** -24)
        err = np.abs(got[lo:hi] - ref)
        assert (err <= tol).all(), (e, (err / np.maximum(tol, 1e-300)).max())
        mine[lo:hi] = True
    assert (got[~mine] == 7).all(), "rows of no expert were written"


@pytest.mark.parametrize("out_dtype", [F32, BF])
@pytest.mark.parametrize("counts,N,M,first,tail", [
    ([1], 64, 16, 0, 0), ([3, 0, 5], 128, 48, 2, 3), ([1, 16, 17, 0, 31, 32, 33], 576, 272, 0, 1),
    ([255, 256, 257, 300], 512, 128, 0, 0), ([700, 0, 1], 2112, 400, 5, 7), ([40] * 70, 1024, 256, 0, 0),
    ([0, 0, 1000], 1088, 1040, 0, 0), ([129] * 3, 4096, 512, 0, 0),
])
def test_experts_shapes(counts, N, M, first, tail, out_dtype):
    c = experts_case(len(counts) + N, counts, N, M, first, tail)
    experts_check(experts_run(*c, out_dtype), *c)


def test_experts_no_rows_and_bad_offsets():
    """Nothing for any expert; offsets outside the rows are clamped, and none counts as less than one before it."""
    off, ac, al, wc, wl = experts_case(3, [10, 10, 10, 10], 256, 64)
    for o in ([5, 5, 5, 5, 5], [-4, 7, 30, 20, 500], [40, 30, 20, 10, 0]):
        o = np.array(o, np.int32)
        experts_check(experts_run(o, ac, al, wc, wl), o, ac, al, wc, wl)


def test_experts_many_experts():
    rng = np.random.default_rng(4)
    c = experts_case(5, list(rng.integers(0, 4, 512)), 128, 32)
    experts_check(experts_run(*c), *c)


def test_experts_non_finite_scales_stay_in_their_row():
    off, ac, al, wc, wl = experts_case(6, [20, 300], 512, 256)
    clean = experts_run(off, ac, al, wc, wl)
    al[7, 3], wl[1, 9, 2] = 255, 255
    out = experts_run(off, ac, al, wc, wl)
    assert out[7].isnan().all() and out[20:, 9].isnan().all()
    keep_r = [r for r in range(320) if r != 7]
    keep_c = [c for c in range(256) if c != 9]
    assert torch.equal(out[keep_r][:, keep_c], clean[keep_r][:, keep_c])


def test_linear_experts_equals_its_two_halves():
    rng = np.random.default_rng(7)
    off, _, _, wc, wl = experts_case(7, [33, 0, 70, 5], 512, 128)
    T, N, M = 108, 512, 128
    X = torch.from_numpy(rng.standard_normal((T, N)).astype(np.float32)).to(BF).cuda()
    A = (np.eye(8) + 0.1 * rng.standard_normal((8, 8))).astype(np.float32)
    B = R.cuda((np.eye(4) + 0.1 * rng.standard_normal((N // 32, 4, 4))).astype(np.float32))
    ratios = torch.full((N // 32 * 2,), 0.95, device="cuda")
    w, s, o = R.cuda(wc), R.cuda(np.stack([R.tile_scales(x) for x in wl])), R.cuda(off)
    out, ref = torch.empty(T, M, device="cuda"), torch.empty(T, M, device="cuda")
    ws = torch.empty(BQ.batq_linear_experts_workspace_size(T, N), dtype=torch.uint8, device="cuda")
    BQ.batq_linear_experts(X, A, B, ratios, w, s, o, M, ws, out)
    codes, scales = BQ.empty_act_buffers(T, N, BQ.BATQ_SCALES_LINEAR)
    BQ.batq_quant_act(X, A, B, ratios, codes, scales, BQ.BATQ_SCALES_LINEAR)
    BQ.batq_gemm_mxfp4_experts(codes, scales, w, s, o, M, N, ref)
    ok()
    assert torch.equal(out, ref)
    experts_check(ref, off, codes.cpu().numpy(), scales.cpu().numpy().reshape(T, -1), wc, wl)
