"""Edges of the serving operators: many tiles per cluster, scales and magnitudes far apart, ranges of rows that
overlap, calls at once from several threads, and calls without rows."""

import numpy as np
import pytest
import torch

from mxfp4_w4a4_post_block_b200 import batq as BQ
import serving_ref as R
from test_gpu_serving import (BF, F32, append_check, append_run, attn_check, attn_run, long_table, ok, w4a16_case,
                              w4a16_check, w4a16_run)
from test_gpu_serving_run import Layer

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ W4A16

@pytest.mark.parametrize("S,N,M,out_dtype,fmt", [
    (16, 512, 37888, F32, "mxfp4"), (16, 1024, 37888, BF, "mxfp4"), (16, 2304, 24576, F32, "nvfp4"),
    (16, 2560, 24576, F32, "mxfp4"), (4, 2560, 37888, BF, "mxfp4"), (4, 4096, 24576, BF, "mxfp4"),
    (16, 4096, 24576, F32, "nvfp4")])
def test_w4a16_many_tiles_per_cluster(S, N, M, out_dtype, fmt):
    """Clusters of two to eight CTAs that exchange the sums of four tiles and more: two buffers in turn, whose sums
    must not be replaced before all of a CTA has read them.  (The values, and bit for bit at every repeat.)"""
    x, A, B, codes, lin, _ = w4a16_case(S, N, M, fmt, BF, False, S + N)
    first = w4a16_run(x, A, B, codes, lin, fmt, out_dtype)
    w4a16_check(first, x, A, B, codes, lin, fmt)
    w, s, xd = R.cuda(codes), R.cuda(R.tile_scales(lin)), x.cuda()
    out = torch.empty_like(first)
    wf = BQ.BATQ_W4_MXFP4 if fmt == "mxfp4" else BQ.BATQ_W4_NVFP4
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(100):
        out.fill_(7.0)
        BQ.batq_linear_w4a16(xd, None, None, w, s, M, out, w_format=wf)
        differ += (out != first).sum()
    assert int(differ) == 0
    ok()


@pytest.mark.parametrize("S", [1, 3])
@pytest.mark.parametrize("out_dtype", [F32, BF])
def test_w4a16_nvfp4_values_on_their_bound(S, out_dtype):
    """The block Hadamard transform of a block whose 32 terms all add up, on a power of two: 32 x 0.70710683 / (2 sqrt 8)
    rounds to 4, and its bound's fp32 products to just below 4, so that the value's exponent is the larger one."""
    N, M, rng = 128, 48, np.random.default_rng(31)
    H2 = np.array([[1, 1], [1, -1]])
    H4, H8 = np.kron(H2, H2), np.kron(np.kron(H2, H2), H2)
    A = (H8 / np.sqrt(8)).astype(np.float32)
    B = np.repeat((H4 / 2).astype(np.float32)[None], N // 32, 0)
    codes, lin = R.random_weights(rng, M, N, "nvfp4")
    x = (rng.standard_normal((S, N)) * 0.01).astype(np.float32)
    x[:, 32:64] = np.kron(H4[:, 1], H8[:, 7]) * np.float32(0.70710683)  # the signs of one column of the block's P
    x = torch.from_numpy(x)
    w4a16_check(w4a16_run(x, A, B, codes, lin, "nvfp4", out_dtype), x, A, B, codes, lin, "nvfp4")


@pytest.mark.parametrize("x_mag,a_mag,b_mag", [(1e30, 1e-30, 1e-20), (1e-20, 1e-10, 1e35), (1e10, 1e30, 1e-30)])
def test_w4a16_nvfp4_transforms_of_far_magnitudes(x_mag, a_mag, b_mag):
    """x, A and B whose product is ordinary, while A times B is not in fp32's range.  (x times B has to be: the
    transform's own sums hold it.)"""
    x, A, B, codes, lin, _ = w4a16_case(3, 256, 32, "nvfp4", F32, True, 32)
    x, A, B = x * x_mag, (A * np.float32(a_mag)).astype(np.float32), (B * np.float32(b_mag)).astype(np.float32)
    w4a16_check(w4a16_run(x, A, B, codes, lin, "nvfp4", F32), x, A, B, codes, lin, "nvfp4")


# ------------------------------------------------------------------ attention

def lse_check(lse, q, cu, lens, table, kc, ks, scale, max_q, digits):
    """lse of each row against fp64, within the row's own score error: every score is off by at most `ds`, and so is
    the logarithm of their exponentials' sum.  ds as in serving_ref.attention; beside it the exponentials (2^-21 each),
    fp32 additions (a lane's share of the keys and the joins), what references leave out (2^-24) and lse's own rounding."""
    page, D = kc.shape[2:]
    T, heads, k = q.shape[0], kc.shape[1], R.e4m3_value(kc) * R.e8m0_value(ks)[..., None, None]
    qd = q.double().numpy().reshape(T, -1, D)
    G, got, rows = qd.shape[1] // heads, lse.double().cpu().numpy(), 0
    q_bits = 23 if q.dtype == BF else 11
    for b in range(len(lens)):
        n, L = cu[b + 1] - cu[b], min(int(lens[b]), table.shape[1] * page)
        kk = k[table[b, :(L + page - 1) // page]].transpose(1, 0, 2, 3).reshape(heads, -1, D)[:, :L]
        for i in range(min(n, max_q)):
            see = L - n + i + 1
            for h in range(qd.shape[1]):
                qq, ke = qd[cu[b] + i, h], kk[h // G][:see]
                s, c = ke @ qq * scale, (np.abs(ke) @ np.abs(qq) * abs(scale)).max()
                ds = c * (2.0 ** -q_bits + (D / 8 + 8) * 2.0 ** -23)
                if digits:
                    top = np.repeat(np.abs(qq).reshape(-1, 32).max(1), 32)
                    eq = top * 2.0 ** -21 if q_bits > 11 else np.abs(qq) * 2.0 ** -12 + top * 2.0 ** -25
                    ds = (np.abs(ke) @ eq).max() * abs(scale) + c * (D / 8 + 8) * 2.0 ** -23
                ds += np.abs(s).max() * 2.0 ** -22 + 2.0 ** -15
                want = s.max() + np.log(np.exp(s - s.max()).sum())
                tol = ds + 2.0 ** -21 + 2.0 ** -24 + (see / 32 + 16) * 2.0 ** -23 + abs(want) * 2.0 ** -22
                assert abs(got[cu[b] + i, h] - want) <= tol, (b, i, h, got[cu[b] + i, h], want, tol)
                rows += 1
    assert rows


def spread_case(seed, kv, G, D, page, lens, scales, q_dtype=BF):
    """One query per sequence; V's page p of each sequence has the scale byte scales(p, pages)."""
    rng = np.random.default_rng(seed)
    lens = np.array(lens, np.int32)
    need = (lens + page - 1) // page
    ids = rng.permutation(int(need.sum())).astype(np.int32)
    table = np.full((len(lens), int(need.max())), -1, np.int32)
    kc, ks = R.cache(rng, len(ids), kv, page, D, 0.0)
    vc, vs = R.cache(rng, len(ids), kv, page, D, 0.0)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
        for p in range(n):
            vs[table[b, p]] = scales(p, n)
    vc[vs[:, 0] == 0] = 0  # what the writer leaves for zeros
    q = torch.from_numpy(rng.standard_normal((len(lens), kv * G * D)).astype(np.float32)).to(q_dtype)
    return [q, np.arange(len(lens) + 1).astype(np.int32), lens, table, kc, ks, vc, vs]


ORDERS = {
    "in turn": lambda lo, hi: lambda p, n: (lo, hi)[p & 1],
    "low first": lambda lo, hi: lambda p, n: lo if 2 * p < n else hi,
    "high first": lambda lo, hi: lambda p, n: hi if 2 * p < n else lo,
    "one high page": lambda lo, hi: lambda p, n: hi if p == n // 2 else lo,
    "one low page": lambda lo, hi: lambda p, n: lo if p == n // 2 else hi,
    "steps": lambda lo, hi: lambda p, n: lo + (hi - lo) * p // max(n - 1, 1),
}


@pytest.mark.parametrize("order", list(ORDERS))
@pytest.mark.parametrize("low,high", [(0, 247), (0, 127), (1, 247), (20, 172), (60, 200), (127, 247), (87, 167), (5, 9)])
@pytest.mark.parametrize("D,G,page,tokens", [(64, 2, 16, 0), (64, 20, 64, 0), (128, 4, 16, 0), (128, 12, 32, 0),
                                             (256, 2, 16, 0), (128, 4, 16, 2049), (128, 12, 64, 2049), (128, 20, 16, 2049),
                                             (128, 40, 32, 2049)])
def test_attention_page_scales_at_both_ends_beside_each_other(D, G, page, tokens, low, high, order):
    """V pages whose scales lie up to 2^247 apart, in one tile and in different tiles, key groups and runs, every
    sequence with a query: the tokens of the small ones count in the sums as the others do."""
    lens = [2 * page, 2 * page - 3, 5 * page + 1, 700, 1, 1900]
    c = long_table(spread_case(40, 1, G, D, page, lens, ORDERS[order](low, high)), page, tokens)
    for b in (0, 2, 3, 5):  # (the single token's sequence has one page)
        seen = c[7][c[3][b, :(lens[b] + page - 1) // page], 0]
        assert seen.min() == low and seen.max() == high
    out, lse = attn_run(*c, 0.05, 1, out_dtype=F32)
    attn_check(out, None, *c, 0.05, 1)
    lse_check(lse, *c[:6], 0.05, 1, tokens > 0)


@pytest.mark.parametrize("low,high", [(0, 247), (1, 240), (40, 200)])
@pytest.mark.parametrize("D,G,tokens", [(64, 2, 0), (128, 4, 0), (256, 4, 0), (128, 4, 2049), (128, 20, 2049), (128, 40, 2049)])
def test_attention_scores_and_page_scales_apart(D, G, tokens, low, high):
    """Scores that rise or fall by up to 60 along the sequence while V's scales change: references move both ways."""
    page, lens = 32, [2000, 1999, 640, 641]
    for order in ("low first", "high first", "steps"):
        c = spread_case(41, 1, G, D, page, lens, ORDERS[order](low, high))
        table, ks = c[3], c[5]
        for b in range(4):
            n = (lens[b] + page - 1) // page
            for p in range(n):  # K's scale moves the scores' size; half of the sequences backwards
                ks[table[b, p]] = 116 + 7 * (p if b & 1 else n - 1 - p) // n
        c = long_table(c, page, tokens)
        out, lse = attn_run(*c, 0.05, 1, out_dtype=F32)
        attn_check(out, None, *c, 0.05, 1)
        lse_check(lse, *c[:6], 0.05, 1, tokens > 0)


@pytest.mark.parametrize("D,G,tokens", [(64, 4, 0), (128, 4, 0), (256, 4, 0), (128, 4, 2049), (128, 40, 2049)])
@pytest.mark.parametrize("q_dtype", [BF, F32])
def test_attention_log_sums(D, G, tokens, q_dtype):
    """lse within its row's own error, one token to thousands."""
    page, lens = 16, [1, 2, 17, 300, 2500 if tokens else 1500]
    c = long_table(spread_case(42, 2, G, D, page, lens, lambda p, n: 119, q_dtype), page, tokens)
    out, lse = attn_run(*c, D ** -0.5, 1, out_dtype=F32)
    attn_check(out, None, *c, D ** -0.5, 1)
    lse_check(lse, *c[:6], D ** -0.5, 1, tokens > 0)


@pytest.mark.parametrize("D,G,tokens", [(128, 4, 2049), (128, 12, 2049), (128, 20, 2049), (128, 40, 2049)])
@pytest.mark.parametrize("q_dtype", [BF, F32])
def test_attention_rows_at_both_ends_of_the_range_share_an_item(D, G, tokens, q_dtype):
    """A head whose query has one value of 3e38 (its scores are finite) beside ordinary heads, whose softmax is their
    own; and that head's other 32-dim blocks, where the keys have zeros under the large value."""
    c = spread_case(43, 2, G, D, 16, [300, 65, 17, 1], lambda p, n: 119, q_dtype)
    q = c[0].view(4, 2 * G, D)
    for h in (0, G, 2 * G - 1):
        q[:, h] = 0.0
        q[:, h, 5] = 3e38
    c = long_table(c, 16, tokens)
    out, lse = attn_run(*c, 0.1, 1, out_dtype=F32)
    attn_check(out, None, *c, 0.1, 1)
    lse_check(lse, *c[:6], 0.1, 1, True)
    c[4] = c[4].copy()
    c[4][..., 5] = 0  # K has nothing there: the row's scores are those of its other blocks
    q[:, 0, 64:] = torch.randn(4, D - 64).to(q_dtype)
    out, lse = attn_run(*c, 0.1, 1, out_dtype=F32)
    attn_check(out, None, *c, 0.1, 1)
    lse_check(lse, *c[:6], 0.1, 1, True)


@pytest.mark.parametrize("mag", [1e-11, 1e3])
@pytest.mark.parametrize("D,G,tokens", [(64, 4, 0), (128, 4, 0), (256, 4, 0), (128, 4, 2049), (128, 40, 2049)])
def test_attention_factors_beyond_the_range_of_scores_within(D, G, tokens, mag):
    """K scales of 2^40 under queries of 3e38 where K's codes are zero, and under ordinary scores of small queries: the
    product of the units is beyond fp32's range, no score is."""
    c = spread_case(44, 1, G, D, 16, [100, 33, 5], lambda p, n: 119)
    q = c[0].view(3, G, D)
    q *= mag
    q[:, 1] = 0.0
    q[:, 1, 7] = 3e38
    c[4] = c[4].copy()
    c[4][..., 7] = 0
    c[5] = np.full_like(c[5], 127 + 40 - 8)
    c = long_table(c, 16, tokens)
    out, lse = attn_run(*c, 0.1, 1, out_dtype=F32)
    attn_check(out, None, *c, 0.1, 1)
    lse_check(lse, *c[:6], 0.1, 1, tokens > 0)


# ------------------------------------------------------------------ the cache

@pytest.mark.parametrize("page,D,dtype", [(16, 64, BF), (64, 128, F32)])
@pytest.mark.parametrize("cu,n", [([0, 70, 0, 70, 0, 70, 0, 70], 70), ([0, 70, 5, 66, 66, 60, 69, 0, 70], 70),
                                  ([0, 3, 0, 3, 0, 3, 0, 3, 0, 3, 0, 3], 3)])
def test_append_rows_of_several_sequences(page, D, dtype, cu, n):
    """Ranges of rows that overlap (every second one decreases and is empty): each sequence gets its rows, though they
    touch more pages than rows or pages of rows."""
    rng = np.random.default_rng(50)
    heads, cu = 2, np.array(cu, np.int32)
    B = len(cu) - 1
    lens = np.array([max(int(cu[b + 1] - cu[b]), 0) + 15 + b for b in range(B)], np.int32)
    each = -(-(n + 16 + B) // page) + 1
    table = rng.permutation(B * each).reshape(B, each).astype(np.int32)
    kc, ks = R.cache(rng, B * each, heads, page, D)
    vc, vs = R.cache(rng, B * each, heads, page, D)
    x = torch.from_numpy(rng.standard_normal((n, heads * D)).astype(np.float32)).to(dtype)
    g = append_run(x.cuda(), x.cuda(), cu, lens, table, kc, ks, vc, vs)
    xs = x.double().numpy().reshape(n, heads, D)
    append_check(xs, cu, lens, table, page, kc, ks, g[0], g[1])
    append_check(xs, cu, lens, table, page, vc, vs, g[2], g[3])


# ------------------------------------------------------------------ threads

def test_waiting_calls_let_other_threads_run():
    """Calls that wait for a place in a full launch queue do not hold the interpreter's lock meanwhile."""
    import threading
    import time
    m = Layer(60, 64, 16, 4, [3, 9])
    b, d = m.buffers(), m.d
    m.step(b)
    torch.cuda.synchronize()
    gaps, done = [0.0], threading.Event()

    def tick():
        last = time.perf_counter()
        while not done.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps[0] = max(gaps[0], now - last)
            last = now

    t = threading.Thread(target=tick)
    t.start()
    torch.cuda._sleep(int(2e9))  # about a second, behind which the calls queue up
    t0, longest = time.perf_counter(), 0.0
    for _ in range(4000):
        t1 = time.perf_counter()
        BQ.batq_linear_w4a16(b["x"], None, None, d["w_qkv"], d["s_qkv"], b["qkv"].shape[1], b["qkv"])
        longest = max(longest, time.perf_counter() - t1)
    done.set()
    t.join()
    torch.cuda.synchronize()
    ok()
    assert longest > 0.3, "no call waited"
    assert gaps[0] < longest / 2, (gaps[0], longest, time.perf_counter() - t0)


FIRST_CALLS = """
import sys, threading
sys.path[:0] = [%r, %r]
import torch
from mxfp4_w4a4_post_block_b200 import batq as BQ
from test_gpu_serving_run import Layer

layers = [Layer(61, D, 32, 70, [900, 33, 2000, 5]) for D in (64, 128, 64, 128)]
bufs, streams = [m.buffers() for m in layers], [torch.cuda.Stream() for _ in layers]
torch.cuda.synchronize()
start, errors = threading.Barrier(len(layers)), []

def work(m, b, s):
    try:
        with torch.cuda.stream(s):
            start.wait()
            for _ in range(50):
                m.step(b)
    except Exception as e:
        errors.append(e)

threads = [threading.Thread(target=work, args=a) for a in zip(layers, bufs, streams)]
for t in threads: t.start()
for t in threads: t.join()
torch.cuda.synchronize()
assert not errors, errors
assert BQ.batq_device_error() == 0
want = []
for D in (64, 128):
    m = Layer(61, D, 32, 70, [900, 33, 2000, 5])
    b = m.buffers()
    m.step(b)
    want.append(b)
for i, b in enumerate(bufs):
    for k in b:
        assert torch.equal(b[k], want[i %% 2][k]), (i, k)
print("as one thread's")
"""


def test_first_calls_of_several_threads():
    """A process whose first serving calls come from four threads at once, each on its own stream (what a launcher finds
    out at its first call is shared by all threads): results as one thread's."""
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS % (os.path.dirname(here), here)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "as one thread's" in r.stdout, r.stderr[-2000:]


# ------------------------------------------------------------------ no rows

def test_calls_without_rows_do_nothing():
    """A layer without rows, a step without new tokens or sequences: nothing is written, nothing raised; what does not fit
    is refused as with rows."""
    m = Layer(62, 64, 16, 4, [3, 9])
    b, d = m.buffers(), m.d
    m.step(b)
    kept = [t.clone() for t in d["cache"]]
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    q, kv, M = m.qh * 64, m.kv * 64, b["qkv"].shape[1]
    BQ.batq_linear_w4a16(b["x"][:0], m.A, d["Bm"], d["w_qkv"], d["s_qkv"], M, b["qkv"][:0])
    BQ.batq_linear_w4a16(torch.empty(0, m.hidden, dtype=BF, device="cuda"), None, None, d["w_qkv"], d["s_qkv"], M,
                         torch.empty(0, M, device="cuda"))
    BQ.batq_kv8_append(b["qkv"][:0, q:q + kv], b["qkv"][:0, q + kv:], none, b["lens"], d["table"], *d["cache"])
    BQ.batq_kv8_append(b["qkv"][:0, q:q + kv], b["qkv"][:0, q + kv:], None, b["lens"][:0], d["table"][:0], *d["cache"])
    BQ.batq_attn_kv8(b["qkv"][:0, :q], none, b["lens"], d["table"], *d["cache"], 0.125, 1, m.ws, b["att"][:0])
    offsets = torch.zeros(m.E + 1, dtype=torch.int32, device="cuda")
    BQ.batq_linear_experts(b["sorted"][:0], m.A, d["Bm"], None, d["w_e"], d["s_e"], offsets, m.M, m.ws_e, b["e"][:0])
    codes, scales = BQ.empty_act_buffers(1, m.hidden, BQ.BATQ_SCALES_LINEAR)
    BQ.batq_gemm_mxfp4_experts(codes[:0], scales[:0], d["w_e"], d["s_e"], offsets, m.M, m.hidden, b["e"][:0])
    torch.cuda.synchronize()
    ok()
    for t, k in zip(d["cache"], kept):
        assert torch.equal(t, k)
    with pytest.raises(ValueError):
        BQ.batq_linear_w4a16(b["x"][:0], m.A, d["Bm"], d["w_qkv"], d["s_qkv"], M, b["qkv"])
    with pytest.raises(ValueError):
        BQ.batq_attn_kv8(b["qkv"][:0, :q], None, b["lens"], d["table"], *d["cache"], 0.125, 1, m.ws, b["att"][:0])


@pytest.mark.parametrize("D,G,tokens", [(64, 2, 0), (128, 2, 2049), (256, 2, 0)])
def test_attention_more_queries_allowed_than_there_are(D, G, tokens):
    """A generous max_q_len: what a call of the most that can be (T rows; one without cu) gives, and as fast."""
    rng = np.random.default_rng(63)
    c = list(spread_case(63, 2, G, D, 16, [300, 1200, 41], lambda p, n: 119))
    c[0] = torch.from_numpy(rng.standard_normal((7, 2 * G * D)).astype(np.float32)).to(BF)
    c[1] = np.array([0, 5, 5, 7], np.int32)
    c = long_table(c, 16, tokens)
    for cu, most in ((c[1], 7), (None, 1)):
        want = attn_run(c[0], cu, *c[2:], 0.1, most)
        for m in (most + 1, 300000):
            got = attn_run(c[0], cu, *c[2:], 0.1, m)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # the time of a call that is told 300000 beside one that is told 1
    d = [R.cuda(a) for a in c[2:]]
    q, out = c[0].cuda(), torch.empty(7, 2 * G * D, dtype=BF, device="cuda")
    ws = torch.empty(BQ.batq_attn_kv8_workspace_size(300000, 2 * G, 2, D), dtype=torch.uint8, device="cuda")
    times = [1e9, 1e9]
    for _ in range(5):
        for k, m in enumerate((1, 300000)):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            for i in range(60):
                if i == 10:
                    a.record()
                BQ.batq_attn_kv8(q, None, *d, 0.1, m, ws, out)
            b.record()
            torch.cuda.synchronize()
            times[k] = min(times[k], a.elapsed_time(b))
    assert times[1] < 2 * times[0] + 0.2, times


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("S", [1, 3, 8, 16])
@pytest.mark.parametrize("x_dtype", [BF, F32])
def test_w4a16_bf16_outputs_beside_an_outlier(S, x_dtype, fmt):
    """A value 2^11 above its block's others, whose weights are zero: the outputs come of the others alone, which are
    kept to 2^-16 of it (and the output to 2^-8 of itself)."""
    N, M, rng = 64, 1040, np.random.default_rng(33)
    codes, lin = R.random_weights(rng, M, N, fmt)
    codes[:, 10 // 2] &= 0xF0  # element 10's codes (the low nibble) are +0
    x = torch.from_numpy(rng.uniform(-1, 1, (S, N)).astype(np.float32)).to(x_dtype)
    x[:, 10] = 2047.0 if x_dtype == F32 else 2040.0  # (below 2^11: the block's power of two is 2^10)
    out = w4a16_run(x, None, None, codes, lin, fmt, BF)
    w, xd = R.weights(codes, lin, fmt), x.double().numpy()
    ref = xd @ w.T
    G = 32 if fmt == "mxfp4" else 16
    each = np.where(np.arange(N) // G == 10 // G, 2.0 ** -16 * 2.0 ** 10, 2.0 ** -16)
    if fmt == "nvfp4":
        each = each + 2.0 ** -33 * 2.0 ** 11
    tol = each @ np.abs(w).T + (np.abs(xd) * (np.arange(N) != 10)) @ np.abs(w).T * (N / 8 + 24) * 2.0 ** -23 + np.abs(ref) * 2.0 ** -8
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("D,G,tokens", [(64, 3, 0), (64, 24, 0), (128, 5, 0), (256, 16, 0), (128, 5, 2049), (128, 20, 2049),
                                        (128, 44, 2049)])
@pytest.mark.parametrize("k_spread", [3.0, 12.0])
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_attention_large_scores_beside_page_scales_apart(D, G, tokens, k_spread, seed):
    """Scores up to 2^40, which fp32 holds in steps that V's exponents are lost in, with V scales anywhere: each row is an
    average of its tokens' values, finite, and where one token is clearly ahead that token's."""
    rng = np.random.default_rng(seed)
    page, lens = 16, [1500, 700, 33, 16, 1501]
    c = spread_case(70 + seed, 1, G, D, page, lens, lambda p, n: int(rng.choice([1, 40, 100, 127, 160, 200, 240])))
    c[5] = np.clip(np.round(rng.standard_normal(c[5].shape) * k_spread + 119), 60, 190).astype(np.uint8)
    c = long_table(c, page, tokens)
    out, lse = attn_run(*c, 0.1, 1, out_dtype=F32)
    attn_check(out, None, *c, 0.1, 1)
    k, v = (R.e4m3_value(a) * R.e8m0_value(s)[..., None, None] for a, s in ((c[4], c[5]), (c[6], c[7])))
    seen = 0
    for b, L in enumerate(lens):
        ids = c[3][b, :(L + page - 1) // page]
        kk, vv = (a[ids, 0].reshape(-1, D)[:L] for a in (k, v))
        for h in range(G):
            s = kk @ c[0].view(-1, G, D)[b, h].double().numpy() * 0.1
            got = out.view(-1, G, D)[b, h].double().cpu().numpy()
            assert np.isfinite(got).all() and (np.abs(got) <= np.abs(vv).max(0) * (1 + 2.0 ** -9)).all()
            order = np.sort(s)
            if L == 1 or order[-1] - order[-2] > 200 + np.abs(s).max() * 2.0 ** -15:  # e^-200 times 2^113 is nothing beside 2^-126
                assert np.abs(got - vv[s.argmax()]).max() <= np.abs(vv[s.argmax()]).max() * 2.0 ** -10 + 2.0 ** -126
                seen += 1
    assert seen or k_spread < 10


@pytest.mark.parametrize("G", [4, 20, 40])
def test_long_attention_partials_of_the_largest_values(G):
    """V near fp32's largest (scale 2^120), scores that rise by about 43 from one 128 keys to the next, which is less than a
    reference's slack, in items cut by run borders: partials stay finite."""
    page, lens = 32, [2200] * 40
    c = spread_case(80, 1, G, 128, page, lens, lambda p, n: 247)
    c[0].abs_()
    c[4] = c[4] & 0x7F  # keys and queries of one sign, so that scores rise with K's scales
    for b in range(len(lens)):
        c[5][c[3][b], 0] = np.where(np.arange(len(c[3][b])) // 4 % 2 == 0, 119, 125).astype(np.uint8)
    c = long_table(c, page)
    out, lse = attn_run(*c, 0.028, 1, out_dtype=F32)
    attn_check(out, None, *c, 0.028, 1)
    lse_check(lse, *c[:6], 0.028, 1, True)
