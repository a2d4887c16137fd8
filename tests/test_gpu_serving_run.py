"""The serving operators as a program uses them: a decode step of all of them, captured graphs, other streams,
calls that overlap, caches beyond 4 GiB, and what the Python calls refuse."""

import numpy as np
import pytest
import torch

from mxfp4_w4a4_post_block_b200 import batq as BQ
import serving_ref as R
from test_gpu_serving import BF, F32, append_check, attn_check, attn_run, experts_check, host, ok, w4a16_check

pytestmark = pytest.mark.gpu


class Layer:
    """One block of a decoder: QKV, cache, attention, output product, and top-2 of 4 experts."""

    def __init__(self, seed, D, page, max_pages, lens):
        rng = np.random.default_rng(seed)
        self.D, self.page, self.qh, self.kv, self.hidden, self.E, self.M = D, page, 8, 2, 512, 4, 256
        self.B = len(lens)
        rows = (self.qh + 2 * self.kv) * D
        self.A = (np.eye(8) + 0.1 * rng.standard_normal((8, 8))).astype(np.float32)
        self.Bm = (np.eye(4) + 0.1 * rng.standard_normal((self.hidden // 32, 4, 4))).astype(np.float32)
        self.w_qkv, self.l_qkv = R.random_weights(rng, rows, self.hidden, "mxfp4")
        self.w_o, self.l_o = R.random_weights(rng, self.hidden, self.qh * D, "nvfp4")
        self.w_e, self.l_e = zip(*(R.random_weights(rng, self.M, self.hidden, "mxfp4") for _ in range(self.E)))
        self.w_e, self.l_e = np.stack(self.w_e), np.stack(self.l_e)
        pages = self.B * max_pages + 2
        self.table = rng.permutation(pages)[:self.B * max_pages].reshape(self.B, max_pages).astype(np.int32)
        self.lens = np.array(lens, np.int32)
        self.cache = [R.cache(rng, pages, self.kv, page, D) for _ in range(2)]
        self.x = torch.from_numpy(rng.standard_normal((self.B, self.hidden)).astype(np.float32)).to(BF)
        self.route = rng.permuted(np.tile(np.arange(self.E), (self.B, 1)), axis=1)[:, :2]
        # on the device
        self.d = dict(Bm=R.cuda(self.Bm), w_qkv=R.cuda(self.w_qkv), s_qkv=R.cuda(R.tile_scales(self.l_qkv)), w_o=R.cuda(self.w_o),
                      s_o=R.cuda(R.tile_scales(self.l_o)), w_e=R.cuda(self.w_e),
                      s_e=R.cuda(np.stack([R.tile_scales(l) for l in self.l_e])), table=R.cuda(self.table),
                      cache=[R.cuda(a) for kv in self.cache for a in kv])
        order = np.argsort(self.route.reshape(-1), kind="stable")
        self.offsets = np.searchsorted(self.route.reshape(-1)[order], np.arange(self.E + 1)).astype(np.int32)
        self.rows_of = order // 2
        self.d.update(offsets=R.cuda(self.offsets), rows_of=torch.from_numpy(self.rows_of).cuda())
        f = dict(dtype=torch.uint8, device="cuda")
        self.ws = torch.empty(BQ.batq_attn_kv8_workspace_size(1, self.qh, self.kv, D), **f)
        self.ws_e = torch.empty(BQ.batq_linear_experts_workspace_size(2 * self.B, self.hidden), **f)

    def buffers(self):
        q = (self.qh + 2 * self.kv) * self.D
        return dict(x=self.x.cuda(), lens=R.cuda(self.lens), qkv=torch.empty(self.B, q, dtype=BF, device="cuda"),
                    att=torch.empty(self.B, self.qh * self.D, dtype=BF, device="cuda"),
                    o=torch.empty(self.B, self.hidden, dtype=F32, device="cuda"),
                    sorted=torch.empty(2 * self.B, self.hidden, dtype=BF, device="cuda"),
                    e=torch.empty(2 * self.B, self.M, dtype=BF, device="cuda"))

    def step(self, b):
        d, q = self.d, self.qh * self.D
        kv = self.kv * self.D
        BQ.batq_linear_w4a16(b["x"], self.A, d["Bm"], d["w_qkv"], d["s_qkv"], b["qkv"].shape[1], b["qkv"])
        BQ.batq_kv8_append(b["qkv"][:, q:q + kv], b["qkv"][:, q + kv:], None, b["lens"], d["table"], *d["cache"])
        BQ.batq_attn_kv8(b["qkv"][:, :q], None, b["lens"], d["table"], *d["cache"], self.D ** -0.5, 1, self.ws, b["att"])
        BQ.batq_linear_w4a16(b["att"], None, None, d["w_o"], d["s_o"], self.hidden, b["o"], w_format=BQ.BATQ_W4_NVFP4)
        torch.index_select(b["o"].to(BF), 0, d["rows_of"], out=b["sorted"])
        BQ.batq_linear_experts(b["sorted"], self.A, d["Bm"], None, d["w_e"], d["s_e"], d["offsets"], self.M, self.ws_e, b["e"])


@pytest.mark.parametrize("D,page,max_pages,lens", [(64, 16, 20, [3, 1, 130, 257, 16]), (128, 32, 70, [5, 700, 1, 64, 33, 90, 128])])
def test_decode_steps_of_all_operators(D, page, max_pages, lens):
    """Three steps; each operator against fp64 of what it was given."""
    m = Layer(1, D, page, max_pages, lens)
    b = m.buffers()
    for step in range(3):
        before = [t.cpu().numpy() for t in m.d["cache"]]
        b["x"].copy_(torch.roll(m.x, step, 0))
        b["lens"].copy_(torch.from_numpy(m.lens + step))
        m.step(b)
        ok()
        q, kv = m.qh * D, m.kv * D
        w4a16_check(b["qkv"], b["x"].cpu(), m.A, m.Bm, m.w_qkv, m.l_qkv, "mxfp4")
        after = [t.cpu().numpy() for t in m.d["cache"]]
        qkv, cu, now = b["qkv"].cpu(), np.arange(m.B + 1), m.lens + step
        for k in range(2):
            new = qkv[:, q + k * kv:q + (k + 1) * kv].double().numpy().reshape(m.B, m.kv, D)
            append_check(new, cu, now, m.table, page, before[2 * k], before[2 * k + 1], after[2 * k], after[2 * k + 1])
        attn_check(b["att"], None, qkv[:, :q], cu, now, m.table, *after, D ** -0.5, 1)
        w4a16_check(b["o"], b["att"].cpu(), None, None, m.w_o, m.l_o, "nvfp4")
        assert torch.equal(b["sorted"], b["o"].to(BF)[m.d["rows_of"]])
        codes, scales = BQ.empty_act_buffers(2 * m.B, m.hidden, BQ.BATQ_SCALES_LINEAR)
        BQ.batq_quant_act(b["sorted"], m.A, m.d["Bm"], None, codes, scales, BQ.BATQ_SCALES_LINEAR)
        experts_check(b["e"], m.offsets, codes.cpu().numpy(), scales.cpu().numpy().reshape(2 * m.B, -1), m.w_e, m.l_e)


@pytest.mark.parametrize("D,page,max_pages,lens", [(64, 16, 20, [3, 1, 130, 257, 16]), (128, 32, 70, [5, 700, 1, 64, 33, 90, 128])])
def test_captured_steps_replay_as_the_eager_ones(D, page, max_pages, lens):
    """A graph of the step, replayed for three steps with inputs and lengths copied in; every byte as without it."""
    eager, graphed = Layer(2, D, page, max_pages, lens), Layer(2, D, page, max_pages, lens)
    be, bg = eager.buffers(), graphed.buffers()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    kept = [t.clone() for t in graphed.d["cache"]]
    with torch.cuda.graph(graph, stream=side):
        graphed.step(bg)
    for t, k in zip(graphed.d["cache"], kept):  # (a capture runs nothing)
        assert torch.equal(t, k)
    for step in range(3):
        for m, b in ((eager, be), (graphed, bg)):
            b["x"].copy_(torch.roll(m.x, step, 0))
            b["lens"].copy_(torch.from_numpy(m.lens + step))
        eager.step(be)
        graph.replay()
        ok()
        for name in be:
            assert torch.equal(be[name], bg[name]), name
        for t, k in zip(eager.d["cache"], graphed.d["cache"]):
            assert torch.equal(t, k)


def test_two_graphs_overlap_with_workspaces_of_their_own():
    layers = [Layer(3 + i, 128, 32, 70, [900, 33, 2000, 5]) for i in range(2)]
    bufs, graphs, streams = [m.buffers() for m in layers], [], [torch.cuda.Stream() for _ in layers]
    for m, b, s in zip(layers, bufs, streams):
        m.step(b)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            m.step(b)
        graphs.append(g)
    torch.cuda.synchronize()
    want = [{k: v.clone() for k, v in b.items()} for b in bufs]
    for _ in range(20):  # (the same token is written again each time)
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    ok()
    for b, w in zip(bufs, want):
        for k in w:
            assert torch.equal(b[k], w[k]), k


def test_graphs_that_share_a_workspace_in_one_stream():
    """Two shapes of attention with one workspace, replayed in turn."""
    rng = np.random.default_rng(5)
    page, kv, D = 16, 2, 128
    cases = []
    ws = torch.empty(BQ.batq_attn_kv8_workspace_size(4, 16, kv, D), dtype=torch.uint8, device="cuda")
    for G, n, lens in ((8, 4, [3000, 70]), (2, 1, [2500, 600, 10])):
        B = len(lens)
        table = R.cuda(rng.permutation(200)[None].repeat(B, 0).astype(np.int32))
        c = [R.cuda(a) for _ in range(2) for a in R.cache(rng, 200, kv, page, D)]
        q = torch.randn(B * n, kv * G * D, device="cuda").to(BF)
        cu, out = R.cuda(np.arange(B + 1).astype(np.int32) * n), torch.empty(B * n, kv * G * D, dtype=BF, device="cuda")
        cases.append((q, cu, R.cuda(np.array(lens, np.int32)), table, *c, 0.088, n, ws, out))
    graphs, want = [], []
    side = torch.cuda.Stream()
    for c in cases:
        BQ.batq_attn_kv8(*c)
        want.append(c[-1].clone())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            BQ.batq_attn_kv8(*c)
        graphs.append(g)
    for _ in range(10):
        for g, c in zip(graphs, cases):
            c[-1].zero_()
            g.replay()
    ok()
    for c, w in zip(cases, want):
        assert torch.equal(c[-1], w)


def test_calls_follow_their_stream():
    """Inputs made by a long queue of another stream's work, the calls issued there without waiting."""
    m = Layer(6, 128, 32, 70, [900, 33, 2000, 5])
    b = m.buffers()
    m.step(b)
    torch.cuda.synchronize()
    want = {k: v.clone() for k, v in b.items()}
    side = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device="cuda")
    x = b["x"].clone()
    for k in b:
        if k not in ("lens",):
            b[k].zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            big = (big @ big).clamp(-1, 1)
        b["x"].copy_(x)
        m.step(b)
    side.synchronize()
    ok()
    for k in want:
        assert torch.equal(b[k], want[k]), k


def test_every_call_repeats_bit_for_bit():
    m = Layer(7, 128, 32, 200, [6000, 33, 2000, 5, 1, 17, 6400, 512])
    b = m.buffers()
    m.step(b)
    want = {k: v.clone() for k, v in b.items()}
    cache = [t.clone() for t in m.d["cache"]]
    for _ in range(10):
        m.ws.random_()
        m.ws_e.random_()
        m.step(b)
        ok()
        for k in want:
            assert torch.equal(b[k], want[k]), k
        for t, k in zip(m.d["cache"], cache):
            assert torch.equal(t, k)


@pytest.mark.parametrize("D,page,heads,table_pages", [(256, 128, 8, 3), (128, 128, 8, 17), (64, 64, 16, 6)])
def test_caches_beyond_four_gibibytes(D, page, heads, table_pages):
    """Pages at the far end of a cache give what the same pages give in a small one."""
    rng = np.random.default_rng(8)
    pages = (1 << 32) // (heads * page * D) + 40
    far = BQ.empty_kv8_cache(pages, heads, page, D)
    assert far[0].numel() > 1 << 32
    near = [R.cuda(a) for _ in range(2) for a in R.cache(rng, 2 * table_pages, heads, page, D)]
    for f, n in zip(far, near):
        f[-2 * table_pages:] = n
    table = torch.arange(2 * table_pages, dtype=torch.int32, device="cuda").view(2, table_pages)
    lens = torch.tensor([2 * page + 7, page - 3], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 5, 8], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(8, heads * D, device="cuda") for _ in range(2))
    q = torch.randn(8, 2 * heads * D, device="cuda").to(BF)
    ws = torch.empty(BQ.batq_attn_kv8_workspace_size(5, 2 * heads, heads, D), dtype=torch.uint8, device="cuda")
    outs = []
    for c, t in ((far, table + (pages - 2 * table_pages)), (near, table)):
        BQ.batq_kv8_append(k, v, cu, lens, t.contiguous(), *c)
        out = torch.empty_like(q)
        BQ.batq_attn_kv8(q, cu, lens, t.contiguous(), *c, D ** -0.5, 5, ws, out)
        outs.append(out)
    ok()
    assert torch.equal(*outs) and outs[0].isfinite().all()
    for f, n in zip(far, near):
        assert torch.equal(f[-2 * table_pages:], n)


def test_largest_page_tables_and_batches():
    """Many sequences, most of them empty; a table that names far more pages than are used."""
    rng = np.random.default_rng(9)
    B, kv, D, page, max_pages = 3000, 1, 128, 16, 2100
    lens = np.where(np.arange(B) % 17 == 0, rng.integers(1, 40, B), 0).astype(np.int32)
    lens[1777] = 33000
    table = rng.integers(0, 2200, (B, max_pages)).astype(np.int32)
    kc, ks = R.cache(rng, 2200, kv, page, D)
    vc, vs = R.cache(rng, 2200, kv, page, D)
    q = torch.from_numpy(rng.standard_normal((B, D)).astype(np.float32)).to(BF)
    c = (q, np.arange(B + 1), lens, table, kc, ks, vc, vs)
    out, lse = attn_run(q, None, *c[2:], 0.088, 1)
    attn_check(out, lse, *c, 0.088, 1)


def test_python_calls_refuse_what_does_not_fit():
    m = Layer(10, 64, 16, 4, [3, 9])
    d, b = m.d, m.buffers()
    x, out, w, s = b["x"], b["qkv"], d["w_qkv"], d["s_qkv"]
    rows = out.shape[1]
    keep = out.clone()

    def refuse(f, *args, error=(ValueError, TypeError, BQ.BatqError), **kw):
        with pytest.raises(error):
            f(*args, **kw)

    lin = BQ.batq_linear_w4a16
    refuse(lin, x.t(), None, None, w, s, rows, out)                                    # columns, not rows
    refuse(lin, x[:, ::2], None, None, w, s, rows, out)
    refuse(lin, x.half(), None, None, w, s, rows, out)
    refuse(lin, x[0], None, None, w, s, rows, out)
    refuse(lin, x[:, :480], None, None, w, s, rows, out)                               # weights of another N
    refuse(lin, x, m.A, None, w, s, rows, out)                                         # A without B
    refuse(lin, x, m.A, d["Bm"][:8], w, s, rows, out)
    refuse(lin, x, None, None, w, s, rows, out[:, :-16])
    refuse(lin, x, None, None, w, s, rows, out[:1])
    refuse(lin, x, None, None, w[:, ::2], s, rows, out)
    refuse(lin, x, None, None, w[:-1], s, rows, out)
    refuse(lin, x, None, None, w, s[:-512], rows, out)
    refuse(lin, x, None, None, w, s, rows, out, w_format=2)
    refuse(lin, x, None, None, w, s, rows, out, w_gs=torch.ones(1, device="cuda"))      # MXFP4 has none
    refuse(lin, x.repeat(9, 1), None, None, w, s, rows, out.repeat(9, 1))              # 18 tokens
    refuse(lin, x.cpu(), None, None, w, s, rows, out)
    refuse(lin, x, None, None, w.cpu(), s, rows, out)
    kv, q = m.kv * 64, m.qh * 64
    k, v, cache = out[:, q:q + kv], out[:, q + kv:], d["cache"]
    app = BQ.batq_kv8_append
    refuse(app, k, v[:1], None, b["lens"], d["table"], *cache)
    refuse(app, k, v.float(), None, b["lens"], d["table"], *cache)
    refuse(app, k[:, :100], v[:, :100], None, b["lens"], d["table"], *cache)
    refuse(app, k, v, b["lens"], b["lens"], d["table"], *cache)                        # cu needs batch + 1
    refuse(app, k, v, None, b["lens"].long(), d["table"], *cache)
    refuse(app, k, v, None, b["lens"], d["table"][:, ::2], *cache)
    refuse(app, k, v, None, b["lens"], d["table"][:1], *cache)
    refuse(app, k, v, None, b["lens"], d["table"], cache[0][:, :, ::2], *cache[1:])
    refuse(app, k, v, None, b["lens"], d["table"], cache[0], cache[1][:1], *cache[2:])
    refuse(app, k, v, None, b["lens"], d["table"], cache[0][:-1], *cache[1:])
    refuse(app, k, v, None, b["lens"], d["table"], cache[0], cache[1], cache[2].cpu(), cache[3])
    refuse(app, k[:1], v[:1], None, b["lens"], d["table"], *cache)                     # fewer rows than sequences
    att = BQ.batq_attn_kv8
    qq = out[:, :q]
    good = [qq, None, b["lens"], d["table"], *cache, 0.125, 1, m.ws, b["att"]]
    for at, bad in ((0, qq[:, :-8]), (0, qq.half()), (1, b["lens"]), (2, b["lens"].float()), (3, d["table"].view(-1)),
                    (4, cache[0].float()), (5, cache[1].t()), (8, float("nan")), (9, 0), (10, m.ws[:1000]),
                    (10, m.ws.view(-1)[1:]), (11, b["att"][:, :-64]), (11, b["att"].half()), (11, b["att"][:1])):
        args = list(good)
        args[at] = bad
        refuse(att, *args)
    refuse(att, *good, lse=torch.empty(m.B, m.qh + 1, device="cuda"))
    refuse(att, *good, lse=torch.empty(m.B, m.qh, dtype=BF, device="cuda"))
    ex = BQ.batq_linear_experts
    good = [b["sorted"], m.A, d["Bm"], None, d["w_e"], d["s_e"], d["offsets"], m.M, m.ws_e, b["e"]]
    for at, bad in ((0, b["sorted"][:, :-32]), (1, None), (2, None), (4, d["w_e"][:3]), (5, d["s_e"][:3]),
                    (6, d["offsets"].float()), (7, 20), (8, m.ws_e[:100]), (9, b["e"][:, :-16])):
        args = list(good)
        args[at] = bad
        refuse(ex, *args)
    torch.cuda.synchronize()
    ok()
    assert torch.equal(keep, out)
    m.step(b)  # the context is as it was
    ok()
