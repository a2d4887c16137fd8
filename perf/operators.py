"""What is measured of the serving operators: 4-bit weight products for few tokens, the 8-bit
cache's writer and the attention that reads it, and the products of ragged groups of experts.

``run`` computes each operator in its plain form (elementary torch operations in fp32), or, with
``own`` set, calls the library.  Cases are plain dicts; ``prepare`` makes the inputs from a seed.

Formats, as in include/batq.h: packed E2M1 codes (element 2j in the low nibble) with E8M0 scales per
32 elements (or E4M3 per 16 and a tensor scale: NVFP4) in the 128-row x 4-column tile layout; cache
pages of E4M3 codes [pages, kv heads, page, head dim] with one E8M0 scale per page and head.
"""

import math
import random

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MIDPOINTS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # One token through a square projection (4096 x 4096): the smallest call of a decode step.
        {"name": "w4a16 1x4096x4096", "op": "w4a16", "S": 1, "N": 4096, "M": 4096, "fmt": "mxfp4", "x": "bf16",
         "out": "bf16", "transform": True},
        # Four sequences through the widest weight of the decode workload (4096 -> 24576).
        {"name": "w4a16 4x4096x24576", "op": "w4a16", "S": 4, "N": 4096, "M": 24576, "fmt": "mxfp4", "x": "bf16",
         "out": "bf16", "transform": True},
        # A down projection of a small odd batch, NVFP4 weights used without a transform, fp32 in and out.
        {"name": "w4a16 nvfp4 7x12288x4096", "op": "w4a16", "S": 7, "N": 12288, "M": 4096, "fmt": "nvfp4", "x": "f32",
         "out": "f32", "transform": False},
        # One new token of each of 64 sequences into pages of 16 tokens: the cache write of a decode step.
        {"name": "kv8 append 64x1", "op": "append", "B": 64, "kv": 8, "D": 128, "page": 16, "new": 1, "old": 700,
         "ragged": 11, "x": "bf16"},
        # Prompts of five sequences (about 8000 tokens in all), some of which continue a partly filled page of 64.
        {"name": "kv8 append 5 prompts", "op": "append", "B": 5, "kv": 8, "D": 128, "page": 64, "new": 2400,
         "old": 900, "ragged": 12, "x": "bf16"},
        # Three short chats with as many KV heads as heads: latency is all that counts.
        {"name": "attn 3 short", "op": "attn", "B": 3, "kv": 8, "G": 1, "D": 64, "page": 16, "len": 100, "q": 1,
         "ragged": 21, "pad": 0},
        # A decode step of 64 ragged sequences of up to 8192 tokens, 32 heads on 8 KV heads, small pages.
        {"name": "attn 64 ragged", "op": "attn", "B": 64, "kv": 8, "G": 4, "D": 128, "page": 16, "len": 8192, "q": 1,
         "ragged": 22, "pad": 0},
        # One sequence of 131072 tokens: the work has to be split along the cache.
        {"name": "attn 1x131072", "op": "attn", "B": 1, "kv": 8, "G": 4, "D": 128, "page": 64, "len": 131072, "q": 1,
         "ragged": 0, "pad": 0},
        # Checking drafted tokens: up to five queries per sequence, eight heads per KV head, a padded batch.
        {"name": "attn 16 drafts", "op": "attn", "B": 16, "kv": 4, "G": 8, "D": 128, "page": 32, "len": 16000, "q": 5,
         "ragged": 23, "pad": 9},
        # A decode step of 64 rows over 64 experts: most experts have none, one or two rows.
        {"name": "experts 64 rows of 64", "op": "experts", "E": 64, "T": 64, "N": 4096, "M": 2048, "ragged": 31,
         "pad": 0, "out": "bf16"},
        # A ragged middle: 128 small experts, odd sizes, about 64 rows each.
        {"name": "experts 8190 rows of 128", "op": "experts", "E": 128, "T": 8190, "N": 2112, "M": 1040, "ragged": 32,
         "pad": 2, "out": "bf16"},
        # A prompt of 16384 rows over eight large experts: the matrix rate counts.
        {"name": "experts 16384 rows of 8", "op": "experts", "E": 8, "T": 16384, "N": 4096, "M": 4096, "ragged": 33,
         "pad": 0, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("w4a16", "append", "attn", "experts"))
    if op == "w4a16":
        while True:
            N, M = 64 * _log(rng, 1, 192), 16 * _log(rng, 1, 2048)
            if N * M <= 4096 * 24576:
                break
        return {"op": op, "S": rng.randint(1, 16), "N": N, "M": M, "fmt": rng.choice(("mxfp4", "nvfp4")),
                "x": rng.choice(("bf16", "f32")), "out": rng.choice(("bf16", "f32")), "transform": rng.random() < 0.6}
    if op == "append":
        B = _log(rng, 1, 64)
        return {"op": op, "B": B, "kv": rng.choice((1, 2, 3, 4, 8)), "D": rng.choice((64, 128, 256)),
                "page": rng.choice((16, 32, 64, 128)), "new": _log(rng, 1, max(1, 8192 // B)), "old": _log(rng, 1, 1500),
                "ragged": rng.randint(1, 10 ** 6), "x": rng.choice(("bf16", "f32"))}
    if op == "attn":
        while True:
            c = {"op": op, "B": _log(rng, 1, 64), "kv": rng.choice((1, 2, 3, 4, 8)), "G": rng.choice((1, 2, 3, 4, 5, 8, 16)),
                 "D": rng.choice((64, 128, 256)), "page": rng.choice((16, 32, 64, 128)), "len": _log(rng, 1, 100000),
                 "q": rng.choice((1, 1, 1, 2, 3, 5, 8)), "ragged": rng.randint(1, 10 ** 6), "pad": rng.choice((0, 0, 3))}
            if c["B"] * c["len"] * c["kv"] * c["D"] <= 131072 * 8 * 128:
                return c
    while True:
        E, T, N, M = rng.choice((1, 2, 5, 8, 16, 60, 128)), _log(rng, 1, 16384), 64 * _log(rng, 1, 64), 16 * _log(rng, 1, 256)
        if E * N * M <= 64 * 4096 * 2048:
            return {"op": op, "E": E, "T": T, "N": N, "M": M, "ragged": rng.randint(1, 10 ** 6), "pad": rng.choice((0, 0, 5)),
                    "out": "bf16"}


def _lengths(case):
    """Of each sequence: the new tokens (or queries) and the tokens in the cache with them."""
    B, rng = case["B"], random.Random(case["ragged"])
    if case["op"] == "append":
        new = [case["new"] if case["new"] == 1 else rng.randint(0 if B > 1 else 1, 2 * case["new"]) for _ in range(B)]
        if case["new"] > 1:  # as many tokens as `new` a sequence says, on average
            over = sum(new) / (B * case["new"])
            new = [max(1 if b == 0 else 0, int(n / max(over, 1e-9))) for b, n in enumerate(new)]
        return new, [rng.randint(0, case["old"]) + n for n in new]
    if not case["ragged"]:
        return [case["q"]] * B, [case["len"]] * B
    new, total = [], []
    for b in range(B):
        n = rng.randint(0 if B > 2 and b else 1, case["q"]) if case["q"] > 1 else 1
        new.append(n)
        total.append(max(n, rng.randint(max(1, case["len"] // 8), case["len"])))
    return new, total


def _counts(case):
    """Rows of each expert: uneven, some experts without any."""
    E, T, rng = case["E"], case["T"], random.Random(case["ragged"])
    w = [0.0 if rng.random() < 0.08 and E > 4 else rng.uniform(0.3, 2.0) for _ in range(E)]
    if sum(w) == 0.0:
        w[0] = 1.0
    if T < 4 * E:  # few rows: each goes to an expert of its own choice
        counts = [0] * E
        for e in rng.choices(range(E), w, k=T):
            counts[e] += 1
        return counts
    counts = [int(T * x / sum(w)) for x in w]
    counts[max(range(E), key=lambda e: w[e])] += T - sum(counts)
    return counts


# --------------------------------------------------------------------------- inputs

def _tile_scales(s):
    """Row-major scales [..., rows, columns] -> the 128 x 4 tile layout [..., bytes], padded with 0x7F."""
    lead, (rows, cols) = s.shape[:-2], s.shape[-2:]
    R, C = (rows + 127) // 128, (cols + 3) // 4
    p = torch.full((*lead, R * 128, C * 4), 0x7F, dtype=torch.uint8, device=s.device)
    p[..., :rows, :cols] = s
    n = len(lead)
    p = p.view(*lead, R, 4, 32, C, 4).permute(*range(n), n, n + 3, n + 2, n + 1, n + 4)
    return p.reshape(*lead, -1).contiguous()


def _pack(q):
    """Nearest E2M1 codes of q (saturating), two to a byte."""
    mid = torch.tensor(MIDPOINTS, device=q.device)
    c = torch.bucketize(q.abs(), mid, out_int32=True).to(torch.uint8) | ((q < 0).to(torch.uint8) << 3)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).contiguous()


def _to_mxfp4(w):
    b = w.view(*w.shape[:-1], -1, 32)
    e = torch.floor(torch.log2(b.abs().amax(-1).clamp_min(1e-30))) - 2
    return _pack((b * torch.exp2(-e)[..., None]).view(w.shape)), (e + 127).to(torch.uint8)


def _to_nvfp4(w):
    gs = 448.0 * 6.0 / w.abs().amax()
    b = w.view(*w.shape[:-1], -1, 16)
    s = (b.abs().amax(-1) * gs / 6.0).to(torch.float8_e4m3fn)
    q = b * (gs / s.float().clamp_min(2.0 ** -9))[..., None]
    return _pack(q.view(w.shape)), s.view(torch.uint8), gs.reshape(1)


def _activations(g, rows, N):
    """Rows of unit variance with a hundredth of the channels 20 times larger."""
    x = torch.randn(rows, N, device="cuda", generator=g)
    return x * (1.0 + 19.0 * (torch.rand(N, device="cuda", generator=g) < 0.01))


def _pages(g, page, lens, page_count):
    """A page table [B, most pages] with the pages of a shuffled pool; -1 behind each sequence's last."""
    need = [(n + page - 1) // page for n in lens]
    ids = torch.randperm(page_count, generator=g)[:sum(need)].to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table.cuda()


def _cache(g, pages, kv, page, D):
    """Pages of E4M3 codes and their scales: each head's values with a spread of its own."""
    x = torch.randn(pages, kv, page, D, device="cuda", generator=g)
    x *= torch.exp2(torch.randn(pages, kv, 1, 1, device="cuda", generator=g))
    m, e = torch.frexp(x.abs().amax((2, 3)))  # m in [0.5, 1): amax <= 448 * 2^s
    s = (e - 9 + (m > 0.875)).to(torch.int32)
    codes = (x * torch.exp2(-s.float())[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, (s + 127).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    h = torch.Generator("cpu").manual_seed(seed)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}
    st = {"case": case}
    if case["op"] == "w4a16":
        S, N, M = case["S"], case["N"], case["M"]
        st["x"] = _activations(g, S, N).to(dt[case["x"]])
        w = torch.randn(M, N, device="cuda", generator=g) * 0.02
        if case["fmt"] == "mxfp4":
            st["codes"], s = _to_mxfp4(w)
            st["gs"] = None
        else:
            st["codes"], s, st["gs"] = _to_nvfp4(w)
        st["scales"] = _tile_scales(s)
        st["A"] = st["A_dev"] = st["B"] = None
        if case["transform"]:
            st["A"] = (torch.eye(8) + 0.1 * torch.randn(8, 8, generator=h)).numpy()
            st["A_dev"] = torch.from_numpy(st["A"]).cuda()
            st["B"] = torch.eye(4, device="cuda") + 0.1 * torch.randn(N // 32, 4, 4, device="cuda", generator=g)
        st["out"] = torch.zeros(S, M, dtype=dt[case["out"]], device="cuda")
        return st
    if case["op"] == "experts":
        E, N, M, T = case["E"], case["N"], case["M"], case["T"]
        counts = _counts(case)
        st["most"] = max(counts)
        st["a_codes"], st["a_scales"] = _to_mxfp4(_activations(g, T + case["pad"], N))
        st["w_codes"], s = _to_mxfp4(torch.randn(E, M, N, device="cuda", generator=g) * 0.02)
        st["w_scales"] = _tile_scales(s)
        st["offsets"] = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
        st["out"] = torch.zeros(T + case["pad"], M, dtype=dt[case["out"]], device="cuda")
        return st
    new, lens = _lengths(case)
    kv, page, D, B = case["kv"], case["page"], case["D"], case["B"]
    pages = sum((n + page - 1) // page for n in lens) + 7
    st["table"] = _pages(h, page, lens, pages)
    st["k"], st["ks"] = _cache(g, pages, kv, page, D)
    st["v"], st["vs"] = _cache(g, pages, kv, page, D)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["cu"] = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
    rows = sum(new)
    st["seq"] = torch.repeat_interleave(torch.arange(B), torch.tensor(new)).cuda()  # the sequence of each row
    if case["op"] == "append":
        qkv = torch.randn(rows, 2 * kv * D, device="cuda", generator=g)
        qkv *= torch.exp2(torch.randn(rows, 1, device="cuda", generator=g))
        qkv = qkv.to(dt[case["x"]])
        st["new_k"], st["new_v"] = qkv[:, :kv * D], qkv[:, kv * D:]  # slices of one projection's output
        return st
    H = kv * case["G"]
    st["q"] = (2.0 * torch.randn(rows + case["pad"], H * D, device="cuda", generator=g)).bfloat16()
    st["out"] = torch.zeros(rows + case["pad"], H * D, dtype=torch.bfloat16, device="cuda")
    st["scale"] = D ** -0.5
    st["row"] = torch.tensor([i for n in new for i in range(n)], device="cuda")  # its place among its sequence's
    st["ws"] = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")  # kept by a server for all its calls
    return st


# --------------------------------------------------------------------------- the plain forms

def _untile(t, rows, cols):
    R, C = (rows + 127) // 128, (cols + 3) // 4
    lead = t.shape[:-1]
    n = len(lead)
    t = t.view(*lead, R, C, 32, 4, 4).permute(*range(n), n, n + 3, n + 2, n + 1, n + 4)
    return t.reshape(*lead, R * 128, C * 4)[..., :rows, :cols]


def _values(codes):
    """fp32 values of packed E2M1 codes."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1)
    return lut[c.int()].view(*codes.shape[:-1], -1)


def _pow2(e8m0):
    return torch.exp2(e8m0.float() - 127.0)


def _mx(codes, scales):
    v = _values(codes)
    return (v.view(*v.shape[:-1], -1, 32) * _pow2(scales)[..., None]).view(v.shape)


def _plain_w4a16(st):
    c, x = st["case"], st["x"].float()
    S, N, M = c["S"], c["N"], c["M"]
    if c["transform"]:
        t = torch.matmul(x.view(S, N // 32, 4, 8), st["A_dev"])
        x = torch.matmul(st["B"].transpose(1, 2), t).reshape(S, N)
    if c["fmt"] == "mxfp4":
        w = _mx(st["codes"], _untile(st["scales"], M, N // 32))
    else:
        s = _untile(st["scales"], M, N // 16).contiguous().view(torch.float8_e4m3fn).float()
        w = (_values(st["codes"]).view(M, N // 16, 16) * s[..., None]).view(M, N)
    out = torch.matmul(x, w.t())
    if st["gs"] is not None:
        out = out / st["gs"]
    return out.to(st["out"].dtype)


def _plain_append(st):
    c = st["case"]
    kv, page, D = c["kv"], c["page"], c["D"]
    rows = st["seq"].numel()
    first = st["lens"] - (st["cu"][1:] - st["cu"][:-1])  # tokens in the cache before
    pos = first[st["seq"]] + torch.arange(rows, device="cuda") - st["cu"][st["seq"]]
    pid, off = st["table"][st["seq"], pos // page].long(), pos % page
    start = torch.full((st["k"].shape[0],), page, device="cuda").scatter_reduce_(0, pid, off.long(), "amin")
    out = []
    for codes, scales, x in ((st["k"], st["ks"], st["new_k"]), (st["v"], st["vs"], st["new_v"])):
        x = x.float().view(rows, kv, D)
        a = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)
        m, e = torch.frexp(a)
        e = torch.where(a > 0, (e - 9 + (m > 0.875)).clamp(min=-127), -127).to(torch.int32)
        need = torch.full(scales.shape, -127, dtype=torch.int32, device="cuda")
        need.scatter_reduce_(0, pid[:, None].expand(rows, kv), e, "amax")
        old = scales.int() - 127
        held = (start > 0)[:, None]  # pages with tokens of before (or without new ones) keep at least their scale
        s = torch.where(held, torch.maximum(old, need), need)
        keep = torch.arange(page, device="cuda")[None, :] < start[:, None]  # rows that were there before
        v = codes.view(torch.float8_e4m3fn).float() * torch.exp2((old - s).float())[:, :, None, None]
        grown = keep[:, None, :] & (s > old)[:, :, None] & (start < page)[:, None, None]
        codes.copy_(torch.where(grown[..., None], v.to(torch.float8_e4m3fn).view(torch.uint8), codes))
        q = (x * torch.exp2(-s[pid].float())[..., None])
        q = torch.where(q.isfinite(), q, float("nan")).to(torch.float8_e4m3fn).view(torch.uint8)
        codes[pid, :, off] = q
        scales.copy_((s + 127).to(torch.uint8))
        out += [codes.view(torch.float8_e4m3fn), scales]
    return out


def _plain_attn(st):
    c = st["case"]
    kv, G, page, D, B, Q = c["kv"], c["G"], c["page"], c["D"], c["B"], c["q"]
    rows = st["seq"].numel()
    table = st["table"].clamp_min(0).long()
    L = table.shape[1] * page
    k = st["k"].view(torch.float8_e4m3fn)[table].float() * _pow2(st["ks"])[table][..., None, None]
    v = st["v"].view(torch.float8_e4m3fn)[table].float() * _pow2(st["vs"])[table][..., None, None]
    k = k.transpose(1, 2).reshape(B, kv, L, D)
    v = v.transpose(1, 2).reshape(B, kv, L, D)
    q = torch.zeros(B, Q, kv, G, D, device="cuda")
    q[st["seq"], st["row"]] = st["q"][:rows].float().view(rows, kv, G, D)
    s = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(B, kv, G * Q, D), k.transpose(2, 3)).view(B, kv, G, Q, L) * st["scale"]
    n = st["cu"][1:] - st["cu"][:-1]
    at = torch.arange(L, device="cuda")
    last = (st["lens"] - n)[:, None] + torch.arange(Q, device="cuda")  # the last token that each query sees
    seen = (at <= last[..., None]) & (at < st["lens"][:, None, None])
    s = torch.where(seen[:, None, None], s, float("-inf"))
    m = s.amax(-1, keepdim=True).clamp_min(-1e30)
    p = torch.exp(s - m)
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-30)
    v = torch.where((at < st["lens"][:, None])[:, None, :, None], v, 0.0)
    o = torch.matmul(p.view(B, kv, G * Q, L), v).view(B, kv, G, Q, D).permute(0, 3, 1, 2, 4)
    out = torch.zeros_like(st["out"])
    out[:rows] = o[st["seq"], st["row"]].reshape(rows, kv * G * D).to(out.dtype)
    return out


def _plain_experts(st):
    c = st["case"]
    E, N, M = c["E"], c["N"], c["M"]
    off = st["offsets"].long()
    a = _mx(st["a_codes"], st["a_scales"])
    w = _mx(st["w_codes"], _untile(st["w_scales"], M, N // 32))
    at = off[:-1, None] + torch.arange(st["most"], device="cuda")  # each expert's rows, padded to the most
    real = at < off[1:, None]
    y = torch.bmm(a[at.clamp_max(a.shape[0] - 1)], w.transpose(1, 2))
    out = torch.zeros_like(st["out"])
    out[at[real]] = y[real].to(out.dtype)
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"w4a16": _plain_w4a16, "append": _plain_append, "attn": _plain_attn, "experts": _plain_experts}[op](state)


def _own(st, op):
    from mxfp4_w4a4_post_block_b200 import batq as BQ
    c = st["case"]
    if op == "w4a16":
        BQ.batq_linear_w4a16(st["x"], st["A"], st["B"], st["codes"], st["scales"], c["M"], st["out"], w_gs=st["gs"],
                             w_format=BQ.BATQ_W4_MXFP4 if c["fmt"] == "mxfp4" else BQ.BATQ_W4_NVFP4)
        return st["out"]
    if op == "append":
        BQ.batq_kv8_append(st["new_k"], st["new_v"], st["cu"], st["lens"], st["table"], st["k"], st["ks"], st["v"],
                           st["vs"])
        return [st["k"].view(torch.float8_e4m3fn), st["ks"], st["v"].view(torch.float8_e4m3fn), st["vs"]]
    if op == "attn":
        BQ.batq_attn_kv8(st["q"], st["cu"], st["lens"], st["table"], st["k"], st["ks"], st["v"], st["vs"], st["scale"],
                         c["q"], st["ws"], st["out"])
        return st["out"]
    BQ.batq_gemm_mxfp4_experts(st["a_codes"], st["a_scales"], st["w_codes"], st["w_scales"], st["offsets"], c["M"],
                               c["N"], st["out"])
    return st["out"]


# --------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "w4a16":
        S, N, M = case["S"], case["N"], case["M"]
        size = {"bf16": 2, "f32": 4}
        w = M * N // 2 + M * N // (32 if case["fmt"] == "mxfp4" else 16)
        return {"bytes": w + S * N * size[case["x"]] + S * M * size[case["out"]], "flops": 2 * S * N * M}
    if case["op"] == "experts":
        counts = _counts(case)
        N, M, T = case["N"], case["M"], sum(counts)
        used = sum(1 for n in counts if n)
        row = N // 2 + N // 32
        return {"bytes": used * M * row + T * row + T * M * 2, "flops": 2 * T * N * M}
    new, lens = _lengths(case)
    kv, D = case["kv"], case["D"]
    if case["op"] == "append":
        size = {"bf16": 2, "f32": 4}[case["x"]]
        return {"bytes": 2 * sum(new) * kv * D * (size + 1), "flops": 4 * sum(new) * kv * D}
    H = kv * case["G"]
    read = sum(n for n, q in zip(lens, new) if q)
    seen = sum(q * (n - q) + q * (q + 1) // 2 for n, q in zip(lens, new))
    return {"bytes": 2 * read * kv * D + 4 * sum(new) * H * D, "flops": 4 * seen * H * D}


# --------------------------------------------------------------------------- the definitions in 64 bits

def _e4m3_64(bits):
    """Values of E4M3 bytes from their fields."""
    b = bits.long()
    e, m = (b >> 3) & 15, (b & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e.double() - 10))
    v = torch.where((b & 127) == 127, float("nan"), v)
    return torch.where(b >= 128, -v, v)


def _e2m1_64(codes):
    """Values of packed E2M1 codes from their fields: s e e m."""
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    e, m = (n >> 1) & 3, (n & 1).double()
    v = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e.double() - 1))
    return torch.where(n >= 8, -v, v)


def _scale_at(t, rows, cols, r, c):
    """Scale bytes (r, c) of the tile layout, by its address formula."""
    kp = (cols + 3) // 4
    return t[((r // 128) * kp + c // 4) * 512 + (r % 32) * 16 + ((r // 32) % 4) * 4 + c % 4]


def _weights_64(codes, tiles, M, N, nv):
    g = 16 if nv else 32
    r, c = torch.arange(M, device="cuda")[:, None], torch.arange(N // g, device="cuda")[None]
    s = _scale_at(tiles, M, N // g, r, c)
    s = _e4m3_64(s) if nv else torch.exp2(s.double() - 127)
    return _e2m1_64(codes) * s.repeat_interleave(g, 1)


def _round_e4m3(v):
    """Nearest E4M3 value (ties to even) of |v| <= 448."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 1).clamp_min(-6).double() - 3)
    return torch.round(v / step) * step


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "w4a16":
        S, N, M = case["S"], case["N"], case["M"]
        x = st["x"].double()
        if case["transform"]:
            P = torch.einsum("iab,cd->iacbd", st["B"].double(), st["A_dev"].double()).reshape(N // 32, 32, 32)
            x = torch.einsum("sia,iab->sib", x.view(S, N // 32, 32), P).reshape(S, N)
        out = torch.empty(S, M, dtype=torch.float64, device="cuda")
        w = _weights_64(st["codes"], st["scales"], M, N, case["fmt"] == "nvfp4")
        out.copy_(x @ w.t())
        return out / st["gs"].double() if st["gs"] is not None else out
    if case["op"] == "experts":
        N, M = case["N"], case["M"]
        out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
        at = 0
        for e, n in enumerate(_counts(case)):
            if n:
                a = _e2m1_64(st["a_codes"][at:at + n]) * torch.exp2(st["a_scales"][at:at + n].double() - 127).repeat_interleave(32, 1)
                out[at:at + n] = a @ _weights_64(st["w_codes"][e], st["w_scales"][e], M, N, False).t()
            at += n
        return out
    new, lens = _lengths(case)
    kv, page, D = case["kv"], case["page"], case["D"]
    table = st["table"].cpu().tolist()
    if case["op"] == "append":
        out = []
        for codes, scales, x in ((st["k"], st["ks"], st["new_k"]), (st["v"], st["vs"], st["new_v"])):
            vals, s, x = _e4m3_64(codes), scales.clone(), x.double().view(-1, kv, D)
            at = 0
            for b, n in enumerate(new):
                p = lens[b] - n
                while n:
                    o, take = p % page, min(n, page - p % page)
                    pid, rows = table[b][p // page], x[at:at + take]
                    a = rows.abs().amax((0, 2))
                    e = torch.ceil(torch.log2(a / 448.0)).clamp_min(-127)
                    e = torch.where(torch.exp2(e - 1) * 448 >= a, e - 1, e).clamp_min(-127)  # log2's own rounding
                    e = torch.where(torch.exp2(e) * 448 < a, e + 1, e)
                    if o:
                        old = s[pid].double() - 127
                        e = torch.maximum(e, old)
                        vals[pid, :, :o] = _round_e4m3(vals[pid, :, :o] * torch.exp2(old - e)[:, None, None])
                    vals[pid, :, o:o + take] = _round_e4m3(rows / torch.exp2(e)[:, None]).transpose(0, 1)
                    s[pid] = (e + 127).to(torch.uint8)
                    p, at, n = p + take, at + take, n - take
            out += [vals, s]
        return out
    H, G = kv * case["G"], case["G"]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, n in enumerate(new):
        if n:
            L = lens[b]
            ids = torch.tensor(table[b][:(L + page - 1) // page], device="cuda")
            k, v = (( _e4m3_64(c[ids]) * torch.exp2(s[ids].double() - 127)[..., None, None]).transpose(0, 1).reshape(kv, -1, D)[:, :L]
                    for c, s in ((st["k"], st["ks"]), (st["v"], st["vs"])))
            q = st["q"][at:at + n].double().view(n, kv, G, D)
            s = torch.einsum("nhgd,hld->hgnl", q, k) * st["scale"]
            hide = torch.ones(n, L, dtype=torch.bool, device="cuda").tril(L - n).logical_not()
            p = torch.softmax(s.masked_fill(hide, float("-inf")), -1)
            out[at:at + n] = torch.einsum("hgnl,hld->nhgd", p, v).reshape(n, H * D)
        at += n
    return out
