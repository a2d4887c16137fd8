"""The serving operators from their definitions, in fp64 numpy / torch on the CPU (no library code)."""

from __future__ import annotations

import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E2M1 = np.concatenate([E2M1, -E2M1])


def e4m3_value(b):
    b = np.asarray(b, dtype=np.int64)
    e, m = (b >> 3) & 15, (b & 7).astype(np.float64)
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b >= 128, -v, v)


def e8m0_value(b):
    b = np.asarray(b, dtype=np.float64)
    return np.where(b == 255, np.nan, np.exp2(b - 127.0))


def e2m1_matrix(codes):
    """Values of packed E2M1 codes, last axis doubled."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    return E2M1[c]


def tile_scales(lin):
    """Row-major scale bytes (rows x columns) into the 128 x 4 tile layout, padding 0x7F."""
    rows, cols = lin.shape
    R, C = (rows + 127) // 128, (cols + 3) // 4
    out = np.full(R * C * 512, 0x7F, np.uint8)
    r, c = np.meshgrid(np.arange(rows), np.arange(cols), indexing="ij")
    out[((r // 128) * C + c // 4) * 512 + (r % 32) * 16 + ((r // 32) % 4) * 4 + c % 4] = lin
    return out


def weights(codes, lin, fmt):
    """fp64 weights of codes (M x N/2) and row-major scale bytes."""
    s = e8m0_value(lin) if fmt == "mxfp4" else e4m3_value(lin)
    return e2m1_matrix(codes) * np.repeat(s, 32 if fmt == "mxfp4" else 16, axis=1)


def random_weights(rng, M, N, fmt):
    codes = rng.integers(0, 256, (M, N // 2), dtype=np.uint8)
    if fmt == "mxfp4":
        lin = rng.integers(117, 126, (M, N // 32)).astype(np.uint8)
    else:
        lin = rng.integers(0x28, 0x7F, (M, N // 16)).astype(np.uint8)
    return codes, lin


def transform(x, A, B):
    """x P in fp64 and the condition |x| |P| of it."""
    S, N = x.shape
    P = np.einsum("iab,cd->iacbd", B.reshape(-1, 4, 4).astype(np.float64), A.astype(np.float64)).reshape(N // 32, 32, 32)
    xb = x.reshape(S, N // 32, 32)
    return (np.einsum("sia,iab->sib", xb, P).reshape(S, N),
            np.einsum("sia,iab->sib", np.abs(xb), np.abs(P)).reshape(S, N))


def round_e4m3(v):
    """Nearest E4M3 value (ties to even), |v| <= 448."""
    _, e = np.frexp(v)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.round(v / step) * step


def block_exponent(amax):
    e = -127
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def append(x, cu, lens, table, page, vals, exps):
    """x: T x heads x D; vals: [pages, heads, page, D] code values, exps: [pages, heads] exponents; in place."""
    pages, heads = exps.shape
    for b in range(len(lens)):
        r0, r1 = cu[b], cu[b + 1]
        if r0 < 0 or r1 > x.shape[0] or r1 < r0 or lens[b] < r1 - r0:
            continue
        first = lens[b] - (r1 - r0)
        for p in range(first // page, min((lens[b] + page - 1) // page, table.shape[1])):
            lo, hi = max(first, p * page), min(lens[b], (p + 1) * page)
            pid = table[b, p]
            if hi <= lo or not 0 <= pid < pages:
                continue
            for h in range(heads):
                rows = x[r0 + lo - first:r0 + hi - first, h].astype(np.float64)
                fin = np.isfinite(rows)
                e = block_exponent(np.abs(rows[fin]).max() if fin.any() else 0.0)
                o = lo - p * page
                if o > 0:
                    e = max(e, int(exps[pid, h]))
                    d = int(exps[pid, h]) - e
                    if d < 0:
                        vals[pid, h, :o] = round_e4m3(vals[pid, h, :o] * 2.0 ** d)
                exps[pid, h] = e
                q = np.full(rows.shape, np.nan)
                q[fin] = round_e4m3(rows[fin] / 2.0 ** e)
                vals[pid, h, o:o + hi - lo] = q


def attention(q, cu, lens, table, page, k, v, vs, scale, max_q, q_bits=24, digits=False):
    """q: T x H x D fp64; k, v: [pages, heads, page, D] fp64 values; vs: [pages, heads] the scales in v.  Returns (out, lse, tol): rows without a
    sequence are NaN in tol.  tol: what f16 probabilities (2^-11 each, weights and none in the sum), scores
    off by their fp32 sums and by queries of `q_bits` bits, and fp32 sums of p v may move an output by.  `digits`:
    of weights that are integers of 20 bits per 32 tokens instead, and of queries in 8-bit parts."""
    T, H, D = q.shape
    heads = k.shape[1]
    G = H // heads
    out, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    tol = np.full((T, H, D), np.nan)
    for b in range(len(lens)):
        r0, r1 = cu[b], cu[b + 1]
        if r0 < 0 or r1 > T or r1 < r0:
            continue
        n = r1 - r0
        L = max(0, min(lens[b], table.shape[1] * page))
        ids = table[b, :(L + page - 1) // page]
        named = np.repeat((ids >= 0) & (ids < k.shape[0]), page)[:L]
        safe = np.where((ids >= 0) & (ids < k.shape[0]), ids, 0)
        kk = k[safe].transpose(1, 0, 2, 3).reshape(heads, -1, D)[:, :L]
        vv = v[safe].transpose(1, 0, 2, 3).reshape(heads, -1, D)[:, :L]
        sv = np.repeat(vs[safe].T, page, axis=1)[:, :L]
        for i in range(min(n, max_q)):
            see = named & (np.arange(L) <= L - n + i)
            for h in range(H):
                tol[r0 + i, h] = 0.0
                if not see.any():
                    continue
                ks, vals, sc, qq = kk[h // G][see], vv[h // G][see], sv[h // G][see], q[r0 + i, h]
                s = ks @ qq * scale
                c = np.abs(ks) @ np.abs(qq) * abs(scale)
                m = np.nanmax(s) if not np.isnan(s).all() else 0.0
                p = np.exp(s - m)
                l = p.sum()
                out[r0 + i, h] = (p / l) @ vals
                lse[r0 + i, h] = m + np.log(l)
                # Every score is off by at most ds: f16 of the query, D fp32 additions, the multiplication by the
                # scales, and sums with the running maximum and the block's exponent (2^-15 covers |ev| <= 127).
                # p_t / sum p then is off by a factor of at most e^(2 ds), since numerator and sum each change by
                # at most e^ds, whatever ds is: |do| <= (e^(2 ds) - 1) sum_t p_t |v_t| (2 ds alone holds only for
                # ds << 1, and scores of 1e5 have ds > 1).
                ds = c.max() * (2.0 ** -q_bits + (D / 8 + 8) * 2.0 ** -23) + np.abs(s).max() * 2.0 ** -22 + 2.0 ** -15
                pv = (p / l) @ np.abs(vals)
                if digits:
                    # A query's parts: E4M3 keeps a value to 2^-4 of it or to 2^-10, where the largest of 32 head dims
                    # is in [2^7, 2^8), and each further part divides that by 16.  Two parts hold bf16's bits but for
                    # the second bound, 2^-14 / 2^7; three keep fp32 to 2^-12 of the value or 2^-18 / 2^7.
                    top = np.repeat(np.abs(qq).reshape(-1, 32).max(1), 32)
                    eq = top * 2.0 ** -21 if q_bits > 11 else np.abs(qq) * 2.0 ** -12 + top * 2.0 ** -25
                    ds = (np.abs(ks) @ eq).max() * abs(scale) + c.max() * (D / 8 + 8) * 2.0 ** -23 + np.abs(s).max() * 2.0 ** -22 + 2.0 ** -15
                    grow = np.expm1(min(2 * ds, 600.0))
                    # The integers are off by half a unit, 2^-21 of a power of two that is less than twice the largest
                    # weight of the 32 tokens; the exponential by 2^-21; each tile's additions round in fp32.
                    at = np.nonzero(see)[0] // 32
                    most = np.zeros(at.max() + 1)
                    np.maximum.at(most, at, p * sc)
                    tol[r0 + i, h] = pv * (2.0 ** -20 + (L / 32 + 8) * 2.0 ** -23 + grow)
                    tol[r0 + i, h] += 2.0 ** -20 / l * (1 + grow) * (most[at] @ np.abs(vals / sc[:, None]))
                    continue
                tol[r0 + i, h] = pv * (2.0 ** -11 + 2.0 ** -20 + np.expm1(min(2 * ds, 600.0)) * (1 + 2.0 ** -11))
                # The f16 weights are p_t 2^ev(t) over the largest such product W, times 2^15: below 2^-14 their
                # rounding is absolute, 2^-25, that is 2^-40 W for each token's code.
                tol[r0 + i, h] += 2.0 ** -40 * (p * sc).max() / l * np.abs(vals / sc[:, None]).sum(0) * (1 + np.expm1(min(2 * ds, 600.0)))
    return out, lse, tol


def cache(rng, pages, heads, page, D, spread=1.0):
    codes = rng.integers(0, 256, (pages, heads, page, D)).astype(np.uint8)
    codes = np.where((codes & 0x7F) > 0x74, codes & 0xF0, codes).astype(np.uint8)  # no NaN
    exps = np.round(rng.standard_normal((pages, heads)) * spread - 8).astype(np.int64)
    return codes, (exps + 127).astype(np.uint8)


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()
