"""64-bit references of the speculative-decoding operators, written from their
formulas, on the CPU."""
from __future__ import annotations

import numpy as np
import torch

DTYPES = {"fp16": torch.float16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
CODE_MAX = {"e4m3": 448.0, "int8": 127.0}


def random_cache(kind, pages, heads, page, dim, gen, spread=1.0):
    """(k, v, k_scale, v_scale) on the CPU; scales None for fp16."""
    out = []
    for _ in range(2):
        x = torch.randn((pages, heads, page, dim), generator=gen) * spread
        if kind == "fp16":
            out += [x.half(), None]
        else:
            s = x.abs().amax(-1) / CODE_MAX[kind]
            y = x / s[..., None]
            out += [y.round().to(torch.int8) if kind == "int8" else y.to(DTYPES[kind]), s]
    return out[0], out[2], out[1], out[3]


def values(cache, scale):
    """The values that a cache stands for, in float64."""
    x = cache.float().double()
    return x if scale is None else x * scale.double()[..., None]


def attention(q, k, v, ks, vs, table, ctx, start, mask, scale):
    """(out, lse, tol_out, tol_lse) in float64.  mask: list of ints or None.

    Tolerances.  A score's fp32 error is at most e_s = 2 (D + 8) 2^-24 scale
    sum|q k| (products exact or rounded once, D sums, scaling, exponent); a
    weight's is then e_s + 2^-20 (exp, the running maximum's factors) relative,
    plus its rounding to fp16, 2^-11 relative or 2^-25 absolute below fp16's
    normal range (the weights of the largest score are 1).  With
    A = sum p|v| / sum p, the weights' errors give at most
    (2^-11 + 2 e_s + 2^-19 + L 2^-24) A (L terms summed in fp32) + L 2^-25 max|v|;
    the output's rounding gives 2^-11 |o| + 2^-25."""
    q = q.double()
    T, Q, D = q.shape
    H, page = k.shape[1], k.shape[2]
    G = Q // H
    kd, vd = values(k, ks), values(v, vs)
    out, lse = torch.zeros_like(q), torch.full((T, Q), -np.inf, dtype=torch.float64)
    tol, tol_l = torch.zeros_like(q), torch.zeros((T, Q), dtype=torch.float64)
    for s in range(len(ctx)):
        a, n, c = start[s], start[s + 1] - start[s], max(0, ctx[s])
        pos = torch.arange(c + n)
        entry = pos // page
        ok = entry < table.shape[1]
        pg = table[s].long()[entry.clamp_max(table.shape[1] - 1)]
        ok &= (pg >= 0) & (pg < k.shape[0])
        pg = torch.where(ok, pg, 0)
        for i in range(n):
            seen = ok.clone()
            for j in range(n):
                bit = (j <= i) if mask is None else bool((mask[a + i] >> j) & 1)
                seen[c + j] &= bit
            at = seen.nonzero()[:, 0]
            if not len(at):
                continue
            for h in range(H):
                kk, vv = kd[pg[at], h, pos[at] % page], vd[pg[at], h, pos[at] % page]
                for g in range(G):
                    qi = q[a + i, h * G + g]
                    x = (kk @ qi) * scale
                    m = x.max()
                    p = torch.exp(x - m)
                    Z = p.sum()
                    o = p @ vv / Z
                    A = p @ vv.abs() / Z
                    es = 2 * (D + 8) * 2.0 ** -24 * abs(scale) * float((kk.abs() @ qi.abs()).max())
                    L = len(at)
                    out[a + i, h * G + g] = o
                    lse[a + i, h * G + g] = m + torch.log(Z)
                    tol[a + i, h * G + g] = ((2.0 ** -11 + 2 * es + 2.0 ** -19 + L * 2.0 ** -24) * A
                                             + L * 2.0 ** -25 * vv.abs().max() + 2.0 ** -11 * o.abs()
                                             + 2.0 ** -25)
                    tol_l[a + i, h * G + g] = es + 2.0 ** -19 + L * 2.0 ** -24 \
                        + 2.0 ** -22 * (abs(m) + torch.log(Z))
    return out, lse, tol, tol_l


def rotate(x, pos, freq, interleaved, mscale=1.0):
    """(rotated, |a| + |b| per element) of x [T][heads][D] in float64."""
    x = x.double()
    h = len(freq)
    ang = pos.double()[:, None] * freq.double()
    c, s = (torch.cos(ang) * mscale)[:, None], (torch.sin(ang) * mscale)[:, None]
    y, size = x.clone(), x.abs()
    ia = torch.arange(0, 2 * h, 2) if interleaved else torch.arange(h)
    ib = ia + 1 if interleaved else ia + h
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = (a.abs() + b.abs()) * mscale
    return y, size


def quantise(x, kind):
    """(values, scales) of rows x in float64."""
    s = x.abs().amax(-1) / CODE_MAX[kind]
    u = x / torch.where(s > 0, s, 1.0)[..., None]
    if kind == "int8":
        u = torch.round(u)
    else:
        step = torch.exp2(torch.floor(torch.log2(u.abs().clamp_min(2.0 ** -6))) - 3)
        u = torch.round(u / step) * step
    return u * s[..., None], s


def code_step(x, s, kind):
    """Distance between neighbouring codes' values at x (scale s)."""
    if kind == "int8":
        return s[..., None].expand_as(x)
    u = x.abs() / torch.where(s > 0, s, 1.0)[..., None]
    return torch.exp2(torch.floor(torch.log2(u.clamp_min(2.0 ** -6))) - 3) * s[..., None]


def verify(logits, ids, parents, start, accept, race, draft, temperature, max_nodes):
    """(path, count, token, margin): margin is the smallest relative distance of
    any decision from its boundary; decisions nearer than fp32 can tell apart
    are not comparable."""
    S = len(start) - 1
    path = np.full((S, max_nodes), -1, np.int32)
    count, token = np.zeros(S, np.int32), np.full(S, -1, np.int32)
    margin = np.inf
    V = logits.shape[1]
    for s in range(S):
        a, n = int(start[s]), int(start[s + 1] - start[s])
        if n == 0:
            continue
        cur, walk = 0, [0]
        while True:
            x = logits[a + cur].astype(np.float64)
            if np.isnan(x).any() or not np.isfinite(x.max()):
                break
            kids = [c for c in range(cur + 1, n) if parents[a + c] == cur and 0 <= ids[a + c] < V]
            nxt = None
            if temperature == 0:
                best = int(np.argmax(x))  # the lowest index of equals
                nxt = next((c for c in kids if ids[a + c] == best), None)
                if nxt is None:
                    token[s] = best
                    break
            else:
                w = np.exp((x - x.max()) / temperature)
                w /= w.sum()
                for c in kids:
                    t = ids[a + c]
                    qt = 1.0 if draft is None else float(draft[a + cur][t])
                    u = float(accept[a + c])
                    margin = min(margin, abs(u * qt - w[t]) / max(u * qt, w[t], 1e-300))
                    if u * qt < w[t]:
                        nxt = c
                        break
                    if draft is None:
                        less = w.copy()
                        less[t] = 0
                    else:
                        less = np.maximum(w - draft[a + cur].astype(np.float64), 0)
                    if less.sum() > 0:
                        w = less / less.sum()
                if nxt is None:
                    r = w / race[s].astype(np.float64)
                    token[s] = int(np.argmax(r))
                    if V > 1:
                        two = np.partition(r, -2)[-2:]
                        margin = min(margin, (two[1] - two[0]) / max(two[1], 1e-300))
                    break
            cur = nxt
            walk.append(cur)
        path[s, :len(walk)] = walk
        count[s] = len(walk)
    return path, count, token, margin
