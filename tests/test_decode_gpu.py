"""GPU parity of the speculative-decoding operators (nm_rope_append,
nm_cache_read, nm_tree_attention, nm_tree_verify) against 64-bit references."""
from __future__ import annotations

import random

import numpy as np
import pytest

import decode_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

KINDS = ["fp16", "e4m3", "int8"]
NAN = float("nan")


@pytest.fixture(scope="module")
def nm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_spmv_memory_gb300 import _build
    _build.build()
    import sparse_spmv_memory_gb300 as m
    m.lib()
    return m


def cuda(*ts):
    out = tuple(None if t is None else t.cuda() for t in ts)
    return out if len(out) > 1 else out[0]


def within(got, want, tol, what):
    got = got.double().cpu()
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    err = (got - want).abs()
    bad = ~(err <= tol) & ~inf
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} beyond tolerance, worst ratio "
                           f"{float((err / tol)[bad].max()):.3g}, first {bad.nonzero()[0].tolist()}")


# ---- attention ---------------------------------------------------------------------
def tree_masks(n, rnd):
    seen = []
    for i in range(n):
        seen.append((seen[rnd.randrange(i)] if i else 0) | (1 << i))
    return seen


def signed(masks):
    return torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64)


class Batch:
    """Inputs of one attention call on the CPU, and the call."""

    def __init__(self, kind, ctx, nodes, q_heads, kv_heads, dim, page, seed=1, masks="tree",
                 q_scale=2.0, spread=1.0, spoil=True):
        gen, rnd = torch.Generator().manual_seed(seed), random.Random(seed)
        self.ctx, self.nodes, self.page = ctx, nodes, page
        need = [max(1, -(-(c + n) // page)) for c, n in zip(ctx, nodes)]
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=gen).to(torch.int32)
        self.table = torch.full((len(ctx), max(need)), -1, dtype=torch.int32)
        at = 0
        for s, m in enumerate(need):
            self.table[s, :m] = order[at:at + m]
            at += m
        self.k, self.v, self.ks, self.vs = ref.random_cache(kind, pages, kv_heads, page, dim, gen,
                                                            spread)
        self.start = [sum(nodes[:s]) for s in range(len(nodes) + 1)]
        self.masks = None if masks is None else [m for n in nodes for m in tree_masks(n, rnd)]
        T = sum(nodes)
        self.q = (torch.randn((T, q_heads, dim), generator=gen) * q_scale).half()
        self.scale = dim ** -0.5
        self.clean = (self.k.clone(), self.v.clone())
        if spoil:  # whatever lies behind the sequences' ends is never used
            for s in range(len(ctx)):
                end = ctx[s] + nodes[s]
                for j in range(end, need[s] * page):
                    self.set_row(s, j, NAN)

    def place(self, s, j):
        return int(self.table[s, j // self.page]), j % self.page

    def set_row(self, s, j, x, head=slice(None), which="kv"):
        p, o = self.place(s, j)
        for name in which:
            cache, scale = (self.k, self.ks) if name == "k" else (self.v, self.vs)
            if scale is None:
                cache[p, head, o] = x
            else:
                scale[p, head, o] = x

    def run(self, nm, **kw):
        k, v, ks, vs = cuda(self.k, self.v, self.ks, self.vs)
        mask = None if self.masks is None else signed(self.masks).cuda()
        return nm.nm_tree_attention(
            self.q.cuda(), k, v, self.table.cuda(),
            torch.tensor(self.ctx, dtype=torch.int32).cuda(),
            torch.tensor(self.start, dtype=torch.int32).cuda(), max(1, max(self.nodes)),
            tree_mask=mask, k_scale=ks, v_scale=vs, scale=self.scale, **kw)

    def want(self):
        def clean(x, scale):  # the reference never reads spoilt rows either, but 0 * nan would
            return x if scale is not None else torch.nan_to_num(x, 0.0)
        ks = None if self.ks is None else torch.nan_to_num(self.ks, 0.0)
        vs = None if self.vs is None else torch.nan_to_num(self.vs, 0.0)
        return ref.attention(self.q, clean(self.k, ks), clean(self.v, vs), ks, vs, self.table,
                             self.ctx, self.start, self.masks, self.scale)

    def check(self, nm, what, **kw):
        out, lse = self.run(nm, **kw)
        torch.cuda.synchronize()
        o, l, to, tl = self.want()
        within(lse, l, tl, what + " lse")
        within(out, o, to, what + " out")
        return out, lse


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("ctx,nodes", [
    ([0], [1]), ([1], [1]), ([7], [1]), ([500], [1]), ([129], [2]), ([63, 64, 65], [3, 1, 5]),
    ([0, 1000, 17], [8, 8, 8]), ([256, 0, 300, 5], [16, 33, 1, 20]), ([1500], [64]),
    ([40] * 9, [4] * 9), ([3000, 2], [7, 1])])
def test_attention_lengths(nm, kind, ctx, nodes):
    Batch(kind, ctx, nodes, 16, 4, 128, 16).check(nm, f"{kind} ctx {ctx} nodes {nodes}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("q_heads,kv_heads,dim", [(1, 1, 64), (7, 1, 64), (28, 4, 64), (8, 8, 128),
                                                  (5, 5, 64), (32, 8, 128), (24, 2, 128),
                                                  (64, 1, 128), (40, 8, 64)])
@pytest.mark.parametrize("nodes", [1, 5, 17])
def test_attention_heads(nm, kind, q_heads, kv_heads, dim, nodes):
    Batch(kind, [211, 34], [nodes, max(1, nodes - 2)], q_heads, kv_heads, dim, 32, seed=3).check(
        nm, f"{kind} {q_heads}/{kv_heads}x{dim} nodes {nodes}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nodes", [3, 9, 18, 33, 64])
@pytest.mark.parametrize("scale", [-0.07, 0.0, 1e-20])
def test_attention_scales(nm, kind, nodes, scale):
    """A scale of any sign, and ones under which every row is averaged."""
    b = Batch(kind, [300, 0], [nodes, 2], 8, 2, 128, 64, seed=41)
    b.scale = scale
    b.check(nm, f"{kind} nodes {nodes} scale {scale}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim,q_heads", [(128, 8), (64, 56)])
@pytest.mark.parametrize("ctx,nodes", [([300, 0, 77], [1, 2, 1]), ([2500], [2]), ([40] * 40, [1] * 40)])
def test_attention_few_rows_of_wide_tables(nm, kind, dim, q_heads, ctx, nodes):
    """Few query rows, and tables that could hold far more than the sequences do."""
    b = Batch(kind, ctx, nodes, q_heads, 8, dim, 64, seed=43)
    wide = torch.full((len(ctx), -(-220 * 2 ** 20 // (len(ctx) * 64 * 8 * dim * 4))), -1, dtype=torch.int32)
    cols = min(wide.shape[1], b.table.shape[1])
    wide[:, :cols] = b.table[:, :cols]
    b.table = wide
    b.check(nm, f"{kind} {q_heads}x{dim} ctx {ctx}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [8, 64, 128, 1024])
@pytest.mark.parametrize("nodes", [2, 40])
def test_attention_pages_and_causal(nm, kind, page, nodes):
    """Pages that end inside any tile, one larger than the context; no mask."""
    Batch(kind, [333, 129], [nodes, 1], 8, 2, 128, page, seed=5, masks=None).check(
        nm, f"{kind} page {page}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nodes", [3, 24])
def test_attention_rows_that_see_nothing(nm, kind, nodes):
    b = Batch(kind, [0, 70, 0], [nodes, nodes, 1], 16, 2, 64, 16, seed=7)
    for t in (0, nodes, nodes + 1, 2 * nodes):  # no bits at all
        b.masks[t] = 0
    out, lse = b.check(nm, f"{kind} empty rows")
    assert torch.isinf(lse[0]).all() and (out[0] == 0).all()
    assert torch.isinf(lse[2 * nodes]).all() and (out[2 * nodes] == 0).all()
    assert torch.isfinite(lse[nodes]).all()  # it sees its context


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nodes", [6, 30])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("bad", [NAN, float("inf")])
def test_attention_spoilt_node(nm, kind, nodes, which, bad):
    """A non-finite row of one node reaches the nodes that see it and no others."""
    b = Batch(kind, [90], [nodes], 8, 2, 128, 16, seed=9)
    want, wl, to, tl = b.want()
    j = 3
    b.set_row(0, 90 + j, bad, which=which)
    out, lse = b.run(nm)
    seen = torch.tensor([bool((m >> j) & 1) for m in b.masks])
    assert seen.any() and not seen.all()
    within(out[~seen], want[~seen], to[~seen], "nodes that do not see it")
    within(lse[~seen], wl[~seen], tl[~seen], "lse of nodes that do not see it")
    if bad != bad or which == "v" or kind == "fp16":  # codes times an infinite scale: the score may
        assert not torch.isfinite(out[seen]).all(-1).any()  # be -inf, which rightly weighs nothing


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nodes", [4, 32])
def test_attention_large_scores_and_outliers(nm, kind, nodes):
    """Scores of several hundred (all weight on few rows) and values whose rows
    differ by orders of magnitude."""
    b = Batch(kind, [400], [nodes], 8, 2, 128, 32, seed=11, q_scale=60.0)
    factor = 10.0 ** (torch.arange(b.v.shape[0] * 32).view(-1, 1, 32) % 7 - 4).float()
    if b.vs is None:
        b.v = (b.v.float() * factor[..., None]).half()
    else:
        b.vs = b.vs * factor
    b.check(nm, f"{kind} large scores")
    b = Batch(kind, [400], [nodes], 8, 2, 128, 32, seed=12)
    b.scale = 0.0  # every row weighs the same
    b.check(nm, f"{kind} scale 0")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nodes,group", [(1, 2), (5, 2), (5, 4), (9, 7), (20, 5), (64, 4)])
@pytest.mark.parametrize("small", [-25.5, -27, -29])
def test_attention_one_dominant_position(nm, kind, nodes, group, small):
    """Nearly all the weight on an early position, whose values are 0 in most columns;
    1023 others of 2^small of its weight make those columns.  Enough sequences, all of
    the same pages, for items that one block has whole.  Tolerance: weights of down to
    2^-24 of the largest are rounded by 2^-11 (below: 2^-35 of it each), A = sum p|v|; a
    score by e_s = 2 (D + 8) 2^-24 scale |q k|; sums are fp32 over at most 2^10 terms;
    the output's rounding."""
    L, D, H, page, S = 1024, 64, 8, 64, 38
    gen = torch.Generator().manual_seed(nodes)
    k = torch.randn((H, L, D), generator=gen)
    v = 64 * (1 + 0.5 * torch.randn((H, L, D), generator=gen))
    at = 5
    k[..., 0] = 0.0
    k[:, at], v[:, at] = 0.0, 0.0
    k[:, at, 0], v[:, at, 5] = 16.0, 200.0

    def stored(x):  # [pages][heads][page][dim], and scales
        x = x.view(H, L // page, page, D).transpose(0, 1).contiguous()
        if kind == "fp16":
            return x.half(), None
        s = x.abs().amax(-1) / ref.CODE_MAX[kind]
        y = x / s[..., None]
        return (y.round().to(torch.int8) if kind == "int8" else y.to(ref.DTYPES[kind])), s
    (kc, ks), (vc, vs) = stored(k), stored(v)
    kd, vd = (ref.values(c, s).transpose(0, 1).reshape(H, L, D) for c, s in ((kc, ks), (vc, vs)))
    T, Q = S * nodes, H * group
    q = torch.zeros((T, Q, D), dtype=torch.float16)
    q[..., 0] = 8.0
    scale = float(np.float32(-small * np.log(2.0) / (8.0 * float(kd[0, at, 0]))))
    table = torch.arange(L // page, dtype=torch.int32).expand(S, -1).contiguous()
    out, lse = nm.nm_tree_attention(
        *cuda(q, kc, vc, table), torch.full((S,), L, dtype=torch.int32).cuda(),
        (torch.arange(S + 1) * nodes).to(torch.int32).cuda(), nodes,
        tree_mask=torch.zeros(T, dtype=torch.int64).cuda(), k_scale=cuda(ks), v_scale=cuda(vs), scale=scale)
    s = kd[..., 0] * 8.0 * scale
    p = torch.softmax(s, -1)[:, None]
    o, A = (p @ vd)[:, 0], (p @ vd.abs())[:, 0]
    es = 2 * (D + 8) * 2.0 ** -24 * float(s.abs().max())
    tol = (2.0 ** -11 + 2 * es + 2.0 ** -14) * A + L * 2.0 ** -35 * vd.abs().max() + 2.0 ** -11 * o.abs() + 2.0 ** -25
    assert (tol[:, 6:] < 0.15 * o[:, 6:]).all()

    def rows(x):  # of every key head, for its query heads and all tokens
        return x.repeat_interleave(group, 0).expand((T,) + (Q,) + x.shape[1:])
    within(out, rows(o), rows(tol), f"{kind} out")
    want = torch.logsumexp(s, -1)
    within(lse, rows(want), rows(es + 2.0 ** -14 + 2.0 ** -22 * want), f"{kind} lse")


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("nodes,q_heads", [(50, 1), (64, 2), (64, 5)])
def test_attention_weights_are_rounded_once(nm, kind, nodes, q_heads):
    """The largest score so far grows by 2^9 to 2^11 inside a tile of 128 positions, at
    one whose value row is 0 in all columns but one, as is that of the largest before:
    the other columns show the weight of one that is neither.  One rounding of it to fp16, one of the output, 2^-11 each, and
    2^-15 for scores, scales and exponentials: two products at most that are not 0,
    exact, then four roundings of numbers up to 42, 2^-24 of them each."""
    D, page = 128, 16
    gen = torch.Generator().manual_seed(nodes)
    L = 100
    k, v = torch.zeros((L, D)), torch.zeros((L, D))
    other = [i for i in range(L) if i not in (3, 7, 45)]
    k[other, 0], v[other] = -1.0, 1e-3
    k[[3, 7, 45], 0] = 1.0
    k[[7, 45], 2] = 1.0
    k[45, 1] = 1.0
    v[3] = 1.0 + torch.rand(D, generator=gen)
    v[[7, 45], 0] = 2.0
    out = []
    for x in (k, v):
        s = x.abs().amax(-1) / ref.CODE_MAX[kind]
        y = x / torch.where(s > 0, s, 1.0)[:, None]
        out += [y.round().to(torch.int8) if kind == "int8" else y.to(ref.DTYPES[kind]), s]
    kc, ks, vc, vs = out
    kd, vd = ref.values(kc, ks), ref.values(vc, vs)
    q = torch.zeros((nodes, q_heads, D))
    q[..., 0] = 20.0
    q[..., 1] = (9 + 2 * torch.rand((nodes, q_heads), generator=gen)) * 0.6931
    q[..., 2] = torch.rand((nodes, q_heads), generator=gen) * 0.6931
    q = q.half()
    pages = -(-(L + nodes) // page)

    def paged(x, shape):
        raw = x.view(torch.uint8) if x.dim() == 2 else x
        y = torch.zeros((pages * page,) + raw.shape[1:], dtype=raw.dtype)
        y[:L] = raw
        return y.view(x.dtype).view(shape).cuda()
    one = (pages, 1, page)
    got, _ = nm.nm_tree_attention(
        q.cuda(), paged(kc, one + (D,)), paged(vc, one + (D,)), torch.arange(pages, dtype=torch.int32)[None].cuda(),
        torch.tensor([L], dtype=torch.int32).cuda(), torch.tensor([0, nodes], dtype=torch.int32).cuda(), nodes,
        tree_mask=torch.zeros(nodes, dtype=torch.int64).cuda(), k_scale=paged(ks, one), v_scale=paged(vs, one),
        scale=1.0)
    s = q.double() @ kd.T
    p = torch.softmax(s, -1)
    o, A = p @ vd, p @ vd.abs()
    within(got, o, 2.0 ** -11 * (A + o.abs()) + 2.0 ** -15 * A + 2.0 ** -25, f"{kind} out")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nodes", [1, 20])
def test_attention_absent_pages(nm, kind, nodes):
    """Entries out of range, and positions beyond the table, are seen by no node."""
    b = Batch(kind, [200, 100], [nodes, nodes], 8, 2, 64, 16, seed=13, spoil=False)
    b.table[0, 2], b.table[0, 5], b.table[1, 0] = -1, b.k.shape[0], 2 ** 31 - 1
    b.check(nm, f"{kind} absent pages")
    b.table = b.table[:, :4].contiguous()
    b.check(nm, f"{kind} short table")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nodes", [3, 18])
def test_attention_strides(nm, kind, nodes):
    """q and out inside wider rows, k and v pages interleaved in one buffer, a
    table that is part of a wider one."""
    b = Batch(kind, [150, 77], [nodes, 2], 8, 2, 128, 16, seed=15)
    T = sum(b.nodes)
    both = torch.stack([b.k.view(torch.uint8 if b.ks is not None else torch.float16),
                        b.v.view(torch.uint8 if b.ks is not None else torch.float16)], 1).cuda()
    both = both.view(b.k.dtype)
    ks = vs = None
    if b.ks is not None:
        sc = torch.stack([b.ks, b.vs], 1).cuda()
        ks, vs = sc[:, 0], sc[:, 1]
    wide_q = torch.full((T, 12 * 128), 7.0, dtype=torch.float16, device="cuda")
    wide_q[:, :8 * 128] = b.q.view(T, -1).cuda()
    wide_o = torch.full((T, 10 * 128), 7.0, dtype=torch.float16, device="cuda")
    wide_t = torch.full((2, b.table.shape[1] + 5), 10 ** 6, dtype=torch.int32, device="cuda")
    wide_t[:, :b.table.shape[1]] = b.table.cuda()
    out, lse = nm.nm_tree_attention(
        wide_q[:, :8 * 128].unflatten(1, (8, 128)), both[:, 0], both[:, 1],
        wide_t[:, :b.table.shape[1]], torch.tensor(b.ctx, dtype=torch.int32).cuda(),
        torch.tensor(b.start, dtype=torch.int32).cuda(), max(b.nodes),
        tree_mask=signed(b.masks).cuda(), k_scale=ks, v_scale=vs,
        out=wide_o[:, :8 * 128].unflatten(1, (8, 128)))
    o, l, to, tl = b.want()
    within(out, o, to, "strided out")
    within(lse, l, tl, "strided lse")
    assert (wide_o[:, 8 * 128:] == 7).all()


def test_attention_ragged_bounds(nm):
    """Nodes beyond max_nodes are not computed, sequences without nodes and
    tokens outside q_start are left alone."""
    b = Batch("fp16", [50, 60, 70], [3, 0, 9], 8, 2, 64, 16, seed=17)
    T = sum(b.nodes)
    out = torch.full((T, 8, 64), 5.0, dtype=torch.float16, device="cuda")
    lse = torch.full((T, 8), 5.0, device="cuda")
    k, v = cuda(b.k, b.v)
    nm.nm_tree_attention(b.q.cuda(), k, v, b.table.cuda(),
                         torch.tensor(b.ctx, dtype=torch.int32).cuda(),
                         torch.tensor(b.start, dtype=torch.int32).cuda(), 4,
                         tree_mask=signed(b.masks).cuda(), out=out, lse=lse)
    # with max_nodes 4 the third sequence's nodes are its first four only
    b.nodes[2] = 4
    b.start = [0, 3, 3, 7]
    b.q, keep = b.q[:7], b.masks
    b.masks = [m & 15 for m in keep[:7]]
    o, l, to, tl = b.want()
    within(out[:7], o, to, "first nodes")
    within(lse[:7], l, tl, "first nodes' lse")
    assert (out[7:] == 5).all() and (lse[7:] == 5).all()


INT_MIN = -2 ** 31


@pytest.mark.parametrize("nodes", [2, 7])
@pytest.mark.parametrize("start,rows", [([0, 3, INT_MIN, 7], [3, 0, 7]), ([0, 3, -5, 7], [3, 0, 7]),
                                        ([INT_MIN, 3, 2 ** 31 - 1, INT_MIN], [3, 9, 0])])
def test_starts_out_of_range(nm, nodes, start, rows):
    """Starts below 0, beyond the tokens or before the last one: the other sequences
    are as ever, and nothing beyond the tokens is read or written."""
    b = Batch("fp16", [50, 60, 70], [3, 0, 9], 8, 2, 64, 16, seed=17, spoil=False)
    T = 12
    k, v, q = cuda(b.k, b.v, b.q)
    st = torch.tensor(start, dtype=torch.int32).cuda()
    ctx = torch.tensor(b.ctx, dtype=torch.int32).cuda()
    wide = torch.full((T + 70, 8, 64), 5.0, dtype=torch.float16, device="cuda")
    lse = torch.full((T + 70, 8), 5.0, device="cuda")
    nm.nm_tree_attention(q, k, v, b.table.cuda(), ctx, st, nodes, out=wide[:T], lse=lse[:T])
    done = set()
    for s in range(3):
        first = max(start[s], 0)
        n = min(nodes, rows[s])
        if n:
            done |= set(range(first, first + n))
    left = [t for t in range(T + 70) if t not in done]
    assert (wide[left] == 5).all() and (lse[left] == 5).all()
    assert (lse[sorted(done)] != 5).all()
    V = 40
    logits = torch.zeros((T, V), device="cuda")
    logits[:, 9] = 30.0
    zero = torch.zeros(T, dtype=torch.int32, device="cuda")
    path, count, token = nm.nm_tree_verify(logits, zero, zero - 1, st, nodes, temperature=0.0)
    assert count.tolist() == [min(1, r) for r in rows]
    assert token.tolist() == [9 if r else -1 for r in rows]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nodes", [1, 4, 32])
def test_attention_workspace_and_repeats(nm, kind, nodes):
    """The same bits every time, through one workspace that other calls used in
    between, on a stream of its own."""
    b = Batch(kind, [5000, 30], [nodes, nodes], 8, 1, 128, 64, seed=19)
    c = Batch(kind, [100] * 20, [2] * 20, 8, 1, 128, 64, seed=20)
    need = max(nm.nm_tree_attention_workspace_bytes(2, 8, 1, 128, nodes),
               nm.nm_tree_attention_workspace_bytes(20, 8, 1, 128, 2))
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
    first = b.check(nm, "first", workspace=ws)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        c.run(nm, workspace=ws)
        second = b.run(nm, workspace=ws)
    side.synchronize()
    assert torch.equal(first[0], second[0]) and torch.equal(first[1], second[1])


@pytest.mark.parametrize("kind", KINDS)
def test_attention_workspace_of_other_shapes(nm, kind):
    """Calls of different shapes through one workspace, zero-filled once: few and
    many items, cut and whole, few and many rows."""
    calls = [Batch(kind, [6000], [1], 8, 1, 128, 64, seed=30),
             Batch(kind, [700 + 61 * i for i in range(25)], [2] * 25, 8, 4, 128, 64, seed=31),
             Batch(kind, [900, 2500, 40], [32, 5, 17], 8, 2, 128, 64, seed=32),
             Batch(kind, [5000, 30], [4, 3], 8, 2, 64, 16, seed=33),
             Batch(kind, [300 + 97 * i for i in range(40)], [12] * 40, 8, 2, 64, 16, seed=34)]
    need = max(nm.nm_tree_attention_workspace_bytes(len(b.nodes), b.q.shape[1], b.k.shape[1], b.q.shape[2], max(b.nodes))
               for b in calls)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for turn in range(2):
        for i in (0, 1, 2, 3, 1, 4, 0, 3, 2):
            calls[i].check(nm, f"turn {turn}, call {i}", workspace=ws)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nodes", [1, 24])
def test_attention_workspace_of_a_given_stream(nm, kind, nodes):
    """The zeros of a workspace that a call makes for itself are there before its
    kernels on the stream that it was given, however busy the current one is."""
    b = Batch(kind, [9000, 400], [nodes, nodes], 8, 2, 128, 64, seed=35)
    want = b.check(nm, "on the current stream")
    need = nm.nm_tree_attention_workspace_bytes(2, 8, 2, 128, nodes)
    args = cuda(b.q, b.k, b.v, b.table, torch.tensor(b.ctx, dtype=torch.int32),
                torch.tensor(b.start, dtype=torch.int32))
    ks, vs = cuda(b.ks, b.vs)
    mask = signed(b.masks).cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        used = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # what the allocator gives next
        torch.cuda.synchronize()
        del used
        torch.cuda._sleep(100_000_000)
        out, lse = nm.nm_tree_attention(*args, nodes, tree_mask=mask, k_scale=ks, v_scale=vs, stream=side)
        side.synchronize()
        with torch.cuda.stream(side):
            same = bool((out == want[0]).all()) and bool((lse == want[1]).all())
        torch.cuda.synchronize()
        assert same


def test_attention_long_offsets(nm):
    """A cache whose byte and element offsets pass 2^32: the sequence's pages lie
    at both of its ends."""
    dim, heads, page = 128, 8, 64
    pages = (1 << 32) // (heads * page * dim) + 50
    k = torch.zeros((pages, heads, page, dim), dtype=torch.int8, device="cuda")
    v = torch.zeros_like(k)
    ks = torch.zeros((pages, heads, page), device="cuda")
    vs = torch.zeros_like(ks)
    b = Batch("int8", [380], [6], 16, heads, dim, page, seed=21)
    far = torch.tensor([pages - 1 - 3 * i if i % 2 == 0 else i for i in range(b.k.shape[0])])
    for a, c in ((k, b.k), (v, b.v), (ks, b.ks), (vs, b.vs)):
        a[far.cuda()] = c.cuda()
    table = torch.where(b.table >= 0, far[b.table.clamp_min(0).long()].to(torch.int32), -1)
    out, lse = nm.nm_tree_attention(b.q.cuda(), k, v, table.cuda(),
                                    torch.tensor(b.ctx, dtype=torch.int32).cuda(),
                                    torch.tensor(b.start, dtype=torch.int32).cuda(), 6,
                                    tree_mask=signed(b.masks).cuda(), k_scale=ks, v_scale=vs)
    o, l, to, tl = b.want()
    within(out, o, to, "far pages out")
    within(lse, l, tl, "far pages lse")
    # and the same rows read back
    slots = (far[:4, None] * page + torch.arange(page)).reshape(-1).cuda()
    rk, rv = nm.nm_cache_read(k, v, slots, k_scale=ks, v_scale=vs)
    want = (b.k[:4].float() * b.ks[:4, ..., None]).half().transpose(1, 2).reshape(-1, heads, dim)
    ok = ~torch.isnan(want)
    assert torch.equal(rk.cpu()[ok], want[ok])


def test_attention_graph(nm):
    """The call replays from a CUDA graph on new contents of its buffers."""
    b = Batch("fp16", [700], [4], 32, 8, 128, 16, seed=23)
    k, v, q = cuda(b.k, b.v, b.q)
    args = (k, v, b.table.cuda(), torch.tensor(b.ctx, dtype=torch.int32).cuda(),
            torch.tensor(b.start, dtype=torch.int32).cuda(), 4)
    mask = signed(b.masks).cuda()
    ws = torch.zeros(max(16, nm.nm_tree_attention_workspace_bytes(1, 32, 8, 128, 4)),
                     dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((4, 32), device="cuda")
    nm.nm_tree_attention(q, *args, tree_mask=mask, workspace=ws, out=out, lse=lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nm.nm_tree_attention(q, *args, tree_mask=mask, workspace=ws, out=out, lse=lse)
    b.q = (b.q.float() * -0.7).half()
    q.copy_(b.q)
    for _ in range(3):
        out.zero_()
        g.replay()
    torch.cuda.synchronize()
    o, l, to, tl = b.want()
    within(out, o, to, "replayed out")
    within(lse, l, tl, "replayed lse")


# ---- rotary positions, cache write and read ------------------------------------------
def append_case(kind, tokens, q_heads, kv_heads, dim, page, seed, top=5000):
    gen = torch.Generator().manual_seed(seed)
    pages = -(-tokens // page) + 3
    x = torch.randn((tokens, q_heads + 2 * kv_heads, dim), generator=gen)
    x[..., 1] *= 15
    pos = torch.randint(0, top, (tokens,), generator=gen).to(torch.int32)
    slots = torch.randperm(pages * page, generator=gen)[:tokens].contiguous()
    shape = (pages, kv_heads, page, dim)
    k, v = (torch.zeros(shape, dtype=ref.DTYPES[kind], device="cuda") for _ in range(2))
    ks = vs = None
    if kind != "fp16":
        ks, vs = (torch.zeros(shape[:3], device="cuda") for _ in range(2))
    return x.half(), pos, slots, k, v, ks, vs


def check_append(nm, kind, x, pos, slots, caches, freq, interleaved, mscale, q):
    """q, and the cache's rows: the rotation's fp32 error is at most 2^-21 (|a| +
    |b|) (cos and sin to 2^-22, two products and a sum); q and fp16 rows are
    rounded once; a code lies within half a step (and the fp32 error of x /
    scale, 2^-21 max|x|) of its value, or a neighbour where that is a tie."""
    k, v, ks, vs = caches
    H, page = k.shape[1], k.shape[2]
    Q = x.shape[1] - 2 * H
    y, size = ref.rotate(x[:, :Q + H], pos, freq, interleaved, mscale)
    if q is not None:
        within(q, y[:, :Q], 2.0 ** -11 * y[:, :Q].abs() + 2.0 ** -21 * size[:, :Q] + 2.0 ** -25, "q")
    for cache, scale, row, sz, name in ((k, ks, y[:, Q:], size[:, Q:], "k"),
                                        (v, vs, x[:, Q + H:].double(), x[:, Q + H:].double().abs(), "v")):
        pg, off = slots // page, slots % page
        got = cache.cpu().view(torch.uint8 if scale is not None else torch.float16)[pg, :, off]
        got = got.view(cache.dtype).float().double()
        eps = 2.0 ** -21 * sz
        if scale is None:
            within(got, row, 2.0 ** -11 * row.abs() + eps + 2.0 ** -25, name)
            continue
        sc = scale.cpu()[pg, :, off].double()
        s = row.abs().amax(-1) / ref.CODE_MAX[kind]
        worst = eps.amax(-1)
        within(sc, s, 2.0 ** -22 * s + worst / ref.CODE_MAX[kind] + 1e-45, name + " scale")
        tol = ref.code_step(row, s, kind) / 2 * (1 + 2.0 ** -20) + eps + 2.0 ** -20 * row.abs() \
            + worst[..., None] / 100 + 1e-45
        within(got * sc[..., None], row, tol, name + " codes")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(128, 128), (128, 64), (128, 36), (64, 64), (64, 20), (64, 0),
                                     (128, 2)])
def test_append_layouts(nm, kind, interleaved, dim, rot):
    x, pos, slots, *caches = append_case(kind, 37, 6, 2, dim, 16, seed=rot + dim)
    freq = nm.nm_rope_inv_freq(rot, 10000.0)
    q = nm.nm_rope_append(x.view(37, -1).cuda(), caches[0], caches[1], pos.cuda(), slots.cuda(),
                          freq, 6, k_scale=caches[2], v_scale=caches[3], interleaved=interleaved,
                          mscale=1.25)
    check_append(nm, kind, x, pos, slots, caches, freq.cpu(), interleaved,
                 1.25 if rot else 1.0, q)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens,q_heads,kv_heads,dim", [(1, 32, 8, 128), (1, 1, 1, 64), (3, 28, 4, 64),
                                                         (700, 8, 1, 128), (64, 64, 8, 128)])
def test_append_sizes(nm, kind, tokens, q_heads, kv_heads, dim):
    x, pos, slots, *caches = append_case(kind, tokens, q_heads, kv_heads, dim, 64, seed=tokens,
                                         top=131072)
    freq = nm.nm_rope_inv_freq(dim, 500000.0, "banded", 8.0)
    q = nm.nm_rope_append(x.view(tokens, -1).cuda(), caches[0], caches[1], pos.cuda(),
                          slots.cuda(), freq, q_heads, k_scale=caches[2], v_scale=caches[3])
    check_append(nm, kind, x, pos, slots, caches, freq.cpu(), False, 1.0, q)


@pytest.mark.parametrize("kind", KINDS)
def test_append_again_commits_the_same_rows(nm, kind):
    """Rows appended again to other slots are the same bits; without q; slots out
    of range are not written; qkv inside wider rows."""
    x, pos, slots, k, v, ks, vs = append_case(kind, 9, 4, 2, 128, 16, seed=3)
    freq = nm.nm_rope_inv_freq(128)
    wide = torch.zeros((9, 9 * 128), dtype=torch.float16, device="cuda")
    wide[:, :8 * 128] = x.view(9, -1).cuda()
    q = nm.nm_rope_append(wide[:, :8 * 128], k, v, pos.cuda(), slots.cuda(), freq, 4, k_scale=ks,
                          v_scale=vs)
    before = [t.clone() for t in (k, v, ks, vs) if t is not None]
    first = nm.nm_cache_read(k, v, slots.cuda(), ks, vs)
    out = slots.clone()
    out[0], out[1], out[2] = -1, k.shape[0] * 16, 1 << 60
    none = nm.nm_rope_append(wide[:, :8 * 128], k, v, pos.cuda(), out.cuda(), freq, 4, k_scale=ks,
                             v_scale=vs, want_q=False)
    assert none is None
    for a, b in zip(before, [t for t in (k, v, ks, vs) if t is not None]):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    free = [i for i in range(k.shape[0] * 16) if i not in set(slots.tolist())][:3]
    dst = torch.tensor(free, device="cuda")
    nm.nm_rope_append(wide[4:7, :8 * 128], k, v, pos[4:7].cuda().contiguous(), dst, freq, 4,
                      k_scale=ks, v_scale=vs, want_q=False)
    again = nm.nm_cache_read(k, v, dst, ks, vs)
    assert torch.equal(again[0], first[0][4:7]) and torch.equal(again[1], first[1][4:7])
    assert q.shape == (9, 4, 128)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("lo,hi", [(2 ** 17, 2 ** 18), (2 ** 20, 2 ** 21), (2 ** 23, 2 ** 24 + 99),
                                   (2 ** 27, 2 ** 28), (2 ** 31 - 5000, 2 ** 31 - 1)])
def test_append_far_positions(nm, interleaved, lo, hi):
    """Positions up to the largest int32, above 2^24 too, where they are no fp32
    numbers.  Tolerance: two pairs of cosine and sine, 2^-23 each, make one, 2^-21.4
    with the roundings; two products and a sum; q and fp16 rows are rounded once."""
    T, Q, H, D = 150, 4, 2, 128
    x, pos, slots, k, v, _, _ = append_case("fp16", T, Q, H, D, 16, seed=lo % 1000)
    gen = torch.Generator().manual_seed(lo % 997)
    pos = torch.randint(lo, hi, (T,), generator=gen).to(torch.int32)
    pos[-1] = hi
    freq = nm.nm_rope_inv_freq(D, 10000.0, device="cpu")
    freq[3] = 1.75  # a frequency may be above 1
    q = nm.nm_rope_append(x.view(T, -1).cuda(), k, v, pos.cuda(), slots.cuda(), freq.cuda(), Q, interleaved=interleaved)
    # the product of 31 and 24 bits does not fit a double
    angle = pos.numpy().astype(np.longdouble)[:, None] * freq.numpy().astype(np.longdouble)
    c, s = (torch.from_numpy(f(angle).astype(np.float64))[:, None] for f in (np.cos, np.sin))
    h = D // 2
    ia = torch.arange(0, D, 2) if interleaved else torch.arange(h)
    ib = ia + 1 if interleaved else ia + h
    y, size = x[:, :Q + H].double(), x[:, :Q + H].double()
    a, b = x[:, :Q + H, ia].double(), x[:, :Q + H, ib].double()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    tol = 2.0 ** -11 * y.abs() + 2.0 ** -20 * size + 2.0 ** -25
    within(q, y[:, :Q], tol[:, :Q], "q")
    within(k.cpu()[slots // 16, :, slots % 16], y[:, Q:], tol[:, Q:], "k")


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_append_zero_and_non_finite_rows(nm, kind):
    x, pos, slots, k, v, ks, vs = append_case(kind, 4, 2, 1, 64, 8, seed=5)
    x[0, 3] = 0                      # token 0's values
    x[1, 3, 5] = float("inf")
    x[2, 3, 6] = NAN
    x[3, 3] = 0
    x[3, 3, 0] = 6e-8                # the smallest subnormal
    nm.nm_rope_append(x.view(4, -1).cuda(), k, v, pos.cuda(), slots.cuda(),
                      nm.nm_rope_inv_freq(64), 2, k_scale=ks, v_scale=vs)
    rk, rv = nm.nm_cache_read(k, v, slots.cuda(), ks, vs)
    assert (rv[0] == 0).all()
    assert torch.isnan(rv[1]).all() and torch.isnan(rv[2]).all()
    assert torch.equal(rv[3].cpu(), x[3, 3:4])
    assert torch.isfinite(rk).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,heads,dim,page", [(1, 1, 64, 8), (77, 8, 128, 16), (1000, 3, 64, 128)])
def test_read_bits(nm, kind, rows, heads, dim, page):
    """code * scale in fp32, rounded once: the same bits as the CPU's."""
    gen = torch.Generator().manual_seed(rows)
    pages = -(-rows // page) + 2
    k, v, ks, vs = ref.random_cache(kind, pages, heads, page, dim, gen, 3.0)
    slots = torch.randint(0, pages * page, (rows,), generator=gen)
    if rows > 5:
        slots[3], slots[5] = -7, pages * page
    gk, gv = nm.nm_cache_read(*cuda(k, v, slots), *(cuda(ks, vs)))
    for got, c, s in ((gk, k, ks), (gv, v, vs)):
        x = c.float() if s is None else c.float() * s[..., None]
        ok = (slots >= 0) & (slots < pages * page)
        at = torch.where(ok, slots, 0)
        want = torch.where(ok[:, None, None], x[at // page, :, at % page], 0.0).half()
        assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("kind", KINDS)
def test_read_of_one_half(nm, kind):
    """Only k or only v asked for: the same rows, and the other half is not read (its
    scales and codes do not matter)."""
    from sparse_spmv_memory_gb300.decode import _Cache
    import ctypes
    gen = torch.Generator().manual_seed(2)
    k, v, ks, vs = cuda(*ref.random_cache(kind, 9, 3, 16, 64, gen))
    slots = torch.randint(0, 9 * 16, (50,), generator=gen).cuda()
    rk, rv = nm.nm_cache_read(k, v, slots, ks, vs)
    P = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    c = _Cache(k=P(k), v=P(v), k_scale=P(ks), v_scale=P(vs), pages=9, page_stride=3 * 16 * 64,
               scale_page_stride=48, kv_heads=3, page_size=16, head_dim=64, type=KINDS.index(kind))
    for want, which in ((rk, 0), (rv, 1)):
        out = torch.zeros_like(want)
        assert nm.lib().nm_cache_read(ctypes.byref(c), P(slots), 50, None if which else P(out),
                                      P(out) if which else None, torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(out, want)


# ---- verification --------------------------------------------------------------------
def verify_case(seed, seqs, nodes, vocab, drafted, temperature, fp32, closeness=0.7, fan=3):
    """Inputs of a walk whose decisions all lie 1e-4 off their boundaries: fp32
    sums of the vocabulary are good to a few 1e-6."""
    while True:
        rng, rnd = np.random.default_rng(seed), random.Random(seed)
        n = [max(1, nodes - rnd.randrange(3)) for _ in range(seqs)]
        start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        N = int(start[-1])
        logits = (rng.standard_normal((N, vocab)) * 2.5).astype(np.float32 if fp32 else np.float16)
        guess = logits.astype(np.float64) + rng.standard_normal((N, vocab)) * closeness
        q = np.exp(guess - guess.max(1, keepdims=True))
        q = (q / q.sum(1, keepdims=True)).astype(np.float32)
        parents, ids = np.full(N, -1, np.int32), np.zeros(N, np.int32)
        for s in range(seqs):
            kids = [0] * n[s]
            for i in range(1, n[s]):
                p = rnd.choice([j for j in range(i) if kids[j] < fan])
                parents[start[s] + i] = p
                row = start[s] + p
                if drafted:
                    ids[start[s] + i] = rng.choice(vocab, p=q[row].astype(np.float64)
                                                   / q[row].astype(np.float64).sum())
                else:
                    ids[start[s] + i] = np.argsort(-guess[row], kind="stable")[min(kids[p], vocab - 1)]
                kids[p] += 1
        accept = rng.random(N).astype(np.float32)
        race = np.maximum(rng.exponential(size=(seqs, vocab)), 1e-30).astype(np.float32)
        want = ref.verify(logits, ids, parents, start, accept, race, q if drafted else None,
                          temperature, nodes)
        if want[3] > 1e-4:
            return logits, ids, parents, start, accept, race, q if drafted else None, want[:3]
        seed += 1000


def run_verify(nm, case, nodes, temperature, **kw):
    logits, ids, parents, start, accept, race, q = (None if a is None else torch.from_numpy(a).cuda()
                                                    for a in case[:7])
    return nm.nm_tree_verify(logits, ids, parents, start, nodes, draft=q, accept=accept, race=race,
                             temperature=temperature, **kw)


def same(got, want):
    for g, w, what in zip(got, want, ("path", "count", "token")):
        assert np.array_equal(g.cpu().numpy(), w), what


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("temperature", [0.0, 0.7, 1.0])
@pytest.mark.parametrize("seqs,nodes,vocab", [(1, 1, 1), (1, 2, 5), (3, 7, 33), (5, 20, 1000),
                                              (2, 64, 32000), (17, 5, 4097)])
def test_verify_walks(nm, fp32, drafted, temperature, seqs, nodes, vocab):
    case = verify_case(seqs * 100 + nodes, seqs, nodes, vocab, drafted, temperature, fp32)
    same(run_verify(nm, case, nodes, temperature), case[7])


@pytest.mark.parametrize("drafted", [True, False])
def test_verify_far_draft_and_repeated_children(nm, drafted):
    """A draft far from the target (most children rejected, several a node) and
    children with equal tokens."""
    for seed in range(6):
        case = list(verify_case(seed, 4, 24, 300, drafted, 1.0, True, closeness=4.0, fan=8))
        same(run_verify(nm, case, 24, 1.0), case[7])


def test_verify_forbidden_tokens_and_bad_rows(nm):
    """Logits of -inf have no weight; a row that is all -inf, or has NaN or +inf,
    ends the walk with token -1; nodes with bad parents or tokens are never
    visited; a sequence without nodes."""
    V = 100
    logits = torch.full((6, V), float("-inf"))
    logits[0, 7] = 0.0                    # token 7 for certain
    logits[1, 50] = NAN                   # sequence 0, node 1
    logits[2, 3] = 1.0                    # sequence 1, node 0: token 3
    logits[4] = 0.0
    logits[4, 9] = float("inf")           # sequence 3, node 0
    ids = torch.tensor([0, 7, 0, 3, 0, 5], dtype=torch.int32)
    par = torch.tensor([-1, 0, -1, 5, -1, 0], dtype=torch.int32)
    start = torch.tensor([0, 2, 4, 4, 6], dtype=torch.int32)
    for temperature in (1.0, 0.0):
        path, count, token = nm.nm_tree_verify(
            *cuda(logits, ids, par, start), 2, accept=torch.full((6,), 0.5).cuda(),
            race=torch.ones((4, V)).cuda(), temperature=temperature)
        assert path.tolist() == [[0, 1], [0, -1], [-1, -1], [0, -1]]
        assert count.tolist() == [2, 1, 0, 1]
        assert token.tolist() == [-1, 3, -1, -1]
    ids[1] = V  # out of the vocabulary
    path, count, token = nm.nm_tree_verify(
        *cuda(logits, ids, par, start), 2, accept=torch.full((6,), 0.5).cuda(),
        race=torch.ones((4, V)).cuda())
    assert path[0].tolist() == [0, -1] and int(token[0]) == 7


@pytest.mark.parametrize("temperature", [0.0, 1.0])
def test_verify_ties_take_the_lowest_index(nm, temperature):
    V = 5000
    logits = torch.zeros((1, V))
    logits[0, 1234] = logits[0, 1111] = logits[0, 4999] = 3.0
    path, count, token = nm.nm_tree_verify(
        logits.cuda(), torch.zeros(1, dtype=torch.int32).cuda(),
        torch.full((1,), -1, dtype=torch.int32).cuda(), torch.tensor([0, 1], dtype=torch.int32).cuda(),
        1, accept=torch.zeros(1).cuda(), race=torch.ones((1, V)).cuda(), temperature=temperature)
    assert int(token[0]) == 1111


@pytest.mark.parametrize("fp32", [False, True])
def test_verify_strides(nm, fp32):
    """Rows inside wider ones, at odd element offsets (no vector loads)."""
    case = verify_case(77, 3, 9, 1001, True, 0.9, fp32)
    logits, ids, parents, start, accept, race, q = (torch.from_numpy(a).cuda() for a in case[:7])

    def inside(t):
        w = torch.full((t.shape[0], t.shape[1] + 6), NAN, dtype=t.dtype, device="cuda")
        w[:, 1:1 + t.shape[1]] = t
        return w[:, 1:1 + t.shape[1]]
    got = nm.nm_tree_verify(inside(logits), ids, parents, start, 9, draft=inside(q), accept=accept,
                            race=inside(race), temperature=0.9)
    same(got, case[7])


@pytest.mark.parametrize("drafted", [True, False])
def test_verify_keeps_the_targets_distribution(nm, drafted):
    """Over many sequences the first kept token is distributed as the target's:
    each frequency within 5 standard deviations."""
    rng = np.random.default_rng(5)
    S, V = 40000, 6
    p = np.array([0.35, 0.25, 0.2, 0.1, 0.07, 0.03])
    q = np.array([0.05, 0.4, 0.1, 0.3, 0.1, 0.05])
    logits = np.tile(np.log(p).astype(np.float32), (3 * S, 1))
    kids = rng.choice(V, size=(S, 2), p=q) if drafted else np.tile([1, 3], (S, 1))
    ids = np.zeros((S, 3), np.int32)
    ids[:, 1:] = kids
    parents = np.tile(np.array([-1, 0, 0], np.int32), S)
    start = np.arange(0, 3 * S + 1, 3, dtype=np.int32)
    draft = np.tile(q.astype(np.float32), (3 * S, 1)) if drafted else None
    case = (logits, ids.reshape(-1), parents, start, rng.random(3 * S).astype(np.float32),
            np.maximum(rng.exponential(size=(S, V)), 1e-30).astype(np.float32), draft)
    path, count, token = run_verify(nm, case, 3, 1.0)
    path, count, token = path.cpu().numpy(), count.cpu().numpy(), token.cpu().numpy()
    kept = np.where(count > 1, ids[np.arange(S), np.maximum(path[:, 1], 0)], token)
    f = np.bincount(kept, minlength=V) / S
    assert (np.abs(f - p) < 5 * np.sqrt(p * (1 - p) / S)).all(), (f, p)
    assert 0.2 < (count > 1).mean() < 0.95


@pytest.mark.parametrize("vocab", [1000, 300007])
@pytest.mark.parametrize("fp32", [True, False])
def test_verify_little_mass_left(nm, vocab, fp32):
    """Without draft, after a rejection of a token of probability 1 - d: what is left, d
    = 2e-6 to 3e-2, is a sum as exact as its terms.  The second child is tried at 0.5 %
    to either side of its share, the race is decided by far: fp32 sums and
    exponentials are good to 1e-5 here."""
    rng = np.random.default_rng(vocab)
    S = 48 if vocab < 10000 else 6
    N = 4 * S
    logits = np.zeros((N, vocab), np.float32)
    ids = np.tile(np.array([0, 3, 8, vocab - 1], np.int32), S)       # node 0 has the children 1, 2, 3
    parents = np.tile(np.array([-1, 0, 0, 0], np.int32), S)
    start = np.arange(0, N + 1, 4, dtype=np.int32)
    accept = np.full(N, 1 - 2.0 ** -24, np.float32)
    race = np.ones((S, vocab), np.float32)
    race[:, 11] = 1e-9
    for s in range(S):
        x = rng.normal(size=vocab) * 0.5
        x[3] = x[8] = x[-1] = -np.inf
        rest = np.exp(x).sum()
        share2, share3 = rng.uniform(0.2, 0.5), rng.uniform(0.2, 0.4)
        x[8], x[-1] = np.log(rest * share2 / (1 - share2 - share3)), np.log(rest * share3 / (1 - share2 - share3))
        x[3] = np.log(np.exp(x).sum()) + np.log(1 / 10 ** rng.uniform(-5.7, -1.5))
        logits[4 * s] = x
    if not fp32:
        logits = logits.astype(np.float16)
    for s in range(S):
        w = np.exp(logits[4 * s].astype(np.float64) - logits[4 * s].max())
        w[3] = 0
        accept[4 * s + 2] = w[8] / w.sum() * (1 + rng.choice([-1, 1]) * 0.005)
        w[8] = 0
        accept[4 * s + 3] = w[-1] / w.sum() * (1 + rng.choice([-1, 1]) * 0.005)
    want = ref.verify(logits, ids, parents, start, accept, race, None, 1.0, 4)
    assert len(set(want[0][:, 1])) == 3 or vocab > 10000
    same(run_verify(nm, (logits, ids, parents, start, accept, race, None), 4, 1.0), want[:3])


@pytest.mark.parametrize("temperature", [1e-45, 1e-40, 1e-30])
@pytest.mark.parametrize("drafted", [True, False])
def test_verify_smallest_temperatures(nm, temperature, drafted):
    """Temperatures down to the smallest number above 0: all the weight is on the
    largest logit (one that no other equals)."""
    case = verify_case(31, 6, 9, 500, drafted, 0.0, True)
    logits, ids, parents, start, accept, race, q, _ = case
    assert all(np.sort(r)[-1] > np.sort(r)[-2] for r in logits)
    got = run_verify(nm, case, 9, temperature)
    want = ref.verify(logits, ids, parents, start, accept, race, q, max(temperature, 1e-12), 9)
    same(got, want[:3])


# ---- wide batches, long vocabularies, the calls' own refusals -------------------------
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nodes,q_heads", [(1, 8), (6, 8), (14, 8), (20, 16), (40, 16)])
def test_attention_many_sequences(nm, kind, nodes, q_heads):
    """More sequences than a warp's lanes, all of their own length, one long, some
    without nodes: rows 4 .. 320 of 2 key heads, every kernel."""
    rnd = random.Random(nodes)
    ctx = [rnd.choice([0, 1, 17, 64, 127, 130]) for _ in range(45)] + [900]
    ns = [rnd.randint(0, nodes) for _ in range(45)] + [nodes]
    Batch(kind, ctx, ns, q_heads, 2, 64, 8, seed=nodes).check(nm, f"{kind} 46 sequences")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nodes", [3, 5, 9, 17, 33, 64])
def test_attention_rows_of_every_tile(nm, kind, nodes):
    """Rows just above 16, 32, 64, 128, 256 a key head: every row tile and its last
    rows; the maximum grows over the positions, so that sums are rescaled."""
    b = Batch(kind, [1300], [nodes], 7, 1, 128, 32, seed=nodes)
    order = torch.zeros(b.k.shape[0], dtype=torch.int64)
    order[b.table[0].clamp_min(0).long()] = torch.arange(b.table.shape[1])
    grow = (0.2 + 0.15 * order.float())[:, None, None]
    if b.ks is None:
        b.k = (b.k.float() * grow[..., None]).half()
    else:
        b.ks = b.ks * grow
    b.check(nm, f"{kind} {7 * nodes} rows")
    b.scale = -b.scale
    b.check(nm, f"{kind} {7 * nodes} rows, negative scale")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("q_heads,kv_heads,nodes,ns", [
    (64, 8, 33, [1, 33, 3, 1, 2, 1, 5, 4] * 2),      # most sequences have one of two row tiles
    (16, 2, 64, [64, 7, 1, 12, 0, 16, 30, 1] * 2),
    (28, 4, 40, [40, 18, 19, 3] * 2),                # 280, 126, 133, 21 rows: last tiles of 24 and 133
    (64, 1, 6, [6] * 12)])                           # 384: every sequence's second tile has 128
def test_attention_batches_with_one_of_two_row_tiles(nm, kind, q_heads, kv_heads, nodes, ns):
    """More than 128 rows a key head at most, but items that have no more than 128,
    and many of them in a block (a long sequence makes the blocks' ranges long): one
    of the block's two streams is idle."""
    rnd = random.Random(q_heads + nodes)
    ctx = [60000 if kv_heads < 4 else 30000] + [rnd.choice([0, 5, 100, 127, 128, 250]) for _ in ns]
    b = Batch(kind, ctx, [1] + ns, q_heads, kv_heads, 64, 16, seed=nodes)
    first = b.check(nm, f"{kind} {q_heads}/{kv_heads}")
    for _ in range(20):
        out, lse = b.run(nm)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert nm.nm_wait_timeouts() == 0


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_heads,nodes", [(8, 3), (16, 5), (64, 3)])
def test_attention_batches_of_edge_tiles(nm, dim, q_heads, nodes):
    """Every value tile of an fp16 cache has nodes or absent rows in it, so that each
    is looked at before the product; many such items follow one another in a block,
    and a page that is missing altogether now and then."""
    rnd = random.Random(q_heads)
    ctx = [rnd.randrange(100) for _ in range(160)] + [40000]
    b = Batch("fp16", ctx, [rnd.randint(1, nodes) for _ in range(160)] + [1], q_heads, 1, dim, 16, seed=q_heads)
    for s in range(0, 160, 7):
        b.table[s, 0] = -1
    first = b.check(nm, f"{q_heads}x{dim}")
    for _ in range(20):
        out, lse = b.run(nm)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert nm.nm_wait_timeouts() == 0


@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("vocab", [131073, 140001, 300007])
def test_verify_long_vocabularies(nm, drafted, vocab):
    """Beyond what a cluster's threads hold with 16 elements each, and with 32."""
    case = verify_case(vocab, 2, 6, vocab, drafted, 0.8, False)
    same(run_verify(nm, case, 6, 0.8), case[7])
    case = verify_case(vocab, 2, 6, vocab, drafted, 0.0, True)
    same(run_verify(nm, case, 6, 0.0), case[7])


def test_verify_many_sequences(nm):
    """More sequences than run at the same time, every one as in the reference."""
    case = verify_case(9, 200, 5, 33000, True, 0.9, False)
    same(run_verify(nm, case, 5, 0.9), case[7])


@pytest.mark.parametrize("kind", KINDS)
def test_append_and_read_interleaved_pages(nm, kind):
    """K and V pages side by side in one buffer, written on a stream of its own."""
    x, pos, slots, k, v, ks, vs = append_case(kind, 21, 4, 2, 64, 8, seed=8)
    raw = torch.zeros((k.shape[0], 2) + k.shape[1:], dtype=torch.uint8 if ks is not None else k.dtype,
                      device="cuda").view(k.dtype)
    k2, v2 = raw[:, 0], raw[:, 1]
    ks2 = vs2 = None
    if ks is not None:
        sc = torch.zeros((k.shape[0], 2) + ks.shape[1:], device="cuda")
        ks2, vs2 = sc[:, 0], sc[:, 1]
    freq = nm.nm_rope_inv_freq(64)
    dx, dp, ds = x.view(21, -1).cuda(), pos.cuda(), slots.cuda()
    nm.nm_rope_append(dx, k, v, dp, ds, freq, 4, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    nm.nm_rope_append(dx, k2, v2, dp, ds, freq, 4, k_scale=ks2, v_scale=vs2, stream=side)
    got = nm.nm_cache_read(k2, v2, ds, k_scale=ks2, v_scale=vs2, stream=side)
    side.synchronize()
    want = nm.nm_cache_read(k, v, ds, k_scale=ks, v_scale=vs)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(k2.contiguous().view(torch.uint8), k.view(torch.uint8))


def test_binding_refusals(nm):
    """Types, shapes and layouts that the marshalling refuses, and a status of the
    library as its exception."""
    b = Batch("e4m3", [40], [3], 8, 2, 64, 16)
    k, v, ks, vs, q = cuda(b.k, b.v, b.ks, b.vs, b.q)
    table, ctx, start = b.table.cuda(), torch.tensor([40], dtype=torch.int32).cuda(), \
        torch.tensor([0, 3], dtype=torch.int32).cuda()

    def attend(q=q, k=k, v=v, table=table, ctx=ctx, start=start, n=3, **kw):
        kw = dict(dict(k_scale=ks, v_scale=vs), **kw)
        return nm.nm_tree_attention(q, k, v, table, ctx, start, n, **kw)
    attend()
    for bad in (dict(q=q.float()), dict(q=q.transpose(0, 1)), dict(k=k.view(torch.uint8)),
                dict(k=k[:, :, ::2]), dict(table=table.long()), dict(ctx=ctx.long()),
                dict(start=start[:1]), dict(k_scale=None), dict(v_scale=vs.half()),
                dict(tree_mask=torch.zeros(2, dtype=torch.int64, device="cuda")),
                dict(out=torch.empty((3, 4, 64), dtype=torch.float16, device="cuda")),
                dict(lse=torch.empty(7, device="cuda")), dict(q=q.cpu())):
        with pytest.raises(ValueError):
            attend(**bad)
    with pytest.raises(TypeError):
        attend(q=None)
    with pytest.raises(nm.NMError) as e:
        attend(n=65)
    assert e.value.status == 2
    with pytest.raises(nm.NMError) as e:
        attend(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 5
    with pytest.raises(nm.NMError) as e:
        attend(scale=float("inf"))
    assert e.value.status == 2
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        nm.nm_cache_read(k, v, slots.int(), ks, vs)
    with pytest.raises(ValueError):
        nm.nm_rope_append(q.view(3, -1)[:, :-64], k, v, start, slots, ctx.float(), 8, ks, vs)
    logits = torch.zeros((3, 10), device="cuda")
    ids = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        nm.nm_tree_verify(logits.double(), ids, ids, start, 3)
    with pytest.raises(ValueError):
        nm.nm_tree_verify(logits, ids, ids, start, 3, draft=logits[:, :5])
    with pytest.raises(nm.NMError) as e:  # sampling without random numbers
        nm.nm_tree_verify(logits, ids, ids, start, 3)
    assert e.value.status == 1


# ---- nothing to do -------------------------------------------------------------------
def test_empty_calls(nm):
    """No tokens, rows or sequences, with tensors that are really empty (their
    address is NULL): no-ops, and a batch whose sequences all have no nodes is
    answered."""
    i32, dev = torch.int32, "cuda"
    for kind in KINDS:
        shape = (4, 2, 8, 64)
        k, v = (torch.zeros(shape, dtype=ref.DTYPES[kind], device=dev) for _ in range(2))
        ks, vs = (None, None) if kind == "fp16" else (torch.zeros(shape[:3], device=dev) for _ in range(2))
        no = torch.zeros(0, dtype=torch.int64, device=dev)
        empty = torch.zeros(0, dtype=i32, device=dev)
        assert no.data_ptr() == 0
        qkv = torch.zeros((0, 8 * 64), dtype=torch.float16, device=dev)
        q = nm.nm_rope_append(qkv, k, v, empty, no, nm.nm_rope_inv_freq(64), 4, k_scale=ks, v_scale=vs)
        assert q.shape == (0, 4, 64)
        assert nm.nm_rope_append(qkv, k, v, empty, no, nm.nm_rope_inv_freq(64), 4, k_scale=ks, v_scale=vs,
                                 want_q=False) is None
        rk, rv = nm.nm_cache_read(k, v, no, ks, vs)
        assert rk.shape == rv.shape == (0, 2, 64)
        for seqs in (0, 3):
            start = torch.zeros(seqs + 1, dtype=i32, device=dev)
            table, ctx = torch.zeros((seqs, 4), dtype=i32, device=dev), torch.full((seqs,), 20, dtype=i32, device=dev)
            mask = no if seqs else None
            out, lse = nm.nm_tree_attention(q, k, v, table, ctx, start, 4, tree_mask=mask, k_scale=ks, v_scale=vs)
            assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
        some = torch.ones((5, 4, 64), dtype=torch.float16, device=dev)
        out, lse = nm.nm_tree_attention(some, k, v, torch.zeros((0, 4), dtype=i32, device=dev), empty,
                                        torch.zeros(1, dtype=i32, device=dev), 4, k_scale=ks, v_scale=vs)
        assert out.shape == (5, 4, 64)
    for seqs in (0, 3):
        for dtype in (torch.float16, torch.float32):
            logits = torch.zeros((0, 33), dtype=dtype, device=dev)
            start = torch.zeros(seqs + 1, dtype=i32, device=dev)
            for kw in (dict(temperature=0.0), dict(accept=logits.float()[:, 0], race=torch.ones((seqs, 33), device=dev)),
                       dict(accept=logits.float()[:, 0], race=torch.ones((seqs, 33), device=dev), draft=logits.float())):
                path, count, token = nm.nm_tree_verify(logits, empty, empty, start, 4, **kw)
                assert path.tolist() == [[-1] * 4] * seqs
                assert count.tolist() == [0] * seqs and token.tolist() == [-1] * seqs
    torch.cuda.synchronize()


def test_verify_refuses_any_number_of_nodes(nm):
    """More nodes than a tree may have, however many: the status of the library, and no
    path of that length is allocated first."""
    logits = torch.zeros((3, 10), device="cuda")
    ids = torch.zeros(3, dtype=torch.int32, device="cuda")
    start = torch.zeros(60001, dtype=torch.int32, device="cuda")
    for n in (65, 10 ** 6, 2 ** 31 - 1, 0, -1, -2 ** 31):
        with pytest.raises(nm.NMError) as e:
            nm.nm_tree_verify(logits, ids, ids, start, n, temperature=0.0)
        assert e.value.status == 2


@pytest.mark.parametrize("nodes", [1, 9])
def test_attention_workspace_over_an_input_refused(nm, nodes):
    """A workspace that meets any array that the call reads or writes."""
    b = Batch("int8", [40, 3], [nodes, 1], 8, 2, 64, 16, seed=2, spoil=False)
    need = nm.nm_tree_attention_workspace_bytes(2, 8, 2, 64, nodes)
    k, v, ks, vs = cuda(b.k, b.v, b.ks, b.vs)
    args = dict(q=b.q.cuda(), block_table=b.table.cuda(), ctx_len=torch.tensor(b.ctx, dtype=torch.int32).cuda(),
                q_start=torch.tensor(b.start, dtype=torch.int32).cuda(), tree_mask=signed(b.masks).cuda(),
                out=torch.empty_like(b.q.cuda()), lse=torch.empty(b.q.shape[:2], device="cuda"))
    ws = torch.zeros(need + (1 << 20), dtype=torch.uint8, device="cuda")
    for name, t in args.items():
        inside = ws[need - 64:].view(t.dtype)[:t.numel()].view(t.shape)
        inside.copy_(t)
        with pytest.raises(nm.NMError) as e:
            nm.nm_tree_attention(k_cache=k, v_cache=v, max_nodes=nodes, k_scale=ks, v_scale=vs, workspace=ws[:need],
                                 **dict(args, **{name: inside}))
        assert e.value.status == 7, name
        ws.zero_()
    nm.nm_tree_attention(k_cache=k, v_cache=v, max_nodes=nodes, k_scale=ks, v_scale=vs, workspace=ws[:need], **args)


@pytest.mark.parametrize("cache", KINDS)
def test_example_decodes_as_one_token_at_a_time(nm, cache):
    """Speculative decoding at temperature 0 gives the tokens of plain decoding, and
    some drafted tokens are accepted; at a temperature it runs."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "speculative_decode.py")
    spec = importlib.util.spec_from_file_location("speculative_decode", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    plain, none = ex.decode(2, cache, 20, 0.0, 3)
    out, accepted = ex.decode(2, cache, 20, 0.0, 3, plain)
    assert out == plain and none == 0 and accepted > 5
    warm, _ = ex.decode(2, cache, 12, 1.0, 3, plain)
    assert len(warm) == 12 and all(0 <= t < ex.VOCAB for t in warm)


# ---- waits that give up -----------------------------------------------------------------
def stalled(nm, call, limit_s=2.0):
    """Runs a call whose arrival never comes: it ends after about its limit (20 ms)
    and is counted, the next call of its kind does nothing, and after a reset the
    count is zero again."""
    import time
    torch.cuda.synchronize()
    nm.nm_wait_timeouts(reset=True)
    t0 = time.time()
    assert call() == 0
    torch.cuda.synchronize()
    assert time.time() - t0 < limit_s
    assert nm.nm_wait_timeouts() > 0


@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("vocab", [300, 20000, 128256])
@pytest.mark.parametrize("temperature", [0.0, 0.9])
def test_verify_wait_that_gives_up(nm, drafted, vocab, temperature):
    """One block of a sequence never hears of another (or of itself): it gives up,
    the others at their next exchange, in every sequence; the kernel ends."""
    case = verify_case(vocab, 5, 9, vocab, drafted, temperature, False)
    logits, ids, parents, start, accept, race, q = cuda(*(None if a is None else torch.from_numpy(a)
                                                          for a in case[:7]))
    path = torch.full((5, 9), -7, dtype=torch.int32, device="cuda")
    count, token = (torch.full((5,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    P = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    stalled(nm, lambda: nm.lib().nm_tree_verify_stall_selftest(
        P(logits), 0, vocab, vocab, P(q), vocab, P(ids), P(parents), P(start), len(ids), 5, 9, P(accept),
        P(race), vocab, temperature, P(path), P(count), P(token), 20000, torch.cuda.current_stream().cuda_stream))
    # until the reset calls return without an answer, all blocks of a cluster alike
    count.fill_(-9)
    token.fill_(-9)
    run_verify(nm, case, 9, temperature, count=count, token=token)
    torch.cuda.synchronize()
    assert (count == -9).all() and (token == -9).all()
    nm.nm_wait_timeouts(reset=True)
    same(run_verify(nm, case, 9, temperature), case[7])
    assert nm.nm_wait_timeouts() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nodes", [3, 6, 12, 40])
def test_attention_wait_that_gives_up(nm, kind, nodes):
    """The loaders of the many-row kernel bring nothing: every role gives up, tensor
    memory is freed, and the call after a reset is right."""
    from sparse_spmv_memory_gb300.decode import _Cache
    import ctypes
    b = Batch(kind, [700, 90, 1500], [nodes, 1, nodes], 16, 2, 128, 16, seed=51)
    k, v, ks, vs, q = cuda(b.k, b.v, b.ks, b.vs, b.q)
    table, ctx, start = cuda(b.table, torch.tensor(b.ctx, dtype=torch.int32), torch.tensor(b.start, dtype=torch.int32))
    mask = signed(b.masks).cuda()
    T = q.shape[0]
    out, lse = torch.zeros_like(q), torch.zeros((T, 16), device="cuda")
    need = nm.nm_tree_attention_workspace_bytes(3, 16, 2, 128, nodes)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    P = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    c = _Cache(k=P(k), v=P(v), k_scale=P(ks), v_scale=P(vs), pages=k.shape[0], page_stride=2 * 16 * 128,
               scale_page_stride=32, kv_heads=2, page_size=16, head_dim=128, type=KINDS.index(kind))
    stalled(nm, lambda: nm.lib().nm_tree_attention_stall_selftest(
        P(q), 16 * 128, T, 16, 3, P(start), nodes, ctypes.byref(c), P(table), table.shape[1], table.shape[1],
        P(ctx), P(mask), b.scale, P(out), 16 * 128, P(lse), P(ws), need, 20000,
        torch.cuda.current_stream().cuda_stream))
    b.run(nm, workspace=ws)  # returns without an answer
    torch.cuda.synchronize()
    nm.nm_wait_timeouts(reset=True)
    b.check(nm, f"{kind} after a reset", workspace=ws)
    assert nm.nm_wait_timeouts() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nodes", [3, 6, 12, 24])
def test_attention_gives_up_with_copies_in_flight(nm, kind, nodes):
    """Half of the blocks give up soon; the others, with milliseconds of work before
    them, then give up in the midst of it, copies and products in flight: they end as
    well, and the next call is right."""
    from sparse_spmv_memory_gb300.decode import _Cache
    import ctypes
    S, H, G, D, page, L = 128, 8, 8, 64, 64, 65536
    gen = torch.Generator("cuda").manual_seed(nodes)
    pages = L // page + 1
    k, v = (torch.randn((pages, H, page, D), generator=gen, device="cuda") for _ in range(2))
    ks = vs = None
    if kind == "fp16":
        k, v = k.half(), v.half()
    else:
        k, v = (x.clamp(-4, 4).mul(30).to(ref.DTYPES[kind]) for x in (k, v))
        ks, vs = (torch.full((pages, H, page), 1 / 30, device="cuda") for _ in range(2))
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(S, -1).contiguous()  # all of one text
    ctx = torch.full((S,), L, dtype=torch.int32, device="cuda")
    start = (torch.arange(S + 1, device="cuda") * nodes).to(torch.int32)
    T = S * nodes
    q = torch.randn((T, H * G, D), generator=gen, device="cuda").half()
    need = nm.nm_tree_attention_workspace_bytes(S, H * G, H, D, nodes)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros((T, H * G), device="cuda")
    P = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    c = _Cache(k=P(k), v=P(v), k_scale=P(ks), v_scale=P(vs), pages=pages, page_stride=H * page * D,
               scale_page_stride=H * page, kv_heads=H, page_size=page, head_dim=D, type=KINDS.index(kind))
    good = nm.nm_tree_attention(q, k, v, table, ctx, start, nodes, k_scale=ks, v_scale=vs, workspace=ws)
    for limit in (1, 500, 3000):
        stalled(nm, lambda: nm.lib().nm_tree_attention_stall_selftest(
            P(q), H * G * D, T, H * G, S, P(start), nodes, ctypes.byref(c), P(table), pages, pages, P(ctx), None,
            D ** -0.5, P(out), H * G * D, P(lse), P(ws), need, limit, torch.cuda.current_stream().cuda_stream), 6.0)
        nm.nm_wait_timeouts(reset=True)
        again = nm.nm_tree_attention(q, k, v, table, ctx, start, nodes, k_scale=ks, v_scale=vs, workspace=ws)
        assert torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])
        assert nm.nm_wait_timeouts() == 0


def test_no_bounded_wait_gave_up(nm):
    assert nm.nm_wait_timeouts() == 0
