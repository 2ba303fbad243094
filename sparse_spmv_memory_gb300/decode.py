"""The operators around the sparse products in a step of speculative decoding
(the C ABI in ``include/nm_decode.h``): rotary positions with the write of keys
and values into a paged cache, reading its rows back, attention of a tree of
drafted tokens over the cache, and the verification of those tokens.

As the rest of the binding this is marshalling only.  A cache is passed as its
tensors: ``k_cache`` and ``v_cache`` [pages][kv_heads][page_size][head_dim] of
float16, float8_e4m3fn or int8 (the dtype names what it holds; any page stride,
the inner three dimensions contiguous), and for the 8-bit types ``k_scale`` and
``v_scale`` float32 [pages][kv_heads][page_size].  A slot is
page * page_size + offset.
"""
from __future__ import annotations

import ctypes

import sparse_spmv_memory_gb300 as _nm

__all__ = ["nm_rope_inv_freq", "nm_rope_append", "nm_cache_read", "nm_tree_attention",
           "nm_tree_attention_workspace_bytes", "nm_tree_verify"]

ROPE_SCALINGS = {None: 0, "linear": 1, "banded": 2}


class _Cache(ctypes.Structure):
    """nm_cache."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("scale_page_stride", ctypes.c_int64),
                ("kv_heads", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("type", ctypes.c_int32)]


def declare(L) -> None:
    """Argument types of the entry points of nm_decode.h."""
    P, I64, I32, SZ, F32 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t,
                            ctypes.c_float)
    F64 = ctypes.c_double
    sig = {
        "nm_rope_inv_freq": ([P, I32, F64, I32, F64, F64, F64, F64], I32),
        "nm_rope_append": ([P, I64, I64, I32, P, P, P, I32, I32, F32, P, I64, P, P], I32),
        "nm_cache_read": ([P, P, I64, P, P, P], I32),
        "nm_tree_attention_workspace_bytes": ([I64, I32, I32, I32, I32], SZ),
        "nm_tree_attention": ([P, I64, I64, I32, I64, P, I32, P, P, I64, I64, P, P, F32, P, I64,
                               P, P, SZ, P], I32),
        "nm_tree_verify": ([P, I32, I64, I64, P, I64, P, P, P, I64, I64, I32, P, P, I64, F32, P,
                            P, P, P], I32),
    }
    for name, (args, res) in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res


def _contiguous_after(t, first: int) -> bool:
    """Whether the dimensions from ``first`` on are laid out densely."""
    want = 1
    for size, stride in zip(reversed(t.shape[first:]), reversed(t.stride()[first:])):
        if size != 1 and stride != want:
            return False
        want *= size
    return True


def _cache(k, v, k_scale, v_scale) -> _Cache:
    torch = _nm._torch()
    _nm._need_cuda(k, v, k_scale, v_scale)
    types = {torch.float16: 0, torch.float8_e4m3fn: 1, torch.int8: 2}
    if k.dtype not in types or v.dtype != k.dtype:
        raise ValueError("k_cache and v_cache must both be float16, float8_e4m3fn or int8")
    if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or \
            not _contiguous_after(k, 1):
        raise ValueError("k_cache and v_cache must be [pages][kv_heads][page_size][head_dim] of one "
                         "shape and stride, contiguous but for the page stride")
    scale_stride = 0
    if k.dtype != torch.float16:
        if k_scale is None or v_scale is None:
            raise ValueError("an 8-bit cache needs k_scale and v_scale")
        for s in (k_scale, v_scale):
            if s.dtype != torch.float32 or s.shape != k.shape[:3] or \
                    s.stride() != k_scale.stride() or not _contiguous_after(s, 1):
                raise ValueError("k_scale and v_scale must be float32 [pages][kv_heads][page_size] "
                                 "of one stride, contiguous but for the page stride")
        scale_stride = k_scale.stride(0) if k.shape[0] > 1 else k.shape[1] * k.shape[2]
    elif k_scale is not None or v_scale is not None:
        raise ValueError("a float16 cache takes no scales")
    pages, heads, page, dim = k.shape
    stride = k.stride(0) if pages > 1 else heads * page * dim
    return _Cache(k.data_ptr(), v.data_ptr(), _nm._ptr(k_scale), _nm._ptr(v_scale), pages, stride,
                  scale_stride, heads, page, dim, types[k.dtype])


def _vector(t, dtype, n, what):
    """A contiguous device vector of ``n`` elements of ``dtype`` (or None)."""
    if t is None:
        return None
    _nm._need_cuda(t)
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of {n} elements")
    return t.data_ptr()


def _heads(t, tokens, dim, what):
    """(pointer, token stride) of fp16 [tokens][heads][dim] with dense heads."""
    torch = _nm._torch()
    _nm._need_cuda(t)
    if t.dtype != torch.float16 or t.dim() != 3 or t.shape[0] != tokens or t.shape[2] != dim or \
            not _contiguous_after(t, 1):
        raise ValueError(f"{what} must be float16 [{tokens}][heads][{dim}], contiguous but for the "
                         "token stride")
    return t.data_ptr(), t.stride(0) if tokens > 1 else t.shape[1] * t.shape[2]


def nm_rope_inv_freq(rot_dim: int, base: float = 10000.0, scaling: str | None = None,
                     factor: float = 1.0, low: float = 1.0, high: float = 4.0,
                     orig_ctx: float = 8192.0, device=None):
    """Angles per position of the rot_dim / 2 rotated pairs (float32), on
    ``device`` (default: the current CUDA device): plain, or for longer contexts
    ``scaling`` "linear" (all divided by ``factor``) or "banded" (by wavelength:
    short ones kept, long ones divided, a linear mix between)."""
    torch = _nm._torch()
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {list(ROPE_SCALINGS)}")
    out = torch.empty(max(0, rot_dim // 2), dtype=torch.float32)
    _nm._check(_nm.lib().nm_rope_inv_freq(out.data_ptr(), rot_dim, base, ROPE_SCALINGS[scaling],
                                          factor, low, high, orig_ctx), "nm_rope_inv_freq")
    return out.to("cuda" if device is None else device)


def nm_rope_append(qkv, k_cache, v_cache, positions, slots, inv_freq, q_heads: int, k_scale=None,
                   v_scale=None, interleaved: bool = False, mscale: float = 1.0, q=None,
                   want_q: bool = True, stream=None):
    """Rotate the query and key heads of qkv fp16 [tokens][(q_heads + 2 kv_heads)
    * head_dim] and write keys and values to the cache rows ``slots`` (int64;
    out of range: not written).  ``positions`` int32; ``inv_freq`` float32, half
    as long as the rotated part of a head.  Returns the rotated queries fp16
    [tokens][q_heads][head_dim] (``q`` if given; None with want_q=False, which
    skips them: the form that commits accepted tokens to their final slots)."""
    torch = _nm._torch()
    c = _cache(k_cache, v_cache, k_scale, v_scale)
    _nm._need_cuda(qkv, inv_freq)
    if qkv.dtype != torch.float16 or qkv.dim() != 2 or qkv.stride(1) != 1 or \
            qkv.shape[1] != (q_heads + 2 * c.kv_heads) * c.head_dim:
        raise ValueError("qkv must be float16 [tokens][(q_heads + 2 kv_heads) * head_dim] with unit "
                         "column stride")
    tokens = qkv.shape[0]
    pos = _vector(positions, torch.int32, tokens, "positions")
    slot = _vector(slots, torch.int64, tokens, "slots")
    freq = _vector(inv_freq, torch.float32, inv_freq.numel(), "inv_freq")
    if q is None and want_q:
        q = torch.empty((tokens, q_heads, c.head_dim), dtype=torch.float16, device=qkv.device)
    qp, ldq = (None, 0) if q is None else _heads(q, tokens, c.head_dim, "q")
    if q is not None and q.shape[1] != q_heads:
        raise ValueError("q must have q_heads heads")
    _nm._check(_nm.lib().nm_rope_append(
        qkv.data_ptr(), qkv.stride(0) if tokens > 1 else qkv.shape[1], tokens, q_heads, pos, slot,
        freq, 2 * inv_freq.numel(), 1 if interleaved else 0, mscale, qp, ldq, ctypes.byref(c),
        _nm._stream(stream)), "nm_rope_append")
    return q


def nm_cache_read(k_cache, v_cache, slots, k_scale=None, v_scale=None, k=None, v=None,
                  stream=None):
    """Rows ``slots`` (int64; out of range: zeros) of the cache as fp16: (k, v),
    each [rows][kv_heads][head_dim]."""
    torch = _nm._torch()
    c = _cache(k_cache, v_cache, k_scale, v_scale)
    rows = slots.numel()
    slot = _vector(slots, torch.int64, rows, "slots")
    shape = (rows, c.kv_heads, c.head_dim)
    if k is None:
        k = torch.empty(shape, dtype=torch.float16, device=slots.device)
    if v is None:
        v = torch.empty(shape, dtype=torch.float16, device=slots.device)
    for t in (k, v):
        _nm._need_cuda(t)
        if t.dtype != torch.float16 or t.shape != shape or not t.is_contiguous():
            raise ValueError("k and v must be contiguous float16 [rows][kv_heads][head_dim]")
    _nm._check(_nm.lib().nm_cache_read(ctypes.byref(c), slot, rows, k.data_ptr(), v.data_ptr(),
                                       _nm._stream(stream)), "nm_cache_read")
    return k, v


def nm_tree_attention_workspace_bytes(seqs: int, q_heads: int, kv_heads: int, head_dim: int,
                                      max_nodes: int) -> int:
    return _nm.lib().nm_tree_attention_workspace_bytes(seqs, q_heads, kv_heads, head_dim, max_nodes)


def nm_tree_attention(q, k_cache, v_cache, block_table, ctx_len, q_start, max_nodes: int,
                      tree_mask=None, k_scale=None, v_scale=None, scale: float | None = None,
                      out=None, lse=None, workspace=None, stream=None):
    """Attention of drafted nodes over their sequences' cached contexts and
    trees: q fp16 [tokens][q_heads][head_dim]; sequence s has the tokens
    q_start[s] .. q_start[s+1] - 1 (int32 [seqs + 1], at most ``max_nodes`` <= 64
    each), ctx_len[s] (int32) cached positions in the pages block_table[s] (int32
    [seqs][entries]), and its node j at position ctx_len[s] + j.  ``tree_mask``
    int64 [tokens]: bit j, the token sees node j (None: nodes up to itself).
    ``scale`` defaults to head_dim ** -0.5.  Returns (out fp16 like q, lse
    float32 [tokens][q_heads]); a node that sees nothing gets zeros and
    -infinity.  The workspace must be zero-filled before its first use (every
    call leaves it ready); a zeroed one of
    nm_tree_attention_workspace_bytes(...) bytes is allocated when none is
    given."""
    torch = _nm._torch()
    c = _cache(k_cache, v_cache, k_scale, v_scale)
    tokens, q_heads, dim = q.shape
    qp, ldq = _heads(q, tokens, c.head_dim, "q")
    seqs = ctx_len.numel()
    ctx = _vector(ctx_len, torch.int32, seqs, "ctx_len")
    start = _vector(q_start, torch.int32, seqs + 1, "q_start")
    mask = _vector(tree_mask, torch.int64, tokens, "tree_mask")
    _nm._need_cuda(block_table, workspace)
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or \
            block_table.shape[0] != seqs or block_table.stride(1) != 1 and block_table.shape[1] != 1:
        raise ValueError("block_table must be int32 [seqs][entries] with unit column stride")
    if out is None:
        out = torch.empty((tokens, q_heads, dim), dtype=torch.float16, device=q.device)
    op, ldo = _heads(out, tokens, c.head_dim, "out")
    if out.shape[1] != q_heads:
        raise ValueError("out must have as many heads as q")
    if lse is None:
        lse = torch.empty((tokens, q_heads), dtype=torch.float32, device=q.device)
    lp = _vector(lse, torch.float32, tokens * q_heads, "lse")
    L = _nm.lib()
    if workspace is None:
        need = L.nm_tree_attention_workspace_bytes(seqs, q_heads, c.kv_heads, dim, max_nodes)
        if need:
            workspace = torch.zeros(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    cols = block_table.shape[1]
    _nm._check(L.nm_tree_attention(
        qp, ldq, tokens, q_heads, seqs, start, max_nodes, ctypes.byref(c), block_table.data_ptr(),
        block_table.stride(0) if seqs > 1 else cols, cols, ctx, mask,
        dim ** -0.5 if scale is None else scale, op, ldo, lp, _nm._ptr(workspace), ws_bytes,
        _nm._stream(stream)), "nm_tree_attention")
    return out, lse


def nm_tree_verify(logits, tokens, parents, node_start, max_nodes: int, draft=None, accept=None,
                   race=None, temperature: float = 1.0, path=None, count=None, token=None,
                   stream=None):
    """Accept or reject drafted tokens against the target's probabilities:
    logits fp16 or fp32 [nodes][vocab] (row i: after node i), ``tokens`` and
    ``parents`` int32 [nodes], node_start int32 [seqs + 1] (at most ``max_nodes``
    <= 64 nodes a sequence, node 0 its last committed token).  ``draft`` float32
    [nodes][vocab]: row n, the distribution that node n's children were drawn
    from (None: proposals without probabilities).  ``accept`` float32 [nodes]
    uniform in [0, 1) and ``race`` float32 [seqs][vocab] exponentially distributed
    are the random numbers; temperature 0 takes the largest logit and neither.
    Returns (path int32 [seqs][max_nodes], the accepted nodes and then -1;
    count int32 [seqs]; token int32 [seqs], the next one)."""
    torch = _nm._torch()
    _nm._need_cuda(logits, draft, race)
    if logits.dtype not in (torch.float16, torch.float32) or logits.dim() != 2 or \
            logits.stride(1) != 1 and logits.shape[1] != 1:
        raise ValueError("logits must be float16 or float32 [nodes][vocab] with unit column stride")
    n, vocab = logits.shape
    seqs = node_start.numel() - 1
    ids = _vector(tokens, torch.int32, n, "tokens")
    par = _vector(parents, torch.int32, n, "parents")
    start = _vector(node_start, torch.int32, seqs + 1, "node_start")
    acc = _vector(accept, torch.float32, n, "accept")
    for t, rows, what in ((draft, n, "draft"), (race, seqs, "race")):
        if t is not None and (t.dtype != torch.float32 or t.shape != (rows, vocab) or
                              t.stride(1) != 1 and vocab != 1):
            raise ValueError(f"{what} must be float32 [{rows}][{vocab}] with unit column stride")
    if path is None:
        path = torch.empty((seqs, max_nodes), dtype=torch.int32, device=logits.device)
    if count is None:
        count = torch.empty(seqs, dtype=torch.int32, device=logits.device)
    if token is None:
        token = torch.empty(seqs, dtype=torch.int32, device=logits.device)

    def ld(t):
        return 0 if t is None else t.stride(0) if t.shape[0] > 1 else vocab

    _nm._check(_nm.lib().nm_tree_verify(
        logits.data_ptr(), 1 if logits.dtype == torch.float32 else 0, ld(logits), vocab,
        _nm._ptr(draft), ld(draft), ids, par, start, n, seqs, max_nodes, acc, _nm._ptr(race),
        ld(race), temperature, _vector(path, torch.int32, seqs * max_nodes, "path"),
        _vector(count, torch.int32, seqs, "count"), _vector(token, torch.int32, seqs, "token"),
        _nm._stream(stream)), "nm_tree_verify")
    return path, count, token
