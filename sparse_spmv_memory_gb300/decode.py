"""The operators around the sparse products in a step of speculative decoding
(the C ABI in ``include/nm_decode.h``): rotary positions with the write of keys
and values into a paged cache, reading its rows back, attention of a tree of
drafted tokens over the cache, and the verification of those tokens.

As the rest of the binding this is marshalling only, compiled (csrc/binding.cpp)
because these calls take a few microseconds each.  A cache is passed as its
tensors: ``k_cache`` and ``v_cache`` [pages][kv_heads][page_size][head_dim] of
float16, float8_e4m3fn or int8 (the dtype names what it holds; any page stride,
the inner three dimensions contiguous), and for the 8-bit types ``k_scale`` and
``v_scale`` float32 [pages][kv_heads][page_size].  A slot is
page * page_size + offset.

All tensors of a call are on one device, current or not.  ``stream`` is a
torch.cuda.Stream or a raw cudaStream_t (None: that device's current one); outputs
and workspaces that a call makes itself are allocated on that stream.
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
    for name in ("nm_tree_attention", "nm_tree_verify"):  # the same and a limit, before the stream
        args, res = sig[name]
        sig[name + "_stall_selftest"] = (args[:-1] + [I64, P], res)
    for name, (args, res) in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res


_ext = None


def _calls():
    """The compiled half of this module (csrc/binding.cpp)."""
    global _ext
    if _ext is None:
        _nm._torch()  # its libraries are the binding's
        _nm.lib()  # the library first: its absence is the clearer message
        from . import _decode_ext
        _ext = _decode_ext
    return _ext


def _given(stream):
    return None if stream is None else _nm._stream(stream)


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
    return _calls().rope_append(qkv, k_cache, v_cache, positions, slots, inv_freq, q_heads, k_scale,
                                v_scale, interleaved, mscale, q, want_q, _given(stream))


def nm_cache_read(k_cache, v_cache, slots, k_scale=None, v_scale=None, k=None, v=None,
                  stream=None):
    """Rows ``slots`` (int64; out of range: zeros) of the cache as fp16: (k, v),
    each [rows][kv_heads][head_dim]."""
    return _calls().cache_read(k_cache, v_cache, slots, k_scale, v_scale, k, v, _given(stream))


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
    return _calls().tree_attention(q, k_cache, v_cache, block_table, ctx_len, q_start, max_nodes,
                                   tree_mask, k_scale, v_scale, scale, out, lse, workspace,
                                   _given(stream))


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
    return _calls().tree_verify(logits, tokens, parents, node_start, max_nodes, draft, accept, race,
                                temperature, path, count, token, _given(stream))
