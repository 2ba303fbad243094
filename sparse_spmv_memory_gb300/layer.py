"""The operators between the sparse products of a decoder layer and at its answer (the
C ABI in ``include/nm_layer.h``): the product with bias, activation and residual in
its epilogue, the residual stream's update with the norms around it, and log
probabilities of tokens.

As decode.py this is marshalling only, compiled (csrc/binding.cpp).  All tensors of a
call are on one device, current or not.  ``stream`` is a torch.cuda.Stream or a raw
cudaStream_t (None: that device's current one); outputs and workspaces that a call
makes itself are allocated on that stream.  Several outputs of a call that have less
than 16 MiB together share one allocation (it lives as long as any of them; resizing or
saving one concerns all).  The operators are for inference: they have no gradients.
"""
from __future__ import annotations

import ctypes

import sparse_spmv_memory_gb300 as _nm

from . import decode as _decode

__all__ = ["nm_linear", "nm_linear_workspace_bytes", "nm_residual_norm", "nm_token_logprobs"]

ACTIVATIONS = {None: 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
NORMS = {None: 0, "rms": 1, "layer": 2}


class _Epilogue(ctypes.Structure):
    """nm_epilogue."""
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("ldres", ctypes.c_int64),
                ("activation", ctypes.c_int32), ("gated", ctypes.c_int32), ("scale", ctypes.c_float)]


class _Norm(ctypes.Structure):
    """nm_norm."""
    _fields_ = [("kind", ctypes.c_int32), ("params_fp32", ctypes.c_int32),
                ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("offset", ctypes.c_float), ("eps", ctypes.c_float)]


def declare(L) -> None:
    """Argument types of the entry points of nm_layer.h."""
    P, I64, I32, SZ, F32 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t,
                            ctypes.c_float)
    sig = {
        "nm_linear_workspace_bytes": ([I64, I64, I64], SZ),
        "nm_linear": ([P, P, I64, I64, P, I64, I64, P, P, I64, P, SZ, P], I32),
        "nm_residual_norm": ([P, I32, I64, P, I64, P, P, I64, F32, F32, P, I64, P, P, I64, I64,
                              I64, P], I32),
        "nm_token_logprobs": ([P, I32, I64, I64, I64, P, I64, I32, F32, P, P, I32, P, P, P], I32),
    }
    args, res = sig["nm_linear"]  # the same and a limit, before the stream
    sig["nm_linear_stall_selftest"] = (args[:-1] + [I64, P], res)
    for name, (args, res) in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res


def _named(kinds, name, what):
    try:
        return kinds[name]
    except (KeyError, TypeError):
        raise ValueError(f"{what} must be one of {list(kinds)}") from None


def nm_linear_workspace_bytes(rows: int, cols: int, tokens: int) -> int:
    """Bytes of workspace of nm_linear on the current device (0: none)."""
    return _nm.lib().nm_linear_workspace_bytes(rows, cols, tokens)


def nm_linear(values, masks, X, bias=None, activation: str | None = None, gated: bool = False,
              scale: float = 1.0, residual=None, Y=None, workspace=None, stream=None,
              cols: int | None = None):
    """Y = residual + scale * act(W X + bias) for any number of tokens: X fp16
    [tokens][ldx] (first ``cols`` columns used), bias fp16 [rows], Y fp16
    [tokens][rows].  ``activation``: None, "relu", "silu", "gelu" or "gelu_tanh".
    ``gated``: rows are interleaved (gate, up) pairs as for nm_spmv_swiglu, and
    Y = residual + scale * act(gate) * up, fp16 [tokens][rows / 2].  ``residual`` is
    fp16 like Y and may be Y itself.  A workspace of nm_linear_workspace_bytes(...)
    bytes is allocated when needed and none is given."""
    return _decode._calls().linear(values, masks, X, bias, _named(ACTIVATIONS, activation, "activation"),
                                   gated, scale, residual, Y, workspace, _decode._given(stream), cols)


def nm_residual_norm(residual, block=None, norm: str | None = "rms", weight=None, bias=None,
                     post_norm: str | None = None, post_weight=None, post_bias=None, gate=None,
                     scale: float = 1.0, residual_scale: float = 1.0, weight_offset: float = 0.0,
                     eps: float = 1e-6, residual_out=None, out=None, stream=None):
    """Between two blocks of a layer: s = residual_scale * residual + scale * gate *
    post_norm(block), and norm(s): returns (norm(s) fp16, s like residual).
    ``residual`` fp16 or fp32 [tokens][width], ``block`` fp16 like it (None: s is the
    scaled residual, returned as it is where residual_scale is 1); ``gate`` fp16
    [width] or [tokens][width].  Norms are None, "rms" or "layer", times
    weight_offset + weight (1 without a weight) plus bias, all fp16 or all fp32
    [width] and given with their norm only; without ``norm`` the first result is
    None.  ``residual_out`` may be ``residual`` itself."""
    return _decode._calls().residual_norm(
        residual, block, _named(NORMS, norm, "norm"), weight, bias, _named(NORMS, post_norm, "post_norm"),
        post_weight, post_bias, gate, scale, residual_scale, weight_offset, eps, residual_out, out,
        _decode._given(stream))


def nm_token_logprobs(logits, tokens=None, top: int = 0, temperature: float = 1.0, logprob=None,
                      entropy=None, top_ids=None, top_logprob=None, stream=None):
    """From rows of logits fp16 or fp32 [rows][vocab] at a temperature: (log
    probabilities float32 of ``tokens`` int32 [rows] or [rows][n], shaped alike; the
    entropy float32 [rows]; the ``top`` <= 32 likeliest tokens int32 [rows][top], the
    lowest id first among equals; their log probabilities float32).  A token outside
    the vocabulary has -infinity; a row without a finite largest logit, or with NaN,
    has NaN and tokens -1."""
    return _decode._calls().token_logprobs(logits, tokens, top, temperature, logprob, entropy, top_ids,
                                           top_logprob, _decode._given(stream))
