"""64-bit references of the operators of nm_layer.h, with error bounds.

Every function returns (value, tolerance) in float64.  E is the rounding of a
float32 operation, 2^-24 relative; H that of a float16 result, 2^-11 relative (and
half of the smallest step, 2^-25).
"""
import math

import torch

E, H, TINY = 2.0 ** -24, 2.0 ** -11, 2.0 ** -25


def half(y, err):
    """A float16 result of a value y computed with error err."""
    return y, err + H * (y.abs() + err) + TINY


def unpacked(values, masks):
    """Dense float64 from the packed arrays."""
    rows, words = masks.shape
    kept = (masks[:, :, None].long() >> torch.arange(32, device=masks.device)) & 1
    rank = kept.cumsum(-1) - kept
    v = values.double().view(rows, words, 16)
    return (torch.gather(v, 2, rank.clamp_max(15)) * kept).flatten(1)


def activation(x, act):
    if act is None:
        return x
    if act == "relu":
        return x.clamp_min(0)
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu":
        return x * torch.special.ndtr(x)
    return x * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))


def linear(W, x, bias, act, gated, scale, residual):
    """W dense float64.  A sum of K products: each addition may be off by one step of the
    running value (tensor cores truncate: 2 E), so 2 E K sum |w x|.  Activations have a
    slope of at most 1.13 and are off by 16 E of their size (an exponential's argument
    carries its rounding, times at most |x| where the result matters: 2 E |x| of it)."""
    x = x.double()
    s, size = x @ W.T, x.abs() @ W.abs().T
    err = 2 * E * (W != 0).sum(1).max() * size
    if bias is not None:
        s, err = s + bias.double(), err + E * (size + bias.double().abs())

    def acted(s, err):
        y = activation(s, act)
        return y, err if act is None else 1.13 * err + (16 + 4 * s.abs()) * E * y.abs()

    if gated:
        y, ey = acted(s[:, 0::2], err[:, 0::2])
        u, eu = s[:, 1::2], err[:, 1::2]
        y, err = y * u, ey * u.abs() + y.abs() * eu + ey * eu + E * (y * u).abs()
    else:
        y, err = acted(s, err)
    y, err = scale * y, abs(scale) * err + E * (scale * y).abs()
    if residual is not None:
        y = y + residual.double()
        err = err + E * y.abs()
    return half(y, err)


def _norm(x, err, kind, weight, bias, offset, eps):
    """The sums have at most 32 terms a thread, then 10 levels: 48 E relative."""
    if kind is None:
        return x, err
    n = x.shape[1]
    if kind == "layer":
        mean = x.mean(1, keepdim=True)
        err = err + err.mean(1, keepdim=True) + 48 * E * x.abs().mean(1, keepdim=True) + E * (x - mean).abs()
        x = x - mean
    r = torch.rsqrt(x.square().mean(1, keepdim=True) + eps)
    # the root mean square moves by at most that of err
    rel = 32 * E + r * (err.square().sum(1, keepdim=True) / n).sqrt()
    w = torch.ones(n, dtype=torch.float64, device=x.device) if weight is None else offset + weight.double()
    y = x * r * w
    err = (err * r * w.abs()) * (1 + rel) + (rel + 4 * E) * y.abs()
    if bias is not None:
        y = y + bias.double()
        err = err + E * y.abs()
    return y, err


def residual_norm(residual, block, norm, weight, bias, post_norm, post_weight, post_bias, gate, scale,
                  residual_scale, weight_offset, eps):
    """((out, tolerance) or None, (stream, tolerance))"""
    s = residual_scale * residual.double()
    err = E * s.abs()
    if block is not None:
        b = block.double()
        b, eb = _norm(b, torch.zeros_like(b), post_norm, post_weight, post_bias, weight_offset, eps)
        g = 1.0 if gate is None else gate.double()
        b, eb = scale * g * b, abs(scale) * (eb * (g if gate is None else g.abs())) + 2 * E * (scale * g * b).abs()
        s = s + b
        err = err + eb + E * s.abs()
    out = None
    if norm is not None:
        out = half(*_norm(s, err, norm, weight, bias, weight_offset, eps))
    stream = half(s, err) if residual.dtype == torch.float16 else (s, err + 2 * E * s.abs())
    return out, stream


def logprobs(logits, ids, top, temperature):
    """(logprob, entropy, top_ids, top_logprob), each (value, tolerance) but top_ids.
    R = sum without the largest: each term's exponent is off by 4 E |t| (log2 e / T, the
    product, a reference up to 64 away: 64 E more) and 2^x by 2^-22; the sum has
    V / 512 + 32 terms a thread and 16 levels.  A term 2^t below 2^-126, float32's
    smallest normal number, may count as 0, as may its product with |t| ln 2 (below
    88 x 2^-126, since 2^t |t| falls with |t|): V of them."""
    x = logits.double()
    V = x.shape[1]
    none = V * 2.0 ** -126
    m = x.amax(1, keepdim=True)
    ok = torch.isfinite(m) & ~torch.isnan(x).any(1, keepdim=True)
    t = (x - m) / temperature
    order = x.nan_to_num(nan=0.0).sort(dim=1, descending=True, stable=True).indices
    e = t.exp()
    e.scatter_(1, order[:, :1], 0.0)
    R = e.sum(1, keepdim=True)
    A = torch.where(e > 0, -e * t, 0.0).sum(1, keepdim=True)
    far = torch.where(R > 0, A / R, 0.0)
    rel = (V / 512 + 32 + 16 + 64 + 8) * E + 6 * E * far
    log_z = torch.log1p(R)
    err_z = rel * R / (1 + R) + 4 * E * log_z + none
    h = log_z + A / (1 + R)
    # A's terms carry |t| more: the mean of t^2 over that of |t|
    t2 = torch.where(e > 0, e * t * t, 0.0).sum(1, keepdim=True)
    err_h = err_z + (2 * rel * A + 6 * E * t2) / (1 + R) + 4 * E * h + 88 * none
    nan = float("nan")

    def lp(at, inside=None):
        y = torch.gather(t, 1, at)
        v = y - log_z
        if inside is not None:
            v = torch.where(inside, v, -math.inf)
        return torch.where(ok, v, nan), 4 * E * y.abs() + err_z + 2 * E * v.abs()

    ids = ids.long()
    inside = (ids >= 0) & (ids < V)
    first = lp(torch.where(inside, ids, 0), inside)
    best = order[:, :top]
    return (first, (torch.where(ok, h, nan).squeeze(1), err_h.squeeze(1)),
            torch.where(ok, best, -1).to(torch.int32), lp(best))
