"""The operators around the sparse products of a decoder layer and at its answer,
in plain form and through the library.

  linear    the product with an N:M matrix, with bias, activation (gated too),
            scale and residual in its epilogue, for one token to a prefill;
  norm      the residual stream's update by a block's output (normed after the
            block, gated, scaled) and the norm before the next block;
  logprobs  log probabilities of given tokens, the entropy and the likeliest
            tokens, from rows of logits.

``run`` takes one pass: elementary torch operations in fp32 where ``own`` is
false, the library's calls where it is true.  ``exact`` gives the definition in
64 bits.  The plain form of a product has the pruned matrix itself in hand, as a
program without packed weights keeps it.  Matrix sizes are those of the 8B and
70B decoder layers of the benchmark, or odd.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"fp16": torch.float16, "fp32": torch.float32}


# ---- the cases ---------------------------------------------------------------
def _linear(name, tokens, rows, cols, pattern, act=None, gated=False, bias=False, residual=False,
            scale=1.0):
    return dict(name=name, op="linear", tokens=tokens, rows=rows, cols=cols, pattern=pattern, act=act,
                gated=gated, bias=bias, residual=residual, scale=scale)


def _norm(name, tokens, width, norm="rms", post=None, gate=None, stream="fp16", scale=1.0,
          residual_scale=1.0, bias=False):
    return dict(name=name, op="norm", tokens=tokens, width=width, norm=norm, post=post, gate=gate,
                stream=stream, scale=scale, residual_scale=residual_scale, bias=bias)


def _logprobs(name, rows, vocab, logits, ids, top, temperature, forbidden=False):
    return dict(name=name, op="logprobs", rows=rows, vocab=vocab, logits=logits, ids=ids, top=top,
                temperature=temperature, forbidden=forbidden)


def listed():
    return [
        # One token's attention output, added to the stream: latency counts.
        _linear("linear 1, 4096x4096 +res", 1, 4096, 4096, 4, residual=True),
        # One token through the 70B layer's gate and up projections.
        _linear("linear 1, 57344x8192 gated", 1, 57344, 8192, 8, act="silu", gated=True),
        # A tree of 8 drafted tokens, a QKV projection with a bias.
        _linear("linear 8, 10240x8192 +bias", 8, 10240, 8192, 32, bias=True),
        # A serving batch through a feed-forward block with biases; odd sizes.
        _linear("linear 100, 4999x2080 gelu", 100, 4999, 2080, 16, act="gelu", bias=True,
                residual=True, scale=0.5),
        # Many sequences' drafted trees through the 70B layer's down projection.
        _linear("linear 300, 8192x28672 +res", 300, 8192, 28672, 4, residual=True),
        # A prompt through the 8B layer's gate and up projections.
        _linear("linear 2048, 28672x4096 gated", 2048, 28672, 4096, 4, act="silu", gated=True),
        # One token between two blocks: latency.
        _norm("norm 1x4096", 1, 4096),
        # A prompt between two blocks of a model with norms before and after each.
        _norm("norm 4096x8192 post, gate", 4096, 8192, post="rms", gate="channel", scale=0.5),
        # A padded batch with a gate for each token, an odd width, an fp32 stream.
        _norm("norm 777x5121 layer fp32", 777, 5121, norm="layer", post="layer", gate="token",
              stream="fp32", residual_scale=0.75, bias=True),
        # One answered token with its alternatives: latency.
        _logprobs("logprobs 1x128256 top 20", 1, 128256, "fp16", 1, 20, 1.0),
        # A prompt's tokens scored, rows without padding of an odd vocabulary.
        _logprobs("logprobs 64x50257 fp32", 64, 50257, "fp32", 4, 0, 0.7, forbidden=True),
        # Many prompts scored at once, with a few alternatives each.
        _logprobs("logprobs 2048x128256 top 5", 2048, 128256, "fp16", 1, 5, 1.0, forbidden=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "norm", "logprobs"])
    if op == "linear":
        cols = 32 * _log_int(rng, 1, 896)
        rows = _log_int(rng, 1, min(57344, 57344 * 8192 // cols))
        tokens = _log_int(rng, 1, max(1, min(2048, 2048 * 28672 * 4096 // (rows * cols))))
        gated = rng.random() < 0.4
        rows += gated and rows % 2
        act = rng.choice(["silu", "gelu", "gelu_tanh", "relu"])
        case = _linear("", tokens, rows, cols, rng.choice([4, 8, 16, 32]),
                       act if gated or rng.random() < 0.5 else None, gated, rng.random() < 0.5,
                       rng.random() < 0.5, rng.choice([1.0, 1.0, 0.25]))
    elif op == "norm":
        width = _log_int(rng, 32, 16384)
        case = _norm("", _log_int(rng, 1, min(16384, 4096 * 8192 // width)), width,
                     rng.choice(["rms", "rms", "layer", None]), rng.choice([None, "rms", "layer"]),
                     rng.choice([None, "channel", "token"]), rng.choice(["fp16", "fp32"]),
                     rng.choice([1.0, 0.22]), rng.choice([1.0, 0.75]), rng.random() < 0.3)
    else:
        vocab = _log_int(rng, 500, 151936)
        case = _logprobs("", _log_int(rng, 1, min(4096, 2048 * 128256 // vocab // 2)), vocab,
                         rng.choice(["fp16", "fp32"]), rng.randint(0, 5), rng.choice([0, 1, 5, 20, 32]),
                         rng.choice([0.6, 1.0, 1.0, 1.3]), rng.random() < 0.5)
    del case["name"]
    return case


def work(case):
    if case["op"] == "linear":
        t, r, c = case["tokens"], case["rows"], case["cols"]
        n = r // 2 if case["gated"] else r
        # packed weights, x, bias, residual in; y out; the kept half of the products
        return {"bytes": r * c * 9 // 8 + 2 * (t * c + case["bias"] * r + t * n * (1 + case["residual"])),
                "flops": t * r * c}
    if case["op"] == "norm":
        t, w = case["tokens"], case["width"]
        stream = 2 if case["stream"] == "fp16" else 4
        gate = {None: 0, "channel": 2 * w, "token": 2 * t * w}[case["gate"]]
        out = 2 if case["norm"] else 0
        return {"bytes": t * w * (2 + 2 * stream + out) + gate, "flops": t * w * 12}
    r, v = case["rows"], case["vocab"]
    return {"bytes": r * (v * (2 if case["logits"] == "fp16" else 4) + 8 * case["ids"] + 4 + 8 * case["top"]),
            "flops": r * v * 6}


# ---- inputs --------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _words(pattern, seed):
    """A few thousand mask words that keep half of every group of ``pattern`` columns."""
    g = torch.Generator().manual_seed(seed)
    keys = torch.rand((4096, 32 // pattern, pattern), generator=g)
    kept = keys.argsort(-1).argsort(-1) < pattern // 2
    return (kept.view(4096, 32).long() << torch.arange(32)).sum(-1).to(torch.int32).to(DEV)


def _bits(masks):
    return ((masks[..., None] >> torch.arange(32, dtype=torch.int32, device=DEV)) & 1).flatten(1).bool()


def _prepare_linear(case, seed):
    g = _gen(seed)
    t, r, c = case["tokens"], case["rows"], case["cols"]
    n = r // 2 if case["gated"] else r
    words = _words(case["pattern"], seed)
    masks = words[torch.randint(0, 4096, (r, c // 32), device=DEV, generator=g)]
    # weights of a layer that keeps its input's size
    values = torch.randn((r, c // 2), dtype=torch.float16, device=DEV, generator=g) * (1.4 * c ** -0.5)
    dense = torch.zeros((r, c), dtype=torch.float16, device=DEV)
    step = max(1, (1 << 28) // c)
    for i in range(0, r, step):  # bounded temporaries
        dense[i:i + step].masked_scatter_(_bits(masks[i:i + step]), values[i:i + step])
    x = torch.randn((t, c), dtype=torch.float16, device=DEV, generator=g)
    x[:, :2] *= 20  # a few channels of activations are far larger than the rest
    rnd = lambda *s: torch.randn(s, dtype=torch.float16, device=DEV, generator=g)  # noqa: E731
    return dict(op="linear", values=values, masks=masks, dense=dense, x=x,
                bias=rnd(r) if case["bias"] else None, residual=rnd(t, n) * 4 if case["residual"] else None,
                act=case["act"], gated=case["gated"], scale=case["scale"])


def _prepare_norm(case, seed):
    g = _gen(seed)
    t, w = case["tokens"], case["width"]
    rnd = lambda *s: torch.randn(s, device=DEV, generator=g)  # noqa: E731
    stream, block = rnd(t, w) * 3, rnd(t, w)
    stream[:, 5 % w] *= 100  # the stream's large channels
    block[t // 2] = 0        # a padding token
    weight = lambda: (1 + 0.2 * rnd(w)).half()  # noqa: E731
    shift = lambda kind: (0.1 * rnd(w)).half() if case["bias"] and kind == "layer" else None  # noqa: E731
    gate = {None: lambda: None, "channel": lambda: rnd(w).half(), "token": lambda: rnd(t, w).half()}
    return dict(op="norm", residual=stream.to(DTYPES[case["stream"]]), block=block.half(),
                gate=gate[case["gate"]](), norm=case["norm"], post=case["post"],
                weight=weight() if case["norm"] else None, bias=shift(case["norm"]),
                post_weight=weight() if case["post"] else None, post_bias=shift(case["post"]),
                scale=case["scale"], residual_scale=case["residual_scale"], eps=1e-5)


def _prepare_logprobs(case, seed):
    g = _gen(seed)
    r, v = case["rows"], case["vocab"]
    logits = torch.randn((r, v), dtype=DTYPES[case["logits"]], device=DEV, generator=g) * 2.5
    # a few likely tokens in most rows
    at = torch.randint(0, v, (r, 8), device=DEV, generator=g)
    logits.scatter_(1, at, (torch.rand((r, 8), device=DEV, generator=g) * 22).to(logits.dtype))
    ids = torch.randint(0, v, (r, case["ids"]), device=DEV, generator=g)
    if case["ids"]:
        ids[:, 0] = at[:, 0]
        ids[r // 2, -1] = -1  # a padding token
    if case["forbidden"]:
        logits[:, 7::97] = float("-inf")  # tokens that the grammar forbids
        logits[::3, 5::11] = torch.finfo(logits.dtype).min
        if r > 4:
            logits[r // 3] = float("-inf")  # no token at all
    if case["ids"]:  # one masked by the type's lowest value would be the output's only size
        lowest = torch.gather(logits, 1, ids.clamp_min(0)) == torch.finfo(logits.dtype).min
        ids = torch.where(lowest, logits.argmax(-1, keepdim=True), ids)
    return dict(op="logprobs", logits=logits, ids=ids.to(torch.int32), top=case["top"],
                temperature=case["temperature"])


def prepare(case, seed):
    return {"linear": _prepare_linear, "norm": _prepare_norm,
            "logprobs": _prepare_logprobs}[case["op"]](case, seed)


# ---- the plain forms -------------------------------------------------------------
def _activate(y, act):
    if act == "silu":
        return y / (1 + torch.exp(-y))
    if act == "relu":
        return torch.where(y > 0, y, 0.0)
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    return y


def _plain_linear(st):
    y = torch.matmul(st["x"].float(), st["dense"].float().T)
    if st["bias"] is not None:
        y = y + st["bias"].float()
    if st["gated"]:
        y = _activate(y[:, 0::2], st["act"]) * y[:, 1::2]
    else:
        y = _activate(y, st["act"])
    y = y * st["scale"]
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.half()


def _normed(x, kind, weight, bias, eps):
    if kind is None:
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.float()
    return y if bias is None else y + bias.float()


def _plain_norm(st):
    b = _normed(st["block"].float(), st["post"], st["post_weight"], st["post_bias"], st["eps"])
    if st["gate"] is not None:
        b = b * st["gate"].float()
    s = st["residual"].float() * st["residual_scale"] + b * st["scale"]
    if st["norm"] is None:
        return s.to(st["residual"].dtype)
    return _normed(s, st["norm"], st["weight"], st["bias"], st["eps"]).half(), s.to(st["residual"].dtype)


def _ordered(x, at):
    """int64 keys that order (x, -index): ties go to the lowest index."""
    b = (x.float() + 0.0).view(torch.int32)
    b = torch.where(b < 0, b ^ 0x7FFFFFFF, b).long()
    return (b << 32) | (0x7FFFFFFF - at)


def _plain_logprobs(st):
    x = st["logits"].float()
    V = x.shape[1]
    m = x.amax(-1, keepdim=True)
    valid = torch.isfinite(m)
    t = (x - m) / st["temperature"]
    e = torch.exp(t)
    z = e.sum(-1, keepdim=True)
    log_z = torch.log(z)
    entropy = log_z - torch.where(e > 0, e * t, 0.0).sum(-1, keepdim=True) / z
    ids = st["ids"].long()
    inside = (ids >= 0) & (ids < V)
    lp = torch.where(inside, torch.gather(t, 1, ids.clamp(0, V - 1)) - log_z, float("-inf"))
    lp = torch.where(valid, lp, float("nan"))
    entropy = torch.where(valid, entropy, float("nan")).squeeze(-1)
    if not st["top"]:
        return lp, entropy
    key = torch.topk(_ordered(st["logits"], torch.arange(V, device=DEV)), st["top"], -1).values
    at = 0x7FFFFFFF - (key & 0x7FFFFFFF)
    top = torch.where(valid, torch.gather(t, 1, at) - log_z, float("nan"))
    return lp, entropy, torch.where(valid, at, -1).to(torch.int32), top


def _own_linear(st):
    import sparse_spmv_memory_gb300 as nm
    return nm.nm_linear(st["values"], st["masks"], st["x"], bias=st["bias"], activation=st["act"],
                        gated=st["gated"], scale=st["scale"], residual=st["residual"])


def _own_norm(st):
    import sparse_spmv_memory_gb300 as nm
    out, s = nm.nm_residual_norm(
        st["residual"], st["block"], norm=st["norm"], weight=st["weight"], bias=st["bias"],
        post_norm=st["post"], post_weight=st["post_weight"], post_bias=st["post_bias"], gate=st["gate"],
        scale=st["scale"], residual_scale=st["residual_scale"], eps=st["eps"])
    return s if st["norm"] is None else (out, s)


def _own_logprobs(st):
    import sparse_spmv_memory_gb300 as nm
    lp, entropy, at, top = nm.nm_token_logprobs(st["logits"], st["ids"], top=st["top"],
                                                temperature=st["temperature"])
    return (lp, entropy, at, top) if st["top"] else (lp, entropy)


def run(state):
    if own:
        return {"linear": _own_linear, "norm": _own_norm, "logprobs": _own_logprobs}[state["op"]](state)
    return {"linear": _plain_linear, "norm": _plain_norm, "logprobs": _plain_logprobs}[state["op"]](state)


# ---- the definitions in 64 bits ----------------------------------------------------
def _exact_linear(st):
    masks, values, x = st["masks"], st["values"].double(), st["x"].double()
    rows, words = masks.shape
    sums = torch.empty((x.shape[0], rows), dtype=torch.float64, device=DEV)
    step = max(1, (1 << 22) // words)
    col = torch.arange(32, device=DEV)
    for i in range(0, rows, step):
        kept = (masks[i:i + step, :, None].long() >> col) & 1
        rank = kept.cumsum(-1) - kept  # of a column among its word's kept ones
        v = values[i:i + step].view(-1, words, 16)
        w = torch.gather(v, 2, rank.clamp_max(15)) * kept
        sums[:, i:i + step] = torch.einsum("tk,rk->tr", x, w.flatten(1))
    if st["bias"] is not None:
        sums += st["bias"].double()
    F = torch.nn.functional
    fn = {None: lambda y: y, "silu": F.silu, "relu": F.relu, "gelu": F.gelu,
          "gelu_tanh": lambda y: F.gelu(y, approximate="tanh")}[st["act"]]
    if st["gated"]:
        pair = sums.view(x.shape[0], rows // 2, 2)
        y = fn(pair[..., 0]) * pair[..., 1]
    else:
        y = fn(sums)
    y = st["scale"] * y
    return y if st["residual"] is None else y.add_(st["residual"].double())


def _exact_norm(st):
    def unit(x, kind, w, b):
        if kind == "rms":
            return x * torch.rsqrt(x.square().mean(1, keepdim=True) + st["eps"]) * w.double()
        if kind == "layer":
            return torch.nn.functional.layer_norm(x, x.shape[1:], w.double(),
                                                  None if b is None else b.double(), st["eps"])
        return x
    y = unit(st["block"].double(), st["post"], st["post_weight"], st["post_bias"]) * st["scale"]
    if st["gate"] is not None:
        y *= st["gate"].double()
    s = torch.add(y, st["residual"].double(), alpha=st["residual_scale"])
    return s if st["norm"] is None else (unit(s, st["norm"], st["weight"], st["bias"]), s)


def _exact_logprobs(st):
    rows, vocab = st["logits"].shape
    lp, entropy, at, top = [], [], [], []
    step = max(1, (1 << 25) // vocab)
    for i in range(0, rows, step):
        x = st["logits"][i:i + step].double()
        ids = st["ids"][i:i + step].long()
        p = torch.log_softmax(x / st["temperature"], -1)
        ok = torch.isfinite(x.amax(-1))
        there = (ids >= 0) & (ids < vocab)
        q = torch.where(there, p.gather(1, torch.where(there, ids, 0)), -math.inf)
        lp.append(torch.where(ok[:, None], q, math.nan))
        entropy.append(torch.where(ok, -(p.exp() * p.clamp_min(-1e300)).sum(-1), math.nan))
        if st["top"]:
            order = x.sort(dim=-1, descending=True, stable=True).indices[:, :st["top"]]
            at.append(torch.where(ok[:, None], order, -1).to(torch.int32))
            top.append(torch.where(ok[:, None], p.gather(1, order), math.nan))
    out = [torch.cat(lp), torch.cat(entropy)]
    return tuple(out + [torch.cat(at), torch.cat(top)] if st["top"] else out)


def exact(case, seed):
    return {"linear": _exact_linear, "norm": _exact_norm,
            "logprobs": _exact_logprobs}[case["op"]](prepare(case, seed))
