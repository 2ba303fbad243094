"""GPU parity of the operators around the sparse products (nm_linear,
nm_residual_norm, nm_token_logprobs) against 64-bit references."""
from __future__ import annotations

import ctypes

import pytest

import layer_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

NAN, INF = float("nan"), float("inf")
PATTERNS = [(2, 4), (4, 8), (8, 16), (16, 32)]


@pytest.fixture(scope="module")
def nm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_spmv_memory_gb300 import _build
    _build.build()
    import sparse_spmv_memory_gb300 as m
    m.lib()
    return m


def generator(seed):
    return torch.Generator("cuda").manual_seed(seed)


def within(got, want, what):
    want, tol = want
    got = got.double()
    assert got.shape == want.shape, f"{what}: {tuple(got.shape)} for {tuple(want.shape)}"
    odd = ~torch.isfinite(want)
    assert torch.equal(got[odd].nan_to_num(nan=7.0), want[odd].nan_to_num(nan=7.0)), f"{what}: infinities or NaN differ"
    err = (got - want).abs()
    bad = ~(err <= tol) & ~odd
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} beyond tolerance, worst ratio "
                           f"{float((err / tol)[bad].max()):.3g}, first {bad.nonzero()[0].tolist()}")


def strided(shape, pad, gen, dtype=torch.float16, spoil=NAN, scale=1.0):
    """A matrix whose rows lie ``pad`` elements further apart, with ``spoil`` between."""
    big = torch.full((shape[0], shape[1] + pad), spoil, dtype=dtype, device="cuda")
    big[:, :shape[1]] = (torch.randn(shape, device="cuda", generator=gen) * scale).to(dtype)
    return big, big[:, :shape[1]]


# ---- nm_linear --------------------------------------------------------------------
class Product:
    def __init__(self, nm, rows, cols, tokens, pattern=(2, 4), act=None, gated=False, bias=False,
                 residual=False, scale=1.0, seed=0, pad=0, x_scale=1.0):
        g = generator(seed)
        W = (torch.randn((rows, cols), device="cuda", generator=g) * 1.4 * cols ** -0.5).half()
        self.values, self.masks = nm.nm_pack(W, *pattern)
        self.x = strided((tokens, cols), pad, g, scale=x_scale)[1]
        self.n = rows // 2 if gated else rows
        rnd = lambda *s: torch.randn(s, device="cuda", generator=g).half()  # noqa: E731
        self.kw = dict(bias=rnd(rows) if bias else None, activation=act, gated=gated, scale=scale,
                       residual=strided((tokens, self.n), pad, g)[1] if residual else None)

    def want(self):
        k = self.kw
        return ref.linear(ref.unpacked(self.values, self.masks), self.x, k["bias"], k["activation"],
                          k["gated"], k["scale"], k["residual"])

    def run(self, nm, **kw):
        return nm.nm_linear(self.values, self.masks, self.x, **{**self.kw, **kw})


ACTS = [None, "relu", "silu", "gelu", "gelu_tanh"]
TOKENS = [1, 2, 3, 5, 6, 8, 9, 16, 37, 65, 130, 300, 520]
SHAPES = [(1, 32), (2, 64), (7, 1024), (300, 1056), (130, 2048), (1000, 4096)]


@pytest.mark.parametrize("tokens", TOKENS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear(nm, shape, tokens):
    rows, cols = shape
    i = TOKENS.index(tokens) + 7 * SHAPES.index(shape)
    for k, gated in enumerate((False, True)):
        if gated and rows % 2:
            continue
        p = Product(nm, rows, cols, tokens, PATTERNS[i % 4], ACTS[(i + k) % 5], gated, bias=i % 3 != 0,
                    residual=i % 2 == 0, scale=(1.0, -0.3)[i // 2 % 2], seed=i, pad=(0, 8)[i % 2])
        within(p.run(nm), p.want(), f"{shape} {tokens} gated={gated}")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("tokens", [1, 4, 20])
def test_linear_activations_over_their_range(nm, act, gated, tokens):
    p = Product(nm, 96, 256, tokens, (4, 8), act, gated, True, True, 0.5, seed=3, x_scale=9.0)
    within(p.run(nm), p.want(), f"{act}")


@pytest.mark.parametrize("tokens,rows,cols", [(1, 20, 53248), (1, 40, 65536), (2, 33, 60000 // 32 * 32),
                                              (8, 40, 28672), (5, 26, 28672 + 32), (7, 3, 13312),
                                              (16, 64, 28672), (300, 256, 16384), (12, 126, 14336 + 64)])
@pytest.mark.parametrize("gated", [False, True])
def test_linear_long_rows(nm, tokens, rows, cols, gated):
    """Rows whose tile leaves no room, column slices, and K splits of the prefill plan."""
    if gated and rows % 2:
        rows += 1
    p = Product(nm, rows, cols, tokens, (8, 16), "silu", gated, True, True, seed=rows)
    within(p.run(nm), p.want(), f"{tokens} {rows} {cols}")


def test_linear_every_kind_of_plan_is_met(nm):
    need = nm.nm_linear_workspace_bytes
    assert need(20, 53248, 1) > 0 and need(4096, 4096, 1) == 0 and need(40, 28672, 8) > 0
    assert need(300, 1056, 8) == 0 and need(64, 28672, 16) == 0 and need(57344, 8192, 2048) == 0
    assert need(0, 64, 4) == need(4, 64, 0) == need(4, 33, 4) == need(-1, 64, 4) == 0


def test_linear_many_rows_beside_a_large_tile(nm):
    """More rows than a block's remaining shared memory holds sums for."""
    rows, cols, tokens = 90112, 12288, 8
    g = generator(1)
    words = torch.tensor([0x0F0F0F0F, 0x33333333, 0x55555555, 0x3C3C3C3C], dtype=torch.int32, device="cuda")
    masks = words[torch.randint(0, 4, (rows, cols // 32), device="cuda", generator=g)]
    values = torch.randn((rows, cols // 2), dtype=torch.float16, device="cuda", generator=g) * 0.02
    x = torch.randn((tokens, cols), dtype=torch.float16, device="cuda", generator=g)
    bias = torch.randn((rows,), dtype=torch.float16, device="cuda", generator=g)
    pick = torch.cat([torch.arange(0, rows, 2 * 347), torch.arange(rows - 40, rows, 2)]).cuda()
    pairs = torch.stack([pick, pick + 1], 1).flatten()
    W = ref.unpacked(values[pairs], masks[pairs])
    assert nm.nm_linear_workspace_bytes(rows, cols, tokens) == 0
    y = nm.nm_linear(values, masks, x, bias=bias)
    within(y[:, pairs], ref.linear(W, x, bias[pairs], None, False, 1.0, None), "plain")
    y = nm.nm_linear(values, masks, x, bias=bias, gated=True, activation="silu")
    within(y[:, pick // 2], ref.linear(W, x, bias[pairs], "silu", True, 1.0, None), "gated")


@pytest.mark.parametrize("tokens", [16, 100, 200, 330, 512])
@pytest.mark.parametrize("late", [0, 1, 2, 3, 30])
def test_linear_words_of_several_patterns(nm, tokens, late):
    """Mask words that keep 4 columns of every byte, but for one row's from a word on:
    16 columns at the word's start, its end, spread, or whole bytes."""
    rows, cols = 200, 64 * 32
    g = generator(late)
    even = torch.tensor([0x33333333, 0x55555555, 0x0F0F0F0F, 0x3C5A6996], dtype=torch.int32, device="cuda")
    odd = torch.tensor([0x0000FFFF, -0x10000, 0x00FF00FF, 0x7F80FF00], dtype=torch.int32, device="cuda")
    masks = even[torch.randint(0, len(even), (rows, 64), device="cuda", generator=g)]
    bits = torch.arange(32, dtype=torch.int32, device="cuda")
    row = 37 * (late + 1) % rows
    masks[row, late:] = odd[torch.randint(0, len(odd), (64 - late,), device="cuda", generator=g)]
    assert bool((((masks[..., None] >> bits) & 1).sum(-1) == 16).all())
    values = torch.randn((rows, cols // 2), dtype=torch.float16, device="cuda", generator=g) * 0.02
    x = torch.randn((tokens, cols), dtype=torch.float16, device="cuda", generator=g)
    within(nm.nm_linear(values, masks, x), ref.linear(ref.unpacked(values, masks), x, None, None, False, 1.0, None),
           "mixed")


@pytest.mark.parametrize("tokens", [1, 8, 20, 200, 300])
@pytest.mark.parametrize("pattern", [(2, 4), (8, 16)], ids=str)
def test_linear_masks_and_rows_off_16_bytes(nm, tokens, pattern):
    """Mask words from any multiple of 4 bytes on, outputs from any multiple of 2."""
    p = Product(nm, 200, 1024, tokens, pattern, "gelu_tanh", bias=True, residual=True, seed=tokens)
    want = p.want()
    moved = torch.zeros(p.masks.numel() + 1, dtype=torch.int32, device="cuda")[1:].view_as(p.masks)
    p.masks = moved.copy_(p.masks)
    big = torch.full((tokens, 203), 7.0, device="cuda").half()
    y = p.run(nm, Y=big[:, 1:201])
    within(y, want, "moved")
    assert bool((big[:, 0] == 7).all()) and bool((big[:, 201:] == 7).all())


@pytest.mark.parametrize("tokens", [1, 3, 8, 9, 100])
@pytest.mark.parametrize("gated", [False, True])
def test_linear_in_place_and_rows_between(nm, tokens, gated):
    """The residual stream is updated where it lies; what lies between its rows stays."""
    p = Product(nm, 202, 1088, tokens, act="gelu", gated=gated, bias=True, seed=5, pad=16)
    big, view = strided((tokens + 2, p.n), 5, generator(9), spoil=123.0)
    before = big.clone()
    stream = view[1:tokens + 1]
    p.kw["residual"] = stream.clone()
    want = p.want()
    out = p.run(nm, residual=stream, Y=stream)
    assert out.data_ptr() == stream.data_ptr()
    within(stream, want, "in place")
    big[1:tokens + 1, :p.n] = before[1:tokens + 1, :p.n]
    assert torch.equal(big, before)


def test_linear_agrees_with_the_products_it_extends(nm):
    """Up to 8 tokens, where the plans are the same, the bits without an epilogue are those
    of nm_spmv and nm_spmm, and gated SiLU of one token has those of nm_spmv_swiglu."""
    for rows, cols in [(300, 1056), (1000, 4096)]:
        for tokens in (1, 2, 4, 6, 8):
            p = Product(nm, rows, cols, tokens, seed=tokens)
            y = p.run(nm)
            if tokens == 1:
                want = nm.nm_spmv(p.values, p.masks, p.x[0])[None]
            else:
                want = nm.nm_spmm(p.values, p.masks, p.x)
            assert torch.equal(y, want), (rows, cols, tokens)
        p = Product(nm, rows, cols, 1, act="silu", gated=True, seed=3)
        assert torch.equal(p.run(nm)[0], nm.nm_spmv_swiglu(p.values, p.masks, p.x[0]))


def test_linear_nonfinite(nm):
    """Up to 8 tokens a non-finite activation reaches the rows that keep its column;
    beyond, every row of its token; other tokens nothing."""
    for tokens in (1, 2, 8, 20):
        p = Product(nm, 64, 256, tokens, seed=tokens)
        clean = p.run(nm)
        p.x[tokens - 1, 37] = INF
        y = p.run(nm)
        keeps = ((p.masks[:, 1] >> 5) & 1).bool()
        assert torch.equal(y[:-1], clean[:-1])
        if tokens <= 8:
            assert torch.equal(y[-1, ~keeps], clean[-1, ~keeps]) and not torch.isfinite(y[-1, keeps]).any()
        else:
            assert not torch.isfinite(y[-1]).any()


def test_linear_empty(nm):
    v, m = nm.nm_pack(torch.randn((8, 64), device="cuda").half(), 2, 4)
    assert nm.nm_linear(v, m, torch.empty((0, 64), dtype=torch.float16, device="cuda")).shape == (0, 8)
    y = nm.nm_linear(v[:0], m[:0], torch.zeros((3, 64), dtype=torch.float16, device="cuda"))
    assert y.shape == (3, 0)


def refuses(call, status=None):
    import sparse_spmv_memory_gb300 as m
    with pytest.raises((m.NMError, ValueError, TypeError)) as e:
        call()
    if status is not None:
        assert isinstance(e.value, m.NMError) and e.value.status == status, e.value


def test_linear_refusals(nm):
    p = Product(nm, 64, 128, 4, bias=True, residual=True)
    y = torch.empty((4, 64), dtype=torch.float16, device="cuda")
    refuses(lambda: p.run(nm, activation="tanh"))
    refuses(lambda: p.run(nm, scale=INF), 2)
    refuses(lambda: p.run(nm, bias=p.kw["bias"][:63]))
    refuses(lambda: p.run(nm, bias=p.kw["bias"].float()))
    refuses(lambda: p.run(nm, residual=p.kw["residual"][:3]))
    refuses(lambda: p.run(nm, Y=y[:, :63]))
    refuses(lambda: p.run(nm, Y=y.float()))
    refuses(lambda: p.run(nm, cols=96))
    refuses(lambda: p.run(nm, gated=True))  # the residual is as wide as all rows
    refuses(lambda: nm.nm_linear(p.values, p.masks[:, :3], p.x))
    refuses(lambda: nm.nm_linear(p.values.float(), p.masks, p.x))
    refuses(lambda: nm.nm_linear(p.values, p.masks, p.x.cpu()))
    refuses(lambda: nm.nm_linear(p.values[:63], p.masks[:63], p.x, gated=True))
    refuses(lambda: nm.nm_linear(p.values, p.masks, p.x, Y=p.x[:, :64]), 7)
    two = torch.zeros((8, 64), dtype=torch.float16, device="cuda")
    refuses(lambda: nm.nm_linear(p.values, p.masks, p.x, residual=two[:4], Y=two[1:5]), 7)
    wide = torch.zeros((4, 128), dtype=torch.float16, device="cuda")
    refuses(lambda: nm.nm_linear(p.values, p.masks, p.x, residual=wide[:, :64], Y=wide.view(8, 64)[:4]), 7)
    off = torch.zeros(4 * 128 + 8, dtype=torch.float16, device="cuda")[1:513].view(4, 128)
    refuses(lambda: nm.nm_linear(p.values, p.masks, off), 4)
    q = Product(nm, 40, 28672, 8)
    small = torch.empty(nm.nm_linear_workspace_bytes(40, 28672, 8) - 16, dtype=torch.uint8, device="cuda")
    refuses(lambda: q.run(nm, workspace=small), 5)
    assert torch.equal(p.run(nm), p.run(nm, workspace=small))  # one that is not needed


# ---- nm_residual_norm ---------------------------------------------------------------
class Norm:
    def __init__(self, tokens, width, norm="rms", post=None, gate=None, stream=torch.float16, block=True,
                 params=torch.float16, bias=False, weight=True, scale=1.0, residual_scale=1.0, offset=0.0,
                 eps=1e-6, pad=0, seed=0):
        g = generator(seed)
        self.residual = strided((tokens, width), pad, g, stream, scale=3.0)[1]
        self.block = strided((tokens, width), pad, g)[1] if block else None
        vec = lambda: (torch.randn(width, device="cuda", generator=g) * 0.3 + 1).to(params)  # noqa: E731
        gates = {None: lambda: None, "channel": lambda: vec().half(),
                 "token": lambda: strided((tokens, width), pad, g)[1]}
        self.kw = dict(norm=norm, weight=vec() if norm and weight else None, bias=vec() if norm and bias else None,
                       post_norm=post, post_weight=vec() if post and weight else None,
                       post_bias=vec() if post and bias else None, gate=gates[gate](), scale=scale,
                       residual_scale=residual_scale, weight_offset=offset, eps=eps)

    def run(self, nm, **kw):
        return nm.nm_residual_norm(self.residual, self.block, **{**self.kw, **kw})

    def want(self):
        return ref.residual_norm(self.residual, self.block, **self.kw)

    def check(self, nm, what, **kw):
        out, stream = self.run(nm, **kw)
        want_out, want_stream = self.want()
        within(stream, want_stream, what + " stream")
        if want_out is None:
            assert out is None
        else:
            within(out, want_out, what + " out")


WIDTHS = [1, 7, 8, 32, 64, 100, 129, 256, 264, 514, 770, 1000, 1024, 1538, 2047, 2050, 4096, 5121, 6146, 8191, 8192, 8193,
          8200, 12290, 12288, 16384, 16386, 16392, 32761, 32768]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("stream", [torch.float16, torch.float32], ids=["fp16", "fp32"])
def test_norm_widths(nm, width, stream):
    i = WIDTHS.index(width)
    for k, tokens in enumerate((1, 5, 67)):
        Norm(tokens, width, ("rms", "layer")[(i + k) % 2], (None, "rms", "layer")[(i + k) % 3],
             (None, "channel", "token")[(i + k) // 2 % 3], stream, seed=i, bias=k == 1,
             params=(torch.float16, torch.float32)[i % 2], pad=(0, 8, 3)[k]).check(nm, f"{tokens}x{width}")


@pytest.mark.parametrize("norm", [None, "rms", "layer"])
@pytest.mark.parametrize("post", [None, "rms", "layer"])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
def test_norm_forms(nm, norm, post, gate):
    for stream in (torch.float16, torch.float32):
        for width, weight in ((512, True), (99, False)):
            Norm(9, width, norm, post, gate, stream, weight=weight, bias=True, scale=-0.4, residual_scale=0.8,
                 offset=1.0, eps=1e-3, seed=width).check(nm, f"{norm} {post} {gate} {stream} {width}")


@pytest.mark.parametrize("tokens", [1, 2, 3, 8, 9, 1000, 4099])
@pytest.mark.parametrize("width", [64, 96, 512, 2048])
def test_norm_rows_a_block(nm, tokens, width):
    Norm(tokens, width, "rms", "rms", "channel", seed=tokens).check(nm, f"{tokens}x{width}")


# rows of whole 16-byte pieces, more than fit the SMs at once, on which blocks stay: one and two
# groups a thread, one to eight rows a block, two to four stages
MANY = [(5000, 256), (2600, 512), (1700, 768), (1300, 1024), (700, 1792), (170, 7936), (200, 8192)]


@pytest.mark.parametrize("tokens,width", MANY)
@pytest.mark.parametrize("stream", [torch.float16, torch.float32], ids=["fp16", "fp32"])
def test_norm_many_rows(nm, tokens, width, stream):
    assert tokens * (width // 8) > 1024 * torch.cuda.get_device_properties(0).multi_processor_count
    k = 0
    for norm in (None, "rms", "layer"):
        for post in (None, "rms", "layer"):
            for gate in (None, "channel", "token"):
                k += 1
                Norm(tokens, width, norm, post, gate, stream, params=(torch.float16, torch.float32)[k % 2],
                     bias=k % 3 == 0, weight=k % 4 != 1, scale=(1.0, -0.4)[k // 2 % 2],
                     residual_scale=(0.8, 1.0)[k // 3 % 2], offset=(0.0, 1.0)[k // 2 % 2], eps=(1e-6, 1e-3)[k % 2],
                     pad=(0, 8, 24)[k % 3], seed=k).check(nm, f"{norm} {post} {gate} {k}")
    for norm in ("rms", "layer"):
        Norm(tokens, width, norm, stream=stream, block=False, bias=True, residual_scale=0.5,
             seed=1).check(nm, f"{norm} alone, scaled")
        n = Norm(tokens, width, norm, stream=stream, block=False, bias=norm == "layer", seed=2)
        n.check(nm, f"{norm} alone")
        assert n.run(nm)[1] is n.residual


@pytest.mark.parametrize("tokens,width", MANY[1::2])
@pytest.mark.parametrize("stream", [torch.float16, torch.float32], ids=["fp16", "fp32"])
def test_norm_many_rows_in_place_and_spoilt(nm, tokens, width, stream):
    n = Norm(tokens, width, "layer", "rms", "token", stream, bias=True, seed=2)
    big, view = strided((tokens + 2, width), 16, generator(4), stream, spoil=55.0)
    before = big.clone()
    n.residual = view[1:tokens + 1].clone()
    want_out, want = n.want()
    n.residual = view[1:tokens + 1]
    out, _ = n.run(nm, residual_out=n.residual)
    within(n.residual, want, "in place")
    within(out, want_out, "out")
    clean, clean_s = out.clone(), n.residual.clone()
    big[1:tokens + 1, :width] = before[1:tokens + 1, :width]
    assert torch.equal(big, before)
    # a row alone is spoilt by what it holds, and rows of nothing have their biases
    n.residual[tokens // 2, 9] = NAN
    n.block[tokens - 1, width - 1] = INF
    n.block[3] = 0
    out, s = n.run(nm)
    assert torch.isnan(out[tokens // 2]).all() and torch.isnan(out[tokens - 1]).all()
    rest = torch.ones(tokens, dtype=torch.bool, device="cuda")
    rest[[3, tokens // 2, tokens - 1]] = False
    assert torch.equal(out[rest], clean[rest]) and torch.equal(s[rest], clean_s[rest])
    w = n.want()
    within(out[3:4], (w[0][0][3:4], w[0][1][3:4]), "a row of nothing")


def test_norm_without_block(nm):
    for stream in (torch.float16, torch.float32):
        n = Norm(7, 1024, stream=stream, block=False)
        n.check(nm, "norm alone")
        assert n.run(nm)[1] is n.residual
        n.check(nm, "norm alone, copied", residual_out=torch.empty_like(n.residual))
        Norm(7, 1024, None, stream=stream, block=False, residual_scale=0.5).check(nm, "scaled")


def test_norm_in_place_and_rows_between(nm):
    n = Norm(6, 777, "layer", "rms", "token", torch.float32, seed=2)
    big, view = strided((8, 777), 5, generator(4), torch.float32, spoil=55.0)
    before = big.clone()
    n.residual = view[1:7].clone()
    want_out, want = n.want()
    n.residual = view[1:7]
    out, s = n.run(nm, residual_out=n.residual)
    within(n.residual, want, "in place")
    within(out, want_out, "out")
    big[1:7, :777] = before[1:7, :777]
    assert torch.equal(big, before)


def test_norm_rows_of_nothing_and_spoilt_rows(nm):
    n = Norm(8, 640, "rms", "layer", "token", seed=6)
    clean, clean_s = n.run(nm)
    n.block[2] = 0
    n.residual[2] = 0
    n.block[3] = 5.0  # no deviation: the layer norm of it is its bias
    n.residual[5, 9] = NAN
    n.block[6, 0] = INF
    out, s = n.run(nm)
    assert torch.equal(out[2], torch.zeros_like(out[2])) and torch.equal(s[2], torch.zeros_like(s[2]))
    assert torch.equal(s[3], n.residual[3])
    assert torch.isnan(out[5]).all() and torch.isnan(s[6]).all()
    for r in (0, 1, 4, 7):
        assert torch.equal(out[r], clean[r]) and torch.equal(s[r], clean_s[r])


# (tokens, width): a row a block, blocks that stay with one and two groups a thread, two and
# four groups a thread, element by element one and two at a time, shifted groups
NORM_KERNELS = [(3, 1792), (900, 1792), (1200, 1536), (2, 12288), (2, 24576), (5, 777), (4, 5121), (6, 1002),
                (3, 13000), (2, 30001), (2, 32767)]


@pytest.mark.parametrize("tokens,width", NORM_KERNELS)
@pytest.mark.parametrize("stream", [torch.float16, torch.float32], ids=["fp16", "fp32"])
def test_layer_norm_of_equal_elements_is_its_bias(nm, tokens, width, stream):
    """A row without deviation, at values where a mean that is one rounding off would count
    against eps.  The mean of x is off by 48 E |x| at most (see layer_ref), the mean of what
    is left of x by 50 E of that, and 1 / sqrt(var + eps) is at most eps^-1/2."""
    values = torch.tensor([1000.0, 30016.0, -60000.0, 1001.0, 0.1, 0.0, -3.3], dtype=torch.float16, device="cuda")
    if stream == torch.float32:
        values = values.float() * 1.2345678
    x = values[torch.arange(tokens, device="cuda") % 7]
    for post in (False, True):
        n = Norm(tokens, width, None if post else "layer", "layer" if post else None, None, stream, block=post,
                 bias=True, seed=width)
        n.residual.copy_(x[:, None].expand(tokens, width) * (0 if post else 1))
        if post:
            x = x.clamp(-65504, 65504).half()
            n.block.copy_(x[:, None].expand(tokens, width))
        out, s = n.run(nm)
        w, b = (n.kw["post_weight"], n.kw["post_bias"]) if post else (n.kw["weight"], n.kw["bias"])
        want = b.double().expand(tokens, width)
        err = 48 * 50 * ref.E ** 2 * x.double().abs()[:, None] * 1e3 * w.double().abs() + 2 * ref.E * want.abs()
        within(s if post else out, ref.half(want, err), f"post={post}")


@pytest.mark.parametrize("tokens,width", NORM_KERNELS)
def test_layer_norm_far_from_zero(nm, tokens, width):
    """Deviations of 1 about a mean of 30000: x - mean is exact, so that the norm is as
    exact as about 0 (the bound of the test above, and 64 E of the value)."""
    n = Norm(tokens, width, "layer", None, None, torch.float32, block=False, bias=True, seed=width)
    n.residual.copy_(torch.randn((tokens, width), device="cuda", generator=generator(3)) + 30000.0)
    out, _ = n.run(nm)
    x = n.residual.double()
    d = x - x.mean(1, keepdim=True)
    r = torch.rsqrt(d.square().mean(1, keepdim=True) + 1e-6)
    w = n.kw["weight"].double()
    want = d * r * w + n.kw["bias"].double()
    err = 48 * 50 * ref.E ** 2 * 31000 * r * w.abs() + 64 * ref.E * (want.abs() + (d * r * w).abs())
    within(out, ref.half(want, err), "far")


def test_norm_empty_and_alignment(nm):
    n = Norm(0, 64)
    out, s = n.run(nm)
    assert out.shape == s.shape == (0, 64)
    for off in (1, 4, 8):  # any alignment of the elements
        n = Norm(5, 256, "rms", "rms", "channel", seed=off)
        n.residual = torch.randn(5 * 256 + off, device="cuda").half()[off:].view(5, 256)
        n.kw["weight"] = torch.randn(256 + off, device="cuda").half()[off:]
        n.check(nm, f"offset {off}")


def test_norm_refuses_a_gate_without_dimensions(nm):
    n = Norm(4, 64)
    for gate in (torch.ones((), device="cuda").half(), torch.ones((4, 64, 1), device="cuda").half()):
        with pytest.raises(ValueError):
            n.run(nm, gate=gate)


def test_norm_refusals(nm):
    n = Norm(4, 64, "rms", "rms", "token")
    refuses(lambda: n.run(nm, norm="group"))
    refuses(lambda: n.run(nm, scale=NAN), 2)
    refuses(lambda: n.run(nm, eps=-1.0), 2)
    refuses(lambda: n.run(nm, weight=n.kw["weight"][:60]))
    refuses(lambda: n.run(nm, weight=n.kw["weight"].double()))
    refuses(lambda: n.run(nm, weight=n.kw["weight"].float(), bias=n.kw["weight"]))
    refuses(lambda: n.run(nm, gate=n.kw["gate"][:3]))
    refuses(lambda: n.run(nm, out=n.block), 7)
    refuses(lambda: n.run(nm, out=n.residual), 7)
    refuses(lambda: n.run(nm, residual_out=n.block), 7)
    refuses(lambda: n.run(nm, residual_out=n.residual.float()))
    refuses(lambda: n.run(nm, norm=None, weight=None, out=torch.empty_like(n.block)))
    refuses(lambda: nm.nm_residual_norm(n.residual, gate=n.kw["gate"]))
    refuses(lambda: n.run(nm, norm=None))  # (with a weight)
    refuses(lambda: n.run(nm, post_norm=None))
    refuses(lambda: nm.nm_residual_norm(n.residual.double()))
    refuses(lambda: nm.nm_residual_norm(n.residual, n.block.float()))
    refuses(lambda: nm.nm_residual_norm(torch.zeros((1, 32776), dtype=torch.float16, device="cuda")), 2)
    two = torch.zeros((9, 64), dtype=torch.float16, device="cuda")
    refuses(lambda: nm.nm_residual_norm(two[:8], n.block.repeat(2, 1), residual_out=two[1:]), 7)


# ---- nm_token_logprobs ----------------------------------------------------------------
def check_logprobs(nm, logits, ids=None, top=0, temperature=1.0, what=""):
    lp, h, at, top_lp = nm.nm_token_logprobs(logits, ids, top=top, temperature=temperature)
    none = torch.zeros((logits.shape[0], 0), dtype=torch.int32, device="cuda")
    want = ref.logprobs(logits, none if ids is None else ids if ids.dim() == 2 else ids[:, None], top, temperature)
    if ids is not None and ids.dim() == 1:
        want = ((want[0][0].squeeze(1), want[0][1].squeeze(1)),) + want[1:]
    assert torch.equal(at, want[2]), f"{what}: top ids"
    within(lp, want[0], what + " logprob")
    within(h, want[1], what + " entropy")
    within(top_lp, want[3], what + " top logprob")


VOCABS = [1, 2, 7, 8, 31, 33, 500, 4096, 4097, 8200, 50257, 128256, 151936]


@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32], ids=["fp16", "fp32"])
def test_logprobs(nm, vocab, dtype):
    for k, rows in enumerate((1, 3, 40, 170)):
        g = generator(vocab + k)
        top = min(vocab, (20, 32, 0, 1)[(VOCABS.index(vocab) + k) % 4])
        x = strided((rows, vocab), (0, 3, 8, 0)[k], g, dtype, spoil=(NAN, INF)[k % 2], scale=3.0)[1]
        ids = torch.randint(-1, vocab + 1, (rows, 1 + k), device="cuda", generator=g).to(torch.int32)
        check_logprobs(nm, x, ids, top, (1.0, 0.7, 1.3, 4.0)[k], f"{rows}x{vocab}")


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32], ids=["fp16", "fp32"])
@pytest.mark.parametrize("rows,vocab", [(1, 128256), (7, 50257), (200, 5000)])
def test_logprobs_ties_and_order(nm, dtype, rows, vocab):
    """Equal logits, ascending and descending rows (one thread or block holds all of the
    best), zeros of both signs: the lowest ids first."""
    g = generator(1)
    at = torch.arange(vocab, device="cuda")
    for what, x in [("equal", torch.zeros(vocab, device="cuda")),
                    ("ascending", at / vocab * 8), ("descending", -at / vocab * 8),
                    ("strided", (at % 512 == 77) * 9.0), ("strided up", (at // 8 % 512 == 3) * at / vocab),
                    ("few values", torch.randint(0, 4, (vocab,), device="cuda", generator=g) * 1.0),
                    ("signs", torch.where(at % 3 == 0, -0.0, 0.0)),
                    ("one", torch.where(at == vocab - 1, 30.0, 0.0))]:
        x = x.to(dtype)[None].repeat(rows, 1)
        ids = torch.randint(0, vocab, (rows,), device="cuda", generator=g).to(torch.int32)
        check_logprobs(nm, x, ids, 32, 1.0, what)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32], ids=["fp16", "fp32"])
@pytest.mark.parametrize("vocab", [40, 9000, 128256])
def test_logprobs_masks_and_spoilt_rows(nm, dtype, vocab):
    low = torch.finfo(dtype).min
    g = generator(vocab)
    x = (torch.randn((12, vocab), device="cuda", generator=g) * 2).to(dtype)
    x[0] = -INF                      # nothing allowed
    x[1] = -INF
    x[1, vocab // 2] = 1.0           # one token
    x[2] = low                       # all masked by the lowest value: all equal
    x[3, ::2] = low
    x[4, 1:] = -INF
    x[5, vocab - 1] = NAN
    x[6, 3] = INF
    x[7, 3:] = -INF                  # fewer than the alternatives
    x[8] = low
    x[8, 9] = -INF
    x[9, 0] = torch.finfo(dtype).max
    x[10] = x[10] - 60000.0 if dtype == torch.float16 else x[10] - 1e6
    ids = torch.full((12, 3), vocab // 2, dtype=torch.int32, device="cuda")
    ids[:, 1] = vocab
    ids[:, 2] = 9
    # where differences of the values reach float32's end only -infinity is left
    want_far = dtype == torch.float32
    lp, h, at, top_lp = nm.nm_token_logprobs(x, ids, top=8)
    w = ref.logprobs(x, ids, 8, 1.0)
    fix = lambda v: (torch.where(v[0] < -3.4028235e38, -INF, v[0]), v[1])  # noqa: E731
    assert torch.equal(at, w[2])
    assert at[0].tolist() == at[5].tolist() == at[6].tolist() == [-1] * 8
    assert at[7, :5].tolist()[3:] == [3, 4]
    within(lp, fix(w[0]) if want_far else w[0], "logprob")
    within(h, w[1], "entropy")
    within(top_lp, fix(w[3]) if want_far else w[3], "top logprob")
    assert float(h[1]) == 0.0 and float(lp[1, 0]) == 0.0


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32], ids=["fp16", "fp32"])
def test_logprobs_of_the_nearly_certain(nm, dtype):
    """1 - p far below float32's step at 1: log p and the entropy keep their digits."""
    for vocab in (1000, 128256):
        for gap in (5.0, 20.0, 30.0, 60.0, 90.0):
            g = generator(int(gap))
            x = torch.randn((3, vocab), device="cuda", generator=g).to(dtype)
            best = torch.tensor([0, vocab // 3, vocab - 1], device="cuda")
            x[torch.arange(3, device="cuda"), best] = gap
            check_logprobs(nm, x, best.to(torch.int32), 2, 1.0, f"{vocab} {gap}")


def test_logprobs_temperatures(nm):
    g = generator(3)
    x = torch.randn((5, 3000), device="cuda", generator=g) * 4
    ids = torch.zeros(5, dtype=torch.int32, device="cuda")
    for t in (2.0 ** -20, 1e-3, 0.1, 7.0, 2.0 ** 20):
        for y in (x, x.half()):
            check_logprobs(nm, y, ids, 3, t, f"temperature {t}")
    for t in (0.0, -1.0, NAN, INF, 1e-7, 2e6):
        refuses(lambda: nm.nm_token_logprobs(x, ids, temperature=t), 2)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32], ids=["fp16", "fp32"])
@pytest.mark.parametrize("rows,vocab", [(1, 128256), (7, 50257), (5, 3000), (200, 5000)])
@pytest.mark.parametrize("peak", [14.3, 21.6, 3002.0, 4001.0, 30016.0, 65504.0])
def test_logprobs_large_and_equal_logits_at_small_temperatures(nm, dtype, rows, vocab, peak):
    """x / T far beyond float32's exact whole numbers: equal largest logits, in different
    blocks of a row too, share the probability; rows of one value are even (of the type's
    lowest too), and one step of fp16 below the largest is as far as it is."""
    g = generator(vocab)
    x = (torch.randn((rows, vocab), device="cuda", generator=g) * 2).to(dtype)
    peak = torch.tensor(peak).half()
    below = float(peak) * (1 - 2.0 ** -10)
    x[:, [3, vocab - 2]] = peak.to(dtype).cuda()
    x[:, vocab // 2] = below
    x[::3, vocab // 3] = float(peak)
    if rows > 1:
        x[1] = -float(peak)
    if rows > 2:
        x[2] = torch.finfo(dtype).min
        x[2, 7] = -INF
    ids = torch.tensor([3, vocab - 2, vocab // 2, 5], dtype=torch.int32, device="cuda").repeat(rows, 1)
    for t in (2.0 ** -20, 1e-6, 1e-5, 1e-4, 1e-3, 0.01, 0.3):
        t = float(torch.tensor(t))  # (the call's float32)
        check_logprobs(nm, x, ids, 4, t, f"{peak} {t}")


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32], ids=["fp16", "fp32"])
@pytest.mark.parametrize("vocab", [16, 33, 90, 250, 257, 263, 270, 300, 511, 513, 1000, 1023, 1500, 1792, 1801, 2100])
def test_logprobs_short_rows_with_many_alternatives(nm, vocab, dtype):
    """Fewer warps than the alternatives need: the bound is then from all threads' largest."""
    g = generator(vocab)
    for off in (0, 3):
        x = torch.randn((5, vocab + 3), device="cuda", generator=g).to(dtype)
        x[1] = x[1].round()
        x[2, 10:] = -INF
        x[3, vocab // 2:] = 9.0
        x = x[:, off:off + vocab]
        for top in (1, 4, 5, 8, 12, 16, 20, 31, 32):
            if top <= vocab:
                check_logprobs(nm, x, x.argmin(1).to(torch.int32), top, 1.0, f"{vocab} {top} {off}")


def test_logprobs_many_ids_and_alignment(nm):
    g = generator(4)
    base = torch.randn(40 * 1001 + 16, device="cuda", generator=g)
    for dtype in (torch.float16, torch.float32):
        for off in (1, 2, 3, 5, 8):
            x = base.to(dtype)[off:off + 40 * 1001].view(40, 1001)
            ids = torch.randint(-5, 1010, (40, 1024), device="cuda", generator=g).to(torch.int32)
            check_logprobs(nm, x, ids, 5, 1.0, f"{dtype} {off}")
    check_logprobs(nm, base[:40 * 1001].view(40, 1001), ids[:, 3:900:1], 5, 1.0, "ids with a stride")
    col = ids[:, 7]
    check_logprobs(nm, base[:40 * 1001].view(40, 1001), col, 0, 1.0, "one column")


def test_logprobs_empty_and_refusals(nm):
    x = torch.randn((4, 100), device="cuda")
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    lp, h, at, tl = nm.nm_token_logprobs(x[:0], ids[:0], top=3)
    assert lp.shape == (0, 2) and h.shape == (0,) and at.shape == (0, 3) and tl.shape == (0, 3)
    lp, h, at, tl = nm.nm_token_logprobs(x)
    assert lp.shape == (4, 0) and at.shape == (4, 0) and h.shape == (4,)
    refuses(lambda: nm.nm_token_logprobs(x, top=33))
    refuses(lambda: nm.nm_token_logprobs(x, top=-1))
    refuses(lambda: nm.nm_token_logprobs(x[:, :5], top=6), 2)
    refuses(lambda: nm.nm_token_logprobs(x.double()))
    refuses(lambda: nm.nm_token_logprobs(x.bfloat16()))
    refuses(lambda: nm.nm_token_logprobs(x, ids.long()))
    refuses(lambda: nm.nm_token_logprobs(x, ids[:3]))
    refuses(lambda: nm.nm_token_logprobs(x.T))
    refuses(lambda: nm.nm_token_logprobs(x, ids, entropy=torch.empty(3, device="cuda")))
    refuses(lambda: nm.nm_token_logprobs(x, entropy=x[0, :4]), 7)
    refuses(lambda: nm.nm_token_logprobs(x, ids, logprob=x.view(-1)[:8].view(4, 2)), 7)
    e = torch.empty(8, device="cuda")
    refuses(lambda: nm.nm_token_logprobs(x, ids, logprob=e.view(4, 2), entropy=e[4:]), 7)
    refuses(lambda: nm.nm_token_logprobs(x, torch.zeros((4, 1025), dtype=torch.int32, device="cuda")), 2)


def test_large_outputs_have_allocations_of_their_own(nm):
    """Keeping one output of a call does not keep the others' memory, but for small ones."""
    own = lambda t: t.untyped_storage().nbytes() == t.nbytes  # noqa: E731
    for tokens, width, apart in ((64, 1024, False), (2048, 4096, True)):
        for stream in (torch.float16, torch.float32):
            n = Norm(tokens, width, stream=stream)
            out, s = n.run(nm)
            assert own(out) == own(s) == apart
            n.check(nm, f"{tokens} {stream}")
    x = torch.randn((4100, 1030), device="cuda")
    ids = torch.randint(0, 1030, (4100, 1024), device="cuda").to(torch.int32)
    for rows, apart in ((10, False), (4100, True)):
        parts = nm.nm_token_logprobs(x[:rows], ids[:rows], top=3)
        assert all(own(t) == apart for t in parts)
        check_logprobs(nm, x[:rows], ids[:rows], 3, 1.0, f"{rows}")


# ---- calls that the documentation allows ---------------------------------------------------
@pytest.mark.parametrize("tokens", [1, 2, 8, 9, 40, 300])
def test_linear_first_columns_of_wider_rows(nm, tokens):
    """``cols``: X is wider than the matrix; what lies behind is not used."""
    p = Product(nm, 70, 96, tokens, act="relu", bias=True, seed=tokens)
    x = torch.full((tokens, 160), NAN, device="cuda").half()
    x[:, :96] = p.x
    y = nm.nm_linear(p.values, p.masks, x, cols=96, **p.kw)
    within(y, p.want(), "wider")
    if tokens == 1:  # rows of any width, since there is no next one
        x = torch.full((1, 101), NAN, device="cuda").half()
        x[:, :96] = p.x
        within(nm.nm_linear(p.values, p.masks, x, cols=96, **p.kw), p.want(), "odd width")


def test_linear_outputs_beyond_32_bits(nm):
    """Outputs and residuals whose offsets pass 2^31 elements, 9 and more tokens and 8."""
    g = generator(1)
    for tokens, rows, ld in ((40000, 57344, 57344), (8, 64, 300000008), (20, 64, 120000008)):
        p = Product(nm, rows, 32, tokens, (4, 8), bias=True, seed=rows)
        y = torch.empty((tokens - 1) * ld + rows, dtype=torch.float16, device="cuda").as_strided((tokens, rows), (ld, 1))
        p.kw["residual"] = torch.randn((tokens, rows), device="cuda", generator=g).half()
        p.run(nm, Y=y)
        for a, b in ((0, 4), (tokens // 2, tokens // 2 + 3), (tokens - 5, tokens)):
            q = Product(nm, 1, 32, 1)
            q.values, q.masks, q.x = p.values, p.masks, p.x[a:b]
            q.kw = {**p.kw, "residual": p.kw["residual"][a:b]}
            within(y[a:b], q.want(), f"{tokens} {a}")
        del y


def test_norm_and_logprobs_beyond_32_bits(nm):
    for width in (8192, 8190, 30001):
        tokens = 2 ** 31 // width + 40
        for stream in (torch.float16, torch.float32):
            n = Norm(tokens, width, "layer", "rms", "token", stream)
            out, s = n.run(nm, residual_out=n.residual.clone())
            for a, b in ((0, 3), (tokens - 70, tokens)):
                m = Norm(1, 1)
                m.residual, m.block, m.kw = n.residual[a:b], n.block[a:b], {**n.kw, "gate": n.kw["gate"][a:b]}
                want_out, want_s = m.want()
                within(out[a:b], want_out, f"{width} {a} out")
                within(s[a:b], want_s, f"{width} {a} stream")
            del n, out, s
    rows, vocab = 2 ** 31 // 50257 + 30, 50257
    for dtype in (torch.float16, torch.float32):
        x = torch.randn((rows, vocab), dtype=dtype, device="cuda", generator=generator(5))
        ids = torch.arange(rows, device="cuda").to(torch.int32)[:, None] % vocab
        parts = nm.nm_token_logprobs(x, ids, top=6)
        for a, b in ((0, 3), (rows - 50, rows)):
            w = ref.logprobs(x[a:b], ids[a:b], 6, 1.0)
            assert torch.equal(parts[2][a:b], w[2])
            for got, want in ((parts[0], w[0]), (parts[1], w[1]), (parts[3], w[3])):
                within(got[a:b], want, f"{dtype} {a}")
        del x


def test_logprobs_many_ids_of_few_rows_and_the_longest(nm):
    """Ids beyond a block's threads where a row is split, the same id twice; 2^24 logits."""
    for rows, vocab in ((1, 128256), (3, 1 << 24)):
        for dtype in (torch.float16, torch.float32):
            x = torch.randn((rows, vocab), device="cuda", generator=generator(rows)).to(dtype)
            ids = torch.randint(-3, vocab + 3, (rows, 1024), device="cuda", generator=generator(7)).to(torch.int32)
            ids[:, 500:600] = ids[:, :100]
            check_logprobs(nm, x, ids, 32, 0.5, f"{rows}x{vocab}")


def test_calls_under_inference_mode_and_of_parameters(nm):
    """Outputs of calls in inference mode are usable after it, and gradients are not asked for."""
    n = Norm(5, 512)
    out, s = n.run(nm)
    x = torch.randn((3, 500), device="cuda")
    want = nm.nm_token_logprobs(x, top=2)
    with torch.inference_mode():
        out2, s2 = n.run(nm)
        got = nm.nm_token_logprobs(x, top=2)
        assert torch.equal(out2 + 0, out)
    assert torch.equal(out2, out) and torch.equal(s2, s) and same(got, want)
    n.kw["weight"] = torch.nn.Parameter(n.kw["weight"])
    out3, s3 = n.run(nm)
    assert not out3.requires_grad and torch.equal(out3, out)
    out3.mul_(2)  # an ordinary tensor, apart from the other output
    assert torch.equal(s3, s)


# ---- waits that give up -------------------------------------------------------------------
def stalled(nm, p, y, limit_us=20000, limit_s=4.0):
    """nm_linear's self-test: half of the blocks get no weights; it ends soon and is counted."""
    import time
    from sparse_spmv_memory_gb300.layer import _Epilogue, ACTIVATIONS
    k = p.kw
    at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    e = _Epilogue(bias=at(k["bias"]), residual=at(k["residual"]), ldres=p.n, activation=ACTIVATIONS[k["activation"]],
                  gated=k["gated"], scale=k["scale"])
    tokens, cols = p.x.shape
    torch.cuda.synchronize()
    nm.nm_wait_timeouts(reset=True)
    t0 = time.time()
    assert nm.lib().nm_linear_stall_selftest(at(p.values), at(p.masks), p.masks.shape[0], cols, at(p.x), p.x.stride(0),
                                             tokens, ctypes.byref(e), at(y), y.stride(0), None, 0, limit_us,
                                             torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert time.time() - t0 < limit_s
    assert nm.nm_wait_timeouts() > 0


# tokens, rows, cols: every size of tile; the masks by TMA and by cp.async; K split over clusters
STALLS = [(16, 128, 1024), (16, 300, 1056), (100, 1000, 4096), (200, 130, 2048), (300, 300, 1056), (520, 1000, 2080),
          (16, 64, 28672), (300, 256, 16384), (12, 126, 14336 + 64), (600, 256, 8192)]


@pytest.mark.parametrize("tokens,rows,cols", STALLS)
def test_linear_wait_that_gives_up(nm, tokens, rows, cols):
    p = Product(nm, rows, cols, tokens, (8, 16), "silu", True, True, True, seed=rows)
    good = p.run(nm)
    y = torch.empty_like(good)
    stalled(nm, p, y)
    # until the reset calls do nothing, all blocks of a cluster alike
    y.fill_(7.0)
    torch.cuda.synchronize()
    for _ in range(3):
        p.run(nm, Y=y)
    torch.cuda.synchronize()
    assert bool((y == 7).all())
    nm.nm_wait_timeouts(reset=True)
    assert torch.equal(p.run(nm, Y=y), good)
    assert nm.nm_wait_timeouts() == 0


@pytest.mark.parametrize("tokens", [16, 128, 256, 300, 512])
@pytest.mark.parametrize("rows,cols", [(57344, 4096), (256, 65536)])
def test_linear_gives_up_with_copies_in_flight(nm, tokens, rows, cols):
    """Half of the blocks give up soon; the others in the midst of their work, copies and
    products in flight, those of a cluster too: they end as well, and the next call is right."""
    p = Product(nm, rows, cols, tokens, (2, 4), seed=tokens)
    good = p.run(nm)
    y = torch.empty_like(good)
    for limit in (1, 50, 500):
        stalled(nm, p, y, limit)
        nm.nm_wait_timeouts(reset=True)
        assert torch.equal(p.run(nm, Y=y), good)
        assert nm.nm_wait_timeouts() == 0


@pytest.mark.parametrize("tokens,rows,cols", [(16, 128, 1024), (300, 256, 16384)])
def test_a_call_that_does_nothing_still_keeps_the_order(nm, tokens, rows, cols):
    """With the flag set nm_linear's blocks leave at once; what follows on the stream is
    after what came before all the same: log probabilities from a long row, read by a norm."""
    p = Product(nm, rows, cols, tokens, seed=1)
    y = p.run(nm)
    g = generator(2)
    x = torch.randn((1, 1 << 24), device="cuda", generator=g)
    ids = torch.randint(0, 1 << 24, (1, 1024), device="cuda", generator=g).to(torch.int32)
    want = nm.nm_token_logprobs(x, ids)[0]
    want_h, _ = nm.nm_residual_norm(want)
    lp = torch.empty_like(want)
    stalled(nm, p, y)
    for _ in range(10):
        lp.fill_(1.0)
        nm.nm_token_logprobs(x, ids, logprob=lp)
        p.run(nm, Y=y)
        h, _ = nm.nm_residual_norm(lp)
        assert torch.equal(h, want_h)
    nm.nm_wait_timeouts(reset=True)
    p.run(nm, Y=y)
    assert nm.nm_wait_timeouts() == 0


# ---- all of them ------------------------------------------------------------------------
def calls(nm):
    g = generator(8)
    out = []
    for tokens in (1, 6, 8, 40, 200, 300, 520):
        p = Product(nm, 130, 2048, tokens, act="silu", gated=True, bias=True, residual=True, seed=tokens)
        out.append((lambda p=p, **kw: [p.run(nm, **kw)]))
    for tokens in (8, 16):
        p = Product(nm, 64, 28672, tokens, act="gelu", seed=tokens)
        out.append((lambda p=p, **kw: [p.run(nm, **kw)]))
    n = Norm(33, 1000, "layer", "rms", "token", torch.float32)
    out.append(lambda **kw: list(n.run(nm, **kw)))
    x = torch.randn((5, 50257), device="cuda", generator=g).half()
    ids = torch.zeros((5, 2), dtype=torch.int32, device="cuda")
    out.append(lambda **kw: list(nm.nm_token_logprobs(x, ids, top=7, **kw)))
    y = torch.randn((400, 3001), device="cuda", generator=g)
    out.append(lambda **kw: list(nm.nm_token_logprobs(y, top=32, **kw)))
    return out


def same(a, b):
    return all(torch.equal(u.nan_to_num(nan=7.0), v.nan_to_num(nan=7.0)) for u, v in zip(a, b))


def test_calls_repeat_bit_for_bit(nm):
    for i, call in enumerate(calls(nm)):
        first = call()
        for _ in range(5):
            assert same(first, call()), i


def test_calls_on_other_streams_at_once(nm):
    cs = calls(nm)
    want = [c() for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = [[c(stream=s) for c, s in zip(cs, streams)] for _ in range(4)]
    torch.cuda.synchronize()
    for turn in got:
        for i, (a, b) in enumerate(zip(want, turn)):
            assert same(a, b), i


def test_calls_captured_and_replayed(nm):
    cs = calls(nm)
    want = [c() for c in cs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [c() for c in cs]
    for _ in range(3):
        for g in got:
            for t in g:
                t.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(want, got)):
        assert same(a, b), i


def test_calls_follow_what_the_stream_writes(nm):
    """Every kernel waits for the one before it: inputs written just before, and outputs
    read just after, on the same stream."""
    p = Product(nm, 512, 2048, 4, residual=True)
    x, res = p.x.clone(), p.kw["residual"].clone()
    want = p.run(nm)
    h, _ = nm.nm_residual_norm(want)
    lp = nm.nm_token_logprobs(h, top=4)
    for _ in range(20):
        p.x.fill_(NAN)
        p.kw["residual"].fill_(NAN)
        p.x.copy_(x)
        p.kw["residual"].copy_(res)
        h2, _ = nm.nm_residual_norm(p.run(nm))
        lp2 = nm.nm_token_logprobs(h2, top=4)
        assert torch.equal(h, h2) and same(lp, lp2)


def test_a_layer_of_them(nm):
    """As a decoder layer uses them, feed-forward block and answer, against the same in
    64 bits: each operator's tolerance is checked on its own inputs above; here the steps'
    outputs feed one another, and every step is checked against its 64-bit form of the
    inputs it was given."""
    g = generator(11)
    for tokens in (1, 5, 24):
        hidden, ffn, vocab = 512, 1024, 3001
        up = Product(nm, 2 * ffn, hidden, tokens, (2, 4), "silu", True, seed=1)
        down = Product(nm, hidden, ffn, tokens, (2, 4), bias=True, scale=0.5, seed=2)
        head = Product(nm, vocab, hidden, tokens, (16, 32), seed=3, scale=4.0)
        stream = torch.randn((tokens, hidden), device="cuda", generator=g).half()
        block = torch.randn((tokens, hidden), device="cuda", generator=g).half()
        n = Norm(tokens, hidden, "rms", "rms")
        n.residual, n.block = stream, block
        want_h, want_s = n.want()
        h, stream = n.run(nm, residual_out=stream)
        within(h, want_h, "norm")
        within(stream, want_s, "stream")
        up.x = h
        a = up.run(nm)
        within(a, up.want(), "gate and up")
        down.x = a
        down.kw["residual"] = stream.clone()
        stream = down.run(nm, Y=stream, residual=stream)
        within(stream, down.want(), "down")
        head.x, _ = nm.nm_residual_norm(stream, weight=n.kw["weight"])
        logits = head.run(nm)
        within(logits, head.want(), "head")
        check_logprobs(nm, logits, logits.float().argmax(1).to(torch.int32), 20, 1.0, "answer")
    assert nm.nm_wait_timeouts() == 0
