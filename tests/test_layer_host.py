"""Host side of the operators around the sparse products: refusals of the C calls that
need no device, at addresses that are never dereferenced."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

OK, NULL, SHAPE, ALIGN, ALIAS = 0, 1, 2, 4, 7
V, M, X, Y, B, R, W = (0x100000000 + (i << 36) for i in range(7))


@pytest.fixture(scope="module")
def nm():
    from sparse_spmv_memory_gb300 import _build
    _build.build()
    import sparse_spmv_memory_gb300 as m
    return m


def linear(nm, epilogue=True, **kw):
    from sparse_spmv_memory_gb300.layer import _Epilogue
    e = dict(bias=B, residual=R, ldres=64, activation=2, gated=0, scale=1.0)
    a = dict(values=V, masks=M, rows=64, cols=128, X=X, ldx=128, tokens=4, Y=Y, ldy=64, workspace=W, ws=1 << 30)
    for k, v in kw.items():
        (e if k in e else a)[k] = v
    ep = ctypes.byref(_Epilogue(**e)) if epilogue else None
    return nm.lib().nm_linear(a["values"], a["masks"], a["rows"], a["cols"], a["X"], a["ldx"], a["tokens"], ep,
                              a["Y"], a["ldy"], a["workspace"], a["ws"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(epilogue=False), NULL), (dict(values=0), NULL), (dict(masks=0), NULL), (dict(X=0), NULL), (dict(Y=0), NULL),
    (dict(rows=-1), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(cols=0), SHAPE), (dict(cols=48), SHAPE),
    (dict(cols=1 << 31), SHAPE), (dict(tokens=-1), SHAPE), (dict(tokens=1 << 31), SHAPE), (dict(ldx=120), SHAPE),
    (dict(ldx=1 << 31), SHAPE), (dict(ldy=63), SHAPE), (dict(ldres=63), SHAPE), (dict(rows=63, gated=1), SHAPE),
    (dict(activation=5), SHAPE), (dict(activation=-1), SHAPE), (dict(scale=math.inf), SHAPE),
    (dict(scale=math.nan), SHAPE), (dict(values=V + 16), ALIGN), (dict(masks=M + 2), ALIGN), (dict(X=X + 8), ALIGN),
    (dict(ldx=132), ALIGN), (dict(Y=Y + 1), ALIGN), (dict(bias=B + 1), ALIGN), (dict(residual=R + 1), ALIGN),
    (dict(workspace=W + 8), ALIGN), (dict(Y=X), ALIAS), (dict(Y=V + 64), ALIAS), (dict(Y=M), ALIAS),
    (dict(Y=B + 2), ALIAS), (dict(Y=R + 2), ALIAS), (dict(Y=R, ldy=72), ALIAS), (dict(rows=0), OK),
    (dict(tokens=0), OK), (dict(tokens=0, X=0, Y=0, values=0, masks=0), OK)], ids=str)
def test_linear(nm, kw, want):
    assert linear(nm, **kw) == want


def test_linear_stall_selftest_refuses_a_limit_out_of_range(nm):
    from sparse_spmv_memory_gb300.layer import _Epilogue
    e = ctypes.byref(_Epilogue(bias=None, residual=None, ldres=0, activation=0, gated=0, scale=1.0))
    for limit, want in ((0, SHAPE), (-1, SHAPE), (2000001, SHAPE), (20000, OK)):
        assert nm.lib().nm_linear_stall_selftest(V, M, 0, 128, X, 128, 16, e, Y, 64, None, 0, limit, None) == want


def norm(nm, pre=True, post=True, **kw):
    from sparse_spmv_memory_gb300.layer import _Norm
    n = dict(kind=1, params_fp32=0, weight=W, bias=None, offset=0.0, eps=1e-6)
    a = dict(residual=R, fp32=0, ldr=64, block=B, ldb=64, gate=V, ldg=64, scale=1.0, rscale=1.0, sout=X, lds=64,
             out=Y, ldo=64, tokens=4, width=64)
    for k, v in kw.items():
        (n if k in n else a)[k] = v
    ref = lambda want: ctypes.byref(_Norm(**n)) if want else None  # noqa: E731
    return nm.lib().nm_residual_norm(a["residual"], a["fp32"], a["ldr"], a["block"], a["ldb"], ref(post), a["gate"],
                                     a["ldg"], a["scale"], a["rscale"], a["sout"], a["lds"], ref(pre), a["out"],
                                     a["ldo"], a["tokens"], a["width"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(residual=0), NULL), (dict(sout=0, out=0), NULL), (dict(tokens=-1), SHAPE), (dict(tokens=1 << 31), SHAPE),
    (dict(width=0), SHAPE), (dict(width=32769, ldr=1 << 20, ldb=1 << 20, ldg=1 << 20, lds=1 << 20, ldo=1 << 20), SHAPE),
    (dict(ldr=63), SHAPE), (dict(ldb=63), SHAPE), (dict(ldg=63), SHAPE), (dict(ldg=-1), SHAPE), (dict(lds=63), SHAPE),
    (dict(ldo=63), SHAPE), (dict(kind=3), SHAPE), (dict(kind=-1), SHAPE), (dict(eps=-1e-6), SHAPE),
    (dict(eps=math.nan), SHAPE), (dict(offset=math.inf), SHAPE), (dict(scale=math.nan), SHAPE),
    (dict(rscale=math.inf), SHAPE), (dict(residual=R + 1), ALIGN), (dict(residual=R + 2, fp32=1), ALIGN),
    (dict(sout=X + 2, fp32=1), ALIGN), (dict(block=B + 1), ALIGN), (dict(gate=V + 1), ALIGN), (dict(out=Y + 1), ALIGN),
    (dict(weight=W + 1), ALIGN), (dict(weight=W + 2, params_fp32=1), ALIGN), (dict(out=R), ALIAS), (dict(out=B + 2), ALIAS),
    (dict(out=V), ALIAS), (dict(out=X), ALIAS), (dict(out=W), ALIAS), (dict(sout=B), ALIAS), (dict(sout=V), ALIAS),
    (dict(sout=W), ALIAS), (dict(sout=R + 2), ALIAS), (dict(sout=R, lds=72), ALIAS), (dict(tokens=0), OK),
    (dict(tokens=0, residual=0, out=0, sout=0), OK)], ids=str)
def test_norm(nm, kw, want):
    assert norm(nm, **kw) == want


def logprobs(nm, **kw):
    a = dict(logits=X, fp32=0, ld=100, rows=4, vocab=100, ids=V, ld_ids=2, n=2, t=1.0, lp=Y, h=B, top=5, at=R, tl=W)
    a.update(kw)
    return nm.lib().nm_token_logprobs(a["logits"], a["fp32"], a["ld"], a["rows"], a["vocab"], a["ids"], a["ld_ids"],
                                      a["n"], a["t"], a["lp"], a["h"], a["top"], a["at"], a["tl"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(logits=0), NULL), (dict(ids=0), NULL), (dict(lp=0), NULL), (dict(at=0), NULL), (dict(tl=0), NULL),
    (dict(rows=-1), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(vocab=0), SHAPE), (dict(vocab=(1 << 24) + 1, ld=1 << 25), SHAPE),
    (dict(ld=99), SHAPE), (dict(n=-1), SHAPE), (dict(n=1025, ld_ids=2000), SHAPE), (dict(ld_ids=1), SHAPE),
    (dict(top=-1), SHAPE), (dict(top=33), SHAPE), (dict(vocab=4), SHAPE), (dict(t=0.0), SHAPE), (dict(t=-1.0), SHAPE),
    (dict(t=math.nan), SHAPE), (dict(t=math.inf), SHAPE), (dict(t=2.0 ** -21), SHAPE), (dict(t=2.0 ** 21), SHAPE),
    (dict(logits=X + 1), ALIGN), (dict(logits=X + 2, fp32=1), ALIGN), (dict(ids=V + 2), ALIGN), (dict(lp=Y + 2), ALIGN),
    (dict(h=B + 2), ALIGN), (dict(at=R + 2), ALIGN), (dict(tl=W + 2), ALIGN), (dict(lp=X), ALIAS), (dict(lp=V), ALIAS),
    (dict(h=X + 4), ALIAS), (dict(at=V + 4), ALIAS), (dict(tl=X), ALIAS), (dict(lp=B), ALIAS), (dict(at=W), ALIAS),
    (dict(h=R + 8), ALIAS), (dict(rows=0), OK), (dict(rows=0, logits=0, ids=0, lp=0, h=0, at=0, tl=0), OK)], ids=str)
def test_logprobs(nm, kw, want):
    assert logprobs(nm, **kw) == want


def test_python_refuses_host_tensors_and_names(nm):
    x = torch.zeros((2, 64), dtype=torch.float16)
    for call in (lambda: nm.nm_residual_norm(x), lambda: nm.nm_token_logprobs(x),
                 lambda: nm.nm_linear(x, x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="norm must be one of"):
        nm.nm_residual_norm(x, norm="group")
    with pytest.raises(ValueError, match="activation must be one of"):
        nm.nm_linear(x, x, x, activation="tanh")
    with pytest.raises(TypeError):
        nm.nm_token_logprobs(7)


def test_no_kernel_leaves_before_it_waited_for_the_one_before_it():
    """A kernel that lets the next one start early and ends without having waited itself
    would let that one read what the kernel before both still writes."""
    import glob
    import os
    import re
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_spmv_memory_gb300", "csrc")
    kernels = 0
    for path in sorted(glob.glob(os.path.join(csrc, "*.cu*"))):
        with open(path) as f:
            code = re.sub(r"//[^\n]*", "", f.read())
        for part in code.split("pdl_launch_dependents();")[1:]:
            assert "pdl_wait_previous();" in part, path
            kernels += 1
            assert not re.search(r"\breturn\b", re.split(r"pdl_wait_previous\(\);", part)[0]), path
    assert kernels >= 15
