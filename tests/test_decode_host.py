"""Host side of the speculative-decoding operators: refusals that need no
device, and the rotary frequencies."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def nm():
    from sparse_spmv_memory_gb300 import _build
    _build.build()
    import sparse_spmv_memory_gb300 as m
    return m


def cache(**kw):
    """A well-formed e4m3 cache at addresses that are never dereferenced."""
    from sparse_spmv_memory_gb300.decode import _Cache
    d = dict(k=0x100000000, v=0x200000000, k_scale=0x300000000, v_scale=0x310000000, pages=10,
             page_stride=2 * 16 * 64, scale_page_stride=32, kv_heads=2, page_size=16, head_dim=64,
             type=1)
    d.update(kw)
    return _Cache(**d)


def ref(c):
    return None if c is None else ctypes.byref(c)


def test_inv_freq(nm):
    f = nm.nm_rope_inv_freq(64, 10000.0, device="cpu")
    want = [10000.0 ** (-2 * i / 64) for i in range(32)]
    assert f.tolist() == torch.tensor(want, dtype=torch.float64).float().tolist()
    lin = nm.nm_rope_inv_freq(64, 10000.0, "linear", 4.0, device="cpu")
    assert torch.allclose(lin * 4, f, rtol=1e-6)
    b = nm.nm_rope_inv_freq(128, 500000.0, "banded", 8.0, 1.0, 4.0, 8192.0, device="cpu")
    p = nm.nm_rope_inv_freq(128, 500000.0, device="cpu")
    kept = mixed = cut = 0
    for x, y in zip(b.tolist(), p.tolist()):
        wave = 2 * math.pi / y
        if wave < 8192 / 4 * 0.999:
            assert x == y
            kept += 1
        elif wave > 8192 * 1.001:
            assert abs(x * 8 - y) < 1e-6 * y
            cut += 1
        else:
            m = (8192 / wave - 1) / 3
            assert abs(x - ((1 - m) * y / 8 + m * y)) < 1e-5 * y
            mixed += 1
    assert kept and mixed and cut
    assert nm.nm_rope_inv_freq(0, device="cpu").numel() == 0
    L = nm.lib()
    buf = (ctypes.c_float * 8)()
    assert L.nm_rope_inv_freq(buf, 7, 1e4, 0, 1.0, 1.0, 4.0, 8192.0) == 2
    assert L.nm_rope_inv_freq(buf, 8, -1.0, 0, 1.0, 1.0, 4.0, 8192.0) == 2
    assert L.nm_rope_inv_freq(buf, 8, 1e4, 3, 1.0, 1.0, 4.0, 8192.0) == 2
    assert L.nm_rope_inv_freq(buf, 8, 1e4, 2, 1.0, 4.0, 4.0, 8192.0) == 2
    assert L.nm_rope_inv_freq(buf, 8, 1e4, 1, 0.0, 1.0, 4.0, 8192.0) == 2
    assert L.nm_rope_inv_freq(None, 8, 1e4, 0, 1.0, 1.0, 4.0, 8192.0) == 1
    with pytest.raises(ValueError):
        nm.nm_rope_inv_freq(8, scaling="other")


BAD_CACHES = [
    (dict(k=0), 1), (dict(v=0), 1), (dict(k_scale=0), 1), (dict(type=3), 2), (dict(type=-1), 2),
    (dict(page_size=12), 2), (dict(page_size=4), 2), (dict(page_size=1 << 21), 2),
    (dict(head_dim=96), 2), (dict(kv_heads=0), 2), (dict(kv_heads=1025), 2), (dict(pages=0), 2),
    (dict(pages=1 << 31), 2), (dict(page_stride=2047), 2), (dict(page_stride=1 << 40), 2),
    (dict(scale_page_stride=31), 2), (dict(page_stride=2064), 4), (dict(k=0x100000010), 4),
    (dict(v_scale=0x310000002), 4)]


@pytest.mark.parametrize("change,code", BAD_CACHES)
def test_caches_refused(nm, change, code):
    L, c = nm.lib(), cache(**change)
    q, o = 0x400000000, 0x500000000
    assert L.nm_rope_append(q, 512, 4, 4, o, o, o, 64, 0, 1.0, None, 0, ref(c), None) == code
    assert L.nm_cache_read(ref(c), o, 4, q, None, None) == code
    assert L.nm_tree_attention(q, 256, 4, 4, 1, o, 4, ref(c), o, 4, 4, o, None, 1.0, q + (1 << 20),
                               256, None, None, 0, None) == code


def test_append_refused(nm):
    L = nm.lib()
    base = dict(qkv=0x400000000, ld=512, tokens=4, q_heads=4, pos=0x500000000, slots=0x510000000,
                freq=0x520000000, rot=64, q=0x600000000, ldq=256, c=cache())

    def call(**kw):
        a = dict(base, **kw)
        return L.nm_rope_append(a["qkv"], a["ld"], a["tokens"], a["q_heads"], a["pos"], a["slots"],
                                a["freq"], a["rot"], 0, 1.0, a["q"], a["ldq"], ref(a["c"]), None)
    for name in ("qkv", "pos", "slots", "freq", "c"):
        assert call(**{name: None}) == 1, name
    assert call(tokens=-1) == 2 and call(tokens=1 << 31) == 2 and call(q_heads=0) == 2
    assert call(ld=504) == 2 and call(ldq=248) == 2
    assert call(rot=66) == 2 and call(rot=63) == 2 and call(rot=-2) == 2
    assert call(qkv=base["qkv"] + 8) == 4 and call(ld=516) == 4 and call(ldq=260) == 4
    assert call(q=base["q"] + 2) == 4 and call(pos=base["pos"] + 1) == 4
    assert call(slots=base["slots"] + 4) == 4
    assert call(q=base["qkv"] + 1024) == 7          # q over qkv
    assert call(qkv=0x100000000) == 7               # qkv over the cache
    assert call(q=0x300000000 - 32) == 7            # q over the scales
    assert call(tokens=0) == 0
    assert call(rot=0, freq=None, tokens=0) == 0


def test_read_refused(nm):
    L = nm.lib()
    c, slots, k, v = cache(), 0x500000000, 0x600000000, 0x610000000
    assert L.nm_cache_read(ref(c), None, 4, k, v, None) == 1
    assert L.nm_cache_read(None, slots, 4, k, v, None) == 1
    assert L.nm_cache_read(ref(c), slots, -1, k, v, None) == 2
    assert L.nm_cache_read(ref(c), slots, 1 << 31, k, v, None) == 2
    assert L.nm_cache_read(ref(c), slots, 4, k + 8, v, None) == 4
    assert L.nm_cache_read(ref(c), slots + 4, 4, k, v, None) == 4
    assert L.nm_cache_read(ref(c), slots, 4, k, k + 16, None) == 7
    assert L.nm_cache_read(ref(c), slots, 4, 0x100000000, v, None) == 7
    assert L.nm_cache_read(ref(c), slots, 0, k, v, None) == 0
    assert L.nm_cache_read(ref(c), slots, 4, None, None, None) == 0


def test_attention_refused(nm):
    L = nm.lib()
    base = dict(q=0x400000000, ldq=256, tokens=8, q_heads=4, seqs=2, start=0x500000000, nodes=4,
                c=cache(), table=0x510000000, ldt=6, cols=6, ctx=0x520000000, mask=0x530000000,
                scale=0.1, out=0x600000000, ldo=256, lse=0x610000000)

    def call(**kw):
        a = dict(base, **kw)
        return L.nm_tree_attention(a["q"], a["ldq"], a["tokens"], a["q_heads"], a["seqs"], a["start"],
                                   a["nodes"], ref(a["c"]), a["table"], a["ldt"], a["cols"], a["ctx"],
                                   a["mask"], a["scale"], a["out"], a["ldo"], a["lse"], None, 0, None)
    for name in ("q", "start", "c", "table", "ctx", "out"):
        assert call(**{name: None}) == 1, name
    assert call(tokens=-1) == 2 and call(seqs=65536) == 2 and call(seqs=-1) == 2
    assert call(q_heads=3) == 2 and call(q_heads=0) == 2 and call(q_heads=130, ldq=130 * 64) == 2
    assert call(nodes=0) == 2 and call(nodes=65) == 2
    assert call(ldq=248) == 2 and call(ldo=200) == 2 and call(cols=0) == 2 and call(ldt=5) == 2
    assert call(scale=float("nan")) == 2 and call(scale=float("inf")) == 2
    assert call(q=base["q"] + 8) == 4 and call(ldq=260) == 4 and call(ldo=268) == 4
    assert call(mask=base["mask"] + 4) == 4 and call(table=base["table"] + 2) == 4
    assert call(tokens=0) == 0 and call(seqs=0) == 0
    assert nm.nm_tree_attention_workspace_bytes(1, 3, 2, 64, 4) == 0
    assert nm.nm_tree_attention_workspace_bytes(1, 4, 2, 96, 4) == 0
    assert nm.nm_tree_attention_workspace_bytes(1, 4, 2, 64, 65) == 0


def test_verify_refused(nm):
    L = nm.lib()
    base = dict(logits=0x400000000, fp32=0, ld=1000, vocab=1000, draft=0x500000000, ldd=1000,
                ids=0x600000000, par=0x601000000, start=0x602000000, n=8, seqs=2, nodes=4,
                acc=0x603000000, race=0x604000000, ldr=1000, t=1.0, path=0x700000000,
                count=0x701000000, token=0x702000000)

    def call(**kw):
        a = dict(base, **kw)
        return L.nm_tree_verify(a["logits"], a["fp32"], a["ld"], a["vocab"], a["draft"], a["ldd"],
                                a["ids"], a["par"], a["start"], a["n"], a["seqs"], a["nodes"],
                                a["acc"], a["race"], a["ldr"], a["t"], a["path"], a["count"],
                                a["token"], None)
    for name in ("logits", "ids", "par", "start", "path", "count", "token", "acc", "race"):
        assert call(**{name: None}) == 1, name
    assert call(t=-0.1) == 2 and call(t=float("nan")) == 2 and call(t=float("inf")) == 2
    assert call(vocab=0) == 2 and call(vocab=(1 << 24) + 1, ld=1 << 25, ldd=1 << 25, ldr=1 << 25) == 2
    assert call(n=-1) == 2 and call(seqs=65536) == 2 and call(nodes=65) == 2 and call(nodes=0) == 2
    assert call(ld=999) == 2 and call(ldd=999) == 2 and call(ldr=999) == 2
    assert call(logits=base["logits"] + 1) == 4 and call(draft=base["draft"] + 2) == 4
    assert call(count=base["count"] + 2) == 4
    assert call(path=base["count"] - 16) == 7 and call(token=base["count"] + 4) == 7
    assert call(seqs=0) == 0
    assert call(t=0.0, acc=None, race=None, draft=None, seqs=0) == 0


def test_empty_calls_take_no_addresses(nm):
    """Arrays without elements: NULL is what an empty tensor has."""
    L, c, N = nm.lib(), cache(), None
    assert L.nm_rope_append(N, 512, 0, 4, N, N, N, 64, 0, 1.0, N, 0, ref(c), N) == 0
    assert L.nm_rope_append(N, 512, 1, 4, N, N, N, 64, 0, 1.0, N, 0, ref(c), N) == 1
    assert L.nm_rope_append(N, 504, 0, 4, N, N, N, 64, 0, 1.0, N, 0, ref(c), N) == 2
    assert L.nm_rope_append(N, 512, 0, 4, N, N, N, 64, 0, 1.0, N, 0, N, N) == 1
    assert L.nm_cache_read(ref(c), N, 0, N, N, N) == 0 and L.nm_cache_read(ref(c), N, 1, N, N, N) == 1
    for tokens, seqs, code in ((0, 0, 0), (0, 3, 0), (5, 0, 0), (5, 3, 1), (-1, 0, 2), (0, -1, 2)):
        assert L.nm_tree_attention(N, 256, tokens, 4, seqs, N, 4, ref(c), N, 4, 4, N, N, 1.0, N, 256, N, N, 0,
                                   N) == code
    for tokens, seqs, t, code in ((0, 0, 0.0, 0), (0, 0, 1.0, 0), (7, 0, 1.0, 0), (0, 2, 1.0, 1), (-1, 0, 1.0, 2)):
        assert L.nm_tree_verify(N, 0, 8, 8, N, 0, N, N, N, tokens, seqs, 4, N, N, 8, t, N, N, N, N) == code


def test_outputs_over_any_input_refused(nm):
    """What a call writes may not meet anything that it reads."""
    L, c = nm.lib(), cache()
    qkv, pos, slots, freq, q = 0x400000000, 0x500000000, 0x510000000, 0x520000000, 0x600000000

    def append(q=q, pos=pos, slots=slots, freq=freq):
        return L.nm_rope_append(qkv, 512, 4, 4, pos, slots, freq, 64, 0, 1.0, q, 256, ref(c), None)
    for over in (dict(pos=q + 16), dict(slots=q + 1024), dict(freq=q + 2040), dict(pos=0x100000000 + 64),
                 dict(slots=0x200000000 + 8), dict(freq=0x310000000 + 4)):
        assert append(**over) == 7, over
    for k, v in ((slots, None), (None, slots + 16), (slots - 64, None)):
        assert L.nm_cache_read(ref(c), slots, 4, k, v, None) == 7

    base = dict(q=0x400000000, start=0x500000000, table=0x510000000, ctx=0x520000000, mask=0x530000000,
                out=0x600000000, lse=0x610000000, ws=0x620000000)

    def attend(**kw):
        a = dict(base, **kw)
        return L.nm_tree_attention(a["q"], 256, 8, 4, 2, a["start"], 4, ref(c), a["table"], 6, 6, a["ctx"],
                                   a["mask"], 0.1, a["out"], 256, a["lse"], a["ws"], 1 << 40, None)
    for written in ("out", "lse"):
        for read in ("q", "start", "table", "ctx", "mask"):
            assert attend(**{read: base[written] + 16}) == 7, (written, read)

    base = dict(logits=0x400000000, draft=0x500000000, ids=0x600000000, par=0x601000000, start=0x602000000,
                acc=0x603000000, race=0x604000000, path=0x700000000, count=0x701000000, token=0x702000000)

    def verify(t=1.0, **kw):
        a = dict(base, **kw)
        return L.nm_tree_verify(a["logits"], 0, 1000, 1000, a["draft"], 1000, a["ids"], a["par"], a["start"], 8, 2,
                                4, a["acc"], a["race"], 1000, t, a["path"], a["count"], a["token"], None)
    for written in ("path", "count", "token"):
        for read in ("logits", "draft", "ids", "par", "start", "acc", "race"):
            assert verify(**{read: base[written]}) == 7, (written, read)
            if read not in ("draft", "acc", "race"):  # not read at temperature 0
                assert verify(t=0.0, **{read: base[written]}) == 7


def test_stall_selftests_refuse_a_limit_out_of_range(nm):
    L, c = nm.lib(), cache()
    o = 0x500000000
    for limit in (0, -5, 2000001):
        assert L.nm_tree_verify_stall_selftest(o, 0, 8, 8, None, 0, o, o, o, 4, 0, 4, None, None, 0, 0.0,
                                               o, o, o, limit, None) == 2
        assert L.nm_tree_attention_stall_selftest(o, 256, 8, 4, 0, o, 4, ref(c), o, 4, 4, o, None, 1.0,
                                                  o, 256, None, None, 0, limit, None) == 2


def test_binding_refuses_cpu_tensors_and_wrong_types(nm):
    k = torch.zeros((2, 1, 8, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        nm.nm_cache_read(k, k, torch.zeros(1, dtype=torch.int64))


@pytest.mark.filterwarnings("ignore")
def test_binding_refuses_tensors_of_two_devices(nm):
    """Tensors that only say which device they are on, and have no memory: the refusal
    comes before anything else is asked of them."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        def t(*shape, dtype=torch.int32, on=0):
            return torch.empty(shape, dtype=dtype, device=f"cuda:{on}")
        h, f, i64 = torch.float16, torch.float32, torch.int64
        k, v = t(4, 1, 8, 64, dtype=h), t(4, 1, 8, 64, dtype=h)
        other = "another device"
        with pytest.raises(ValueError, match=other):
            nm.nm_cache_read(k, v, t(3, dtype=i64, on=1))
        with pytest.raises(ValueError, match=other):
            nm.nm_cache_read(k, t(4, 1, 8, 64, dtype=h, on=1), t(3, dtype=i64))
        with pytest.raises(ValueError, match=other):
            nm.nm_rope_append(t(3, 256, dtype=h), k, v, t(3), t(3, dtype=i64, on=1), t(32, dtype=f), 2)
        with pytest.raises(ValueError, match=other):
            nm.nm_tree_attention(t(3, 2, 64, dtype=h), k, v, t(1, 4), t(1), t(2), 3,
                                 workspace=t(64, dtype=torch.uint8, on=1))
        with pytest.raises(ValueError, match=other):
            nm.nm_tree_verify(t(3, 9, dtype=h), t(3), t(3), t(2), 3, temperature=0.0, token=t(1, on=2))
