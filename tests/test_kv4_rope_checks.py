"""What the 4-bit cache and the norm and rotation calls refuse (CPU): the C ABI before any launch, and the
binding's checks of layouts on ``meta`` tensors (shapes, no storage)."""
import ctypes

import pytest
import torch

from gated_block_sparse_gate_b200 import binding as gb
from gated_block_sparse_gate_b200.build import build

BF, F32, I32, U8, F16 = torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.float16
OK, ODD = 4096, 4100


def meta(*shape, dtype=BF):
    return torch.empty(*shape, dtype=dtype, device="meta")


@pytest.fixture(scope="module")
def lib():
    build()
    return gb.load_library()


@pytest.fixture
def on_meta(monkeypatch):
    """The calls run on meta tensors, with a library that returns success for everything."""
    class Library:
        def __getattr__(self, name):
            return (lambda *a: 256) if name.endswith("_bytes") else lambda *a: 0

    monkeypatch.setattr(gb, "_DEVICE_TYPES", ("meta",))
    monkeypatch.setattr(gb, "load_library", Library)
    monkeypatch.setattr(gb, "_current", lambda device: 0)


def rejected(fn, *args, status=1, **kw):
    with pytest.raises(gb.GbsError) as e:
        fn(*args, **kw)
    assert e.value.status == status
    return str(e.value)


# ------------------------------------------------------------------ the C ABI


def rope_params(**kw):
    a = dict(B=2, N=8, Hq=4, Hkv=2, d=64, rot=64, interleaved=0, n_axes=1, axis=(), max_pos=16, dtype=0, w_dtype=1,
             eps=1e-6)
    a.update(kw)
    a["axis"] = (ctypes.c_ubyte * 64)(*a["axis"])
    return gb.RopeParams(**a)


def heads(ptr=OK, b=4096, h=1024, n=64):
    return ctypes.byref(gb.Heads(ptr, b, h, n))


def fwd(lib, p, t=None, side=(OK, OK, OK, OK, OK), ws=OK):
    t = t or {}
    return lib.gbs_qkv_rope_fwd(ctypes.byref(p), *(t.get(n, heads()) for n in "qkv"), *side,
                                *(t.get(n, heads()) for n in "QKV"), ws, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(B=0), 1, b"positive"), (dict(N=0), 1, b"positive"), (dict(Hkv=-1), 1, b"positive"),
    (dict(d=96), 2, b"d 96"), (dict(rot=12), 1, b"rot 12"), (dict(rot=72), 1, b"rot 72"), (dict(rot=-8), 1, b"rot"),
    (dict(interleaved=2), 1, b"interleaved"), (dict(n_axes=0), 1, b"n_axes"), (dict(n_axes=5), 1, b"n_axes"),
    (dict(axis=(0, 1)), 1, b"axis[1]"), (dict(max_pos=0), 1, b"max_pos"), (dict(dtype=2), 1, b"dtype"),
    (dict(w_dtype=7), 1, b"w_dtype"), (dict(eps=-1.0), 1, b"eps"), (dict(eps=float("nan")), 1, b"eps"),
    (dict(eps=float("inf")), 1, b"eps"), (dict(B=1 << 20, N=1 << 12), 1, b"too large"),
])
def test_rope_parameters(lib, kw, status, text):
    p = rope_params(**kw)
    assert lib.gbs_qkv_rope_workspace_bytes(ctypes.byref(p)) == 0
    assert fwd(lib, p) == status and text in lib.gbs_last_error()


def test_rope_tensors(lib):
    p = rope_params()
    for n in "qkQK":
        assert fwd(lib, p, {n: None}) == 1 and n.encode() + b" is NULL" in lib.gbs_last_error()
    for n in "qkvQKV":
        assert fwd(lib, p, {n: heads(ODD)}) == 1 and b"16-byte" in lib.gbs_last_error()
        for bad in (dict(b=4), dict(h=-64), dict(n=65), dict(b=1 << 43)):
            assert fwd(lib, p, {n: heads(**bad)}) == 1 and b"stride" in lib.gbs_last_error()
    assert fwd(lib, p, {"v": None}) == 1 and b"both v and V" in lib.gbs_last_error()
    assert fwd(lib, p, side=(OK, None, OK, OK, OK)) == 1 and b"both weights" in lib.gbs_last_error()
    for i in (2, 3, 4):
        side = [OK] * 5
        side[i] = None
        assert fwd(lib, p, side=side) == 1 and b"is NULL" in lib.gbs_last_error()
        side[i] = 4098 if i == 4 else 4104
        assert fwd(lib, p, side=side) == 1 and b"aligned" in lib.gbs_last_error()
    assert fwd(lib, p, ws=4096 + 16) == 5


def test_rope_backward_workspace(lib):
    p = rope_params()
    need = lib.gbs_qkv_rope_workspace_bytes(ctypes.byref(p))
    assert need > 256

    def bwd(ws=OK, n=need, dw=OK, dv=heads()):
        return lib.gbs_qkv_rope_bwd(ctypes.byref(p), heads(), heads(), OK, OK, OK, OK, OK, heads(), heads(), heads(),
                                    heads(), heads(), dv, dw, OK, ws, n, None)

    assert bwd(ws=None) == 5 and bwd(n=need - 1) == 5 and bwd(ws=OK + 128) == 5
    assert bwd(dw=None) == 1 and b"dwq" in lib.gbs_last_error()
    assert bwd(dv=None) == 1 and b"both dV and dv" in lib.gbs_last_error()


def cache(**kw):
    a = dict(kc=OK, kp=OK, vc=OK, vp=OK, block_table=None, max_blocks=0, num_pages=0, cap=256)
    a.update(kw)
    return gb.Kv4CacheDesc(**a)


@pytest.mark.parametrize("kw,text", [
    (dict(kc=None), b"kc is NULL"), (dict(vp=ODD), b"vp is not 16"), (dict(cap=192), b"cap"), (dict(cap=250), b"cap"),
    (dict(block_table=OK, max_blocks=3, num_pages=9), b"max_blocks"),
    (dict(block_table=OK, max_blocks=4, num_pages=0), b"num_pages"),
    (dict(block_table=4098, max_blocks=4, num_pages=9), b"block_table"),
])
def test_cache_descriptions(lib, kw, text):
    p = gb.make_params(2, 4, 2, 250, 64, 64, 4, "sparse")
    c = cache(**kw)
    ws = lib.gbs_kv4_workspace_bytes(ctypes.byref(p))
    assert ws > 0
    calls = [lambda: lib.gbs_kv4_decode(ctypes.byref(p), ctypes.byref(c), None, 0, OK, OK, OK, OK, 0, OK, ws, None)]
    for f in (lib.gbs_kv4_append, lib.gbs_kv4_read):
        calls.append(lambda f=f: f(ctypes.byref(p), ctypes.byref(c), heads(), heads(), 8, OK, None, None, None))
    for call in calls:
        assert call() == 1 and text in lib.gbs_last_error(), lib.gbs_last_error()


def test_append_and_read_arguments(lib):
    p = gb.make_params(2, 4, 2, 250, 64, 64, 4, "sparse")

    def call(f, K=heads(), V=heads(), T=8, start=OK, count=None, ws=None, p=p, c=cache()):
        return f(ctypes.byref(p), ctypes.byref(c), K, V, T, start, count, ws, None)

    for f in (lib.gbs_kv4_append, lib.gbs_kv4_read):
        assert call(f, K=None) == 1 and call(f, V=heads(ODD)) == 1 and call(f, K=heads(n=60)) == 1
        assert call(f, T=-1) == 1 and call(f, start=None) == 1 and call(f, start=4097) == 1
        assert call(f, count=4098) == 1 and call(f, ws=OK + 8) == 5
        assert call(f, T=1 << 30) == 1 and b"too large" in lib.gbs_last_error()
        assert call(f, T=0) == 0  # nothing to do, nothing launched
        assert call(f, p=gb.make_params(2, 4, 2, 250, 96, 64, 4, "sparse")) == 2


def test_decode_arguments(lib):
    def call(p=None, c=cache(), lens=None, shared=0, q=OK, S=OK, O=OK, LSE=OK, splits=0, ws=OK, n=None):
        p = p or gb.make_params(2, 4, 2, 250, 64, 64, 4, "sparse")
        n = lib.gbs_kv4_workspace_bytes(ctypes.byref(p)) if n is None else n
        return lib.gbs_kv4_decode(ctypes.byref(p), ctypes.byref(c), lens, shared, q, S, O, LSE, splits, ws, n, None)

    for kw in (dict(q=None), dict(S=None), dict(O=ODD), dict(LSE=ODD), dict(shared=2), dict(splits=-1),
               dict(splits=33), dict(lens=4098),
               dict(p=gb.make_params(2, 4, 2, 250, 64, 64, 300, "sparse"), n=1 << 30),
               dict(p=gb.make_params(2, 4, 2, 250, 64, 64, 4, "threshold", tau=0.0), n=1 << 30),
               dict(p=gb.make_params(2, 3, 2, 250, 64, 64, 4, "sparse"), n=1 << 30)):
        assert call(**kw) == 1, kw
    assert call(ws=None) == 5 and call(ws=OK + 64) == 5 and call(n=255) == 5
    assert call(p=gb.make_params(2, 4, 2, 250, 64, 32, 4, "sparse"), n=1 << 30) == 2


# ------------------------------------------------------------------ the binding


def rope_args(B=2, N=9, Hq=4, Hkv=2, d=64, rot=64, axes=None, **kw):
    qkv = meta(B, N, Hq + 2 * Hkv, d)
    a = dict(zip("qkv", qkv.split((Hq, Hkv, Hkv), 2)), cos=meta(32, rot // 2, dtype=F32),
             sin=meta(32, rot // 2, dtype=F32), pos=meta(B, N, dtype=I32))
    a.update(kw)
    return a


def test_rope_layouts(on_meta):
    assert [t.shape for t in gb.qkv_rope(**rope_args())] == [(2, 4, 9, 64), (2, 2, 9, 64), (2, 2, 9, 64)]
    gb.qkv_rope(**rope_args(pos=meta(2, 9, 3, dtype=I32)), axes=[i % 3 for i in range(32)])
    w = dict(wq=meta(64, dtype=F32), wk=meta(64, dtype=F32))
    gb.qkv_rope(**rope_args(), **w)
    for kw, text in ((dict(k=meta(2, 9, 2, 64, dtype=F32)), "k has dtype"), (dict(v=meta(2, 9, 3, 64)), "v has shape"),
                     (dict(q=meta(2, 9, 64, 4).transpose(2, 3)), "contiguous channels"),
                     (dict(pos=meta(2, 9, dtype=torch.int64)), "pos has dtype"), (dict(pos=meta(2, 8, dtype=I32)), "pos"),
                     (dict(sin=meta(32, 16, dtype=F32)), "sin has shape"), (dict(cos=meta(32, 32)), "cos has dtype"),
                     (dict(axes=[0] * 31), "axes has 31"), (dict(axes=[1] * 32), "axis is outside"),
                     (dict(wq=meta(64, dtype=F32)), "both weights"), (dict(out=(1, 2)), "out must be"),
                     (dict(wq=meta(64, dtype=F32), wk=meta(64)), "wk has dtype"),
                     (dict(q=meta(2, 9, 4, 64, dtype=F16)), "float16"), (dict(ws=meta(8, dtype=U8)), "256")):
        with pytest.raises(gb.GbsError, match=text):
            gb.qkv_rope(**{**rope_args(), **kw})


def test_outputs_whose_elements_share_memory(on_meta):
    dev = torch.device("meta")
    h = lambda t, out: gb.Heads.from_buffer_copy(  # noqa: E731
        gb._heads("t", "X", t, tuple(t.shape), (BF,), dev, out=out))
    shared = meta(2, 1, 9, 64).expand(2, 4, 9, 64)
    assert h(shared, False).stride_h == 0
    assert "share memory" in rejected(h, shared, True)
    window = torch.empty(1, device="meta", dtype=BF).expand(4096).as_strided((2, 2, 9, 64), (2048, 512, 64, 1))
    assert "share memory" in rejected(h, window, True)
    assert h(meta(2, 9, 4, 64).transpose(1, 2), True).stride_n == 256


@pytest.mark.skipif(gb._marshal is None, reason="built without the headers")
def test_native_checks_say_what_those_in_python_say():
    """On host tensors (device index -1), whose answers need no GPU."""
    x = torch.zeros(2, 3, 5, 64, dtype=BF)
    views = [x, x.transpose(1, 2), x[:, :, :, ::2], x[:, :1].expand(2, 3, 5, 64), x[:1], x.float(), x.view(-1),
             torch.nn.Parameter(x.float()), None, 3, torch.zeros(0, 3, 5, 64, dtype=BF)]
    python_fits = lambda t, dt, i, s: (isinstance(t, torch.Tensor) and t.get_device() == i and t.dtype in dt  # noqa: E731
                                       and (s is None or t.shape == s) and t.is_contiguous())
    for t in views:
        for dt in ((BF,), (F32, BF), (F32,)):
            for shape in (None, (2, 3, 5, 64), (2, 5, 3, 64), (1, 3, 5, 64)):
                for index in (-1, 0, None):
                    assert gb._marshal.fits(t, dt, index, shape) == python_fits(t, dt, index, shape)
    h = lambda t, **kw: gb.Heads.from_buffer_copy(gb._marshal.heads(  # noqa: E731
        t, (BF,), -1, tuple(t.shape), kw.get("token_major", False), kw.get("written", False)))
    for t in views[:5]:
        for token_major in (False, True):
            if t.stride(3) != 1:
                assert gb._marshal.heads(t, (BF,), -1, tuple(t.shape), token_major, False) is None
                continue
            got = h(t, token_major=token_major)
            st = [0 if n == 1 else s for n, s in zip(t.shape, t.stride())]
            want = (st[0], st[2], st[1]) if token_major else (st[0], st[1], st[2])
            assert (got.ptr, got.stride_b, got.stride_h, got.stride_n) == (t.data_ptr(), *want)
    assert gb._marshal.heads(views[1], (BF,), -1, (2, 5, 3, 64), True, True) is None  # written, and not contiguous
    assert h(x, written=True).stride_h == 5 * 64
    with pytest.raises(TypeError):
        gb._marshal.heads(x, (BF,), -1)
    with pytest.raises(TypeError):
        gb._marshal.fits(x, BF, -1, None)


def test_kv4_layouts(on_meta):
    B, Hkv, d, L = 3, 2, 64, 200
    flat = gb.kv4_cache(B, Hkv, d, L=L, device="meta")
    pages = gb.kv4_cache(B, Hkv, d, num_pages=20, device="meta")
    assert flat[0].shape == (B, Hkv, 256, 32) and pages[3].shape == (20, Hkv, 64, 2, 2)
    table, start = meta(B, 4, dtype=I32), meta(B, dtype=I32)
    K = meta(B, Hkv, 5, d)
    assert gb.kv4_append(K, K, flat, start) is None
    for args, kw, text in (((K, K, pages, start), {}, "key codes have shape"),
                           ((K, K, flat[:3], start), {}, "cache must be"),
                           ((K, K, (flat[0], flat[1].float(), *flat[2:]), start), {}, "key parameters has dtype"),
                           ((K, K, (*flat[:2], flat[2][:, :, :64], flat[3]), start), {}, "value codes has shape"),
                           ((K, K, pages, start), dict(block_table=meta(B + 1, 4, dtype=I32)), "block_table must"),
                           ((K, K, pages, start), dict(block_table=table.long()), "block_table has dtype"),
                           ((K, K, flat, start[:2]), {}, "start has shape"),
                           ((K, K, flat, start), dict(count=start.float()), "count has dtype"),
                           ((K, K[:, :, :4], flat, start), {}, "V has shape"),
                           ((K.half(), K.half(), flat, start), {}, "float16")):
        with pytest.raises(gb.GbsError, match=text):
            gb.kv4_append(*args, **kw)
    q, S = meta(B, 4, d), meta(B, 4, 4, dtype=F32)
    assert [t.shape for t in gb.kv4_decode(q, flat, S, L)] == [(B, 4, d), (B, 4)]
    gb.kv4_decode(q, pages, S, L, block_table=table, seq_lens=start)
    assert [t.shape for t in gb.kv4_read(flat, start, 5)] == [(B, Hkv, 5, d)] * 2
    with pytest.raises(gb.GbsError, match="out must be"):
        gb.kv4_read(flat, start, 5, out=(K[:, :, :4], K[:, :, :4]))
    for kw, text in ((dict(L=257), "outside"), (dict(L=0), "outside"), (dict(S=meta(B, 2, 4, dtype=F32)), "S has"),
                     (dict(group_shared=True), "S has"), (dict(seq_lens=start[:1]), "seq_lens"),
                     (dict(out=meta(B, 4, d, dtype=F32)), "O has dtype"), (dict(q=q.half()), "float16")):
        with pytest.raises(gb.GbsError, match=text):
            gb.kv4_decode(**{**dict(q=q, cache=flat, S=S, L=L), **kw})
    with pytest.raises(gb.GbsError, match="either"):
        gb.kv4_cache(B, Hkv, d, L=4, num_pages=4, device="meta")


def test_axes_and_tables():
    assert gb.rope_axes((2, 1, 1)) == (0, 0, 1, 2)
    assert gb.rope_axes((3, 1, 2), interleaved=True) == (0, 1, 2, 0, 2, 0)
    cos, sin = gb.rope_tables(200001, 8, 10000.0, "cpu")
    angle = torch.tensor(200000.0, dtype=torch.float64) * 10000.0 ** -0.25
    assert cos.dtype == F32 and abs(float(cos[200000, 1]) - float(angle.cos())) < 2 ** -24
    assert abs(float(sin[200000, 1]) - float(angle.sin())) < 2 ** -24
    assert gb.rope_tables(5, 0, device="cpu")[0].shape == (5, 0)


def test_host_tensors_never_reach_the_library(lib):
    z = torch.zeros(1, 2, 4, 64, dtype=BF)
    t = torch.zeros(4, 32)
    pos = torch.zeros(1, 2, dtype=I32)
    assert "CUDA" in rejected(gb.qkv_rope, z, z, z, t, t, pos)
    start = torch.zeros(1, dtype=I32)
    c = gb.kv4_cache(1, 2, 64, L=64, device="cpu")
    assert "CUDA" in rejected(gb.kv4_append, z, z, c, start)
    assert "CUDA" in rejected(gb.kv4_read, c, start, 4)
    assert "CUDA" in rejected(gb.kv4_decode, torch.zeros(1, 2, 64, dtype=BF), c, torch.zeros(1, 2, 1), 64)
