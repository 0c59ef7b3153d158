"""Limits and refusals of the 4-bit cache and the norm and rotation calls (CPU): the C ABI before any launch, and the
binding on ``meta`` tensors."""
import ctypes

import pytest
import torch

from gated_block_sparse_gate_b200 import binding as gb
from tests.test_kv4_rope_checks import BF, F32, I32, OK, cache, heads, lib, meta, on_meta, rejected, rope_params  # noqa: F401


def test_the_cache_sets_its_own_limits(lib):
    """B * Hq * N of 2^31 and more, which gbs_decode_ex refuses for its tensor maps; a row's blocks are counted in int."""
    for B, Hq, Hkv, N in ((128, 64, 8, 262144), (1, 1, 1, 2 ** 31 - 1), (4096, 128, 8, 1 << 20)):
        p = gb.make_params(B, Hq, Hkv, N, 128, 64, 32, "sparse")
        assert lib.gbs_kv4_workspace_bytes(ctypes.byref(p)) >= 256
        assert lib.gbs_workspace_bytes(ctypes.byref(p), gb.OP_DECODE) == 0
        c = cache(block_table=OK, max_blocks=-(-N // 64), num_pages=1 << 20)
        for f in (lib.gbs_kv4_append, lib.gbs_kv4_read):
            assert f(ctypes.byref(p), ctypes.byref(c), heads(), heads(), 0, OK, None, None, None) == 0
    p = gb.make_params(1 << 20, 1 << 11, 1, 64, 128, 64, 32, "sparse")
    assert lib.gbs_kv4_workspace_bytes(ctypes.byref(p)) == 0 and b"B * Hq" in lib.gbs_last_error()


def test_a_block_table_of_more_rows_than_int32_holds(on_meta):
    """The binding names a length that the library can be told."""
    wide = meta(2, 2 ** 25 + 8, dtype=I32)
    pages = gb.kv4_cache(2, 2, 64, num_pages=8, device="meta")
    assert gb._check_kv4("x", pages, 2, 64, torch.device("meta"), 64, wide)[2] == 2 ** 31 - 1
    gb.kv4_append(meta(2, 2, 5, 64), meta(2, 2, 5, 64), pages, meta(2, dtype=I32), block_table=wide)


def test_calls_enter_the_device_and_the_stream_of_their_tensors(monkeypatch):
    """With stand-ins for the current device, for entering one and for streams."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "device", lambda d: ("device", d))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: ("stream", s))
    here, there = torch.device("cuda", 0), torch.device("cuda", 1)
    assert gb._elsewhere("x", here, None) is None
    assert gb._elsewhere("x", there, None) == ("device", there)

    class Stream:
        device = there

    side = Stream()
    assert gb._elsewhere("x", there, side) == ("stream", side)
    assert "stream is on cuda:1" in rejected(gb._elsewhere, "x", here, side)


# ------------------------------------------------------------------ outputs apart from inputs

B, N, HQ, HKV, D = 2, 8, 4, 2, 64
PACKED = dict(b=N * (HQ + 2 * HKV) * D, h=D, n=(HQ + 2 * HKV) * D)  # of a projection's q, k and v
FAR = 1 << 30


def parts(at, es=2):
    return [heads(at + i * D * es, **PACKED) for i in (0, HQ, HQ + HKV)]


def planes(at, es=2):
    """Three head-major tensors, one after another."""
    return [heads(at + i * B * N * D * es, b=h * N * D, h=N * D, n=D) for i, h in ((0, HQ), (HQ, HKV), (HQ + HKV, HKV))]


def apart(call):
    """The library's answer: True where the tensors' places are accepted (and the launch fails without a GPU)."""
    s = call()
    assert s in (1, 3) if not torch.cuda.is_available() else s == 1
    return s == 3


def test_outputs_that_share_memory_are_refused(lib):
    if torch.cuda.is_available():
        pytest.skip("the accepted calls have no memory behind them")
    p = rope_params(B=B, N=N, Hq=HQ, Hkv=HKV, d=D)
    ws = lib.gbs_qkv_rope_workspace_bytes(ctypes.byref(p))

    def fwd(ins, outs):
        return apart(lambda: lib.gbs_qkv_rope_fwd(ctypes.byref(p), *ins, OK, OK, OK, OK, OK, *outs, None, None))

    def bwd(x, ins, outs, w=OK):
        return apart(lambda: lib.gbs_qkv_rope_bwd(ctypes.byref(p), *x[:2], w, w, OK, OK, OK, *ins, *outs, OK, OK, OK,
                                                  ws, None))

    total = B * N * (HQ + 2 * HKV) * D * 2
    assert fwd(parts(FAR), planes(FAR + total)) and fwd(parts(FAR + total), planes(FAR))
    assert not fwd(parts(FAR), planes(FAR)) and not fwd(parts(FAR), parts(FAR))
    assert not fwd(parts(FAR), planes(FAR + total - 16)) and not fwd(parts(FAR + total - 16), planes(FAR))
    q, k, v = planes(FAR + total)
    assert not fwd(parts(FAR), [q, q, v]) and not fwd(parts(FAR), [q, k, k])
    assert b"K and V share memory" in lib.gbs_last_error()
    # the heads of outputs between those of the inputs, in tokens of both
    wide = dict(b=2 * PACKED["b"], h=D, n=2 * PACKED["n"])
    ins = [heads(FAR + i * D * 2, **wide) for i in (0, HQ, HQ + HKV)]
    outs = [heads(FAR + (i + HQ + 2 * HKV) * D * 2, **wide) for i in (0, HQ, HQ + HKV)]
    assert fwd(ins, outs) and fwd(outs, ins)
    assert not fwd(ins, [heads(FAR + (i + HQ + 2 * HKV - 1) * D * 2, **wide) for i in (0, HQ, HQ + HKV)])
    # the gradient where the projection is: refused where it is read, not without a norm
    assert bwd(parts(FAR + total), planes(FAR), parts(FAR + 2 * total))
    assert not bwd(parts(FAR + total), planes(FAR), parts(FAR + total))
    assert b"q and dq share memory" in lib.gbs_last_error()
    assert bwd(parts(FAR + total), planes(FAR), parts(FAR + total), w=None)
    assert not bwd(parts(FAR + total), planes(FAR), parts(FAR), w=None)
    c = cache(kc=FAR, kp=FAR, vc=FAR, vp=FAR)
    params = gb.make_params(B, HKV, HKV, 250, D, 64, 4, "sparse")

    def read(K, V):
        return apart(lambda: lib.gbs_kv4_read(ctypes.byref(params), ctypes.byref(c), K, V, N, OK, None, None, None))

    assert read(k, v) and not read(k, k)


def test_what_is_found_to_share_memory(lib):
    """Random places and strides against the elements themselves: nothing that shares one is accepted."""
    if torch.cuda.is_available():
        pytest.skip("the accepted calls have no memory behind them")
    import random

    rng, found = random.Random(0), {False: 0, True: 0}
    params = gb.make_params(2, 2, 2, 250, D, 64, 4, "sparse")
    c = cache(kc=FAR, kp=FAR, vc=FAR, vp=FAR)
    for _ in range(3000):
        places, args = [], []
        for _ in "kv":
            steps = rng.sample([D, 2 * D, 4 * D, 8 * D, 3 * D, 24 * D], 3)
            at = rng.randrange(0, 40) * D // rng.choice((1, 2))
            places.append({at + b * steps[0] + h * steps[1] + n * steps[2] + x for b in range(2) for h in range(2)
                           for n in range(3) for x in range(0, D, 8)})
            args.append(heads(FAR + 2 * at, *steps))
        ok = apart(lambda: lib.gbs_kv4_read(ctypes.byref(params), ctypes.byref(c), *args, 3, OK, None, None, None))
        shares = bool(places[0] & places[1])
        assert not (ok and shares)
        found[ok == (not shares)] += 1
    assert found[True] > 2000  # and most that share none are


# ------------------------------------------------------------------ the binding's own refusals


def test_arguments_of_another_kind_are_refused_in_words(on_meta):
    """GbsError where an argument has a form that nothing can be made of: what is not a tuple, a number or that large."""
    qkv = meta(2, 9, 8, 64)
    q, k, v = qkv.split((4, 2, 2), 2)
    t, pos = meta(32, 32, dtype=F32), meta(2, 9, dtype=I32)
    rope = lambda **kw: gb.qkv_rope(q, k, v, t, t, pos, **kw)  # noqa: E731
    back = lambda **kw: gb.qkv_rope_backward(q, k, t, t, pos, meta(2, 4, 9, 64), meta(2, 2, 9, 64), None,  # noqa: E731
                                             **kw)
    flat, start = gb.kv4_cache(3, 2, 64, L=200, device="meta"), meta(3, dtype=I32)
    qs, S = meta(3, 4, 64), meta(3, 4, 4, dtype=F32)
    decode = lambda **kw: gb.kv4_decode(qs, flat, S, 200, **kw)  # noqa: E731
    for call, text in ((lambda: rope(axes=[0.0] * 32), "whole numbers"), (lambda: rope(axes=3), "whole numbers"),
                       (lambda: rope(out=3), "out must be"), (lambda: back(grads=q), "grads must be"),
                       (lambda: rope(eps="a"), "cannot be passed"), (lambda: decode(topk=2 ** 40), "cannot be passed"),
                       (lambda: decode(topk=2.5), "cannot be passed"),
                       (lambda: gb.kv4_read(flat, start[0], 4), "start must be"),
                       (lambda: gb.kv4_read(flat, start, 4.0), "T must be"),
                       (lambda: gb.kv4_read(flat, start, 4, out=(qs,)), "out must be"),
                       (lambda: gb.kv4_read(flat, start, 4, out=qs), "out must be")):
        assert text in rejected(call)
    rope(axes=torch.zeros(32, dtype=torch.int64))  # anything that counts as whole numbers


def test_ranges_beyond_64_bits_are_not_taken_for_apart(lib):
    """The largest strides with the most tokens: the same place is refused whatever its end would be."""
    if torch.cuda.is_available():
        pytest.skip("no memory behind them")
    for n in (1 << 28, 3 << 26, (1 << 29) - 1):
        p = rope_params(B=1, N=n, Hq=HQ, Hkv=HKV, d=D)
        t = [heads(FAR, b=0, h=D, n=1 << 42) for _ in "qkv"]
        s = lib.gbs_qkv_rope_fwd(ctypes.byref(p), *t, None, None, OK, OK, OK, *t, None, None)
        assert s == 1 and b"share memory" in lib.gbs_last_error()
