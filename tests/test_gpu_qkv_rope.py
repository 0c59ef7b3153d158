"""qkv_rope and its backward against a float64 form.

Tolerances. A stored result is rounded once: half a step of its type (eps / 2 of
the value). Before that the fp32 work on a row of d channels is off by a few
roundings of its terms (the norm's sum by at most d of them, in tree order far
fewer): 2^-19 of the row's largest value is allowed for all of it. dw sums R rows:
each row's term carries those roundings, and the sum's own are at most its depth
(under 2^10 adds in sequence here): 2^-13 of the sum of the terms' sizes.
"""
import pytest
import torch

from gated_block_sparse_gate_b200 import binding as gb
from gated_block_sparse_gate_b200.build import build
from tests.operator_refs import rope_forward

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    gb.load_library()


def _case(seed, B, N, Hq, Hkv, d, rot, dtype, axes=1, norm=True, packed=True, w_dtype=F32, max_pos=512):
    g = torch.Generator().manual_seed(seed)
    x = dict(cos=None, sin=None, eps=1e-6)
    x["cos"], x["sin"] = gb.rope_tables(max_pos, rot, 1000.0, "cpu")
    shape = (B, N) if axes == 1 else (B, N, axes)
    x["pos"] = torch.randint(0, max_pos, shape, generator=g).to(torch.int32)
    x["axes"] = [i % axes for i in range(rot // 2)]
    if packed:
        qkv = torch.randn(B, N, Hq + 2 * Hkv, d, generator=g).to(dtype)
        x["q"], x["k"], x["v"] = qkv.split((Hq, Hkv, Hkv), 2)
    else:
        x["q"], x["k"], x["v"] = (torch.randn(B, N, h, d, generator=g).to(dtype) for h in (Hq, Hkv, Hkv))
    x["wq"] = x["wk"] = None
    if norm:
        x["wq"], x["wk"] = (1 + 0.3 * torch.randn(2, d, generator=g)).to(w_dtype)
    x["dQ"], x["dK"], x["dV"] = (torch.randn(B, h, N, d, generator=g).to(dtype) for h in (Hq, Hkv, Hkv))
    return x


def _dev(x):
    return {n: t.to(DEV) if isinstance(t, torch.Tensor) else t for n, t in x.items()}


def _close(got, want, scale=None, slack=2.0 ** -19):
    half = torch.finfo(got.dtype).eps / 2
    got, want = got.double().cpu(), want.detach().double()
    scale = want.abs().amax(-1, keepdim=True) if scale is None else scale
    off = (got - want).abs() - half * want.abs() - slack * scale
    assert got.shape == want.shape and bool((off <= 0).all()), float(off.max())


def _check(x, interleaved=False, backward=True, out=None, grads=None):
    how = dict(axes=x["axes"], interleaved=interleaved, eps=x["eps"])
    dev = _dev(x)
    Q, K, V = gb.qkv_rope(*(dev[n] for n in ("q", "k", "v", "cos", "sin", "pos", "wq", "wk")), out=out, **how)
    leaves = {n: x[n].double().requires_grad_() for n in ("q", "k", "v", "wq", "wk") if x[n] is not None}
    ref = {h: rope_forward(leaves[h], leaves.get("w" + h), x["cos"], x["sin"], x["pos"], x["axes"], interleaved,
                           x["eps"]).transpose(1, 2) for h in "qk"}
    _close(Q, ref["q"])
    _close(K, ref["k"])
    assert torch.equal(V.cpu(), x["v"].transpose(1, 2))
    if not backward:
        return
    got = gb.qkv_rope_backward(*(dev[n] for n in ("q", "k", "cos", "sin", "pos", "dQ", "dK", "dV", "wq", "wk")),
                               grads=grads, **how)
    loss = (ref["q"] * x["dQ"].double()).sum() + (ref["k"] * x["dK"].double()).sum()
    names = [n for n in leaves if n != "v"]
    want = dict(zip(names, torch.autograd.grad(loss, [leaves[n] for n in names])))
    # the row's terms before h - xh mean(h xh) cancels: r w g
    for n, dz, t in (("q", x["dQ"], got[0]), ("k", x["dK"], got[1])):
        rows = leaves[n].detach()
        r = 1 / (rows.pow(2).mean(-1, keepdim=True) + x["eps"]).sqrt() if x["wq"] is not None else 1
        w = x["w" + n].double().abs().max() if x["wq"] is not None else 1
        size = r * w * dz.double().transpose(1, 2).abs().amax(-1, keepdim=True) * 2
        _close(t, want[n], size)
    assert torch.equal(got[2].cpu(), x["dV"].transpose(1, 2))
    for n, dz, t in (("q", x["dQ"], got[3]), ("k", x["dK"], got[4])):
        if x["wq"] is None:
            assert t is None
            continue
        rows = leaves[n].detach()
        xh = rows / (rows.pow(2).mean(-1, keepdim=True) + x["eps"]).sqrt()
        size = (xh.abs() * dz.double().transpose(1, 2).abs().amax(-1, keepdim=True)).sum((0, 1, 2))
        assert t.dtype == F32
        _close(t, want["w" + n], size, 2.0 ** -13)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,N,Hq,Hkv,d,rot", [
    (1, 1, 1, 1, 64, 64),       # one token of one head
    (64, 1, 32, 8, 128, 128),   # a decode step
    (2, 37, 5, 3, 128, 128),    # head counts that no lane split divides
    (3, 130, 6, 2, 64, 16),     # most channels not rotated
    (1, 517, 4, 2, 128, 56),    # half a rotated part that is no power of two
    (2, 65, 2, 1, 64, 0),       # a norm alone
])
@pytest.mark.parametrize("interleaved", [False, True])
def test_forward_and_backward(B, N, Hq, Hkv, d, rot, dtype, interleaved):
    _check(_case(B + N, B, N, Hq, Hkv, d, rot, dtype), interleaved)


@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("norm", [False, True])
def test_several_axes(axes, norm):
    _check(_case(axes, 2, 41, 8, 2, 128, 128, BF, axes=axes, norm=norm))


def test_many_tokens_go_round_the_grid():
    """More tokens than one turn of the backward's CTAs takes."""
    _check(_case(9, 2, 9001, 2, 1, 64, 64, F32, max_pos=9001))


def test_bf16_weights_and_separate_tensors():
    _check(_case(3, 2, 70, 4, 2, 128, 128, BF, packed=False, w_dtype=BF))


def test_strided_outputs_and_gradients():
    """Keys and values into their places of a contiguous cache, gradients into one packed tensor; what lies
    around them is left as it was."""
    B, N, Hq, Hkv, d, L, at = 2, 19, 4, 2, 128, 64, 23
    x = _case(5, B, N, Hq, Hkv, d, 128, BF)
    Kc, Vc = (torch.full((B, Hkv, L, d), 7.0, dtype=BF, device=DEV) for _ in range(2))
    Q = torch.empty(B, N, Hq, d, dtype=BF, device=DEV).transpose(1, 2)  # token-major again
    dqkv = torch.empty(B, N, Hq + 2 * Hkv, d, dtype=BF, device=DEV)
    _check(x, out=(Q, Kc[:, :, at:at + N], Vc[:, :, at:at + N]), grads=dqkv.split((Hq, Hkv, Hkv), 2))
    for c in (Kc, Vc):
        assert bool((c[:, :, :at] == 7).all()) and bool((c[:, :, at + N:] == 7).all())


def test_queries_and_keys_alone():
    x = _dev(_case(6, 1, 33, 4, 2, 64, 64, BF))
    a = (x["q"], x["k"], None, x["cos"], x["sin"], x["pos"])
    Q, K, V = gb.qkv_rope(*a)
    full = gb.qkv_rope(x["q"], x["k"], x["v"], x["cos"], x["sin"], x["pos"])
    assert V is None and torch.equal(Q, full[0]) and torch.equal(K, full[1])
    dq, dk, dv, dwq, dwk = gb.qkv_rope_backward(x["q"], x["k"], x["cos"], x["sin"], x["pos"], x["dQ"], x["dK"])
    assert dv is None and dwq is None and dwk is None and dq.shape == x["q"].shape


def test_zero_rows_and_large_values():
    """A row of zeros stays zero with a finite gradient; values whose squares fit fp32 keep their norm."""
    x = _case(7, 1, 8, 2, 2, 128, 128, F32)
    x["q"][0, 3] = 0
    x["q"][0, 4] *= 1e15
    _check(x, backward=False)
    dev = _dev(x)
    dq = gb.qkv_rope_backward(*(dev[n] for n in ("q", "k", "cos", "sin", "pos", "dQ", "dK", "dV", "wq", "wk")))[0]
    assert bool(torch.isfinite(dq).all())


def test_gradient_against_differences():
    """Central differences of the loss sum(z dz) computed from the kernel's own fp32 forward. With a step of
    2^-5 the loss changes by about 0.06 |gradient|; its fp32 terms are each off by 2^-23 of values of a few
    units and the curvature term is (step^2 / 6) f''' with f''' below 20: 0.01 in all."""
    x = _dev(_case(8, 1, 5, 2, 1, 64, 64, F32))
    how = dict(wq=x["wq"], wk=x["wk"], eps=x["eps"])
    dq = gb.qkv_rope_backward(x["q"], x["k"], x["cos"], x["sin"], x["pos"], x["dQ"], x["dK"], x["dV"], **how)[0]
    h = 2.0 ** -5
    for t, head, c in ((0, 0, 0), (1, 1, 33), (4, 0, 63), (2, 1, 31)):
        loss = []
        for sign in (1, -1):
            q = x["q"].clone()
            q[0, t, head, c] += sign * h
            Q = gb.qkv_rope(q, x["k"], x["v"], x["cos"], x["sin"], x["pos"], **how)[0]
            loss.append(float((Q.double() * x["dQ"].double()).sum()))
        assert abs((loss[0] - loss[1]) / (2 * h) - float(dq[0, t, head, c])) < 0.01


def test_weight_gradients_repeat_bit_for_bit():
    x = _dev(_case(10, 1, 5000, 8, 2, 128, 128, BF))
    a = [x[n] for n in ("q", "k", "cos", "sin", "pos", "dQ", "dK", "dV", "wq", "wk")]
    one, two = (gb.qkv_rope_backward(*a) for _ in range(2))
    assert all(torch.equal(p, q) for p, q in zip(one, two))


def test_bad_position_is_clamped_and_reported():
    x = _dev(_case(11, 1, 6, 2, 1, 64, 64, F32, max_pos=16))
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    a = [x[n] for n in ("q", "k", "v", "cos", "sin")]
    want = gb.qkv_rope(*a, x["pos"].clamp(0, 15), ws=ws)
    gb.check(ws)
    for bad, good in ((16, 15), (-1, 0), (2 ** 31 - 1, 15)):
        pos = x["pos"].clone()
        pos[0, 2] = bad
        fine = x["pos"].clone()
        fine[0, 2] = good
        want = gb.qkv_rope(*a, fine)
        got = gb.qkv_rope(*a, pos, ws=ws)
        with pytest.raises(gb.GbsError) as e:
            gb.check(ws)
        assert e.value.status == 1
        gb.clear_error(ws)
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_on_another_stream_and_in_a_graph():
    x = _dev(_case(12, 2, 50, 4, 2, 128, 128, BF))
    fwd = [x[n] for n in ("q", "k", "v", "cos", "sin", "pos", "wq", "wk")]
    bwd = [x[n] for n in ("q", "k", "cos", "sin", "pos", "dQ", "dK", "dV", "wq", "wk")]
    want = [*gb.qkv_rope(*fwd), *gb.qkv_rope_backward(*bwd)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [*gb.qkv_rope(*fwd, stream=side), *gb.qkv_rope_backward(*bwd, stream=side)]
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = [*gb.qkv_rope(*fwd), *gb.qkv_rope_backward(*bwd)]
    for t in kept:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(kept, want))


@pytest.mark.parametrize("B,N,Hq,Hkv", [(1, 1, 3, 1), (2, 37, 5, 3), (1, 700, 3, 1)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_no_eps(B, N, Hq, Hkv, dtype):
    """Lanes without a row of their own add nothing to the weights' gradients, eps = 0 included."""
    _check(dict(_case(31, B, N, Hq, Hkv, 64, 64, dtype), eps=0.0))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("axes,norm,values", [(1, True, True), (3, False, True), (2, True, False)])
def test_native_calls_give_what_the_bindings_own_path_gives(axes, norm, values, dtype, monkeypatch):
    """csrc/marshal.cpp's calls and the Python path behind them: the same results and refusals."""
    x = _dev(_case(41, 2, 37, 6, 2, 64, 48, dtype, axes=axes, norm=norm))
    if not values:
        x["v"] = x["dV"] = None
    ws = torch.zeros(gb.qkv_rope_workspace_bytes(x["q"], x["k"], 48), dtype=torch.uint8, device=DEV)
    fwd, bwd = ("q", "k", "v", "cos", "sin", "pos", "wq", "wk"), ("q", "k", "cos", "sin", "pos", "dQ", "dK", "dV", "wq", "wk")

    def results():
        out = []
        for kw in ({}, dict(ws=ws)):
            z = gb.qkv_rope(*(x[n] for n in fwd), axes=x["axes"], **kw)
            out += [*z, *gb.qkv_rope(*(x[n] for n in fwd), axes=tuple(x["axes"]), out=tuple(
                t if t is None else torch.empty_like(t) for t in z))]
            g = gb.qkv_rope_backward(*(x[n] for n in bwd), axes=x["axes"], **kw)
            out += [*g, *gb.qkv_rope_backward(*(x[n] for n in bwd), axes=x["axes"], grads=tuple(
                t if t is None else torch.empty_like(t) for t in g[:3]))]
        return out

    def refusals():
        text = []
        for change in (dict(cos=x["cos"][:, :8]), dict(pos=x["pos"].long()), dict(wq=x["cos"][0]), dict(q=x["q"][:1]),
                       dict(sin=None), dict(k=x["k"][:, :, :1].transpose(2, 3))):
            y = {**x, **change}
            with pytest.raises(gb.GbsError) as e:
                gb.qkv_rope(*(y[n] for n in fwd), axes=x["axes"])
            text.append(str(e.value))
        for kw in (dict(axes=[9] * 24), dict(axes=[0]), dict(axes=x["axes"], eps=-1.0),
                   dict(axes=x["axes"], ws=ws[:128]), dict(axes=x["axes"], interleaved=2)):
            if "interleaved" in kw:  # any truth value is taken
                assert gb.qkv_rope(*(x[n] for n in fwd), **kw) is not None
                continue
            with pytest.raises(gb.GbsError) as e:
                gb.qkv_rope(*(x[n] for n in fwd), **kw)
            text.append(str(e.value))
        return text

    native = results(), refusals()
    monkeypatch.setattr(gb, "_native", gb._NoCalls)
    own = results(), refusals()
    assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(native[0], own[0]))
    assert native[1] == own[1]


def test_plain_calls_are_native(monkeypatch):
    """Plain arguments do not reach the Python checks."""
    x = _dev(_case(43, 1, 5, 4, 2, 64, 64, BF))
    monkeypatch.setattr(gb, "_rope_call", None)
    Q, K, V = gb.qkv_rope(*(x[n] for n in ("q", "k", "v", "cos", "sin", "pos", "wq", "wk")))
    gb.qkv_rope_backward(*(x[n] for n in ("q", "k", "cos", "sin", "pos", "dQ", "dK", "dV", "wq", "wk")))
    packed = torch.zeros(1, 5, 8, 64, dtype=BF, device=DEV)
    gb.qkv_rope_backward(*(x[n] for n in ("q", "k", "cos", "sin", "pos", "dQ", "dK", "dV", "wq", "wk")),
                         grads=packed.split((4, 2, 2), 2))
    monkeypatch.undo()
    for grads in ((packed[:, :, :1].expand(1, 5, 4, 64), None, None), (packed.as_strided((1, 5, 4, 64), (2560, 256, 32, 1)),
                                                                      None, None)):
        with pytest.raises(gb.GbsError, match="share memory"):
            gb.qkv_rope_backward(*(x[n] for n in ("q", "k", "cos", "sin", "pos", "dQ", "dK")), None, x["wq"], x["wk"],
                                 grads=(grads[0], packed[:, :, 4:6], None))
    assert Q.shape == (1, 4, 5, 64)
