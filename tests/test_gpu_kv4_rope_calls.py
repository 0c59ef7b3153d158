"""Calls of the norm, rotation and 4-bit cache operators that a program makes beside the plain ones: outputs of any
strides, tensors of more than 2^31 elements, several threads at once."""
import threading

import pytest
import torch

from gated_block_sparse_gate_b200 import binding as gb
from gated_block_sparse_gate_b200.build import build
from tests.test_gpu_kv4 import DEV, _decode_case, _run

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    gb.load_library()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_read_into_tensors_of_any_strides(d, dtype):
    """Token-major keys, values inside a larger tensor; what lies between is left as it was."""
    g = torch.Generator().manual_seed(d)
    B, Hkv, T = 3, 2, 70
    K, V = (torch.randn(B, Hkv, T, d, generator=g).to(dtype).to(DEV) for _ in "kv")
    start = torch.tensor([0, 9, 30], dtype=torch.int32, device=DEV)
    count = torch.tensor([70, 0, 33], dtype=torch.int32, device=DEV)
    cache = gb.kv4_cache(B, Hkv, d, L=100, device=DEV)
    gb.kv4_append(K, V, cache, start)
    want = gb.kv4_read(cache, start, T, count=count, dtype=dtype)
    tokens = torch.full((B, T, Hkv, d), 7.0, dtype=dtype, device=DEV)
    wide = torch.full((B, Hkv, T + 2, 2 * d), 7.0, dtype=dtype, device=DEV)
    out = tokens.transpose(1, 2), wide[:, :, 1:-1, d:]
    got = gb.kv4_read(cache, start, T, count=count, dtype=dtype, out=out)
    assert got[0] is out[0] and got[1] is out[1]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    wide[:, :, 1:-1, d:] = 7.0
    assert bool((wide == 7.0).all())
    with pytest.raises(gb.GbsError, match="share memory"):
        gb.kv4_read(cache, start, T, dtype=dtype, out=(out[0], out[0]))


def test_projections_of_more_than_2_to_the_31_elements():
    """The tokens at both ends give the bits that they give alone, forward and backward."""
    N, Hq, d, n = 540000, 32, 128, 40
    assert N * Hq * d > 2 ** 31
    g = torch.Generator(device=DEV).manual_seed(1)
    q = torch.randn(1, N // 100, Hq, d, generator=g, device=DEV).to(BF).repeat(1, 100, 1, 1)
    k = torch.randn(1, N, 1, d, generator=g, device=DEV).to(BF)
    q[:, -n:] = torch.randn(1, n, Hq, d, generator=g, device=DEV).to(BF)
    cos, sin = gb.rope_tables(N, d, device=DEV)
    pos = torch.arange(N, dtype=torch.int32, device=DEV)[None]
    w = 1 + 0.1 * torch.randn(2, d, generator=g, device=DEV)
    Q, K, V = gb.qkv_rope(q, k, k, cos, sin, pos, *w)
    for at in (slice(0, n), slice(N - n, N)):
        alone = gb.qkv_rope(q[:, at], k[:, at], k[:, at], cos, sin, pos[:, at].contiguous(), *w)
        assert all(torch.equal(a[:, :, at], b) for a, b in zip((Q, K, V), alone))
    dq, dk, dv = gb.qkv_rope_backward(q, k, cos, sin, pos, Q, K, V, *w)[:3]
    for at in (slice(0, n), slice(N - n, N)):
        alone = gb.qkv_rope_backward(q[:, at], k[:, at], cos, sin, pos[:, at].contiguous(), Q[:, :, at], K[:, :, at],
                                     V[:, :, at], *w)
        assert all(torch.equal(a[:, at], b) for a, b in zip((dq, dk, dv), alone))


def test_several_threads_at_once():
    """Each on a stream of its own, with its own workspaces; a refused call of one leaves the others' messages alone."""
    x = [_decode_case(40 + i, 2, 4, 2, 128, 900, [900, 80], bool(i % 2), BF if i < 2 else F32) for i in range(4)]
    want = [_run(x[i], 900, 8, bool(i % 2)) for i in range(4)]
    on = [{n: t.to(DEV) if isinstance(t, torch.Tensor) else t for n, t in y.items()} for y in x]
    caches = [[t.to(DEV) for t in y["cache"]] for y in x]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                for turn in range(100):
                    got = gb.kv4_decode(on[i]["q"], caches[i], on[i]["S"], 900, topk=8, block_table=on[i]["table"],
                                        seq_lens=on[i]["lens"], group_shared=bool(i % 2))
                    try:
                        gb.kv4_decode(on[i]["q"], caches[i], on[i]["S"], 900, topk=300 + i, seq_lens=on[i]["lens"],
                                      block_table=on[i]["table"], group_shared=bool(i % 2))
                    except gb.GbsError as e:
                        assert f"topk {300 + i}" in str(e)
                    else:
                        raise AssertionError("not refused")
                    side.synchronize()
                    assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
        except BaseException as e:  # noqa: BLE001
            wrong.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
