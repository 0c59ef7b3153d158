"""Scores at the ends of fp32's range, as masks make them: the decode over a 4-bit cache gives the definition's result.

Tolerances are those of tests/test_gpu_kv4.py (_check).
"""
import pytest
import torch

from gated_block_sparse_gate_b200 import binding as gb
from gated_block_sparse_gate_b200.build import build
from tests.test_gpu_kv4 import _check, _decode_case, _run

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
LOWEST = torch.finfo(F32).min


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    gb.load_library()


@pytest.mark.parametrize("splits", [1, 3, 0])
@pytest.mark.parametrize("dtype,shared", [(BF, False), (BF, True), (F32, False)])
@pytest.mark.parametrize("masked", [[0], [0, 1, 2, 3], [0, 5, 9], [4, 12]])
def test_blocks_masked_by_the_lowest_score(masked, dtype, shared, splits):
    """All blocks are kept, the masked ones with a weight of 0, wherever they come first."""
    x = _decode_case(sum(masked), 2, 8, 2, 128, 900, [900, 870], shared, dtype)
    x["S"][..., masked] = LOWEST
    _check(x, 900, 20, shared, splits=splits)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_masked_blocks_in_the_longest_rows(dtype):
    """Rows that are selected from before the decode: five blocks that are not masked, fifteen that are."""
    x = _decode_case(3, 1, 2, 1, 64, 530000, None, True, dtype, paged=False)
    x["S"][..., [i for i in range(x["S"].shape[-1]) if i % 1700 != 1]] = LOWEST
    _check(x, 530000, 20, True)


# blocks a row, budget: rows that a warp, one warp after the others, all warps, and a kernel before select from
ROWS = [(900, 6), (900, 20), (40000, 32), (40000, 200), (530000, 32)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("L,k", ROWS)
@pytest.mark.parametrize("shift", [2.0 ** 20, -2.0 ** 20])
def test_gates_do_not_depend_on_the_scores_level(shift, L, k, dtype):
    """Scores in steps of 1 / 4, which fp32 holds beside 2^20: the log gates are those without it."""
    x = _decode_case(k, 1, 2, 1, 64, L, None, True, dtype, paged=False)
    x["S"] = (4 * x["S"]).round() / 4 + shift
    _check(x, L, k, True)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("L,k", ROWS)
@pytest.mark.parametrize("level", [1e8, LOWEST, -LOWEST])
def test_equal_scores_of_any_size(level, L, k, dtype):
    x = _decode_case(k, 1, 2, 1, 64, L, None, True, dtype, paged=False)
    x["S"].zero_()
    want = _run(x, L, k, True)
    x["S"].fill_(level)
    assert all(torch.equal(a, b) for a, b in zip(_run(x, L, k, True), want))


@pytest.mark.parametrize("L", [1000, 20000, 140000, 530000])
@pytest.mark.parametrize("k", [0, 20, 96, 256])
def test_nan_scores_keep_every_index_in_range(L, k):
    """Scores have to be finite; with NaNs among them (the one of all bits set too) the debug build finds every kept
    block inside its row all the same. It clamps a bad index before it is used."""
    saved, gb._lib = gb._lib, None
    try:
        gb.load_library(build(debug=True))
        for dtype in (BF, F32):
            for shared in (False, True):
                x = _decode_case(11, 2, 4, 2, 64, L, [L, L // 3], shared, dtype, paged=False)
                bits = x["S"].view(torch.int32)
                bits[0, :1] = -1
                bits[0, 1, ::3] = 0x7fffffff
                bits[1, 0, 5::7] = -1
                p = gb.make_params(2, 4, 2, L, 64, 64, k, "sparse", dtype)
                ws = torch.zeros(gb.kv4_workspace_bytes(p), dtype=torch.uint8, device="cuda:0")
                _run(x, L, k, shared, ws=ws)
                gb.check(ws)
                _run(x, L, k, shared, tau=1e-3, ws=ws)
                gb.check(ws)
    finally:
        gb._lib = saved
