"""A wait of the 4-bit decode that runs out: its rows are NaN, in one CTA and in several, and the error word tells.

The debug build takes a call's first waits for expired where its error word already holds GBS_ERR_TIMEOUT; the
copies themselves arrive, so nothing hangs.
"""
import pytest
import torch

from gated_block_sparse_gate_b200 import binding as gb
from gated_block_sparse_gate_b200.build import build
from tests.test_gpu_kv4 import DEV, _decode_case, _run

pytestmark = pytest.mark.gpu
TIMEOUT = 4


@pytest.fixture
def debug_library():
    saved = gb._lib
    gb._lib = None
    try:
        yield gb.load_library(build(debug=True))
    finally:
        gb._lib = saved


@pytest.mark.parametrize("splits", [1, 2, 5])
@pytest.mark.parametrize("d,shared", [(128, False), (128, True), (64, False), (64, True)])
def test_a_wait_that_runs_out_shows_in_the_results(debug_library, d, shared, splits):
    x = _decode_case(splits, 2, 8, 2, d, 1500, [1500, 40], shared)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    want = _run(x, 1500, 12, shared, splits=splits, ws=ws)
    gb.check(ws)
    ws[0] = TIMEOUT
    O, LSE = _run(x, 1500, 12, shared, splits=splits, ws=ws)
    assert bool(torch.isnan(O).all()) and bool(torch.isnan(LSE).all())
    with pytest.raises(gb.GbsError) as e:
        gb.check(ws)
    assert e.value.status == TIMEOUT
    gb.clear_error(ws)
    assert all(torch.equal(a, b) for a, b in zip(_run(x, 1500, 12, shared, splits=splits, ws=ws), want))
    gb.check(ws)
