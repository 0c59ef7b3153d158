"""The bf16 decode over a 4-bit cache holds its weights, products and sums in as many bits as fp32 does.

Logits are kept small (a scale of 1 / 256), so that their own rounding leaves room to see the rest. Tolerances: a
logit and the exponential of it are off by e = d 2^-23 scale sum |q k| + 2^-18, twice in numerator and sum. p and s p as
two fp16 terms leave 2^-21, and each of at most 32 products added to a sum of these tests may cut a step of 2^-23 of it:
2^-18 + 2^-21 of sum s p n <= sum p |v| + sum p |m|, |m| <= 6. In all (2 e + 2^-17) sum p |v| + 6 2^-17, and half a step
of bf16. (With one fp16 term for each of the two, 2^-12 of a key's s n would be left: up to 24 times that.)
"""
import numpy as np
import pytest
import torch

from gated_block_sparse_gate_b200 import binding as gb
from gated_block_sparse_gate_b200.build import build
from tests.test_gpu_kv4 import _decode_case, _reference, _run, _within

pytestmark = pytest.mark.gpu
SCALE = 1 / 256


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    gb.load_library()


@pytest.mark.parametrize("L", [2, 70, 200])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_weights_and_products_keep_fp32s_bits(d, shared, L):
    x = _decode_case(100 + L, 16, 8, 2, d, L, None, shared)
    O, LSE = _run(x, L, 3, shared, scale=SCALE)
    Or, Lr, A, Z = _reference(x, L, 3, shared, None, SCALE)
    e = d * 2.0 ** -23 * Z + 2.0 ** -18
    _within(O, Or, (2 * e[..., None] + 2.0 ** -17) * A + 6 * 2.0 ** -17)
    assert (np.abs(LSE.double().cpu().numpy() - Lr) <= e + 2.0 ** -23 * np.abs(Lr)).all()


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_low_codes_beside_high_ones(d, shared):
    """A low nibble of 0, at one key in 64 of 1, beside any high one. 40 blocks are 20 half blocks to a warp, with up to
    16 products of both terms to a sum for each: 320 steps of 2^-23 of a sum of values that are not negative, so less
    than 2^-14 of the result."""
    L = 64 * 40
    x = _decode_case(7, 4, 8, 2, d, L, None, shared)
    g = torch.Generator().manual_seed(1)
    for i in (0, 2):
        x["cache"][i] = x["cache"][i] & 0xf0 | (torch.rand(x["cache"][i].shape, generator=g) < 1 / 64).to(torch.uint8)
        x["cache"][i + 1][..., 1] = 0
    O, _ = _run(x, L, 40, shared, scale=SCALE)
    Or, _, A, Z = _reference(x, L, 40, shared, None, SCALE)
    e = d * 2.0 ** -23 * Z + 2.0 ** -18
    _within(O, Or, (2 * e[..., None] + 2.0 ** -14) * A)
