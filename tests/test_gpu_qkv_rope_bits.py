"""qkv_rope of fp32 rows keeps the bits of fp32.

A normed channel is x r w with r = 1 / sqrt(mean x^2 + eps): three roundings to nearest, as many as x / sqrt(..) * w
takes. Over 2^15 rows the two have the same mean square error but for what chance does, well below 1 % (2^22 channels,
and 2^15 values of r); 2 % are allowed. (A square root of 2^-22 instead shows as 5 %.)
"""
import pytest
import torch

from gated_block_sparse_gate_b200 import binding as gb
from gated_block_sparse_gate_b200.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    gb.load_library()


@pytest.mark.parametrize("d", [64, 128])
def test_normed_rows_round_as_often_as_the_formula(d):
    g = torch.Generator().manual_seed(d)
    x = torch.randn(1, 4096, 8, d, generator=g)
    w = 1 + 0.3 * torch.randn(d, generator=g)
    cos, sin = gb.rope_tables(1, 0, device=DEV)
    pos = torch.zeros(1, 4096, dtype=torch.int32, device=DEV)
    Q, K, _ = gb.qkv_rope(x.to(DEV), x.to(DEV), None, cos, sin, pos, w.to(DEV), w.to(DEV))
    exact = x.double() / (x.double().pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
    plain = x / (x.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w
    off = lambda y: float(((y.double() - exact) / exact).pow(2).mean().sqrt())  # noqa: E731
    for y in (Q, K):
        assert off(y.cpu().transpose(1, 2)) <= 1.02 * off(plain)


def _dq(x, w, dz, eps=1e-6):
    """dx of the norm alone in x's type."""
    r = 1 / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    h, xh = dz * w, x * r
    return r * (h - xh * (h * xh).mean(-1, keepdim=True))


@pytest.mark.parametrize("d", [64, 128])
def test_gradients_round_no_more_than_the_formula(d):
    g = torch.Generator().manual_seed(d)
    x, dz = torch.randn(2, 1, 4096, 8, d, generator=g)
    w = 1 + 0.3 * torch.randn(d, generator=g)
    cos, sin = gb.rope_tables(1, 0, device=DEV)
    pos = torch.zeros(1, 4096, dtype=torch.int32, device=DEV)
    to = [t.to(DEV) for t in (x, dz.transpose(1, 2), w)]
    dq = gb.qkv_rope_backward(to[0], to[0], cos, sin, pos, to[1], to[1], None, to[2], to[2])[0]
    exact = _dq(x.double(), w.double(), dz.double())
    off = lambda y: float((y.double() - exact).norm())  # noqa: E731
    assert off(dq.cpu()) <= 1.02 * off(_dq(x, w, dz))
