"""The 4-bit cache's calls on batches and lengths that the tensor maps of the other decode could not address."""
import math

import pytest
import torch

from gated_block_sparse_gate_b200 import binding as gb
from gated_block_sparse_gate_b200.build import build
from tests.test_gpu_kv4 import DEV, _check, _decode_case

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    gb.load_library()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_large_batch_gives_what_its_halves_give(dtype):
    """B * Hq * L = 2^31; sequences share a pool of few pages."""
    B, Hq, Hkv, d, L, pages = 128, 64, 8, 64, 262144, 40
    g = torch.Generator(device=DEV).manual_seed(1)
    cache = gb.kv4_cache(B, Hkv, d, num_pages=pages, device=DEV)
    K, V = (torch.randn(pages, Hkv, 64, d, generator=g, device=DEV).to(dtype) for _ in "kv")
    gb.kv4_append(K, V, cache, torch.zeros(pages, dtype=torch.int32, device=DEV),
                  block_table=torch.arange(pages, dtype=torch.int32, device=DEV)[:, None].contiguous())
    table = torch.randint(0, pages, (B, L // 64), generator=g, device=DEV, dtype=torch.int32)
    lens = torch.randint(1, L + 1, (B,), generator=g, device=DEV).to(torch.int32)
    lens[3], lens[70] = L, 0
    q = torch.randn(B, Hq, d, generator=g, device=DEV).to(dtype)
    S = math.sqrt(2) * torch.randn(B, Hkv, L // 64, generator=g, device=DEV)
    call = lambda s: gb.kv4_decode(q[s], cache, S[s], L, topk=8, num_splits=1, block_table=table[s],  # noqa: E731
                                   seq_lens=lens[s], group_shared=True)
    whole, parts = call(slice(None)), [call(slice(0, 64)), call(slice(64, 128))]
    assert all(torch.equal(w, torch.cat(p)) for w, p in zip(whole, zip(*parts)))
    # rows of a block table that allows them are read where they are
    back = gb.kv4_read(cache, lens - 1, 1, block_table=table, count=(lens > 0).to(torch.int32), dtype=F32)
    rows = gb.kv4_read(cache, torch.zeros(pages, dtype=torch.int32, device=DEV), 64, dtype=F32,
                       block_table=torch.arange(pages, dtype=torch.int32, device=DEV)[:, None].contiguous())
    at = (lens - 1).clamp(min=0).long()
    page = table[torch.arange(B, device=DEV), at // 64].long()
    for got, r in zip(back, rows):
        want = torch.where((lens > 0)[:, None, None], r[page, :, at % 64], 0)
        assert torch.equal(got[:, :, 0], want)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_block_table_of_the_longest_rows(dtype):
    """A row of 2^31 - 64 positions, of which a sequence fills a part."""
    L = 2 ** 31 - 64
    x = _decode_case(2, 1, 2, 1, 64, 70000, [70000], True, dtype)
    x["S"] = torch.cat([x["S"], torch.full((1, 1, L // 64 - x["S"].shape[2]), 99.0)], 2)
    x["table"] = torch.cat([x["table"], torch.full((1, L // 64 - x["table"].shape[1]), -1, dtype=torch.int32)], 1)
    _check(x, L, 12, True)
