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
