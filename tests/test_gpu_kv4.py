"""The 4-bit cache: rows written and read back, and the decode over it, against float64 forms.

Tolerances. What is stored is defined to the bit, so rows read back equal the
float64 form's values rounded once: half a step of the output's type plus one of
fp32 for the value itself.
Decode, for one query over the kept keys (p the weights, v the values):
  LSE  a logit sums d products in fp32 in any order: off by at most d 2^-23 of
       scale sum |q k| (a tensor core may cut instead of round: one step, not half),
       and the sums of exponentials and the logarithm by 2^-18 in all.
  O    the weights inherit the logits' error e (twice, in numerator and sum):
       2 e sum p |v|; sums of fp32 as above with at most 2^-16 of the same. With bf16
       queries weights p are rounded to fp16 (2^-11 of |v|), then products s p (2^-11 of
       s n <= |v| + |m|, with |m| <= 6 spread in the caches below); a product below
       fp16's normal range is cut to steps of 2^-24, off by 2^-25 times a code of at most
       15, against weights of which the largest is at least 2^10 over twice the largest
       scale, if that is above 1: 2^-30 (1 + spread) a key.
       In all (2 e + 2^-16) sum p |v|, with bf16 queries 2^-10 sum p |v| + 2^-11 6 spread
       + 2^-30 (1 + spread) keys more, and half a step of the output's type.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from gated_block_sparse_gate_b200 import binding as gb
from gated_block_sparse_gate_b200.build import build
from tests.operator_refs import kv4_quantised, kv4_values

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    gb.load_library()


def _within(got, want, slack=0.0):
    half = torch.finfo(got.dtype).eps / 2 + 2.0 ** -24
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    off = np.abs(got - want) - half * np.abs(want) - slack
    assert not (off > 0).any(), np.nanmax(off)


def _table(g, B, nb, extra=3):
    return torch.randperm(B * nb + extra, generator=g)[:B * nb].view(B, nb).to(torch.int32)


# ------------------------------------------------------------------ append, read


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("B,Hkv,T,L", [(1, 1, 1, 64), (3, 2, 130, 260), (64, 8, 1, 300), (2, 3, 77, 100)])
def test_rows_written_are_the_definitions(B, Hkv, T, L, paged, d, dtype):
    g = torch.Generator().manual_seed(T + L + d)
    x = [(torch.randn(B, Hkv, T, d, generator=g) * torch.exp(torch.randn(d, generator=g))).to(dtype) for _ in "kv"]
    nb = -(-L // 64)
    start = torch.randint(0, L - T + 1, (B,), generator=g).to(torch.int32)
    table = _table(g, B, nb).to(DEV) if paged else None
    cache = gb.kv4_cache(B, Hkv, d, **(dict(num_pages=B * nb + 3) if paged else dict(L=L)), device=DEV)
    for t in cache:
        t.fill_(3)
    before = [t.clone() for t in cache]
    gb.kv4_append(x[0].to(DEV), x[1].to(DEV), cache, start.to(DEV), block_table=table)
    back = gb.kv4_read(cache, start.to(DEV), T, block_table=table, dtype=dtype)
    for got, t in zip(back, x):
        _within(got, kv4_quantised(t))
    # rows that no token went to keep their contents
    rows = torch.zeros(cache[0].shape[:3], dtype=torch.bool)
    for b in range(B):
        for t in range(T):
            pos = int(start[b]) + t
            if paged:
                rows[int(table[b, pos // 64]), :, pos % 64] = True
            else:
                rows[b, :, pos] = True
    for t, old in zip(cache, before):
        assert torch.equal(t.cpu()[~rows], old.cpu()[~rows])


def test_codes_next_to_a_border_and_ties():
    """Values half way between two codes (ties go to the even one) and the fp32 neighbours of them."""
    m, s = -2.0, 0.25
    edge = m + s * (np.arange(15) + 0.5)
    near = np.concatenate([edge, np.nextafter(edge.astype(np.float32), np.float32(9)),
                           np.nextafter(edge.astype(np.float32), np.float32(-9))]).astype(np.float32)
    x = torch.zeros(1, 1, 2, 64)
    x[..., 0::32], x[..., 1::32] = m, m + 15 * s
    x[0, 0, 0, 2:32] = torch.from_numpy(near[:30])
    x[0, 0, 0, 34:49] = torch.from_numpy(near[30:])
    x[0, 0, 1] = torch.linspace(-1, 1, 64) ** 3
    cache = gb.kv4_cache(1, 1, 64, L=64, device=DEV)
    start = torch.zeros(1, dtype=torch.int32, device=DEV)
    gb.kv4_append(x.to(DEV), x.to(DEV), cache, start)
    assert np.array_equal(kv4_values(cache[0], cache[1])[0, 0, :2], kv4_quantised(x)[0, 0])


def test_random_codes_equal_the_64_bit_rounding():
    g = torch.Generator().manual_seed(0)
    for dtype in (BF, F32):
        x = (torch.randn(2, 4, 4096, 128, generator=g) * 4 ** torch.randn(2, 4, 4096, 1, generator=g)).to(dtype)
        cache = gb.kv4_cache(2, 4, 128, L=4096, device=DEV)
        gb.kv4_append(x.to(DEV), x.to(DEV), cache, torch.zeros(2, dtype=torch.int32, device=DEV))
        assert np.array_equal(kv4_values(cache[2], cache[3]), kv4_quantised(x))


def test_extreme_values():
    """Equal values, zeros, tiny and huge values, infinities (limited) and a NaN (its group alone)."""
    x = torch.zeros(1, 1, 8, 64)
    x[0, 0, 0] = 1.7
    x[0, 0, 2] = torch.linspace(0, 1e-7, 64)
    # in 64 bits: the difference of the ends, 6e38, is beyond fp32's 3.4e38 and would make the row NaN
    x[0, 0, 3] = torch.linspace(-3e38, 3e38, 64, dtype=torch.float64)
    x[0, 0, 4] = torch.linspace(-1, 1, 64)
    x[0, 0, 4, 5], x[0, 0, 4, 40] = math.inf, -math.inf
    x[0, 0, 5] = torch.linspace(-1, 1, 64)
    x[0, 0, 5, 33] = math.nan
    x[0, 0, 6] = 70000.0
    x[0, 0, 7] = torch.linspace(1000, 1000.01, 64)
    cache = gb.kv4_cache(1, 1, 64, L=64, device=DEV)
    gb.kv4_append(x.to(DEV), x.to(DEV), cache, torch.zeros(1, dtype=torch.int32, device=DEV))
    K, V = gb.kv4_read(cache, torch.zeros(1, dtype=torch.int32, device=DEV), 8, dtype=F32)
    want = kv4_quantised(x)
    _within(K, want)
    assert np.isnan(want[0, 0, 5]).sum() == 32 and np.isfinite(want[0, 0, 3]).all()
    assert torch.equal(torch.nan_to_num(K), torch.nan_to_num(V))


def test_ragged_counts_and_strides():
    """Only the first count[b] tokens are written; token-major (strided) keys and a shared value head."""
    g = torch.Generator().manual_seed(4)
    B, Hkv, T, d = 4, 3, 50, 64
    K = torch.randn(B, T, Hkv, d, generator=g).to(BF).to(DEV).transpose(1, 2)
    V = torch.randn(B, 1, T, d, generator=g).to(BF).to(DEV).expand(B, Hkv, T, d)
    count = torch.tensor([0, 50, 1, 17], dtype=torch.int32, device=DEV)
    start = torch.tensor([0, 14, 63, 31], dtype=torch.int32, device=DEV)
    cache = gb.kv4_cache(B, Hkv, d, L=128, device=DEV)
    gb.kv4_append(K, V, cache, start, count=count)
    K1, V1 = gb.kv4_read(cache, start, T, count=count, dtype=F32)
    K0, V0 = gb.kv4_read(cache, start, T, dtype=F32)
    live = (torch.arange(T, device=DEV) < count[:, None])[:, None, :, None]
    want = [np.where(live.cpu().numpy(), kv4_quantised(t), 0) for t in (K, V)]
    for got, w in ((K1, want[0]), (V1, want[1]), (K0, want[0]), (V0, want[1])):
        _within(got, w)


def _reported(ws):
    """Whether a bad argument was recorded in ``ws``, which is cleared."""
    try:
        gb.check(ws)
    except gb.GbsError as e:
        assert e.status == 1
        gb.clear_error(ws)
        return True
    return False


def test_bad_positions_pages_and_counts_are_left_out_and_reported():
    B, Hkv, T, d = 2, 1, 4, 64
    x = torch.ones(B, Hkv, T, d, dtype=BF, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    good = dict(start=[0, 60], count=[4, 4], table=[[0, 1], [2, 3]])
    for name, value in (("start", [0, 126]), ("start", [-1, 60]), ("start", [0, 2 ** 31 - 1]),
                        ("start", [-2 ** 31, 0]), ("count", [5, 4]), ("count", [4, -1]),
                        ("table", [[0, 1], [4, 3]]), ("table", [[0, 1], [-1, 3]]),
                        ("table", [[0, 1], [2, -1]])):  # the last: positions 60 .. 63, the entry is not read
        a = {k: torch.tensor(v, dtype=torch.int32, device=DEV) for k, v in {**good, name: value}.items()}
        cache = gb.kv4_cache(B, Hkv, d, num_pages=4, device=DEV)
        gb.kv4_append(x, x, cache, a["start"], block_table=a["table"], count=a["count"], ws=ws)
        reported = value != [[0, 1], [2, -1]]
        assert _reported(ws) == reported
        K, _ = gb.kv4_read(cache, a["start"], T, block_table=a["table"], count=a["count"], ws=ws)
        assert _reported(ws) == reported
        for b in range(B):
            for t in range(T):
                pos, n = int(a["start"][b]) + t, min(max(int(a["count"][b]), 0), T)
                fine = 0 <= pos < 128 and t < n and 0 <= int(a["table"][b, pos // 64]) < 4
                assert float(K[b, 0, t].float().min()) == float(K[b, 0, t].float().max()) == (1.0 if fine else 0.0)


# ------------------------------------------------------------------ decode


def _decode_case(seed, B, Hq, Hkv, d, L, lens, shared, dtype=BF, paged=True, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    nb = -(-L // 64)
    shape = (B * nb + 3, Hkv, 64) if paged else (B, Hkv, nb * 64)
    x = dict(table=_table(g, B, nb) if paged else None, lens=None if lens is None else
             torch.tensor(lens, dtype=torch.int32))
    cache = []
    for _ in "kv":
        cache += [torch.randint(0, 256, (*shape, d // 2), generator=g, dtype=torch.uint8),
                  torch.stack((0.2 + 0.1 * torch.rand(*shape, d // 32, generator=g),
                               -2 + torch.randn(*shape, d // 32, generator=g)), -1).mul(spread).half()]
    x["cache"] = cache
    x["q"] = torch.randn(B, Hq, d, generator=g).to(dtype)
    x["S"] = torch.randn(B, Hkv if shared else Hq, nb, generator=g) * math.sqrt(2)
    return x


def _reference(x, L, k, shared, tau, scale=None):
    """(O, LSE, sum p |v|, scale max sum |q k|) in float64 through the oracle's decode."""
    B, Hq, d = x["q"].shape
    Hkv = x["cache"][0].shape[1]
    kv = [kv4_values(*x["cache"][i:i + 2]) for i in (0, 2)]
    if x["table"] is None:  # a contiguous cache as pages
        nb = kv[0].shape[2] // 64
        kv = [t.reshape(B, Hkv, nb, 64, d).transpose(0, 2, 1, 3, 4).reshape(B * nb, Hkv, 64, d) for t in kv]
        table = np.arange(B * nb).reshape(B, nb)
    else:
        table = x["table"].numpy()
    lens = np.full(B, L) if x["lens"] is None else x["lens"].numpy()
    q = x["q"].double().numpy()
    live = np.nonzero(lens > 0)[0]
    O, A = np.zeros((B, Hq, d)), np.zeros((B, Hq, d))
    LSE, Z = np.full((B, Hq), -np.inf), np.zeros((B, Hq))
    mode = oracle.SPARSE if tau is None else oracle.THRESHOLD
    run = lambda V: oracle.gated_decode_paged(  # noqa: E731
        q[live], kv[0], V, table[live], lens[live], x["S"].numpy()[live], 64, k, group_shared=shared, mode=mode,
        tau=tau, **({} if scale is None else dict(scale=scale)))
    O[live], LSE[live] = run(kv[1])
    A[live] = run(np.abs(kv[1]))[0]
    with np.errstate(invalid="ignore"):
        for b in live:
            for h in range(Hq):
                rows = kv[0][table[b, :-(-lens[b] // 64)], h * Hkv // Hq].reshape(-1, d)[:lens[b]]
                Z[b, h] = np.abs(rows).dot(np.abs(q[b, h])).max() * (d ** -0.5 if scale is None else scale)
    return O, LSE, A, Z


def _run(x, L, k, shared, tau=None, splits=0, scale=0.0, **kw):
    on = {n: t.to(DEV) if isinstance(t, torch.Tensor) else t for n, t in x.items()}
    return gb.kv4_decode(on["q"], [t.to(DEV) for t in x["cache"]], on["S"], L, topk=k, block_table=on["table"],
                         seq_lens=on["lens"], group_shared=shared, tau=tau, num_splits=splits, scale=scale, **kw)


def _check(x, L, k, shared, tau=None, splits=0, scale=0.0, spread=1.0):
    O, LSE = _run(x, L, k, shared, tau, splits, scale)
    Or, Lr, A, Z = _reference(x, L, k, shared, tau, scale or None)
    d = x["q"].shape[2]
    e = d * 2.0 ** -23 * Z + 2.0 ** -18
    LSE = LSE.double().cpu().numpy()
    live = np.isfinite(Lr)
    assert np.array_equal(np.isfinite(LSE), live) and bool((LSE[~live] == -np.inf).all())
    off = np.abs(LSE - Lr)[live] - e[live] - 2.0 ** -23 * np.abs(Lr[live])
    assert (off <= 0).all(), off.max()
    slack = (2 * e[..., None] + 2.0 ** -16) * A
    if x["q"].dtype == BF:
        slack += 2.0 ** -10 * A + 2.0 ** -11 * 6 * spread + 2.0 ** -30 * (1 + spread) * min(L, 64 * (k + 1))
    _within(O, Or, slack)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_decode(d, paged, shared, dtype):
    x = _decode_case(d, 4, 8, 2, d, 2133, [2133, 64, 1000, 65], shared, dtype, paged)
    _check(x, 2133, 8, shared)


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 63, 64, 65, 129, 1000])
@pytest.mark.parametrize("shared", [False, True])
def test_decode_lengths(L, shared):
    _check(_decode_case(L, 2, 4, 2, 128, L, None, shared, paged=False), L, 4, shared)


@pytest.mark.parametrize("splits", [1, 2, 3, 7, 32])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_splits(splits, dtype):
    x = _decode_case(splits, 2, 4, 1, 64, 3000, [3000, 700], False, dtype)
    _check(x, 3000, 20, False, splits=splits)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (12, 1), (16, 2), (10, 2), (40, 2), (4, 4)])
@pytest.mark.parametrize("shared", [False, True])
def test_decode_group_sizes(Hq, Hkv, shared):
    _check(_decode_case(Hq, 2, Hq, Hkv, 128, 900, [900, 333], shared), 900, 5, shared)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("k", [0, 1, 256])
def test_decode_budgets(k, dtype):
    _check(_decode_case(k, 2, 4, 2, 64, 1500, [1500, 20], True, dtype), 1500, k, True)


@pytest.mark.parametrize("shared", [False, True])
def test_decode_threshold(shared):
    x = _decode_case(21, 3, 6, 2, 128, 2500, [2500, 1800, 640], shared)
    S, tau = x["S"].numpy(), 0.02
    for b, n in enumerate(x["lens"].tolist()):
        cur = (n - 1) // 64
        for h in range(S.shape[1]):  # no gate so near to tau that fp32 may decide otherwise
            band = [oracle.threshold_count(S[b, h], cur, tau * math.exp(s)) for s in (1e-4, -1e-4)]
            assert band[0] == band[1]
    _check(x, 2500, 16, shared, tau=tau)


def _scores(kind, S):
    """Scores of a kind, in the shape of S."""
    n = S.shape[-1]
    if kind == "ties":
        return (2 * S).round() / 2
    if kind == "equal":
        return torch.zeros_like(S)
    if kind == "ascending":
        return torch.arange(n).float().expand_as(S).contiguous() / 64
    if kind == "one high":
        return torch.where(torch.arange(n) == n // 2, 50.0, -0.0 * S)
    if kind == "wide":
        return S * 10 ** (6 * S)
    return S


@pytest.mark.parametrize("kind", ["normal", "ties", "equal", "ascending", "one high", "wide"])
@pytest.mark.parametrize("k", [1, 32, 96, 97, 256])
def test_decode_selects_in_rows_of_many_blocks(kind, k):
    L = [16500, 20011, 70000][k % 3]  # 258, 313 and 1094 blocks
    x = _decode_case(k, 1, 4, 2, 64, L, None, False, paged=False)
    x["S"] = _scores(kind, x["S"]).clamp(-80, 80)
    _check(x, L, k, False)


@pytest.mark.parametrize("L", [131072, 131137, 200000, 524289, 530000])
@pytest.mark.parametrize("kind", ["normal", "ties"])
def test_decode_rows_at_the_borders_of_the_selections(L, kind):
    """2048 and 2049 blocks, 8192 and more: the selections that the kernel does itself, and the one before it."""
    x = _decode_case(L, 1, 2, 1, 64, L, None, True, paged=False)
    x["S"] = _scores(kind, x["S"])
    _check(x, L, 20, True)


@pytest.mark.parametrize("tau", [1e-6, 1e-3, 0.01])
def test_decode_threshold_in_long_rows(tau):
    x = _decode_case(1, 2, 2, 2, 64, 40000, [40000, 17000], False)
    S = x["S"].numpy()
    for b, n in enumerate(x["lens"].tolist()):
        cur = (n - 1) // 64
        for h in range(2):
            band = [oracle.threshold_count(S[b, h], cur, tau * math.exp(s)) for s in (1e-4, -1e-4)]
            assert min(band[0], 40) == min(band[1], 40)
    _check(x, 40000, 40, False, tau=tau)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_idle_slots(dtype):
    """Length 0 gives 0 and -infinity, whatever the slot's pages hold."""
    x = _decode_case(5, 5, 4, 2, 64, 300, [0, 300, 0, 1, 0], True, dtype)
    _check(x, 300, 3, True)
    _check(_decode_case(6, 1, 4, 2, 64, 300, [0], False, dtype), 300, 3, False)


@pytest.mark.parametrize("spread", [1e-5, 1e-3, 30.0, 6000.0])
def test_decode_small_and_large_values(spread):
    _check(_decode_case(7, 2, 4, 2, 128, 700, None, True, spread=spread), 700, 6, True, scale=0.02, spread=spread)


def test_rows_behind_the_sequence_may_hold_anything():
    """NaN parameters behind the last token and in pages of other sequences do not reach the result."""
    for dtype in (BF, F32):
        for n in (1, 17, 64, 100):
            x = _decode_case(n, 1, 4, 2, 128, 128, [n], False, dtype)
            want = _run(x, 128, 4, False)
            for i in (1, 3):
                for page in set(range(x["cache"][i].shape[0])) - set(x["table"][0].tolist()):
                    x["cache"][i][page] = float("nan")
                for c, page in enumerate(x["table"][0].tolist()):
                    x["cache"][i][page, :, max(0, min(64, n - 64 * c)):] = float("nan")
            got = _run(x, 128, 4, False)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            assert bool(torch.isfinite(got[0]).all())


def test_a_nan_row_that_counts_shows():
    x = _decode_case(3, 2, 4, 2, 64, 128, None, True)
    x["cache"][1][int(x["table"][0, 1]), 0, 63, 0, 1] = float("nan")
    O, LSE = _run(x, 128, 4, True)
    assert bool(torch.isnan(LSE[0, :2]).all()) and bool(torch.isfinite(LSE[0, 2:]).all())
    assert bool(torch.isnan(O[0, :2]).all()) and bool(torch.isfinite(O[1]).all())


def test_bad_pages_and_lengths_are_reported():
    x = _decode_case(8, 2, 4, 2, 64, 200, [200, 100], True)
    p = gb.make_params(2, 4, 2, 200, 64, 64, 8, "sparse")
    ws = torch.zeros(gb.kv4_workspace_bytes(p), dtype=torch.uint8, device=DEV)
    want = _run(x, 200, 8, True, ws=ws)
    gb.check(ws)
    for page in (-1, x["cache"][0].shape[0]):
        y = dict(x, table=x["table"].clone())
        y["table"][1, 0] = page
        got = _run(y, 200, 8, True, ws=ws)
        with pytest.raises(gb.GbsError):
            gb.check(ws)
        gb.clear_error(ws)
        assert torch.equal(got[0][0], want[0][0])
    for n, same in ((-1, 0), (201, 200)):
        y = dict(x, lens=torch.tensor([n, 100], dtype=torch.int32))
        got = _run(y, 200, 8, True, ws=ws)
        with pytest.raises(gb.GbsError):
            gb.check(ws)
        gb.clear_error(ws)
        z = dict(x, lens=torch.tensor([same, 100], dtype=torch.int32))
        assert torch.equal(got[0], _run(z, 200, 8, True)[0])


def test_pages_give_the_contiguous_bits():
    B, Hq, Hkv, d, L = 3, 8, 2, 128, 1000
    x = _decode_case(9, B, Hq, Hkv, d, L, [1000, 999, 130], False, paged=False)
    g = torch.Generator().manual_seed(1)
    nb = -(-L // 64)
    table = _table(g, B, nb)
    pools = []
    for t in x["cache"]:
        pool = torch.zeros(B * nb + 3, Hkv, 64, *t.shape[3:], dtype=t.dtype)
        pool[table.long()] = t.view(B, Hkv, nb, 64, *t.shape[3:]).transpose(1, 2)
        pools.append(pool)
    y = dict(x, cache=pools, table=table)
    for shared in (False, True):
        x["S"] = y["S"] = torch.randn(B, Hkv if shared else Hq, nb, generator=g)
        assert all(torch.equal(a, b) for a, b in zip(_run(x, L, 6, shared), _run(y, L, 6, shared)))


def test_rows_beyond_32_bit_offsets():
    """A pool of more than 2^32 code bytes: pages at its end are written, read and decoded like those at its
    beginning."""
    B, Hq, Hkv, d, L, pages = 2, 2, 1, 128, 200, 1 << 20
    g = torch.Generator().manual_seed(3)
    cache = [torch.empty(pages, Hkv, 64, d // 2, dtype=torch.uint8, device=DEV),
             torch.empty(pages, Hkv, 64, d // 32, 2, dtype=torch.float16, device=DEV)]
    cache += [torch.empty_like(t) for t in cache]
    assert cache[0].numel() == 1 << 32
    K, V = (torch.randn(1, Hkv, L, d, generator=g).to(BF).to(DEV).expand(B, Hkv, L, d) for _ in "kv")
    table = torch.tensor([[0, 1, 2, 3], [pages - 1, pages - 3, pages - 4, pages - 2]], dtype=torch.int32, device=DEV)
    start = torch.zeros(B, dtype=torch.int32, device=DEV)
    gb.kv4_append(K, V, cache, start, block_table=table)
    back = gb.kv4_read(cache, start, L, block_table=table, dtype=F32)
    assert all(torch.equal(t[0], t[1]) for t in back)
    _within(back[0][0], kv4_quantised(K[0]))
    q = torch.randn(1, Hq, d, generator=g).expand(B, Hq, d).contiguous().to(DEV)
    S = torch.randn(1, Hq, 4, generator=g).expand(B, Hq, 4).contiguous().to(DEV)
    for dtype in (BF, F32):
        O, LSE = gb.kv4_decode(q.to(dtype), cache, S, L, topk=2, block_table=table)
        assert torch.equal(O[0], O[1]) and torch.equal(LSE[0], LSE[1]) and bool(torch.isfinite(LSE).all())


def test_decode_on_another_stream_in_a_graph_and_twice():
    x = _decode_case(10, 2, 4, 2, 128, 900, [900, 80], True)
    want = _run(x, 900, 8, True)
    torch.cuda.synchronize()
    on = {n: t.to(DEV) if isinstance(t, torch.Tensor) else t for n, t in x.items()}
    cache = [t.to(DEV) for t in x["cache"]]
    torch.cuda.synchronize()
    call = lambda **kw: gb.kv4_decode(on["q"], cache, on["S"], 900, topk=8, block_table=on["table"],  # noqa: E731
                                      seq_lens=on["lens"], group_shared=True, **kw)
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = [call(stream=s) for s in sides for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in got for a, b in zip(r, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = call()
    # the graph reads the lengths at replay
    on["lens"].copy_(torch.tensor([80, 900], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    again = call()
    assert all(torch.equal(a, b) for a, b in zip(kept, again)) and not torch.equal(kept[0], want[0])


def test_debug_build_finds_every_index_in_range():
    """libgbs_debug.so checks what is read from lists and must give the same bits."""
    saved, out = gb._lib, []
    cases = [(_decode_case(30, 2, 4, 2, 64, 3000, [3000, 65], False), 3000, 8),
             (_decode_case(31, 1, 2, 1, 64, 530000, None, True, paged=False), 530000, 20),
             (_decode_case(32, 2, 4, 2, 128, 500, [500, 0], True, F32), 500, 3)]
    try:
        for debug in (False, True):
            gb._lib = None
            gb.load_library(build(debug=debug))
            for x, L, k in cases:
                B, Hq, d = x["q"].shape
                p = gb.make_params(B, Hq, x["cache"][0].shape[1], L, d, 64, k, "sparse", x["q"].dtype)
                ws = torch.zeros(gb.kv4_workspace_bytes(p), dtype=torch.uint8, device=DEV)
                out.append(_run(x, L, k, x["S"].shape[1] < Hq, ws=ws))
                gb.check(ws)
    finally:
        gb._lib = saved
    for a, b in zip(out[:3], out[3:]):
        assert all(torch.equal(t, u) for t, u in zip(a, b))


# ------------------------------------------------------------------ together


def test_a_prompt_and_steps_through_all_of_it():
    """Projection -> norms and rotation -> cache -> decode, one token after another, against the same through
    float64: the cache's rows are compared through what was written (their rounding to 4 bits is exact), the
    attention against the oracle over them."""
    B, Hq, Hkv, d, T, steps = 2, 8, 2, 128, 150, 3
    g = torch.Generator().manual_seed(2)
    L = T + steps
    nb = -(-L // 64)
    table = _table(g, B, nb).to(DEV)
    cache = gb.kv4_cache(B, Hkv, d, num_pages=B * nb + 3, device=DEV)
    cos, sin = gb.rope_tables(L, d, device=DEV)
    wq, wk = (1 + 0.1 * torch.randn(2, d, generator=g)).to(DEV)
    lens = torch.tensor([T, T - 70], dtype=torch.int32, device=DEV)  # a padded batch

    def tokens(n, pos):
        qkv = torch.randn(B, n, Hq + 2 * Hkv, d, generator=g).to(BF).to(DEV)
        return gb.qkv_rope(*qkv.split((Hq, Hkv, Hkv), 2), cos, sin, pos, wq, wk)

    _, K, V = tokens(T, torch.arange(T, dtype=torch.int32, device=DEV).expand(B, T).contiguous())
    gb.kv4_append(K, V, cache, torch.zeros_like(lens), block_table=table, count=lens)
    for _ in range(steps):
        Q, K, V = tokens(1, lens[:, None].contiguous())
        gb.kv4_append(K, V, cache, lens, block_table=table)
        lens += 1
        x = dict(q=Q[:, :, 0].cpu(), cache=[t.cpu() for t in cache], table=table.cpu(), lens=lens.cpu(),
                 S=torch.randn(B, Hkv, nb, generator=g))
        _check(x, L, 1, True)


@pytest.mark.parametrize("L", [1000, 20000, 140000])
@pytest.mark.parametrize("k", [0, 20, 96, 256])
def test_a_nan_score_keeps_the_selection_in_range(L, k):
    """Scores have to be finite; any NaN among them, the one of all bits set too, still gives blocks of the row."""
    x = _decode_case(11, 2, 4, 2, 64, L, None, False, paged=False)
    bits = x["S"].view(torch.int32)
    bits[0, :2] = -1
    bits[0, 2, ::3] = 0x7fffffff
    O, LSE = _run(x, L, k, False)
    y = dict(x, S=torch.zeros_like(x["S"]))
    y["S"][1] = x["S"][1]
    want = _run(y, L, k, False)
    assert torch.equal(O[1], want[0][1]) and torch.equal(LSE[1], want[1][1])


def test_groups_of_one_value_whose_minimum_rounds_up():
    """0.3 is 0.30005 in fp16, so such a group has a scale below 0 (and codes 0). One key with 8,255 others of 2^-18 of
    its weight, which together make up 3 % of the sum: the weights have to keep them."""
    L, d = 64 * 130, 64
    K, V = torch.zeros(1, 1, L, d), torch.full((1, 1, L, d), 5.0)
    K[0, 0, 0], V[0, 0, 0] = 12.5, 0.3
    cache = gb.kv4_cache(1, 1, d, L, device=DEV)
    gb.kv4_append(K.to(DEV), V.to(DEV), cache, torch.zeros(1, dtype=torch.int32, device=DEV))
    assert float(cache[3][0, 0, 0, 0, 0]) < 0
    x = dict(table=None, lens=None, cache=[t.cpu() for t in cache], q=torch.ones(1, 1, d, dtype=BF),
             S=torch.zeros(1, 1, 130))
    _check(x, L, 256, False, scale=1 / d)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("power,scale", [(-124, 0.0), (-124, 2.0 ** 120), (-60, 2.0 ** 57), (60, 2.0 ** -63),
                                         (118, 2.0 ** -121)])
def test_decode_of_small_and_large_queries(power, scale, dtype):
    """Queries near both ends of fp32's range, with a scale that makes their logits ordinary (or leaves them small)."""
    x = _decode_case(13, 2, 4, 2, 64, 300, [300, 77], True, dtype)
    x["q"] *= 2.0 ** power
    _check(x, 300, 3, True, scale=scale)


def _rows_case():
    g = torch.Generator().manual_seed(3)
    K, V = (torch.randn(2, 2, 5, 64, generator=g).to(BF).to(DEV) for _ in "kv")
    return K, V, torch.tensor([60, 0], dtype=torch.int32, device=DEV), torch.tensor([5, 3], dtype=torch.int32, device=DEV)


def test_native_calls_give_what_the_bindings_own_path_gives(monkeypatch):
    """csrc/marshal.cpp's calls and the Python path behind them: the same results, for given and new outputs, and the
    same refusals."""
    K, V, start, count = _rows_case()
    table = torch.tensor([[2, 0], [1, 3]], dtype=torch.int32, device=DEV)
    x = _decode_case(17, 2, 4, 2, 64, 300, [300, 77], True)
    x = {n: t.to(DEV) if isinstance(t, torch.Tensor) else t for n, t in x.items()}
    x["cache"] = tuple(t.to(DEV) for t in x["cache"])
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)

    def results():
        out = []
        for pages, block_table in ((None, None), (4, table)):
            cache = gb.kv4_cache(2, 2, 64, L=None if pages else 128, num_pages=pages, device=DEV)
            for n in (None, count):
                gb.kv4_append(K, V, cache, start, block_table, n, ws=ws if n is None else None)
                out += [*cache, *gb.kv4_read(cache, start, 5, block_table, n, dtype=F32)]
        for tau, splits, lens in ((None, 0, x["lens"]), (0.1, 2, None)):
            given = dict(out=torch.empty_like(x["q"]), lse=torch.empty(2, 4, device=DEV), ws=ws)
            for kw in ({}, given):
                O, LSE = gb.kv4_decode(x["q"], x["cache"], x["S"], 300, topk=3, block_table=x["table"], seq_lens=lens,
                                       group_shared=True, tau=tau, num_splits=splits, **kw)
                assert not kw or O is kw["out"] and LSE is kw["lse"]
                out += [O, LSE]
        return [t.clone() for t in out]

    def refusals():
        text = []
        cache = gb.kv4_cache(2, 2, 64, 128, device=DEV)
        for call in (lambda: gb.kv4_append(K, V[:, :, :4], cache, start),
                     lambda: gb.kv4_append(K, V, cache[:3], start),
                     lambda: gb.kv4_append(K, V, cache, start.long()),
                     lambda: gb.kv4_read(cache, start, 5, dtype=torch.float16),
                     lambda: gb.kv4_read(cache, start[:1], 5),
                     lambda: gb.kv4_decode(x["q"], x["cache"], x["S"], 301, topk=3, block_table=x["table"]),
                     lambda: gb.kv4_decode(x["q"], x["cache"], x["S"], 300, topk=257, block_table=x["table"],
                                           group_shared=True),
                     lambda: gb.kv4_decode(x["q"], x["cache"], x["S"], 300, topk=3, block_table=x["table"],
                                           group_shared=True, scale=-1.0),
                     lambda: gb.kv4_decode(x["q"], x["cache"], x["S"], 300, topk=3, block_table=x["table"],
                                           group_shared=True, ws=ws[:128])):
            with pytest.raises(gb.GbsError) as e:
                call()
            text.append(str(e.value))
        return text

    assert gb._native is not gb._NoCalls
    native = results(), refusals()
    monkeypatch.setattr(gb, "_native", gb._NoCalls)
    own = results(), refusals()
    assert all(torch.equal(a, b) for a, b in zip(native[0], own[0])) and native[1] == own[1]


def test_plain_calls_are_native(monkeypatch):
    """Plain arguments do not reach the Python checks."""
    K, V, start, count = _rows_case()
    cache = gb.kv4_cache(2, 2, 64, 128, device=DEV)
    q, S = torch.randn(2, 4, 64, device=DEV), torch.randn(2, 4, 2, device=DEV)
    monkeypatch.setattr(gb, "_check_kv4", None)
    gb.kv4_append(K, V, cache, start, count=count)
    gb.kv4_read(cache, start, 5)
    gb.kv4_decode(q, cache, S, 100, topk=1)
    gb.kv4_decode(q.to(BF), cache, S, 100, topk=1, tau=0.5, scale=1)
