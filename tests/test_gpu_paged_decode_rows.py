"""Decodes of more rows than one unit of work has, vs the fp64 oracle: units of 16 rows, which large calls take, and
several units of 8 rows whose work is split among blocks. Which form runs is asserted: the library's rule may change.

A block table much wider than its sequences need makes a call count as large while the oracle stays cheap. Tolerance as
for the other decodes: 2^-8 of the output, and of A = sum_j p_j |v_j| the weights' rounding (2^-11 in 8-bit caches,
2^-16 in 16-bit ones) and twice their logits' error (2^-12)."""
import ctypes

import numpy as np
import pytest
import torch

import gpu_util as G
import transformer_attention_relative_gb300 as rp
from test_gpu_paged_decode import MODES, _case, _check, _ref

pytestmark = pytest.mark.gpu
BF, E4 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def _split(cache, B, Hq, Lq, pages):
    """(rows of a unit, launches) of such a call"""
    rows, launches = ctypes.c_int(), ctypes.c_int()
    assert rp.relpos_selftest_paged_decode_split(cache._ref, B, Hq, Lq, pages, ctypes.byref(rows),
                                                 ctypes.byref(launches)) == 0
    return rows.value, launches.value


def _widened(table, pages):
    return torch.cat([table, torch.full((table.shape[0], max(0, pages - table.shape[1])), -1, dtype=torch.int32)], 1)


def _run(cache, q, table, lens, bias, mode, pages, rows, launches, **kw):
    table = _widened(table, pages)
    assert _split(cache, q.shape[0], q.shape[1], q.shape[2], table.shape[1]) == (rows, launches)
    got = rp.paged_decode(q.cuda(), cache, table.cuda(), lens.cuda(), bias=None if bias is None else bias.cuda(),
                          mode=MODES[mode], **kw)
    torch.cuda.synchronize()
    return got


SHAPES = [(9, 1, 1), (16, 1, 1), (8, 2, 4), (8, 2, 5), (20, 1, 1), (10, 2, 8), (17, 1, 2)]  # Hq, Hkv, Lq


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("d,page", [(64, 32), (64, 128), (128, 64)])
@pytest.mark.parametrize("Hq,Hkv,Lq", SHAPES)
@pytest.mark.parametrize("rows", [8, 16])
def test_shared_units(dtype, d, page, Hq, Hkv, Lq, rows):
    """Ragged and empty sequences, some shorter than the new rows, some split among many blocks; every bias."""
    lens = [3000, 0, 1, 5, 700, 33, 64, 0, 1029]
    for mode in ("t5", "alibi", "none"):
        case = _case(lens, Hq, Hkv, Lq, d, page, dtype, mode, 100 * Hq + Lq)
        got = _run(*case, mode, (1 << 18) // page if rows == 16 else 0, rows, 2)
        assert rp.check_status() == 0
        _check(got, *_ref(*case, mode), dtype == E4)
        assert not got[1].float().any() and not got[7].float().any() and not got[2, :, :Lq - 1].float().any()


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,Lq", [(16, 8, 5), (72, 8, 1), (160, 8, 1)])
def test_a_block_for_each_unit_of_16_rows(dtype, d, Hq, Hkv, Lq):
    """Many short sequences: one launch, no scratch."""
    pages = 2 if dtype == BF and d == 128 else 4
    lens = [(37 * b) % 61 for b in range(398)] + [pages * 128, pages * 128 - 1]
    for mode in ("t5", "alibi"):
        cache, q, table, n, bias = _case(lens, Hq, Hkv, Lq, d, 128, dtype, mode, 7)
        table = table[:, :pages].contiguous()
        got = _run(cache, q, table, n, bias, mode, 0, 16, 1)
        assert rp.check_status() == 0
        for some in (slice(0, 12), slice(390, 400)):
            ref = _ref(cache, q[some], table[some], n[some], bias, mode)
            _check(got[some], *ref, dtype == E4)


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("bad", ["nan", "largest"])
def test_16_rows_that_see_a_bad_value_and_rows_that_do_not(dtype, d, where, bad):
    """A new token's NaN (in a 16-bit cache also an infinity) reaches the rows that see it and no other."""
    for n in (70, 1300):
        cache, q, table, lens, bias = _case([n, 20], 8, 2, 5, d, 32, dtype, "none", 12)
        ref, size = _ref(cache, q, table, lens, bias, "none")
        t = getattr(cache, where)
        p, s = int(table[0, (n - 3) // 32]), (n - 3) % 32  # the key of query row 2
        if dtype == E4:
            t.view(torch.uint8)[p, :, s] = 0x7f if bad == "nan" else 0xff
        else:
            t.view(torch.int16)[p, :, s] = 0x7fc0 if bad == "nan" else 0x7f80
        got = _run(cache, q, table, lens, bias, "none", (1 << 18) // 32, 16, 2)
        _check(got[:, :, :2], ref[:, :, :2], size[:, :, :2], dtype == E4)
        _check(got[1], ref[1], size[1], dtype == E4)
        if bad == "nan" or dtype == E4 or where == "v":
            assert not got[0, :, 2:].isfinite().any()
        assert rp.check_status() == 0


@pytest.mark.parametrize("nb,md", [(32, 128), (8, 20), (64, 3000), (128, 5000)])
@pytest.mark.parametrize("Hq,Lq", [(16, 1), (20, 1), (4, 5)])
@pytest.mark.parametrize("rows", [8, 16])
def test_bias_tables(nb, md, Hq, Lq, rows):
    """Near distances from a table in shared memory where it fits, from the buckets where it does not."""
    cache, q, table, lens, _ = _case([4000, 40], Hq, 1, Lq, 64, 64, E4, "t5", 10)
    bias = torch.randn(nb, Hq, generator=torch.Generator().manual_seed(1))
    kw = dict(num_buckets=nb, max_distance=md)
    got = _run(cache, q, table, lens, bias, "t5", (1 << 21) // 64 if rows == 16 else 0, rows, 2, **kw)
    _check(got, *_ref(cache, q, table, lens, bias, "t5", **kw), True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [8, 16])
def test_pages_of_very_different_scales(d, rows):
    """Zero pages, very large and very small values between ordinary ones, for 16 rows of a key/value head."""
    g = torch.Generator().manual_seed(3)
    cache, q, table, lens, bias = _case([1500, 300], 8, 2, 4, d, 32, E4, "none", 23)
    e = torch.randint(-9, -4, cache.v_scale.shape, generator=g).float()
    odd = torch.rand(e.shape, generator=g) < 0.3
    e[odd] = torch.randint(-120, 60, (int(odd.sum()),), generator=g).float()
    e[odd & (torch.rand(e.shape, generator=g) < 0.5)] = -120.0
    cache.v_scale.copy_(torch.exp2(e).cuda())
    got = _run(cache, q, table, lens, bias, "none", (1 << 18) // 32 if rows == 16 else 0, rows, 2)
    _check(got, *_ref(cache, q, table, lens, bias, "none"), True)
    assert rp.check_status() == 0


def test_long_shares_of_16_rows():
    """A batch that is large by its tokens: tens of tiles a warp, whole and shared units, 16 and 20 rows a head."""
    for dtype, d, Hq, Lq in ((E4, 64, 16, 1), (BF, 128, 10, 2)):
        H, B, page, n = 8, 40, 64, 4096
        g = torch.Generator().manual_seed(4)
        cache, q, table, _, _ = _case([n], Hq * H, H, Lq, d, page, dtype, "none", 31)
        q = q.expand(B, -1, -1, -1)
        lens = torch.randint(n - 500, n + 1, (B,), generator=g, dtype=torch.int32)
        many = table.expand(B, -1).contiguous()  # every sequence over the same pages
        got = _run(cache, q, many, lens, None, "none", 0, 16, 2)
        for b in (0, 7, 23, B - 1):
            ref = _ref(cache, q[b:b + 1], table, lens[b:b + 1], None, "none")
            _check(got[b:b + 1], *ref, dtype == E4)
    assert rp.check_status() == 0


def test_repeats_of_16_rows_are_equal():
    case = _case([3000, 500, 20, 1700], 8, 2, 5, 64, 64, E4, "alibi", 17)
    runs = [_run(*case, "alibi", (1 << 18) // 64, 16, 2) for _ in range(5)]
    assert all(torch.equal(r, runs[0]) for r in runs)


def test_missing_pages_and_long_lengths_with_16_rows():
    """As with 8 rows: the keys of missing pages are left out, an over-long sequence is skipped."""
    cache, q, table, lens, bias = _case([900, 300, 40], 8, 2, 4, 64, 32, BF, "none", 18)
    t = _widened(table, (1 << 18) // 32)
    t[0, 0], t[0, 9] = -1, cache.num_pages
    lens[2] = (1 << 18) + 1
    got = _run(cache, q, t, lens, bias, "none", 0, 16, 2)
    assert rp.check_status() == rp.RELPOS_ERR_PAGE and rp.check_status() == 0
    ref, size = _ref(cache, q[1:2], table[1:2], lens[1:2], bias, "none")
    _check(got[1:2], ref, size, False)
    assert not got[2].float().any()
    keep = np.array([j for j in range(900) if j // 32 not in (0, 9)])
    k, v = (getattr(cache, x).double().cpu().numpy() for x in ("k", "v"))
    pages = [int(p) if j not in (0, 9) else 0 for j, p in enumerate(table[0, :29])]
    for h in range(8):
        kk, vv = k[pages, h // 4].reshape(-1, 64), v[pages, h // 4].reshape(-1, 64)
        for i in range(4):
            at = keep[keep <= 896 + i]
            z = kk[at] @ q[0, h, i].double().numpy() / 8.0
            e = np.exp(z - z.max())
            e /= e.sum()
            _check(got[0, h, i], e @ vv[at], e @ np.abs(vv[at]), False)


def test_split_of_bad_arguments():
    cache = rp.PagedCache.empty(4, 2, 64)
    rows, launches = ctypes.c_int(), ctypes.c_int()
    out = ctypes.byref(rows), ctypes.byref(launches)
    f = rp.relpos_selftest_paged_decode_split
    assert f(cache._ref, 2, 4, 1, 100, *out) == 0 and f(None, 2, 4, 1, 100, *out) == rp.RELPOS_ERR_INVALID_ARG
    for a in ((0, 4, 1, 9), (2, 3, 1, 9), (2, 4, 0, 9), (2, 4, 1, 0)):
        assert f(cache._ref, *a, *out) == rp.RELPOS_ERR_INVALID_ARG
    assert f(cache._ref, 2, 4, 9, 9, *out) == rp.RELPOS_ERR_UNSUPPORTED
    assert f(cache._ref, 2, 4, 1, 9, None, out[1]) == rp.RELPOS_ERR_INVALID_ARG
