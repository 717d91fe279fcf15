"""What a decode makes of pages and lengths outside its cache, in the sequence that has them: the keys of a page that
does not exist are left out, a sequence longer than its block table is skipped (zero rows), and the status says so.

Tolerance as for the other decodes: 2^-8 of the output, and of A = sum_j p_j |v_j| the weights' rounding (2^-11 in
8-bit caches, 2^-16 in 16-bit ones) and twice their logits' error (2^-12)."""
import numpy as np
import pytest
import torch

import gpu_util as G
import transformer_attention_relative_gb300 as rp
from test_gpu_paged_decode import _case, _gpu, _ref

pytestmark = pytest.mark.gpu
BF, E4 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def _without(cache, q, table, lens, bias, mode, gone):
    """The oracle's attention of sequence 0 without the keys of the pages `gone`."""
    n, page = int(lens[0]), cache.page_size
    keep = np.array([j for j in range(n) if j // page not in gone], dtype=int)
    _, Hq, Lq, d = q.shape
    out, size = np.zeros((Hq, Lq, d)), np.zeros((Hq, Lq, d))
    for h in range(Hq):
        kv = []
        for name in ("k", "v"):
            x = getattr(cache, name)[:, h // (Hq // cache.heads)].double().cpu().numpy()
            if cache.k_scale is not None:
                x = x * getattr(cache, name + "_scale")[:, h // (Hq // cache.heads)].double().cpu().numpy()[:, None, None]
            pages = [int(i) if j not in gone else 0 for j, i in enumerate(table[0, :(n + page - 1) // page])]
            kv.append(x[pages].reshape(-1, d))
        for i in range(Lq):
            at = keep[keep <= n - Lq + i]
            if len(at) == 0:
                continue
            z = kv[0][at] @ q[0, h, i].double().numpy() / np.sqrt(d)
            if mode == "alibi":
                z = z - float(bias[h]) * (n - Lq + i - at)
            e = np.exp(z - z.max())
            e /= e.sum()
            out[h, i], size[h, i] = e @ kv[1][at], e @ np.abs(kv[1][at])
    return out, size


def _near(got, ref, size, eight):
    got = got.double().cpu().numpy()
    assert np.all(np.isfinite(got))
    tol = 2.0 ** -8 * np.abs(ref) + size * ((2.0 ** -11 if eight else 2.0 ** -16) + 2.0 ** -12)
    assert np.all(np.abs(got - ref) <= tol), float((np.abs(got - ref) - tol).max())


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("mode", ["none", "alibi"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,gone", [((100, 90), (1,)), ((100, 90), (0, 3)), ((100, 90), (0, 1, 2, 3)),
                                       ((3000, 90), (0, 1, 2, 3, 4, 5, 6, 7, 40, 93)), ((3000, 90), tuple(range(60)))])
def test_keys_of_missing_pages_are_left_out(dtype, mode, d, lens, gone):
    """Page 0 of the pool belongs to nobody and holds NaN, scales too; so the other sequence stays as it was."""
    cache, q, table, lens, bias = _case(list(lens), 4, 2, 2, d, 32, dtype, mode, 51)
    free = sorted(set(range(cache.num_pages)) - set(table[table >= 0].tolist()))[0]
    swap = torch.arange(cache.num_pages)
    swap[0], swap[free] = free, 0  # the unused page to the front
    parts = [t if t.dtype != E4 else t.view(torch.uint8) for t in (cache.k, cache.v, cache.k_scale, cache.v_scale) if t is not None]
    for t in parts:
        t.copy_(t[swap.cuda()])
    moved = table.clone()
    moved[table == 0] = free
    table = moved
    broken = table.clone()
    for i, p in enumerate(gone):
        broken[0, p] = (-1, cache.num_pages, 2 ** 31 - 1, -2 ** 31)[i % 4]
    q = 4 * q  # keys that are left out must not dilute the rest
    got = _gpu(cache, q, broken, lens, bias, mode)
    assert rp.check_status() == rp.RELPOS_ERR_PAGE
    assert rp.check_status() == 0
    _near(got[0], *_without(cache, q, table, lens, bias, mode, gone), dtype == E4)
    ref, size = _ref(cache, q, table, lens, bias, mode)
    _near(got[1], ref[1], size[1], dtype == E4)


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("cols", [3, 40])
def test_a_sequence_longer_than_its_table_is_skipped(dtype, cols):
    """Short tables (one launch) and long ones (two)."""
    lens = [32 * cols, 90, 32 * cols - 5]
    cache, q, table, lens, bias = _case(lens, 4, 2, 2, 64, 32, dtype, "none", 52)
    ref, size = _ref(cache, q, table, lens, bias, "none")
    table = table[:, :cols].contiguous()
    for over in (32 * cols + 1, 2 ** 31 - 1):
        lens[0] = over
        got = _gpu(cache, q, table, lens, bias, "none")
        assert rp.check_status() == rp.RELPOS_ERR_PAGE and rp.check_status() == 0
        assert not got[0].float().any()
        _near(got[1:], ref[1:], size[1:], dtype == E4)
    lens[:] = 2 ** 31 - 1
    got = _gpu(cache, q, table, lens, bias, "none")
    assert rp.check_status() == rp.RELPOS_ERR_PAGE and not got.float().any()
