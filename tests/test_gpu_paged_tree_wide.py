"""Trees with many rows a key/value head, on the wide products: how a call is cut up, sequences that leave a part of a
unit's rows or none, many units a block, streams and captured graphs. The tolerance is that of test_gpu_paged_tree."""
import ctypes

import numpy as np
import pytest
import torch

import gpu_util as G
import transformer_attention_relative_gb300 as rp
from test_gpu_paged_decode import MODES, _case, _check
from test_gpu_paged_tree import _ref, _tree

pytestmark = pytest.mark.gpu
BF, E4 = torch.bfloat16, torch.float8_e4m3fn
LONG = 160 * 128  # slots of a table that is long enough for the wide products whatever the sequences hold


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def _split(cache, B, Hq, n, pages, mode=0):
    out = [ctypes.c_int(-1) for _ in range(3)]
    assert rp.relpos_selftest_paged_tree_split(cache._ref, B, Hq, n, pages, mode, *(ctypes.byref(x) for x in out)) == 0
    return tuple(x.value for x in out)


def _long(table, page):
    return torch.nn.functional.pad(table, (0, max(0, LONG // page - table.shape[1])), value=-1)


def _run(cache, q, table, lens, parents, bias, mode, nodes=None, short=False, **kw):
    table = table if short else _long(table, cache.page_size)
    B, Hq, n, _ = q.shape
    assert _split(cache, B, Hq, n, table.shape[1], MODES[mode] or 0)[2] == 1
    o = rp.paged_tree_decode(q.cuda(), cache, table.cuda(), lens.cuda(), parents.cuda(),
                             nodes=None if nodes is None else torch.tensor(nodes, dtype=torch.int32).cuda(),
                             bias=None if bias is None else bias.cuda(), mode=MODES[mode], **kw)
    torch.cuda.synchronize()
    assert rp.check_status() == 0
    return o


def _parity(lens, Hq, Hkv, n, d, page, dtype, mode, seed, nodes=None, **kw):
    cache, q, table, lens, bias = _case(lens, Hq, Hkv, n, d, page, dtype, mode, seed)
    parents = _tree("random", len(lens), n, seed)
    got = _run(cache, q, table, lens, parents, bias, mode, nodes, **kw)
    kw.pop("short", None)
    _check(got, *_ref(cache, q, table, lens, parents, bias, mode, nodes, **kw), dtype == E4)


def test_which_products_run():
    for dtype, none, alibi in ((BF, 9, 9), (E4, 33, 17)):
        cache = rp.PagedCache.empty(4, 2, 64, page_size=64, dtype=dtype)
        for mode, first in ((0, none), (rp.MODE_T5, none), (rp.MODE_ALIBI, alibi)):
            assert _split(cache, 1, 2 * (first - 1), 1, 512, mode)[2] == 0
            assert _split(cache, 1, 2 * first, 1, 512, mode) == (first, 2, 1)
            # up to a tile of 128 keys an SM: the others
            sms = torch.cuda.get_device_properties(0).multi_processor_count
            assert _split(cache, 1, 2 * first, 1, 2 * (sms // 2), mode)[2] == 0
            assert _split(cache, 1, 2 * first, 1, 2 * (sms // 2 + 1), mode)[2] == 1
        assert _split(cache, 1, 2 * 8, 64, 512) == (256, 2, 1)
        assert _split(cache, 1, 2 * 5, 64, 512) == (160, 2, 1)
        assert _split(cache, 1, 2 * 9, 64, 512) == (192, 2, 1)
        assert _split(cache, 100, 2 * 9, 64, 4) == (192, 1, 1)


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,n", [(1, 9), (1, 32), (3, 11), (2, 32), (65, 1), (2, 64), (43, 3), (4, 64), (257, 1), (9, 57)])
def test_rows_of_a_unit(dtype, d, G, n):
    """Four, two and no copies; one tile for both warpgroups; pairs; several units a head."""
    if dtype == E4 and G * n < 33:
        n = 33
    _parity([n + 700, n, 130 + n], 2 * G, 2, n, d, 64, dtype, "t5" if G < 20 else "none", 31)


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("mode", ["none", "t5", "alibi"])
def test_sequences_that_leave_a_part_of_the_rows(dtype, mode):
    """Units of 256 rows with 0, 1, .. of them in use: the same unit as pair, with the second half short, and as single."""
    nodes = [32, 0, 1, 8, 16, 17, 31, 4]
    lens = [500, 300, 1, 8, 400, 129, 800, 128]
    _parity(lens, 16, 2, 32, 64, 32, dtype, mode, 32, nodes)
    _parity(lens, 18, 2, 32, 128, 32, dtype, mode, 33, nodes)  # two units of 144


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("n,Hq", [(12, 8), (40, 2), (33, 8)])
def test_more_sequences_than_a_warp_has_lanes(dtype, n, Hq):
    lens = [0 if b % 9 == 4 else n + (53 * b) % 400 for b in range(77)]
    nodes = [0 if b % 9 == 4 or b % 13 < 3 else 1 + (5 * b) % n for b in range(77)]
    mode = "alibi" if n * Hq // 2 < 33 else "t5"
    _parity(lens, Hq, 2, n, 64, 32, dtype, mode, 34, nodes)


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("G", [1, 4])
def test_a_block_for_each_unit(dtype, G):
    """Tables of up to two tiles: no joining launch."""
    B, n = 90, 40
    lens = [0 if b == 3 else n + (31 * b) % (256 - n + 1) for b in range(B)]
    cache = _case([1], 2, 2, 1, 64, 64, dtype, "none", 0)[0]
    assert _split(cache, B, 2 * G, n, 4) == (G * n, 1, 1)
    for mode in ("t5", "alibi"):
        cache, q, table, ln, bias = _case(lens, 2 * G, 2, n, 64, 64, dtype, mode, 35)
        parents = _tree("random", B, n, 35)
        nodes = [0 if b in (3, 7) else 1 + b % n for b in range(B)]
        got = _run(cache, q, table[:, :4], ln, parents, bias, mode, nodes, short=True)
        _check(got, *_ref(cache, q, table, ln, parents, bias, mode, nodes), dtype == E4)


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("mode", ["none", "t5", "alibi"])
@pytest.mark.parametrize("scale", [-0.2, 2.0 ** -20, 0.9])
def test_scales_of_any_sign(dtype, mode, scale):
    _parity([300, 40], 8, 2, 40, 64, 64, dtype, mode, 36, scale=scale)


@pytest.mark.parametrize("dtype", [E4, BF])
def test_slopes_of_any_sign_and_large_biases(dtype):
    cache, q, table, lens, _ = _case([700, 64], 8, 2, 40, 64, 64, dtype, "alibi", 37)
    parents = _tree("random", 2, 40, 37)
    slopes = torch.tensor([0.0, -0.01, 0.5, 30.0, 1e-20, -1e-3, 3.0, 0.1])
    got = _run(cache, q, table, lens, parents, slopes, "alibi")
    # logits of up to 30 * 700 log2(e), in fp32: 2^-24 of them, a few times over, beside the usual 2^-12
    _check(got, *_ref(cache, q, table, lens, parents, slopes, "alibi"), dtype == E4)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,n", [(1, 40), (2, 64), (4, 64)])
def test_foul_scales_and_pages_of_zeros(d, G, n):
    """Pages whose scales have no power of two beside the others' fall back to bf16 products."""
    cache, q, table, lens, bias = _case([700, 300], 2 * G, 2, n, d, 32, E4, "none", 38)
    cache.k_scale[table[0, 1].item()] = 0.0
    cache.v_scale[table[0, 2].item()] = 2.0 ** -140
    cache.v_scale[table[1, 3].item()] = -2.0 ** -6
    cache.k_scale[table[1, 4].item()] = 2.0 ** -60
    parents = _tree("random", 2, n, 38)
    got = _run(cache, q, table, lens, parents, bias, "none")
    _check(got, *_ref(cache, q, table, lens, parents, bias, "none"), True)


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -30, 2.0 ** 20])
def test_query_rows_of_any_size(size):
    """(With keys as much smaller, where the rows are large.)"""
    cache, q, table, lens, bias = _case([500, 100], 4, 2, 40, 64, 64, E4, "none", 39)
    q = (q.float() * size).to(BF)
    if size > 1:
        cache.k_scale.mul_(1 / size)
    parents = _tree("random", 2, 40, 39)
    got = _run(cache, q, table, lens, parents, bias, "none")
    _check(got, *_ref(cache, q, table, lens, parents, bias, "none"), True)


@pytest.mark.parametrize("dtype", [E4, BF])
def test_streams_captures_and_replays(dtype):
    """The first call of its sizes under capture; two graphs and two streams at once; other lengths at a replay."""
    n, Hq = 36, 8
    a, b = (_case([900, 257], Hq, 2, n, 64, 64, dtype, "t5", s) for s in (40, 41))
    parents = _tree("random", 2, n, 40)
    gpu = []
    for cache, q, table, lens, bias in (a, b):
        gpu.append((q.cuda(), cache, _long(table, 64).cuda(), lens.cuda(), parents.cuda(), bias.cuda()))
    outs = [torch.zeros_like(g[0]) for g in gpu]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()

    def call(i, **kw):
        q, cache, table, lens, par, bias = gpu[i]
        return rp.paged_tree_decode(q, cache, table, lens, par, bias=bias, mode=rp.MODE_T5, out=outs[i], **kw)

    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i in range(2):
        with torch.cuda.graph(graphs[i], stream=streams[i]):
            call(i)
    want = [_ref(c, q, t, ln, parents, bi, "t5") for c, q, t, ln, bi in (a, b)]
    for _ in range(3):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        _check(outs[i], *want[i], dtype == E4)
    first = [o.clone() for o in outs]
    torch.cuda.synchronize()
    for _ in range(3):
        for i in range(2):
            call(i, stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, outs))
    lens = torch.tensor([100, 36], dtype=torch.int32)
    gpu[0][3].copy_(lens.cuda())
    torch.cuda.synchronize()
    graphs[0].replay()
    torch.cuda.synchronize()
    cache, q, table, _, bias = a
    _check(outs[0], *_ref(cache, q, table, lens, parents, bias, "t5"), dtype == E4)
    assert rp.check_status() == 0


def test_the_same_bits_in_another_place():
    """What a block does not depend on: pages elsewhere, other table columns."""
    cache, q, table, lens, bias = _case([3000, 500], 8, 2, 40, 128, 64, E4, "alibi", 42)
    parents = _tree("random", 2, 40, 42)
    a = _run(cache, q, table, lens, parents, bias, "alibi")
    perm = torch.randperm(cache.num_pages, generator=torch.Generator().manual_seed(1))
    moved = rp.PagedCache(*(x.view(torch.uint8)[perm.argsort().cuda()].view(E4) for x in (cache.k, cache.v)),
                          *(x[perm.argsort().cuda()].contiguous() for x in (cache.k_scale, cache.v_scale)))
    to = torch.where(table >= 0, perm[table.clamp(min=0).long()].to(torch.int32), table)
    b = _run(moved, q, torch.nn.functional.pad(to, (0, 999), value=-7), lens, parents, bias, "alibi")
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [E4, BF])
def test_a_long_context_of_many_rows(dtype):
    """Units that go over many blocks, in pairs; the last shares in the midst of a unit."""
    cache, q, table, lens, bias = _case([30011, 64], 4, 1, 64, 64, 128, dtype, "t5", 43)
    parents = _tree("random", 2, 64, 43)
    got = _run(cache, q, table, lens, parents, bias, "t5", [64, 64])
    _check(got, *_ref(cache, q, table, lens, parents, bias, "t5", [64, 64]), dtype == E4)
    np.testing.assert_array_equal(got.isfinite().cpu(), True)


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("n", [3, 40])
def test_pages_past_4_gb(dtype, n):
    """The same pages at the end of a pool whose keys take more than 4 GB: the same bits, whichever products run."""
    size = 1 if dtype == E4 else 2
    pages = (1 << 32) // (2 * 128 * 128 * size) + 40
    cache, q, table, lens, bias = _case([900, 300], 4, 2, n, 128, 128, dtype, "alibi", 44)
    parents = _tree("random", 2, n, 44)
    far = rp.PagedCache.empty(pages, 2, 128, page_size=128, dtype=dtype)
    at = pages - cache.num_pages
    for name in ("k", "v"):
        getattr(far, name).view(torch.uint8)[at:] = getattr(cache, name).view(torch.uint8)
        if dtype == E4:
            getattr(far, name + "_scale")[at:] = getattr(cache, name + "_scale")
    outs = [rp.paged_tree_decode(q.cuda(), c, _long(t, 128).cuda(), lens.cuda(), parents.cuda(), bias=bias.cuda(),
                                 mode=rp.MODE_ALIBI)
            for c, t in ((cache, table), (far, torch.where(table >= 0, table + at, table)))]
    assert rp.check_status() == 0 and torch.equal(*outs)
    _check(outs[1], *_ref(cache, q, table, lens, parents, bias, "alibi"), dtype == E4)


@pytest.mark.parametrize("dtype", [E4, BF])
def test_sequences_that_share_pages_and_a_shared_query(dtype):
    """One context under several trees, and one query row for all of them (strides of 0)."""
    cache, q, table, lens, bias = _case([500], 8, 2, 40, 64, 64, dtype, "t5", 45)
    B = 5
    parents = _tree("random", B, 40, 45)
    got = _run(cache, q.cuda().expand(B, -1, -1, -1), table.expand(B, -1), lens.expand(B).contiguous(), parents, bias, "t5")
    for b in range(B):
        _check(got[b:b + 1], *_ref(cache, q, table, lens, parents[b:b + 1], bias, "t5"), dtype == E4)
