"""Attention of trees of drafted tokens over a paged cache vs the fp64 oracle.

Tolerance as for the other decodes, with A = sum_j p_j |v_j|: half a bf16 step of the output (2^-8 of it), the weights'
rounding before p v, 2^-11 A in 8-bit caches or 2^-16 A in 16-bit ones, and twice the logits' error, 2^-12 A."""
import numpy as np
import pytest
import torch

import gpu_util as G
import transformer_attention_relative_gb300 as rp
from oracle import serving_oracle as so
from test_gpu_paged_decode import MODES, _case, _check

pytestmark = pytest.mark.gpu
BF, E4 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


@pytest.fixture(autouse=True, params=["short table", "long table"])
def _tables(request):
    """Each case with its own table, and with one of so many columns that the library counts on long sequences and takes
    the wide products where there are rows enough for them."""
    global _columns
    _columns = 0 if request.param == "short table" else 160 * 128
    yield


_columns = 0


def _table(table, page):
    more = max(0, _columns // page - table.shape[1])
    return torch.nn.functional.pad(table, (0, more), value=-1).cuda()


def _tree(kind, B, n, seed=0):
    if kind == "chain":
        return torch.arange(-1, n - 1, dtype=torch.int32).expand(B, n).contiguous()
    if kind == "star":
        return torch.full((B, n), -1, dtype=torch.int32)
    g = torch.Generator().manual_seed(seed)
    t = (torch.rand(B, n, generator=g) * (torch.arange(n) + 1)).floor().to(torch.int32) - 1
    t[:, 0] = -1
    return t


def _gpu(cache, q, table, lens, parents, bias, mode, nodes=None, **kw):
    o = rp.paged_tree_decode(q.cuda(), cache, _table(table, cache.page_size), lens.cuda(), parents.cuda(),
                             nodes=None if nodes is None else torch.tensor(nodes, dtype=torch.int32).cuda(),
                             bias=None if bias is None else bias.cuda(), mode=MODES[mode], **kw)
    torch.cuda.synchronize()
    return o


def _values(cache):
    c = {"k": cache.k.double().cpu().numpy(), "v": cache.v.double().cpu().numpy()}
    if cache.k_scale is not None:
        c |= {"k_scale": cache.k_scale.double().cpu().numpy(), "v_scale": cache.v_scale.double().cpu().numpy()}
    return c


def _ref(cache, q, table, lens, parents, bias, mode, nodes=None, **kw):
    parents = parents if parents.dim() == 2 else parents.expand(len(lens), -1)
    return so.paged_tree_decode(q.double().numpy(), _values(cache), table.numpy(), lens.tolist(), cache.page_size,
                                parents.tolist(), nodes, None if bias is None else bias.double().numpy(), mode, **kw)


def _parity(lens, Hq, Hkv, n, d, page, dtype, mode, seed, kind="random", nodes=None, **kw):
    cache, q, table, lens, bias = _case(lens, Hq, Hkv, n, d, page, dtype, mode, seed)
    parents = _tree(kind, len(lens), n, seed)
    got = _gpu(cache, q, table, lens, parents, bias, mode, nodes, **kw)
    assert rp.check_status() == 0
    _check(got, *_ref(cache, q, table, lens, parents, bias, mode, nodes, **kw), dtype == E4)
    return got


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("d,page", [(64, 32), (64, 64), (64, 128), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("mode", ["none", "t5", "alibi"])
def test_types_pages_biases(dtype, d, page, mode):
    _parity([7, 8, 32, 39, 127, 135, 200, 515], 4, 2, 7, d, page, dtype, mode, 1)


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("Hq,Hkv,n", [(1, 1, 1), (3, 3, 2), (8, 1, 5), (16, 2, 16), (4, 4, 33), (16, 2, 64), (12, 4, 25),
                                      (33, 1, 9), (40, 1, 64)])
def test_heads_and_nodes(dtype, Hq, Hkv, n):
    """Rows of a key/value head from one to many tiles of them."""
    _parity([n, n + 3, 97, 300], Hq, Hkv, n, 64, 32, dtype, "t5", 2)
    _parity([n, n + 2, 97, 300], Hq, Hkv, n, 128, 64, dtype, "alibi", 3)


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("kind", ["chain", "star"])
@pytest.mark.parametrize("mode", ["none", "t5", "alibi"])
def test_chains_and_stars(dtype, kind, mode):
    _parity([64, 150, 1000], 4, 2, 64, 64, 32, dtype, mode, 4, kind)


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (16, 2)])
def test_trees_of_different_sizes(dtype, Hq, Hkv):
    """Sequences without nodes, of nodes alone, and none at all; rows without a node are zero whatever they hold."""
    lens, nodes = [0, 60, 5, 12, 200, 3], [4, 0, 5, 1, 12, 2]
    cache, q, table, lens, bias = _case(lens, Hq, Hkv, 12, 64, 32, dtype, "t5", 5)
    parents = _tree("random", 6, 12, 5)
    for b, m in enumerate(nodes):
        if lens[b] > 0:
            q[b, :, m:] = float("nan")
            parents[b, m:] = 77
    got = _gpu(cache, q, table, lens, parents, bias, "t5", nodes)
    assert rp.check_status() == 0
    ref, size = _ref(cache, q, table, lens, parents, bias, "t5", nodes)
    _check(got, ref, size, dtype == E4)
    for b, m in enumerate(nodes):
        assert not got[b, :, m if lens[b] > 0 else 0:].any()


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("Hq,n", [(2, 3), (8, 21), (4, 64)])
def test_long_contexts_split_over_blocks(dtype, Hq, n):
    _parity([20011, 97], Hq, 1, n, 64, 128, dtype, "t5", 6)
    _parity([4096], Hq, 1, n, 128, 32, dtype, "none", 7)


def test_many_short_sequences():
    _parity([6 + (37 * b) % 90 for b in range(150)], 2, 2, 6, 64, 32, E4, "alibi", 8)


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("n", [4, 40])
def test_sharp_logits(dtype, n):
    """Keys of larger magnitude: a few keys carry the softmax and the running maximum moves from tile to tile."""
    cache, q, table, lens, bias = _case([1000, 70], 8, 2, n, 64, 64, dtype, "none", 9, 2, 3.0)
    parents = _tree("random", 2, n, 9)
    got = _gpu(cache, q, table, lens, parents, bias, "none")
    _check(got, *_ref(cache, q, table, lens, parents, bias, "none"), dtype == E4)


@pytest.mark.parametrize("nb,md", [(8, 20), (64, 1000), (128, 5000)])
@pytest.mark.parametrize("Hq,n", [(4, 9), (32, 9)])
def test_buckets_and_scale(nb, md, Hq, n):
    cache, q, table, lens, _ = _case([900, 40], Hq, 2, n, 64, 64, E4, "t5", 10)
    bias = torch.randn(nb, Hq, generator=torch.Generator().manual_seed(1))
    parents = _tree("random", 2, n, 10)
    kw = dict(num_buckets=nb, max_distance=md, scale=0.3)
    _check(_gpu(cache, q, table, lens, parents, bias, "t5", **kw), *_ref(cache, q, table, lens, parents, bias, "t5", **kw), True)


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("where", ["k", "v", "v_inf"])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (32, 1, 64), (32, 1, 128)])
def test_nan_of_a_node_stays_on_its_branch(dtype, where, Hq, Hkv, d):
    """A drafted token's NaN or infinity reaches its descendants' rows and no other."""
    if where == "v_inf" and dtype == E4:
        pytest.skip("e4m3 has no infinity")
    n, bad = 12, 3
    cache, q, table, lens, bias = _case([70], Hq, Hkv, n, d, 32, dtype, "none", 12)
    parents = _tree("random", 1, n, 12)
    ref, size = _ref(cache, q, table, lens, parents, bias, "none")
    slot = 70 - n + bad
    p, s = int(table[0, slot // 32]), slot % 32
    t = cache.k if where == "k" else cache.v
    (t.view(torch.uint8) if dtype == E4 else t.view(torch.int16))[p, :, s] = \
        0x7f if dtype == E4 else 0x7f80 if where == "v_inf" else 0x7fc0
    got = _gpu(cache, q, table, lens, parents, bias, "none")
    on = [i for i, line in enumerate(so.tree_lines(parents[0].tolist())) if bad in line]
    off = [i for i in range(n) if i not in on]
    assert len(on) > 1 and len(off) > 1
    _check(got[:, :, off], ref[:, :, off], size[:, :, off], dtype == E4)
    assert (got[:, :, on].isinf() if where == "v_inf" else got[:, :, on].isnan()).all()
    assert rp.check_status() == 0


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("Hq", [2, 32])
def test_a_foul_scale_of_drafted_pages_stays_on_its_branches(value, Hq):
    """The second page holds the last nodes only; nodes of the first page that are nobody's descendants there are clean."""
    n = 10
    cache, q, table, lens, bias = _case([36], Hq, 1, n, 64, 32, E4, "none", 13)  # nodes 0..5 in page 0, 6..9 in page 1
    parents = torch.tensor([[-1, 0, 0, 1, 1, 2, 3, 0, 6, -1]], dtype=torch.int32)
    ref, size = _ref(cache, q, table, lens, parents, bias, "none")
    cache.v_scale[table[0, 1].item()] = value
    got = _gpu(cache, q, table, lens, parents, bias, "none")
    _check(got[:, :, :6], ref[:, :, :6], size[:, :, :6], True)
    assert not got[:, :, 6:].isfinite().any()


@pytest.mark.parametrize("Hq,n", [(2, 5), (16, 30)])
@pytest.mark.parametrize("d", [64, 128])
def test_page_scales_far_apart(Hq, n, d):
    """Values from 2^-25 to 2^15 of one another in the pages of one tile and of one sequence. The weights of small pages
    keep their bits: rows whose keys of large pages are masked away by their logits stay exact."""
    cache, q, table, lens, bias = _case([600], Hq, 1, n, d, 32, E4, "none", 14)
    g = torch.Generator().manual_seed(3)
    e = torch.randint(-25, 16, cache.v_scale.shape, generator=g).float()
    cache.v_scale.copy_(torch.exp2(e).cuda())
    parents = _tree("random", 1, n, 14)
    got = _gpu(cache, q, table, lens, parents, bias, "none")
    _check(got, *_ref(cache, q, table, lens, parents, bias, "none"), True)


@pytest.mark.parametrize("Hq,n", [(2, 5), (16, 30)])
def test_scales_that_are_no_powers_of_two(Hq, n):
    cache, q, table, lens, bias = _case([333, 90], Hq, 1, n, 128, 64, E4, "alibi", 15)
    g = torch.Generator().manual_seed(4)
    for s in (cache.k_scale, cache.v_scale):
        s.copy_((torch.rand(s.shape, generator=g) * 0.05 + 0.01).cuda())
    parents = _tree("random", 2, n, 15)
    got = _gpu(cache, q, table, lens, parents, bias, "alibi")
    _check(got, *_ref(cache, q, table, lens, parents, bias, "alibi"), True)


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (32, 2)])
def test_bad_parents_and_counts_are_reported(dtype, Hq, Hkv):
    cache, q, table, lens, bias = _case([70, 50, 40], Hq, Hkv, 9, 64, 32, dtype, "t5", 16)
    parents = _tree("random", 3, 9, 16)
    broken, meant = parents.clone(), parents.clone()
    for i, a in ((3, 3), (5, 8), (7, -2), (8, 2 ** 31 - 1)):
        broken[0, i], meant[0, i] = a, -1
    got = _gpu(cache, q, table, lens, broken, bias, "t5")
    assert rp.check_status() == rp.RELPOS_ERR_TREE and rp.check_status() == 0
    ref, size = _ref(cache, q, table, lens, meant, bias, "t5")
    _check(got, ref, size, dtype == E4)
    for count in (-1, 10, 2 ** 31 - 1, -2 ** 31):
        got = _gpu(cache, q, table, lens, meant, bias, "t5", [9, count, 9])
        assert rp.check_status() == rp.RELPOS_ERR_TREE and rp.check_status() == 0
        assert not got[1].any()
        _check(got[::2], ref[::2], size[::2], dtype == E4)
    lens[1] = 8  # fewer tokens than nodes
    got = _gpu(cache, q, table, lens, meant, bias, "t5")
    assert rp.check_status() == rp.RELPOS_ERR_TREE and not got[1].any()
    lens[1] = 2 ** 31 - 1
    got = _gpu(cache, q, table, lens, meant, bias, "t5")
    assert rp.check_status() == rp.RELPOS_ERR_PAGE and not got[1].any()
    _check(got[::2], ref[::2], size[::2], dtype == E4)


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("Hq,d", [(2, 64), (24, 64), (24, 128)])
@pytest.mark.parametrize("gone", [(1,), (0, 3), (2, 3), tuple(range(4))])
def test_keys_of_missing_pages_are_left_out(dtype, Hq, d, gone):
    cache, q, table, lens, bias = _case([100, 90], Hq, 1, 6, d, 32, dtype, "alibi", 17)
    parents = _tree("random", 2, 6, 17)
    broken = table.clone()
    for i, p in enumerate(gone):
        broken[0, p] = (-1, cache.num_pages, 2 ** 31 - 1, -2 ** 31)[i % 4]
    got = _gpu(cache, q, broken, lens, parents, bias, "alibi")
    assert rp.check_status() == rp.RELPOS_ERR_PAGE and rp.check_status() == 0
    _check(got, *_ref(cache, q, table, lens, parents, bias, "alibi", gone=gone), dtype == E4)


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("Hq", [4, 32])
def test_strides_alignment_and_a_shared_tree(dtype, Hq):
    n = 10
    cache, q, table, lens, bias = _case([100, 50], Hq, 2, n, 64, 32, dtype, "t5", 18)
    parents = _tree("random", 1, n, 18)[0]
    ref, size = _ref(cache, q, table, lens, parents, bias, "t5")
    wide = torch.zeros(2, n, Hq, 2 * 64 + 1, dtype=BF)
    wide[..., 1:65] = q.transpose(1, 2)
    out = torch.full((2, n, Hq, 2 * 64 + 1), 7.0, dtype=BF, device="cuda")
    x = rp.paged_tree_decode(wide.cuda()[..., 1:65].transpose(1, 2), cache, _table(table, 32), lens.cuda(), parents.cuda(),
                             bias=bias.cuda(), mode=rp.MODE_T5, out=out[..., 65:].transpose(1, 2))
    _check(x, ref, size, dtype == E4)
    assert (out[..., :65] == 7.0).all()


@pytest.mark.parametrize("Hq", [4, 32])
def test_the_same_bits_every_time(Hq):
    cache, q, table, lens, bias = _case([5000, 300, 77], Hq, 2, 20, 128, 64, E4, "t5", 19)
    parents = _tree("random", 3, 20, 19)
    a = _gpu(cache, q, table, lens, parents, bias, "t5")
    for _ in range(3):
        assert torch.equal(a, _gpu(cache, q, table, lens, parents, bias, "t5"))
    # nor on what stands in the slots behind the sequences, or in other sequences
    b = _gpu(cache, q[:1], table[:1], lens[:1], parents[:1], bias, "t5")
    np.testing.assert_allclose(a[:1].double().cpu(), b.double().cpu(), rtol=2.0 ** -6, atol=2.0 ** -9)
