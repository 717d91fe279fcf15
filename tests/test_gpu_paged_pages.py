"""Keeping drafted tokens, giving out pages and copying them vs the oracle: all of it exact. And the operators together:
steps of speculative decoding and of beam search over a paged cache."""
import numpy as np
import pytest
import torch

import gpu_util as G
import transformer_attention_relative_gb300 as rp
from oracle import serving_oracle as so
from test_gpu_paged_tree import _tree, _values

pytestmark = pytest.mark.gpu
BF, E4 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def _cache(pages, H, page, d, dtype, seed, pow2=True, spread=4):
    g = torch.Generator().manual_seed(seed)
    shape = (pages, H, page, d)
    if dtype == BF:
        return rp.PagedCache(*(torch.randn(shape, generator=g).to(BF).cuda() for _ in range(2)))
    codes = [(torch.randn(shape, generator=g) * 60).clamp(-448, 448).to(E4).cuda() for _ in range(2)]
    scales = [torch.exp2(torch.randint(-spread, spread, shape[:2], generator=g).float()) for _ in range(2)]
    if not pow2:
        scales = [s * (1 + torch.rand(s.shape, generator=g)) for s in scales]
    return rp.PagedCache(*codes, *(s.cuda() for s in scales))


def _table(lens, page, pages, seed, width=None):
    counts = [-(-n // page) for n in lens]
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
    t = torch.full((len(lens), width or max(max(counts), 1)), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts):
        t[b, :c] = order[at:at + c]
        at += c
    return t


def _same(cache, want):
    for name, x in _values(cache).items():
        np.testing.assert_array_equal(x, want[name], err_msg=name)


def _bytes(cache):
    return [t.clone().view(torch.uint8) for t in (cache.k, cache.v, cache.k_scale, cache.v_scale) if t is not None]


# ------------------------------------------------------------------ compact

@pytest.mark.parametrize("dtype,pow2", [(BF, True), (E4, True), (E4, False)])
@pytest.mark.parametrize("page,d", [(32, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("n,m", [(1, 1), (7, 3), (40, 40), (64, 64), (200, 64)])
def test_compact(dtype, pow2, page, d, n, m):
    """Trees that begin anywhere in a page, nodes kept in any order and more than once."""
    lens = [n, n + 5, n + 31, n + 100]
    pages = sum(-(-x // page) for x in lens) + 2
    cache = _cache(pages, 3, page, d, dtype, n, pow2)
    table = _table(lens, page, pages, n)
    g = torch.Generator().manual_seed(m)
    kept = torch.randint(0, n, (4, m), generator=g, dtype=torch.int32)
    counts = [m, m // 2, 0, (m + 1) // 2]
    want = so.paged_compact(_values(cache), table.numpy(), lens, [n] * 4, kept.tolist(), counts, page)
    rp.paged_compact(cache, table.cuda(), _i32(lens), kept.cuda(), n, counts=_i32(counts))
    assert rp.check_status() == 0
    _same(cache, want)


@pytest.mark.parametrize("dtype", [BF, E4])
def test_compact_with_counts_of_their_own(dtype):
    """Numbers of nodes of each sequence, kept rows with a stride, all of them kept by default; empty sequences."""
    lens, nodes = [50, 0, 33, 20], [9, 4, 33, 2]
    cache = _cache(9, 2, 32, 64, dtype, 1)
    table = _table(lens, 32, 9, 1, 3)
    kept = torch.full((4, 10), 99, dtype=torch.int32)
    kept[:, :5] = torch.tensor([0, 3, 1, 8, 4])
    kept[3, :2] = torch.tensor([1, 0])
    want = so.paged_compact(_values(cache), table.numpy(), lens, nodes, kept.tolist(), [5, 0, 5, 2], 32)
    rp.paged_compact(cache, table.cuda(), _i32(lens), kept.cuda()[:, :5], _i32(nodes))
    assert rp.check_status() == 0
    _same(cache, want)


def test_compact_foul_scales():
    """NaN in a page's scale or codes goes with the tokens that have it; a page never takes a NaN for its scale."""
    cache = _cache(2, 1, 32, 64, E4, 2)
    table = _i32([[0, 1]])
    cache.v_scale.copy_(torch.tensor([[0.5], [float("nan")]]))
    cache.k.view(torch.uint8)[1, 0, 3] = 0x7f
    cache.k_scale.copy_(torch.tensor([[0.25], [2.0]]))
    rp.paged_compact(cache, table, _i32([38]), _i32([[9, 0]]), 10)  # slot 28 <- 37, slot 29 <- 28
    assert rp.check_status() == 0
    v = cache.v.double().cpu() * cache.v_scale.double().cpu()[..., None, None]
    assert v[0, 0, 28].isnan().all() and v[0, 0, :28].isfinite().all() and v[0, 0, 29:].isfinite().all()
    assert cache.v_scale[0].item() == 0.5 and cache.k_scale[0].item() == 2.0
    rp.paged_compact(cache, table, _i32([38]), _i32([[0, 7]]), 10)  # slot 29 <- 35, whose key is NaN
    assert cache.k[0, 0, 29].float().isnan().all() and cache.k[0, 0, :29].float().isfinite().all()


def test_compact_reports_what_is_outside():
    lens = [50, 40, 60]
    cache = _cache(8, 2, 32, 64, BF, 3)
    table = _table(lens, 32, 8, 3, 2)
    kept = torch.tensor([[4, 10, -1, 2 ** 31 - 1, 2]] * 3, dtype=torch.int32)  # of 9 nodes
    meant = [[4, 1, 2, 3, 2]] * 3
    want = so.paged_compact(_values(cache), table.numpy(), lens, [9] * 3, meant, [5] * 3, 32)
    rp.paged_compact(cache, table.cuda(), _i32(lens), kept.cuda(), 9)
    assert rp.check_status() == rp.RELPOS_ERR_TREE and rp.check_status() == 0
    _same(cache, want)
    was = _bytes(cache)
    for kw, args in ((dict(counts=_i32([6, -1, 2 ** 31 - 1])), 9), ({}, _i32([51, -1, 2 ** 31 - 1]))):
        rp.paged_compact(cache, table.cuda(), _i32(lens), kept.cuda(), args, **kw)
        assert rp.check_status() == rp.RELPOS_ERR_TREE
    rp.paged_compact(cache, table.cuda(), _i32([65, 2 ** 31 - 1, -2 ** 31]), kept.cuda(), 9)
    assert rp.check_status() == rp.RELPOS_ERR_PAGE
    # pages that are none: neither written nor read
    broken = table.clone()
    broken[:, 1] = torch.tensor([-1, 8, 2 ** 31 - 1], dtype=torch.int32)
    rp.paged_compact(cache, broken.cuda(), _i32(lens), _i32([[4, 3]] * 3), 9)
    assert rp.check_status() == rp.RELPOS_ERR_PAGE
    for b in (0, 2):  # drafted slots 41 .. and 51 .. lie in the second page alone; 31 of sequence 1 in the first
        for x, y in zip(was, _bytes(cache)):
            for p in table[b].tolist():
                assert torch.equal(x[p], y[p])


# ------------------------------------------------------------------ assign

def _assign(refs, table, lens, source, new_lens, page, width=None):
    width = width or table.shape[1]
    new, left, copies = rp.paged_assign(_i32(refs), table.cuda(), _i32(lens), _i32(new_lens), page,
                                        source=None if source is None else _i32(source), max_pages=width)
    src = list(range(len(lens))) if source is None else source
    want = so.paged_assign(refs, table.tolist(), lens, src, new_lens, page, width)
    assert new.tolist() == want[0]
    assert left.tolist() == want[1]
    assert [tuple(c) for c in copies.tolist()] == want[2]
    return new, left, copies


def _refs(table, lens, page, pages, outside=()):
    refs = [0] * pages
    for row, n in zip(table.tolist(), lens):
        for p in row[:-(-n // page)]:
            refs[p] += 1
    for p in outside:
        refs[p] += 1
    return refs


@pytest.mark.parametrize("page", [32, 64, 128])
@pytest.mark.parametrize("seed", range(8))
def test_assign(page, seed):
    """Sequences that share pages, take new parents, grow, shrink, begin and end; pages held elsewhere; several calls one
    after another."""
    r = np.random.default_rng(seed)
    B = int(r.integers(1, 60))
    pages = int(r.integers(1500, 5000))
    lens = [int(r.integers(0, 6 * page)) for _ in range(B)]
    table = _table(lens, page, pages, seed, 12)
    refs = _refs(table, lens, page, pages, r.integers(0, pages, 5))
    for _ in range(4):
        B2 = int(r.integers(1, 60))
        source = [int(s) for s in r.integers(-1, len(lens), B2)]
        new_lens = [int(min(12 * page, max(-3, (lens[s] if s >= 0 else 0) + r.integers(-2 * page, 3 * page)))) for s in source]
        new_lens = [n if r.random() > 0.1 else 0 for n in new_lens]
        new_lens = [max(n, 0) for n in new_lens]
        new, left, _ = _assign(refs, table, lens, source, new_lens, page)
        assert rp.check_status() == 0
        table, refs, lens = new.cpu(), left.tolist(), new_lens


@pytest.mark.parametrize("B,pages", [(1, 1), (1, 31), (2000, 70001), (8192, 100000)])
def test_assign_sizes(B, pages):
    """One row and one page, and more of both than the cluster has threads."""
    lens = [(7 * b) % 300 + 1 if pages > 31 else 20 for b in range(B)]
    table = _table(lens, 64, pages, 1, 6)
    refs = _refs(table, lens, 64, pages)
    _assign(refs, table, lens, None, [n + 1 + (b % 64) for b, n in enumerate(lens)], 64)
    _assign(refs, table, lens, [b // 4 * 4 for b in range(B)], lens, 64)
    assert rp.check_status() == 0
    _assign(refs, table, lens, None, [0] * B, 64, 1)


def test_assign_new_sequences_alone_and_no_rows():
    none = torch.empty(0, 4, dtype=torch.int32)
    new, left, copies = _assign([1, 0, 2, 0, 0], none, [], [-1, -1], [33, 1], 32, 4)
    assert new.tolist() == [[1, 3, -1, -1], [4, -1, -1, -1]]
    new, left, copies = rp.paged_assign(left, new, _i32([33, 1]), _i32([]), 32, source=_i32([]))
    assert left.tolist() == [1, 0, 2, 0, 0] and new.shape == (0, 4) and copies.shape == (0, 3)
    assert rp.check_status() == 0


def test_assign_too_few_pages():
    """Requests in order as long as there are pages; the rest is -1, copies too, and reported."""
    table = torch.tensor([[2, 0], [3, -1]], dtype=torch.int32)
    _assign([1, 0, 1, 1, 1], table, [40, 20], [0, 0, 1, 1], [80, 80, 20, 64], 32, 4)
    assert rp.check_status() == rp.RELPOS_ERR_PAGE and rp.check_status() == 0


def test_assign_reports_what_is_outside():
    table = torch.tensor([[2, 9], [-4, 1], [0, 1]], dtype=torch.int32)
    refs = _i32([1, 1, 1, 0, 0])
    new, left, copies = rp.paged_assign(refs, table.cuda(), _i32([40, 40, 65]), _i32([41, 64, 70, 10, 30]), 32,
                                        source=_i32([0, 1, 0, 5, -2]))
    assert rp.check_status() == rp.RELPOS_ERR_PAGE and rp.check_status() == 0
    # row 0: page 2 and, for 9, a fresh one without a copy; row 1: -1 shared as it is, its last page kept; row 2 does not
    # fit its table; rows 3 and 4 are new. Old row 2 does not fit: page 0's reference stays.
    assert new.tolist() == [[2, 3], [-1, 1], [-1, -1], [4, -1], [-1, -1]]
    assert left.tolist() == [1, 1, 1, 1, 1]
    assert (copies == -1).all()
    # a count below the rows that refer to a page, and a negative one: never below nothing
    new, left, copies = rp.paged_assign(_i32([1, -5, 0]), _i32([[0, 1], [0, 2]]), _i32([64, 64]), _i32([0, 0]), 32)
    assert rp.check_status() == rp.RELPOS_ERR_PAGE and left.tolist() == [0, 0, 0]


def test_assign_in_place_and_strided():
    lens = [100, 30, 64]
    table = _table(lens, 32, 40, 5, 9)
    refs = _refs(table, lens, 32, 40)
    want = so.paged_assign(refs, table.tolist(), lens, [2, 2, 0], [65, 70, 129], 32, 9)
    wide = torch.full((3, 20), 5, dtype=torch.int32)
    wide[:, 3:12] = table
    r, out, copies = _i32(refs), torch.full((3, 12), 7, dtype=torch.int32, device="cuda"), torch.empty(3, 3, dtype=torch.int32, device="cuda")
    t, w, s, n = wide.cuda(), _i32(lens), _i32([2, 2, 0]), _i32([65, 70, 129])
    rc = rp.relpos_paged_assign(r.data_ptr(), 40, 32, t[:, 3:].data_ptr(), 20, 9, w.data_ptr(), 3, s.data_ptr(), n.data_ptr(), 3,
                                out.data_ptr(), 12, 9, r.data_ptr(), copies.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and rp.check_status() == 0
    assert out[:, :9].tolist() == want[0] and (out[:, 9:] == 7).all()
    assert r.tolist() == want[1] and [tuple(c) for c in copies.tolist()] == want[2]


# ------------------------------------------------------------------ copy

@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("page,H,d", [(32, 1, 64), (64, 5, 128), (128, 16, 64)])
def test_copy(dtype, page, H, d):
    cache = _cache(20, H, page, d, dtype, 6)
    copies = [(3, 4, page), (-1, -1, -1), (5, 6, 1), (3, 7, page - 1), (8, 9, 0), (-1, 2, 5), (10, 10, 3), (11, 12, 17)]
    want = _values(cache)
    for f, t, n in copies:
        if f >= 0 and n > 0 and f != t:
            for x in ("k", "v"):
                want[x][t, :, :n] = want[x][f, :, :n]
                if dtype == E4:
                    want[x + "_scale"][t] = want[x + "_scale"][f]
    rp.paged_copy(cache, _i32(copies))
    assert rp.check_status() == 0
    _same(cache, want)
    was = _bytes(cache)
    for bad in ((20, 1, 2), (1, 20, 2), (-2, 1, 2), (1, -1, 2), (1, 2, -1), (1, 2, page + 1), (2 ** 31 - 1, 0, 1)):
        rp.paged_copy(cache, _i32([bad]))
        assert rp.check_status() == rp.RELPOS_ERR_PAGE
    assert all(torch.equal(x, y) for x, y in zip(was, _bytes(cache)))


def test_copy_past_4_gb():
    """Byte offsets beyond 32 bits."""
    cache = rp.PagedCache.empty(5000, 32, 128, page_size=128)
    cache.k[4998] = torch.randn(32, 128, 128, device="cuda").to(BF)
    cache.v[4998] = 3.0
    rp.paged_copy(cache, _i32([(4998, 4999, 100), (4998, 0, 128)]))
    for x in (cache.k, cache.v):
        assert torch.equal(x[4999, :, :100], x[4998, :, :100]) and not x[4999, :, 100:].any()
        assert torch.equal(x[0], x[4998]) and not x[1:4998:501].any()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", [BF, E4])
def test_speculative_decoding(dtype):
    """Prompt, then steps of: pages for the drafts, append the tree (keys turned at its positions), attention of its
    nodes, keep a branch, forget the rest. Each step's attention is that of each branch's tokens as a sequence of its own;
    in 8 bits the values of the codes that the cache holds count, within the tolerance of the tree's attention."""
    B, Hq, Hkv, d, page, n = 3, 4, 2, 64, 32, 12
    g = torch.Generator().manual_seed(7)
    plan = rp.RotaryPlan(64)
    cache = rp.PagedCache.empty(60, Hkv, d, page_size=page, dtype=dtype)
    refs, table, lens = _i32([0] * 60), torch.full((B, 12), -1, dtype=torch.int32, device="cuda"), _i32([0] * B)
    prompt = _i32([40, 63, 5])
    table, refs, _ = rp.paged_assign(refs, table, lens, prompt, page)
    rows = [torch.randn(B, Hkv, 63, d, generator=g).to(BF).cuda() for _ in range(2)]
    for b in range(B):  # ragged prompts one by one
        m = int(prompt[b])
        rp.paged_append(cache, rows[0][b:b + 1, :, :m], rows[1][b:b + 1, :, :m], table[b:b + 1], prompt[b:b + 1], plan=plan)
    held, lens = prompt.clone(), prompt.clone()
    # what each sequence's tokens are, exactly: 16 bits only
    dense = [[[], []] for _ in range(B)]
    for b in range(B):
        for x, y in zip(dense[b], (rp.rotary(rows[0], plan)[b], rows[1][b])):
            x.extend(y[:, j].double().cpu().numpy() for j in range(int(prompt[b])))
    for step in range(5):
        total = lens + n
        table, refs, copies = rp.paged_assign(refs, table, held, total, page)
        assert (copies == -1).all()
        held = total
        parents = _tree("random", B, n, 100 + step)
        depth = torch.tensor([[len(x) - 1 for x in so.tree_lines(p)] for p in parents.tolist()])
        k, v = (torch.randn(B, Hkv, n, d, generator=g).to(BF).cuda() for _ in range(2))
        q = torch.randn(B, Hq, n, d, generator=g).to(BF).cuda()
        place = (lens.cpu()[:, None] + depth).to(torch.int32).cuda()
        q, k = rp.rotary(q, plan, k, positions=place)
        rp.paged_append(cache, k, v, table, total)
        got = rp.paged_tree_decode(q, cache, table, total, parents.cuda())
        ref, size = so.paged_tree_decode(q.double().cpu().numpy(), _values(cache), table.cpu().numpy(), total.tolist(), page,
                                         parents.tolist())
        eight = dtype == E4
        tol = 2.0 ** -8 * np.abs(ref) + size * ((2.0 ** -11 if eight else 2.0 ** -16) + 2.0 ** -12)
        assert np.all(np.abs(got.double().cpu().numpy() - ref) <= tol)
        kept, counts = torch.zeros(B, n, dtype=torch.int32), []
        for b in range(B):
            lines = so.tree_lines(parents[b].tolist())
            line = max(lines, key=len) if step % 2 else lines[-1]
            kept[b, :len(line)] = torch.tensor(line)
            counts.append(len(line))
            for x, y in zip(dense[b], (k, v)):
                x.extend(y[b, :, j].double().cpu().numpy() for j in line)
        counts = _i32(counts)
        rp.paged_compact(cache, table, total, kept.cuda(), n, counts=counts)
        lens = lens + counts
        if dtype == BF:
            values = _values(cache)
            for b in range(B):
                pages = table[b, :-(-int(lens[b]) // page)].tolist()
                for name, x in zip("kv", dense[b]):
                    now = np.concatenate([values[name][p] for p in pages], 1)[:, :int(lens[b])]
                    np.testing.assert_array_equal(now, np.stack(x, 1))
    table, refs, _ = rp.paged_assign(refs, table, held, _i32([0] * B), page)
    assert not refs.any() and rp.check_status() == 0


@pytest.mark.parametrize("dtype", [BF, E4])
def test_beam_search(dtype):
    """Beams over shared pages: each step takes new parents, copies the pages that two beams would write, appends a token
    and attends; every beam stays the sequence that its history says."""
    W, H, d, page, layers = 6, 2, 64, 32, 2
    g = torch.Generator().manual_seed(8)
    caches = [rp.PagedCache.empty(80, H, d, page_size=page, dtype=dtype) for _ in range(layers)]
    refs, table = _i32([0] * 80), torch.full((1, 8), -1, dtype=torch.int32, device="cuda")
    table, refs, _ = rp.paged_assign(refs, table, _i32([0]), _i32([70]), page)
    hist = [[[(c, j) for j in range(70)] for _ in range(W)] for c in range(layers)]
    tokens = {}
    for c, cache in enumerate(caches):
        k, v = (torch.randn(1, H, 70, d, generator=g).to(BF).cuda() for _ in range(2))
        rp.paged_append(cache, k, v, table, _i32([70]))
        for j in range(70):
            tokens[c, j] = (k[0, :, j], v[0, :, j])
    lens, fresh = _i32([70]), 1000
    for step in range(45):
        source = [0] * W if step == 0 else [int(s) for s in torch.randint(0, W, (W,), generator=g)]
        new = lens[_i32(source).long()] + 1
        table, refs, copies = rp.paged_assign(refs, table, lens, new, page, source=_i32(source))
        lens = new
        for c, cache in enumerate(caches):
            rp.paged_copy(cache, copies)
            k, v, q = (torch.randn(W, H, 1, d, generator=g).to(BF).cuda() for _ in range(3))
            rp.paged_append(cache, k, v, table, lens)
            hist[c] = [hist[c][s] + [(c, fresh + w)] for w, s in enumerate(source)]
            for w in range(W):
                tokens[c, fresh + w] = (k[w, :, 0], v[w, :, 0])
            if step % 15 == 14:
                got = rp.paged_decode(q, cache, table, lens).double().cpu()
                if dtype == E4:  # the values of the codes in the cache
                    ref, size = so.paged_decode(q.double().cpu().numpy(), _values(cache), table.cpu().numpy(), lens.tolist(), page)
                    tol = 2.0 ** -8 * np.abs(ref) + size * (2.0 ** -11 + 2.0 ** -12)
                    assert np.all(np.abs(got.numpy() - ref) <= tol)
                values = _values(cache)
                for w in range(W):
                    kk, vv = (torch.stack([tokens[t][i] for t in hist[c][w]], 1).double().cpu() for i in range(2))
                    if dtype == BF:
                        p = torch.softmax(q[w].double().cpu() @ kk.transpose(1, 2) / 8.0, -1)
                        want, size = (p @ vv)[:, 0], (p @ vv.abs())[:, 0]
                        assert ((got[w, :, 0] - want).abs() <= 2.0 ** -8 * want.abs() + size * 2.0 ** -12).all()
                        continue
                    # half a step of e4m3 for each rounding: to its page's scale when appended, and each time it grew (to
                    # twice at most three times here: the largest of 32 x 64 normal values lies within 2 .. 8)
                    for name, x in (("k", kk), ("v", vv)):
                        at = table[w, :-(-x.shape[1] // page)].tolist()
                        now = np.concatenate([values[name][i] * values[name + "_scale"][i][:, None, None] for i in at], 1)
                        now = torch.from_numpy(now[:, :x.shape[1]])
                        assert ((now - x).abs() <= 4 * (2.0 ** -4 * x.abs() + 2.0 ** -10 * 2.0 ** -5)).all()
        fresh += W
    alive = sorted(p for p, r in enumerate(refs.tolist()) if r)
    assert alive == sorted({p for row, n in zip(table.tolist(), lens.tolist()) for p in row[:-(-n // page)]})
    assert rp.check_status() == 0
