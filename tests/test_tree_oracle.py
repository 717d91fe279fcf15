"""Pins of the oracle's tree decode, compaction and page assignment (CPU)."""
import numpy as np
import pytest

from oracle import serving_oracle as so


def _cache(B, lens, page, H, d, seed):
    r = np.random.default_rng(seed)
    counts = [-(-n // page) for n in lens]
    order = r.permutation(sum(counts) + 2)
    table, at = -np.ones((B, max(counts) + 1), dtype=int), 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    shape = (len(order), H, page, d)
    return {"k": r.standard_normal(shape), "v": r.standard_normal(shape)}, table, r


@pytest.mark.parametrize("mode", ["none", "t5", "alibi"])
def test_a_chain_is_a_plain_decode(mode):
    lens, n = [40, 9, 4], 4
    cache, table, r = _cache(3, lens, 8, 2, 16, 1)
    q = r.standard_normal((3, 4, n, 16))
    bias = r.standard_normal((32, 4)) if mode == "t5" else r.random(4)
    a = so.paged_tree_decode(q, cache, table, lens, 8, [list(range(-1, n - 1))] * 3, bias=bias, mode=mode)
    b = so.paged_decode(q, cache, table, lens, 8, bias, mode)
    np.testing.assert_allclose(a[0], b[0], rtol=1e-12)
    np.testing.assert_allclose(a[1], b[1], rtol=1e-12)


@pytest.mark.parametrize("mode", ["none", "t5", "alibi"])
def test_each_branch_is_a_sequence_of_its_own(mode):
    """Row i of a tree is the last row of a sequence that holds the context and the line of node i."""
    parents, base, page, d = [-1, 0, 0, 1, -1, 3], 21, 8, 16
    n = len(parents)
    cache, table, r = _cache(2, [base + n, base + n], page, 2, d, 2)
    q = r.standard_normal((1, 4, n, d))
    bias = r.standard_normal((32, 4)) if mode == "t5" else r.random(4)
    got, _ = so.paged_tree_decode(q, cache, table[:1], [base + n], page, [parents], bias=bias, mode=mode)
    rows = {x: np.concatenate([cache[x][p] for p in table[0, :4]], 1)[:, :base + n] for x in "kv"}  # [H, tokens, d]
    for i, line in enumerate(so.tree_lines(parents)):
        for x in "kv":
            flat = np.concatenate([rows[x][:, :base], rows[x][:, [base + j for j in line]]], 1)
            for s in range(flat.shape[1]):
                cache[x][table[1, s // page], :, s % page] = flat[:, s]
        want, _ = so.paged_decode(q[:, :, i:i + 1], cache, table[1:], [base + len(line)], page, bias, mode)
        np.testing.assert_allclose(got[0, :, i], want[0, :, 0], rtol=1e-12)


def test_kept_nodes_are_their_line():
    """Attention of a chain over what is kept equals that of its nodes in the tree."""
    parents, base, page = [-1, 0, 0, 2, 2, 4], 13, 8
    cache, table, r = _cache(1, [base + 6], page, 1, 8, 3)
    q = r.standard_normal((1, 1, 6, 8))
    want, _ = so.paged_tree_decode(q, cache, table, [base + 6], page, [parents])
    line = [0, 2, 4, 5]
    so.paged_compact(cache, table, [base + 6], [6], [line], [4], page)
    got, _ = so.paged_decode(q[:, :, line], cache, table, [base + 4], page)
    np.testing.assert_allclose(got, want[:, :, line], rtol=1e-12)


def test_assign_by_hand():
    # two beams share page 5, their last pages are 2 and 7; page 5 is held elsewhere too
    refs = [0, 0, 1, 0, 0, 3, 0, 1]
    table = [[5, 2], [5, 7]]
    new, left, copies = so.paged_assign(refs, table, [12, 11], [1, 1, 0, -1], [12, 12, 0, 3], 8, 3)
    assert new == [[5, 7, -1], [5, 0, -1], [-1, -1, -1], [1, -1, -1]]
    assert left == [1, 1, 0, 0, 0, 3, 0, 1] and copies == [(-1,) * 3, (7, 0, 3), (-1,) * 3, (-1,) * 3]
    # growing over a page's end and shrinking, nothing free but what was given up
    new, left, copies = so.paged_assign([1, 1, 1, 1], [[3, 1], [0, 2]], [16, 9], [0, 1], [17, 8], 8, 3)
    assert new == [[3, 1, 2], [0, -1, -1]] and left == [1, 1, 1, 1]
    assert so.paged_assign([1], [[0]], [3], [0, 0], [4, 4], 8, 1) == ([[0], [-1]], [1], [(-1,) * 3] * 2)
