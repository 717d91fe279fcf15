"""Refusals of the tree decode, compaction, page assignment and page copy: host-side checks that answer before anything
reaches the GPU (CPU only)."""
import ctypes
import os

import pytest
import torch

import transformer_attention_relative_gb300 as rp
from test_serving_args import BAD, CACHES, NO, OK, _cache, v
from transformer_attention_relative_gb300 import build as rpbuild


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(rpbuild.LIB_PATH):
        rpbuild.build()
    return rp.load_library()


def _tree(cache=None, **kw):
    a = dict(Q=16, B=2, Hq=4, n=5, table=16, stride=4, pages=4, lens=16, nodes=0, parents=16, up=5, mode=-1, bias=0, nb=32,
             md=128, scale=0.0, out=64, strides=True, row=64)
    a.update(kw)
    s = rp._RowStrides(64, 64, a["row"])
    ref = ctypes.byref(s) if a["strides"] else None
    c = _cache(**(cache or {}))
    return rp.relpos_paged_tree_decode(ctypes.byref(c), v(a["Q"]), ref, a["B"], a["Hq"], a["n"], v(a["table"]), a["stride"],
                                       a["pages"], v(a["lens"]), v(a["nodes"]), v(a["parents"]), a["up"], a["mode"],
                                       v(a["bias"]), a["nb"], a["md"], a["scale"], v(a["out"]), ref, None)


@pytest.mark.parametrize("cache,code", CACHES)
def test_tree_cache(cache, code):
    assert _tree(cache) == code


@pytest.mark.parametrize("kw,code", [
    (dict(mode=1), BAD), (dict(mode=0, bias=16, nb=31), BAD), (dict(mode=0, bias=16, md=16), BAD), (dict(mode=0), BAD),
    (dict(mode=3), BAD), (dict(mode=3, bias=18), BAD), (dict(strides=False), BAD), (dict(B=-1), BAD), (dict(Hq=-2), BAD),
    (dict(n=-1), BAD), (dict(n=65), NO), (dict(Hq=3), BAD), (dict(Q=0), BAD), (dict(out=0), BAD), (dict(Q=17), BAD),
    (dict(lens=0), BAD), (dict(table=0), BAD), (dict(table=18), BAD), (dict(pages=0), BAD), (dict(stride=2), BAD),
    (dict(parents=0), BAD), (dict(parents=18), BAD), (dict(nodes=18), BAD), (dict(up=-1), BAD), (dict(row=63), BAD),
    (dict(row=0), BAD), (dict(scale=float("nan")), BAD), (dict(pages=1 << 24, stride=1 << 24), NO),
    (dict(B=1 << 22, pages=1 << 10, stride=1 << 10), NO),
    (dict(B=0, Q=0, parents=0), OK), (dict(Hq=0, Q=0), OK), (dict(n=0, Q=0, parents=0), OK),
])
def test_tree(kw, code):
    assert _tree(**kw) == code


def test_tree_without_pages_or_heads():
    assert _tree(dict(num_pages=0, k=0)) == BAD and _tree(dict(H=0, k=0)) == BAD


def _compact(cache=None, **kw):
    a = dict(B=2, table=16, stride=4, pages=4, lens=16, nodes=0, n=5, kept=16, ks=3, m=3, counts=0)
    a.update(kw)
    c = _cache(**(cache or {}))
    return rp.relpos_paged_compact(ctypes.byref(c), a["B"], v(a["table"]), a["stride"], a["pages"], v(a["lens"]), v(a["nodes"]),
                                   a["n"], v(a["kept"]), a["ks"], a["m"], v(a["counts"]), None)


@pytest.mark.parametrize("cache,code", CACHES)
def test_compact_cache(cache, code):
    assert _compact(cache) == code


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), BAD), (dict(n=-1), BAD), (dict(m=-1), BAD), (dict(pages=-1), BAD), (dict(table=0), BAD), (dict(lens=0), BAD),
    (dict(kept=0), BAD), (dict(kept=17), BAD), (dict(nodes=18), BAD), (dict(counts=18), BAD), (dict(stride=3), BAD),
    (dict(ks=2), BAD), (dict(pages=0), BAD), (dict(m=65, ks=65), NO), (dict(B=65536), NO),
    (dict(pages=1 << 24, stride=1 << 24), NO), (dict(B=0, kept=0), OK), (dict(m=0, kept=0), OK),
])
def test_compact(kw, code):
    assert _compact(**kw) == code


def test_compact_pool_sizes():
    assert _compact(dict(num_pages=1 << 27)) == NO and _compact(dict(num_pages=0, k=0)) == BAD
    assert _compact(dict(H=0, k=0)) == OK


def _assign(**kw):
    a = dict(refs=16, P=9, page=32, table=32, stride=4, pages=4, lens=16, B=2, source=16, new=16, B2=3, to=64, ts=4, width=4,
             nr=16, copies=16)
    a.update(kw)
    return rp.relpos_paged_assign(v(a["refs"]), a["P"], a["page"], v(a["table"]), a["stride"], a["pages"], v(a["lens"]), a["B"],
                                  v(a["source"]), v(a["new"]), a["B2"], v(a["to"]), a["ts"], a["width"], v(a["nr"]),
                                  v(a["copies"]), None)


@pytest.mark.parametrize("kw,code", [
    (dict(P=-1), BAD), (dict(B=-1), BAD), (dict(B2=-1), BAD), (dict(pages=-1), BAD), (dict(width=-1), BAD), (dict(page=0), BAD),
    (dict(page=48), NO), (dict(page=256), NO), (dict(refs=0), BAD), (dict(nr=0), BAD), (dict(lens=0), BAD), (dict(table=0), BAD),
    (dict(new=0), BAD), (dict(copies=0), BAD), (dict(to=0), BAD), (dict(to=32), BAD), (dict(refs=18), BAD), (dict(source=18), BAD),
    (dict(copies=18), BAD), (dict(stride=3), BAD), (dict(ts=3), BAD), (dict(B2=8193), NO),
    (dict(width=1 << 24, ts=1 << 24), NO), (dict(B=1 << 20, pages=1 << 12, stride=1 << 12), NO),
    (dict(P=0, refs=0, nr=0, B2=0, new=0, copies=0, to=0), OK),
])
def test_assign(kw, code):
    assert _assign(**kw) == code


def _copy(cache=None, copies=16, N=3):
    return rp.relpos_paged_copy(ctypes.byref(_cache(**(cache or {}))), v(copies), N, None)


@pytest.mark.parametrize("cache,code", CACHES)
def test_copy_cache(cache, code):
    assert _copy(cache) == code


def test_copy():
    assert _copy(copies=0) == BAD and _copy(copies=18) == BAD and _copy(N=-1) == BAD and _copy(N=1 << 30) == NO
    assert _copy(copies=0, N=0) == OK and _copy(dict(H=0, k=0), 0) == OK and _copy(dict(num_pages=0, k=0), 0) == OK


class _Handle:
    heads, head_dim, page_size, num_pages, _index = 2, 64, 32, 4, 0


def test_python_refuses_wrong_shapes_and_types():
    c, i = _Handle(), torch.int32
    q, table, lens, up = torch.zeros(2, 4, 5, 64).bfloat16(), torch.zeros(2, 3, dtype=i), torch.zeros(2, dtype=i), torch.zeros(2, 5, dtype=i)
    for bad in (dict(Q=q.float()), dict(parents=up.long()), dict(out=q.float())):
        with pytest.raises(TypeError):
            rp.paged_tree_decode(**{**dict(Q=q, cache=c, block_table=table, lens=lens, parents=up), **bad})
    for bad in (dict(Q=q[..., :32]), dict(parents=up[:1]), dict(parents=up[:, :4]), dict(parents=up.t().contiguous().t()),
                dict(lens=lens[:1]), dict(out=q[:1]), dict(block_table=table[:1]), dict(Q=q.transpose(2, 3)), dict()):
        with pytest.raises(ValueError):  # the last one: host tensors
            rp.paged_tree_decode(**{**dict(Q=q, cache=c, block_table=table, lens=lens, parents=up), **bad})
    kept = torch.zeros(2, 3, dtype=i)
    with pytest.raises(TypeError):
        rp.paged_compact(c, table, lens, kept.long(), 5)
    for bad in (dict(n=-1), dict(lens=lens[:1]), dict(kept=kept[:1]), dict(kept=kept.t().contiguous().t()), dict()):
        with pytest.raises(ValueError):
            rp.paged_compact(**{**dict(cache=c, block_table=table, lens=lens, kept=kept, n=5), **bad})
    refs = torch.zeros(9, dtype=i)
    for bad in (dict(refs=refs.long()), dict(new_lens=lens.long()), dict(block_table=table.long())):
        with pytest.raises(TypeError):
            rp.paged_assign(**{**dict(refs=refs, block_table=table, lens=lens, new_lens=lens, page_size=32), **bad})
    for bad in (dict(refs=refs[::2]), dict(lens=lens[:1]), dict(new_lens=lens[:1]), dict(max_pages=-1), dict()):
        with pytest.raises(ValueError):
            rp.paged_assign(**{**dict(refs=refs, block_table=table, lens=lens, new_lens=lens, page_size=32), **bad})
    with pytest.raises(TypeError):
        rp.paged_copy(c, torch.zeros(2, 3))
    for bad in (torch.zeros(2, 4, dtype=i), torch.zeros(6, dtype=i), torch.zeros(2, 3, dtype=i)):
        with pytest.raises(ValueError):
            rp.paged_copy(c, bad)
