"""Refusals of the rotary and paged-cache entry points: host-side checks that
answer before anything reaches the GPU (CPU only)."""
import ctypes
import os

import pytest
import torch

import transformer_attention_relative_gb300 as rp
from transformer_attention_relative_gb300 import build as rpbuild

BAD, NO, OK = rp.RELPOS_ERR_INVALID_ARG, rp.RELPOS_ERR_UNSUPPORTED, rp.RELPOS_OK


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(rpbuild.LIB_PATH):
        rpbuild.build()
    return rp.load_library()


def v(x):
    return ctypes.c_void_p(x) if x else None


@pytest.mark.parametrize("kw,code", [
    (dict(), OK),
    (dict(rot=63), BAD), (dict(rot=0), BAD), (dict(rot=258), BAD), (dict(rot=256), OK),
    (dict(layout=2), BAD), (dict(base=1.0), BAD), (dict(base=float("nan")), BAD), (dict(base=float("inf")), BAD),
    (dict(scaling=4), BAD), (dict(scaling=-1), BAD),
    (dict(scaling=1, factor=0.5), BAD), (dict(scaling=1, factor=float("nan")), BAD), (dict(scaling=0, factor=0.0), OK),
    (dict(scaling=2, factor=4.0, rot=2), BAD),
    (dict(scaling=3, factor=4.0), BAD), (dict(scaling=3, factor=4.0, olen=4096.0), OK),
    (dict(scaling=3, factor=4.0, olen=4096.0, fast=1.0, slow=1.0), BAD),
    (dict(scaling=3, factor=4.0, olen=float("inf")), BAD),
])
def test_plan(kw, code):
    a = dict(rot=64, layout=0, base=1e4, scaling=0, factor=1.0, olen=0.0, fast=32.0, slow=1.0)
    a.update(kw)
    plan = rp._RotaryPlan()
    assert rp.relpos_rotary_plan_init(ctypes.byref(plan), a["rot"], a["layout"], a["base"], a["scaling"], a["factor"],
                                      a["olen"], a["fast"], a["slow"]) == code
    assert rp.relpos_rotary_plan_init(None, 64, 0, 1e4, 0, 1.0, 0.0, 32.0, 1.0) == BAD


def test_plan_in_python():
    with pytest.raises(ValueError):
        rp.RotaryPlan(64, layout="thirds")
    with pytest.raises(ValueError):
        rp.RotaryPlan(64, scaling="more")
    with pytest.raises(rp.RelposError) as e:
        rp.RotaryPlan(63)
    assert e.value.code == BAD


def _rotary(**kw):
    a = dict(plan=rp.RotaryPlan(64)._ref, dtype=0, inverse=0, n=1, B=1, L=2, d=64, x=16, out=32, H=2, sl=64, pos=0,
             offset=0, ten=True)
    a.update(kw)
    t = (rp._RotaryTensor * 2)()
    for e in t:
        e.x, e.out, e.H = a["x"] or None, a["out"] or None, a["H"]
        e.x_row = e.out_row = a["sl"]
    return rp.relpos_rotary(a["plan"], a["dtype"], a["inverse"], t if a["ten"] else None, a["n"], a["B"], a["L"],
                            a["d"], v(a["pos"]), 0, a["offset"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(plan=None), BAD), (dict(plan=ctypes.byref(rp._RotaryPlan())), BAD),  # a plan that was never filled
    (dict(dtype=2), BAD), (dict(inverse=2), BAD), (dict(n=0), BAD), (dict(n=3), BAD), (dict(ten=False), BAD),
    (dict(B=-1), BAD), (dict(L=-1), BAD), (dict(d=62), BAD), (dict(d=65), BAD), (dict(H=-1), BAD), (dict(H=70000), NO),
    (dict(x=0), BAD), (dict(out=0), BAD), (dict(x=17), BAD), (dict(dtype=1, x=18), BAD), (dict(pos=2), BAD),
    (dict(offset=0x7fffffff), BAD), (dict(B=1 << 20, L=1 << 20), NO),
    (dict(B=0, x=0), OK), (dict(L=0, x=0), OK), (dict(H=0, x=0), OK),
])
def test_rotary(kw, code):
    assert _rotary(**kw) == code


def _cache(**kw):
    a = dict(k=16, v=32, ks=48, vs=64, num_pages=4, H=2, page=32, d=64, dtype=2)
    a.update(kw)
    return rp._PagedCache(a["k"] or None, a["v"] or None, a["ks"] or None, a["vs"] or None, a["num_pages"], a["H"],
                          a["page"], a["d"], a["dtype"])


CACHES = [
    (dict(dtype=1), BAD), (dict(dtype=3), BAD), (dict(num_pages=-1), BAD), (dict(H=-1), BAD), (dict(d=0), BAD),
    (dict(page=0), BAD), (dict(d=96), NO), (dict(d=256), NO), (dict(page=16), NO), (dict(page=48), NO),
    (dict(page=256), NO), (dict(H=70000), NO), (dict(k=0), BAD), (dict(v=0), BAD), (dict(k=24), BAD), (dict(v=34), BAD),
    (dict(ks=0), BAD), (dict(vs=0), BAD), (dict(ks=50), BAD),
]


def _append(cache=None, **kw):
    a = dict(plan=None, K=16, V=32, cu=0, rows=0, n=1, B=2, table=16, stride=4, pages=4, lens=16, strides=True)
    a.update(kw)
    s = rp._RowStrides(64, 64, 64)
    ref = ctypes.byref(s) if a["strides"] else None
    c = _cache(**(cache or {}))
    return rp.relpos_paged_append(ctypes.byref(c), a["plan"], v(a["K"]), v(a["V"]), ref, ref, v(a["cu"]), a["rows"],
                                  a["n"], a["B"], v(a["table"]), a["stride"], a["pages"], v(a["lens"]), None)


@pytest.mark.parametrize("cache,code", CACHES)
def test_append_cache(cache, code):
    assert _append(cache) == code


@pytest.mark.parametrize("kw,code", [
    (dict(plan=ctypes.byref(rp._RotaryPlan())), BAD), (dict(strides=False), BAD), (dict(B=-1), BAD), (dict(n=-1), BAD),
    (dict(pages=-1), BAD), (dict(K=0), BAD), (dict(V=0), BAD), (dict(K=17), BAD), (dict(table=0), BAD),
    (dict(lens=0), BAD), (dict(lens=18), BAD), (dict(cu=18, rows=3), BAD), (dict(stride=3), BAD), (dict(pages=0), BAD),
    (dict(n=1 << 29), NO), (dict(pages=1 << 24, stride=1 << 24), NO),
    (dict(n=0, K=0), OK), (dict(B=0, K=0), OK), (dict(cu=16, rows=0, K=0), OK),
])
def test_append(kw, code):
    assert _append(**kw) == code


def test_append_plan_fits_the_head():
    assert _append(plan=rp.RotaryPlan(128)._ref) == BAD
    assert _append(plan=rp.RotaryPlan(24)._ref) == NO


def _decode(cache=None, **kw):
    a = dict(Q=16, B=2, Hq=4, Lq=1, table=16, stride=4, pages=4, lens=16, mode=-1, bias=0, nb=32, md=128, scale=0.0,
             out=64, strides=True)
    a.update(kw)
    s = rp._RowStrides(64, 64, 64)
    ref = ctypes.byref(s) if a["strides"] else None
    c = _cache(**(cache or {}))
    return rp.relpos_paged_decode(ctypes.byref(c), v(a["Q"]), ref, a["B"], a["Hq"], a["Lq"], v(a["table"]),
                                  a["stride"], a["pages"], v(a["lens"]), a["mode"], v(a["bias"]), a["nb"], a["md"],
                                  a["scale"], v(a["out"]), ref, None)


@pytest.mark.parametrize("cache,code", CACHES)
def test_decode_cache(cache, code):
    assert _decode(cache) == code


@pytest.mark.parametrize("kw,code", [
    (dict(mode=1), BAD), (dict(mode=0, bias=16, nb=31), BAD), (dict(mode=0, bias=16, md=16), BAD), (dict(mode=0), BAD),
    (dict(mode=3), BAD), (dict(mode=3, bias=18), BAD), (dict(strides=False), BAD), (dict(B=-1), BAD), (dict(Hq=-2), BAD),
    (dict(Lq=-1), BAD), (dict(Lq=9), NO), (dict(Hq=3), BAD), (dict(Q=0), BAD), (dict(out=0), BAD), (dict(Q=17), BAD),
    (dict(lens=0), BAD), (dict(table=0), BAD), (dict(table=18), BAD), (dict(pages=0), BAD), (dict(stride=2), BAD),
    (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD), (dict(pages=1 << 24, stride=1 << 24), NO),
    (dict(B=1 << 22, pages=1 << 10, stride=1 << 10), NO),
    (dict(B=0, Q=0), OK), (dict(Hq=0, Q=0), OK), (dict(Lq=0, Q=0), OK),
])
def test_decode(kw, code):
    assert _decode(**kw) == code


def test_decode_without_pages_or_heads():
    assert _decode(dict(num_pages=0, k=0)) == BAD and _decode(dict(H=0, k=0)) == BAD


def test_python_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    plan = rp.RotaryPlan(64)
    with pytest.raises(ValueError):
        rp.rotary(x, plan)
    with pytest.raises(TypeError):
        rp.rotary(x.half(), plan)
    k = torch.zeros(2, 2, 32, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        rp.PagedCache(k, k.clone())  # not on a GPU
    with pytest.raises(TypeError):
        rp.PagedCache(k.float(), k.float())
    with pytest.raises(ValueError):
        rp.PagedCache(k, k[:1])
    with pytest.raises(ValueError):
        rp.PagedCache(k, k, torch.ones(2, 2), torch.ones(2, 2))  # scales of a 16-bit cache
    q = k.view(torch.uint8)[..., :64].contiguous().view(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        rp.PagedCache(q, q)
    with pytest.raises(TypeError):
        rp.PagedCache(q, q, torch.ones(2, 2).double(), torch.ones(2, 2))


@pytest.mark.parametrize("B,H,L,strides", [
    (2, 1, 1, (0, 64, 64)), (1, 2, 1, (64, 0, 64)), (1, 1, 2, (64, 64, 0)), (1, 1, 2, (64, 64, 63)), (1, 2, 1, (64, -63, 64)),
])
def test_outputs_whose_rows_overlap(B, H, L, strides):
    """An expanded tensor as the output: blocks would write one row at a time of several."""
    t = (rp._RotaryTensor * 1)()
    t[0].x, t[0].out, t[0].H = 16, 32, H
    t[0].x_batch = t[0].x_head = t[0].x_row = 64
    t[0].out_batch, t[0].out_head, t[0].out_row = strides
    assert rp.relpos_rotary(rp.RotaryPlan(64)._ref, 0, 0, t, 1, B, L, 64, None, 0, 0, None) == BAD
    c = _cache(H=1)
    q, o = rp._RowStrides(0, 0, 0), rp._RowStrides(*strides)
    assert rp.relpos_paged_decode(ctypes.byref(c), v(16), ctypes.byref(q), B, H, L, v(16), 4, 4, v(16), -1, None, 32,
                                  128, 0.0, v(64), ctypes.byref(o), None) == BAD
