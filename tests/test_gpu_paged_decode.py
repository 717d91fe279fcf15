"""Decoding over a paged cache vs the fp64 oracle.

Tolerance, with A = sum_j p_j |v_j| (the oracle returns it): half a bf16 step of
the output (2^-8 of it); the weights' rounding before p v, 2^-11 A in fp16 (8-bit
caches) or 2^-16 A in two bf16 parts; and the weights' error from the logits, at
most twice the logits' (2^-13 for |logit| up to 30: d products and their sum in
fp32, the exponential's 2^-22) of A."""
import numpy as np
import pytest
import torch

import gpu_util as G
import transformer_attention_relative_gb300 as rp
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu
BF, E4 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def _case(lens, Hq, Hkv, Lq, d, page, dtype, mode, seed, spare=2, k_sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    per = max(1, max((n + page - 1) // page for n in lens)) + 1
    pages = sum((n + page - 1) // page for n in lens) + spare
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((B, per), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        c = (n + page - 1) // page
        table[b, :c] = order[at:at + c]
        at += c
    shape = (pages, Hkv, page, d)
    if dtype == E4:
        # NaN wherever no token lies: unused slots, pages and scales
        codes, scales = [], []
        for sigma in (k_sigma, 1.0):
            x = torch.randn(shape, generator=g)
            s = torch.exp2(torch.randint(-8, -4, shape[:2], generator=g).float())
            codes.append((x * sigma / s[..., None, None]).clamp(-448, 448).to(E4).view(torch.uint8))
            scales.append(s)
        hole = 0x7f
    else:
        codes = [(torch.randn(shape, generator=g) * sigma).to(BF).view(torch.int16) for sigma in (k_sigma, 1.0)]
        scales, hole = [], 0x7fc0
    used = torch.zeros(pages, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range(n):
            used[table[b, j // page], j % page] = True
    for c in codes:
        c.masked_fill_(~used[:, None, :, None], hole)
    for s in scales:
        s[~used.any(1)] = float("nan")
    view = (lambda t: t.cuda().view(E4)) if dtype == E4 else (lambda t: t.cuda().view(BF))
    cache = rp.PagedCache(view(codes[0]), view(codes[1]), *(s.cuda() for s in scales))
    q = torch.randn(B, Lq, Hq, d, generator=g).to(BF).transpose(1, 2)
    bias = {"none": None, "t5": torch.randn(32, Hq, generator=g),
            "alibi": torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)])}[mode]
    return cache, q, table, torch.tensor(lens, dtype=torch.int32), bias


MODES = {"none": None, "t5": rp.MODE_T5, "alibi": rp.MODE_ALIBI}


def _gpu(cache, q, table, lens, bias, mode, **kw):
    o = rp.paged_decode(q.cuda(), cache, table.cuda(), lens.cuda(), bias=None if bias is None else bias.cuda(),
                        mode=MODES[mode], **kw)
    torch.cuda.synchronize()
    return o


def _ref(cache, q, table, lens, bias, mode, **kw):
    c = {"k": cache.k.double().cpu().numpy(), "v": cache.v.double().cpu().numpy()}
    if cache.k_scale is not None:
        c |= {"k_scale": cache.k_scale.double().cpu().numpy(), "v_scale": cache.v_scale.double().cpu().numpy()}
    return so.paged_decode(q.double().numpy(), c, table.numpy(), lens.tolist(), cache.page_size,
                           None if bias is None else bias.double().numpy(), mode, **kw)


def _check(got, ref, size, eight):
    got = got.double().cpu().numpy()
    tol = 2.0 ** -8 * np.abs(ref) + size * ((2.0 ** -11 if eight else 2.0 ** -16) + 2.0 ** -12)
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - ref) <= tol), (float(np.abs(got - ref).max()), float((np.abs(got - ref) / np.maximum(tol, 1e-30)).max()))


def _parity(*a, **kw):
    cache, q, table, lens, bias = _case(*a)
    mode = a[7]
    got = _gpu(cache, q, table, lens, bias, mode, **kw)
    assert rp.check_status() == 0
    _check(got, *_ref(cache, q, table, lens, bias, mode, **kw), a[6] == E4)
    return got


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("d,page", [(64, 32), (64, 64), (64, 128), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("mode", ["none", "t5", "alibi"])
def test_types_pages_biases(dtype, d, page, mode):
    _parity([1, 31, 32, 33, 127, 128, 200, 515], 4, 2, 1, d, page, dtype, mode, 1)


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("Hq,Hkv,Lq", [(1, 1, 1), (3, 3, 2), (8, 1, 1), (16, 2, 2), (5, 1, 3), (12, 4, 8), (16, 1, 2),
                                       (32, 2, 8), (34, 2, 1)])
def test_heads_and_rows(dtype, Hq, Hkv, Lq):
    """Groups and new rows below, at and beyond one 16-row tile."""
    _parity([40, 3, 97, 300], Hq, Hkv, Lq, 64, 32, dtype, "t5", 2)
    _parity([40, 2, 97, 300], Hq, Hkv, Lq, 128, 64, dtype, "alibi", 3)


@pytest.mark.parametrize("dtype", [E4, BF])
def test_rows_before_the_start_and_empty_sequences(dtype):
    got = _parity([0, 1, 5, 0, 8, 200], 4, 2, 8, 64, 32, dtype, "none", 4).float().cpu()
    assert not got[0].any() and not got[3].any() and not got[1, :, :7].any() and got[1, :, 7].any()
    assert not _parity([0, 0], 4, 2, 1, 64, 32, dtype, "none", 5).float().any()


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("n", [4096, 20011])
def test_long_contexts_split_over_blocks(dtype, n):
    _parity([n, 77], 4, 1, 1, 64, 128, dtype, "t5", 6)
    _parity([n], 2, 1, 2, 128, 128, dtype, "none", 7)


def test_many_short_sequences():
    _parity([1 + (37 * b) % 90 for b in range(150)], 2, 2, 1, 64, 32, E4, "alibi", 8)


@pytest.mark.parametrize("dtype", [E4, BF])
def test_sharp_logits(dtype):
    """Keys of larger magnitude: a few keys carry the softmax and the running
    maximum moves from tile to tile."""
    _parity([1000, 70], 4, 2, 2, 64, 64, dtype, "none", 9, 2, 3.0)


@pytest.mark.parametrize("nb,md", [(8, 20), (32, 128), (64, 1000), (128, 5000)])
def test_buckets(nb, md):
    cache, q, table, lens, _ = _case([900, 40], 4, 2, 2, 64, 64, E4, "t5", 10)
    bias = torch.randn(nb, 4, generator=torch.Generator().manual_seed(1))
    kw = dict(num_buckets=nb, max_distance=md)
    _check(_gpu(cache, q, table, lens, bias, "t5", **kw), *_ref(cache, q, table, lens, bias, "t5", **kw), True)


def test_scale_argument():
    cache, q, table, lens, bias = _case([300, 40], 4, 2, 1, 128, 64, BF, "none", 11)
    _check(_gpu(cache, q, table, lens, bias, "none", scale=0.3), *_ref(cache, q, table, lens, bias, "none", scale=0.3), False)


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("where", ["k", "v"])
def test_nan_in_a_later_row_stays_there(dtype, where):
    """A new token's NaN reaches the rows that see it and no other."""
    cache, q, table, lens, bias = _case([70], 4, 2, 4, 64, 32, dtype, "none", 12)
    ref, size = _ref(cache, q, table, lens, bias, "none")
    t = getattr(cache, where)
    p, s = int(table[0, 68 // 32]), 68 % 32  # the key of query row 2 (position 68)
    (t.view(torch.uint8) if dtype == E4 else t.view(torch.int16))[p, :, s] = 0x7f if dtype == E4 else 0x7fc0
    got = _gpu(cache, q, table, lens, bias, "none")
    _check(got[:, :, :2], ref[:, :, :2], size[:, :, :2], dtype == E4)
    assert got[:, :, 2:].isnan().all()
    assert rp.check_status() == 0


def test_lowest_values_in_the_bias():
    """The fp32 type's lowest value as a mask in the table: no overflow to
    minus infinity, an even softmax where every key has it; minus infinity
    itself gives a key no weight."""
    low = torch.finfo(torch.float32).min
    cache, q, table, lens, _ = _case([50], 2, 1, 1, 64, 32, E4, "t5", 13)
    v = cache.v.double().cpu().numpy()
    vs = cache.v_scale.double().cpu().numpy()
    seq = np.concatenate([v[p, 0] * vs[p, 0] for p in table[0, :2].tolist()])[:50]
    got = _gpu(cache, q, table, lens, torch.full((32, 2), low), "t5").double().cpu().numpy()
    tol = 2.0 ** -8 * np.abs(seq.mean(0)) + np.abs(seq).mean(0) * 2.0 ** -10
    assert np.all(np.abs(got[0, :, 0] - seq.mean(0)) <= tol)
    bias = torch.full((32, 2), low)
    bias[0] = 0.0  # its own key alone
    got = _gpu(cache, q, table, lens, bias, "t5").double().cpu().numpy()
    assert np.all(np.abs(got[0, :, 0] - seq[49]) <= 2.0 ** -8 * np.abs(seq[49]) + 2.0 ** -11 * np.abs(seq[49]))
    bias[1:] = -float("inf")
    again = _gpu(cache, q, table, lens, bias, "t5").double().cpu().numpy()
    np.testing.assert_array_equal(got, again)


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("mask", [-1e9, torch.finfo(torch.float32).min])
def test_masks_over_many_tiles(dtype, mask):
    """Every key masked by a bias that fp32 cannot add a product to without
    losing it: an even softmax over all tiles, near ones and far ones. (|q.k| /
    sqrt(d) stays below 32, half a step of fp32 at 1e9, so each logit is the mask
    itself.)"""
    cache, q, table, lens, _ = _case([1500, 40], 4, 2, 1, 64, 64, dtype, "t5", 25)
    got = _gpu(cache, q, table, lens, torch.full((32, 4), mask), "t5").double().cpu().numpy()
    ref, size = _ref(cache, 0 * q, table, lens, torch.zeros(32, 4), "t5")  # equal logits
    _check(torch.from_numpy(got), ref, size, dtype == E4)


@pytest.mark.parametrize("scale_exp", [-100, 60])
def test_far_scales(scale_exp):
    """Page scales far from 1 on the values (and back on q for the keys)."""
    cache, q, table, lens, bias = _case([100], 4, 2, 1, 64, 32, E4, "none", 14)
    cache.v_scale.mul_(2.0 ** scale_exp)
    _check(_gpu(cache, q, table, lens, bias, "none"), *_ref(cache, q, table, lens, bias, "none"), True)
    cache.v_scale.mul_(2.0 ** -scale_exp)
    cache.k_scale.mul_(2.0 ** scale_exp)
    q2 = (q.double() * 2.0 ** -scale_exp).to(BF)
    _check(_gpu(cache, q2, table, lens, bias, "none"), *_ref(cache, q2, table, lens, bias, "none"), True)


def test_pages_of_very_different_scales():
    """Values whose pages differ in scale by far more than a weight's bits, in
    both directions, a page of scale zero and one of negative scale."""
    for d in (64, 128):
        cache, q, table, lens, bias = _case([700, 130], 4, 2, 1, d, 32, E4, "none", 23)
        g = torch.Generator().manual_seed(24)
        for s in (cache.v_scale,):
            s.copy_(torch.exp2(torch.randint(-60, 30, s.shape, generator=g).float()).cuda())
            s[table[0, 3], 0] = 0.0
            s[table[0, 5], 1] *= -1.0
            s[table[1, 0]] = 2.0 ** -40
        _check(_gpu(cache, q, table, lens, bias, "none"), *_ref(cache, q, table, lens, bias, "none"), True)


def test_strides_and_out():
    cache, q, table, lens, bias = _case([100, 9], 4, 2, 2, 64, 32, E4, "none", 15)
    want = _gpu(cache, q, table, lens, bias, "none")
    fused = torch.randn(2, 2, 4 * 64 + 7).to(BF).cuda()
    odd = fused[..., 3:3 + 256].unflatten(2, (4, 64)).transpose(1, 2)
    odd.copy_(q)
    out = torch.full((2, 4, 5, 67), 3.0, dtype=BF, device="cuda")
    o = rp.paged_decode(odd, cache, table.cuda(), lens.cuda(), out=out[:, :, 1:3, 2:66])
    assert torch.equal(o, want)
    rest = out.clone()
    rest[:, :, 1:3, 2:66] = 3.0
    assert (rest == 3.0).all()  # nothing beside the rows was touched


def test_bad_pages_are_skipped_and_reported():
    for dtype in (E4, BF):
        cache, q, table, lens, bias = _case([100, 90], 4, 2, 1, 64, 32, dtype, "none", 16)
        ref, size = _ref(cache, q, table, lens, bias, "none")
        for bad in (-1, cache.num_pages, 2 ** 31 - 1, -2 ** 31):
            t = table.clone()
            t[0, 1] = bad
            got = _gpu(cache, q, t, lens, bias, "none")
            assert rp.check_status() == rp.RELPOS_ERR_PAGE
            _check(got[1:], ref[1:], size[1:], dtype == E4)
        got = _gpu(cache, q, table[:, :3].contiguous(), torch.tensor([97, 90], dtype=torch.int32), bias, "none")
        assert rp.check_status() == rp.RELPOS_ERR_PAGE  # a length beyond the table's pages
        _check(got[1:], ref[1:], size[1:], dtype == E4)
        assert rp.check_status() == 0


def test_repeats_are_equal_and_streams_do_not_mix():
    a = _case([3000, 500, 20], 8, 2, 1, 64, 64, E4, "alibi", 17)
    b = _case([2500, 900], 8, 2, 2, 128, 64, BF, "t5", 18)
    da = [x.cuda() if torch.is_tensor(x) else x for x in a]
    db = [x.cuda() if torch.is_tensor(x) else x for x in b]
    run_a = lambda: rp.paged_decode(da[1], da[0], da[2], da[3], bias=da[4], mode=rp.MODE_ALIBI)  # noqa: E731
    run_b = lambda: rp.paged_decode(db[1], db[0], db[2], db[3], bias=db[4], mode=rp.MODE_T5)  # noqa: E731
    want_a, want_b = run_a(), run_b()
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i in range(20):
        for st, run in zip(s, (run_a, run_b)):
            with torch.cuda.stream(st):
                got.append(run())
    torch.cuda.synchronize()
    assert all(torch.equal(g, want_a) for g in got[0::2]) and all(torch.equal(g, want_b) for g in got[1::2])
    _check(want_a, *_ref(*a, "alibi"), True)
    _check(want_b, *_ref(*b, "t5"), False)


def test_captured_graphs():
    """Two graphs, replayed in turn and with lengths that grew since capture."""
    cache, q, table, lens, bias = _case([700, 33], 4, 2, 1, 64, 64, E4, "t5", 19)
    qd, td, bd = q.cuda(), table.cuda(), bias.cuda()
    ld = torch.tensor([10, 0], dtype=torch.int32, device="cuda")
    run = lambda: rp.paged_decode(qd, cache, td, ld, bias=bd, mode=rp.MODE_T5)  # noqa: E731
    run()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run())
        graphs.append(g)
    for n in ([700, 33], [65, 1], [0, 32]):
        ld.copy_(torch.tensor(n, dtype=torch.int32))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        ref = _ref(cache, q, table, torch.tensor(n), bias, "t5")
        for o in outs:
            _check(o, *ref, True)
    assert rp.check_status() == 0


def test_offsets_beyond_32_bits():
    """The last pages of a pool of over 4 GB."""
    page, d, H = 128, 128, 8
    pages = (1 << 32) // (page * d * H) + 40
    k = torch.zeros(pages, H, page, d, dtype=torch.uint8, device="cuda").view(E4)
    v = torch.zeros(pages, H, page, d, dtype=torch.uint8, device="cuda").view(E4)
    cache = rp.PagedCache(k, v, torch.ones(pages, H, device="cuda"), torch.ones(pages, H, device="cuda"))
    table = torch.tensor([[pages - 1, pages - 2, pages - 7]], dtype=torch.int32)
    n = 300
    g = torch.Generator().manual_seed(20)
    kv = torch.randn(n, 2 * H, d, generator=g).to(BF)
    rp.paged_append(cache, kv.cuda()[:, :H], kv.cuda()[:, H:], table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(),
                    cu_new=torch.tensor([0, n], dtype=torch.int32).cuda())
    q = torch.randn(1, H, 1, d, generator=g).to(BF)
    got = _gpu(cache, q, table, torch.tensor([n], dtype=torch.int32), None, "none")
    small = rp.PagedCache(*(x[[pages - 1, pages - 2, pages - 7]].contiguous() if x.dtype != E4 else
                            x.view(torch.uint8)[[pages - 1, pages - 2, pages - 7]].contiguous().view(E4)
                            for x in (k, v, cache.k_scale, cache.v_scale)))
    _check(got, *_ref(small, q, torch.tensor([[0, 1, 2]]), torch.tensor([n]), None, "none"), True)
    assert k.view(torch.uint8)[:pages - 7].sum() == 0 and rp.check_status() == 0


def test_a_decode_loop():
    """Prompt and steps as a server runs them: rotate, append, decode; against
    dense attention in fp64 over the same tokens. 16-bit cache: keys rounded
    once (2^-8 relative), so logits move by up to 2^-8 sum |q||k| / sqrt(d)."""
    B, Hq, H, d, page = 2, 4, 2, 64, 32
    g = torch.Generator().manual_seed(21)
    N = [45, 70]
    steps = 6
    plan = rp.RotaryPlan(d)
    X = [torch.randn(n + steps, Hq + 2 * H, d, generator=g).to(BF) for n in N]
    table = torch.tensor([[3, 0, 5], [1, 4, 2]], dtype=torch.int32).cuda()
    for dtype in (BF, E4):
        cache = rp.PagedCache.empty(6, H, d, page_size=page, dtype=dtype)
        prompt = torch.cat([x[:n] for x, n in zip(X, N)]).cuda()
        lens = torch.tensor(N, dtype=torch.int32).cuda()
        rp.paged_append(cache, prompt[:, Hq:Hq + H], prompt[:, Hq + H:], table, lens,
                        cu_new=torch.tensor([0, N[0], sum(N)], dtype=torch.int32).cuda(), plan=plan)
        for t in range(steps):
            row = torch.stack([x[n + t] for x, n in zip(X, N)])[:, :, None].cuda()  # [B, heads, 1, d]
            lens += 1
            rp.paged_append(cache, row[:, Hq:Hq + H], row[:, Hq + H:], table, lens, plan=plan)
            q = rp.rotary(row[:, :Hq], plan, positions=(lens - 1)[:, None])
            o = rp.paged_decode(q, cache, table, lens)
            _check(o, *_ref(cache, q.cpu(), table.cpu(), lens.cpu(), None, "none"), dtype == E4)
            if dtype == BF:
                for b in range(B):
                    n = N[b] + t + 1
                    x = X[b].double().numpy()[:n].transpose(1, 0, 2)
                    k = so.rotary(x[Hq:Hq + H], np.arange(n), d)
                    qq = so.rotary(x[:Hq, -1:], [n - 1], d)
                    for h in range(Hq):
                        z = k[h // 2] @ qq[h, 0] / 8.0
                        e = np.exp(z - z.max())
                        e /= e.sum()
                        vv = x[Hq + H + h // 2]
                        dz = 2 * 2.0 ** -8 * (np.abs(k[h // 2]) @ np.abs(qq[h, 0]) / 8.0).max()
                        tol = 2.0 ** -8 * np.abs(e @ vv) + (2.1 * dz + 2.0 ** -12) * (e @ np.abs(vv))
                        assert np.all(np.abs(o[b, h, 0].double().cpu().numpy() - e @ vv) <= tol)
    assert rp.check_status() == 0


def test_refusals():
    cache, q, table, lens, _ = _case([40], 4, 2, 1, 64, 32, E4, "none", 22)
    q, table, lens = q.cuda(), table.cuda(), lens.cuda()
    slopes = torch.ones(4, device="cuda")
    for call in (lambda: rp.paged_decode(q[..., :32], cache, table, lens), lambda: rp.paged_decode(q, cache, table, lens, bias=slopes),
                 lambda: rp.paged_decode(q, cache, table, lens, bias=slopes, mode=rp.MODE_T5),
                 lambda: rp.paged_decode(q, cache, table, lens, bias=slopes, mode=rp.MODE_SHAW),
                 lambda: rp.paged_decode(q.cpu(), cache, table, lens), lambda: rp.paged_decode(q, cache, table, lens[:0]),
                 lambda: rp.paged_decode(q, cache, table, lens, out=q[:, :2])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: rp.paged_decode(q.float(), cache, table, lens), lambda: rp.paged_decode(q, cache, table.long(), lens),
                 lambda: rp.paged_decode(q, cache, table, lens, mode=rp.MODE_ALIBI),
                 lambda: rp.paged_decode(q, cache, table, lens, bias=slopes.half(), mode=rp.MODE_ALIBI)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(rp.RelposError) as e:
        rp.paged_decode(q.expand(1, 4, 9, 64), cache, table, lens)
    assert e.value.code == rp.RELPOS_ERR_UNSUPPORTED
    with pytest.raises(rp.RelposError):
        rp.paged_decode(q[:, :3], cache, table, lens)


def test_broadcast_queries():
    cache, q, table, lens, _ = _case([300, 70], 4, 2, 3, 64, 64, E4, "none", 31)
    one = q[:, :1, :1].cuda().expand(2, 4, 3, 64)
    args = cache, table.cuda(), lens.cuda()
    assert torch.equal(rp.paged_decode(one, *args), rp.paged_decode(one.contiguous(), *args))
    with pytest.raises(rp.RelposError) as e:
        rp.paged_decode(one.contiguous(), *args, out=one)
    assert e.value.code == rp.RELPOS_ERR_INVALID_ARG
    assert rp.check_status() == 0


def test_calls_from_several_threads():
    """Threads with streams and T5 parameters of their own: what calls share on the host does not mix."""
    import threading

    cache, q, table, lens, bias = _case([2000, 130, 5], 8, 2, 1, 64, 64, E4, "t5", 32)
    qd, td, ld, bd = q.cuda(), table.cuda(), lens.cuda(), bias.cuda()
    shapes = [(32, 128), (32, 500), (16, 64), (8, 20), (24, 1000), (30, 77), (4, 9), (32, 33), (12, 300), (28, 128)]
    run = lambda nb, md: rp.paged_decode(qd, cache, td, ld, bias=bd[:nb], mode=rp.MODE_T5, num_buckets=nb,  # noqa: E731
                                         max_distance=md)
    want = [run(*s) for s in shapes]
    torch.cuda.synchronize()
    same = []

    def work(k):
        with torch.cuda.stream(torch.cuda.Stream()):
            got = [(i, run(*shapes[i])) for i in ((k + 3 * j) % len(shapes) for j in range(60))]
            torch.cuda.current_stream().synchronize()
            same.extend(torch.equal(o, want[i]) for i, o in got)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(same) == 4 * 60 and all(same) and rp.check_status() == 0


def test_graphs_replayed_at_once():
    """Two graphs, each with calls that need scratch, on two streams at the same time."""
    cases = [_case([3000, 700, 1], 8, 2, 1, 64, 64, E4, "none", 33), _case([2600, 900], 8, 2, 2, 128, 64, BF, "none", 34)]
    graphs, outs, want, inputs = [], [], [], []
    for cache, q, table, lens, _ in cases:
        args = q.cuda(), cache, table.cuda(), lens.cuda()
        inputs.append(args)
        want.append(rp.paged_decode(*args))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append([rp.paged_decode(*args) for _ in range(4)])
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(15):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for w, os in zip(want, outs):
        assert all(torch.equal(w, o) for o in os)
    assert rp.check_status() == 0
