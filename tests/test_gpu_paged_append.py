"""Appending to a paged cache vs the fp64 oracle.

8-bit caches: scales and codes equal the oracle's exactly (codes are the
correctly rounded ones). 16-bit caches: values exactly, turned keys within half
a bf16 step (2^-8) plus the fp32 rotation's 2^-21 (|x1| + |x2|)."""
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


def _bytes(t):
    return t.view(torch.uint8) if t.dtype == E4 else t.view(torch.int16)


def _snapshot(c):
    s = {"k": c.k.double().cpu().numpy().copy(), "v": c.v.double().cpu().numpy().copy()}
    if c.k_scale is not None:
        s |= {"k_scale": c.k_scale.double().cpu().numpy().copy(), "v_scale": c.v_scale.double().cpu().numpy().copy()}
    return s


def _case(new, old, H, d, page, dtype, seed, spread=2.0):
    """A cache whose sequences hold old[b] tokens, and new[b] more rows."""
    g = torch.Generator().manual_seed(seed)
    B = len(new)
    per = max(1, max((n + o + page - 1) // page for n, o in zip(new, old)))
    pages = B * per + 3
    table = torch.full((B, per), -1, dtype=torch.int32)
    order = torch.randperm(pages, generator=g).to(torch.int32)
    at = 0
    for b in range(B):
        c = (new[b] + old[b] + page - 1) // page
        table[b, :c] = order[at:at + c]
        at += c
    cache = rp.PagedCache.empty(pages, H, d, page_size=page, dtype=dtype)
    if dtype == E4:
        codes = torch.randint(0, 256, (2, pages, H, page, d), generator=g, dtype=torch.uint8)
        codes[(codes & 0x7f) == 0x7f] = 0x30  # no NaN
        cache.k.view(torch.uint8).copy_(codes[0].cuda())
        cache.v.view(torch.uint8).copy_(codes[1].cuda())
        for s in (cache.k_scale, cache.v_scale):
            s.copy_(torch.exp2(torch.randint(-9, -5, (pages, H), generator=g).float()).cuda())
    else:
        cache.k.copy_(torch.randn(cache.k.shape, generator=g).to(BF).cuda())
        cache.v.copy_(torch.randn(cache.k.shape, generator=g).to(BF).cuda())
    T = sum(new)
    kv = (torch.randn(T + 2, 2 * H, d, generator=g) * torch.exp2(spread * torch.randn(T + 2, 2 * H, 1, generator=g))).to(BF)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
    lens = torch.tensor([n + o for n, o in zip(new, old)], dtype=torch.int32)
    return cache, kv, table, cu, lens


def _expect(before, kv, table, cu, lens, page, H, rot=0, layout="half", **freq):
    K, V = kv.double().numpy()[:, :H].transpose(1, 0, 2), kv.double().numpy()[:, H:].transpose(1, 0, 2)
    for b in range(len(lens)):
        a, z = int(cu[b]), int(cu[b + 1])
        if z > a and lens[b] > 0:
            so.paged_append(before, K[:, a:z], V[:, a:z], table[b].tolist(), int(lens[b]) - (z - a), page, rot, layout, **freq)
    return before


def _same(cache, want, kv=None, H=0, turned=False):
    got = _snapshot(cache)
    for n in want:
        if turned and n == "k" and "k_scale" not in want:
            size = float(kv.float().abs().max())
            assert np.all(np.abs(got[n] - want[n]) <= 2.0 ** -8 * np.abs(want[n]) + 2.0 ** -20 * size)
        else:
            np.testing.assert_array_equal(got[n], want[n], err_msg=n)


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("d,page,H", [(64, 32, 3), (64, 64, 16), (64, 128, 5), (128, 32, 9), (128, 64, 2), (128, 128, 1)])
@pytest.mark.parametrize("rot,layout", [(0, "half"), (64, "half"), (64, "interleaved"), (16, "half"), (48, "interleaved")])
def test_ragged(dtype, d, page, H, rot, layout):
    new, old = [1, 0, 5, 97, 1, 130, 33], [0, 40, 31, 3, 64, 7, 127]
    cache, kv, table, cu, lens = _case(new, old, H, d, page, dtype, 100 * d + page + rot)
    want = _expect(_snapshot(cache), kv, table, cu, lens, page, H, rot, layout)
    plan = rp.RotaryPlan(rot, layout=layout) if rot else None
    kv_d = kv.cuda()
    args = (cache, kv_d[:, :H], kv_d[:, H:], table.cuda(), lens.cuda())
    rp.paged_append(*args, cu_new=cu.cuda(), plan=plan)
    assert rp.check_status() == 0
    _same(cache, want, kv, H, turned=rot > 0)
    # appending the same tokens again writes the same bytes
    held = [_bytes(t).clone() for t in (cache.k, cache.v)]
    rp.paged_append(*args, cu_new=cu.cuda(), plan=plan)
    assert all(torch.equal(a, _bytes(t)) for a, t in zip(held, (cache.k, cache.v)))


@pytest.mark.parametrize("dtype", [E4, BF])
@pytest.mark.parametrize("B", [1, 33, 70])
def test_one_token_steps(dtype, B):
    """A decode loop's steps over a page border, 32-bit strides of a [B,H,1,d]
    batch, unused entries among them."""
    H, d, page = 4, 64, 32
    old = [(29 + 5 * b) % 70 for b in range(B)]
    cache, _, table, _, _ = _case([8] * B, old, H, d, page, dtype, B)
    want = _snapshot(cache)
    plan = rp.RotaryPlan(64)
    g = torch.Generator().manual_seed(B)
    idle = [b % 7 == 3 for b in range(B)]
    for step in range(8):
        k, v = (torch.randn(B, H, 1, d, generator=g) * 2.0 ** step).to(BF), torch.randn(B, H, 1, d, generator=g).to(BF)
        lens = torch.tensor([0 if i else o + step + 1 for i, o in zip(idle, old)], dtype=torch.int32)
        rp.paged_append(cache, k.cuda(), v.cuda(), table.cuda(), lens.cuda(), plan=plan)
        _expect(want, torch.cat([k, v], 1)[:, :, 0], table, torch.arange(B + 1), lens, page, H, 64)
    assert rp.check_status() == 0
    _same(cache, want, torch.tensor(2.0 ** 10), H, turned=True)


def test_uniform_chunks_and_strides():
    H, d, page = 3, 128, 64
    new, old = [50, 50], [0, 90]
    cache, kv, table, cu, lens = _case(new, old, H, d, page, E4, 5)
    want = _expect(_snapshot(cache), kv, table, cu, lens, page, H, 128)
    K = kv[:100, :H].reshape(2, 50, H, d).transpose(1, 2).cuda()
    V = kv[:100, H:].reshape(2, 50, H, d).transpose(1, 2).contiguous().cuda()
    wide = torch.full((2, table.shape[1] + 3), -7, dtype=torch.int32)
    wide[:, 1:1 + table.shape[1]] = table
    rp.paged_append(cache, K, V, wide.cuda()[:, 1:1 + table.shape[1]], lens.cuda(), plan=rp.RotaryPlan(128))
    assert rp.check_status() == 0
    _same(cache, want)


@pytest.mark.parametrize("cut", [1, 4])
def test_unaligned_rows(cut):
    H, d, page = 2, 64, 32
    cache, kv, table, cu, lens = _case([40], [10], H, d, page, E4, 6)
    want = _expect(_snapshot(cache), kv, table, cu, lens, page, H, 64)
    flat = torch.zeros(42, 2 * H * d + 9, dtype=BF)
    flat[:, cut:cut + 2 * H * d] = kv.reshape(42, -1)
    w = flat.cuda()
    k = w[:, cut:cut + H * d].unflatten(1, (H, d))
    v = w[:, cut + H * d:cut + 2 * H * d].unflatten(1, (H, d))
    rp.paged_append(cache, k, v, table.cuda(), lens.cuda(), cu_new=cu.cuda(), plan=rp.RotaryPlan(64))
    assert rp.check_status() == 0
    _same(cache, want)


def test_codes_next_to_borders():
    """Half a million turned keys at far positions and a stretched plan with an
    amplitude: every code the correctly rounded one."""
    H, d, page = 8, 64, 64
    freq = dict(scaling="yarn", factor=16.0, original_len=4096.0)
    cache, kv, table, cu, lens = _case([1000], [30000], H, d, page, E4, 7, spread=0.0)
    table[:] = torch.randperm(cache.num_pages)[:table.shape[1]].to(torch.int32)
    want = _expect(_snapshot(cache), kv, table, cu, lens, page, H, 64, **freq)
    rp.paged_append(cache, kv.cuda()[:, :H], kv.cuda()[:, H:], table.cuda(), lens.cuda(), cu_new=cu.cuda(),
                    plan=rp.RotaryPlan(64, **freq))
    _same(cache, want)


def _pairs_next_to_borders(second):
    """(position, frequency, first member) of pairs with this second member whose y1 lies within the fp32 rotation's
    error 2^-22 (|x1| + |x2|) of a border between codes, but not within 2^-36 of it: the oracle's angles, of up to
    4096 in 64 bits, are off by 2^-40."""
    w, _ = so.rotary_frequencies(64)
    pos = np.arange(1, 4096, dtype=np.float64)
    found = []
    for m in range(32):
        c, s = np.cos(pos * w[m]), np.sin(pos * w[m])
        for x1 in 1.0 + np.arange(128) / 128.0:
            y = np.abs(x1 * c - second * s) / so.e4m3_scale(max(x1, second) * 2.0 ** 0.5)
            step = np.ldexp(1.0, np.maximum(np.frexp(y)[1] - 1, -6) - 3)
            gap = np.abs(y / step - np.floor(y / step) - 0.5) * step * so.e4m3_scale(max(x1, second) * 2.0 ** 0.5)
            size = x1 + second
            found += [(int(pos[i]), m, x1) for i in np.nonzero((gap < 2.0 ** -22 * size) & (gap > 2.0 ** -36 * size))[0]]
    return found


@pytest.mark.parametrize("second", [0.0, 1.0])
def test_pairs_next_to_borders(second):
    """Keys made of the pairs that the fp32 rotation cannot decide."""
    found = _pairs_next_to_borders(second)
    assert len(found) > 40
    B, page = len(found), 32
    cache = rp.PagedCache.empty(B, 1, 64, page_size=page, dtype=E4)
    cache.k_scale.fill_(2.0 ** -40)
    cache.v_scale.fill_(2.0 ** -40)
    table = torch.full((B, 4096 // page), -1, dtype=torch.int32)
    kv = torch.zeros(B, 2, 64)
    for b, (pos, m, x1) in enumerate(found):
        table[b, pos // page] = b
        kv[b, 0, m], kv[b, 0, 32 + m] = x1, second
    kv = kv.to(BF)
    cu, lens = torch.arange(B + 1, dtype=torch.int32), torch.tensor([f[0] + 1 for f in found], dtype=torch.int32)
    want = _expect(_snapshot(cache), kv, table, cu, lens, page, 1, 64)
    rp.paged_append(cache, kv.cuda()[:, :1], kv.cuda()[:, 1:], table.cuda(), lens.cuda(), cu_new=cu.cuda(),
                    plan=rp.RotaryPlan(64))
    assert rp.check_status() == 0
    _same(cache, want)


def test_odd_values():
    """Zeros, the smallest and largest magnitudes, infinities and NaN."""
    H, d, page = 1, 64, 32
    for x, rot in [(0.0, 64), (1e-38, 64), (3e38, 64), (float("inf"), 0), (float("nan"), 0), (9.2e-41, 0)]:
        cache, kv, table, cu, lens = _case([3], [2], H, d, page, E4, 8)
        cache.k_scale.fill_(2.0 ** -130 if x == 0 else 2.0 ** -8)
        cache.v_scale.copy_(cache.k_scale)
        kv[1] = 0.0
        kv[1, :, 7] = x
        want = _expect(_snapshot(cache), kv, table, cu, lens, page, H, rot)
        rp.paged_append(cache, kv.cuda()[:, :1], kv.cuda()[:, 1:], table.cuda(), lens.cuda(), cu_new=cu.cuda(),
                        plan=rp.RotaryPlan(rot) if rot else None)
        assert rp.check_status() == 0
        _same(cache, want)


@pytest.mark.parametrize("old", [0, 40])
def test_infinities_that_are_turned(old):
    """From position 0 on, where a rotation changes nothing, and further out: they saturate, beside their partners'
    NaN where the formula has one."""
    H, d, page = 2, 64, 32
    cache, kv, table, cu, lens = _case([5], [old], H, d, page, E4, 41)
    kv[0, 0, 3], kv[0, 0, 40], kv[2, 0, 9] = float("inf"), float("-inf"), float("-inf")
    want = _expect(_snapshot(cache), kv, table, cu, lens, page, H, 64)
    rp.paged_append(cache, kv.cuda()[:, :H], kv.cuda()[:, H:], table.cuda(), lens.cuda(), cu_new=cu.cuda(),
                    plan=rp.RotaryPlan(64))
    assert rp.check_status() == 0
    _same(cache, want)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_many_open_codes(layout):
    """Infinities leave the codes of their pairs open, thousands of them here; the heads beside theirs keep their own."""
    H, d, page, n = 16, 64, 64, 500
    cache, kv, table, cu, lens = _case([n] * 8, [33 * b for b in range(8)], H, d, page, E4, 42)
    kv[600:700, 5] = float("inf")
    kv[640, 5, ::3] = float("-inf")
    kv[650:660, 6, 4:20] = float("-inf")
    want = _expect(_snapshot(cache), kv, table, cu, lens, page, H, 64, layout)
    rp.paged_append(cache, kv.cuda()[:, :H], kv.cuda()[:, H:], table.cuda(), lens.cuda(), cu_new=cu.cuda(),
                    plan=rp.RotaryPlan(64, layout=layout))
    assert rp.check_status() == 0
    _same(cache, want)


def test_bad_pages_and_lengths_are_skipped_and_reported():
    """The kernel's own checks of page numbers, lengths and row ranges: nothing
    is written, the status says so once, good sequences are served."""
    H, d, page = 2, 64, 32
    for dtype in (E4, BF):
        for break_ in ("page", "negative page", "short", "long", "rows", "order"):
            cache, kv, table, cu, lens = _case([4, 4], [30, 3], H, d, page, dtype, 9)
            want = _snapshot(cache)
            good = want
            if break_ == "page":
                table[0, 1] = cache.num_pages
            elif break_ == "negative page":
                table[0, 1] = -1
            elif break_ == "short":
                lens[0] = 3
            elif break_ == "long":
                lens[0] = table.shape[1] * page + 1
            elif break_ == "rows":
                cu[2] = 4 + 100
            elif break_ == "order":
                cu[1] = -3
            if "page" in break_:  # the sequence's first page is in order
                half = _expect(good, kv[:2], table, torch.tensor([0, 2]), torch.tensor([32]), page, H)
                want = _expect(half, kv[4:], table[1:], torch.tensor([0, 4]), lens[1:], page, H)
            elif break_ in ("short", "long"):
                want = _expect(good, kv[4:], table[1:], torch.tensor([0, 4]), lens[1:], page, H)
            elif break_ == "rows":
                want = _expect(good, kv, table, torch.tensor([0, 4]), lens[:1], page, H)
            kv_d = kv.cuda()
            rp.paged_append(cache, kv_d[:, :H], kv_d[:, H:], table.cuda(), lens.cuda(), cu_new=cu.cuda())
            assert rp.check_status() == rp.RELPOS_ERR_PAGE, break_
            assert rp.check_status() == 0
            if break_ != "order":
                _same(cache, want)


def test_side_stream_and_graph():
    H, d, page = 4, 64, 64
    cache, kv, table, cu, lens = _case([70, 9], [5, 0], H, d, page, E4, 10)
    first = [t.clone() for t in (_bytes(cache.k), _bytes(cache.v), cache.k_scale, cache.v_scale)]
    kv_d, table_d, cu_d, lens_d, plan = kv.cuda(), table.cuda(), cu.cuda(), lens.cuda(), rp.RotaryPlan(64)

    def call():
        rp.paged_append(cache, kv_d[:, :H], kv_d[:, H:], table_d, lens_d, cu_new=cu_d, plan=plan)

    def restore():
        for t, f in zip((_bytes(cache.k), _bytes(cache.v), cache.k_scale, cache.v_scale), first):
            t.copy_(f)

    want = _expect(_snapshot(cache), kv, table, cu, lens, page, H, 64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    _same(cache, want)
    restore()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    _same(cache, _snapshot(cache))
    restore()
    g.replay()
    torch.cuda.synchronize()
    _same(cache, want)


def test_empty_calls():
    cache, kv, table, cu, lens = _case([4], [0], 2, 64, 32, E4, 11)
    want = _snapshot(cache)
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    rp.paged_append(cache, kv.cuda()[:0, :2], kv.cuda()[:0, 2:], table.cuda(), lens.cuda(), cu_new=torch.zeros(2, dtype=torch.int32).cuda())
    rp.paged_append(cache, kv.cuda()[:, :2], kv.cuda()[:, 2:], table.cuda()[:0], lens.cuda()[:0], cu_new=z)
    _same(cache, want)


def test_refusals():
    cache, kv, table, cu, lens = _case([4], [0], 2, 64, 32, E4, 12)
    kv, table, cu, lens = kv.cuda(), table.cuda(), cu.cuda(), lens.cuda()
    k, v = kv[:, :2], kv[:, 2:]
    for call in (lambda: rp.paged_append(cache, k, v, table, lens), lambda: rp.paged_append(cache, k, v[:2], table, lens, cu_new=cu),
                 lambda: rp.paged_append(cache, k[:, :1], v[:, :1], table, lens, cu_new=cu),
                 lambda: rp.paged_append(cache, k, v, table, lens[:0], cu_new=cu),
                 lambda: rp.paged_append(cache, k.cpu(), v, table, lens, cu_new=cu),
                 lambda: rp.paged_append(cache, k, v, table[0], lens, cu_new=cu)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: rp.paged_append(cache, k.float(), v, table, lens, cu_new=cu),
                 lambda: rp.paged_append(cache, k, v, table.long(), lens, cu_new=cu),
                 lambda: rp.paged_append(cache, k, v, table, lens, cu_new=cu.long())):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(rp.RelposError):
        rp.paged_append(cache, k, v, table, lens, cu_new=cu, plan=rp.RotaryPlan(24))
