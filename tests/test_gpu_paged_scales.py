"""Decoding over 8-bit pages whose scales lie far apart, vs the fp64 oracle.

Tolerance as for the other decodes: half a bf16 step of the output (2^-8 of it),
and of A = sum_j p_j |v_j| the weights' rounding to fp16, 2^-11, and twice their
logits' error, 2^-12. That holds for weights down to 2^-18 of a row's largest; what
lies below goes into fp16's subnormal numbers. Sums of weights (up to 2^13) and values
are fp32 before the division by the weights' sum: values stay below 2^108 here."""
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


def _check(cache, q, table, lens, got, dims=slice(None)):
    c = {n: getattr(cache, n).double().cpu().numpy() for n in ("k", "v", "k_scale", "v_scale")}
    with np.errstate(over="ignore"):
        ref, size = so.paged_decode(q.double().numpy(), c, table.numpy(), lens, cache.page_size)
    got, ref, size = got.double().cpu().numpy()[..., dims], ref[..., dims], size[..., dims]
    assert np.all(np.isfinite(got)), int((~np.isfinite(got)).sum())
    bad = np.abs(got - ref) / (2.0 ** -8 * np.abs(ref) + size * (2.0 ** -11 + 2.0 ** -12) + 2.0 ** -133)
    assert bad.max() <= 1.0, float(bad.max())


def _filled(d, page, H, sizes, g, positive=True):
    """A cache with one sequence appended through the library: page i holds values of magnitude sizes[i]."""
    n = page * len(sizes)
    cache = rp.PagedCache.empty(len(sizes) + 1, H, d, page_size=page, dtype=E4)
    table = torch.randperm(len(sizes) + 1, generator=g)[None, :len(sizes)].to(torch.int32)
    k, v = torch.randn(n, H, d, generator=g), torch.randn(n, H, d, generator=g)
    v = (v.abs() if positive else v) * torch.tensor(sizes).repeat_interleave(page)[:, None, None]
    rp.paged_append(cache, k.to(BF).cuda(), v.to(BF).cuda(), table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(),
                    cu_new=torch.tensor([0, n], dtype=torch.int32).cuda())
    return cache, table, n


def _decode(cache, table, n, q):
    lens = torch.tensor(n, dtype=torch.int32).cuda()
    got = rp.paged_decode(q.cuda(), cache, table.cuda(), lens)
    assert rp.check_status() == 0
    return got


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [32, 64, 128])
@pytest.mark.parametrize("tokens", [512, 4096])
def test_a_page_of_zero_values(d, page, tokens):
    """Padding tokens with zero values fill a page between ordinary ones: the library gives it the scale 2^-120."""
    g = torch.Generator().manual_seed(d + page)
    sizes = [1.0] * (tokens // page)
    for i in range(len(sizes) // 4, len(sizes), 3):
        sizes[i] = 0.0
    cache, table, n = _filled(d, page, 2, sizes, g)
    assert float(cache.v_scale.min()) == 2.0 ** -120
    q = torch.randn(1, 4, 1, d, generator=g).to(BF)
    _check(cache, q, table, [n], _decode(cache, table, [n], q))


@pytest.mark.parametrize("d", [64, 128])
def test_a_zero_page_in_long_shares(d):
    """Blocks with tens of tiles a warp (many sequences over the same pages), one zero page in the middle."""
    page, H, B, g = 64, 8, 64, torch.Generator().manual_seed(5)
    sizes = [1.0] * 64
    sizes[37] = 0.0
    cache, table, n = _filled(d, page, H, sizes, g, positive=False)
    q = torch.randn(1, H, 1, d, generator=g).to(BF)
    got = _decode(cache, table.expand(B, -1).contiguous(), [n] * B, q.expand(B, -1, -1, -1))
    for b in (0, 1, 17, B - 1):
        _check(cache, q, table, [n], got[b:b + 1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), 3e38, -2.0 ** 105])
def test_a_very_large_value(d, value):
    """An infinite one saturates at the largest scale. The dims beside it keep what the other pages give them (its own
    may pass fp32 in a sum of weights and values)."""
    g = torch.Generator().manual_seed(6)
    page, pages = 64, 8
    n = page * pages
    cache = rp.PagedCache.empty(pages, 1, d, page_size=page, dtype=E4)
    table = torch.arange(pages, dtype=torch.int32)[None]
    k, v = torch.randn(n, 1, d, generator=g), torch.randn(n, 1, d, generator=g).abs()
    v[200, 0, 5] = value
    rp.paged_append(cache, k.to(BF).cuda(), v.to(BF).cuda(), table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(),
                    cu_new=torch.tensor([0, n], dtype=torch.int32).cuda())
    assert float(cache.v_scale.max()) >= 2.0 ** 96
    q = torch.randn(1, 2, 1, d, generator=g).to(BF)
    got = _decode(cache, table, [n], q)
    _check(cache, q, table, [n], got, [i for i in range(d) if i != 5] if abs(value) > 1e38 else slice(None))
    assert bool((got[..., 5] * value > 0).all())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
def test_scales_over_their_whole_range(d, order):
    """Values of 2^-112 to 2^98, in turn."""
    g = torch.Generator().manual_seed(7)
    sizes = [2.0 ** e for e in range(-112, 99, 7)]
    if order == "falling":
        sizes = sizes[::-1]
    if order == "mixed":
        sizes = [sizes[i] for i in torch.randperm(len(sizes), generator=g).tolist()]
    cache, table, n = _filled(d, 32, 1, sizes, g, positive=False)
    q = (0.3 * torch.randn(1, 2, 1, d, generator=g)).to(BF)
    _check(cache, q, table, [n], _decode(cache, table, [n], q))
    # and each alone with its neighbours, where the largest does not hide the rest
    for i in range(0, len(sizes) - 4, 4):
        m = 4 * 32
        _check(cache, q, table[:, i:i + 4], [m], _decode(cache, table[:, i:i + 4].contiguous(), [m], q))


@pytest.mark.parametrize("exponent", [-140, -127, -100, 99])
def test_scales_at_the_ends_of_fp32(exponent):
    """A cache from elsewhere: very large scales, and subnormal ones, on every page."""
    g = torch.Generator().manual_seed(8)
    codes = torch.randn(2, 3, 1, 32, 64, generator=g)
    codes[1] *= 64.0
    codes = codes.clamp(-448, 448).to(E4)
    scale = torch.full((3, 1), 2.0 ** exponent, dtype=torch.float64).float()
    cache = rp.PagedCache(codes[0].cuda(), codes[1].cuda(), torch.ones(3, 1).cuda(), scale.cuda())
    q = torch.randn(1, 1, 1, 64, generator=g).to(BF)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32)
    _check(cache, q, table, [90], _decode(cache, table, [90], q))


@pytest.mark.parametrize("factor", [64.0, 32.0, 4.0])
@pytest.mark.parametrize("d", [64, 128])
def test_weak_keys_behind_a_page_of_larger_scale(d, factor):
    """The first page has a larger value scale and holds, in each of its four tiles, a key that dominates the softmax
    and has zero values; the output is the sum over the equal weak keys of the other pages, 2^-17.9 of the largest
    weight each (8.25 x 12 / 8 nats). Each warp meets the first page before them."""
    g = torch.Generator().manual_seed(9)
    pages, page = 4, 128
    k = torch.zeros(pages, 1, page, d)
    k[0, 0, ::32, 0] = 12.0
    v = torch.randn(pages, 1, page, d, generator=g).abs() * 64.0
    v[0] = 0.0
    scale = torch.full((pages, 1), 2.0 ** -6)
    scale[0] *= factor
    cache = rp.PagedCache(k.to(E4).cuda(), v.clamp(0, 448).to(E4).cuda(), torch.ones(pages, 1).cuda(), scale.cuda())
    q = torch.zeros(1, 1, 1, d)
    q[..., 0] = 8.25
    table = torch.arange(pages, dtype=torch.int32)[None]
    lens = torch.tensor([pages * page], dtype=torch.int32)
    got = rp.paged_decode(q.to(BF).cuda(), cache, table.cuda(), lens.cuda(), scale=0.125)
    assert rp.check_status() == 0
    c = {n: getattr(cache, n).double().cpu().numpy() for n in ("k", "v", "k_scale", "v_scale")}
    ref, size = so.paged_decode(q.double().numpy(), c, table.numpy(), [pages * page], page, scale=0.125)
    bad = np.abs(got.double().cpu().numpy() - ref) / (2.0 ** -8 * ref + size * (2.0 ** -11 + 2.0 ** -12))
    assert bad.max() <= 1.0, float(bad.max())


@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_scale_that_is_not_finite_stays_with_its_page(rows, bad):
    """The newest token starts a page whose value scale is not finite: the rows before it do not see that page."""
    g = torch.Generator().manual_seed(10)
    codes = torch.randn(2, 3, 1, 32, 64, generator=g).to(E4)
    scales = torch.ones(2, 3, 1)
    n = 65  # the last token alone in the third page
    table = torch.tensor([[1, 2, 0]], dtype=torch.int32)
    q = torch.randn(1, 2, rows, 64, generator=g).to(BF)
    good = rp.PagedCache(codes[0].cuda(), codes[1].cuda(), scales[0].cuda(), scales[1].cuda())
    want = _decode(good, table, [n], q)
    scales[1, 0] = bad
    cache = rp.PagedCache(codes[0].cuda(), codes[1].cuda(), scales[0].cuda(), scales[1].cuda())
    got = _decode(cache, table, [n], q)
    assert not got[:, :, -1].isfinite().any()
    if rows > 1:
        c = {x: getattr(good, x).double().cpu().numpy() for x in ("k", "v", "k_scale", "v_scale")}
        ref, size = so.paged_decode(q.double().numpy(), c, table.numpy(), [n], 32)
        got, ref, size = got[:, :, :-1].double().cpu().numpy(), ref[:, :, :-1], size[:, :, :-1]
        assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + size * (2.0 ** -11 + 2.0 ** -12))
    assert want.isfinite().all()
