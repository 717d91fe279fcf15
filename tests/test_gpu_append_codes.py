"""Codes of an 8-bit append where fp32 arithmetic alone would miss them: pairs whose
rotation overflows, and pages whose scale is not a power of two. They equal the fp64
oracle's, bit for bit."""
import numpy as np
import pytest
import torch

import gpu_util as G
import transformer_attention_relative_gb300 as rp
from oracle import serving_oracle as so
from test_gpu_paged_append import _expect, _same, _snapshot

pytestmark = pytest.mark.gpu
BF, E4 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def _append(cache, kv, table, cu, lens, H, plan=None):
    d = kv.cuda()
    rp.paged_append(cache, d[:, :H], d[:, H:], table.cuda(), lens.cuda(), cu_new=cu.cuda(), plan=plan)
    assert rp.check_status() == 0


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("freq", [{}, dict(scaling="yarn", factor=8.0, original_len=4096.0)])
def test_pairs_whose_rotation_overflows(layout, freq):
    """One or both members of a pair near 3e38: turned, and with an amplitude above 1, they pass fp32's largest value;
    their quotients by the page's scale do not pass 448."""
    page, n = 32, 64
    g = torch.Generator().manual_seed(1)
    cache = rp.PagedCache.empty(3, 1, 64, page_size=page, dtype=E4)
    sign = torch.randint(0, 2, (n, 2, 64), generator=g) * 2 - 1
    kv = ((2.0 + 1.38 * torch.rand(n, 2, 64, generator=g)) * 1e38 * sign).to(BF)
    kv[::3, 0, :20] *= 0.01  # pairs with one large member, whose magnitudes' sum is still finite
    kv[::5] = (torch.randn(kv[::5].shape, generator=g) * 1e37).to(BF)
    table, cu = torch.tensor([[2, 0]], dtype=torch.int32), torch.tensor([0, n], dtype=torch.int32)
    lens = torch.tensor([n], dtype=torch.int32)
    want = _expect(_snapshot(cache), kv, table, cu, lens, page, 1, 64, layout, **freq)
    _append(cache, kv, table, cu, lens, 1, rp.RotaryPlan(64, layout=layout, **freq))
    _same(cache, want)


def _ties(scale):
    """bf16 values whose quotient by the scale lies on, or next to, a border between codes."""
    x = torch.arange(0x3000, 0x4200, dtype=torch.int16).view(BF).double().numpy()
    q = x / scale
    q, x = q[(q > 2.0 ** -9) & (q < 440)], x[(q > 2.0 ** -9) & (q < 440)]
    step = np.ldexp(1.0, np.maximum(np.frexp(q)[1] - 1, -6) - 3)
    return x[np.abs(q / step - np.floor(q / step) - 0.5) < 2.0 ** -6]


SCALES = [7 * 2.0 ** -9, float(np.float32(1.3 * 2.0 ** -9)), float(np.float32(0.011)), 3 * 2.0 ** -12,
          float(np.float32(1.7e-4)), 1.5 * 2.0 ** 20, 1.25 * 2.0 ** -119]


@pytest.mark.parametrize("rot", [0, 64])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("scale", SCALES)
def test_scales_that_are_no_powers_of_two(rot, layout, scale):
    """Pages quantised elsewhere, half full: the tokens appended to them keep the scale and divide by it exactly."""
    page, old, H, B = 128, 3, 2, 12
    g = torch.Generator().manual_seed(2)
    cache = rp.PagedCache.empty(B, H, 64, page_size=page, dtype=E4)
    cache.k_scale.fill_(scale)
    cache.v_scale.fill_(scale)
    shift = 2.0 ** (-27 if scale > 1 else 110 if scale < 1e-30 else 0)
    near = torch.from_numpy(_ties(scale * shift) / shift)
    assert len(near) > 20
    n = page - old
    # the power of two below the scale has to hold sqrt(2) times them: a larger one would replace it
    most = 448 * 2.0 ** np.floor(np.log2(scale)) / 1.4143
    near = near[near <= most]
    kv = near[torch.randint(0, len(near), (B * n, 2 * H, 64), generator=g)]
    kv *= torch.randint(0, 2, kv.shape, generator=g) * 2 - 1
    kv[::3] = torch.randn(kv[::3].shape, generator=g, dtype=torch.float64) * most / 3
    kv = kv.to(BF).double().clamp(-0.99 * most, 0.99 * most).to(BF)
    cu = torch.arange(B + 1, dtype=torch.int32) * n
    table, lens = torch.randperm(B, generator=g).to(torch.int32)[:, None], torch.full((B,), page, dtype=torch.int32)
    want = _expect(_snapshot(cache), kv, table, cu, lens, page, H, rot, layout)
    assert np.all(want["k_scale"] == scale) and np.all(want["v_scale"] == scale)
    _append(cache, kv, table, cu, lens, H, rp.RotaryPlan(rot, layout=layout) if rot else None)
    _same(cache, want)


def _misleading():
    """Scales m 2^-32 whose product with a code, rounded to fp32 first, lands on a border that it is next to."""
    found = []
    for c in (9, 11, 13, 15):
        for border in range(17 * 2 ** 22, 64 * 2 ** 22, 2 ** 22):
            for m in (border // c, border // c + 1):
                y = c * m / 2.0 ** 26
                if 2 ** 23 <= m < 2 ** 24 and so.e4m3_round(y) != so.e4m3_round(float(np.float32(y))):
                    found.append(m * 2.0 ** -32)
    return found


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale", SCALES + _misleading()[::3])
def test_codes_that_leave_such_a_scale(d, scale):
    """A larger token moves the codes that are there to a power of two."""
    page, old = 64, 40
    g = torch.Generator().manual_seed(3)
    cache = rp.PagedCache.empty(8, 1, d, page_size=page, dtype=E4)
    codes = torch.randint(0, 256, (2, *cache.k.shape), generator=g, dtype=torch.uint8)
    codes[(codes & 0x7f) == 0x7f] = 0x30  # no NaN
    cache.k.view(torch.uint8).copy_(codes[0].cuda())
    cache.v.view(torch.uint8).copy_(codes[1].cuda())
    cache.k_scale.fill_(scale)
    cache.v_scale.fill_(scale)
    big = torch.tensor([450.0, 500.0, 1000.0, 2500.0, 9000.0, 450.0, 40000.0, 3e5])
    kv = (scale * big[:, None, None] * torch.ones(8, 2, d)).to(BF)
    cu, lens = torch.arange(9, dtype=torch.int32), torch.full((8,), old + 1, dtype=torch.int32)
    table = torch.randperm(8, generator=g).to(torch.int32)[:, None]
    want = _expect(_snapshot(cache), kv, table, cu, lens, page, 1)
    _append(cache, kv, table, cu, lens, 1)
    _same(cache, want)
