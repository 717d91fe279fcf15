"""Codes of an 8-bit append where fp32 arithmetic alone would miss them: pairs whose
rotation overflows. They equal the fp64 oracle's, bit for bit."""
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
