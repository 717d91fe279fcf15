"""Pins of the serving operators' oracle (CPU): closed forms, library
reductions, and the attention oracle on a contiguous cache."""
import math

import numpy as np
import pytest
import torch

from oracle import relpos_oracle as orc
from oracle import serving_oracle as so

rng = np.random.default_rng(11)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_two_dimensions_turn_by_the_position(layout):
    """rot = 2: one pair at frequency 1, so position p turns it by p radians."""
    x = np.array([[[1.0, 0.0, 5.0, -3.0], [0.0, 1.0, 5.0, -3.0]]])
    y = so.rotary(x, [2, 2], 2, layout)
    np.testing.assert_allclose(y[0, 0], [math.cos(2), math.sin(2), 5, -3], atol=1e-15)
    np.testing.assert_allclose(y[0, 1], [-math.sin(2), math.cos(2), 5, -3], atol=1e-15)


def test_layouts_name_the_same_pairs():
    x = rng.standard_normal((3, 8))
    paired = np.concatenate([x[:, 0::2], x[:, 1::2]], -1)
    a, b = so.rotary(x, [1, 2, 3], 8, "interleaved"), so.rotary(paired, [1, 2, 3], 8, "half")
    np.testing.assert_allclose(np.concatenate([a[:, 0::2], a[:, 1::2]], -1), b, atol=1e-14)


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
def test_products_depend_on_the_offset_alone(scaling):
    f = dict(scaling=scaling, factor=4.0, original_len=64.0)
    q, k = rng.standard_normal((2, 1, 16))
    at = [float((so.rotary(q, [p], 16, **f) * so.rotary(k, [p - 5], 16, **f)).sum()) for p in (5, 77, 4000)]
    np.testing.assert_allclose(at, at[0], rtol=1e-10)
    back = so.rotary(so.rotary(q, [9], 16, **f), [9], 16, inverse=True, **f)
    np.testing.assert_allclose(back, q * so.rotary_frequencies(16, **f)[1] ** 2, atol=1e-13)


def test_stretched_frequencies():
    w, a = so.rotary_frequencies(8)
    np.testing.assert_allclose(w, [1.0, 0.1, 0.01, 0.001])
    assert a == 1.0
    np.testing.assert_allclose(so.rotary_frequencies(8, scaling="linear", factor=4.0)[0], w / 4)
    # NTK: the fastest frequency stays, the slowest is divided by the factor
    n = so.rotary_frequencies(8, scaling="ntk", factor=4.0)[0]
    np.testing.assert_allclose([n[0], n[-1]], [1.0, 0.001 / 4])
    # by parts: over 32 turns kept, under one turn interpolated
    y, a = so.rotary_frequencies(8, scaling="yarn", factor=4.0, original_len=300.0)
    np.testing.assert_allclose([y[0], y[-1], y[-2]], [1.0, 0.001 / 4, 0.01 / 4])
    turns = 300 * 0.1 / (2 * math.pi)
    g = (turns - 1) / 31
    np.testing.assert_allclose(y[1], (1 - g) * 0.1 / 4 + g * 0.1)
    np.testing.assert_allclose(a, 0.1 * math.log(4.0) + 1.0)


def test_gradient_is_the_inverse_turn():
    x, dy = rng.standard_normal((2, 3, 12))
    f = dict(scaling="yarn", factor=8.0, original_len=40.0)
    g = so.rotary(dy, [3, 50, 7], 8, "interleaved", inverse=True, **f)
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = 1e-3
        d = ((so.rotary(x + e, [3, 50, 7], 8, "interleaved", **f) -
              so.rotary(x - e, [3, 50, 7], 8, "interleaved", **f)) * dy).sum() / 2e-3
        assert abs(d - g[i]) < 1e-9


def test_e4m3_rounding_against_torch():
    x = np.concatenate([rng.standard_normal(2000) * 10.0 ** rng.uniform(-4, 2, 2000), [0.0, 448.0, 1e-9, 2.0 ** -10]])
    codes = np.arange(127, dtype=np.uint8)
    grid = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    x = np.concatenate([x, grid, -grid, (grid[1:] + grid[:-1]) / 2])  # the grid, and its ties
    x = np.clip(x, -448, 448)
    want = torch.from_numpy(x.astype(np.float32).astype(np.float64)).float().to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(so.e4m3_round(x.astype(np.float32).astype(np.float64)), want)
    assert so.e4m3_round(1e9) == 448 and np.isnan(so.e4m3_round(np.nan))


def test_scales_are_the_smallest_powers_that_hold():
    for most in (448.0, 447.9, 448.1, 896.0, 1.0, 3e-5, 1e30):
        s = so.e4m3_scale(most)
        assert most <= 448 * s and (most > 448 * s / 2) and math.log2(s) == round(math.log2(s))
    assert so.e4m3_scale(0.0) == 2.0 ** -120 and so.e4m3_scale(1e300) == 2.0 ** 120


def _contiguous(B, H, n, page, d):
    """K, V [B, H, n, d] and the same in pages handed out in a mixed order."""
    K, V = rng.standard_normal((2, B, H, n, d))
    per = (n + page - 1) // page
    table = rng.permutation(B * per + 2)[:B * per].reshape(B, per)
    cache = {x: np.full((B * per + 2, H, page, d), np.nan) for x in ("k", "v")}
    for b in range(B):
        so.paged_append(cache, K[b, :, :5], V[b, :, :5], table[b], 0, page)
        so.paged_append(cache, K[b, :, 5:], V[b, :, 5:], table[b], 5, page)
    return K, V, cache, table


@pytest.mark.parametrize("mode", ["none", "t5", "alibi"])
def test_decode_is_the_attention_of_the_last_rows(mode):
    B, H, n, d = 2, 3, 75, 8
    K, V, cache, table = _contiguous(B, H, n, 32, d)
    Q = rng.standard_normal((B, H, 2, d))
    bias = {"none": None, "t5": rng.standard_normal((32, H)), "alibi": np.abs(rng.standard_normal(H))}[mode]
    got, size = so.paged_decode(Q, cache, table, [n, n], 32, bias, mode)
    if mode == "none":
        mask = torch.arange(n)[None] <= torch.tensor([[n - 2], [n - 1]])
        ref = torch.nn.functional.scaled_dot_product_attention(*map(torch.from_numpy, (Q, K, V)), attn_mask=mask).numpy()
    else:
        ref = orc.attention(orc.MODE_T5 if mode == "t5" else orc.MODE_ALIBI, Q, K, V, bias, causal=True, q_offset=n - 2)
    np.testing.assert_allclose(got, ref, atol=1e-12)
    assert np.all(size >= np.abs(got) - 1e-12)


def test_decode_groups_heads_and_leaves_early_rows_zero():
    K, V, cache, table = _contiguous(1, 2, 6, 32, 8)
    Q = rng.standard_normal((1, 4, 3, 8))
    got, _ = so.paged_decode(Q, cache, table, [2], 32)
    assert np.all(got[:, :, 0] == 0)  # position -1
    for hq in range(4):
        np.testing.assert_allclose(got[0, hq, 1], V[0, hq // 2, 0])  # position 0 sees itself alone
    assert np.all(so.paged_decode(Q, cache, table, [0], 32)[0] == 0)


def test_append_grows_a_page_scale_and_moves_its_codes():
    cache = {x: np.zeros((1, 1, 32, 8)) for x in ("k", "v")} | {x: np.ones((1, 1)) for x in ("k_scale", "v_scale")}
    small, large = np.full((1, 1, 8), 1.0), np.full((1, 1, 8), 600.0)
    so.paged_append(cache, small, small, [0], 0, 32)
    assert cache["v_scale"][0, 0] == 2.0 ** -8 and np.all(cache["v"][0, 0, 0] == 256.0)
    so.paged_append(cache, large, large, [0], 1, 32)
    assert cache["v_scale"][0, 0] == 2.0 and np.all(cache["v"][0, 0, 0] == 0.5) and np.all(cache["v"][0, 0, 1] == 288.0)
    so.paged_append(cache, small, small, [0], 2, 32)
    assert cache["v_scale"][0, 0] == 2.0  # it does not shrink
    so.paged_append(cache, small, small, [0], 0, 32)
    assert cache["v_scale"][0, 0] == 2.0 ** -8  # a page taken anew
