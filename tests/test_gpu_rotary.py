"""Rotary positions and their gradient vs the fp64 oracle.

Tolerances: one rounding of the result, half a step of its type (2^-8 of it in
bf16, 2^-24 in fp32), and the fp32 arithmetic before it: sine and cosine off by
at most 2^-23 (angle and series), amplitude, two products and a sum, each off by
2^-24 of |x1| + |x2| <= 2 max(|x1|, |x2|): under 2^-21 amplitude (|x1| + |x2|)."""
import numpy as np
import pytest
import torch

import gpu_util as G
import transformer_attention_relative_gb300 as rp
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def _x(shape, dtype, seed, order="bhld"):
    g = torch.Generator().manual_seed(seed)
    B, H, L, d = shape
    if order == "bhld":
        return torch.randn(B, H, L, d, generator=g).to(dtype).cuda()
    return torch.randn(B, L, H, d, generator=g).to(dtype).cuda().transpose(1, 2)


def _check(got, x, pos, rot, layout="half", inverse=False, **freq):
    f = dict(freq)
    xd = x.double().cpu().numpy()
    pos = np.broadcast_to(np.asarray(pos, dtype=np.int64), (x.shape[0], x.shape[2]))[:, None]
    ref = so.rotary(xd, pos, rot, layout, inverse, **f)
    amp = so.rotary_frequencies(rot, **f)[1]
    size = np.abs(xd)
    if layout == "half":
        h = rot // 2
        pair = size[..., :h] + size[..., h:rot]
        size = np.concatenate([pair, pair, 0 * size[..., rot:]], -1)
    else:
        pair = size[..., 0:rot:2] + size[..., 1:rot:2]
        size = np.concatenate([np.repeat(pair, 2, -1), 0 * size[..., rot:]], -1)
    got_d = got.double().cpu().numpy()
    assert got.shape == x.shape and got.dtype == x.dtype
    tol = np.abs(ref) * torch.finfo(x.dtype).eps / 2 + 2.0 ** -21 * amp * size
    assert np.all(np.abs(got_d - ref) <= tol), float((np.abs(got_d - ref) - tol).max())
    np.testing.assert_array_equal(got_d[..., rot:], xd[..., rot:])  # the rest of the head as it was


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 64), (80, 40), (32, 8), (6, 2), (10, 6), (256, 256)])
def test_sizes(dtype, layout, d, rot):
    q, k = _x((2, 3, 5, d), dtype, 1), _x((2, 1, 5, d), dtype, 2, "blhd")
    plan = rp.RotaryPlan(rot, layout=layout)
    yq, yk = rp.rotary(q, plan, k, offset=11)
    for y, x in ((yq, q), (yk, k)):
        _check(y, x, np.arange(11, 16), rot, layout)
    assert torch.equal(rp.rotary(q, plan, offset=11), yq)  # one tensor, the same bits


@pytest.mark.parametrize("L", [1, 2, 31, 33, 257, 2048])
@pytest.mark.parametrize("order", ["bhld", "blhd"])
def test_lengths_and_orders(L, order):
    q = _x((2, 5, L, 64), BF, 3, order)
    y = rp.rotary(q, rp.RotaryPlan(64))
    assert y.stride() == q.stride()
    _check(y, q, np.arange(L), 64)


@pytest.mark.parametrize("freq", [dict(scaling="linear", factor=8.0), dict(scaling="ntk", factor=4.0),
                                  dict(scaling="yarn", factor=32.0, original_len=4096.0),
                                  dict(scaling="yarn", factor=2.0, original_len=100.0, fast_turns=8.0, slow_turns=0.5),
                                  dict(base=500000.0)])
@pytest.mark.parametrize("backward", [False, True])
def test_scalings(freq, backward):
    q = _x((1, 4, 70, 128), F32, 4)
    call = rp.rotary_backward if backward else rp.rotary
    y = call(q, rp.RotaryPlan(128, **freq), offset=5000)
    _check(y, q, np.arange(5000, 5070), 128, inverse=backward, **freq)


def test_far_and_negative_positions():
    """Angles of positions up to 2^31: frequencies and angles in 64 bits are off
    by a few 2^-53 relative on both sides (power, division, product: six in
    all), which the bound adds, 4 p 2^-52."""
    pos = torch.tensor([0, 1, -1, -1000003, 10 ** 6, 10 ** 7 + 1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    q = _x((1, 2, 8, 64), F32, 5)
    y = rp.rotary(q, rp.RotaryPlan(64), positions=pos.cuda())
    ref = so.rotary(q.double().cpu().numpy(), pos.numpy(), 64)
    size = np.abs(q.double().cpu().numpy())
    size = np.tile(size[..., :32] + size[..., 32:], 2)
    tol = np.abs(ref) * 2.0 ** -24 + size * (2.0 ** -21 + np.abs(pos.numpy().astype(float))[:, None] * 2.0 ** -50)
    assert np.all(np.abs(y.double().cpu().numpy() - ref) <= tol)


@pytest.mark.parametrize("shared", [True, False])
def test_positions(shared):
    q = _x((3, 2, 9, 64), BF, 6)
    g = torch.Generator().manual_seed(7)
    pos = torch.randint(0, 100000, (9,) if shared else (3, 9), generator=g, dtype=torch.int32)
    plan = rp.RotaryPlan(64, layout="interleaved")
    _check(rp.rotary(q, plan, positions=pos.cuda()), q, pos.numpy(), 64, "interleaved")
    wide = torch.zeros(3, 20, dtype=torch.int32).cuda()  # a slice of a wider table
    wide[:, 4:13] = pos.cuda()
    _check(rp.rotary(q, plan, positions=wide[:, 4:13]), q, pos.numpy(), 64, "interleaved")


@pytest.mark.parametrize("cut", [0, 1, 4])
def test_slices_of_a_projection(cut):
    """Heads sliced out of a fused projection at odd places: rows that start on
    16, 2 and 8 bytes."""
    B, L, H, d = 2, 7, 3, 64
    fused = _x((B, 1, L, 3 * H * d + 8), BF, 8)[:, 0]
    q = fused[..., cut:cut + H * d].view(B, L, H, d) if cut == 0 else fused[..., cut:].as_strided(
        (B, L, H, d), (fused.stride(0), fused.stride(1), d, 1), fused.storage_offset() + cut)
    q = q.transpose(1, 2)
    _check(rp.rotary(q, rp.RotaryPlan(64)), q, np.arange(L), 64)


def test_in_place_and_out():
    q, k = _x((2, 3, 40, 64), BF, 9), _x((2, 2, 40, 64), BF, 10)
    plan = rp.RotaryPlan(32)
    want = rp.rotary(q, plan, k)
    out = (torch.empty_like(q), torch.full((2, 40, 2, 64), 7.0, dtype=BF, device="cuda").transpose(1, 2))
    assert rp.rotary(q, plan, k, out=out)[1] is out[1]
    a, b = q.clone(), k.clone()
    rp.rotary(a, plan, b, out=(a, b))
    for w, o, i in zip(want, out, (a, b)):
        assert torch.equal(w, o) and torch.equal(w, i)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient(layout):
    freq = dict(scaling="yarn", factor=8.0, original_len=64.0)
    plan = rp.RotaryPlan(48, layout=layout, **freq)
    x, dy = _x((2, 3, 33, 64), F32, 11), _x((2, 3, 33, 64), F32, 12)
    g = rp.rotary_backward(dy, plan, offset=3)
    _check(g, dy, np.arange(3, 36), 48, layout, True, **freq)
    # against differences: the map is linear, so a large step has no truncation
    # error; each output is off by less than 2^-21 amplitude (|x1| + |x2|), on
    # both sides of the difference and in the gradient
    e = _x((2, 3, 33, 64), F32, 13)
    y = (rp.rotary(x + e, plan, offset=3).double() - rp.rotary(x, plan, offset=3).double()) * dy.double()
    want = (g.double() * ((x + e).double() - x.double())).sum()
    largest = float(x.abs().max() + (x + e).abs().max())
    assert abs(float(y.sum() - want)) <= 2.0 ** -21 * 1.21 * float(dy.abs().double().sum()) * 4 * largest


def test_odd_values():
    """Infinities and NaN stay within their pair; the largest finite values turn
    without overflow on the way."""
    q = torch.zeros(1, 1, 2, 64, dtype=F32, device="cuda")
    q[0, 0, 1, 3] = float("nan")
    q[0, 0, 1, 5] = float("inf")
    q[0, 0, 1, 7] = 1e38
    y = rp.rotary(q, rp.RotaryPlan(64))[0, 0, 1].cpu()
    assert y[3].isnan() and y[35].isnan() and not y[5].isfinite() and not y[37].isfinite()
    assert y[7].isfinite() and y[39].isfinite() and torch.count_nonzero(y) == 6


def test_empty_sizes():
    plan = rp.RotaryPlan(64)
    for shape in ((0, 2, 3, 64), (2, 0, 3, 64), (2, 2, 0, 64)):
        assert rp.rotary(torch.zeros(shape, dtype=BF, device="cuda"), plan).shape == shape


def test_more_heads_than_a_launch_dimension():
    """One token of 80000 heads: more groups of heads than a grid is high."""
    q, k = _x((1, 40000, 1, 2), BF, 16), _x((1, 40000, 1, 2), BF, 17)
    plan = rp.RotaryPlan(2)
    for y, x in zip(rp.rotary(q, plan, k, offset=3), (q, k)):
        _check(y, x, [3], 2)


def test_side_stream_and_graph():
    q = _x((2, 4, 100, 64), BF, 14)
    plan, pos = rp.RotaryPlan(64), torch.arange(100, dtype=torch.int32, device="cuda")
    want = rp.rotary(q, plan, positions=pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = rp.rotary(q, plan, positions=pos)
    s.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = rp.rotary(q, plan, positions=pos)
        z = rp.rotary_backward(y, plan, positions=pos)
    pos += 7
    g.replay()
    _check(y, q, np.arange(7, 107), 64)
    torch.cuda.synchronize()
    assert (z.float() - q.float()).abs().max() <= 2.0 ** -7 * 1.5 * q.abs().max()  # two bf16 roundings of a pair


def test_refusals():
    q = _x((1, 2, 4, 64), BF, 15)
    plan = rp.RotaryPlan(64)
    for call in (lambda: rp.rotary(q, plan, q[:, :, :3]), lambda: rp.rotary(q, plan, out=q[:, :1]),
                 lambda: rp.rotary(q, plan, positions=torch.arange(5, dtype=torch.int32, device="cuda")),
                 lambda: rp.rotary(q, plan, positions=torch.arange(4, dtype=torch.int32)),
                 lambda: rp.rotary(q.transpose(2, 3), plan), lambda: rp.rotary(q, plan, q, out=(q,))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: rp.rotary(q, plan, q.float()), lambda: rp.rotary(q, plan, out=q.float()),
                 lambda: rp.rotary(q, plan, positions=torch.arange(4, device="cuda"))):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(rp.RelposError):
        rp.rotary(q, rp.RotaryPlan(128))


def test_broadcast_rows():
    """One row for every head and position: read as it lies, never written over."""
    plan = rp.RotaryPlan(64)
    x = torch.randn(2, 1, 1, 64, device="cuda").to(torch.bfloat16).expand(2, 3, 9, 64)
    assert torch.equal(rp.rotary(x, plan), rp.rotary(x.contiguous(), plan))
    with pytest.raises(rp.RelposError) as e:
        rp.rotary(x, plan, out=x)
    assert e.value.code == rp.RELPOS_ERR_INVALID_ARG
