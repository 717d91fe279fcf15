"""fp64 oracle of the serving operators: rotary positions, the paged key/value
cache and decoding over it -- test infrastructure only.

Written from the definitions ("Relative Position Embeddings, in depth",
sections "ALiBi and RoPE: the two endpoints" and "Kernels and the KV cache",
and the readings stated in the C header); shares no code with the library.
"""
from __future__ import annotations

import math

import numpy as np

from .relpos_oracle import t5_bucket

E4M3_MAX = 448.0


def rotary_frequencies(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                       original_len: float = 0.0, fast_turns: float = 32.0, slow_turns: float = 1.0):
    """(w_m for m < rot / 2, amplitude)."""
    m = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2.0))
    w = base ** (-2.0 * m / rot)
    if scaling == "linear":
        return w / factor, 1.0
    if scaling == "yarn":
        turns = original_len * w / (2.0 * math.pi)
        g = np.clip((turns - slow_turns) / (fast_turns - slow_turns), 0.0, 1.0)
        return (1.0 - g) * w / factor + g * w, 0.1 * math.log(factor) + 1.0
    return w, 1.0


def rotary(x, positions, rot: int, layout: str = "half", inverse: bool = False, **freq):
    """x [..., L, d] turned at positions [L] (or broadcastable [..., L])."""
    w, amp = rotary_frequencies(rot, **freq)
    ang = np.asarray(positions, dtype=np.float64)[..., None] * w
    cos, sin = amp * np.cos(ang), amp * np.sin(ang) * (-1.0 if inverse else 1.0)
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    return y


def e4m3_round(x):
    """Nearest e4m3 value, ties to even, saturating; NaN stays."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        _, e = np.frexp(np.where(np.isfinite(x), x, 1.0))
        step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
        return np.where(np.isnan(x), np.nan, np.clip(np.rint(x / step) * step, -E4M3_MAX, E4M3_MAX))


def e4m3_scale(most: float) -> float:
    """The smallest power of two s, within 2^-120 .. 2^120, with most <= 448 s."""
    if not most > 0.0:
        return 2.0 ** -120
    if math.isinf(most):
        return 2.0 ** 120
    e = -120
    while e < 120 and most / E4M3_MAX > 2.0 ** e:
        e += 1
    return 2.0 ** e


def paged_append(cache, K, V, table, start: int, page: int, rot: int = 0, layout: str = "half", **freq):
    """Write one sequence's new tokens K, V [H, n, d] at positions start ..
    into `cache`: a dict of "k", "v" (values of the codes where it is 8 bits)
    [pages, H, page, d] and, for an 8-bit cache, "k_scale", "v_scale"."""
    n = K.shape[1]
    pos = np.arange(start, start + n)
    amp = rotary_frequencies(rot, **freq)[1] if rot else 1.0
    reach = math.sqrt(2.0) * amp if rot else 1.0
    turned = rotary(K, pos, rot, layout, **freq) if rot else np.asarray(K, dtype=np.float64)
    at = 0
    while at < n:
        p = start + at
        lo = p % page
        m = min(page - lo, n - at)
        i = table[p // page]
        for name, x, raw, g in (("k", turned, K, reach), ("v", np.asarray(V, dtype=np.float64), V, 1.0)):
            x = x[:, at:at + m]
            if "k_scale" not in cache:
                cache[name][i, :, lo:lo + m] = x
                continue
            for h in range(K.shape[0]):
                mag = np.abs(np.asarray(raw[h, at:at + m], dtype=np.float64))
                mag = mag[~np.isnan(mag)]
                want = e4m3_scale(float(mag.max()) * g if mag.size else 0.0)
                if lo > 0:
                    had = cache[name + "_scale"][i, h]
                    want = max(want, had)
                    cache[name][i, h, :lo] = e4m3_round(cache[name][i, h, :lo] * (had / want))
                cache[name + "_scale"][i, h] = want
                cache[name][i, h, lo:lo + m] = e4m3_round(x[h] / want)
        at += m
    return cache


def paged_decode(Q, cache, table, lens, page: int, bias=None, mode: str = "none", num_buckets: int = 32,
                 max_distance: int = 128, scale: float = 0.0):
    """(out, weight): out [B, Hq, Lq, d], and sum_j p_j |v_j| beside it, the
    size that errors of the weights scale with."""
    B, Hq, Lq, d = Q.shape
    Hkv = cache["k"].shape[1]
    G = Hq // Hkv
    s = scale if scale else 1.0 / math.sqrt(d)
    out, size = np.zeros(Q.shape), np.zeros(Q.shape)
    for b in range(B):
        n = int(lens[b])
        if n <= 0:
            continue
        pages = [int(i) for i in table[b][:(n + page - 1) // page]]
        for h in range(Hkv):
            kv = []
            for name in ("k", "v"):
                x = cache[name][pages, h].astype(np.float64)
                if "k_scale" in cache:
                    x = x * cache[name + "_scale"][pages, h].astype(np.float64)[:, None, None]
                kv.append(x.reshape(-1, d)[:n])
            for hq in range(h * G, (h + 1) * G):
                for i in range(Lq):
                    p = n - Lq + i
                    if p < 0:
                        continue
                    z = kv[0][:p + 1] @ Q[b, hq, i].astype(np.float64) * s
                    back = p - np.arange(p + 1)
                    if mode == "alibi":
                        z = z - float(bias[hq]) * back
                    elif mode == "t5":
                        ids = [t5_bucket(-int(t), False, num_buckets, max_distance) for t in back]
                        z = z + np.asarray(bias, dtype=np.float64)[ids, hq]
                    e = np.exp(z - z.max())
                    e /= e.sum()
                    out[b, hq, i] = e @ kv[1][:p + 1]
                    size[b, hq, i] = e @ np.abs(kv[1][:p + 1])
    return out, size
