"""Measured cases of the serving operators: rotary positions (and their gradient), appending to a paged
key/value cache with the rotation on the way, and decoding over that cache.

``own = False`` computes each operator in elementary torch operations; ``own = True`` makes the calls a
user makes of the library. ``listed()`` are the cases, ``draw()`` gives more of the same ranges.

Definitions
  rotary   pairs (x1, x2) of the first ``rot`` dimensions of a head, at position p and frequency w_m:
           (x1 cos(p w_m) - x2 sin(p w_m), x1 sin(p w_m) + x2 cos(p w_m)) times the plan's amplitude.
           "half": x1 = x[m], x2 = x[m + rot / 2]; "interleaved": x1 = x[2m], x2 = x[2m + 1].
           w_m = base^(-2m / rot); "linear" divides it by the factor, "ntk" stretches the base, "yarn"
           interpolates by parts (rotations over the original length between 1 and 32) with amplitude
           0.1 ln(factor) + 1. The gradient is the rotation by -p.
  append   the last n_b of sequence b's len_b tokens are written to the pages its block table names: keys
           rotated at their positions, values as they are. 8-bit caches hold e4m3 codes and, for each page
           and head, a power-of-two scale: the smallest that holds the largest new magnitude (of keys, sqrt(2)
           and the amplitude times it: any rotation fits) in 448 times it, never smaller than the page's scale
           so far (a page whose first token is written starts afresh; codes there move to a larger scale).
  decode   softmax(q.k / sqrt(d) + bias) v over the first len_b tokens of the cache, grouped heads; query
           row i of Lq sits at position len_b - Lq + i and sees the keys up to its own position; bias none,
           T5 buckets (causal) or ALiBi. A row before the sequence's start is zero.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
BASE = 10000.0
ORIGINAL_LEN = 4096  # the length a stretched plan was trained at


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one new token of one sequence: the query's and key's heads of a decode step
        dict(name="rotary_one_token", op="rotary", B=1, L=1, Hq=16, Hk=16, d=64, rot=64, layout="half", scaling="none",
             factor=1.0, dtype="bf16", first=4095, order="blhd", backward=False),
        # a training batch, heads first as the attention kernels take it
        dict(name="rotary_train", op="rotary", B=4, L=2048, Hq=16, Hk=16, d=64, rot=64, layout="half", scaling="none",
             factor=1.0, dtype="bf16", first=0, order="bhld", backward=False),
        # the gradient of a ragged training batch: part of the head, interleaved, grouped keys
        dict(name="rotary_gradient", op="rotary", B=8, L=509, Hq=12, Hk=4, d=128, rot=64, layout="interleaved",
             scaling="none", factor=1.0, dtype="bf16", first=0, order="blhd", backward=True),
        # a long document in 32 bits with stretched positions, far from the origin
        dict(name="rotary_far_fp32", op="rotary", B=1, L=16411, Hq=16, Hk=4, d=128, rot=128, layout="half",
             scaling="yarn", factor=32.0, dtype="fp32", first=1000003, order="blhd", backward=False),
        # a decode step of a serving batch: one token of each sequence
        dict(name="append_step_8bit", op="append", B=32, new=1, old=4096, H=16, d=64, page=64, cache="e4m3", rot=64,
             layout="half", dtype="bf16"),
        # ragged prompts written at once
        dict(name="append_prompts_8bit", op="append", B=8, new=2048, old=0, H=16, d=64, page=64, cache="e4m3", rot=64,
             layout="half", dtype="bf16"),
        # chunks of long prompts behind what is cached, 16 bits, part of the head rotated
        dict(name="append_chunks_16bit", op="append", B=4, new=1001, old=3001, H=8, d=128, page=32, cache="bf16", rot=64,
             layout="interleaved", dtype="bf16"),
        # one short sequence: latency
        dict(name="decode_one_short", op="decode", B=1, len=113, ragged=False, Hq=16, Hkv=16, Lq=1, d=64, page=32,
             cache="bf16", bias="t5"),
        # the serving batch with the T5 bias, 8 bits
        dict(name="decode_t5_8bit", op="decode", B=32, len=4096, ragged=False, Hq=16, Hkv=16, Lq=1, d=64, page=64,
             cache="e4m3", bias="t5"),
        # ragged lengths, grouped heads
        dict(name="decode_ragged_grouped_8bit", op="decode", B=24, len=8191, ragged=True, Hq=32, Hkv=8, Lq=1, d=128,
             page=64, cache="e4m3", bias="none"),
        # few long contexts
        dict(name="decode_long_8bit", op="decode", B=2, len=131075, ragged=False, Hq=16, Hkv=4, Lq=1, d=128, page=128,
             cache="e4m3", bias="alibi"),
        # several new rows a sequence (drafted tokens to be checked), 16 bits
        dict(name="decode_rows_16bit", op="decode", B=16, len=4099, ragged=True, Hq=16, Hkv=4, Lq=5, d=64, page=32,
             cache="bf16", bias="t5"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "decode"])
    if op == "rotary":
        d = rng.choice([64, 64, 128, 128, 80, 32])
        L, Hq = _log_int(rng, 1, 8192), rng.choice([4, 8, 12, 16, 32])
        most = max(1, (1 << 26) // (L * Hq * d))
        return dict(op=op, B=min(_log_int(rng, 1, 32), most), L=L, Hq=Hq, Hk=rng.choice([1, 2, Hq]), d=d,
                    rot=rng.choice([d, d, d // 2]), layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "none", "linear", "ntk", "yarn"]), factor=rng.choice([2.0, 8.0, 40.0]),
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), first=rng.choice([0, _log_int(rng, 1, 1 << 20)]),
                    order=rng.choice(["bhld", "blhd"]), backward=rng.random() < 0.4)
    if op == "append":
        d, H = rng.choice([64, 128]), rng.choice([1, 4, 8, 16])
        new = 1 if rng.random() < 0.4 else _log_int(rng, 2, 4096)
        B = min(_log_int(rng, 1, 64), max(1, (1 << 24) // (new * H * d)))
        return dict(op=op, B=B, new=new, old=rng.choice([0, _log_int(rng, 1, 4096)]), H=H, d=d,
                    page=rng.choice([32, 64, 128]), cache=rng.choice(["e4m3", "bf16"]), rot=rng.choice([d, d, d // 2]),
                    layout=rng.choice(["half", "interleaved"]), dtype="bf16")
    d, Hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8, 16])
    n = _log_int(rng, 1, 65536)
    B = min(_log_int(rng, 1, 48), max(1, (1 << 27) // (n * Hkv * d)))
    return dict(op=op, B=B, len=n, ragged=rng.random() < 0.6, Hq=Hkv * rng.choice([1, 2, 4, 8]), Hkv=Hkv,
                Lq=rng.choice([1, 1, 1, 2, 3, 8]), d=d, page=rng.choice([32, 64, 128]), cache=rng.choice(["e4m3", "bf16"]),
                bias=rng.choice(["none", "t5", "alibi"]))


def _spread(case, most, b):
    """Element b's share of `most` in a ragged batch: between a sixth and all of it."""
    B = case["B"]
    return most if B == 1 else max(1, most * (1 + 5 * ((7 * b) % B) // (B - 1)) // 6) if (7 * b) % B else max(1, most // 6)


def _append_lens(case):
    """(new tokens, tokens in all) of each sequence."""
    new = [1 if case["new"] == 1 else _spread(case, case["new"], b) for b in range(case["B"])]
    old = [0 if case["old"] == 0 else max(0, case["old"] - 13 * b) for b in range(case["B"])]
    return new, [n + o for n, o in zip(new, old)]


def _decode_lens(case):
    return [max(1, _spread(case, case["len"], b)) if case["ragged"] else case["len"] for b in range(case["B"])]


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"rotary": _prepare_rotary, "append": _prepare_append, "decode": _prepare_decode}[case["op"]](case, g)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _dtype(name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}[name]


def _plan(case):
    import transformer_attention_relative_gb300 as rp
    return rp.RotaryPlan(case["rot"], layout=case["layout"], base=BASE, scaling=case.get("scaling", "none"),
                         factor=case.get("factor", 1.0), original_len=ORIGINAL_LEN)


def _prepare_rotary(case, g):
    B, L, d = case["B"], case["L"], case["d"]
    x = []
    for H in (case["Hq"], case["Hk"]):
        if case["order"] == "bhld":
            x.append(_randn(g, B, H, L, d).to(_dtype(case["dtype"])))
        else:
            x.append(_randn(g, B, L, H, d).to(_dtype(case["dtype"])).transpose(1, 2))
    # sequences of a batch start at different positions
    start = case["first"] + torch.arange(B, device="cuda") * 17
    pos = (start[:, None] + torch.arange(L, device="cuda")[None]).to(torch.int32)
    s = dict(case=case, q=x[0], k=x[1], pos=pos)
    if own:
        s["plan"] = _plan(case)
    return s


def _pages(case, lens, g):
    """A block table over a shuffled pool; -1 where a sequence has no page."""
    counts = [-(-n // case["page"]) for n in lens]
    pool = sum(counts) + 7
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, max(counts))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    return table, pool


def _quantised(x):
    """e4m3 codes and power-of-two scales of pages x [..., page, d]."""
    amax = x.abs().amax(dim=(-1, -2)).clamp(min=1e-30)
    scale = torch.exp2(torch.ceil(torch.log2(amax / E4M3_MAX)))
    return (x / scale[..., None, None]).to(torch.float8_e4m3fn), scale


def _pool(case, pool, H, g):
    """The cache's pages with keys and values in them, each page and head of a magnitude of its own."""
    s, shape = {}, (pool, H, case["page"], case["d"])
    for name, sigma in (("k", 1.5), ("v", 1.0)):
        if case["cache"] == "bf16":
            s[name] = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        else:
            s[name] = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
            s[name + "_scale"] = torch.empty(pool, H, device="cuda")
        step = max(1, (1 << 26) // (H * case["page"] * case["d"]))
        for a in range(0, pool, step):
            n = min(step, pool - a)
            x = _randn(g, n, *shape[1:]) * (sigma * torch.exp2(torch.randint(-1, 2, (n, H), generator=g, device="cuda").float() * 0.5))[..., None, None]
            if case["cache"] == "bf16":
                s[name][a:a + n] = x.to(torch.bfloat16)
            else:
                codes, s[name + "_scale"][a:a + n] = _quantised(x)
                s[name].view(torch.uint8)[a:a + n] = codes.view(torch.uint8)
    return s


def _handle(s, case):
    import transformer_attention_relative_gb300 as rp
    return rp.PagedCache(s["k"], s["v"], s.get("k_scale"), s.get("v_scale"))


def _prepare_append(case, g):
    new, lens = _append_lens(case)
    H, d = case["H"], case["d"]
    table, pool = _pages(case, lens, g)
    s = dict(case=case, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), **_pool(case, pool, H, g))
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    # one projection's output holds the keys' and the values' heads of every token
    kv = _randn(g, cu[-1], 2 * H, d) * torch.exp2(_randn(g, cu[-1], 2 * H, 1))
    kv = kv.to(_dtype(case["dtype"]))
    s["new_k"], s["new_v"] = kv[:, :H], kv[:, H:]
    if own:
        s["plan"], s["handle"] = _plan(case), _handle(s, case)
    return s


def _prepare_decode(case, g):
    lens = _decode_lens(case)
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    table, pool = _pages(case, lens, g)
    s = dict(case=case, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), **_pool(case, pool, Hkv, g))
    s["q"] = _randn(g, B, case["Lq"], Hq, d).to(torch.bfloat16).transpose(1, 2)
    if case["bias"] == "t5":
        s["bias"] = 0.5 * _randn(g, 32, Hq)
    elif case["bias"] == "alibi":
        s["bias"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], device="cuda")
    if own:
        s["handle"] = _handle(s, case)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return {"rotary": _run_rotary, "append": _run_append, "decode": _run_decode}[s["case"]["op"]](s)


def _frequencies(case, device):
    """w_m in 64 bits, and the amplitude."""
    rot, f = case["rot"], case.get("factor", 1.0)
    scaling, base = case.get("scaling", "none"), BASE
    if scaling == "ntk":
        base = BASE * f ** (rot / (rot - 2))
    w = base ** (-torch.arange(0, rot, 2, device=device, dtype=torch.float64) / rot)
    if scaling == "linear":
        w = w / f
    if scaling == "yarn":
        turns = ORIGINAL_LEN * w / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        return w / f * (1 - keep) + w * keep, 0.1 * math.log(f) + 1.0
    return w, 1.0


def _pairs(x, case):
    rot = case["rot"]
    if case["layout"] == "half":
        return x[..., :rot // 2], x[..., rot // 2:rot]
    return x[..., 0:rot:2], x[..., 1:rot:2]


def _joined(a, b, x, case):
    if case["layout"] == "half":
        return torch.cat([a, b, x[..., case["rot"]:]], -1)
    return torch.cat([torch.stack([a, b], -1).flatten(-2), x[..., case["rot"]:]], -1)


def _run_rotary(s):
    case = s["case"]
    if own:
        import transformer_attention_relative_gb300 as rp
        call = rp.rotary_backward if case["backward"] else rp.rotary
        return call(s["q"], s["plan"], s["k"], positions=s["pos"])
    w, amp = _frequencies(case, s["pos"].device)
    angle = s["pos"].double()[:, None, :, None] * w
    cos, sin = (torch.cos(angle) * amp).float(), (torch.sin(angle) * amp).float()
    if case["backward"]:
        sin = -sin
    out = []
    for x in (s["q"], s["k"]):
        x1, x2 = _pairs(x.float(), case)
        out.append(_joined(x1 * cos - x2 * sin, x1 * sin + x2 * cos, x.float(), case).to(x.dtype))
    return tuple(out)


def _round_e4m3(x):
    """x (64 bits) to the nearest e4m3 value, ties to even, saturating."""
    e = torch.frexp(x)[1].clamp(min=-5) - 4
    step = ((e.long() + 1023) << 52).view(torch.float64)  # 2^e
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX).float().to(torch.float8_e4m3fn)


def _scale_for(most):
    """The smallest power of two s with most <= 448 s."""
    f, e = torch.frexp(most / E4M3_MAX)
    e = torch.where(f == 0.5, e - 1, e)
    e = torch.where(most > 0, e, torch.full_like(e, -120)).clamp(-120, 120)
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)  # 2^e


def _run_append(s):
    case = s["case"]
    if own:
        import transformer_attention_relative_gb300 as rp
        rp.paged_append(s["handle"], s["new_k"], s["new_v"], s["table"], s["lens"], cu_new=s["cu"], plan=s["plan"])
        return [s[n] for n in ("k", "v", "k_scale", "v_scale") if n in s]
    page, cu, lens = case["page"], s["cu"].long(), s["lens"].long()
    new = cu[1:] - cu[:-1]
    b = torch.repeat_interleave(torch.arange(len(lens), device=cu.device), new, output_size=s["new_k"].shape[0])
    pos = torch.arange(s["new_k"].shape[0], device=cu.device) - cu[b] + (lens - new)[b]
    at, slot = s["table"][b, pos // page].long(), pos % page
    w, amp = _frequencies(case, pos.device)
    angle = pos.double()[:, None, None] * w
    k = s["new_k"].double()  # 64 bits: values next to a border of the 8-bit grid
    x1, x2 = _pairs(k, case)
    cos, sin = torch.cos(angle) * amp, torch.sin(angle) * amp
    rotated = _joined(x1 * cos - x2 * sin, x1 * sin + x2 * cos, k, case)
    if case["cache"] == "bf16":
        s["k"][at, :, slot] = rotated.float().to(torch.bfloat16)
        s["v"][at, :, slot] = s["new_v"].to(torch.bfloat16)
        return [s["k"], s["v"]]
    # no rotation takes a value beyond sqrt(2) times the largest one
    size_k = k.abs().amax(-1) * (math.sqrt(2.0) * amp)
    size_v = s["new_v"].double().abs().amax(-1)
    first = at.new_zeros(s["k"].shape[0], dtype=torch.bool)
    first[at[slot == 0]] = True
    touched = torch.zeros_like(first)
    touched[at] = True
    start = (lens - new)
    head = s["table"].gather(1, (start // page).clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0].long()
    head, upto = head[start % page > 0], (start % page)[start % page > 0]
    for name, size, x in (("k", size_k, rotated), ("v", size_v, s["new_v"].double())):
        codes, scale = s[name], s[name + "_scale"]
        most = torch.zeros(scale.shape, dtype=torch.float64, device=scale.device)
        most.scatter_reduce_(0, at[:, None].expand_as(size), size, "amax")
        want = _scale_for(most)
        want = torch.where(first[:, None], want, torch.maximum(want, scale))
        want = torch.where(touched[:, None], want, scale)
        # the codes that were in a page move to its new scale
        moved = (codes[head].float() * (scale[head] / want[head])[..., None, None]).to(torch.float8_e4m3fn)
        keep = torch.arange(page, device=at.device)[None] >= upto[:, None]
        held = codes.view(torch.uint8)
        held[head] = torch.where(keep[:, None, :, None], held[head], moved.view(torch.uint8))
        scale.copy_(want)
        held[at, :, slot] = _round_e4m3(x / want[at][..., None].double()).view(torch.uint8)
    return [s["k"], s["v"], s["k_scale"], s["v_scale"]]


def _t5_bucket(distance, slots=32, most=128):
    exact = slots // 2
    far = exact + (torch.log(distance.clamp(min=exact).double() / exact) / math.log(most / exact) * (slots - exact)).long()
    return torch.where(distance < exact, distance, far.clamp(max=slots - 1))


def _run_decode(s):
    case = s["case"]
    if own:
        import transformer_attention_relative_gb300 as rp
        mode = {"none": None, "t5": rp.MODE_T5, "alibi": rp.MODE_ALIBI}[case["bias"]]
        return rp.paged_decode(s["q"], s["handle"], s["table"], s["lens"], bias=s.get("bias"), mode=mode)
    B, Hq, Hkv, Lq, d = (case[n] for n in ("B", "Hq", "Hkv", "Lq", "d"))
    table = s["table"].long().clamp(min=0)
    n = table.shape[1] * case["page"]
    k, v = s["k"][table].float(), s["v"][table].float()  # [B, pages, Hkv, page, d]
    if case["cache"] != "bf16":
        k = k * s["k_scale"][table][..., None, None]
        v = v * s["v_scale"][table][..., None, None]
    k = k.transpose(1, 2).reshape(B, Hkv, n, d)
    v = v.transpose(1, 2).reshape(B, Hkv, n, d)
    q = s["q"].float().reshape(B, Hkv, Hq // Hkv * Lq, d)
    score = (q @ k.transpose(-1, -2)).view(B, Hq, Lq, n) / math.sqrt(d)
    key = torch.arange(n, device=q.device)
    back = (s["lens"].long()[:, None] - Lq + torch.arange(Lq, device=q.device))[:, :, None] - key  # query - key position
    if case["bias"] == "t5":
        score = score + s["bias"][_t5_bucket(back.clamp(min=0))].permute(0, 3, 1, 2)
    elif case["bias"] == "alibi":
        score = score - s["bias"][None, :, None, None] * back.abs().float()[:, None]
    hidden = (back < 0)[:, None]
    score = score.masked_fill(hidden, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-38)
    v = v.masked_fill((key[None] >= s["lens"][:, None])[:, None, :, None], 0.0)
    return (p.view(B, Hkv, -1, n) @ v).view(B, Hq, Lq, d).to(torch.bfloat16)


# ------------------------------------------------------------------ work and exact values

def work(case):
    if case["op"] == "rotary":
        n = case["B"] * case["L"] * (case["Hq"] + case["Hk"])
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": 2 * n * case["d"] * size + 4 * case["B"] * case["L"], "flops": 3 * n * case["rot"]}
    size = 1 if case["cache"] == "e4m3" else 2
    if case["op"] == "append":
        new, lens = _append_lens(case)
        n = sum(new) * case["H"]
        touched = sum(-(-t // case["page"]) - (t - c) // case["page"] for c, t in zip(new, lens))
        return {"bytes": 2 * n * case["d"] * (2 + size) + (16 * touched * case["H"] if size == 1 else 0) + 4 * touched + 8 * case["B"],
                "flops": 3 * n * case["rot"] + (4 * n * case["d"] if size == 1 else 0)}
    lens, d = _decode_lens(case), case["d"]
    pages = sum(-(-n // case["page"]) for n in lens)
    rows = case["B"] * case["Hq"] * case["Lq"]
    return {"bytes": 2 * sum(lens) * case["Hkv"] * d * size + (8 * pages * case["Hkv"] if size == 1 else 0) + 4 * pages + 4 * rows * d,
            "flops": 4 * sum(lens) * case["Hq"] * case["Lq"] * d}


def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "append": _exact_append, "decode": _exact_decode}[case["op"]](case, s)


def _exact_angles(case, positions):
    """cos and sin, amplitude included, [positions, rot / 2] in 64 bits."""
    rot, f, kind = case["rot"], case.get("factor", 1.0), case.get("scaling", "none")
    w, amp = [], 1.0
    for m in range(rot // 2):
        if kind == "ntk":
            w.append(math.pow(BASE * math.pow(f, rot / (rot - 2.0)), -2.0 * m / rot))
            continue
        x = math.pow(BASE, -2.0 * m / rot)
        if kind == "linear":
            x /= f
        elif kind == "yarn":
            part = min(1.0, max(0.0, (ORIGINAL_LEN * x / (2 * math.pi) - 1.0) / 31.0))
            x = x * part + x / f * (1.0 - part)
        w.append(x)
    if kind == "yarn":
        amp = 0.1 * math.log(f) + 1.0
    a = torch.outer(positions.double(), torch.tensor(w, dtype=torch.float64, device=positions.device))
    return torch.polar(torch.full_like(a, amp), a)


def _exact_rotation(x, turn, case):
    """x [..., d] in 64 bits times the unit complex numbers `turn` [..., rot / 2]."""
    rot, y = case["rot"], x.clone()
    a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if case["layout"] == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    z = torch.complex(x[..., a].contiguous(), x[..., b].contiguous()) * turn
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_rotary(case, s):
    turn = _exact_angles(case, s["pos"].reshape(-1)).view(case["B"], 1, case["L"], -1)
    turn = turn.conj() if case["backward"] else turn
    return tuple(_exact_rotation(s[n].double(), turn, case) for n in ("q", "k"))


def _exact_append(case, s):
    page = case["page"]
    new, lens = _append_lens(case)
    table = s["table"].tolist()
    cache = {n: s[n].double() for n in ("k", "v", "k_scale", "v_scale") if n in s}
    grid = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().to(s["k"].device)  # 0 .. 448
    middle = (grid[1:] + grid[:-1]) / 2

    def nearest(x):
        a = x.abs().contiguous()
        low, high = torch.searchsorted(middle, a), torch.searchsorted(middle, a, right=True)  # they differ on a tie
        return torch.where(torch.signbit(x), -1.0, 1.0).double() * grid[torch.where(low == high, low, low + low % 2)]

    def scale_of(length):
        e = torch.ceil(torch.log2(length.clamp(min=1e-60) / E4M3_MAX))
        e = torch.where(length > E4M3_MAX * torch.exp2(e), e + 1, e)
        e = torch.where(length <= E4M3_MAX * torch.exp2(e - 1), e - 1, e)
        return torch.exp2(e.clamp(-120, 120))

    at = 0
    for b, (n, total) in enumerate(zip(new, lens)):
        p = total - n
        while p < total:
            upto = min(total, (p // page + 1) * page)
            i, lo, hi = table[b][p // page], p % page, (upto - 1) % page + 1
            x = s["new_k"][at:at + upto - p].double().transpose(0, 1)  # [H, tokens, d]
            turn = _exact_angles(case, torch.arange(p, upto, device=x.device))
            y = _exact_rotation(x, turn, case)
            length = x.abs().amax((-1, -2)) * (math.sqrt(2.0) * abs(complex(turn.flatten()[0])))
            v = s["new_v"][at:at + upto - p].double().transpose(0, 1)
            for name, z, size in (("k", y, length), ("v", v, v.abs().amax((-1, -2)))):
                if case["cache"] == "bf16":
                    cache[name][i, :, lo:hi] = z
                    continue
                want, had = scale_of(size), cache[name + "_scale"][i].clone()
                if lo > 0:
                    want = torch.maximum(want, had)
                    cache[name][i, :, :lo] = nearest(cache[name][i, :, :lo] * (had / want)[:, None, None])
                cache[name + "_scale"][i] = want
                cache[name][i, :, lo:hi] = nearest((z / want[:, None, None]).clamp(-E4M3_MAX, E4M3_MAX))
            at += upto - p
            p = upto
    return [cache[n] for n in ("k", "v", "k_scale", "v_scale") if n in cache]


def _exact_decode(case, s):
    lens = _decode_lens(case)
    Hq, Hkv, Lq, d, page = (case[n] for n in ("Hq", "Hkv", "Lq", "d", "page"))
    out = torch.zeros(case["B"], Hq, Lq, d, dtype=torch.float64, device=s["q"].device)
    for b, n in enumerate(lens):
        i = s["table"][b, :-(-n // page)].long()
        for h in range(Hkv):
            k, v = s["k"][i, h].double(), s["v"][i, h].double()
            if case["cache"] != "bf16":
                k, v = k * s["k_scale"][i, h].double()[:, None, None], v * s["v_scale"][i, h].double()[:, None, None]
            k, v = k.reshape(-1, d)[:n], v.reshape(-1, d)[:n]
            for r in range(Lq):
                sees = n - Lq + r + 1
                if sees <= 0:
                    continue
                G = Hq // Hkv
                q = s["q"][b, h * G:(h + 1) * G, r].double()
                z = q @ k[:sees].T / math.sqrt(d)
                back = torch.arange(sees - 1, -1, -1, device=z.device)
                if case["bias"] == "alibi":
                    z -= s["bias"][h * G:(h + 1) * G].double()[:, None] * back
                elif case["bias"] == "t5":
                    ids = torch.where(back < 16, back, 31)
                    near = back[(back >= 16) & (back < 128)].tolist()
                    ids[(back >= 16) & (back < 128)] = torch.tensor(
                        [min(31, 16 + int(math.log(t / 16) / math.log(8) * 16)) for t in near], dtype=ids.dtype, device=ids.device)
                    z += s["bias"].double()[ids][:, h * G:(h + 1) * G].T
                out[b, h * G:(h + 1) * G, r] = torch.softmax(z, -1) @ v[:sees]
    return out
