"""Measured cases of the operators around drafted tokens and the pages of a paged key/value cache: attention of a tree
of drafted tokens over the cache, keeping the accepted ones, giving pages to sequences (growing, freeing, forking) and
copying pages.

``own = False`` computes each operator in elementary torch operations; ``own = True`` makes the calls a user makes of
the library. ``listed()`` are the cases, ``draw()`` gives more of the same ranges.

Definitions
  tree     the last n_b of sequence b's len_b tokens are drafted: node i lies in slot base + i (base = len_b - n_b) and
           has the parent a(i) < i, or -1. Its depth is 0 without a parent, else one more than its parent's; its position
           is base + depth. Row i sees the slots below base, itself and its ancestors:
           softmax(q.k / sqrt(d) + bias) v over those, grouped heads; bias none, T5 buckets (causal) of the distance
           between positions, or ALiBi. Rows from n_b on are zero.
  compact  of the n_b drafted tokens the `count` listed ones are kept: slot base + i takes what slot base + kept[i] held,
           keys and values. In 8-bit pages a page that gets tokens of another page takes the larger of its own and those
           pages' scales; its codes move to it, rounded to nearest.
  assign   pages for new rows of a block table. The old rows give up their references; new row i continues old row
           source[i] for the first keep = min(its length, new_lens[i]) tokens: pages that those fill are shared; a last
           page that they fill in part stays with the lowest such row unless somebody else holds the page (another new
           row as a full page, or a reference from elsewhere), the others get a fresh page and an entry (from, to,
           tokens) in the list of copies. What new_lens[i] needs beyond is fresh. Fresh pages are those without a
           reference, lowest number first, to the rows in order; entries behind a row's last page are -1.
  copy     of each listed (from, to, tokens): the first `tokens` slots' keys and values of page `from`, and its scales,
           go to page `to`; an entry of -1 is none.
"""
import math

import torch

own = False

E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one short sequence with a small tree: latency
        dict(name="tree_one_short", op="tree", B=1, len=113, ragged=False, nodes=8, Hq=16, Hkv=16, d=64, page=32,
             cache="bf16", bias="t5"),
        # the serving batch with the T5 bias, 8 bits, 16 drafted tokens each
        dict(name="tree_t5_8bit", op="tree", B=32, len=4096, ragged=False, nodes=16, Hq=16, Hkv=16, d=64, page=64,
             cache="e4m3", bias="t5"),
        # ragged lengths and trees, grouped heads: up to 132 rows of a key/value head
        dict(name="tree_ragged_grouped_8bit", op="tree", B=24, len=8191, ragged=True, nodes=33, Hq=32, Hkv=8, d=128,
             page=64, cache="e4m3", bias="none"),
        # few long contexts, wide trees: 256 rows of a key/value head
        dict(name="tree_long_8bit", op="tree", B=2, len=131075, ragged=False, nodes=64, Hq=16, Hkv=4, d=128, page=128,
             cache="e4m3", bias="alibi"),
        # 16 bits, ragged, 100 rows of a key/value head
        dict(name="tree_ragged_16bit", op="tree", B=16, len=4099, ragged=True, nodes=25, Hq=16, Hkv=4, d=64, page=32,
             cache="bf16", bias="t5"),
        # after a step of the serving batch: up to 5 of 16 drafted tokens were right
        dict(name="compact_step_8bit", op="compact", B=32, len=4096, nodes=16, keep=5, H=16, d=64, page=64, cache="e4m3"),
        # large batch, wide trees over several pages, 16 bits
        dict(name="compact_batch_16bit", op="compact", B=256, len=611, nodes=64, keep=17, H=8, d=128, page=32, cache="bf16"),
        # a step of beam search: 16 groups of 4 beams take new parents and grow by a token
        dict(name="assign_beams", op="assign", B=64, len=1000, new=1, group=4, page=32, pool=4096, outside=0),
        # a large batch grows by a page or so each, some end, some are forked, over a shared prefix
        dict(name="assign_batch", op="assign", B=512, len=16384, new=70, group=2, page=64, pool=262144, outside=33),
        # the beams' unfilled pages
        dict(name="copy_tails_8bit", op="copy", N=64, every=3, whole=False, H=16, d=64, page=64, pool=256, cache="e4m3"),
        # long sequences forked into pages of their own
        dict(name="copy_pages_16bit", op="copy", N=1024, every=1, whole=True, H=8, d=128, page=64, pool=2100, cache="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "compact", "assign", "copy"])
    page = rng.choice([32, 64, 128])
    if op == "tree":
        d, Hkv, G = rng.choice([64, 128]), rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 1, 2, 4, 8])
        nodes = _log_int(rng, 1, 64)
        # no more keys and products than the largest listed case
        cache = rng.choice(["e4m3", "bf16"])
        keys, rows = (1 << (27 if cache == "e4m3" else 26)) // (Hkv * d), (1 << 34) // (Hkv * G * nodes * d)
        n = min(nodes + _log_int(rng, 1, 65536), keys, rows)
        most = min(keys, rows) // n
        return dict(op=op, B=min(_log_int(rng, 1, 48), max(1, most)), len=n, ragged=rng.random() < 0.6, nodes=nodes,
                    Hq=Hkv * G, Hkv=Hkv, d=d, page=page, cache=cache,
                    bias=rng.choice(["none", "t5", "alibi"]))
    if op == "compact":
        keep = _log_int(rng, 1, 24)
        nodes = rng.randint(2 * keep, 64)
        return dict(op=op, B=_log_int(rng, 1, 256), len=nodes + rng.choice([0, _log_int(rng, 1, 4096)]), nodes=nodes,
                    keep=keep, H=rng.choice([1, 4, 8]), d=rng.choice([64, 128]), page=page,
                    cache=rng.choice(["e4m3", "bf16"]))
    if op == "assign":
        B, n, new = _log_int(rng, 1, 512), _log_int(rng, 1, 7000), rng.choice([1, _log_int(rng, 1, 300)])
        return dict(op=op, B=B, len=n, new=new, group=rng.choice([1, 2, 4, 5]), page=page,
                    pool=2 * B * ((n + new) // page + 2) + rng.randint(0, 9999), outside=rng.choice([0, 0, 7]))
    N, H, d = _log_int(rng, 1, 512), rng.choice([1, 4, 8, 16]), rng.choice([64, 128])
    N = min(N, max(1, (1 << 26) // (H * page * d)))
    return dict(op=op, N=N, every=rng.choice([1, 1, 2, 3]), whole=rng.random() < 0.5, H=H, d=d, page=page,
                pool=2 * N + rng.randint(0, 50), cache=rng.choice(["e4m3", "bf16"]))


def _share(b, B):
    """Element b's share in a ragged batch, in sixths: between one and six."""
    return 6.0 if B == 1 else 1.0 + 5.0 * ((7 * b) % B) / (B - 1)


def _tree_sizes(case):
    """(nodes, tokens in all) of each sequence."""
    B = case["B"]
    nodes = [max(1, int(case["nodes"] * _share(B - 1 - b, B) / 6)) if case["ragged"] else case["nodes"] for b in range(B)]
    lens = [max(nodes[b], int(case["len"] * _share(b, B) / 6)) if case["ragged"] else case["len"] for b in range(B)]
    return nodes, lens


def _compact_sizes(case):
    """(kept tokens, tokens in all) of each sequence."""
    return ([1 + (3 * b) % case["keep"] for b in range(case["B"])],
            [max(case["nodes"], case["len"] - 13 * (b % 40)) for b in range(case["B"])])


def _assign_sizes(case):
    """(tokens of the old rows, of the new rows)."""
    old = [max(0, case["len"] - (37 * (b // case["group"])) % (1 + case["len"] // 2)) for b in range(case["B"])]
    # every 11th sequence ends
    return old, [0 if b % 11 == 10 else n + case["new"] for b, n in enumerate(old)]


def _copied(case):
    """Tokens of each listed copy, 0 where there is none."""
    return [0 if i % case["every"] else case["page"] if case["whole"] else 1 + (29 * i) % case["page"] for i in range(case["N"])]


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"tree": _prepare_tree, "compact": _prepare_compact, "assign": _prepare_assign, "copy": _prepare_copy}[case["op"]](case, g)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _table(page, lens, g):
    """A block table over a shuffled pool; -1 where a sequence has no page."""
    counts = [-(-n // page) for n in lens]
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
            size = torch.exp2(torch.randint(-1, 2, (n, H), generator=g, device="cuda").float() * 0.5)
            x = _randn(g, n, *shape[1:]) * (sigma * size)[..., None, None]
            if case["cache"] == "bf16":
                s[name][a:a + n] = x.to(torch.bfloat16)
            else:
                codes, s[name + "_scale"][a:a + n] = _quantised(x)
                s[name].view(torch.uint8)[a:a + n] = codes.view(torch.uint8)
    return s


def _handle(s):
    import transformer_attention_relative_gb300 as rp
    return rp.PagedCache(s["k"], s["v"], s.get("k_scale"), s.get("v_scale"))


def _prepare_tree(case, g):
    nodes, lens = _tree_sizes(case)
    B, n, Hq, d = case["B"], case["nodes"], case["Hq"], case["d"]
    table, pool = _table(case["page"], lens, g)
    s = dict(case=case, table=table, lens=_ints(lens), nodes=_ints(nodes), **_pool(case, pool, case["Hkv"], g))
    s["q"] = _randn(g, B, n, Hq, d).to(torch.bfloat16).transpose(1, 2)
    # node 0 is the token after the context; the others hang from any earlier one
    u = torch.rand(B, n, generator=g, device="cuda")
    s["parents"] = (u * torch.arange(n, device="cuda")).floor().to(torch.int32)
    s["parents"][:, 0] = -1
    if case["bias"] == "t5":
        s["bias"] = 0.5 * _randn(g, 32, Hq)
    elif case["bias"] == "alibi":
        s["bias"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], device="cuda")
    if own:
        s["handle"] = _handle(s)
    return s


def _prepare_compact(case, g):
    counts, lens = _compact_sizes(case)
    B, n, keep = case["B"], case["nodes"], case["keep"]
    table, pool = _table(case["page"], lens, g)
    s = dict(case=case, table=table, lens=_ints(lens), counts=_ints(counts), **_pool(case, pool, case["H"], g))
    # the first node and, behind the last slot that is written, one of each later rank in ascending order
    rest = torch.rand(B, n - keep, generator=g, device="cuda").argsort(-1)[:, :keep - 1].sort(-1)[0] + keep
    s["kept"] = torch.cat([torch.zeros(B, 1, dtype=torch.int64, device="cuda"), rest], 1).to(torch.int32)
    if own:
        s["handle"] = _handle(s)
    return s


def _prepare_assign(case, g):
    old, new = _assign_sizes(case)
    B, page, pool, group = case["B"], case["page"], case["pool"], case["group"]
    counts = [-(-n // page) for n in old]
    width = max(max(counts), max(-(-n // page) for n in new), 1)
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(counts):
        # sequences of a group have their first half in common
        shared = c // 2 if b % group else 0
        if shared:
            table[b, :shared] = table[b - 1, :shared]
        table[b, shared:c] = order[at:at + c - shared]
        at += c - shared
    refs = torch.zeros(pool + 1, dtype=torch.int32, device="cuda")
    refs.scatter_add_(0, torch.where(table < 0, pool, table).flatten().long(), torch.ones(table.numel(), dtype=torch.int32, device="cuda"))
    if case["outside"]:  # pages that a store of prefixes holds too
        refs[:pool:case["outside"]] += 1
    # each sequence goes on from one of its group
    first = torch.arange(B, device="cuda") // group * group
    source = first + (torch.rand(B, generator=g, device="cuda") * group).floor().long()
    source = torch.minimum(source, torch.full_like(source, B - 1)).to(torch.int32)
    return dict(case=case, table=table, refs=refs[:pool].contiguous(), lens=_ints(old), new_lens=_ints(new), source=source)


def _prepare_copy(case, g):
    tokens = _copied(case)
    s = dict(case=case, **_pool(case, case["pool"], case["H"], g))
    order = torch.randperm(case["pool"], generator=g, device="cuda").to(torch.int32)
    n = _ints(tokens)
    copies = torch.stack([order[:case["N"]], order[case["N"]:2 * case["N"]], n], 1)
    s["copies"] = torch.where(n[:, None] > 0, copies, -1).contiguous()
    if own:
        s["handle"] = _handle(s)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return {"tree": _run_tree, "compact": _run_compact, "assign": _run_assign, "copy": _run_copy}[s["case"]["op"]](s)


def _t5_bucket(distance, slots=32, most=128):
    exact = slots // 2
    far = exact + (torch.log(distance.clamp(min=exact).double() / exact) / math.log(most / exact) * (slots - exact)).long()
    return torch.where(distance < exact, distance, far.clamp(max=slots - 1))


def _run_tree(s):
    case = s["case"]
    if own:
        import transformer_attention_relative_gb300 as rp
        mode = {"none": None, "t5": rp.MODE_T5, "alibi": rp.MODE_ALIBI}[case["bias"]]
        return rp.paged_tree_decode(s["q"], s["handle"], s["table"], s["lens"], s["parents"], nodes=s["nodes"],
                                    bias=s.get("bias"), mode=mode)
    B, Hq, Hkv, n, d = (case[x] for x in ("B", "Hq", "Hkv", "nodes", "d"))
    table = s["table"].long().clamp(min=0)
    N = table.shape[1] * case["page"]
    k, v = s["k"][table].float(), s["v"][table].float()  # [B, pages, Hkv, page, d]
    if case["cache"] != "bf16":
        k = k * s["k_scale"][table][..., None, None]
        v = v * s["v_scale"][table][..., None, None]
    k = k.transpose(1, 2).reshape(B, Hkv, N, d)
    v = v.transpose(1, 2).reshape(B, Hkv, N, d)
    # sees[b, i, j]: node j is node i or an ancestor of it
    node = torch.arange(n, device=k.device)
    up = (s["parents"][:, :, None] == node) | (node[:, None] == node)
    sees = torch.linalg.matrix_power(up.double(), 64) > 0
    depth = sees.sum(-1) - 1  # [B, n]
    base = (s["lens"] - s["nodes"]).long()[:, None]
    key = torch.arange(N, device=k.device)[None]
    drafted = (key >= base) & (key < s["lens"][:, None])
    at = (key - base).clamp(0, n - 1)
    place = torch.where(drafted, base + depth.gather(1, at), key)  # positions of the keys
    back = (base + depth)[:, :, None] - place[:, None]             # [B, n, N]
    seen = torch.where(drafted[:, None], sees.gather(2, at[:, None].expand(B, n, N)), (key < base)[:, None])
    seen = seen & (node[None] < s["nodes"][:, None])[:, :, None]
    score = (s["q"].float().reshape(B, Hkv, Hq // Hkv * n, d) @ k.transpose(-1, -2)).view(B, Hq, n, N) / math.sqrt(d)
    if case["bias"] == "t5":
        score = score + s["bias"][_t5_bucket(back.clamp(min=0))].permute(0, 3, 1, 2)
    elif case["bias"] == "alibi":
        score = score - s["bias"][None, :, None, None] * back.abs().float()[:, None]
    score = score.masked_fill(~seen[:, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-38)
    v = v.masked_fill((key >= s["lens"][:, None])[:, None, :, None], 0.0)
    return (p.view(B, Hkv, -1, N) @ v).view(B, Hq, n, d).to(torch.bfloat16)


def _run_compact(s):
    case = s["case"]
    if own:
        import transformer_attention_relative_gb300 as rp
        rp.paged_compact(s["handle"], s["table"], s["lens"], s["kept"], case["nodes"], counts=s["counts"])
        return [s[n] for n in ("k", "v", "k_scale", "v_scale") if n in s]
    B, page, keep = case["B"], case["page"], case["keep"]
    base = (s["lens"] - case["nodes"]).long()[:, None]
    i = torch.arange(keep, device=base.device)[None]
    live = i < s["counts"][:, None]
    # an entry that is not kept stays where it is
    to, of = base + i, base + torch.where(live, s["kept"].long(), i)
    table = s["table"].long()
    to_page, of_page = table.gather(1, to // page), table.gather(1, of // page)
    if case["cache"] == "bf16":
        for name in ("k", "v"):
            s[name][to_page, :, to % page] = s[name][of_page, :, of % page]
        return [s["k"], s["v"]]
    # the pages that the kept tokens go to, and what they held
    far = -(-keep // page) + 1
    spot = (base // page + torch.arange(far, device=base.device)).clamp(max=table.shape[1] - 1)
    mine = table.gather(1, spot)
    held_page = torch.where(mine < 0, table.gather(1, base // page), mine).flatten()  # twice the same: the same is written
    for name in ("k", "v"):
        codes, scale = s[name], s[name + "_scale"]
        token, was = codes[of_page, :, of % page].float(), scale[of_page]  # [B, keep, H, d], [B, keep, H]
        want = scale.clone()
        want.scatter_reduce_(0, to_page.flatten()[:, None].expand(-1, scale.shape[1]), was.flatten(0, 1), "amax")
        moved = (codes[held_page].double() * (scale[held_page].double() / want[held_page].double())[..., None, None]).float()
        bytes_ = codes.view(torch.uint8)
        bytes_[held_page] = moved.to(torch.float8_e4m3fn).view(torch.uint8)
        new = (token.double() * (was.double() / want[to_page].double())[..., None]).float().to(torch.float8_e4m3fn)
        bytes_[to_page, :, to % page] = new.view(torch.uint8)
        scale.copy_(want)
    return [s["k"], s["v"], s["k_scale"], s["v_scale"]]


def _run_assign(s):
    case = s["case"]
    page = case["page"]
    if own:
        import transformer_attention_relative_gb300 as rp
        return rp.paged_assign(s["refs"], s["table"], s["lens"], s["new_lens"], page, source=s["source"])
    table, refs, width = s["table"].long(), s["refs"], s["table"].shape[1]
    entry = torch.arange(width, device=table.device)[None]
    # references from elsewhere
    none = refs.shape[0]
    holds = entry < ((s["lens"].long() + page - 1) // page)[:, None]
    left = torch.cat([refs, refs.new_zeros(1)])
    one = torch.ones(table.numel(), dtype=left.dtype, device=left.device)
    left = left.scatter_add(0, torch.where(holds, table, none).flatten(), -one)
    # what the new rows continue
    source = s["source"].long()
    rows = table[source]
    keep = torch.minimum(s["lens"].long()[source], s["new_lens"].long())
    full, part = keep // page, keep % page
    shared = entry < full[:, None]
    left = left.scatter_add(0, torch.where(shared, rows, none).flatten(), one[:1].expand(rows.numel()))
    last = rows.gather(1, full.clamp(max=width - 1)[:, None])[:, 0]
    last = torch.where(part > 0, last, none)
    i = torch.arange(len(source), device=table.device)
    lowest = torch.full((none + 1,), len(source), device=table.device).scatter_reduce(0, last, i, "amin")
    stays = (part > 0) & (left[last] <= 0) & (lowest[last] == i)
    left = left.scatter(0, torch.where(stays, last, none), 1)[:none]
    # fresh pages
    pages = (s["new_lens"].long() + page - 1) // page
    wants = (entry >= (full + stays)[:, None]) & (entry < pages[:, None])
    rank = (wants.flatten().cumsum(0) - 1).view_as(wants)
    free = (left == 0).sum()
    order = torch.argsort((left != 0).to(torch.int32), stable=True)
    fresh = torch.where(rank < free, order[rank.clamp(0, none - 1)], -1)
    new = torch.where(shared | (stays[:, None] & (entry == full[:, None])), rows, torch.where(wants, fresh, -1))
    got = wants & (rank < free)
    left = torch.cat([left, left[:1]]).scatter(0, torch.where(got, fresh, none).flatten(), 1)[:none]
    to = new.gather(1, full.clamp(max=width - 1)[:, None])[:, 0]
    copies = torch.stack([last, to, part], 1)
    copies = torch.where(((part > 0) & ~stays & (to >= 0))[:, None], copies, -1)
    return new.to(torch.int32), left.to(torch.int32), copies.to(torch.int32)


def _run_copy(s):
    case = s["case"]
    if own:
        import transformer_attention_relative_gb300 as rp
        rp.paged_copy(s["handle"], s["copies"])
        return [s[n] for n in ("k", "v", "k_scale", "v_scale") if n in s]
    of, to, n = s["copies"].long().unbind(1)
    # an entry that is none copies the pool's last page, which nothing else touches, onto itself
    last = case["pool"] - 1
    of, to = torch.where(n > 0, of, last), torch.where(n > 0, to, last)
    takes = torch.arange(case["page"], device=of.device) < n[:, None]
    for name in ("k", "v"):
        x = s[name] if case["cache"] == "bf16" else s[name].view(torch.uint8)
        x[to] = torch.where(takes[:, None, :, None], x[of], x[to])
        if name + "_scale" in s:
            s[name + "_scale"][to] = s[name + "_scale"][of]
    return [s[n] for n in ("k", "v", "k_scale", "v_scale") if n in s]


# ------------------------------------------------------------------ work and exact values

def work(case):
    if case["op"] == "assign":
        old, new = _assign_sizes(case)
        page, B = case["page"], case["B"]
        held = sum(-(-n // page) for n in old)
        width = max(-(-n // page) for n in old + new + [1])
        return {"bytes": 4 * (held + B * width + 2 * case["pool"] + 3 * B + 3 * B), "flops": 0}
    size = 1 if case["cache"] == "e4m3" else 2
    if case["op"] == "tree":
        nodes, lens = _tree_sizes(case)
        d, Hkv, Hq = case["d"], case["Hkv"], case["Hq"]
        pages = sum(-(-n // case["page"]) for n in lens)
        rows = Hq * sum(nodes)
        return {"bytes": 2 * sum(lens) * Hkv * d * size + (8 * pages * Hkv if size == 1 else 0) + 4 * pages
                + 2 * rows * d + 2 * case["B"] * Hq * case["nodes"] * d + 4 * sum(nodes) + 8 * case["B"],
                "flops": 4 * d * Hq * sum(a * b for a, b in zip(nodes, lens))}
    if case["op"] == "compact":
        counts, lens = _compact_sizes(case)
        moved = sum(c - 1 for c in counts)  # the first kept one is where it belongs
        return {"bytes": 4 * moved * case["H"] * case["d"] * size + 4 * sum(counts) + 8 * case["B"], "flops": 0}
    tokens = _copied(case)
    some = sum(t > 0 for t in tokens)
    return {"bytes": 4 * sum(tokens) * case["H"] * case["d"] * size + (16 * some * case["H"] if size == 1 else 0)
            + 12 * case["N"], "flops": 0}


def exact(case, seed):
    if case["op"] == "assign":
        return None  # whole numbers
    s = prepare(case, seed)
    return {"tree": _exact_tree, "compact": _exact_compact, "copy": _exact_copy}[case["op"]](case, s)


def _exact_tree(case, s):
    nodes, lens = _tree_sizes(case)
    Hq, Hkv, d, page = (case[x] for x in ("Hq", "Hkv", "d", "page"))
    G = Hq // Hkv
    parents = s["parents"].tolist()
    out = torch.zeros(case["B"], Hq, case["nodes"], d, dtype=torch.float64, device=s["q"].device)
    for b, (n, total) in enumerate(zip(nodes, lens)):
        base, lines = total - n, []
        for i in range(n):
            lines.append((lines[parents[b][i]] if parents[b][i] >= 0 else []) + [i])
        depth = torch.tensor([len(x) - 1 for x in lines], device=out.device)
        hidden = torch.zeros(n, total, dtype=torch.bool)
        for i, line in enumerate(lines):
            hidden[i, base:] = True
            hidden[i, [base + j for j in line]] = False
        hidden = hidden.to(out.device)
        place = torch.cat([torch.arange(base, device=out.device), base + depth])
        back = (base + depth)[:, None] - place[None]
        i = s["table"][b, :-(-total // page)].long()
        if case["bias"] == "t5":
            near = [x if x < 16 else min(31, 16 + int(math.log(x / 16) / math.log(8) * 16)) for x in range(128)]
            ids = torch.tensor(near, device=out.device)[back.clamp(0, 127)]
        for h in range(Hkv):
            k, v = s["k"][i, h].double(), s["v"][i, h].double()
            if case["cache"] != "bf16":
                k, v = k * s["k_scale"][i, h].double()[:, None, None], v * s["v_scale"][i, h].double()[:, None, None]
            k, v = k.reshape(-1, d)[:total], v.reshape(-1, d)[:total]
            for hq in range(h * G, (h + 1) * G):
                z = s["q"][b, hq, :n].double() @ k.T / math.sqrt(d)
                if case["bias"] == "alibi":
                    z -= s["bias"][hq].double() * back.abs()
                elif case["bias"] == "t5":
                    z += s["bias"][:, hq].double()[ids]
                out[b, hq, :n] = torch.softmax(z.masked_fill(hidden, -math.inf), -1) @ v
    return out


def _exact_compact(case, s):
    page, n = case["page"], case["nodes"]
    counts, lens = _compact_sizes(case)
    table, kept = s["table"].tolist(), s["kept"].tolist()
    cache = {x: s[x].double() for x in ("k", "v", "k_scale", "v_scale") if x in s}
    grid = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().to(s["k"].device)  # 0 .. 448
    middle = (grid[1:] + grid[:-1]) / 2

    def nearest(x):
        a = x.abs().contiguous()
        low, high = torch.searchsorted(middle, a), torch.searchsorted(middle, a, right=True)  # they differ on a tie
        return torch.where(torch.signbit(x), -1.0, 1.0).double() * grid[torch.where(low == high, low, low + low % 2)]

    for b, (count, total) in enumerate(zip(counts, lens)):
        base = total - n
        pages, slots = zip(*[divmod(base + j, page) for j in kept[b][:count]])
        of = torch.tensor([table[b][p] for p in pages], device=grid.device)
        slots = torch.tensor(slots, device=grid.device)
        for name in ("k", "v"):
            token = cache[name][of, :, slots]  # [count, H, d]
            had = cache[name + "_scale"][of] if name + "_scale" in cache else None
            for p in range(base // page, (base + count - 1) // page + 1):
                lo, hi = max(base, p * page), min(base + count, (p + 1) * page)
                to, x = table[b][p], token[lo - base:hi - base].transpose(0, 1)
                if had is not None:
                    was, got = cache[name + "_scale"][to].clone(), had[lo - base:hi - base].T
                    want = torch.maximum(was, got.amax(1))
                    cache[name][to] = nearest(cache[name][to] * (was / want)[:, None, None])
                    cache[name + "_scale"][to] = want
                    x = nearest(x * (got / want[:, None])[..., None])
                cache[name][to, :, lo - p * page:hi - p * page] = x
    return [cache[x] for x in ("k", "v", "k_scale", "v_scale") if x in cache]


def _exact_copy(case, s):
    cache = {x: s[x].double() for x in ("k", "v", "k_scale", "v_scale") if x in s}
    for of, to, n in s["copies"].tolist():
        if n <= 0:
            continue
        for name in cache:
            if name.endswith("scale"):
                cache[name][to] = cache[name][of]
            else:
                cache[name][to, :, :n] = cache[name][of, :, :n]
    return [cache[x] for x in ("k", "v", "k_scale", "v_scale") if x in cache]
