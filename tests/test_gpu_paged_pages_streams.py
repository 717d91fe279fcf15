"""The operators on pages and trees on streams and in captured graphs, a process's first calls among them."""
import subprocess
import sys

import numpy as np
import pytest
import torch

import gpu_util as G
import transformer_attention_relative_gb300 as rp
from oracle import serving_oracle as so
from test_gpu_paged_pages import _assign, _bytes, _cache, _i32, _refs, _table

pytestmark = pytest.mark.gpu
BF, E4 = torch.bfloat16, torch.float8_e4m3fn

FIRST = """
import torch, transformer_attention_relative_gb300 as rp
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
cache = rp.PagedCache.empty(40, 2, 64, page_size=32, dtype=torch.{dtype})
cache.k.view(torch.uint8).copy_(torch.randint(0, 100, (40, 2, 32, cache.k.view(torch.uint8).shape[-1]), device="cuda"))
cache.v.copy_(cache.k)
table, lens, refs = i32([[0, 1] + [-1] * 700, [2, 3] + [-1] * 700]), i32([40, 64]), i32([1] * 4 + [0] * 36)
grown, parents, kept = i32([65, 80]), i32([-1, 0, 1, 1, -1, 4, 5, 6, 7]), i32([[0, 2], [1, 8]])
q, out = torch.randn(2, 16, 9, 64, device="cuda").bfloat16(), torch.empty(2, 16, 9, 64, device="cuda", dtype=torch.bfloat16)
few = torch.empty(2, 2, 9, 64, device="cuda", dtype=torch.bfloat16)
before = [x.clone() for x in (cache.k.view(torch.uint8), cache.v.view(torch.uint8))]
torch.cuda.synchronize()
def calls():
    rp.paged_tree_decode(q, cache, table, lens, parents, out=out)
    rp.paged_tree_decode(q[:, :2], cache, table, lens, parents, out=few)
    rp.paged_compact(cache, table, lens, kept, 9)
    new = rp.paged_assign(refs, table, lens, grown, 32)
    rp.paged_copy(cache, new[2])
    return new
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    new = calls()
g.replay()
torch.cuda.synchronize()
got = [x.clone() for x in (out, few, *new, cache.k.view(torch.uint8), cache.v.view(torch.uint8))]
for x, y in zip((cache.k, cache.v), before):
    x.view(torch.uint8).copy_(y)
new = calls()
torch.cuda.synchronize()
for x, y in zip(got, (out, few, *new, cache.k.view(torch.uint8), cache.v.view(torch.uint8))):
    assert torch.equal(x.view(torch.uint8), y.contiguous().view(torch.uint8))
assert rp.check_status() == 0 and new[1].sum() == 6
print("fine")
"""


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


@pytest.mark.parametrize("dtype", ["bfloat16", "float8_e4m3fn"])
def test_first_calls_of_a_process_under_capture(dtype):
    r = subprocess.run([sys.executable, "-c", FIRST.format(dtype=dtype)], capture_output=True, text=True, timeout=110)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


def test_assign_of_two_streams_at_once():
    streams = [torch.cuda.Stream() for _ in range(2)]
    cases = []
    for seed in range(2):
        lens = [(31 * b + 7 * seed) % 400 for b in range(300)]
        table = _table(lens, 64, 9000, seed, 9)
        refs = _refs(table, lens, 64, 9000)
        new_lens = [n + 50 for n in lens]
        source = [b // 3 * 3 for b in range(300)]
        new_lens = [new_lens[s] for s in source]
        want = so.paged_assign(refs, table.tolist(), lens, source, new_lens, 64, 9)
        cases.append(((_i32(refs), table.cuda(), _i32(lens), _i32(new_lens), 64), _i32(source), want))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for s, (args, source, _) in enumerate(cases):
            got[s].append(rp.paged_assign(*args, source=source, stream=streams[s]))
    torch.cuda.synchronize()
    for s, (_, _, want) in enumerate(cases):
        for new, left, copies in got[s]:
            assert new.tolist() == want[0] and left.tolist() == want[1]
            assert [tuple(c) for c in copies.tolist()] == want[2]
    assert rp.check_status() == 0


@pytest.mark.parametrize("entries", [65536, 65537])
def test_assign_on_either_side_of_its_thread_counts(entries):
    lens, page = [300, 40, 0, 65], 32
    pages = entries - 2 * 4 * 16
    table = _table(lens, page, pages, 3, 16)
    refs = _refs(table, lens, page, pages, [5, 9])
    _assign(refs, table, lens, [0, 0, 1, 3], [330, 310, 64, 0], page)
    assert rp.check_status() == 0


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m", [16, 17, 32, 33, 63, 64])
def test_compact_on_either_side_of_its_variants(dtype, d, m):
    cache = _cache(12, 3, 32, d, dtype, 8)
    lens, n = [100, 64, 90], 64
    table = _table(lens, 32, 12, 8, 4)
    kept = torch.sort(torch.rand(3, n, generator=torch.Generator().manual_seed(m)).argsort(1)[:, :m], 1).values.to(torch.int32)
    was = [x.view(torch.uint8).cpu().numpy().copy() if dtype == E4 else x.view(torch.int16).cpu().numpy().copy()
           for x in (cache.k, cache.v)]
    if dtype == E4:
        cache.k_scale.fill_(0.25)
        cache.v_scale.fill_(0.5)
    rp.paged_compact(cache, table.cuda(), _i32(lens), kept.cuda(), n)
    assert rp.check_status() == 0
    for x, want in zip((cache.k, cache.v), was):
        had = want.copy()
        for b, ln in enumerate(lens):
            for i, j in enumerate(kept[b].tolist()):
                s, t = ln - n + j, ln - n + i
                want[table[b, t // 32], :, t % 32] = had[table[b, s // 32], :, s % 32]
        np.testing.assert_array_equal((x.view(torch.uint8) if dtype == E4 else x.view(torch.int16)).cpu().numpy(), want)


def test_copies_and_compacts_in_replayed_graphs():
    """Two graphs over one pool, in turn; what a replay does goes by the lists' present entries."""
    cache = _cache(16, 2, 32, 64, BF, 9)
    copies, lens, kept = _i32([[0, 1, 32]]), _i32([40]), _i32([[2, 3]])
    table = _i32([[4, 5]])
    rp.paged_copy(cache, _i32([[0, 0, 0]]))
    torch.cuda.synchronize()
    a, b = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(a):
        rp.paged_copy(cache, copies)
    with torch.cuda.graph(b):
        rp.paged_compact(cache, table, lens, kept, 5)
    for of, to, ln in ((2, 3, 40), (6, 7, 37), (0, 9, 64)):
        copies.copy_(_i32([[of, to, 32]]))
        lens.copy_(_i32([ln]))
        want = cache.k.clone()
        want[to] = want[of]
        for i, j in enumerate((2, 3)):
            s, t = ln - 5 + j, ln - 5 + i
            want[4 + t // 32, :, t % 32] = want[4 + s // 32, :, s % 32]
        a.replay()
        b.replay()
        torch.cuda.synchronize()
        assert torch.equal(cache.k, want)
    assert rp.check_status() == 0 and len(_bytes(cache)) == 2
