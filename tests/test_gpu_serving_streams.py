"""Serving calls on a stream that is not the current one, and as the first of a process under capture."""
import os
import subprocess
import sys
import textwrap

import pytest
import torch

import gpu_util as G
import transformer_attention_relative_gb300 as rp

pytestmark = pytest.mark.gpu
BF, E4 = torch.bfloat16, torch.float8_e4m3fn
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def _calls():
    """name -> (call with a stream, shape and dtype of what it allocates)"""
    g = torch.Generator().manual_seed(1)
    q = torch.randn(2, 4, 64, 64, generator=g).to(BF).cuda()
    plan = rp.RotaryPlan(64)
    k = torch.randn(9, 2, 32, 64, generator=g).to(BF).cuda()
    cache = rp.PagedCache(k, k.clone())
    table = torch.arange(8, dtype=torch.int32).view(2, 4).cuda()
    lens = torch.tensor([100, 128], dtype=torch.int32).cuda()
    rows = q[:, :, :4].contiguous()
    slopes = torch.tensor([0.5, 0.25, 0.125, 0.0625], device="cuda")
    bias = torch.randn(32, 4, generator=g).cuda()
    at = torch.arange(64, dtype=torch.int32, device="cuda").expand(2, 4, 64).contiguous()
    return {
        "rotary": lambda s: rp.rotary(q, plan, stream=s),
        "rotary_pair": lambda s: rp.rotary(q, plan, q, stream=s)[1],
        "rotary_backward": lambda s: rp.rotary_backward(q, plan, stream=s),
        "paged_decode": lambda s: rp.paged_decode(rows, cache, table, lens, stream=s),
        "attention": lambda s: rp.attention(q, q, q, bias, stream=s),
        "index_ids": lambda s: rp.index_ids(rp.MODE_T5, -8192, 16384, stream=s),
        "t5_decode_positions": lambda s: rp.t5_decode_positions(rows, q, q, bias, at, stream=s),
        "alibi_decode_positions": lambda s: rp.alibi_decode_positions(rows, q, q, slopes, at, stream=s),
        "t5_attention_backward": lambda s: rp.t5_attention_backward(q, q, q, q, bias, stream=s)[1],
    }


NAMES = ["rotary", "rotary_pair", "rotary_backward", "paged_decode", "attention", "index_ids", "t5_decode_positions",
         "alibi_decode_positions", "t5_attention_backward"]


@pytest.mark.parametrize("name", NAMES)
def test_outputs_are_not_memory_that_the_current_stream_still_uses(name):
    """The current stream is behind: it has yet to write a tensor whose memory is free on the host already. A call on
    another stream must not be given that memory for its output."""
    call = _calls()[name]
    want = call(torch.cuda.current_stream())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        old = [torch.empty_like(want) for _ in range(8)]
        torch.cuda.synchronize()
        torch.cuda._sleep(40_000_000)  # some 20 ms of the current stream
        for t in old:
            t.fill_(7)
        del old, t
        got = call(s)
        s.synchronize()
        torch.cuda.synchronize()
        if name == "t5_attention_backward":  # its sums' order is not fixed
            assert torch.allclose(got.float(), want.float(), atol=1e-2, rtol=1e-2)
        else:
            assert torch.equal(got, want)
        del got
    assert rp.check_status() == 0


def test_outputs_outlive_their_use_on_the_current_stream():
    """An output of another stream, read by the current one and dropped: its memory is not given out before that read."""
    call = _calls()["rotary"]
    want = call(torch.cuda.current_stream())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        got = call(s)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda._sleep(40_000_000)
        copy = got.clone()
        del got
        with torch.cuda.stream(s):
            others = [torch.full_like(want, 7.0) for _ in range(8)]
        torch.cuda.synchronize()
        assert torch.equal(copy, want)
        del others


def _python(code):
    r = subprocess.run([sys.executable, "-c", textwrap.dedent(code)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]


@pytest.mark.parametrize("before", ["append", "short decode"])
def test_a_capture_may_hold_the_first_long_decode(before):
    """The process has made a call before (the status word is looked up), but none that takes scratch."""
    _python(f"""
        import torch, transformer_attention_relative_gb300 as rp
        g = torch.Generator().manual_seed(3)
        for dtype in (torch.bfloat16, torch.float8_e4m3fn):
            cache = rp.PagedCache.empty(40, 2, 64, page_size=32, dtype=dtype)
            kv = torch.randn(1200, 4, 64, generator=g).to(torch.bfloat16).cuda()
            table = torch.arange(40, dtype=torch.int32).view(1, 40).cuda()
            lens, cu = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([1200], [0, 1200]))
            rp.paged_append(cache, kv[:, :2], kv[:, 2:], table, lens, cu_new=cu)
            q = torch.randn(1, 4, 1, 64, generator=g).to(torch.bfloat16).cuda()
            if {before!r} == "short decode":
                rp.paged_decode(q, cache, table[:, :1], torch.ones_like(lens))
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = rp.paged_decode(q, cache, table, lens)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, rp.paged_decode(q, cache, table, lens))
        assert rp.check_status() == 0
    """)


def test_a_capture_may_hold_the_first_wide_append():
    """The first append of a process that takes more shared memory than a launch has by default."""
    _python("""
        import torch, transformer_attention_relative_gb300 as rp
        assert rp.check_status() == 0
        cache = rp.PagedCache.empty(4, 2, 128, page_size=128, dtype=torch.float8_e4m3fn)
        kv = torch.randn(300, 4, 128).to(torch.bfloat16).cuda()
        table = torch.arange(4, dtype=torch.int32).view(1, 4).cuda()
        lens, cu = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([300], [0, 300]))
        run = lambda: rp.paged_append(cache, kv[:, :2], kv[:, 2:], table, lens, cu_new=cu, plan=rp.RotaryPlan(128))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        graph.replay()
        torch.cuda.synchronize()
        held = [t.view(torch.uint8).clone() for t in (cache.k, cache.v)]
        assert held[0].any() and held[1].any()
        for t in (cache.k, cache.v):
            t.view(torch.uint8).zero_()
        run()
        assert all(torch.equal(a, t.view(torch.uint8)) for a, t in zip(held, (cache.k, cache.v)))
        assert rp.check_status() == 0
    """)
