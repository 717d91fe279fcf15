"""Serving calls under stream capture that are the first of their kind in a process."""
import os
import subprocess
import sys
import textwrap

import pytest

import gpu_util as G

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


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
