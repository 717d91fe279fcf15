"""The serving functions on a torch without the private functions that they prefer."""
import importlib.util

import pytest
import torch

import transformer_attention_relative_gb300 as rp
from transformer_attention_relative_gb300 import serving


@pytest.fixture
def public_only(monkeypatch):
    """A second copy of the module, imported without them."""
    spec = importlib.util.spec_from_file_location(serving.__name__ + "_public", serving.__file__)
    copy = importlib.util.module_from_spec(spec)
    with monkeypatch.context() as without:  # torch's own wrappers need them afterwards
        for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
            without.delattr(torch._C, name, raising=False)
        spec.loader.exec_module(copy)
    return copy


def test_public_functions_take_their_place(public_only, monkeypatch):
    assert public_only._device is torch.cuda.current_device

    class Stream:
        cuda_stream = 1234

    monkeypatch.setattr(torch.cuda, "current_stream", lambda index: Stream if index == 3 else None)
    assert public_only._raw_stream(3) == 1234


@pytest.mark.gpu
def test_calls_are_the_same(public_only):
    import gpu_util as G
    G.ensure_built()
    g = torch.Generator().manual_seed(1)
    q = torch.randn(2, 4, 1, 64, generator=g).to(torch.bfloat16).cuda()
    plan = rp.RotaryPlan(64)
    pages = torch.randn(2, 3, 2, 32, 64, generator=g).to(torch.bfloat16).cuda()
    table, lens = torch.tensor([[0, 2], [1, -1]], dtype=torch.int32).cuda(), torch.tensor([40, 9], dtype=torch.int32).cuda()
    with torch.cuda.stream(torch.cuda.Stream()):
        for module in (rp, public_only):
            cache = module.PagedCache(pages[0].clone(), pages[1].clone())
            module.paged_append(cache, q[:, :2], q[:, 2:], table, lens, plan=plan)
            out = module.rotary(q, plan, offset=5), cache.k, cache.v, module.paged_decode(q, cache, table, lens)
            if module is rp:
                want = out
        torch.cuda.current_stream().synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert rp.check_status() == 0
