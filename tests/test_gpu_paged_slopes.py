"""ALiBi slopes of any finite size in the paged decode, vs the fp64 oracle (tolerance as for the other decodes: 2^-8 of
the output, and of A = sum_j p_j |v_j| 2^-11 or 2^-16 for the weights' rounding and 2^-12 for the logits' error)."""
import pytest
import torch

import gpu_util as G
import transformer_attention_relative_gb300 as rp
from test_gpu_paged_decode import _case, _check, _gpu, _ref

pytestmark = pytest.mark.gpu
LARGEST = torch.finfo(torch.float32).max


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 31, 32, 33, 64, 500, 2048, 2049])
def test_slopes_up_to_the_largest(dtype, n):
    """The largest leave a row its own key; zero is no bias."""
    cache, q, table, lens, _ = _case([n, 40], 8, 2, 2, 64, 32, dtype, "none", 61)
    for slopes in ([LARGEST, 2.5e38, 1e38, 1e30, 1e10, 1e3, 1.0, 0.0], [2.0 ** -e for e in (3, 9, 20, 60, 100, 126, 140, 1)]):
        bias = torch.tensor(slopes)
        got = _gpu(cache, q, table, lens, bias, "alibi")
        assert rp.check_status() == 0
        _check(got, *_ref(cache, q, table, lens, bias, "alibi"), dtype != torch.bfloat16)
