"""Arguments of the windowed attention and the 8-bit cache at the edges of what the C entry takes, on
the GPU."""
import pytest
import torch

import laplacian_nystr_linear_gb300 as lap

from tests.test_window_gpu import make

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("wide", [2 ** 31, 2 ** 32, 2 ** 32 + 5])
def test_windows_wider_than_32_bits(wide):
    """No bound, not the low 32 bits of the width."""
    q, k, v, _ = make(1, 2, 1, 70, 70, 32, BF)
    for a, b in ((dict(left=wide), dict(left=-1)), (dict(left=3, right=wide), dict(left=3, right=-1)),
                 (dict(left=3, sinks=wide), dict(left=-1))):
        assert torch.equal(lap.window_attention(q, k, v, **a), lap.window_attention(q, k, v, **b))
    cache = lap.cache_alloc(2, 1, 32, 64)
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    n = torch.tensor([70], dtype=torch.int32, device="cuda")
    lap.cache_append(cache, k, v, table, torch.zeros_like(n))
    want = lap.cache_attention(q, cache, table, n, left=-1)
    assert torch.equal(lap.cache_attention(q, cache, table, n, left=wide), want)
    assert torch.equal(lap.cache_attention(q, cache, table, n, left=3, sinks=wide), want)
