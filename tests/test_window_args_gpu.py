"""Arguments of the windowed attention and the 8-bit cache at the edges of what the C entry takes, on
the GPU."""
import pytest
import torch

import laplacian_nystr_linear_gb300 as lap

from tests._window_ref import check, reference
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


@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["f32", "bf16"])
def test_first_tokens_of_many_heads(dtype):
    """Key tiles with first tokens whose queries are not cut, since there are as many as fill the GPU."""
    q, k, v, do = make(80, 4, 4, 600, 600, 16, dtype)
    p = lap.WindowParams.of(q, k, 63, 0, 200)
    assert lap.window_workspace_bytes(p, dtype, True) == 4 * 80 * 4 * 600
    out, lse = lap.window_fwd(q, k, v, p)
    ref = reference(q, k, v, 63, 0, 200, dout=do)
    check("out", out, ref["out"])
    for name, x in zip(("dq", "dk", "dv"), lap.window_bwd(q, k, v, out, do, lse, p)):
        check(name, x, ref[name])
