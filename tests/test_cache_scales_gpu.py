"""Attention over the 8-bit cache where the blocks' value scales lie far apart, against the plain
64-bit form on the values that the cache stands for (allowed errors: tests/_window_ref.py)."""
import pytest
import torch

import laplacian_nystr_linear_gb300 as lap
from laplacian_nystr_linear_gb300 import _lib, api

from tests._window_ref import check, reference
from tests.test_cache_gpu import clone, filled, gathered

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
DTYPES = pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
ROWS = pytest.mark.parametrize("Nq", [1, 4], ids=["4rows", "16rows"])   # of 4 heads a key head


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    assert api.device_status(clear=True) == _lib.LAPNYS_OK


def compare(q, cache, table, lens):
    """cache_attention against the 64-bit form.  P is held to 2^-21 of itself with fp32 queries (two
    f16 parts), and q to 2^-22 of its row's largest feature."""
    out = lap.cache_attention(q, cache, table, lens)
    k, v = gathered(cache, table)
    ref = reference(q, k, v, -1, 0, 0, None, lens, lens - q.shape[2], extra_p=2.0 ** -21,
                    extra_s=2.0 ** -22 * 8)
    check("out", out, ref["out"])
    return out


@DTYPES
@ROWS
@pytest.mark.parametrize("order", ["down", "up"])
@pytest.mark.parametrize("place", ["in_a_group", "across_groups"])
@pytest.mark.parametrize("gap", [17, 20, 40])
def test_neighbouring_blocks_far_apart(gap, place, order, Nq, dtype):
    """Blocks of 16 tokens, two of them to a group of 32 keys, `gap` powers of two apart."""
    exps = [-7, -7 - gap] * 4 if place == "in_a_group" else [-7, -7, -7 - gap, -7 - gap] * 2
    exps = torch.tensor(exps if order == "down" else exps[::-1])
    cache = clone(filled(8, 2, 16, 64, seed=gap), "cuda")
    cache.v_scale.copy_((2.0 ** exps)[:, None].expand(8, 2))
    q = torch.randn((1, 8, Nq, 64), generator=torch.Generator().manual_seed(gap)).cuda().to(dtype) * 0.7
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None].contiguous()
    compare(q, cache, table, torch.tensor([125], dtype=torch.int32, device="cuda"))
