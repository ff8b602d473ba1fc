"""The feed-forward block where test_mlp_gpu.py allows more than the contract does."""
import pytest
import torch

import laplacian_nystr_linear_gb300 as lap
from tests._bounds import check
from tests._mlp_ref import check_scale, reference
from tests.test_mlp_gpu import DTYPES, NAMES, SIZES, _inputs, _step

pytestmark = pytest.mark.gpu


def test_far_magnitudes_in_fp32():
    """1e-30 is 2^-99.7: three parts hold it and its gradients, though products of two such values are nothing."""
    t, dy = _inputs(65, 64, 96, torch.float32, False, 3, 1e-30)
    ref = reference(**t, kind="silu", dy=dy)
    y, grads = _step(t, dy, "silu")
    check("y", y, ref["y"], torch.float32)
    for n, g in grads.items():
        check("d" + n, g, ref[n], torch.float32)
    assert float(grads["x"].abs().mean()) > 1e-31


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 8, 9, 64, 65, 100, 128, 129, 300])
@pytest.mark.parametrize("C,Fh", [(512, 2048), (66, 70)])
def test_what_the_backward_needs_changes_nothing(dtype, T, C, Fh):
    t, dy = _inputs(T, C, Fh, dtype, True, 6)
    assert torch.equal(lap.gated_mlp(**t), _step(t, dy, "silu")[0])


@pytest.mark.parametrize("T,C,Fh", SIZES + [(17931, 32, 1), (2, 1, 344), (3, 21, 2699), (60000, 2, 2), (46795, 17, 3)])
def test_gradients_by_the_blocks_that_are_scaled(T, C, Fh):
    """p and q are scaled by rows of 16 features and rounded to 11 bits, 2^-11 at the most; and the errors allowed are those of a working kernel: below a tenth
    of the values (rows of one feature apart, whose values may cancel)."""
    t, dy = _inputs(T, C, Fh, torch.bfloat16, True)
    ref = reference(**t, kind="gelu", dy=dy, block=16, kept=2.0 ** -11)
    y, grads = _step(t, dy, "gelu")
    for n, g in (("y", y), *grads.items()):
        check(n, g, ref[n], torch.bfloat16)
        assert min(C, Fh) < 8 or check_scale(ref[n]) < 0.1, n
    assert set(grads) == set(NAMES)
