"""What the windowed attention and the 8-bit cache refuse or put right in Python, before anything is
enqueued (no GPU)."""
import pytest
import torch
import torch.autograd.forward_ad as fwAD

import laplacian_nystr_linear_gb300 as lap
from laplacian_nystr_linear_gb300 import window


def _operands():
    q, k, v = (torch.randn(1, 2, 8, 16) for _ in range(3))
    return q, k, v, lap.cache_alloc(4, 2, 16, 16, device="cpu"), torch.zeros((1, 1), dtype=torch.int32)


@pytest.mark.parametrize("which", range(3))
@pytest.mark.parametrize("grad", [True, False])
def test_forward_mode_derivatives_are_refused(which, grad):
    q, k, v, cache, table = _operands()
    with torch.set_grad_enabled(grad), fwAD.dual_level():
        x = [q, k, v]
        x[which] = fwAD.make_dual(x[which], torch.ones_like(q))
        with pytest.raises(ValueError, match="forward-mode"):
            lap.window_attention(*x, 4)
        with pytest.raises(ValueError, match="forward-mode"):
            if which == 0:
                lap.cache_attention(x[0], cache, table, table[0])
            else:
                lap.cache_append(cache, x[1], x[2], table, table[0])
        # plain tensors within a dual level are as ever: refused only as not on a GPU
        with pytest.raises(ValueError, match="CUDA"):
            lap.window_attention(q, k, v, 4)


def test_forward_mode_through_the_backward_is_refused():
    dout = torch.randn(1, 2, 8, 16)
    with fwAD.dual_level(), pytest.raises(ValueError, match="forward-mode"):
        window._Window.backward(object(), fwAD.make_dual(dout, torch.ones_like(dout)))


def test_function_transforms_are_refused():
    q, k, v, _, _ = _operands()
    with pytest.raises(ValueError, match="forward-mode"):
        torch.func.jvp(lambda q: lap.window_attention(q, k, v, 4), (q,), (torch.ones_like(q),))


@pytest.mark.parametrize("which", ["k", "v"])
def test_append_refuses_what_requires_a_gradient(which):
    _, k, v, cache, table = _operands()
    x = {"k": k, "v": v}
    x[which].requires_grad_(True)
    with pytest.raises(ValueError, match="gradient"):
        lap.cache_append(cache, k, v, table, table[0])
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):   # refused only as not on a GPU
        lap.cache_append(cache, k, v, table, table[0])
