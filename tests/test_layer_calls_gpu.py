"""Calls of the layer's operators that their documentation allows, beside the ordinary ones."""
import pytest
import torch

import laplacian_nystr_linear_gb300 as lap
from laplacian_nystr_linear_gb300 import layer

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16]


def _rand(*shape, seed=0, dtype=torch.float32):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


@pytest.mark.parametrize("which", [0, 1])
def test_rotary_turns_back_only_what_needs_a_gradient(which, monkeypatch):
    q, k, dq, dk = (_rand(2, h, 9, 32, seed=i) for i, h in enumerate((4, 2, 4, 2)))
    f = lap.rotary_frequencies(32)
    both = [x.clone().requires_grad_(True) for x in (q, k)]
    want = torch.autograd.grad(lap.rotary(*both, f), both, [dq, dk])
    some = [x.clone().requires_grad_(i == which) for i, x in enumerate((q, k))]
    out = lap.rotary(*some, f)
    turned, real = [], layer._rotary
    monkeypatch.setattr(layer, "_rotary", lambda q, k, *a: (turned.append((q.shape, k)), real(q, k, *a))[1])
    got, = torch.autograd.grad(out, some[which], [dq, dk])
    assert torch.equal(got, want[which])
    assert turned == [((dq, dk)[which].shape, None)]
