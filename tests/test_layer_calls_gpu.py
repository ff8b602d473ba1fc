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


@pytest.mark.parametrize("given,pre,post", [(("weight",), "rms", None), (("u", "weight", "gate"), "layer", None),
                                            (("u", "post_weight"), None, "rms"), (("u",), None, None),
                                            (("u", "weight", "post_weight", "post_bias", "gate", "scale"), "rms", "layer")])
def test_norm_bwd_gives_the_gradients_of_what_there_is(given, pre, post):
    B, N, C = 2, 11, 64
    shapes = dict(u=(B, N, C), weight=(C,), post_weight=(C,), post_bias=(C,), gate=(B, C), scale=(C,))
    t = {n: _rand(*s, seed=i) if n in given else None for i, (n, s) in enumerate(shapes.items())}
    x, dh, dy = (_rand(B, N, C, seed=i) for i in (7, 8, 9))
    dh, dy = dh if "u" in given else None, dy if pre else None
    p = lap.NormParams(B, N, C, False, pre, post, 1e-6)
    vec = {n: t[n] for n in ("post_weight", "post_bias", "gate", "scale")}
    _, _, st = lap.norm_fwd(x, t["u"], t["weight"], None, p, **vec)
    got = lap.norm_bwd(x, t["u"], t["weight"], st, dh, dy, p, **vec)
    want = (True, "u" in given, "weight" in given, pre is not None,
            *(n in given for n in ("post_weight", "post_bias", "gate", "scale")))
    again = lap.norm_bwd(x, t["u"], t["weight"], st, dh, dy, p, **vec, want=want)
    assert [g is not None for g in got] == list(want)
    assert all(torch.equal(a, b) for a, b in zip(got, again) if a is not None)


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("T,C", [(5, 33), (130, 33)])
def test_rows_that_are_a_piece_of_others(dtype, T, C):
    """gated_mlp of rows behind the first one, whose storage starts anywhere."""
    whole = _rand(T + 1, C, seed=1, dtype=dtype)
    w_in, w_out = _rand(C, 80, seed=2, dtype=dtype), _rand(40, C, seed=3, dtype=dtype)
    dy = _rand(T, C, seed=4, dtype=dtype)
    out = []
    for x in (whole[1:], whole[1:].clone()):
        leaves = [v.detach().requires_grad_(True) for v in (x, w_in, w_out)]
        y = lap.gated_mlp(leaves[0], leaves[1], None, leaves[2], None)
        out.append([y.detach(), lap.gated_mlp(x, w_in, None, w_out, None), *torch.autograd.grad(y, leaves, dy)])
    assert whole[1:].data_ptr() % 16
    assert all(torch.equal(a, b) for a, b in zip(*out))


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan"), 3.4e38])
@pytest.mark.parametrize("T", [3, 40, 300])
def test_values_that_are_not_finite_in_fp32(T, bad):
    """They stay in the sums that they are part of: a row of x in its row, a column of w_out in its column, a row of dy
    in dx's row, in all of the weights' gradients and its column of b_out's."""
    C, F = 64, 96
    t = dict(x=_rand(T, C, seed=1), w_in=_rand(C, 2 * F, seed=2) / 8, b_in=_rand(2 * F, seed=3),
             w_out=_rand(F, C, seed=4) / 8, b_out=_rand(C, seed=5))
    dy = _rand(T, C, seed=6)
    p = lap.MlpParams(T, C, F)
    y, ctx = lap.mlp_fwd(**t, p=p)
    grads = lap.mlp_bwd(t["x"], t["w_in"], t["w_out"], dy, ctx, p)

    def put(name, *at):
        v = t[name].clone()
        v[at] = bad
        return lap.mlp_fwd(**{**t, name: v}, p=p)[0]

    rows, cols = torch.arange(T, device="cuda") != 2, torch.arange(C, device="cuda") != 5
    got = put("x", 2, 7)
    assert torch.equal(got[rows], y[rows]) and not got[2].isfinite().any()
    got = put("w_out", 11, 5)
    itself = T <= 8 and bad == 3.4e38       # few rows take weights in fp32: finite sums
    assert torch.equal(got[:, cols], y[:, cols]) and (itself or not got[:, 5].isfinite().any())
    assert itself or not put("w_in", 3, 20).isfinite().any()
    dy[2, 5] = bad
    dx, dw_in, db_in, dw_out, db_out = lap.mlp_bwd(t["x"], t["w_in"], t["w_out"], dy, ctx, p)
    assert torch.equal(dx[rows], grads[0][rows]) and not dx[2].isfinite().any()
    assert not dw_in.isfinite().any() and not db_in.isfinite().any() and not dw_out[:, 5].isfinite().any()
    assert torch.equal(dw_out[:, cols], grads[3][:, cols]) and torch.equal(db_out[cols], grads[4][cols])
