"""The feed-forward block's sums over very many rows or features, all of one sign.

Operands are made so that every factor of a sum is exact: the gate is 16 throughout (act(16) = 16 and
act'(16) = 1 to more than 24 bits), the other half is x itself or its bias, so h = 16 u, and the gradient of
h is dy itself.

The tensor cores cut a sum off at each instruction of 16 k, by up to 2^-22 of it, half of that over a sum
that grows from nothing.  bf16: 1024 instructions make 2^-13 of the sum, what is added up beyond is rounded
to nearest (fewer than 2^8 additions of 2^-24 each).  fp32: 640 instructions for the smaller products, 2^-7 of the
sum, 8 for the leading one; 4096 roundings to nearest beyond, which do not know of one another: 4 sqrt(4096 / 3)
2^-24.  Below 2^-16 in all.
"""
import pytest
import torch

import laplacian_nystr_linear_gb300 as lap
from tests._bounds import check
from tests._mlp_ref import reference

pytestmark = pytest.mark.gpu


def _values(shape, dtype, seed):
    """bf16: in [0.5, 1.5]; fp32: all parts behind the first of one sign, up to 2^-8 of it."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(shape, dtype=dtype, device="cuda")
    for part in t.split(1 << 22):
        r = torch.rand(part.shape, generator=gen, device="cuda")
        part.copy_(0.5 + r if dtype == torch.bfloat16 else 1 + 2.0 ** -8 - r * 2.0 ** -10)
    return t


def _off(got, want):
    return float((got.double() / want - 1).abs().max())


@pytest.mark.parametrize("dtype,T,limit", [(torch.bfloat16, 1 << 26, 2.0 ** -8 + 2.0 ** -12), (torch.bfloat16, 1 << 21, 2.0 ** -8 + 2.0 ** -12),
                                           (torch.float32, 1 << 24, 2.0 ** -16), (torch.float32, 1 << 20, 2.0 ** -16)],
                         ids=["bf16-2^26", "bf16-2^21", "f32-2^24", "f32-2^20"])
def test_weights_gradients_over_many_rows(dtype, T, limit):
    C = F = 8
    x, dy = _values((T, C), dtype, 1), _values((T, C), dtype, 2)
    eye = torch.eye(C, device="cuda")
    w_in = torch.cat([torch.zeros_like(eye), eye], 1).to(dtype)
    b_in = torch.cat([torch.full((F,), 16.0, device="cuda"), torch.zeros(F, device="cuda")]).to(dtype)
    w_out = eye.to(dtype)
    p = lap.MlpParams(T, C, F, "gelu")
    y, ctx = lap.mlp_fwd(x, w_in, b_in, w_out, None, p)
    _, dw_in, db_in, dw_out, db_out = lap.mlp_bwd(x, w_in, w_out, dy, ctx, p)
    assert torch.equal(y, 16 * x)
    want = torch.zeros((C, C), dtype=torch.float64, device="cuda")
    for a, b in zip(x.split(1 << 22), dy.split(1 << 22)):
        want += a.double().T @ b.double()
    assert _off(dw_in[:, F:], 16 * want) <= limit         # du = 16 dy
    assert _off(dw_out, 16 * want) <= limit
    assert _off(db_out, sum(b.double().sum(0) for b in dy.split(1 << 22))) <= limit


@pytest.mark.parametrize("T,limit", [(4, 2.0 ** -8), (64, 2.0 ** -8)])
def test_few_rows_over_many_features(T, limit):
    """A CTA's stretch of one column block is longer than an accumulator takes.  (The mean over the columns says no
    more than a column: the sums are 2^21 within 0.3 / sqrt(131072) of it, a fifth of a bf16 step, so that
    their roundings are much alike and do not cancel.)  A bias that takes a sum's leading bits away leaves
    2^-8 of it to be rounded to 2^-16, and shows what the sum itself has lost."""
    C, F = 16384, 131072
    u, w_out = _values((F,), torch.bfloat16, 3), _values((F, C), torch.bfloat16, 4)
    b_in = torch.cat([torch.full_like(u, 16.0), u])
    x = torch.zeros((T, C), dtype=torch.bfloat16, device="cuda")
    w_in = torch.zeros((C, 2 * F), dtype=torch.bfloat16, device="cuda")
    y = lap.gated_mlp(x, w_in, b_in, w_out, None, act="gelu")
    want = sum(16 * a.double() @ b.double() for a, b in zip(u.split(4096), w_out.split(4096)))
    assert float((y.double() / want - 1).abs().max()) <= limit + 2.0 ** -12
    assert torch.equal(y, y[:1].expand_as(y))
    b_out = -want.bfloat16()
    y = lap.gated_mlp(x, w_in, b_in, w_out, b_out, act="gelu")
    left = want + b_out.double()
    assert float(((y.double() - left).abs() - limit * left.abs()).div(want).max()) <= 2.0 ** -12
    assert torch.equal(y, y[:1].expand_as(y))


@pytest.mark.parametrize("T", [16, 100])
def test_few_rows_over_many_features_f32(T):
    C, F = 16384, 32768
    u, w_out = _values((F,), torch.float32, 3), _values((F, C), torch.float32, 4)
    b_in = torch.cat([torch.full_like(u, 16.0), u])
    x = torch.zeros((T, C), dtype=torch.float32, device="cuda")
    y = lap.gated_mlp(x, torch.zeros((C, 2 * F), device="cuda"), b_in, w_out, None, act="gelu")
    want = sum(16 * a.double() @ b.double() for a, b in zip(u.split(4096), w_out.split(4096)))
    assert float((y.double() / want - 1).abs().max()) <= 2.0 ** -17
    assert torch.equal(y, y[:1].expand_as(y))


@pytest.mark.parametrize("act,C", [("silu", 1024), ("gelu", 1024), ("silu", 1001)])
def test_rows_summed_over_many_features(act, C):
    """y and dx over more features than an accumulator takes, without ranges of them."""
    T, F = 4864, 20480
    gen = torch.Generator(device="cuda").manual_seed(5)
    r = lambda s, *shape: (torch.randn(shape, generator=gen, device="cuda") * s).bfloat16()  # noqa: E731
    t = dict(x=r(1.0, T, C), w_in=r(C ** -0.5, C, 2 * F), b_in=None, w_out=r(F ** -0.5, F, C), b_out=r(0.3, C))
    dy = r(1.0, T, C)
    p = lap.MlpParams(T, C, F, act)
    y, ctx = lap.mlp_fwd(**t, p=p)
    dx, *_ = lap.mlp_bwd(t["x"], t["w_in"], t["w_out"], dy, ctx, p, want=(True, False, False, False, False))
    ref = reference(**t, kind=act, dy=dy)
    check("y", y, ref["y"], torch.bfloat16)
    check("dx", dx, ref["x"], torch.bfloat16)


@pytest.mark.parametrize("dtype,T", [(torch.bfloat16, 3), (torch.float32, 3), (torch.float32, 20), (torch.float32, 200)])
def test_wide_rows(dtype, T):
    """C beyond what one accumulator of a large bf16 product sums."""
    C, F = 131080, 40
    gen = torch.Generator(device="cuda").manual_seed(5)
    r = lambda s, *shape: (torch.randn(shape, generator=gen, device="cuda") * s).to(dtype)  # noqa: E731
    t = dict(x=r(1.0, T, C), w_in=r(C ** -0.5, C, 2 * F), b_in=r(0.3, 2 * F), w_out=r(F ** -0.5, F, C), b_out=r(0.3, C))
    dy = r(1.0, T, C)
    p = lap.MlpParams(T, C, F)
    y, ctx = lap.mlp_fwd(**t, p=p)
    ref = reference(**t, kind="silu", dy=dy)
    check("y", y, ref["y"], dtype)
    for n, g in zip(("x", "w_in", "b_in", "w_out", "b_out"), lap.mlp_bwd(t["x"], t["w_in"], t["w_out"], dy, ctx, p)):
        check("d" + n, g, ref[n], dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_many_rows_of_odd_sizes(dtype):
    T, C, F = (1 << 21) + 77, 33, 21
    gen = torch.Generator(device="cuda").manual_seed(5)
    r = lambda s, *shape: (torch.randn(shape, generator=gen, device="cuda") * s).to(dtype)  # noqa: E731
    t = dict(x=r(1.0, T, C), w_in=r(C ** -0.5, C, 2 * F), b_in=r(0.3, 2 * F), w_out=r(F ** -0.5, F, C), b_out=r(0.3, C))
    dy = r(1.0, T, C)
    p = lap.MlpParams(T, C, F)
    y, ctx = lap.mlp_fwd(**t, p=p)
    grads = lap.mlp_bwd(t["x"], t["w_in"], t["w_out"], dy, ctx, p)
    again = lap.mlp_bwd(t["x"], t["w_in"], t["w_out"], dy, ctx, p)
    ref = reference(**t, kind="silu", dy=dy, block=16, kept=2.0 ** -11)
    check("y", y, ref["y"], dtype)
    for n, g, h in zip(("x", "w_in", "b_in", "w_out", "b_out"), grads, again):
        check("d" + n, g, ref[n], dtype)
        assert torch.equal(g, h), n
        # the bounds grow with the sum; the errors are those of roundings (fp32: 5 2^-24 of parts left out, and as much
        # again for each of activation, sums in registers and ranges, whose signs are mixed: below 32 2^-24)
        if n in ("w_in", "w_out"):
            off = float((g.double() - ref[n].v).norm() / ref[n].v.norm())
            assert off < (2.0 ** -19 if dtype == torch.float32 else 2.0 ** -8), (n, off)
