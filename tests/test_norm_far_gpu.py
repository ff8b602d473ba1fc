"""Layer norms of rows whose mean is far above their deviation: the backward from the forward's statistics.

The statistics are taken as they are (fp32), so that their own rounding is in the reference too: what is left is
a subtraction, a product and the sums (errors carried along by _bounds.py; DEEP: a row's sum)."""
import pytest
import torch

import laplacian_nystr_linear_gb300 as lap
from tests._bounds import Off, check

pytestmark = pytest.mark.gpu
DEEP = 53
DTYPES = [torch.float32, torch.bfloat16]
WIDTHS = [8, 40, 64, 100, 128, 320, 321, 512, 1000, 1001, 1024, 2048, 4096, 6144, 8192, 12288]
NONE = (False,) * 8


def _inputs(N, C, dtype):
    gen = torch.Generator(device="cuda").manual_seed(C + N)
    r = lambda s, m, *shape: (torch.randn(shape, generator=gen, device="cuda") * s + m).to(dtype)  # noqa: E731
    return r(1.0, 4000.0, 2, N, C), r(0.2, 1.0, C), r(0.2, 0.0, C), r(1.0, 0.0, 2, N, C)


def _through(e, z, mean, r):
    """(unit(z), the gradient of z) of a layer norm with these statistics"""
    hat = (Off.of(z) - Off.of(mean)) * Off.of(r)
    t = e - hat * (e * hat).mean(DEEP) - e.mean(DEEP)
    return hat, Off.of(r) * t


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("N", [3, 40])
@pytest.mark.parametrize("C", WIDTHS)
def test_norm_of_the_sum(dtype, N, C):
    x, w, _, dy = _inputs(N, C, dtype)
    p = lap.NormParams(2, N, C, False, "layer", None, 1e-6)
    _, _, st = lap.norm_fwd(x, None, w, None, p)
    e = Off.of(dy) * Off.of(w)
    hat, want = _through(e, x, st[..., 2:3], st[..., 3:4])
    for biased in (True, False):
        dx, _, dw, db, *_ = lap.norm_bwd(x, None, w, st, None, dy, p, want=(True, False, True, biased) + NONE[4:])
        check("dx", dx, want, dtype)
        check("dweight", dw, (Off.of(dy) * hat).sum((0, 1), 2 * N + 64), dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("N", [3, 40])
@pytest.mark.parametrize("C", WIDTHS)
def test_norm_of_the_block(dtype, N, C):
    u, w, b, dh = _inputs(N, C, dtype)
    p = lap.NormParams(2, N, C, False, None, "layer", 1e-6)
    _, _, st = lap.norm_fwd(dh, u, None, None, p, post_weight=w, post_bias=b)
    e = Off.of(dh) * Off.of(w)
    hat, want = _through(e, u, st[..., 0:1], st[..., 1:2])
    for biased in (True, False):
        _, du, _, _, dw, db, _, _ = lap.norm_bwd(dh, u, None, st, dh, None, p, post_weight=w, post_bias=b,
                                                 want=(False, True, False, False, True, biased, False, False))
        check("du", du, want, dtype)
        check("dpost_weight", dw, (Off.of(dh) * hat).sum((0, 1), 2 * N + 64), dtype)
