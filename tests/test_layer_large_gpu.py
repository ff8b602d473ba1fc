"""Tensors of more than 2^31 elements: what lies behind that is what a call of the last rows alone gives."""
import pytest
import torch

import laplacian_nystr_linear_gb300 as lap

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16]


def _rand(shape, seed, dtype):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(shape, dtype=dtype, device="cuda")
    for part in t.view(-1).split(1 << 28):
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda"))
    return t


@pytest.fixture(autouse=True)
def _room():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("layout,d,rot", [("half", 128, 128), ("interleaved", 64, 32), ("half", 33, 10)])
def test_rotary(dtype, layout, d, rot):
    N, last = (1 << 31) // (2 * d) + 5, 300
    q = _rand((1, 2, N, d), 1, dtype)
    f = lap.rotary_frequencies(rot)
    tail = q[:, :, -last:].contiguous()
    start = torch.tensor([N - last], dtype=torch.int32, device="cuda")
    want, _ = lap.rotary_apply(tail, None, f, start=start, layout=layout)
    lap.rotary_apply(q, None, f, layout=layout, q_out=q)
    assert torch.equal(q[:, :, -last:], want)


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("C", [512, 1001, 64, 9216])
def test_norms(dtype, C):
    """A tail of whole tiles and sequences of its own, so that its rows go the same way."""
    N, last = 1 << 10, 2
    B = (1 << 31) // (N * C) + last + 1
    x, u = _rand((B, N, C), 1, dtype), _rand((B, N, C), 2, dtype)
    vec = dict(post_weight=_rand((C,), 3, dtype), post_bias=None, gate=_rand((B, C), 4, dtype), scale=None)
    w = _rand((C,), 5, dtype)
    cut = lambda t: t[-last:].contiguous()  # noqa: E731
    out = []
    for x, u, g, b in ((x, u, vec["gate"], B), (cut(x), cut(u), cut(vec["gate"]), last)):
        p = lap.NormParams(b, N, C, False, "layer", "rms", 1e-6)
        v = {**vec, "gate": g}
        h, y, st = lap.norm_fwd(x, u, w, None, p, **v)
        dx, du, *_, dgate, _ = lap.norm_bwd(x, u, w, st, u, x, p, **v,
                                            want=(True, True, False, False, False, False, True, False))
        out.append([t[-last:].clone() for t in (h, y, st, dx, du, dgate)])
        del h, y, st, dx, du
    for n, a, b in zip(("h", "y", "stats", "dx", "du"), *out):
        assert torch.equal(a, b), n
    # the sums' rows are shared among the blocks otherwise
    off = (out[0][5].double() - out[1][5].double()).norm() / out[1][5].double().norm()
    assert float(off) < (1e-5 if dtype == torch.float32 else 2.0 ** -7)


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("C,F", [(512, 8), (8, 520)])
def test_feed_forward(dtype, C, F):
    """Both x and the hidden values: the last 2^20 rows alone are rounded between the products alike."""
    T, last = (1 << 31) // max(C, F) + 259, 1 << 20
    x, dy = _rand((T, C), 1, dtype), _rand((T, C), 2, dtype)
    w_in, w_out = _rand((C, 2 * F), 3, dtype) * C ** -0.5, _rand((F, C), 4, dtype) * F ** -0.5
    out = []
    for x, dy, n in ((x, dy, T), (x[-last:].clone(), dy[-last:].clone(), last)):
        p = lap.MlpParams(n, C, F)
        y, ctx = lap.mlp_fwd(x, w_in, None, w_out, None, p)
        dx, *_ = lap.mlp_bwd(x, w_in, w_out, dy, ctx, p, want=(True, False, False, False, False))
        out.append([t[-last:].clone() for t in (y, dx)])
        del y, ctx, dx
    for n, a, b in zip(("y", "dx"), *out):
        assert torch.equal(a, b), n
    assert lap.api.load().lapnys_device_status(0) == 0
