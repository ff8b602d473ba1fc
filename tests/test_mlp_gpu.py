"""The gated feed-forward block against its definition in 64 bits; errors: _mlp_ref.py."""
import pytest
import torch

import laplacian_nystr_linear_gb300 as lap
from tests._bounds import check
from tests._mlp_ref import reference

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16]
NAMES = ("x", "w_in", "b_in", "w_out", "b_out")


def _inputs(T, C, Fh, dtype, bias, seed=0, spread=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed + T + C + Fh)
    r = lambda s, *shape: (torch.randn(shape, generator=gen, device="cuda") * s).to(dtype)  # noqa: E731
    return dict(x=r(spread, T, C), w_in=r(C ** -0.5, C, 2 * Fh), b_in=r(0.3, 2 * Fh) if bias else None,
                w_out=r(Fh ** -0.5, Fh, C), b_out=r(0.3, C) if bias else None), r(1.0, T, C)


def _step(t, dy, act, names=NAMES):
    leaves = {n: None if v is None else v.clone().requires_grad_(n in names) for n, v in t.items()}
    y = lap.gated_mlp(**leaves, act=act)
    names = [n for n in names if t[n] is not None]
    return y.detach(), dict(zip(names, torch.autograd.grad(y, [leaves[n] for n in names], dy)))


SIZES = [(1, 8, 8), (3, 16, 24), (1, 64, 64), (31, 64, 128), (33, 72, 136), (128, 128, 256), (130, 40, 341),
         (256, 256, 64), (257, 512, 1408), (300, 100, 50), (64, 1, 1), (5, 7, 3), (513, 33, 129), (1000, 200, 264),
         (70, 1032, 40), (2, 520, 2056), (17, 64, 72)]


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("T,C,Fh", SIZES)
@pytest.mark.parametrize("act,bias", [("silu", False), ("gelu", True), ("gelu_tanh", False)])
def test_forward_and_gradients(dtype, T, C, Fh, act, bias):
    t, dy = _inputs(T, C, Fh, dtype, bias)
    ref = reference(**t, kind=act, dy=dy)
    y, grads = _step(t, dy, act)
    check("y", y, ref["y"], dtype)
    for n, g in grads.items():
        check("d" + n, g, ref[n], dtype)
    with torch.no_grad():
        check("y alone", lap.gated_mlp(**t, act=act), ref["y"], dtype)


@pytest.mark.parametrize("T,C,Fh", [(2, 24, 40), (6, 32, 72), (16, 32, 64), (200, 64, 128), (256, 512, 2048), (40, 2048, 4096)])
def test_small_calls_add_next_to_nothing_to_the_roundings_of_their_results(T, C, Fh):
    """h and the gradient of (g | u) in two parts: the 2-norm of the error is that of rounding the exact
    values, but for 2^-12 (p, q) and 2^-16, a tenth of a rounding's 2^-9 or so, squared beside it."""
    t, dy = _inputs(T, C, Fh, torch.bfloat16, True, 8)
    ref = reference(**t, kind="silu", dy=dy)
    y, grads = _step(t, dy, "silu")
    for n, got in (("y", y), *grads.items()):
        v = ref[n].v
        own, off = (v.bfloat16().double() - v).norm(), (got.double() - v).norm()
        # 2^-10 of the values: above what 2^-12 of every factor can add up to
        assert off <= 1.05 * own + 2.0 ** -10 * v.norm(), (n, float(off / own))


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 5, 8, 9, 16, 17, 33, 48, 63, 64, 65, 100, 128, 129])
@pytest.mark.parametrize("C,Fh,act", [(512, 2048, "silu"), (2048, 520, "gelu"), (1000, 3000, "gelu_tanh"), (66, 70, "silu"),
                                      (333, 1021, "silu")])
def test_few_rows(dtype, T, C, Fh, act):
    """Few rows go their own way (weights read once, split over all SMs), up to 64 in bf16, 128 in fp32."""
    t, dy = _inputs(T, C, Fh, dtype, T % 2 == 0, 6)
    ref = reference(**t, kind=act, dy=dy)
    first = lap.gated_mlp(**t, act=act)
    check("y", first, ref["y"], dtype)
    assert torch.equal(lap.gated_mlp(**t, act=act), first)
    y, grads = _step(t, dy, act)
    assert torch.equal(y, first) or T > 64
    for n, g in grads.items():
        check("d" + n, g, ref[n], dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
def test_long_sums_stay_close(dtype):
    """The drift of long sums, measured as a whole: 2-norm of the error over the value's."""
    t, dy = _inputs(4096, 1024, 1536, dtype, False)
    y, grads = _step(t, dy, "silu")
    w = {n: v.double() for n, v in t.items() if v is not None}
    z = w["x"] @ w["w_in"]
    g, u = z[:, :1536], z[:, 1536:]
    s = torch.sigmoid(g)
    h = g * s * u
    dh = dy.double() @ w["w_out"].T
    dz = torch.cat([dh * u * s * (1 + g * (1 - s)), dh * g * s], 1)
    want = {"y": (y, h @ w["w_out"]), "x": (grads["x"], dz @ w["w_in"].T), "w_in": (grads["w_in"], w["x"].T @ dz),
            "w_out": (grads["w_out"], h.T @ dy.double())}
    # bf16: two roundings of at most 2^-9 of a step's middle (uniform: 2^-8 / sqrt 3 / 2 of the values each);
    # fp32: 24-bit parts and sums cut off a few hundred times, far from one side
    for n, (a, b) in want.items():
        off = float((a.double() - b).norm() / b.norm())
        assert off < (1e-6 if dtype == torch.float32 else 2.0 ** -8), (n, off)


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("spread", [1e-30, 1e-4, 30.0, 1e8])
def test_far_magnitudes(dtype, spread):
    """Hidden values of any size: the factors kept for the backward are scaled row by row."""
    t, dy = _inputs(65, 64, 96, dtype, False, 3, spread)
    ref = reference(**t, kind="silu", dy=dy)
    y, grads = _step(t, dy, "silu")
    if spread > 1e-20 or dtype == torch.bfloat16:   # fp32: three parts reach down to 2^-110
        check("y", y, ref["y"], dtype)
        for n, g in grads.items():
            check("d" + n, g, ref[n], dtype)
    else:
        assert all(g.isfinite().all() for g in grads.values())


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
def test_repeats_and_partial_gradients(dtype):
    t, dy = _inputs(700, 96, 200, dtype, True, 1)
    y, whole = _step(t, dy, "gelu")
    y2, again = _step(t, dy, "gelu")
    assert torch.equal(y, y2) and all(torch.equal(whole[n], again[n]) for n in NAMES)
    for n in NAMES:
        assert torch.equal(_step(t, dy, "gelu", (n,))[1][n], whole[n]), n


def test_shapes_of_x_and_rows_that_are_not_finite():
    t, dy = _inputs(30, 64, 128, torch.bfloat16, False, 2)
    y = lap.gated_mlp(**t)
    x3 = t["x"].view(2, 5, 3, 64)
    assert torch.equal(lap.gated_mlp(**{**t, "x": x3}), y.view(x3.shape))
    t["x"][4, 9], t["x"][20, 0] = float("nan"), float("inf")
    got = lap.gated_mlp(**t)
    keep = [i for i in range(30) if i not in (4, 20)]
    assert torch.equal(got[keep], y[keep]) and got[4].isnan().all() and not got[20].isfinite().any()


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("T,C", [(5, 33), (130, 33)])
def test_gradient_that_is_a_piece_of_another(dtype, T, C):
    """Rows of no whole 16-byte pieces, concatenated: the second part's gradient starts anywhere."""
    t, dy = _inputs(T, C, 40, dtype, False, 9)
    leaves = {n: None if v is None else v.clone().requires_grad_(True) for n, v in t.items()}
    y = torch.cat([torch.zeros((1, C), dtype=dtype, device="cuda"), lap.gated_mlp(**leaves)])
    whole = torch.cat([dy[:1], dy])
    assert whole[1:].data_ptr() % 16 and whole[1:].is_contiguous()
    got = torch.autograd.grad(y, [v for v in leaves.values() if v is not None], whole)
    want = _step(t, dy, "silu", ("x", "w_in", "w_out"))[1]
    assert all(torch.equal(a, b) for a, b in zip(got, want.values()))


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("T", [3, 40])
def test_partial_gradients_of_few_rows(dtype, T):
    t, dy = _inputs(T, 96, 200, dtype, True, 1)
    whole = _step(t, dy, "gelu")[1]
    for n in NAMES:
        assert torch.equal(_step(t, dy, "gelu", (n,))[1][n], whole[n]), n


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
def test_two_streams_at_once(dtype):
    """Calls of few and of many rows side by side on two streams, each with its own workspace."""
    torch.cuda.synchronize()
    a, b = (_inputs(T, 1024, 2048, dtype, True, 7)[0] for T in (6, 40))
    c = _inputs(300, 128, 256, dtype, True, 7)[0]
    want = [lap.gated_mlp(**t) for t in (a, b, c)]
    torch.cuda.synchronize()
    streams, got = (torch.cuda.Stream(), torch.cuda.Stream()), []
    for i in range(8):
        with torch.cuda.stream(streams[i % 2]):
            got.append([lap.gated_mlp(**t) for t in (a, b, c)])
    torch.cuda.synchronize()
    for run in got:
        assert all(torch.equal(x, y) for x, y in zip(run, want))
    assert lap.api.load().lapnys_device_status(0) == 0


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 40, 300])
def test_captured_and_on_another_stream(T, dtype):
    t, dy = _inputs(T, 128, 256, dtype, True, 5)
    p = lap.MlpParams(T, 128, 256, "silu")

    def step():
        y, ctx = lap.mlp_fwd(**t, p=p)
        alone, _ = lap.mlp_fwd(**t, p=p, need_ctx=False)
        return [y, alone, *lap.mlp_bwd(t["x"], t["w_in"], t["w_out"], dy, ctx, p)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    t["x"].neg_()
    dy.mul_(2)
    g.replay()
    for a, b in zip(got, step()):
        assert torch.equal(a, b)
    assert lap.api.load().lapnys_device_status(0) == 0


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("T,C,Fh", [(130, 72, 136), (1, 64, 64), (40, 33, 50)])
def test_nothing_is_written_beside_the_outputs(dtype, T, C, Fh):
    """Outputs, ctx and workspace between guard bytes, filled with NaN before."""
    t, dy = _inputs(T, C, Fh, dtype, True, 4)
    p = lap.MlpParams(T, C, Fh, "silu")
    guards = []

    def room(nbytes):
        buf = torch.full((nbytes + 2048,), 0xFF, dtype=torch.uint8, device="cuda")
        buf[:1024] = 0x5A
        buf[1024 + nbytes:] = 0x5A
        guards.append((buf, nbytes))
        return buf[1024:1024 + nbytes]

    y = room(t["x"].nbytes).view(dtype).view(T, C)
    ctx = room(lap.mlp_ctx_bytes(p, dtype))
    lap.mlp_fwd(**t, p=p, y=y, ctx=ctx, ws=room(lap.mlp_workspace_bytes(p, dtype)))
    grads = lap.mlp_bwd(t["x"], t["w_in"], t["w_out"], dy, ctx, p, ws=room(lap.mlp_workspace_bytes(p, dtype, True)))
    y2, want = _step(t, dy, "silu")
    assert torch.equal(y, y2) and all(torch.equal(a, want[n]) for n, a in zip(NAMES, grads))
    for buf, n in guards:
        assert (buf[:1024] == 0x5A).all() and (buf[1024 + n:] == 0x5A).all()
