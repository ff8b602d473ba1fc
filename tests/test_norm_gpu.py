"""The residual with its norms against its definition, with errors carried along (_bounds.py).

A row's sum goes through at most 16 additions in a thread, 5 in its warp and 32 over the warps; a sum over
rows through the rows of a group, 8 groups, 32 threads of 10 parts or sequences each at the sizes here."""
import pytest
import torch

import laplacian_nystr_linear_gb300 as lap
from tests._bounds import Off, check

pytestmark = pytest.mark.gpu
DEEP = 53
DTYPES = [torch.float32, torch.bfloat16]
NAMES = ("x", "u", "weight", "bias", "post_weight", "post_bias", "gate", "scale")


def _unit(z, kind, eps):
    """(unit norm, 1 / deviation)"""
    if kind == "layer":
        z = z - z.mean(DEEP)
    r = ((z * z).mean(DEEP) + eps).rsqrt()
    return z * r, r


def _through(e, hat, r, kind):
    t = e - hat * (e * hat).mean(DEEP)
    if kind == "layer":
        t = t - e.mean(DEEP)
    return r * t


def _reference(t, pre, post, eps, dh=None, dy=None):
    o = {n: None if v is None else Off.of(v) for n, v in t.items()}
    seq = lambda v: v[:, None] if v is not None and v.v.dim() == 2 else v  # noqa: E731
    w, b, gate = seq(o["weight"]), seq(o["bias"]), seq(o["gate"])
    mul = lambda z, f: z if f is None else z * f  # noqa: E731
    h = o["x"]
    if t["u"] is not None:
        uh, ur = _unit(o["u"], post, eps) if post else (o["u"], None)
        n = mul(uh, o["post_weight"])
        n = n if o["post_bias"] is None else n + o["post_bias"]
        h = h + mul(mul(n, gate), o["scale"])
    out = {"h": h}
    if pre:
        hh, hr = _unit(h, pre, eps)
        y = mul(hh, w)
        out["y"] = y if b is None else y + b
    if dh is None and dy is None:
        return out
    B, N, C = t["x"].shape
    rows = N * B + 64
    dt = Off.of(torch.zeros_like(t["x"]) if dh is None else dh)
    if pre and dy is not None:
        d = Off.of(dy)
        dt = dt + _through(mul(d, w), hh, hr, pre)
        wide = t["weight"] is not None and t["weight"].dim() == 2
        dims = 1 if wide else (0, 1)
        out["weight"] = (d * hh).sum(dims, rows)
        out["bias"] = d.sum(1 if t["bias"] is not None and t["bias"].dim() == 2 else (0, 1), rows)
    out["x"] = dt
    if t["u"] is not None:
        dn = mul(mul(dt, gate), o["scale"])
        out["u"] = _through(mul(dn, o["post_weight"]), uh, ur, post) if post else dn
        S3, S4 = (dt * uh).sum(1, rows), dt.sum(1, rows)                  # [B, C]
        m = mul(mul(Off.of(torch.ones((B, C), device="cuda")), o["gate"]), o["scale"])
        out["post_weight"], out["post_bias"] = (m * S3).sum(0, 64 + B), (m * S4).sum(0, 64 + B)
        G = mul(S3, o["post_weight"])
        G = G if o["post_bias"] is None else G + o["post_bias"] * S4
        out["gate"] = mul(G, o["scale"])
        out["scale"] = mul(G, o["gate"]).sum(0, 64 + B)
    return out


def _inputs(B, N, C, dtype, seed, given):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    shapes = dict(x=(B, N, C), u=(B, N, C), weight=(C,), bias=(C,), post_weight=(C,), post_bias=(C,),
                  gate=(B, C), scale=(C,))
    if "per_seq" in given:
        shapes.update(weight=(B, C), bias=(B, C))
    return {n: (torch.randn(s, generator=gen, device="cuda") * 0.5 + 0.5).to(dtype)
            if n == "x" or n in given else None for n, s in shapes.items()}


ALL = ("u", "weight", "bias", "post_weight", "post_bias", "gate", "scale")
SHAPES = [(1, 1, 1), (2, 3, 8), (1, 40, 16), (3, 37, 100), (2, 65, 256), (2, 33, 264), (1, 50, 512),
          (4, 19, 520), (2, 21, 1000), (1, 9, 1032), (1, 3, 2048), (2, 5, 4104), (1, 2, 8192), (1, 3, 16384),
          (70, 2, 64), (400, 1, 24), (1, 3, 4101), (2, 2, 9001)]


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("B,N,C", SHAPES)
@pytest.mark.parametrize("pre,post,given", [
    ("rms", None, ("weight",)), ("layer", "layer", ALL), ("rms", "rms", ("u", "post_weight", "scale")),
    ("layer", None, ("u", "gate", "bias")), (None, "rms", ("u", "gate", "post_weight")),
    ("layer", "rms", ALL + ("per_seq",)), (None, None, ("u", "scale"))],
    ids=["norm", "all", "rms2", "gate", "post", "per_seq", "add"])
def test_forward_and_gradients(dtype, B, N, C, pre, post, given):
    t = _inputs(B, N, C, dtype, B + N + C, given)
    leaves = {n: None if v is None else v.clone().requires_grad_(True) for n, v in t.items()}
    h, y = lap.residual_norm(**leaves, pre=pre, post=post, eps=1e-5)
    assert (y is None) == (pre is None)
    gen = torch.Generator(device="cuda").manual_seed(1)
    dh, dy = (torch.randn(t["x"].shape, generator=gen, device="cuda").to(dtype) for _ in range(2))
    dh = dh if t["u"] is not None else None
    dy = dy if pre else None
    ref = _reference(t, pre, post, 1e-5, dh, dy)
    outs, grads = zip(*[(o, g) for o, g in ((h, dh), (y, dy)) if g is not None])
    if t["u"] is not None:
        check("h", h.detach(), ref["h"], dtype)
    else:
        assert h is leaves["x"]
    if pre:
        check("y", y.detach(), ref["y"], dtype)
    names = [n for n in NAMES if t[n] is not None]
    for n, g in zip(names, torch.autograd.grad(outs, [leaves[n] for n in names], grads)):
        check("d" + n, g, ref[n], dtype)
    with torch.no_grad():
        h2, y2 = lap.residual_norm(**t, pre=pre, post=post, eps=1e-5)
    assert torch.equal(h2, h) and (pre is None or torch.equal(y2, y))


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
def test_many_rows_repeat_bit_for_bit(dtype):
    t = _inputs(3, 1500, 320, dtype, 5, ALL)
    dh, dy = torch.randn_like(t["x"]), torch.randn_like(t["x"])
    ref = _reference(t, "layer", "layer", 1e-6, dh, dy)
    runs = []
    for _ in range(2):
        leaves = {n: v.clone().requires_grad_(True) for n, v in t.items()}
        h, y = lap.residual_norm(**leaves, pre="layer", post="layer")
        runs.append([h, y, *torch.autograd.grad([h, y], list(leaves.values()), [dh, dy])])
    for n, a, b in zip(("h", "y") + NAMES, *runs):
        assert torch.equal(a, b), n
        check(n, a.detach(), ref[n], dtype)


def test_only_one_output_or_one_input_wanted():
    t = _inputs(2, 33, 96, torch.float32, 3, ALL)
    dh, dy = torch.randn_like(t["x"]), torch.randn_like(t["x"])
    leaves = {n: v.clone().requires_grad_(True) for n, v in t.items()}
    h, y = lap.residual_norm(**leaves, pre="rms", post="rms")
    zero = torch.zeros_like(dh)
    whole = torch.autograd.grad([h, y], list(leaves.values()), [dh, zero], retain_graph=True)
    alone = torch.autograd.grad(h, list(leaves.values()), dh, retain_graph=True, allow_unused=True)
    for n, a, b in zip(NAMES, whole, alone):
        assert torch.equal(a, b) if b is not None else n in ("weight", "bias"), n
    whole = torch.autograd.grad([h, y], list(leaves.values()), [zero, dy], retain_graph=True)
    alone = torch.autograd.grad(y, list(leaves.values()), dy)
    assert all(torch.equal(a, b) for a, b in zip(whole, alone))
    for n in NAMES:
        leaf = t[n].clone().requires_grad_(True)
        h, y = lap.residual_norm(**{**t, n: leaf}, pre="rms", post="rms")
        g, = torch.autograd.grad([h, y], [leaf], [zero, dy])
        assert torch.equal(g, whole[NAMES.index(n)]), n


def test_the_same_tensor_twice():
    x = torch.randn((2, 8, 64), device="cuda", requires_grad=True)
    h, y = lap.residual_norm(x, x)
    g, = torch.autograd.grad((h.sum() + (y * y.detach()).sum()), x)
    a, b = (x.detach().clone().requires_grad_(True) for _ in range(2))
    h, y = lap.residual_norm(a, b)
    ga, gb = torch.autograd.grad((h.sum() + (y * y.detach()).sum()), [a, b])
    assert torch.equal(g, ga + gb)


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
def test_unaligned_storage_gives_the_same(dtype):
    """Single elements instead of 16-byte pieces: other sums, within the same bounds."""
    t = _inputs(2, 11, 136, dtype, 9, ALL)
    ref = _reference(t, "layer", "rms", 1e-6)
    for n in NAMES:
        buf = torch.empty(t[n].numel() + 1, dtype=dtype, device="cuda")
        moved = buf[1:].view(t[n].shape)
        moved.copy_(t[n])
        h, y = lap.residual_norm(**{**t, n: moved}, pre="layer", post="rms")
        check("h", h, ref["h"], dtype)
        check("y", y, ref["y"], dtype)


def test_non_finite_rows_stay_their_own():
    t = _inputs(1, 40, 128, torch.bfloat16, 2, ("u", "weight"))
    want = lap.residual_norm(**t)
    t["u"][0, 7, 3] = float("nan")
    t["x"][0, 20, 5] = float("inf")
    got = lap.residual_norm(**t)
    keep = [i for i in range(40) if i not in (7, 20)]
    for a, b in zip(got, want):
        assert torch.equal(a[:, keep], b[:, keep])
    assert got[1][0, 7].isnan().all()


def test_captured_step():
    t = _inputs(2, 64, 128, torch.bfloat16, 4, ALL)
    dh, dy = torch.randn_like(t["x"]), torch.randn_like(t["x"])
    p = lap.NormParams(2, 64, 128, False, "layer", "layer", 1e-6)
    ws = torch.empty(lap.norm_workspace_bytes(2, 64, 128, True), dtype=torch.uint8, device="cuda")
    vec = {n: t[n] for n in ("post_weight", "post_bias", "gate", "scale")}

    def step():
        h, y, st = lap.norm_fwd(t["x"], t["u"], t["weight"], t["bias"], p, **vec)
        return [h, y, *lap.norm_bwd(t["x"], t["u"], t["weight"], st, dh, dy, p, **vec, ws=ws)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    t["x"].mul_(-1)
    g.replay()
    for a, b in zip(got, step()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("B,N,C", [(1, 3, 1), (3, 5, 1), (2, 7, 3), (1, 17, 5), (3, 33, 7), (5, 16, 2), (1, 129, 9),
                                   (2, 100, 33), (4, 37, 514), (2, 301, 321), (1, 29, 1001), (2, 13, 2047), (3, 9, 4095),
                                   (2, 700, 258), (1, 2000, 301)])
def test_rows_that_are_no_whole_pieces(dtype, B, N, C):
    """Rows that start anywhere in 16 bytes, tensors that end anywhere; guard rows behind the inputs hold NaN,
    which no sum may meet; the gradients of inputs that start at an odd element agree within the same bounds."""
    t = _inputs(B, N, C, dtype, B + N + C, ALL)
    dh, dy = torch.randn_like(t["x"]), torch.randn_like(t["x"])
    ref = _reference(t, "layer", "layer", 1e-6, dh, dy)
    p = lap.NormParams(B, N, C, False, "layer", "layer", 1e-6)
    vec = {n: t[n] for n in ("post_weight", "post_bias", "gate", "scale")}
    for off in (0, 1):
        def put(v):
            buf = torch.full((v.numel() + off + 64,), float("nan"), dtype=dtype, device="cuda")
            moved = buf[off:off + v.numel()].view(v.shape)
            moved.copy_(v)
            return moved

        x, u, gh, gy = (put(v) for v in (t["x"], t["u"], dh, dy))
        h, y, st = lap.norm_fwd(x, u, t["weight"], t["bias"], p, **vec)
        check("h", h, ref["h"], dtype)
        check("y", y, ref["y"], dtype)
        for n, g in zip(NAMES, lap.norm_bwd(x, u, t["weight"], st, gh, gy, p, **vec)):
            check("d" + n, g, ref[n], dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("B,N,C", [(2, 200, 512), (3, 77, 1000), (1, 333, 514), (2, 300, 321), (2, 200, 2048), (2, 100, 4096),
                                   (1, 90, 4608), (2, 60, 5001), (2, 80, 6144), (1, 170, 8192)])
def test_weights_without_biases(dtype, B, N, C):
    """Two kinds of sums over the rows instead of four: more rows at once, and wider ones."""
    t = _inputs(B, N, C, dtype, B + N + C, ("u", "weight", "post_weight", "gate"))
    dh, dy = torch.randn_like(t["x"]), torch.randn_like(t["x"])
    p = lap.NormParams(B, N, C, False, "rms", "rms", 1e-6)
    ref = _reference(t, "rms", "rms", 1e-6, dh, dy)
    vec = {n: t[n] for n in ("post_weight", "post_bias", "gate", "scale")}
    _, _, st = lap.norm_fwd(t["x"], t["u"], t["weight"], None, p, **vec)
    want = tuple(t[n] is not None for n in NAMES)
    grads = lap.norm_bwd(t["x"], t["u"], t["weight"], st, dh, dy, p, **vec, want=want)
    for n, g in zip(NAMES, grads):
        assert (g is not None) == (t[n] is not None)
        if g is not None:
            check("d" + n, g, ref[n], dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("B,N,C", [(1, 1000, 64), (4, 300, 128), (2, 777, 18), (3, 500, 40), (1, 3000, 5), (2, 130, 127),
                                   (1, 600, 8), (2, 1025, 1), (3, 33, 96), (40, 17, 64)])
@pytest.mark.parametrize("pre,post,given", [
    ("rms", None, ("weight",)), ("layer", "layer", ALL), ("layer", "rms", ALL + ("per_seq",)),
    ("rms", "rms", ("u", "weight", "post_weight"))], ids=["norm", "all", "per_seq", "rms2"])
def test_narrow_rows(dtype, B, N, C, pre, post, given):
    """Several rows to a warp (a head's features), tiles that a sequence ends in."""
    test_forward_and_gradients(dtype, B, N, C, pre, post, given)
