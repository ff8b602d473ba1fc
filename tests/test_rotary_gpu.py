"""Rotary positions against their definition in 64 bits.

A cosine is off by the phase's (cut to 2^-32 of a turn, rounded to fp32 as half turns in [-1, 1)): at most
pi (2^-31 + 2^-25), by sincospif (2 ulp) and by the factor's product: below 5 * 2^-24 in all.  Two products
and a sum add three roundings, so an output is within 8 * 2^-24 factor (|a| + |b|) of its value, before it
is rounded to the tensors' type (half a step)."""
import math

import pytest
import torch

import laplacian_nystr_linear_gb300 as lap

pytestmark = pytest.mark.gpu
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
DTYPES = [torch.float32, torch.bfloat16]


def _angles(freqs):
    return [(t % 2 ** 64) * 2.0 * math.pi / 2.0 ** 64 for t in freqs.turns.tolist()]


def _check(x, got, p, w, factor, layout, sign=1):
    """p: [B, N] positions on the host (whole numbers), w: radians of the pairs."""
    B, H, N, d = x.shape
    r = len(w)
    # whole turns taken off in whole numbers, so far positions stay exact
    angle = torch.tensor([[[math.fmod(int(a) * f, 2 * math.pi) for f in w] for a in row] for row in p.tolist()],
                         dtype=torch.float64, device=x.device)[:, None] * sign
    cos, sin = torch.cos(angle) * factor, torch.sin(angle) * factor
    i = torch.arange(r, device=x.device)
    first, second = (i, i + r) if layout == "half" else (2 * i, 2 * i + 1)
    v = x.double()
    a, b = v[..., first], v[..., second]
    ref, off = v.clone(), torch.zeros_like(v)
    ref[..., first], ref[..., second] = a * cos - b * sin, b * cos + a * sin
    off[..., first] = off[..., second] = 8 * 2.0 ** -24 * abs(factor) * (a.abs() + b.abs())
    off += U[x.dtype] * (ref.abs() + off)
    off[..., 2 * r:] = 0
    assert got.dtype == x.dtype and got.shape == x.shape
    assert ((got.double() - ref).abs() <= 1.01 * off).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,Hq,Hkv,N,d,rot", [
    (1, 1, 1, 1, 16, 16), (2, 4, 2, 37, 64, 64), (3, 5, 1, 1, 128, 128), (1, 12, 3, 130, 96, 64),
    (2, 3, 3, 9, 80, 24), (1, 2, 1, 17, 30, 6), (2, 1, 1, 5, 7, 2), (1, 33, 11, 3, 64, 48)])
def test_forward_and_gradients(dtype, layout, B, Hq, Hkv, N, d, rot):
    gen = torch.Generator(device="cuda").manual_seed(B * 1000 + N)
    q = torch.randn((B, Hq, N, d), generator=gen, device="cuda").to(dtype).requires_grad_(True)
    k = torch.randn((B, Hkv, N, d), generator=gen, device="cuda").to(dtype).requires_grad_(True)
    dq, dk = (torch.randn(x.shape, generator=gen, device="cuda").to(dtype) for x in (q, k))
    f = lap.rotary_frequencies(rot, scaling="parts", factor=8.0, context=4096)
    start = torch.tensor([7 + 100003 * b for b in range(B)], dtype=torch.int32, device="cuda")
    p = start.cpu().long()[:, None] + torch.arange(N)
    oq, ok = lap.rotary(q, k, f, start=start, layout=layout)
    w = _angles(f)
    _check(q.detach(), oq.detach(), p, w, f.factor, layout)
    _check(k.detach(), ok.detach(), p, w, f.factor, layout)
    gq, gk = torch.autograd.grad([oq, ok], [q, k], [dq, dk])
    _check(dq, gq, p, w, f.factor, layout, -1)
    _check(dk, gk, p, w, f.factor, layout, -1)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_positions_one_by_one_negative_and_far(layout):
    p = torch.tensor([[0, 1, -1, 5], [2 ** 31 - 1, -2 ** 31, 1 << 20, 999983]])
    q = torch.randn((2, 3, 4, 32), device="cuda")
    f = lap.rotary_frequencies(32)
    got = lap.rotary(q, None, f, positions=p.to(torch.int32).cuda(), layout=layout)
    assert got[1] is None
    # p w modulo a turn, in whole numbers of 2^-64
    turns = [t % 2 ** 64 for t in f.turns.tolist()]
    phase = torch.tensor([[[(int(a) * t % 2 ** 64) / 2.0 ** 64 for t in turns] for a in r] for r in p.tolist()],
                         dtype=torch.float64, device="cuda")[:, None] * (2 * math.pi)
    i = torch.arange(16, device="cuda")
    a, b = (i, i + 16) if layout == "half" else (2 * i, 2 * i + 1)
    z = torch.complex(q.double()[..., a], q.double()[..., b]) * torch.polar(torch.ones_like(phase), phase)
    off = 8 * 2.0 ** -24 * (q[..., a].abs() + q[..., b].abs()).double() * 1.2
    assert ((got[0][..., a].double() - z.real).abs() <= off).all()
    assert ((got[0][..., b].double() - z.imag).abs() <= off).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16"])
@pytest.mark.parametrize("layout,d,rot", [("half", 64, 64), ("half", 40, 20), ("interleaved", 64, 32),
                                          ("interleaved", 33, 10)])
def test_in_place_back_and_elsewhere(dtype, layout, d, rot):
    """In place and unaligned give the same bits; turned back it is what it was, up to roundings."""
    q, k = (torch.randn((2, h, 19, d), device="cuda").to(dtype) for h in (4, 2))
    f = lap.rotary_frequencies(rot)
    want = lap.rotary_apply(q, k, f, layout=layout)
    buf = torch.empty(q.numel() + 1, dtype=dtype, device="cuda")
    off = buf[1:].view(q.shape)
    off.copy_(q)
    got = lap.rotary_apply(off, k, f, layout=layout, q_out=off)
    assert torch.equal(off, want[0]) and torch.equal(got[1], want[1])
    q2, k2 = q.clone(), k.clone()
    lap.rotary_apply(q2, k2, f, layout=layout, q_out=q2, k_out=k2)
    assert torch.equal(q2, want[0]) and torch.equal(k2, want[1])
    back, _ = lap.rotary_apply(want[0], None, f, layout=layout, inverse=True)
    u = 2 * U[dtype] + 40 * 2.0 ** -24
    i = torch.arange(rot // 2, device="cuda")
    a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    size = q.double().abs()
    size[..., a] = size[..., b] = size[..., a] + size[..., b]
    assert ((back.double() - q.double()).abs() <= 2 * u * size).all()


def test_a_start_whose_last_positions_pass_32_bits():
    q = torch.randn((1, 2, 6, 32), device="cuda")
    f = lap.rotary_frequencies(32)
    got, _ = lap.rotary(q, None, f, start=torch.tensor([2 ** 31 - 3], dtype=torch.int32, device="cuda"))
    turns = [t % 2 ** 64 for t in f.turns.tolist()]
    phase = torch.tensor([[((2 ** 31 - 3 + n) * t % 2 ** 64) / 2.0 ** 64 for t in turns] for n in range(6)],
                         dtype=torch.float64, device="cuda") * (2 * math.pi)
    z = torch.complex(q.double()[..., :16], q.double()[..., 16:]) * torch.polar(torch.ones_like(phase), phase)
    off = 10 * 2.0 ** -24 * (q[..., :16].abs() + q[..., 16:].abs()).double()
    assert ((got[..., :16].double() - z.real).abs() <= off).all()
    assert ((got[..., 16:].double() - z.imag).abs() <= off).all()


def test_more_heads_than_a_grid_has_rows():
    q = torch.randn((1, 70000, 1, 8), device="cuda")
    f = lap.rotary_frequencies(8)
    start = torch.tensor([5], dtype=torch.int32, device="cuda")
    got, _ = lap.rotary(q, None, f, start=start)
    want, _ = lap.rotary(q.view(10, 7000, 1, 8), None, f, start=start.expand(10).contiguous())
    assert torch.equal(got.view(10, 7000, 1, 8), want)


def test_one_gradient_alone_and_none():
    q, k = (torch.randn((1, 2, 6, 16), device="cuda", requires_grad=True) for _ in range(2))
    f = lap.rotary_frequencies(16)
    oq, ok = lap.rotary(q, k, f)
    both = torch.autograd.grad([oq, ok], [q, k], [torch.ones_like(q), torch.ones_like(k)], retain_graph=True)
    assert torch.equal(torch.autograd.grad(oq.sum(), q, retain_graph=True)[0], both[0])
    assert torch.equal(torch.autograd.grad(ok.sum(), k, retain_graph=True)[0], both[1])
    assert torch.autograd.grad(ok.sum(), q, allow_unused=True)[0] is None


def test_captured_and_on_another_stream():
    q, k = (torch.randn((2, h, 40, 64), device="cuda").bfloat16() for h in (8, 2))
    f = lap.rotary_frequencies(64)
    start = torch.zeros(2, dtype=torch.int32, device="cuda")
    oq, ok = torch.empty_like(q), torch.empty_like(k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lap.rotary_apply(q, k, f, start=start, q_out=oq, k_out=ok)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lap.rotary_apply(q, k, f, start=start, q_out=oq, k_out=ok)
    start += 77
    q.neg_()
    g.replay()
    want = lap.rotary_apply(q, k, f, start=start)
    assert torch.equal(oq, want[0]) and torch.equal(ok, want[1])
