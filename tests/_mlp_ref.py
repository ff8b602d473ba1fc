"""The gated feed-forward block in 64 bits, with how far the kernels may be from it (_bounds.Off).

Products.  The tensor instruction adds 16 products at a time to its fp32 sum and cuts the result off: taken
as 2^-22 of the magnitudes summed, each time.  bf16 operands are exact, a sum over K is K / 16 such steps
(and up to 32 more additions where K is split).  fp32 operands are three bf16 parts, 2^-24 of each is left
out, and of nine products of parts three, below 3 * 2^-24; a0 b0 is summed over 128 of K by the instruction
(8 steps), and by fp32 additions beyond; the other five products, 2^-8 of the magnitudes together at most
(2^-7 with both orders), in K / 16 * 5 steps: (8 + K / 128 / 4 + 2^-7 K / 3.2) 2^-22 + 5 * 2^-24.
Activation.  An activation's and its slope's own error is taken as 2^-19 (bf16 calls: approximate
exponential and reciprocal, 2^-22 each, times small factors) or 2^-21 (fp32) of 1 + |g|; their slopes are
below 1.2.
Between the products bf16 calls round h and the gradient of (g | u), half a step; with two parts (up to 64
rows of whole 16-byte pieces, or T C F <= 2^28) half a step of what the first left, 2^-16 in all, and their products
run over both parts, one after the other: twice the steps.  Kept for the backward: p, q rounded to f16 (bf16 calls), `kept` of the value and 2^-38 of the
largest of a block (`block` features: 16 in the kernels).
"""
import math

import torch

from tests._bounds import F, U, Off


def steps(K, f32):
    if f32:
        return (8 + K / 512 + K / 400) * 4 * F + 5 * F
    return (K / 16 + 34) * 4 * F


def mm(a, b, f32):
    s = steps(a.v.shape[-1], f32)
    A, B = a.v.abs() + a.off, b.v.abs() + b.off
    return Off(a.v @ b.v, a.off @ B + A @ b.off + s * (A @ B) + 1e-37)


def tr(a):
    return Off(a.v.mT, a.off.mT)


def act(g, kind):
    """act(g), act'(g) in 64 bits"""
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if kind == "gelu":
        c = 0.5 * torch.special.erfc(-g / math.sqrt(2))
        return g * c, c + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


def mm2(a, b, two):
    """mm of bf16 values that are kept in one part or two (rounded here), summed over both"""
    def kept(o):
        return Off(o.v, o.off + (2.0 ** -16 if two else 2.0 ** -8) * (o.v.abs() + o.off))
    a, b = (kept(a[0]), b) if isinstance(a, tuple) else (a, kept(b[0]))
    s = steps(a.v.shape[-1], False) * (2 if two else 1)
    A, B = a.v.abs() + a.off, b.v.abs() + b.off
    return Off(a.v @ b.v, a.off @ B + A @ b.off + s * (A @ B) + 1e-37)


def reference(x, w_in, b_in, w_out, b_out, kind, dy=None, block=32, kept=2.0 ** -12):
    """{name: Off} of y and, with dy, of the gradients; x, dy [T, C]; block: features of a row with one scale;
    kept: how far an f16 value may be off (half a step of its 11 bits is up to 2^-11)"""
    f32, dt = x.dtype == torch.float32, x.dtype
    Fh = w_out.shape[0]
    T, C = x.shape
    two = T * C * Fh <= 2 ** 28 or (T <= 64 and C % 8 == 0 and Fh % 8 == 0)
    part = lambda o: (o,)  # noqa: E731
    X, W, V = Off.of(x), Off.of(w_in), Off.of(w_out)
    z = mm(X, W, f32)
    if b_in is not None:
        z = z + Off.of(b_in)
    g, u = z[:, :Fh], z[:, Fh:]
    p, s = act(g.v, kind)
    own = (2.0 ** -21 if f32 else 2.0 ** -19) * (1 + g.v.abs())
    p, s = Off(p, 1.2 * g.off + own), Off(s, 1.2 * g.off + own)
    h = p * u
    y = mm(h, V, True) if f32 else mm2(part(h), V, two)
    out = {"y": y if b_out is None else y + Off.of(b_out)}
    if dy is None:
        return out
    q = u * s
    if not f32:
        for o in (p, q):
            pad = (-Fh) % block
            big = torch.nn.functional.pad(o.v.abs(), (0, pad)).unflatten(1, (-1, block)).amax(-1)
            o.off = o.off + kept * (o.v.abs() + o.off) + 2.0 ** -38 * big.repeat_interleave(block, 1)[:, :Fh]
    D = Off.of(dy)
    dh = mm(D, tr(V), f32)
    dg, du = dh * q, dh * p
    dz = Off(torch.cat([dg.v, du.v], 1), torch.cat([dg.off, du.off], 1))
    if f32:
        out["x"], out["w_in"], out["w_out"] = mm(dz, tr(W), True), mm(tr(X), dz, True), mm(tr(h), D, True)
    else:
        out["x"], out["w_in"] = mm2(part(dz), tr(W), two), mm2(tr(X), part(dz), two)
        out["w_out"] = mm2(part(tr(h)), D, two)
        dz = Off(dz.v, dz.off + (2.0 ** -16 if two else 2.0 ** -8) * (dz.v.abs() + dz.off))
    rows = x.shape[0] + 64
    out["b_in"], out["b_out"] = dz.sum(0, rows), D.sum(0, rows)
    return out


def check_scale(ref: Off):
    """The errors allowed are those of a working kernel, not of any: below a tenth of the values' size."""
    return float(ref.off.norm() / ref.v.norm())


__all__ = ["U", "reference", "check_scale"]
