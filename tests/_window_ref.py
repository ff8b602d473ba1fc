"""Windowed attention in 64 bits, plainly, and how far fp32 / bf16 kernels may be from it.

A rounding to a type is off by at most u = finfo.eps / 2 of the value (bf16 2^-8, fp32 2^-24).
With P the exact probabilities, |.| elementwise:

bf16 forward   the operands' products are exact in fp32, P is rounded once (u), the output once (u):
               |o - ref| <= u |ref| + u P|v|, and fp32 sums on top.
bf16 backward  dv: P and the result rounded once:            u |dv| + u P^T|do|
               dq, dk: dS and the result rounded once; D = do.o uses the rounded output, which is
               off by do_i = u (|o| + P|v|), so dS is off by P D_off with D_off = |do|.o_off:
               u |dq| + scale (u |dS| + P D_off) |K|, and the same transposed for dk.
with rest      the backward reads out + rest, off by u^2 |o| + u P|v| only, and dq takes dS in two
               parts (u^2); dk as before.
fp32 sums      a score is off by at most (d + 4) 2^-24 scale |q|.|k| =: E (twice in P, twice more
               through the log-sum), a sum of n terms by (n + 16) 2^-24 of its terms' magnitudes.
"""
import math

import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def visible(Nq, Nk, left, right, sinks, lens, q_pos, device):
    p = q_pos[:, None, None].long() + torch.arange(Nq, device=device)[None, :, None]
    j = torch.arange(Nk, device=device)[None, None, :]
    n = lens[:, None, None].long().clamp(0, Nk)
    ok = (p >= 0) & (p < n) & (j < n)
    if right >= 0:
        ok &= j <= p + right
    if left >= 0:
        ok &= (j >= p - left) | (j < sinks)
    return ok                                             # [B, Nq, Nk]


def reference(q, k, v, left, right, sinks, scale=None, lens=None, q_pos=None, dout=None,
              extra_p=0.0, extra_s=0.0, rest=False):
    """{name: (64-bit value, allowed error)} of out, lse and, with dout, dq, dk, dv.
    extra_p, extra_s: further relative error of P and of the scores' magnitudes |q|.|k|.
    rest: the gradients' errors with the forward's rest, and ref["both"] for out + rest."""
    dt, dev = q.dtype, q.device
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1:3]
    g = Hq // Hkv
    scale = d ** -0.5 if scale is None else scale
    lens = torch.full((B,), Nk, device=dev) if lens is None else lens
    q_pos = torch.full((B,), Nk - Nq, device=dev) if q_pos is None else q_pos
    ok = visible(Nq, Nk, left, right, sinks, lens, q_pos, dev)[:, None]
    alive = (torch.arange(Nk, device=dev)[None] < lens[:, None])[:, None, :, None]

    def heads(x):   # what lies behind a sequence may be anything
        return torch.where(alive, x.double(), 0.0).repeat_interleave(g, dim=1)

    rows = ok.any(-1)[..., None]                           # [B, 1, Nq, 1]
    Q, K, V = torch.where(rows, q.double(), 0.0), heads(k), heads(v)
    s = Q @ K.transpose(-1, -2) * scale
    mag = (Q.abs() @ K.abs().transpose(-1, -2)) * scale    # |q|.|k|
    s = torch.where(ok, s, -math.inf)
    mx = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(mx.isinf(), 0.0, mx))
    t = e.sum(-1, keepdim=True)
    P = torch.where(t > 0, e / t, 0.0)
    o = P @ V
    u, f = U[dt], 2.0 ** -24
    E = torch.where(ok, mag, 0.0).amax(-1, keepdim=True) * ((d + 4) * f + extra_s)
    n = Nk
    pr = 4 * E + (n + 16) * f + extra_p                    # relative error of P by the sums
    up = u if dt == torch.bfloat16 else 0.0                # P and dS rounded between products
    Pv = P @ V.abs()
    o_off = u * o.abs() + (up + pr) * Pv
    lse = torch.where(t > 0, mx + torch.log(t), -math.inf)[..., 0] / math.log(2)
    lse_off = torch.where(lse.isinf(), 0.0, 1.5 * pr[..., 0] + 4 * f * lse.abs() + 1e-30)
    got = {"out": (o, 1.01 * o_off + 1e-30), "lse": (lse, lse_off)}
    if rest:
        o_off = u * u * o.abs() + (up + pr) * Pv
        got["both"] = (o, 1.01 * o_off + 1e-30)
    if dout is None:
        return got
    dO = torch.where(rows, dout.double(), 0.0)
    dP = dO @ V.transpose(-1, -2)
    D = (dO * o).sum(-1, keepdim=True)
    dS = P * (dP - D)
    back = (d + 16) * f
    dPm = dO.abs() @ V.abs().transpose(-1, -2)             # magnitudes of the sums in dP
    D_off = (dO.abs() * o_off).sum(-1, keepdim=True) + back * (dO.abs() * o.abs()).sum(-1, keepdim=True)
    dS_off = P * (D_off + back * dPm) + 2 * pr * P * (dP.abs() + D.abs())
    up_q = up * up if rest else up
    tr = lambda x: x.transpose(-1, -2)  # noqa: E731
    kv = lambda x: x.reshape(B, Hkv, g, Nk, d).sum(2)      # noqa: E731
    n2 = (Nq * g + 16) * f
    dq, dk, dv = dS @ K * scale, kv(tr(dS) @ Q) * scale, kv(tr(P) @ dO)
    dS_n = dS_off + (up_q + (n + 16) * f) * dS.abs()
    dS_g = dS_off + (up + n2) * dS.abs()
    dq_off = u * dq.abs() + scale * (dS_n @ K.abs())
    dk_off = u * dk.abs() + scale * kv(tr(dS_g) @ Q.abs())
    dv_off = u * dv.abs() + kv(tr(P * (up + 2 * pr + n2)) @ dO.abs())
    got.update(dq=(dq, 1.01 * dq_off + 1e-30), dk=(dk, 1.01 * dk_off + 1e-30),
               dv=(dv, 1.01 * dv_off + 1e-30))
    return got


def check(name, got, ref):
    value, off = ref
    assert got.shape == value.shape, (name, got.shape, value.shape)
    x = got.double()
    same = x.isinf() & (x == value)
    far = torch.where(same, 0.0, (x - value).abs() / off.clamp(min=1e-300))
    far = torch.where(same | ((x == value) & ~x.isnan()), 0.0, far)
    worst = float(torch.nan_to_num(far, nan=math.inf).max()) if far.numel() else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3g} times the allowed error"
    return worst
