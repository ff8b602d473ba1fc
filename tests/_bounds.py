"""Values in 64 bits that carry how far a computation in 32 bits may be from them.

Every operation adds what one rounding to nearest may add (2^-24 of the result) to what its operands'
errors make of it; a sum of n terms adds at most `deep` roundings to each term, where deep is the longest
chain of additions that a term goes through.  `stored` is a rounding to the tensors' type.
"""
import math

import torch

F = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


class Off:
    def __init__(self, v, off=None):
        self.v = v
        self.off = torch.zeros_like(v) if off is None else off

    @staticmethod
    def of(t):
        return Off(t.double())

    def _up(self, v, off):
        return Off(v, off + F * v.abs() + 1e-37)      # products may be flushed below the normal range

    def __add__(self, o):
        o = o if isinstance(o, Off) else Off(torch.as_tensor(float(o), dtype=torch.float64, device=self.v.device))
        return self._up(self.v + o.v, self.off + o.off)

    def __sub__(self, o):
        return self + Off(-o.v, o.off)

    def __mul__(self, o):
        o = o if isinstance(o, Off) else Off(torch.as_tensor(float(o), dtype=torch.float64, device=self.v.device))
        return self._up(self.v * o.v, self.v.abs() * o.off + self.off * o.v.abs() + self.off * o.off)

    def __getitem__(self, i):
        return Off(self.v[i], self.off[i])

    def sum(self, dim, deep, keepdim=False):
        v = self.v.sum(dim, keepdim)
        return Off(v, (self.off + deep * F * (self.v.abs() + self.off)).sum(dim, keepdim) + 1e-37)

    def mean(self, deep):
        return self.sum(-1, deep, True) * (1.0 / self.v.shape[-1])

    def rsqrt(self):
        lo = (self.v - self.off).clamp(min=1e-300)
        v = self.v ** -0.5
        return Off(v, lo ** -0.5 - v + 4 * F * v)     # rsqrtf: within 2 ulp

    def stored(self, dtype):
        return Off(self.v, self.off + U[dtype] * (self.v.abs() + self.off))


def check(name, got, ref: Off, dtype):
    """got (of dtype) within the allowed error of ref's values, rounded once to dtype."""
    ref = ref.stored(dtype)
    assert got.shape == ref.v.shape, (name, got.shape, ref.v.shape)
    assert got.dtype == dtype, name
    far = (got.double() - ref.v).abs() / (1.01 * ref.off + 1e-35)
    worst = float(torch.nan_to_num(far, nan=math.inf).max()) if far.numel() else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3g} times the allowed error"
    return worst
