"""What stands around the attentions in a layer: rotary positions, the residual with its norms, and the
gated feed-forward block.  Marshalling only: every step runs in liblapnys kernels."""
from __future__ import annotations

import functools
import math
from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._lib import check, load
from .api import _DT, _dtype
from .window import _at, _nbytes, _no_tangent, _on, _on_stream, _sizes, _tensor, _workspace

_LAYOUT = {"half": _lib.LAPNYS_HALF, "interleaved": _lib.LAPNYS_INTERLEAVED}
_ACT = {"silu": _lib.LAPNYS_SILU, "gelu": _lib.LAPNYS_GELU, "gelu_tanh": _lib.LAPNYS_GELU_TANH}
_NORM = {None: _lib.LAPNYS_NONE, "rms": _lib.LAPNYS_RMS, "layer": _lib.LAPNYS_LAYER}


def _chosen(table, name, what):
    try:
        return table[name]
    except (KeyError, TypeError):
        raise ValueError(f"unknown {what} {name!r}: one of {', '.join(map(repr, table))}") from None


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
class RotaryFrequencies(NamedTuple):
    """turns: int64 [pairs], turns a position in units of 2^-64; factor: of the turned features."""
    turns: torch.Tensor
    factor: float

    @staticmethod
    def of(radians, factor: float = 1.0, device="cuda") -> "RotaryFrequencies":
        """From angles a position, one for each pair (numbers or a tensor)."""
        if isinstance(radians, torch.Tensor):
            radians = radians.double().cpu().tolist()
        turns = []
        for w in radians:
            w = float(w)
            if not math.isfinite(w):
                raise ValueError(f"angles must be finite: {w}")
            n = round(math.ldexp(math.fmod(w / (2.0 * math.pi), 1.0), 64)) % 2 ** 64
            turns.append(n - 2 ** 64 if n >= 2 ** 63 else n)
        if not turns:
            raise ValueError("no pairs")
        return RotaryFrequencies(torch.tensor(turns, dtype=torch.int64, device=device), float(factor))


def rotary_frequencies(rot, base=10000.0, scaling=None, factor=1.0, context=None, low=1.0, high=32.0,
                       device="cuda") -> RotaryFrequencies:
    """The angles base^(-2 i / rot) of rot / 2 pairs, as they are or scaled for contexts `factor` times
    longer than those trained on:
      "linear"  all angles divided by factor;
      "base"    base raised to base * factor^(rot / (rot - 2)): the slowest pair slows down by factor, the
                fastest stays;
      "parts"   a pair that makes `high` turns or more over `context` positions (the length trained on)
                stays, one of `low` turns or fewer is divided by factor, others in between linearly;
                turned features are multiplied by 1 + 0.1 ln(factor).
    """
    rot = int(rot)
    if rot < 2 or rot % 2:
        raise ValueError(f"rot must be even and at least 2: {rot}")
    base, f = float(base), float(factor)
    if not (base > 0 and math.isfinite(base) and f > 0 and math.isfinite(f)):
        raise ValueError("base and factor must be positive")
    if scaling not in (None, "linear", "base", "parts"):
        raise ValueError(f"unknown scaling {scaling!r}: None, 'linear', 'base' or 'parts'")
    if scaling == "base" and rot > 2:
        base *= f ** (rot / (rot - 2.0))
    w = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    grow = 1.0
    if scaling == "linear":
        w = [x / f for x in w]
    elif scaling == "parts":
        if context is None or not context > 0 or not high > low:
            raise ValueError("'parts' takes the context trained on, and high > low")
        for i, x in enumerate(w):
            turns = context * x / (2.0 * math.pi)
            keep = min(1.0, max(0.0, (turns - low) / (high - low)))
            w[i] = x * (keep + (1.0 - keep) / f)
        grow = 1.0 + 0.1 * math.log(f) if f > 1.0 else 1.0
    return RotaryFrequencies.of(w, grow, device)


def rotary_apply(q, k, freqs: RotaryFrequencies, start=None, positions=None, layout="half", inverse=False,
                 q_out=None, k_out=None):
    """lapnys_rotary: returns (q, k) turned; q_out, k_out may be q and k themselves.  No derivatives."""
    if q.dim() != 4 or (k is not None and k.dim() != 4):
        raise ValueError("q and k must be [B, H, N, d] tensors")
    B, Hq, N, d = q.shape
    dev, dt = q.device, _dtype(q)
    lay = _chosen(_LAYOUT, layout, "layout")
    Hkv = 0 if k is None else k.shape[1]
    _tensor(q, "q", q.shape, q.dtype, dev)
    if k is not None:
        _tensor(k, "k", (B, Hkv, N, d), q.dtype, dev)
    if not isinstance(freqs, RotaryFrequencies) or freqs.turns.dim() != 1:
        raise ValueError("freqs must be RotaryFrequencies (rotary_frequencies makes them)")
    _tensor(freqs.turns, "freqs.turns", freqs.turns.shape, torch.int64, dev)
    if start is not None and positions is not None:
        raise ValueError("start or positions, not both")
    if start is not None:
        _tensor(start, "start", (B,), torch.int32, dev)
    if positions is not None:
        _tensor(positions, "positions", (B, N), torch.int32, dev)
    if q_out is not None:
        _tensor(q_out, "q_out", q.shape, q.dtype, dev)
    if k_out is not None:
        if k is None:
            raise ValueError("k_out without k")
        _tensor(k_out, "k_out", k.shape, q.dtype, dev)
    with _on(dev):
        q_out = torch.empty_like(q) if q_out is None else q_out
        if k is not None and k_out is None:
            k_out = torch.empty_like(k)
        rc = load().lapnys_rotary(
            q.data_ptr(), _at(k), q_out.data_ptr(), _at(k_out), freqs.turns.data_ptr(), _at(start),
            _at(positions), *_sizes(B, Hq, Hkv, N, d, 2 * freqs.turns.shape[0]), lay, freqs.factor,
            int(inverse), _on_stream(dev), dt)
    check(rc, "lapnys_rotary")
    return q_out, k_out


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(fctx, q, k, turns, start, positions, factor, layout):
        fctx.save_for_backward(turns, start, positions)
        fctx.how = factor, layout
        fctx.set_materialize_grads(False)
        return rotary_apply(q, k, RotaryFrequencies(turns, factor), start, positions, layout)

    @staticmethod
    @once_differentiable
    def backward(fctx, dq, dk):
        _no_tangent("rotary's backward", dq, dk)
        turns, start, positions = fctx.saved_tensors
        factor, layout = fctx.how
        freqs = RotaryFrequencies(turns, factor)
        grads = [None if g is None else g.contiguous() for g in (dq, dk)]
        if grads[0] is not None:
            grads = rotary_apply(*grads, freqs, start, positions, layout, True)
        elif grads[1] is not None:      # one tensor is enough to the call
            grads[1] = rotary_apply(grads[1], None, freqs, start, positions, layout, True)[0]
        return *grads, None, None, None, None, None


def rotary(q, k, freqs: RotaryFrequencies, start=None, positions=None, layout="half"):
    """Queries and keys turned by their positions, with autograd: returns (q, k).

    q: [B, Hq, N, d], k: [B, Hkv, N, d] CUDA tensors (float32 or bfloat16), or k None.  freqs (from
    rotary_frequencies) turns the first 2 * pairs features of a head, the others pass.  Token n of
    sequence b stands at start[b] + n (start: int32 [B], default 0) or at positions[b, n] (int32 [B, N]).
    layout: "half" pairs features (i, i + pairs), "interleaved" (2 i, 2 i + 1).  Gradients are of first
    order, by reverse mode only.  rotary_apply does the same in place.
    """
    _no_tangent("rotary", q, k)
    if not isinstance(freqs, RotaryFrequencies):
        raise ValueError("freqs must be RotaryFrequencies (rotary_frequencies makes them)")
    if torch.is_grad_enabled() and (q.requires_grad or (k is not None and k.requires_grad)):
        return _Rotary.apply(q, k, freqs.turns, start, positions, freqs.factor, layout)
    return rotary_apply(q, k, freqs, start, positions, layout)


# ---------------------------------------------------------------------------
# the residual of a block with the norms around it
# ---------------------------------------------------------------------------
class NormParams(NamedTuple):
    """Shape and norms of one call: x [B, N, C]; per_seq: weight and bias are [B, C]."""
    B: int
    N: int
    C: int
    per_seq: bool
    pre: Optional[str]
    post: Optional[str]
    eps: float

    def dims(self):
        return (*_sizes(self.B, self.N, self.C), int(self.per_seq), _chosen(_NORM, self.pre, "norm"),
                _chosen(_NORM, self.post, "norm"))


def _vector(t, name, shape, x):
    if t is not None:
        _tensor(t, name, shape, x.dtype, x.device)


def _check_norm(x, u, weight, bias, post_weight, post_bias, gate, scale, p: NormParams):
    _dtype(x)
    _tensor(x, "x", (p.B, p.N, p.C), x.dtype, x.device)
    _vector(u, "u", x.shape, x)
    wide = (p.B, p.C) if p.per_seq else (p.C,)
    _vector(weight, "weight", wide, x)
    _vector(bias, "bias", wide, x)
    for t, name in ((post_weight, "post_weight"), (post_bias, "post_bias"), (scale, "scale")):
        _vector(t, name, (p.C,), x)
    _vector(gate, "gate", (p.B, p.C), x)


@functools.lru_cache(maxsize=256)
def norm_workspace_bytes(B, N, C, seqs) -> int:
    """seqs: with a gate or per_seq."""
    return load().lapnys_norm_workspace_bytes(*_sizes(B, N, C), int(seqs))


def norm_fwd(x, u, weight, bias, p: NormParams, post_weight=None, post_bias=None, gate=None, scale=None,
             h=None, y=None, stats=None, need_stats=True):
    """lapnys_norm_fwd: returns (h, y, stats); h is None without u, y without a norm of h, stats when
    need_stats is False."""
    _check_norm(x, u, weight, bias, post_weight, post_bias, gate, scale, p)
    dims, dev = p.dims(), x.device
    if u is None and h is not None:
        raise ValueError("h without u")
    if p.pre is None and y is not None:
        raise ValueError("y without a norm")
    _vector(h, "h", x.shape, x)
    _vector(y, "y", x.shape, x)
    if stats is not None:
        _tensor(stats, "stats", (p.B, p.N, 4), torch.float32, dev)
    with _on(dev):
        h = torch.empty_like(x) if h is None and u is not None else h
        y = torch.empty_like(x) if y is None and p.pre is not None else y
        if not need_stats:
            stats = None
        elif stats is None:
            stats = torch.empty((p.B, p.N, 4), dtype=torch.float32, device=dev)
        rc = load().lapnys_norm_fwd(
            x.data_ptr(), _at(u), _at(weight), _at(bias), _at(post_weight), _at(post_bias), _at(gate),
            _at(scale), _at(h), _at(y), _at(stats), *dims, p.eps, _on_stream(dev), _dtype(x))
    check(rc, "lapnys_norm_fwd")
    return h, y, stats


def norm_bwd(x, u, weight, stats, dh, dy, p: NormParams, post_weight=None, post_bias=None, gate=None,
             scale=None, want=(True,) * 8, ws=None):
    """lapnys_norm_bwd: the gradients of (x, u, weight, bias, post_weight, post_bias, gate, scale), those
    wanted; dh, dy: the outputs', or None."""
    _check_norm(x, u, weight, None, post_weight, post_bias, gate, scale, p)
    dims, dev = p.dims(), x.device
    _tensor(stats, "stats", (p.B, p.N, 4), torch.float32, dev)
    _vector(dh, "dh", x.shape, x)
    _vector(dy, "dy", x.shape, x)
    wide = (p.B, p.C) if p.per_seq else (p.C,)
    shapes = (x.shape, x.shape, wide, wide, (p.C,), (p.C,), (p.B, p.C), (p.C,))
    with _on(dev):
        grads = [torch.empty(s, dtype=x.dtype, device=dev) if w else None for s, w in zip(shapes, want)]
        if any(want[2:]):
            ws = _workspace(ws, norm_workspace_bytes(p.B, p.N, p.C, p.per_seq or gate is not None), dev)
        rc = load().lapnys_norm_bwd(
            x.data_ptr(), _at(u), _at(weight), _at(post_weight), _at(post_bias), _at(gate), _at(scale),
            stats.data_ptr(), _at(dh), _at(dy), *(_at(g) for g in grads), *dims, _on_stream(dev),
            _dtype(x), _at(ws), _nbytes(ws))
    check(rc, "lapnys_norm_bwd")
    return grads


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(fctx, x, u, weight, bias, post_weight, post_bias, gate, scale, p: NormParams):
        h, y, stats = norm_fwd(x, u, weight, bias, p, post_weight, post_bias, gate, scale)
        fctx.p = p
        fctx.set_materialize_grads(False)
        fctx.save_for_backward(x, u, weight, stats, post_weight, post_bias, gate, scale)
        return h, y

    @staticmethod
    @once_differentiable
    def backward(fctx, dh, dy):
        _no_tangent("residual_norm's backward", dh, dy)
        x, u, weight, stats, post_weight, post_bias, gate, scale = fctx.saved_tensors
        if dh is None and dy is None:
            return (None,) * 9
        dh, dy = (None if g is None else g.contiguous() for g in (dh, dy))
        want = list(fctx.needs_input_grad[:8])
        if dy is None:
            want[2] = want[3] = False
        return *norm_bwd(x, u, weight, stats, dh, dy, fctx.p, post_weight, post_bias, gate, scale,
                         want), None


def residual_norm(x, u=None, weight=None, bias=None, post_weight=None, post_bias=None, gate=None, scale=None,
                  pre="rms", post=None, eps=1e-6):
    """A block's output u taken into the residual x, and the next block's input, with autograd:
    h = x + gate scale post(u), y = pre(h); returns (h, y).

    x, u: [B, N, C] CUDA tensors (float32 or bfloat16), u None: h is x itself.  pre, post: "rms",
    "layer" (centred) or None (post: u as it is; pre: no y), with weight, bias: [C], or [B, C] for each
    sequence its own; post_weight, post_bias, scale: [C]; gate: [B, C]; each optional, all of x's type.
    C is at most 16384.  Gradients are of first order, by reverse mode only.
    """
    tensors = (x, u, weight, bias, post_weight, post_bias, gate, scale)
    _no_tangent("residual_norm", *tensors)
    if x.dim() != 3:
        raise ValueError("x must be [B, N, C]")
    if u is None and pre is None:
        raise ValueError("neither u nor a norm: nothing to do")
    per_seq = any(t is not None and t.dim() == 2 for t in (weight, bias))
    p = NormParams(*x.shape, per_seq, pre, post, float(eps))
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        h, y = _ResidualNorm.apply(*tensors, p)
    else:
        h, y, _ = norm_fwd(x, u, weight, bias, p, post_weight, post_bias, gate, scale, need_stats=False)
    return x if u is None else h, y


# ---------------------------------------------------------------------------
# the gated feed-forward block
# ---------------------------------------------------------------------------
class MlpParams(NamedTuple):
    """Shape of one call: T rows of C features, F hidden."""
    T: int
    C: int
    F: int
    act: str = "silu"

    def sizes(self):
        return _sizes(self.T, self.C, self.F)


@functools.lru_cache(maxsize=256)
def mlp_ctx_bytes(p: MlpParams, dtype: torch.dtype) -> int:
    return load().lapnys_mlp_ctx_bytes(*p.sizes(), _DT[dtype])


@functools.lru_cache(maxsize=256)
def mlp_workspace_bytes(p: MlpParams, dtype: torch.dtype, backward: bool = False) -> int:
    return load().lapnys_mlp_workspace_bytes(*p.sizes(), _DT[dtype], int(backward))


def _check_mlp(x, w_in, b_in, w_out, b_out, p: MlpParams):
    _dtype(x)
    dev, dt = x.device, x.dtype
    if not isinstance(x, torch.Tensor) or x.dim() < 2 or x.shape[-1] != p.C or x.numel() != p.T * p.C:
        raise ValueError(f"x must be a tensor of {p.T} rows of {p.C}")
    _tensor(x, "x", x.shape, dt, dev)
    _tensor(w_in, "w_in", (p.C, 2 * p.F), dt, dev)
    _tensor(w_out, "w_out", (p.F, p.C), dt, dev)
    _vector(b_in, "b_in", (2 * p.F,), x)
    _vector(b_out, "b_out", (p.C,), x)


def mlp_fwd(x, w_in, b_in, w_out, b_out, p: MlpParams, y=None, ctx=None, ws=None, need_ctx=True):
    """lapnys_mlp_fwd: returns (y, ctx); ctx is None when need_ctx is False."""
    _check_mlp(x, w_in, b_in, w_out, b_out, p)
    act, dev = _chosen(_ACT, p.act, "activation"), x.device
    _vector(y, "y", x.shape, x)
    with _on(dev):
        y = torch.empty_like(x) if y is None else y
        ctx = _workspace(ctx, mlp_ctx_bytes(p, x.dtype), dev) if need_ctx else None
        ws = _workspace(ws, mlp_workspace_bytes(p, x.dtype), dev)
        rc = load().lapnys_mlp_fwd(
            x.data_ptr(), w_in.data_ptr(), _at(b_in), w_out.data_ptr(), _at(b_out), y.data_ptr(),
            *p.sizes(), act, _on_stream(dev), _dtype(x), _at(ctx), _nbytes(ctx), _at(ws), _nbytes(ws))
    check(rc, "lapnys_mlp_fwd")
    return y, ctx


def mlp_bwd(x, w_in, w_out, dy, ctx, p: MlpParams, want=(True,) * 5, ws=None):
    """lapnys_mlp_bwd: the gradients of (x, w_in, b_in, w_out, b_out), those wanted."""
    _check_mlp(x, w_in, None, w_out, None, p)
    dev = x.device
    _tensor(dy, "dy", x.shape, x.dtype, dev)
    need = mlp_ctx_bytes(p, x.dtype)
    if ctx is None or not ctx.is_cuda or ctx.device != dev or not ctx.is_contiguous() or ctx.nbytes < need:
        raise ValueError(f"ctx must be the forward's, {need} bytes on {dev}")
    shapes = (x.shape, w_in.shape, (2 * p.F,), w_out.shape, (p.C,))
    with _on(dev):
        grads = [torch.empty(s, dtype=x.dtype, device=dev) if w else None for s, w in zip(shapes, want)]
        ws = _workspace(ws, mlp_workspace_bytes(p, x.dtype, True), dev)
        rc = load().lapnys_mlp_bwd(
            x.data_ptr(), w_in.data_ptr(), w_out.data_ptr(), dy.data_ptr(), ctx.data_ptr(),
            *(_at(g) for g in grads), *p.sizes(), _on_stream(dev), _dtype(x), _at(ws), _nbytes(ws))
    check(rc, "lapnys_mlp_bwd")
    return grads


class _Mlp(torch.autograd.Function):
    @staticmethod
    def forward(fctx, x, w_in, b_in, w_out, b_out, p: MlpParams):
        y, ctx = mlp_fwd(x, w_in, b_in, w_out, b_out, p)
        fctx.p = p
        fctx.save_for_backward(x, w_in, w_out, ctx)
        return y

    @staticmethod
    @once_differentiable
    def backward(fctx, dy):
        _no_tangent("gated_mlp's backward", dy)
        x, w_in, w_out, ctx = fctx.saved_tensors
        return *mlp_bwd(x, w_in, w_out, dy.contiguous(), ctx, fctx.p, fctx.needs_input_grad[:5]), None


def gated_mlp(x, w_in, b_in, w_out, b_out, act="silu"):
    """The gated feed-forward block, with autograd: (g | u) = x w_in + b_in,
    y = (act(g) * u) w_out + b_out.

    x: CUDA tensor (float32 or bfloat16) of rows of C features, [.., C]; w_in: [C, 2 F], the gate's
    columns, then the others; w_out: [F, C]; biases [2 F] and [C] or None; act: "silu", "gelu" or
    "gelu_tanh".  Gradients are of first order, by reverse mode only.
    """
    tensors = (x, w_in, b_in, w_out, b_out)
    _no_tangent("gated_mlp", *tensors)
    if x.dim() < 2 or w_out.dim() != 2:
        raise ValueError("x must be [.., C] and w_out [F, C]")
    p = MlpParams(x.numel() // max(1, x.shape[-1]), x.shape[-1], w_out.shape[0], act)
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        return _Mlp.apply(*tensors, p)
    return mlp_fwd(*tensors, p, need_ctx=False)[0]
