"""What stands around the attentions in a layer: rotary positions, the residual with its norms, and the
gated feed-forward block.  Marshalling only: every step runs in liblapnys kernels.

A step that is captured into a CUDA graph takes leaves that no eager autograd graph still holds, as
window_attention's does (their gradients would be added up on that graph's stream).
"""
from __future__ import annotations

import functools
import math
from decimal import Context, Decimal, localcontext
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


def _any_requires_grad(tensors):
    for t in tensors:
        if t is not None and t.requires_grad:
            return True
    return False


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
# far positions multiply what an angle is off by, and doubles (2^-53 of it) would be a quarter of a
# feature's 24 bits off at 2^31: angles are computed to 60 digits and rounded once, to 2^-64 of a turn
_DIGITS = Context(prec=60)
_TURN = Decimal("6.28318530717958647692528676655900576839433879875021164194988918461563281257")


class RotaryFrequencies(NamedTuple):
    """turns: int64 [pairs], turns a position in units of 2^-64; factor: of the turned features."""
    turns: torch.Tensor
    factor: float

    @staticmethod
    def of(radians, factor: float = 1.0, device="cuda") -> "RotaryFrequencies":
        """From angles a position, one for each pair (numbers, Decimal ones as they are, or a tensor)."""
        if isinstance(radians, torch.Tensor):
            radians = radians.double().cpu().tolist()
        turns = []
        with localcontext(_DIGITS):
            for w in radians:
                w = w if isinstance(w, Decimal) else Decimal(float(w))
                if not w.is_finite():
                    raise ValueError(f"angles must be finite: {w}")
                w /= _TURN
                n = int(((w - w.to_integral_value()) * 2 ** 64).to_integral_value()) % 2 ** 64
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
                turned features are multiplied by 1 + 0.1 ln(factor) (factors above 1).
    Other rules (by a pair's index, or without a factor of the features): RotaryFrequencies.of, which
    takes any angles and any factor.
    """
    rot = int(rot)
    if rot < 2 or rot % 2:
        raise ValueError(f"rot must be even and at least 2: {rot}")
    base, f = float(base), float(factor)
    if not (base > 0 and math.isfinite(base) and f > 0 and math.isfinite(f)):
        raise ValueError("base and factor must be positive")
    if scaling not in (None, "linear", "base", "parts"):
        raise ValueError(f"unknown scaling {scaling!r}: None, 'linear', 'base' or 'parts'")
    if scaling == "parts" and (context is None or not context > 0 or not high > low):
        raise ValueError("'parts' takes the context trained on, and high > low")
    with localcontext(_DIGITS):
        grow, by = 1.0, Decimal(f)
        log = Decimal(base).ln()
        if scaling == "base" and rot > 2:
            log += by.ln() * rot / (rot - 2)
        step, w = (log * -2 / rot).exp(), [Decimal(1)]
        for _ in range(rot // 2 - 1):
            w.append(w[-1] * step)
        if scaling == "linear":
            w = [x / by for x in w]
        elif scaling == "parts":
            low, high, context = (Decimal(float(x)) for x in (low, high, context))
            for i, x in enumerate(w):
                turns = context * x / _TURN
                keep = min(Decimal(1), max(Decimal(0), (turns - low) / (high - low)))
                w[i] = x * (keep + (1 - keep) / by)
            grow = 1.0 + 0.1 * math.log(f) if f > 1.0 else 1.0
    return RotaryFrequencies.of(w, grow, device)


@functools.lru_cache(maxsize=256)
def _rotary_plan(q_shape, k_shape, pairs, layout, dtype):
    """What the C call takes of one kind of call, checked once: sizes, layout, element type."""
    if len(q_shape) != 4 or (k_shape is not None and len(k_shape) != 4):
        raise ValueError("q and k must be [B, H, N, d] tensors")
    B, Hq, N, d = q_shape
    Hkv = 0 if k_shape is None else k_shape[1]
    if k_shape is not None and k_shape != (B, Hkv, N, d):
        raise ValueError(f"k must be {(B, Hkv, N, d)}: {tuple(k_shape)}")
    return (*_sizes(B, Hq, Hkv, N, d, 2 * pairs), _chosen(_LAYOUT, layout, "layout")), _DT[dtype]


def _check_rotary(q, k, freqs, start, positions, layout):
    _dtype(q)
    dev, dt, shape = q.device, q.dtype, q.shape
    if not isinstance(freqs, RotaryFrequencies) or freqs.turns.dim() != 1:
        raise ValueError("freqs must be RotaryFrequencies (rotary_frequencies makes them)")
    turns = freqs.turns
    plan = _rotary_plan(shape, None if k is None else k.shape, turns.shape[0], layout, dt)
    _tensor(q, "q", shape, dt, dev)
    if k is not None:
        _tensor(k, "k", k.shape, dt, dev)
    _tensor(turns, "freqs.turns", turns.shape, torch.int64, dev)
    if start is not None:
        if positions is not None:
            raise ValueError("start or positions, not both")
        _tensor(start, "start", shape[:1], torch.int32, dev)
    elif positions is not None:
        _tensor(positions, "positions", (shape[0], shape[2]), torch.int32, dev)
    return plan


def _rotary(q, k, turns, start, positions, plan, factor, inverse, q_out=None, k_out=None):
    dev = q.device
    with _on(dev):
        if q_out is None:
            q_out = torch.empty_like(q)
        if k is not None and k_out is None:
            k_out = torch.empty_like(k)
        check(load().lapnys_rotary(
            q.data_ptr(), _at(k), q_out.data_ptr(), _at(k_out), turns.data_ptr(), _at(start),
            _at(positions), *plan[0], factor, inverse, _on_stream(dev), plan[1]), "lapnys_rotary")
    return q_out, k_out


def rotary_apply(q, k, freqs: RotaryFrequencies, start=None, positions=None, layout="half", inverse=False,
                 q_out=None, k_out=None):
    """lapnys_rotary: returns (q, k) turned; q_out, k_out may be q and k themselves.  No derivatives."""
    plan = _check_rotary(q, k, freqs, start, positions, layout)
    if q_out is not None:
        _tensor(q_out, "q_out", q.shape, q.dtype, q.device)
    if k_out is not None:
        if k is None:
            raise ValueError("k_out without k")
        _tensor(k_out, "k_out", k.shape, q.dtype, q.device)
    return _rotary(q, k, freqs.turns, start, positions, plan, freqs.factor, int(inverse), q_out, k_out)


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(fctx, q, k, freqs, start, positions, layout):
        plan = _check_rotary(q, k, freqs, start, positions, layout)
        fctx.save_for_backward(freqs.turns, start, positions)
        fctx.how = plan, freqs.factor
        fctx.set_materialize_grads(False)
        return _rotary(q, k, freqs.turns, start, positions, plan, freqs.factor, 0)

    @staticmethod
    @once_differentiable
    def backward(fctx, dq, dk):
        _no_tangent("rotary's backward", dq, dk)
        turns, start, positions = fctx.saved_tensors
        plan, factor = fctx.how
        dq, dk = (g.contiguous() if g is not None and need else None
                  for g, need in zip((dq, dk), fctx.needs_input_grad))
        if dq is None:                  # the call takes one tensor or two
            if dk is not None:
                B, _, Hkv, *rest = plan[0]
                plan = (B, Hkv, 0, *rest), plan[1]
                dk = _rotary(dk, None, turns, start, positions, plan, factor, 1)[0]
        else:
            if dk is None:
                B, Hq, _, *rest = plan[0]
                plan = (B, Hq, 0, *rest), plan[1]
            dq, dk = _rotary(dq, dk, turns, start, positions, plan, factor, 1)
        return dq, dk, None, None, None, None


def rotary(q, k, freqs: RotaryFrequencies, start=None, positions=None, layout="half"):
    """Queries and keys turned by their positions, with autograd: returns (q, k).

    q: [B, Hq, N, d], k: [B, Hkv, N, d] CUDA tensors (float32 or bfloat16), or k None.  freqs (from
    rotary_frequencies) turns the first 2 * pairs features of a head, the others pass.  Token n of
    sequence b stands at start[b] + n (start: int32 [B], default 0) or at positions[b, n] (int32 [B, N]).
    layout: "half" pairs features (i, i + pairs), "interleaved" (2 i, 2 i + 1).  Gradients are of first
    order, by reverse mode only.  rotary_apply does the same in place.
    """
    _no_tangent("rotary", q, k)
    if torch.is_grad_enabled() and (q.requires_grad or (k is not None and k.requires_grad)):
        return _Rotary.apply(q, k, freqs, start, positions, layout)
    plan = _check_rotary(q, k, freqs, start, positions, layout)
    return _rotary(q, k, freqs.turns, start, positions, plan, freqs.factor, 0)


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


@functools.lru_cache(maxsize=256)
def _norm_dims(p: NormParams):
    return p.dims()


def _check_norm(x, u, weight, bias, post_weight, post_bias, gate, scale, p: NormParams):
    _dtype(x)
    C = (p.C,)
    _tensor(x, "x", p[:3], x.dtype, x.device)
    wide = (p.B, p.C) if p.per_seq else C
    for t, name, shape in ((u, "u", p[:3]), (weight, "weight", wide), (bias, "bias", wide),
                           (post_weight, "post_weight", C), (post_bias, "post_bias", C),
                           (gate, "gate", (p.B, p.C)), (scale, "scale", C)):
        if t is not None:
            _tensor(t, name, shape, x.dtype, x.device)


@functools.lru_cache(maxsize=256)
def norm_workspace_bytes(B, N, C, seqs) -> int:
    """seqs: with a gate or per_seq."""
    return load().lapnys_norm_workspace_bytes(*_sizes(B, N, C), int(seqs))


def _norm_fwd(x, u, weight, bias, post_weight, post_bias, gate, scale, p, h, y, stats, need_stats):
    dev = x.device
    with _on(dev):
        if h is None and u is not None:
            h = torch.empty_like(x)
        if y is None and p.pre is not None:
            y = torch.empty_like(x)
        if not need_stats:
            stats = None
        elif stats is None:
            stats = torch.empty((p.B, p.N, 4), dtype=torch.float32, device=dev)
        check(load().lapnys_norm_fwd(
            x.data_ptr(), _at(u), _at(weight), _at(bias), _at(post_weight), _at(post_bias), _at(gate),
            _at(scale), _at(h), _at(y), _at(stats), *_norm_dims(p), p.eps, _on_stream(dev),
            _DT[x.dtype]), "lapnys_norm_fwd")
    return h, y, stats


def norm_fwd(x, u, weight, bias, p: NormParams, post_weight=None, post_bias=None, gate=None, scale=None,
             h=None, y=None, stats=None, need_stats=True):
    """lapnys_norm_fwd: returns (h, y, stats); h is None without u, y without a norm of h, stats when
    need_stats is False."""
    _check_norm(x, u, weight, bias, post_weight, post_bias, gate, scale, p)
    if u is None and h is not None:
        raise ValueError("h without u")
    if p.pre is None and y is not None:
        raise ValueError("y without a norm")
    _vector(h, "h", x.shape, x)
    _vector(y, "y", x.shape, x)
    if stats is not None:
        _tensor(stats, "stats", (p.B, p.N, 4), torch.float32, x.device)
    return _norm_fwd(x, u, weight, bias, post_weight, post_bias, gate, scale, p, h, y, stats, need_stats)


def _norm_bwd(x, u, weight, stats, dh, dy, p, post_weight, post_bias, gate, scale, want, ws):
    dev = x.device
    C = (p.C,)
    wide = (p.B, p.C) if p.per_seq else C
    shapes = (None, None, wide, wide, C, C, (p.B, p.C), C)
    with _on(dev):
        grads = [(torch.empty_like(x) if s is None else torch.empty(s, dtype=x.dtype, device=dev)) if w else None
                 for s, w in zip(shapes, want)]
        if ws is None and any(want[2:]):
            ws = torch.empty(norm_workspace_bytes(p.B, p.N, p.C, p.per_seq or gate is not None),
                             dtype=torch.uint8, device=dev)
        check(load().lapnys_norm_bwd(
            x.data_ptr(), _at(u), _at(weight), _at(post_weight), _at(post_bias), _at(gate), _at(scale),
            stats.data_ptr(), _at(dh), _at(dy), *map(_at, grads), *_norm_dims(p), _on_stream(dev),
            _DT[x.dtype], _at(ws), _nbytes(ws)), "lapnys_norm_bwd")
    return grads


def norm_bwd(x, u, weight, stats, dh, dy, p: NormParams, post_weight=None, post_bias=None, gate=None,
             scale=None, want=None, ws=None):
    """lapnys_norm_bwd: the gradients of (x, u, weight, bias, post_weight, post_bias, gate, scale), those
    wanted (None: of all that there are, and of a bias where there is a norm); dh, dy: the outputs', or None."""
    if want is None:
        there = (u, weight, post_weight, post_bias, gate, scale)
        has_u, has_w, *others = (t is not None for t in there)
        want = (True, has_u, has_w, p.pre is not None, *others)
    _check_norm(x, u, weight, None, post_weight, post_bias, gate, scale, p)
    _tensor(stats, "stats", (p.B, p.N, 4), torch.float32, x.device)
    _vector(dh, "dh", x.shape, x)
    _vector(dy, "dy", x.shape, x)
    if ws is not None:
        _workspace(ws, 0, x.device)
    return _norm_bwd(x, u, weight, stats, dh, dy, p, post_weight, post_bias, gate, scale, want, ws)


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(fctx, x, u, weight, bias, post_weight, post_bias, gate, scale, p: NormParams):
        h, y, stats = _norm_fwd(x, u, weight, bias, post_weight, post_bias, gate, scale, p, None, None, None,
                                True)
        fctx.p = p
        fctx.set_materialize_grads(False)
        fctx.save_for_backward(x, u, weight, stats, post_weight, post_bias, gate, scale)
        return h, y

    @staticmethod
    @once_differentiable
    def backward(fctx, dh, dy):
        _no_tangent("residual_norm's backward", dh, dy)
        x, u, weight, stats, *others = fctx.saved_tensors
        if dh is None and dy is None:
            return (None,) * 9
        dh, dy = (None if g is None else g.contiguous() for g in (dh, dy))
        want = list(fctx.needs_input_grad[:8])
        if dy is None:
            want[2] = want[3] = False
        return *_norm_bwd(x, u, weight, stats, dh, dy, fctx.p, *others, want, None), None


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
    per_seq = (weight is not None and weight.dim() == 2) or (bias is not None and bias.dim() == 2)
    p = NormParams(*x.shape, per_seq, pre, post, float(eps))
    _norm_dims(p)
    _check_norm(*tensors, p)
    if torch.is_grad_enabled() and _any_requires_grad(tensors):
        h, y = _ResidualNorm.apply(*tensors, p)
    else:
        h, y, _ = _norm_fwd(*tensors, p, None, None, None, False)
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


@functools.lru_cache(maxsize=256)
def _mlp_plan(shape, F, act):
    """(parameters, sizes and activation as the C call takes them) of x's shape."""
    if len(shape) < 2:
        raise ValueError("x must be [.., C]")
    C = shape[-1]
    T = math.prod(shape[:-1])
    p = MlpParams(T, C, F, act)
    return p, p.sizes(), _chosen(_ACT, act, "activation")


def _check_mlp(x, w_in, b_in, w_out, b_out, p: MlpParams):
    _dtype(x)
    dev, dt, C, F = x.device, x.dtype, p.C, p.F
    if x.dim() < 2 or x.shape[-1] != C or x.numel() != p.T * C:
        raise ValueError(f"x must be a tensor of {p.T} rows of {C}")
    _tensor(x, "x", x.shape, dt, dev)
    _tensor(w_in, "w_in", (C, 2 * F), dt, dev)
    _tensor(w_out, "w_out", (F, C), dt, dev)
    if b_in is not None:
        _tensor(b_in, "b_in", (2 * F,), dt, dev)
    if b_out is not None:
        _tensor(b_out, "b_out", (C,), dt, dev)


def _mlp_fwd(x, w_in, b_in, w_out, b_out, plan, y, ctx, ws, need_ctx):
    p, sizes, act = plan
    dev, dt = x.device, x.dtype
    with _on(dev):
        if y is None:
            y = torch.empty_like(x)
        if not need_ctx:
            ctx = None
        elif ctx is None:
            ctx = torch.empty(mlp_ctx_bytes(p, dt), dtype=torch.uint8, device=dev)
        if ws is None:
            ws = torch.empty(mlp_workspace_bytes(p, dt), dtype=torch.uint8, device=dev)
        check(load().lapnys_mlp_fwd(
            x.data_ptr(), w_in.data_ptr(), _at(b_in), w_out.data_ptr(), _at(b_out), y.data_ptr(), *sizes,
            act, _on_stream(dev), _DT[dt], _at(ctx), _nbytes(ctx), ws.data_ptr(), ws.nbytes),
            "lapnys_mlp_fwd")
    return y, ctx


def mlp_fwd(x, w_in, b_in, w_out, b_out, p: MlpParams, y=None, ctx=None, ws=None, need_ctx=True):
    """lapnys_mlp_fwd: returns (y, ctx); ctx is None when need_ctx is False."""
    _check_mlp(x, w_in, b_in, w_out, b_out, p)
    _vector(y, "y", x.shape, x)
    for t in (ctx, ws):
        if t is not None:
            _workspace(t, 0, x.device)
    return _mlp_fwd(x, w_in, b_in, w_out, b_out, (p, p.sizes(), _chosen(_ACT, p.act, "activation")), y, ctx,
                    ws, need_ctx)


def _mlp_bwd(x, w_in, w_out, dy, ctx, plan, want, ws):
    p, sizes, _ = plan
    dev, dt = x.device, x.dtype
    like = (x, w_in, (2 * p.F,), w_out, (p.C,))
    with _on(dev):
        grads = [(torch.empty(t, dtype=dt, device=dev) if isinstance(t, tuple) else torch.empty_like(t)) if w
                 else None for t, w in zip(like, want)]
        if ws is None:
            ws = torch.empty(mlp_workspace_bytes(p, dt, True), dtype=torch.uint8, device=dev)
        check(load().lapnys_mlp_bwd(
            x.data_ptr(), w_in.data_ptr(), w_out.data_ptr(), dy.data_ptr(), ctx.data_ptr(),
            *map(_at, grads), *sizes, _on_stream(dev), _DT[dt], ws.data_ptr(), ws.nbytes), "lapnys_mlp_bwd")
    return grads


def mlp_bwd(x, w_in, w_out, dy, ctx, p: MlpParams, want=(True,) * 5, ws=None):
    """lapnys_mlp_bwd: the gradients of (x, w_in, b_in, w_out, b_out), those wanted."""
    _check_mlp(x, w_in, None, w_out, None, p)
    dev = x.device
    _tensor(dy, "dy", x.shape, x.dtype, dev)
    need = mlp_ctx_bytes(p, x.dtype)
    if ctx is None or not ctx.is_cuda or ctx.device != dev or not ctx.is_contiguous() or ctx.nbytes < need:
        raise ValueError(f"ctx must be the forward's, {need} bytes on {dev}")
    if ws is not None:
        _workspace(ws, 0, dev)
    return _mlp_bwd(x, w_in, w_out, dy, ctx, (p, p.sizes(), None), want, ws)


class _Mlp(torch.autograd.Function):
    @staticmethod
    def forward(fctx, x, w_in, b_in, w_out, b_out, plan):
        y, ctx = _mlp_fwd(x, w_in, b_in, w_out, b_out, plan, None, None, None, True)
        fctx.plan = plan
        fctx.save_for_backward(x, w_in, w_out, ctx)
        return y

    @staticmethod
    @once_differentiable
    def backward(fctx, dy):
        _no_tangent("gated_mlp's backward", dy)
        x, w_in, w_out, ctx = fctx.saved_tensors
        dy = dy.contiguous()
        if dy.data_ptr() % 16:      # a piece of another tensor, as a concatenation's gradient is
            dy = dy.clone()
        return *_mlp_bwd(x, w_in, w_out, dy, ctx, fctx.plan, fctx.needs_input_grad, None), None


def gated_mlp(x, w_in, b_in, w_out, b_out, act="silu"):
    """The gated feed-forward block, with autograd: (g | u) = x w_in + b_in,
    y = (act(g) * u) w_out + b_out.

    x: CUDA tensor (float32 or bfloat16) of rows of C features, [.., C] (copied where it does not start on
    16 bytes); w_in: [C, 2 F], the gate's columns, then the others; w_out: [F, C]; biases [2 F] and [C] or
    None; all these 16-byte aligned; act: "silu", "gelu" or "gelu_tanh".  bf16 calls of more than 2^28
    multiply-adds a product and more than 64 rows (or C or F no multiple of 8) hold the hidden values in bf16
    between the products, others in 16 bits, so a row's last bits depend on how many are in the call.
    Gradients are of first order, by reverse mode only.
    """
    tensors = (x, w_in, b_in, w_out, b_out)
    _no_tangent("gated_mlp", *tensors)
    if w_out.dim() != 2:
        raise ValueError("w_out must be [F, C]")
    plan = _mlp_plan(x.shape, w_out.shape[0], act)
    _check_mlp(*tensors, plan[0])
    if x.data_ptr() % 16:           # a piece of another tensor
        tensors = (x.clone(), *tensors[1:])
    if torch.is_grad_enabled() and _any_requires_grad(tensors):
        return _Mlp.apply(*tensors, plan)
    return _mlp_fwd(*tensors, plan, None, None, None, False)[0]
