"""Softmax attention over a window and the first tokens, for training, prompts
and single tokens, and the same attention over a cache held in 8 bits.

Key j is visible to the query at position p of a sequence of n tokens iff
0 <= p < n, j < n, j <= p + right and (j >= p - left or j < sinks); -1 as left or
right is no bound.  Marshalling only: every step runs in liblapnys kernels.
"""
from __future__ import annotations

import contextlib
import functools
import math
from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import _lib
from ._lib import check, load
from .api import _DT, _dtype


def _sizes(*sizes):
    """Sizes as the C entries take them: ctypes would cut them to 32 bits."""
    if max(sizes) >= 2 ** 31 or min(sizes) < -2 ** 31:
        raise ValueError(f"sizes must be below 2**31: {sizes}")
    return sizes


@functools.lru_cache(maxsize=256)
def _reach(*tokens):
    """Sides and first tokens the same way: from 2^28 tokens on they are as good as any."""
    return tuple(max(-2 ** 31, min(int(t), 2 ** 31 - 1)) for t in tokens)


class WindowParams(NamedTuple):
    """Shape and mask of one call: q [B, Hq, Nq, d], k and v [B, Hkv, Nk, d]."""
    B: int
    Hq: int
    Hkv: int
    Nq: int
    Nk: int
    d: int
    left: int
    right: int
    sinks: int
    scale: float

    @functools.lru_cache(maxsize=256)
    def dims(self):
        return *_sizes(*self[:6]), *_reach(*self[6:9])

    @staticmethod
    def of(q: torch.Tensor, k: torch.Tensor, left: int, right: int = 0, sinks: int = 0,
           scale: Optional[float] = None) -> "WindowParams":
        if q.dim() != 4 or k.dim() != 4:
            raise ValueError("q and k must be [B, H, N, d] tensors")
        B, Hq, Nq, d = q.shape
        return WindowParams(B, Hq, k.shape[1], Nq, k.shape[2], d, int(left), int(right), int(sinks),
                            _scale(scale, d))


class KVCache(NamedTuple):
    """Keys and values in 8 bits: k, v float8_e4m3fn [blocks, Hkv, block, d] and their scales
    float32 [blocks, Hkv] (powers of two); a key is k * k_scale."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


def _scale(scale, d):
    return 1.0 / math.sqrt(d) if scale is None else float(scale)


def _tensor(t, name, shape, dtype, device):
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape
            or not t.is_cuda or not t.is_contiguous() or t.device != device):
        raise ValueError(f"{name} must be a contiguous CUDA tensor of shape {tuple(shape)} and {dtype}"
                         f" on {device}")


def _batch(t, name, B, device):
    if t is not None:
        _tensor(t, name, (B,), torch.int32, device)


def _no_tangent(name, *tensors):
    """Refuses dual tensors, whose tangents the kernels would drop.  (Outside a dual level there are
    none; three tensors looked at take 1 to 2 us of a call's 25.)"""
    if getattr(forward_ad, "_current_level", 0) < 0:
        return
    for t in tensors:
        if isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None:
            raise ValueError(f"{name} has no forward-mode derivative")


_HERE = contextlib.nullcontext()


def _at(t):
    return None if t is None else t.data_ptr()


def _on_stream(device):
    return torch._C._cuda_getCurrentRawStream(device.index)


def _on(device):
    """The tensors' device as the current one."""
    return _HERE if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _workspace(ws, need, device):
    if ws is None:
        return torch.empty(need, dtype=torch.uint8, device=device) if need else None
    if not ws.is_cuda or ws.device != device or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous CUDA tensor on {device}")
    return ws


def _nbytes(ws):
    return 0 if ws is None else ws.nbytes


def _check_window(q, k, v, lens, q_pos, p: WindowParams):
    dev, dt = q.device, q.dtype
    _dtype(q)
    _tensor(q, "q", (p.B, p.Hq, p.Nq, p.d), dt, dev)
    _tensor(k, "k", (p.B, p.Hkv, p.Nk, p.d), dt, dev)
    _tensor(v, "v", (p.B, p.Hkv, p.Nk, p.d), dt, dev)
    _batch(lens, "lens", p.B, dev)
    _batch(q_pos, "q_pos", p.B, dev)


@functools.lru_cache(maxsize=256)
def window_workspace_bytes(p: WindowParams, dtype: torch.dtype, backward: bool = False) -> int:
    return load().lapnys_window_workspace_bytes(*p.dims(), _DT[dtype], int(backward))


def window_fwd(q, k, v, p: WindowParams, lens=None, q_pos=None, out=None, lse=None, ws=None,
               need_lse=True, rest=None):
    """lapnys_window_fwd: returns (out, lse); lse is None when need_lse is False.  rest (bf16, like
    out): filled with what the rounding of out left, for window_bwd."""
    _check_window(q, k, v, lens, q_pos, p)
    dev = q.device
    if out is not None:
        _tensor(out, "out", q.shape, q.dtype, dev)
    if lse is not None:
        _tensor(lse, "lse", q.shape[:3], torch.float32, dev)
    if rest is not None:
        _tensor(rest, "rest", q.shape, torch.bfloat16, dev)
    with _on(dev):
        out = torch.empty_like(q) if out is None else out
        if not need_lse:
            lse = None
        elif lse is None:
            lse = torch.empty(q.shape[:3], dtype=torch.float32, device=dev)
        ws = _workspace(ws, window_workspace_bytes(p, q.dtype), dev)
        rc = load().lapnys_window_fwd(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), _at(lse), _at(rest), _at(lens),
            _at(q_pos), *p.dims(), p.scale, _on_stream(dev), _dtype(q), _at(ws), _nbytes(ws))
    check(rc, "lapnys_window_fwd")
    return out, lse


def window_bwd(q, k, v, out, dout, lse, p: WindowParams, lens=None, q_pos=None, dq=None, dk=None,
               dv=None, ws=None, rest=None):
    """lapnys_window_bwd: returns (dq, dk, dv); rest: the forward's, if it kept one."""
    _check_window(q, k, v, lens, q_pos, p)
    dev = q.device
    _tensor(out, "out", q.shape, q.dtype, dev)
    _tensor(lse, "lse", q.shape[:3], torch.float32, dev)
    for t, name, like in ((dq, "dq", q), (dk, "dk", k), (dv, "dv", v)):
        if t is not None:
            _tensor(t, name, like.shape, q.dtype, dev)
    if rest is not None:
        _tensor(rest, "rest", q.shape, torch.bfloat16, dev)
    return _bwd(q, k, v, out, dout, lse, rest, p, lens, q_pos, dq, dk, dv, ws)


def _bwd(q, k, v, out, dout, lse, rest, p, lens, q_pos, dq, dk, dv, ws):
    dev = q.device
    _tensor(dout, "dout", q.shape, q.dtype, dev)
    with _on(dev):
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        dv = torch.empty_like(v) if dv is None else dv
        ws = _workspace(ws, window_workspace_bytes(p, q.dtype, True), dev)
        rc = load().lapnys_window_bwd(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), dout.data_ptr(), lse.data_ptr(),
            _at(rest), _at(lens), _at(q_pos), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
            *p.dims(), p.scale, _on_stream(dev), _dtype(q), _at(ws), _nbytes(ws))
    check(rc, "lapnys_window_bwd")
    return dq, dk, dv


class _Window(torch.autograd.Function):
    @staticmethod
    def forward(fctx, q, k, v, lens, q_pos, p: WindowParams):
        rest = torch.empty_like(q) if q.dtype == torch.bfloat16 else None
        out, lse = window_fwd(q, k, v, p, lens, q_pos, rest=rest)
        fctx.p = p
        fctx.save_for_backward(q, k, v, out, lse, rest, lens, q_pos)
        return out

    @staticmethod
    @once_differentiable
    def backward(fctx, dout):
        _no_tangent("window_attention's backward", dout)
        q, k, v, out, lse, rest, lens, q_pos = fctx.saved_tensors   # checked by the forward
        return *_bwd(q, k, v, out, dout.contiguous(), lse, rest, fctx.p, lens, q_pos, None, None,
                     None, None), None, None, None


def window_attention(q, k, v, left, right=0, sinks=0, scale=None, lens=None, q_pos=None):
    """Softmax attention over a window and the first tokens, with autograd.

    q: [B, Hq, Nq, d], k, v: [B, Hkv, Nk, d] CUDA tensors (float32 or bfloat16), Hq a multiple of
    Hkv, d a multiple of 16 up to 128.  A query sees `left` keys before it, `right` after it (-1:
    all) and the first `sinks` of its sequence, never beyond p + right.  lens: int32 [B], tokens of
    each sequence of a padded batch; q_pos: int32 [B], position of each sequence's first query
    (default Nk - Nq).  Queries that see nothing give zeros.  scale defaults to 1 / sqrt(d).
    Gradients are of first order, by reverse mode only.  A step that is captured into a CUDA graph takes leaves that no
    eager autograd graph still holds (their gradients would be added up on that graph's stream).
    """
    _no_tangent("window_attention", q, k, v)
    p = WindowParams.of(q, k, left, right, sinks, scale)
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad):
        return _Window.apply(q, k, v, lens, q_pos, p)
    return window_fwd(q, k, v, p, lens, q_pos, need_lse=False)[0]


# ---------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------
def cache_alloc(blocks, heads, d, block=64, device="cuda") -> KVCache:
    """An empty cache of `blocks` blocks of `block` tokens (16, 32, 64 or 128)."""
    kv = (torch.zeros((blocks, heads, block, d), dtype=torch.float8_e4m3fn, device=device)
          for _ in range(2))
    sc = (torch.zeros((blocks, heads), dtype=torch.float32, device=device) for _ in range(2))
    return KVCache(*kv, *sc)


def _check_cache(cache: KVCache, table, heads, d, B, device):
    if cache.k.dim() != 4:
        raise ValueError("the cache's k must be [blocks, heads, block, d]")
    blocks, _, block, _ = cache.k.shape
    for name in ("k", "v"):
        _tensor(getattr(cache, name), f"cache.{name}", (blocks, heads, block, d), torch.float8_e4m3fn,
                device)
        _tensor(getattr(cache, f"{name}_scale"), f"cache.{name}_scale", (blocks, heads),
                torch.float32, device)
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be an int32 tensor [B, max_blocks]")
    _tensor(table, "table", (B, table.shape[1]), torch.int32, device)
    return block, blocks, table.shape[1]


def cache_append(cache: KVCache, k, v, table, start, lens=None) -> None:
    """lapnys_cache_append: rounds the new tokens k, v [B, Hkv, N, d] (float32 or bfloat16) into the
    cache; token i of sequence b goes to position start[b] + i while that is below lens[b].
    table: int32 [B, max_blocks]; start, lens: int32 [B].  No derivatives."""
    _no_tangent("cache_append", k, v)
    if torch.is_grad_enabled() and (k.requires_grad or v.requires_grad):
        raise ValueError("cache_append has no gradient: detach k and v")
    if k.dim() != 4:
        raise ValueError("k must be [B, Hkv, N, d]")
    B, Hkv, N, d = k.shape
    dev = k.device
    dt = _dtype(k)
    _tensor(k, "k", k.shape, k.dtype, dev)
    _tensor(v, "v", k.shape, k.dtype, dev)
    geometry = _check_cache(cache, table, Hkv, d, B, dev)
    _tensor(start, "start", (B,), torch.int32, dev)
    _batch(lens, "lens", B, dev)
    with _on(dev):
        rc = load().lapnys_cache_append(
            _at(k), _at(v), _at(cache.k), _at(cache.v), _at(cache.k_scale), _at(cache.v_scale),
            _at(table), _at(start), _at(lens), *_sizes(B, Hkv, N, d, *geometry), _on_stream(dev), dt)
    check(rc, "lapnys_cache_append")


@functools.lru_cache(maxsize=256)
def _cache_workspace(*sizes) -> int:
    return load().lapnys_cache_workspace_bytes(*sizes)


def cache_workspace_bytes(q, cache: KVCache, table, left=-1, right=0, sinks=0) -> int:
    B, Hq, Nq, d = q.shape
    blocks, Hkv, block, _ = cache.k.shape
    return _cache_workspace(*_sizes(B, Hq, Hkv, Nq, d, block, blocks, table.shape[1]),
                            *_reach(left, right, sinks), _dtype(q))


def cache_attention(q, cache: KVCache, table, lens, left=-1, right=0, sinks=0, scale=None,
                    q_pos=None, out=None, ws=None):
    """lapnys_cache_attention: attention of a few queries q [B, Hq, Nq, d] (float32 or bfloat16) over
    the cache, with window_attention's mask.  lens: int32 [B], the sequences' tokens in the cache;
    q_pos: int32 [B], default lens - Nq (the queries are the last tokens).  No derivatives."""
    _no_tangent("cache_attention", q)
    if q.dim() != 4:
        raise ValueError("q must be [B, Hq, Nq, d]")
    if torch.is_grad_enabled() and q.requires_grad:
        raise ValueError("cache_attention has no gradient: detach q")
    B, Hq, Nq, d = q.shape
    dev = q.device
    dt = _dtype(q)
    _tensor(q, "q", q.shape, q.dtype, dev)
    Hkv = cache.k.shape[1] if cache.k.dim() == 4 else 0
    geometry = _check_cache(cache, table, Hkv, d, B, dev)
    _tensor(lens, "lens", (B,), torch.int32, dev)
    _batch(q_pos, "q_pos", B, dev)
    sizes, reach = _sizes(B, Hq, Hkv, Nq, d, *geometry), _reach(left, right, sinks)
    with _on(dev):
        out = torch.empty_like(q) if out is None else out
        _tensor(out, "out", q.shape, q.dtype, dev)
        ws = _workspace(ws, _cache_workspace(*sizes, *reach, dt), dev)
        rc = load().lapnys_cache_attention(
            _at(q), _at(cache.k), _at(cache.v), _at(cache.k_scale), _at(cache.v_scale),
            _at(table), _at(lens), _at(q_pos), _at(out), *sizes, *reach,
            _scale(scale, d), _on_stream(dev), dt, _at(ws), _nbytes(ws))
    check(rc, "lapnys_cache_attention")
    return out
