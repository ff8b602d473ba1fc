"""Refusals of the rotary positions, the residual with its norms and the gated feed-forward block, before
anything is enqueued (no GPU), and the frequencies that are computed on the host."""
import ctypes
import math

import pytest
import torch
import torch.autograd.forward_ad as fwAD

import laplacian_nystr_linear_gb300 as lap
from laplacian_nystr_linear_gb300 import _lib

FAKE = ctypes.c_void_p(1 << 20)   # aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 1)
HALF = ctypes.c_void_p((1 << 20) + 2)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from laplacian_nystr_linear_gb300 import build as b
    b.build()
    return _lib.load()


ROT = dict(B=2, Hq=4, Hkv=2, N=10, d=64, rot=32)


def _rotary(lib, **kw):
    a = dict(ROT, q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, turns=FAKE, start=None, positions=None, layout=0,
             factor=1.0, inverse=0, dtype=1)
    a.update(kw)
    return lib.lapnys_rotary(a["q"], a["k"], a["qo"], a["ko"], a["turns"], a["start"], a["positions"],
                             *(a[n] for n in ROT), a["layout"], a["factor"], a["inverse"], None, a["dtype"])


@pytest.mark.parametrize("bad", [
    dict(B=0), dict(Hq=0), dict(Hkv=-1), dict(Hkv=0), dict(N=0), dict(d=0), dict(rot=0), dict(rot=31),
    dict(rot=66), dict(q=None), dict(q=ODD), dict(k=None), dict(k=ODD), dict(qo=None), dict(ko=None),
    dict(ko=ODD), dict(turns=None), dict(turns=HALF), dict(start=HALF), dict(positions=ODD),
    dict(start=FAKE, positions=FAKE), dict(layout=2), dict(factor=NAN), dict(factor=INF), dict(dtype=2),
    dict(q=HALF, dtype=0), dict(B=1 << 20, N=1 << 20)], ids=str)
def test_rotary_refuses(lib, bad):
    before = lib.lapnys_launch_count()
    assert _rotary(lib, **bad) == _lib.LAPNYS_EINVAL
    assert lib.lapnys_launch_count() == before


NORM = dict(B=2, N=8, C=64, per_seq=0, pre=1, post=1)
VECS = ("weight", "bias", "pw", "pb", "gate", "scale")


def _fwd(lib, **kw):
    a = dict(NORM, x=FAKE, u=FAKE, h=FAKE, y=FAKE, stats=FAKE, eps=1e-6, dtype=1, **{v: None for v in VECS})
    a.update(kw)
    return lib.lapnys_norm_fwd(a["x"], a["u"], *(a[v] for v in VECS), a["h"], a["y"], a["stats"],
                               *(a[n] for n in NORM), a["eps"], None, a["dtype"])


def _bwd(lib, **kw):
    a = dict(NORM, x=FAKE, u=FAKE, stats=FAKE, dh=FAKE, dy=FAKE, dx=FAKE, du=FAKE, dtype=1, ws=None, ws_bytes=0,
             **{v: None for v in VECS}, **{"d" + v: None for v in VECS})
    a.update(kw)
    return lib.lapnys_norm_bwd(a["x"], a["u"], a["weight"], a["pw"], a["pb"], a["gate"], a["scale"], a["stats"],
                               a["dh"], a["dy"], a["dx"], a["du"], *(a["d" + v] for v in VECS),
                               *(a[n] for n in NORM), None, a["dtype"], a["ws"], a["ws_bytes"])


@pytest.mark.parametrize("bad", [
    dict(B=0), dict(N=0), dict(C=0), dict(B=1 << 16, N=1 << 16), dict(pre=3), dict(post=-1), dict(dtype=5),
    dict(x=None), dict(x=ODD), dict(stats=HALF), dict(gate=ODD), dict(pre=0), dict(pre=0, weight=FAKE),
    dict(pre=0, y=None, dy=None, per_seq=1), dict(u=None), dict(u=None, post=0, gate=FAKE),
    dict(u=None, post=0, scale=FAKE), dict(post=0, pw=FAKE), dict(post=0, pb=FAKE)], ids=str)
def test_norm_refuses(lib, bad):
    before = lib.lapnys_launch_count()
    kw = {k: v for k, v in bad.items() if k != "dy"}
    assert _fwd(lib, **kw) == _lib.LAPNYS_EINVAL
    assert _bwd(lib, **{k: v for k, v in bad.items() if k != "y"}) == _lib.LAPNYS_EINVAL
    assert lib.lapnys_launch_count() == before


def test_norm_refuses_more(lib):
    assert _fwd(lib, C=16385) == _lib.LAPNYS_ENOTSUP and _bwd(lib, C=16385) == _lib.LAPNYS_ENOTSUP
    for bad in (dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(y=None), dict(h=None, y=None), dict(bias=ODD)):
        assert _fwd(lib, **bad) == _lib.LAPNYS_EINVAL
    for bad in (dict(stats=None), dict(dgate=FAKE), dict(dscale=FAKE), dict(dpw=FAKE), dict(dx=ODD),
                dict(pre=0, dy=FAKE), dict(u=None, post=0), dict(dweight=FAKE),
                dict(post=0, dpb=FAKE), dict(pre=0, dy=None, dweight=FAKE)):
        assert _bwd(lib, **bad) == _lib.LAPNYS_EINVAL
    need = lib.lapnys_norm_workspace_bytes(2, 8, 64, 0)
    assert need >= 4 * 64 * 4
    assert _bwd(lib, dweight=FAKE, ws=FAKE, ws_bytes=need - 1) == _lib.LAPNYS_ENOSPC
    assert lib.lapnys_norm_workspace_bytes(2, 8, 16385, 0) == 0
    assert lib.lapnys_norm_workspace_bytes(0, 8, 64, 0) == 0


def test_norm_rows_stay_countable(lib):
    """Rows, and the places just behind the last one, are counted in 32 bits."""
    most = 2 ** 31 - 1024
    for B, N in ((1, most + 1), (most + 1, 1), (1, 2 ** 31 - 1)):
        assert _fwd(lib, B=B, N=N) == _lib.LAPNYS_EINVAL and _bwd(lib, B=B, N=N) == _lib.LAPNYS_EINVAL
        assert lib.lapnys_norm_workspace_bytes(B, N, 1, 1) == 0
    # a sequence a row: sums of four kinds of every slot and sequence
    assert 2 * 16 * most < lib.lapnys_norm_workspace_bytes(most, 1, 1, 1) < 2 * 16 * (most + 1024)


MLP = dict(T=100, C=64, F=128)
BIG = 1 << 40


def _mlp_fwd(lib, **kw):
    a = dict(MLP, x=FAKE, w_in=FAKE, b_in=None, w_out=FAKE, b_out=None, y=FAKE, act=0, dtype=1, ctx=None, ctx_bytes=0,
             ws=FAKE, ws_bytes=0)
    a.update(kw)
    return lib.lapnys_mlp_fwd(a["x"], a["w_in"], a["b_in"], a["w_out"], a["b_out"], a["y"], *(a[n] for n in MLP),
                              a["act"], None, a["dtype"], a["ctx"], a["ctx_bytes"], a["ws"], a["ws_bytes"])


def _mlp_bwd(lib, **kw):
    a = dict(MLP, x=FAKE, w_in=FAKE, w_out=FAKE, dy=FAKE, ctx=FAKE, dx=FAKE, dw_in=FAKE, db_in=None, dw_out=FAKE,
             db_out=None, dtype=1, ws=FAKE, ws_bytes=0)
    a.update(kw)
    return lib.lapnys_mlp_bwd(a["x"], a["w_in"], a["w_out"], a["dy"], a["ctx"], a["dx"], a["dw_in"], a["db_in"],
                              a["dw_out"], a["db_out"], *(a[n] for n in MLP), None, a["dtype"], a["ws"],
                              a["ws_bytes"])


@pytest.mark.parametrize("bad", [
    dict(T=0), dict(C=0), dict(F=-1), dict(T=(1 << 28) + 1), dict(C=1 << 21), dict(F=1 << 21),
    dict(T=1 << 28, C=1 << 20), dict(C=1 << 20, F=1 << 20, T=1), dict(dtype=2), dict(x=None), dict(w_in=ODD),
    dict(w_out=None), dict(x=HALF), dict(ws=None), dict(ws=HALF)], ids=str)
def test_mlp_refuses(lib, bad):
    before = lib.lapnys_launch_count()
    assert _mlp_fwd(lib, **bad) == _lib.LAPNYS_EINVAL
    assert _mlp_bwd(lib, **bad) == _lib.LAPNYS_EINVAL
    assert lib.lapnys_launch_count() == before


def test_mlp_refuses_more(lib):
    for bad in (dict(act=-1), dict(act=3), dict(y=None), dict(y=ODD), dict(b_in=HALF), dict(ctx=HALF)):
        assert _mlp_fwd(lib, **bad) == _lib.LAPNYS_EINVAL
    for bad in (dict(dy=None), dict(ctx=None), dict(dx=HALF), dict(db_in=ODD), dict(dw_out=HALF)):
        assert _mlp_bwd(lib, **bad) == _lib.LAPNYS_EINVAL
    for dtype in (0, 1):
        fwd, bwd = (lib.lapnys_mlp_workspace_bytes(100, 64, 128, dtype, b) for b in (0, 1))
        ctx = lib.lapnys_mlp_ctx_bytes(100, 64, 128, dtype)
        assert min(fwd, bwd, ctx) > 0
        assert _mlp_fwd(lib, dtype=dtype, ws_bytes=fwd - 1) == _lib.LAPNYS_ENOSPC
        assert _mlp_fwd(lib, dtype=dtype, ws_bytes=fwd, ctx=FAKE, ctx_bytes=ctx - 1) == _lib.LAPNYS_ENOSPC
        assert _mlp_bwd(lib, dtype=dtype, ws_bytes=bwd - 1) == _lib.LAPNYS_ENOSPC
    assert lib.lapnys_mlp_ctx_bytes(0, 64, 128, 1) == 0 and lib.lapnys_mlp_workspace_bytes(1, 64, 128, 7, 0) == 0


def test_mlp_sizes(lib):
    """h, p and q of a training step, 6 bytes a hidden value in bf16; the backward's partial sums bounded."""
    T, C, F = 131072, 512, 1408
    assert 6 * T * F < lib.lapnys_mlp_ctx_bytes(T, C, F, 1) < 6.3 * T * F
    assert 4 * T * F < lib.lapnys_mlp_workspace_bytes(T, C, F, 1, 1) < 4 * T * F + (1 << 28)
    assert lib.lapnys_mlp_workspace_bytes(1, 4096, 10880, 1, 0) < 1 << 24   # no copy of the weights


def test_python_refuses():
    q, f = torch.zeros((1, 2, 4, 16)), lap.rotary_frequencies(16, device="cpu")
    x, w = torch.zeros((2, 4, 16)), torch.ones(16)
    wi, wo = torch.zeros((16, 16)), torch.zeros((8, 16))
    for bad in (lambda: lap.rotary(q, q, f), lambda: lap.rotary(q[0], q, f), lambda: lap.rotary(q, q, None),
                lambda: lap.rotary(q, q, f, layout="pairs"), lambda: lap.rotary_frequencies(7),
                lambda: lap.rotary_frequencies(0), lambda: lap.rotary_frequencies(8, base=0),
                lambda: lap.rotary_frequencies(8, scaling="none"), lambda: lap.rotary_frequencies(8, factor=-1),
                lambda: lap.rotary_frequencies(8, scaling="parts", factor=2.0),
                lambda: lap.rotary_frequencies(8, scaling="parts", factor=2.0, context=100, low=3, high=2),
                lambda: lap.RotaryFrequencies.of([INF], device="cpu"),
                lambda: lap.RotaryFrequencies.of([], device="cpu"),
                lambda: lap.residual_norm(x, None, w), lambda: lap.residual_norm(x[0], None, w),
                lambda: lap.residual_norm(x, pre=None), lambda: lap.residual_norm(x, x, w, pre="batch"),
                lambda: lap.residual_norm(x, x, w, post="l2"),
                lambda: lap.gated_mlp(x, wi, None, wo, None), lambda: lap.gated_mlp(x[0, 0], wi, None, wo, None),
                lambda: lap.gated_mlp(x, wi, None, wo[0], None), lambda: lap.gated_mlp(x, wi, None, wo, None, "relu"),
                lambda: lap.mlp_fwd(x, wi, None, wo, None, lap.MlpParams(BIG, 16, 8)),
                lambda: lap.mlp_ctx_bytes(lap.MlpParams(BIG, 16, 8), torch.bfloat16),
                lambda: lap.norm_workspace_bytes(BIG, 1, 16, False)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: lap.rotary(q.half(), q.half(), f), lambda: lap.residual_norm(x.half(), None, w.half()),
                lambda: lap.gated_mlp(x.half(), wi.half(), None, wo.half(), None)):
        with pytest.raises(TypeError):
            bad()


def test_forward_mode_derivatives_are_refused():
    q, f = torch.zeros((1, 2, 4, 16)), lap.rotary_frequencies(16, device="cpu")
    x, w = torch.zeros((2, 4, 16)), torch.ones(16)
    with fwAD.dual_level():
        dual = fwAD.make_dual(q, torch.ones_like(q))
        for call in (lambda: lap.rotary(dual, q, f), lambda: lap.rotary(q, dual, f),
                     lambda: lap.residual_norm(x, None, fwAD.make_dual(w, w)),
                     lambda: lap.residual_norm(fwAD.make_dual(x, x), x),
                     lambda: lap.gated_mlp(fwAD.make_dual(x, x), torch.zeros((16, 16)), None, torch.zeros((8, 16)),
                                           None)):
            with pytest.raises(ValueError, match="forward-mode"):
                call()


def test_frequencies():
    turns = lambda f: [t % 2 ** 64 / 2.0 ** 64 for t in f.turns.tolist()]  # noqa: E731
    w = [10000.0 ** (-2 * i / 16) for i in range(8)]
    plain = lap.rotary_frequencies(16, device="cpu")
    assert turns(plain) == pytest.approx([x / (2 * math.pi) for x in w], rel=1e-14) and plain.factor == 1.0
    assert turns(lap.rotary_frequencies(16, scaling="linear", factor=4, device="cpu")) == pytest.approx(
        [x / (8 * math.pi) for x in w], rel=1e-14)
    base = turns(lap.rotary_frequencies(16, scaling="base", factor=4, device="cpu"))
    assert base[0] == turns(plain)[0] and base[-1] == pytest.approx(turns(plain)[-1] / 4, rel=1e-12)
    parts = lap.rotary_frequencies(16, scaling="parts", factor=4, context=4096, device="cpu")
    assert turns(parts)[0] == turns(plain)[0] and turns(parts)[-1] == pytest.approx(turns(plain)[-1] / 4)
    assert parts.factor == pytest.approx(1 + 0.1 * math.log(4))
    back = lap.RotaryFrequencies.of([-0.5, 7.0], device="cpu")
    assert turns(back) == pytest.approx([1 - 0.5 / (2 * math.pi), 7 / (2 * math.pi) - 1])


def test_mlp_refuses_more_features_than_an_accumulator_sums(lib):
    for C in ((1 << 16) + 1, 1 << 17, 1 << 20):
        assert _mlp_fwd(lib, C=C) == _lib.LAPNYS_EINVAL and _mlp_bwd(lib, C=C) == _lib.LAPNYS_EINVAL
        assert lib.lapnys_mlp_ctx_bytes(100, C, 128, 1) == 0 and lib.lapnys_mlp_ctx_bytes(64, C | 1, 128, 1) == 0
        # few rows and fp32 sum such products up in registers
        assert lib.lapnys_mlp_ctx_bytes(100, C, 128, 0) > 0 and lib.lapnys_mlp_ctx_bytes(64, C & -8, 128, 1) > 0
    assert lib.lapnys_mlp_ctx_bytes(100, 1 << 16, 128, 1) > 0


def _turn(digits):
    """2 pi 10^digits, in whole numbers: pi / 4 = 4 atan(1 / 5) - atan(1 / 239)"""
    one = 10 ** (digits + 10)

    def atan(n):
        t = s = one // n
        k = 1
        while t:
            t //= -n * n
            k += 2
            s += t // k
        return s

    return 8 * (4 * atan(5) - atan(239)) // 10 ** 10


def test_frequencies_to_the_last_bit():
    """base^(-2 i / 16) with base 10^4 is 10^(-i / 2): square roots in whole numbers, to 60 digits."""
    D = 60
    turn = _turn(D)
    for scaling, by in ((None, 1), ("linear", 7)):
        got = lap.rotary_frequencies(16, scaling=scaling, factor=by, device="cpu").turns.tolist()
        for i, t in enumerate(got):
            w = math.isqrt(10 ** (2 * D - i)) // by
            assert abs(t % 2 ** 64 - w * 2 ** 64 / turn) <= 2 ** 12      # (a double's view of it)
            assert abs(t % 2 ** 64 - (w * 2 ** 64 + turn // 2) // turn) <= 1, (scaling, i)
    # the slowest pair with a raised base: exactly divided by the factor
    base = lap.rotary_frequencies(16, scaling="base", factor=4, device="cpu").turns.tolist()
    assert abs(base[-1] - (math.isqrt(10 ** (2 * D - 7)) // 4 * 2 ** 64 + turn // 2) // turn) <= 1
    # given angles are taken as the numbers they are
    got = lap.RotaryFrequencies.of([0.1, -3.0, 1e6], device="cpu").turns.tolist()
    for w, t in zip((0.1, -3.0, 1e6), got):
        n, d = w.as_integer_ratio()
        want = (n * 10 ** D * 2 ** 64 + d * turn // 2) // (d * turn)
        assert (t - want + 1) % 2 ** 64 <= 2, w
