"""Refusals of the windowed attention and the 8-bit cache, found on the host before anything is
enqueued (no GPU)."""
import ctypes

import pytest
import torch

from laplacian_nystr_linear_gb300 import _lib

FAKE = ctypes.c_void_p(1 << 20)   # aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 4)
ODD2 = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    from laplacian_nystr_linear_gb300 import build as b
    b.build()
    return _lib.load()


DIMS = dict(B=2, Hq=4, Hkv=2, Nq=100, Nk=100, d=64, left=10, right=0, sinks=1)


def _fwd(lib, **kw):
    a = dict(DIMS, q=FAKE, k=FAKE, v=FAKE, out=FAKE, lse=FAKE, rest=None, lens=None, q_pos=None, scale=0.1,
             dtype=1, ws=None, ws_bytes=0)
    a.update(kw)
    return lib.lapnys_window_fwd(a["q"], a["k"], a["v"], a["out"], a["lse"], a["rest"], a["lens"],
                                 a["q_pos"], *(a[n] for n in DIMS), a["scale"], None, a["dtype"], a["ws"],
                                 a["ws_bytes"])


def _bwd(lib, **kw):
    a = dict(DIMS, q=FAKE, k=FAKE, v=FAKE, out=FAKE, dout=FAKE, lse=FAKE, rest=None, lens=None, q_pos=None, dq=FAKE,
             dk=FAKE, dv=FAKE, scale=0.1, dtype=1, ws=FAKE, ws_bytes=0)
    a.update(kw)
    return lib.lapnys_window_bwd(a["q"], a["k"], a["v"], a["out"], a["dout"], a["lse"], a["rest"], a["lens"],
                                 a["q_pos"], a["dq"], a["dk"], a["dv"], *(a[n] for n in DIMS), a["scale"],
                                 None, a["dtype"], a["ws"], a["ws_bytes"])


BAD = [dict(B=0), dict(Hq=0), dict(Hq=3), dict(Hkv=-1), dict(Nq=0), dict(Nk=0), dict(Nk=(1 << 28) + 1),
       dict(left=-2), dict(right=-2), dict(sinks=-1), dict(scale=0.0), dict(scale=float("nan")),
       dict(scale=float("inf")), dict(scale=-1.0), dict(dtype=2), dict(q=None), dict(k=ODD), dict(v=None),
       dict(out=ODD), dict(lse=ODD2), dict(rest=ODD),
       dict(rest=FAKE, dtype=0), dict(lens=ODD2), dict(q_pos=ODD2), dict(B=1 << 20, Hq=1 << 10)]


@pytest.mark.parametrize("bad", BAD, ids=str)
def test_window_refuses(lib, bad):
    before = lib.lapnys_launch_count()
    assert _fwd(lib, **bad) == _lib.LAPNYS_EINVAL
    assert _bwd(lib, **bad) == _lib.LAPNYS_EINVAL
    assert lib.lapnys_launch_count() == before


def test_window_refuses_widths_and_small_workspaces(lib):
    for d in (8, 24, 144, 256):
        assert _fwd(lib, d=d) == _lib.LAPNYS_ENOTSUP
        assert _bwd(lib, d=d) == _lib.LAPNYS_ENOTSUP
    for bad in (dict(dq=None), dict(dk=ODD), dict(dv=None), dict(dout=ODD), dict(ws=None), dict(lse=None)):
        assert _bwd(lib, **bad) == _lib.LAPNYS_EINVAL
    need = lib.lapnys_window_workspace_bytes(*DIMS.values(), 1, 1)
    assert need >= 2 * 4 * 100 * 4
    assert _bwd(lib, ws_bytes=need - 1) == _lib.LAPNYS_ENOSPC
    token = dict(DIMS, Nq=1, Nk=100000, left=-1)
    need = lib.lapnys_window_workspace_bytes(*token.values(), 1, 0)
    assert need > 0
    assert _fwd(lib, **token, ws=FAKE, ws_bytes=need - 1) == _lib.LAPNYS_ENOSPC
    assert _fwd(lib, **token) == _lib.LAPNYS_EINVAL          # needs one
    assert lib.lapnys_window_workspace_bytes(*dict(DIMS, d=24).values(), 1, 1) == 0
    # many first tokens on a long sequence: the partials stay bounded
    far = dict(DIMS, Nq=1 << 16, Nk=1 << 16, left=127, sinks=1 << 14)
    assert lib.lapnys_window_workspace_bytes(*far.values(), 1, 1) < 1 << 30


CACHE = dict(B=2, Hkv=2, N=5, d=64, block=32, blocks=10, max_blocks=4)


def _append(lib, **kw):
    a = dict(CACHE, k=FAKE, v=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, table=FAKE, start=FAKE, lens=None,
             dtype=1)
    a.update(kw)
    return lib.lapnys_cache_append(a["k"], a["v"], a["kc"], a["vc"], a["ks"], a["vs"], a["table"],
                                   a["start"], a["lens"], *(a[n] for n in CACHE), None, a["dtype"])


def _attend(lib, **kw):
    a = dict(CACHE, Hq=4, q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, table=FAKE, lens=FAKE, q_pos=None,
             out=FAKE, left=-1, right=0, sinks=0, scale=0.1, dtype=1, ws=None, ws_bytes=0)
    a.update(kw)
    return lib.lapnys_cache_attention(a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["table"], a["lens"],
                                      a["q_pos"], a["out"], a["B"], a["Hq"], a["Hkv"], a["N"], a["d"],
                                      a["block"], a["blocks"], a["max_blocks"], a["left"], a["right"],
                                      a["sinks"], a["scale"], None, a["dtype"], a["ws"], a["ws_bytes"])


@pytest.mark.parametrize("bad", [dict(B=0), dict(Hkv=0), dict(N=0), dict(block=8), dict(block=48),
                                 dict(blocks=0), dict(max_blocks=0), dict(max_blocks=1 << 27), dict(dtype=3),
                                 dict(kc=None), dict(vc=ODD), dict(ks=ODD2), dict(vs=None), dict(table=None),
                                 dict(lens=ODD2)], ids=str)
def test_cache_refuses(lib, bad):
    before = lib.lapnys_launch_count()
    assert _append(lib, **bad) == _lib.LAPNYS_EINVAL
    assert _attend(lib, **bad) == _lib.LAPNYS_EINVAL
    assert lib.lapnys_launch_count() == before


def test_cache_refuses_more(lib):
    assert _append(lib, d=24) == _lib.LAPNYS_ENOTSUP and _attend(lib, d=160) == _lib.LAPNYS_ENOTSUP
    assert _append(lib, k=ODD) == _lib.LAPNYS_EINVAL and _append(lib, start=None) == _lib.LAPNYS_EINVAL
    for bad in (dict(Hq=3), dict(q=ODD), dict(out=None), dict(lens=None), dict(left=-3), dict(sinks=-1),
                dict(scale=0.0), dict(q_pos=ODD2)):
        assert _attend(lib, **bad) == _lib.LAPNYS_EINVAL
    need = lib.lapnys_cache_workspace_bytes(2, 4, 2, 1, 64, 32, 4000, 4000, -1, 0, 0, 1)
    assert need > 0
    assert _attend(lib, N=1, blocks=4000, max_blocks=4000, ws=FAKE, ws_bytes=need - 1) == _lib.LAPNYS_ENOSPC
    assert lib.lapnys_cache_workspace_bytes(2, 4, 2, 1, 64, 31, 4000, 4000, -1, 0, 0, 1) == 0


def test_status_texts(lib):
    assert b"block" in lib.lapnys_strerror(_lib.LAPNYS_EPAGE)


def test_python_refuses():
    import laplacian_nystr_linear_gb300 as lap
    x = torch.zeros((1, 2, 8, 16))
    with pytest.raises(ValueError):          # not on a GPU
        lap.window_attention(x, x, x, 4)
    with pytest.raises(ValueError):
        lap.window_attention(x[0], x, x, 4)
    with pytest.raises(TypeError):
        lap.window_attention(x.half(), x.half(), x.half(), 4)
    cache = lap.cache_alloc(4, 2, 16, 16, device="cpu")
    assert cache.k.shape == (4, 2, 16, 16) and cache.k_scale.shape == (4, 2)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        lap.cache_append(cache, x, x, i[None], i)
    with pytest.raises(ValueError):
        lap.cache_attention(x, cache, i[None], i)
    with pytest.raises(ValueError):          # no gradient
        lap.cache_attention(x.clone().requires_grad_(True), cache, i[None], i)
