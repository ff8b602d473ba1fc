"""What the windowed attention and the 8-bit cache refuse or put right in Python, before anything is
enqueued (no GPU)."""
import pytest
import torch
import torch.autograd.forward_ad as fwAD

import laplacian_nystr_linear_gb300 as lap
from laplacian_nystr_linear_gb300 import window


def _operands():
    q, k, v = (torch.randn(1, 2, 8, 16) for _ in range(3))
    return q, k, v, lap.cache_alloc(4, 2, 16, 16, device="cpu"), torch.zeros((1, 1), dtype=torch.int32)


@pytest.mark.parametrize("which", range(3))
@pytest.mark.parametrize("grad", [True, False])
def test_forward_mode_derivatives_are_refused(which, grad):
    q, k, v, cache, table = _operands()
    with torch.set_grad_enabled(grad), fwAD.dual_level():
        x = [q, k, v]
        x[which] = fwAD.make_dual(x[which], torch.ones_like(q))
        with pytest.raises(ValueError, match="forward-mode"):
            lap.window_attention(*x, 4)
        with pytest.raises(ValueError, match="forward-mode"):
            if which == 0:
                lap.cache_attention(x[0], cache, table, table[0])
            else:
                lap.cache_append(cache, x[1], x[2], table, table[0])
        # plain tensors within a dual level are as ever: refused only as not on a GPU
        with pytest.raises(ValueError, match="CUDA"):
            lap.window_attention(q, k, v, 4)


def test_forward_mode_through_the_backward_is_refused():
    dout = torch.randn(1, 2, 8, 16)
    with fwAD.dual_level(), pytest.raises(ValueError, match="forward-mode"):
        window._Window.backward(object(), fwAD.make_dual(dout, torch.ones_like(dout)))


def test_function_transforms_are_refused():
    q, k, v, _, _ = _operands()
    with pytest.raises(ValueError, match="forward-mode"):
        torch.func.jvp(lambda q: lap.window_attention(q, k, v, 4), (q,), (torch.ones_like(q),))


@pytest.mark.parametrize("which", ["k", "v"])
def test_append_refuses_what_requires_a_gradient(which):
    _, k, v, cache, table = _operands()
    x = {"k": k, "v": v}
    x[which].requires_grad_(True)
    with pytest.raises(ValueError, match="gradient"):
        lap.cache_append(cache, k, v, table, table[0])
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):   # refused only as not on a GPU
        lap.cache_append(cache, k, v, table, table[0])


BIG = 2 ** 32      # cut to 32 bits: 0


@pytest.mark.parametrize("given,kept", [(BIG, 2 ** 31 - 1), (BIG + 5, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1),
                                        (2 ** 31 - 1, 2 ** 31 - 1), (-1, -1), (7, 7), (-BIG, -2 ** 31),
                                        (1 - 2 ** 33, -2 ** 31)])
def test_wide_windows_do_not_wrap(given, kept):
    q = torch.zeros((1, 2, 8, 16))
    assert lap.WindowParams.of(q, q, given, given, given).dims()[6:] == (kept, kept, kept)
    p = lap.WindowParams(1, 2, 2, 8, 8, 16, given, given, given, 1.0)
    assert p.dims()[6:] == (kept, kept, kept)


def test_wide_windows_over_the_cache_do_not_wrap():
    q, cache = torch.zeros((1, 2, 1, 16)), lap.cache_alloc(2000, 2, 16, 16, device="cpu")
    table = torch.zeros((1, 2000), dtype=torch.int32)
    need = lap.cache_workspace_bytes(q, cache, table, left=-1, right=0)
    assert lap.cache_workspace_bytes(q, cache, table, left=0, right=0) < need
    for wide in (BIG, BIG + 5, 2 ** 31):
        assert lap.cache_workspace_bytes(q, cache, table, left=wide, right=0) == need
        assert lap.cache_workspace_bytes(q, cache, table, left=0, right=wide) == need
        assert lap.cache_workspace_bytes(q, cache, table, left=0, right=0, sinks=wide) == need
    assert lap.cache_workspace_bytes(q, cache, table, left=-BIG) == 0      # not a window


def test_sizes_beyond_32_bits_are_refused():
    for i in range(6):
        dims = [1, 2, 2, 8, 8, 16]
        dims[i] += BIG
        with pytest.raises(ValueError, match="2\\*\\*31"):
            lap.window_workspace_bytes(lap.WindowParams(*dims, 4, 0, 0, 1.0), torch.bfloat16)
    with pytest.raises(ValueError, match="2\\*\\*31"):
        window._sizes(1, BIG + 5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_no_partials_where_the_first_tokens_tiles_are_not_cut(dtype):
    """As many key tiles with first tokens as blocks run at once: their queries stay whole, and the
    backward needs D (4 bytes a query row) alone."""
    rows = 32 * 8 * 4096
    p = lap.WindowParams(32, 8, 8, 4096, 4096, 128, 511, 0, 1024, 0.1)
    assert lap.window_workspace_bytes(p, dtype, True) == 4 * rows
    p = p._replace(B=1, Hq=2, Hkv=2)      # few tiles: cut
    assert lap.window_workspace_bytes(p, dtype, True) > 4 * rows / 128
