"""Attention over the 8-bit cache where the blocks' value scales lie far apart, against the plain
64-bit form on the values that the cache stands for (allowed errors: tests/_window_ref.py)."""
import pytest
import torch

import laplacian_nystr_linear_gb300 as lap
from laplacian_nystr_linear_gb300 import _lib, api

from tests._window_ref import check, reference
from tests.test_cache_gpu import clone, filled, gathered

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
DTYPES = pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
ROWS = pytest.mark.parametrize("Nq", [1, 4], ids=["4rows", "16rows"])   # of 4 heads a key head


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    assert api.device_status(clear=True) == _lib.LAPNYS_OK


def compare(q, cache, table, lens):
    """cache_attention against the 64-bit form.  P is held to 2^-21 of itself with fp32 queries (two
    f16 parts), and q to 2^-22 of its row's largest feature."""
    out = lap.cache_attention(q, cache, table, lens)
    k, v = gathered(cache, table)
    ref = reference(q, k, v, -1, 0, 0, None, lens, lens - q.shape[2], extra_p=2.0 ** -21,
                    extra_s=2.0 ** -22 * 8)
    check("out", out, ref["out"])
    return out


@DTYPES
@ROWS
@pytest.mark.parametrize("order", ["down", "up"])
@pytest.mark.parametrize("place", ["in_a_group", "across_groups"])
@pytest.mark.parametrize("gap", [17, 20, 40])
def test_neighbouring_blocks_far_apart(gap, place, order, Nq, dtype):
    """Blocks of 16 tokens, two of them to a group of 32 keys, `gap` powers of two apart."""
    exps = [-7, -7 - gap] * 4 if place == "in_a_group" else [-7, -7, -7 - gap, -7 - gap] * 2
    exps = torch.tensor(exps if order == "down" else exps[::-1])
    cache = clone(filled(8, 2, 16, 64, seed=gap), "cuda")
    cache.v_scale.copy_((2.0 ** exps)[:, None].expand(8, 2))
    q = torch.randn((1, 8, Nq, 64), generator=torch.Generator().manual_seed(gap)).cuda().to(dtype) * 0.7
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None].contiguous()
    compare(q, cache, table, torch.tensor([125], dtype=torch.int32, device="cuda"))


def weighed(T, dtype, Nq, codes, exps, B=1, Hkv=2, seed=0):
    """q, cache, table for B sequences: a key of block j scores 20 codes[b][j] bits above one of code 0
    in every second query row (0 in the others, but for some noise), its block's value scale is
    2^exps[b][j].  Every sequence has blocks of its own."""
    gen = torch.Generator().manual_seed(seed)
    codes, exps = torch.tensor(codes).view(B, -1), torch.tensor(exps).view(B, -1)
    nb, d = codes.shape[1], 64
    cache = filled(B * nb, Hkv, T, d, seed=seed)
    k = torch.randn((B * nb, Hkv, T, d), generator=gen) / 4
    k[..., 0] = codes.reshape(-1, 1, 1).float()
    cache.k.copy_(k.to(torch.float8_e4m3fn))
    cache.k_scale.fill_(1)
    cache.v_scale.copy_((2.0 ** exps).reshape(-1, 1).expand(-1, Hkv))
    q = torch.randn((B, 4 * Hkv, Nq, d), generator=gen)
    q[..., 0] = 0
    q[:, ::2, :, 0] = 20 * 0.6931 * d ** 0.5
    table = torch.arange(B * nb, dtype=torch.int32).view(B, nb)
    return q.cuda().to(dtype), clone(cache, "cuda"), table.cuda()


def order_of(name, n, seed=0):
    """Seven codes over n blocks."""
    x = torch.arange(n) * 7 // n
    if name == "falling":
        x = x.flip(0)
    elif name == "mixed":
        x = x[torch.randperm(n, generator=torch.Generator().manual_seed(seed))]
    elif name == "turns":
        x = torch.arange(n) % 2 * 6
    return x.tolist()


@DTYPES
@ROWS
@pytest.mark.parametrize("order", ["rising", "falling", "mixed", "turns"])
@pytest.mark.parametrize("T", [16, 64])
def test_small_values_of_large_weight(T, order, Nq, dtype):
    """Weights from 2^-120 to 1 on values from 2^20 to 2^-100: in every second row each block adds as
    much to the output as any other, in the rest the large values are all that counts."""
    codes = order_of(order, 448 // T)
    q, cache, table = weighed(T, dtype, Nq, codes, [20 - 20 * c for c in codes])
    compare(q, cache, table, torch.tensor([448 - 5], dtype=torch.int32, device="cuda"))


@DTYPES
@ROWS
@pytest.mark.parametrize("T", [16, 64])
def test_scales_within_a_long_stretch(T, Nq, dtype):
    """So many keys that a warp's stretch spans blocks of several scales: 2^-40 to 2^20 by the weights,
    and by chance up to 2^4 beside that."""
    B, Hkv, n = 8, 4, 4096
    gen = torch.Generator().manual_seed(T)
    codes = torch.randint(0, 4, (B, n // T), generator=gen)
    exps = 20 - 20 * codes + torch.randint(-4, 5, codes.shape, generator=gen)
    q, cache, table = weighed(T, dtype, Nq, codes.tolist(), exps.tolist(), B, Hkv, seed=T)
    lens = torch.arange(n - 7 * B, n, 7, dtype=torch.int32, device="cuda")
    compare(q, cache, table, lens)


@DTYPES
@pytest.mark.parametrize("size", [1e-18, 1e-25])
def test_tiny_values(size, dtype):
    """Appended and attended: scales down to 2^-91 where nothing else has been seen."""
    gen = torch.Generator().manual_seed(1)
    k, v = (torch.randn((2, 2, 200, 64), generator=gen).cuda().to(dtype) for _ in range(2))
    cache = lap.cache_alloc(8, 2, 64, 64)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    lens = torch.tensor([200, 70], dtype=torch.int32, device="cuda")
    lap.cache_append(cache, k, v * size, table, torch.zeros_like(lens), lens)
    q = torch.randn((2, 8, 1, 64), generator=gen).cuda().to(dtype)
    out = compare(q, cache, table, lens)
    assert bool((out != 0).any(-1).all())


@DTYPES
@ROWS
@pytest.mark.parametrize("T", [16, 128])
def test_the_values_unit_does_not_matter(T, Nq, dtype):
    """Values 2^n times as large give an output 2^n times as large, bit for bit."""
    gen = torch.Generator().manual_seed(T)
    cache = clone(filled(1536 // T, 2, T, 64, seed=T), "cuda")
    table = torch.randperm(1536 // T, generator=gen).to(torch.int32).view(2, -1).cuda()
    lens = torch.tensor([765, 300], dtype=torch.int32, device="cuda")
    q = (torch.randn((2, 8, Nq, 64), generator=gen) * 4).cuda().to(dtype)
    want = lap.cache_attention(q, cache, table, lens)
    for n in (-80, -20, -9, 20, 70):
        other = cache._replace(v_scale=cache.v_scale * 2.0 ** n)
        assert torch.equal(lap.cache_attention(q, other, table, lens).double() * 2.0 ** -n, want.double()), n


def compare_many(B, q, cache, table, lens):
    """The same for B sequences alike, over the same blocks (so many that a warp takes long stretches)."""
    k, v = gathered(cache, table)
    ref = reference(q, k, v, -1, 0, 0, None, lens, lens - q.shape[2], extra_p=2.0 ** -21,
                    extra_s=2.0 ** -22 * 8)["out"]
    q, table, lens = (x.expand(B, *x.shape[1:]).contiguous() for x in (q, table, lens))
    check("out", lap.cache_attention(q, cache, table, lens), [x.expand(q.shape) for x in ref])


@DTYPES
@ROWS
def test_a_long_tail_of_small_values(Nq, dtype):
    """One token of weight 1 and 65536 of 2^-20, 6 % of the sum, at scales of 2^-16; a warp takes some
    18000 keys."""
    T, nb = 128, 513
    q, cache, table = weighed(T, dtype, Nq, [1] + [0] * (nb - 1), [-16] * nb, Hkv=8)
    cache.k.view(torch.uint8)[0, :, 1:, 0] = 0          # one token of the first block alone
    cache.v.view(torch.uint8).fill_(0x38)               # all values 1 ..
    cache.v.view(torch.uint8)[0, :, 0, :] = 0xB8        # .. but that token's, -1
    compare_many(64, q, cache, table, torch.tensor([nb * T], dtype=torch.int32, device="cuda"))


@DTYPES
@ROWS
@pytest.mark.parametrize("small", [-45, -70])
def test_weights_that_rise_little_by_little(small, Nq, dtype):
    """A block of ordinary values, then small ones whose weights rise by half a bit a block: after 120
    blocks they are all that counts (2^-45 beside 2^-59), or the first block is (2^-70)."""
    T, nb = 16, 121
    q, cache, table = weighed(T, dtype, Nq, [0] * nb, [0] + [small] * (nb - 1), Hkv=8)
    level = torch.arange(nb, device="cuda").view(-1, 1, 1) / 40
    k = cache.k.float()
    k[..., 0], k[..., 1] = level.floor(), (level - level.floor())   # the sum rises by 20 / 40 bits
    q[..., 1] = q[..., 0]
    cache = cache._replace(k=k.to(torch.float8_e4m3fn))
    compare_many(512, q, cache, table, torch.tensor([nb * T], dtype=torch.int32, device="cuda"))


@DTYPES
def test_a_negative_scale_turns_the_sign(dtype):
    """Not what cache_append stores, but a cache of a user's own: its scales are factors."""
    cache = clone(filled(8, 2, 16, 64), "cuda")
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None].contiguous()
    lens = torch.tensor([125], dtype=torch.int32, device="cuda")
    q = torch.randn((1, 8, 1, 64), generator=torch.Generator().manual_seed(2)).cuda().to(dtype)
    want = lap.cache_attention(q, cache, table, lens)
    assert torch.equal(lap.cache_attention(q, cache._replace(v_scale=-cache.v_scale), table, lens), -want)
    cache.v_scale[::2] *= -1.5
    compare(q, cache, table, lens)
