"""The 8-bit cache: appended values bit for bit, attention over them against the plain 64-bit form
(allowed errors: tests/_window_ref.py, on the values that the cache stands for)."""
import math

import pytest
import torch

import laplacian_nystr_linear_gb300 as lap
from laplacian_nystr_linear_gb300 import _lib, api

from tests._window_ref import check, reference

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    assert api.device_status(clear=True) == _lib.LAPNYS_OK


def scale_of(amax):
    """2^ceil(log2(amax / 448)), by whole numbers."""
    if amax == 0:
        return 2.0 ** -100
    m, e = math.frexp(amax)          # amax = m 2^e, 448 = 0.875 2^9
    return 2.0 ** max(-100, e - 9 + (1 if m > 0.875 else 0))


def append_ref(cache, k, v, table, start, lens):
    """cache_append on the host in python floats and torch's own rounding."""
    T = cache.k.shape[2]
    for x8, xs, x in ((cache.k, cache.k_scale, k), (cache.v, cache.v_scale, v)):
        B, H, N, d = x.shape
        for b in range(B):
            end = min(start[b] + N, table.shape[1] * T, 1 << 30 if lens is None else lens[b])
            for lb in range(max(start[b], 0) // T, (max(end, 1) - 1) // T + 1):
                fs, fe = max(start[b], lb * T, 0), min(end, lb * T + T)
                if fs >= fe:
                    continue
                blk, held = int(table[b, lb]), max(0, fs - lb * T) if start[b] > lb * T else 0
                for h in range(H):
                    new = x[b, h, fs - start[b]:fe - start[b]].float()
                    fin = new[torch.isfinite(new)].abs()
                    s = scale_of(float(fin.max()) if fin.numel() else 0.0)
                    if held:
                        s = max(s, float(xs[blk, h]))
                        old = x8[blk, h, :held].float() * (float(xs[blk, h]) / s)
                        x8[blk, h, :held] = old.to(torch.float8_e4m3fn)
                    xs[blk, h] = s
                    x8[blk, h, fs - lb * T:fe - lb * T] = (new / s).clamp(-448, 448).to(torch.float8_e4m3fn)


def values(cache):
    return [(x.float() * s[..., None, None]) for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]


def clone(cache, device=None):
    return lap.KVCache(*(x.detach().clone().to(device or x.device) for x in cache))


def equal(a, b):
    for x, y in zip(a, b):
        x, y = x.cpu(), y.cpu()
        if x.dtype == torch.float8_e4m3fn:
            x, y = x.view(torch.uint8), y.view(torch.uint8)
        assert torch.equal(x, y)


def filled(blocks, H, T, d, seed=0):
    """A cache whose every slot holds something."""
    g = torch.Generator().manual_seed(seed)
    c = lap.cache_alloc(blocks, H, d, T, device="cpu")
    for x8, xs in ((c.k, c.k_scale), (c.v, c.v_scale)):
        x8.copy_((torch.randn(x8.shape, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn))
        xs.copy_(2.0 ** torch.randint(-9, -5, xs.shape, generator=g))
    return c


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,d,N,start,lens", [
    (16, 16, 1, [0, 5, 15], None),
    (32, 48, 3, [31, 30, 0], [34, 31, 0]),
    (64, 128, 70, [0, 63, 100], None),
    (128, 112, 200, [1, 128, 255], [120, 300, 400]),
    (16, 64, 40, [-10, -40, 3], None),
    (64, 128, 5, [190, 188, 1000], None),      # the table ends at 192
])
def test_append(T, d, N, start, lens, dtype):
    g = torch.Generator().manual_seed(T + N)
    H, nb = 2, 192 // T if N < 10 and T == 64 else 448 // T + 1
    c = filled(3 * nb + 2, H, T, d)
    table = torch.randperm(3 * nb + 2, generator=g)[:3 * nb].reshape(3, nb).to(torch.int32)
    k = (torch.randn((3, H, N, d), generator=g) * torch.tensor([1e-3, 1.0, 300.0]).view(3, 1, 1, 1)).to(dtype)
    v = torch.randn((3, H, N, d), generator=g).to(dtype)
    v[0] = 0
    v[1, :, 0, 0], v[1, :, 0, 1], v[1, :, 0, 2] = float("inf"), float("-inf"), float("nan")
    want, got = clone(c), clone(c, "cuda")
    append_ref(want, k, v, table, start, lens)
    i = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    lap.cache_append(got, k.cuda(), v.cuda(), table.cuda(), i(start), i(lens))
    equal(got, want)


def test_append_token_by_token():
    """One token at a time gives one call's values but for what becomes subnormal at a larger scale:
    within 2^-10 of 2^-6 scales, so 2^-9 / 2 scales a re-rounding, at most 3 of them here."""
    H, T, d, n = 2, 32, 64, 100
    k = torch.randn((1, H, n, d), device="cuda") * torch.linspace(0.5, 4, n, device="cuda").view(1, 1, n, 1)
    v = torch.randn((1, H, n, d), device="cuda")
    table = torch.tensor([[3, 0, 2, 1]], dtype=torch.int32, device="cuda")
    one, many = lap.cache_alloc(4, H, d, T), lap.cache_alloc(4, H, d, T)
    at = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")  # noqa: E731
    lap.cache_append(one, k, v, table, at(0))
    for t in range(n):
        lap.cache_append(many, k[:, :, t:t + 1].contiguous(), v[:, :, t:t + 1].contiguous(), table, at(t))
    assert torch.equal(one.k_scale, many.k_scale) and torch.equal(one.v_scale, many.v_scale)
    for x, y, s in zip(values(one), values(many), (one.k_scale, one.v_scale)):
        assert bool(((x - y).abs() <= 3 * 2.0 ** -10 * s[..., None, None]).all())


# B, Hq, Hkv, Nq, d, T, left, right, sinks, lens, q_pos
CASES = {
    "one": (1, 1, 1, 1, 16, 16, -1, 0, 0, [1], None),
    "batch": (4, 8, 2, 1, 128, 64, -1, 0, 0, [700, 64, 65, 1], None),
    "window": (3, 4, 4, 1, 64, 32, 100, 0, 4, [600, 90, 3], None),
    "empty": (3, 4, 2, 2, 96, 16, 30, 0, 1, [0, 1, 40], None),
    "few": (2, 6, 2, 4, 112, 128, -1, 0, 0, [513, 300], None),
    "positions": (3, 2, 1, 3, 80, 16, 50, 7, 20, [200, 180, 150], [100, 178, -1]),
    "rows_over_one_tile": (2, 16, 1, 3, 128, 64, 200, 0, 5, [400, 333], None),
    "prompt": (2, 4, 2, 90, 64, 64, 64, 0, 4, [300, 90], None),
    "long": (2, 8, 1, 1, 128, 64, -1, 0, 0, [20000, 7], None),
}


def gathered(cache, table):
    t = table.long()
    return [x[t].transpose(1, 2).reshape(t.shape[0], x.shape[1], -1, x.shape[3]) for x in values(cache)]


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("name", list(CASES))
def test_attention(name, dtype):
    B, Hq, Hkv, Nq, d, T, left, right, sinks, lens, q_pos = CASES[name]
    nb = -(-max(lens) // T)
    cache = clone(filled(B * nb + 3, Hkv, T, d, seed=nb), "cuda")
    g = torch.Generator().manual_seed(7)
    table = torch.randperm(B * nb + 3, generator=g)[:B * nb].reshape(B, nb).to(torch.int32).cuda()
    q = torch.randn((B, Hq, Nq, d), generator=g).cuda().to(dtype) * 0.7
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    pos = n - Nq if q_pos is None else torch.tensor(q_pos, dtype=torch.int32, device="cuda")
    k, v = gathered(cache, table)
    # q is held to 2^-22 of its row's largest feature (score error scale |q|max sum |k|, as mag times
    # d at the very most), P to 2^-22 of itself and 2^-35 of the row's largest
    ref = reference(q.float() if dtype == F32 else q, k.to(dtype), v.to(dtype), left, right, sinks, None,
                    n, pos, extra_p=2.0 ** -21, extra_s=2.0 ** -22 * 8)
    # what lies behind a sequence, in its blocks and in its table, may be anything
    for b in range(B):
        if lens[b] % T:
            cache.k.view(torch.uint8)[table[b, lens[b] // T].long(), :, lens[b] % T:] = 0x7F
            cache.v.view(torch.uint8)[table[b, lens[b] // T].long(), :, lens[b] % T:] = 0x7F
        table[b, -(-lens[b] // T):] = -1 if b % 2 else 10 ** 9
    out = lap.cache_attention(q, cache, table, n, left, right, sinks,
                              q_pos=None if q_pos is None else pos)
    check("out", out, ref["out"])


def test_blocks_outside_the_window_are_not_read():
    T, n = 16, 400
    cache = clone(filled(30, 1, T, 64), "cuda")
    table = torch.arange(25, dtype=torch.int32, device="cuda")[None].contiguous()
    q = torch.randn((1, 2, 1, 64), device="cuda", dtype=BF)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    want = lap.cache_attention(q, cache, table, lens, left=50, sinks=4)
    table[0, 1:(n - 51) // T] = -7
    cache.k.view(torch.uint8)[1:(n - 51) // T] = 0x7F
    assert torch.equal(lap.cache_attention(q, cache, table, lens, left=50, sinks=4), want)


def test_blocks_that_are_not_there():
    """Reported, never read or written; the other sequences' results stay."""
    T, d = 16, 32
    cache = clone(filled(12, 2, T, d), "cuda")
    table = torch.arange(12, dtype=torch.int32, device="cuda").reshape(2, 6)
    q = torch.randn((2, 4, 1, d), device="cuda", dtype=BF)
    lens = torch.tensor([90, 90], dtype=torch.int32, device="cuda")
    good = lap.cache_attention(q, cache, table, lens)
    for bad in (12, -1, 2 ** 31 - 1):
        t = table.clone()
        t[0, 2] = bad
        out = lap.cache_attention(q, cache, t, lens)
        assert api.device_status(clear=True) == _lib.LAPNYS_EPAGE
        assert torch.equal(out[1], good[1])
        k, v = gathered(cache, table[:1])
        keep = [j for j in range(90) if j // T != 2]
        ref = reference(q[:1], k[:, :, keep].to(BF), v[:, :, keep].to(BF), -1, 0, 0)
        check("out", out[:1], ref["out"])
        before = clone(cache)
        x = torch.randn((2, 2, 1, d), device="cuda", dtype=BF)
        lap.cache_append(cache, x, x, t, torch.tensor([40, 40], dtype=torch.int32, device="cuda"))
        assert api.device_status(clear=True) == _lib.LAPNYS_EPAGE
        assert torch.equal(cache.k[:6].view(torch.uint8), before.k[:6].view(torch.uint8))
        assert not torch.equal(cache.k[8].view(torch.uint8), before.k[8].view(torch.uint8))
        cache = before


def test_long_offsets():
    """A cache of over 2^32 bytes: its last blocks."""
    T, d, H = 128, 128, 8
    blocks = 2 ** 32 // (T * d * H) + 3
    cache = lap.cache_alloc(blocks, H, d, T)
    table = torch.tensor([[blocks - 1, blocks - 2]], dtype=torch.int32, device="cuda")
    k, v = (torch.randn((1, H, 200, d), device="cuda", dtype=BF) for _ in range(2))
    n = torch.tensor([200], dtype=torch.int32, device="cuda")
    lap.cache_append(cache, k, v, table, torch.zeros_like(n))
    small = lap.KVCache(*(x[-2:].contiguous() for x in cache))
    q = torch.randn((1, H, 1, d), device="cuda", dtype=BF)
    ts = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    assert torch.equal(lap.cache_attention(q, cache, table, n), lap.cache_attention(q, small, ts, n))
    ks, _ = gathered(small, ts)
    assert float((ks[:, :, :200] - k.float()).abs().max()) <= 2.0 ** -4 * float(k.float().abs().max())


def test_prompt_then_tokens_as_a_user_runs_them():
    """A prompt through window_attention and into the cache, then tokens one by one in a captured
    graph; each answer against the plain form over the values that the cache holds."""
    B, Hq, Hkv, d, T, n0 = 2, 8, 2, 64, 32, 150
    left, sinks = 63, 4
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda").to(BF)  # noqa: E731
    q, k, v = r(B, Hq, n0, d), r(B, Hkv, n0, d), r(B, Hkv, n0, d)
    lens = torch.tensor([n0, 101], dtype=torch.int32, device="cuda")
    out = lap.window_attention(q, k, v, left, 0, sinks, lens=lens)
    check("out", out, reference(q, k, v, left, 0, sinks, None, lens)["out"])
    cache = lap.cache_alloc(20, Hkv, d, T)
    table = torch.randperm(20, generator=gen, device="cuda")[:16].reshape(B, 8).to(torch.int32)
    lap.cache_append(cache, k, v, table, torch.zeros_like(lens), lens)
    q1, k1, v1 = r(B, Hq, 1, d), r(B, Hkv, 1, d), r(B, Hkv, 1, d)
    count, start = lens.clone(), lens.clone()

    def token():
        start.copy_(count)
        count.add_(1)
        lap.cache_append(cache, k1, v1, table, start, count)
        return lap.cache_attention(q1, cache, table, count, left, 0, sinks)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        answer = token()
    for _ in range(40):
        for x in (q1, k1, v1):
            x.copy_(r(*x.shape))
        graph.replay()
        kk, vv = gathered(cache, table)
        ref = reference(q1, kk.to(BF), vv.to(BF), left, 0, sinks, None, count, count - 1)
        check("out", answer, ref["out"])
    assert count.tolist() == [n0 + 40, 141]
