"""Windowed attention (forward, backward, few tokens) against the plain 64-bit form; the allowed
errors are derived in tests/_window_ref.py."""
import pytest
import torch

import laplacian_nystr_linear_gb300 as lap

from tests._window_ref import check, reference

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def make(B, Hq, Hkv, Nq, Nk, d, dtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(1000 * Nq + 10 * d + B + seed)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    q, k, v, do = r(B, Hq, Nq, d), r(B, Hkv, Nk, d), r(B, Hkv, Nk, d), r(B, Hq, Nq, d)
    k = k + 0.5 * r(1, Hkv, 1, d)
    return [x.to(dtype) for x in (q, k, v, do)]


def ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


# B, Hq, Hkv, Nq, Nk, d, left, right, sinks, lens, q_pos
CASES = {
    "one_key": (1, 1, 1, 1, 1, 16, 0, 0, 0, None, None),
    "self_only": (2, 2, 1, 33, 33, 32, 0, 0, 0, None, None),
    "causal_all": (1, 2, 2, 200, 200, 64, -1, 0, 0, None, None),
    "both_all": (2, 3, 1, 130, 130, 48, -1, -1, 0, None, None),
    "window": (1, 4, 2, 517, 517, 64, 100, 0, 4, None, None),
    "window_128": (1, 2, 1, 700, 700, 128, 255, 0, 4, None, None),
    "two_sided": (2, 2, 2, 301, 301, 80, 37, 90, 1, None, None),
    "right_only": (1, 1, 1, 260, 260, 112, 0, 70, 3, None, None),
    "many_first": (1, 2, 1, 600, 600, 64, 63, 0, 200, None, None),
    "first_touch": (1, 2, 2, 300, 300, 96, 64, 5, 64, None, None),
    "ragged": (4, 4, 2, 190, 190, 64, 40, 10, 2, [190, 0, 1, 97], None),
    "ragged_128": (3, 2, 2, 384, 384, 128, -1, 0, 0, [384, 129, 128], None),
    "lens_odd_values": (3, 1, 1, 70, 70, 32, 20, 0, 1, [-5, 1000, 35], None),
    "chunk": (2, 4, 4, 100, 400, 64, 150, 0, 4, None, None),
    "chunk_positions": (3, 2, 1, 64, 300, 128, 90, 7, 4, [300, 150, 280], [236, 120, -20]),
    "positions_off": (2, 2, 2, 40, 100, 16, 30, 0, 0, [100, 50], [90, 2000000000]),
    "group_8": (1, 16, 2, 140, 140, 128, 64, 0, 4, None, None),
    "queries_cut": (1, 8, 1, 700, 700, 64, -1, -1, 0, None, None),
    "queries_cut_causal": (2, 4, 1, 333, 333, 128, -1, 0, 4, [333, 200], None),
    "long_first": (1, 1, 1, 2500, 2500, 64, 50, 0, 4, None, None),
    "one_token": (3, 8, 2, 1, 777, 128, 300, 0, 4, [777, 1, 300], [776, 0, 299]),
    "one_token_64": (2, 4, 4, 1, 1000, 64, -1, 0, 0, None, None),
    "five_tokens": (2, 6, 2, 5, 515, 96, 200, 2, 17, [515, 200], [510, 195]),
    "one_token_empty": (3, 2, 1, 1, 50, 32, 8, 0, 1, [0, 50, 20], [0, 60, -1]),
    "rows_over_one_tile": (1, 24, 1, 3, 260, 48, -1, 0, 0, None, None),
}


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("name", list(CASES))
def test_forward_and_backward(name, dtype):
    B, Hq, Hkv, Nq, Nk, d, left, right, sinks, lens, q_pos = CASES[name]
    q, k, v, do = make(B, Hq, Hkv, Nq, Nk, d, dtype)
    lens, q_pos = ints(lens), ints(q_pos)
    if lens is not None:   # behind a sequence: anything
        for b in range(B):
            n = max(0, int(lens[b]))
            k[b, :, n:] = float("nan")
            v[b, :, n:] = float("inf")
            if Nq == Nk:
                q[b, :, n:] = float("nan")
                do[b, :, n:] = float("nan")
    ref = reference(q, k, v, left, right, sinks, None, lens, q_pos, do)
    p = lap.WindowParams.of(q, k, left, right, sinks)
    out, lse = lap.window_fwd(q, k, v, p, lens, q_pos)
    check("out", out, ref["out"])
    check("lse", lse, ref["lse"])
    for name_, x in zip(("dq", "dk", "dv"), lap.window_bwd(q, k, v, out, do, lse, p, lens, q_pos)):
        check(name_, x, ref[name_])


@pytest.mark.parametrize("name", list(CASES))
def test_rest_of_the_output(name):
    """out + rest is the output before its rounding, and the gradients are the nearer for it."""
    B, Hq, Hkv, Nq, Nk, d, left, right, sinks, lens, q_pos = CASES[name]
    q, k, v, do = make(B, Hq, Hkv, Nq, Nk, d, BF)
    lens, q_pos = ints(lens), ints(q_pos)
    ref = reference(q, k, v, left, right, sinks, None, lens, q_pos, do, rest=True)
    p = lap.WindowParams.of(q, k, left, right, sinks)
    rest = torch.full_like(q, float("nan"))
    out, lse = lap.window_fwd(q, k, v, p, lens, q_pos, rest=rest)
    assert torch.equal(out, lap.window_fwd(q, k, v, p, lens, q_pos)[0])
    check("both", out.double() + rest.double(), ref["both"])
    for name_, x in zip(("dq", "dk", "dv"),
                        lap.window_bwd(q, k, v, out, do, lse, p, lens, q_pos, rest=rest)):
        check(name_, x, ref[name_])


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_autograd_agrees_with_differences(dtype):
    """<grad, step> against the 64-bit loss's central difference along the same step.  The truncation
    is of order h^2 = 1e-8 of the third derivative; what remains is the gradient's allowed error."""
    q, k, v, do = make(2, 4, 2, 90, 90, 64, dtype)
    args = dict(left=30, right=5, sinks=2)
    leaves = [x.detach().requires_grad_(True) for x in (q, k, v)]
    grads = torch.autograd.grad(lap.window_attention(*leaves, **args), leaves, do)
    ref = reference(q, k, v, 30, 5, 2, dout=do)
    h = 1e-4
    for i, name in enumerate(("dq", "dk", "dv")):
        step = torch.randn(grads[i].shape, dtype=torch.float64, device="cuda")
        loss = []
        for sgn in (1, -1):
            x = [t.double() for t in (q, k, v)]
            x[i] = x[i] + sgn * h * step
            s = x[0] @ x[1].repeat_interleave(2, 1).transpose(-1, -2) / 8
            j, p = torch.arange(90, device="cuda")[None], torch.arange(90, device="cuda")[:, None]
            s = s.masked_fill(~((j <= p + 5) & ((j >= p - 30) | (j < 2))), float("-inf"))
            loss.append(float(((torch.softmax(s, -1) @ x[2].repeat_interleave(2, 1)) * do.double()).sum()))
        want = (loss[0] - loss[1]) / (2 * h)
        off = float((ref[name][1] * step.abs()).sum()) + 1e-5 * abs(want) + 1e-4
        assert abs(float((grads[i].double() * step).sum()) - want) <= off


@pytest.mark.parametrize("fill", ["lowest", "large"])
def test_scores_of_extreme_size(fill):
    """Scores far apart (up to 1e4) and keys of the type's lowest value: one key takes all."""
    q, k, v, _ = make(1, 2, 1, 64, 200, 64, BF)
    if fill == "large":
        q, k = q * 64, k * 64
    else:
        q[:] = 0
        k[:, :, 10:20] = torch.finfo(BF).min
    ref = reference(q, k, v, 50, 0, 4)
    out = lap.window_attention(q, k, v, 50, 0, 4)
    if fill == "lowest":   # 0 * lowest = 0: every score is 0, the scores' error as well
        ref["out"] = (ref["out"][0], 2.0 ** -7 * v.float().abs().amax().double().expand_as(ref["out"][0]))
    check("out", out, ref["out"])


def test_streams_graphs_and_two_at_once():
    q, k, v, do = make(2, 4, 2, 300, 300, 64, BF)
    a = dict(left=60, right=0, sinks=4)

    def step():
        leaves = [x.detach().requires_grad_(True) for x in (q, k, v)]
        o = lap.window_attention(*leaves, **a)
        return [o.detach(), *torch.autograd.grad(o, leaves, do)]

    want = [x.clone() for x in step()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(step())
    torch.cuda.synchronize()
    for r in got:
        for x, y in zip(r, want):
            assert torch.equal(x, y)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = step()
        graphs.append((g, r))
    for x in (q, k, v, do):
        x.copy_(torch.roll(x, 1, 0))
    want = [x.clone() for x in step()]
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    for _, r in graphs:
        for x, y in zip(r, want):
            assert torch.equal(x, y)


def test_shared_inputs_partial_gradients_and_second_order():
    """One tensor as queries, keys and values; gradients asked of some inputs only; a broadcast
    output gradient; second derivatives are refused."""
    q, k, v, _ = make(2, 2, 2, 70, 70, 32, BF)
    a = dict(left=20, right=3, sinks=1)
    ones = torch.ones_like(q)
    p = lap.WindowParams.of(q, k, 20, 3, 1)

    def grads(q, k, v):
        rest = torch.empty_like(q)
        out, lse = lap.window_fwd(q, k, v, p, rest=rest)
        return lap.window_bwd(q, k, v, out, ones, lse, p, rest=rest)

    x = q.detach().requires_grad_(True)
    lap.window_attention(x, x, x, **a).sum().backward()
    parts = [g.float() for g in grads(q, q, q)]
    # two sums of bf16 values, each rounded (2^-8 of at most the magnitudes' sum)
    assert bool(((x.grad.float() - sum(parts)).abs() <= 2.0 ** -6 * sum(g.abs() for g in parts)).all())
    want = grads(q, k, v)
    for i in range(3):
        t = [y.detach().requires_grad_(j == i) for j, y in enumerate((q, k, v))]
        lap.window_attention(*t, **a).sum().backward()
        assert torch.equal(t[i].grad, want[i])
        assert all(y.grad is None for j, y in enumerate(t) if j != i)
    y = q.detach().requires_grad_(True)
    g, = torch.autograd.grad(lap.window_attention(y, k, v, **a).sum(), y, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_guarded_outputs_and_repeatability():
    """Every output element is written, nothing beside it, and twice the same."""
    for Nq, Nk in ((150, 150), (1, 150)):
        q, k, v, do = make(2, 4, 2, Nq, Nk, 80, BF)
        p = lap.WindowParams.of(q, k, 33, 0, 3)

        def guarded(like):
            pad = 64
            buf = torch.full((like.numel() + 2 * pad,), 7.0, dtype=like.dtype, device="cuda")
            t = buf[pad:pad + like.numel()].view(like.shape)
            t.fill_(float("nan"))
            return buf, t, pad

        runs = []
        for _ in range(2):
            bo, out, pad = guarded(q)
            _, lse = lap.window_fwd(q, k, v, p, out=out)
            bufs = [guarded(x) for x in (q, k, v)]
            lap.window_bwd(q, k, v, out, do, lse, p, dq=bufs[0][1], dk=bufs[1][1], dv=bufs[2][1])
            for buf, t, _ in [(bo, out, pad)] + bufs:
                assert bool(torch.isfinite(t).all())
                assert bool((buf[:pad] == 7).all()) and bool((buf[-pad:] == 7).all())
            runs.append([out] + [b[1] for b in bufs])
        for x, y in zip(*runs):
            assert torch.equal(x, y)


def test_long_sums_of_fp32():
    """One query over 2.9 M keys: its parts add up some 300 groups of 16 keys each, the parts (of 608
    warps, four at a time) some 150.  Sums rounded to nearest walk at random: with n = 450 steps of
    numerator and of denominator, each off by 2^-24 at most (uniform: a third of its square), four
    standard deviations are below 4 sqrt(2 n) 2^-24.  Sums that are cut off drift by n 2^-24 and more."""
    n, d = 608 * 16 * 300, 16
    gen = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.rand(s, generator=gen, device="cuda")  # noqa: E731
    q, k, v = r(1, 1, 1, d) - 0.5, r(1, 1, n, d), 1 + r(1, 1, n, d)
    out = lap.window_attention(q, k, v, -1)
    s = (k[0, 0].double() @ q[0, 0, 0].double()) / 4
    want = torch.softmax(s, 0) @ v[0, 0].double()
    assert float((out[0, 0, 0].double() / want - 1).abs().max()) <= 4 * (2 * 450) ** 0.5 * 2.0 ** -24


def test_long_offsets():
    """Keys beyond 2^31 elements: the last of many sequences."""
    B, Nk, d = 2, 2 ** 23 + 40, 128
    k = torch.zeros((B, 1, Nk, d), dtype=BF, device="cuda")
    q, kk, v, _ = make(B, 2, 1, 100, 600, d, BF)
    k[:, :, -600:] = kk
    vv = torch.zeros_like(k)
    vv[:, :, -600:] = v
    for n in (100, 1):
        qn = q[:, :, :n].contiguous()
        ref = reference(qn, kk, v, 200, 0, 0)
        check("out", lap.window_attention(qn, k, vv, 200, 0, 0), ref["out"])
