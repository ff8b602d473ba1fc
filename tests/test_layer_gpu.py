"""The operators of a layer together, as they are used: norms and residuals around an attention and the
gated feed-forward block; a prompt and single tokens over the 8-bit cache with rotary positions."""
import pytest
import torch

import laplacian_nystr_linear_gb300 as lap

pytestmark = pytest.mark.gpu


def _plain_norm(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w


def test_two_blocks_train():
    """x -> attention block -> feed-forward block against the same layer with plain norms and products."""
    B, gh, gw, C, H, Fh, m = 2, 16, 16, 128, 2, 200, 16
    N = gh * gw
    gen = torch.Generator(device="cuda").manual_seed(0)
    r = lambda s, *shape: torch.randn(shape, generator=gen, device="cuda") * s  # noqa: E731
    par = dict(n1=1 + r(0.1, C), n2=1 + r(0.1, C), n3=1 + r(0.1, C), s1=0.5 + r(0.1, C), s2=0.5 + r(0.1, C),
               w_qkv=r(C ** -0.5, C, 3 * C), w_o=r(C ** -0.5, C, C), w_in=r(C ** -0.5, C, 2 * Fh),
               w_out=r(Fh ** -0.5, Fh, C))
    x, d = r(1.0, B, N, C), r(1.0, B, N, C)

    def attend(y, p):
        return lap.attention_block(y, p["w_qkv"], None, p["w_o"], None, grid=(gh, gw), heads=H, m=m, iters=12)

    def ours(x, p):
        _, y = lap.residual_norm(x, None, p["n1"])
        h, y = lap.residual_norm(x, attend(y, p), p["n2"], scale=p["s1"])
        h, y = lap.residual_norm(h, lap.gated_mlp(y, p["w_in"], None, p["w_out"], None), p["n3"], scale=p["s2"])
        return h, y

    def plain(x, p):
        h = x + attend(_plain_norm(x, p["n1"]).contiguous(), p) * p["s1"]
        z = _plain_norm(h, p["n2"]) @ p["w_in"]
        h = h + ((torch.nn.functional.silu(z[..., :Fh]) * z[..., Fh:]) @ p["w_out"]) * p["s2"]
        return h, _plain_norm(h, p["n3"])

    out = []
    for f in (ours, plain):
        leaves = {n: v.clone().requires_grad_(True) for n, v in par.items()}
        xl = x.clone().requires_grad_(True)
        h, y = f(xl, leaves)
        out.append([h, y, *torch.autograd.grad((h * d).sum() + (y * d).sum(), [xl, *leaves.values()])])
    # the attention's own fp32 tolerance against 64 bits, on both sides of the comparison
    for n, a, b in zip(["h", "y", "x", *par], *out):
        assert float((a - b).detach().norm() / b.detach().norm()) < 2e-4, n


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_prompt_then_tokens(layout):
    """Turned keys of a prompt and of single tokens, through the cache, against all at once through
    window_attention; the cache holds e4m3 of at most 2^-4 off, which bounds the scores' and values' errors."""
    B, Hq, Hkv, d, N, new = 2, 4, 2, 64, 50, 3
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn((B, h, N + new, d), generator=gen, device="cuda").bfloat16() for h in (Hq, Hkv, Hkv))
    f = lap.rotary_frequencies(d, scaling="linear", factor=2.0)
    qt, kt = lap.rotary(q, k, f, layout=layout)
    cache = lap.cache_alloc(16, Hkv, d, 16)
    table = torch.arange(16, dtype=torch.int32, device="cuda").view(B, 8)
    at = lambda n: torch.full((B,), n, dtype=torch.int32, device="cuda")  # noqa: E731
    outs = []
    for lo, hi in ((0, N), *((N + i, N + i + 1) for i in range(new))):
        qs, ks = (t[:, :, lo:hi].contiguous() for t in (q, k))
        lap.rotary_apply(qs, ks, f, start=at(lo), layout=layout, q_out=qs, k_out=ks)
        assert torch.equal(qs, qt[:, :, lo:hi]) and torch.equal(ks, kt[:, :, lo:hi])
        lap.cache_append(cache, ks, v[:, :, lo:hi].contiguous(), table, at(lo), at(hi))
        if lo:
            outs.append(lap.cache_attention(qs, cache, table, at(hi)))
    held = [c.float() * s[:, :, None, None] for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
    ck, cv = (h.view(B, 8, Hkv, 16, d).transpose(1, 2).reshape(B, Hkv, 128, d)[:, :, :N + new].contiguous()
              for h in held)
    want = lap.window_attention(qt.float().contiguous(), ck, cv, -1)[:, :, N:]
    assert float((torch.cat(outs, 2).float() - want).norm() / want.norm()) < 2.0 ** -7
