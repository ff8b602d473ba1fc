"""Sliding-window attention with first tokens that stay visible, and attention over a cache held
in 8 bits: the cases that are measured, their inputs, their plain forms in torch, and their values
in 64 bits.

A case is one of four calls:
  op "window"  window_attention forward (train False) or forward and backward (train True)
  op "append"  cache_append: new keys and values rounded into the cache's blocks
  op "cache"   cache_attention: a few tokens per sequence over the cache
Key j is visible to the query at position p of a sequence of n tokens iff
  0 <= p < n, j < n, j <= p + right and (j >= p - left or j < sinks);  -1: no bound.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
MIN_EXP = -100  # the smallest scale is 2 ** MIN_EXP


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _window(name, B, Hq, Hkv, Nq, Nk, d, left, right, sinks, dtype, train, ragged=False):
    return {"name": name, "op": "window", "B": B, "Hq": Hq, "Hkv": Hkv, "Nq": Nq, "Nk": Nk, "d": d,
            "left": left, "right": right, "sinks": sinks, "dtype": dtype, "train": train,
            "ragged": ragged}


def _cache(name, op, B, Hq, Hkv, Nq, n, T, d, left, sinks, dtype, ragged):
    return {"name": name, "op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "Nq": Nq, "Nk": n, "T": T, "d": d,
            "left": left, "right": 0, "sinks": sinks, "dtype": dtype, "ragged": ragged}


def listed():
    return [
        # a float32 training step on the smallest token grid (14 x 14), window over 3 grid rows
        _window("train_f32_196", 1, 1, 1, 196, 196, 32, 21, 21, 1, "float32", True),
        # inference on 56 x 56 token grids: local branch with one class token, both directions
        _window("grid_fwd_bf16", 32, 1, 1, 3136, 3136, 64, 112, 112, 1, "bfloat16", False),
        # a padded batch of odd length in training, both directions, heads that share keys
        _window("train_ragged_bf16", 4, 10, 5, 1001, 1001, 96, 100, 28, 2, "bfloat16", True, True),
        # causal training on long sequences (16384 tokens, heads of 64)
        _window("train_16k_bf16", 2, 16, 16, 16384, 16384, 64, 1023, 0, 4, "bfloat16", True),
        # causal training with shared keys, heads of 128
        _window("train_gqa_bf16", 1, 16, 4, 8192, 8192, 128, 2047, 0, 4, "bfloat16", True),
        # a long prompt
        _window("prompt_32k_bf16", 1, 8, 2, 32768, 32768, 128, 4095, 0, 4, "bfloat16", False),
        # one token of each sequence against plain keys and values
        _window("token_bf16", 16, 32, 8, 1, 4096, 128, 1023, 0, 4, "bfloat16", False, True),
        # one new token a sequence into the cache
        _cache("append_token", "append", 32, 8, 8, 1, 2049, 64, 128, -1, 0, "bfloat16", True),
        # a batch of prompts into the cache
        _cache("append_prompt", "append", 4, 8, 8, 4099, 4099, 64, 128, -1, 0, "bfloat16", True),
        # the smallest answer: one sequence, one shared head, window and first tokens
        _cache("cache_token_small", "cache", 1, 8, 1, 1, 2000, 16, 64, 511, 4, "float32", False),
        # an ordinary batch that answers, one token each
        _cache("cache_token_batch", "cache", 32, 32, 8, 1, 8192, 64, 128, -1, 0, "bfloat16", True),
        # a few tokens at once over long sequences
        _cache("cache_long", "cache", 4, 16, 4, 4, 131072, 64, 128, -1, 0, "bfloat16", True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window", "window", "train", "train", "token", "append", "cache", "cache"])
    d = rng.choice([16, 32, 48, 64, 64, 80, 96, 112, 128, 128])
    Hkv = _log_int(rng, 1, 8)
    g = rng.choice([1, 1, 2, 3, 4, 8])
    dtype = rng.choice(["bfloat16", "bfloat16", "bfloat16", "float32"])
    ragged = rng.random() < 0.5
    sinks = rng.choice([0, 1, 4, 4, rng.randint(5, 130)])
    if op in ("window", "train"):
        N = _log_int(rng, 2, 6000)
        B = _log_int(rng, 1, max(1, min(16, 20000 // (N * Hkv * g) + 1)))
        left = rng.choice([-1, _log_int(rng, 1, 2047)])
        right = rng.choice([0, 0, _log_int(rng, 1, 512) - 1, -1])
        whole, part = op == "train" or ragged or rng.random() < 0.7, rng.random()
        while True:
            Nq = N if whole else max(1, int(part * N))
            c = _window("", B, Hkv * g, Hkv, Nq, N, d, left, right, sinks, dtype, op == "train", ragged)
            if work(c)["flops"] < 2e11:
                return {k: v for k, v in c.items() if k != "name"}
            N = max(2, N * 3 // 4)
    if op == "token":
        N = _log_int(rng, 16, 16384)
        c = _window("", _log_int(rng, 1, 16), Hkv * g, Hkv, rng.choice([1, 1, 2, 5]), N, d,
                    rng.choice([-1, _log_int(rng, 1, 4096) - 1]), 0, sinks, dtype, False, ragged)
        return {k: v for k, v in c.items() if k != "name"}
    N = _log_int(rng, 1, 16384)
    Nq = min(N, rng.choice([1, 1, 1, 2, 4, 7]) if op == "cache" or rng.random() < 0.5
             else _log_int(rng, 1, 2048))
    c = _cache("", op, _log_int(rng, 1, 32), Hkv * g, Hkv, Nq, N, rng.choice([16, 32, 64, 128]), d,
               rng.choice([-1, _log_int(rng, 1, 4096) - 1]), sinks, dtype, ragged)
    return {k: v for k, v in c.items() if k != "name"}


def _lens(case):
    """Tokens of each sequence (known from the case alone)."""
    B, N = case["B"], case["Nk"]
    if not case["ragged"]:
        return [N] * B
    # the first is whole, the last one short; never fewer than the tokens of a cache call
    least = min(N, case["Nq"]) if case["op"] != "window" else 1
    return [max(least, N - (b * N * 3) // (4 * max(1, B - 1)) - (b % 3)) if b else N for b in range(B)]


def _pairs(case):
    """Visible (query, key) pairs of one head, summed over the batch."""
    total = 0
    for n in _lens(case):
        p0 = (n - case["Nq"]) if _q_at_end(case) else case["Nk"] - case["Nq"]
        left = n if case["left"] < 0 else case["left"]
        right = n if case["right"] < 0 else case["right"]
        for i in range(case["Nq"]):
            p = p0 + i
            if not 0 <= p < n:
                continue
            lo, hi = max(0, p - left), min(n - 1, p + right)
            total += hi - lo + 1 + min(case["sinks"], lo)
    return total


def _q_at_end(case):
    """Queries are the sequence's last tokens (single tokens), not the rows of a padded batch."""
    return case["op"] != "window" or (case["ragged"] and case["Nq"] < case["Nk"])


def work(case):
    e = 4 if case["dtype"] == "float32" else 2
    B, Hq, Hkv, Nq, d = (case[k] for k in ("B", "Hq", "Hkv", "Nq", "d"))
    if case["op"] == "append":
        n, T = B * Hkv * Nq, case["T"]
        return {"bytes": 2.0 * n * d * (e + 1) + 2 * 4 * n / T, "flops": 4.0 * n * d}
    pairs = _pairs(case)
    keys = 0  # tokens that some query sees
    for n in _lens(case):
        p0 = (n - Nq) if _q_at_end(case) else case["Nk"] - Nq
        lo = 0 if case["left"] < 0 else max(0, p0 - case["left"])
        keys += max(0, n - lo) + min(case["sinks"], lo, n)
    q = B * Hq * Nq * d
    if case["op"] == "cache":
        return {"bytes": 2.0 * q * e + 2.0 * keys * Hkv * d + 8.0 * keys * Hkv / case["T"],
                "flops": 4.0 * pairs * Hq * d}
    kv = keys * Hkv * d
    if not case["train"]:
        return {"bytes": e * (2.0 * q + 2.0 * kv), "flops": 4.0 * pairs * Hq * d}
    return {"bytes": e * (4.0 * q + 4.0 * kv), "flops": 14.0 * pairs * Hq * d}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _keys(shape, gen, sinks):
    """Keys as a layer makes them: unit spread, a shift of each channel, larger first tokens."""
    B, H, N, d = shape
    k = torch.randn(shape, generator=gen, device=DEV)
    k += 0.5 * torch.randn((1, H, 1, d), generator=gen, device=DEV)
    if sinks:
        k[:, :, :sinks] *= 1.5
    return k


def _pow2_scale(amax):
    """The smallest power of two s with amax / s <= 448, at least 2 ** MIN_EXP."""
    m, e = torch.frexp(amax)
    ex = torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype), torch.full_like(e, MIN_EXP))
    return ((ex.clamp(min=MIN_EXP) + 127) << 23).to(torch.int32).view(torch.float32)


def _fill_cache(case, gen, B, nb):
    """A cache whose blocks hold rounded keys and values, blocks of a sequence scattered."""
    Hkv, T, d = case["Hkv"], case["T"], case["d"]
    blocks = B * nb + 3
    shape = (blocks, Hkv, T, d)
    out = []
    for spread in (1.0, 1.0):
        x = torch.randn(shape, generator=gen, device=DEV) * spread
        s = _pow2_scale(x.abs().amax(dim=(2, 3)))
        out += [(x / s[:, :, None, None]).to(torch.float8_e4m3fn), s]
        del x
    table = torch.randperm(blocks, generator=gen, device=DEV)[:B * nb].reshape(B, nb).to(torch.int32)
    return out[0], out[2], out[1], out[3], table


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    B, Hq, Hkv, Nq, Nk, d = (case[k] for k in ("B", "Hq", "Hkv", "Nq", "Nk", "d"))
    dt = getattr(torch, case["dtype"])
    s = {"case": case}
    lens = torch.tensor(_lens(case), dtype=torch.int32, device=DEV)
    if case["op"] == "window":
        s["q"] = torch.randn((B, Hq, Nq, d), generator=gen, device=DEV).to(dt)
        s["k"] = _keys((B, Hkv, Nk, d), gen, case["sinks"]).to(dt)
        s["v"] = torch.randn((B, Hkv, Nk, d), generator=gen, device=DEV).to(dt)
        s["lens"] = lens if case["ragged"] else None
        s["q_pos"] = lens - Nq if _q_at_end(case) else None
        if case["train"]:
            s["dout"] = torch.randn((B, Hq, Nq, d), generator=gen, device=DEV).to(dt)
        return s
    T = case["T"]
    nb = -(-Nk // T)
    s["lens"] = lens
    s["k8"], s["v8"], s["ks"], s["vs"], s["table"] = _fill_cache(case, gen, B, nb)
    if case["op"] == "cache":
        s["q"] = torch.randn((B, Hq, Nq, d), generator=gen, device=DEV).to(dt)
    else:
        s["start"] = lens - Nq
        s["k"] = _keys((B, Hkv, Nq, d), gen, 0).to(dt)
        s["v"] = torch.randn((B, Hkv, Nq, d), generator=gen, device=DEV).to(dt)
    return s


# ---------------------------------------------------------------------------
# plain forms (32 bits, rounded once at the end)
# ---------------------------------------------------------------------------
def _softmax_products(s, visible):
    """exp(s - max) over the visible keys and its sum; rows that see nothing give zeros."""
    s = s.masked_fill(~visible, float("-inf"))
    mx = s.detach().amax(dim=-1, keepdim=True)
    e = torch.exp(s - torch.where(torch.isinf(mx), torch.zeros_like(mx), mx))
    total = e.sum(dim=-1, keepdim=True)
    return e / torch.where(total == 0, torch.ones_like(total), total)


def _plain_dense(q, k, v, case, lens, q_pos):
    """Every query against every key. q [B, Hkv, g, Nq, d], k and v [B, Hkv, Nk, d]."""
    B, Nq, Nk = q.shape[0], q.shape[3], k.shape[2]
    p = (q_pos[:, None] + torch.arange(Nq, device=DEV))[:, None, None, :, None]
    j = torch.arange(Nk, device=DEV)[None, None, None, None, :]
    n = lens[:, None, None, None, None]
    left = Nk if case["left"] < 0 else case["left"]
    right = Nk if case["right"] < 0 else case["right"]
    visible = (p >= 0) & (p < n) & (j < n) & (j <= p + right) & ((j >= p - left) | (j < case["sinks"]))
    s = torch.matmul(q, k[:, :, None].transpose(-1, -2)) / math.sqrt(case["d"])
    return torch.matmul(_softmax_products(s, visible), v[:, :, None])


def _plain_band(q, k, v, case, lens):
    """Blocks of queries against the keys that their windows reach, and the first tokens."""
    B, Hkv, g, N, d = q.shape
    left = N if case["left"] < 0 else min(case["left"], N)
    right = N if case["right"] < 0 else min(case["right"], N)
    S = min(case["sinks"], N)
    blk = min(N, max(64, left + right + 1))
    nb = -(-N // blk)
    width = blk + left + right
    pad = torch.nn.functional.pad
    qb = pad(q, (0, 0, 0, nb * blk - N)).reshape(B, Hkv, g, nb, blk, d)
    kb = pad(k, (0, 0, left, nb * blk - N + right)).unfold(2, width, blk)[:, :, None]  # ... nb, d, width
    vb = pad(v, (0, 0, left, nb * blk - N + right)).unfold(2, width, blk)[:, :, None]
    p = torch.arange(nb * blk, device=DEV).reshape(nb, blk, 1)
    j = (torch.arange(nb, device=DEV) * blk - left)[:, None, None] + torch.arange(width, device=DEV)
    n = lens.reshape(B, 1, 1, 1, 1, 1)
    near = (p < n) & (j >= 0) & (j < n) & (j <= p + right) & (j >= p - left)
    f = torch.arange(S, device=DEV)
    first = (p < n) & (f < n) & (f < p - left)
    s = torch.cat([torch.matmul(qb, kb),
                   torch.matmul(qb, k[:, :, None, None, :S].transpose(-1, -2))], dim=-1) / math.sqrt(d)
    P = _softmax_products(s, torch.cat([near, first], dim=-1))
    o = torch.matmul(P[..., :width], vb.transpose(-1, -2)) + torch.matmul(P[..., width:], v[:, :, None, None, :S])
    return o.reshape(B, Hkv, g, nb * blk, d)[:, :, :, :N]


def _plain_window(s):
    c = s["case"]
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    B, Nq, Nk = c["B"], c["Nq"], c["Nk"]
    lens = s["lens"] if s["lens"] is not None else torch.full((B,), Nk, device=DEV, dtype=torch.int32)
    q_pos = s["q_pos"] if s["q_pos"] is not None else torch.full((B,), Nk - Nq, device=DEV, dtype=torch.int32)
    leaves = [x.requires_grad_(c["train"]) for x in (q, k, v)]
    qg = q.reshape(B, c["Hkv"], c["Hq"] // c["Hkv"], Nq, c["d"])
    reach = (Nk if c["left"] < 0 else c["left"]) + (Nk if c["right"] < 0 else c["right"])
    o = (_plain_band(qg, k, v, c, lens) if Nq == Nk and 2 * reach < Nk
         else _plain_dense(qg, k, v, c, lens, q_pos))
    o = o.reshape(q.shape)
    dt = s["q"].dtype
    if not c["train"]:
        return o.to(dt)
    grads = torch.autograd.grad(o, leaves, s["dout"].float())
    return [o.detach().to(dt)] + [x.to(dt) for x in grads]


def _plain_append(s):
    """Every block that gets tokens is taken out, joined with them, rounded and put back."""
    c = s["case"]
    B, Hkv, n, T, d = c["B"], c["Hkv"], c["Nq"], c["T"], c["d"]
    nt = (n + T - 2) // T + 1                                  # blocks a sequence may touch
    first = torch.div(s["start"], T, rounding_mode="floor")
    lb = first[:, None] + torch.arange(nt, device=DEV)         # logical blocks [B, nt]
    pos = lb[:, :, None] * T + torch.arange(T, device=DEV)     # positions [B, nt, T]
    i = pos - s["start"][:, None, None]
    fresh = (i >= 0) & (i < n) & (pos < s["lens"][:, None, None])
    old = i < 0                                                # tokens that were there
    gets = fresh.any(dim=2)
    blk = torch.gather(s["table"], 1, lb.clamp(max=s["table"].shape[1] - 1).long()).long()
    sel = blk[gets]
    at = i.clamp(0, n - 1)[:, None, :, :, None].expand(B, Hkv, nt, T, d).reshape(B, Hkv, nt * T, d)
    out = []
    for x, x8, xs in ((s["k"], s["k8"], s["ks"]), (s["v"], s["v8"], s["vs"])):
        new = torch.gather(x.float(), 2, at).reshape(B, Hkv, nt, T, d).transpose(1, 2)[gets]
        fr, ol = fresh[gets][:, None, :, None], old[gets][:, None, :, None]
        new = torch.where(fr, new, torch.zeros_like(new))
        scale = _pow2_scale(new.abs().amax(dim=(2, 3)))
        scale = torch.where(old[gets].any(dim=1)[:, None], torch.maximum(scale, xs[sel]), scale)
        was = x8[sel].float()
        got = torch.where(fr, new / scale[:, :, None, None],
                          torch.where(ol, was * (xs[sel] / scale)[:, :, None, None], was))
        x8.view(torch.uint8)[sel] = got.to(torch.float8_e4m3fn).view(torch.uint8)
        xs[sel] = scale
        out += [x8, xs]
    return out


def _plain_cache(s):
    """The sequences' blocks gathered and multiplied out, then dense attention."""
    c = s["case"]
    B, Hkv, T, d = c["B"], c["Hkv"], c["T"], c["d"]
    t = s["table"].long()
    k, v = ((x8.view(torch.uint8)[t].view(torch.float8_e4m3fn).float() * xs[t][..., None, None])
            .transpose(1, 2).reshape(B, Hkv, -1, d) for x8, xs in ((s["k8"], s["ks"]), (s["v8"], s["vs"])))
    q = s["q"].float().reshape(B, Hkv, c["Hq"] // Hkv, c["Nq"], d)
    return _plain_dense(q, k, v, c, s["lens"], s["lens"] - c["Nq"]).reshape(s["q"].shape).to(s["q"].dtype)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    c = state["case"]
    if own:
        import laplacian_nystr_linear_gb300 as lap
        mask = {k: c[k] for k in ("left", "right", "sinks")}
        if c["op"] == "window":
            q, k, v = state["q"], state["k"], state["v"]
            mask.update(lens=state["lens"], q_pos=state["q_pos"])
            if not c["train"]:
                return lap.window_attention(q, k, v, **mask)
            leaves = [x.detach().requires_grad_(True) for x in (q, k, v)]
            o = lap.window_attention(*leaves, **mask)
            return [o.detach(), *torch.autograd.grad(o, leaves, state["dout"])]
        cache = lap.KVCache(state["k8"], state["v8"], state["ks"], state["vs"])
        if c["op"] == "append":
            lap.cache_append(cache, state["k"], state["v"], state["table"], state["start"],
                             lens=state["lens"])
            return [cache.k, cache.k_scale, cache.v, cache.v_scale]
        return lap.cache_attention(state["q"], cache, state["table"], state["lens"], **mask)
    if c["op"] == "window":
        return _plain_window(state)
    return _plain_append(state) if c["op"] == "append" else _plain_cache(state)


# ---------------------------------------------------------------------------
# values in 64 bits, from the definitions
# ---------------------------------------------------------------------------
def _exact_rows(q, k, v, p, n, c, dout=None):
    """Queries q [Hkv, g, R, d] at positions p [R] over the keys of one sequence, with gradients."""
    left = k.shape[1] if c["left"] < 0 else c["left"]
    right = k.shape[1] if c["right"] < 0 else c["right"]
    lo = max(0, int(p[0]) - left)
    hi = max(lo, min(n, int(p[-1]) + right + 1))
    S = min(c["sinks"], lo)
    j = torch.cat([torch.arange(S, device=DEV), torch.arange(lo, hi, device=DEV)])
    ok = (j[None] < n) & (j[None] <= p[:, None] + right) & (p[:, None] >= 0) & (p[:, None] < n)
    ok &= (j[None] >= p[:, None] - left) | (j[None] < c["sinks"])
    kj, vj = k[:, j], v[:, j]
    sc = c["d"] ** -0.5
    s = torch.einsum("hgrd,hjd->hgrj", q, kj) * sc
    w = torch.where(ok, torch.exp(s - torch.where(ok, s, -1e300).amax(-1, keepdim=True).clamp(min=-1e299)), 0.0)
    t = w.sum(-1, keepdim=True)
    w = torch.where(t > 0, w / t, 0.0)
    o = torch.einsum("hgrj,hjd->hgrd", w, vj)
    if dout is None:
        return o, None
    dw = torch.einsum("hgrd,hjd->hgrj", dout, vj)
    ds = w * (dw - (w * dw).sum(-1, keepdim=True)) * sc
    dq = torch.einsum("hgrj,hjd->hgrd", ds, kj)
    return o, (j, dq, torch.einsum("hgrj,hgrd->hjd", ds, q), torch.einsum("hgrj,hgrd->hjd", w, dout))


def _exact_attention(q, k_of, v_of, case, lens, q_pos, dout=None):
    B, Hq, Nq, d = q.shape
    Hkv = case["Hkv"]
    o = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    dq = torch.zeros_like(o) if dout is not None else None
    dks, dvs = [], []
    rows = 512
    for b in range(B):
        k, v = k_of(b), v_of(b)
        dk, dv = (torch.zeros_like(k), torch.zeros_like(v)) if dout is not None else (None, None)
        for r in range(0, Nq, rows):
            at = slice(r, min(Nq, r + rows))
            p = int(q_pos[b]) + torch.arange(at.start, at.stop, device=DEV)
            split = lambda x: x[b, :, at].double().reshape(Hkv, Hq // Hkv, -1, d)  # noqa: E731
            ob, g = _exact_rows(split(q), k, v, p, int(lens[b]), case, None if dout is None else split(dout))
            o[b, :, at] = ob.reshape(Hq, -1, d)
            if g is not None:
                dq[b, :, at] = g[1].reshape(Hq, -1, d)
                dk.index_add_(1, g[0], g[2])
                dv.index_add_(1, g[0], g[3])
        dks.append(dk)
        dvs.append(dv)
    return o if dout is None else [o, dq, torch.stack(dks), torch.stack(dvs)]


def _exact_append(s, c):
    """Token by token positions on the host's side of the table, block by block in 64 bits."""
    T, n = c["T"], c["Nq"]
    start, lens, table = (s[x].tolist() for x in ("start", "lens", "table"))
    out = []
    for x, x8, xs in ((s["k"], s["k8"], s["ks"]), (s["v"], s["v8"], s["vs"])):
        got, sc = x8.double().clone(), xs.double().clone()
        src, dst, groups = [], [], {}
        for b in range(c["B"]):
            for i in range(min(n, lens[b] - start[b])):
                p = start[b] + i
                blk = table[b][p // T]
                groups.setdefault(blk, []).append((b * n + i, p % T))
        blocks = sorted(groups)
        idx = torch.full((len(blocks), T), -1, dtype=torch.int64)
        for r, blk in enumerate(blocks):
            for token, slot in groups[blk]:
                idx[r, slot] = token
        idx, sel = idx.to(DEV), torch.tensor(blocks, device=DEV)
        fresh = (idx >= 0)[:, None, :, None]
        lead = (idx >= 0).to(torch.int8).argmax(dim=1)
        held = (torch.arange(T, device=DEV)[None] < lead[:, None])[:, None, :, None]
        rows = x.double().transpose(1, 2).reshape(c["B"] * n, c["Hkv"], c["d"])
        new = torch.where(fresh, rows[idx.clamp(min=0)].transpose(1, 2), 0.0)
        top = new.abs().amax(dim=(2, 3))
        e = torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / E4M3_MAX) - 1e-13)
        want = torch.where(top > 0, torch.exp2(e), 0.0).clamp(min=2.0 ** MIN_EXP)
        want = torch.where(lead[:, None] > 0, torch.maximum(want, sc[sel]), want)
        old = got[sel]
        val = torch.where(fresh, new / want[:, :, None, None],
                          torch.where(held, old * (sc[sel] / want)[:, :, None, None], old))
        # nearest value of 3 mantissa bits, exponents from -6, ties to even
        ex = torch.floor(torch.log2(val.abs().clamp(min=2.0 ** -6)) + 1e-13).clamp(min=-6)
        unit = torch.exp2(ex - 3)
        got[sel] = torch.round(val / unit) * unit
        sc[sel] = want
        out += [got, sc]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s, case)
    B, Nq, Nk = case["B"], case["Nq"], case["Nk"]
    if case["op"] == "window":
        lens = s["lens"].tolist() if s["lens"] is not None else [Nk] * B
        q_pos = s["q_pos"].tolist() if s["q_pos"] is not None else [Nk - Nq] * B
        return _exact_attention(s["q"], lambda b: s["k"][b].double(), lambda b: s["v"][b].double(), case,
                                lens, q_pos, s.get("dout"))

    def rows(x8, xs, b):
        t = s["table"][b].long()
        x = x8.view(torch.uint8)[t].view(torch.float8_e4m3fn).double() * xs[t].double()[..., None, None]
        return x.transpose(0, 1).reshape(case["Hkv"], -1, case["d"])

    lens = s["lens"].tolist()
    return _exact_attention(s["q"], lambda b: rows(s["k8"], s["ks"], b), lambda b: rows(s["v8"], s["vs"], b),
                            case, lens, [n - Nq for n in lens])
