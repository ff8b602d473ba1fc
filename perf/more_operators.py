"""What stands around the attentions in a layer: rotary positions, the residual with its norms, and
the gated feed-forward block.  The cases that are measured, their inputs, their plain forms in torch,
and their values in 64 bits.

A case is one of three calls, forward (train False) or forward and backward (train True):
  op "rotary"  rotary: queries and keys turned by their positions
  op "norm"    residual_norm: h = x + scale gate post(u), y = pre(h)
  op "mlp"     gated_mlp: y = (act(x Wg + bg) * (x Wu + bu)) Wo + bo, w_in = [Wg | Wu]
"""
import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _rotary(name, B, Hq, Hkv, N, d, rot, layout, scaling, far, given, dtype, train):
    """far: the sequences' last positions lie below it; given: positions one by one, not from a start."""
    return {"name": name, "op": "rotary", "B": B, "Hq": Hq, "Hkv": Hkv, "N": N, "d": d, "rot": rot,
            "layout": layout, "scaling": scaling, "far": far, "given": given, "dtype": dtype, "train": train}


def _norm(name, B, N, C, pre, post, gate, scale, bias, dtype, train):
    """gate: of each sequence [B, C]; scale: of each feature [C]; bias: of the norms."""
    return {"name": name, "op": "norm", "B": B, "N": N, "C": C, "pre": pre, "post": post, "gate": gate,
            "scale": scale, "bias": bias, "dtype": dtype, "train": train}


def _mlp(name, B, N, C, F, act, bias, dtype, train):
    return {"name": name, "op": "mlp", "B": B, "N": N, "C": C, "F": F, "act": act, "bias": bias,
            "dtype": dtype, "train": train}


def listed():
    return [
        # one new token of each of 32 sequences that are far along, frequencies scaled by parts
        _rotary("rotary_token", 32, 32, 8, 1, 128, 128, "half", "parts", 131072, False, "bfloat16", False),
        # a training step on sequences of 8192, heads of 128 that share keys
        _rotary("rotary_train", 2, 16, 4, 8192, 128, 128, "half", "none", 8192, False, "bfloat16", True),
        # a padded batch in fp32, pairs side by side, part of the head, positions given
        _rotary("rotary_part_f32", 4, 10, 5, 1001, 96, 64, "interleaved", "linear", 4004, True, "float32", True),
        # between two blocks of one answering token of each of 32 sequences
        _norm("norm_token", 32, 1, 1024, "rms", "none", False, False, False, "bfloat16", False),
        # 128 x 128 token grids, 8 heads of 64: both norms, the gate and the residual scale, trained
        _norm("norm_grid_train", 8, 16384, 512, "layer", "layer", True, True, True, "bfloat16", True),
        # 5 heads of 64, an odd length, fp32
        _norm("norm_odd_f32_train", 4, 1001, 320, "layer", "none", False, True, True, "float32", True),
        # a long prompt through a wide model
        _norm("norm_prompt", 1, 32768, 4096, "rms", "rms", False, False, False, "bfloat16", False),
        # the smallest answer: one token
        _mlp("mlp_token", 1, 1, 512, 2048, "silu", False, "bfloat16", False),
        # 16 sequences that answer, a wide model
        _mlp("mlp_token_batch", 16, 1, 4096, 10880, "silu", False, "bfloat16", False),
        # a prompt of odd length, biases
        _mlp("mlp_prompt", 1, 4099, 2048, 5504, "gelu", True, "bfloat16", False),
        # 128 x 128 token grids, 8 heads of 64, trained
        _mlp("mlp_grid_train", 8, 16384, 512, 1408, "silu", False, "bfloat16", True),
        # 28 x 28 grids, 2 heads of 64, fp32, a hidden width that nothing divides
        _mlp("mlp_odd_f32_train", 4, 784, 128, 341, "gelu", True, "float32", True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "norm", "mlp", "mlp"])
    dtype = rng.choice(["bfloat16", "bfloat16", "bfloat16", "float32"])
    train = rng.random() < 0.6
    if op == "rotary":
        d = rng.choice([16, 32, 48, 64, 64, 80, 96, 112, 128, 128])
        Hkv = _log_int(rng, 1, 8)
        g = rng.choice([1, 1, 2, 3, 4, 8])
        N = 1 if rng.random() < 0.25 else _log_int(rng, 1, 16384)
        B = _log_int(rng, 1, max(1, min(32, 400000 // (N * Hkv * g))))
        rot = d if rng.random() < 0.6 else 2 * rng.randint(1, d // 2)
        c = _rotary("", B, Hkv * g, Hkv, N, d, rot, rng.choice(["half", "interleaved"]),
                    rng.choice(["none", "linear", "base", "parts"]), N + _log_int(rng, 1, 1 << 20),
                    rng.random() < 0.3, dtype, train and N > 1)
    elif op == "norm":
        C = rng.choice([_log_int(rng, 8, 8192), 8 * _log_int(rng, 1, 1024), 64 * _log_int(rng, 1, 128)])
        rows = _log_int(rng, 1, max(1, (1 << 26) // C))
        B = min(rows, _log_int(rng, 1, 32))
        pre = rng.choice(["rms", "layer"])
        post = rng.choice(["none", "none", pre])
        c = _norm("", B, max(1, rows // B), C, pre, post, rng.random() < 0.5, rng.random() < 0.5,
                  pre == "layer" and rng.random() < 0.7, dtype, train)
    else:
        C = rng.choice([_log_int(rng, 16, 4096), 8 * _log_int(rng, 4, 512), 64 * _log_int(rng, 1, 64)])
        F = rng.choice([_log_int(rng, C, 4 * C), 8 * _log_int(rng, max(1, C // 8), C // 2 + 1), 4 * C])
        most = (1.5e12 if dtype == "bfloat16" else 3e11) / (18.0 * C * F)
        rows = rng.choice([_log_int(rng, 1, 64), _log_int(rng, 1, max(1, min(65536, int(most))))])
        B = min(rows, _log_int(rng, 1, 16))
        c = _mlp("", B, max(1, rows // B), C, F, rng.choice(["silu", "silu", "gelu", "gelu_tanh"]),
                 rng.random() < 0.4, dtype, train)
    return {k: v for k, v in c.items() if k != "name"}


def work(case):
    e = 4.0 if case["dtype"] == "float32" else 2.0
    twice = 2.0 if case["train"] else 1.0
    T = float(case["B"] * case["N"])
    if case["op"] == "rotary":
        n = T * (case["Hq"] + case["Hkv"])
        return {"bytes": twice * 2.0 * n * case["d"] * e, "flops": twice * 3.0 * n * case["rot"]}
    if case["op"] == "norm":
        # x, u in, h, y out; backward dh, dy in, dx, du out
        n = T * case["C"]
        return {"bytes": twice * 4.0 * n * e, "flops": (40.0 if case["train"] else 16.0) * n}
    C, F = case["C"], case["F"]
    wide = T * C * F
    if not case["train"]:
        return {"bytes": e * (2.0 * T * C + 3.0 * C * F), "flops": 6.0 * wide}
    return {"bytes": e * (4.0 * T * C + 6.0 * C * F), "flops": 18.0 * wide}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
BASE = 10000.0
PARTS = {"factor": 16.0, "context": 8192, "low": 1.0, "high": 32.0}


def _frequencies(case):
    """Radians a position, one for each pair, and the factor of the turned features."""
    rot, scaling, f = case["rot"], case["scaling"], PARTS["factor"]
    base = BASE
    if scaling == "base" and rot > 2:
        base = BASE * f ** (rot / (rot - 2.0))
    w = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        w = [x / f for x in w]
    if scaling != "parts":
        return w, 1.0
    out = []
    for x in w:
        turns = PARTS["context"] * x / (2.0 * math.pi)
        keep = min(1.0, max(0.0, (turns - PARTS["low"]) / (PARTS["high"] - PARTS["low"])))
        out.append(x * (keep + (1.0 - keep) / f))
    return out, 1.0 + 0.1 * math.log(f)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    dt = getattr(torch, case["dtype"])
    B, N = case["B"], case["N"]
    s = {"case": case}

    def rand(*shape, spread=1.0, shift=0.0):
        return (torch.randn(shape, generator=gen, device=DEV) * spread + shift).to(dt)

    if case["op"] == "rotary":
        s["q"] = rand(B, case["Hq"], N, case["d"])
        s["k"] = rand(B, case["Hkv"], N, case["d"])
        far = case["far"]
        last = torch.randint(far // 2, far, (B,), generator=gen, device=DEV)
        s["start"] = (last - N + 1).clamp(min=0).to(torch.int32)
        s["positions"] = None
        if case["given"]:   # several documents in a row: positions begin anew
            cut = torch.randint(1, N + 1, (B, 1), generator=gen, device=DEV)
            i = torch.arange(N, device=DEV)[None]
            s["positions"] = torch.where(i < cut, i + s["start"][:, None], i - cut).to(torch.int32)
            s["start"] = None
        if case["train"]:
            s["dq"], s["dk"] = rand(*s["q"].shape), rand(*s["k"].shape)
        w, s["factor"] = _frequencies(case)
        s["w"] = torch.tensor(w, dtype=torch.float64, device=DEV)
        if own:
            import laplacian_nystr_linear_gb300 as lap
            scaling = case["scaling"]
            given = {} if scaling == "none" else {"scaling": scaling, "factor": PARTS["factor"]}
            if scaling == "parts":
                given.update(context=PARTS["context"], low=PARTS["low"], high=PARTS["high"])
            s["freqs"] = lap.rotary_frequencies(case["rot"], base=BASE, device=DEV, **given)
        return s
    if case["op"] == "norm":
        C = case["C"]
        # a residual stream that has grown, some features larger than others, and a block's output
        s["x"] = (torch.randn((B, N, C), generator=gen, device=DEV)
                  * (2.0 * torch.exp(0.5 * torch.randn((C,), generator=gen, device=DEV))) + 0.1).to(dt)
        s["u"] = rand(B, N, C, spread=0.7)
        s["weight"] = rand(C, spread=0.2, shift=1.0)
        s["bias"] = rand(C, spread=0.1) if case["bias"] else None
        s["post_weight"] = rand(C, spread=0.2, shift=1.0) if case["post"] != "none" else None
        s["post_bias"] = rand(C, spread=0.1) if case["bias"] and case["post"] != "none" else None
        s["gate"] = rand(B, C, spread=0.5, shift=0.5) if case["gate"] else None
        s["scale"] = rand(C, spread=0.05, shift=0.2) if case["scale"] else None
        if case["train"]:
            s["dh"], s["dy"] = rand(B, N, C), rand(B, N, C)
        return s
    C, F = case["C"], case["F"]
    s["x"] = rand(B, N, C)
    s["w_in"] = rand(C, 2 * F, spread=C ** -0.5)
    s["w_out"] = rand(F, C, spread=F ** -0.5)
    s["b_in"] = rand(2 * F, spread=0.1) if case["bias"] else None
    s["b_out"] = rand(C, spread=0.1) if case["bias"] else None
    if case["train"]:
        s["dy"] = rand(B, N, C)
    return s


# ---------------------------------------------------------------------------
# plain forms (32 bits, angles in 64, rounded once at the end)
# ---------------------------------------------------------------------------
def _plain_rotary(s):
    c = s["case"]
    rot, N, dt = c["rot"], c["N"], s["q"].dtype
    p = s["positions"] if s["positions"] is not None else s["start"][:, None] + torch.arange(N, device=DEV)
    angle = p.double()[:, None, :, None] * s["w"]                     # [B, 1, N, rot / 2]
    cos, sin = ((f(angle) * s["factor"]).float() for f in (torch.cos, torch.sin))

    def turn(x):
        t = x[..., :rot]
        if c["layout"] == "half":
            a, b = t[..., :rot // 2], t[..., rot // 2:]
            t = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
        else:
            a, b = t[..., 0::2], t[..., 1::2]
            t = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        return torch.cat([t, x[..., rot:]], dim=-1)

    leaves = [s[n].float().requires_grad_(c["train"]) for n in ("q", "k")]
    out = [turn(x) for x in leaves]
    grads = torch.autograd.grad(out, leaves, [s["dq"].float(), s["dk"].float()]) if c["train"] else []
    return [x.detach().to(dt) for x in (*out, *grads)]


NORM_LEAVES = ("x", "u", "weight", "bias", "post_weight", "post_bias", "gate", "scale")
EPS = 1e-6


def _plain_norm(s):
    c = s["case"]
    dt = s["x"].dtype
    t = {n: None if s[n] is None else s[n].float().requires_grad_(c["train"]) for n in NORM_LEAVES}

    def norm(z, kind, weight, bias):
        if kind == "layer":
            z = z - z.mean(dim=-1, keepdim=True)
        z = z * torch.rsqrt((z * z).mean(dim=-1, keepdim=True) + EPS) * weight
        return z if bias is None else z + bias

    z = t["u"] if c["post"] == "none" else norm(t["u"], c["post"], t["post_weight"], t["post_bias"])
    if t["gate"] is not None:
        z = z * t["gate"][:, None]
    if t["scale"] is not None:
        z = z * t["scale"]
    h = t["x"] + z
    y = norm(h, c["pre"], t["weight"], t["bias"])
    out = [h, y]
    leaves = [x for x in t.values() if x is not None]
    grads = torch.autograd.grad(out, leaves, [s["dh"].float(), s["dy"].float()]) if c["train"] else []
    return [x.detach().to(dt) for x in (*out, *grads)]


def _act(x, kind):
    if kind == "silu":
        return x / (1.0 + torch.exp(-x))
    if kind == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))


MLP_LEAVES = ("x", "w_in", "b_in", "w_out", "b_out")


def _plain_mlp(s):
    c = s["case"]
    dt = s["x"].dtype
    t = {n: None if s[n] is None else s[n].float().requires_grad_(c["train"]) for n in MLP_LEAVES}
    z = torch.matmul(t["x"], t["w_in"])
    if t["b_in"] is not None:
        z = z + t["b_in"]
    y = torch.matmul(_act(z[..., :c["F"]], c["act"]) * z[..., c["F"]:], t["w_out"])
    if t["b_out"] is not None:
        y = y + t["b_out"]
    if not c["train"]:
        return y.to(dt)
    leaves = [x for x in t.values() if x is not None]
    return [x.detach().to(dt) for x in (y, *torch.autograd.grad(y, leaves, s["dy"].float()))]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _own(s):
    import laplacian_nystr_linear_gb300 as lap
    c = s["case"]
    train = c["train"]

    def leaf(x):
        return None if x is None else x.detach().requires_grad_(train)

    if c["op"] == "rotary":
        leaves = [leaf(s["q"]), leaf(s["k"])]
        out = lap.rotary(*leaves, s["freqs"], start=s["start"], positions=s["positions"], layout=c["layout"])
        back = [s["dq"], s["dk"]] if train else None
    elif c["op"] == "norm":
        t = {n: leaf(s[n]) for n in NORM_LEAVES}
        out = lap.residual_norm(t["x"], t["u"], t["weight"], t["bias"], post_weight=t["post_weight"],
                                post_bias=t["post_bias"], gate=t["gate"], scale=t["scale"], pre=c["pre"],
                                post=None if c["post"] == "none" else c["post"], eps=EPS)
        leaves = [x for x in t.values() if x is not None]
        back = [s["dh"], s["dy"]] if train else None
    else:
        t = {n: leaf(s[n]) for n in MLP_LEAVES}
        out = lap.gated_mlp(t["x"], t["w_in"], t["b_in"], t["w_out"], t["b_out"], act=c["act"])
        if not train:
            return out
        leaves, out, back = [x for x in t.values() if x is not None], [out], [s["dy"]]
    if not train:
        return list(out)
    return [*(x.detach() for x in out), *torch.autograd.grad(out, leaves, back)]


def run(state):
    if own:
        return _own(state)
    return {"rotary": _plain_rotary, "norm": _plain_norm, "mlp": _plain_mlp}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# values in 64 bits, from the definitions
# ---------------------------------------------------------------------------
def _exact_rotary(s):
    """Pairs as complex numbers; the gradient turns the other way."""
    c = s["case"]
    rot, N = c["rot"], c["N"]
    p = s["positions"] if s["positions"] is not None else s["start"][:, None] + torch.arange(N, device=DEV)[None]
    e = torch.polar(torch.full((), s["factor"], dtype=torch.float64, device=DEV).expand(c["B"], N, rot // 2),
                    p.double()[..., None] * s["w"])[:, None]
    first = torch.arange(rot // 2, device=DEV) * (2 if c["layout"] == "interleaved" else 1)
    second = first + (1 if c["layout"] == "interleaved" else rot // 2)

    def turn(x, e):
        o = x.double().clone()
        z = torch.complex(o[..., first], o[..., second]) * e
        o[..., first], o[..., second] = z.real, z.imag
        return o

    out = [turn(s["q"], e), turn(s["k"], e)]
    return out + [turn(s["dq"], e.conj()), turn(s["dk"], e.conj())] if c["train"] else out


def _exact_norm(s):
    c = s["case"]
    x, u = s["x"].double(), s["u"].double()
    one = torch.ones((), dtype=torch.float64, device=DEV)
    g = {n: one if s[n] is None else s[n].double() for n in ("weight", "post_weight", "gate", "scale")}
    zero = torch.zeros((), dtype=torch.float64, device=DEV)
    pb, qb = (zero if s[n] is None else s[n].double() for n in ("bias", "post_bias"))
    gate = g["gate"][:, None] if s["gate"] is not None else one
    m = gate * g["scale"]

    def unit(z, kind):
        if kind == "none":
            return z, None
        z = z - z.mean(-1, keepdim=True) if kind == "layer" else z
        r = (z.square().mean(-1, keepdim=True) + EPS) ** -0.5
        return z * r, r

    def back(d, hat, r, kind):     # through the unit norm
        if kind == "none":
            return d
        t = d - hat * (d * hat).mean(-1, keepdim=True)
        return r * (t - d.mean(-1, keepdim=True) if kind == "layer" else t)

    uh, ur = unit(u, c["post"])
    n = uh * g["post_weight"] + qb
    h = x + m * n
    hh, hr = unit(h, c["pre"])
    out = [h, hh * g["weight"] + pb]
    if not c["train"]:
        return out
    dh, dy = s["dh"].double(), s["dy"].double()
    dt = dh + back(dy * g["weight"], hh, hr, c["pre"])
    dn = dt * m
    out += [dt, back(dn * g["post_weight"], uh, ur, c["post"]), (dy * hh).sum((0, 1))]
    if s["bias"] is not None:
        out.append(dy.sum((0, 1)))
    if s["post_weight"] is not None:
        out.append((dn * uh).sum((0, 1)))
    if s["post_bias"] is not None:
        out.append(dn.sum((0, 1)))
    if s["gate"] is not None:
        out.append((dt * n * g["scale"]).sum(1))
    if s["scale"] is not None:
        out.append((dt * n * gate).sum((0, 1)))
    return out


def _exact_mlp(s):
    c = s["case"]
    F = c["F"]
    x = s["x"].double().flatten(0, 1)
    wi, wo = s["w_in"].double(), s["w_out"].double()
    z = x @ wi
    if s["b_in"] is not None:
        z += s["b_in"].double()
    a, b = z[:, :F], z[:, F:]
    if c["act"] == "silu":
        sg = torch.sigmoid(a)
        act, slope = a * sg, sg * (1 + a * (1 - sg))
    elif c["act"] == "gelu":
        cdf = 0.5 * torch.special.erfc(-a / math.sqrt(2.0))
        act, slope = a * cdf, cdf + a * torch.exp(-0.5 * a * a) / math.sqrt(2.0 * math.pi)
    else:
        k = math.sqrt(2.0 / math.pi)
        th = torch.tanh(k * (a + 0.044715 * a ** 3))
        act = 0.5 * a * (1 + th)
        slope = 0.5 * (1 + th) + 0.5 * a * (1 - th * th) * k * (1 + 3 * 0.044715 * a * a)
    hid = act * b
    y = hid @ wo
    if s["b_out"] is not None:
        y += s["b_out"].double()
    shape = s["x"].shape
    if not c["train"]:
        return y.reshape(shape)
    dy = s["dy"].double().flatten(0, 1)
    dhid = dy @ wo.T
    dz = torch.cat([dhid * b * slope, dhid * act], dim=1)
    out = [y.reshape(shape), (dz @ wi.T).reshape(shape), x.T @ dz]
    if s["b_in"] is not None:
        out.append(dz.sum(0))
    out.append(hid.T @ dy)
    if s["b_out"] is not None:
        out.append(dy.sum(0))
    return out


def exact(case, seed):
    if case["op"] == "mlp" and work(case)["flops"] > 4e12:
        return None
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "norm": _exact_norm, "mlp": _exact_mlp}[case["op"]](s)
