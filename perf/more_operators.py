"""The operators of a recurrent block and of attention's inputs, and the cases they are measured on: the gated linear
recurrence (prompt, training and single-token form), norms of queries and keys with their rotary positions in the same pass,
and the short causal convolution that stands before a recurrence.

With ``own`` false, ``run`` computes an operator in its plain form, elementary torch operations in
float32 rounded once at the end; with ``own`` true it calls the framework's kernels.  ``exact`` gives
the same outputs from the definitions in float64.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}

# Largest work of a drawn case in bytes, below the largest listed one's.
MOST_BYTES = 8.0e8


# ---- cases ----------------------------------------------------------------------------------------

def listed():
    return [
        # a batch of prompts through a recurrent layer: decay a rate times a gate, inputs gated and scaled to keep the norm
        {"name": "scan_prompt_bf16", "op": "scan", "B": 8, "N": 2048, "C": 4096, "gate": "rate", "mix": "norm",
         "gated": True, "state": False, "ragged": False, "dtype": "bf16"},
        # one long sequence continued from a kept state: few rows of channels to share out
        {"name": "scan_long_bf16", "op": "scan", "B": 1, "N": 65536, "C": 2048, "gate": "sigmoid", "mix": "convex",
         "gated": False, "state": True, "ragged": False, "dtype": "bf16"},
        # a small fp32 batch of prompts of different lengths (0 and 1 among them), an odd width, the plain recurrence
        {"name": "scan_ragged_f32", "op": "scan", "B": 5, "N": 777, "C": 333, "gate": "log", "mix": "plain",
         "gated": False, "state": True, "ragged": True, "dtype": "f32"},
        # a training step's forward and gradients
        {"name": "scan_train_bf16", "op": "scan_train", "B": 8, "N": 2048, "C": 2048, "gate": "rate", "mix": "norm",
         "gated": True, "state": False, "ragged": False, "dtype": "bf16"},
        # a smaller one, of odd lengths, with a state on both ends (a sequence cut in pieces)
        {"name": "scan_train_f16", "op": "scan_train", "B": 3, "N": 1001, "C": 1000, "gate": "sigmoid", "mix": "convex",
         "gated": False, "state": True, "ragged": True, "dtype": "f16"},
        # one token of a serving batch, its states in a pool
        {"name": "scan_token_bf16", "op": "scan_step", "B": 64, "C": 2048, "gate": "rate", "mix": "norm", "gated": True,
         "dtype": "bf16"},
        # q and k of a training batch, half layout, whole head
        {"name": "qknorm_bf16", "op": "qknorm", "B": 4, "H": 16, "G": 16, "N": 4096, "D": 128, "rot": 128, "dtype": "bf16",
         "order": "bnhd", "interleaved": False, "centred": False, "start": 0},
        # forward and gradients: shared k heads, half of the head turned, interleaved, centred norms, an odd length
        {"name": "qknorm_train_f16", "op": "qknorm_train", "B": 2, "H": 12, "G": 4, "N": 1023, "D": 96, "rot": 48,
         "dtype": "f16", "order": "bnhd", "interleaved": True, "centred": True, "start": 1000},
        # single tokens deep in their contexts
        {"name": "qknorm_token_bf16", "op": "qknorm", "B": 64, "H": 16, "G": 4, "N": 1, "D": 128, "rot": 128, "dtype": "bf16",
         "order": "bhnd", "interleaved": False, "centred": False, "start": 30000},
        # the convolution before the recurrence of a training batch, forward and gradients
        {"name": "conv_train_bf16", "op": "conv_train", "B": 8, "N": 2048, "C": 4096, "K": 4, "silu": True, "bias": True,
         "state": False, "ragged": False, "dtype": "bf16"},
        # prompts of different lengths (0 and 1 among them) continued from kept inputs, an odd width
        {"name": "conv_ragged_f32", "op": "conv", "B": 5, "N": 777, "C": 333, "K": 3, "silu": False, "bias": False,
         "state": True, "ragged": True, "dtype": "f32"},
        # one token of a serving batch
        {"name": "conv_token_bf16", "op": "conv_step", "B": 64, "C": 2048, "K": 4, "silu": True, "bias": True,
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_train", "scan_train", "scan_step", "qknorm", "qknorm_train", "qknorm_train",
                     "conv", "conv_train", "conv_step"])
    while True:
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        if op.startswith("qknorm"):
            D = 8 * rng.randint(2, 32)
            G = rng.choice([1, 2, 4, 8, 16])
            c = {"op": op, "B": _log(rng, 1, 64), "H": G * rng.choice([1, 2, 4]), "G": G, "N": _log(rng, 1, 16384), "D": D,
                 "rot": D if rng.random() < 0.5 else 2 * rng.randint(0, D // 2), "dtype": dtype,
                 "order": rng.choice(["bhnd", "bnhd"]), "interleaved": rng.random() < 0.5, "centred": rng.random() < 0.3,
                 "start": rng.choice([0, 1000, 30000])}
        else:
            c = {"op": op, "B": _log(rng, 1, 256 if op.endswith("step") else 16)}
            if not op.endswith("step"):
                c["N"] = _log(rng, 1, 65536)
            c["C"] = 8 * _log(rng, 2, 1024) if rng.random() < 0.6 else _log(rng, 1, 8192)
            if op.startswith("scan"):
                c.update(gate=rng.choice(["log", "sigmoid", "rate"]), mix=rng.choice(["plain", "convex", "norm"]),
                         gated=rng.random() < 0.5)
            else:
                c.update(K=rng.randint(2, 8), silu=rng.random() < 0.5, bias=rng.random() < 0.5)
            if not op.endswith("step"):
                c.update(state=rng.random() < 0.5, ragged=rng.random() < 0.3)
            c["dtype"] = dtype
        if work(c)["bytes"] <= MOST_BYTES:
            return c


# ---- inputs ---------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(1000003 * (seed % 9973) + 29)


def _randn(gen, shape, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _lengths(gen, B, N):
    n = torch.randint(0, N + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    n[:2] = torch.tensor([0, 1], device="cuda", dtype=torch.int32)[:B]
    n[B - 1] = N
    return n


def _slots(gen, B):
    """Places of B rows in a pool half as large again: (slots int32, the pool's size)."""
    size = B + B // 2 + 1
    return torch.randperm(size, generator=gen, device="cuda")[:B].to(torch.int32), size


def _gate(gen, case, shape):
    """What a projection gives a decay gate: memories of a few to some hundred tokens."""
    dt = DTYPES[case["dtype"]]
    if case["gate"] == "log":
        return (-torch.exp(_randn(gen, shape) - 3.0)).to(dt)
    return (_randn(gen, shape) * 1.2 + (2.5 if case["gate"] == "sigmoid" else 0.0)).to(dt)


def prepare(case, seed):
    gen, op = _gen(seed), case["op"]
    dt = DTYPES[case["dtype"]]
    s = {"case": dict(case)}
    if op.startswith("qknorm"):
        B, N, D, rot = (case[x] for x in ("B", "N", "D", "rot"))
        for name, heads in (("q", case["H"]), ("k", case["G"])):
            kinds = (name, "d" + name) if op == "qknorm_train" else (name,)
            for t in kinds:
                x = _randn(gen, (B, N, heads, D) if case["order"] == "bnhd" else (B, heads, N, D), dt)
                s[t] = x.transpose(1, 2) if case["order"] == "bnhd" else x
            s["w" + name] = (1.0 + 0.2 * _randn(gen, (D,))).to(dt)
        first = torch.randint(0, case["start"] + 1, (B, 1), generator=gen, device="cuda", dtype=torch.int32)
        s["positions"] = first + torch.arange(N, device="cuda", dtype=torch.int32)[None, :]
        p = torch.arange(rot // 2, device="cuda", dtype=torch.float32)
        s["inv_freq"] = torch.exp(p * (-2.0 / max(rot, 1) * math.log(10000.0)))
        s["eps"] = 1e-6
        return s
    B, C = case["B"], case["C"]
    single = op.endswith("step")
    shape = (B, C) if single else (B, case["N"], C)
    s["x"] = _randn(gen, shape, dt)
    if op.startswith("scan"):
        s["z"] = _gate(gen, case, shape)
        s["i"] = _randn(gen, shape, dt) if case["gated"] else None
        # decays of 0.9 to 0.999 at a half-open gate
        u = torch.rand((C,), generator=gen, device="cuda")
        s["rate"] = -2.0 * torch.log(0.9 + 0.099 * u) if case["gate"] == "rate" else None
        entry, wide = (C,), torch.float32
    else:
        K = case["K"]
        s["w"] = (_randn(gen, (C, K)) / math.sqrt(K)).to(dt)
        s["b"] = (0.1 * _randn(gen, (C,))).to(dt) if case["bias"] else None
        entry, wide = (K - 1, C), dt
    if single:
        s["slots"], size = _slots(gen, B)
        s["state"] = _randn(gen, (size,) + entry, wide)
        return s
    s["state"] = _randn(gen, (B,) + entry, wide) if case["state"] else None
    s["lengths"] = _lengths(gen, B, case["N"]) if case["ragged"] else None
    if op.endswith("train"):
        s["dy"] = _randn(gen, shape, dt)
        s["dstate"] = _randn(gen, (B,) + entry, wide) if case["state"] else None
    return s


# ---- the plain forms: the recurrence ----------------------------------------------------------------

def _plain_gates(s):
    """a, 1 - a, what multiplies the input and the input's gate, in float32."""
    c, z = s["case"], s["z"].float()
    if c["gate"] == "sigmoid":
        a, d = torch.sigmoid(z), torch.sigmoid(-z)
    else:
        la = z if c["gate"] == "log" else -s["rate"] * torch.sigmoid(z)
        a, d = torch.exp(la), -torch.expm1(la)
    m = {"plain": lambda: torch.ones_like(a), "convex": lambda: d, "norm": lambda: torch.sqrt(d * (1.0 + a))}[c["mix"]]()
    return a, d, m, None if s["i"] is None else torch.sigmoid(s["i"].float())


def _live(lengths, shape):
    """[B, N, 1], true at a row's tokens; None where every row is full."""
    if lengths is None:
        return None
    return (torch.arange(shape[1], device="cuda")[None, :] < lengths[:, None])[..., None]


def _doubling(a, u):
    """h_t = a_t h_{t-1} + u_t from zero along dim 1, and the products of a up to t, by doubling the reach."""
    step, N = 1, a.shape[1]
    while step < N:
        u = torch.cat((u[:, :step], u[:, step:] + a[:, step:] * u[:, :-step]), 1)
        a = torch.cat((a[:, :step], a[:, step:] * a[:, :-step]), 1)
        step *= 2
    return u, a


def _plain_scan(s):
    c, dt = s["case"], s["x"].dtype
    live = _live(s["lengths"], s["x"].shape)
    a, d, m, g = _plain_gates(s)
    x = s["x"].float()
    u = m * x if g is None else m * g * x
    if live is not None:
        a, u = torch.where(live, a, 1.0), torch.where(live, u, 0.0)
    h, reach = _doubling(a, u)
    if s["state"] is not None:
        h = h + reach * s["state"][:, None]
    y = h if live is None else torch.where(live, h, 0.0)
    out = {"y": y.to(dt), "state": h[:, -1].clone()}
    if c["op"] == "scan":
        return out
    dy = s["dy"].float() if live is None else torch.where(live, s["dy"].float(), 0.0)
    after = torch.zeros_like(dy[:, 0]) if s["dstate"] is None else s["dstate"]
    # G_t = dy_t + a_{t+1} G_{t+1}, backwards, with the gradient of the state that leaves behind the last token
    nxt = torch.cat((a[:, 1:], torch.ones_like(a[:, :1])), 1)
    G, reach = _doubling(nxt.flip(1), dy.flip(1))
    G = (G + reach * after[:, None]).flip(1)
    first = torch.zeros_like(after) if s["state"] is None else s["state"]
    before = torch.cat((first[:, None], h[:, :-1]), 1)
    if s["state"] is not None:
        out["dstate"] = a[:, 0] * G[:, 0]
    gx = x if g is None else g * x
    dl = a * G * before                            # gradient of log a
    if c["mix"] == "convex":
        dl = dl - G * gx * a
    elif c["mix"] == "norm":
        dl = dl - torch.where(m > 0, G * gx * a * a / m, 0.0)
    z = s["z"].float()
    if c["gate"] == "sigmoid":
        dz = dl * d
    elif c["gate"] == "log":
        dz = dl
    else:
        p = torch.sigmoid(z)
        out["drate"] = -(dl * p if live is None else torch.where(live, dl * p, 0.0)).sum((0, 1))
        dz = -dl * s["rate"] * p * torch.sigmoid(-z)
    cut = (lambda t: t.to(dt)) if live is None else (lambda t: torch.where(live, t, 0.0).to(dt))
    out["dx"], out["dz"] = cut(G * m if g is None else G * m * g), cut(dz)
    if g is not None:
        out["di"] = cut(G * m * x * g * torch.sigmoid(-s["i"].float()))
    return out


def _plain_scan_step(s):
    a, d, m, g = _plain_gates(s)
    u = m * s["x"].float()
    at = s["slots"].long()
    h = a * s["state"][at] + (u if g is None else g * u)
    s["state"][at] = h
    return {"y": h.to(s["x"].dtype), "state": s["state"]}


# ---- the plain forms: norms of q and k with their positions --------------------------------------------

def _plain_turn(f, s, inverse):
    c, R = s["case"], s["case"]["rot"]
    if R == 0:
        return f
    angle = (s["positions"].double()[..., None] * s["inv_freq"].double())[:, None]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float() * (-1.0 if inverse else 1.0)
    if c["interleaved"]:
        a, b = f[..., 0:R:2], f[..., 1:R:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = f[..., : R // 2], f[..., R // 2: R]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, f[..., R:]), -1)


def _plain_qknorm(s):
    c, out = s["case"], {}
    for name in ("q", "k"):
        x, w = s[name].float(), s["w" + name].float()
        if c["centred"]:
            x = x - x.mean(-1, keepdim=True)
        rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
        xhat = x * rstd
        out[name] = _plain_turn(xhat * w, s, False).to(s[name].dtype)
        if c["op"] == "qknorm_train":
            dn = _plain_turn(s["d" + name].float(), s, True)
            out["dw" + name] = (dn * xhat).sum((0, 1, 2))
            h = dn * w
            dx = h - xhat * (h * xhat).mean(-1, keepdim=True)
            if c["centred"]:
                dx = dx - h.mean(-1, keepdim=True)
            out["d" + name] = (rstd * dx).to(s[name].dtype)
    return out


# ---- the plain forms: the short convolution ------------------------------------------------------------

def _plain_conv(s):
    c, dt = s["case"], s["x"].dtype
    B, N, C, K = (c[x] for x in ("B", "N", "C", "K"))
    live = _live(s["lengths"], s["x"].shape)
    zero = torch.zeros((), device="cuda")
    w = s["w"].float()
    first = torch.zeros((B, K - 1, C), device="cuda") if s["state"] is None else s["state"].float()
    x = s["x"].float() if live is None else torch.where(live, s["x"].float(), zero)
    x = torch.cat((first, x), 1)                   # token t stands at t + K - 1
    p = sum(w[:, j] * x[:, j:j + N] for j in range(K))
    if s["b"] is not None:
        p = p + s["b"].float()
    gate = torch.sigmoid(p)
    y = p * gate if c["silu"] else p
    if live is not None:
        y = torch.where(live, y, zero)
    n = torch.full((B,), N, device="cuda") if s["lengths"] is None else s["lengths"].long()
    at = (n[:, None] + torch.arange(K - 1, device="cuda"))[..., None].expand(B, K - 1, C)      # the last K - 1 inputs
    out = {"y": y.to(dt), "state": torch.gather(x, 1, at).to(dt)}
    if c["op"] == "conv":
        return out
    dp = s["dy"].float()
    if c["silu"]:
        dp = dp * gate * (1.0 + p * (1.0 - gate))
    if live is not None:
        dp = torch.where(live, dp, zero)
    dx = torch.zeros((B, N + K - 1, C), device="cuda")
    if s["dstate"] is not None:
        dx.scatter_(1, at, s["dstate"].float())
    for j in range(K):
        dx[:, j:j + N] += dp * w[:, j]
    out["dw"] = torch.stack([(dp * x[:, j:j + N]).sum((0, 1)) for j in range(K)], 1)
    if s["b"] is not None:
        out["db"] = dp.sum((0, 1))
    out["dx"] = (dx[:, K - 1:] if live is None else torch.where(live, dx[:, K - 1:], zero)).to(dt)
    if s["state"] is not None:
        out["dstate"] = dx[:, :K - 1].to(dt)
    return out


def _plain_conv_step(s):
    at = s["slots"].long()
    x = torch.cat((s["state"][at], s["x"][:, None]), 1)
    p = (x.float() * s["w"].float().t()).sum(1)
    if s["b"] is not None:
        p = p + s["b"].float()
    if s["case"]["silu"]:
        p = p * torch.sigmoid(p)
    s["state"][at] = x[:, 1:]
    return {"y": p.to(s["x"].dtype), "state": s["state"]}


# ---- one pass -------------------------------------------------------------------------------------

def _run_plain(s):
    op = s["case"]["op"]
    if op in ("scan", "scan_train"):
        return _plain_scan(s)
    if op == "scan_step":
        return _plain_scan_step(s)
    if op.startswith("qknorm"):
        return _plain_qknorm(s)
    return _plain_conv_step(s) if op == "conv_step" else _plain_conv(s)


def _own_scan(lconv, s):
    c = s["case"]
    how = dict(gate=c["gate"], mix=c["mix"], input_gate=s["i"], rate=s["rate"])
    if c["op"] == "scan_step":
        return {"y": lconv.gated_scan_step(s["x"], s["z"], s["state"], slots=s["slots"], **how), "state": s["state"]}
    train = c["op"] == "scan_train"
    y, state, marks = lconv.gated_scan(s["x"], s["z"], state=s["state"], lengths=s["lengths"], need_marks=train, **how)
    out = {"y": y, "state": state}
    if train:
        g = lconv.gated_scan_bwd(s["dy"], s["x"], s["z"], marks, dstate=s["dstate"], lengths=s["lengths"],
                                 need_dstate=s["state"] is not None, **how)
        out.update(dx=g.dx, dz=g.dz)
        for name, t in (("di", g.dinput_gate), ("drate", g.drate), ("dstate", g.dstate)):
            if t is not None:
                out[name] = t
    return out


def _own_qknorm(lconv, s):
    c = s["case"]
    how = dict(eps=s["eps"], centred=c["centred"], interleaved=c["interleaved"])
    q, k = lconv.qk_norm_rotary(s["q"], s["k"], s["wq"], s["wk"], s["positions"], s["inv_freq"], **how)
    out = {"q": q, "k": k}
    if c["op"] == "qknorm_train":
        g = lconv.qk_norm_rotary_bwd(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], s["positions"], s["inv_freq"], **how)
        out.update(dq=g.dq, dk=g.dk, dwq=g.dq_weight, dwk=g.dk_weight)
    return out


def _own_conv(lconv, s):
    c = s["case"]
    how = dict(bias=s["b"], activation="silu" if c["silu"] else None)
    if c["op"] == "conv_step":
        return {"y": lconv.short_conv_step(s["x"], s["w"], s["state"], slots=s["slots"], **how), "state": s["state"]}
    y, state = lconv.short_conv(s["x"], s["w"], state=s["state"], lengths=s["lengths"], **how)
    out = {"y": y, "state": state}
    if c["op"] == "conv_train":
        g = lconv.short_conv_bwd(s["dy"], s["x"], s["w"], state=s["state"], dstate=s["dstate"], lengths=s["lengths"], **how)
        out.update(dx=g.dx, dw=g.dweight)
        for name, t in (("db", g.dbias), ("dstate", g.dstate)):
            if t is not None:
                out[name] = t
    return out


def run(state):
    if not own:
        return _run_plain(state)
    from fft_long_convolution_amd import lconv
    op = state["case"]["op"]
    return (_own_scan if op.startswith("scan") else _own_qknorm if op.startswith("qknorm") else _own_conv)(lconv, state)


# ---- what a pass cannot do without -------------------------------------------------------------------

def work(case):
    c, e = case, SIZE[case["dtype"]]
    op = c["op"]
    if op.startswith("qknorm"):
        n = c["B"] * c["N"] * (c["H"] + c["G"]) * c["D"]
        side = 4 * c["B"] * c["N"] + 2 * e * c["D"]
        if op == "qknorm":
            return {"bytes": 2 * e * n + side, "flops": 7 * n}
        return {"bytes": 5 * e * n + side + 8 * c["D"], "flops": 22 * n}        # x, dy in; y, dx and the weights' gradients out
    rows, n = c["B"] * c["C"], c["B"] * c["C"] * c.get("N", 1)
    train = op.endswith("train")
    if op.startswith("scan"):
        inputs = 3 if c["gated"] else 2
        side = (4 * c["C"] if c["gate"] == "rate" else 0) * (2 if train else 1)
        if op == "scan_step":
            return {"bytes": e * n * (inputs + 1) + 8 * rows + side + 4 * c["B"], "flops": 20 * n}
        states = 4 * rows * (2 if c["state"] else 1)
        if op == "scan":
            return {"bytes": e * n * (inputs + 1) + states + side, "flops": 20 * n}
        return {"bytes": e * n * (2 * inputs + 2) + 2 * states + side, "flops": 55 * n}      # inputs, dy; y and the gradients
    K = c["K"]
    side = e * c["C"] * (K + (1 if c["bias"] else 0))
    if op == "conv_step":
        return {"bytes": e * n * 2 + 2 * e * rows * (K - 1) + side + 4 * c["B"], "flops": (2 * K + 5) * n}
    states = e * rows * (K - 1) * (2 if c["state"] else 1)
    if op == "conv":
        return {"bytes": 2 * e * n + states + side, "flops": (2 * K + 5) * n}
    return {"bytes": 4 * e * n + 2 * states + side + 4 * c["C"] * (K + (1 if c["bias"] else 0)), "flops": (6 * K + 14) * n}


# ---- the definitions in 64 bits -----------------------------------------------------------------------

def _exact_scan(s):
    """The recurrence token by token; the gradients by the chain rule, backwards."""
    c = s["case"]
    op = c["op"]
    wide = lambda t: None if t is None else t.double().reshape(c["B"], -1, c["C"])  # noqa: E731
    x, z, i = wide(s["x"]), wide(s["z"]), wide(s["i"])
    N = x.shape[1]
    n = [N] * c["B"] if s.get("lengths") is None else s["lengths"].tolist()
    n = torch.tensor(n, device="cuda")
    expit = lambda t: 1.0 / (1.0 + torch.exp(-t))  # noqa: E731
    rate = None if s["rate"] is None else s["rate"].double()

    def at(t):
        """Everything of token t: log a, a, 1 - a, m, the input's gate."""
        if c["gate"] == "log":
            la = z[:, t]
        elif c["gate"] == "sigmoid":
            la = -torch.log1p(torch.exp(-z[:, t]))
        else:
            la = -rate * expit(z[:, t])
        a, d = torch.exp(la), -torch.expm1(la)
        m = torch.ones_like(a) if c["mix"] == "plain" else d if c["mix"] == "convex" else torch.sqrt(-torch.expm1(2.0 * la))
        return la, a, d, m, torch.ones_like(a) if i is None else expit(i[:, t])

    if op == "scan_step":
        h = s["state"].double()
        h = h[s["slots"].long()] if "slots" in s else h
    else:
        h = torch.zeros(c["B"], c["C"], dtype=torch.float64, device="cuda") if s["state"] is None else s["state"].double()
    kept, y = [], torch.zeros_like(x)
    for t in range(N):
        la, a, d, m, g = at(t)
        on = (t < n)[:, None]
        if op == "scan_train":
            kept.append(h)
        new = a * h + m * g * x[:, t]
        y[:, t] = torch.where(on, new, 0.0)
        h = torch.where(on, new, h)
    if op == "scan_step":
        pool = s["state"].double()
        pool[s["slots"].long()] = h
        return {"y": y[:, 0], "state": pool}
    out = {"y": y, "state": h}
    if op == "scan":
        return out
    G = torch.zeros_like(h) if s["dstate"] is None else s["dstate"].double()      # of the state that follows
    dx, dz, di = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    drate = torch.zeros(c["C"], dtype=torch.float64, device="cuda")
    for t in range(N - 1, -1, -1):
        la, a, d, m, g = at(t)
        on = (t < n)[:, None]
        now = G + s["dy"][:, t].double()
        dx[:, t] = torch.where(on, now * m * g, 0.0)
        di[:, t] = torch.where(on, now * m * x[:, t] * g * (1.0 - g), 0.0)
        da = now * kept[t]
        if c["mix"] == "convex":
            da = da - now * g * x[:, t]
        elif c["mix"] == "norm":
            da = da - now * g * x[:, t] * a / m
        dla = da * a
        if c["gate"] == "sigmoid":
            dla = dla * d
        elif c["gate"] == "rate":
            p = expit(z[:, t])
            drate -= torch.where(on, dla * p, 0.0).sum(0)
            dla = -dla * rate * p * (1.0 - p)
        dz[:, t] = torch.where(on, dla, 0.0)
        G = torch.where(on, a * now, G)
    out.update(dx=dx, dz=dz)
    if i is not None:
        out["di"] = di
    if rate is not None:
        out["drate"] = drate
    if s["state"] is not None:
        out["dstate"] = G
    return out


def _exact_qknorm(s):
    """Rows as vectors, turned pairs as complex numbers; the norm's gradient as its Jacobian's product."""
    c, R, D, out = s["case"], s["case"]["rot"], s["case"]["D"], {}
    lo, hi = (slice(0, R, 2), slice(1, R, 2)) if c["interleaved"] else (slice(0, R // 2), slice(R // 2, R))
    angle = s["positions"].double()[:, None, :, None] * s["inv_freq"].double()
    turn = torch.polar(torch.ones_like(angle), angle)

    def turned(x, by):
        x = x.clone()
        if R:
            z = torch.complex(x[..., lo].contiguous(), x[..., hi].contiguous()) * by
            x[..., lo], x[..., hi] = z.real, z.imag
        return x

    for name in ("q", "k"):
        x, w = s[name].double(), s["w" + name].double()
        u = x - x.sum(-1, keepdim=True) / D if c["centred"] else x
        size = torch.sqrt((u * u).sum(-1, keepdim=True) / D + s["eps"])
        out[name] = turned(u / size * w, turn)
        if c["op"] == "qknorm_train":
            dn = turned(s["d" + name].double(), turn.conj())
            out["dw" + name] = (dn * u / size).sum((0, 1, 2))
            v = dn * w
            dx = v / size - u * (u * v).sum(-1, keepdim=True) / (D * size ** 3)
            out["d" + name] = dx - dx.sum(-1, keepdim=True) / D if c["centred"] else dx
    return out


def _exact_conv(s):
    """One row at a time, only its own tokens."""
    c = s["case"]
    K, C, w = c["K"], c["C"], s["w"].double()
    bias = torch.zeros(C, dtype=torch.float64, device="cuda") if s["b"] is None else s["b"].double()
    if c["op"] == "conv_step":
        at = s["slots"].long()
        pool = s["state"].double()
        x = torch.cat((pool[at], s["x"].double()[:, None]), 1)
        p = torch.einsum("bkc,ck->bc", x, w) + bias
        pool[at] = x[:, 1:]
        return {"y": p / (1.0 + torch.exp(-p)) if c["silu"] else p, "state": pool}
    B, N = c["B"], c["N"]
    zeros = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    out = {"y": zeros(B, N, C), "state": zeros(B, K - 1, C)}
    if c["op"] == "conv_train":
        out.update(dw=zeros(C, K), dx=zeros(B, N, C))
        if s["b"] is not None:
            out["db"] = zeros(C)
        if s["state"] is not None:
            out["dstate"] = zeros(B, K - 1, C)
    for b in range(B):
        n = N if s["lengths"] is None else int(s["lengths"][b])
        x = torch.cat((zeros(K - 1, C) if s["state"] is None else s["state"][b].double(), s["x"][b, :n].double()))
        out["state"][b] = x[n:]
        p = bias.expand(n, C).clone()
        for j in range(K):
            p += x[j:j + n] * w[:, j]
        sig = 1.0 / (1.0 + torch.exp(-p))
        out["y"][b, :n] = p * sig if c["silu"] else p
        if c["op"] == "conv":
            continue
        dp = s["dy"][b, :n].double()
        if c["silu"]:
            dp = dp * (sig + p * sig * (1.0 - sig))
        dx = zeros(n + K - 1, C)
        if s["dstate"] is not None:
            dx[n:] += s["dstate"][b].double()
        for j in range(K):
            dx[j:j + n] += dp * w[:, j]
            out["dw"][:, j] += (dp * x[j:j + n]).sum(0)
        out["dx"][b, :n] = dx[K - 1:]
        if s["b"] is not None:
            out["db"] += dp.sum(0)
        if s["state"] is not None:
            out["dstate"][b] = dx[:K - 1]
    return out


def exact(case, seed):
    op = case["op"]
    if op in ("scan", "scan_train"):
        # the recurrence is a few dozen passes over the states for every token; the gradients keep every state
        cost = case["N"] * (2e-4 + case["B"] * case["C"] * 4e-10) * (3 if op == "scan_train" else 1)
        if cost > 15.0 or (op == "scan_train" and 8 * case["B"] * case["C"] * case["N"] > 4e9):
            return None
    s = prepare(case, seed)
    return _exact_scan(s) if op.startswith("scan") else _exact_qknorm(s) if op.startswith("qknorm") else _exact_conv(s)
