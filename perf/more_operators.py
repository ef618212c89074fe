"""Workloads of the operators that a block of a sequence model needs between its recurrent layers, its linear attention
and its norms: the gated linear recurrence (prompts, training, single tokens), the norm of each head with its rotary
position (prompts, training, single tokens) and the gated feed-forward block (forward and backward).

`run` computes each in plain torch operations, in 32 bits (angles in 64), or (``own``) through this library's entry
points.  Sizes follow the library's recurrent workloads: widths 512, 1024 and 2048, heads of 64 or 128, sequences of 128
to 512 steps, batches of 1 to 256, longer sequences where the operator is meant for them, and feed-forward layers 2.75
times as wide as the model.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token for four users of a width-1024 layer, where only latency counts
        {"name": "rec_step_b4_w1024_bf16", "op": "rec_step", "B": 4, "slots": 5, "W": 1024, "dtype": "bf16",
         "gates": 1},
        # a long prompt of one request: few channels, so the sequence itself has to be spread over the card
        {"name": "rec_prompt_t16384_b1_w2048_bf16", "op": "rec_prompt", "T": 16384, "B": 1, "W": 2048,
         "dtype": "bf16", "gates": 1, "ragged": False, "state": False, "packed": True, "batch_first": False},
        # training at the shape of the width-2048 benchmark layer
        {"name": "rec_train_t512_b256_w2048_bf16", "op": "rec_train", "T": 512, "B": 256, "W": 2048, "dtype": "bf16",
         "gates": 1, "ragged": False, "state": False, "packed": False, "batch_first": False},
        # ragged training windows that continue earlier ones, an input gate of its own, odd width, fp32, batch-first
        {"name": "rec_train_t333_b5_w1001_f32", "op": "rec_train", "T": 333, "B": 5, "W": 1001, "dtype": "f32",
         "gates": 2, "ragged": True, "state": True, "packed": True, "batch_first": True},
        # a token for each of 16 requests, far into their texts
        {"name": "rot_step_b16_16x128_bf16", "op": "rot_forward", "T": 1, "B": 16, "H": 16, "Hkv": 8, "D": 128,
         "rot": 128, "interleaved": False, "norm": True, "far": 131072, "dtype": "bf16", "packed": True,
         "batch_first": False},
        # queries and keys of a long prompt
        {"name": "rot_prompt_t16384_b1_16x128_bf16", "op": "rot_forward", "T": 16384, "B": 1, "H": 16, "Hkv": 16,
         "D": 128, "rot": 128, "interleaved": False, "norm": True, "far": 0, "dtype": "bf16", "packed": True,
         "batch_first": False},
        # training over 512 steps of 256 rows, norm weights included
        {"name": "rot_train_t512_b256_16x128_bf16", "op": "rot_train", "T": 512, "B": 256, "H": 16, "Hkv": 8,
         "D": 128, "rot": 128, "interleaved": False, "norm": True, "far": 0, "dtype": "bf16", "packed": False,
         "batch_first": False},
        # training with odd head counts, part of the head rotated in neighbouring pairs, windows of longer texts, fp32
        {"name": "rot_train_t333_b5_6x72_f32", "op": "rot_train", "T": 333, "B": 5, "H": 6, "Hkv": 3, "D": 72,
         "rot": 40, "interleaved": True, "norm": True, "far": 1000000, "dtype": "f32", "packed": True,
         "batch_first": True},
        # the block for the tokens of four users: the weights' traffic
        {"name": "mlp_4x1024x2816_bf16", "op": "mlp_forward", "rows": 4, "in": 1024, "hidden": 2816, "out": 1024,
         "act": "silu", "dtype": "bf16"},
        # a serving batch of 256 tokens at width 2048
        {"name": "mlp_256x2048x5632_bf16", "op": "mlp_forward", "rows": 256, "in": 2048, "hidden": 5632, "out": 2048,
         "act": "silu", "dtype": "bf16"},
        # a training step over 16384 tokens at width 2048
        {"name": "mlp_train_16384x2048x5632_bf16", "op": "mlp_train", "rows": 16384, "in": 2048, "hidden": 5632,
         "out": 2048, "act": "silu", "dtype": "bf16"},
        # a training step in fp32 at the width of the fp32 benchmark layer, an odd number of tokens
        {"name": "mlp_train_8191x512x1408_f32", "op": "mlp_train", "rows": 8191, "in": 512, "hidden": 1408,
         "out": 512, "act": "gelu", "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    op = rng.choice(["rec_step", "rec_prompt", "rec_train", "rot_forward", "rot_train", "mlp_forward", "mlp_train"])
    dtype = rng.choice(["f32", "bf16", "bf16"])
    c = {"op": op, "dtype": dtype}
    if op == "rec_step":
        B = _log(rng, 1, 256)
        c.update(B=B, slots=B + rng.randint(0, B), W=rng.choice([512, 1024, 2048, _log(rng, 16, 4096)]),
                 gates=rng.choice([1, 2]))
    elif op.startswith("rec_"):
        W = rng.choice([512, 1024, 2048, _log(rng, 16, 4096)])
        T = _log(rng, 2, 16384 if op == "rec_prompt" else 2048)
        B = _log(rng, 1, max(1, min(256, (1 << (25 if dtype == "f32" else 27)) // (T * W))))
        c.update(T=T, B=B, W=W, gates=rng.choice([1, 2]), ragged=rng.random() < 0.4, state=rng.random() < 0.5,
                 packed=rng.random() < 0.5, batch_first=rng.random() < 0.5)
    elif op.startswith("rot_"):
        kv = rng.choice([1, 2, 3, 4, 8, 16])
        H = kv * rng.choice([g for g in (1, 1, 2, 4) if kv * g <= 16])
        D = rng.choice([64, 128, 128, 2 * rng.randint(4, 64), rng.randint(9, 256)])
        T = _log(rng, 1, 16384)
        B = _log(rng, 1, max(1, min(256, (1 << (25 if dtype == "f32" else 27)) // (T * (H + kv) * D))))
        c.update(T=T, B=B, H=H, Hkv=kv, D=D, rot=rng.choice([D // 2 * 2, D // 2 * 2, 2 * rng.randint(1, D // 2)]),
                 interleaved=rng.random() < 0.4, norm=rng.random() < 0.7, far=rng.choice([0, 4096, 131072, 1000000]),
                 packed=rng.random() < 0.5, batch_first=rng.random() < 0.5)
    else:
        wide = rng.choice([512, 1024, 2048, _log(rng, 24, 2048)])
        hidden = rng.choice([wide * 11 // 4, wide * 4, _log(rng, 32, 8192)])
        most = (1 << 34) if dtype == "f32" else (1 << 36)
        c.update({"rows": _log(rng, 1, max(1, min(16384, most // (wide * hidden)))), "in": wide, "hidden": hidden,
                  "out": rng.choice([wide, wide, _log(rng, 24, 2048)]), "act": rng.choice(["silu", "gelu", "sigmoid"])})
    return c


# ----------------------------------------------------------------- inputs
def _normal(gen, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * std).to(dtype)


def _frequencies(rot):
    return 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(1, rot)).to(DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 1000003 + 29)
    op, dt = case["op"], TYPES[case["dtype"]]
    s = {"case": dict(case)}
    if op.startswith("rec_"):
        B, W, gates = case["B"], case["W"], case["gates"]
        lead = (B,) if op == "rec_step" else (B, case["T"]) if case["batch_first"] else (case["T"], B)
        # channels that remember from about 2 to about 400 tokens
        keep = torch.linspace(0.0, 6.0, W, device=DEV)
        parts = [torch.randn(lead + (W,), generator=gen, device=DEV) for _ in range(1 + gates)]
        parts[1] += keep
        if op != "rec_step" and case["packed"]:  # one projection gave them side by side
            parts = torch.cat(parts, -1).to(dt).split(W, -1)
        else:
            parts = [p.to(dt) for p in parts]
        s["x"], s["forget"], s["input"] = parts[0], parts[1], parts[2] if gates == 2 else None
        if op == "rec_step":
            N = case["slots"]
            s["pool"] = _normal(gen, (N, W), torch.float32)
            # requests keep the slot that was free when they came; every ninth row of a larger batch is idle
            order = torch.randperm(N, generator=gen, device=DEV)[:B].to(torch.int32)
            s["slots"] = torch.where(torch.arange(B, device=DEV) % 9 == 8, torch.full_like(order, -1), order)
            return s
        s["state"] = _normal(gen, (B, W), torch.float32) if case["state"] else None
        s["lengths"] = None
        if case["ragged"]:  # any length from none to all of it, the first row full
            n = torch.randint(0, case["T"] + 1, (B,), generator=gen, device=DEV, dtype=torch.int32)
            n[0] = case["T"]
            s["lengths"] = n
        if op == "rec_train":
            s["dy"] = _normal(gen, lead + (W,), dt)
            s["dstate"] = _normal(gen, (B, W), torch.float32) if case["state"] else None
    elif op.startswith("rot_"):
        T, B, H, G, D = (case[n] for n in ("T", "B", "H", "Hkv", "D"))
        lead = (B, T) if case["batch_first"] else (T, B)
        if case["packed"]:  # queries, keys and values of one projection
            wide = _normal(gen, lead + ((H + 2 * G) * D,), dt)
            s["q"], s["k"] = wide[..., :H * D].unflatten(-1, (H, D)), wide[..., H * D:(H + G) * D].unflatten(-1, (G, D))
        else:
            s["q"], s["k"] = _normal(gen, lead + (H, D), dt), _normal(gen, lead + (G, D), dt)
        s["frequencies"] = _frequencies(case["rot"])
        s["positions"] = None
        if case["far"]:  # each row goes on where its text stands
            start = torch.randint(0, case["far"], (B,), generator=gen, device=DEV, dtype=torch.int32)
            at = torch.arange(T, device=DEV, dtype=torch.int32)
            s["positions"] = start.view(B, 1) + at if case["batch_first"] else at.view(T, 1) + start
        s["wq"] = s["wk"] = None
        if case["norm"]:
            s["wq"] = (1.0 + _normal(gen, (D,), torch.float32, 0.1)).to(dt)
            s["wk"] = (1.0 + _normal(gen, (D,), torch.float32, 0.1)).to(dt)
        if op == "rot_train":
            s["dq"], s["dk"] = _normal(gen, lead + (H, D), dt), _normal(gen, lead + (G, D), dt)
    else:
        rows, K, F, O = (case[n] for n in ("rows", "in", "hidden", "out"))
        s["x"] = _normal(gen, (rows, K), dt)
        s["w_gate"], s["w_up"] = _normal(gen, (F, K), dt, K ** -0.5), _normal(gen, (F, K), dt, K ** -0.5)
        s["w_down"] = _normal(gen, (O, F), dt, F ** -0.5)
        if op == "mlp_train":
            s["dy"] = _normal(gen, (rows, O), dt)
    return s


# ------------------------------------------------------------- plain forms
def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the first axis: spans of twice the length each time."""
    span = 1
    while span < a.shape[0]:
        b = torch.cat([b[:span], torch.addcmul(b[span:], a[span:], b[:-span])])
        a = torch.cat([a[:span], a[span:] * a[:-span]])
        span *= 2
    return b


def _plain_recurrence(s, grads):
    case = s["case"]
    dt, T, B = s["x"].dtype, case["T"], case["B"]
    seq = (lambda t: t.transpose(0, 1)) if case["batch_first"] else (lambda t: t)
    x, f = seq(s["x"]).float(), seq(s["forget"]).float()
    z, a = torch.sigmoid(-f), torch.sigmoid(f)
    w = z if s["input"] is None else torch.sigmoid(seq(s["input"]).float())
    live = None
    if s["lengths"] is not None:
        live = (torch.arange(T, device=x.device).view(T, 1) < s["lengths"].view(1, B)).unsqueeze(-1)
        # tokens past a row's end leave the state as it is
        a, x = torch.where(live, a, torch.ones_like(a)), torch.where(live, x, torch.zeros_like(x))
    first = torch.zeros_like(x[0]) if s["state"] is None else s["state"]
    b = w * x
    b[0] += a[0] * first
    h = _scan(a, b)
    shown = h if live is None else torch.where(live, h, torch.zeros_like(h))
    out = {"y": seq(shown.to(dt)), "state": h[-1].clone()}
    if not grads:
        return out
    d = seq(s["dy"]).float()
    if live is not None:
        d = torch.where(live, d, torch.zeros_like(d))
    if s["dstate"] is not None:
        d = torch.cat([d[:-1], d[-1:] + s["dstate"]])
    after = torch.cat([torch.zeros_like(a[:1]), a.flip(0)[:-1]])  # what the token before it passes back
    d = _scan(after, d.flip(0)).flip(0)
    if s["state"] is not None:
        out["dstate"] = a[0] * d[0]
    if live is not None:
        d = torch.where(live, d, torch.zeros_like(d))
    before = torch.cat([first.unsqueeze(0), h[:-1]])
    out["dx"] = seq((w * d).to(dt))
    if s["input"] is None:
        out["dforget"] = seq((d * (before - x) * z * (1 - z)).to(dt))
    else:
        out["dforget"] = seq((d * before * z * (1 - z)).to(dt))
        out["dinput"] = seq((d * x * w * (1 - w)).to(dt))
    return out


def _plain_recurrence_step(s):
    busy, at = (s["slots"] >= 0).unsqueeze(-1), s["slots"].clamp(min=0).long()
    x, f = s["x"].float(), s["forget"].float()
    z = torch.sigmoid(-f)
    w = z if s["input"] is None else torch.sigmoid(s["input"].float())
    h = torch.sigmoid(f) * s["pool"][at] + w * x
    N = s["pool"].shape[0]
    of = torch.full((N + 1,), -1, device=h.device)  # the row of each slot; idle rows name the place past the last
    of[torch.where(s["slots"] >= 0, at, N)] = torch.arange(s["case"]["B"], device=h.device)
    s["pool"].copy_(torch.where(of[:N].unsqueeze(-1) >= 0, h[of[:N].clamp(min=0)], s["pool"]))
    return {"y": torch.where(busy, h, torch.zeros_like(h)).to(s["x"].dtype), "pool": s["pool"]}


def _turn(u, cos, sin, rot, interleaved):
    """Pairs of the first `rot` values turned by their angles."""
    if interleaved:
        a, b = u[..., 0:rot:2], u[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = u[..., :rot // 2], u[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, u[..., rot:]], -1)


def _angles(s):
    case = s["case"]
    T, B = case["T"], case["B"]
    p = s["positions"]
    if p is None:
        p = torch.arange(T, device=DEV).view((1, T) if case["batch_first"] else (T, 1))
    angle = p.double().unsqueeze(-1).unsqueeze(-1) * s["frequencies"]
    return torch.cos(angle).float(), torch.sin(angle).float()


def _plain_rotary(s, grads):
    case = s["case"]
    rot, pairs, norm = case["rot"], case["interleaved"], case["norm"]
    cos, sin = _angles(s)
    out = {}
    for name, weight in (("q", "wq"), ("k", "wk")):
        x = s[name].float()
        u = x
        if norm:
            r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
            unit, w = x * r, s[weight].float()
            u = unit * w
        out[name] = _turn(u, cos, sin, rot, pairs).to(s[name].dtype)
        if grads:
            g = _turn(s["d" + name].float(), cos, -sin, rot, pairs)
            if norm:
                out["d" + weight] = (g * unit).sum((0, 1, 2)).to(s[name].dtype)
                g = g * w
                g = r * (g - unit * (g * unit).mean(-1, keepdim=True))
            out["d" + name] = g.to(s[name].dtype)
    return out


def _act(g, kind):
    """The activation and its slope."""
    if kind == "gelu":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g * g * g))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)
    p = torch.sigmoid(g)
    if kind == "sigmoid":
        return p, p * (1 - p)
    return g * p, p * (1 + g * (1 - p))


def _plain_mlp(s, grads):
    dt, kind = s["x"].dtype, s["case"]["act"]
    x, wg, wu, wd = (s[n].float() for n in ("x", "w_gate", "w_up", "w_down"))
    g, u = torch.matmul(x, wg.T), torch.matmul(x, wu.T)
    a, slope = _act(g, kind)
    h = a * u
    out = {"y": torch.matmul(h, wd.T).to(dt)}
    if grads:
        dy = s["dy"].float()
        dh = torch.matmul(dy, wd)
        dg, du = dh * u * slope, dh * a
        out["dx"] = (torch.matmul(dg, wg) + torch.matmul(du, wu)).to(dt)
        out["dw_gate"], out["dw_up"] = torch.matmul(dg.T, x).to(dt), torch.matmul(du.T, x).to(dt)
        out["dw_down"] = torch.matmul(dy.T, h).to(dt)
    return out


# -------------------------------------------------------------------- run
def _run_own(s):
    import layer_lstm_forward_amd as lib
    case = s["case"]
    op = case["op"]
    if op == "rec_step":
        y = lib.gated_recurrence_step(s["x"], s["forget"], s["pool"], input_gate=s["input"], slots=s["slots"])
        return {"y": y, "pool": s["pool"]}
    if op.startswith("rec_"):
        more = {"input_gate": s["input"], "state": s["state"], "lengths": s["lengths"],
                "batch_first": case["batch_first"]}
        y, last = lib.gated_recurrence(s["x"], s["forget"], **more)
        out = {"y": y, "state": last}
        if op == "rec_train":
            dx, df, di, dstate = lib.gated_recurrence_backward(s["x"], s["forget"], y, s["dy"], dstate=s["dstate"],
                                                               **more)
            out.update(dx=dx, dforget=df)
            if di is not None:
                out["dinput"] = di
            if dstate is not None:
                out["dstate"] = dstate
        return out
    if op.startswith("rot_"):
        more = {"positions": s["positions"], "q_weight": s["wq"], "k_weight": s["wk"], "norm": case["norm"],
                "eps": EPS, "interleaved": case["interleaved"], "batch_first": case["batch_first"]}
        q, k = lib.rotary(s["q"], s["k"], s["frequencies"], **more)
        out = {"q": q, "k": k}
        if op == "rot_train":
            dq, dk, dwq, dwk = lib.rotary_backward(s["q"], s["k"], s["frequencies"], s["dq"], s["dk"], **more)
            out.update(dq=dq, dk=dk)
            if case["norm"]:
                out.update(dwq=dwq, dwk=dwk)
        return out
    weights = (s["w_gate"], s["w_up"], s["w_down"])
    if op == "mlp_forward":
        return {"y": lib.gated_mlp(s["x"], *weights, activation=case["act"])}
    y, kept = lib.gated_mlp_train(s["x"], *weights, activation=case["act"])
    dx, dg, du, dd = lib.gated_mlp_backward(s["dy"], s["x"], *weights, kept, activation=case["act"])
    return {"y": y, "dx": dx, "dw_gate": dg, "dw_up": du, "dw_down": dd}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "rec_step":
        return _plain_recurrence_step(state)
    if op.startswith("rec_"):
        return _plain_recurrence(state, op == "rec_train")
    if op.startswith("rot_"):
        return _plain_rotary(state, op == "rot_train")
    return _plain_mlp(state, op == "mlp_train")


# ------------------------------------------------------------------- work
def work(case):
    op, size = case["op"], 4 if case["dtype"] == "f32" else 2
    if op == "rec_step":
        rows, W = case["B"] - case["B"] // 9, case["W"]  # the others are idle
        return {"bytes": rows * W * (8 + size * (1 + case["gates"])) + case["B"] * W * size, "flops": 10 * rows * W}
    if op.startswith("rec_"):
        T, B, W, gates = case["T"], case["B"], case["W"], case["gates"]
        n = T * B * W
        read = n * (0.5 + 0.5 / B if case["ragged"] else 1.0)
        states = B * W * 4
        nbytes, flops = size * (read * (1 + gates) + n) + states * (2 if case["state"] else 1), 10 * read
        if op == "rec_train":
            nbytes += size * (read * (3 + gates) + n * (1 + gates)) + states * (3 if case["state"] else 0)
            flops += 16 * read
        return {"bytes": nbytes, "flops": flops}
    if op.startswith("rot_"):
        n = case["T"] * case["B"] * (case["H"] + case["Hkv"]) * case["D"]
        train = op == "rot_train"
        return {"bytes": size * n * (5 if train else 2), "flops": n * (20 if train else 8)}
    rows, K, F, O = (case[n] for n in ("rows", "in", "hidden", "out"))
    product = 2 * rows * F * (2 * K + O)
    weights = F * (2 * K + O)
    nbytes = size * (rows * (K + O) + weights)
    if op == "mlp_forward":
        return {"bytes": nbytes, "flops": product}
    return {"bytes": nbytes + size * (rows * (2 * K + O) + 2 * weights), "flops": 3 * product}


# ------------------------------------------------------------------ exact
def _exact_recurrence(case, s):
    T, B, W = case["T"], case["B"], case["W"]
    at = (lambda t, i: t[:, i]) if case["batch_first"] else (lambda t, i: t[i])
    n = torch.full((B,), T, device=DEV) if s["lengths"] is None else s["lengths"]
    h = torch.zeros(B, W, dtype=torch.float64, device=DEV) if s["state"] is None else s["state"].double()
    shape = (B, T, W) if case["batch_first"] else (T, B, W)
    y = torch.zeros(shape, dtype=torch.float64, device=DEV)
    grads = case["op"] == "rec_train"
    kept = []
    for t in range(T):
        on = (t < n)[:, None]
        x, keep = at(s["x"], t).double(), 1 / (1 + torch.exp(-at(s["forget"], t).double()))
        take = 1 - keep if s["input"] is None else 1 / (1 + torch.exp(-at(s["input"], t).double()))
        if grads:
            kept.append(h)
        new = keep * h + take * x
        h = torch.where(on, new, h)
        at(y, t).copy_(torch.where(on, new, 0.0))
    out = {"y": y, "state": h}
    if grads:
        dx, df, di = (torch.zeros(shape, dtype=torch.float64, device=DEV) for _ in range(3))
        D = torch.zeros_like(h) if s["dstate"] is None else s["dstate"].double()
        for t in range(T - 1, -1, -1):
            on = (t < n)[:, None]
            x, keep = at(s["x"], t).double(), 1 / (1 + torch.exp(-at(s["forget"], t).double()))
            take = 1 - keep if s["input"] is None else 1 / (1 + torch.exp(-at(s["input"], t).double()))
            total = D + at(s["dy"], t).double()
            at(dx, t).copy_(torch.where(on, take * total, 0.0))
            slope = keep * (1 - keep)
            if s["input"] is None:
                at(df, t).copy_(torch.where(on, total * (kept[t] - x) * slope, 0.0))
            else:
                at(df, t).copy_(torch.where(on, total * kept[t] * slope, 0.0))
                at(di, t).copy_(torch.where(on, total * x * take * (1 - take), 0.0))
            D = torch.where(on, keep * total, D)
        out.update(dx=dx, dforget=df)
        if s["input"] is not None:
            out["dinput"] = di
        if s["state"] is not None:
            out["dstate"] = D
    return out


def _exact_recurrence_step(case, s):
    pool, y = s["pool"].double(), torch.zeros(case["B"], case["W"], dtype=torch.float64, device=DEV)
    for b in range(case["B"]):
        i = int(s["slots"][b])
        if i >= 0:
            keep = 1 / (1 + torch.exp(-s["forget"][b].double()))
            take = 1 - keep if s["input"] is None else 1 / (1 + torch.exp(-s["input"][b].double()))
            pool[i] = keep * pool[i] + take * s["x"][b].double()
            y[b] = pool[i]
    return {"y": y, "pool": pool}


def _exact_rotary(case, s):
    """Pairs as complex numbers."""
    rot, D = case["rot"], case["D"]
    if s["positions"] is not None:
        p = s["positions"].double()
    else:
        p = torch.arange(case["T"], dtype=torch.float64, device=DEV)
        p = p[None, :] if case["batch_first"] else p[:, None]
    angle = p[:, :, None, None] * s["frequencies"]
    wheel = torch.complex(torch.cos(angle), torch.sin(angle))
    if case["interleaved"]:
        order = torch.arange(rot, device=DEV)
    else:
        order = torch.arange(rot, device=DEV).view(2, rot // 2).T.reshape(-1)

    def turned(u, by):
        out = u.clone()
        pair = u[..., order]
        pair = torch.view_as_real(torch.complex(pair[..., 0::2], pair[..., 1::2]) * by).flatten(-2)
        out[..., order] = pair
        return out

    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        unit = x
        if case["norm"]:
            power = (x ** 2).sum(-1, keepdim=True) / D + EPS
            unit, w = x * power ** -0.5, s["w" + name].double()
            out[name] = turned(unit * w, wheel)
        else:
            out[name] = turned(x, wheel)
        if case["op"] == "rot_train":
            g = turned(s["d" + name].double(), wheel.conj())
            if case["norm"]:
                out["dw" + name] = (g * unit).flatten(0, 2).sum(0)
                v = g * w
                g = (v - x * ((v * x).sum(-1, keepdim=True) / (D * power))) * power ** -0.5
            out["d" + name] = g
    return out


def _exact_mlp(case, s):
    def slope(g):
        """act(g) and act'(g) from their definitions."""
        if case["act"] == "gelu":
            k = (2 / math.pi) ** 0.5
            inner, rise = k * (g + 0.044715 * g ** 3), k * (1 + 0.134145 * g ** 2)
            p = 1 / (1 + torch.exp(-2 * inner))  # (1 + tanh) / 2
            return g * p, p + g * 2 * p * (1 - p) * rise
        p = 1 / (1 + torch.exp(-g))
        return (p, p - p ** 2) if case["act"] == "sigmoid" else (p * g, p + p * g - p ** 2 * g)

    x, wg, wu, wd = (s[n].double() for n in ("x", "w_gate", "w_up", "w_down"))
    g, u = x @ wg.T, x @ wu.T
    a, rise = slope(g)
    out = {"y": (a * u) @ wd.T}
    if case["op"] == "mlp_train":
        dy = s["dy"].double()
        out["dw_down"] = dy.T @ (a * u)
        dh = dy @ wd
        du = dh * a
        dg = dh * u * rise
        out["dx"] = dg @ wg + du @ wu
        out["dw_gate"], out["dw_up"] = dg.T @ x, du.T @ x
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rec_step":
        return _exact_recurrence_step(case, s)
    if case["op"].startswith("rec_"):
        return _exact_recurrence(case, s)
    if case["op"].startswith("rot_"):
        return _exact_rotary(case, s)
    return _exact_mlp(case, s)
