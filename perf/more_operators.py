"""Cases, plain forms and exact values of the operators that mix a sequence along
time beside the linear attention: the short causal convolution, the selective
state space scan that follows it, and the rotary positions of the attention's
queries and keys.

Layouts.  Token rows are (batch, length, channels); B and C of the scan are
(batch, length, groups, states); heads are (batch, length, heads, head width).
"""
import math
import random

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one frame of 64 running simulations out of 96 slots: the last inputs of
        # each are kept between calls, and the call itself is the cost
        {"name": "conv_step", "op": "conv_step", "batch": 64, "slots": 96, "channels": 1024,
         "width": 4, "silu": True, "bias": True, "dtype": "bf16"},
        # 12 frames at each point of a 64 x 64 grid, the channels of the FNO stack:
        # very many short sequences
        {"name": "conv_frames", "op": "conv_fwd", "batch": 4096, "length": 12, "channels": 64,
         "width": 4, "silu": True, "bias": True, "ragged": False, "state": False,
         "dtype": "f32"},
        # a long prompt that continues earlier ones
        {"name": "conv_prompt", "op": "conv_fwd", "batch": 4, "length": 8192, "channels": 2048,
         "width": 4, "silu": True, "bias": True, "ragged": False, "state": True,
         "dtype": "bf16"},
        # training on uneven sequences, one of them empty; odd sizes
        {"name": "conv_grad", "op": "conv_bwd", "batch": 5, "length": 4099, "channels": 1001,
         "width": 3, "silu": True, "bias": True, "ragged": True, "state": False,
         "dtype": "f16"},
        # one frame of the same 64 simulations through the scan
        {"name": "scan_step", "op": "scan_step", "batch": 64, "slots": 96, "channels": 1024,
         "states": 16, "groups": 1, "gate": True, "skip": True, "dtype": "bf16"},
        # 12 frames at each point of a 64 x 64 grid
        {"name": "scan_frames", "op": "scan_fwd", "batch": 4096, "length": 12, "channels": 64,
         "states": 16, "groups": 1, "gate": False, "skip": True, "ragged": False,
         "state": False, "dtype": "f32"},
        # one long prompt, odd length: few rows, so the time axis has to be split
        {"name": "scan_prompt", "op": "scan_fwd", "batch": 1, "length": 8191, "channels": 2048,
         "states": 16, "groups": 1, "gate": True, "skip": True, "ragged": False,
         "state": True, "dtype": "bf16"},
        # training on the frames of a 32 x 32 grid, two samples
        {"name": "scan_frames_grad", "op": "scan_bwd", "batch": 2048, "length": 12,
         "channels": 64, "states": 16, "groups": 1, "gate": True, "skip": True,
         "ragged": False, "state": False, "dtype": "f32"},
        # training on long sequences
        {"name": "scan_grad", "op": "scan_bwd", "batch": 2, "length": 4096, "channels": 1024,
         "states": 16, "groups": 1, "gate": True, "skip": True, "ragged": False,
         "state": False, "dtype": "bf16"},
        # the queries and keys of one frame of 64 simulations, far into their run, by
        # frequencies that are scaled for long contexts
        {"name": "rotary_step", "op": "rotary_fwd", "batch": 64, "length": 1, "heads": 16,
         "kv_heads": 4, "dim": 64, "rotary_dim": 64, "layout": "half", "scaling": "ramp",
         "positions": "offset", "dtype": "f16"},
        # a prompt with shared key heads
        {"name": "rotary_prompt", "op": "rotary_fwd", "batch": 4, "length": 8192, "heads": 16,
         "kv_heads": 4, "dim": 128, "rotary_dim": 128, "layout": "half", "scaling": "none",
         "positions": "none", "dtype": "bf16"},
        # gradients of a rotation of half of each head, neighbouring pairs, positions
        # of every token (sequences packed behind one another), odd length
        {"name": "rotary_grad", "op": "rotary_bwd", "batch": 3, "length": 4097, "heads": 12,
         "kv_heads": 12, "dim": 80, "rotary_dim": 40, "layout": "interleaved",
         "scaling": "linear", "positions": "token", "dtype": "f32"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv_step", "conv_fwd", "conv_bwd", "scan_step", "scan_fwd", "scan_bwd",
                     "rotary_fwd", "rotary_bwd"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    half = 2 if dtype == "f32" else 1
    if op.startswith("rotary"):
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 1, 2, 4])
        dim = rng.choice([32, 48, 64, 80, 128, 256])
        batch = _log_int(rng, 1, 64)
        most = 4 * 8192 * 20 * 128 // (half * batch * (heads + kv) * dim)
        return {"op": op, "batch": batch, "length": _log_int(rng, 1, max(1, min(16384, most))),
                "heads": heads, "kv_heads": kv, "dim": dim,
                "rotary_dim": rng.choice([dim, dim // 2, 2 * (dim // 3)]),
                "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["none", "linear", "base", "ramp"]),
                "positions": rng.choice(["none", "offset", "token"]), "dtype": dtype}
    if op.startswith("conv"):
        case = {"op": op, "width": rng.choice([2, 3, 4, 4, 5, 8]), "silu": rng.random() < 0.7,
                "bias": rng.random() < 0.7, "dtype": dtype}
    else:
        states = rng.choice([1, 4, 8, 16, 16, 16, 24, 64])
        groups = rng.choice([1, 1, 1, 2, 4])
        case = {"op": op, "states": states, "groups": groups, "gate": rng.random() < 0.6,
                "skip": rng.random() < 0.7, "dtype": dtype}
    unit = case.get("groups", 1)
    if op.endswith("step"):
        batch = _log_int(rng, 1, 128)
        case.update(batch=batch, slots=batch + rng.randrange(0, 33),
                    channels=unit * max(1, _log_int(rng, 16, 2048) // unit))
        return case
    channels = unit * max(1, _log_int(rng, 8, 2048) // unit)
    most = 4 * 8192 * 2048 // (half * (2 if op == "conv_bwd" else 1))
    if op.startswith("scan"):
        most = min(most // 4, 8191 * 2048 * 16 // (case["states"] * (2 if op == "scan_bwd"
                                                                       else 1)))
    batch = _log_int(rng, 1, min(4096, most // channels))
    case.update(batch=batch, channels=channels,
                length=_log_int(rng, 1, max(1, min(16384, most // (batch * channels)))),
                ragged=rng.random() < 0.5, state=rng.random() < 0.5)
    return case


def _lengths(case):
    """Valid tokens of each sequence: the first is full, the second empty, the
    others in between (a property of the case, not of the seed)."""
    if not case["ragged"] or case["batch"] == 1:
        return [case["length"]] * case["batch"]
    r = random.Random(case["batch"] * 1000003 + case["length"])
    return [case["length"], 0] + [r.randint(1, case["length"])
                                  for _ in range(case["batch"] - 2)]


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    if op.startswith("rotary"):
        rows = case["batch"] * case["length"]
        heads = case["heads"] + case["kv_heads"]
        where = {"none": 0, "offset": 4 * case["batch"], "token": 4 * rows}[case["positions"]]
        return {"bytes": 2 * e * rows * heads * case["dim"] + where,
                "flops": 3 * rows * heads * case["rotary_dim"]}
    D, B = case["channels"], case["batch"]
    if op.startswith("conv"):
        W = case["width"]
        per = 2 * W + (6 if case["silu"] else 0)
        weights = 4 * D * (W + 1)
        state = e * B * (W - 1) * D
        if op == "conv_step":
            return {"bytes": 2 * e * B * D + 2 * state + weights, "flops": per * B * D}
        n, every = sum(_lengths(case)) * D, B * case["length"] * D
        if op == "conv_fwd":
            return {"bytes": e * (n + every) + (2 if case["state"] else 1) * state + weights,
                    "flops": per * n}
        return {"bytes": e * (2 * n + every) + (3 if case["state"] else 0) * state + 2 * weights,
                "flops": (per + 4 * W + 6) * n}
    N, G = case["states"], case["groups"]
    state = 4 * B * D * N
    weights = 4 * D * (N + 2)
    rows = 3 if case["gate"] else 2               # x, dt and the gate
    if op == "scan_step":
        return {"bytes": e * B * (D * (rows + 1) + 2 * G * N) + 2 * state + weights,
                "flops": 7 * B * D * N + 20 * B * D}
    n, every = sum(_lengths(case)), B * case["length"]
    if op == "scan_fwd":
        return {"bytes": e * (n * (rows * D + 2 * G * N) + every * D) + weights
                + (2 if case["state"] else 1) * state,
                "flops": n * D * (7 * N + 20)}
    return {"bytes": e * (n * ((rows + 1) * D + 2 * G * N) + every * (rows * D + 2 * G * N))
            + 2 * weights + (3 if case["state"] else 0) * state,
            "flops": n * D * (22 * N + 40)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        s["plan"] = _plan(case)
    return s


ROTARY = {"base": 10000.0, "factor": 8.0, "original": 4096, "fast": 32.0, "slow": 1.0}


def _plan(case):
    """The plan (a description of the shapes) that a program makes once."""
    import fft_gemm_ifft_gb300 as fno
    op = case["op"]
    if op.startswith("rotary"):
        r = ROTARY
        scaling = {"none": None, "linear": ("linear", r["factor"]),
                   "base": ("base", r["factor"]),
                   "ramp": ("ramp", r["factor"], r["original"], r["fast"], r["slow"])}
        return fno.Rotary(case["batch"], case["length"], case["heads"], case["kv_heads"],
                          case["dim"], rotary_dim=case["rotary_dim"], layout=case["layout"],
                          base=r["base"], scaling=scaling[case["scaling"]], dtype=case["dtype"])
    back = op.endswith("bwd")
    if op.startswith("conv"):
        return fno.CausalConv(case["batch"], case.get("length", 1), case["channels"],
                              case["width"], act="silu" if case["silu"] else "none",
                              dtype=case["dtype"], backward=back)
    return fno.SelectiveScan(case["batch"], case.get("length", 1), case["channels"],
                             case["states"], groups=case["groups"], softplus=True,
                             dtype=case["dtype"], backward=back)


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DT[case["dtype"]]
    op = case["op"]
    s = {"case": case}

    def rnd(*shape, scale=1.0, mean=0.0):
        return mean + scale * torch.randn(shape, generator=g, device="cuda")

    if op.startswith("rotary"):
        B, T = case["batch"], case["length"]
        for name, h in (("q", case["heads"]), ("k", case["kv_heads"])):
            s[name] = rnd(B, T, h, case["dim"]).to(dt)
        s["offsets"] = s["positions"] = None
        if case["positions"] == "offset":
            s["offsets"] = torch.randint(0, 1 << 20, (B,), generator=g, device="cuda",
                                         dtype=torch.int32)
        elif case["positions"] == "token":
            # several sequences behind one another in each row
            start = torch.randint(0, 2 * T, (B, 1), generator=g, device="cuda")
            s["positions"] = ((torch.arange(T, device="cuda")[None] + start) % (T // 2 + 1)
                              ).to(torch.int32).contiguous()
        return s

    B, D = case["batch"], case["channels"]
    step = op.endswith("step")
    T = 1 if step else case["length"]

    def rows(*width, scale=1.0, mean=0.0):
        t = rnd(B, T, *width, scale=scale, mean=mean)
        return (t[:, 0] if step else t).contiguous().to(dt)

    s["x"] = rows(D)
    if op.startswith("conv"):
        W = case["width"]
        s["w"] = rnd(D, W, scale=W ** -0.5)
        s["bias"] = rnd(D, scale=0.2) if case["bias"] else None
        shape, kind = (W - 1, D), dt
    else:
        N, G = case["states"], case["groups"]
        # steps of 0.001 to 0.1 around which the data moves, decays of 1 .. N a unit
        s["dt"] = rows(D, scale=0.5)
        low, high = math.log(1e-3), math.log(1e-1)
        unit = torch.exp(low + (high - low) * torch.rand(D, generator=g, device="cuda"))
        s["dt_bias"] = torch.log(torch.expm1(unit))
        s["A"] = (-torch.arange(1, N + 1, device="cuda").float()
                  * torch.exp(rnd(D, N, scale=0.1))).contiguous()
        s["B"], s["C"] = rows(G, N), rows(G, N)
        s["D"] = rnd(D, scale=0.2, mean=1.0) if case["skip"] else None
        s["z"] = rows(D) if case["gate"] else None
        shape, kind = (D, N), torch.float32
    if step:
        n = case["slots"]
        s["state"] = rnd(n, *shape).to(kind)
        s["new"] = s["state"].clone()
        # each running simulation's slot; about one row in sixteen is idle (-1)
        slot = torch.randperm(n, generator=g, device="cuda")[:B].to(torch.int32)
        idle = torch.rand(B, generator=g, device="cuda") < 1.0 / 16
        s["slots"] = torch.where(idle, torch.full_like(slot, -1), slot)
        return s
    s["lengths"] = (torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
                    if case["ragged"] else None)
    s["s0"] = rnd(B, *shape).to(kind) if case["state"] else None
    if op.endswith("bwd"):
        s["dy"] = rows(D)
        s["dsT"] = rnd(B, *shape).to(kind) if case["state"] else None
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    op, p = s["case"]["op"], s["plan"]
    if op.startswith("rotary"):
        call = p.forward if op == "rotary_fwd" else p.backward
        q, k = call(s["q"], s["k"], positions=s["positions"], offsets=s["offsets"])
        return {"q": q, "k": k}
    if op == "conv_step":
        y = p.step(s["x"], s["w"], s["state"], bias=s["bias"], slots=s["slots"],
                   new_state=s["new"])
        return {"y": y, "state": s["new"]}
    if op == "conv_fwd":
        y, sT = p.forward(s["x"], s["w"], bias=s["bias"], lengths=s["lengths"], state=s["s0"],
                          want_state=True)
        return {"y": y, "state": sT}
    if op == "conv_bwd":
        d = p.backward(s["x"], s["w"], s["dy"], bias=s["bias"], lengths=s["lengths"],
                       state=s["s0"], dstate=s["dsT"])
        return {k: v for k, v in zip(("dx", "dw", "dbias", "dstate"), d) if v is not None}
    more = {"D": s["D"], "z": s["z"], "dt_bias": s["dt_bias"]}
    if op == "scan_step":
        y = p.step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], slots=s["slots"],
                   new_state=s["new"], **more)
        return {"y": y, "state": s["new"]}
    more.update(lengths=s["lengths"], state=s["s0"])
    if op == "scan_fwd":
        y, sT = p.forward(s["x"], s["dt"], s["A"], s["B"], s["C"], want_state=True, **more)
        return {"y": y, "state": sT}
    return p.backward(s["x"], s["dt"], s["A"], s["B"], s["C"], s["dy"], dstate=s["dsT"], **more)


# --- the plain form: elementary operations in 32 bits (64 for the angles) ----
def _run_plain(s):
    op = s["case"]["op"]
    if op.startswith("rotary"):
        return _plain_rotary(s)
    if op.endswith("step"):
        return _plain_step(s)
    return _plain_conv(s) if op.startswith("conv") else _plain_scan(s)


def _frequencies(case, device):
    """Radians a position of each pair, in 64 bits."""
    r, p = case["rotary_dim"], ROTARY
    base = p["base"]
    if case["scaling"] == "base" and r > 2:
        base = base * p["factor"] ** (r / (r - 2))
    f = base ** (-torch.arange(0, r, 2, device=device, dtype=torch.float64) / r)
    if case["scaling"] == "linear":
        f = f / p["factor"]
    elif case["scaling"] == "ramp":
        # turns over the original length: many keep their frequency, few are slowed
        turns = p["original"] * f / (2.0 * math.pi)
        keep = ((turns - p["slow"]) / (p["fast"] - p["slow"])).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / p["factor"])
    return f


def _magnitude(case):
    return 1.0 + 0.1 * math.log(ROTARY["factor"]) if case["scaling"] == "ramp" else 1.0


def _plain_rotary(s):
    case = s["case"]
    dt, r = DT[case["dtype"]], case["rotary_dim"]
    at = torch.arange(case["length"], device="cuda")[None]
    if s["positions"] is not None:
        at = s["positions"].long()
    elif s["offsets"] is not None:
        at = at + s["offsets"].long()[:, None]
    angle = at.double()[..., None] * _frequencies(case, "cuda")
    mag = _magnitude(case)
    cos = (mag * torch.cos(angle)).float()[:, :, None]
    sin = (mag * torch.sin(angle)).float()[:, :, None]
    if case["op"] == "rotary_bwd":
        sin = -sin
    out = {}
    for name in ("q", "k"):
        x = s[name].float()
        if case["layout"] == "half":
            a, b = x[..., :r // 2], x[..., r // 2:r]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = x[..., 0:r:2], x[..., 1:r:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        out[name] = torch.cat([y, x[..., r:]], -1).to(dt)
    return out


def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _softplus(v):
    return v.clamp(min=0.0) + torch.log1p(torch.exp(-v.abs()))


def _mask(s):
    case = s["case"]
    if s["lengths"] is None:
        return torch.ones((case["batch"], case["length"], 1), device="cuda")
    at = torch.arange(case["length"], device="cuda")[None]
    return (at < s["lengths"][:, None]).float()[..., None]


def _plain_conv(s):
    case, dt = s["case"], DT[s["case"]["dtype"]]
    B, T, D, W = (case[k] for k in ("batch", "length", "channels", "width"))
    m = _mask(s)
    x, w = s["x"].float() * m, s["w"]
    first = torch.zeros((B, W - 1, D), device="cuda") if s["s0"] is None else s["s0"].float()
    full = torch.cat([first, x], 1)
    pre = sum(full[:, j:j + T] * w[:, j] for j in range(W))
    if s["bias"] is not None:
        pre = pre + s["bias"]
    # the last W - 1 inputs of a sequence of n tokens are full[n : n + W - 1]
    n = (torch.full((B,), T, device="cuda") if s["lengths"] is None else s["lengths"].long())
    tail = (n[:, None] + torch.arange(W - 1, device="cuda"))[..., None].expand(B, W - 1, D)
    if case["op"] == "conv_fwd":
        y = pre * _sigmoid(pre) if case["silu"] else pre
        return {"y": (y * m).to(dt), "state": torch.gather(full, 1, tail).to(dt)}
    dp = s["dy"].float() * m
    if case["silu"]:
        g = _sigmoid(pre)
        dp = dp * g * (1.0 + pre * (1.0 - g))
    dfull = torch.zeros_like(full)
    for j in range(W):
        dfull[:, j:j + T] += dp * w[:, j]
    if s["dsT"] is not None:
        dfull.scatter_add_(1, tail, s["dsT"].float())
    out = {"dx": (dfull[:, W - 1:] * m).to(dt),
           "dw": torch.stack([(dp * full[:, j:j + T]).sum((0, 1)) for j in range(W)], 1)}
    if s["bias"] is not None:
        out["dbias"] = dp.sum((0, 1))
    if s["s0"] is not None:
        out["dstate"] = dfull[:, :W - 1].to(dt)
    return out


def _walk(a, b):
    """h_t = a_t h_{t-1} + b_t along axis 1 by doubling steps (h_{-1} = 0)."""
    k, T = 1, a.shape[1]
    while k < T:
        b = torch.cat([b[:, :k], b[:, k:] + a[:, k:] * b[:, :-k]], 1)
        if 2 * k < T:
            a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def _plain_scan(s):
    case, dt = s["case"], DT[s["case"]["dtype"]]
    per = case["channels"] // case["groups"]
    m = _mask(s)
    x = s["x"].float() * m
    v = s["dt"].float() + s["dt_bias"]
    v = torch.where(m > 0, v, torch.zeros_like(v))
    step = _softplus(v) * m
    Bc, Cc = ((s[k].float() * m[..., None]).repeat_interleave(per, 2) for k in ("B", "C"))
    a = torch.exp(step[..., None] * s["A"])
    b = (step * x)[..., None] * Bc
    s0 = torch.zeros_like(a[:, 0]) if s["s0"] is None else s["s0"]
    b[:, 0] += a[:, 0] * s0
    h = _walk(a, b)
    if case["op"] == "scan_fwd":
        del a, b
        y = (h * Cc).sum(-1)
        last = h[:, -1].clone()
        if s["D"] is not None:
            y = y + s["D"] * x
        if s["z"] is not None:
            z = s["z"].float()
            y = y * z * _sigmoid(z)
        return {"y": torch.where(m > 0, y, torch.zeros_like(y)).to(dt), "state": last}
    del b
    dy = s["dy"].float() * m
    out = {}
    if s["z"] is not None:
        z = torch.where(m > 0, s["z"].float(), torch.zeros_like(x))
        g = _sigmoid(z)
        y = (h * Cc).sum(-1)
        if s["D"] is not None:
            y = y + s["D"] * x
        out["dz"] = (dy * y * g * (1.0 + z * (1.0 - g))).to(dt)
        dy = dy * z * g
    # the gradient of every state: gh_t = C_t dy_t + a_{t+1} gh_{t+1}
    own_part = Cc * dy[..., None]
    if s["dsT"] is not None:
        own_part[:, -1] += s["dsT"]
    later = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    gh = _walk(later.flip(1), own_part.flip(1)).flip(1)
    del later, own_part
    before = torch.cat([s0[:, None], h[:, :-1]], 1)
    if s["s0"] is not None:
        out["dstate"] = a[:, 0] * gh[:, 0]
    through = gh * a * before
    del a, before
    out["dA"] = (through * step[..., None]).sum((0, 1))
    dstep = (through * s["A"]).sum(-1)
    del through
    shape = (case["batch"], case["length"], case["groups"], per, case["states"])
    out["dC"] = (h * dy[..., None]).view(shape).sum(3).to(dt)
    del h
    out["dB"] = (gh * (step * x)[..., None]).view(shape).sum(3).to(dt)
    inner = (gh * Bc).sum(-1)
    dx = step * inner
    if s["D"] is not None:
        dx = dx + s["D"] * dy
        out["dD"] = (dy * x).sum((0, 1))
    ddt = (dstep + x * inner) * _sigmoid(v) * m
    out["ddt_bias"] = ddt.sum((0, 1))
    out["dx"], out["ddt"] = (dx * m).to(dt), ddt.to(dt)
    return out


def _scatter_rows(s, new):
    """``s["state"]`` with row b's new state in its slot; idle rows change nothing."""
    live, n = s["slots"] >= 0, s["case"]["slots"]
    at = s["slots"].long()
    row = torch.full((n + 1,), -1, device="cuda").scatter(
        0, torch.where(live, at, torch.full_like(at, n)),
        torch.arange(s["case"]["batch"], device="cuda"))[:n]
    return torch.where((row >= 0)[:, None, None], new[row.clamp(min=0)], s["state"])


def _plain_step(s):
    case, dt = s["case"], DT[s["case"]["dtype"]]
    live = (s["slots"] >= 0)[:, None]
    x, state = s["x"].float(), s["state"][s["slots"].clamp(min=0).long()]
    if case["op"] == "conv_step":
        full = torch.cat([state, s["x"][:, None]], 1)
        y = (full.float() * s["w"].t()).sum(1)
        if s["bias"] is not None:
            y = y + s["bias"]
        if case["silu"]:
            y = y * _sigmoid(y)
        new = full[:, 1:]
    else:
        per = case["channels"] // case["groups"]
        step = _softplus(s["dt"].float() + s["dt_bias"])
        Bc, Cc = (s[k].float().repeat_interleave(per, 1) for k in ("B", "C"))
        new = state * torch.exp(step[..., None] * s["A"]) + (step * x)[..., None] * Bc
        y = (new * Cc).sum(-1)
        if s["D"] is not None:
            y = y + s["D"] * x
        if s["z"] is not None:
            z = s["z"].float()
            y = y * z * _sigmoid(z)
    return {"y": (y * live).to(dt), "state": _scatter_rows(s, new)}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op.startswith("rotary"):
        return _exact_rotary(case, s)
    if op.endswith("step"):
        return _exact_step(case, s)
    if op.startswith("conv"):
        return _exact_conv(case, s)
    return _exact_scan(case, s)


def _exact_rotary(case, s):
    # a pair as a complex number, times e^{i angle}
    r, p, mag = case["rotary_dim"], ROTARY, 1.0
    freq = []
    for i in range(r // 2):
        f = p["base"] ** (-2.0 * i / r)
        if case["scaling"] == "linear":
            f /= p["factor"]
        elif case["scaling"] == "base" and r > 2:
            f = (p["base"] * p["factor"] ** (r / (r - 2.0))) ** (-2.0 * i / r)
        elif case["scaling"] == "ramp":
            turns = p["original"] * f / (2.0 * math.pi)
            share = min(1.0, max(0.0, (turns - p["slow"]) / (p["fast"] - p["slow"])))
            f = share * f + (1.0 - share) * f / p["factor"]
        freq.append(f)
    if case["scaling"] == "ramp":
        mag = 0.1 * math.log(p["factor"]) + 1.0
    freq = torch.tensor(freq, dtype=torch.float64, device="cuda")
    B, T = case["batch"], case["length"]
    at = torch.arange(T, dtype=torch.float64, device="cuda").expand(B, T)
    if s["positions"] is not None:
        at = s["positions"].double()
    if s["offsets"] is not None:
        at = at + s["offsets"].double()[:, None]
    angle = at[:, :, None, None] * freq
    if case["op"] == "rotary_bwd":
        angle = -angle
    turn = torch.polar(torch.full_like(angle, mag), angle)
    out = {}
    for name in ("q", "k"):
        y = s[name].double()
        head = y[..., :r]
        pairs = (head.unflatten(-1, (2, r // 2)).transpose(-1, -2) if case["layout"] == "half"
                 else head.unflatten(-1, (r // 2, 2)))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = (z.transpose(-1, -2) if case["layout"] == "half" else z).flatten(-2)
        out[name] = torch.cat([z, y[..., r:]], -1)
    return out


def _exact_step(case, s):
    new = s["state"].double()
    x = s["x"].double()
    y = torch.zeros_like(x)
    for b, at in enumerate(s["slots"].tolist()):
        if at < 0:
            continue
        if case["op"] == "conv_step":
            window = torch.cat([s["state"][at].double(), x[b:b + 1]])
            v = torch.einsum("wd,dw->d", window, s["w"].double())
            if s["bias"] is not None:
                v = v + s["bias"].double()
            y[b] = torch.nn.functional.silu(v) if case["silu"] else v
            new[at] = window[1:]
            continue
        h, y[b] = _exact_token(case, s, s["state"][at].double(), x[b], s["dt"][b].double(),
                               s["B"][b].double(), s["C"][b].double(),
                               None if s["z"] is None else s["z"][b].double())
        new[at] = h
    return {"y": y, "state": new}


def _exact_token(case, s, h, x, dt, B, C, z, A=None, D=None, bias=None):
    """One token of the scan's definition; h (..., channels, states)."""
    A = s["A"].double() if A is None else A
    bias = s["dt_bias"].double() if bias is None else bias
    if D is None and s["D"] is not None:
        D = s["D"].double()
    per = case["channels"] // case["groups"]
    v = dt + bias
    delta = torch.logaddexp(v, torch.zeros_like(v))
    B, C = B.repeat_interleave(per, -2), C.repeat_interleave(per, -2)
    h = torch.exp(delta[..., None] * A) * h + (delta * x)[..., None] * B
    y = torch.matmul(h[..., None, :], C[..., :, None])[..., 0, 0]
    if D is not None:
        y = y + D * x
    if z is not None:
        y = y * torch.nn.functional.silu(z)
    return h, y


def _exact_conv(case, s):
    # the library's convolution in 64 bits, sequence by sequence where they are
    # uneven; the gradients by differentiating it
    W, B, T, D = case["width"], case["batch"], case["length"], case["channels"]
    back = case["op"] == "conv_bwd"
    x, w = s["x"].double(), s["w"].double()
    bias = None if s["bias"] is None else s["bias"].double()
    first = (torch.zeros((B, W - 1, D), dtype=torch.float64, device="cuda")
             if s["s0"] is None else s["s0"].double())
    wrt = [x, w, first] + ([] if bias is None else [bias])
    if back:
        for t in wrt:
            t.requires_grad_()

    def apply(x, first):
        seq = torch.cat([first, x], 1)
        pre = torch.nn.functional.conv1d(seq.transpose(1, 2), w[:, None], bias, groups=D)
        y = (torch.nn.functional.silu(pre) if case["silu"] else pre).transpose(1, 2)
        return y, seq[:, seq.shape[1] - (W - 1):]

    n = _lengths(case)
    if len(set(n)) == 1:
        y, last = apply(x, first)
    else:
        order = {}
        for b, length in enumerate(n):
            order.setdefault(length, []).append(b)
        if len(order) > 600:
            return None
        ys, lasts = [None] * B, [None] * B
        for length, members in order.items():
            yy, ll = ((None, first[members]) if length == 0
                      else apply(x[members, :length], first[members]))
            for i, b in enumerate(members):
                ys[b] = torch.zeros((T, D), dtype=torch.float64, device="cuda")
                if length:
                    ys[b] = torch.cat([yy[i], ys[b][length:]])
                lasts[b] = ll[i]
        y, last = torch.stack(ys), torch.stack(lasts)
    if not back:
        return {"y": y, "state": last}
    loss = (y * s["dy"].double()).sum()
    if s["dsT"] is not None:
        loss = loss + (last * s["dsT"].double()).sum()
    d = torch.autograd.grad(loss, wrt, allow_unused=True)
    d = [torch.zeros_like(t) if v is None else v for t, v in zip(wrt, d)]
    out = {"dx": d[0], "dw": d[1]}
    if bias is not None:
        out["dbias"] = d[3]
    if s["s0"] is not None:
        out["dstate"] = d[2]
    return out


def _exact_scan(case, s):
    # token by token; the gradients by differentiating that
    B, T = case["batch"], case["length"]
    back = case["op"] == "scan_bwd"
    # about 60 us a token forward, four times that with gradients
    if T > (16400 if back else 40000):
        return None
    x, dt, Bm, Cm = (s[k].double() for k in ("x", "dt", "B", "C"))
    z = None if s["z"] is None else s["z"].double()
    A, bias = s["A"].double(), s["dt_bias"].double()
    D = None if s["D"] is None else s["D"].double()
    h0 = (torch.zeros((B, case["channels"], case["states"]), dtype=torch.float64, device="cuda")
          if s["s0"] is None else s["s0"].double())
    n = torch.tensor(_lengths(case), device="cuda")
    even = len(set(_lengths(case))) == 1
    rows = {"dx": x, "ddt": dt, "dB": Bm, "dC": Cm, **({} if z is None else {"dz": z})}
    wrt = {"dA": A, "ddt_bias": bias, **({} if D is None else {"dD": D}),
           **({} if s["s0"] is None else {"dstate": h0})}
    # each token's rows as leaves of their own: their gradients are collected in place
    parts = {k: list(t.unbind(1)) for k, t in rows.items()}
    if back:
        parts = {k: [t.detach().clone().requires_grad_() for t in p] for k, p in parts.items()}
        for t in wrt.values():
            t.requires_grad_()
    h, ys = h0, []
    for t in range(T):
        new, y = _exact_token(case, s, h, parts["dx"][t], parts["ddt"][t], parts["dB"][t],
                              parts["dC"][t], None if z is None else parts["dz"][t], A, D, bias)
        if even:
            h = new
        else:
            on = (t < n)[:, None]
            h = torch.where(on[..., None], new, h)
            y = torch.where(on, y, torch.zeros_like(y))
        ys.append(y)
    y = torch.stack(ys, 1)
    if not back:
        return {"y": y, "state": h}
    loss = (y * s["dy"].double()).sum()
    if s["dsT"] is not None:
        loss = loss + (h * s["dsT"].double()).sum()
    leaves = list(wrt.values()) + [t for p in parts.values() for t in p]
    d = list(torch.autograd.grad(loss, leaves))
    out = dict(zip(wrt, d))
    d = d[len(wrt):]
    for k in parts:
        out[k], d = torch.stack(d[:T], 1), d[T:]
    return out
