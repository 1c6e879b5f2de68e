"""Cases, plain forms and exact values of the sequence operators: the sandwich
norm (norms before and after a block with its gate and residual scale), the
8-bit activation checkpoints and what the backward pass reads of them, and
linear attention with a decay for each head.

Layouts.  "grid" fields are (batch, channels, points), the spectral layers'
channels-first tensors with the space flattened; "tokens" are (batch, points,
channels).  Heads are (batch, length, heads, head width).
"""
import math
import random

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5
GROUP = 128          # elements that share one 8-bit scale, along the last axis


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one frame's latent tokens between two blocks of an autoregressive
        # rollout: a handful of rows, where the call itself is the cost
        {"name": "norm_step", "op": "norm_fwd", "layout": "tokens", "batch": 4, "points": 1,
         "channels": 512, "norm": "rms", "gate": "none", "sigmoid": False, "save8": False,
         "dtype": "bf16"},
        # the FNO stack's 128 x 128 field (16 x 64 channels) after a spectral
        # layer, conditioned by a gate per sample and channel; the layer's
        # output is kept in 8 bits for the backward
        {"name": "norm_grid", "op": "norm_fwd", "layout": "grid", "batch": 16, "points": 16384,
         "channels": 64, "norm": "rms", "gate": "channel", "sigmoid": False, "save8": True,
         "dtype": "f32"},
        # the 256 x 256 workload's field (32 x 64 channels) in the backward,
        # from the 8-bit checkpoint
        {"name": "norm_grid_grad", "op": "norm_bwd", "layout": "grid", "batch": 32,
         "points": 65536, "channels": 64, "norm": "layer", "gate": "channel", "sigmoid": False,
         "save8": True, "dtype": "bf16"},
        # patch tokens with a learned sigmoid gate per element, odd token count
        {"name": "norm_tokens_grad", "op": "norm_bwd", "layout": "tokens", "batch": 3,
         "points": 4099, "channels": 1024, "norm": "layer", "gate": "full", "sigmoid": True,
         "save8": False, "dtype": "f16"},
        # a 1-D layer's activations (4 x 16 channels, 257 points: odd, the
        # last group of a row is one element)
        {"name": "pack_small", "op": "pack", "rows": 64, "cols": 257, "dtype": "f32"},
        # the pre-activations of the 256 x 256 workload kept in 8 bits, and the
        # GELU's backward from them
        {"name": "gelu_grad", "op": "gelu_bwd", "rows": 2048, "cols": 65536, "dtype": "f16"},
        # the 1x1 linear of the FNO stack: weight and bias gradients from the
        # 8-bit input of the layer
        {"name": "linear_grad", "op": "linear_bwd", "batch": 16, "cin": 64, "cout": 64,
         "points": 16384, "dtype": "f32"},
        # the same over 64^3 volumes with uneven channel counts (40 -> 60)
        {"name": "linear_grad_3d", "op": "linear_bwd", "batch": 8, "cin": 40, "cout": 60,
         "points": 262144, "dtype": "bf16"},
        # one rollout step of 64 running simulations out of 96 slots
        {"name": "attn_step", "op": "attn_step", "batch": 64, "slots": 96, "heads": 16,
         "kv_heads": 16, "dk": 64, "dv": 64, "dtype": "bf16"},
        # a prompt of past frames' tokens, ragged lengths (one of them empty)
        {"name": "attn_prompt", "op": "attn_fwd", "batch": 4, "length": 4096, "heads": 16,
         "kv_heads": 16, "dk": 64, "dv": 64, "ragged": True, "state": True, "dtype": "bf16"},
        # one long history in float32, few heads, odd length
        {"name": "attn_long_f32", "op": "attn_fwd", "batch": 1, "length": 16383, "heads": 8,
         "kv_heads": 4, "dk": 64, "dv": 64, "ragged": False, "state": False, "dtype": "f32"},
        # training: gradients with key/value heads shared by groups of query heads
        {"name": "attn_grad", "op": "attn_bwd", "batch": 2, "length": 8192, "heads": 16,
         "kv_heads": 8, "dk": 128, "dv": 128, "ragged": False, "state": False, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "pack", "gelu_bwd", "linear_bwd", "attn_step",
                     "attn_fwd", "attn_bwd"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op in ("norm_fwd", "norm_bwd"):
        layout = rng.choice(["grid", "tokens"])
        channels = _log_int(rng, 16, 512 if layout == "grid" else 4096)
        most = 32 * 64 * 65536 // (2 if dtype == "f32" else 1)
        batch = _log_int(rng, 1, 32)
        points = _log_int(rng, 1, max(1, min(65536, most // (batch * channels))))
        return {"op": op, "layout": layout, "batch": batch, "points": points,
                "channels": channels, "norm": rng.choice(["rms", "layer"]),
                "gate": rng.choice(["none", "channel", "full"]),
                "sigmoid": rng.random() < 0.5, "save8": rng.random() < 0.5, "dtype": dtype}
    if op in ("pack", "gelu_bwd"):
        rows = _log_int(rng, 1, 2048)
        return {"op": op, "rows": rows, "dtype": dtype,
                "cols": _log_int(rng, 16, 65536 // (2 if dtype == "f32" else 1))}
    if op == "linear_bwd":
        cin, cout = _log_int(rng, 3, 128), _log_int(rng, 3, 128)
        batch = _log_int(rng, 1, 16)
        return {"op": op, "batch": batch, "cin": cin, "cout": cout, "dtype": dtype,
                "points": _log_int(rng, 64, min(262144, 8 * 262144 * 100 // (cin + cout)
                                                // batch // (2 if dtype == "f32" else 1)))}
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 1, 2, 4])
    dk, dv = rng.choice([(32, 32), (64, 64), (128, 128), (64, 128), (48, 80)])
    if op == "attn_step":
        batch = _log_int(rng, 1, 128)
        return {"op": op, "batch": batch, "slots": batch + rng.randrange(0, 33), "heads": heads,
                "kv_heads": kv, "dk": dk, "dv": dv, "dtype": dtype}
    batch = _log_int(rng, 1, 8)
    most = 2 * 8192 * 16 * 128 * 128 // (batch * heads * dk * dv * (2 if dtype == "f32" else 1))
    return {"op": op, "batch": batch, "length": _log_int(rng, 1, max(1, min(16384, most))),
            "heads": heads, "kv_heads": kv, "dk": dk, "dv": dv, "ragged": rng.random() < 0.5,
            "state": rng.random() < 0.5, "dtype": dtype}


def _lengths(case):
    """Valid tokens of each sequence: the first is full, the second empty, the
    others in between (a property of the case, not of the seed)."""
    if not case["ragged"] or case["batch"] == 1:
        return [case["length"]] * case["batch"]
    r = random.Random(case["batch"] * 1000003 + case["length"])
    return [case["length"], 0] + [r.randint(1, case["length"])
                                  for _ in range(case["batch"] - 2)]


def _groups(n):
    return -(-n // GROUP)


def work(case):
    e = 4 if case.get("dtype") == "f32" else 2
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        B, C, P = case["batch"], case["channels"], case["points"]
        n = B * C * P
        rows, cols = (B * C, P) if case["layout"] == "grid" else (B * P, C)
        packed = n + 4 * rows * _groups(cols)        # 8-bit codes and their scales
        gate = {"none": 0, "channel": 4 * B * C, "full": e * n}[case["gate"]]
        if op == "norm_fwd":        # x, f, gate -> y, u (and the checkpoint of f, and its values)
            return {"bytes": 4 * e * n + gate + (2 * packed + e * n if case["save8"] else 0)
                    + 12 * C,
                    "flops": 12 * n}
        # y, f, gate, dy, du -> dx, df, dgate, parameter gradients
        return {"bytes": 5 * e * n + (packed if case["save8"] else e * n) + 2 * gate + 32 * C,
                "flops": 30 * n}
    if op in ("pack", "gelu_bwd"):
        n = case["rows"] * case["cols"]
        packed = n + 4 * case["rows"] * _groups(case["cols"])
        if op == "pack":            # x -> codes, scales, and the values read back
            return {"bytes": 2 * e * n + 2 * packed, "flops": 5 * n}
        return {"bytes": 2 * e * n + packed, "flops": 20 * n}
    if op == "linear_bwd":
        B, P, ci, co = case["batch"], case["points"], case["cin"], case["cout"]
        return {"bytes": B * P * (e * co + ci) + 4 * B * ci * _groups(P) + 4 * co * (ci + 1),
                "flops": 2 * B * P * co * (ci + 1)}
    H, K, dk, dv, B = case["heads"], case["kv_heads"], case["dk"], case["dv"], case["batch"]
    state = 4 * B * H * dk * dv
    if op == "attn_step":
        return {"bytes": 2 * state + e * B * (H * (dk + dv) + K * (dk + dv)),
                "flops": 5 * B * H * dk * dv}
    valid, every = sum(_lengths(case)), B * case["length"]
    read = valid * (H * dk + K * (dk + dv))
    if op == "attn_fwd":
        return {"bytes": e * (read + every * H * dv) + (2 if case["state"] else 1) * state,
                "flops": 4 * valid * H * dk * dv}
    return {"bytes": e * (read + valid * H * dv + every * (H * dk + K * (dk + dv)))
            + (3 if case["state"] else 0) * state,
            "flops": 10 * valid * H * dk * dv}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _field(g, shape, axis, dtype, spread=0.5):
    """Activations: normal, with a spread of sizes over the channels."""
    size = [1] * len(shape)
    size[axis] = shape[axis]
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    x *= torch.exp(spread * torch.randn(size, generator=g, device="cuda"))
    return x.to(dtype)


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        s["plan"] = _plan(case)
    return s


def _plan(case):
    """The plan (a description of the shapes) that a program makes once."""
    import fft_gemm_ifft_gb300 as fno
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        return fno.SandwichNorm(case["channels"], case["points"], case["batch"],
                                layout=case["layout"], norm=case["norm"], gate=case["gate"],
                                gate_sigmoid=case["sigmoid"], eps=EPS, dtype=case["dtype"])
    if op == "linear_bwd":
        return fno.LinearGrad(case["batch"], case["cin"], case["cout"], case["points"],
                              dtype=case["dtype"])
    if op in ("attn_step", "attn_fwd", "attn_bwd"):
        return fno.LinearAttention(case["batch"], case.get("length", 1), case["heads"],
                                   case["kv_heads"], case["dk"], case["dv"],
                                   dtype=case["dtype"], backward=op == "attn_bwd")
    return None


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DT[case["dtype"]]
    op = case["op"]
    s = {"case": case}

    def vec(n, mean, sd):
        return mean + sd * torch.randn(n, generator=g, device="cuda")

    if op in ("norm_fwd", "norm_bwd"):
        B, C, P = case["batch"], case["channels"], case["points"]
        shape, ax = ((B, C, P), 1) if case["layout"] == "grid" else ((B, P, C), 2)
        s["params"] = {"s": vec(C, 0.2, 0.1), "w2": vec(C, 1.0, 0.2), "w1": vec(C, 1.0, 0.2)}
        if case["norm"] == "layer":
            s["params"].update(b2=vec(C, 0.0, 0.2), b1=vec(C, 0.0, 0.2))
        s["gate"] = None
        if case["gate"] == "channel":
            s["gate"] = vec((B, C), 1.0 if not case["sigmoid"] else 0.0, 0.5)
        elif case["gate"] == "full":
            s["gate"] = _field(g, shape, ax, dt)
        s["x"] = _field(g, shape, ax, dt)        # the residual stream (y in the backward)
        s["f"] = _field(g, shape, ax, dt, 1.0)   # the block's output
        if op == "norm_bwd":
            s["dy"] = _field(g, shape, ax, dt)
            s["du"] = _field(g, shape, ax, dt)
            if case["save8"]:
                s["f8"] = _pack(s["f"])
                del s["f"]
        return s
    if op in ("pack", "gelu_bwd"):
        shape = (case["rows"], case["cols"])
        s["x"] = _field(g, shape, 0, dt)
        if op == "gelu_bwd":
            s["dy"] = _field(g, shape, 0, dt)
            s["x8"] = _pack(s["x"])
            del s["x"]
        return s
    if op == "linear_bwd":
        B, P, ci, co = case["batch"], case["points"], case["cin"], case["cout"]
        s["x8"] = _pack(_field(g, (B, ci, P), 1, dt))
        s["dy"] = _field(g, (B, co, P), 1, dt)
        return s

    B, H, K, dk, dv = (case[k] for k in ("batch", "heads", "kv_heads", "dk", "dv"))
    T = 1 if op == "attn_step" else case["length"]

    def heads(n, d, scale=1.0):
        t = torch.randn((B, T, n, d), generator=g, device="cuda") * scale
        return (t[:, 0] if op == "attn_step" else t).contiguous().to(dt)

    s["q"], s["k"], s["v"] = heads(H, dk), heads(K, dk), heads(K, dv)
    # memory of about 2 tokens in the first head to about 1000 in the last
    span = 2.0 ** (1.0 + 9.0 * torch.arange(H, device="cuda") / max(1, H - 1))
    s["log_decay"] = torch.log1p(-1.0 / span).float()
    s["scale"] = dk ** -0.5
    if op == "attn_step":
        n = case["slots"]
        s["state"] = torch.randn((n, H, dk, dv), generator=g, device="cuda")
        s["new"] = s["state"].clone()
        # each running simulation's slot; about one row in sixteen is idle (-1)
        slot = torch.randperm(n, generator=g, device="cuda")[:B].to(torch.int32)
        idle = torch.rand(B, generator=g, device="cuda") < 1.0 / 16
        s["slots"] = torch.where(idle, torch.full_like(slot, -1), slot)
    else:
        s["lengths"] = (torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
                        if case["ragged"] else None)
        s["s0"] = (torch.randn((B, H, dk, dv), generator=g, device="cuda")
                   if case["state"] else None)
        if op == "attn_bwd":
            s["do"] = heads(H, dv)
            s["dsT"] = (torch.randn((B, H, dk, dv), generator=g, device="cuda")
                        if case["state"] else None)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from fft_gemm_ifft_gb300 import PackedActivation, pack_activation
    op, dt = s["case"]["op"], DT[s["case"]["dtype"]]
    if op == "norm_fwd":
        y, u, f8 = s["plan"].forward(s["x"], s["f"], s["params"], gate=s["gate"],
                                     save8=s["case"]["save8"])
        return {"y": y, "u": u} if f8 is None else {"y": y, "u": u, "f8": f8.values()}
    if op == "norm_bwd":
        f = PackedActivation(*s["f8"], dt) if "f8" in s else s["f"]
        return s["plan"].backward(s["x"], f, s["params"], s["dy"], s["du"], gate=s["gate"])
    if op == "pack":
        return pack_activation(s["x"]).values()
    if op == "gelu_bwd":
        return PackedActivation(*s["x8"], dt).gelu_backward(s["dy"])
    if op == "linear_bwd":
        dw, db = s["plan"](s["dy"], PackedActivation(*s["x8"], dt))
        return {"dw": dw, "db": db}
    if op == "attn_step":
        o = s["plan"].step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], slots=s["slots"],
                           new_state=s["new"], scale=s["scale"])
        return {"o": o, "state": s["new"]}
    if op == "attn_fwd":
        o, sT = s["plan"].forward(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"],
                                  lengths=s["lengths"], state=s["s0"], want_state=True)
        return {"o": o, "state": sT}
    d = s["plan"].backward(s["q"], s["k"], s["v"], s["log_decay"], s["do"], scale=s["scale"],
                           lengths=s["lengths"], state=s["s0"], dstate=s["dsT"])
    return {"dq": d[0], "dk": d[1], "dv": d[2], **({} if d[3] is None else {"dstate": d[3]})}


# --- the plain form: elementary operations in 32 bits ------------------------
def _pack(x):
    """codes (int8) and scales: per GROUP consecutive elements of the last axis
    scale = max|x| / 127 and code = round(x (127 / max|x|)), half to even; a
    group below 1e-30 gets scale 0."""
    n = x.shape[-1]
    pad = _groups(n) * GROUP - n
    v = torch.nn.functional.pad(x.float(), (0, pad)).unflatten(-1, (-1, GROUP))
    amax = v.abs().amax(-1)
    keep = ~(amax < 1e-30)
    top = torch.full_like(amax, 127.0)     # divided as tensors: not by way of a reciprocal
    inv = torch.where(keep, top / amax, torch.zeros_like(amax))
    q = torch.round(v * inv[..., None]).to(torch.int8).flatten(-2)[..., :n].contiguous()
    return q, torch.where(keep, amax / top, torch.zeros_like(amax))


def _unpack(q, sc):
    n = q.shape[-1]
    v = torch.nn.functional.pad(q.float(), (0, _groups(n) * GROUP - n))
    return (v.unflatten(-1, (-1, GROUP)) * sc[..., None]).flatten(-2)[..., :n]


def _norm(v, kind, ax):
    if kind == "layer":
        v = v - v.mean(ax, keepdim=True)
    r = torch.rsqrt((v * v).mean(ax, keepdim=True) + EPS)
    return v * r, r


def _norm_grad(dn, n, r, kind, ax):
    """Gradient of a norm's input, given that of its normalised value n."""
    d = dn - n * (dn * n).mean(ax, keepdim=True)
    if kind == "layer":
        d = d - dn.mean(ax, keepdim=True)
    return d * r


def _run_plain(s):
    case = s["case"]
    op, dt = case["op"], DT[case["dtype"]]
    if op in ("norm_fwd", "norm_bwd"):
        grid, kind, p = case["layout"] == "grid", case["norm"], s["params"]
        ax = 1 if grid else 2
        view = (1, -1, 1) if grid else (1, 1, -1)
        g = s["gate"]
        if g is not None:
            g = g.float()
            if case["gate"] == "channel":
                g = g[:, :, None] if grid else g[:, None, :]
        a = 1.0 if g is None else (torch.sigmoid(g) if case["sigmoid"] else g)
        sc, w2, w1 = (p[k].view(view) for k in ("s", "w2", "w1"))
        b2, b1 = ((p["b2"].view(view), p["b1"].view(view)) if kind == "layer" else (0.0, 0.0))
        if op == "norm_fwd":
            y = s["x"].float() + sc * a * (_norm(s["f"].float(), kind, ax)[0] * w2 + b2)
            u = _norm(y, kind, ax)[0] * w1 + b1
            out = {"y": y.to(dt), "u": u.to(dt)}
            if case["save8"]:
                out["f8"] = _unpack(*_pack(s["f"])).to(dt)
            return out
        over = (0, 2) if grid else (0, 1)
        n1, r1 = _norm(s["x"].float(), kind, ax)
        n2, r2 = _norm(_unpack(*s["f8"]) if "f8" in s else s["f"].float(), kind, ax)
        du = s["du"].float()
        dY = s["dy"].float() + _norm_grad(du * w1, n1, r1, kind, ax)
        dz = dY * sc * a
        out = {"dx": dY.to(dt), "df": _norm_grad(dz * w2, n2, r2, kind, ax).to(dt)}
        z = n2 * w2 + b2
        out["ds"] = (dY * a * z).sum(over)
        out["dw2"] = (dz * n2).sum(over)
        out["dw1"] = (du * n1).sum(over)
        if kind == "layer":
            out["db2"], out["db1"] = dz.sum(over), du.sum(over)
        if g is not None:
            dg = dY * sc * z
            if case["sigmoid"]:
                dg = dg * a * (1.0 - a)
            out["dgate"] = dg.to(dt) if case["gate"] == "full" else dg.sum(2 if grid else 1)
        return out
    if op == "pack":
        return _unpack(*_pack(s["x"])).to(dt)
    if op == "gelu_bwd":
        v = _unpack(*s["x8"])
        slope = (0.5 * (1.0 + torch.erf(v * math.sqrt(0.5)))
                 + v * torch.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi))
        return (s["dy"].float() * slope).to(dt)
    if op == "linear_bwd":
        dy = s["dy"].float()
        return {"dw": torch.matmul(dy, _unpack(*s["x8"]).transpose(1, 2)).sum(0),
                "db": dy.sum((0, 2))}
    if op == "attn_step":
        G = case["heads"] // case["kv_heads"]
        q = s["q"].float()
        k, v = (s[n].float().repeat_interleave(G, 1) for n in ("k", "v"))
        live, n = s["slots"] >= 0, case["slots"]
        at = s["slots"].clamp(min=0).long()
        S = (s["state"][at] * torch.exp(s["log_decay"])[None, :, None, None]
             + k[..., None] * v[..., None, :])
        o = s["scale"] * (q[..., None] * S).sum(2) * live[:, None, None]
        row = torch.full((n + 1,), -1, device="cuda").scatter(
            0, torch.where(live, at, torch.full_like(at, n)),
            torch.arange(case["batch"], device="cuda"))[:n]
        mine = (row >= 0)[:, None, None, None]
        return {"o": o.to(dt), "state": torch.where(mine, S[row.clamp(min=0)], s["state"])}

    G = case["heads"] // case["kv_heads"]
    B, T, H = s["q"].shape[:3]
    if s["lengths"] is None:
        m = torch.ones((B, T), device="cuda")
    else:
        m = (torch.arange(T, device="cuda")[None] < s["lengths"][:, None]).float()
    q = s["q"].float() * m[..., None, None]
    k, v = (s[n].float().repeat_interleave(G, 2) * m[..., None, None] for n in ("k", "v"))
    decay = m[..., None] * s["log_decay"]                     # (B, T, H)
    s0 = s["s0"]
    if op == "attn_fwd":
        o, S = _scan(q, k, v, decay, s0)
        return {"o": (s["scale"] * o).to(dt), "state": S}
    do = s["scale"] * s["do"].float() * m[..., None, None]
    dq, _ = _scan(do, v, k, decay, None if s0 is None else s0.transpose(2, 3))
    # the reversed scan: a token's own step comes before its decay
    later = torch.nn.functional.pad(decay[:, 1:], (0, 0, 0, 1)).flip(1)
    q, k, v, do = (t.flip(1) for t in (q, k, v, do))
    dsT = s["dsT"]
    dk, _ = _scan(v, do, q, later, None if dsT is None else dsT.transpose(2, 3))
    dv, S = _scan(k, q, do, later, dsT)
    dk, dv = (t.flip(1).unflatten(2, (-1, G)).sum(3).to(dt) for t in (dk, dv))
    out = {"dq": dq.to(dt), "dk": dk, "dv": dv}
    if s0 is not None:
        out["dstate"] = S * torch.exp(decay[:, 0])[..., None, None]
    return out


def _scan(q, k, v, decay, s0, n=128):
    """o_t = q_t S_t, S_t = e^{decay_t} S_{t-1} + k_t v_t^T, in chunks of n tokens."""
    B, T, H, dk = q.shape
    pad = -T % n
    q, k, v = (torch.nn.functional.pad(t, (0, 0, 0, 0, 0, pad))
               .unflatten(1, (-1, n)).permute(0, 3, 1, 2, 4) for t in (q, k, v))
    c = torch.nn.functional.pad(decay, (0, 0, 0, pad)).unflatten(1, (-1, n))
    c = c.permute(0, 3, 1, 2).cumsum(-1)                       # (B, H, chunks, n)
    low = torch.ones((n, n), device=q.device).tril().bool()
    gap = (c[..., :, None] - c[..., None, :]).masked_fill(~low, -math.inf)
    o = torch.matmul(torch.matmul(q, k.transpose(-1, -2)) * torch.exp(gap), v)
    add = torch.matmul((k * torch.exp(c[..., -1:] - c)[..., None]).transpose(-1, -2), v)
    # the state after each chunk: the earlier chunks' sums, decayed over the chunks between
    if s0 is None:
        s0 = torch.zeros((B, H, dk, v.shape[-1]), device=q.device)
    e = c[..., -1].cumsum(-1)
    low = torch.ones((e.shape[-1],) * 2, device=q.device).tril().bool()
    gap = (e[..., :, None] - e[..., None, :]).masked_fill(~low, -math.inf)
    S = (torch.matmul(torch.exp(gap), add.flatten(-2)).unflatten(-1, (dk, -1))
         + torch.exp(e)[..., None, None] * s0[:, :, None])
    before = torch.cat([s0[:, :, None], S[:, :, :-1]], 2)
    o = o + torch.matmul(q * torch.exp(c)[..., None], before)
    return o.permute(0, 2, 3, 1, 4).flatten(1, 2)[:, :T].contiguous(), S[:, :, -1]


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        return _exact_norm(case, s)
    if op == "pack":
        return None                       # codes: rounding to the nearest is part of the definition
    if op == "gelu_bwd":
        v = _values64(s["x8"]).requires_grad_()
        phi = 0.5 * torch.special.erfc(-v / math.sqrt(2.0))
        (d,) = torch.autograd.grad(v * phi, v, s["dy"].double())
        return d
    if op == "linear_bwd":
        dw = torch.zeros((case["cout"], case["cin"]), dtype=torch.float64, device="cuda")
        q, sc = s["x8"]
        for b in range(case["batch"]):
            dw += s["dy"][b].double() @ _values64((q[b], sc[b])).T
        return {"dw": dw, "db": s["dy"].double().sum((0, 2))}
    return _exact_attn(case, s)


def _values64(x8):
    q, sc = x8
    at = torch.arange(q.shape[-1], device=q.device) // GROUP
    return q.double() * sc.double()[..., at]


def _exact_norm(case, s):
    # channels last throughout; the gradients by differentiating the definition
    def last(t):
        return t.transpose(1, 2) if case["layout"] == "grid" else t

    def norm(v, w, b):
        if case["norm"] == "layer":
            return (v - v.mean(-1, keepdim=True)) / (v.var(-1, correction=0, keepdim=True)
                                                     + EPS).sqrt() * w + b
        return v / (v.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w

    def block(x, f, g, p):
        z = norm(f, p["w2"], p.get("b2"))
        if g is not None:
            a = 1.0 / (1.0 + torch.exp(-g)) if case["sigmoid"] else g
            z = z * (a[:, None, :] if case["gate"] == "channel" else a)
        return x + p["s"] * z

    p = {k: v.double() for k, v in s["params"].items()}
    g = s["gate"]
    if g is not None:
        g = g.double() if case["gate"] == "channel" else last(g.double())
    if case["op"] == "norm_fwd":
        y = block(last(s["x"].double()), last(s["f"].double()), g, p)
        out = {"y": last(y), "u": last(norm(y, p["w1"], p.get("b1")))}
        if case["save8"]:
            out["f8"] = None
        return out
    y = last(s["x"].double()).requires_grad_()
    u = norm(y, p["w1"].requires_grad_(), p["b1"].requires_grad_() if "b1" in p else None)
    names = [n for n in ("w1", "b1") if n in p]
    d = torch.autograd.grad(u, [y] + [p[n] for n in names], last(s["du"].double()))
    out = {"d" + n: t for n, t in zip(names, d[1:])}
    dY = d[0] + last(s["dy"].double())
    del u, d, y
    f = (last(_values64(s["f8"])) if "f8" in s else last(s["f"].double())).requires_grad_()
    p = {k: v.detach().requires_grad_() for k, v in p.items()}
    if g is not None:
        g.requires_grad_()
    wrt = {"df": f, "ds": p["s"], "dw2": p["w2"]}
    if "b2" in p:
        wrt["db2"] = p["b2"]
    if g is not None:
        wrt["dgate"] = g
    d = torch.autograd.grad(block(0.0, f, g, p), list(wrt.values()), dY)
    out.update(zip(wrt, d))
    out["dx"] = last(dY)
    out["df"] = last(out["df"])
    if case["gate"] == "full":
        out["dgate"] = last(out["dgate"])
    return out


def _exact_attn(case, s):
    # token by token
    G = case["heads"] // case["kv_heads"]
    gamma = torch.exp(s["log_decay"].double())
    step = case["op"] == "attn_step"
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    k, v = k.repeat_interleave(G, k.dim() - 2), v.repeat_interleave(G, v.dim() - 2)
    if step:
        o, new = torch.zeros_like(v), s["new"].double()
        for b, at in enumerate(s["slots"].tolist()):
            if at >= 0:
                new[at] = gamma[:, None, None] * s["state"][at].double() + torch.einsum(
                    "hd,he->hde", k[b], v[b])
                o[b] = s["scale"] * torch.einsum("hd,hde->he", q[b], new[at])
        return {"o": o, "state": new}
    B, T, H, dk = q.shape
    if T > 20000:
        return None
    length = torch.tensor(_lengths(case), device="cuda")

    def walk(order, a, b, c, S, own_first):
        """out_t = a_t Z where Z gathers b_s c_s^T with a factor gamma per step between;
        own_first: the decay precedes the token (forward), else it follows (reverse)."""
        out = torch.zeros(a.shape[:3] + (c.shape[3],), dtype=torch.float64, device="cuda")
        for t in order:
            on = (t < length).double()[:, None, None, None]
            keep = on * gamma[None, :, None, None] + (1.0 - on)
            if own_first:
                S = S * keep
            S = S + on * b[:, t, :, :, None] * c[:, t, :, None, :]
            out[:, t] = on[..., 0] * torch.matmul(a[:, t, :, None, :], S)[:, :, 0]
            if not own_first:
                S = S * keep
        return out, S

    def start(m, d0, d1):
        return (torch.zeros((B, H, d0, d1), dtype=torch.float64, device="cuda") if m is None
                else m.double())

    dv_ = v.shape[3]
    if case["op"] == "attn_fwd":
        o, S = walk(range(T), q, k, v, start(s["s0"], dk, dv_), True)
        return {"o": s["scale"] * o, "state": S}
    do = s["scale"] * s["do"].double()
    back = range(T - 1, -1, -1)
    dq, _ = walk(range(T), do, v, k, start(s["s0"], dk, dv_).transpose(2, 3), True)
    end = start(s["dsT"], dk, dv_)
    gk, _ = walk(back, v, do, q, end.transpose(2, 3), False)
    gv, S = walk(back, k, q, do, end, False)
    gk, gv = (t.unflatten(2, (-1, G)).sum(3) for t in (gk, gv))
    return {"dq": dq, "dk": gk, "dv": gv, **({"dstate": S} if case["state"] else {})}
