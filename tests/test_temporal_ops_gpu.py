"""Causal convolution, selective scan and rotary positions on the GPU against their
definitions in 64 bits (``temporal_ref.py``), at the sizes, types and masks where they can
go wrong; a run of them together; and their refusals."""
import itertools

import pytest
import torch

import ops_ref as R
import temporal_ref as M

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def pkg(fno):
    return fno


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def rand(g, shape, dtype="f32", scale=1.0, mean=0.0):
    return (mean + scale * torch.randn(shape, generator=g)).to(R.TORCH[dtype])


def cuda(v):
    return None if v is None else v.cuda()


def d64(v):
    return None if v is None else v.double()


def leaf(v):
    return None if v is None else v.double().requires_grad_()


def lengths_of(g, B, T):
    """Uneven lengths: a full one, an empty one, one beyond what there is, a negative one."""
    n = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32)
    for b, v in zip(range(B), (T, 0, T + 7, -3)):
        n[b] = v
    return n


def spoil(t, n):
    """NaN in the tokens beyond the lengths."""
    if n is not None:
        t = t.clone()
        for b, k in enumerate(n.tolist()):
            t[b, max(0, min(k, t.shape[1])):] = float("nan")
    return t


def close(got, ref, bound, scale=None):
    """Relative 2-norm error, or against ``scale`` where the exact value may cancel."""
    if scale is None:
        assert R.rel(got, ref) < bound, R.rel(got, ref)
        return
    got = got.detach().double().cpu()
    assert torch.isfinite(got).all() and got.shape == ref.shape
    assert (got - ref).norm().item() <= bound * max(scale, ref.norm().item())


# ---------------------------------------------------------------------------
# causal convolution
# ---------------------------------------------------------------------------
CONVS = [  # batch, length, channels, width
    (1, 1, 1, 2), (2, 1, 33, 4), (4, 2, 64, 4), (5, 3, 8, 8), (2, 17, 1001, 3), (1, 300, 96, 8),
    (4, 37, 40, 5), (2, 129, 130, 2), (5, 64, 256, 4), (1, 3000, 16, 4), (3, 40, 7, 6),
    (2, 33, 24, 7), (300, 12, 32, 4), (2, 70, 6, 3),
]


def conv_inputs(shape, dtype, bias, ragged, state, seed=0):
    B, T, D, W = shape
    g = gen(seed + 13 * B + 7 * T + D + W)
    t = {"x": rand(g, (B, T, D), dtype), "w": rand(g, (D, W), scale=W ** -0.5),
         "bias": rand(g, (D,), scale=0.3) if bias else None,
         "dy": rand(g, (B, T, D), dtype),
         "state": rand(g, (B, W - 1, D), dtype) if state else None,
         "dstate": rand(g, (B, W - 1, D), dtype) if state else None,
         "lengths": lengths_of(g, B, T) if ragged else None}
    return t


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("i", range(len(CONVS)))
def test_conv(pkg, dtype, i):
    B, T, D, W = CONVS[i]
    k = i + {"f32": 0, "f16": 1, "bf16": 3}[dtype]
    silu, bias, ragged, state = k % 3 != 0, k % 4 != 1, k % 2 == 1 and B > 1, k % 5 < 3
    t = conv_inputs(CONVS[i], dtype, bias, ragged, state)
    n = t["lengths"]
    p = pkg.CausalConv(B, T, D, W, act="silu" if silu else "none", dtype=dtype, backward=True)
    c = {name: cuda(v) for name, v in t.items()}
    x = cuda(spoil(t["x"], n))
    y, sT = p.forward(x, c["w"], bias=c["bias"], lengths=c["lengths"], state=c["state"],
                      want_state=True)
    lx, lw, lb, ls = leaf(t["x"]), leaf(t["w"]), leaf(t["bias"]), leaf(t["state"])
    ry, rs = M.conv(lx, lw, lb, silu, n, ls)
    close(y, ry, R.tol(dtype))
    assert torch.equal(sT.cpu().double(), rs.detach())          # copies of inputs
    loss = (ry * d64(t["dy"])).sum()
    if state:
        loss = loss + (rs * d64(t["dstate"])).sum()
    names = [m for m, v in (("dx", lx), ("dw", lw), ("dbias", lb), ("ds", ls)) if v is not None]
    want = dict(zip(names, torch.autograd.grad(
        loss, [v for v in (lx, lw, lb, ls) if v is not None], allow_unused=True)))
    got = dict(zip(("dx", "dw", "dbias", "ds"),
                   p.backward(x, c["w"], cuda(spoil(t["dy"], n)), bias=c["bias"],
                              lengths=c["lengths"], state=c["state"], dstate=c["dstate"])))
    for name in ("dbias", "ds"):
        assert (got[name] is None) == (name not in want)
    for name, ref in want.items():
        got_ = got[name]
        ref = torch.zeros_like(got_.cpu().double()) if ref is None else ref
        # sums of a few terms of either sign may cancel: against the terms' size
        scale = d64(t["dy"]).norm().item() if name in ("dw", "dbias") else None
        close(got_, ref, R.tol(dtype if name in ("dx", "ds") else "f32"), scale)
    p.close()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("W,D", [(2, 5), (4, 64), (8, 33), (3, 18)])
def test_conv_steps_are_the_sequence(pkg, dtype, W, D):
    """Token by token through slots, in place, against the whole sequence; idle rows and
    slots of no row are left alone."""
    B, T, slots = 5, 11, 8
    t = conv_inputs((B, T, D, W), dtype, True, False, True)
    c = {k: cuda(v) for k, v in t.items()}
    whole = pkg.CausalConv(B, T, D, W, dtype=dtype)
    y, sT = whole.forward(c["x"], c["w"], bias=c["bias"], state=c["state"], want_state=True)
    step = pkg.CausalConv(B, 1, D, W, dtype=dtype)
    at = torch.tensor([6, 1, -1, 0, 8], dtype=torch.int32)      # rows 2 and 4 are idle
    live = [0, 1, 3]
    state = torch.full((slots, W - 1, D), 7.0, dtype=R.TORCH[dtype])
    for b in live:
        state[at[b]] = t["state"][b]
    state = state.cuda()
    for k in range(T):
        out = step.step(c["x"][:, k].contiguous(), c["w"], state, bias=c["bias"],
                        slots=at.cuda())
        assert torch.equal(out[live], y[live, k])
        assert not out[[2, 4]].any()
    for b in live:
        assert torch.equal(state[at[b]], sT[b])
    rest = [s for s in range(slots) if s not in (6, 1, 0)]
    assert (state[rest] == 7.0).all()


# ---------------------------------------------------------------------------
# selective scan
# ---------------------------------------------------------------------------
SCANS = [  # batch, length, channels, states, groups
    (1, 1, 1, 1, 1), (2, 1, 33, 16, 1), (4, 7, 64, 16, 1), (5, 8, 32, 4, 1), (4, 9, 40, 8, 2),
    (1, 300, 96, 16, 1), (2, 200, 130, 24, 1), (1, 65, 34, 3, 2), (4, 40, 48, 64, 3),
    (1, 130, 20, 64, 1), (3, 50, 12, 50, 4), (2, 100, 300, 16, 1), (1, 2000, 8, 16, 1),
    (64, 12, 32, 16, 1), (3, 150, 5, 2, 1), (2, 77, 257, 7, 1), (2, 33, 64, 12, 1),
    # many short sequences: a block holds several, and goes on with further ones
    (700, 3, 10, 16, 1), (9, 40, 24, 4, 2), (2600, 2, 33, 5, 1),
]
# A decay is good to 2^-22 of itself, and the steps and rates below make the memory at most
# 40 tokens (step 0.05 or more, rate 0.5 or more): the states are off by 40 2^-22 < 1e-5,
# which adds to the sums' 1e-5.
SCAN_EXTRA = 1e-5


def scan_inputs(shape, dtype, skip, gate, bias, plus, ragged, state, seed=0):
    B, T, D, N, G = shape
    g = gen(seed + 13 * B + 7 * T + D + 3 * N + G)
    t = {"x": rand(g, (B, T, D), dtype),
         "A": -(0.5 + 3.0 * torch.rand((D, N), generator=g)),
         "B": rand(g, (B, T, G, N), dtype), "C": rand(g, (B, T, G, N), dtype),
         "D": rand(g, (D,)) if skip else None, "z": rand(g, (B, T, D), dtype) if gate else None}
    # steps of 0.05 to 0.4: log(e^s - 1) before softplus
    s = 0.05 + 0.35 * torch.rand((B, T, D), generator=g)
    v = torch.log(torch.expm1(s)) if plus else s
    t["bias"] = rand(g, (D,), scale=0.01) if bias else None
    t["dt"] = (v if plus else v + 0.05).to(R.TORCH[dtype])
    t["dy"] = rand(g, (B, T, D), dtype)
    t["state"] = rand(g, (B, D, N)) if state else None
    t["dstate"] = rand(g, (B, D, N)) if state else None
    t["lengths"] = lengths_of(g, B, T) if ragged else None
    return t


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("i", range(len(SCANS)))
def test_scan(pkg, dtype, i):
    B, T, D, N, G = SCANS[i]
    k = i + {"f32": 0, "f16": 1, "bf16": 3}[dtype]
    skip, gate, bias, plus = k % 3 != 0, k % 2 == 0, k % 4 != 1, k % 5 != 2
    ragged, state = k % 3 == 1 and B > 1, k % 4 < 2
    t = scan_inputs(SCANS[i], dtype, skip, gate, bias, plus, ragged, state)
    n = t["lengths"]
    p = pkg.SelectiveScan(B, T, D, N, groups=G, softplus=plus, dtype=dtype, backward=True)
    c = {name: cuda(v) for name, v in t.items()}
    for name in ("x", "dt", "B", "C", "z", "dy"):
        c[name] = None if t[name] is None else cuda(spoil(t[name], n))
    more = dict(D=c["D"], z=c["z"], dt_bias=c["bias"], lengths=c["lengths"], state=c["state"])
    y, sT = p.forward(c["x"], c["dt"], c["A"], c["B"], c["C"], want_state=True, **more)
    f32 = R.tol("f32") + SCAN_EXTRA
    stored = R.tol(dtype) + SCAN_EXTRA
    leaves = {m: leaf(t[m]) for m in ("x", "dt", "A", "B", "C", "D", "z", "bias", "state")}
    two = leaf(t["dt"])
    ry, rs = M.scan(leaves["x"], leaves["dt"], leaves["A"], leaves["B"], leaves["C"],
                    leaves["D"], leaves["z"], leaves["bias"], plus, n, leaves["state"],
                    dt_input=two)
    close(y, ry, stored)
    close(sT, rs, f32)
    loss = (ry * d64(t["dy"])).sum()
    if state:
        loss = loss + (rs * d64(t["dstate"])).sum()
    wrt = {m: v for m, v in leaves.items() if v is not None}
    grads = torch.autograd.grad(loss, list(wrt.values()) + [two], allow_unused=True)
    want = {m: torch.zeros_like(v) if d is None else d
            for (m, v), d in zip(wrt.items(), grads)}
    first = want["dt"]
    second = torch.zeros_like(first) if grads[-1] is None else grads[-1]
    want["dt"] = first + second
    parts = (first.norm() + second.norm()).item()          # dt's gradient is a difference
    got = p.backward(c["x"], c["dt"], c["A"], c["B"], c["C"], c["dy"], dstate=c["dstate"], **more)
    names = {"bias": "ddt_bias", "state": "dstate"}
    assert set(got) == {names.get(m, "d" + m) for m in wrt}
    for m, ref in want.items():
        g = got[names.get(m, "d" + m)]
        kind = m in ("x", "dt", "B", "C", "z")
        # sums of few terms of either sign: against the terms
        scale = {"dt": parts, "bias": parts, "D": (d64(t["dy"]).norm() * 0.5).item(),
                 "A": parts, "B": want["B"].norm().item() + 1e-3, "C": None}.get(m)
        close(g, ref, stored if kind else f32, scale)
    p.close()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,N,G", [(5, 1, 1), (64, 16, 1), (36, 10, 3), (8, 64, 2), (33, 64, 1)])
def test_scan_steps_are_the_sequence(pkg, dtype, D, N, G):
    B, T, slots = 5, 9, 8
    t = scan_inputs((B, T, D, N, G), dtype, True, True, True, True, False, True)
    c = {k: cuda(v) for k, v in t.items()}
    args = dict(D=c["D"], dt_bias=c["bias"])
    ry, rs = M.scan(*(d64(t[k]) for k in ("x", "dt", "A", "B", "C", "D", "z", "bias")),
                    True, None, d64(t["state"]))
    step = pkg.SelectiveScan(B, 1, D, N, groups=G, dtype=dtype)
    at = torch.tensor([6, 1, -1, 0, 8], dtype=torch.int32)
    live = [0, 1, 3]
    state = torch.full((slots, D, N), 7.0)
    for b in live:
        state[at[b]] = t["state"][b]
    state = state.cuda()
    got = []
    for k in range(T):
        row = {m: c[m][:, k].contiguous() for m in ("x", "dt", "B", "C", "z")}
        if k % 2:                                          # in place, or to another buffer
            out = step.step(row["x"], row["dt"], c["A"], row["B"], row["C"], state, z=row["z"],
                            slots=at.cuda(), **args)
        else:
            new = state.clone()
            out = step.step(row["x"], row["dt"], c["A"], row["B"], row["C"], state, z=row["z"],
                            slots=at.cuda(), new_state=new, **args)
            state = new
        assert not out[[2, 4]].any()
        got.append(out)
    close(torch.stack(got, 1)[live], ry[live], R.tol(dtype) + SCAN_EXTRA)
    close(state[at[live].long()], rs[live], R.tol("f32") + SCAN_EXTRA)
    rest = [s for s in range(slots) if s not in (6, 1, 0)]
    assert (state[rest] == 7.0).all()


def test_scan_carries_over(pkg):
    """Two halves with the state between them are the whole, also where one is split in time."""
    B, T, D, N = 1, 1500, 40, 16
    t = scan_inputs((B, T, D, N, 1), "f32", True, True, True, True, False, True)
    ry, rs = M.scan(*(d64(t[k]) for k in ("x", "dt", "A", "B", "C", "D", "z", "bias")),
                    True, None, d64(t["state"]))
    c = {k: cuda(v) for k, v in t.items()}
    cut = 1403
    state, out = c["state"], []
    for a, b in ((0, cut), (cut, T)):
        p = pkg.SelectiveScan(B, b - a, D, N)
        row = {m: c[m][:, a:b].contiguous() for m in ("x", "dt", "B", "C", "z")}
        y, state = p.forward(row["x"], row["dt"], c["A"], row["B"], row["C"], D=c["D"],
                             z=row["z"], dt_bias=c["bias"], state=state, want_state=True)
        out.append(y)
    close(torch.cat(out, 1), ry, R.tol("f32") + SCAN_EXTRA)
    close(state, rs, R.tol("f32") + SCAN_EXTRA)


def test_scan_steps_at_the_ends_of_softplus(pkg):
    """Steps from 1e-9 to 90, from softplus of -20 to 90; NaN stays where it is."""
    v = torch.tensor([-100.0, -20.0, -15.0, -1.0, -1e-3, 0.0, 1e-3, 1.0, 15.0, 20.0, 90.0])
    D = len(v)
    p = pkg.SelectiveScan(1, 1, D, 1)
    one = torch.ones(1, 1, 1, 1).cuda()
    y, _ = p.forward(torch.ones(1, 1, D).cuda(), v.view(1, 1, D).cuda(),
                     -torch.ones(D, 1).cuda(), one, one)
    want = M.softplus(v.double())                          # y = d x B C
    # (softplus(-100) = e^-100 = 3.7e-44 lies below 2^-126 = 1.2e-38, the least normal
    # float32: 24 significant bits end there, and such a step is 0)
    assert ((y.cpu().double().view(-1) - want).abs() <= 1e-6 * want + 2.0 ** -126).all()


def test_scan_nan_stays_in_its_channel(pkg):
    B, T, D, N = 2, 100, 33, 16
    t = scan_inputs((B, T, D, N, 1), "f32", True, False, True, True, False, False)
    c = {k: cuda(v) for k, v in t.items()}
    p = pkg.SelectiveScan(B, T, D, N, backward=True)
    args = (c["dt"], c["A"], c["B"], c["C"])
    clean, _ = p.forward(c["x"], *args, D=c["D"], dt_bias=c["bias"])
    x = c["x"].clone()
    x[1, 40, 7] = float("nan")
    y, _ = p.forward(x, *args, D=c["D"], dt_bias=c["bias"])
    hit = torch.zeros(B, T, D, dtype=torch.bool, device="cuda")
    hit[1, 40:, 7] = True
    assert torch.isnan(y[hit]).all() and torch.equal(y[~hit], clean[~hit])


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
ROTARIES = [  # batch, length, heads, kv heads, dim, rotary dim
    (1, 1, 1, 1, 2, 2), (3, 5, 4, 2, 64, 64), (2, 33, 6, 3, 80, 40), (2, 7, 3, 0, 48, 32),
    (1, 9, 5, 5, 7, 6), (2, 300, 8, 1, 128, 128), (1, 4, 2, 1, 300, 256), (64, 1, 16, 4, 64, 64),
    (2, 17, 2, 2, 20, 10),
]
SCALINGS = [None, ("linear", 4.0), ("base", 8.0), ("ramp", 8.0, 256, 8.0, 1.0)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("i", range(len(ROTARIES)))
def test_rotary(pkg, dtype, layout, i):
    B, T, H, K, dim, r = ROTARIES[i]
    k = i + (layout == "half") + 2 * (dtype == "f16")
    scaling, where = SCALINGS[k % 4], ("none", "offsets", "positions")[k % 3]
    if scaling and scaling[0] == "base" and r == 2:
        scaling = None
    g = gen(5 * i + B)
    q = rand(g, (B, T, H, dim), dtype)
    kk = rand(g, (B, T, K, dim), dtype) if K else None
    pos, kw = torch.arange(T).expand(B, T), {}
    if where == "offsets":
        off = torch.randint(-1 << 31, (1 << 31) - 1, (B,), generator=g).to(torch.int32)
        pos, kw = pos + off.long()[:, None], {"offsets": off.cuda()}
    elif where == "positions":
        at = torch.randint(0, 1 << 20, (B, T), generator=g).to(torch.int32)
        pos, kw = at.long(), {"positions": at.cuda()}
    p = pkg.Rotary(B, T, H, K, dim, rotary_dim=r, layout=layout, scaling=scaling, dtype=dtype)
    for call, sign in ((p.forward, 1), (p.backward, -1)):
        # in place, and into new tensors
        a, b = q.cuda(), cuda(kk)
        oq, ok = call(a, b, **kw)
        iq, ik = call(a, b, q_out=a, k_out=b, **kw)
        assert iq.data_ptr() == a.data_ptr() and torch.equal(iq, oq)
        # angles to 2^-32 of a turn and 2^31 positions' 53 bits: below 1e-6
        close(oq, M.rotate(d64(q), sign * pos, r, layout, scaling=scaling), R.tol(dtype))
        if K:
            assert torch.equal(ik, ok)
            close(ok, M.rotate(d64(kk), sign * pos, r, layout, scaling=scaling), R.tol(dtype))
        assert torch.equal(oq[..., r:].cpu(), q[..., r:])
    p.close()


# ---------------------------------------------------------------------------
# together, and as they are called
# ---------------------------------------------------------------------------
def test_a_mixer_of_them(pkg):
    """Norm, convolution and scan beside rotary linear attention on one stream, whole and
    token by token, against the definitions."""
    B, T, C, N, W, H, K, d = 3, 70, 64, 16, 4, 4, 2, 16
    g = gen(11)
    x = rand(g, (B, T, C))
    w1 = rand(g, (C,), mean=1.0, scale=0.1)
    cw, cb = rand(g, (C, W), scale=0.5), rand(g, (C,), scale=0.1)
    A = -(0.5 + 3.0 * torch.rand((C, N), generator=g))
    wdt, wb, wc = (rand(g, (C, m), scale=0.3 * C ** -0.5) for m in (C, N, N))
    wq, wk, wv = (rand(g, (C, h * d), scale=C ** -0.5) for h in (H, K, K))
    skip, decay = rand(g, (C,)), torch.tensor([-0.5, -0.1, -0.05, -0.02])

    # 64 bits
    u = R.norm(d64(x), "rms", 1e-5, d64(w1), None, 2)
    v, _ = M.conv(u, d64(cw), d64(cb), True)
    Bm, Cm = ((v @ d64(m)).unsqueeze(2) for m in (wb, wc))
    y, sT = M.scan(v, v @ d64(wdt), d64(A), Bm, Cm, d64(skip), u)
    q, k, val = ((u @ d64(m)).unflatten(-1, (-1, d)) for m in (wq, wk, wv))
    pos = torch.arange(T).expand(B, T)
    o, S = R.attention(M.rotate(q, pos, d, "half"), M.rotate(k, pos, d, "half"), val, decay,
                       d ** -0.5)

    X, P = x.cuda(), {m: t.cuda() for m, t in dict(
        w1=w1, cw=cw, cb=cb, A=A, wdt=wdt, wb=wb, wc=wc, wq=wq, wk=wk, wv=wv, D=skip,
        decay=decay).items()}

    def mix(n, rows, conv, scan, rot, attn, offsets=None):
        """The same calls on `n` tokens a sequence; the last four are how each is called."""
        u = pkg.SandwichNorm(C, n, B, layout="tokens").pre(rows, P)
        v = conv(u)
        Bm, Cm = ((v @ P[m]).view(B, n, 1, N) for m in ("wb", "wc"))
        y = scan(v, v @ P["wdt"], Bm, Cm, u)
        q, k, val = ((u @ P[m]).view(B, n, -1, d) for m in ("wq", "wk", "wv"))
        q, k = rot(q, k)
        return y, attn(q, k, val)

    cv, sc = pkg.CausalConv(B, T, C, W), pkg.SelectiveScan(B, T, C, N)
    at, ro = pkg.LinearAttention(B, T, H, K, d, d), pkg.Rotary(B, T, H, K, d)
    kept = {}

    def scan_all(v, dt, b, c, z):
        out, kept["h"] = sc.forward(v, dt, P["A"], b, c, D=P["D"], z=z, want_state=True)
        return out

    def attn_all(q, k, val):
        out, kept["S"] = at.forward(q, k, val, P["decay"], want_state=True)
        return out

    gy, go = mix(T, X, lambda u: cv.forward(u, P["cw"], bias=P["cb"])[0], scan_all, ro.forward,
                 attn_all)
    for got, ref in ((gy, y), (go, o), (kept["h"], sT), (kept["S"], S)):
        # float32 through norm, convolution, products of 64 terms (library) and the operator:
        # each within 1e-5, and the scan's decays
        close(got, ref, 5e-5)

    cs, ss = pkg.CausalConv(B, 1, C, W), pkg.SelectiveScan(B, 1, C, N)
    as_, rs = pkg.LinearAttention(B, 1, H, K, d, d), pkg.Rotary(B, 1, H, K, d)
    inputs = torch.zeros(B, W - 1, C).cuda()
    h, Sx = torch.zeros(B, C, N).cuda(), torch.zeros(B, H, d, d).cuda()
    ys, os_ = [], []
    for t in range(T):
        off = torch.full((B,), t, dtype=torch.int32).cuda()
        a, b = mix(1, X[:, t:t + 1].contiguous(),
                   lambda u: cs.step(u[:, 0], P["cw"], inputs, bias=P["cb"]).view(B, 1, C),
                   lambda v, dt, bm, cm, z: ss.step(v[:, 0], dt[:, 0], P["A"], bm[:, 0],
                                                    cm[:, 0], h, D=P["D"],
                                                    z=z[:, 0]).view(B, 1, C),
                   lambda q, k: rs.forward(q, k, offsets=off),
                   lambda q, k, val: as_.step(q[:, 0], k[:, 0], val[:, 0], P["decay"],
                                              Sx).view(B, 1, H, d))
        ys.append(a)
        os_.append(b)
    for got, ref in ((torch.cat(ys, 1), y), (torch.cat(os_, 1), o), (h, sT), (Sx, S)):
        close(got, ref, 5e-5)


def test_captured_and_on_another_stream(pkg):
    """The same bits eagerly, on a side stream and from a replayed graph whose inputs
    changed after the capture."""
    B, T, D, N, W = 2, 700, 72, 16, 4
    t = scan_inputs((B, T, D, N, 1), "bf16", True, True, True, True, False, True)
    v = conv_inputs((B, T, D, W), "bf16", True, False, True)
    other = scan_inputs((B, T, D, N, 1), "bf16", True, True, True, True, False, True, seed=1)
    c, cv, oc = ({k: cuda(x) for k, x in m.items()} for m in (t, v, other))
    scan = pkg.SelectiveScan(B, T, D, N, dtype="bf16", backward=True)
    conv = pkg.CausalConv(B, T, D, W, dtype="bf16", backward=True)
    rot = pkg.Rotary(B, T, 6, 3, 8, dtype="bf16")

    def run(stream=None):
        kw = {"stream": stream}
        x, s1 = conv.forward(c["x"], cv["w"], bias=cv["bias"], state=cv["state"],
                             want_state=True, **kw)
        more = dict(D=c["D"], z=c["z"], dt_bias=c["bias"], state=c["state"], **kw)
        y, s2 = scan.forward(x, c["dt"], c["A"], c["B"], c["C"], want_state=True, **more)
        d = scan.backward(x, c["dt"], c["A"], c["B"], c["C"], c["dy"], dstate=c["dstate"], **more)
        e = conv.backward(c["x"], cv["w"], d["dx"], bias=cv["bias"], state=cv["state"],
                          dstate=cv["dstate"], **kw)
        q, k = rot.forward(y.view(B, T, 9, 8)[:, :, :6].contiguous(),
                           y.view(B, T, 9, 8)[:, :, 6:].contiguous(), **kw)
        return [x, s1, y, s2, *d.values(), *e, q, k]

    def same(a, b):
        assert all(torch.equal(u, w) for u, w in zip(a, b))

    first = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = run()
    side.synchronize()
    same(first, second)
    same(first, run())                                       # the same bits every time
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    names = ("x", "dt", "A", "B", "C", "D", "z", "bias", "dy", "state", "dstate")
    for name in names:
        c[name].copy_(oc[name])
    graph.replay()
    torch.cuda.synchronize()
    replayed = [u.clone() for u in out]
    same(replayed, run())
    assert not torch.equal(replayed[2], first[2])


def test_outputs_stay_in_bounds(pkg):
    """What lies around the outputs is left alone, at sizes that end inside tiles."""
    B, T, D, N, W = 3, 13, 21, 5, 3
    t = scan_inputs((B, T, D, N, 1), "bf16", True, True, True, True, True, False)
    c = {k: cuda(x) for k, x in t.items()}
    n = B * T * D
    buf = torch.full((n + 1024,), 3.0, dtype=torch.bfloat16, device="cuda")
    out = buf[512:512 + n].view(B, T, D)
    pkg.SelectiveScan(B, T, D, N, dtype="bf16").forward(
        c["x"], c["dt"], c["A"], c["B"], c["C"], D=c["D"], z=c["z"], dt_bias=c["bias"],
        lengths=c["lengths"], out=out)
    assert (buf[:512] == 3.0).all() and (buf[512 + n:] == 3.0).all()
    buf.fill_(3.0)
    pkg.CausalConv(B, T, D, W, dtype="bf16").forward(
        c["x"], torch.ones(D, W).cuda(), lengths=c["lengths"], out=out)
    assert (buf[:512] == 3.0).all() and (buf[512 + n:] == 3.0).all()
    buf.fill_(3.0)
    q = c["x"].view(B, T, 3, 7)
    pkg.Rotary(B, T, 3, 0, 7, rotary_dim=4, dtype="bf16").forward(q, q_out=out.view(B, T, 3, 7))
    assert (buf[:512] == 3.0).all() and (buf[512 + n:] == 3.0).all()


def test_more_than_32_bits_of_elements(pkg):
    """Rows whose offsets pass 2^31 elements (and 2^32 bytes) are those of a small call."""
    T, D = 1 << 17, 1 << 10
    B = 17                                                  # 2^31 + 2^27 elements
    x = torch.zeros(B, T, D, dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.randn(T, D, device="cuda").bfloat16()
    w = torch.randn(D, 4, device="cuda")
    y, _ = pkg.CausalConv(B, T, D, 4, dtype="bf16").forward(x, w)
    z, _ = pkg.CausalConv(1, T, D, 4, dtype="bf16").forward(x[-1:], w)
    assert torch.equal(y[-1], z[0]) and not y[:-1].any()
    heads = x.view(B, T, 8, 128)
    q, _ = pkg.Rotary(B, T, 8, 0, 128, dtype="bf16").forward(heads, q_out=y.view(heads.shape))
    r, _ = pkg.Rotary(1, T, 8, 0, 128, dtype="bf16").forward(heads[-1:])
    assert torch.equal(q[-1], r[0]) and not q[:-1].any()


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
def test_refusals(pkg):
    z = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")   # noqa: E731
    conv = pkg.CausalConv(2, 5, 6, 3)
    x, w = z(2, 5, 6), z(6, 3)
    for bad in (z(2, 5, 7), z(2, 5, 12)[..., ::2], z(2, 5, 6).half(), x.cpu(), None):
        with pytest.raises((TypeError, ValueError)):
            conv.forward(bad, w)
    with pytest.raises(ValueError):
        conv.forward(x, z(6, 4))
    with pytest.raises(TypeError):
        conv.forward(x, w, lengths=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        conv.forward(x, w, state=z(2, 3, 6))
    with pytest.raises(pkg.FnoError):
        conv.forward(x, w, out=x)                            # an output over an input
    with pytest.raises(pkg.FnoError):
        conv.backward(x, w, x)                               # made without backward=True
    row = z(2, 6)
    with pytest.raises(ValueError):
        conv.step(row, w, z(1, 2, 6))                        # fewer slots than rows
    with pytest.raises(ValueError):
        conv.step(row, w, z(0, 2, 6), slots=z(2, dtype=torch.int32))
    for kw in (dict(width=1), dict(channels=0), dict(batch=0), dict(length=0)):
        with pytest.raises(pkg.FnoError):
            pkg.CausalConv(**{**dict(batch=1, length=1, channels=4, width=3), **kw})
    for kw in (dict(act="relu"), dict(dtype="f64"), dict(channels=2 ** 32 + 4)):
        with pytest.raises(ValueError):
            pkg.CausalConv(**{**dict(batch=1, length=1, channels=4, width=3), **kw})

    scan = pkg.SelectiveScan(2, 5, 6, 4, groups=2)
    A, b = z(6, 4), z(2, 5, 2, 4)
    ok = dict(x=x, dt=x, A=A, B=b, C=b)
    for name, bad in (("x", z(2, 5, 5)), ("dt", x.half()), ("A", A.half()), ("B", z(2, 5, 1, 4)),
                      ("C", b.transpose(2, 3)), ("x", z(2, 5, 12)[..., ::2])):
        with pytest.raises((TypeError, ValueError)):
            scan.forward(**{**ok, name: bad})
    with pytest.raises(ValueError):
        scan.forward(**ok, state=z(2, 6, 5))
    with pytest.raises(pkg.FnoError):
        scan.forward(**ok, out=x)
    with pytest.raises(pkg.FnoError):
        scan.backward(**ok, dy=x)
    for kw in (dict(groups=4), dict(states=0), dict(states=65), dict(groups=0)):
        with pytest.raises(pkg.FnoError):
            pkg.SelectiveScan(**{**dict(batch=1, length=1, channels=6, states=4), **kw})

    rot = pkg.Rotary(2, 5, 4, 2, 8)
    q, k = z(2, 5, 4, 8), z(2, 5, 2, 8)
    for args, kw in (((q,), {}), ((q, q), {}), ((q, k[:1]), {}),
                     ((q, k), dict(positions=z(2, dtype=torch.int32))),
                     ((q, k), dict(offsets=z(2, dtype=torch.int64))),
                     ((q, k), dict(offsets=z(2, dtype=torch.int32),
                                   positions=z(2, 5, dtype=torch.int32)))):
        with pytest.raises((TypeError, ValueError)):
            rot.forward(*args, **kw)
    flat = z(2 * 2 * 5 * 4 * 8)
    with pytest.raises(pkg.FnoError):                        # over a part of the input
        rot.forward(flat[:320].view(2, 5, 4, 8), k, q_out=flat[160:480].view(2, 5, 4, 8))
    with pytest.raises(ValueError):
        pkg.Rotary(2, 5, 4, 0, 8).forward(q, k)
    for kw in (dict(rotary_dim=3), dict(rotary_dim=10), dict(base=1.0), dict(dim=0),
               dict(scaling=("linear", 0.5)), dict(scaling=("ramp", 2.0, 100, 1.0, 1.0)),
               dict(rotary_dim=2, scaling=("base", 2.0))):
        with pytest.raises(pkg.FnoError):
            pkg.Rotary(**{**dict(batch=1, length=1, heads=1, kv_heads=1, dim=8), **kw})
    for kw in (dict(scaling=("linear",)), dict(scaling=("other", 1.0)), dict(layout="pairs")):
        with pytest.raises(ValueError):
            pkg.Rotary(**{**dict(batch=1, length=1, heads=1, kv_heads=1, dim=8), **kw})
