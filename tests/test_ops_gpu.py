"""The sequence operators on the GPU against their definitions in 64 bits
(``ops_ref.py``), at the sizes, types, masks and layouts where they can go
wrong, and their refusals."""
import itertools

import pytest
import torch

import ops_ref as R
from fft_gemm_ifft_gb300 import capi

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


# ---------------------------------------------------------------------------
# sandwich norm
# ---------------------------------------------------------------------------
SHAPES = [  # batch, points, channels
    (1, 1, 1), (2, 1, 33), (1, 3, 512), (3, 257, 7), (2, 130, 64), (1, 513, 96), (2, 64, 1000),
    (1, 40, 2056), (2, 1024, 128), (5, 9, 4099),
    # the tiles of half and quarter warps, the tiles read again with an odd point
    # count, and rows past every kernel that holds them
    (2, 70, 200), (1, 77, 130), (1, 33, 700), (1, 3, 9000),
]


def norm_inputs(layout, B, P, C, dtype, kind, gate, seed=0):
    g = gen(seed + 17 * B + 31 * P + C)
    shape = (B, C, P) if layout == "grid" else (B, P, C)
    t = {n: rand(g, shape, dtype) for n in ("x", "f", "dy", "du")}
    p = {"s": rand(g, (C,), scale=0.3), "w2": rand(g, (C,), mean=1.0, scale=0.2),
         "w1": rand(g, (C,), mean=1.0, scale=0.2)}
    if kind == "layer":
        p["b2"], p["b1"] = rand(g, (C,), scale=0.2), rand(g, (C,), scale=0.2)
    if gate == "channel":
        t["gate"] = rand(g, (B, C))
    elif gate == "full":
        t["gate"] = rand(g, shape, dtype)
    else:
        t["gate"] = None
    return t, p


def cuda(v):
    if isinstance(v, dict):
        return {k: cuda(x) for k, x in v.items()}
    return None if v is None else v.cuda()


def d64(v):
    return None if v is None else v.double()


def check_norm(pkg, layout, B, P, C, dtype, kind, gate, sigmoid, packed, eps=1e-5):
    t, p = norm_inputs(layout, B, P, C, dtype, kind, gate)
    n = pkg.SandwichNorm(C, P, B, layout=layout, norm=kind, gate=gate, gate_sigmoid=sigmoid,
                         eps=eps, dtype=dtype)
    T, PR = cuda(t), cuda(p)
    y, u, f8 = n.forward(T["x"], T["f"], PR, gate=T["gate"], save8=packed)
    p64 = {k: v.double().requires_grad_() for k, v in p.items()}
    ry, ru = R.sandwich(d64(t["x"]), d64(t["f"]), p64, kind, eps, layout, d64(t["gate"]), sigmoid)
    assert R.rel(y, ry) < R.tol(dtype) and R.rel(u, ru) < R.tol(dtype)
    if packed:
        codes, scales = R.pack(t["f"])
        assert torch.equal(f8.codes.cpu(), codes) and torch.equal(f8.scales.cpu(), scales)
    # the gradients at a given stream y (any field) and the values f stands for
    yv = d64(t["x"]).requires_grad_()
    fv = (R.values(f8.codes, f8.scales) if packed else d64(t["f"])).requires_grad_()
    gv = None if t["gate"] is None else d64(t["gate"]).requires_grad_()
    _, ru = R.sandwich(yv, None, p64, kind, eps, layout)
    first = [yv, p64["w1"]] + ([p64["b1"]] if kind == "layer" else [])
    g1 = torch.autograd.grad(ru, first, d64(t["du"]))
    dY = g1[0] + d64(t["dy"])
    ry, _ = R.sandwich(torch.zeros_like(yv), fv, p64, kind, eps, layout, gv, sigmoid, False)
    names = ["df", "ds", "dw2"] + ["db2"] * (kind == "layer") + ["dgate"] * (gv is not None)
    wrt = [fv, p64["s"], p64["w2"]] + ([p64["b2"]] if kind == "layer" else []) + \
        ([gv] if gv is not None else [])
    want = dict(zip(names, torch.autograd.grad(ry, wrt, dY)))
    want["dx"], want["dw1"] = dY, g1[1]
    if kind == "layer":
        want["db1"] = g1[2]
    got = n.backward(T["x"], f8 if packed else T["f"], PR, T["dy"], T["du"], gate=T["gate"])
    assert set(got) == set(want)
    for k, w in want.items():
        stored = k in ("dx", "df") or (k == "dgate" and gate == "full")
        bound = R.tol(dtype if stored else "f32")
        # where the exact gradient cancels to (nearly) nothing its error is
        # measured against what was added up
        if C == 1 and k in ("df", "ds", "dw2", "dw1", "dgate"):
            scale = (d64(t["dy"]).norm() + d64(t["du"]).norm()).item() / eps ** 0.5
            assert (got[k].double().cpu() - w).norm().item() < bound * scale
            continue
        assert R.rel(got[k], w) < bound, (k, R.rel(got[k], w))
    n.close()


@pytest.mark.parametrize("layout", ["grid", "tokens"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_norm(pkg, layout, dtype, i):
    kinds, gates = ["rms", "layer"], ["none", "channel", "full"]
    k = i + (layout == "grid") + 2 * (dtype == "f16")
    check_norm(pkg, layout, *SHAPES[i], dtype, kinds[k % 2], gates[k % 3], k % 4 == 1, k % 5 < 2)


# rows of some lanes, of three to fourteen warps, by pairs and single elements, with
# row counts that leave a CTA's last rows out; tiles of every part of a warp, whose
# rows start on 8, 4 and fewer bytes
EDGES = [("tokens", 2, 67, c) for c in (3, 22, 40, 63, 300, 518, 1300, 2303, 3500)] + \
        [("tokens", 1, 5, 6150)] + \
        [("grid", 2, 100, 300), ("grid", 1, 101, 400), ("grid", 2, 66, 40), ("grid", 1, 67, 20),
         ("grid", 1, 131, 97), ("grid", 1, 134, 160), ("grid", 1, 65, 289)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("i", range(len(EDGES)))
def test_norm_edges(pkg, dtype, i):
    layout, B, P, C = EDGES[i]
    check_norm(pkg, layout, B, P, C, dtype, "layer", "full", True, dtype != "f16")
    check_norm(pkg, layout, B, P, C, dtype, "rms", "channel", False, dtype == "f16")


@pytest.mark.parametrize("layout,kind,gate,sigmoid,packed", [
    c for c in itertools.product(["grid", "tokens"], ["rms", "layer"], ["none", "channel", "full"],
                                 [False, True], [False, True]) if c[2] != "none" or not c[3]])
def test_norm_every_form(pkg, layout, kind, gate, sigmoid, packed):
    check_norm(pkg, layout, 3, 133, 72, "bf16", kind, gate, sigmoid, packed)
    check_norm(pkg, layout, 2, 256, 128, "f32", kind, gate, sigmoid, packed)


@pytest.mark.parametrize("layout", ["grid", "tokens"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_alone_and_parts(pkg, layout, kind):
    # the norm in front of the first block; the block without the next norm;
    # gradients with either of dy and du absent
    B, P, C = 2, 65, 40
    t, p = norm_inputs(layout, B, P, C, "f32", kind, "none")
    n = pkg.SandwichNorm(C, P, B, layout=layout, norm=kind)
    T, PR = cuda(t), cuda(p)
    p64 = {k: v.double().requires_grad_() for k, v in p.items()}
    x = d64(t["x"]).requires_grad_()
    _, ru = R.sandwich(x, None, p64, kind, 1e-5, layout)
    assert R.rel(n.pre(T["x"], PR), ru) < R.tol("f32")
    (dx, dw1) = torch.autograd.grad(ru, [x, p64["w1"]], d64(t["du"]))
    got = n.backward(T["x"], None, PR, None, T["du"])
    assert set(got) == {"dx", "dw1"} | ({"db1"} if kind == "layer" else set())
    assert R.rel(got["dx"], dx) < R.tol("f32") and R.rel(got["dw1"], dw1) < R.tol("f32")
    y, u, f8 = n.forward(T["x"], T["f"], PR, want_u=False)
    assert u is None and f8 is None
    f = d64(t["f"]).requires_grad_()
    ry, _ = R.sandwich(x, f, p64, kind, 1e-5, layout, want_u=False)
    assert R.rel(y, ry) < R.tol("f32")
    (df,) = torch.autograd.grad(ry, [f], d64(t["dy"]))
    got = n.backward(T["x"], T["f"], PR, T["dy"])
    assert torch.equal(got["dx"], T["dy"]) and "dw1" not in got
    assert R.rel(got["df"], df) < R.tol("f32")


@pytest.mark.parametrize("layout", ["grid", "tokens"])
def test_norm_gradient_against_differences(pkg, layout):
    # L = <cy, y> + <cu, u> along random directions; central differences of the
    # kernel's own float32 forward at step h are off by O(h^2) and by
    # 2^-24 |y| sqrt(n) / h: with h = 2e-2 both are under 1e-3 of |L'|
    B, P, C = 2, 33, 24
    t, p = norm_inputs(layout, B, P, C, "f32", "layer", "channel", seed=5)
    n = pkg.SandwichNorm(C, P, B, layout=layout, norm="layer", gate="channel", gate_sigmoid=True)
    T, PR = cuda(t), cuda(p)

    def loss(x, f, gate, params):
        y, u, _ = n.forward(x, f, params, gate=gate)
        return ((y.double() * T["dy"].double()).sum() + (u.double() * T["du"].double()).sum())

    y, _, _ = n.forward(T["x"], T["f"], PR, gate=T["gate"])
    g = n.backward(y, T["f"], PR, T["dy"], T["du"], gate=T["gate"])
    h = 2e-2
    for name, key in [("x", "dx"), ("f", "df"), ("gate", "dgate"), ("s", "ds"), ("w2", "dw2"),
                      ("b2", "db2"), ("w1", "dw1"), ("b1", "db1")]:
        d = rand(gen(77), g[key].shape).cuda()
        d = d * (1.0 / d.norm())
        # a direction with a sizeable slope: half random, half along the gradient
        d = d + g[key] / g[key].norm()

        def at(e):
            a = {"x": T["x"], "f": T["f"], "gate": T["gate"]}
            q = dict(PR)
            if name in a:
                a[name] = a[name] + e * d
            else:
                q[name] = q[name] + e * d
            return loss(a["x"], a["f"], a["gate"], q)

        slope = ((at(h) - at(-h)) / (2 * h)).item()
        want = (g[key].double() * d.double()).sum().item()
        assert abs(slope - want) < 3e-3 * abs(want) + 1e-3, (name, slope, want)


def test_norm_large_mean_and_zero_rows(pkg):
    # a mean 1000 times the spread must not cancel; a row of zeros has n = 0
    B, P, C = 1, 50, 320
    g = gen(3)
    x = torch.zeros(B, P, C)
    f = 1000.0 + rand(g, (B, P, C))
    f[0, 7] = 0.0
    p = {"s": torch.ones(C), "w2": torch.ones(C), "b2": torch.zeros(C), "w1": torch.ones(C),
         "b1": torch.zeros(C)}
    for layout in ("tokens", "grid"):
        def lay(t):
            return t.transpose(1, 2).contiguous() if layout == "grid" else t
        n = pkg.SandwichNorm(C, P, B, layout=layout, norm="layer")
        y, u, _ = n.forward(lay(x).cuda(), lay(f).cuda(), cuda(p))
        ry, ru = R.sandwich(lay(x).double(), lay(f).double(), {k: v.double() for k, v in p.items()},
                            "layer", 1e-5, layout)
        # float32 holds f only to 2^-24 * 1000 = 6e-5 of its spread
        assert R.rel(y, ry) < 1e-4 and R.rel(u, ru) < 1e-4


def test_norm_in_place_and_repeatable(pkg):
    t, p = norm_inputs("grid", 2, 300, 64, "bf16", "rms", "channel")
    n = pkg.SandwichNorm(64, 300, 2, gate="channel", dtype="bf16")
    T, PR = cuda(t), cuda(p)
    y, u, _ = n.forward(T["x"], T["f"], PR, gate=T["gate"])
    x = T["x"].clone()
    y2, u2, _ = n.forward(x, T["f"], PR, gate=T["gate"], y=x)
    assert torch.equal(y, x) and torch.equal(u, u2) and y2 is x
    a = n.backward(y, T["f"], PR, T["dy"], T["du"], gate=T["gate"])
    b = n.backward(y, T["f"], PR, T["dy"], T["du"], gate=T["gate"])
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_norm_infinite_and_nan_points_stay_apart(pkg):
    # one bad point spoils its own channels and no other point
    for layout in ("grid", "tokens"):
        t, p = norm_inputs(layout, 1, 200, 48, "f32", "rms", "none")
        n = pkg.SandwichNorm(48, 200, 1, layout=layout)
        T, PR = cuda(t), cuda(p)
        y, u, _ = n.forward(T["x"], T["f"], PR)
        at = (0, slice(None), 77) if layout == "grid" else (0, 77)
        f = T["f"].clone()
        f[at][5] = float("nan")
        y2, u2, _ = n.forward(T["x"], f, PR)
        assert torch.isnan(y2[at]).all() and torch.isnan(u2[at]).all()
        y2[at], u2[at] = y[at], u[at]
        assert torch.equal(y, y2) and torch.equal(u, u2)


def test_norm_refusals(pkg):
    n = pkg.SandwichNorm(16, 8, 2, norm="layer", gate="channel")
    t, p = norm_inputs("grid", 2, 8, 16, "f32", "layer", "channel")
    T, PR = cuda(t), cuda(p)
    with pytest.raises(ValueError):
        n.forward(T["x"], T["f"], {k: v for k, v in PR.items() if k != "b2"}, gate=T["gate"])
    with pytest.raises(TypeError):
        n.forward(T["x"], T["f"], PR)                               # no gate
    with pytest.raises(TypeError):
        n.forward(T["x"].half(), T["f"], PR, gate=T["gate"])
    with pytest.raises(ValueError):
        n.forward(T["x"][:1], T["f"], PR, gate=T["gate"])
    with pytest.raises(ValueError):
        n.forward(T["x"].transpose(0, 1).contiguous().transpose(0, 1), T["f"], PR,
                  gate=T["gate"])
    with pytest.raises(pkg.FnoError) as e:
        n.forward(T["x"], T["f"], PR, gate=T["gate"], y=T["f"])     # over an input
    assert e.value.status == capi.FNO_ERR_ALIASING
    with pytest.raises(pkg.FnoError):
        n.backward(T["x"], T["f"], PR, None, None, gate=T["gate"])  # no gradient at all
    h, x, f, s = n.handle, T["x"].data_ptr(), T["f"].data_ptr(), PR["s"].data_ptr()
    w = PR["w2"].data_ptr()
    y, g = T["dy"].data_ptr(), T["gate"].data_ptr()
    fwd = capi.fno_sandwich_forward
    assert fwd(h, x, f, g, s, w, None, w, s, y, None, None, None, None) == \
        capi.FNO_ERR_INVALID_ARG                                     # b2 missing
    assert fwd(h, x, f, g, s, w, s, None, None, None, None, None, None, None) == \
        capi.FNO_ERR_INVALID_ARG                                     # y missing
    assert fwd(h, x + 4, f, g, s, w, s, None, None, y, None, None, None, None) == \
        capi.FNO_ERR_MISALIGNED


# ---------------------------------------------------------------------------
# 8-bit checkpoints
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(1,), (3, 1), (2, 127), (5, 128), (2, 129), (7, 257), (64, 4),
                                   (3, 5, 1000), (2, 4096), (33, 8191), (1, 100003)])
def test_pack_and_unpack(pkg, dtype, shape):
    x = rand(gen(len(shape) + shape[-1]), shape, dtype)
    flat = x.view(-1)
    flat[::7] *= 30.0                          # outliers
    if x.shape[-1] > 200:
        x[..., 128:190] = 0.0                  # part of a group, and
        x[..., 128:256] *= 0.0                 # a group of zeros
    p = pkg.pack_activation(x.cuda())
    codes, scales = R.pack(x)
    assert torch.equal(p.codes.cpu(), codes) and torch.equal(p.scales.cpu(), scales)
    got = p.values()
    assert torch.equal(got.cpu(), (codes.float() * scales[..., torch.arange(shape[-1]) // 128])
                       .to(x.dtype))
    # within half a step of the group's scale, and the storage type's rounding
    step = R.values(torch.ones_like(codes), scales)
    bound = (0.5 + 1e-5) * step + R.HALF_ULP[dtype] * 127 * step
    assert ((got.cpu().double() - x.double()).abs() <= bound).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pack_special_groups(pkg, dtype):
    x = rand(gen(1), (3, 512), dtype)
    x[0, 5], x[1, 130], x[2, 511] = float("nan"), float("inf"), -float("inf")
    x[0, 128:256] = 1e-38                      # below the smallest scale: reads back as 0
    x[0, 256:384] = -0.0
    p = pkg.pack_activation(x.cuda())
    v = p.values().cpu()
    assert torch.isnan(v[0, :128]).all() and torch.isnan(v[1, 128:256]).all()
    assert torch.isnan(v[2, 384:]).all()
    assert (v[0, 128:384] == 0).all() and torch.isfinite(v[0, 384:]).all()
    assert torch.isfinite(v[1, :128]).all() and torch.isfinite(v[2, :384]).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1), (3, 127), (2, 130), (64, 3), (5, 1001), (16, 4096)])
def test_gelu_backward(pkg, dtype, shape):
    g = gen(9 + shape[1])
    x, dy = rand(g, shape, dtype, scale=2.0), rand(g, shape, dtype)
    p = pkg.pack_activation(x.cuda())
    want = dy.double() * R.gelu_slope(R.values(p.codes, p.scales))
    d = dy.cuda()
    got = p.gelu_backward(d)
    assert R.rel(got, want) < R.tol(dtype)
    assert p.gelu_backward(d, out=d) is d and torch.equal(d, got)


def test_gelu_backward_against_differences(pkg):
    # the slope of the exact GELU at the code values, by differences in 64 bits
    v = torch.linspace(-6, 6, 1281).view(1, -1)
    p = pkg.pack_activation(v.cuda())
    x = R.values(p.codes, p.scales)

    def gelu(t):
        return 0.5 * t * torch.special.erfc(-t / 2.0 ** 0.5)
    h = 1e-5
    want = (gelu(x + h) - gelu(x - h)) / (2 * h)
    got = p.gelu_backward(torch.ones_like(v).cuda()).cpu().double()
    assert (got - want).abs().max() < 1e-6


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,ci,co,P", [(1, 1, 1, 1), (2, 3, 5, 127), (1, 64, 64, 128),
                                       (3, 40, 60, 1000), (2, 128, 128, 640), (1, 130, 33, 257),
                                       (2, 16, 200, 4096), (1, 300, 129, 384), (1, 127, 128, 515)])
def test_linear_grad(pkg, dtype, B, ci, co, P):
    g = gen(ci + co + P)
    x, dy = rand(g, (B, ci, P), dtype), rand(g, (B, co, P), dtype)
    p = pkg.pack_activation(x.cuda())
    n = pkg.LinearGrad(B, ci, co, P, dtype=dtype)
    dw, db = n(dy.cuda(), p)
    v = R.values(p.codes, p.scales)
    # exact products summed in float32: the float32 bound for every type
    assert R.rel(dw, torch.einsum("bop,bip->oi", dy.double(), v)) < R.tol("f32")
    want = dy.double().sum((0, 2))
    assert ((db.cpu().double() - want).abs() <= 1e-5 * dy.double().abs().sum((0, 2))).all()
    a, b = n(dy.cuda(), p)
    assert torch.equal(a, dw) and torch.equal(b, db)
    assert n.device_error() == 0
    n.close()


def test_linear_grad_refusals(pkg):
    n = pkg.LinearGrad(2, 8, 4, 50)
    x8 = pkg.pack_activation(torch.randn(2, 8, 50, device="cuda"))
    dy = torch.randn(2, 4, 50, device="cuda")
    with pytest.raises(TypeError):
        n(dy.half(), x8)
    with pytest.raises(TypeError):
        n(dy, torch.randn(2, 8, 50, device="cuda"))
    with pytest.raises(ValueError):
        n(dy, pkg.pack_activation(torch.randn(2, 8, 49, device="cuda")))
    c, s = x8.codes.data_ptr(), x8.scales.data_ptr()
    d, ws = dy.data_ptr(), torch.empty(n.workspace_bytes, dtype=torch.uint8, device="cuda")
    assert capi.fno_linear_grad(n.handle, d, c, s, d, None, ws.data_ptr(), None) == \
        capi.FNO_ERR_ALIASING
    assert capi.fno_linear_grad(n.handle, d, c, s, None, None, ws.data_ptr(), None) == \
        capi.FNO_ERR_INVALID_ARG
    with pytest.raises(TypeError):
        pkg.PackedActivation(x8.codes, x8.scales, torch.float64)
    with pytest.raises(ValueError):
        pkg.PackedActivation(x8.codes, x8.scales[..., :0], torch.float32)
    with pytest.raises(TypeError):
        pkg.pack_activation(torch.zeros(3, 4))
    with pytest.raises(ValueError):
        pkg.pack_activation(torch.zeros(0, 4, device="cuda"))


def test_offsets_beyond_32_bits(pkg):
    # 2^31 + some elements: the last rows are where 32-bit offsets would wrap
    rows, cols = 65537, 32800
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn((2, cols), device="cuda").bfloat16()
    x[-2:] = tail
    p = pkg.pack_activation(x)
    q = pkg.pack_activation(tail)
    assert torch.equal(p.codes[-2:], q.codes) and torch.equal(p.scales[-2:], q.scales)
    assert not p.codes[:-2].any()
    p.values(out=x)
    assert torch.equal(x[-2:], q.values())
    dy = torch.ones_like(x)
    p.gelu_backward(dy, out=dy)
    assert torch.equal(dy[-2:], q.gelu_backward(torch.ones_like(tail)))
    del dy
    n = pkg.SandwichNorm(cols, rows, 1, layout="tokens", dtype="bf16")
    w = {k: torch.ones(cols, device="cuda") for k in ("s", "w2", "w1")}
    u = n.pre(x.view(1, rows, cols), w)
    small = pkg.SandwichNorm(cols, 2, 1, layout="tokens", dtype="bf16")
    assert torch.equal(u[:, -2:], small.pre(x[-2:].view(1, 2, cols).clone(), w))


# ---------------------------------------------------------------------------
# linear attention
# ---------------------------------------------------------------------------
def attn_inputs(B, T, H, K, dk, dv, dtype, state, seed=0):
    g = gen(seed + B + T + 3 * H + dk)
    t = {"q": rand(g, (B, T, H, dk), dtype), "k": rand(g, (B, T, K, dk), dtype, dk ** -0.5),
         "v": rand(g, (B, T, K, dv), dtype), "do": rand(g, (B, T, H, dv), dtype)}
    span = 2.0 ** (1.0 + 8.0 * torch.arange(H) / max(1, H - 1))
    t["log_decay"] = torch.log1p(-1.0 / span).float()
    t["s0"] = rand(g, (B, H, dk, dv)) if state else None
    t["dsT"] = rand(g, (B, H, dk, dv)) if state else None
    return t


# roundings of a 16-bit path: the output, the weights of a chunk's tokens and
# the state in front of it
def attn_tol(dtype, stored=True):
    return R.tol(dtype, 3) if stored else R.tol("f32")


def check_attn(pkg, B, T, H, K, dk, dv, dtype, lengths=None, state=True, grad=True, decay=None):
    t = attn_inputs(B, T, H, K, dk, dv, dtype, state)
    if decay is not None:
        t["log_decay"] = torch.tensor(decay, dtype=torch.float32).expand(H).contiguous()
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    a = pkg.LinearAttention(B, T, H, K, dk, dv, dtype=dtype, backward=grad)
    C = cuda(t)
    scale = 0.37
    if ln is not None:        # what lies beyond a sequence is not looked at
        for b, n in enumerate(lengths):
            for x in ("q", "k", "v", "do"):
                C[x][b, max(0, min(n, T)):] = float("nan")
    kw = dict(scale=scale, lengths=cuda(ln), state=C["s0"])
    o, sT = a.forward(C["q"], C["k"], C["v"], C["log_decay"], want_state=True, **kw)
    w = {x: d64(t[x]).requires_grad_() for x in ("q", "k", "v")}
    s0 = None if not state else t["s0"].double().requires_grad_()
    ro, rS = R.attention(w["q"], w["k"], w["v"], t["log_decay"], scale, ln, s0)
    assert R.rel(o, ro) < attn_tol(dtype), R.rel(o, ro)
    assert R.rel(sT, rS) < attn_tol(dtype, False), R.rel(sT, rS)
    if grad:
        loss = (ro * d64(t["do"])).sum() + ((rS * t["dsT"].double()).sum() if state else 0.0)
        wrt = list(w.values()) + ([s0] if state else [])
        want = torch.autograd.grad(loss, wrt)
        got = a.backward(C["q"], C["k"], C["v"], C["log_decay"], C["do"], dstate=C["dsT"], **kw)
        for i, name in enumerate("qkv"):
            assert R.rel(got[i], want[i]) < attn_tol(dtype), (name, R.rel(got[i], want[i]))
        assert (got[3] is None) == (not state)
        if state:      # (below float32's range it is 0)
            assert R.rel(got[3], want[3].float()) < attn_tol(dtype, False)
    assert a.device_error() == 0
    a.close()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,T,H,K,dk,dv", [
    (1, 1, 1, 1, 1, 1), (2, 1, 4, 2, 64, 64), (1, 2, 2, 1, 5, 3), (2, 63, 2, 2, 64, 64),
    (1, 64, 4, 1, 128, 128), (2, 65, 2, 1, 32, 32), (1, 127, 2, 2, 64, 128), (1, 128, 2, 2, 64, 64),
    (2, 129, 4, 2, 48, 80), (1, 300, 2, 2, 128, 64), (1, 257, 1, 1, 256, 200), (3, 700, 2, 2, 64, 64),
    (1, 530, 4, 2, 128, 128),
])
def test_attention(pkg, dtype, B, T, H, K, dk, dv):
    check_attn(pkg, B, T, H, K, dk, dv, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dk,dv,group", [(64, 64, 1), (128, 128, 2), (24, 40, 3)])
def test_attention_ragged(pkg, dtype, dk, dv, group):
    # empty, one token, the chunk's edges, all, and lengths outside the range
    lengths = [0, 1, 63, 64, 65, 127, 128, 129, 333, 334, 1000, -5]
    check_attn(pkg, len(lengths), 334, 2 * group, 2, dk, dv, dtype, lengths=lengths)
    check_attn(pkg, 3, 334, group, 1, dk, dv, dtype, lengths=[0, 0, 0], state=True)
    check_attn(pkg, 3, 200, group, 1, dk, dv, dtype, lengths=[200, 0, 7], state=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", [0.0, -1e-4, -5.0, -200.0, -float("inf")])
def test_attention_decays(pkg, dtype, decay):
    # no decay, hardly any, nothing left of the last token but one, none at all
    check_attn(pkg, 2, 333, 2, 2, 64, 64, dtype, decay=decay, grad=decay > -1e30)
    check_attn(pkg, 1, 200, 2, 1, 40, 24, dtype, decay=decay, grad=decay > -1e30)


def test_attention_decay_of_zero_gradient(pkg):
    # gamma = 0: o_t = scale (q_t . k_t) v_t; the state has no gradient
    t = attn_inputs(1, 150, 2, 2, 64, 64, "f32", True)
    C = cuda(t)
    ninf = torch.full((2,), -float("inf"), device="cuda")
    a = pkg.LinearAttention(1, 150, 2, 2, 64, 64, backward=True)
    zero = torch.zeros_like(C["dsT"])
    dq, dk, dv, ds = a.backward(C["q"], C["k"], C["v"], ninf, C["do"], scale=1.0, state=C["s0"],
                                dstate=zero)
    q, k, v, do = (d64(t[x]) for x in ("q", "k", "v", "do"))
    vd = (v * do).sum(-1, keepdim=True)
    assert R.rel(dq, vd * k) < 1e-5 and R.rel(dk, vd * q) < 1e-5
    assert R.rel(dv, (q * k).sum(-1, keepdim=True) * do) < 1e-5
    assert not ds.any()


@pytest.mark.parametrize("dtype,dk,dv", [("f32", 64, 64), ("bf16", 64, 64), ("bf16", 128, 128),
                                         ("f16", 64, 128)])
def test_attention_long(pkg, dtype, dk, dv):
    # long enough that the time axis is split, and the parts joined
    check_attn(pkg, 1, 5000, 2, 1, dk, dv, dtype)
    check_attn(pkg, 2, 3001, 2, 2, dk, dv, dtype, lengths=[3001, 1234])


def test_attention_in_two_parts(pkg):
    # a prompt in two calls, the state handed over, is the prompt in one
    t = cuda(attn_inputs(2, 500, 4, 2, 64, 64, "f32", True))
    a, b, c = (pkg.LinearAttention(2, n, 4, 2, 64, 64) for n in (500, 217, 283))
    o, s = a.forward(t["q"], t["k"], t["v"], t["log_decay"], state=t["s0"], want_state=True)

    def cut(lo, hi):
        return [t[n][:, lo:hi].contiguous() for n in ("q", "k", "v")] + [t["log_decay"]]
    o1, s1 = b.forward(*cut(0, 217), state=t["s0"], want_state=True)
    o2, s2 = c.forward(*cut(217, 500), state=s1, want_state=True)
    assert R.rel(torch.cat([o1, o2], 1), o.cpu()) < 2e-6 and R.rel(s2, s.cpu()) < 2e-6


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("H,K,dk,dv", [(4, 2, 64, 64), (2, 2, 128, 128), (3, 1, 5, 33),
                                       (1, 1, 256, 250), (8, 8, 48, 80)])
def test_attention_step(pkg, dtype, H, K, dk, dv):
    B, n = 5, 9
    g = gen(dk + dv)
    a = pkg.LinearAttention(B, 1, H, K, dk, dv, dtype=dtype)
    state = rand(g, (n, H, dk, dv))
    slots = torch.tensor([3, -1, 8, 0, 9], dtype=torch.int32)     # two rows are idle
    t = attn_inputs(B, 1, H, K, dk, dv, dtype, False)
    q, k, v = (t[x][:, 0].contiguous() for x in ("q", "k", "v"))
    live = [0, 2, 3]
    ro, rS = R.attention(*(d64(t[x])[live] for x in ("q", "k", "v")), t["log_decay"], 0.5,
                         state=state[slots[live].long()])
    S = state.cuda()
    new = torch.full_like(S, 7.0)
    args = [x.cuda() for x in (q, k, v, t["log_decay"])]
    o = a.step(*args, S, slots=slots.cuda(), new_state=new, scale=0.5)
    assert torch.equal(S.cpu(), state)
    assert R.rel(o.cpu()[live], ro[:, 0]) < R.tol(dtype)
    assert not o.cpu()[[1, 4]].any()
    assert R.rel(new.cpu()[slots[live].long()], rS) < R.tol("f32")
    rest = [i for i in range(n) if i not in (3, 8, 0)]
    assert (new.cpu()[rest] == 7.0).all()
    # in place, without slots
    S2 = state.cuda()
    o2 = a.step(*args, S2, scale=0.5)
    ro, rS = R.attention(*(d64(t[x]) for x in ("q", "k", "v")), t["log_decay"], 0.5,
                         state=state[:B])
    assert R.rel(o2, ro[:, 0]) < R.tol(dtype) and R.rel(S2[:B], rS) < R.tol("f32")
    assert torch.equal(S2[B:].cpu(), state[B:])


def test_attention_steps_follow_the_prompt(pkg):
    # 40 single tokens after a prompt give what the longer prompt gives
    t = cuda(attn_inputs(2, 140, 4, 2, 64, 64, "f32", False))
    a, b = pkg.LinearAttention(2, 140, 4, 2, 64, 64), pkg.LinearAttention(2, 100, 4, 2, 64, 64)
    o, s = a.forward(t["q"], t["k"], t["v"], t["log_decay"], want_state=True)
    _, S = b.forward(*(t[n][:, :100].contiguous() for n in ("q", "k", "v")), t["log_decay"],
                     want_state=True)
    for i in range(100, 140):
        oi = b.step(*(t[n][:, i].contiguous() for n in ("q", "k", "v")), t["log_decay"], S)
        assert R.rel(oi, o[:, i].cpu()) < 5e-6
    assert R.rel(S, s.cpu()) < 5e-6


def test_attention_gradient_against_differences(pkg):
    # o and the final state are linear in each of q, k, v and s0, so a central
    # difference is exact but for float32: 2^-24 |o| sqrt(n) / h, under 1e-4 here
    t = cuda(attn_inputs(1, 150, 2, 1, 32, 32, "f32", True))
    a = pkg.LinearAttention(1, 150, 2, 1, 32, 32, backward=True)

    def loss(q, k, v, s0):
        o, s = a.forward(q, k, v, t["log_decay"], state=s0, want_state=True)
        return (o.double() * t["do"].double()).sum() + (s.double() * t["dsT"].double()).sum()

    base = [t["q"], t["k"], t["v"], t["s0"]]
    grads = a.backward(t["q"], t["k"], t["v"], t["log_decay"], t["do"], state=t["s0"],
                       dstate=t["dsT"])
    for i, gr in enumerate(grads):
        d = rand(gen(i), gr.shape).cuda()
        d = d / d.norm() + gr / gr.norm()
        hi, lo = list(base), list(base)
        hi[i], lo[i] = base[i] + d, base[i] - d
        slope = ((loss(*hi) - loss(*lo)) / 2).item()
        want = (gr.double() * d.double()).sum().item()
        assert abs(slope - want) < 1e-3 * abs(want) + 1e-3, (i, slope, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_repeatable_and_any_stream(pkg, dtype):
    t = cuda(attn_inputs(2, 2000, 4, 2, 64, 64, dtype, True))
    a = pkg.LinearAttention(2, 2000, 4, 2, 64, 64, dtype=dtype, backward=True)
    args = (t["q"], t["k"], t["v"], t["log_decay"])
    o, s = a.forward(*args, state=t["s0"], want_state=True)
    d = a.backward(*args, t["do"], state=t["s0"], dstate=t["dsT"])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        o2, s2 = a.forward(*args, state=t["s0"], want_state=True)
        d2 = a.backward(*args, t["do"], state=t["s0"], dstate=t["dsT"])
    st.synchronize()
    assert torch.equal(o, o2) and torch.equal(s, s2)
    assert all(torch.equal(x, y) for x, y in zip(d, d2))
    # the same calls in a CUDA graph
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o3, s3 = a.forward(*args, state=t["s0"], want_state=True)
    o3.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, o3) and torch.equal(s, s3)


def test_attention_refusals(pkg):
    t = cuda(attn_inputs(2, 20, 4, 2, 16, 16, "f32", True))
    a = pkg.LinearAttention(2, 20, 4, 2, 16, 16)
    args = [t["q"], t["k"], t["v"], t["log_decay"]]
    with pytest.raises(TypeError):
        a.forward(t["q"].half(), *args[1:])
    with pytest.raises(ValueError):
        a.forward(t["q"][:, :19].contiguous(), *args[1:])
    with pytest.raises(ValueError):
        a.forward(*args[:3], t["log_decay"][:1])
    with pytest.raises(TypeError):
        a.forward(*args, lengths=torch.tensor([1, 2], device="cuda"))      # int64
    with pytest.raises(pkg.FnoError) as e:
        a.backward(*args, t["do"])                                         # plan without it
    assert e.value.status == capi.FNO_ERR_INVALID_ARG
    with pytest.raises(pkg.FnoError) as e:
        a.forward(*args, out=t["q"].view(2, 20, 4, 16))
    assert e.value.status == capi.FNO_ERR_ALIASING
    with pytest.raises(ValueError):
        a.step(*(x[:, 0].contiguous() for x in args[:3]), args[3], t["s0"][..., :8])
    with pytest.raises(pkg.FnoError):     # fewer states than rows
        a.step(*(x[:, 0].contiguous() for x in args[:3]), args[3], t["s0"][:1].clone())
    with pytest.raises(pkg.FnoError):
        pkg.LinearAttention(2, 20, 4, 3, 16, 16)
