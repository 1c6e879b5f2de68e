"""The sequence operators on the GPU where a call goes wrong without a sign: the
digits of 16-bit results, operands that are also results, infinities and NaN,
several tiles or rows for each block of threads, other streams."""
import pytest
import torch

import ops_ref as R
from fft_gemm_ifft_gb300 import capi
from test_ops_gpu import attn_inputs, check_norm, cuda, d64, gen, norm_inputs, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def pkg(fno):
    return fno


# ---------------------------------------------------------------------------
# sandwich norm
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("C", [300, 1024, 2300])
def test_norm_alone_over_many_rows(pkg, dtype, kind, C):
    # rows of several warps, several rows for each: the rows' sums follow one another
    # in the same shared memory
    P = 4099
    t, p = norm_inputs("tokens", 1, P, C, dtype, kind, "none")
    n = pkg.SandwichNorm(C, P, 1, layout="tokens", norm=kind, dtype=dtype)
    T, PR = cuda(t), cuda(p)
    p64 = {k: v.double().requires_grad_() for k, v in p.items()}
    x = d64(t["x"]).requires_grad_()
    _, ru = R.sandwich(x, None, p64, kind, 1e-5, "tokens")
    names = ["dx", "dw1"] + ["db1"] * (kind == "layer")
    want = torch.autograd.grad(ru, [x] + [p64[k[1:]] for k in names[1:]], d64(t["du"]))
    got = n.backward(T["x"], None, PR, None, T["du"])
    for k, w in zip(names, want):
        assert R.rel(got[k], w) < R.tol(dtype if k == "dx" else "f32"), k
    for _ in range(3):
        again = n.backward(T["x"], None, PR, None, T["du"])
        assert all(torch.equal(again[k], got[k]) for k in got)


@pytest.mark.parametrize("layout,C", [("grid", 24), ("grid", 130), ("grid", 700), ("grid", 4099),
                                      ("tokens", 40), ("tokens", 300), ("tokens", 4099)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("where", ["x", "f", "dy", "du"])
def test_norm_gradients_of_nan(pkg, layout, C, kind, where):
    # a NaN of one element is a NaN wherever the definition has one, and nowhere else
    B, P = 2, 70
    t, p = norm_inputs(layout, B, P, C, "f32", kind, "none")
    at = (1, C // 2, 33) if layout == "grid" else (1, 33, C // 2)
    t[where][at] = float("nan")
    p64 = {k: v.double().requires_grad_() for k, v in p.items()}
    y, f = d64(t["x"]).requires_grad_(), d64(t["f"]).requires_grad_()
    _, ru = R.sandwich(y, None, p64, kind, 1e-5, layout)
    layer = kind == "layer"
    g1 = torch.autograd.grad(ru, [y, p64["w1"]] + ([p64["b1"]] if layer else []), d64(t["du"]))
    dY = g1[0] + d64(t["dy"])
    ry, _ = R.sandwich(torch.zeros_like(y), f, p64, kind, 1e-5, layout, want_u=False)
    g2 = torch.autograd.grad(ry, [f, p64["s"], p64["w2"]] + ([p64["b2"]] if layer else []), dY)
    want = dict(zip(["df", "ds", "dw2", "db2"], g2), dx=dY, dw1=g1[1])
    if layer:
        want["db1"] = g1[2]
    n = pkg.SandwichNorm(C, P, B, layout=layout, norm=kind)
    T = cuda(t)
    got = n.backward(T["x"], T["f"], cuda(p), T["dy"], T["du"])
    assert set(got) == set(want)
    for k, w in want.items():
        assert torch.equal(torch.isnan(got[k]).cpu(), torch.isnan(w)), k


@pytest.mark.parametrize("B", [2 ** 31 + 9, 2 ** 32 + 5])
def test_norm_of_more_samples_than_a_grid_has_blocks(pkg, B):
    # one point and channel a sample: 9 to 17 GB
    x = torch.ones((B, 1, 1), dtype=torch.float16, device="cuda")
    x[-3:, 0, 0] = torch.tensor([-2.0, 0.0, 0.003], dtype=torch.float16)
    u = torch.full_like(x, float("nan"))
    n = pkg.SandwichNorm(1, 1, B, dtype="f16")
    n.pre(x, {"w1": torch.ones(1, device="cuda")}, u=u)
    t = x[-4:, 0, 0].double().cpu()
    want = t / torch.sqrt(t * t + 1e-5)
    assert (u[-4:, 0, 0].double().cpu() - want).abs().max() < 2.0 ** -11
    one = u[-4]
    for i in range(0, B - 3, 1 << 30):
        assert (u[i:min(i + (1 << 30), B - 3)] == one).all()


def test_norm_in_place_over_two_inputs(pkg):
    # y may be x, but not while x is f as well: f's codes are taken after y is stored
    n = pkg.SandwichNorm(8, 65, 2)
    x = torch.randn(2, 8, 65, device="cuda")
    one = torch.ones(8, device="cuda")
    w = {"s": one, "w2": one, "w1": one}
    before = x.clone()
    with pytest.raises(pkg.FnoError) as e:
        n.forward(x, x, w, y=x, save8=True)
    assert e.value.status == capi.FNO_ERR_ALIASING and torch.equal(x, before)
    y, _, f8 = n.forward(x, x, w, save8=True)               # apart from y: as any f
    assert torch.equal(f8.codes, pkg.pack_activation(x).codes)


@pytest.mark.parametrize("layout,P,C", [("grid", 400, 24), ("grid", 401, 40), ("grid", 20001, 40),
                                        ("grid", 333, 200), ("grid", 130, 300), ("grid", 200, 600),
                                        ("grid", 33, 4099), ("tokens", 4099, 40),
                                        ("tokens", 4099, 300), ("tokens", 700, 1025),
                                        ("tokens", 50, 4099), ("tokens", 9, 9000)])
@pytest.mark.parametrize("dtype,kind,gate", [("f32", "layer", "full"), ("bf16", "rms", "channel"),
                                             ("f16", "layer", "none")])
def test_norm_over_its_operands(pkg, layout, P, C, dtype, kind, gate):
    # y over x and dx over dy (the C ABI) are what they are apart
    B = 2
    t, p = norm_inputs(layout, B, P, C, dtype, kind, gate)
    n = pkg.SandwichNorm(C, P, B, layout=layout, norm=kind, gate=gate, dtype=dtype)
    T, PR = cuda(t), cuda(p)
    y, u, f8 = n.forward(T["x"], T["f"], PR, gate=T["gate"], save8=True)
    x = T["x"].clone()
    y2, u2, g8 = n.forward(x, T["f"], PR, gate=T["gate"], save8=True, y=x)
    assert torch.equal(x, y) and torch.equal(u, u2) and torch.equal(f8.codes, g8.codes)
    for f in (T["f"], f8):
        want = n.backward(y, f, PR, T["dy"], T["du"], gate=T["gate"])
        got = {k: torch.full_like(v, float("nan")) for k, v in want.items()}
        got["dx"] = T["dy"].clone()
        packed = f is f8
        ptr = lambda v: None if v is None else v.data_ptr()
        assert capi.fno_sandwich_backward(
            n.handle, ptr(y), None if packed else ptr(f), ptr(f8.codes) if packed else None,
            ptr(f8.scales) if packed else None, ptr(T["gate"]), ptr(PR["s"]), ptr(PR["w2"]),
            ptr(PR.get("b2")), ptr(PR["w1"]), ptr(got["dx"]), ptr(T["du"]), ptr(got["dx"]),
            ptr(got["df"]), ptr(got.get("dgate")), ptr(got["ds"]), ptr(got["dw2"]),
            ptr(got.get("db2")), ptr(got["dw1"]), ptr(got.get("db1")), n.workspace.data_ptr(),
            torch.cuda.current_stream().cuda_stream) == capi.FNO_OK
        for k, w in want.items():
            assert torch.equal(got[k], w), k


# Rows, tiles and blocks for several turns of every CTA (one wave has 152 SMs' worth),
# the last of them in part: what is on its way while a CTA works, the buffers' second
# use, sums over turns.
TURNS = [("tokens", 1, 4099, 300), ("tokens", 1, 4099, 1024), ("tokens", 3, 21001, 40),
         ("tokens", 1, 3001, 2500), ("grid", 2, 39999, 64), ("grid", 2, 40000, 64),
         ("grid", 1, 60000, 20), ("grid", 2, 12010, 200), ("grid", 1, 12003, 300),
         ("grid", 1, 25002, 600), ("grid", 1, 12001, 520)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("i", range(len(TURNS)))
def test_norm_of_several_turns(pkg, dtype, i):
    layout, B, P, C = TURNS[i]
    kinds, gates = ["rms", "layer"], ["none", "channel", "full"]
    k = i + ["f32", "f16", "bf16"].index(dtype)
    check_norm(pkg, layout, B, P, C, dtype, kinds[k % 2], gates[k % 3], k % 4 < 2, False)
    check_norm(pkg, layout, B, P, C, dtype, kinds[1 - k % 2], gates[(k + 1) % 3], k % 4 > 1, True)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("layout,P,C", [("tokens", 4099, 300), ("tokens", 20001, 40),
                                        ("grid", 39999, 24), ("grid", 12003, 300),
                                        ("grid", 25002, 520)])
def test_norm_of_several_turns_is_repeatable(pkg, dtype, layout, P, C):
    t, p = norm_inputs(layout, 1, P, C, dtype, "layer", "full")
    n = pkg.SandwichNorm(C, P, 1, layout=layout, norm="layer", gate="full", dtype=dtype)
    T, PR = cuda(t), cuda(p)
    for f in (T["f"], pkg.pack_activation(T["f"])):
        a = n.backward(T["x"], f, PR, T["dy"], T["du"], gate=T["gate"])
        for _ in range(3):
            b = n.backward(T["x"], f, PR, T["dy"], T["du"], gate=T["gate"])
            assert all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("layout,B,P,C", [("tokens", 100, 3, 40), ("grid", 33, 70, 24),
                                          ("tokens", 3001, 12, 32), ("grid", 1000, 5, 300),
                                          ("tokens", 65535, 2, 8), ("grid", 65535, 2, 3)])
def test_norm_gate_of_many_samples(pkg, layout, B, P, C):
    # a gate per sample and channel, up to the most samples it takes
    check_norm(pkg, layout, B, P, C, "f32", "layer", "channel", True, False)
    check_norm(pkg, layout, B, P, C, "bf16", "rms", "channel", False, True)


def test_packed_activation_refusals(pkg):
    c, s = (torch.zeros((3, 0), dtype=t, device="cuda") for t in (torch.int8, torch.float32))
    with pytest.raises(TypeError):
        pkg.PackedActivation(None, s, torch.float32)
    with pytest.raises(ValueError):
        pkg.PackedActivation(c, s, torch.float32)               # no element
    with pytest.raises(ValueError):
        pkg.PackedActivation(c.new_zeros(()), s.new_zeros(()), torch.float32)
    with pytest.raises(TypeError):
        pkg.PackedActivation(c.new_zeros((3, 4)).float(), s.new_zeros((3, 1)), torch.float32)


# ---------------------------------------------------------------------------
# weight and bias gradient
# ---------------------------------------------------------------------------
def check_linear_grad(pkg, B, ci, co, P, dtype):
    g = gen(B + ci + co + P)
    x, dy = rand(g, (B, ci, P), dtype), rand(g, (B, co, P), dtype)
    p = pkg.pack_activation(x.cuda())
    n = pkg.LinearGrad(B, ci, co, P, dtype=dtype)
    dw, db = n(dy.cuda(), p)
    v = R.values(p.codes, p.scales)
    assert R.rel(dw, torch.einsum("bop,bip->oi", dy.double(), v)) < R.tol("f32")
    want = dy.double().sum((0, 2))
    assert ((db.cpu().double() - want).abs() <= 1e-5 * dy.double().abs().sum((0, 2))).all()
    assert n.device_error() == 0


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("P", [1, 2, 3, 5, 7, 9, 129, 131])
def test_linear_grad_of_few_elements(pkg, dtype, P):
    # rows that end within a word, samples of a row or two
    for B, ci, co in ((5, 1, 1), (6, 1, 2), (9, 3, 1), (700, 1, 1)):
        check_linear_grad(pkg, B, ci, co, P, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,ci,co,P", [(2, 64, 64, 50048), (3, 40, 60, 50001), (1, 128, 33, 99999),
                                       (2, 130, 200, 40008), (700, 5, 7, 129)])
def test_linear_grad_of_several_blocks(pkg, dtype, B, ci, co, P):
    # five blocks and more for every CTA: each stage and accumulator again
    check_linear_grad(pkg, B, ci, co, P, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("ci", [40, 128])                # the bias by a row of ones, by threads
@pytest.mark.parametrize("P", [256, 301])
def test_linear_grad_of_infinities(pkg, dtype, ci, P):
    # codes of no element are 0: an infinity in dy is one in every weight of its output,
    # two of opposite signs are NaN, and no other output sees them
    B, co = 2, 24
    g = gen(P + ci)
    x = rand(g, (B, ci, P), dtype)
    x = torch.where(x < 0, x - 0.5, x + 0.5)
    dy = rand(g, (B, co, P), dtype)
    inf = float("inf")
    dy[0, 3, 17], dy[1, 5, P - 1], dy[1, 20, 130] = inf, -inf, inf
    dy[0, 9, 0], dy[1, 9, 0] = inf, -inf
    dy[1, 11, 200] = float("nan")
    p = pkg.pack_activation(x.cuda())
    assert p.codes.bool().all()
    dw, db = pkg.LinearGrad(B, ci, co, P, dtype=dtype)(dy.cuda(), p)
    v = R.values(p.codes, p.scales)
    want = torch.stack([(dy[:, o, None].double() * v).sum((0, 2)) for o in range(co)])
    for got, w in ((dw.cpu(), want), (db.cpu(), dy.double().sum((0, 2)))):
        for kind in (torch.isnan, torch.isposinf, torch.isneginf):
            assert torch.equal(kind(got), kind(w)), kind
        fine = torch.isfinite(w)
        assert R.rel(got[fine], w[fine]) < R.tol("f32")


# ---------------------------------------------------------------------------
# linear attention
# ---------------------------------------------------------------------------
def close(got, want, size, name):
    """Element by element: a bfloat16 result is its exact value rounded once (half
    an ulp, 2^-8 of the value at most), and what the sums' terms were off by: the
    weights of a chunk, the state in front of it and what is added to that are held
    to 16 bits each, 2^-16 of a term, under 2^-14 of the terms' sizes together
    with the float32 sums."""
    d = (got.detach().double().cpu() - want).abs()
    bound = R.HALF_ULP["bf16"] * want.abs() + 2.0 ** -14 * size
    assert (d <= bound).all(), (name, (d / bound).max().item())


@pytest.mark.parametrize("B,T,H,K,dk,dv", [(2, 300, 4, 4, 64, 64), (1, 700, 4, 2, 128, 128),
                                           (1, 300, 2, 2, 48, 80), (2, 200, 2, 1, 20, 36)])
@pytest.mark.parametrize("state", [False, True])
def test_attention_bfloat16_digits(pkg, B, T, H, K, dk, dv, state):
    t = attn_inputs(B, T, H, K, dk, dv, "bf16", state)
    a = pkg.LinearAttention(B, T, H, K, dk, dv, dtype="bf16", backward=True)
    C = cuda(t)
    args = (C["q"], C["k"], C["v"], C["log_decay"])
    o, sT = a.forward(*args, scale=0.5, state=C["s0"], want_state=state)
    grads = a.backward(*args, C["do"], scale=0.5, state=C["s0"], dstate=C["dsT"])

    def run(f):             # results of f(inputs), and the gradients
        w = [f(d64(t[x])).requires_grad_() for x in ("q", "k", "v")]
        s0 = f(d64(t["s0"])).requires_grad_() if state else None
        ro, rS = R.attention(*w, t["log_decay"], 0.5, None, s0)
        loss = (ro * f(d64(t["do"]))).sum()
        if state:
            loss = loss + (rS * f(d64(t["dsT"]))).sum()
        return [ro.detach()] + list(torch.autograd.grad(loss, w))
    want, size = run(lambda x: x.clone()), run(torch.abs)
    for got, w, s, name in zip([o, *grads[:3]], want, size, ("o", "dq", "dk", "dv")):
        close(got, w, s, name)
    assert a.device_error() == 0


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 64), ("f16", 128)])
@pytest.mark.parametrize("T", [200, 1024, 2500, 4096, 9000])     # 1, 2, 5, 8 and more segments
def test_attention_states_in_place(pkg, dtype, d, T):
    # sT = s0 and ds0 = gsT (the C ABI allows them): every part of the time axis starts
    # from the state as it was.  The parts are joined in the same order by either way,
    # but for the rounding of the initial state's product
    t = attn_inputs(1, T, 2, 1, d, d, dtype, True)
    t["log_decay"] = torch.tensor([-1e-4, -2e-3])       # the initial state counts to the end
    C = cuda(t)
    a = pkg.LinearAttention(1, T, 2, 1, d, d, dtype=dtype, backward=True)
    args = (C["q"], C["k"], C["v"], C["log_decay"])
    o, sT = a.forward(*args, state=C["s0"], want_state=True)
    grads = a.backward(*args, C["do"], state=C["s0"], dstate=C["dsT"])
    space = torch.empty(a.workspace_bytes, dtype=torch.uint8, device="cuda")
    ws = space.data_ptr()
    p = [x.data_ptr() for x in args] + [d ** -0.5, None]
    st = torch.cuda.current_stream().cuda_stream
    for _ in range(3):
        s, o2 = C["s0"].clone(), torch.empty_like(o)
        assert capi.fno_linattn_forward(a.handle, *p, s.data_ptr(), o2.data_ptr(), s.data_ptr(),
                                        ws, st) == capi.FNO_OK
        assert R.rel(o2, o.cpu()) < (2e-6 if dtype == "f32" else R.HALF_ULP[dtype] / 8)
        assert R.rel(s, sT.cpu()) < 2e-6
        ds, g = C["dsT"].clone(), [torch.empty_like(x) for x in grads[:3]]
        assert capi.fno_linattn_backward(a.handle, *p, C["s0"].data_ptr(), C["do"].data_ptr(),
                                         ds.data_ptr(), *(x.data_ptr() for x in g),
                                         ds.data_ptr(), ws, st) == capi.FNO_OK
        for x, y in zip(g, grads):
            assert R.rel(x, y.cpu()) < (2e-6 if dtype == "f32" else R.HALF_ULP[dtype] / 8)
        assert R.rel(ds, grads[3].cpu()) < 2e-6
    assert a.device_error() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 129), (33, 130), (7, 255), (200, 131), (256, 256)])
def test_attention_step_of_wide_values(pkg, dtype, dk, dv):
    # more value columns than threads: a second round, which some threads have no column of
    B, H = 3, 2
    t = attn_inputs(B, 1, H, 1, dk, dv, dtype, True)
    C = cuda(t)
    a = pkg.LinearAttention(B, 1, H, 1, dk, dv, dtype=dtype)
    ro, rS = R.attention(*(d64(t[x]) for x in ("q", "k", "v")), t["log_decay"], 0.5, state=t["s0"])
    o = a.step(*(C[x][:, 0].contiguous() for x in ("q", "k", "v")), C["log_decay"], C["s0"],
               scale=0.5)
    assert R.rel(o, ro[:, 0]) < R.tol(dtype) and R.rel(C["s0"], rS) < R.tol("f32")
