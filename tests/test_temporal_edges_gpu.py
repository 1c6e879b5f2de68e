"""Convolution, scan and rotary positions where they can go wrong without a sign: every way of
dividing a scan's work, gradients by differences, states that die or never fade, infinities
behind a sequence's end, graphs that share a plan, positions at the ends of 32 bits."""
import pytest
import torch

import ops_ref as R
import temporal_ref as M
import test_temporal_ops_gpu as base

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def pkg(fno):
    return fno


def scan_call(pkg, t, shape, dtype, plus=True):
    """(forward and backward results of the operator, the same in 64 bits) of `t`."""
    B, T, D, N, G = shape
    n = t["lengths"]
    p = pkg.SelectiveScan(B, T, D, N, groups=G, softplus=plus, dtype=dtype, backward=True)
    c = {name: base.cuda(v) for name, v in t.items()}
    for name in ("x", "dt", "B", "C", "z", "dy"):
        c[name] = None if t[name] is None else base.cuda(base.spoil(t[name], n))
    more = dict(D=c["D"], z=c["z"], dt_bias=c["bias"], lengths=c["lengths"], state=c["state"])
    y, sT = p.forward(c["x"], c["dt"], c["A"], c["B"], c["C"], want_state=True, **more)
    got = p.backward(c["x"], c["dt"], c["A"], c["B"], c["C"], c["dy"], dstate=c["dstate"], **more)
    got.update(y=y, sT=sT)
    names = [m for m in ("x", "dt", "A", "B", "C", "D", "z", "bias", "state")
             if t[m] is not None]
    with torch.device("cuda"):                           # the definition, on the GPU for speed
        leaf = {m: t[m].cuda().double().requires_grad_() for m in names}
        two = t["dt"].cuda().double().requires_grad_()
        y, sT = M.scan(*(leaf.get(m) for m in ("x", "dt", "A", "B", "C", "D", "z", "bias")),
                       plus, c["lengths"], leaf.get("state"), dt_input=two)
        loss = (y * c["dy"].double().nan_to_num()).sum()
        if t["dstate"] is not None:
            loss = loss + (sT * c["dstate"].double()).sum()
        grads = torch.autograd.grad(loss, [*leaf.values(), two])
    rename = {"bias": "ddt_bias", "state": "dstate"}
    want = {rename.get(m, "d" + m): v.cpu() for m, v in zip(names, grads)}
    parts = (want["ddt"].norm() + grads[-1].norm().cpu()).item()
    want["ddt"] = want["ddt"] + grads[-1].cpu()
    want.update(y=y.detach().cpu(), sT=sT.detach().cpu())
    return got, want, parts


REGIMES = [  # batch, length, channels, states, groups
    # segments beyond what a lane of the joining holds
    (1, 8300, 4, 16, 1), (2, 8290, 3, 2, 1),
    # spans of several segments in the backward's last pass
    (10, 1160, 640, 2, 1), (10, 700, 640, 16, 2),
    # as many sequences as fill the GPU, of one tile, two, and more
    (300, 8, 64, 16, 1), (300, 13, 64, 16, 1), (500, 16, 66, 4, 1), (260, 16, 32, 64, 2),
    (700, 41, 70, 16, 1), (420, 33, 40, 24, 1), (1000, 17, 5, 9, 1),
    # more groups than a wave has blocks, odd ones of several sequences a block, many channels
    (5, 9, 2400, 4, 600), (900, 5, 42, 8, 7), (6, 9, 20002, 2, 1),
    # groups of 32 channels and fewer, whose blocks hold several sequences
    (37, 30, 96, 16, 3), (11, 90, 16, 3, 4),
]


# (a definition of thousands of tokens takes half a minute)
@pytest.mark.parametrize("i,ragged,dtype", [(0, False, "f32"), (0, False, "bf16"), (1, True, "f16")]
                         + [(i, r, d) for i in range(2, len(REGIMES)) for r in (False, True)
                            for d in ("f32", "f16", "bf16")])
def test_scan_however_its_work_is_divided(pkg, i, ragged, dtype):
    B, T, D, N, G = REGIMES[i]
    k = i + ragged + {"f32": 0, "f16": 1, "bf16": 2}[dtype]
    skip, gate, bias, state = k % 3 != 1, k % 2 == 0, k % 3 != 2, k % 4 != 3
    t = base.scan_inputs(REGIMES[i], dtype, skip, gate, bias, True, ragged and B > 1, state)
    got, want, parts = scan_call(pkg, t, REGIMES[i], dtype)
    assert set(got) == set(want)
    f32, stored = R.tol("f32") + base.SCAN_EXTRA, R.tol(dtype) + base.SCAN_EXTRA
    for name, ref in want.items():
        # sums of terms of either sign: against the terms (as in test_scan)
        scale = {"ddt": parts, "ddt_bias": parts, "dA": parts,
                 "dD": (t["dy"].double().norm() * 0.5).item(),
                 "dB": want["dB"].norm().item() + 1e-3}.get(name)
        base.close(got[name], ref, stored if name in ("y", "dx", "ddt", "dB", "dC", "dz")
                   else f32, scale)


def test_scan_gradients_are_differences(pkg):
    """Along each gradient's own direction, of the loss as the forward computes it."""
    shape = B, T, D, N, G = 2, 45, 12, 5, 2
    t = base.scan_inputs(shape, "f32", True, True, True, True, False, True)
    c = {k: base.cuda(v) for k, v in t.items()}
    p = pkg.SelectiveScan(B, T, D, N, groups=G, backward=True)
    names = {"x": "dx", "dt": "ddt", "A": "dA", "B": "dB", "C": "dC", "D": "dD", "z": "dz",
             "bias": "ddt_bias", "state": "dstate"}

    def call(f, **kw):
        v = {**c, **kw}
        return f(v["x"], v["dt"], v["A"], v["B"], v["C"], D=v["D"], z=v["z"],
                 dt_bias=v["bias"], state=v["state"])

    def loss(**kw):
        y, sT = call(lambda *a, **m: p.forward(*a, want_state=True, **m), **kw)
        return ((y.double() * c["dy"].double()).sum()
                + (sT.double() * c["dstate"].double()).sum()).item()

    y, sT = call(lambda *a, **m: p.forward(*a, want_state=True, **m))
    size = (y.norm() * c["dy"].norm() + sT.norm() * c["dstate"].norm()).item()
    grads = call(lambda *a, **m: p.backward(*a, c["dy"], dstate=c["dstate"], **m))
    for name, g in names.items():
        d = grads[g] / grads[g].abs().max()
        slope = (grads[g].double() * d.double()).sum().item()

        def difference(eps):
            return (loss(**{name: c[name] + eps * d}) - loss(**{name: c[name] - eps * d})) / (
                2 * eps)
        eps = 2.0 ** -5
        near, far = difference(eps), difference(2 * eps)
        # the third derivative's share is a third of far - near; the outputs are good to 2e-5
        # of their size (rounding and decays), twice, over 2 eps
        bound = abs(far - near) + 2e-5 * size / eps
        assert abs(near - slope) <= bound, (name, near, slope, bound)
        assert bound < 0.1 * slope, (name, bound, slope)       # (the test says something)


def test_conv_gradients_are_differences(pkg):
    B, T, D, W = 2, 37, 10, 4
    t = base.conv_inputs((B, T, D, W), "f32", True, False, True)
    c = {k: base.cuda(v) for k, v in t.items()}
    p = pkg.CausalConv(B, T, D, W, backward=True)

    def loss(**kw):
        v = {**c, **kw}
        y, sT = p.forward(v["x"], v["w"], bias=v["bias"], state=v["state"], want_state=True)
        return ((y.double() * c["dy"].double()).sum()
                + (sT.double() * c["dstate"].double()).sum()).item()

    y, sT = p.forward(c["x"], c["w"], bias=c["bias"], state=c["state"], want_state=True)
    size = (y.norm() * c["dy"].norm() + sT.norm() * c["dstate"].norm()).item()
    grads = p.backward(c["x"], c["w"], c["dy"], bias=c["bias"], state=c["state"],
                       dstate=c["dstate"])
    for name, g in zip(("x", "w", "bias", "state"), grads):
        d = g / g.abs().max()
        slope = (g.double() * d.double()).sum().item()

        def difference(eps):
            return (loss(**{name: c[name] + eps * d}) - loss(**{name: c[name] - eps * d})) / (
                2 * eps)
        eps = 2.0 ** -5
        near, far = difference(eps), difference(2 * eps)
        # the third derivative's share is a third of far - near; the outputs are good to 1e-5
        bound = abs(far - near) + 1e-5 * size / eps
        assert abs(near - slope) <= bound, (name, near, slope, bound)
        assert bound < 0.1 * slope, (name, bound, slope)


@pytest.mark.parametrize("shape", [(2, 100, 33, 16, 1), (300, 12, 64, 5, 1), (1, 700, 8, 4, 2)])
def test_scan_states_that_die_at_once(pkg, shape):
    """Rates of -10^4: every decay is 0, and so is what each token leaves to the next."""
    t = base.scan_inputs(shape, "f32", True, True, True, True, False, True)
    t["A"] = torch.full_like(t["A"], -1e4)
    got, want, parts = scan_call(pkg, t, shape, "f32")
    for name, ref in want.items():
        scale = {"ddt": parts, "ddt_bias": parts, "dA": parts,
                 "dstate": t["dstate"].norm().item(),
                 "dD": (t["dy"].double().norm() * 0.5).item()}.get(name)
        base.close(got[name], ref, R.tol("f32") + base.SCAN_EXTRA, scale)


@pytest.mark.parametrize("T,D", [(3000, 8), (15, 40)])
def test_scan_states_that_never_fade(pkg, T, D):
    """A of 0: a sum of all tokens.  Terms of one sign, so that nothing cancels: a sum of T
    of them is off by T roundings at most."""
    shape = (2, T, D, 4, 1)
    t = base.scan_inputs(shape, "f32", False, False, False, False, True, False)
    for m in ("x", "B", "C", "dt", "dy"):
        t[m] = t[m].abs() + 0.1
    t["A"] = torch.zeros_like(t["A"])
    got, want, parts = scan_call(pkg, t, shape, "f32", plus=False)
    for name, ref in want.items():
        # (dA is a sum of products of two such sums)
        base.close(got[name], ref, R.tol("f32") + 3 * T * 2.0 ** -24,
                   parts if name in ("ddt", "dA") else None)


@pytest.mark.parametrize("T", [9, 600])
def test_what_lies_behind_the_end_is_not_looked_at(pkg, T):
    """Infinities there, lengths of nothing everywhere, and no state of its own."""
    B, D, N, W = 3, 40, 16, 4
    t = base.scan_inputs((B, T, D, N, 1), "f32", True, True, True, True, False, True)
    c = {k: base.cuda(v) for k, v in t.items()}
    ok = torch.tensor([T, 4, 0], dtype=torch.int32).cuda()
    scan = pkg.SelectiveScan(B, T, D, N, backward=True)
    conv = pkg.CausalConv(B, T, D, W, backward=True)
    w = torch.randn(D, W).cuda()

    def run(v, n):
        more = dict(D=c["D"], z=v["z"], dt_bias=c["bias"], lengths=n, state=c["state"])
        args = (v["x"], v["dt"], c["A"], v["B"], v["C"])
        y, sT = scan.forward(*args, want_state=True, **more)
        d = scan.backward(*args, v["dy"], dstate=c["dstate"], **more)
        u, s2 = conv.forward(v["x"], w, lengths=n, want_state=True)
        e = conv.backward(v["x"], w, v["dy"], lengths=n)
        return [y, sT, u, s2, *d.values(), *e[:2]]

    inf = dict(c)
    for name in ("x", "dt", "B", "C", "z", "dy"):
        inf[name] = c[name].clone()
        inf[name][1, 4:] = float("inf")
        inf[name][2] = float("-inf")
    for a, b in zip(run(c, ok), run(inf, ok)):
        assert torch.isfinite(b).all() and torch.equal(a, b)
    for name in ("x", "dt", "B", "C", "z", "dy"):
        inf[name].fill_(float("nan"))
    y, sT, u, s2, *rest = run(inf, torch.zeros(B, dtype=torch.int32).cuda())
    assert not y.any() and not u.any() and not s2.any() and torch.equal(sT, c["state"])
    d = dict(zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dstate"), rest))
    assert torch.equal(d.pop("dstate"), c["dstate"])
    assert not any(v.any() for v in d.values()) and not any(v.any() for v in rest[9:])


def test_two_graphs_of_one_plan(pkg):
    """They share its workspace; replayed one after the other, in any order, each gives the
    results of its own inputs."""
    shape = B, T, D, N, G = 1, 900, 40, 16, 1
    scan = pkg.SelectiveScan(B, T, D, N, dtype="f16", backward=True)
    graphs = []
    for seed in (0, 1):
        t = base.scan_inputs(shape, "f16", True, True, True, True, False, False, seed=seed)
        c = {k: base.cuda(v) for k, v in t.items()}

        def run(c=c):
            kw = dict(D=c["D"], z=c["z"], dt_bias=c["bias"])
            args = (c["x"], c["dt"], c["A"], c["B"], c["C"])
            return [scan.forward(*args, **kw)[0], *scan.backward(*args, c["dy"], **kw).values()]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):                       # (the first makes the workspace)
            out = run()
        graphs.append((graph, out, run))
    for k in (0, 1, 1, 0):
        graphs[k][0].replay()
    torch.cuda.synchronize()
    for _, out, run in graphs:
        for a, b in zip(out, run()):
            assert torch.equal(a, b)
    assert not torch.equal(graphs[0][1][0], graphs[1][1][0])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_positions_at_the_ends_of_32_bits(pkg, layout):
    """Tokens of an offset of 2^31 - 1 are at 2^31 - 1 + t, which is not wrapped."""
    B, T, H, dim = 3, 70, 2, 64
    q = torch.randn(B, T, H, dim, generator=base.gen(3))
    off = torch.tensor([2 ** 31 - 1, -2 ** 31, 0], dtype=torch.int32)
    out, _ = pkg.Rotary(B, T, H, 0, dim, layout=layout).forward(q.cuda(), offsets=off.cuda())
    pos = torch.arange(T) + off.long()[:, None]
    base.close(out, M.rotate(q.double(), pos, dim, layout), R.tol("f32"))


def test_rotary_of_a_gradient_undoes_it(pkg):
    """Turned and turned back: the identity, times m^2."""
    q = torch.randn(2, 33, 3, 48, generator=base.gen(4)).cuda()
    p = pkg.Rotary(2, 33, 3, 0, 48, scaling=("ramp", 4.0, 128, 8.0, 1.0))
    off = torch.tensor([5, 100000], dtype=torch.int32).cuda()
    back, _ = p.backward(p.forward(q, offsets=off)[0], offsets=off)
    m = M.frequencies(48, 10000.0, ("ramp", 4.0, 128, 8.0, 1.0))[1]
    base.close(back, q.cpu().double() * m * m, R.tol("f32"))


def test_addresses_off_their_alignment_are_refused(pkg):
    B, T, D, N = 1, 6, 8, 4
    buf = torch.zeros(B * T * D + 1, dtype=torch.bfloat16, device="cuda")
    odd, x = buf[1:].view(B, T, D), torch.zeros(B, T, D, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(B, T, 1, N, dtype=torch.bfloat16, device="cuda")
    A, w = torch.zeros(D, N, device="cuda"), torch.zeros(D, 3, device="cuda")
    with pytest.raises(pkg.FnoError):
        pkg.CausalConv(B, T, D, 3, dtype="bf16").forward(odd, w)
    with pytest.raises(pkg.FnoError):
        pkg.CausalConv(B, T, D, 3, dtype="bf16").forward(x, w, out=odd)
    scan = pkg.SelectiveScan(B, T, D, N, dtype="bf16")
    with pytest.raises(pkg.FnoError):
        scan.forward(odd, x, A, b, b)
    with pytest.raises(pkg.FnoError):
        scan.forward(x, x, A, b, b, out=odd)
    with pytest.raises(pkg.FnoError):
        pkg.Rotary(B, T, 1, 0, D, dtype="bf16").forward(odd.view(B, T, 1, D))


def test_workspaces_are_of_the_plan(pkg):
    scan = pkg.SelectiveScan(1, 900, 40, 16, backward=True)
    assert scan.workspace is None and scan.workspace_bytes > 0
    scan._workspace()
    assert scan.workspace.get_device() == scan.device
    if torch.cuda.device_count() > 1:
        with torch.cuda.device(1), pytest.raises(ValueError):
            z = torch.zeros(1, 900, 40, device="cuda:0")
            scan.forward(z, z, torch.zeros(40, 16, device="cuda:0"),
                         torch.zeros(1, 900, 1, 16, device="cuda:0"),
                         torch.zeros(1, 900, 1, 16, device="cuda:0"))
