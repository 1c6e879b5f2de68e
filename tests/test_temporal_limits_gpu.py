"""Convolution, scan and rotary positions at the ends of what their plans take: products of
sizes that pass 32 bits, workspaces, digits, what lies around the operands, streams."""
import pytest
import torch

import ops_ref as R
import temporal_ref as M
import test_temporal_edges_gpu as edges
import test_temporal_ops_gpu as base
from fft_gemm_ifft_gb300 import capi

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def pkg(fno):
    return fno


def room(gigabytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gigabytes * 1e9:
        pytest.skip(f"wants {gigabytes} GB of device memory")


def test_scan_rows_of_b_and_c_of_more_than_31_bits(pkg):
    """groups x states = 2^31 + 512: the last groups' outputs and gradients, of both tokens,
    are those of a plan that has these groups alone, and the others' are zero."""
    room(100)
    T, N, K = 2, 32, 64
    G = (1 << 26) + 16                                  # one channel each
    t = base.scan_inputs((1, T, K, N, K), "bf16", True, False, True, True, False, False)
    few = {k: v.cuda() for k, v in t.items() if v is not None}

    def many(name, shape):
        v = torch.zeros(shape, dtype=few[name].dtype, device="cuda")
        v.narrow(v.dim() - 1 if name in ("x", "dt", "dy", "D", "bias") else
                 0 if name == "A" else 2, G - K, K).copy_(few[name])
        return v

    def run(v, groups):
        p = pkg.SelectiveScan(1, T, groups, N, groups=groups, dtype="bf16", backward=True)
        args, more = [v[k] for k in ("x", "dt", "A", "B", "C")], dict(D=v["D"], dt_bias=v["bias"])
        out = {"y": p.forward(*args, **more)[0]}
        out.update(p.backward(*args, v["dy"], **more))
        p.close()
        return out

    want = run(few, K)
    shapes = {"x": (1, T, G), "dt": (1, T, G), "dy": (1, T, G), "A": (G, N), "D": (G,),
              "bias": (G,), "B": (1, T, G, N), "C": (1, T, G, N)}
    got = run({k: many(k, s) for k, s in shapes.items()}, G)
    assert set(got) == set(want)
    for name, ref in want.items():
        axis = {"dB": 2, "dC": 2}.get(name, 0 if name in ("dA", "dD", "ddt_bias") else 2)
        assert torch.equal(got[name].narrow(axis, G - K, K), ref), name
        rest = got[name].narrow(axis, 0, G - K)
        for row in (rest[0].unbind(0) if axis == 2 else (rest,)):
            assert not row.any(), name


@pytest.mark.parametrize("per_group", [1, 2, 3, 16, 33, 64, 100])
@pytest.mark.parametrize("N", [4, 16, 40])
def test_scan_workspace_goes_by_the_channels(pkg, per_group, N):
    """What the backward keeps for every 8 tokens is a state of each channel, padded to twice
    the channels and the next power of two of the states at most, however many groups there
    are; nothing is allocated for it here."""
    B, T, G = 4, 4096, 2048 // per_group
    p = pkg.SelectiveScan(B, T, G * per_group, N, groups=G, backward=True)
    padded = 1 << max(2, (N - 1).bit_length())
    kept = 4 * B * (T // 8) * G * per_group * padded
    # besides: a sum of the steps for each kept state, the segments' states (64 tokens at
    # least, forwards and backwards), the blocks' parts of the gradients
    chblocks = -(-per_group // 64)
    rest = kept // padded + 3 * kept // 8 + 4 * B * (T // 64) * G * per_group * (padded + 2)
    if chblocks > 1:
        rest += 4 * chblocks * B * T * G * 2 * N
    assert p.workspace is None and p.workspace_bytes <= 2 * kept + rest
    p.close()


@pytest.mark.parametrize("shape", [(2, 90, 6, 5, 3), (1, 200, 35, 16, 7), (3, 40, 102, 8, 6),
                                   (2, 33, 130, 16, 2), (1, 70, 9, 24, 9), (2, 64, 132, 4, 4)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scan_kept_states_of_small_groups(pkg, shape, dtype):
    """Groups of 1 to 65 channels keep their states in units of 2 to 64 channels."""
    t = base.scan_inputs(shape, dtype, True, True, True, True, shape[0] > 1, True)
    got, want, parts = edges.scan_call(pkg, t, shape, dtype)
    f32, stored = R.tol("f32") + base.SCAN_EXTRA, R.tol(dtype) + base.SCAN_EXTRA
    for name, ref in want.items():
        # sums of terms of either sign: against the terms
        scale = {"ddt": parts, "ddt_bias": parts, "dA": parts,
                 "dD": (t["dy"].double().norm() * 0.5).item(),
                 "dB": want["dB"].norm().item() + 1e-3}.get(name)
        base.close(got[name], ref, stored if name in ("y", "dx", "ddt", "dB", "dC", "dz")
                   else f32, scale)


def test_scan_workspaces_that_no_gpu_has_are_refused(pkg):
    """2^38 bytes: 64 sequences of 2^17 tokens keep 2^20 states of 4096 x 64."""
    with pytest.raises(pkg.FnoError):
        pkg.SelectiveScan(64, 1 << 17, 4096, 64, backward=True)
    pkg.SelectiveScan(64, 1 << 17, 4096, 64).close()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 3, 2, 1, 3, 2), (2, 50, 7, 3, 9, 4), (3, 7, 40, 9, 33, 32),
                                   (1, 400, 5, 5, 5, 2), (2, 19, 3, 2, 10, 6), (1, 21, 4, 4, 6, 6)])
def test_rotary_of_neighbours_element_by_element(pkg, dtype, shape):
    """Pairs of neighbours in heads of odd (or odd numbers of pairs of) elements, which are read
    one or two at a time; in place, and beside elements that are copied."""
    B, T, H, K, dim, r = shape
    g = base.gen(sum(shape))
    q, k = base.rand(g, (B, T, H, dim), dtype), base.rand(g, (B, T, K, dim), dtype)
    p = pkg.Rotary(B, T, H, K, dim, rotary_dim=r, layout="interleaved", dtype=dtype)
    pos = torch.arange(T).expand(B, T)
    for call, sign in ((p.forward, 1), (p.backward, -1)):
        a, b = q.cuda(), k.cuda()
        oq, ok = call(a, b)
        call(a, b, q_out=a, k_out=b)
        assert torch.equal(a, oq) and torch.equal(b, ok)
        for got, x in ((oq, q), (ok, k)):
            # element by element, besides half a step of the type (2^-25 below fp16's normal
            # numbers), relative to the pair: in float32 pi 2^-25 of the angle, a unit (2^-24) of
            # cosine and sine each, and 2^-24 of the product: below 2^-21; in 16 bits the angle's
            # product with pi (2^-21) and the fast cosines (2^-21 each): below 2^-19
            want = M.rotate(x.double(), sign * pos, r, "interleaved")
            eps = torch.finfo(x.dtype).eps / 2
            size = want.abs() + 0
            size[..., :r] = x.double()[..., :r].unflatten(-1, (-1, 2)).norm(
                dim=-1, keepdim=True).expand(B, T, x.shape[2], r // 2, 2).flatten(-2)
            bound = (eps * want.abs() + 2.0 ** (-21 if dtype == "f32" else -19) * size
                     + (2.0 ** -25 if dtype == "f16" else 0.0))
            assert ((got.cpu().double() - want).abs() <= bound).all()
            assert torch.equal(got[..., r:].cpu(), x[..., r:])
    p.close()


@pytest.mark.parametrize("call", ["step", "forward"])
def test_scan_decays(pkg, call):
    """One token without an input: the state times e^{d A}, for |d A| from 0.001 to 100.  The
    exponent is d times A log2 e, each product rounded (2^-24) and log2 e itself (1.4e-8), which
    is 1.4e-7 |d A| of the result, and the power of two is good to 1.5e-7."""
    D, N = 64, 16
    g = base.gen(5)
    x = torch.exp(torch.empty(D, N).uniform_(-6.9, 4.6, generator=g))            # |d A|
    d = torch.exp(torch.empty(1, 1, D).uniform_(-7, 3, generator=g))
    A = -(x / d.view(D, 1)).contiguous()
    zero, h = torch.zeros(1, 1, D).cuda(), torch.ones(1, D, N).cuda()
    bc = torch.ones(1, 1, 1, N).cuda()
    p = pkg.SelectiveScan(1, 1, D, N, softplus=False)
    if call == "forward":
        _, h = p.forward(zero, d.cuda(), A.cuda(), bc, bc, state=h, want_state=True)
    else:
        p.step(zero[:, 0], d[:, 0].cuda(), A.cuda(), bc[:, 0], bc[:, 0], h)
    dA = A.double() * d.double().view(D, 1)
    want = torch.exp(dA)
    bound = (1.5e-7 + 1.4e-7 * dA.abs()) * want + 2.0 ** -126
    assert ((h.cpu().double()[0] - want).abs() <= bound).all()


@pytest.mark.parametrize("B,T,D", [(1, 4000, 8), (40, 3000, 64)])
def test_scan_that_remembers_a_thousand_tokens(pkg, B, T, D):
    """Steps of 0.001 at a rate of 1, with terms of one sign, so that nothing cancels."""
    N, memory = 8, 1000.0
    g = base.gen(T)

    def some(*shape):
        return (0.5 + torch.rand(shape, generator=g)).cuda()

    x, Bm, Cm, dy = some(B, T, D), some(B, T, 1, N), some(B, T, 1, N), some(B, T, D)
    d, A = torch.full((B, T, D), 1e-3, device="cuda"), -torch.ones(D, N, device="cuda")
    p = pkg.SelectiveScan(B, T, D, N, softplus=False, backward=True)
    y, sT = p.forward(x, d, A, Bm, Cm, want_state=True)
    got = p.backward(x, d, A, Bm, Cm, dy)
    # 64 bits: all decays are a = e^{d A}, so that sums over earlier tokens are products with
    # powers of a, here by blocks of 500 tokens
    a = torch.exp(d[0, 0, 0].double() * A[0, 0].double())

    def run(u, reverse=False):
        """s_t = a s_{t-1} + u_t along axis 1."""
        u = u.flip(1) if reverse else u
        out, s = [], torch.zeros_like(u[:, 0])
        for part in u.split(500, 1):
            n = part.shape[1]
            i = torch.arange(n, device="cuda")
            low = torch.where(i[:, None] >= i, a ** (i[:, None] - i).clamp(min=0), 0.0 * a)
            o = torch.einsum("ts,bs...->bt...", low, part)
            o = o + torch.einsum("t,b...->bt...", a ** (i + 1), s)
            out.append(o)
            s = o[:, -1]
        o = torch.cat(out, 1)
        return o.flip(1) if reverse else o

    dd = d.double()
    u = (dd * x.double())[..., None] * Bm.double()
    h = run(u)
    # a decay is good to 1.5e-7 and a sum's rounding is 2^-24, for each token remembered
    bound = memory * (1.5e-7 + 2.0 ** -24) + 1e-5
    base.close(y, (h * Cm.double()).sum(-1).cpu(), bound)
    base.close(sT, h[:, -1].cpu(), bound)
    gr = run(Cm.double() * dy.double()[..., None], reverse=True)
    s1 = (gr * Bm.double()).sum(-1)
    base.close(got["dx"], (dd * s1).cpu(), bound)
    base.close(got["dB"], (gr * (dd * x.double())[..., None]).sum(2, keepdim=True).cpu(), bound)
    base.close(got["dC"], (h * dy.double()[..., None]).sum(2, keepdim=True).cpu(), bound)
    before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    e = a * gr * before                                  # of two such sums
    base.close(got["dA"], (dd[..., None] * e).sum((0, 1)).cpu(), 2 * bound)
    first, second = x.double() * s1, (A.double() * e).sum(-1)
    base.close(got["ddt"], (first + second).cpu(), 2 * bound,
               (first.norm() + second.norm()).item())


# ---------------------------------------------------------------------------
# what lies around the operands
# ---------------------------------------------------------------------------
ZONE = 4096                                            # bytes in front and behind


class Zones:
    """Operands between zones of bytes 0xff (a NaN in every type), which no call writes; what
    an operand holds before it is written is NaN as well."""

    def __init__(self):
        self.bufs = []

    def new(self, nbytes):
        buf = torch.full((2 * ZONE + -(-nbytes // 256) * 256,), 0xff, dtype=torch.uint8,
                         device="cuda")
        self.bufs.append((buf, nbytes))
        return buf[ZONE:ZONE + nbytes]

    def empty(self, shape, dtype):
        n = torch.Size(shape).numel() * torch.empty((), dtype=dtype).element_size()
        return self.new(n).view(dtype).view(shape)

    def of(self, t):
        return None if t is None else self.empty(t.shape, t.dtype).copy_(t)

    def check(self):
        for buf, n in self.bufs:
            assert (buf[:ZONE] == 0xff).all() and (buf[ZONE + n:] == 0xff).all()


def ptr(t):
    return None if t is None else t.data_ptr()


def ws_of(plan, zones):
    return zones.new(plan.workspace_bytes).data_ptr() if plan.workspace_bytes else None


def same(got, want):
    for name, t in want.items():
        assert torch.equal(got[name], t), name


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(3, 13, 21, 5, 1), (1, 300, 33, 16, 3), (2, 90, 130, 24, 2),
                                   (5, 17, 10, 4, 5), (1, 700, 7, 64, 7), (300, 9, 34, 16, 1),
                                   (2, 1, 3, 2, 1)])
def test_scan_leaves_what_lies_around(pkg, dtype, shape):
    """Every output and a workspace of exactly its size, filled with NaN beforehand."""
    B, T, D, N, G = shape
    t = base.scan_inputs(shape, dtype, True, True, True, True, B > 1, True)
    c = {k: base.cuda(v) for k, v in t.items()}
    p = pkg.SelectiveScan(B, T, D, N, groups=G, dtype=dtype, backward=True)
    more = dict(D=c["D"], z=c["z"], dt_bias=c["bias"], lengths=c["lengths"], state=c["state"])
    args = [c[k] for k in ("x", "dt", "A", "B", "C")]
    y, sT = p.forward(*args, want_state=True, **more)
    back = p.backward(*args, c["dy"], dstate=c["dstate"], **more)
    zones, s = Zones(), torch.cuda.current_stream().cuda_stream
    ins = [ptr(zones.of(v)) for v in (*args, c["D"], c["z"], c["bias"], c["lengths"], c["state"])]
    got = {"y": zones.empty(y.shape, y.dtype), "sT": zones.empty(sT.shape, sT.dtype)}
    pkg.check(capi.fno_scan_forward(p.handle, *ins, ptr(got["y"]), ptr(got["sT"]),
                                    ws_of(p, zones), s))
    got.update({k: zones.empty(v.shape, v.dtype) for k, v in back.items()})
    order = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dstate")
    pkg.check(capi.fno_scan_backward(p.handle, *ins, ptr(zones.of(c["dy"])),
                                     ptr(zones.of(c["dstate"])), *(ptr(got[k]) for k in order),
                                     ws_of(p, zones), s))
    torch.cuda.synchronize()
    zones.check()
    same(got, {"y": y, "sT": sT, **back})


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(3, 13, 21, 3), (1, 300, 33, 8), (2, 90, 130, 4), (5, 1, 1, 2),
                                   (300, 9, 34, 5)])
def test_conv_leaves_what_lies_around(pkg, dtype, shape):
    B, T, D, W = shape
    c = {k: base.cuda(v) for k, v in
         base.conv_inputs(shape, dtype, True, B > 1, True).items()}
    p = pkg.CausalConv(B, T, D, W, dtype=dtype, backward=True)
    more = dict(bias=c["bias"], lengths=c["lengths"], state=c["state"])
    y, sT = p.forward(c["x"], c["w"], want_state=True, **more)
    back = p.backward(c["x"], c["w"], c["dy"], dstate=c["dstate"], **more)
    zones, s = Zones(), torch.cuda.current_stream().cuda_stream
    ins = [ptr(zones.of(c[k])) for k in ("x", "w", "bias", "lengths", "state")]
    got = {"y": zones.empty(y.shape, y.dtype), "sT": zones.empty(sT.shape, sT.dtype)}
    pkg.check(capi.fno_causal_conv_forward(p.handle, *ins, ptr(got["y"]), ptr(got["sT"]), s))
    outs = {k: zones.empty(v.shape, v.dtype) for k, v in zip(("dx", "dw", "db", "ds"), back)}
    pkg.check(capi.fno_causal_conv_backward(
        p.handle, *ins, ptr(zones.of(c["dy"])), ptr(zones.of(c["dstate"])),
        *(ptr(v) for v in outs.values()), ws_of(p, zones), s))
    torch.cuda.synchronize()
    zones.check()
    same({**got, **outs}, {"y": y, "sT": sT, **dict(zip(outs, back))})


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,N,G,W", [(21, 5, 1, 3), (34, 16, 2, 4), (3, 64, 3, 8), (1, 1, 1, 2)])
def test_steps_leave_what_lies_around(pkg, dtype, D, N, G, W):
    B, slots = 4, 6
    at = torch.tensor([5, -1, 0, 6], dtype=torch.int32).cuda()            # two rows are idle
    t = {k: base.cuda(v) for k, v in base.scan_inputs(
        (B, 1, D, N, G), dtype, True, True, True, True, False, False).items()}
    row = [t[k][:, 0].contiguous() for k in ("x", "dt", "B", "C", "z")]
    s = torch.cuda.current_stream().cuda_stream
    scan = pkg.SelectiveScan(B, 1, D, N, groups=G, dtype=dtype)
    conv = pkg.CausalConv(B, 1, D, W, dtype=dtype)
    state = torch.randn(slots, D, N, device="cuda")
    inputs = torch.randn(slots, W - 1, D, device="cuda").to(row[0].dtype)
    w, bias = torch.randn(D, W, device="cuda"), torch.randn(D, device="cuda")
    h, u = state.clone(), inputs.clone()
    y = scan.step(row[0], row[1], t["A"], row[2], row[3], h, D=t["D"], z=row[4],
                  dt_bias=t["bias"], slots=at)
    v = conv.step(row[0], w, u, bias=bias, slots=at)
    zones = Zones()
    oy, ov = zones.empty(y.shape, y.dtype), zones.empty(v.shape, v.dtype)
    nh, nu = zones.of(state), zones.of(inputs)
    ins = [ptr(zones.of(x)) for x in (row[0], row[1], t["A"], row[2], row[3], t["D"], row[4],
                                      t["bias"], at)]
    pkg.check(capi.fno_scan_step(scan.handle, *ins, slots, ptr(zones.of(state)), ptr(nh), ptr(oy),
                                 s))
    pkg.check(capi.fno_causal_conv_step(
        conv.handle, *(ptr(zones.of(x)) for x in (row[0], w, bias, at)), slots,
        ptr(zones.of(inputs)), ptr(nu), ptr(ov), s))
    torch.cuda.synchronize()
    zones.check()
    same({"y": oy, "v": ov, "h": nh, "u": nu}, {"y": y, "v": v, "h": h, "u": u})


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("shape", [(3, 13, 3, 2, 7, 4), (1, 65, 5, 1, 20, 10),
                                   (2, 9, 4, 4, 64, 64)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rotary_leaves_what_lies_around(pkg, dtype, shape, layout):
    B, T, H, K, dim, r = shape
    g = base.gen(7)
    q = base.rand(g, (B, T, H, dim), dtype).cuda()
    k = base.rand(g, (B, T, K, dim), dtype).cuda()
    off = torch.arange(B, dtype=torch.int32).cuda() * 1000
    p = pkg.Rotary(B, T, H, K, dim, rotary_dim=r, layout=layout, dtype=dtype)
    want = dict(zip("qk", p.forward(q, k, offsets=off)))
    zones = Zones()
    got = {n: zones.empty(v.shape, v.dtype) for n, v in want.items()}
    pkg.check(capi.fno_rotary_apply(p.handle, ptr(zones.of(q)), ptr(zones.of(k)), None,
                                    ptr(zones.of(off)), 0, ptr(got["q"]), ptr(got["k"]),
                                    torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    zones.check()
    same(got, want)


# ---------------------------------------------------------------------------
# streams
# ---------------------------------------------------------------------------
def test_calls_go_to_the_stream_they_are_given(pkg):
    """Inputs that arrive late on a side stream: a call that went to the current stream in place
    of stream= would have read what was there before."""
    B, T, D, N, W, H = 2, 300, 72, 16, 4, 9
    t = {k: base.cuda(v) for k, v in base.scan_inputs(
        (B, T, D, N, 1), "bf16", True, True, True, True, False, True).items()}
    w, busy = torch.randn(D, W, device="cuda"), torch.randn(4096, 4096, device="cuda")
    scan = pkg.SelectiveScan(B, T, D, N, dtype="bf16", backward=True)
    conv = pkg.CausalConv(B, T, D, W, dtype="bf16", backward=True)
    one, first = pkg.SelectiveScan(B, 1, D, N, dtype="bf16"), pkg.CausalConv(B, 1, D, W,
                                                                             dtype="bf16")
    rot = pkg.Rotary(B, T, H, 0, D // H, dtype="bf16")
    h, u = t["state"].clone(), torch.ones(B, W - 1, D, device="cuda").bfloat16()
    x = torch.zeros_like(t["x"])
    rows = {k: t[k][:, 0].contiguous() for k in ("x", "dt", "B", "C")}
    x0 = torch.zeros_like(rows["x"])
    args = (t["dt"], t["A"], t["B"], t["C"])
    CALLS = {
        "conv": lambda s: conv.forward(x, w, want_state=True, stream=s),
        "conv.backward": lambda s: conv.backward(x, w, t["dy"], stream=s)[:2],
        "conv.step": lambda s: (first.step(x0, w, u, new_state=torch.empty_like(u), stream=s),),
        "scan": lambda s: scan.forward(x, *args, state=t["state"], want_state=True, stream=s),
        "scan.backward": lambda s: tuple(scan.backward(x, *args, t["dy"], stream=s).values()),
        "scan.step": lambda s: (one.step(x0, rows["dt"], t["A"], rows["B"], rows["C"], h,
                                         new_state=torch.empty_like(h), stream=s),),
        "rotary": lambda s: (rot.forward(x.view(B, T, H, D // H), stream=s)[0],),
        "rotary.backward": lambda s: (rot.backward(x.view(B, T, H, D // H), stream=s)[0],),
    }
    side, current = torch.cuda.Stream(), torch.cuda.current_stream()
    for name, call in CALLS.items():
        x.copy_(t["x"])
        x0.copy_(rows["x"])
        want = [v.clone() for v in call(None)]
        x.zero_()
        x0.zero_()
        zero = [v.clone() for v in call(None)]
        assert any(not torch.equal(a, b) for a, b in zip(want, zero)), name
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(30):                                 # some milliseconds
                torch.mm(busy, busy)
            x.copy_(t["x"])
            x0.copy_(rows["x"])
        got = call(side)
        current.wait_stream(side)
        for a, b in zip(got, want):
            assert torch.equal(a, b), name
        torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# offsets of more than 31 bits
# ---------------------------------------------------------------------------
def test_scan_and_conv_rows_of_more_than_31_bits(pkg):
    """2^31 + 2^27 elements a field, and twice as many in the states that the backward keeps:
    the first and the last sequence have the same tokens and give the same bits; those between
    have none."""
    room(100)
    B, T, D, N = 17, 1 << 17, 1 << 10, 16
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
    lengths[0] = lengths[-1] = T

    def rows(*width, scale=1.0, mean=0.0):
        t = torch.full((B, T, *width), float("nan"), dtype=torch.bfloat16, device="cuda")
        t[0] = mean + scale * torch.randn(T, *width, device="cuda")
        t[-1] = t[0]
        return t

    def check(t, name):
        assert torch.isfinite(t[0]).all() and t[0].any(), name
        assert torch.equal(t[0], t[-1]), name
        for row in t[1:-1]:
            assert not row.any(), name

    x, dy = rows(D), rows(D)
    w = torch.randn(D, 4, device="cuda")
    conv = pkg.CausalConv(B, T, D, 4, dtype="bf16", backward=True)
    check(conv.forward(x, w, lengths=lengths)[0], "conv")
    dx, dw, _, _ = conv.backward(x, w, dy, lengths=lengths)
    check(dx, "conv dx")
    assert torch.isfinite(dw).all()
    del dx, conv
    dt, Bm, Cm = rows(D, scale=0.5, mean=-2.0), rows(1, N), rows(1, N)
    A = -(0.5 + torch.rand(D, N, device="cuda"))
    scan = pkg.SelectiveScan(B, T, D, N, dtype="bf16", backward=True)
    y, sT = scan.forward(x, dt, A, Bm, Cm, lengths=lengths, want_state=True)
    check(y, "y")
    check(sT, "state")
    del y
    for name, t in scan.backward(x, dt, A, Bm, Cm, dy, lengths=lengths).items():
        if name == "dA":
            assert torch.isfinite(t).all()
        else:
            check(t, name)


def test_slots_of_more_than_31_bits(pkg):
    """States of 2^31 elements and more: a slot behind them is as one in front."""
    room(40)
    D, N, W = 1024, 64, 8
    slots = (1 << 31) // (D * N) + 3
    state = torch.zeros(slots, D, N, device="cuda")
    state[0] = torch.randn(D, N, device="cuda")
    state[-1] = state[0]
    g = base.scan_inputs((1, 1, D, N, 1), "bf16", True, True, True, True, False, False)
    row = {k: (v[:, 0] if k in ("x", "dt", "B", "C", "z") else v).cuda()
           for k, v in g.items() if v is not None}
    two = {k: row[k].expand(2, *row[k].shape[1:]).contiguous()
           for k in ("x", "dt", "B", "C", "z")}
    at = torch.tensor([0, slots - 1], dtype=torch.int32).cuda()
    p = pkg.SelectiveScan(2, 1, D, N, dtype="bf16")
    before = state[0].clone()
    y = p.step(two["x"], two["dt"], row["A"], two["B"], two["C"], state, D=row["D"], z=two["z"],
               dt_bias=row["bias"], slots=at)
    assert torch.equal(y[0], y[1]) and torch.equal(state[0], state[-1])
    assert not torch.equal(state[0], before)
    for part in state[1:-1].split(4096):
        assert not part.any()
    del state
    slots = (1 << 31) // (D * (W - 1)) + 3
    inputs = torch.zeros(slots, W - 1, D, dtype=torch.bfloat16, device="cuda")
    inputs[0] = torch.randn(W - 1, D, device="cuda")
    inputs[-1] = inputs[0]
    old = inputs[0].clone()
    at = torch.tensor([0, slots - 1], dtype=torch.int32).cuda()
    y = pkg.CausalConv(2, 1, D, W, dtype="bf16").step(two["x"], torch.randn(D, W, device="cuda"),
                                                      inputs, slots=at)
    assert torch.equal(y[0], y[1]) and torch.equal(inputs[0], inputs[-1])
    assert torch.equal(inputs[0, :-1], old[1:]) and torch.equal(inputs[0, -1], two["x"][0])
    for part in inputs[1:-1].split(65536):
        assert not part.any()


# ---------------------------------------------------------------------------
# one more way of dividing a scan's work
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("shape", [(400, 130, 4, 16, 1), (160, 200, 70, 16, 1),
                                   (100, 70, 6, 40, 2)])
def test_scan_split_in_front_of_one_span(pkg, dtype, ragged, shape):
    """Sequences that fill the last pass backward without a split in time but not the passes in
    front of it, which are split: the gradient of the final state goes past the segments."""
    t = base.scan_inputs(shape, dtype, True, True, True, True, ragged, True)
    got, want, parts = edges.scan_call(pkg, t, shape, dtype)
    f32, stored = R.tol("f32") + base.SCAN_EXTRA, R.tol(dtype) + base.SCAN_EXTRA
    for name, ref in want.items():
        # sums of terms of either sign: against the terms
        scale = {"ddt": parts, "ddt_bias": parts, "dA": parts,
                 "dD": (t["dy"].double().norm() * 0.5).item(),
                 "dB": want["dB"].norm().item() + 1e-3}.get(name)
        base.close(got[name], ref, stored if name in ("y", "dx", "ddt", "dB", "dC", "dz")
                   else f32, scale)
