"""Convolution, scan and rotary positions at the ends of what their plans take: products of
sizes that pass 32 bits."""
import pytest
import torch

import ops_ref as R
import temporal_ref as M
import test_temporal_edges_gpu as edges
import test_temporal_ops_gpu as base

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
