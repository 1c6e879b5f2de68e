"""The sequence operators on the GPU where a call goes wrong without a sign: the
digits of 16-bit results, operands that are also results, infinities and NaN,
several tiles or rows for each block of threads, other streams."""
import pytest
import torch

import ops_ref as R
from test_ops_gpu import attn_inputs, cuda, d64, norm_inputs

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
