"""Definitions in 64 bits of the sequence operators, on the CPU, for the tests."""
import math

import torch

GROUP = 128
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# half an ulp of the storage type, relative (24, 11 and 8 significant bits)
HALF_ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def rel(got, ref):
    got, ref = got.detach().double().cpu(), ref.detach().double()
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert torch.isfinite(got).all()
    norm = ref.norm().item()
    diff = (got - ref).norm().item()
    return diff / norm if norm else diff


def tol(dtype, roundings=1):
    """Bound on the relative 2-norm error: every rounding to the storage type is
    off by at most half an ulp of its value; the float32 sums of these tests
    (up to some thousand terms) stay under 1e-5, the library's own bound."""
    return 1e-5 + (0.0 if dtype == "f32" else roundings * HALF_ULP[dtype])


# ----- 8-bit checkpoints (the codes are those of float32 arithmetic) -----
def pack(x):
    x = x.detach().cpu().float()
    n = x.shape[-1]
    pad = -n % GROUP
    v = torch.nn.functional.pad(x, (0, pad)).unflatten(-1, (-1, GROUP))
    m = v.abs().amax(-1)
    keep = ~(m < 1e-30)
    # tensor by tensor: a division by (or of) a Python number is carried out as
    # a product with a rounded reciprocal
    top = torch.full_like(m, 127.0)
    inv = torch.where(keep, top / m, torch.zeros_like(m))
    q = torch.round(v * inv[..., None])
    q = torch.nan_to_num(q, nan=0.0).to(torch.int8).flatten(-2)[..., :n]
    return q.contiguous(), torch.where(keep, m / top, torch.zeros_like(m))


def values(codes, scales):
    at = torch.arange(codes.shape[-1]) // GROUP
    return codes.cpu().double() * scales.cpu().double()[..., at]


def gelu_slope(v):
    return (0.5 * torch.special.erfc(-v / math.sqrt(2.0))
            + v * torch.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi))


# ----- sandwich norm; fields as (batch, channels, points) or (batch, points, channels) -----
def norm(v, kind, eps, w, b, ax):
    shape = [1] * v.dim()
    shape[ax] = -1
    if kind == "layer":
        v = v - v.mean(ax, keepdim=True)
    n = v / torch.sqrt((v * v).mean(ax, keepdim=True) + eps) * w.view(shape)
    return n + b.view(shape) if kind == "layer" else n


def sandwich(x, f, p, kind, eps, layout, gate=None, sigmoid=False, want_u=True):
    """(y, u) in 64 bits; differentiable."""
    ax = 1 if layout == "grid" else 2
    shape = [1, 1, 1]
    shape[ax] = -1
    y = x
    if f is not None:
        z = norm(f, kind, eps, p["w2"], p.get("b2"), ax)
        if gate is not None:
            a = 1.0 / (1.0 + torch.exp(-gate)) if sigmoid else gate
            z = z * (a.unsqueeze(2 if layout == "grid" else 1) if a.dim() == 2 else a)
        y = x + p["s"].view(shape) * z
    return y, norm(y, kind, eps, p["w1"], p.get("b1"), ax) if want_u else None


# ----- linear attention, token by token; differentiable -----
def attention(q, k, v, log_decay, scale, lengths=None, state=None):
    B, T, H, dk = q.shape
    G = H // k.shape[2]
    k, v = k.repeat_interleave(G, 2), v.repeat_interleave(G, 2)
    gamma = torch.exp(log_decay.double())[None, :, None, None]
    S = (torch.zeros(B, H, dk, v.shape[3], dtype=torch.float64) if state is None
         else state.double())
    n = (torch.full((B,), T) if lengths is None else lengths.long().clamp(0, T))
    out = []
    for t in range(T):
        on = (t < n)[:, None, None, None]
        new = gamma * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        S = torch.where(on, new, S)
        o = scale * torch.einsum("bhd,bhde->bhe", q[:, t], S)
        out.append(torch.where(on[..., 0], o, torch.zeros_like(o)))
    return torch.stack(out, 1), S
