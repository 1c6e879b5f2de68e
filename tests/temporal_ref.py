"""Definitions in 64 bits of the operators that mix a sequence along time (causal
convolution, selective scan, rotary positions), on the CPU and differentiable."""
import math

import torch


def _valid(B, T, lengths):
    n = torch.full((B,), T) if lengths is None else lengths.long().clamp(0, T)
    return n, (torch.arange(T)[None] < n[:, None])[..., None]


def conv(x, w, bias, silu, lengths=None, state=None):
    """(y, final state); what lies beyond a sequence's length is not looked at."""
    B, T, D = x.shape
    W = w.shape[1]
    n, m = _valid(B, T, lengths)
    x = torch.where(m, x, torch.zeros_like(x))
    first = torch.zeros(B, W - 1, D, dtype=torch.float64) if state is None else state
    full = torch.cat([first, x], 1)
    pre = sum(full[:, j:j + T] * w[:, j] for j in range(W))
    if bias is not None:
        pre = pre + bias
    y = pre / (1.0 + torch.exp(-pre)) if silu else pre
    at = (n[:, None] + torch.arange(W - 1))[..., None].expand(B, W - 1, D)
    return torch.where(m, y, torch.zeros_like(y)), torch.gather(full, 1, at)


def softplus(v):
    return torch.logaddexp(v, torch.zeros_like(v))


def scan(x, dt, A, B, C, D=None, z=None, bias=None, plus=True, lengths=None, state=None,
         dt_input=None):
    """(y, final state), token by token.  ``dt_input``: the dt of the inputs' steps where
    it is told apart from that of the decays (for the parts of its gradient)."""
    n_b, T, ch = x.shape
    per = ch // B.shape[2]

    def steps(v):
        v = v if bias is None else v + bias
        return softplus(v) if plus else v

    h = (torch.zeros(n_b, ch, A.shape[1], dtype=torch.float64) if state is None else state)
    n, _ = _valid(n_b, T, lengths)
    out = []
    for t in range(T):
        on = (t < n)[:, None]
        zero = torch.zeros_like(x[:, t])
        pick = lambda v: torch.where(on, v, zero)           # noqa: E731
        d = steps(pick(dt[:, t]))
        du = d if dt_input is None else steps(pick(dt_input[:, t]))
        xt = pick(x[:, t])
        wide = on[..., None]
        Bt, Ct = (torch.where(wide, v[:, t], torch.zeros_like(v[:, t])).repeat_interleave(per, 1)
                  for v in (B, C))
        new = torch.exp(d[..., None] * A) * h + (du * xt)[..., None] * Bt
        h = torch.where(wide, new, h)
        y = (Ct * h).sum(-1)
        if D is not None:
            y = y + D * xt
        if z is not None:
            zt = pick(z[:, t])
            y = y * zt / (1.0 + torch.exp(-zt))
        out.append(torch.where(on, y, zero))
    return torch.stack(out, 1), h


def frequencies(r, base, scaling=None):
    """(radians a position of each pair, magnitude)."""
    kind, *v = ("none",) if scaling is None else scaling
    if kind == "base":
        base = base * v[0] ** (r / (r - 2))
    f = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if kind == "linear":
        f = [x / v[0] for x in f]
    if kind == "ramp":
        factor, original, fast, slow = v
        keep = [min(1.0, max(0.0, (original * x / (2 * math.pi) - slow) / (fast - slow)))
                for x in f]
        f = [x * (k + (1 - k) / factor) for x, k in zip(f, keep)]
    return torch.tensor(f, dtype=torch.float64), (1 + 0.1 * math.log(v[0]) if kind == "ramp"
                                                   else 1.0)


def rotate(x, pos, r, layout, base=10000.0, scaling=None):
    """x (batch, length, heads, dim) at positions pos (batch, length)."""
    f, mag = frequencies(r, base, scaling)
    angle = pos.double()[:, :, None, None] * f
    cos, sin = mag * torch.cos(angle), mag * torch.sin(angle)
    out = x.clone()
    first, second = ((slice(0, r // 2), slice(r // 2, r)) if layout == "half"
                     else (slice(0, r, 2), slice(1, r, 2)))
    a, b = x[..., first], x[..., second]
    out[..., first], out[..., second] = a * cos - b * sin, b * cos + a * sin
    return out
