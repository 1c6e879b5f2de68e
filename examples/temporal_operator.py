"""A time-dependent neural operator on the library's operators, trained with
8-bit activation checkpoints and rolled out one frame at a time.

One block of the model maps frames x (batch, time, channels, n, n) to the next
frame's features:

    u  = n1(x)                                  norm in front of the block
    y  = x + s (n2(SpectralConv(u)) w2)         over space, each frame by itself
    z  = y + s' a (n2'(A y) w2')                over time, each point by itself: A is
                                                decayed linear attention, a a gate
    out = P GELU(L z + l)                       pointwise head, one output channel

The training step keeps the spectral layer's output and the head's input and
pre-activation in 8 bits; every gradient is taken by the library's backward
calls.  The rollout carries the attention's state instead of the past frames.
A gate per channel of each point makes every point a sample of the norm over time,
which takes batch n^2 up to 65535.

    python examples/temporal_operator.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from fft_gemm_ifft_gb300 import (LinearAttention, LinearGrad, SandwichNorm,  # noqa: E402
                                 SpectralConv, capi, pack_activation)


class TemporalOperator:
    def __init__(self, batch, time, n=32, channels=32, modes=8, heads=4, kv_heads=2, width=16,
                 seed=0):
        self.b, self.t, self.n, self.c = batch, time, n, channels
        self.p, self.frames, self.heads, self.kv, self.d = n * n, batch * time, heads, kv_heads, width
        g = torch.Generator().manual_seed(seed)

        def rnd(*shape, scale=1.0):
            return (scale * torch.randn(shape, generator=g)).cuda()

        c = channels
        self.w = {
            "spec": rnd(2, c, c, modes, modes, 2, scale=0.5 / c),
            "q": rnd(c, heads * width, scale=c ** -0.5), "k": rnd(c, kv_heads * width, scale=c ** -0.5),
            "v": rnd(c, kv_heads * width, scale=c ** -0.5),
            "o": rnd(heads * width, c, scale=(heads * width) ** -0.5),
            "lin": rnd(c, c, scale=c ** -0.5), "bias": torch.zeros(c, device="cuda"),
            "proj": rnd(c, scale=c ** -0.5), "gate": torch.zeros(batch * self.p, c, device="cuda"),
        }
        one = torch.ones(c, device="cuda")
        self.space = {"s": 0.5 * one, "w2": one.clone(), "w1": one.clone()}
        self.time = {"s": 0.5 * one, "w2": one.clone()}
        span = 2.0 ** torch.linspace(1.0, 5.0, heads)            # memory of 2 to 32 frames
        self.log_decay = torch.log1p(-1.0 / span).float().cuda()
        self._plans(batch, time)

    def _plans(self, b, t):
        n, c, p = self.n, self.c, self.p
        self.conv = SpectralConv((n, n), self.w["spec"].shape[3:5], b * t, c, c,
                                 flags=capi.FNO_PLAN_BACKWARD)
        self.norm_space = SandwichNorm(c, p, b * t, layout="grid")
        self.norm_time = SandwichNorm(c, t, b * p, layout="tokens", gate="channel",
                                      gate_sigmoid=True)
        self.attention = LinearAttention(b * p, t, self.heads, self.kv, self.d, self.d,
                                         backward=True)
        self.head = LinearGrad(b * t, c, c, p)

    # frames (b t, c, p) <-> a sequence for each point (b p, t, c)
    def _to_time(self, x):
        return (x.view(self.b, self.t, self.c, self.p).permute(0, 3, 1, 2)
                .reshape(self.b * self.p, self.t, self.c).contiguous())

    def _to_space(self, x):
        return (x.view(self.b, self.p, self.t, self.c).permute(0, 2, 3, 1)
                .reshape(self.frames, self.c, self.p).contiguous())

    def _qkv(self, y):
        shape = y.shape[:-1]
        return [(y @ self.w[k]).view(*shape, h, self.d).contiguous()
                for k, h in (("q", self.heads), ("k", self.kv), ("v", self.kv))]

    def forward(self, x):
        """x (batch, time, channels, n, n) -> (batch, time, n, n) and what the
        backward needs."""
        w, keep = self.w, {}
        x = x.reshape(self.frames, self.c, self.p)
        u = self.norm_space.pre(x, self.space)
        f = self.conv(u.view(-1, self.c, self.n, self.n), w["spec"]).view(x.shape)
        y, _, keep["f8"] = self.norm_space.forward(x, f, self.space, save8=True, want_u=False)
        y = self._to_time(y)
        q, k, v = self._qkv(y)
        o, keep["state"] = self.attention.forward(q, k, v, self.log_decay, want_state=True)
        a = (o.flatten(2) @ w["o"]).contiguous()
        z, _, keep["a8"] = self.norm_time.forward(y, a, self.time, gate=w["gate"], save8=True,
                                                  want_u=False)
        zs = self._to_space(z)
        t = torch.matmul(w["lin"], zs) + w["bias"][:, None]
        keep.update(x=x, u=u, y=y, q=q, k=k, v=v, o=o, z=z, z8=pack_activation(zs),
                    t8=pack_activation(t))
        h = torch.nn.functional.gelu(t)
        keep["h"] = h
        out = torch.einsum("c,bcp->bp", w["proj"], h)
        return out.view(self.b, self.t, self.n, self.n), keep

    def backward(self, dout, keep):
        """Gradients of every weight (the norms' under ``space.*`` / ``time.*``)."""
        w, g = self.w, {}
        dout = dout.reshape(self.frames, 1, self.p)
        g["proj"] = (dout * keep["h"]).sum((0, 2))
        dt = keep["t8"].gelu_backward((w["proj"][:, None] * dout).contiguous())
        g["lin"], g["bias"] = self.head(dt, keep["z8"])
        dz = self._to_time(torch.matmul(w["lin"].t(), dt))
        d = self.norm_time.backward(keep["z"], keep["a8"], self.time, dz, gate=w["gate"])
        g.update({"time." + k: d["d" + k] for k in self.time}, gate=d["dgate"])
        g["o"] = keep["o"].flatten(2).flatten(0, 1).t() @ d["df"].flatten(0, 1)
        do = (d["df"] @ w["o"].t()).view_as(keep["o"]).contiguous()
        dq, dk, dv, _ = self.attention.backward(keep["q"], keep["k"], keep["v"], self.log_decay, do)
        dy = d["dx"]
        for k, x in (("q", dq), ("k", dk), ("v", dv)):
            x = x.flatten(2)
            g[k] = keep["y"].flatten(0, 1).t() @ x.flatten(0, 1)
            dy = dy + x @ w[k].t()
        dy = self._to_space(dy)
        # y enters only through its own stream here: x's gradient comes in two parts
        d = self.norm_space.backward(keep["x"], keep["f8"], self.space, dy)
        g.update({"space." + k: d["d" + k] for k in ("s", "w2")})
        du, g["spec"] = self.conv.backward(keep["u"].view(-1, self.c, self.n, self.n), w["spec"],
                                           d["df"].view(-1, self.c, self.n, self.n))
        e = self.norm_space.backward(keep["x"], None, self.space, d["dx"], du.view(keep["u"].shape))
        g["space.w1"], g["x"] = e["dw1"], e["dx"]
        return g

    def apply(self, grads, rate):
        for k, v in grads.items():
            if k == "x":
                continue
            group, _, name = k.rpartition(".")
            target = {"space": self.space, "time": self.time}[group] if group else self.w
            target[name] -= rate * v

    def start_rollout(self, batch):
        """Plans for single frames; returns the empty history."""
        self._step = {
            "conv": SpectralConv((self.n, self.n), self.w["spec"].shape[3:5], batch, self.c, self.c),
            "space": SandwichNorm(self.c, self.p, batch, layout="grid"),
            "time": SandwichNorm(self.c, 1, batch * self.p, layout="tokens", gate="channel",
                                 gate_sigmoid=True),
            "attention": LinearAttention(batch * self.p, 1, self.heads, self.kv, self.d, self.d),
        }
        return torch.zeros((batch * self.p, self.heads, self.d, self.d), device="cuda")

    def step(self, x, state):
        """One frame x (batch, channels, n, n) -> (batch, n, n); the history in
        ``state`` is updated in place."""
        s, w, b = self._step, self.w, x.shape[0]
        x = x.reshape(b, self.c, self.p).contiguous()
        u = s["space"].pre(x, self.space)
        f = s["conv"](u.view(-1, self.c, self.n, self.n), w["spec"]).view(x.shape)
        y, _, _ = s["space"].forward(x, f, self.space, want_u=False)
        y = y.transpose(1, 2).reshape(b * self.p, 1, self.c).contiguous()
        q, k, v = (t[:, 0].contiguous() for t in self._qkv(y))
        o = s["attention"].step(q, k, v, self.log_decay, state)
        a = (o.flatten(1) @ w["o"])[:, None].contiguous()
        z, _, _ = s["time"].forward(y, a, self.time, gate=w["gate"], want_u=False)
        z = z.view(b, self.p, self.c).transpose(1, 2)
        h = torch.nn.functional.gelu(torch.matmul(w["lin"], z) + w["bias"][:, None])
        return torch.einsum("c,bcp->bp", w["proj"], h).view(b, self.n, self.n)


def travelling_waves(batch, time, n, channels, seed=1):
    """Frames whose channel 0 is a field moving over a periodic grid, the others
    its fixed random features; the target is the next frame's field."""
    g = torch.Generator().manual_seed(seed)
    k = torch.arange(n).float() * (2.0 * torch.pi / n)
    phase = 6.28 * torch.rand((batch, 3, 2), generator=g)
    speed = 0.5 + torch.rand((batch, 3), generator=g)
    t = torch.arange(time + 1).float()
    field = sum(torch.cos((m + 1) * (k[:, None] + k[None, :])[None, None]
                          - speed[:, m, None, None, None] * t[None, :, None, None]
                          + phase[:, m, 0, None, None, None]) / (m + 1) for m in range(3))
    mix = torch.randn((channels,), generator=g)
    bias = 0.1 * torch.randn((channels, n, n), generator=g)
    x = field[:, :-1, None] * mix[:, None, None] + bias
    return x.cuda(), field[:, 1:].cuda()


def main(steps=40, batch=2, time=12, n=32, channels=32, rate=0.05):
    x, target = travelling_waves(batch, time, n, channels)
    model = TemporalOperator(batch, time, n, channels)
    losses = []
    for _ in range(steps):
        out, keep = model.forward(x)
        err = out - target
        losses.append(float((err * err).mean()))
        model.apply(model.backward(2.0 / err.numel() * err, keep), rate)
    out, _ = model.forward(x)
    state = model.start_rollout(batch)
    frames = torch.stack([model.step(x[:, i], state) for i in range(time)], 1)
    gap = float((frames - out).norm() / out.norm())
    return losses, gap


if __name__ == "__main__":
    losses, gap = main()
    print(f"mean squared error {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps; "
          f"frame by frame against the whole sequence: {gap:.1e}")
