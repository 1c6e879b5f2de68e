"""Operands and plans of another device than the current one are refused before anything is
launched.  The current device is reported as another one here, so that one GPU is enough."""
import pytest
import torch

from fft_gemm_ifft_gb300 import sequence

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def pkg(fno):
    return fno


def calls(pkg):
    """Name -> a valid call of every entry point."""
    def z(*s, dtype=torch.float32):
        return torch.zeros(s, dtype=dtype, device="cuda")

    x, f8 = z(2, 8, 4), pkg.pack_activation(z(2, 8, 4))
    v = {k: z(8) for k in ("s", "w2", "w1")}
    norm, lin = pkg.SandwichNorm(8, 4, 2), pkg.LinearGrad(2, 8, 3, 4)
    att = pkg.LinearAttention(2, 5, 2, 1, 8, 8, backward=True)
    q, k, decay, st = z(2, 5, 2, 8), z(2, 5, 1, 8), z(2), z(2, 2, 8, 8)
    conv = pkg.CausalConv(2, 5, 6, 3, backward=True)
    scan = pkg.SelectiveScan(2, 5, 6, 4, backward=True)
    rot = pkg.Rotary(2, 5, 2, 1, 8)
    t, w, A, b = z(2, 5, 6), z(6, 3), z(6, 4), z(2, 5, 1, 4)
    return {
        "pack": lambda: pkg.pack_activation(x),
        "values": lambda: f8.values(),
        "gelu": lambda: f8.gelu_backward(x),
        "norm.pre": lambda: norm.pre(x, v),
        "norm": lambda: norm.forward(x, x, v, y=z(2, 8, 4)),
        "norm.backward": lambda: norm.backward(x, f8, v, x),
        "linear": lambda: lin.backward(z(2, 3, 4), f8),
        "attention": lambda: att.forward(q, k, k, decay),
        "attention.backward": lambda: att.backward(q, k, k, decay, q),
        "attention.step": lambda: att.step(q[:, 0].contiguous(), k[:, 0].contiguous(),
                                           k[:, 0].contiguous(), decay, st),
        "rotary": lambda: rot.forward(q, k),
        "conv": lambda: conv.forward(t, w),
        "conv.backward": lambda: conv.backward(t, w, t),
        "conv.step": lambda: conv.step(z(2, 6), w, z(2, 2, 6)),
        "scan": lambda: scan.forward(t, t, A, b, b),
        "scan.backward": lambda: scan.backward(t, t, A, b, b, t),
        "scan.step": lambda: scan.step(z(2, 6), z(2, 6), A, z(2, 1, 4), z(2, 1, 4), z(2, 6, 4)),
    }


def test_another_current_device(pkg, monkeypatch):
    every = calls(pkg)
    for call in every.values():
        call()
    monkeypatch.setattr(sequence, "_current_device", lambda: 1)
    for name, call in every.items():
        with pytest.raises(ValueError, match="not the current device"):
            call()
            pytest.fail(name)


def test_operands_of_another_device(pkg, monkeypatch):
    """Plans of device 1 while it is current, tensors of device 0."""
    for name, call in calls(pkg).items():
        if name not in ("pack", "values", "gelu"):
            call()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)       # plans are made on it
    every = calls(pkg)
    monkeypatch.setattr(sequence, "_current_device", lambda: 1)
    for name, call in every.items():
        if name not in ("pack", "values", "gelu"):                     # (these have no plan)
            with pytest.raises(ValueError, match="must be on cuda:1"):
                call()
                pytest.fail(name)
