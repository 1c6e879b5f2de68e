"""The example that runs the sequence operators together: a training step with
8-bit checkpoints, and the rollout of single frames."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(fno):
    spec = importlib.util.spec_from_file_location(
        "temporal_operator", os.path.join(ROOT, "examples", "temporal_operator.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_trains_and_rolls_out(example):
    losses, gap = example.main(steps=25, batch=2, time=6, n=16, channels=16, rate=0.2)
    assert losses[-1] < 0.5 * losses[0]
    # single frames carry float32 states through the same arithmetic: 1e-5
    assert gap < 1e-5


def test_gradients_against_differences(example):
    # The checkpoints are within half a step of 1/127 of their group's largest
    # value, so a weight's gradient is off by about 1 %: 5 % is asked for, along
    # directions with a sizeable slope.
    x, target = example.travelling_waves(1, 5, 16, 16)
    m = example.TemporalOperator(1, 5, 16, 16)

    def loss():
        return float(((m.forward(x)[0] - target).double() ** 2).mean())

    out, keep = m.forward(x)
    err = out - target
    grads = m.backward(2.0 / err.numel() * err, keep)
    for name, g in grads.items():
        if name == "x":
            continue
        group, _, key = name.rpartition(".")
        w = ({"space": m.space, "time": m.time}[group] if group else m.w)[key]
        d = g / g.norm()
        h = 1e-2
        w += h * d
        hi = loss()
        w -= 2 * h * d
        lo = loss()
        w += h * d
        slope, want = (hi - lo) / (2 * h), float((g * d).sum())
        assert abs(slope - want) < 0.05 * abs(want) + 1e-4, (name, slope, want)
