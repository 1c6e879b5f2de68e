"""Convolution, scan and rotary positions at the ends of what their plans take: products of
sizes that pass 32 bits."""
import pytest
import torch

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
