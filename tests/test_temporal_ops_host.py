"""Argument checks of the causal convolution, the selective scan and the rotary positions;
no GPU is needed: descriptions and addresses are checked before any CUDA call."""
import ctypes

import pytest

from fft_gemm_ifft_gb300 import capi

BAD, UNS, OK = capi.FNO_ERR_INVALID_ARG, capi.FNO_ERR_UNSUPPORTED, capi.FNO_OK


@pytest.fixture(scope="module", autouse=True)
def L():
    from fft_gemm_ifft_gb300 import build
    build.build()
    return capi.lib()


def scan_desc(**kw):
    d = capi.fno_scan_desc_t()
    for name, x in {**dict(batch=2, length=5, channels=6, states=4, groups=2, softplus=1, dtype=0,
                           flags=0), **kw}.items():
        setattr(d, name, x)
    return d


def rotary_desc(**kw):
    d = capi.fno_rotary_desc_t()
    for name, x in {**dict(batch=2, length=5, heads=4, kv_heads=2, dim=8, rotary_dim=8, layout=0,
                           scaling=0, base=10000.0, factor=0.0, original=0.0, fast=0.0, slow=0.0,
                           dtype=0), **kw}.items():
        setattr(d, name, x)
    return d


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), BAD), (dict(length=0), BAD), (dict(channels=0), BAD), (dict(states=0), BAD),
    (dict(groups=0), BAD), (dict(groups=4), BAD), (dict(dtype=3), BAD), (dict(flags=2), BAD),
    (dict(batch=-1), BAD), (dict(states=65), UNS), (dict(length=1 << 40), UNS),
    (dict(batch=1 << 36), UNS),
])
def test_scan_plan_rejects(kw, code):
    st, h = capi.fno_scan_plan(scan_desc(**kw))
    assert st == code and not h


INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), BAD), (dict(length=0), BAD), (dict(heads=0), BAD), (dict(kv_heads=-1), BAD),
    (dict(dim=0), BAD), (dict(rotary_dim=0), BAD), (dict(rotary_dim=7), BAD),
    (dict(rotary_dim=10), BAD), (dict(layout=2), BAD), (dict(scaling=4), BAD),
    (dict(base=1.0), BAD), (dict(base=NAN), BAD), (dict(base=INF), BAD), (dict(dtype=-1), BAD),
    (dict(scaling=1), BAD), (dict(scaling=1, factor=NAN), BAD), (dict(scaling=2, factor=INF), BAD),
    (dict(scaling=2, factor=2.0, rotary_dim=2), BAD),
    (dict(scaling=3, factor=2.0), BAD),
    (dict(scaling=3, factor=2.0, original=64.0, fast=1.0, slow=1.0), BAD),
    (dict(scaling=3, factor=2.0, original=64.0, fast=INF, slow=1.0), BAD),
    (dict(dim=1025), UNS), (dict(dim=512, rotary_dim=258), UNS), (dict(length=1 << 40), UNS),
])
def test_rotary_plan_rejects(kw, code):
    st, h = capi.fno_rotary_plan(rotary_desc(**kw))
    assert st == code and not h


@pytest.mark.parametrize("args,code", [
    ((0, 5, 6, 3, 1, 0), BAD), ((1, 0, 6, 3, 1, 0), BAD), ((1, 5, 0, 3, 1, 0), BAD),
    ((1, 5, 6, 1, 1, 0), BAD), ((1, 5, 6, 3, 2, 0), BAD), ((1, 5, 6, 3, 1, 7), BAD),
    ((1, 5, 6, 3, 1, 0, 2), BAD), ((1, 5, 6, 9, 1, 0), UNS), ((1, 1 << 40, 6, 3, 1, 0), UNS),
    ((1 << 36, 5, 6, 3, 1, 0), UNS),
])
def test_conv_plan_rejects(args, code):
    st, h = capi.fno_causal_conv_plan(*args)
    assert st == code and not h


def test_null_arguments(L):
    assert L.fno_scan_plan(None, None) == BAD and L.fno_rotary_plan(None, None) == BAD
    h = ctypes.c_void_p(0)
    assert L.fno_scan_plan(ctypes.byref(h), None) == BAD
    assert L.fno_rotary_plan(ctypes.byref(h), None) == BAD
    assert capi.fno_scan_workspace_size(None)[0] == BAD
    assert capi.fno_causal_conv_workspace_size(None)[0] == BAD
    assert capi.fno_rotary_apply(None, 16, 16, None, None, 0, 16, 16, None) == BAD
    assert capi.fno_causal_conv_forward(None, *[16] * 8) == BAD
    assert capi.fno_causal_conv_backward(None, *[16] * 13) == BAD
    assert capi.fno_causal_conv_step(None, 16, 16, 16, 16, 1, 16, 16, 16, None) == BAD
    assert capi.fno_scan_forward(None, *[16] * 14) == BAD
    assert capi.fno_scan_backward(None, *[16] * 23) == BAD
    assert capi.fno_scan_step(None, *[16] * 9, 1, *[16] * 4) == BAD
    for name in ("scan", "causal_conv", "rotary"):
        assert getattr(capi, f"fno_{name}_destroy")(None) == OK


def test_failed_allocation_is_reported(monkeypatch):
    monkeypatch.setenv("FNO_FAULT_INJECT", "plan_alloc")
    oom = capi.FNO_ERR_OUT_OF_MEMORY
    assert capi.fno_scan_plan(scan_desc()) == (oom, None)
    assert capi.fno_rotary_plan(rotary_desc()) == (oom, None)
    assert capi.fno_causal_conv_plan(1, 5, 6, 3, 1, 0) == (oom, None)


def test_python_classes_check_names_and_ranges():
    import fft_gemm_ifft_gb300 as pkg
    for name in ("Rotary", "CausalConv", "SelectiveScan"):
        assert name in pkg.__all__ and getattr(pkg, name) is not None
    # values that a 32-bit field would wrap
    for kw in (dict(channels=2 ** 32 + 4), dict(states=2 ** 32 + 4), dict(groups=-2 ** 32 + 1)):
        with pytest.raises(ValueError):
            pkg.SelectiveScan(**{**dict(batch=1, length=1, channels=4, states=4), **kw})
    with pytest.raises(ValueError):
        pkg.CausalConv(1, 1, 4, 3, act="gelu")
    with pytest.raises(ValueError):
        pkg.Rotary(1, 1, 1, 1, 8, scaling=("ramp", 2.0))
    with pytest.raises(ValueError):
        pkg.Rotary(1, 1, 1, 1, 8, dtype="f64")
