"""Argument checks of the sequence operators' C ABI; no GPU is needed: every
description is checked before any CUDA call."""
import ctypes

import pytest

from fft_gemm_ifft_gb300 import capi

BAD, UNS, OK = capi.FNO_ERR_INVALID_ARG, capi.FNO_ERR_UNSUPPORTED, capi.FNO_OK


@pytest.fixture(scope="module", autouse=True)
def L():
    from fft_gemm_ifft_gb300 import build
    build.build()
    return capi.lib()


def desc(**kw):
    d = capi.fno_sandwich_desc_t()
    v = dict(batch=2, points=5, channels=7, layout=0, norm=0, gate=0, gate_sigmoid=0, eps=1e-5,
             dtype=0)
    v.update(kw)
    for name, x in v.items():
        setattr(d, name, x)
    return d


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), BAD), (dict(points=0), BAD), (dict(channels=0), BAD), (dict(batch=-1), BAD),
    (dict(layout=2), BAD), (dict(norm=2), BAD), (dict(gate=3), BAD), (dict(dtype=3), BAD),
    (dict(eps=-1e-6), BAD), (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD),
    (dict(channels=65537), UNS), (dict(points=1 << 41), UNS), (dict(gate=1, batch=65536), UNS),
])
def test_sandwich_plan_rejects(kw, code):
    st, h = capi.fno_sandwich_plan(desc(**kw))
    assert st == code and not h


def test_sandwich_null_arguments(L):
    assert L.fno_sandwich_plan(None, None) == BAD
    h = ctypes.c_void_p(0)
    assert L.fno_sandwich_plan(ctypes.byref(h), None) == BAD
    assert capi.fno_sandwich_workspace_size(None)[0] == BAD
    assert capi.fno_sandwich_forward(None, *[None] * 13) == BAD
    assert capi.fno_sandwich_backward(None, *[None] * 21) == BAD
    assert capi.fno_sandwich_destroy(None) == OK


@pytest.mark.parametrize("rows,cols,dtype,code", [
    (0, 5, 0, BAD), (5, 0, 0, BAD), (-1, 5, 0, BAD), (5, 5, 3, BAD), (1 << 30, 1 << 30, 0, UNS),
    (5, 5, 0, BAD),                                    # null pointers
])
def test_act8_rejects(rows, cols, dtype, code):
    assert capi.fno_act8_pack(rows, cols, dtype, None, None, None, None) == code
    assert capi.fno_act8_unpack(rows, cols, dtype, None, None, None, None) == code
    assert capi.fno_act8_gelu_backward(rows, cols, dtype, None, None, None, None, None) == code


def test_act8_alignment_and_overlap():
    # addresses are compared, never followed
    A, B, C = 1 << 20, 2 << 20, 3 << 20
    MIS, ALI = capi.FNO_ERR_MISALIGNED, capi.FNO_ERR_ALIASING
    assert capi.fno_act8_pack(4, 100, 0, A + 4, B, C, None) == MIS
    assert capi.fno_act8_pack(4, 100, 0, A, A + 16, C, None) == ALI
    assert capi.fno_act8_pack(4, 100, 0, A, B, B + 384, None) == ALI
    assert capi.fno_act8_unpack(4, 100, 0, A, B, A, None) == ALI
    # dx may be dy, but not a part of it
    assert capi.fno_act8_gelu_backward(4, 100, 0, A, B, C, C + 16, None) == ALI


@pytest.mark.parametrize("args,code", [
    ((0, 3, 3, 10, 0), BAD), ((1, 0, 3, 10, 0), BAD), ((1, 3, 0, 10, 0), BAD),
    ((1, 3, 3, 0, 0), BAD), ((1, 3, 3, 10, 7), BAD), ((1, 4097, 3, 10, 0), UNS),
    ((1, 3, 4097, 10, 0), UNS), ((1 << 20, 64, 64, 1 << 20, 0), UNS),
])
def test_linear_grad_plan_rejects(args, code):
    st, h = capi.fno_linear_grad_plan(*args)
    assert st == code and not h


@pytest.mark.parametrize("args,code", [
    ((0, 5, 2, 1, 8, 8, 0), BAD), ((1, 0, 2, 1, 8, 8, 0), BAD), ((1, 5, 0, 1, 8, 8, 0), BAD),
    ((1, 5, 2, 0, 8, 8, 0), BAD), ((1, 5, 3, 2, 8, 8, 0), BAD), ((1, 5, 2, 4, 8, 8, 0), BAD),
    ((1, 5, 2, 1, 0, 8, 0), BAD), ((1, 5, 2, 1, 8, 0, 0), BAD), ((1, 5, 2, 1, 8, 8, 5), BAD),
    ((1, 5, 2, 1, 257, 8, 0), UNS), ((1, 5, 2, 1, 8, 257, 0), UNS),
    ((1, 1 << 40, 2, 1, 8, 8, 0), UNS),
])
def test_linattn_plan_rejects(args, code):
    st, h = capi.fno_linattn_plan(*args)
    assert st == code and not h
    assert capi.fno_linattn_plan(1, 5, 2, 1, 8, 8, 0, flags=2)[0] == BAD


def test_null_handles():
    assert capi.fno_linear_grad_destroy(None) == OK and capi.fno_linattn_destroy(None) == OK
    assert capi.fno_linear_grad(None, 16, 16, 16, 16, 16, 16, None) == BAD
    assert capi.fno_linear_grad_workspace_size(None)[0] == BAD
    assert capi.fno_linear_grad_get_device_error(None, None) == BAD
    assert capi.fno_linattn_workspace_size(None)[0] == BAD
    assert capi.fno_linattn_get_device_error(None, None) == BAD
    assert capi.fno_linattn_forward(None, 16, 16, 16, 16, 1.0, *[None] * 6) == BAD
    assert capi.fno_linattn_backward(None, 16, 16, 16, 16, 1.0, *[None] * 10) == BAD
    assert capi.fno_linattn_step(None, 16, 16, 16, 16, 1.0, None, 1, 16, 16, 16, None) == BAD


def test_failed_allocation_is_reported(monkeypatch):
    monkeypatch.setenv("FNO_FAULT_INJECT", "plan_alloc")
    oom = capi.FNO_ERR_OUT_OF_MEMORY
    assert capi.fno_sandwich_plan(desc()) == (oom, None)
    assert capi.fno_linear_grad_plan(1, 3, 3, 10, 0) == (oom, None)
    assert capi.fno_linattn_plan(1, 5, 2, 1, 8, 8, 0) == (oom, None)


def test_failed_launch_is_reported(monkeypatch):
    monkeypatch.setenv("FNO_FAULT_INJECT", "launch")
    A, B, C = 1 << 20, 2 << 20, 3 << 20
    assert capi.fno_act8_pack(4, 100, 0, A, B, C, None) == capi.FNO_ERR_CUDA
    assert capi.fno_act8_gelu_backward(4, 100, 0, A, B, C, C, None) == capi.FNO_ERR_CUDA


def test_python_classes_are_reachable():
    import fft_gemm_ifft_gb300 as pkg
    for name in ("SandwichNorm", "PackedActivation", "pack_activation", "LinearGrad",
                 "LinearAttention"):
        assert name in pkg.__all__ and getattr(pkg, name) is not None
    with pytest.raises(AttributeError):
        pkg.NoSuchOperator
