"""Argument checks of the sequence operators that need no GPU."""
import pytest

from fft_gemm_ifft_gb300 import capi


@pytest.fixture(scope="module", autouse=True)
def L():
    from fft_gemm_ifft_gb300 import build
    build.build()
    return capi.lib()


def test_an_update_in_place_has_one_input(monkeypatch):
    # dx may be dy, but not when another input lies there too (addresses are compared,
    # never followed; the launch is made to fail)
    monkeypatch.setenv("FNO_FAULT_INJECT", "launch")
    A, B, C = 1 << 20, 2 << 20, 3 << 20
    call = capi.fno_act8_gelu_backward
    assert call(4, 100, 0, A, B, C, C, None) == capi.FNO_ERR_CUDA
    assert call(4, 100, 0, C, B, C, C, None) == capi.FNO_ERR_ALIASING
    assert call(4, 100, 0, A, C, C, C, None) == capi.FNO_ERR_ALIASING
