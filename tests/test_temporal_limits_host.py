"""What the plans of convolution, scan and rotary positions refuse at the ends of their sizes;
no GPU is needed: descriptions are checked before any CUDA call."""
import pytest

from fft_gemm_ifft_gb300 import capi
from test_temporal_ops_host import BAD, UNS, rotary_desc, scan_desc


@pytest.fixture(scope="module", autouse=True)
def L():
    from fft_gemm_ifft_gb300 import build
    build.build()
    return capi.lib()


@pytest.mark.parametrize("channels", [2 ** 31 - 2, 2 ** 31 - 1, 2 ** 31 - 256])
def test_scan_channels_whose_blocks_end_behind_31_bits(channels):
    """A block's last channel, of up to 256, has to be a 32-bit number."""
    st, h = capi.fno_scan_plan(scan_desc(batch=1, length=1, channels=channels, states=1, groups=1))
    assert st == UNS and not h


@pytest.mark.parametrize("kw", [dict(base=1e300, factor=1e6, rotary_dim=4),
                                dict(base=1e308, factor=2.0, rotary_dim=8),
                                dict(base=1e4, factor=1e200, rotary_dim=4)])
def test_rotary_base_beyond_float64(kw):
    """base factor^(rotary_dim / (rotary_dim - 2)) that is infinite: every pair but the first
    would stand still."""
    st, h = capi.fno_rotary_plan(rotary_desc(scaling=2, **kw))
    assert st == BAD and not h
