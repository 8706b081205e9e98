"""C-ABI checks of the attention's arguments at their limits that need no GPU:
refused on the host before any launch."""
import ctypes

import pytest

from mxfp4_precision_numerics_amd import mx
from test_abi_cache import FAKE, SHAPE, cache, caller


@pytest.fixture(scope="module")
def L():
    return mx.lib()


def attention(L):
    c = cache()
    call = caller(L.mx_cache_attention, c=ctypes.addressof(c), q=FAKE, qt=mx.MX_BF16, n=3, h=4, ld=0, hl=0, off=None, mq=1,
                  seqs=3, table=FAKE, tld=0, pages=2, len=FAKE, scale=0.125, causal=1, window=0, sinks=None, out=FAKE,
                  old=0, ohl=0, lse=None, ws=FAKE, s=None)
    call.cache = c
    return call


@pytest.mark.parametrize("scale", [2.0 ** 127 * (1 + 2.0 ** -23), 2.4e38, 3.4e38])
def test_scales_whose_exponent_passes_fp32_are_refused(L, scale):
    """Times log2 e they are infinite: a score of 0 would be NaN."""
    assert attention(L)(n=0, seqs=0, scale=scale) == SHAPE


def test_the_largest_scale_is_not_refused(L):
    assert attention(L)(n=0, seqs=0, scale=2.0 ** 127) == 0
