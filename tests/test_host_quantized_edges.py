"""More of the quantised cache's and the logits' argument checks through the C
ABI, with no GPU work: every call here is refused before anything is launched."""
import ctypes

import pytest

from huffman_decode_df11_amd import _lib
from test_host_quantized import ARG, PTR, _attend, _cache


@pytest.mark.parametrize("scale", [1e38, 3e38, -1e38])
def test_scales_that_would_leave_float32_are_refused(scale):
    L, c, a = _lib.lib(), _cache(), _attend(scale=scale)
    assert L.df11_quantized_attention(ctypes.byref(c), ctypes.byref(a), PTR, 1 << 40, None) == ARG
    assert b"scale" in L.df11_last_error()
