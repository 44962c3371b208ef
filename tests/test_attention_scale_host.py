"""Scales that w4_tree_attention cannot apply in f32 are refused, on the host (made-up pointers, nothing is launched)."""
import ctypes as C

import pytest

P = 0x10000


@pytest.mark.parametrize("scale", [2.4e38, 3.4e38, float("inf"), float("nan"), 0.0, -1.0])
def test_scale_is_refused(scale):
    from w4a16_int4_quantized_gb300 import build
    build.build()
    from w4a16_int4_quantized_gb300 import ops
    c = ops.PagedCache(P, P, 10, 16, 2, 64, ops.BF16, 2048, 128, 64)

    def call(s, wsb):
        return ops.raw.w4_tree_attention(P, 256, C.byref(c), P, 3, P, P, P, 2, 8, 4, s, 100, 8, P, P, wsb, None)

    assert call(scale, 1 << 40) == ops.W4_EINVAL
    # the largest that is applied gets as far as the check of its other sizes
    c.page_size = 4
    assert call(2.3e38, 1 << 40) == ops.W4_ESHAPE
    c.page_size = 16
    assert ops.raw.w4_tree_attention(None, 256, C.byref(c), None, 3, None, None, None, 0, 8, 4, 2.3e38, 100, 8, None, None,
                                     0, None) == ops.W4_OK
