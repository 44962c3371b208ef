"""Sizes that the 8-bit cache's store and read-back refuse by their shape, on the host: a launch of them would not
fit 32 bits.  What is accepted is seen by the refusal that comes next, of a NULL pointer: nothing is launched."""
import ctypes

import pytest

from tests.test_step8_host import P, cache, lib  # noqa: F401


def store(lib, T=4, B=2, Hq=4, **kw):  # noqa: F811
    c = cache(lib, **kw)
    ld = (Hq + 2 * c.heads) * c.head_dim
    return lib.raw.w4_qk_norm_rope_kv8(None, 0, ld, T, Hq, P, P, 1e-6, P, None, 100, 0, 0, P, 3, P, P, B,
                                       ctypes.byref(c), P, 1, None)


@pytest.mark.parametrize("kw,fits", [
    # blocks of keys and values: (T / 16 + 2 B) heads
    (dict(heads=1 << 19, head_dim=16, B=1024), False), (dict(heads=1 << 19, head_dim=16, B=1000), True),
    (dict(heads=1 << 19, head_dim=16, T=1 << 15, B=1), False), (dict(heads=1 << 19, head_dim=16, T=1 << 14, B=1), True),
    ((dict(T=(1 << 31) - 1, B=(1 << 29) - 1, heads=1 << 19, head_dim=16)), False),
    # warps of queries: 128 heads of 64 are 8 to a token
    (dict(T=(1 << 31) - 1, Hq=128), False), (dict(T=1 << 28, Hq=128, heads=1), True),
    (dict(T=(1 << 29) - 64, Hq=128, heads=1), False),
    # as heads of 48 are, whose lanes are rounded up
    (dict(T=(1 << 29) - 64, Hq=128, heads=1, head_dim=48), False), (dict(T=1 << 28, Hq=128, heads=1, head_dim=48), True),
    (dict(T=0, B=1 << 28, heads=1 << 19, head_dim=16), None), (dict(T=1 << 30, B=0, heads=1 << 19, head_dim=16), None)])
def test_store(lib, kw, fits):  # noqa: F811
    assert store(lib, **kw) == {True: lib.W4_EINVAL, False: lib.W4_ESHAPE, None: lib.W4_OK}[fits], kw


@pytest.mark.parametrize("kw,fits", [
    (dict(page_size=1 << 20, heads=1 << 8, head_dim=128), False), (dict(page_size=1 << 20, heads=1 << 7, head_dim=128, pages=1), True),
    (dict(page_size=1 << 20, heads=1 << 7, head_dim=128, pages=1 << 11), False),
    (dict(page_size=1 << 20, heads=1 << 7, head_dim=128, pages=(1 << 11) - 1), True),
    (dict(page_size=16, heads=1, head_dim=16, pages=(1 << 31) - 1), True),
    (dict(page_size=32, heads=3, head_dim=256, pages=(1 << 30) - 1), True),      # 1,536 chunks: two CTAs a page
    (dict(page_size=32, heads=3, head_dim=256, pages=(1 << 30)), False),
    (dict(page_size=1 << 30, heads=(1 << 20) - 1, head_dim=256, pages=(1 << 31) - 1), False),
    (dict(page_size=1 << 30, heads=(1 << 20) - 1, head_dim=256, pages=0), None)])
def test_read_back(lib, kw, fits):  # noqa: F811
    got = lib.raw.w4_dequantize_kv8(ctypes.byref(cache(lib, **kw)), None, P, 1, None)
    assert got == {True: lib.W4_EINVAL, False: lib.W4_ESHAPE, None: lib.W4_OK}[fits], kw
