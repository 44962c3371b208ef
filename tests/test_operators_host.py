"""Refusals of the MXFP4 and drafted-token calls, on the host: nothing is launched
or read (the pointers are made up), in the order that include/w4.h documents."""
import ctypes as C

import pytest

P = 0x10000   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from w4a16_int4_quantized_gb300 import build
    build.build()
    from w4a16_int4_quantized_gb300 import ops
    return ops


def test_mxfp4_quantizers(lib):
    r = lib.raw
    for f, a in ((r.w4_quantize_mxfp4, lambda R, K, x=P, t=0, c=P, s=P: (x, t, R, K, c, s, None)),
                 (r.w4_dequantize_mxfp4, lambda R, K, x=P, t=0, c=P, s=P: (c, s, R, K, x, t, None))):
        assert f(*a(-1, 4)) == lib.W4_EINVAL and f(*a(4, -1)) == lib.W4_EINVAL
        assert f(*a(4, 4, t=3)) == lib.W4_EINVAL and f(*a(4, 4, t=-1)) == lib.W4_EINVAL
        assert f(*a(1 << 31, 4)) == lib.W4_ESHAPE and f(*a(4, 1 << 31)) == lib.W4_ESHAPE
        assert f(*a(0, 4, x=None, c=None, s=None)) == lib.W4_OK and f(*a(4, 0, x=None)) == lib.W4_OK
        for missing in ("x", "c", "s"):
            assert f(*a(4, 4, **{missing: None})) == lib.W4_EINVAL
        assert f(*a(4, 4, c=P + 8)) == lib.W4_EINVAL
        assert f(*a(4, 4, x=P + 2)) == lib.W4_EINVAL and f(*a(4, 4, x=P + 1, t=1)) == lib.W4_EINVAL


def test_mxfp4_linears(lib):
    r = lib.raw

    def a16(M, N, K, x=P, w=P, s=P, y=P, t=0, fl=0):
        return r.w4_linear_mxfp4(x, w, s, y, t, M, N, K, fl, None)

    def a4(M, N, K, x=P, w=P, s=P, y=P, t=0, fl=0, sx=P):
        return r.w4_linear_mxfp4_a4(x, sx, w, s, y, t, M, N, K, fl, None)

    for f in (a16, a4):
        for dims in ((-1, 1, 1), (1, -1, 1), (1, 1, -1)):
            assert f(*dims) == lib.W4_EINVAL
        assert f(1, 1, 1, t=5) == lib.W4_EINVAL and f(1, 1, 1, fl=2) == lib.W4_EINVAL
        for dims in ((1 << 31, 1, 1), (1, 1 << 31, 1), (1, 1, 1 << 31)):
            assert f(*dims) == lib.W4_ESHAPE
        assert f(0, 4, 4, x=None, w=None, s=None, y=None) == lib.W4_OK
        assert f(4, 0, 4, x=None, w=None, s=None, y=None) == lib.W4_OK
        for missing in ("x", "w", "s", "y"):
            assert f(4, 4, 4, **{missing: None}) == lib.W4_EINVAL
        assert f(4, 4, 4, w=P + 8) == lib.W4_EINVAL and f(4, 4, 4, x=P + 8) == lib.W4_EINVAL
        assert f(4, 4, 4, y=P + 2) == lib.W4_EINVAL
    assert a4(4, 4, 4, sx=None) == lib.W4_EINVAL


def test_plan(lib):
    r = lib.raw

    def f(B=2, width=4, n_free=3, page=16, cap=8, ctx=P, new=P, par=None, free=P, table=P, cu=P, slots=P, pos=P, mask=P,
          taken=P):
        return r.w4_draft_plan(ctx, new, par, free, n_free, table, B, width, page, cap, cu, slots, pos, mask, taken, None)

    for bad in (dict(B=-1), dict(width=-1), dict(n_free=-1), dict(cap=-1), dict(page=0)):
        assert f(**bad) == lib.W4_EINVAL
    for bad in (dict(B=1 << 24), dict(width=1 << 31), dict(cap=1 << 31)):
        assert f(**bad) == lib.W4_ESHAPE
    for name in ("ctx", "new", "free", "table", "cu", "slots", "pos", "mask", "taken"):
        assert f(**{name: None}) == lib.W4_EINVAL
    assert f(mask=P + 4) == lib.W4_EINVAL


def cache(lib, **kw):
    d = dict(k=P, v=P, pages=10, page_size=16, heads=2, head_dim=64, type=lib.BF16, page_stride=16 * 2 * 64,
             token_stride=2 * 64, head_stride=64)
    d.update(kw)
    return lib.PagedCache(*(d[n] for n, _ in lib.PagedCache._fields_))


CACHE_EINVAL = [dict(type=7), dict(pages=-1), dict(page_size=0), dict(heads=0), dict(head_dim=0), dict(head_stride=4),
                dict(token_stride=-64), dict(page_stride=1), dict(k=None), dict(v=None), dict(k=P + 8)]
CACHE_ESHAPE = [dict(pages=1 << 31), dict(head_dim=12), dict(head_dim=264)]


def test_rope(lib):
    r = lib.raw

    def f(T=4, Hq=4, ld=8 * 64, t=0, rot=64, pos=P, cs=P, slots=P, q=P, x=P, wq=P, wk=P, top=100, **kw):
        c = cache(lib, **kw)
        return r.w4_qk_norm_rope(x, t, ld, T, Hq, wq, wk, 1e-6, pos, cs, top, rot, 0, slots, C.byref(c), q, None)

    for kw in CACHE_EINVAL:
        assert f(**kw) == lib.W4_EINVAL, kw
    for kw in CACHE_ESHAPE:
        assert f(**kw) == lib.W4_ESHAPE, kw
    for kw in (dict(T=-1), dict(Hq=0), dict(rot=-16), dict(t=9), dict(ld=8 * 64 - 4), dict(ld=8 * 64 + 2), dict(top=-1),
               dict(x=None), dict(pos=None), dict(slots=None), dict(q=None), dict(cs=None), dict(x=P + 4), dict(wq=P + 4),
               dict(wk=P + 8), dict(q=P + 2), dict(cs=P + 4)):
        assert f(**kw) == lib.W4_EINVAL, kw
    for kw in (dict(rot=24), dict(rot=80), dict(T=1 << 31), dict(Hq=1 << 30, ld=1 << 40)):
        assert f(**kw) == lib.W4_ESHAPE, kw
    assert f(T=0, x=None, q=None) == lib.W4_OK
    assert r.w4_qk_norm_rope(P, 0, 512, 1, 4, P, P, 1e-6, P, P, 9, 64, 0, P, None, P, None) == lib.W4_EINVAL


def test_tree_attention(lib):
    r = lib.raw

    def f(B=2, T=8, Hq=4, ld=4 * 64, width=3, scale=0.125, max_len=100, max_new=8, q=P, table=P, ctx=P, cu=P, mask=P,
          out=P, ws=P, wsb=1 << 40, **kw):
        c = cache(lib, **kw)
        return r.w4_tree_attention(q, ld, C.byref(c), table, width, ctx, cu, mask, B, T, Hq, scale, max_len, max_new, out,
                                   ws, wsb, None)

    for kw in CACHE_EINVAL + [dict(type=0), dict(pages=0)]:
        assert f(**kw) == lib.W4_EINVAL, kw
    for kw in CACHE_ESHAPE + [dict(page_size=4), dict(page_size=24), dict(Hq=3), dict(Hq=512, ld=512 * 64),
                              dict(B=1 << 24), dict(T=1 << 31), dict(width=1 << 31), dict(max_len=(1 << 31) - 1)]:
        assert f(**kw) == lib.W4_ESHAPE, kw
    for kw in (dict(B=-1), dict(T=-1), dict(Hq=0), dict(width=-1), dict(max_len=-1), dict(max_new=-1), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(ld=4 * 64 - 8),
               dict(ld=4 * 64 + 4), dict(width=0), dict(q=None), dict(table=None), dict(ctx=None), dict(cu=None),
               dict(mask=None), dict(out=None), dict(q=P + 8), dict(mask=P + 4), dict(out=P + 2), dict(ws=P + 8)):
        assert f(**kw) == lib.W4_EINVAL, kw
    for kw in (dict(B=0), dict(T=0), dict(max_new=0), dict(max_len=0)):
        assert f(q=None, out=None, **kw) == lib.W4_OK, kw
    # parts of a unit go through the workspace
    need = lib.tree_attention_workspace_bytes(2, 4, 2, 64, 10000, 8)
    assert need > 0
    assert f(max_len=10000, wsb=need - 1) == lib.W4_EINVAL and f(max_len=10000, ws=None) == lib.W4_EINVAL


def test_workspace_query(lib):
    f = lib.tree_attention_workspace_bytes
    huge = (1 << 64) - 1
    assert f(0, 8, 2, 128, 1000, 1) == f(1, 8, 2, 128, 0, 1) == f(1, 8, 2, 128, 1000, 0) == 0
    assert 0 < f(1, 8, 2, 128, 60, 1) < f(64, 8, 2, 128, 10000, 1) < 64 << 20
    for bad in ((-1, 8, 2, 128, 10, 1), (1, 8, 3, 128, 10, 1), (1, 8, 2, 12, 10, 1), (1, 8, 0, 64, 10, 1),
                (1, 8, 2, 512, 10, 1), (1, 512, 2, 64, 10, 1)):
        assert f(*bad) == huge


def test_python_checks(lib):
    torch = pytest.importorskip("torch")
    k = torch.zeros((2, 16, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lib.paged_cache(k, k.transpose(1, 2))
    with pytest.raises(ValueError):
        lib.paged_cache(k, k.half())
    with pytest.raises(ValueError):
        lib.paged_cache(k.transpose(2, 3), k.transpose(2, 3))
    c = lib.paged_cache(k.transpose(1, 2).contiguous().transpose(1, 2), k.transpose(1, 2).contiguous().transpose(1, 2))
    assert (c.pages, c.page_size, c.heads, c.head_dim) == (2, 16, 2, 64)
    assert (c.page_stride, c.token_stride, c.head_stride) == (2048, 64, 1024)
    codes, scales = torch.zeros((3, 32), dtype=torch.uint8), torch.zeros((3, 2), dtype=torch.uint8)
    for K in (32, 65):
        with pytest.raises(ValueError):
            lib.dequantize_mxfp4(codes, scales, K)
    for bad in (torch.zeros((3, 63)), torch.zeros((64, 3)).T):
        with pytest.raises(ValueError):
            lib.dequantize_mxfp4(codes, scales, 64, out=bad)
