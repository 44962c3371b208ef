"""Refusals of the 8-bit decoder step's calls, on the host: nothing is launched or read
(the pointers are made up), in the order that include/w4.h documents."""
import pytest

P = 0x10000   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from w4a16_int4_quantized_gb300 import build
    build.build()
    from w4a16_int4_quantized_gb300 import ops
    return ops


def test_norm(lib):
    def f(T=4, H=64, ld=64, x=P, xt=1, res=P, out=P, rt=1, w=P, q=P, sx=P, y=P, yt=0):
        return lib.raw.w4_add_rmsnorm_q8(x, xt, ld, res, out, rt, w, 1e-6, T, H, q, sx, y, yt, None)

    for kw in (dict(T=-1), dict(H=-1), dict(xt=3), dict(rt=-1), dict(yt=9), dict(ld=63), dict(x=None), dict(w=None),
               dict(q=None), dict(sx=None), dict(res=None), dict(out=None), dict(x=P + 1), dict(res=P + 1), dict(out=P + 1),
               dict(x=P + 2, xt=0), dict(y=P + 2), dict(w=P + 2), dict(sx=P + 1)):
        assert f(**kw) == lib.W4_EINVAL, kw
    for kw in (dict(T=1 << 31), dict(H=1 << 31, ld=1 << 31), dict(ld=1 << 31)):
        assert f(**kw) == lib.W4_ESHAPE, kw
    assert f(T=0, x=None, w=None, q=None) == f(H=0, x=None) == lib.W4_OK


def cache(lib, **kw):
    d = dict(k=P, v=P, k_scale=P, v_scale=P, pages=10, page_size=32, heads=2, head_dim=64, reserved=0,
             page_stride=32 * 2 * 64, token_stride=2 * 64, head_stride=64)
    d.update(kw)
    return lib.Kv8CacheStruct(*(d[n] for n, _ in lib.Kv8CacheStruct._fields_))


CACHE_EINVAL = [dict(pages=-1), dict(page_size=0), dict(heads=0), dict(head_dim=0), dict(reserved=1), dict(head_stride=8),
                dict(token_stride=-64), dict(page_stride=1), dict(k=None), dict(v=None), dict(k_scale=None),
                dict(v_scale=None), dict(k=P + 8), dict(v=P + 8)]
CACHE_ESHAPE = [dict(pages=1 << 31), dict(head_dim=24), dict(head_dim=272), dict(page_size=8), dict(page_size=48)]


def test_struct_layout(lib):
    import ctypes
    assert ctypes.sizeof(lib.Kv8CacheStruct) == lib._KV8_STRUCT.size
    at = {n: getattr(lib.Kv8CacheStruct, n).offset for n, _ in lib.Kv8CacheStruct._fields_}
    assert at["pages"] == 32 and at["page_size"] == 40 and at["reserved"] == 52 and at["page_stride"] == 56


def test_store(lib):
    import ctypes

    def f(T=4, Hq=4, ld=8 * 64, t=0, rot=64, pos=P, cs=P, table=P, ctx=P, cu=P, B=2, width=3, q=P, qt=1, x=P, wq=P, wk=P,
          top=100, **kw):
        c = cache(lib, **kw)
        return lib.raw.w4_qk_norm_rope_kv8(x, t, ld, T, Hq, wq, wk, 1e-6, pos, cs, top, rot, 0, table, width, ctx, cu, B,
                                           ctypes.byref(c), q, qt, None)

    for kw in CACHE_EINVAL:
        assert f(**kw) == lib.W4_EINVAL, kw
    for kw in CACHE_ESHAPE:
        assert f(**kw) == lib.W4_ESHAPE, kw
    for kw in (dict(T=-1), dict(B=-1), dict(width=-1), dict(Hq=0), dict(rot=-16), dict(t=9), dict(qt=0), dict(qt=5),
               dict(ld=8 * 64 - 4), dict(ld=8 * 64 + 2), dict(top=-1), dict(x=None), dict(pos=None), dict(table=None),
               dict(ctx=None), dict(cu=None), dict(q=None), dict(cs=None), dict(x=P + 4), dict(wq=P + 4), dict(wk=P + 8),
               dict(q=P + 2), dict(cs=P + 4)):
        assert f(**kw) == lib.W4_EINVAL, kw
    for kw in (dict(rot=24), dict(rot=80), dict(T=1 << 31), dict(B=1 << 30), dict(width=1 << 31),
               dict(Hq=1 << 30, ld=1 << 40)):
        assert f(**kw) == lib.W4_ESHAPE, kw
    assert f(T=0, x=None, q=None) == f(B=0, ctx=None) == lib.W4_OK
    assert lib.raw.w4_qk_norm_rope_kv8(P, 0, 512, 1, 4, P, P, 1e-6, P, P, 9, 64, 0, P, 3, P, P, 1, None, P, 1,
                                       None) == lib.W4_EINVAL


def test_dequantize(lib):
    import ctypes

    def f(k_out=P, v_out=P, t=1, **kw):
        return lib.raw.w4_dequantize_kv8(ctypes.byref(cache(lib, **kw)), k_out, v_out, t, None)

    for kw in CACHE_EINVAL + [dict(k_out=None), dict(v_out=None), dict(k_out=P + 8), dict(v_out=P + 2), dict(t=4)]:
        assert f(**kw) == lib.W4_EINVAL, kw
    for kw in CACHE_ESHAPE:
        assert f(**kw) == lib.W4_ESHAPE, kw
    assert f(pages=0, k=None, k_out=None) == lib.W4_OK


def test_attention(lib):
    import ctypes

    def f(B=2, T=8, Hq=4, ld=4 * 64, width=3, scale=0.125, max_len=100, max_new=8, window=0, sinks=0, q=P, qt=1, table=P,
          ctx=P, cu=P, out=P, ws=P, wsb=1 << 40, **kw):
        c = cache(lib, **kw)
        return lib.raw.w4_attention_kv8(q, qt, ld, ctypes.byref(c), table, width, ctx, cu, B, T, Hq, scale, max_len,
                                        max_new, window, sinks, out, ws, wsb, None)

    for kw in CACHE_EINVAL + [dict(pages=0)]:
        assert f(**kw) == lib.W4_EINVAL, kw
    for kw in CACHE_ESHAPE + [dict(Hq=3), dict(B=1 << 30), dict(T=1 << 31), dict(width=1 << 31),
                              dict(max_len=(1 << 31) - 1), dict(max_new=1 << 31), dict(window=1 << 31), dict(sinks=1 << 31)]:
        assert f(**kw) == lib.W4_ESHAPE, kw
    for kw in (dict(B=-1), dict(T=-1), dict(Hq=0), dict(width=-1), dict(max_len=-1), dict(max_new=-1), dict(window=-1),
               dict(sinks=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(scale=3e38), dict(qt=0), dict(ld=4 * 64 - 8), dict(ld=4 * 64 + 4), dict(width=0), dict(q=None),
               dict(table=None), dict(ctx=None), dict(cu=None), dict(out=None), dict(q=P + 8), dict(out=P + 2),
               dict(ws=P + 8)):
        assert f(**kw) == lib.W4_EINVAL, kw
    for kw in (dict(B=0), dict(T=0), dict(max_new=0), dict(max_len=0)):
        assert f(q=None, out=None, **kw) == lib.W4_OK, kw
    # parts of a unit go through the workspace: few rows over long contexts, many rows
    for max_len, max_new in ((300000, 8), (10000, 40)):
        need = lib.attention_kv8_workspace_bytes(2, 4, 2, 64, max_len, max_new)
        assert need > 0
        kw = dict(max_len=max_len, max_new=max_new)
        assert f(wsb=need - 1, **kw) == lib.W4_EINVAL and f(ws=None, **kw) == lib.W4_EINVAL


def test_workspace_query(lib):
    f = lib.attention_kv8_workspace_bytes
    huge = (1 << 64) - 1
    assert f(0, 8, 2, 128, 1000, 1) == f(1, 8, 2, 128, 0, 1) == f(1, 8, 2, 128, 1000, 0) == 0
    assert 0 < f(1, 8, 2, 128, 300000, 1) < 64 << 20 and 0 < f(64, 8, 2, 128, 10000, 4096) < 64 << 20
    assert f(1, 8, 2, 128, 300000, 1, 64, 4) == 0     # a window leaves too little to be cut
    for bad in ((-1, 8, 2, 128, 10, 1), (1, 8, 3, 128, 10, 1), (1, 8, 2, 24, 10, 1), (1, 8, 0, 64, 10, 1),
                (1, 8, 2, 512, 10, 1), (1, 8, 2, 128, 10, 1, -1), (1, 8, 2, 128, 10, 1, 0, 1 << 31)):
        assert f(*bad) == huge


def test_work_beyond_32_bits(lib):
    """B * heads * rows of a request (rounded up to 32, above that to 256s) below 2^31, also where the product passes 64 bits."""
    import ctypes
    f, huge = lib.attention_kv8_workspace_bytes, (1 << 64) - 1
    for B, Hq, Hkv, max_new in ((1 << 22, 16, 16, 32), (1 << 28, 8, 1, 4), (1 << 15, 4, 4, 1 << 14),
                                ((1 << 29) - 1, 1 << 19, 1 << 19, 2047), (1, 2, 2, (1 << 30) - 255)):
        assert f(B, Hq, Hkv, 64, 1000, max_new) == huge, (B, Hq, Hkv, max_new)
        st = lib.raw.w4_attention_kv8(P, lib.BF16, Hq * 64, ctypes.byref(cache(lib, heads=Hkv)), P, 4, P, P, B, 6, Hq, 0.1,
                                      1000, max_new, 0, 0, P, P, huge, None)
        assert st == lib.W4_ESHAPE, (B, Hq, Hkv, max_new)
    for B, Hq, Hkv, max_new in (((1 << 22) - 1, 16, 16, 32), ((1 << 15) - 1, 4, 4, 1 << 14), (1, 2, 2, (1 << 30) - 256)):
        assert f(B, Hq, Hkv, 64, 1000, max_new) != huge, (B, Hq, Hkv, max_new)


def test_copies_and_products_are_waited_for():
    from tests.test_pipeline_drain import test_what_was_begun_is_waited_for as check
    check("attn8_tc.cu")


def test_logprobs(lib):
    def f(T=4, V=100, ld=100, t=0, top=5, x=P, ids=P, lp=P, en=P, ti=P, tl=P):
        return lib.raw.w4_token_logprobs(x, t, ld, T, V, ids, top, lp, en, ti, tl, None)

    for kw in (dict(T=-1), dict(V=-1), dict(top=-1), dict(t=3), dict(ld=99), dict(V=0), dict(x=None), dict(ids=None),
               dict(lp=None), dict(en=None), dict(ti=None), dict(tl=None), dict(x=P + 2), dict(x=P + 1, t=1),
               dict(ids=P + 2), dict(lp=P + 1), dict(en=P + 2), dict(ti=P + 2), dict(tl=P + 2)):
        assert f(**kw) == lib.W4_EINVAL, kw
    for kw in (dict(T=1 << 31), dict(V=(1 << 31) - 16, ld=1 << 32), dict(top=33)):
        assert f(**kw) == lib.W4_ESHAPE, kw
    assert f(T=0, x=None, ids=None) == lib.W4_OK


def test_python_checks(lib):
    torch = pytest.importorskip("torch")
    c = lib.Kv8Cache.empty(3, 32, 2, 64, device="cpu")
    assert c.k.shape == (3, 32, 2, 64) and c.k_scale.shape == (3, 2, 2)
    with pytest.raises(ValueError):
        lib.Kv8Cache(c.k, c.v.contiguous(), c.k_scale, c.v_scale)
    with pytest.raises(ValueError):
        lib.Kv8Cache(c.k, c.v, c.k_scale, c.v_scale[:, :, :1])
    with pytest.raises(ValueError):
        lib.Kv8Cache(c.k.float(), c.v.float(), c.k_scale, c.v_scale)
    x, w = torch.zeros((2, 8)), torch.zeros(8)
    for bad in (dict(w=torch.zeros(7)), dict(w=w.double()), dict(residual=torch.zeros((2, 7))),
                dict(residual=torch.zeros((8, 2)).T), dict(residual_out=x),
                dict(residual=x, residual_out=torch.zeros((2, 8), dtype=torch.float16)), dict(x=torch.zeros((8, 2)).T)):
        with pytest.raises(ValueError):
            lib.add_rmsnorm_q8(**{"x": x, "residual": None, "w": w, **bad})
    i32 = torch.int32
    q, table, ctx, cu = torch.zeros((2, 4, 64), dtype=torch.bfloat16), torch.zeros((1, 4), dtype=i32), torch.zeros(1, dtype=i32), torch.zeros(2, dtype=i32)
    for bad in (dict(q=q[..., :32]), dict(q=q.transpose(0, 1)), dict(block_table=table.long()), dict(ctx_len=ctx[:0]),
                dict(cu_new=cu[:1]), dict(out=q.half()), dict(out=q[:1])):
        with pytest.raises(ValueError):
            lib.attention_kv8(**{"q": q, "cache": c, "block_table": table, "ctx_len": ctx, "cu_new": cu, "scale": 1.0,
                                 "max_len": 8, "max_new": 1, **bad})
    for bad in ((torch.zeros((4, 2)).T, torch.zeros(2, dtype=i32)), (torch.zeros((2, 4)), torch.zeros(2)),
                (torch.zeros((2, 4)), torch.zeros(3, dtype=i32))):
        with pytest.raises(ValueError):
            lib.token_logprobs(*bad)
