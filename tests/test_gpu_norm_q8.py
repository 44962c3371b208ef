"""w4_add_rmsnorm_q8 against its formula in 64 bits.

The residual is the rounded sum, bit for bit.  y: the sum of squares runs over at most
8 * 33 values of a thread in pairs and 10 more sums over the CTA, 2^-24 each (its root halves
that), the reciprocal root 2 steps of 2^-23, the two products 2^-24 each: 2^-17 covers it.
Codes and scale are those of quantize_row_q8 for the f32 y, bit for bit."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_int4_quantized_gb300 import build
    build.build()
    from w4a16_int4_quantized_gb300 import ops
    return ops


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def check(ops, x, res, w, q, sx, h, y, eps=1e-6):
    if res is None:
        assert h is None
        hd = x.double()
    else:
        assert torch.equal(h, (x.float() + res.float()).to(res.dtype))
        hd = h.double()
    want = hd / torch.sqrt((hd * hd).mean(-1, keepdim=True) + eps) * w.double()
    assert ((y.double() - want).abs() <= (2.0 ** -17 + U[y.dtype]) * want.abs() + 1e-37).all()
    if y.dtype == F32:
        q2, sx2, _ = ops.quantize_row_q8(y)
        assert torch.equal(q, q2) and torch.equal(sx, sx2)


@pytest.mark.parametrize("T,H", [(1, 1), (1, 2048), (3, 7), (13, 5121), (2, 8), (5, 100), (151, 264), (153, 8192), (2, 16384),
                                 (3, 40008), (2, 40007), (300, 1024)])
@pytest.mark.parametrize("xt,rt", [(F32, BF16), (BF16, BF16), (F16, F32), (BF16, None), (F32, F16), (F32, F32)])
def test_formula(ops, T, H, xt, rt):
    x, w = randn((T, H), xt, 1), randn((H,), F32, 2)
    res = None if rt is None else randn((T, H), rt, 3, 3.0)
    check(ops, x, res, w, *ops.add_rmsnorm_q8(x, res, w, out_dtype=F32))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_strides_and_places(ops, dtype):
    # rows of another stride, odd starts, each output type, the residual in place
    T, H = 9, 264
    wide = randn((T, H + 21), dtype, 4)
    res, w = randn((T, H), BF16, 5), randn((H,), F32, 6)
    for start in (0, 1, 8):
        x = wide[:, start: start + H]
        q, sx, h, y = ops.add_rmsnorm_q8(x, res, w, out_dtype=F32)
        check(ops, x, res, w, q, sx, h, y)
        for t in (BF16, F16):
            q2, sx2, h2, y2 = ops.add_rmsnorm_q8(x, res, w, out_dtype=t)
            assert torch.equal(q, q2) and torch.equal(sx, sx2) and torch.equal(h, h2) and torch.equal(y2, y.to(t))
        place = res.clone()
        q3, sx3, h3, y3 = ops.add_rmsnorm_q8(x, place, w, residual_out=place)
        assert h3 is place and y3 is None and torch.equal(place, h) and torch.equal(q3, q) and torch.equal(sx3, sx)


def test_long_rows_in_place(ops):
    T, H = 2, 70000   # beyond what the threads hold: the new residual is read again
    for H in (70000, 70001):
        x, res, w = randn((T, H), BF16, 7), randn((T, H), F16, 8), randn((H,), F32, 9)
        want = ops.add_rmsnorm_q8(x, res, w, out_dtype=F32)
        place = res.clone()
        got = ops.add_rmsnorm_q8(x, place, w, out_dtype=F32, residual_out=place)
        for a, b in zip(want, got):
            assert torch.equal(a, b)
        assert ((got[3].double() / (place.double() / (place.double() ** 2).mean(-1, keepdim=True).add(1e-6).sqrt()
                                    * w.double()) - 1).abs().nan_to_num(0.0) <= 2.0 ** -16).all()


def test_zeros_and_not_finite(ops):
    H = 512
    x, w = randn((6, H), F32, 10), torch.ones(H, device="cuda")
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    x[3] = 3e38      # its squares are beyond f32
    x[4] *= 1e-30    # eps decides
    q, sx, _, y = ops.add_rmsnorm_q8(x, None, w, out_dtype=F32)
    assert sx[0] == 0 and (q[0] == 0).all() and (y[0] == 0).all()
    assert sx[1:4].isnan().all() and (q[1:4] == 0).all()
    check(ops, x[4:], None, w, q[4:], sx[4:], None, y[4:])
    w[3] = float("nan")
    q, sx, _, _ = ops.add_rmsnorm_q8(x, None, w)
    assert sx.isnan().all() and (q == 0).all()
    q, sx, _, _ = ops.add_rmsnorm_q8(x[:0], None, w)
    assert q.shape == (0, H)


def test_other_stream_and_graph(ops):
    x, res, w = randn((4, 2048), BF16, 11), randn((4, 2048), BF16, 12), randn((2048,), F32, 13)
    want = ops.add_rmsnorm_q8(x, res, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ops.add_rmsnorm_q8(x, res, w, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want[:3], got[:3]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = ops.add_rmsnorm_q8(x, res, w)
    x.copy_(randn((4, 2048), BF16, 14))
    g.replay()
    want = ops.add_rmsnorm_q8(x, res, w)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want[:3], got[:3]))
