"""GPU tests of microscaled 4-bit floating point against plain definitions in 64 bits.

Quantizer: bit-exact.  Products: the operands' values are exact, so
|y - y_exact| <= 1e-5 * sum_k |x_k W_nk| (f32 accumulation in any order, 2^-17
of the sum of magnitudes) + u |y| for the rounding to the output type (u =
2^-24 f32, 2^-8 bf16, 2^-11 f16)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_int4_quantized_gb300 import build
    build.build()
    from w4a16_int4_quantized_gb300 import ops as o
    o.device_status(clear=True)
    return o


def quantize_reference(x):
    """(values [R, nb, 32] f64, scale bytes, codes [R, nb * 16]) by the definition, in numpy."""
    x = x.detach().cpu().double().numpy()
    R, K = x.shape
    nb = -(-K // 32)
    p = np.zeros((R, nb * 32))
    p[:, :K] = x
    p = p.reshape(R, nb, 32)
    top = np.abs(p).max(-1)
    bad = ~np.isfinite(p).all(-1)
    safe = np.where(bad | (top == 0), 1.0, top)
    e = np.maximum(np.floor(np.log2(safe)) - 2, -127)
    # floor(log2) by the exact exponent (log2 may round up just below a power of two)
    e = np.maximum(np.frexp(safe)[1] - 1 - 2, -127).astype(np.int64)
    e = np.where(top == 0, -127, e)
    a = np.abs(np.where(bad[..., None], 0.0, p)) * np.exp2(-e.astype(np.float64))[..., None]
    grid = np.array(GRID)
    dist = np.abs(a[..., None] - grid)
    best = dist.min(-1, keepdims=True)
    near = dist == best
    even = near & (np.arange(8) % 2 == 0)
    idx = np.where(near.sum(-1) == 2, even.argmax(-1), near.argmax(-1))
    neg = np.signbit(p) & ~bad[..., None]
    code = idx + 8 * neg
    code[bad] = 0
    flat = code.reshape(R, -1)
    codes = (flat[:, 0::2] | (flat[:, 1::2] << 4)).astype(np.uint8)
    s = np.where(bad, 255, e + 127).astype(np.uint8)
    val = np.where(neg, -1.0, 1.0) * grid[idx] * np.exp2(e.astype(np.float64))[..., None]
    val[bad] = np.nan
    return val, s, codes


def values(codes, scales, K):
    """f64 values of packed codes and scale bytes, [R, K]."""
    grid = torch.tensor(GRID + tuple(-g for g in GRID), dtype=torch.float64, device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(1).long()
    return (grid[c] * torch.exp2(scales.double() - 127).repeat_interleave(32, 1))[:, :K]


@pytest.mark.parametrize("R,K", [(1, 1), (1, 31), (3, 32), (5, 33), (7, 2047), (2, 2048), (300, 64), (1, 20000),
                                 (33, 40), (1000, 8), (1300, 2048), (1301, 2044)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_quantize_is_exact(ops, R, K, dtype):
    gen = torch.Generator(device="cuda").manual_seed(R * 31 + K)
    x = torch.randn((R, K), generator=gen, device="cuda")
    x *= torch.exp2(torch.randint(-12, 8, (R, 1), generator=gen, device="cuda").float())
    x = x.to(dtype)
    codes, scales = ops.quantize_mxfp4(x)
    val, s, c = quantize_reference(x)
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), c)
    want = torch.from_numpy(val.reshape(R, -1)[:, :K]).cuda()
    for out in (torch.float32, torch.bfloat16, torch.float16):
        y = ops.dequantize_mxfp4(codes, scales, K, out)
        assert torch.equal(y, want.to(out)), out  # exact in f32 and bf16, rounded once in f16


def test_quantize_ties_and_extremes(ops):
    rows = []
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 7.999, 4.0]
    for scale in (2.0 ** -130, 2.0 ** -126, 1.0, 2.0 ** 100, 2.0 ** 125):
        rows.append([t * scale for t in ties] + [-t * scale for t in ties] + [0.0, -0.0] + [2.0 ** -149] * 10)
    rows.append([0.0] * 32)
    rows.append([-0.0] * 32)
    rows.append([2.0 ** -149] * 32)               # the smallest subnormal alone
    rows.append([3.4028234e38] * 16 + [-1e38] * 16)
    rows.append([float("nan")] + [1.0] * 31)
    rows.append([1.0] * 31 + [float("inf")])
    rows.append([-float("inf")] + [2.0] * 31)
    x = torch.tensor(rows, dtype=torch.float32).cuda()
    codes, scales = ops.quantize_mxfp4(x)
    val, s, c = quantize_reference(x)
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), c)
    y = ops.dequantize_mxfp4(codes, scales, 32).double().cpu().numpy()
    assert np.array_equal(y, val.reshape(len(rows), 32), equal_nan=True)


def test_dequantize_every_code_and_scale(ops):
    """All 16 codes under all 256 scales, exact in f32 and bf16."""
    codes = torch.arange(256, dtype=torch.uint8).view(1, 256).repeat(256, 1)[:, :256].cuda().contiguous()  # 16 blocks of 16 bytes
    scales = torch.arange(256, dtype=torch.uint8).view(256, 1).repeat(1, 16).cuda().contiguous()
    want = values(codes, scales, 512)
    want[255] = float("nan")
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        y = ops.dequantize_mxfp4(codes, scales, 512, dt)
        w = want.to(dt)
        assert bool(((y == w) | (torch.isnan(y) & torch.isnan(w))).all()), dt


@pytest.mark.parametrize("shift", [0, 1, 4, 8])
@pytest.mark.parametrize("R,K", [(3, 40), (5000, 64)])
def test_dequantize_into_a_shifted_buffer(ops, R, K, shift):
    """The widest stores need alignment that a caller's buffer may lack; nothing around it is written."""
    gen = torch.Generator(device="cuda").manual_seed(R + shift)
    codes, scales = ops.quantize_mxfp4(torch.randn((R, K), generator=gen, device="cuda"))
    want = ops.dequantize_mxfp4(codes, scales, K)
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        buf = torch.full((R * K + 16,), -7.0, dtype=dt, device="cuda")
        ops.dequantize_mxfp4(codes, scales, K, dt, out=buf[shift:shift + R * K].view(R, K))
        assert torch.equal(buf[shift:shift + R * K].view(R, K), want.to(dt))
        assert bool((buf[:shift] == -7).all()) and bool((buf[shift + R * K:] == -7).all())


def weights(ops, N, K, seed, spread=6):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randn((N, K), generator=gen, device="cuda")
    w *= torch.exp2(torch.randint(-spread, spread + 1, (N, 1), generator=gen, device="cuda").float()) * 0.02
    return ops.quantize_mxfp4(w)


def check(y, x, w):
    want, size = x @ w.T, x.abs() @ w.abs().T
    tol = 1e-5 * size + U[y.dtype] * want.abs() * 1.01 + (2.0 ** -24 if y.dtype == torch.float16 else 0) + 1e-30
    err = (y.double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


SHAPES = [(1, 1), (16, 32), (100, 31), (257, 2048), (2048, 2080), (33, 4096), (130, 6000), (5000, 96), (9800, 256),
          (700, 2047)]


@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 40])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16, torch.float16])
def test_linear_bf16(ops, M, N, K, out):
    w, sw = weights(ops, N, K, N + K)
    gen = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn((M, K), generator=gen, device="cuda").bfloat16()
    y = ops.linear_mxfp4(x, w, sw, out_dtype=out)
    check(y, x.double(), values(w, sw, K))
    assert torch.equal(ops.linear_mxfp4(x, w, sw, out_dtype=out, flags=ops.FLAG_PDL), y)


@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("M", [1, 3, 9, 16, 17, 64, 65, 128, 129, 300])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16, torch.float16])
def test_linear_4bit(ops, M, N, K, out):
    w, sw = weights(ops, N, K, N + K + 1)
    gen = torch.Generator(device="cuda").manual_seed(M + 5)
    x = torch.randn((M, K), generator=gen, device="cuda")
    x *= torch.exp2(torch.randint(-3, 4, (M, 1), generator=gen, device="cuda").float())
    xq, sx = ops.quantize_mxfp4(x)
    y = ops.linear_mxfp4_a4(xq, sx, w, sw, K, out_dtype=out)
    check(y, values(xq, sx, K), values(w, sw, K))
    assert ops.device_status() == 0


@pytest.mark.parametrize("N,K", [(9, 20011), (130, 12320), (300, 8192), (600, 5000), (2048, 6144), (2048, 13312)])
@pytest.mark.parametrize("M", [1, 8, 13, 16])
def test_few_rows_and_long_sums(ops, M, N, K):
    """The sum over K shared between blocks: any split, large and NaN scales in one block's part alone.

    At most 24 products of 16 columns follow one another in an accumulator, then 8 warps and 8 blocks:
    40 roundings of 2^-23 stay under the 1e-5 of `check` (2048 x 13312: 56 + 10 of them, 8e-6)."""
    w, sw = weights(ops, N, K, N + M)
    sw[N // 2, -3:] = 140  # a factor that takes two steps
    gen = torch.Generator(device="cuda").manual_seed(M + K)
    x = torch.randn((M, K), generator=gen, device="cuda").bfloat16()
    y = ops.linear_mxfp4(x, w, sw)
    check(y, x.double(), values(w, sw, K))
    assert torch.equal(ops.linear_mxfp4(x, w, sw, flags=ops.FLAG_PDL), y)
    xq, sx = ops.quantize_mxfp4(x)
    check(ops.linear_mxfp4_a4(xq, sx, w, sw, K), values(xq, sx, K), values(w, sw, K))
    sw[N // 3, -1] = 255
    for z in (ops.linear_mxfp4(x, w, sw), ops.linear_mxfp4_a4(xq, sx, w, sw, K)):
        assert bool(torch.isnan(z[:, N // 3]).all())
        z[:, N // 3] = 0
        assert bool(torch.isfinite(z).all())


@pytest.mark.parametrize("M", [1, 7, 8, 9, 16])
@pytest.mark.parametrize("N,K", [(9728, 160), (9729, 160), (19457, 96), (20000, 2080)])
def test_linear_4bit_few_rows_of_x_and_many_of_w(ops, M, N, K):
    """Both kernels on either side of the heights of W at which one follows the other."""
    w, sw = weights(ops, N, K, N)
    xq, sx = ops.quantize_mxfp4(torch.randn((M, K), generator=torch.Generator(device="cuda").manual_seed(M),
                                            device="cuda"))
    y = ops.linear_mxfp4_a4(xq, sx, w, sw, K)
    check(y, values(xq, sx, K), values(w, sw, K))
    assert torch.equal(ops.linear_mxfp4_a4(xq, sx, w, sw, K, flags=ops.FLAG_PDL), y)
    assert ops.device_status() == 0


def test_linear_4bit_large(ops):
    """Several tiles a CTA, odd in every direction."""
    M, N, K = 1111, 5003, 1056
    w, sw = weights(ops, N, K, 8)
    xq, sx = ops.quantize_mxfp4(torch.randn((M, K), generator=torch.Generator(device="cuda").manual_seed(9),
                                            device="cuda"))
    y = ops.linear_mxfp4_a4(xq, sx, w, sw, K)
    check(y, values(xq, sx, K), values(w, sw, K))
    assert torch.equal(ops.linear_mxfp4_a4(xq, sx, w, sw, K), y)


@pytest.mark.parametrize("M", [4, 16, 60])
def test_scales_place_by_place(ops, M):
    """One column at a time: each 32 columns under a scale of their own, rows and blocks all different."""
    N, K = 160, 1024
    nb = K // 32
    gen = torch.Generator(device="cuda").manual_seed(3)
    w = torch.randint(0, 256, (N, nb * 16), generator=gen, device="cuda", dtype=torch.uint8)
    xq = torch.randint(0, 256, (M, nb * 16), generator=gen, device="cuda", dtype=torch.uint8)
    sw = torch.randint(110, 145, (N, nb), generator=gen, device="cuda", dtype=torch.uint8)
    sx = torch.randint(110, 145, (M, nb), generator=gen, device="cuda", dtype=torch.uint8)
    check(ops.linear_mxfp4_a4(xq, sx, w, sw, K), values(xq, sx, K), values(w, sw, K))
    x = torch.randn((M, K), generator=gen, device="cuda").bfloat16()
    check(ops.linear_mxfp4(x, w, sw), x.double(), values(w, sw, K))


@pytest.mark.parametrize("M", [2, 40])
def test_extreme_scales_and_nan(ops, M):
    """Products whose factors are near the ends of the range, and a NaN block."""
    N, K = 64, 128
    w = torch.full((N, 64), 0x22, dtype=torch.uint8, device="cuda")      # ones
    xq = torch.full((M, 64), 0x22, dtype=torch.uint8, device="cuda")
    sw = torch.full((N, 4), 254, dtype=torch.uint8, device="cuda")
    sx = torch.full((M, 4), 1, dtype=torch.uint8, device="cuda")
    y = ops.linear_mxfp4_a4(xq, sx, w, sw, K)
    assert bool((y == 128 * 2.0).all())                                    # 2^127 * 2^-126 * 128
    sw[5, 2] = 255
    y = ops.linear_mxfp4_a4(xq, sx, w, sw, K)
    assert bool(torch.isnan(y[:, 5]).all()) and bool((y[:, :5] == 256).all()) and bool((y[:, 6:] == 256).all())
    x = torch.full((M, K), 2.0 ** -126, device="cuda").bfloat16()
    y = ops.linear_mxfp4(x, w, sw)
    assert bool(torch.isnan(y[:, 5]).all()) and bool((y[:, :5] == 256).all()) and bool((y[:, 6:] == 256).all())


def test_other_stream_and_empty(ops):
    w, sw = weights(ops, 300, 512, 1)
    x = torch.randn((3, 512), device="cuda").bfloat16()
    base = ops.linear_mxfp4(x, w, sw)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y = ops.linear_mxfp4(x, w, sw, stream=st)
    st.synchronize()
    assert torch.equal(y, base)
    assert ops.linear_mxfp4(x[:0], w, sw).shape == (0, 300)
    nothing = torch.empty((3, 0), dtype=torch.uint8, device="cuda")
    y = torch.full((3, 3), 7.0, device="cuda")
    assert ops.raw.w4_linear_mxfp4_a4(None, None, None, None, y.data_ptr(), 0, 3, 3, 0, 0, None) == ops.W4_OK
    torch.cuda.synchronize()
    assert bool((y == 0).all())
    assert ops.quantize_mxfp4(torch.empty((3, 0), device="cuda"))[0].shape == nothing.shape
