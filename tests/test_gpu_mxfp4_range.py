"""GPU tests of the MXFP4 products over the whole range of the scales and of K, against 64 bits.

The bound is the header's: max(1e-5, 2.5e-9 K) sum |x W| + K 2^-120 + the rounding of y."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_mxfp4 import U, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_int4_quantized_gb300 import build
    build.build()
    from w4a16_int4_quantized_gb300 import ops as o
    o.device_status(clear=True)
    return o


def check(y, x, w):
    K = x.shape[1]
    want, size = x @ w.T, x.abs() @ w.abs().T
    tol = max(1e-5, 2.5e-9 * K) * size + K * 2.0 ** -120 + U[y.dtype] * want.abs() * 1.01
    err = (y.double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


def codes(rows, K, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, 256, (rows, -(-K // 32) * 16), generator=gen, device="cuda", dtype=torch.uint8)


@pytest.mark.parametrize("M", [1, 9, 16, 40])
@pytest.mark.parametrize("s", [0, 1, 2, 3, 4, 127, 128, 129, 130, 131, 132, 133, 250, 251, 252, 253, 254])
def test_one_scale(ops, M, s):
    """All codes under one scale, with x of about its reciprocal."""
    N, K = 70, 416
    w, sw = codes(N, K, s), torch.full((N, K // 32), s, dtype=torch.uint8, device="cuda")
    W = values(w, sw, K)
    gen = torch.Generator(device="cuda").manual_seed(M)
    x = (torch.randn((M, K), generator=gen, device="cuda").double() * 2.0 ** min(max(127 - s, -120), 120)).bfloat16()
    for dt in (torch.float32, torch.bfloat16):
        check(ops.linear_mxfp4(x, w, sw, out_dtype=dt), x.double(), W)
    xq, sx = codes(M, K, 1000 + M), torch.full((M, K // 32), 254 - s, dtype=torch.uint8, device="cuda")
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        check(ops.linear_mxfp4_a4(xq, sx, w, sw, K, out_dtype=dt), values(xq, sx, K), W)
    assert ops.device_status() == 0


@pytest.mark.parametrize("M", [2, 16, 30])
@pytest.mark.parametrize("N,K", [(64, 4096), (300, 8192)])
def test_all_scales_in_a_row(ops, M, N, K):
    """Blocks under scales from 2^-127 to 2^127 side by side, x of about each one's reciprocal."""
    nb = K // 32
    gen = torch.Generator(device="cuda").manual_seed(K)
    s = torch.randint(0, 255, (nb,), generator=gen, device="cuda")
    s[:2] = torch.tensor([0, 254], device="cuda")
    w, sw = codes(N, K, N), s.to(torch.uint8).repeat(N, 1).contiguous()
    W = values(w, sw, K)
    e = (127 - s).clamp(-120, 120).repeat_interleave(32).double()
    x = (torch.randn((M, K), generator=gen, device="cuda").double() * torch.exp2(e)).bfloat16()
    check(ops.linear_mxfp4(x, w, sw), x.double(), W)
    xq, sx = codes(M, K, M), (254 - s).to(torch.uint8).repeat(M, 1).contiguous()
    check(ops.linear_mxfp4_a4(xq, sx, w, sw, K), values(xq, sx, K), W)
    assert ops.device_status() == 0


@pytest.mark.parametrize("M", [1, 16, 17])
def test_weights_beyond_bf16(ops, M):
    """4 * 2^127 and the like are numbers, whatever M: times 2^-126 they give 8, times zero 0."""
    N, K = 40, 64
    for code, value in ((0x44, 2.0), (0x55, 3.0), (0x66, 4.0), (0x77, 6.0)):
        w = torch.full((N, K // 2), code, dtype=torch.uint8, device="cuda")
        sw = torch.full((N, K // 32), 254, dtype=torch.uint8, device="cuda")
        x = torch.full((M, K), 2.0 ** -126, device="cuda").bfloat16()
        assert bool((ops.linear_mxfp4(x, w, sw) == 2 * value * K).all())
        assert bool((ops.linear_mxfp4(torch.zeros_like(x), w, sw) == 0).all())
        xq = torch.full((M, K // 2), 0x22, dtype=torch.uint8, device="cuda")
        sx = torch.full((M, K // 32), 1, dtype=torch.uint8, device="cuda")
        assert bool((ops.linear_mxfp4_a4(xq, sx, w, sw, K) == 2 * value * K).all())
        assert bool((ops.linear_mxfp4_a4(w[:M].contiguous(), sw[:M].contiguous(), torch.zeros_like(w), sw, K) == 0).all())


@pytest.mark.parametrize("M", [1, 13, 16, 40, 300])
@pytest.mark.parametrize("N,K", [(2048, 2048), (9800, 4096), (9800, 13312), (300, 13312), (300, 28672), (130, 65536)])
def test_long_sums_of_one_sign(ops, M, N, K):
    """Every product positive and under scales of its own, so that each rounding counts and none cancels."""
    gen = torch.Generator(device="cuda").manual_seed(M + K)

    def matrix(R):
        c = codes(R, K, R + K) & 0x77
        return c, torch.randint(121, 133, (R, K // 32), generator=gen, device="cuda", dtype=torch.uint8)

    w, sw = matrix(N)
    W = values(w, sw, K)
    x = (torch.rand((M, K), generator=gen, device="cuda") + 0.1).bfloat16()
    if M <= 40:
        check(ops.linear_mxfp4(x, w, sw), x.double(), W)
    xq, sx = matrix(M)
    check(ops.linear_mxfp4_a4(xq, sx, w, sw, K), values(xq, sx, K), W)
    assert ops.device_status() == 0


def test_values_beyond_the_output_type(ops):
    """Which codes under which of the largest scales are infinite, as the header lists them."""
    grid = torch.arange(16, dtype=torch.uint8, device="cuda")
    w = torch.cat([grid[0::2] | (grid[1::2] << 4), torch.zeros(8, dtype=torch.uint8, device="cuda")]).repeat(3, 1)
    s = torch.tensor([[252], [253], [254]], dtype=torch.uint8, device="cuda")
    far = {252: (), 253: (4.0, 6.0), 254: (2.0, 3.0, 4.0, 6.0)}
    for dt in (torch.float32, torch.bfloat16):
        y = ops.dequantize_mxfp4(w.contiguous(), s, 16, dt)
        for row, byte in enumerate((252, 253, 254)):
            for c, v in enumerate((0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)):
                want = float("inf") if v in far[byte] else v * 2.0 ** (byte - 127)
                assert float(y[row, c]) == want and float(y[row, 8 + c]) == -want, (dt, byte, v)
