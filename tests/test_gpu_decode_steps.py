"""The MXFP4 decode product takes no step up in time where one more row tile would not run at once.

Times of a height of W against a slightly smaller one: within 1.4, where blocks that wait
for a cluster's place take 1.48 to 1.6 (and a change of the split 1.25 at most)."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_int4_quantized_gb300 import build
    build.build()
    from w4a16_int4_quantized_gb300 import ops as o
    return o


def time_of(ops, N, K):
    """The middle of 9 replays of 24 calls, over more weights than the L2 holds."""
    nb = K // 32
    W = [(torch.full((N, nb * 16), 0x22, dtype=torch.uint8, device="cuda"),
          torch.full((N, nb), 127, dtype=torch.uint8, device="cuda")) for _ in range(150_000_000 // (N * nb * 17) + 1)]
    x, y = torch.ones((1, K), device="cuda").bfloat16(), torch.empty((1, N), device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        ops.linear_mxfp4(x, *W[0], out=y)
        torch.cuda.synchronize()
        assert bool((y == K).all())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for i in range(24):
                ops.linear_mxfp4(x, *W[i % len(W)], out=y)
        g.replay()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        ts = []
        for _ in range(9):
            a.record(st)
            g.replay()
            b.record(st)
            torch.cuda.synchronize()
            ts.append(a.elapsed_time(b))
    return sorted(ts)[4]


@pytest.mark.parametrize("K", [8192, 13312])
@pytest.mark.parametrize("small,large", [(2304, 2400), (2304, 2432), (1152, 1200), (1152, 1216), (544, 592), (544, 608)])
def test_one_more_tile(ops, small, large, K):
    assert time_of(ops, large, K) <= 1.4 * time_of(ops, small, K)


@pytest.mark.parametrize("N,K", [(608, 8192), (1216, 8192), (1250, 8192), (2048, 8192), (2400, 13312), (300, 16384), (1024, 16384)])
def test_rows_do_not_depend_on_each_other(ops, N, K):
    """The split over K is one for every M: a row of x gives the same bits alone and among others."""
    gen = torch.Generator(device="cuda").manual_seed(N)
    w, sw = ops.quantize_mxfp4(torch.randn((N, K), generator=gen, device="cuda"))
    x = torch.randn((40, K), generator=gen, device="cuda").bfloat16()
    whole = ops.linear_mxfp4(x, w, sw)
    for m0, m1 in ((0, 1), (3, 11), (7, 20), (30, 40)):
        assert torch.equal(ops.linear_mxfp4(x[m0:m1].contiguous(), w, sw), whole[m0:m1])
