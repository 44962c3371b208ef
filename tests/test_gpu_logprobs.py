"""w4_token_logprobs against log_softmax in 64 bits; the top indices are exact.

A lane sums at most V / 512 values in a row of one CTA, 2^-24 each, and 12 joins follow:
(V / 512 + 16) 2^-24 of s, as much again of t.  An exponent d log2(e) is rounded twice, and
the power of two has 2^-22: 2^-20 (1 + |log p|)."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
INF = float("inf")


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_int4_quantized_gb300 import build
    build.build()
    from w4a16_int4_quantized_gb300 import ops
    return ops


def randn(shape, dtype, seed, scale=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def check(ops, x, ids, top):
    T, V = x.shape
    logp, entropy, top_ids, top_logp = ops.token_logprobs(x, ids, top=top)
    lp = torch.log_softmax(x.double(), -1)
    p = lp.exp()
    ent = -torch.where(p > 0, p * lp, 0.0).sum(-1)
    sums = (V / 512 + 16) * 2.0 ** -24

    def near(got, want):
        fine = want.isfinite()
        assert torch.equal(got[~fine].double(), want[~fine])
        assert ((got.double() - want)[fine].abs() <= 2.0 ** -20 * (1 + want[fine].abs()) + sums).all()

    near(logp, lp.gather(1, ids.long()[:, None])[:, 0])
    assert ((entropy.double() - ent).abs() <= (2.0 ** -20 + 2 * sums) * (1 + ent)).all()
    k = min(top, V)
    order = torch.sort(x.float() + 0.0, dim=-1, descending=True, stable=True)[1][:, :k]
    assert torch.equal(top_ids[:, :k].long(), order)
    near(top_logp[:, :k], lp.gather(1, order))
    assert (top_ids[:, k:] == -1).all() and top_logp[:, k:].isnan().all()


@pytest.mark.parametrize("T,V", [(1, 1), (1, 2), (2, 33), (1, 32000), (3, 4097), (32, 100003), (200, 5001), (160, 32768),
                                 (1, 262144), (5, 65537), (151, 1024), (152, 1024)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("top", [0, 1, 20, 32])
def test_rows(ops, T, V, dtype, top):
    x = randn((T, V), dtype, T + V)
    ids = torch.randint(0, V, (T,), device="cuda", dtype=torch.int32)
    check(ops, x, ids, top)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_strides_and_starts(ops, dtype):
    wide = randn((7, 3001), dtype, 5)
    ids = torch.arange(7, device="cuda", dtype=torch.int32) * 100
    for start in (0, 1, 2, 3, 5, 8):
        for V in (2000, 2001, 2990):
            check(ops, wide[:, start: start + V], ids, 7)


@pytest.mark.parametrize("V", [1000, 70001])
def test_orders_and_ties(ops, V):
    ramp = torch.arange(V, device="cuda", dtype=F32) / V
    rows = torch.stack([ramp, ramp.flip(0), torch.zeros_like(ramp), (ramp * 10).round(), -ramp,
                        torch.where(torch.arange(V, device="cuda") % 2 == 0, 0.0, -0.0)])
    ids = torch.arange(6, device="cuda", dtype=torch.int32)
    for dtype in (F32, BF16):
        check(ops, rows.to(dtype), ids, 32)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_masked(ops, dtype):
    V = 5000
    x = randn((6, V), dtype, 9)
    low = torch.finfo(dtype).min
    x[0, 100:] = -INF
    x[1, ::2] = low
    x[2, 1:] = -INF
    x[3, :-1] = low
    x[4] = low      # every logit masked by the same number: uniform
    x[5, 3:] = -INF  # fewer real ones than alternatives
    check(ops, x, torch.tensor([3, 7, 0, V - 1, 11, 4], device="cuda", dtype=torch.int32), 20)


def test_not_finite(ops):
    V = 3000
    x = randn((5, V), F32, 10)
    x[0, 17] = float("nan")
    x[1, 20] = INF
    x[2] = -INF
    x[3] = float("nan")
    ids = torch.tensor([1, 2, 3, 4, 5], device="cuda", dtype=torch.int32)
    logp, entropy, top_ids, top_logp = ops.token_logprobs(x, ids, top=4)
    assert logp[:4].isnan().all() and entropy[:4].isnan().all() and top_logp[:4].isnan().all()
    assert logp[4].isfinite() and entropy[4].isfinite()
    order = torch.sort(x[0].nan_to_num(nan=-INF), descending=True, stable=True)[1][:4]
    assert torch.equal(top_ids[0].long(), order)
    assert top_ids[1, 0] == 20 and top_ids[2].tolist() == [0, 1, 2, 3] and top_ids[3].tolist() == [-1] * 4


def test_ids_outside(ops):
    x = randn((4, 300), F32, 11)
    logp, entropy, _, _ = ops.token_logprobs(x, torch.tensor([-1, 300, 2 ** 31 - 1, 5], device="cuda", dtype=torch.int32))
    assert logp[:3].isnan().all() and logp[3].isfinite() and entropy.isfinite().all()
    assert ops.token_logprobs(x[:0], torch.zeros(0, device="cuda", dtype=torch.int32), top=3)[2].shape == (0, 3)


def test_far_offsets(ops):
    # a row whose values lie beyond 2^32 bytes
    T, V = 3, 1000
    big = torch.empty((T, 800_000_000), device="cuda", dtype=F32)
    x = big[:, -V:]
    x.copy_(randn((T, V), F32, 12))
    check(ops, x, torch.tensor([0, 500, 999], device="cuda", dtype=torch.int32), 5)


def test_same_bits_and_graph(ops):
    x = randn((6, 50001), BF16, 13)
    ids = torch.zeros(6, device="cuda", dtype=torch.int32)
    a = ops.token_logprobs(x, ids, top=20)
    for _ in range(3):
        assert all(torch.equal(u, v) for u, v in zip(a, ops.token_logprobs(x, ids, top=20)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = ops.token_logprobs(x, ids, top=20, stream=s)
    s.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = ops.token_logprobs(x, ids, top=20)
    x.copy_(randn((6, 50001), BF16, 14))
    g.replay()
    a = ops.token_logprobs(x, ids, top=20)
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(a, c))
