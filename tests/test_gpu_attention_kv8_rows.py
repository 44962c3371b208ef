"""w4_attention_kv8 with many rows to a key head (the tensor-core kernel), and where the choice between the
kernels and between their ways of sharing the work falls; limits as in test_gpu_attention_kv8.py."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from tests import kv8_reference as ref  # noqa: E402
from tests.test_gpu_attention_kv8 import BF16, F16, Batch, ops  # noqa: E402, F401


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D,page", [(16, 16), (48, 32), (64, 64), (64, 256), (80, 16), (128, 32), (128, 128), (144, 16), (256, 64), (256, 32)])
@pytest.mark.parametrize("heads_first", [True, False])
def test_heads_and_pages(ops, dtype, D, page, heads_first):  # noqa: F811
    b = Batch(ops, [130, 0, 61], [40, 129, 1], 6, 2, D, page, dtype, heads_first, seed=D)
    b.check(b.run(ops))


@pytest.mark.parametrize("new", [1, 2, 4, 5, 8, 9, 16, 17, 31, 32, 33, 64, 65])
@pytest.mark.parametrize("G", [1, 4, 7])
def test_rows_around_the_tiles(ops, new, G):  # noqa: F811
    # 16 and 32 rows of the small tiles, 128 and 256 of the large ones
    b = Batch(ops, [100, 700], [new, max(1, new // 2)], 2 * G, 2, 64, 32, F16, seed=new * G)
    b.check(b.run(ops))


@pytest.mark.parametrize("window,sinks", [(1, 0), (63, 1), (64, 64), (65, 65), (200, 70), (1000, 129), (17, 4000)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_window(ops, window, sinks, D):  # noqa: F811
    b = Batch(ops, [1500, 90, 0], [70, 200, 33], 4, 2, D, 16, BF16, seed=window)
    for i, c in enumerate((1500, 90, 0)):
        lo, hi = -(-min(sinks, c) // 16), max(0, c - window + 1) // 16
        if lo < hi:
            b.table[i, lo:hi] = -1
    b.check(b.run(ops, window, sinks), window, sinks)


@pytest.mark.parametrize("order", [(2, 0, 1, 3), (1, 0, 2, 3), (1, 2, 0, 3), (2, 1, 0, 3), (0, 2, 1, 3)])
@pytest.mark.parametrize("new", [2, 40])
def test_any_order_of_pages_tokens_and_heads(ops, order, new):  # noqa: F811
    # the cache's axes (page, token, head, value) in memory in another order, with gaps
    b = Batch(ops, [100, 30], [new, 1], 4, 2, 64, 32, F16)
    want, c = b.run(ops), b.cache
    back = [order.index(i) for i in range(4)]
    k, v = (torch.nn.functional.pad(x.permute(order), (0, 16, 0, 3)).contiguous()[:, :, : x.shape[order[2]], :64].permute(back)
            for x in (c.k, c.v))
    assert torch.equal(k, c.k)
    b.cache = ops.Kv8Cache(k, v, c.k_scale, c.v_scale)
    assert torch.equal(b.run(ops), want)
    got, _ = ops.dequantize_kv8(b.cache, torch.float32)
    assert torch.equal(got.double(), ref.values(c.k, c.k_scale))


def test_units_cut_anywhere(ops):  # noqa: F811
    # fewer units than CTAs, and lengths that leave a part of one step here and there
    for ctx, new, G in (([20000], [16], 4), ([9000, 40, 3000, 17], [40, 1, 33, 64], 4), ([1], [1000], 1)):
        b = Batch(ops, ctx, new, 2 * G, 2, 64, 64, BF16, seed=len(ctx))
        want = b.run(ops)
        b.check(want)
        need = ops.attention_kv8_workspace_bytes(len(ctx), 2 * G, 2, 64, b.max_len, b.max_new)
        ws = torch.full((need // 4 + 4,), float("nan"), device="cuda")
        for _ in range(2):
            assert torch.equal(b.run(ops, workspace=ws), want)


def test_hidden_keys_and_nan_blocks(ops):  # noqa: F811
    b = Batch(ops, [200], [80], 4, 2, 128, 16, F16)
    want = b.run(ops, window=50, sinks=3)
    c = b.cache
    for j in range(16, 144, 16):      # behind every window, not among the first tokens
        page = int(b.table[0, j // 16])
        c.k_scale[page], c.v_scale[page] = 255, 255
    free = [p for p in range(c.k.shape[0]) if p not in b.table.flatten().tolist()]
    c.k_scale[free], c.v_scale[free] = 255, 255
    assert torch.equal(b.run(ops, window=50, sinks=3), want)
    # a block that some rows see: those are NaN, the others as before
    for which in ("k_scale", "v_scale"):
        s = getattr(c, which)
        old = s.clone()
        s[int(b.table[0, 15])] = 255    # keys 240 .. 255: the rows from token 40 on see the first of them
        out = b.run(ops, window=50, sinks=3)
        assert torch.equal(out[:40], want[:40]) and out[40:].isnan().all()
        s.copy_(old)
    b.q[7, 1, 3] = float("inf")
    out = b.run(ops, window=50, sinks=3)
    assert not out[7, 1].isfinite().all() and torch.equal(out[8:], want[8:]) and torch.equal(out[:7], want[:7])


@pytest.mark.parametrize("new", [3, 80])
def test_a_large_scale_touches_only_rows_that_see_it(ops, new):  # noqa: F811
    # values 2^80 times the others' in the last block (its first key is the last token's own), behind all
    # windows and on a page that nobody has
    b = Batch(ops, [193 - new], [new], 4, 2, 64, 16, F16)
    want = b.run(ops, window=20, sinks=2)
    c, free = b.cache, [p for p in range(b.cache.k.shape[0]) if p not in b.table.flatten().tolist()]
    for page in [int(b.table[0, 12]), int(b.table[0, 2])] + free:
        c.v_scale[page] += 80
    out = b.run(ops, window=20, sinks=2)
    assert torch.equal(out[:-1], want[:-1])
    c.v_scale[int(b.table[0, 12])] -= 80
    assert torch.equal(b.run(ops, window=20, sinks=2), want)


@pytest.mark.parametrize("new", [4, 70])
def test_scores_far_from_zero(ops, new):  # noqa: F811
    # one key a million times larger than the others along the query: all of the weight; the same
    # far below: none of it, and beside such keys alone nothing is left
    b = Batch(ops, [40], [new], 2, 1, 64, 16, BF16)
    c, p0 = b.cache, int(b.table[0, 0])
    c.k.zero_()
    b.q.zero_()
    b.q[:, :, 0] = 2.0 ** 30
    c.k[p0, 5, 0, 0] = 100
    out = b.run(ops)
    want = c.v[p0, 5, 0].double() * 2.0 ** (int(c.v_scale[p0, 0, 0]) - 127)
    assert (out.double() - want).abs().max() <= 2.0 ** -8 * want.abs().max()
    c.k[p0, 5, 0, 0] = -100
    b.check(b.run(ops))
    c.k[..., 0] = -100
    assert (b.run(ops) == 0).all()
    c.k[..., 0] = 100     # scores as large as their block's scale: the mean over the keys of the largest one
    want = ref.attention(b.q, ref.values(c.k, c.k_scale), ref.values(c.v, c.v_scale), b.table.cpu(), b.ctx, b.cu, b.scale, 16)[0]
    assert (b.run(ops).double() - want).abs().max() <= 2.0 ** -6


def test_missing_pages(ops):  # noqa: F811
    for page in (16, 32, 128):
        b = Batch(ops, [600, 90], [50, 70], 4, 2, 64, page)
        b.table[0, 1:3] = -1
        b.table[1, 0] = 10 ** 6
        b.check(b.run(ops))
        b.table[:] = -1
        assert (b.run(ops) == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_scales_far_apart(ops, dtype):  # noqa: F811
    b = Batch(ops, [400], [70], 4, 2, 64, page=16, dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(5)
    b.cache.v_scale.copy_(torch.randint(27, 128 if dtype == F16 else 188, b.cache.v_scale.shape, generator=g, device="cuda"))
    b.check(b.run(ops))
    b.cache.v_scale.zero_()
    b.cache.k_scale.zero_()
    assert b.run(ops).isfinite().all()
    b = Batch(ops, [400], [70], 4, 2, 64, page=16, dtype=dtype, scales=(110, 127))
    b.check(b.run(ops))


def test_many_requests(ops):  # noqa: F811
    # more (request, tile) pairs than threads to a CTA, some without rows
    ctx = [(37 * i) % 150 for i in range(700)]
    b = Batch(ops, ctx, [i % 40 for i in range(700)], 2, 2, 64, page=16)
    b.check(b.run(ops))
    # and than are dealt out by their blocks
    b = Batch(ops, [i % 30 for i in range(5000)], [1] * 5000, 2, 2, 16, page=16)
    b.check(b.run(ops))


def test_padding_and_bounds(ops):  # noqa: F811
    b = Batch(ops, [3000, 10, 5], [40, 200, 0], 4, 2, 64, page=16)
    full = b.run(ops)
    b.check(full)
    part = torch.full_like(full, 7.0)
    b.run(ops, max_len=100, max_new=130, out=part)
    assert (part[40 + 130:] == 7.0).all()
    b.check(part, max_new=130)
    pad, q = torch.full((250, 4, 64), 7.0, device="cuda", dtype=BF16), b.q
    b.q = torch.cat([q, torch.full((10, 4, 64), float("nan"), device="cuda", dtype=BF16)])
    b.run(ops, out=pad)
    assert torch.equal(pad[:240], full) and (pad[240:] == 7.0).all()
    assert ops.device_status() == 0


def test_captured_beside_eager(ops):  # noqa: F811
    a, b = Batch(ops, [2000], [64], 8, 2, 128, page=64), Batch(ops, [800, 50], [90, 2], 8, 2, 128, page=64, seed=3)
    wa, wb = a.run(ops), b.run(ops)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = a.run(ops)
    st = torch.cuda.Stream()
    for _ in range(3):
        out.zero_()
        st.wait_stream(torch.cuda.current_stream())
        g.replay()
        got = b.run(ops, stream=st)
        torch.cuda.synchronize()
        assert torch.equal(out, wa) and torch.equal(got, wb)
    assert ops.device_status() == 0
