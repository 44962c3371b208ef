"""w4_attention_kv8 against plain attention in 64 bits on the values that the cache holds.

With V the largest |v| a row sees and S its largest sum |q k| scale: the output is rounded once
(u), a weight to f16 (2^-11), and a score is off by D/16 truncated sums of f32 and its own
roundings, 2^-18 (S + 1), in numerator and denominator: (u + 2^-11 + 2^-17 (S + 1)) V."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from tests import kv8_reference as ref  # noqa: E402

BF16, F16 = torch.bfloat16, torch.float16
U = {BF16: 2.0 ** -8, F16: 2.0 ** -11}


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_int4_quantized_gb300 import build
    build.build()
    from w4a16_int4_quantized_gb300 import ops
    return ops


class Batch:
    def __init__(self, ops, ctx, new, Hq=4, Hkv=2, D=64, page=32, dtype=BF16, heads_first=True, seed=0, scales=(121, 124)):
        g = torch.Generator(device="cuda").manual_seed(seed)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
        pages = sum(need) + 2
        ids = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        table = torch.full((len(ctx), max(need + [1])), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = ids[at: at + n]
            at += n
        self.table, self.ctx, self.page = table.cuda(), i32(ctx), page
        self.cu = i32([sum(new[:i]) for i in range(len(new) + 1)])
        self.max_len, self.max_new = max(c + n for c, n in zip(ctx, new)), max(new)
        self.q = (1.5 * torch.randn((sum(new), Hq, D), generator=g, device="cuda")).to(dtype)
        shape = (pages, Hkv, page, D) if heads_first else (pages, page, Hkv, D)
        code = lambda: (32 * torch.randn(shape, generator=g, device="cuda")).round().clamp(-127, 127).to(torch.int8)  # noqa: E731
        view = (lambda t: t.transpose(1, 2)) if heads_first else (lambda t: t)
        byte = lambda: torch.randint(*scales, (pages, Hkv, page // 16), generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
        self.cache = ops.Kv8Cache(view(code()), view(code()), byte(), byte())
        self.scale = 1 / math.sqrt(D)

    def run(self, ops, window=0, sinks=0, **kw):
        kw = dict(dict(scale=self.scale, max_len=self.max_len, max_new=self.max_new), **kw)
        return ops.attention_kv8(self.q, self.cache, self.table, self.ctx, self.cu, window=window, sinks=sinks, **kw)

    def check(self, out, window=0, sinks=0, max_new=1 << 30):
        c = self.cache
        want, v, s = ref.attention(self.q, ref.values(c.k, c.k_scale), ref.values(c.v, c.v_scale), self.table.cpu(),
                                   self.ctx, self.cu, self.scale, self.page, window, sinks, max_new)
        live = want.isfinite().all(-1)
        assert live.any()
        bound = ((U[self.q.dtype] + 2.0 ** -11 + 2.0 ** -17 * (s + 1)) * v)[..., None]
        assert ((out.double() - want).abs() <= bound + 2.0 ** -25)[live].all(), ((out.double() - want).abs() / bound)[live].max()
        return want


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,page,heads_first", [
    ([0], [1], 1, 1, 64, 16, True), ([1000], [1], 16, 4, 64, 16, True), ([15, 16, 17, 0], [1, 1, 1, 1], 4, 2, 128, 16, False),
    ([700, 3, 0, 64], [4, 1, 7, 0], 28, 4, 128, 64, False), ([0], [100], 4, 2, 80, 32, True), ([50, 9], [33, 70], 5, 5, 96, 16, True),
    ([2000], [3], 2, 1, 256, 128, False), ([300] * 9, [1] * 9, 8, 8, 16, 16, True), ([129], [5], 40, 1, 128, 32, True),
    ([5000], [1], 8, 1, 128, 32, True), ([4097, 1], [17, 40], 16, 2, 112, 16, False), ([31], [2], 6, 3, 48, 256, True),
    ([0, 77], [300, 260], 8, 2, 128, 64, True)])
def test_against_64_bits(ops, dtype, ctx, new, Hq, Hkv, D, page, heads_first):
    b = Batch(ops, ctx, new, Hq, Hkv, D, page, dtype, heads_first, seed=Hq + D)
    b.check(b.run(ops))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (17, 16), (100, 17), (256, 0), (300, 400), (5000, 4), (64, 2 ** 30)])
@pytest.mark.parametrize("ctx,new,Hq,Hkv,D", [([900, 40, 0], [1, 3, 1], 8, 2, 64), ([500], [150], 4, 2, 128), ([4000, 2000], [1, 1], 7, 1, 128)])
def test_window_and_first_tokens(ops, window, sinks, ctx, new, Hq, Hkv, D):
    b = Batch(ops, ctx, new, Hq, Hkv, D, page=16, dtype=F16, seed=window)
    # pages that every window has left, and that no first token is on, are given up
    for i, (c, n) in enumerate(zip(ctx, new)):
        lo, hi = -(-min(sinks, c) // 16), max(0, c - window + 1) // 16
        if lo < hi:
            b.table[i, lo:hi] = -1
    b.check(b.run(ops, window, sinks), window, sinks)


def test_strides(ops):
    b = Batch(ops, [60, 7], [2, 9], 4, 2, 64)
    wide = torch.randn((11, 3, 4, 64), device="cuda").to(BF16)
    b.q = wide[:, 1]
    want = b.check(b.run(ops))
    out = torch.empty((11, 4, 64), device="cuda", dtype=BF16)
    assert b.run(ops, out=out) is out and want is not None
    b.q = b.q.contiguous()
    assert torch.equal(b.run(ops), out)


def test_hidden_keys_never_count(ops):
    # NaN scales and the largest codes where no row sees them: behind the end, behind a row's own place in
    # another block, outside the window
    b = Batch(ops, [40, 200], [3, 20], 4, 2, 128, page=16, dtype=F16)
    want = b.run(ops, window=30, sinks=3)
    c = b.cache
    for i, (ctx, n) in enumerate(((40, 3), (200, 20))):
        for j in range(0, b.table.shape[1] * 16, 16):
            page = int(b.table[i, j // 16])
            if page < 0:
                continue
            seen = [k for k in range(j, j + 16) if k < ctx + n and (k < 3 or k > ctx - 30)]
            if not seen:
                c.k_scale[page], c.v_scale[page] = 255, 255
            for k in range(j, j + 16):
                if k not in seen:
                    c.k[page, k - j], c.v[page, k - j] = 127, -127
    free = [p for p in range(c.k.shape[0]) if p not in b.table.flatten().tolist()]
    c.k_scale[free], c.v_scale[free] = 255, 255
    assert torch.equal(b.run(ops, window=30, sinks=3), want)


def test_not_finite_keys_that_are_seen(ops):
    # a block of NaN gives NaN to the rows that see it, and to those alone
    b = Batch(ops, [0], [64], 2, 1, 64, page=16)
    for which in ("k_scale", "v_scale"):
        s = getattr(b.cache, which)
        old = s.clone()
        s[int(b.table[0, 2])] = 255
        out = b.run(ops)
        assert out[:32].isfinite().all() and out[32:].isnan().all()
        s.copy_(old)
    b.q[5, 1, 3] = float("nan")
    out = b.run(ops)
    assert out[5, 1].isnan().all() and out[5, 0].isfinite().all() and out[6].isfinite().all() and out[:5].isfinite().all()


def test_nothing_seen_is_zero(ops):
    b = Batch(ops, [40, 10], [2, 3], 4, 2, 64, page=16)
    b.table[0] = -1
    b.table[1, 0] = 10 ** 6
    out = b.run(ops)
    assert (out == 0).all()
    # pages in the middle missing: the rest counts
    b = Batch(ops, [100, 90], [2, 70], 4, 2, 64, page=16)
    b.table[:, 2:4] = -1
    b.check(b.run(ops))


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_scales_far_apart(ops, dtype):
    # values of blocks from 2^-100 to 2^60: each row to its own largest
    b = Batch(ops, [400], [2], 4, 2, 64, page=16, dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(5)
    b.cache.v_scale.copy_(torch.randint(27, 128 if dtype == F16 else 188, b.cache.v_scale.shape, generator=g, device="cuda"))
    b.check(b.run(ops))
    b.cache.v_scale.zero_()      # the smallest scale
    out = b.run(ops)
    assert out.isfinite().all()
    # keys of very different size: scores up to some hundreds
    b = Batch(ops, [400], [2], 4, 2, 64, page=16, dtype=dtype, scales=(110, 127))
    b.check(b.run(ops))


def test_long_tail_beside_a_dominant_key(ops):
    # 30,000 keys of weight 2^-20 beside one: their share of the sum is not lost
    n = 30000
    b = Batch(ops, [n], [1], 1, 1, 64, page=64, dtype=F16)
    c = b.cache
    c.k.zero_(), c.v.fill_(64), c.k_scale.fill_(127), c.v_scale.fill_(127)
    c.k[int(b.table[0, 0]), 3, 0, 0] = 100
    c.v[int(b.table[0, 0]), 3] = 0
    b.q.zero_()
    b.scale = 1.0
    b.q[0, 0, 0] = 20 * math.log(2) / 100
    want = b.check(b.run(ops))
    assert (want > 1).all()


def test_small_and_large_queries(ops):
    b = Batch(ops, [50], [4], 2, 1, 64, page=16)
    b.q[0] *= 2.0 ** -120
    b.q[1] = 0
    b.q[2, 0] *= 2.0 ** 40
    out = b.run(ops)
    keep = [0, 1, 3]
    c = b.cache
    want, v, s = ref.attention(b.q, ref.values(c.k, c.k_scale), ref.values(c.v, c.v_scale), b.table.cpu(), b.ctx, b.cu,
                               b.scale, b.page)
    bound = ((2.0 ** -8 + 2.0 ** -11 + 2.0 ** -17 * (s + 1)) * v)[..., None]
    assert ((out.double() - want).abs() <= bound)[keep].all()
    assert out[2].isfinite().all()


def test_bounds_and_padding(ops):
    # a request longer than max_len is read whole; tokens beyond max_new and rows behind the last one stay
    b = Batch(ops, [3000, 10], [2, 40], 4, 2, 64, page=16)
    full = b.run(ops)
    b.check(full)
    part = torch.full_like(full, 7.0)
    b.run(ops, max_len=500, max_new=30, out=part)
    assert (part[2 + 30:] == 7.0).all()
    b.check(part, max_new=30)
    pad = torch.full((50, 4, 64), 7.0, device="cuda", dtype=BF16)
    q = b.q
    b.q = torch.cat([q, torch.full((8, 4, 64), float("nan"), device="cuda", dtype=BF16)])
    b.run(ops, out=pad)
    assert torch.equal(pad[:42], full) and (pad[42:] == 7.0).all()
    b.q = q
    b.cu[2] = 1000       # counts as the number of rows
    assert torch.equal(b.run(ops), full)


def test_workspace_of_any_content(ops):
    b = Batch(ops, [20000, 3], [1, 1], 8, 1, 128, page=64)
    want = b.run(ops)
    b.check(want)
    need = ops.attention_kv8_workspace_bytes(2, 8, 1, 128, b.max_len, 1)
    assert need > 0
    ws = torch.full((need // 4,), float("nan"), device="cuda")
    assert torch.equal(b.run(ops, workspace=ws), want)
    assert torch.equal(b.run(ops, workspace=ws), want)


def test_far_pages(ops):
    pages, stride = 5, (1 << 32) // 4 + 4096
    b = Batch(ops, [30], [2], 4, 2, 64, page=16)
    flat = [torch.zeros(pages * stride, dtype=torch.int8, device="cuda") for _ in range(2)]
    k, v = (f.as_strided((pages, 16, 2, 64), (stride, 128, 64, 1)) for f in flat)
    k.copy_(torch.randint(-127, 128, k.shape, device="cuda")), v.copy_(torch.randint(-127, 128, v.shape, device="cuda"))
    sc = [torch.full((pages, 2, 1), 121, dtype=torch.uint8, device="cuda") for _ in range(2)]
    b.cache = ops.Kv8Cache(k, v, *sc)
    b.table = torch.tensor([[4, 3]], dtype=torch.int32, device="cuda")
    b.check(b.run(ops))


def test_many_requests(ops):
    ctx = [(37 * i) % 200 for i in range(300)]
    b = Batch(ops, ctx, [1 + i % 3 for i in range(300)], 4, 2, 64, page=16)
    b.check(b.run(ops))


def test_other_stream_and_graphs_that_share_a_workspace(ops):
    a, b = Batch(ops, [9000], [1], 8, 1, 128, page=64), Batch(ops, [8000, 50], [1, 2], 8, 1, 128, page=64, seed=3)
    wa, wb = a.run(ops), b.run(ops)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = a.run(ops, stream=st)
    st.synchronize()
    assert torch.equal(got, wa)
    need = max(ops.attention_kv8_workspace_bytes(x.table.shape[0], 8, 1, 128, x.max_len, x.max_new) for x in (a, b))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graphs = []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = x.run(ops, workspace=ws)
        graphs.append((g, o))
    for _ in range(2):
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(graphs[0][1], wa) and torch.equal(graphs[1][1], wb)
        graphs[0][1].zero_(), graphs[1][1].zero_()
    assert ops.device_status() == 0
