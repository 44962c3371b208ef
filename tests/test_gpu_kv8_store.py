"""w4_qk_norm_rope_kv8 and w4_dequantize_kv8 against plain forms in 64 bits.

Values that the store takes as they are (values; keys without norm and rotation) give exact codes
and scale bytes.  With norm and rotation a key is off by 2^-19 of its head's largest value at
most (sum of squares, reciprocal root, two products, two products and a sum: under 32 steps
of 2^-24), so a code is within half a step and 127 * 2^-19 * 2 of the exact quotient."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from tests import kv8_reference as ref  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
U = {BF16: 2.0 ** -8, F16: 2.0 ** -11}


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_int4_quantized_gb300 import build
    build.build()
    from w4a16_int4_quantized_gb300 import ops
    return ops


class Step:
    """A batch with contexts and new tokens over a cache of random codes."""

    def __init__(self, ops, ctx, new, Hq=4, Hkv=2, D=64, page=32, inp=F32, heads_first=True, seed=0, spare=3, width=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
        pages = sum(need) + spare
        ids = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        width = width or max(need + [1])
        table = torch.full((len(ctx), width), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :min(n, width)] = ids[at: at + min(n, width)]
            at += n
        self.ctx_list, self.new_list, self.page, self.Hq, self.Hkv, self.D = ctx, new, page, Hq, Hkv, D
        self.table, self.ctx = table.cuda(), i32(ctx)
        self.cu = i32([sum(new[:i]) for i in range(len(new) + 1)])
        self.T = sum(new)
        self.positions = i32([c + i for c, n in zip(ctx, new) for i in range(n)])
        self.qkv = torch.randn((self.T, (Hq + 2 * Hkv) * D), generator=g, device="cuda").to(inp)
        shape = (pages, Hkv, page, D) if heads_first else (pages, page, Hkv, D)
        code = lambda: torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
        view = (lambda t: t.transpose(1, 2)) if heads_first else (lambda t: t)
        byte = lambda: torch.randint(118, 124, (pages, Hkv, page // 16), generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
        self.cache = ops.Kv8Cache(view(code()), view(code()), byte(), byte())

    def angles(self, rot):
        top = max(c + n for c, n in zip(self.ctx_list, self.new_list)) + 1
        a = torch.arange(top, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(rot // 2, device="cuda", dtype=torch.float64) / max(1, rot // 2))
        return torch.cat([a.cos(), a.sin()], 1).float().contiguous()

    def run(self, ops, wq=None, wk=None, cos_sin=None, **kw):
        return ops.qk_norm_rope_kv8(self.qkv, self.Hq, wq, wk, self.positions, cos_sin, self.table, self.ctx, self.cu,
                                    self.cache, **kw)

    def state(self):
        c = self.cache
        return c.k.double(), c.k_scale.long(), c.v.double(), c.v_scale.long()

    def appended(self, before, k, v):
        """The state after an exact store of k, v [T, head, value]."""
        kc, ks, vc, vs = (t.clone() for t in before)
        for b, (c, n) in enumerate(zip(self.ctx_list, self.new_list)):
            t0 = int(self.cu[b])
            ref.append(kc, ks, k[t0: t0 + n], self.table[b], c, n, self.page)
            ref.append(vc, vs, v[t0: t0 + n], self.table[b], c, n, self.page)
        return kc, ks, vc, vs


def same(a, b):
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("inp", [F32, BF16, F16])
@pytest.mark.parametrize("ctx,new,page,D,heads_first", [
    ([0], [1], 16, 64, True), ([1000], [1], 16, 64, True), ([15, 16, 17, 31], [1, 1, 1, 1], 16, 128, False),
    ([0, 5, 100, 7], [40, 3, 0, 17], 32, 128, True), ([3], [200], 64, 80, False), ([14, 1], [2, 33], 16, 256, True),
    ([9, 40], [16, 32], 128, 16, True), ([2] * 70, [1] * 70, 16, 96, False), ([6] * 40, [5, 0] * 20, 32, 48, True)])
def test_codes_exact(ops, inp, ctx, new, page, D, heads_first):
    s = Step(ops, ctx, new, D=D, page=page, inp=inp, heads_first=heads_first, seed=len(ctx))
    before = s.state()
    x = s.qkv.view(s.T, -1, D)
    q = s.run(ops, out_dtype=F16)
    assert torch.equal(q, x[:, :4].half())
    same(s.state(), s.appended(before, x[:, 4:6], x[:, 6:8]))
    # once more: nothing is left to change
    after = s.state()
    s.run(ops)
    same(s.state(), after)


@pytest.mark.parametrize("D,rot,inter,Hq,Hkv", [(64, 64, False, 4, 2), (128, 128, True, 8, 8), (128, 64, False, 7, 1),
                                                (80, 32, True, 5, 5), (256, 256, False, 3, 1), (96, 96, False, 40, 8)])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("out", [BF16, F16])
def test_norm_and_rotation(ops, D, rot, inter, Hq, Hkv, norm, out):
    s = Step(ops, [5, 0, 30], [20, 1, 3], Hq=Hq, Hkv=Hkv, D=D, seed=D + rot, inp=BF16)
    g = torch.Generator(device="cuda").manual_seed(1)
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g, device="cuda")) for _ in range(2)) if norm else (None, None)
    cs = s.angles(rot)
    before = s.state()
    q = s.run(ops, wq, wk, cs, interleaved=inter, out_dtype=out)
    x = s.qkv.double().view(s.T, -1, D)

    def head(h, w):
        if w is not None:
            h = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * w.double()
        c, sn = cs.double()[s.positions.long()][:, None].chunk(2, -1)
        r, rest = h[..., :rot], h[..., rot:]
        a, b = (r[..., 0::2], r[..., 1::2]) if inter else r.chunk(2, -1)
        u, v = a * c - b * sn, b * c + a * sn
        return torch.cat([torch.stack([u, v], -1).flatten(-2) if inter else torch.cat([u, v], -1), rest], -1)

    want_q, want_k = head(x[:, :Hq], wq), head(x[:, Hq: Hq + Hkv], wk)
    top = want_q.abs().amax(-1, keepdim=True)
    assert ((q.double() - want_q).abs() <= U[out] * want_q.abs() + 2.0 ** -19 * top + 2.0 ** -25).all()
    want = s.appended(before, want_k, x[:, Hq + Hkv:])
    got = s.state()
    same(got[2:], want[2:])
    assert torch.equal(got[1], want[1])      # no largest value of these inputs lies at a border
    assert (got[0] - want[0]).abs().max() <= 1   # another code only next to a tie:
    kv = ref.values(*(t for t in got[:2]))
    for b, (c, n) in enumerate(zip(s.ctx_list, s.new_list)):
        rows, _ = ref.rows_of(kv, s.table[b], c + n, s.page)
        unit, _ = ref.rows_of(torch.exp2(got[1].double() - 127).transpose(1, 2).repeat_interleave(16, 1)[..., None],
                              s.table[b], c + n, s.page)
        exact = want_k[int(s.cu[b]): int(s.cu[b + 1])]
        assert ((rows[c:] - exact).abs() <= unit[c:] * (0.5 + 127 * 2.0 ** -18)).all()


def test_scale_borders(ops):
    # the largest value of a block at and next to 127 * 2^e; tiny, zero and huge blocks
    tops = [127.0, 127.00001, 126.99999, 63.5, 63.500004, 1.0, 0.0, 1e-38, 2.0 ** -126, 1e-45, 3.4e38, 2.0 ** -121, 127 * 2.0 ** -127]
    s = Step(ops, [0] * len(tops), [3] * len(tops), Hq=2, Hkv=1, D=16, page=16)
    x = s.qkv.view(s.T, 4, 16)
    for i, t in enumerate(tops):
        x[3 * i: 3 * i + 3] = x[3 * i: 3 * i + 3].clamp(-1, 1) * t
        x[3 * i + 1, 2:, 7] = -t
    before = s.state()
    s.run(ops)
    same(s.state(), s.appended(before, x[:, 2:3], x[:, 3:4]))


def test_growing_block(ops):
    # 16 single tokens into one block, each larger than all before it: the codes of the plain form, and
    # no value further off than one step of the last scale
    s = Step(ops, [0], [16], Hq=1, Hkv=1, D=32, page=16)
    x = s.qkv.view(16, 3, 32)
    x *= 1.7 ** torch.arange(16, device="cuda")[:, None, None]
    for i in range(16):
        one = Step.__new__(Step)
        one.__dict__.update(s.__dict__)
        one.ctx_list, one.new_list, one.T = [i], [1], 1
        one.ctx, one.cu = torch.tensor([i], dtype=torch.int32, device="cuda"), torch.tensor([0, 1], dtype=torch.int32, device="cuda")
        one.qkv, one.positions = s.qkv[i: i + 1], s.positions[i: i + 1]
        before = one.state()
        one.run(ops)
        same(one.state(), one.appended(before, x[i: i + 1, 1:2], x[i: i + 1, 2:3]))
    got = ref.values(s.cache.k, s.cache.k_scale)[s.table[0, 0].long(), :, 0]
    step = torch.exp2(s.cache.k_scale[s.table[0, 0].long(), 0, 0].double() - 127)
    assert ((got - x[:, 1].double()).abs() <= step).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_not_finite(ops, bad):
    s = Step(ops, [10, 40], [3, 20], Hq=2, Hkv=2, D=64)
    x = s.qkv.view(s.T, 6, 64)
    x[1, 2, 5] = bad      # a key of head 0, in a block with kept tokens
    x[9, 5, 60] = bad     # a value of head 1, in a new block or the first one
    before = s.state()
    s.run(ops)
    want = s.appended(before, x[:, 2:4], x[:, 4:6])
    same(s.state(), want)
    assert (want[1] == 255).sum() == 1 and (want[3] == 255).sum() == 1
    k, v = ops.dequantize_kv8(s.cache, F32)
    assert torch.equal(k.isnan(), ref.values(s.cache.k, s.cache.k_scale).isnan())


def test_bad_pages_positions_and_padding(ops):
    s = Step(ops, [10, 0, 33, 5], [30, 20, 3, 8], Hq=2, Hkv=2, D=64, page=16)
    s.table[0, 1], s.table[1, 0], s.table[2, 2] = -1, 10 ** 6, -5    # tokens without a place
    x = s.qkv.view(s.T, 6, 64)
    before = s.state()
    out = torch.full((s.T + 5, 2, 64), 7.0, device="cuda", dtype=BF16)
    # rows behind the last token, which a padded batch has
    pad = torch.cat([s.qkv, torch.full((5, s.qkv.shape[1]), float("nan"), device="cuda")])
    pos = torch.cat([s.positions, torch.full((5,), 3, dtype=torch.int32, device="cuda")])
    ops.qk_norm_rope_kv8(pad, 2, None, None, pos, None, s.table, s.ctx, s.cu, s.cache, out=out)
    same(s.state(), s.appended(before, x[:, 2:4], x[:, 4:6]))
    assert torch.equal(out[: s.T], x[:, :2].to(BF16)) and (out[s.T:] == 7.0).all()
    # a position outside the table of angles: the token is left out, its codes stay
    s = Step(ops, [0], [4], Hq=2, Hkv=2, D=64)
    cs = s.angles(64)
    s.positions[2] = cs.shape[0]
    s.positions[3] = -1
    before, out = s.state(), torch.full((4, 2, 64), 7.0, device="cuda", dtype=BF16)
    s.run(ops, cos_sin=cs, out=out)
    assert (out[2:] == 7.0).all() and not (out[:2] == 7.0).all(2).any()
    at = s.table[0, 0].long()
    assert torch.equal(s.cache.k[at, 2:].double(), before[0][at, 2:]) and torch.equal(s.cache.v[at, 2:].double(), before[2][at, 2:])
    # a block table too narrow, offsets that run past the rows
    s = Step(ops, [30, 3], [10, 6], Hq=2, Hkv=2, D=64, page=16, width=2)
    x, before = s.qkv.view(s.T, 6, 64), s.state()
    s.run(ops)
    same(s.state(), s.appended(before, x[:, 2:4], x[:, 4:6]))
    s.cu[2] = 1000
    before = s.state()
    s.run(ops)
    same(s.state(), s.appended(before, x[:, 2:4], x[:, 4:6]))


def test_far_pages(ops):
    # codes beyond 2^32 bytes
    g = torch.Generator(device="cuda").manual_seed(3)
    pages, stride = 5, (1 << 32) // 4 + 4096
    flat = [torch.zeros(pages * stride, dtype=torch.int8, device="cuda") for _ in range(2)]
    k, v = (f.as_strided((pages, 16, 2, 64), (stride, 128, 64, 1)) for f in flat)
    sc = [torch.full((pages, 2, 1), 120, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache = ops.Kv8Cache(k, v, *sc)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    qkv = torch.randn((3, 6 * 64), generator=g, device="cuda")
    table = i32([[4]])
    ops.qk_norm_rope_kv8(qkv, 2, None, None, i32([0, 1, 2]), None, table, i32([0]), i32([0, 3]), cache)
    want_k, want_ks = torch.zeros((pages, 16, 2, 64), dtype=torch.float64, device="cuda"), sc[0].long() * 0 + 120
    ref.append(want_k, want_ks, qkv.view(3, 6, 64)[:, 2:4], table[0], 0, 3, 16)
    assert torch.equal(k.double(), want_k) and torch.equal(sc[0].long(), want_ks)
    got, _ = ops.dequantize_kv8(cache, F32)
    assert torch.equal(got.double(), ref.values(k, sc[0]))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("heads_first", [True, False])
def test_dequantize(ops, dtype, heads_first):
    s = Step(ops, [100], [1], Hkv=3, Hq=3, D=48, page=32, heads_first=heads_first)
    c = s.cache
    c.k_scale.view(-1)[:6] = torch.tensor([0, 1, 255, 254, 247, 112], dtype=torch.uint8, device="cuda")
    k, v = ops.dequantize_kv8(c, dtype)
    for got, codes, scales in ((k, c.k, c.k_scale), (v, c.v, c.v_scale)):
        assert got.is_contiguous() and torch.equal(got.double().nan_to_num(7e300), ref.values(codes, scales).to(dtype).double().nan_to_num(7e300))


def test_other_stream_and_graph(ops):
    s = Step(ops, [20, 3], [1, 1], Hq=4, Hkv=2, D=64)
    before = s.state()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    q = s.run(ops, stream=st)
    st.synchronize()
    x = s.qkv.view(2, 8, 64)
    same(s.state(), s.appended(before, x[:, 4:6], x[:, 6:8]))
    assert torch.equal(q, x[:, :4].to(BF16))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run(ops)
    s.qkv.mul_(3.0)
    before = s.state()
    g.replay()
    torch.cuda.synchronize()
    same(s.state(), s.appended(before, x[:, 4:6], x[:, 6:8]))
    assert ops.device_status() == 0 and math.isfinite(1.0)


@pytest.mark.parametrize("cols", (1, 5, 8))
def test_one_wider_row(ops, cols):
    """The stride of a lone row is not looked at, whatever its width."""
    a, b = (Step(ops, [20], [1], inp=BF16, seed=4) for _ in range(2))
    b.qkv = torch.cat([b.qkv, torch.full((1, cols), math.nan, dtype=BF16, device="cuda")], 1)
    assert torch.equal(a.run(ops), b.run(ops))
    for x, y in zip(a.state(), b.state()):
        assert torch.equal(x, y)
