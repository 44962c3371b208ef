"""GPU tests of the step of drafted tokens: the plan (exact), head norms with the
rotation and the cache store, and tree attention, against plain definitions in
64 bits.

Tolerances.  u is the unit roundoff of the output type (2^-8 bf16, 2^-11 f16,
2^-24 f32).
  rope       one rounding (u |y|) of an f32 result: at most about 20 roundings of
             2^-24 relative to the pair's magnitude |a| + |b| <= 2 max|h|, the sum
             of squares (256 terms) included: 2^-18 max|h|.
  attention  with A = sum p |v| / sum p: the output's rounding (u |o|), that of
             each p (u A), and the f32 scores: |s| stays below 40, its error
             below 256 * 2^-24 * 40 = 6e-4, so 2e-3 A covers p and sum p.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

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


def i32(a):
    return torch.tensor(np.asarray(a, dtype=np.int32)).cuda()


# ---------------------------------------------------------------- plan

def plan_reference(ctx, new, parents, free, table, page, cap):
    table = table.copy()
    width = table.shape[1]
    cu, slots, pos, mask, taken = [0], [], [], [], 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        c, n = max(int(c), 0), min(max(int(n), 0), 128)
        for blk in range(-(-c // page), min(-(-(c + n) // page), width)):
            table[b, blk] = free[taken] if taken < len(free) else -1
            taken += 1
        rows = []
        for i in range(n):
            t = cu[-1] + i
            p = i - 1 if parents is None else int(parents[t]) if t < cap else -1
            rows.append((1 << i) | (rows[p] if 0 <= p < i else 0))
            blk, off = divmod(c + i, page)
            pid = int(table[b, blk]) if blk < width else -1
            slots.append(pid * page + off if pid >= 0 else -1)
            pos.append(c + bin(rows[i]).count("1") - 1)
        mask += rows
        cu.append(cu[-1] + n)
    pad = cap - len(slots)
    slots, pos, mask = slots[:cap] + [-1] * pad, pos[:cap] + [0] * pad, mask[:cap] + [0] * pad
    words = np.array([[(r >> (32 * w)) & 0xFFFFFFFF for w in range(4)] for r in mask], np.uint32).reshape(cap, 4)
    return cu, table, slots, pos, words.view(np.int32), taken


PLANS = [
    # ctx, new, page, width, free pages, capacity beyond the tokens
    ([0], [1], 16, 1, 1, 0),
    ([5, 0, 16, 31], [3, 0, 1, 128], 16, 12, 40, 5),
    ([7] * 9, [128] * 9, 8, 20, 200, 0),                  # more requests than one block holds
    (list(range(100, 137)), list(range(37)), 64, 4, 50, 11),
    ([3, 1000, 17], [64, 64, 64], 16, 64, 2, 0),          # free pages run out
    ([30, 31, 40], [9, 9, 9], 16, 2, 9, 0),               # the table is too narrow
    ([-4, 10], [-3, 200], 16, 16, 20, 0),                 # lengths that are clamped
    ([12, 1], [5, 6], 7, 9, 9, 3),                        # a page size that is no power of two
]


@pytest.mark.parametrize("ctx,new,page,width,n_free,more", PLANS)
@pytest.mark.parametrize("kind", ["tree", "chain", "none", "junk"])
def test_plan(ops, ctx, new, page, width, n_free, more, kind):
    g = np.random.default_rng(len(ctx) * 7 + page)
    B, total = len(ctx), sum(min(max(n, 0), 128) for n in new)
    cap = total + more
    table = np.full((B, width), -1, np.int32)
    ids = g.permutation(B * width + n_free).astype(np.int32)
    for b, c in enumerate(ctx):
        h = min(-(-max(c, 0) // page), width)
        table[b, :h] = ids[b * width: b * width + h]
    free = ids[B * width:]
    parents = None
    if kind != "none":
        parents = np.full(cap, -1, np.int32)
        at = 0
        for n in new:
            n = min(max(n, 0), 128)
            i = np.arange(n)
            if kind == "chain":
                parents[at: at + n] = i - 1
            elif kind == "tree":
                parents[at: at + n] = np.maximum(i - 1 - g.integers(0, 5, n), -1)
            else:  # itself, later tokens, far out: all roots
                parents[at: at + n] = g.integers(-500, 500, n)
            at += n
    d_table = i32(table)
    got = ops.draft_plan(i32(ctx), i32(new), None if parents is None else i32(parents), i32(free), d_table, page,
                         max_tokens=cap)
    cu, want_table, slots, pos, mask, taken = plan_reference(ctx, new, parents, free, table, page, cap)
    assert got[0].tolist() == cu
    assert np.array_equal(d_table.cpu().numpy(), want_table)
    assert got[1].tolist() == slots and got[2].tolist() == pos
    assert np.array_equal(got[3].cpu().numpy(), mask)
    assert got[4].tolist() == [taken]
    again = ops.draft_plan(i32(ctx), i32(new), None if parents is None else i32(parents), i32(free), d_table, page,
                           max_tokens=cap)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_plan_capacity_too_small_and_no_requests(ops):
    table = i32(np.full((2, 4), -1))
    buf = torch.full((6,), 77, dtype=torch.int64, device="cuda")
    got = ops.draft_plan(i32([0, 0]), i32([4, 4]), None, i32([3, 2, 1]), table, 16, max_tokens=5)
    assert got[0].tolist() == [0, 4, 8] and got[1].tolist() == [48, 49, 50, 51, 32] and got[4].tolist() == [2]
    assert buf.tolist() == [77] * 6
    got = ops.draft_plan(i32([]), i32([]), None, i32([]), i32(np.zeros((0, 4))), 16, max_tokens=3)
    assert got[0].tolist() == [0] and got[1].tolist() == [-1] * 3 and got[2].tolist() == [0] * 3
    assert got[3].abs().sum().item() == 0 and got[4].tolist() == [0]


# ---------------------------------------------------------------- norm, rotation, store

def make_cache(P, page, H, D, dtype, layout, fill=0.0):
    if layout == "heads_first":
        return torch.full((P, H, page, D), fill, dtype=dtype, device="cuda").transpose(1, 2)
    if layout == "padded":  # strides larger than dense, tokens first
        return torch.full((P, page + 1, H + 1, D + 8), fill, dtype=dtype, device="cuda")[:, :page, :H, :D]
    return torch.full((P, page, H, D), fill, dtype=dtype, device="cuda")


def rope_reference(x, w, cos_sin, pos, inter, eps):
    """x [T, H, D] f64 -> normed and rotated."""
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    if cos_sin is None:
        return x
    R = cos_sin.shape[1]
    cs = cos_sin.double()[pos.long()][:, None]
    c, s = cs[..., : R // 2], cs[..., R // 2:]
    y = x.clone()
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if inter else (x[..., : R // 2], x[..., R // 2: R])
    ya, yb = a * c - b * s, b * c + a * s
    if inter:
        y[..., 0:R:2], y[..., 1:R:2] = ya, yb
    else:
        y[..., : R // 2], y[..., R // 2: R] = ya, yb
    return y


def close_rope(got, want, dtype):
    tol = U[dtype] * want.abs() + 2.0 ** -18 * want.abs().amax() + 1e-30
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25  # subnormal outputs
    return bool(((got.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("T,Hq,Hkv,D,R,layout", [
    (1, 1, 1, 64, 64, "dense"), (3, 4, 2, 128, 128, "heads_first"), (37, 7, 1, 80, 80, "dense"),
    (5, 6, 3, 96, 32, "padded"), (130, 14, 2, 256, 256, "heads_first"), (9, 5, 5, 8, 0, "dense"),
    (2, 3, 1, 32, 16, "padded"), (11, 2, 2, 200, 48, "dense")])
@pytest.mark.parametrize("inp,out", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.bfloat16),
                                     (torch.float16, torch.float16), (torch.float32, torch.float32),
                                     (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("inter", [False, True])
def test_qk_norm_rope(ops, T, Hq, Hkv, D, R, layout, inp, out, inter):
    gen = torch.Generator(device="cuda").manual_seed(T * 1000 + D + R)
    page, P, eps = 16, T // 16 + 3, 1e-5
    cols = (Hq + 2 * Hkv) * D
    big = torch.randn((T, cols + 16), generator=gen, device="cuda").mul_(3).to(inp)  # rows wider than the heads
    qkv = big[:, :cols]
    wq = 1 + 0.3 * torch.randn(D, generator=gen, device="cuda")
    wk = 1 + 0.3 * torch.randn(D, generator=gen, device="cuda")
    pos = torch.randint(0, 50, (T,), generator=gen, device="cuda", dtype=torch.int32)
    ang = torch.randn((50, max(R // 2, 1)), generator=gen, device="cuda") * 9
    cos_sin = torch.cat([ang.cos(), ang.sin()], 1).contiguous() if R else None
    slots = torch.randperm(P * page, generator=gen, device="cuda")[:T].contiguous()
    skip = T > 4  # some tokens without a place, some with a slot outside the cache
    if skip:
        slots[1], slots[3] = -1, P * page
    kc, vc = (make_cache(P, page, Hkv, D, out, layout, fill=5.0) for _ in range(2))
    q = ops.qk_norm_rope(qkv, Hq, wq, wk, pos, cos_sin, slots, kc, vc, eps=eps, interleaved=inter)
    x = qkv.double().view(T, Hq + 2 * Hkv, D)
    assert close_rope(q, rope_reference(x[:, :Hq], wq, cos_sin, pos, inter, eps), out)
    kept = torch.ones(T, dtype=torch.bool, device="cuda")
    if skip:
        kept[1] = kept[3] = False
    pg, off = slots[kept] // page, slots[kept] % page
    want = rope_reference(x[:, Hq: Hq + Hkv], wk, cos_sin, pos, inter, eps)[kept]
    assert close_rope(kc[pg, off], want, out)
    assert torch.equal(vc[pg, off], qkv.view(T, -1)[:, (Hq + Hkv) * D:].reshape(T, Hkv, D).to(out)[kept])
    rest = torch.ones((P, page), dtype=torch.bool, device="cuda")
    rest[pg, off] = False
    assert bool((kc[rest] == 5).all()) and bool((vc[rest] == 5).all())
    if layout == "padded":  # nothing between the rows is touched
        assert bool((kc._base[:, page:] == 5).all()) and bool((vc._base[..., D:] == 5).all())


def test_qk_norm_rope_without_norm_and_left_out_tokens(ops):
    T, Hq, Hkv, D = 6, 2, 1, 64
    qkv = torch.randn((T, (Hq + 2 * Hkv) * D), device="cuda").bfloat16()
    cos_sin = torch.ones((4, D), device="cuda")
    pos = i32([0, 3, 4, -1, 2, 1])
    slots = torch.arange(T, device="cuda")
    kc, vc = (make_cache(1, 16, Hkv, D, torch.bfloat16, "dense", 9.0) for _ in range(2))
    q = torch.full((T, Hq, D), 9.0, dtype=torch.bfloat16, device="cuda")
    ops.qk_norm_rope(qkv, Hq, None, None, pos, cos_sin, slots, kc, vc, out=q)
    assert bool((q[2:4] == 9).all()) and bool((kc[0, 2:4] == 9).all()) and bool((vc[0, 2:4] == 9).all())
    x = qkv.double().view(T, Hq + 2 * Hkv, D)
    keep = [0, 1, 4, 5]
    want = rope_reference(x, None, cos_sin, pos.clamp(0, 3), False, 0.0)
    assert close_rope(q[keep], want[keep, :Hq], torch.bfloat16)
    assert close_rope(kc[0, keep], want[keep, Hq: Hq + 1], torch.bfloat16)
    zero = ops.qk_norm_rope(torch.zeros_like(qkv), Hq, torch.ones(D, device="cuda"), torch.ones(D, device="cuda"), pos,
                            cos_sin, slots, kc, vc, eps=1e-6)
    assert bool((zero[keep] == 0).all())


# ---------------------------------------------------------------- attention

def attention_reference(q, k, v, table, ctx, cu, mask, scale, page):
    """(out, A) in f64: A = sum p |v| / sum p per output value."""
    Hq, Hkv, D = q.shape[1], k.shape[2], q.shape[2]
    G = Hq // Hkv
    out, size = (torch.zeros(q.shape, dtype=torch.float64, device=q.device) for _ in range(2))
    bits = ((mask.long()[:, :, None] >> torch.arange(32, device=q.device)) & 1).view(-1, 128).bool()
    for b, c in enumerate(ctx):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        key = torch.arange(c + n, device=q.device)
        pid = table[b].long()[key // page]
        kk, vv = k[pid, key % page].double(), v[pid, key % page].double()
        for i in range(n):
            t = cu[b] + i
            see = torch.cat([torch.ones(c, dtype=torch.bool, device=q.device), bits[t, :n]])
            if not bool(see.any()):
                continue
            ks, vs = kk[see].repeat_interleave(G, 1), vv[see].repeat_interleave(G, 1)
            s = torch.einsum("hd,lhd->hl", q[t].double(), ks) * scale
            p = torch.softmax(s, -1)
            out[t] = torch.einsum("hl,lhd->hd", p, vs)
            size[t] = torch.einsum("hl,lhd->hd", p, vs.abs())
    return out, size


def attention_inputs(ops, ctx, new, Hq, Hkv, D, page, dtype, layout, seed, spare=2):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    g = np.random.default_rng(seed)
    B = len(ctx)
    need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    P, width = sum(need) + spare, max(max(need), 1)
    ids = g.permutation(P).astype(np.int32)
    table = np.full((B, width), -1, np.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = ids[at: at + m]
        at += m
    parents = np.concatenate([np.maximum(np.arange(n) - 1 - g.integers(0, 4, n), -1) for n in new]).astype(np.int32)
    d_table = i32(table)
    cu, slots, pos, mask, taken = ops.draft_plan(i32(ctx), i32(new), i32(parents), i32(ids), d_table, page)
    d_table = i32(table)  # the pages are all there already
    T = int(sum(new))
    q = (1.5 * torch.randn((T, Hq, D), generator=gen, device="cuda")).to(dtype)
    k, v = (make_cache(P, page, Hkv, D, dtype, layout) for _ in range(2))
    k.copy_(torch.randn(k.shape, generator=gen, device="cuda"))
    v.copy_(torch.randn(v.shape, generator=gen, device="cuda"))
    return q, k, v, d_table, i32(ctx), cu, mask


def check_attention(ops, ctx, new, Hq, Hkv, D, page, dtype, layout, seed, args=None, max_len=None, max_new=None):
    q, k, v, table, c, cu, mask = args or attention_inputs(ops, ctx, new, Hq, Hkv, D, page, dtype, layout, seed)
    scale = 1 / math.sqrt(D)
    max_len, max_new = max_len or max(a + b for a, b in zip(ctx, new)), max_new or max(new)
    # what the workspace holds before the call does not matter: NaN
    ws = torch.full((ops.tree_attention_workspace_bytes(len(ctx), Hq, Hkv, D, max_len, max_new),), 255,
                    dtype=torch.uint8, device="cuda")
    out = ops.tree_attention(q, k, v, table, c, cu, mask, scale, max_len, max_new, workspace=ws)
    want, size = attention_reference(q, k, v, table, ctx, cu.tolist(), mask, scale, page)
    err = (out.double() - want).abs()
    tol = U[dtype] * (want.abs() + size) * 1.01 + 2e-3 * size + 1e-7
    assert bool(torch.isfinite(out).all())
    assert bool((err <= tol).all()), float((err / tol).max())
    assert ops.device_status() == 0
    return out


CASES = [
    # ctx, new, Hq, Hkv, D, page
    ([0], [1], 1, 1, 64, 16),
    ([1], [1], 4, 1, 64, 16),
    ([63], [1], 8, 2, 128, 16),
    ([64], [1], 8, 2, 128, 64),
    ([127, 1, 0], [1, 3, 2], 4, 4, 128, 32),
    ([500, 77, 1025], [17, 64, 5], 14, 2, 128, 16),
    ([200], [128], 8, 1, 64, 128),                        # 8 row tiles
    ([33, 0, 90], [0, 128, 31], 6, 3, 80, 16),            # a request without drafted tokens
    ([129, 300], [33, 40], 5, 1, 96, 8),
    ([257, 3], [20, 100], 4, 2, 256, 16),
    ([100], [9], 2, 2, 40, 256),
    ([700], [3], 128, 1, 64, 32),                         # 128 query heads to a key head
    ([65], [128], 1, 1, 32, 64),
    ([4000, 1], [6, 2], 8, 2, 128, 16),                   # split over keys, one request much shorter
]


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,page", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("layout", ["dense", "heads_first", "padded"])
def test_tree_attention(ops, ctx, new, Hq, Hkv, D, page, dtype, layout):
    check_attention(ops, ctx, new, Hq, Hkv, D, page, dtype, layout, seed=len(ctx) + D + page)


@pytest.mark.parametrize("ctx,new", [([20000], [1]), ([9001], [70]), ([6000] * 5, [8, 1, 0, 64, 3])])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_tree_attention_long(ops, ctx, new, dtype):
    check_attention(ops, ctx, new, 8, 2, 128, 32, dtype, "heads_first", seed=ctx[0])


def test_bounds_larger_than_the_lengths(ops):
    """max_len and max_new are bounds: more than the lengths changes only the split of the work."""
    check_attention(ops, [100, 900], [5, 2], 8, 2, 128, 16, torch.bfloat16, "dense", 3, max_len=9000, max_new=128)


def test_many_requests(ops):
    """More requests than a block has threads, most of them short, some without drafted tokens."""
    g = np.random.default_rng(9)
    ctx = g.integers(0, 70, 600).tolist()
    new = g.integers(0, 3, 600).tolist()
    ctx[17], new[17], ctx[599], new[599] = 1500, 9, 800, 5
    check_attention(ops, ctx, new, 2, 1, 64, 16, torch.float16, "dense", 4)
    new[300] = 100  # two row tiles
    check_attention(ops, ctx, new, 2, 1, 64, 16, torch.float16, "dense", 5)


def test_rows_that_see_nothing_or_little(ops):
    ctx, new = [0, 70], [40, 66]
    args = list(attention_inputs(ops, ctx, new, 4, 2, 64, 16, torch.bfloat16, "dense", 5))
    mask = torch.zeros_like(args[6])
    mask[1, 0] = 1          # token 1 sees token 0 alone
    mask[2, 1] = 1 << 7     # token 39, a later one: any mask is taken as it stands
    mask[50, 3] = -1        # bits past the request's drafted tokens mean nothing
    args[6] = mask
    out = check_attention(ops, ctx, new, 4, 2, 64, 16, torch.bfloat16, "dense", 5, args=args)
    assert bool((out[0] == 0).all()) and bool((out[3:40] == 0).all()) and bool((out[1:3] != 0).any())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("ctx,D", [(70, 128), (0, 64), (3000, 64), (61, 256)])
def test_what_is_not_seen_does_not_matter(ops, bad, dtype, ctx, D):
    """NaN and infinities behind the request's end and in drafted tokens off a row's path."""
    n, page = 37, 16
    q, k, v, table, c, cu, mask = attention_inputs(ops, [ctx], [n], 4, 2, D, page, dtype, "heads_first", 11)
    clean = ops.tree_attention(q, k, v, table, c, cu, mask, 0.1, ctx + n, n)
    used = torch.zeros(k.shape[:2], dtype=torch.bool, device="cuda")
    key = torch.arange(ctx + n, device="cuda")
    used[table[0].long()[key // page], key % page] = True
    k[~used], v[~used] = bad, bad
    out = ops.tree_attention(q, k, v, table, c, cu, mask, 0.1, ctx + n, n)
    assert torch.equal(out, clean)
    # drafted token 20 gets a bad key and a bad value: rows that do not see it keep their bits, rows that do show it
    j = ctx + 20
    pg, off = int(table[0, j // page]), j % page
    v[pg, off, :, 3] = bad
    out = ops.tree_attention(q, k, v, table, c, cu, mask, 0.1, ctx + n, n)
    sees = ((mask[:, 0] >> 20) & 1).bool()
    assert 0 < int(sees.sum()) < n
    assert torch.equal(out[~sees], clean[~sees])
    assert bool((~torch.isfinite(out[sees][:, :, 3])).all())
    if math.isinf(bad):
        assert bool((out[sees][:, :, 3] == bad).all())
    rest = [d for d in range(D) if d != 3]
    assert torch.equal(out[sees][:, :, rest], clean[sees][:, :, rest])
    k[pg, off] = bad
    out = ops.tree_attention(q, k, v, table, c, cu, mask, 0.1, ctx + n, n)
    assert torch.equal(out[~sees], clean[~sees])
    assert ops.device_status() == 0


def test_large_scores_and_growing_maxima(ops):
    """Scores that climb along the context, so that the running maximum is renewed many times."""
    ctx, new, D = [1500], [5], 64
    q, k, v, table, c, cu, mask = attention_inputs(ops, ctx, new, 2, 1, D, 16, torch.float16, "dense", 21)
    key = torch.arange(1505, device="cuda")
    rows = (table[0].long()[key // 16], key % 16)
    k[rows] = (k[rows].float() * 0.1 + (key[:, None, None] / 1505.0) * 4 * torch.sign(q[0, :1].float())).half()
    check_attention(ops, ctx, new, 2, 1, D, 16, torch.float16, "dense", 21, args=(q, k, v, table, c, cu, mask))


def test_strided_queries_streams_and_repeats(ops):
    ctx, new = [300, 2000], [9, 30]
    q, k, v, table, c, cu, mask = attention_inputs(ops, ctx, new, 8, 2, 128, 32, torch.bfloat16, "dense", 31)
    base = ops.tree_attention(q, k, v, table, c, cu, mask, 0.09, 2030, 30)
    wide = torch.zeros((39, 3, 8, 128), dtype=torch.bfloat16, device="cuda")
    wide[:, 1] = q
    assert torch.equal(ops.tree_attention(wide[:, 1], k, v, table, c, cu, mask, 0.09, 2030, 30), base)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        outs = [ops.tree_attention(q, k, v, table, c, cu, mask, 0.09, 2030, 30) for _ in range(20)]
    st.synchronize()
    assert all(torch.equal(o, base) for o in outs)
    # a stream by argument: the workspace of the call is not handed out again before it is through
    for _ in range(20):
        o = ops.tree_attention(q, k, v, table, c, cu, mask, 0.09, 2030, 30, stream=st)
        junk = torch.full((ops.tree_attention_workspace_bytes(2, 8, 2, 128, 2030, 30),), 255, dtype=torch.uint8, device="cuda")
        st.synchronize()
        assert torch.equal(o, base)
    del junk


def test_cache_beyond_32_bit_offsets(ops):
    """Pages whose elements lie past 2^32 from the cache's start."""
    page, Hkv, D = 64, 8, 128
    P = (1 << 32) // (page * Hkv * D) + 40
    if torch.cuda.mem_get_info()[0] < 3 * P * page * Hkv * D * 2:
        pytest.skip("needs about 26 GB of device memory")
    k = torch.empty((P, page, Hkv, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    n_ctx, n = 1000, 4
    ids = torch.arange(P - 17, P, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(4)
    k[ids] = torch.randn((17, page, Hkv, D), generator=gen, device="cuda").bfloat16()
    v[ids] = torch.randn((17, page, Hkv, D), generator=gen, device="cuda").bfloat16()
    q = torch.randn((n, 16, D), generator=gen, device="cuda").bfloat16()
    table = ids.int().view(1, 17).contiguous()
    cu, slots, pos, mask, _ = ops.draft_plan(i32([n_ctx]), i32([n]), None, i32([]), table, page, max_tokens=n)
    qkv = torch.randn((n, (16 + 16) * D), generator=gen, device="cuda").bfloat16()
    w = torch.ones(D, device="cuda")
    cos_sin = torch.cat([torch.ones((2000, D // 2)), torch.zeros((2000, D // 2))], 1).cuda()
    ops.qk_norm_rope(qkv, 16, w, w, pos, cos_sin, slots, k, v)
    at = slots.tolist()
    assert torch.equal(v[at[0] // page, at[0] % page], qkv[0, 24 * D:].view(8, D))
    small_k, small_v = k[ids].clone(), v[ids].clone()
    small = torch.arange(17, device="cuda", dtype=torch.int32).view(1, 17)
    a = ops.tree_attention(q, k, v, table, i32([n_ctx]), cu, mask, 0.088, n_ctx + n, n)
    b = ops.tree_attention(q, small_k, small_v, small, i32([n_ctx]), cu, mask, 0.088, n_ctx + n, n)
    assert torch.equal(a, b)


def test_step_runs_together(ops):
    """plan -> norm, rotation and store -> attention, against the same step in 64 bits."""
    ctx, new, Hq, Hkv, D, page = [90, 5], [12, 7], 8, 2, 64, 16
    gen = torch.Generator(device="cuda").manual_seed(77)
    T = sum(new)
    k, v = (torch.randn((20, page, Hkv, D), generator=gen, device="cuda").bfloat16() for _ in range(2))
    table = np.full((2, 8), -1, np.int32)
    table[0, :6], table[1, :1] = [9, 4, 7, 0, 2, 11], [5]
    d_table = i32(table)
    parents = i32([-1, 0, 0, 1, 1, 2, 3, 3, 5, 8, 8, 4] + [-1, -1, 0, 1, 2, 2, 4])
    cu, slots, pos, mask, taken = ops.draft_plan(i32(ctx), i32(new), parents, i32([17, 18, 19]), d_table, page)
    assert taken.item() == 1 and d_table[0, 6].item() == 17
    qkv = torch.randn((T, (Hq + 2 * Hkv) * D), generator=gen, device="cuda")
    wq, wk = torch.rand(D, generator=gen, device="cuda") + 0.5, torch.rand(D, generator=gen, device="cuda") + 0.5
    ang = torch.arange(200, device="cuda")[:, None] * (10000.0 ** (-torch.arange(D // 2, device="cuda") / (D // 2)))
    cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
    q = ops.qk_norm_rope(qkv, Hq, wq, wk, pos, cos_sin, slots, k, v)
    check_attention(ops, ctx, new, Hq, Hkv, D, page, torch.bfloat16, "dense", 0,
                    args=(q, k, v, d_table, i32(ctx), cu, mask))
    x = qkv.double().view(T, -1, D)
    assert close_rope(q, rope_reference(x[:, :Hq], wq, cos_sin, pos, False, 1e-6), torch.bfloat16)
    assert close_rope(k[slots // page, slots % page], rope_reference(x[:, Hq: Hq + Hkv], wk, cos_sin, pos, False, 1e-6),
                      torch.bfloat16)
