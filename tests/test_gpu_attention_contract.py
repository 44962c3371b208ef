"""GPU tests of what include/w4.h says of w4_tree_attention beyond ordinary inputs.

Tolerances: u is the unit roundoff of the output type, A = sum p |v| / sum p.  As in
test_gpu_draft.py: the output's rounding (u |o|), that of each p (u A), 2e-3 A for the
f32 scores.  A weight below f16's normal numbers is rounded by at most 2^-32 of the
largest weight: L keys together 2^-32 L max |v|.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


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


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("requests", [304, 1])   # a unit to a CTA, or cut into many
@pytest.mark.parametrize("at", [0, 15000])
@pytest.mark.parametrize("drop", [25.5, 20.25, 30.0])
def test_long_tail_beside_a_dominant_key(ops, dtype, requests, at, drop):
    """One key at weight 1 with value 0 and 30,000 at weight 2^-drop with value 1: the output is the tail's share."""
    L, page, D = 30000, 64, 64
    pages = -(-L // page)
    k = torch.zeros((pages, page, 1, D), dtype=dtype, device="cuda")
    v = torch.ones((pages, page, 1, D), dtype=dtype, device="cuda")
    k[..., 0] = -drop
    k[at // page, at % page], v[at // page, at % page] = 0, 0
    q = torch.zeros((requests, 1, D), dtype=dtype, device="cuda")
    q[..., 0] = 1
    table = torch.arange(pages, device="cuda", dtype=torch.int32).repeat(requests, 1)  # all read the same pages
    cu = torch.arange(requests + 1, device="cuda", dtype=torch.int32)
    mask = torch.zeros((requests, 4), dtype=torch.int32, device="cuda")
    mask[:, 0] = 1
    out = ops.tree_attention(q, k, v, table, i32([L - 1] * requests), cu, mask, math.log(2.0), L, 1).double()
    tail = (L - 1) * 2.0 ** -drop
    want = tail / (1 + tail)
    tol = U[dtype] * 2 * want * 1.01 + 2e-3 * want + 2.0 ** -32 * L + 1e-7
    if dtype == torch.float16:
        tol += 2.0 ** -25  # a subnormal output's rounding
    assert float((out - want).abs().max()) <= tol
    assert ops.device_status() == 0


# ---------------------------------------------------------------- bounds, pages and tokens at the edges

from tests.test_gpu_draft import attention_inputs, attention_reference  # noqa: E402


def close(out, want, size, dtype):
    tol = U[dtype] * (want.abs() + size) * 1.01 + 2e-3 * size + 1e-7
    return bool(((out.double() - want).abs() <= tol).all())


def run(ops, args, T, Hq, D, max_len, max_new):
    """The call into the middle of a larger buffer: (output rows, everything around them untouched)."""
    q, k, v, table, c, cu, mask = args
    buf = torch.full((T + 4, Hq, D), 9.0, dtype=q.dtype, device="cuda")
    ws = torch.full((ops.tree_attention_workspace_bytes(len(c), Hq, k.shape[2], D, max_len, max_new),), 255,
                    dtype=torch.uint8, device="cuda")
    out = ops.tree_attention(q[:T], k, v, table, c, cu, mask, 1 / math.sqrt(D), max_len, max_new, out=buf[2:T + 2],
                             workspace=ws)
    assert ops.device_status() == 0
    return out, bool((buf[:2] == 9).all()) and bool((buf[T + 2:] == 9).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("ctx,new,max_new", [([100, 40], [20, 5], 7), ([300, 2], [60, 90], 37), ([5], [3], 1),
                                             ([2000, 70], [128, 1], 100)])
def test_tokens_beyond_max_new_get_no_output(ops, ctx, new, max_new, dtype):
    Hq, Hkv, D, page = 8, 1, 64, 16
    args = attention_inputs(ops, ctx, new, Hq, Hkv, D, page, dtype, "dense", 3)
    T = sum(new)
    out, clean = run(ops, args, T, Hq, D, max(a + b for a, b in zip(ctx, new)), max_new)
    want, size = attention_reference(*args[:4], ctx, args[5].tolist(), args[6], 1 / math.sqrt(D), page)
    i = torch.cat([torch.arange(n, device="cuda") for n in new])
    assert clean and close(out[i < max_new], want[i < max_new], size[i < max_new], dtype)
    assert bool((out[i >= max_new] == 9).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("ctx,new,max_len", [([3000, 50], [4, 9], 64), ([700], [70], 1), ([9000], [1], 300)])
def test_request_longer_than_max_len_is_read_whole(ops, ctx, new, max_len, dtype):
    Hq, Hkv, D, page = 8, 2, 128, 32
    args = attention_inputs(ops, ctx, new, Hq, Hkv, D, page, dtype, "heads_first", 5)
    out, clean = run(ops, args, sum(new), Hq, D, max_len, max(new))
    want, size = attention_reference(*args[:4], ctx, args[5].tolist(), args[6], 1 / math.sqrt(D), page)
    assert clean and close(out, want, size, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("page", [8, 16, 64, 128])
def test_page_outside_the_cache_reads_as_zeros(ops, page, dtype):
    ctx, new, Hq, Hkv, D = [500, 33], [9, 40], 4, 2, 64
    q, k, v, table, c, cu, mask = attention_inputs(ops, ctx, new, Hq, Hkv, D, page, dtype, "dense", 7)
    P = k.shape[0]
    away = table.clone()
    last = (ctx[1] + new[1] - 1) // page
    for (b, j), bad in zip(((0, 0), (0, 3), (0, (ctx[0] + 8) // page), (1, last)), (-1, P, 2 ** 31 - 1, -2 ** 31)):
        away[b, j] = bad
    out, clean = run(ops, (q, k, v, away, c, cu, mask), sum(new), Hq, D, 509, 40)
    zero = torch.zeros((1,) + k.shape[1:], dtype=dtype, device="cuda")
    there = torch.where((away < 0) | (away >= P), P, away)
    want, size = attention_reference(q, torch.cat([k, zero]), torch.cat([v, zero]), there, ctx, cu.tolist(), mask,
                                     1 / math.sqrt(D), page)
    assert clean and close(out, want, size, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("new", [[3, 0, 20], [70, 5, 1]])
def test_tokens_behind_the_last_request(ops, new, dtype):
    """Rows of q at and after cu_new[B] are not written; cu_new past T counts as T."""
    ctx, Hq, Hkv, D, page = [40, 7, 200], 4, 1, 64, 16
    args = list(attention_inputs(ops, ctx, new, Hq, Hkv, D, page, dtype, "dense", 9))
    n = sum(new)
    want, size = attention_reference(*args[:4], ctx, args[5].tolist(), args[6], 1 / math.sqrt(D), page)
    wide = list(args)
    wide[0] = torch.cat([args[0], torch.full((11, Hq, D), float("nan"), dtype=dtype, device="cuda")])
    wide[6] = torch.cat([args[6], torch.full((11, 4), -1, dtype=torch.int32, device="cuda")])
    out, clean = run(ops, wide, n + 11, Hq, D, 300, max(new))
    assert clean and close(out[:n], want, size, dtype) and bool((out[n:] == 9).all())
    out, clean = run(ops, args, n - 1, Hq, D, 300, max(new))
    short = args[5].clamp(max=n - 1)
    want, size = attention_reference(args[0], *args[1:4], ctx, short.tolist(), args[6], 1 / math.sqrt(D), page)
    assert clean and close(out, want[:n - 1], size[:n - 1], dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_scores_of_minus_infinity_alone(ops, dtype):
    ctx, new, Hq, Hkv, D, page = [90], [20], 4, 2, 64, 16
    q, k, v, table, c, cu, mask = attention_inputs(ops, ctx, new, Hq, Hkv, D, page, dtype, "dense", 13)
    q = q.abs() + 0.5
    k.fill_(-float("inf"))
    out, clean = run(ops, (q, k, v, table, c, cu, mask), 20, Hq, D, 110, 20)
    assert clean and bool((out == 0).all())
