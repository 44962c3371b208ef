"""w4_attention_kv8 over batches of requests of very different lengths, with parts of many steps to a CTA:
prompts whose last row tile is not full, one after another, and beside decode tokens.  Scales differ from block
to block by up to 2^5, so that a block's scale taken for another's shows; limits as in test_gpu_attention_kv8.py."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from tests import kv8_reference as ref  # noqa: E402
from tests.test_gpu_attention_kv8 import BF16, F16, U, Batch, ops  # noqa: E402, F401


def long_reference(b, window=0, sinks=0):
    """kv8_reference.attention for long contexts: a key head at a time, all of its rows in one product."""
    c, dev = b.cache, b.q.device
    kv, vv = ref.values(c.k, c.k_scale), ref.values(c.v, c.v_scale)
    T, Hq, D = b.q.shape
    H = kv.shape[2]
    G = Hq // H
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=dev)
    vmax, smax = (torch.zeros((T, Hq), dtype=torch.float64, device=dev) for _ in range(2))
    ctx, cu, table = b.ctx.tolist(), b.cu.tolist(), b.table.cpu()
    for i, n0 in enumerate(ctx):
        t0, n = cu[i], cu[i + 1] - cu[i]
        k, ok = ref.rows_of(kv, table[i], n0 + n, b.page)
        v, _ = ref.rows_of(vv, table[i], n0 + n, b.page)
        assert ok.all()
        j = torch.arange(n0 + n, device=dev)
        for a in range(0, n, 512):
            m = min(512, n - a)
            back = (n0 + a + torch.arange(m, device=dev))[:, None] - j
            see = back >= 0
            if window:
                see &= (back < window) | (j < sinks)
            see = see.repeat_interleave(G, 0)
            rows = slice(t0 + a, t0 + a + m)
            for h in range(H):
                q = b.q[rows, h * G:(h + 1) * G].double().reshape(m * G, D)
                s = torch.where(see, q @ k[:, h].T * b.scale, -float("inf"))
                p = torch.exp(s - s.amax(-1, keepdim=True))
                o = p @ v[:, h] / p.sum(-1, keepdim=True)
                out[rows, h * G:(h + 1) * G] = o.reshape(m, G, D)
                size = torch.where(see, v[:, h].abs().amax(-1), 0.0).amax(-1)
                vmax[rows, h * G:(h + 1) * G] = size.reshape(m, G)
                size = torch.where(see, q.abs() @ k[:, h].abs().T * b.scale, 0.0).amax(-1)
                smax[rows, h * G:(h + 1) * G] = size.reshape(m, G)
    return out, vmax, smax


def check(ops, b, **kw):  # noqa: F811
    got = b.run(ops, **kw)
    for _ in range(2):
        assert torch.equal(b.run(ops, **kw), got)
    want, v, s = long_reference(b, **kw)
    bound = ((U[b.q.dtype] + 2.0 ** -11 + 2.0 ** -17 * (s + 1)) * v)[..., None] + 2.0 ** -25
    bad = (got.double() - want).abs() > bound
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:8].tolist())
    assert ops.device_status() == 0


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,page", [
    # 384 rows a key head: a full pair of tiles, then half of one; 216 steps a CTA
    ([4000] * 32, [96] * 32, 32, 8, 128, 64),
    # prompts from their beginning, the last tokens a tile of their own
    ([0] * 8, [1056] * 8, 32, 8, 128, 32),
    # decode tokens over long contexts before a prompt, and in turn with prompts
    ([6000, 6000], [1, 2048], 32, 8, 128, 64), ([1040, 1040], [1, 1040], 32, 8, 128, 16),
    ([16000, 0] * 8, [1, 300] * 8, 32, 8, 128, 64), ([9001, 17, 6000, 5, 4000] * 4, [2, 400, 1, 33, 70] * 4, 28, 4, 64, 32),
    # the same with one row tile to a CTA: 256 values, and 128 rows at most
    ([5000, 0, 3000] * 3, [1, 150, 9] * 3, 16, 4, 256, 64), ([8000, 100, 3000] * 4, [1, 32, 7] * 4, 32, 8, 128, 64)])
def test_ragged_batches(ops, dtype, ctx, new, Hq, Hkv, D, page):  # noqa: F811
    b = Batch(ops, ctx, new, Hq, Hkv, D, page, dtype, seed=len(ctx) + D, scales=(119, 125))
    check(ops, b)


@pytest.mark.parametrize("window,sinks", [(700, 4), (4096, 100)])
def test_ragged_batches_through_a_window(ops, window, sinks):  # noqa: F811
    b = Batch(ops, [16000, 0, 9000, 3000] * 6, [1, 300, 70, 600] * 6, 32, 8, 128, 64, BF16, seed=window, scales=(119, 125))
    check(ops, b, window=window, sinks=sinks)


def test_a_missing_block_of_the_decode_token_is_not_the_prompts(ops):  # noqa: F811
    # pages outside the cache and blocks of NaN in requests whose segments a tile skips: the prompts behind them stay
    b = Batch(ops, [12000, 0] * 6, [1, 300] * 6, 32, 8, 128, 64, BF16, seed=11, scales=(119, 125))
    want = b.run(ops)
    for i in range(0, 12, 2):
        b.table[i, ::2] = -1
        for page in b.table[i, 1::2].tolist():
            if page >= 0:
                b.cache.v_scale[page] = 255
    got = b.run(ops)
    cu = b.cu.tolist()
    prompt = torch.zeros(cu[-1], dtype=torch.bool, device="cuda")
    for i in range(1, 12, 2):
        prompt[cu[i]: cu[i + 1]] = True
    assert got[~prompt].isnan().all()
    # (the line of all steps is cut by lengths alone: the same bits)
    assert torch.equal(got[prompt], want[prompt])
