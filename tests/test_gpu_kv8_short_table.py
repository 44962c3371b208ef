"""Requests longer than their block table: positions are those of the request, so a window reaches back from
there, keys beyond the table are not seen, and new tokens beyond it are not stored."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from tests.test_gpu_attention_kv8 import BF16, F16, Batch, ops  # noqa: E402, F401


def shorten(b, columns):
    b.table = b.table[:, :columns].contiguous()
    return b


@pytest.mark.parametrize("new", [1, 5, 70])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 0), (40, 3), (300, 20), (1000, 0), (1, 1), (90, 100)])
def test_window_over_a_short_table(ops, window, sinks, new):  # noqa: F811
    # 96 of about 400 keys on the table, and 96 of 110: the window ends beyond the table, or in it
    for page, columns in ((16, 6), (32, 3)):
        b = shorten(Batch(ops, [400, 110 - new, 90], [new, new, 3], 4, 2, 64, page, F16, seed=window + new), columns)
        b.check(b.run(ops, window, sinks), window, sinks)


@pytest.mark.parametrize("new", [2, 40])
def test_a_window_beyond_the_table_sees_nothing(ops, new):  # noqa: F811
    b = shorten(Batch(ops, [500], [new], 4, 2, 128, 32, BF16), 4)
    assert (b.run(ops, window=128) == 0).all()
    b.check(b.run(ops, window=128, sinks=5), 128, 5)
    b.check(b.run(ops))


def test_new_tokens_beyond_the_table_are_not_stored(ops):  # noqa: F811
    from w4a16_int4_quantized_gb300 import ops as o
    b = Batch(ops, [300, 60, 61, 64], [5, 3, 8, 20], 4, 2, 64, 32, seed=2)
    shorten(b, 2)      # 64 tokens: requests 0 and 3 begin beyond it, request 2 crosses its end
    c = b.cache
    before = [t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale)]
    qkv = torch.randn((36, 8 * 64), device="cuda")
    pos = torch.arange(36, dtype=torch.int32, device="cuda")
    o.qk_norm_rope_kv8(qkv, 4, None, None, pos, None, b.table, b.ctx, b.cu, c)
    free = set(range(c.k.shape[0])) - {int(b.table[1, 1]), int(b.table[2, 1])}
    for t, old in zip((c.k, c.v, c.k_scale, c.v_scale), before):
        assert torch.equal(t[sorted(free)], old[sorted(free)])
    got, _ = o.dequantize_kv8(c, torch.float32)
    for r, t0, lo, n in ((1, 5, 60, 3), (2, 8, 61, 3)):
        page = int(b.table[r, 1])
        x = qkv[t0: t0 + n, 4 * 64: 6 * 64].reshape(n, 2, 64)
        step = torch.exp2(c.k_scale[page, :, 1].float() - 127)[None, :, None]
        assert ((got[page, lo - 32: lo - 32 + n] - x).abs() <= step / 2).all()
