"""w4_attention_kv8 at the ends of what bf16 queries and scale bytes hold; limits as in test_gpu_attention_kv8.py."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from tests import kv8_reference as ref  # noqa: E402
from tests.test_gpu_attention_kv8 import BF16, F16, Batch, ops  # noqa: E402, F401


@pytest.mark.parametrize("new", [3, 12, 80])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("up", [100, 116, 121, 124])
def test_large_queries_over_small_keys(ops, up, D, new):  # noqa: F811
    # scores of the usual size: keys 2^-up times as large
    b = Batch(ops, [300], [new], 4, 2, D, 16, BF16, seed=up, scales=(124 - up, 128 - up))
    b.cache.v_scale.fill_(120)
    b.q *= 2.0 ** up
    assert b.q.isfinite().all()
    b.check(b.run(ops))


@pytest.mark.parametrize("new", [3, 12, 80])
def test_small_queries_over_large_keys(ops, new):  # noqa: F811
    # rows whose largest value is below 2^-113 are taken to f16 with 2^126: off by 2^-151, times 64 values of 127 times
    # a scale of 2^98 at most: 2^-40
    b = Batch(ops, [300], [new], 4, 2, 64, 16, BF16, seed=new, scales=(223, 226))
    b.cache.v_scale.fill_(120)
    b.q *= 2.0 ** -104
    b.check(b.run(ops))
    b.q *= 2.0 ** -12
    b.check(b.run(ops))


@pytest.mark.parametrize("new", [3, 12, 80])
@pytest.mark.parametrize("up", [100, 110, 121])
def test_large_queries_over_usual_keys(ops, up, new):  # noqa: F811
    # one key far above the others for every row: all of the weight; and all keys alike: their mean
    b = Batch(ops, [200], [new], 4, 2, 64, 16, BF16, seed=up, scales=(120, 121))
    c = b.cache
    b.q.zero_()
    b.q[:, :, 5] = 2.0 ** up
    c.k[..., 5].clamp_(max=60)
    page = int(b.table[0, 3])
    c.k[page, 7, :, 5] = 120
    out = b.run(ops)
    want = (c.v[page, 7].double() * 2.0 ** (120 - 127)).repeat_interleave(2, 0)
    assert ((out.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -11) * want.abs().amax()).all()
    c.k.zero_()
    values = ref.values(c.v, c.v_scale)
    rows, _ = ref.rows_of(values, b.table[0].cpu(), 200 + new, 16)
    mean = rows.cumsum(0)[200:] / torch.arange(201, 201 + new, device="cuda", dtype=torch.float64)[:, None, None]
    out = b.run(ops)
    assert ((out.double() - mean.repeat_interleave(2, 1)).abs() <= 2.0 ** -8 * mean.abs().amax() + 2.0 ** -11 * rows.abs().amax()).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 12, 80])
def test_far_score_beside_blocks_without_one(ops, new, D, dtype):  # noqa: F811
    # a key of 2^63 times the others' size, and pages outside the cache, blocks of the least scale and keys
    # behind the rows beside it: that key's value, whichever block it lies in
    for block in range(13):
        b = Batch(ops, [200], [new], 4, 2, D, 16, dtype, seed=block, scales=(120, 121))
        c = b.cache
        b.q.zero_()
        b.q[:, :, 5] = 1.0
        c.k[..., 5].clamp_(max=60)
        page = int(b.table[0, block])
        c.k[page, 7, :, 5] = 120
        c.k_scale[page] = 190
        want = (c.v[page, 7].double() * 2.0 ** (120 - 127)).repeat_interleave(2, 0)
        for other in range(13):
            if other != block and other % 2 != block % 2:
                b.table[0, other] = -1
            elif other != block:
                c.k_scale[int(b.table[0, other])] = 0
        out = b.run(ops)
        rows = max(0, 16 * block + 7 - 200)     # those before the key do not see it
        assert ((out.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -11) * want.abs().amax())[rows:].all(), block
        assert out.isfinite().all()


@pytest.mark.parametrize("new", [1, 12, 80])
@pytest.mark.parametrize("up", [22, 40, 90])
def test_weight_of_a_score_near_a_far_one(ops, up, new):  # noqa: F811
    # scores 2^(up + 6) and a d-th less: the second has a weight of 2^(-2^21 d) at most; in the output, which is
    # rounded to 2^-9 of it, (100 - 100 w) / (1 + w)
    for low in (11, 13, 14, 15):
        d = 2.0 ** -(low + 6)
        b = Batch(ops, [60], [new], 2, 1, 64, 16, BF16, seed=low)
        c, p0, p1 = b.cache, int(b.table[0, 0]), int(b.table[0, 2])
        b.scale = 1.0
        b.q.zero_(), c.k.zero_(), c.k_scale.fill_(127), c.v.zero_(), c.v_scale.fill_(127)
        b.q[:, :, 5], b.q[:, :, 6] = 2.0 ** up, 2.0 ** (up - low)
        c.k[p0, 3, 0, 5], c.k[p1, 9, 0, 5], c.k[p1, 9, 0, 6] = 64, 64, -1
        c.v[p0, 3, 0], c.v[p1, 9, 0] = 100, -100
        out = b.run(ops).double()
        w = (100 - out) / (100 + out)
        assert (w >= 0).all() and (w <= 2.0 ** (-2.0 ** 21 * d) + 2.0 ** -7).all(), (low, w.max())


@pytest.mark.parametrize("new", [3, 12, 80])
@pytest.mark.parametrize("byte", [229, 231, 240, 253])
def test_small_queries_over_the_largest_keys(ops, byte, new):  # noqa: F811
    # queries of about 2^(122 - byte); what f16 takes from them is 2^-151, times 64 values of 127 times the scale
    # up to 2^-12 of a score's unit, in numerator and denominator
    b = Batch(ops, [300], [new], 4, 2, 64, 16, BF16, seed=byte, scales=(byte - 2, byte + 1))
    b.cache.v_scale.fill_(120)
    b.q *= 2.0 ** (122 - byte)
    c = b.cache
    want, v, s = ref.attention(b.q, ref.values(c.k, c.k_scale), ref.values(c.v, c.v_scale), b.table.cpu(), b.ctx, b.cu, b.scale, 16)
    err = b.scale * 2.0 ** (-151 + 13 + byte - 127)
    bound = ((2.0 ** -8 + 2.0 ** -11 + 2 * err + 2.0 ** -17 * (s + 1)) * v)[..., None]
    assert ((b.run(ops).double() - want).abs() <= bound).all()
