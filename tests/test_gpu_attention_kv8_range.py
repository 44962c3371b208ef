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
