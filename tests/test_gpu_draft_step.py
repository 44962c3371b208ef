"""examples/draft_step.py: the calls of a decode step of drafted tokens, one after
another, against the same step in plain torch.  The step rounds to bf16 three
times on the way (the queries, keys and values; p; the attention output), 2^-8
each in the worst case and independent, so 3 * 2^-8 of the result's norm covers it."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def step():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_int4_quantized_gb300 import build
    build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import draft_step
    return draft_step


@pytest.mark.parametrize("contexts,parents", [
    ((37, 180, 5), ((-1, 0, 0, 1, 1, 2), (-1,), (-1, -1, 0, 1, 3))),
    ((0,), ((-1,),)),
    ((16, 1500), (tuple(range(-1, 15)), (-1,) * 9))])
def test_step(step, contexts, parents):
    got, want = step.run(contexts, parents, seed=len(contexts))
    assert got.shape == want.shape
    assert ((got - want).norm() / want.norm()).item() <= 3 * 2.0 ** -8
    from w4a16_int4_quantized_gb300 import ops
    assert ops.device_status() == 0
