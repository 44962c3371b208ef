"""examples/decode8_step.py: the calls of a decode step in 8 bits, one after another, against the
same step on dense weights in 32 bits.

What differs are roundings to 8 bits: a row of n normal values has its largest at 4.5 of their spread
at most (n up to 1024), so a Q8 row is off by 4.5 / 127 / sqrt(12) = 1 % of its norm, three times in
the step, and keys and values under a power of two by twice that: 5 % of the logits' spread together,
were they all to fall the same way and the residual to carry nothing past them.  Five such spreads bound
a single log probability."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_int4_quantized_gb300 import build
    build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import decode8_step
    return decode8_step


@pytest.mark.parametrize("contexts,new,window,sinks", [
    ((37, 500, 5), (3, 1, 20), 64, 4), ((0,), (1,), 0, 0), ((16, 1500), (100, 40), 0, 0), ((300,) * 9, (1,) * 9, 100, 1)])
def test_step(example, contexts, new, window, sinks):
    (logp, entropy, ids, top_logp), nexts, want = example.run(contexts, new, window, sinks, top=20, seed=len(contexts))
    assert logp.shape == entropy.shape == (sum(new),) and ids.shape == top_logp.shape == (sum(new), 20)
    limit = 5 * 0.05 * want.std().item()
    assert ((logp - want.gather(1, nexts.long()[:, None])[:, 0]).abs() <= limit).all()
    assert ((top_logp - want.gather(1, ids.long())).abs() <= limit).all()
    assert (top_logp[:, 1:] <= top_logp[:, :-1]).all()
    p = want.exp()
    assert ((entropy + (p * want).sum(-1)).abs() <= limit).all()
    from w4a16_int4_quantized_gb300 import ops
    assert ops.device_status() == 0


def test_steps_in_turn(example):
    """A prompt in one piece, and in pieces and single tokens: the same cache but for the growth of a block's
    scale (a kept code is off by a step of it at most), so the same answers within the limit above."""
    from w4a16_int4_quantized_gb300 import ops
    n = 40
    layer, batch, cache, x, residual = example.make(ops, (0,), (n,), 3)
    whole = example.step(ops, layer, x, residual, batch, cache, 0, 0, 3)[0]
    table, _, _, positions, cos_sin, max_len, _, nexts = batch
    parts, at = [], 0
    other = ops.Kv8Cache.empty(cache.k.shape[0], example.PAGE, example.KV_HEADS, example.HEAD_DIM)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for m in (17, 1, 1, 5, 1, 15):
        b = (table, i32([at]), i32([0, m]), positions[at: at + m].contiguous(), cos_sin, max_len, m, nexts[at: at + m].contiguous())
        parts.append(example.step(ops, layer, x[at: at + m].contiguous(), residual[at: at + m].contiguous(), b, other, 0, 0, 3)[0])
        at += m
    got = torch.cat(parts)
    assert ((got - whole).abs() <= 0.05 * 5 * 2.0).all()
    assert ops.device_status() == 0
