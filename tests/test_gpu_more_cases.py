"""The cases of perf/more_operators.py: the library's calls and the plain forms against the file's
definitions in 64 bits, at its smaller cases and some drawn ones.

Indices are equal.  The error's norm over the result's: queries, attention and the bf16 values one
rounding to the type (u), attention another u of f16 for the weights; a code that lies next to a tie
may be the other one, a step of at most 1/63 of its block's largest value, which is met for no more
than one value in 2^10: 2^-5 * 1/63 * 5.  Log probabilities 2^-18 (see test_gpu_logprobs.py), Q8 scales
and norms 2^-17."""
import importlib.util
import os
import random

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -17}
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "more_operators.py")


def load():
    spec = importlib.util.spec_from_file_location("perf_more_operators", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.fixture(scope="module")
def cases():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_int4_quantized_gb300 import build
    build.build()
    return load()


def cost(m, c):
    w = m.work(c)
    return w["bytes"] + w["flops"] / 250


def chosen():
    m = load()
    small = [c for c in m.listed() if cost(m, c) < 1e8]
    rng, drawn = random.Random(7), {op: [] for op in ("norm", "store", "attn", "logp")}
    while min(map(len, drawn.values())) < 6:
        c = m.draw(rng)
        if len(drawn[c["op"]]) < 6 and cost(m, c) < 6e7:
            drawn[c["op"]].append(dict(c, name="drawn_%s%d" % (c["op"], len(drawn[c["op"]]))))
    return small + sum(drawn.values(), [])


@pytest.mark.parametrize("case", chosen(), ids=lambda c: c["name"])
@pytest.mark.parametrize("own", [True, False], ids=["library", "plain"])
def test_case(cases, case, own):
    cases.own = own
    got = cases.run(cases.prepare(case, 5))
    want = cases.exact(case, 5)
    assert got.keys() == want.keys()
    for name, g in got.items():
        w = want[name]
        assert g.shape == w.shape
        if not g.is_floating_point():
            assert np.array_equal(g.cpu().numpy(), w.cpu().numpy()), name
            continue
        if g.numel() == 0:
            continue
        limit = U[g.dtype]
        if case["op"] == "attn":
            limit += 2.0 ** -11
        if name in ("values", "k", "v"):
            limit += 2.0 ** -5 * 5 / 63
        off = (g.double() - w.double()).norm().item()
        assert off <= limit * w.double().norm().item(), name
