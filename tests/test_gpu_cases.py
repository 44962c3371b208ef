"""The cases of perf/operators.py: the library's calls and the plain forms against the
file's definitions in 64 bits, at its smaller cases and some drawn ones.

Whole numbers are equal.  For computed numbers, the error's norm over the result's: one
rounding to the type (u), for attention another u for the rounded weights, and of the f32
sums 1e-5 of a norm that is larger than the result's by sqrt(K) at most (products), or
2^-18 sqrt(D) and 2e-3 u' (rotation, scores) as in test_gpu_draft.py."""
import importlib.util
import math
import os
import random

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "operators.py")


def load():
    spec = importlib.util.spec_from_file_location("perf_operators", PATH)
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


def chosen():
    m = load()
    small = [c for c in m.listed() if m.work(c)["bytes"] + m.work(c)["flops"] / 250 < 1e8]
    rng, drawn = random.Random(11), {op: [] for op in ("plan", "rope", "attn", "quant", "linear")}
    while min(map(len, drawn.values())) < 5:
        c = m.draw(rng)
        if len(drawn[c["op"]]) < 5 and m.work(c)["bytes"] + m.work(c)["flops"] / 250 < 3e7:
            drawn[c["op"]].append(dict(c, name="drawn_%s%d" % (c["op"], len(drawn[c["op"]]))))
    return small + sum(drawn.values(), [])


def limit(case, dtype):
    u = U[dtype]
    return {"rope": u + 2.0 ** -18 * math.sqrt(case.get("D", 1)), "attn": 2 * u + 2e-3 * u + 1e-5, "quant": 0.0,
            "linear": u + 1e-5 * math.sqrt(case.get("K", 1))}[case["op"]]


@pytest.mark.parametrize("case", chosen(), ids=lambda c: c["name"])
@pytest.mark.parametrize("own", [True, False], ids=["library", "plain"])
def test_case(cases, case, own):
    cases.own = own
    got, want = cases.run(cases.prepare(case, 3)), cases.exact(case, 3)
    if not isinstance(want, dict):
        got, want = dict(y=got), dict(y=want)
    assert got.keys() == want.keys()
    for name in want:
        g, w = got[name], torch.as_tensor(want[name]).cuda()
        assert g.shape == w.shape, name
        if not g.dtype.is_floating_point:
            assert torch.equal(g.long(), w.long()), name
        elif case["op"] == "quant":
            assert torch.equal(g.double(), w), name  # exact in bf16
        else:
            err = float((g.double() - w).norm() / w.norm())
            assert err <= limit(case, g.dtype), (name, err)
    # the same call gives the same bits
    again = cases.run(cases.prepare(case, 3))
    again = again if isinstance(again, dict) else dict(y=again)
    assert all(torch.equal(got[k], again[k]) for k in got)
