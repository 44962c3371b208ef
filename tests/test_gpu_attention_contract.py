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
