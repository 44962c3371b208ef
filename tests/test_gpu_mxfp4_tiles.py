"""The 4-bit GEMM in each tile width, with one and several tiles to a CTA, its scales read in pairs
and one by one, y stored by TMA and value by value; against 64 bits, within 1e-5 sum |x W| and the
rounding of y.

The width that the rule in mxfp4.cu picks is worked out here from the rule's own numbers, so that a
change of the rule cannot leave one of these forms untested."""
import os
import re

import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_mxfp4 import check, values, weights

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4a16_int4_quantized_gb300", "csrc")


def rule():
    with open(os.path.join(CSRC, "mxfp4.cu")) as h:
        s = h.read()
    c = re.search(r"c64 = cost\(64, (\d+)\), c128 = cost\(128, (\d+)\), c256 = cost\(256, (\d+)\)", s)
    assert c and "if (c256 <= c128 && c256 <= c64)" in s and "if (c128 <= c64)" in s
    assert "return ceil_div(ntm * ceil_div(N, bn), sms) * c;" in s
    return {bn: int(v) for bn, v in zip((64, 128, 256), c.groups())}


def picked(M, N, sms):
    """(width, the most tiles of a CTA)."""
    ntm = -(-M // 128)
    rounds = {bn: -(-ntm * -(-N // bn) // sms) for bn in (64, 128, 256)}
    cost = {bn: rounds[bn] * c for bn, c in rule().items()}
    bn = 256 if cost[256] <= min(cost[128], cost[64]) else 128 if cost[128] <= cost[64] else 64
    return bn, rounds[bn]


# M, N, the width, at least so many tiles to a CTA (152 SMs)
SHAPES = [(300, 192, 64, 1), (200, 4000, 64, 1), (12750, 192, 64, 2), (12750, 186, 64, 2),
          (512, 4864, 128, 1), (1000, 6400, 128, 3), (999, 6389, 128, 3),
          (1100, 4096, 256, 1), (1111, 13304, 256, 4), (1111, 13300, 256, 4)]


@pytest.mark.parametrize("M,N,width,tiles", SHAPES)
def test_the_rule_picks_these(M, N, width, tiles):
    bn, most = picked(M, N, 152)
    assert bn == width and most >= tiles


def test_every_form_is_among_them():
    assert {(w, t > 1) for _, _, w, t in SHAPES} == {(w, m) for w in (64, 128, 256) for m in (False, True)}
    for w in (64, 128, 256):  # 16-bit rows that TMA can store and that it cannot
        assert {N * 2 % 16 == 0 for _, N, v, t in SHAPES if v == w and t > 1} == {True, False}


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_int4_quantized_gb300 import build
    build.build()
    from w4a16_int4_quantized_gb300 import ops as o
    o.device_status(clear=True)
    return o


def run(ops, M, N, K, out):
    w, sw = weights(ops, N, K, N + K)
    xq, sx = ops.quantize_mxfp4(torch.randn((M, K), generator=torch.Generator(device="cuda").manual_seed(M), device="cuda"))
    y = ops.linear_mxfp4_a4(xq, sx, w, sw, K, out_dtype=out)
    check(y, values(xq, sx, K), values(w, sw, K))
    assert torch.equal(ops.linear_mxfp4_a4(xq, sx, w, sw, K, out_dtype=out), y)
    assert ops.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,width,tiles", SHAPES)
@pytest.mark.parametrize("K", [256, 512, 544, 1536, 1530])  # 8, 16, 17, 48, 48 blocks: pairs from 16 and 48
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16, torch.float16])
def test_tiles(ops, M, N, width, tiles, K, out):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    bn, most = picked(M, N, sms)
    assert bn == width and most >= tiles
    run(ops, M, N, K, out)


@pytest.mark.gpu
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K", [(2048, 13312, 2048), (1025, 13305, 2048)])
def test_prompt(ops, M, N, K, out):
    assert picked(M, N, torch.cuda.get_device_properties(0).multi_processor_count)[0] == 256
    run(ops, M, N, K, out)
