"""Kernels with copies or products in flight wait for them before they end, after an abort too (read from
the source: making a device wait run out there would need a fault).  tcgen05.cuh checks the ring's
arithmetic when it is compiled."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4a16_int4_quantized_gb300", "csrc")


@pytest.mark.parametrize("name", ["gemm_tc.cu", "mxfp4.cu", "tree_attn.cu"])
def test_what_was_begun_is_waited_for(name):
    with open(os.path.join(CSRC, name)) as h:
        source = h.read()
    end = source.rindex("tmem_dealloc(")
    body = source[source.rindex("__global__", 0, end):end]
    at = body.rindex("if (__builtin_expect(")
    roles, drain = body[:at], body[at:]
    # the block stands between two barriers of the CTA, with no role's code after it
    assert roles.rstrip().endswith("__syncthreads();") and drain.count("__syncthreads();") == 1
    # every barrier that a copy completes on
    rings = set(re.findall(r"expect_tx\(&(?:sh|ctl)->(\w+)", roles)) | set(re.findall(r"expect_tx\(&(\w+)\[", roles))
    assert rings
    for r in rings:
        assert re.search(r"drain_ring\(&?(?:sh|ctl)->%s\b" % r, drain), r
    # and the products, on a barrier of their own
    assert re.search(r"mbar_init\(&(?:sh|ctl)->drained(?:\[r\])?, 1\)", roles)
    assert re.search(r"(?:drain_products|umma_commit)\(&(?:sh|ctl)->drained", drain)
    assert not re.search(r"->drained", roles.replace("mbar_init(&sh->drained", "").replace("mbar_init(&ctl->drained", ""))
