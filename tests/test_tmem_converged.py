"""Every wrapper of a TMEM read or write brings its warp together first: the instructions are undefined for a
warp whose lanes are apart, and their callers branch by row (read from the source)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4a16_int4_quantized_gb300", "csrc")
WHOLE_WARP = re.compile(r"tcgen05\.(?:ld|st)\.sync\.aligned")


def test_reads_and_writes_of_tmem_begin_with_a_whole_warp():
    found = 0
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as h:
            source = re.sub(r"//[^\n]*", "", h.read())
        for part in re.split(r"\n(?=W4_DEV|static __device__|template|__global__)", source):
            if not WHOLE_WARP.search(part):
                continue
            assert name == "tcgen05.cuh", name      # one place
            body = part[part.index("{") + 1:]
            assert body.lstrip().startswith("__syncwarp();"), part[:80]
            found += len(WHOLE_WARP.findall(part))
    assert found == 3
