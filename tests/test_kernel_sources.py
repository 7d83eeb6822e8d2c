"""Properties of the kernels' sources that no run shows (CPU)."""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(glob.glob(os.path.join(ROOT, "moe_expert_dispatch_online_gb300", "csrc", "*.cu*")))


def code(path):
    with open(path) as f:
        text = f.read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_warps_converge_before_warp_wide_instructions(path):
    """An instruction that all threads of a warp execute together comes right behind a __syncwarp (or another such
    instruction): the end of a branch or of a loop that lanes left at different times does not bring them together."""
    lines = code(path).split("\n")
    start, inside = 0, ""                      # of the statement; the function it is in
    for i, line in enumerate(lines):
        name = re.match(r"(?:template|__device__|__global__)[^(]* (\w+)\(", line)
        if name:
            inside = name.group(1)
        if re.search(r"asm volatile\(", line):
            start = i
        if re.search(r"\.aligned|\bbar\.(sync|red)|\belect\.sync", line) and not inside.endswith("_converged"):
            before = [x for x in lines[max(0, start - 8):start] if x.strip()]
            assert any("__syncwarp();" in x or ".aligned" in x for x in before[-4:]), (os.path.basename(path), i + 1, line)
        # a helper that relies on its caller: no lane has branched off since the warp was last together
        if re.search(r"_converged\(", line) and not name:
            for j in range(i - 1, -1, -1):
                if re.search(r"__syncwarp\(\)|__all_sync\(", lines[j]):
                    break
                assert not re.search(r"\bif \((lane|threadIdx)|\bwhile\b", lines[j]), (os.path.basename(path), i + 1, line)


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_load_is_multicast(path):
    """A tensor copy with cluster multicast may only read this GPU's own memory, and the calls take whatever device
    pointers they are given. (A multicast commit is a signal between the two CTAs and reads nothing.)"""
    text = re.sub(r'"\s*"', "", code(path))
    assert not re.findall(r"cp\.async\.bulk[^;\"]*multicast", text)
