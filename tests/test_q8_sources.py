"""Rules that the kernels of the 8-bit operators keep in their source."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "orthonormal_optimizer_step_gb300", "csrc")


def kernels():
    """(name, body) of every __global__ function of the 8-bit operators."""
    for path in sorted(glob.glob(os.path.join(CSRC, "q8_*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__[^;{]*?(\w+)\s*\(\s*const[^{;]*\)\s*\{", text):
            depth, i = 1, m.end()
            while depth:
                depth += {"{": 1, "}": -1}.get(text[i], 0)
                i += 1
            yield m.group(1), text[m.end():i - 1]


KERNELS = dict(kernels())


def test_all_kernels_are_found():
    assert len(KERNELS) >= 10 and {"q8_gemm_kernel", "q8_gemm_split_kernel", "q8_quant_kernel"} <= set(KERNELS)


def outer_blocks(body):
    """The text between a body's outermost braces' ends: a statement or an if with its block each."""
    depth, start = 0, 0
    for i, ch in enumerate(body):
        depth += {"{": 1, "}": -1}.get(ch, 0)
        if depth == 0 and ch in ";}":
            yield body[start:i + 1]
            start = i + 1


@pytest.mark.parametrize("name", sorted(KERNELS))
def test_waits_for_the_previous_kernel_come_first(name):
    """A thread calls wait_previous() before it loads operands or waits on a barrier: a wait's time limit counts from
    its start, so it must not start while an earlier kernel of the stream still runs.  Either every thread calls it
    before the warps part, or each warp's branch does."""
    uses = re.compile(r"mbar_wait|wait_peer|tma_load|scale_words")
    waited = False
    for block in outer_blocks(KERNELS[name]):
        first = block.find("wait_previous()")
        use = uses.search(block)
        assert waited or use is None or 0 <= first < use.start(), block[:200]
        waited = waited or block.strip() == "wait_previous();"
    assert waited or uses.search(KERNELS[name])
