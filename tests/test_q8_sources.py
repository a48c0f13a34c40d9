"""Rules that the kernels of the 8-bit operators keep in their source."""
import ctypes
import glob
import os
import re
import subprocess

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


def test_shares_of_a_split_contraction_have_blocks(tmp_path):
    """The rule itself, compiled for the host, with the kernel's division of the blocks: only the last of eight may have none."""
    text = open(os.path.join(CSRC, "q8_gemm.cu")).read()
    m = re.search(r"^int shares\(long long tiles, int kblocks\)\n\{.*?^\}", text, re.S | re.M)
    src = tmp_path / "shares.cc"
    src.write_text("static long long cdiv(long long a, long long b) { return (a + b - 1) / b; }\n"
                   'extern "C" ' + m.group(0) + "\n")
    subprocess.run(["g++", "-shared", "-fPIC", "-o", str(tmp_path / "shares.so"), str(src)], check=True)
    shares = ctypes.CDLL(str(tmp_path / "shares.so")).shares
    shares.argtypes = [ctypes.c_longlong, ctypes.c_int]
    seen = set()
    for kblocks in range(1, 700):
        for tiles in (1, 15, 16, 23, 28, 29, 36, 46, 47, 200):
            s = shares(tiles, kblocks)
            assert s == 1 or 3 <= s <= 8
            per = -(-kblocks // s)
            with_blocks = -(-kblocks // per)
            assert with_blocks == s or (s == 8 and with_blocks == 7), (kblocks, tiles, s)
            seen.add(s)
    assert seen == {1, 3, 4, 5, 6, 7, 8}
