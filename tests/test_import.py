"""What an import of the package needs."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)


def test_package_and_library_need_no_torch():
    r = run("""
import sys
sys.modules["torch"] = None
import orthonormal_optimizer_step_gb300 as od
from orthonormal_optimizer_step_gb300 import build
build.build()
assert od.status_string(od.DION_OK) and od.dion_workspace_size(1, 64, 64, 8, od.DION_F32) > 0
assert "dion_q8_matmul" in dir(od)
""")
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("first", ["import orthonormal_optimizer_step_gb300.q8",
                                   "from orthonormal_optimizer_step_gb300 import dion_q8_matmul, q8"])
def test_torch_without_cuda_is_enough_for_the_host_side(first):
    r = run(f"""
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
{first}
import orthonormal_optimizer_step_gb300 as od
assert od.q8.dion_q8_matmul is od.dion_q8_matmul
assert od.new_q8(4, 256, device="cpu").data.shape == (4, 256)
try:
    od.dion_q8_quantize(torch.zeros(4, 256))
except ValueError as e:
    assert "CUDA" in str(e)
else:
    raise AssertionError("accepted a CPU tensor")
""")
    assert r.returncode == 0, r.stderr


def test_unknown_names_are_refused():
    import orthonormal_optimizer_step_gb300 as od
    with pytest.raises(AttributeError, match="no attribute 'dion_q9'"):
        od.dion_q9
