"""The digest that ties a committed DRAM-traffic capture to the step's sources."""
import os
import shutil

import bench

CSRC = os.path.join("orthonormal_optimizer_step_gb300", "csrc")


def test_digest_follows_the_steps_sources_alone(tmp_path, monkeypatch):
    shutil.copytree(os.path.join(bench.ROOT, CSRC), tmp_path / CSRC)
    want = bench.csrc_digest()
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.csrc_digest() == want
    for name in ("q8_gemm.cu", "q8.cuh"):          # kernels that no step launches
        with open(tmp_path / CSRC / name, "a") as f:
            f.write("// changed\n")
    assert bench.csrc_digest() == want
    for name in ("dion_tc.cu", "tc.cuh", "common.cuh"):
        before = bench.csrc_digest()
        with open(tmp_path / CSRC / name, "a") as f:
            f.write("// changed\n")
        assert bench.csrc_digest() != before
