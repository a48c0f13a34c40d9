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


def test_the_committed_capture_describes_the_sources():
    """The default workload's figure is reported (it is null when the step's sources have changed since)."""
    value, source = bench.profiled_traffic("llama3-8b-megabatch", "dion_update_tc")
    assert value and value > 1e10, source
