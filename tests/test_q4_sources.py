"""Numbers that the 4-bit product's header states and its sources hold to."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def text(*path):
    with open(os.path.join(ROOT, *path)) as f:
        return f.read()


def test_longest_rows_of_one_pass():
    """The header's bound is the one that the sources check against their shared memory when they are compiled."""
    source = text("orthonormal_optimizer_step_gb300", "csrc", "q4_gemv.cu")
    bound = re.search(r"kLongestOfAllColumns = (\d+);", source).group(1)
    assert re.search(r"static_assert\(all_columns_fit<32>\(\) && all_columns_fit<64>\(\) && all_columns_fit<128>\(\)", source)
    assert re.search(r"fewer for k beyond (\d+)", text("include", "dion_q4.h")).group(1) == bound
