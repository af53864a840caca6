"""The paged kernels are programmatic dependents of one another: a kernel may let the next be set
up only behind its own wait, in every path, or what the next one reads early could be older work
that has not ended. Checked in the source, since no call shows it."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "long_context_decode_02_b200", "csrc")


@pytest.mark.parametrize("name,kernels", [("paged_attend.cu", 2), ("paged_cache.cu", 2)])
def test_dependents_are_let_in_right_behind_the_wait(name, kernels):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    bodies = code.split("__global__")[1:]
    assert len(bodies) == kernels
    for body in bodies:
        statements = [s.strip() for s in re.split(r"[;{}]", body)]
        statements = [s for s in statements if s]
        at = [i for i, s in enumerate(statements) if s == "grid_launch_dependents()"]
        assert len(at) == 1
        assert statements[at[0] - 1] == "grid_dependency_wait()"
