"""Rules of the unary loss's kernels that no run can show, from their source text.

Kernels that wait (griddepcontrol.wait) may begin while the kernel before them still writes what
they will read.  A load through the read-only path asks for memory that nothing writes during
the kernel's whole life, from its start on, so these kernels have none."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dflash2_draft_block_gb300", "csrc")


def functions(name):
    """The text of every function of a file of the loss, comments left out."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    found, depth, start = [], 0, 0
    body = text[text.index("namespace {") + len("namespace {"):]
    for i, c in enumerate(body):
        depth += (c == "{") - (c == "}")
        if depth < 0:
            break
        if c == "}" and depth == 0:
            found.append(body[start:i + 1])
            start = i + 1
    return found


@pytest.mark.parametrize("name, waiting", [("unary_loss.cu", 2), ("loss_gemm.cu", 1)])
def test_no_read_only_loads_beside_the_writer(name, waiting):
    kernels = [f for f in functions(name) if "__global__" in f and "griddepcontrol.wait" in f]
    assert len(kernels) == waiting
    helpers = [f for f in functions(name) if "__device__" in f]
    for f in kernels + helpers:
        assert not re.search(r"__ldg\s*\(|ld\.global\.nc|const\s+\w+\s*\*\s*__restrict__", f), f[:200]
