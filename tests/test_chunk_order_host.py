"""What orders one kernel's (or one SM's) memory accesses before another's, read from the source: a
run that happens to go right does not show it."""
import os
import re

import pytest

import fp8_mla_latent_gb300 as pkg

CSRC = os.path.join(os.path.dirname(os.path.abspath(pkg.__file__)), "csrc")


def source(name):
    """The file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(text, kernel):
    """From the kernel's name to the closing brace of its body (in the first column)."""
    at = text.index(kernel + "(const ChunkArgs")
    return text[at: text.index("\n}", at)]


@pytest.mark.parametrize("kernel", ["chunk_kernel", "join_kernel"])
def test_nothing_of_an_earlier_kernel_is_read_before_the_wait_for_it(kernel):
    """Both start while the kernel before them runs; its writes are promised after the wait alone."""
    b = body(source("chunk.cu"), kernel)
    before = b[b.index("{"): b.index("grid_dependency_wait()")]
    assert "ws." not in before and "a.out" not in before
    assert kernel != "join_kernel" or "return" not in before, "a block that leaves without the wait"
