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


def test_what_another_cta_has_to_see_is_released_and_acquired_at_cluster_scope():
    """A CTA's payload, query, operand and accumulator buffers are read and written by its own warps
    and, at the word of another CTA, by that CTA's stores or MMAs: a barrier of another CTA is arrived
    at, and waited for, at cluster scope."""
    assert "release.cta.shared::cluster" not in source("tc_ptx.cuh")
    b = body(source("chunk.cu"), "chunk_kernel")
    assert "arrive_cluster_local" not in b
    # shared memory: a relay of the other CTA arrives, released at cluster scope
    for bar in ("B_QREADY", "B_PFREE", "B_OP"):
        waits = set(re.findall(r"\b(wait\w*|relay)\(%s" % bar, b))
        assert waits == {"wait_cluster", "relay"}, (bar, waits)
    relay = b[b.index("auto relay"):]
    assert "arrive_cluster(to)" in relay[: relay.index("};")]
    # TMEM alone: the warps arrive themselves, behind the wait for their accesses and the fence
    for bar in ("B_SEMPTY", "B_RS"):
        assert set(re.findall(r"\b(wait\w*)\(%s" % bar, b)) == {"wait_cluster"}, bar
    for at in [m.start() for m in re.finditer(r"arrive_cluster_relaxed\(", b)]:
        assert "tc_fence_before();" in b[at - 300: at]
