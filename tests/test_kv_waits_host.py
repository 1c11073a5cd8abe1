"""The prompt kernel's roles wait for one another only with a limit: read from its source (CPU only).

A role whose wait has run out leaves its loop one warp at a time.  A barrier of the hardware (bar.sync), which has no
limit, would then never be complete for the warps that stand at it; an mbarrier's wait gives up like the others."""
import os
import re

import hadamard_incoherence_transforms_b200 as hit

SRC = os.path.join(os.path.dirname(hit.__file__), "csrc", "kv_prompt.cu")


def code():
    text = open(SRC).read()
    return re.sub(r"//[^\n]*", "", text)


def test_no_barrier_without_a_limit_between_the_roles():
    found = re.findall(r"\b(?:bar|barrier(?:\.cta)?)\.(?:sync|red)\b[^;]*", code())
    assert not found, found


def test_barriers_of_the_block_stand_outside_the_roles():
    """Every thread passes exactly two: after the set-up, and after the roles have ended."""
    body = code()
    body = body[body.index("k_kv_prompt("):]
    body = body[:body.index("cudaError_t prepare(")]
    roles = body[body.index("Follow w{&ring};"):body.index("tcgen05.dealloc")]
    assert body.count("__syncthreads()") == 2 and roles.count("__syncthreads()") == 1
    assert roles.rindex("__syncthreads()") > roles.rindex("give_up()")


def test_waits_are_checked():
    """No mbarrier wait whose outcome is dropped, but for the waits in conditions and assignments."""
    lines = [x.strip() for x in code().splitlines() if "mbar_wait(" in x]
    assert len(lines) >= 12
    for x in lines:
        assert re.search(r"(=|\bif \(|&&|\|\|).*mbar_wait\(", x), x
