"""The prompt kernel's roles wait for one another only with a limit: read from its source (CPU only).

A role whose wait has run out leaves its loop.  The four warps that unpack codes meet at a barrier of the hardware, which
has no limit, so they have to come to it equally often: a warp one of whose waits has run out comes to the next meeting
all the same and says so there, and all of them leave."""
import itertools
import os
import re

import pytest

import hadamard_incoherence_transforms_b200 as hit

SRC = os.path.join(os.path.dirname(hit.__file__), "csrc", "kv_prompt.cu")


def code():
    return re.sub(r"//[^\n]*", "", open(SRC).read())


def kernel():
    body = code()
    body = body[body.index("void __launch_bounds__(kThreads, 1) k_kv_prompt("):]
    return body[:body.index("cudaError_t prepare(")]


def unpacking():
    """The loops of the warps that unpack codes: the one role whose warps share a barrier."""
    body = kernel()
    return body[body.index("auto unpack = ["):body.index("if constexpr (F::HALVES == 2) unpack(")]


def test_one_barrier_inside_the_roles():
    found = re.findall(r"\b(?:bar|barrier(?:\.cta)?)\.(?:sync|red|arrive)[\w.]*", code())
    assert found == ["bar.sync"], found
    assert "auto meet = [&]() { asm volatile(\"bar.sync" in unpacking()


def test_unpacking_warps_meet_equally_often():
    """One meeting for every unit of the group's segments, on every path; a way out of the loop only by what was said
    there; and one more meeting for a warp that leaves by any other way."""
    lines = [x.strip() for x in unpacking().splitlines() if x.strip()]
    assert not any(re.search(r"\b(return;|goto|continue)\b", x) for x in lines)
    loops = [x for x in lines if re.match(r"(while|do)\b", x)]
    assert loops == ["while (ok && !told && (more = w.next(lane)) > 0) {"]
    units = [x for x in lines if x.startswith("for (int j = ")]
    assert units == ["for (int j = ub; j < ue; ++j, ++kv) {"]  # of the segment, which is the same for all four
    assert [x for x in lines if "break" in x] == ["if (told) break;"]
    meets = [i for i, x in enumerate(lines) if x.startswith("meet();")]
    assert len(meets) == 2 and lines.index(units[0]) < meets[0] < lines.index("if (told) break;") < meets[1]
    # inside the loop over units the meeting is under no condition
    depth = 0
    for x in lines[lines.index(units[0]) + 1:meets[0]]:
        depth += x.count("{") - x.count("}")
    assert depth == 0
    assert [x for x in lines[:meets[1]] if x.startswith("if (!told) {")] and lines[meets[1] + 1] == "}"
    # each warp says whether its waits were fine
    assert re.search(r"ok \? \w+ : kFailed|ok \? 0u : kFailed", unpacking())


class Warp:
    """The loop's meetings: segments of 0, 1 or 3 units, each wait failing where `bad` says."""

    def __init__(self, who, bad, segments):
        self.steps = self.run(who, bad, segments)

    @staticmethod
    def run(who, bad, segments):
        n, ok, told, kv = 0, True, False, 0

        def wait():
            nonlocal n
            n += 1
            return (who, n) not in bad

        for units in [*segments, None]:  # None: there are no more
            if not wait():  # for the segment
                ok = False
            if not ok or units is None:
                break
            for _ in range(units):
                ok = ok and wait()
                told = yield kv, not ok  # the meeting, and what was said there
                if told:
                    break
                ok = ok and wait()
                kv += 1
            if told or not ok:
                break
        if not told:
            yield kv, not ok


@pytest.mark.parametrize("segments", [[], [0], [3], [1, 0, 3], [0, 0, 1]])
def test_meetings_of_every_failing_pair_come_to_an_end(segments):
    """The model of that loop, with every pair of failing waits: all four warps come to equally many meetings, nobody is
    left at one, and those of a unit are all at the same unit."""
    waits = 2 * sum(segments) + len(segments) + 1
    places = list(itertools.product(range(4), range(1, waits + 1)))
    for bad in [(), *((p,) for p in places), *itertools.combinations(places, 2)]:
        warps = [Warp(i, bad, segments).steps for i in range(4)]
        at = [next(w, None) for w in warps]
        while any(x is not None for x in at):
            assert all(x is not None for x in at), (segments, bad)
            assert len({kv for kv, _ in at}) == 1
            told = any(fails for _, fails in at)
            after = []
            for w in warps:
                try:
                    after.append(w.send(told))
                except StopIteration:
                    after.append(None)
            at = after


def test_barriers_of_the_block_stand_outside_the_roles():
    """Every thread passes exactly two: after the set-up, and after the roles have ended."""
    body = kernel()
    roles = body[body.index("Follow w{&ring};"):body.index("tcgen05.dealloc")]
    assert body.count("__syncthreads()") == 2 and roles.count("__syncthreads()") == 1
    assert roles.rindex("__syncthreads()") > roles.rindex("give_up()")


def test_waits_are_checked():
    """No mbarrier wait whose outcome is dropped."""
    lines = [x.strip() for x in code().splitlines() if "mbar_wait(" in x]
    assert len(lines) >= 12
    for x in lines:
        assert re.search(r"(=|\bif \(|&&|\|\|).*mbar_wait\(", x), x
