"""The ring of the paged attention's loads as a model on the host: the roles that
wait on mbarriers by parity, in every order that their steps can take.  A wait by
parity is right only for a thread that sees every phase: the waiter of phase k must
find k or k + 1 phases completed.  With more it has been lapped and waits for a
phase that may never come, with fewer it passes early."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def explore(stages, loads, owns, arrivals, second_arrives):
    """All states of: a first loading warp (waits for `empty`, arms, loads), a
    second one (waits for `empty`, has a part of load j where owns[j], arrives at
    `empty` if second_arrives), and the products (wait for `full`, arrive at
    `empty`).  `empty` takes `arrivals` a phase.  Returns what is wrong, or None."""
    start = (0, 0, 0)
    seen, todo = {start}, [start]
    while todo:
        first, second, used = todo.pop()

        def phases(st):
            """Completed phases of a stage's `empty`: arrivals so far over those of a phase."""
            done = sum(1 for j in range(used) if j % stages == st)
            if second_arrives:
                done += sum(1 for j in range(second) if j % stages == st)
            return done // arrivals

        def passes(j):
            """Whether the wait before load j lets a warp through, or what is wrong with it."""
            if j < stages:
                return True
            k, c = j // stages - 1, phases(j % stages)
            if not k <= c <= k + 1:
                return f"load {j}: waits for phase {k} of its stage with {c} completed"
            return c == k + 1
        after = []
        for who, j, step in (("first", first, (1, 0, 0)), ("second", second, (0, 1, 0))):
            if j < loads:
                ok = passes(j)
                if isinstance(ok, str):
                    return f"{who} warp, {ok}"
                if ok:
                    after.append(step)
        # `full` of load `used`: armed by the first warp, and every byte of it is in
        if used < loads and used < first and (not owns[used] or used < second):
            after.append((0, 0, 1))
        if not after and (first, second, used) != (loads, loads, loads):
            return f"stuck at {first}, {second}, {used}"
        for a, b, c in after:
            x = (first + a, second + b, used + c)
            if x not in seen:
                seen.add(x)
                todo.append(x)
    return None


def protocol():
    """The arrivals that a phase of `empty` takes and whether the second loading warp
    makes one for every load, as the kernel has them."""
    with open(os.path.join(ROOT, "sparse_kv_verify_gb300", "csrc", "paged.cu")) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    arrivals = int(re.search(r"mbar_init\(&empty\[s\], (\d+)\)", code).group(1))
    loads = code[code.index("if (warp == C::load_warp || warp == C::load_warp2) {"):code.index("} else if (warp == C::land_warp) {")]
    # in the statement list of a load, not behind the ownership of a page
    second = re.search(r"^ {12}if \(!lead && lane_id == 0\) mbar_arrive\(&empty\[st\]\);", loads, re.M)
    return arrivals, second is not None


OWNS = {"none": lambda j: False, "all": lambda j: True, "a run of single pages": lambda j: not 4 <= j < 15,
        "late": lambda j: j > 12, "odd": lambda j: j % 2 == 1}


@pytest.mark.parametrize("owns", OWNS)
@pytest.mark.parametrize("stages", [2, 3, 5])
def test_no_wait_of_the_ring_can_be_lapped(stages, owns):
    loads = 17
    assert explore(stages, loads, [OWNS[owns](j) for j in range(loads)], *protocol()) is None


def test_the_model_finds_a_warp_that_nothing_waits_for():
    """Where `empty` takes the products' arrival alone, a second warp without a part
    in a load is lapped; one with a part in every load is not."""
    assert "second warp" in explore(3, 17, [False] * 17, 1, False)
    assert "second warp" in explore(3, 17, [OWNS["a run of single pages"](j) for j in range(17)], 1, False)
    assert explore(3, 17, [True] * 17, 1, False) is None
    # and an arrival that is counted but never made, or the other way round
    assert "stuck" in explore(3, 17, [True] * 17, 2, False)
    assert explore(3, 17, [True] * 17, 1, True) is not None
