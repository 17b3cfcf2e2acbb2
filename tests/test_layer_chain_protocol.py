"""Hand-offs of the selective scan's kernels (csrc/ssm_tc.cuh, csrc/ssm_tc_bwd.cuh) under random
schedules, on the CPU.  The order of a role's steps is taken from the kernel's source, so a step
moved across a hand-off there moves here too."""
import os
import re

import pytest

from tests.protocol_model import Model, count_caught

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "delta_rule_recurrent_osdn_b200", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", lambda m: m.group(0) if "-----" in m.group(0) else "", f.read())


def section(text, title, until):
    """The source between two role headings ('// ------ title')."""
    at = re.search(r"// -{20,} " + re.escape(title) + r"\n", text).end()
    return text[at:re.compile(r"// -{20,} " + re.escape(until) + r"\n").search(text, at).start()]


def events(text, patterns):
    """Names of the patterns in the order in which they occur."""
    found = [(m.start(), name) for name, p in patterns.items() for m in re.finditer(p, text)]
    return [name for _, name in sorted(found)]


# ------------------------------------------------------------- the ring of gates (segment launches)
# Two warps make every other chunk's gates in a ring of slots; the state's warps and V's read a
# chunk's slot and give it back.
RING = int(re.search(r"TCS_GATES = (\d+)", source("ssm_tc.cuh")).group(1))


def state_order():
    text = section(source("ssm_tc.cuh"), "state", "V'")
    loop = text[text.index("for (int i = 0; i < nch; ++i)"):]
    return events(loop, {"read": r"gate\(i\)->", "free": r"mbar_arrive\(&gate_free"})


def gate_warp(w, N):
    for i in range(w, N, 2):
        if i >= RING:
            yield ("wait", f"free{i % RING}", i // RING - 1)
        yield ("write", ("gate", i % RING), i)
        yield ("arrive", f"full{i % RING}", i // RING)


def gate_reader(order, N):
    for i in range(N):
        yield ("wait", f"full{i % RING}", i // RING)
        for step in order:
            if step == "read":
                yield ("read", ("gate", i % RING), i)
            else:
                yield ("arrive", f"free{i % RING}", i // RING)


def ring(order, N, seed):
    bars = {f"{k}{s}": c for s in range(RING) for k, c in (("full", 1), ("free", 2))}
    return Model(bars, {"G0": gate_warp(0, N), "G1": gate_warp(1, N),
                        "state": gate_reader(order, N),
                        "V": gate_reader(["read", "free"], N)}, seed)


def test_state_reads_its_gates_before_it_gives_them_back():
    order = state_order()
    assert order.count("free") == 1 and "read" in order
    for seed in range(300):
        ring(order, 3 * RING + 3, seed).run()


def test_a_read_behind_the_release_is_caught():
    assert count_caught(lambda seed: ring(["read", "free", "read"], 3 * RING, seed), range(300)) > 0


# ------------------------------------------------- tensor memory between products (chunk gradients)
# Products with different accumulators may complete in any order: a score tile that one product
# reads is overwritten by another only behind a wait for a commit that covers the first.
def tile_hazards(text):
    """Score tiles overwritten by a product while one issued before may still read them."""
    pattern = re.compile(r"(?P<weighted>weighted\((?P<acc>\w+), (?P<src>\w+),)"
                         r"|(?P<over>(?:scores|state_k)\((?P<dst>\w+),)"
                         r"|mma_commit\((?P<commit>\w+)\)|tcs_wait\((?P<wait>\w+),")
    pending, covered, bad, steps = set(), {}, [], []
    for m in pattern.finditer(text):
        if m.group("weighted"):
            steps += [m.group("acc"), m.group("src")]
            if m.group("acc") in pending:
                bad.append(m.group("acc"))
            pending.add(m.group("src"))
        elif m.group("over"):
            steps.append(m.group("dst"))
            if m.group("dst") in pending:
                bad.append(m.group("dst"))
        elif m.group("commit"):
            covered[m.group("commit")] = set(pending)
        else:
            pending -= covered.pop(m.group("wait"), set())
    return bad, steps


def issue_order():
    text = source("ssm_tc_bwd.cuh")
    at = text.index("bool ok = tcs_wait(tiles, 0)")
    return text[at:text.index("tc::mma_commit(drain)", at)]


def test_score_tiles_are_overwritten_once_used_up():
    bad, steps = tile_hazards(issue_order())
    assert {"T0", "T1", "A0", "A1"} <= set(steps)  # the source was understood
    assert not bad


def test_an_early_overwrite_is_caught():
    assert tile_hazards("weighted(A1, T1, ac); tc::mma_commit(acc1); scores(T1, ady);")[0] == ["T1"]
    assert not tile_hazards("weighted(A1, T1, ac); tc::mma_commit(acc1); tcs_wait(acc1, 0); scores(T1, ady);")[0]


# ------------------------------------------------------------ copies seen by the warps that read them
def test_the_warps_that_read_token_tiles_wait_for_the_copies():
    """A copy's bytes are visible to threads that saw its barrier complete: the element-wise warps of
    the chunk gradients, which read rows of the tiles, wait for it whatever the chunk's length."""
    text = source("ssm_tc_bwd.cuh")
    role = text[text.index("bool ok", text.index("auto arrive = [&]")):]
    first = role[:role.index("tile16(")]
    assert re.match(r"bool ok = wait\(tiles, 0\);", first)
