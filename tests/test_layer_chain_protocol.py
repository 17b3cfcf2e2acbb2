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


# ------------------------------------------------------------------- the forward chain, all its roles
# Transcribed from ssm_tc_chain_kernel in its forward form; what a role reads or writes of shared and
# tensor memory is versioned by chunk.
FWD_BARS = {**{f"{k}{s}": 1 for k in ("q_full", "k_full", "v_full", "q_empty", "k_empty", "v_empty", "g_full")
               for s in (0, 1)},
            "p_full0": 2, "p_full1": 2, "vp_full": 2, "vp_free": 1, "u_full": 1, "u_free": 1, "s_full": 1,
            "y1_done": 1, "y_full": 1, "y_free": 1, "drain": 1,
            **{f"{k}{s}": 1 for k in ("full", "free") for s in range(RING)}}


def gate_wait(i):
    return ("wait", f"full{i % RING}", i // RING)


def gate_read(i):
    return ("read", ("gate", i % RING), i)


def f_tma(N, mut):
    got = {"q": 0, "k": 0, "v": 0}
    ok = True
    for i in range(N):
        for t in "kqv":
            if i >= 2 and not (ok := (yield ("wait", f"{t}_empty{i & 1}", (i >> 1) - 1))):
                break
            yield ("tma", [(t, i & 1)], i, f"{t}_full{i & 1}", i >> 1)
            got[t] = i + 1
        if not ok:
            break
    for t in "kqv":
        for i in range(max(got[t] - 2, 0), got[t]):
            yield ("wait", f"{t}_full{i & 1}", i >> 1, "drain")


def f_mma(N, mut):
    def body():
        def g(i):
            for t in "qk":
                if not (yield ("wait", f"{t}_full{i & 1}", i >> 1)):
                    return False
            yield ("mma", [(("q", i & 1), i), (("k", i & 1), i)], [(("G", i & 1), ("G", i))])
            yield ("commit", f"g_full{i & 1}", i >> 1)
            return True

        if N and not (yield from g(0)):
            return
        for i in range(N):
            s, ph = i & 1, i >> 1
            if not (yield ("wait", "vp_full", i)):
                return
            if i and not (yield ("wait", "u_free", i - 1)):
                return
            yield ("mma", [(("k", s), i), (("vp", 0), ("V", i)), (("vp", 1), ("V", i))], [("U", i)])
            yield ("commit", "u_full", i)
            yield ("commit", "vp_free", i)
            yield ("commit", f"k_empty{s}", ph)
            if not (yield ("wait", "s_full", i)):
                return
            if i and not (yield ("wait", "y_free", i - 1)):
                return
            yield ("mma", [(("q", s), i), ("S", i)], [("Y1", i)])
            yield ("commit", "y1_done", i)
            yield ("commit", f"q_empty{s}", ph)
            if i + 1 < N and not (yield from g(i + 1)):
                return
            if not (yield ("wait", f"p_full{s}", ph)):
                return
            yield ("mma", [(("G", s), ("P", i)), (("v", s), i)], [("Y2", i)])
            yield ("commit", "y_full", i)
            yield ("commit", f"v_empty{s}", ph)

    yield from body()
    yield ("commit", "drain", 0)
    yield ("wait", "drain", 0, "drain")


def f_gates(w):
    def role(N, mut):
        for i in range(w, N, 2):
            if i >= RING and not (yield ("wait", f"free{i % RING}", i // RING - 1)):
                return
            yield ("write", ("gate", i % RING), i)
            yield ("arrive", f"full{i % RING}", i // RING)
    return role


def f_state(N, mut):
    for i in range(N):
        if not (yield gate_wait(i)):
            return
        yield gate_read(i)
        if mut != "state_does_not_wait" and i and not (yield ("wait", "y1_done", i - 1)):
            return
        yield ("write", "S", i)
        yield ("arrive", "s_full", i)
        if not (yield ("wait", "u_full", i)):
            return
        yield ("read", "U", i)
        yield ("arrive", "u_free", i)


def f_v(half):
    def role(N, mut):
        for i in range(N):
            if not (yield gate_wait(i)) or not (yield ("wait", f"v_full{i & 1}", i >> 1)):
                return
            yield gate_read(i)
            yield ("read", ("v", i & 1), i)
            if mut != "values_do_not_wait" and i and not (yield ("wait", "vp_free", i - 1)):
                return
            yield ("write", ("vp", half), ("V", i))
            yield ("arrive", "vp_full", i)
    return role


def f_out(N, mut):
    for i in range(N):
        if not (yield gate_wait(i)):
            return
        yield gate_read(i)
        if not (yield ("wait", "y_full", i)):
            return
        yield ("read", "Y1", i)
        yield ("read", "Y2", i)
        yield ("arrive", "y_free", i)
        yield ("arrive", f"free{i % RING}", i // RING)


def f_p(half):
    def role(N, mut):
        for i in range(N):
            if not (yield gate_wait(i)):
                return
            yield gate_read(i)
            if not (yield ("wait", f"g_full{i & 1}", i >> 1)):
                return
            if half == 0:  # the other half's columns are not told apart: it only arrives
                yield ("rmw", ("G", i & 1), ("G", i), ("P", i))
            yield ("arrive", f"p_full{i & 1}", i >> 1)
    return role


FWD = {"T": f_tma, "M": f_mma, "G0": f_gates(0), "G1": f_gates(1), "S": f_state, "V0": f_v(0),
       "V1": f_v(1), "O": f_out, "P0": f_p(0), "P1": f_p(1)}


def forward(N, seed, mut=None, **kw):
    return Model(FWD_BARS, {k: f(N, mut) for k, f in FWD.items()}, seed, **kw)


@pytest.mark.parametrize("N", [0, 1, 2, 3, 5, RING + 3])
def test_forward_chain_in_every_schedule(N):
    for seed in range(200):
        forward(N, seed).run()


@pytest.mark.parametrize("mut", ["state_does_not_wait", "values_do_not_wait"])
def test_forward_chain_without_a_wait_is_caught(mut):
    assert count_caught(lambda seed: forward(5, seed, mut), range(200)) > 0


@pytest.mark.parametrize("N", [1, 3])
def test_forward_chain_leaves_nothing_in_flight(N):
    for seed in range(200):
        forward(N, seed, timeouts=True).run()
