"""The barrier schedule of the tensor-core tree attention, as a model: whoever is
slow, nobody waits for a phase that has gone by.

A CTA's tensor-core issuer and its two softmax groups meet on mbarriers that are
told apart by parity alone: a wait for parity p passes while the number of
completed phases has the other parity, so a waiter that misses a phase and the
one after it waits for ever.  The issuer and the groups are programs of signals
and waits; every interleaving of them is walked for short lists of segments."""
import itertools

import pytest

# (mode, key tiles): alternate tiles of one Q tile, two Q tiles, a pair of items
SEGMENTS = [("alternate", 1), ("alternate", 2), ("alternate", 3), ("shared", 1), ("shared", 2), ("pair", 1)]


def steps_of(mode, tiles):
    """Softmax groups of a segment's steps, in order."""
    return [u & 1 for u in range(tiles if mode == "alternate" else 2 * tiles)]


def programs(segments, one_step_commits_both):
    """Issuer and groups as lists of ("wait", barrier, phase) and ("signal",
    barrier); a phase of `stat` and `epi` is two signals, of the others one.
    Step u of a segment: scores s, then weights ready, then the product with V,
    whose last one of each group completes a phase of its accumulator, done."""
    issuer, group = [], [[], []]
    n_s, both, joins = [0, 0], 0, 0
    for nd, (mode, tiles) in enumerate(segments):
        order = steps_of(mode, tiles)
        first = list(n_s)                    # phases of s and ready before the segment
        for u in range(-2, len(order)):
            if u >= 0:
                issuer.append(("wait", f"ready{order[u]}", first[order[u]] + u // 2))
                if u + 2 >= len(order):
                    issuer.append(("signal", f"done{order[u]}"))
            if u + 2 < len(order):
                issuer.append(("signal", f"s{order[u + 2]}"))
        for g in order:
            group[g] += [("wait", f"s{g}", n_s[g]), ("signal", f"ready{g}")]
            n_s[g] += 1
        one_step = len(order) == 1
        if one_step and one_step_commits_both:
            issuer.append(("signal", "done1"))
        skip = one_step and not one_step_commits_both
        phase = (nd, nd if one_step_commits_both else both)
        for g in range(2):
            if not (g and skip):
                group[g].append(("wait", f"done{g}", phase[g]))
            if mode == "alternate":
                group[g] += [("signal", "stat"), ("wait", "stat", joins)]
                if g or not skip:
                    group[g].append(("wait", f"done{g ^ 1}", phase[g ^ 1]))
                group[g] += [("signal", "epi"), ("wait", "epi", joins)]
        both += not one_step
        joins += mode == "alternate"
    return [issuer, *group]


def stuck(progs):
    """A reachable state in which somebody is not done and nobody can go on, or None."""
    seen, todo = set(), [(0, 0, 0)]
    while todo:
        at = todo.pop()
        if at in seen:
            continue
        seen.add(at)
        count = {}
        for prog, pc in zip(progs, at):
            for op in prog[:pc]:
                if op[0] == "signal":
                    count[op[1]] = count.get(op[1], 0) + 1
        moved = False
        for i, (prog, pc) in enumerate(zip(progs, at)):
            if pc == len(prog):
                continue
            op = prog[pc]
            phases = count.get(op[1], 0) // (2 if op[1] in ("stat", "epi") else 1)
            if op[0] == "wait" and phases & 1 == op[2] & 1:
                continue                     # by parity: this phase is still open
            if op[0] == "wait":              # passes: the phase meant has completed
                assert phases > op[2], (progs, at)
            todo.append(tuple(p + (j == i) for j, p in enumerate(at)))
            moved = True
        if not moved and any(pc < len(p) for p, pc in zip(progs, at)):
            return at
    return None


@pytest.mark.parametrize("length", [1, 2, 3, 4])
def test_no_interleaving_misses_a_phase(length):
    for segments in itertools.product(SEGMENTS, repeat=length):
        assert stuck(programs(segments, False)) is None, segments


def test_a_phase_without_a_step_of_its_group_can_be_missed():
    """Why a segment of one step has no phase of the second group's accumulator."""
    assert stuck(programs([("pair", 1), ("alternate", 1)], True)) is not None
    assert stuck(programs([("alternate", 2), ("alternate", 1)], True)) is None
