"""The order of writers and readers of the two angle tables of the ring prefill with first tokens
(prefill_first.cuh), as a model on the CPU: every warp's reads, writes, arrivals and waits in program
order, and vector clocks that only the barriers join. Two accesses of one table, one of them a write,
of different meaning, have to be ordered."""

import random

import pytest

ROPE, SOFTMAX = range(4), range(4, 12)


def _programs(starts, wait_for_run_start):
    """Steps of each warp for row blocks with starts[i]: block i begins a run. A step is (kind, what):
    tables are 0 / 1, the meaning of a write is the block it belongs to and whether it holds turns."""
    programs = {}
    for w in ROPE:
        steps = []
        for i, first in enumerate(starts):
            if i > 0 and starts[i - 1] and wait_for_run_start:
                steps.append(("wait", (f"ready{(i - 1) & 1}", (i - 1) >> 1)))
            if i == 1:
                steps.append(("wait", ("start", 0)))
            steps += [("write", (i & 1, ("angles", i))), ("arrive", f"tab{i & 1}"), ("wait", (f"tab{i & 1}", i >> 1))]
            if first:
                run = sum(starts[:i])
                steps += [("write", ((i + 1) & 1, ("turns", i))), ("arrive", "turn"), ("wait", ("turn", run))]
            steps += [("read", (i & 1, ("angles", i)))] * 2
            if first:
                steps += [("read", ((i + 1) & 1, ("turns", i)))] * 3
            steps.append(("arrive", f"ready{i & 1}"))
        programs[w] = steps
    for w in SOFTMAX:
        programs[w] = [("wait", ("turn", 0)), ("read", (1, ("turns", 0))), ("arrive", "start")]
    return programs


def _counts(name):
    return 8 if name == "start" else 4


def _unordered(programs, seed):
    """Runs one schedule; the pairs of accesses that no barrier orders."""
    rng = random.Random(seed)
    clock = {w: [0] * 12 for w in programs}
    at = dict.fromkeys(programs, 0)
    arrivals, phases = {}, {}            # per barrier: clocks of the open phase; joined clocks of complete ones
    history = {0: [], 1: []}             # accesses of a table: (warp, time, meaning, is a write)
    bad = set()
    while True:
        ready = []
        for w, steps in programs.items():
            if at[w] < len(steps):
                kind, what = steps[at[w]]
                if kind != "wait" or len(phases.get(what[0], [])) > what[1]:
                    ready.append(w)
        if not ready:
            assert all(at[w] == len(s) for w, s in programs.items()), "a wait never ends"
            return bad
        w = rng.choice(ready)
        kind, what = programs[w][at[w]]
        at[w] += 1
        clock[w][w] += 1
        if kind == "arrive":
            arrivals.setdefault(what, []).append(list(clock[w]))
            if len(arrivals[what]) == _counts(what):
                phases.setdefault(what, []).append([max(c) for c in zip(*arrivals.pop(what))])
        elif kind == "wait":
            # (a wait on a parity would not see that its phase is over once the next one is too)
            assert len(phases[what[0]]) == what[1] + 1
            clock[w] = [max(a, b) for a, b in zip(clock[w], phases[what[0]][what[1]])]
        else:
            table, meaning = what
            for other, time, theirs, wrote in history[table]:
                if other != w and theirs != meaning and (wrote or kind == "write") and clock[w][other] < time:
                    bad.add((theirs, meaning))
            history[table].append((w, clock[w][w], meaning, kind == "write"))


RUNS = [[True, False, False, False, False], [True, True, True, True], [True, False, True, False, True, False],
        [True, False, False, True, False, False, True], [True, False, False, False, True, True, False, False]]


@pytest.mark.parametrize("starts", RUNS)
def test_tables_are_ordered(starts):
    for seed in range(60):
        assert not _unordered(_programs(starts, True), seed)


@pytest.mark.parametrize("starts", RUNS)
def test_the_wait_for_the_run_start_is_needed(starts):
    """Without it the table of the block behind a run's start is written while its turns are read."""
    bad = set().union(*(_unordered(_programs(starts, False), seed) for seed in range(60)))
    assert (("turns", 0), ("angles", 1)) in bad
