"""The loads and waits of the tile kernel of ep_expert_linear_w4, on the CPU.

A wave's loads are a queue: those asked for first arrive first.  The model runs a
tile's steps by the library's own table (csrc/w4_plan.h) and asks at every barrier
whether the next step's token rows are surely in.  Loads into shared memory are
always made.  Loads into registers for a step that does not come may or may not be:
what no code reads the compiler leaves out, so a wait must hold either way."""
import pytest

import w4_plan


def run(tiles, steps, table, idle=False, dead=False):
    """Steps whose barrier does not wait for the next step's rows.  dead: loads
    after the loop for steps that do not come are made too."""
    lines = tiles < 4
    queue = []                                      # ("rows", step), ("weights" or "scales", steps it is for)
    arrived = 0                                     # loads at the queue's head that are surely in
    bad, rows_asked = [], set()

    def ask_rows(step, n):
        queue.extend([("rows", step)] * n)
        rows_asked.update([step] if n else [])

    def ask_weights(for_steps, n, surely, kind="weights"):
        if not idle and (surely or dead or min(for_steps) < steps):
            queue.extend([(kind, for_steps)] * n)

    # Before the first step: its weights (small tiles: two steps' codes, four steps'
    # scales), three steps' rows, and a wait for the first of those.
    ask_weights((0, 1) if lines else (0,), 8 if lines else 6, True)
    if lines:
        ask_weights((0, 1, 2, 3), 2, True, "scales")
    for s in range(3):
        ask_rows(s, tiles)
    arrived = max(arrived, len(queue) - 2 * tiles)
    assert all(q != ("rows", 0) for q in queue[arrived:])
    for s in range(steps):
        loop = s < steps // 4 * 4
        weights, late, fills, later, idle_later = table(tiles, s % 4, 0 if loop else s % 4 + 1)

        def ask():
            if lines and weights >= 4:              # the codes of two steps, in halves
                for i in range(weights // 4):
                    ask_weights((s + 2 + i,), 4, loop)
            elif lines and weights:
                ask_weights(tuple(range(s + 1, s + 5)), weights, loop, "scales")
            elif weights:
                ask_weights((s + 1,), weights, loop)

        if not idle:
            # Its products have begun, so the first of its weights and its scales are in.
            for kind in ("weights", "scales") if lines else ("weights",):
                mine = [i for i, q in enumerate(queue) if q[0] == kind and s in q[1]]
                assert mine, f"the {kind} of step {s} were not asked for"
                arrived = max(arrived, mine[0] + 1)
        if not late:
            ask()
        arrived = max(arrived, len(queue) - (idle_later if idle else later))
        if s + 1 < steps:
            assert s + 1 in rows_asked, f"the rows of step {s + 1} were not asked for"
            if ("rows", s + 1) in queue[arrived:]:
                bad.append(s)
        if late:
            ask()
        ask_rows(s + 3, fills)
    return bad


CASES = [(tiles, steps) for tiles in (1, 2, 3, 4) for steps in range(4 if tiles < 4 else 1, 30)]


@pytest.mark.parametrize("tiles,steps", CASES)
def test_rows_have_arrived_at_every_barrier(tiles, steps):
    for idle in (False, True):
        for dead in (False, True):
            assert run(tiles, steps, w4_plan.tile_step, idle, dead) == []


def test_the_model_sees_a_count_of_loads_that_are_not_made():
    """The same with the steps after the loop asking for what the loop's do, and
    counting it: right while every load is made, wrong where those for a fourth step
    are left out (K % 512 == 384, up to 96 rows)."""
    def table(tiles, buf, rest):
        return w4_plan.tile_step(tiles, buf, 0)

    for tiles in (1, 2, 3):
        for steps in range(4, 30):
            assert run(tiles, steps, table, dead=True) == []
            assert run(tiles, steps, table) == ([steps - 2] if steps % 4 == 3 else [])
