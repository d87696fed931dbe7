"""The loads and waits of the tile kernel of ep_expert_linear_i8, on the CPU.

A wave's accesses are a queue: those asked for first are done first.  The model runs the
stages of items one after the other by the library's own table (csrc/i8_plan.h), with
each item's stores and loads of scales between them, and asks behind every quarter
whether what the next one reads is surely in, and before every load whether every wave
has read what it writes over."""
import itertools

import pytest

import i8_plan

LOADS = 16
TOKENS, TILE = range(8), [(8 + 2 * q, 9 + 2 * q) for q in range(4)]


def run(items, table, early=1):
    """items: (stages, stores) of each; early: the stages of an item in which the stores
    before it are counted.  Waits that leave something on the way, as (item, stage,
    quarter)."""
    queue, arrived, bad = [], 0, []
    rest = table(0)[0]                              # quarter 0 asks for a next stage's loads from here on
    queue += [(0, g) for g in range(LOADS)] + [(1, g) for g in range(rest)]
    arrived = LOADS                                 # stage 0 is waited for
    flat, before = 0, 0
    # When each part of a stage was read, in quarters, and behind which barrier that is
    # known: behind its own quarter, but those of quarter 3 one later.
    known = {}

    def reads(stage, parts, quarter):
        for g in parts:
            known[stage, g] = quarter + 1 + (quarter % 4 == 3)

    for n, (stages, stores) in enumerate(items):
        queue += [("scales", n)] * 2
        # an item begins with its token tiles and weight tiles 0
        assert all((flat, g) in queue[:arrived] for g in (*TOKENS, *TILE[0]))
        for s in range(stages):
            for q in range(4):
                first, last, later = table(q)
                now = 4 * flat + q
                reads(flat + (q == 3), TILE[(q + 1) % 4], now)
                if q == 3:
                    reads(flat + 1, TOKENS, now)
                for g in range(first, last):
                    # into the slot of this stage (quarter 0: of the one before): its rows
                    # have been read by every wave (those of stage 0's beginning before
                    # the loop, and in stage 0 the other slot is empty)
                    over = flat - (q == 0)
                    assert over < 0 or known.get((over, g), 0) <= now, (n, s, q, g)
                    queue.append((over + 2, g))
                more = stores + 2 if before == stores and s < early else 0
                arrived = max(arrived, len(queue) - later - more)
                need = [(flat, g) for g in TILE[q + 2]] if q < 2 else [(flat + 1, g) for g in (*TOKENS, *TILE[0])] if q == 2 \
                    else [(flat + 1, g) for g in TILE[1]]
                if any(x not in queue[:arrived] for x in need):
                    bad.append((n, s, q))
            flat += 1
        arrived = max(arrived, len(queue) - LOADS)
        assert all(x in queue[:arrived] for x in [("scales", n)]), "scales"
        queue += [("store", n)] * stores
        before = stores
    return bad


@pytest.mark.parametrize("stores", [4, 8, 12, 16, 24, 32])
def test_every_wait_holds(stores):
    for stages in itertools.product((1, 2, 3, 5), repeat=4):
        assert run([(s, stores) for s in stages], i8_plan.quarter) == []
    for heights in itertools.product((stores, 8), repeat=4):
        for stages in (1, 2, 4):
            assert run([(stages, h) for h in heights], i8_plan.quarter) == []


def test_counts_fit_their_field():
    assert max(i8_plan.quarter(q)[2] for q in range(4)) + 32 + 2 <= 63


def test_each_load_is_asked_for_once():
    assert sorted(g for q in range(4) for g in range(*i8_plan.quarter(q)[:2])) == list(range(LOADS))


def test_the_model_sees_stores_counted_a_stage_too_long():
    """In an item's second stage too, some of whose rows were asked for behind them."""
    bad = run([(4, 32)] * 3, i8_plan.quarter, early=2)
    assert bad and {s for _, s, _ in bad} == {1}


def test_the_model_sees_a_load_too_many():
    for q in range(4):
        def table(p):
            first, last, later = i8_plan.quarter(p)
            return first, last, later + (p == q)
        assert run([(4, 16)] * 3, table)
