"""CPU checks of how a linear product ends when one of its waits runs out: a replay of a pair of CTAs, and the test
hook's arguments."""
import random

import pytest

from trainable_block_sparse_cube_b200 import build as vsa_build
from trainable_block_sparse_cube_b200 import vsa


@pytest.fixture(scope="module")
def lib():
    vsa_build.build()
    return vsa.load()


def test_refusals_of_the_test_hook(lib):
    for limit, stall in ((0, 0), (1, 3), (1, -1)):
        assert lib.vsa_linear_set_limits(limit, stall) == 1
    assert lib.vsa_linear_set_limits(2 ** 64 - 1, 2) == 0
    assert lib.vsa_linear_set_limits(10 ** 9, 0) == 0


def _in_flight_at_the_end(rule, stages, total, rng):
    """Replay of a pair's loads and MMAs, step by step: how many loads (of either CTA) land after the pair has
    ended. The MMAs' warp waits `limit` for a step's loads. `rule` "own": a CTA's loads stop when their own wait for
    a free stage runs out, and only then does the even CTA wait for what it knows of; "stop": the kernel's rule, loads
    go on to the step that the MMAs' warp names when it gives up, which waits for them."""
    limit, never = 1.0, float("inf")
    slow = rng.randrange(total)                       # from this step on loads take long
    issue, land, commit = [[], []], [[], []], []
    now, gave_up, m = 0.0, None, total                # the MMAs' warp
    given = [None, None]
    for j in range(total):
        free = commit[j - stages] if j >= stages else 0.0
        for r in (0, 1):
            before = issue[r][-1] if j else 0.0
            at = max(before, free) + rng.uniform(0, 0.01)
            if rule == "own" and (given[r] is not None or free > before + limit):
                given[r] = given[r] or before + limit
                at = never
            if rule == "stop" and j >= m + stages:
                at = never
            issue[r].append(at)
            land[r].append(at + rng.uniform(0.1, 0.4) + (rng.uniform(0, 5) if j >= slow else 0))
        there = max(land[0][j], land[1][j])
        if gave_up is None and there > now + limit:
            gave_up, m = now + limit, j
        if gave_up is None:
            now = max(now, there) + 0.05
            commit.append(now + 0.1)
        else:
            commit.append(never)
    issued = [[t for t, i in zip(land[r], issue[r]) if i < never] for r in (0, 1)]
    end = max([now + 0.1, gave_up or 0.0] + [i for r in (0, 1) for i in issue[r] if i < never])
    if rule == "own":
        end = max([end] + [g for g in given if g])
        if given[0]:                                  # waits for its stages, whose loads it issued itself
            end = max([end] + [min(t, end + limit) for t in issued[0]])
    elif gave_up is not None:
        end = max([end] + [t for r in (0, 1) for t in land[r][m:min(total, m + stages)]])
    return sum(t > end for r in (0, 1) for t in issued[r])


def test_no_load_is_in_flight_when_a_pair_has_given_up():
    rng = random.Random(1)
    cases = [(rng.randint(2, 16), rng.randint(1, 60), rng.random()) for _ in range(2000)]
    left = {rule: [_in_flight_at_the_end(rule, st, n, random.Random(seed)) for st, n, seed in cases]
            for rule in ("own", "stop")}
    assert not any(left["stop"])
    assert any(x for x, (st, n, _) in zip(left["own"], cases) if n <= st)     # what the replay is able to find
    assert any(x for x, (st, n, _) in zip(left["own"], cases) if n > st)
