"""The plan on a B200 when tables or the ring hold ids of no block: the step
does not happen, bit for bit as in the oracle."""
import numpy as np
import pytest

from test_gpu_paged import check_plan, pool_state

pytestmark = pytest.mark.gpu


def step(seed=0, B=40, bs=16, width=30):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, 200, B)
    new = np.where(rng.random(B) < 0.3, -1, rng.integers(0, 60, B))
    ctx[:4], new[:4] = [10, 0, 33, 32], [7, 20, -1, 5]
    table, ring, state, n = pool_state(rng, ctx, bs, 200, width)
    return ctx, new, table, ring, state, bs, n


@pytest.mark.parametrize("capacity", [2048, 5000])       # either side of one block's work
@pytest.mark.parametrize("bad", ["-1", "n", "2^31-1", "-2^31"])
@pytest.mark.parametrize("where", ["ring, first", "ring, last", "leaving", "part-filled"])
def test_a_bad_id_stops_the_step(cuda, where, bad, capacity):
    ctx, new, table, ring, state, bs, n = step()
    bad = {"-1": -1, "n": n, "2^31-1": 2 ** 31 - 1, "-2^31": -2 ** 31}[bad]
    assert check_plan(ctx, new, table, ring, state, bs, capacity)["status"] == "ok"
    grow = np.maximum(new, 0)
    take = int(np.where(new < 0, 0, -(-(ctx + grow) // bs) - -(-ctx // bs)).sum())
    if where.startswith("ring"):
        ring[(state[0] + (0 if "first" in where else take - 1)) % n] = bad
    else:
        table[(2, 2) if where == "leaving" else (0, 0)] = bad
    for in_place in (False, True):
        want = check_plan(ctx, new, table, ring, state, bs, capacity, in_place=in_place)
        assert want["status"] == "shape"


def test_ids_that_the_step_does_not_use_are_not_looked_at(cuda):
    ctx, new, table, ring, state, bs, n = step(1)
    grow = np.maximum(new, 0)
    take = int(np.where(new < 0, 0, -(-(ctx + grow) // bs) - -(-ctx // bs)).sum())
    ring[(state[0] + take) % n] = n                # the first that stays free
    table[3, 1] = -7                               # a full block of a request that goes on
    table[0, 29] = n + 5                           # past the request's blocks
    assert check_plan(ctx, new, table, ring, state, bs, 4000)["status"] == "ok"


@pytest.mark.parametrize("where", ["ring", "leaving", "part-filled"])
@pytest.mark.parametrize("capacity", [2048, 4000])
def test_too_few_blocks_come_before_a_bad_id(cuda, capacity, where):
    """What does not fit is reported as such; the ids are then not looked at."""
    ctx, new, table, ring, state, bs, n = step(2)
    if where == "ring":
        ring[state[0]] = -1
    else:
        table[(2, 2) if where == "leaving" else (0, 0)] = -1
    assert check_plan(ctx, new, table, ring, [state[0], 3], bs, capacity)["status"] == "blocks"
