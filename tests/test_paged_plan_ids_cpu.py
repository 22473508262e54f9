"""The plan's oracle on tables and rings that hold ids of no block: a step
that would take, give back or fill further such a block does not happen."""
import numpy as np
import pytest

from oracle import paged as O

CASE = dict(ctx=[10, 0, 33, 32], new=[7, 20, -1, 5], bs=16, capacity=40)
TABLE = np.array([[3, -1, -1], [-1, -1, -1], [4, 5, 6], [7, 8, -1]])
RING = np.array([0, 1, 2, 9, 10, 11, 12, 3, 4, 5, 6, 7, 8])


def plan(table, ring, state=(0, 7)):
    return O.plan(CASE["ctx"], CASE["new"], table, ring, state, CASE["bs"], CASE["capacity"])


def test_the_step_without_a_bad_id_happens():
    assert plan(TABLE, RING)["status"] == "ok"


@pytest.mark.parametrize("bad", [-1, 13, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("where", ["ring", "leaving", "part-filled"])
def test_a_bad_id_stops_the_step(bad, where):
    table, ring = TABLE.copy(), RING.copy()
    if where == "ring":
        ring[3] = bad                             # the step takes four blocks
    else:
        table[(2, 1) if where == "leaving" else (0, 0)] = bad
    r = plan(table, ring)
    assert r["status"] == "shape"
    assert np.array_equal(r["table"], table) and np.array_equal(r["ring"], ring)
    assert (r["slots"] == -1).all() and not r["cu"].any()
    assert r["ctx"].tolist() == CASE["ctx"] and r["state"].tolist() == [0, 7]


def test_ids_that_the_step_does_not_use_are_not_looked_at():
    table, ring = TABLE.copy(), RING.copy()
    ring[4] = 99                                  # behind the four that it takes
    table[3, 1] = 99                              # a full block of a request that goes on
    table[0, 1] = -5                              # past the request's blocks
    assert plan(table, ring)["status"] == "ok"
