"""The calls of linear_plans.py reach every kernel instance (host only)."""
from __future__ import annotations

import pytest

import linear_plans as lp


@pytest.fixture(scope="module")
def reached():
    return {k for row in lp.ROWS for k in lp.plans(row)}


def test_every_instance_is_reached(reached):
    want = set(lp.instances())
    assert len(want) == 157
    got = {k[:-1] for k in reached}
    assert want - got == set(), "no call of linear_plans.py launches these: search again"
    assert got - want == set(), "instances that linear_plans.py does not know"


def test_every_split_is_reached(reached):
    # pairs of an instance and a split: none, all tiles, those of the last round
    assert len(reached) == lp.PAIRS, "search again"
    for split in ("no", "all", "last"):
        assert sum(k[-1] == split for k in reached) > 90


def test_rows_are_small_enough_to_check():
    # sums of integers up to 9 stay exact in binary32, also times a scale of 2^12
    for M, N, K, *_ in lp.ROWS:
        assert max(M, 2 * N, K) * 12 < 1 << 24 and max(M * N, N * K, M * K) <= 1.4e8
