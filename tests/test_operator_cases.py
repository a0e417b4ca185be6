"""The measured cases' inputs (perf/operators.py) on the CPU: what the calls of
include/moe_block.h require of them."""

import random

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import perf.operators as cases
import w4_dequant_expert_amd as moe


def test_routing_tables_hold_every_entry_the_calls_may_read(monkeypatch):
    monkeypatch.setattr(cases, "DEV", "cpu")
    rng = random.Random(4)
    some = [(1, 256, 8, 32), (37, 300, 8, 32), (64, 1024, 4, 16), (511, 256, 8, 128)]
    some += [(rng.randint(1, 400), E, rng.randint(1, min(E, 8)), rng.choice([16, 32, 64, 128, 256]))
             for E in (4, 9, 64, 200) for _ in range(4)]
    for T, E, k, tile in some:
        r = cases._routing(cases._gen(T), T, E, k, tile)
        d = moe.make_dims(T, 64, 64, E, k, 1, tile, 16)
        n, rows = int(r["n_blocks"]), r["blocks"].numpy()
        assert rows.shape == (moe.moe_max_blocks(d), 4), (T, E, k, tile)
        # the entries in use cover every row once, and those behind them are empty
        assert rows[:n, 2].sum() == T * (k + 1) and (rows[:n, 2] > 0).all() and not rows[n:].any()
        assert np.array_equal(rows[:n, 1], np.cumsum(rows[:n, 2]) - rows[:n, 2])
