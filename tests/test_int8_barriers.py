"""The barrier protocols of the 8-bit products under random schedules: nobody waits for ever, and no phase is taken for another."""
import random

import barrier_model as M
import pytest


def parts(rng):
    """Whole tiles, and shares of tiles of at least one step behind them."""
    return [rng.choice([1, 1, 2, 3, 5])] * rng.randint(1, 8) + [rng.randint(1, 4) for _ in range(rng.randint(0, 3))]


def test_the_persistent_kernel():
    for seed in range(120):
        rng = random.Random(seed)
        M.run(M.persistent(parts(rng), rng.choice([2, 4, 6, 10]), rng.choice([2, 4, 6])), rng)


def test_tiles_of_one_step_need_the_barrier_of_all_products():
    """Every other tile of one step lacks a converting warp's work: its accumulators' phases go on without it."""
    with pytest.raises(M.Stuck):
        for seed in range(200):
            rng = random.Random(seed)
            M.run(M.persistent([1] * 5, 10, 12, last_by_accumulators=True), rng)
