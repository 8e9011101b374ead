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
        M.run(M.persistent(rng, parts(rng), rng.choice([2, 4, 6, 10]), rng.choice([2, 4, 6])), rng)


def test_tiles_of_one_step_need_the_barrier_of_all_products():
    """Every other tile of one step lacks a converting warp's work: its accumulators' phases go on without it."""
    with pytest.raises(M.Stuck):
        for seed in range(200):
            rng = random.Random(seed)
            M.run(M.persistent(rng, [1] * 5, 10, 12, last_by_accumulators=True), rng)


def test_the_kernel_of_clusters():
    for seed in range(200):
        rng = random.Random(seed)
        M.run(M.cluster(rng, rng.randint(1, 30), rng.randint(4, 10)), rng)


def test_converting_warps_wait_for_their_own_steps_alone():
    """The copies of another's step can be followed by the next ones in their place before a warp looks."""
    with pytest.raises(M.Stuck):
        for seed in range(200):
            rng = random.Random(seed)
            M.run(M.cluster(rng, 30, rng.choice([4, 5]), waits_for_all=True), rng)
