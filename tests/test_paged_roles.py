"""The roles of a paged-attention CTA under random schedules (paged_roles.py)."""
import random

import pytest

from paged_roles import LAYOUTS, RING, run

EMPTY_RUNS = {
    "first": [0] * 40 + [3, 1, 2],
    "between": [5] + [0] * (2 * RING) + [1] + [0] * RING + [2, 2],
    "last": [1, 4] + [0] * 30,
    "all": [0] * 20,
    "scattered": [0, 1, 0, 0, 2, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 1, 0] * 3,
}


@pytest.mark.parametrize("layout", list(LAYOUTS))
def test_random_units(layout):
    rng = random.Random(0)
    for seed in range(60):
        most = rng.choice([1, 1, 2, 3, 9, 30])
        units = [rng.choice([0, rng.randint(1, most)]) for _ in range(rng.randint(1, 20))]
        assert run(units, LAYOUTS[layout], seed) == "ok", (units, seed)


@pytest.mark.parametrize("units", list(EMPTY_RUNS))
@pytest.mark.parametrize("layout", list(LAYOUTS))
def test_units_without_a_key(layout, units):
    for seed in range(5):
        assert run(EMPTY_RUNS[units], LAYOUTS[layout], seed) == "ok"


@pytest.mark.parametrize("units", ["first", "between"])
@pytest.mark.parametrize("layout", list(LAYOUTS))
def test_units_without_a_key_have_to_stay_out_of_the_ring(layout, units):
    # with them in it, an issuer's look-ahead for the next S waits for places that only its own
    # P V cursor gives back
    assert run(EMPTY_RUNS[units], LAYOUTS[layout], 0, empty_in_ring=True) == "deadlock"
