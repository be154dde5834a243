"""The waits of fa_kv_weights_tile_kernel's roles on one another, in a model without a GPU (weights_roles)."""
import random

import pytest

import weights_roles as roles


def case(B, H, Hk, T, d, page, lens, new, left):
    return (B, H, Hk, T, d, lens, new, left, 0), -(-max(lens) // page) * page


@pytest.mark.parametrize("decay", [1.0, 0.5, 0.0])
@pytest.mark.parametrize("c", roles.CASES)
def test_units_without_row_blocks_behind_one_that_has_some(c, decay):
    """Every cluster comes to its end; had the side warp looked for its next block before it handed over the one it
    holds, some would not, so these are cases of the GPU tests."""
    args, capacity = case(*c)
    bad, ranks, uneven, units = roles.stalls(False, *args, decay, capacity)
    assert bad == 0
    if decay == 0.5:
        assert units > (3 if uneven else roles.UNITS)
        assert roles.stalls(True, *args, decay, capacity)[0] > 0


def test_the_cases_cover_both_orders_and_clusters_of_two():
    kinds = [roles.stalls(False, *case(*c)[0], 0.5, case(*c)[1])[1:3] for c in roles.CASES]
    assert {(1, False), (2, True), (2, False)} <= set(kinds)


def test_the_waits_can_be_met_whatever_the_sizes():
    rng = random.Random(3)
    seen = set()
    for _ in range(250):
        B, Hk = rng.randint(1, 24), rng.choice([1, 2, 4, 8])
        H, T = Hk * rng.choice([1, 2, 4, 8]), rng.choice([rng.randint(7, 127), rng.randint(128, 2048)])
        if H // Hk * T <= 48:
            continue
        most = rng.choice([500, 4000, 30000])
        lens = [rng.randint(-1, most) for _ in range(B)]
        new = None if rng.random() < 0.4 else [rng.choice([0, 1, rng.randint(0, T), T]) for _ in range(B)]
        bad, ranks, uneven, units = roles.stalls(
            False, B, H, Hk, T, rng.choice([64, 128]), lens, new, rng.choice([-1, -1, 0, rng.randint(1, 3000)]),
            rng.choice([-1, 0, 0, 5]), rng.choice([1.0, 0.5]), max(max(lens), 1), rng.choice([152, 152, 8]))
        assert bad == 0
        seen.add((ranks, uneven, units > roles.UNITS))
    assert {(1, False, True), (2, False, True), (2, True, True), (4, False, False)} <= seen
