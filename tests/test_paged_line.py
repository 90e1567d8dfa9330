"""The many-row kernel's schedule, replayed on the host."""

import numpy as np
import pytest

from tests._paged_line import runs, waits_for_itself

BLOCKING = [([8192, 8192, 0, 8192, 8192], [512, 512, 1, 512, 512], 4, 8, -1, -1),
            ([100, 8192], [4000, 512], 4, 8, -1, 0)]


@pytest.mark.parametrize("batch", BLOCKING)
def test_items_without_keys_stay_out_of_the_ring(batch):
    """With them as segments a loader's look-ahead would come back to the slot of the tile
    that it still holds; without them it reaches two slots at most."""
    parts = runs(*batch)
    assert any(waits_for_itself(p, True) for p in parts)
    assert not any(waits_for_itself(p, False) for p in parts)


def test_random_batches_never_wait_for_themselves():
    rng = np.random.default_rng(0)
    longest = 0
    for _ in range(400):
        B = int(rng.integers(1, 80))
        lens = rng.integers(0, rng.choice([50, 500, 9000]), B) * (rng.random(B) > 0.3)
        n = rng.integers(0, rng.choice([3, 40, 400]), B)
        parts = runs(lens, n, int(rng.choice([1, 4, 16])), int(rng.choice([1, 3, 8])), int(rng.choice([-1, 30])),
                     int(rng.choice([-1, 0])))
        longest = max(longest, max(len(p) for p in parts))
        assert not any(waits_for_itself(p, False) for p in parts)
    assert longest > 8
