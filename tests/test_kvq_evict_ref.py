"""The sorted form of eviction's reference is the slot-by-slot one (no GPU needed)."""

import numpy as np
import pytest

import kvq_ref as ref
from test_gpu_kvq_evict_limits import fast_evict, make_scores


@pytest.mark.parametrize("S,keep,sink,recent", [(1, 1, 0, 0), (50, 20, 3, 4), (200, 199, 0, 0), (200, 7, 30, 100), (90, 45, 0, 90)])
def test_same_plans(S, keep, sink, recent):
    rng = np.random.default_rng(S + keep)
    scores, pos = make_scores(rng, 4, 2, S)
    scores[2] = rng.integers(0, 3, (2, S))
    scores[2, 1, ::4] = -np.inf
    lens, seen = [S, max(S - 1, 0), S // 2, S + 1], [S, S, S // 2, S]
    for a, b in zip(ref.evict(scores, pos, lens, seen, keep, sink, recent), fast_evict(scores, pos, lens, seen, keep, sink, recent)):
        assert np.array_equal(a, b)
