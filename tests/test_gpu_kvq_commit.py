"""The four-bit cache's commit for every head size (rows of scales have 2, 4 and 8 bytes), and for a cache of one slot."""

import numpy as np
import pytest

from test_gpu_kvq import R, arrays, dev, ints, make_cache  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["heads", "rows", "slots"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_commit_of_every_head_size(R, D, layout):
    rng = np.random.default_rng(D)
    B, H, S, N = 5, 3, 90, 64
    cache = make_cache(R, rng, B, H, S, D, layout)
    old = arrays(cache)
    path = np.full((B, 40), -1, np.int32)
    path[0, :40] = [0, *np.sort(rng.choice(np.arange(1, N), 39, replace=False))]     # rows past one turn of a workgroup
    path[1, :3] = [0, 1, 2]                              # stays in place
    path[2, :2] = [0, 63]
    path[3, :3] = [0, 5, 4]                              # not increasing
    path[4, :2] = [0, 63]                                # past the cache
    alen, prefix = [39, 2, 1, 2, 1], [3, 0, 26, 4, 27]
    n = R.kvq_commit(cache, ints(*prefix), dev(path), ints(*alen), N)
    assert n.tolist() == [43, 3, 28, -1, -1]
    for x0, x1 in zip(old, arrays(cache)):
        for b in (0, 2):
            p = path[b, :alen[b] + 1]
            x0[b][:, prefix[b]:prefix[b] + len(p)] = x0[b][:, prefix[b] + p].copy()
        assert np.array_equal(x0, x1)


@pytest.mark.parametrize("step", [0, 16, 1 << 25])
def test_commit_of_one_slot(R, step):
    rng = np.random.default_rng(3)
    cache = make_cache(R, rng, 2, 2, 1, 64)
    old = arrays(cache)
    odd = R.KVQCache(*(t.as_strided(t.shape, (t.stride(0), t.stride(1), step, 1))
                       for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)))
    n = R.kvq_commit(odd, ints(0, 1), dev(np.zeros((2, 1), np.int32)), ints(0, 0), 1)
    assert n.tolist() == [1, -1]
    assert all(np.array_equal(a, b) for a, b in zip(old, arrays(cache)))
