"""Eviction at the limits of its forms: four waves hold a head's keys up to 4096 slots of capacity, sixteen up to 36864,
longer heads are read again every pass; a plan of at most 256 moves is carried out by the selecting workgroup."""

import numpy as np
import pytest

from test_gpu_kvq import R, make_cache, run_evict  # noqa: F401

pytestmark = pytest.mark.gpu


def rank(scores, pos, n, seen, keep, sink, recent):
    """kvq_ref.evict's plan for one head of n slots, by sorting arrays (its loop over slots is slow for long heads)."""
    s, p = scores[:n].astype(np.float64), pos[:n].astype(np.int64)
    protected = (p < sink) | (p >= seen - recent)
    kind = np.where(protected, 0, np.where(np.isnan(s), 2, 1))
    by = np.where(kind == 1, -np.nan_to_num(s, nan=0.0, posinf=np.inf, neginf=-np.inf), 0.0)
    m = min(n, keep)
    kept = np.sort(np.lexsort((np.arange(n), by, kind))[:m])
    source = np.arange(m)
    source[np.setdiff1d(np.arange(m), kept)] = kept[kept >= m]
    return source


def fast_evict(scores, positions, lengths, seen, keep, sink, recent):
    B, H, S = scores.shape
    new_len, source = np.full(B, -1, np.int32), np.full((B, H, keep), -1, np.int32)
    for b in range(B):
        n = int(lengths[b])
        if not 0 <= n <= S:
            continue
        new_len[b] = min(n, keep)
        for h in range(H):
            source[b, h, :new_len[b]] = rank(scores[b, h], positions[b, h], n, int(seen[b]), keep, sink, recent)
    return new_len, source


@pytest.fixture(autouse=True)
def sorted_reference(monkeypatch):
    import kvq_ref as ref
    monkeypatch.setattr(ref, "evict", fast_evict)


def make_scores(rng, B, H, S):
    scores = np.exp(2 * rng.standard_normal((B, H, S))).astype(np.float32)
    scores[0, 1] = np.round(scores[0, 1])                # great ties, across waves
    scores[1, 0, ::5] = np.nan
    scores[1, 0, 3::11] = np.inf
    pos = np.tile(np.arange(S, dtype=np.int32), (B, H, 1))
    pos[1, 1] = pos[1, 1][::-1]                          # the protected ones at the other end
    return scores, pos


@pytest.mark.parametrize("S", [4095, 4096, 4097, 20001, 32768, 36863, 36864, 36865])
@pytest.mark.parametrize("moves", ["few", "half", "few kept"])
@pytest.mark.parametrize("D", [128, 256])
def test_capacities_on_both_sides_of_each_form(R, S, moves, D):
    """Lengths equal to the capacity, one less, and a step's rows above what is kept."""
    keep = {"few": S - 200, "half": S // 2 + 1, "few kept": 255}[moves]
    rng = np.random.default_rng(S + D + keep)
    B, H = 3, 2
    cache = make_cache(R, rng, B, H, S, D)
    scores, pos = make_scores(rng, B, H, S)
    run_evict(R, cache, scores, pos, [S, S - 1, min(S, keep + 6)], [S] * B, keep, 4, 30, moves == "few")


@pytest.mark.parametrize("S,gap", [(4096, 256), (4096, 257), (36864, 256), (36864, 257), (40000, 256), (40000, 257)])
@pytest.mark.parametrize("apart", [False, True])
def test_one_launch_and_two(R, S, gap, apart):
    """The most moves that one launch makes, and one more, as the rows that leave and as the rows that stay."""
    for keep in (S - gap, gap):
        rng = np.random.default_rng(S + keep)
        cache = make_cache(R, rng, 2, 2, S, 64)
        scores, pos = make_scores(rng, 2, 2, S)
        run_evict(R, cache, scores, pos, [S, S - 1], [S, S], keep, 2, 5, apart)


@pytest.mark.parametrize("S", [4096, 36864, 40000])
def test_short_rows_in_long_caches(R, S):
    """Lengths far below the capacity that chose the form, nothing to evict among them."""
    rng = np.random.default_rng(S)
    B, H, keep = 5, 2, 300
    cache = make_cache(R, rng, B, H, S, 64)
    scores, pos = make_scores(rng, B, H, S)
    run_evict(R, cache, scores, pos, [1, keep, keep + 1, 1000, 0], [S] * B, keep, 0, 0, True)
