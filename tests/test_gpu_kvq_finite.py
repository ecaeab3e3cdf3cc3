"""Attention over the four-bit cache answers numbers: the attention tests once more under a comparison that a NaN fails,
and rows whose unseen slots hold bytes that are no values."""

import numpy as np
import pytest

import kvq_ref as ref
import test_gpu_kvq as base
from kvq_check import assert_within
from test_gpu_kvq import (R, dev, f64, ints, make_cache, queries, tree_masks, values,  # noqa: F401
                          test_attention, test_attention_batches_past_64, test_attention_masks_that_leave_a_row_empty,
                          test_attention_prompt, test_attention_ragged_batch_and_error_rows,
                          test_attention_scale_and_sharp_softmax, test_attention_strided_queries_and_given_outputs,
                          test_offsets_past_32_bits, test_one_query_for_all, test_speculative_steps)

pytestmark = pytest.mark.gpu

loose = base.check_attention


def strict(out, lse, q, cache, prefix, counts, mask, scale):
    """base.check_attention, whose comparison of `out` lets a NaN pass, and what that leaves out."""
    loose(out, lse, q, cache, prefix, counts, mask, scale)
    assert np.isfinite(f64(out)).all()
    assert not np.isnan(f64(lse)).any()


@pytest.fixture(autouse=True)
def numbers_only(monkeypatch):
    monkeypatch.setattr(base, "check_attention", strict)


@pytest.mark.parametrize("S", [700, 4000])
@pytest.mark.parametrize("G,N", [(1, 9), (4, 9), (3, 40)])
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "bf16"), (256, "bf16"), (64, "f32"), (128, "f32"), (256, "f32")])
def test_unseen_slots_may_hold_any_bytes(R, D, dtype, G, N, S):
    """Slots behind the row and tree nodes that a query does not see, filled with every scale byte that stands for no
    float32 number: each query's row is what it is over zeros there."""
    rng = np.random.default_rng(D + G + N + S)
    B, H = 2, 2
    prefix = [S - N - 37, 45]
    cache = make_cache(R, rng, B, H, S, D)
    mask = tree_masks(rng, B, N)[0]
    hidden = [3, N - 2]                                  # nodes that only one query sees each: 0 and 1
    mask[:, :, hidden] = 0
    mask[:, 0, hidden[0]] = mask[:, 1, hidden[1]] = 1
    for b in range(B):
        for at, byte in ((slice(prefix[b] + N, None), 255), (prefix[b] + hidden[0], 254), (prefix[b] + hidden[1], 253)):
            for t in (cache.k_scales, cache.v_scales):
                t[b, :, at] = byte
            for t in (cache.k_codes, cache.v_codes):
                t[b, :, at] = 255                        # -6 everywhere
    q = queries(rng, B, N, H * G, D, dtype)
    out, lse = R.kvq_attention(q, cache, ints(*prefix), mask=dev(mask))
    K, V = values(cache)
    K, V = K.copy(), V.copy()
    for b in range(B):
        for at in (slice(prefix[b] + N, None), prefix[b] + hidden[0], prefix[b] + hidden[1]):
            K[b, :, at], V[b, :, at] = 0, 0
    want, wlse, tol, ltol = ref.attend(f64(q), K, V, prefix, [N] * B, mask, D ** -0.5)
    size = ref.attend_abs(f64(q), K, V, prefix, [N] * B, mask, D ** -0.5)
    # a bf16 probability and a bf16 output are off by half a step each, 2^-8; float32 ones by 2^-24
    step = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    tol = tol + step * size + step * np.abs(want) * 1.01 + 1e-37
    clean = slice(2, None)                               # the queries that see neither node
    assert_within(f64(out)[:, clean], want[:, clean], tol[:, clean])
    assert_within(f64(lse)[:, clean], wlse[:, clean], ltol[:, clean])
