"""The four-bit cache on the GPU against its 64-bit reference (kvq_ref): append and read back (exact), attention,
scores, eviction (exact), and a speculative step that uses them together."""

import numpy as np
import pytest

import kvq_ref as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def R():
    import torch
    import rejection_sampling_verify_10_amd as R
    assert torch.cuda.is_available(), "GPU test without a GPU"
    R.lib()
    return R


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def ints(*v):
    return dev(np.array(v, np.int32))


def f64(t):
    return t.double().cpu().numpy()


def make_cache(R, rng, B, H, S, D, layout="heads", lo=120, hi=129, fill=None):
    """A cache of random codes, scales 2^(lo-127) .. 2^(hi-127); `fill` sets every byte instead."""
    import torch
    lead = {"heads": (B, H, S), "rows": (B, S, H), "slots": (S, B, H)}[layout]
    order = {"heads": (0, 1, 2), "rows": (0, 2, 1), "slots": (1, 2, 0)}[layout]
    parts = []
    for _ in range(2):
        for last, low, high in ((D // 2, 0, 256), (D // 32, lo, hi + 1)):
            a = rng.integers(low, high, (*lead, last)).astype(np.uint8) if fill is None else np.full((*lead, last), fill, np.uint8)
            parts.append(torch.from_numpy(a).cuda().permute(*order, 3))
    return R.KVQCache(*parts)


def values(cache):
    """The cache's rows as float64 [B, H, S, D], K and V."""
    n = [t.cpu().numpy() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
    return ref.decode(n[0], n[1]), ref.decode(n[2], n[3])


def arrays(cache):
    return [t.cpu().numpy().copy() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]


def queries(rng, B, N, Hq, D, dtype, size=1.0):
    import torch
    q = torch.from_numpy((size * rng.standard_normal((B, N, Hq, D))).astype(np.float32)).cuda()
    return q.bfloat16() if dtype == "bf16" else q


def tree_masks(rng, B, N):
    m = np.zeros((B, N, N), np.uint8)
    par = np.zeros((B, N), np.int64)
    for b in range(B):
        for n in range(N):
            if n:
                par[b, n] = rng.integers(max(0, n - 5), n)
                m[b, n] = m[b, par[b, n]]
            m[b, n, n] = 1
    return m, par


def check_attention(out, lse, q, cache, prefix, counts, mask, scale):
    """Every output within the roundings that the arithmetic allows."""
    import torch
    K, V = values(cache)
    K, V = np.nan_to_num(K, nan=0.0), np.nan_to_num(V, nan=0.0)      # rows no query sees may hold anything
    B, N, Hq, D = q.shape
    counts = [N] * B if counts is None else counts
    want, wlse, tol, ltol = ref.attend(f64(q), K, V, prefix, counts, mask, scale)
    size = ref.attend_abs(f64(q), K, V, prefix, counts, mask, scale)
    # with bf16 queries a probability rounds to bf16 before it meets V (2^-8), and so does the output
    p_round, o_round = (2.0 ** -8, 2.0 ** -8) if q.dtype == torch.bfloat16 else (U, U)
    tol = tol + p_round * size + o_round * np.abs(want) * 1.01
    got, glse = f64(out), f64(lse)
    bad = np.abs(got - want) > tol + 1e-37
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], want[bad][:3], tol[bad][:3])
    assert np.array_equal(np.isneginf(glse), np.isneginf(wlse))
    live = ~np.isneginf(wlse)
    off = np.abs(glse - np.where(live, wlse, 0.0))[live]
    assert (off <= ltol[live] + 1e-30).all(), (off.max(), ltol[live][off.argmax()])
    assert (got[~live] == 0).all()


# ---- append and read ----

@pytest.mark.parametrize("layout", ["heads", "rows", "slots"])
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "bf16"), (256, "bf16"), (64, "f32"), (128, "f32"), (256, "f32")])
def test_append_and_read(R, D, dtype, layout):
    import torch
    rng = np.random.default_rng(D)
    B, N, H, S = 5, 13, 3, 40
    x = rng.standard_normal((B, N, 2, H, D)) * np.exp2(rng.integers(-20, 20, (B, N, 2, H, 1)))
    x[0, 0, 0, 0, :32] = 0                                           # an empty block
    x[0, 1, 1, 1, 32:64] = np.repeat([7, 6, 5, 3.5, 2.5, 1.75, 1.25, .75], 4)      # ties, the largest value
    x[0, 2, 0, 2, :32] = np.array([7.03125, -7, .25, -.25] * 8)
    x[1, 3, 0, 0, :] *= 2.0 ** -100                                  # below the smallest scale
    x[1, 4, 1, 0, :] *= 2.0 ** 90
    kv = torch.from_numpy(x.astype(np.float32)).cuda()
    kv = kv.bfloat16() if dtype == "bf16" else kv
    k, v = kv[:, :, 0], kv[:, :, 1]                                  # strided views of one projection
    cache = make_cache(R, rng, B, H, S, D, layout, fill=0xEE)
    before = arrays(cache)
    prefix, counts = [3, 27, 0, -1, 28], [13, 13, 7, 13, 13]         # fits, fits exactly, partial, unused, too far
    R.kvq_append(cache, k, v, ints(*prefix), counts=ints(*counts))
    for out_type in (torch.bfloat16, torch.float32):
        rk, rv = R.kvq_read(cache, ints(*prefix), N, counts=ints(*counts), dtype=out_type)
        for got, src in ((rk, k), (rv, v)):
            want, _ = ref.quantise(f64(src))
            for b in range(B):
                n = counts[b] if prefix[b] >= 0 and prefix[b] + counts[b] <= S else 0
                assert np.array_equal(f64(got[b, :n]), want[b, :n]), (b, out_type)
                assert (f64(got[b, n:]) == 0).all()
    scales = ref.quantise(f64(k))[1]
    after = arrays(cache)
    for b in range(B):
        n = counts[b] if prefix[b] >= 0 and prefix[b] + counts[b] <= S else 0
        for i, (x0, x1) in enumerate(zip(before, after)):
            assert np.array_equal(x0[b, :, :max(prefix[b], 0)], x1[b, :, :max(prefix[b], 0)])
            assert np.array_equal(x0[b, :, max(prefix[b], 0) + n:], x1[b, :, max(prefix[b], 0) + n:]), (b, i)
        if n:
            assert np.array_equal(after[1][b, :, prefix[b]:prefix[b] + n], scales[b, :n].swapaxes(0, 1))
    # all of it again without counts: batch row 2's remaining rows appear
    R.kvq_append(cache, k, v, ints(*prefix))
    rk, _ = R.kvq_read(cache, ints(*prefix), N)
    assert np.array_equal(f64(rk[2]), ref.quantise(f64(k))[0][2])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_rows_that_are_not_finite(R, dtype):
    import torch
    rng = np.random.default_rng(3)
    x = rng.standard_normal((1, 6, 2, 1, 128)).astype(np.float32)
    x[0, 1, 0, 0, 70] = np.nan
    x[0, 2, 1, 0, 5] = np.inf
    x[0, 4, 0, 0, 0] = -np.inf
    kv = torch.from_numpy(x).cuda()
    kv = kv.bfloat16() if dtype == "bf16" else kv
    cache = make_cache(R, rng, 1, 1, 8, 128)
    R.kvq_append(cache, kv[:, :, 0], kv[:, :, 1], ints(1))
    rk, rv = R.kvq_read(cache, ints(1), 6)
    nk, nv = np.isnan(f64(rk))[0, :, 0].reshape(6, 4, 32), np.isnan(f64(rv))[0, :, 0].reshape(6, 4, 32)
    want_k, want_v = np.zeros((6, 4), bool), np.zeros((6, 4), bool)
    want_k[1, [0, 2]] = want_k[2, 0] = want_k[4, 0] = True           # the K row's first block says so in every case
    want_v[2, 0] = True
    assert np.array_equal(nk.all(-1), want_k) and np.array_equal(nk.any(-1), want_k)
    assert np.array_equal(nv.all(-1), want_v) and np.array_equal(nv.any(-1), want_v)
    fine, _ = ref.quantise(f64(kv[0, [0, 3, 5], 0]))
    assert np.array_equal(f64(rk)[0, [0, 3, 5]], fine)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_next_to_the_largest(R, dtype):
    """Elements past 7 * 2^125 have no larger scale to go to: they become the largest value, never an infinity, and a
    query that does not see them is what it is without them."""
    import torch
    rng = np.random.default_rng(31)
    top = 6 * 2.0 ** 125
    x = np.zeros((1, 3, 2, 1, 64), np.float32)
    x[0, 0, :, 0, :4] = [3.38e38, -3.0e38, 7 * 2.0 ** 125, 2.0 ** 123]       # one step is 2^124 near zero: a tie, to zero
    x[0, 1, :, 0, 40] = -3.38e38
    x[0, 2] = rng.standard_normal((2, 1, 64))
    kv = torch.from_numpy(x).cuda()
    kv = kv.bfloat16() if dtype == "bf16" else kv
    cache = make_cache(R, rng, 1, 1, 24, 64)
    R.kvq_append(cache, kv[:, :, 0], kv[:, :, 1], ints(20))
    for t in R.kvq_read(cache, ints(20), 3, dtype=torch.float32):
        got = f64(t)[0, :, 0]
        assert np.array_equal(got[0, :4], [top, -top, top, 0]) and (got[0, 4:] == 0).all()
        assert got[1, 40] == -top and (np.delete(got[1], 40) == 0).all()
    mask = np.array([[1, 0, 0], [0, 1, 0], [0, 0, 1]], np.uint8)
    q = queries(rng, 1, 3, 2, 64, dtype)
    out, lse = R.kvq_attention(q, cache, ints(20), mask=dev(mask))
    assert torch.isfinite(out[0, 2]).all() and torch.isfinite(lse[0, 2]).all()
    K, V = values(cache)
    K, V = K.copy(), V.copy()
    K[:, :, 20:22], V[:, :, 20:22] = 0, 0
    want, wlse, tol, ltol = ref.attend(f64(q), K, V, [20], [3], mask[None], 64 ** -0.5)
    size = ref.attend_abs(f64(q), K, V, [20], [3], mask[None], 64 ** -0.5)
    tol = tol + ((2.0 ** -8) * (size + 1.01 * np.abs(want)) if dtype == "bf16" else U * (size + 1.01 * np.abs(want)))
    assert (np.abs(f64(out) - want)[0, 2] <= tol[0, 2] + 1e-37).all()
    assert (np.abs(f64(lse) - wlse)[0, 2] <= ltol[0, 2]).all()


def test_one_slot_whatever_its_stride(R):
    """A cache of one slot: the stride of a dimension of one element never counts."""
    import torch
    rng = np.random.default_rng(32)
    D = 128
    cache = R.new_kvq_cache(2, 2, 1, D, "cuda")
    k, v = (torch.from_numpy(rng.standard_normal((2, 1, 2, D)).astype(np.float32)).cuda() for _ in range(2))
    R.kvq_append(cache, k, v, ints(0, 0))
    q = queries(rng, 2, 1, 4, D, "f32")
    want, wlse = R.kvq_attention(q, cache, ints(0, 0))
    assert wlse.isfinite().all() and (want != 0).any()
    for step in (0, 16, 1 << 25):
        odd = R.KVQCache(*(t.as_strided(t.shape, (t.stride(0), t.stride(1), step, 1))
                           for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)))
        got, lse = R.kvq_attention(q, odd, ints(0, 0))
        assert (got == want).all() and (lse == wlse).all()
        assert all((x == y).all() for x, y in zip(R.kvq_read(odd, ints(0, 0), 1), R.kvq_read(cache, ints(0, 0), 1)))
        sums = [torch.zeros((2, 2, 1), device="cuda") for _ in range(2)]
        for c, s in zip((cache, odd), sums):
            R.kvq_score(q, wlse, c, ints(0, 0), ints(0, 0), s, torch.zeros((2, 2, 1), dtype=torch.int32, device="cuda"),
                        ints(0, 0))
        assert (sums[0] == sums[1]).all() and (sums[0] > 0).all()


# ---- attention ----

ATTEND = [
    # B, N, G, H, D, dtype, layout, prefixes, capacity
    (1, 1, 1, 1, 128, "bf16", "heads", [0], 1),
    (1, 1, 4, 2, 128, "bf16", "heads", [1], 2),
    (3, 1, 4, 2, 128, "bf16", "heads", [31, 32, 33], 64),
    (3, 2, 8, 2, 64, "bf16", "rows", [127, 128, 0], 131),
    (2, 5, 3, 3, 128, "bf16", "slots", [129, 400], 405),
    (2, 27, 4, 2, 128, "bf16", "heads", [300, 3], 400),
    (1, 64, 5, 1, 64, "bf16", "rows", [77], 200),
    (2, 3, 7, 2, 256, "bf16", "heads", [65, 511], 600),
    (1, 33, 2, 1, 256, "bf16", "heads", [40], 100),
    (2, 1, 1, 2, 64, "f32", "heads", [0, 90], 128),
    (2, 9, 5, 2, 128, "f32", "rows", [33, 257], 300),
    (1, 20, 3, 1, 256, "f32", "heads", [130], 150),
    (1, 27, 1, 1, 128, "f32", "slots", [64], 91),
    (1, 1, 16, 1, 128, "bf16", "heads", [2999], 5000),
]


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attention(R, case, tree):
    B, N, G, H, D, dtype, layout, prefix, S = ATTEND[case]
    rng = np.random.default_rng(100 + case)
    cache = make_cache(R, rng, B, H, S, D, layout)
    q = queries(rng, B, N, H * G, D, dtype)
    mask = tree_masks(rng, B, N)[0] if tree else None
    out, lse = R.kvq_attention(q, cache, ints(*prefix), mask=None if mask is None else dev(mask))
    check_attention(out, lse, q, cache, prefix, None, mask, D ** -0.5)
    again = R.kvq_attention(q, cache, ints(*prefix), mask=None if mask is None else dev(mask))
    assert (again[0] == out).all() and (again[1] == lse).all()        # the same bits


@pytest.mark.parametrize("dtype,D,G", [("bf16", 128, 4), ("f32", 64, 2), ("bf16", 256, 3)])
def test_attention_prompt(R, dtype, D, G):
    """Many tokens, several row tiles, ragged counts: padded tokens answer zeros."""
    rng = np.random.default_rng(7)
    B, N, H, S = 3, 150, 2, 400
    cache = make_cache(R, rng, B, H, S, D)
    q = queries(rng, B, N, H * G, D, dtype)
    prefix, counts = [70, 0, 250], [150, 1, 97]
    out, lse = R.kvq_attention(q, cache, ints(*prefix), counts=ints(*counts))
    check_attention(out, lse, q, cache, prefix, counts, None, D ** -0.5)


@pytest.mark.parametrize("splits_up", [False, True])
def test_attention_ragged_batch_and_error_rows(R, splits_up):
    """Empty, unused and over-long batch rows beside ordinary ones; slots behind each row hold bytes that would be
    NaN or infinite if they were read as values."""
    rng = np.random.default_rng(8)
    B, N, G, H, D, S = 6, 4, 4, 2, 128, (4000 if splits_up else 300)
    prefix = [0, 5, -1, S - 3, S - 4, 200]
    counts = [4, 0, 4, 4, 4, 2]
    cache = make_cache(R, rng, B, H, S, D)
    for b in range(B):
        end = max(prefix[b], 0) + counts[b] if 0 <= prefix[b] <= S - counts[b] else 0
        for t in (cache.k_scales, cache.v_scales, cache.k_codes, cache.v_codes):
            t[b, :, end:] = 255
    q = queries(rng, B, N, H * G, D, "bf16")
    out, lse = R.kvq_attention(q, cache, ints(*prefix), counts=ints(*counts))
    check_attention(out, lse, q, cache, prefix, counts, None, D ** -0.5)
    assert not (lse[0] == -np.inf).any() and (lse[1:4] == -np.inf).all()


@pytest.mark.parametrize("B,H,N,S,dtype", [(65, 1, 1, 1300, "bf16"), (130, 1, 3, 1300, "f32"), (129, 2, 1, 1100, "bf16"),
                                           (130, 2, 2, 300, "bf16")])
def test_attention_batches_past_64(R, B, H, N, S, dtype):
    """More batch rows than a wave has lanes: a few long ones, many short ones, unused ones at both ends."""
    rng = np.random.default_rng(B + S)
    prefix = rng.integers(0, 60, B)
    prefix[rng.choice(B, 12, replace=False)] = rng.integers(S - 200, S - N, 12)
    prefix[[0, 63, B - 2]] = [S - N, S - N - 1, S - N]
    prefix[[1, 62, B - 1]] = [-1, S - N + 1, -7]
    counts = rng.integers(0, N + 1, B)
    counts[[0, 63, B - 2]] = N
    cache = make_cache(R, rng, B, H, S, 64)
    q = queries(rng, B, N, 3 * H, 64, dtype)
    out, lse = R.kvq_attention(q, cache, ints(*prefix), counts=ints(*counts))
    check_attention(out, lse, q, cache, prefix.tolist(), counts.tolist(), None, 0.125)


def test_attention_masks_that_leave_a_row_empty(R):
    rng = np.random.default_rng(9)
    B, N, G, H, D = 2, 6, 2, 2, 64
    cache = make_cache(R, rng, B, H, 40, D)
    q = queries(rng, B, N, H * G, D, "bf16")
    mask = tree_masks(rng, B, N)[0]
    mask[0, 3] = 0                                       # sees nothing: no prefix, no node
    mask[1, 2] = 0                                       # sees the prefix alone
    mask[1, 4, 5] = 7                                    # any non-zero byte is a yes, forward too
    out, lse = R.kvq_attention(q, cache, ints(0, 9), mask=dev(mask))
    check_attention(out, lse, q, cache, [0, 9], None, mask, D ** -0.5)
    assert (lse[0, 3] == -np.inf).all() and (out[0, 3] == 0).all() and (lse[1, 2] > -np.inf).all()
    one = dev(mask[0])                                   # one mask for all batch rows
    out, lse = R.kvq_attention(q, cache, ints(0, 9), mask=one)
    check_attention(out, lse, q, cache, [0, 9], None, np.stack([mask[0]] * 2), D ** -0.5)


def test_attention_poisoned_rows_reach_only_queries_that_see_them(R):
    import torch
    rng = np.random.default_rng(10)
    B, N, H, D = 1, 7, 1, 128
    cache = make_cache(R, rng, B, H, 64, D)
    mask, _ = tree_masks(rng, B, N)
    for bad_v in (False, True):
        k, v = (torch.from_numpy(rng.standard_normal((B, N, H, D)).astype(np.float32)).cuda() for _ in range(2))
        (v if bad_v else k)[0, 2, 0, 77] = float("nan")
        R.kvq_append(cache, k, v, ints(20))
        q = queries(rng, B, N, 4, D, "bf16")
        out, lse = R.kvq_attention(q, cache, ints(20), mask=dev(mask))
        sees = mask[0, :, 2] != 0
        assert np.array_equal(np.isnan(f64(out))[0].all((-1, -2)), sees)
        assert np.array_equal(np.isnan(f64(out))[0].any((-1, -2)), sees)
        assert np.array_equal(np.isnan(f64(lse))[0].all(-1), sees)
        assert sees.any() and not sees.all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_scale_and_sharp_softmax(R, dtype):
    """Scores in the hundreds (one key takes all), and a scale near zero (a mean)."""
    rng = np.random.default_rng(11)
    cache = make_cache(R, rng, 2, 1, 300, 64, lo=127, hi=131)
    q = queries(rng, 2, 3, 2, 64, dtype, size=3.0)
    for scale in (1.0, 1e-6, 0.3):
        out, lse = R.kvq_attention(q, cache, ints(250, 17), scale=scale)
        check_attention(out, lse, q, cache, [250, 17], None, None, scale)


def test_attention_strided_queries_and_given_outputs(R):
    import torch
    rng = np.random.default_rng(12)
    B, N, H, G, D = 2, 4, 2, 3, 64
    cache = make_cache(R, rng, B, H, 100, D)
    qkv = queries(rng, B, N, H * (G + 2), D, "bf16")
    q = qkv[:, :, :H * G]                                # the queries of a fused projection
    ws = torch.full((R.kvq_attention_workspace_bytes(cache, N, H * G) + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((B, N, H * G, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, N, H * G), float("nan"), device="cuda")
    got = R.kvq_attention(q, cache, ints(50, 96), out=(out, lse), workspace=ws)
    assert got[0] is out and got[1] is lse
    check_attention(out, lse, q, cache, [50, 96], None, None, D ** -0.5)
    hn = q.transpose(1, 2).contiguous().transpose(1, 2)  # heads outermost
    out2, _ = R.kvq_attention(hn, cache, ints(50, 96))
    assert (out2 == out).all()


def test_offsets_past_32_bits(R):
    """Slots, heads and batch rows further apart than 2^32 bytes."""
    import torch
    rng = np.random.default_rng(13)
    B, N, H, D, S = 2, 3, 2, 64, 280
    step = 1 << 24                                       # bytes from slot to slot: the last slot lies past 4 GiB
    room = torch.empty((S * step + 4096,), dtype=torch.uint8, device="cuda")
    def part(off, last):
        return room[off:].as_strided((B, H, S, last), (2048, 1024, step, 1))
    cache = R.KVQCache(part(0, 32), part(512, 2), part(256, 32), part(768, 2))
    k, v = (torch.from_numpy(rng.standard_normal((B, S, H, D)).astype(np.float32)).cuda() for _ in range(2))
    R.kvq_append(cache, k, v, ints(0, 0))
    rk, rv = R.kvq_read(cache, ints(0, 0), S)
    assert np.array_equal(f64(rk), ref.quantise(f64(k))[0]) and np.array_equal(f64(rv), ref.quantise(f64(v))[0])
    q = queries(rng, B, N, 2 * H, D, "bf16")
    out, lse = R.kvq_attention(q, cache, ints(S - N, 270))
    check_attention(out, lse, q, cache, [S - N, 270], None, None, D ** -0.5)
    scores = torch.zeros((B, H, S), device="cuda")
    pos = torch.zeros((B, H, S), dtype=torch.int32, device="cuda")
    R.kvq_score(q, lse, cache, ints(S - N, 270), ints(2, 2), scores, pos, ints(0, 0))
    want, wpos, tol = ref.score(f64(q), f64(lse), values(cache)[0], [S - N, 270], None, [2, 2], D ** -0.5,
                                np.zeros((B, H, S)), np.zeros((B, H, S), np.int32), [0, 0])
    assert (np.abs(f64(scores) - want) <= tol).all() and np.array_equal(pos.cpu().numpy(), wpos)
    old = arrays(cache)
    wn, wsrc = ref.evict(scores.cpu().numpy(), wpos, [S, 273], [S, 273], 100, 0, 0)
    n, src = R.kvq_evict(cache, scores, pos, ints(S, 273), ints(S, 273), 100)
    assert np.array_equal(n.cpu().numpy(), wn) and np.array_equal(src.cpu().numpy(), wsrc)
    for x0, x1 in zip(old, arrays(cache)):
        assert np.array_equal(ref.move(x0, wsrc, wn), x1)


# ---- scores ----

@pytest.mark.parametrize("D,G,dtype,layout", [(128, 4, "bf16", "heads"), (64, 1, "f32", "rows"), (256, 3, "bf16", "heads"),
                                              (128, 7, "f32", "slots"), (256, 2, "f32", "rows")])
def test_score_paths(R, D, G, dtype, layout):
    rng = np.random.default_rng(D + G)
    B, N, H, S, width = 8, 12, 2, 300, 5
    cache = make_cache(R, rng, B, H, S, D, layout)
    q = queries(rng, B, N, H * G, D, dtype)
    prefix = [100, 0, 255, -1, S - 4, 64, 31, 17]
    path = np.full((B, width), -1, np.int32)
    alen = [4, 0, 2, 1, 4, 3, -1, 2]
    path[0] = [0, 2, 3, 7, 11]
    path[1, 0] = 0
    path[2, :3] = [0, 1, 5]
    path[3, :2] = [0, 1]
    path[4] = [0, 1, 2, 3, 4]                            # its rows would pass the cache's end
    path[5, :4] = [0, 4, 4, 6]                           # not increasing
    path[7, :3] = [0, 3, 12]                             # no such token
    lse = (8 + rng.standard_normal((B, N, H * G))).astype(np.float32)
    lse[0, 3, 1] = -np.inf                               # a query that saw nothing
    scores = rng.random((B, H, S)).astype(np.float32)
    pos = rng.integers(0, 1000, (B, H, S)).astype(np.int32)
    seen = [1000 + b for b in range(B)]
    ds, dp = dev(scores), dev(pos)
    R.kvq_score(q, dev(lse), cache, ints(*prefix), ints(*alen), ds, dp, ints(*seen), path=dev(path))
    want, wpos, tol = ref.score(f64(q), lse, values(cache)[0], prefix, path, alen, D ** -0.5, scores, pos, seen)
    assert np.array_equal(dp.cpu().numpy(), wpos)
    assert (np.abs(f64(ds) - want) <= tol).all(), np.abs(f64(ds) - want).max()
    for b in (3, 4, 5, 6, 7):
        assert np.array_equal(ds[b].cpu().numpy(), scores[b])


@pytest.mark.parametrize("D,G,N,prefix,alen", [(128, 4, 70, [0, 33], [69, 40]), (64, 5, 33, [200, 7], [0, 32]),
                                               (256, 1, 17, [1, 128], [16, 33])])
def test_score_prompt(R, D, G, N, prefix, alen):
    """Without a path: tokens 0 .. accept_len, more of them than a tree has; a length past N is an error row."""
    rng = np.random.default_rng(N)
    B, H, S = 2, 2, 300
    cache = make_cache(R, rng, B, H, S, D)
    q = queries(rng, B, N, H * G, D, "bf16")
    lse = (6 + rng.standard_normal((B, N, H * G))).astype(np.float32)
    scores = rng.random((B, H, S)).astype(np.float32)
    pos = np.full((B, H, S), -5, np.int32)
    ds, dp = dev(scores), dev(pos)
    R.kvq_score(q, dev(lse), cache, ints(*prefix), ints(*alen), ds, dp, ints(3, 4), scale=0.05)
    want, wpos, tol = ref.score(f64(q), lse, values(cache)[0], prefix, None, alen, 0.05, scores, pos, [3, 4])
    assert np.array_equal(dp.cpu().numpy(), wpos)
    assert (np.abs(f64(ds) - want) <= tol).all()
    ds2, dp2 = dev(scores), dev(pos)
    R.kvq_score(q, dev(lse), cache, ints(*prefix), ints(*alen), ds2, dp2, ints(3, 4), scale=0.05)
    assert (ds2 == ds).all()                             # the same bits


@pytest.mark.parametrize("B,H,G,D,N,prefix,dtype", [
    (8, 8, 4, 64, 2400, 0, "bf16"),      # rows in two segments, several key blocks a workgroup, lots older than all keys
    (1, 2, 4, 128, 700, 1500, "bf16"), (1, 1, 3, 256, 300, 90, "f32"), (2, 2, 2, 128, 150, 40, "f32"),
    (1, 16, 16, 64, 40, 3000, "bf16"), (16, 4, 8, 128, 9, 9000, "bf16")])
def test_score_many_rows(R, B, H, G, D, N, prefix, dtype):
    """Prompts and long chains against the definition in 64 bits (torch on the GPU, one head at a time)."""
    import torch
    rng = np.random.default_rng(N)
    S = prefix + N + 3
    cache = make_cache(R, rng, B, H, S, D)
    q = queries(rng, B, N, H * G, D, dtype, size=0.5)
    lse = torch.from_numpy((4 + rng.standard_normal((B, N, H * G))).astype(np.float32)).cuda()
    pre = [prefix] * B
    alen = [N - 1 - b for b in range(B)]
    scores = torch.from_numpy(rng.random((B, H, S)).astype(np.float32)).cuda()
    pos = torch.zeros((B, H, S), dtype=torch.int32, device="cuda")
    before = scores.double()
    R.kvq_score(q, lse, cache, ints(*pre), ints(*alen), scores, pos, ints(*pre))
    table = torch.tensor(list(ref.GRID) + [-v for v in ref.GRID], dtype=torch.float64, device="cuda")
    slot = torch.arange(S, device="cuda")
    u = 2.0 ** -24
    for b in range(B):
        T = alen[b] + 1
        if T < 1:                                        # an error row: left as it was
            assert torch.equal(scores[b].double(), before[b]) and (pos[b] == 0).all()
            continue
        sees = slot <= prefix + torch.arange(T, device="cuda").view(-1, 1)
        for h in range(H):
            c = cache.k_codes[b, h].long()
            K = table[torch.stack((c & 15, c >> 4), -1).flatten(-2)]
            K = K * torch.exp2(cache.k_scales[b, h].double() - 127).repeat_interleave(32, -1)
            w = torch.zeros(S, dtype=torch.float64, device="cuda")
            err = torch.zeros_like(w)
            for g in range(G):
                x, z = q[b, :T, h * G + g].double(), lse[b, :T, h * G + g].double().view(-1, 1)
                s = (x @ K.T) * D ** -0.5
                e = torch.where(sees, torch.exp(s - z), 0.0)
                w += e.sum(0)
                # as in kvq_ref.score: D products, a rounded exponent, exp2
                err += (e * (D * (x.abs() @ K.abs().T) * D ** -0.5 + 8 * s.abs() + 8 * z.abs() + 8)).sum(0) * u
            err += w * (T * G + 24) * u                  # the sums, over at most T*G terms and a few segments
            want = torch.where(slot < prefix, before[b, h] + w, torch.where(slot < prefix + T, w, before[b, h]))
            off = (scores[b, h].double() - want).abs()
            assert (off <= err + 2 * u * want.abs()).all(), (b, h, off.max())
        assert (pos[b, :, prefix:prefix + T] == prefix + torch.arange(T, device="cuda")).all()
        assert (pos[b, :, :prefix] == 0).all() and (pos[b, :, prefix + T:] == 0).all()


def test_scores_of_attention_sum_to_the_queries(R):
    """With attention's own lse the weights of a query sum to one: the new scores hold (d + 1) * G in total."""
    import torch
    rng = np.random.default_rng(21)
    B, N, H, G, D, S = 2, 9, 2, 4, 128, 700
    cache = make_cache(R, rng, B, H, S, D)
    q = queries(rng, B, N, H * G, D, "f32")
    _, lse = R.kvq_attention(q, cache, ints(600, 5))
    scores = torch.zeros((B, H, S), device="cuda")
    pos = torch.zeros((B, H, S), dtype=torch.int32, device="cuda")
    R.kvq_score(q, lse, cache, ints(600, 5), ints(8, 8), scores, pos, ints(600, 5))
    # each weight is off by a few dozen roundings of its exponent's arithmetic, as bounded in kvq_ref
    assert np.allclose(f64(scores).sum(-1), 9 * G, rtol=1e-4)


# ---- eviction ----

def run_evict(R, cache, scores, pos, lens, seen, keep, sink, recent, apart):
    import torch
    ds, dp = dev(scores), dev(pos)
    old = arrays(cache)
    kw = {}
    os, op = ds, dp
    if apart:
        os, op = torch.full_like(ds, -7.0), torch.full_like(dp, -7)
        kw = dict(out_scores=os, out_positions=op)
    n, src = R.kvq_evict(cache, ds, dp, ints(*lens), ints(*seen), keep, sink=sink, recent=recent, **kw)
    wn, wsrc = ref.evict(scores, pos, lens, seen, keep, sink, recent)
    assert np.array_equal(n.cpu().numpy(), wn)
    assert np.array_equal(src.cpu().numpy(), wsrc)
    for x0, x1 in zip(old, arrays(cache)):
        assert np.array_equal(ref.move(x0, wsrc, wn), x1)
    moved_s, moved_p = ref.move(scores, wsrc, wn), ref.move(pos, wsrc, wn)
    if apart:
        assert np.array_equal(ds.cpu().numpy(), scores, equal_nan=True) and np.array_equal(dp.cpu().numpy(), pos)
        for b in range(len(lens)):
            at = max(int(wn[b]), 0)
            moved_s[b, :, at:], moved_p[b, :, at:] = -7, -7
    assert np.array_equal(os.cpu().numpy(), moved_s, equal_nan=True)
    assert np.array_equal(op.cpu().numpy(), moved_p)


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("D,layout,S,keep", [(128, "heads", 40, 16), (64, "rows", 1500, 1000), (256, "slots", 3000, 77),
                                             (128, "rows", 9, 9), (64, "heads", 5000, 1), (128, "heads", 2100, 2048)])
def test_evict(R, D, layout, S, keep, apart):
    rng = np.random.default_rng(S)
    B, H = 7, 2
    cache = make_cache(R, rng, B, H, S, D, layout)
    lens = [S, S - 1, keep, 0, -1, S + 1, min(S, keep + 3)]
    scores = np.exp(2 * rng.standard_normal((B, H, S))).astype(np.float32)
    pos = np.tile(np.arange(S, dtype=np.int32), (B, H, 1))
    run_evict(R, cache, scores, pos, lens, [S] * B, keep, 4, 8, apart)


@pytest.mark.parametrize("keep", [1, 5, 100, 1023, 1024, 1500])
def test_evict_ties_and_special_scores(R, keep):
    rng = np.random.default_rng(keep)
    B, H, S = 4, 2, 2000
    cache = make_cache(R, rng, B, H, S, 64)
    scores = rng.integers(0, 4, (B, H, S)).astype(np.float32)        # great ties
    scores[1] = 0.5                                                  # all alike
    scores[2, :, ::3] = np.nan
    scores[2, :, 1::7] = np.inf
    scores[2, :, 2::7] = -np.inf
    scores[2, :, 4::7] = -0.0
    scores[3] = np.nan
    pos = np.argsort(rng.random((B, H, S)), -1).astype(np.int32)     # positions in any order
    run_evict(R, cache, scores, pos, [S, S, S, S - 5], [S] * B, keep, 3, 10, False)


def test_evict_more_protected_than_kept_and_none(R):
    rng = np.random.default_rng(5)
    cache = make_cache(R, rng, 2, 1, 300, 64)
    scores = rng.random((2, 1, 300)).astype(np.float32)
    pos = np.argsort(rng.random((2, 1, 300)), -1).astype(np.int32)
    run_evict(R, cache, scores, pos, [300, 300], [300, 2 ** 31 - 1], 20, 30, 200, False)
    run_evict(R, cache, scores, pos, [300, 299], [300, -2 ** 31], 20, 0, 2 ** 31 - 1, True)


@pytest.mark.parametrize("S,keep", [(60, 20), (3000, 1000)])
def test_evict_one_array_in_place(R, S, keep):
    """The scores in place and the positions elsewhere, and the other way round."""
    import torch
    rng = np.random.default_rng(S)
    for which in range(2):
        cache = make_cache(R, rng, 2, 2, S, 64)
        scores = rng.random((2, 2, S)).astype(np.float32)
        pos = np.tile(np.arange(S, dtype=np.int32), (2, 2, 1))
        ds, dp = dev(scores), dev(pos)
        other = torch.full_like(dp if which else ds, -7)
        n, src = R.kvq_evict(cache, ds, dp, ints(S, S - 1), ints(S, S), keep, sink=1, recent=3,
                             **{"out_positions" if which else "out_scores": other})
        wn, wsrc = ref.evict(scores, pos, [S, S - 1], [S, S], keep, 1, 3)
        assert np.array_equal(src.cpu().numpy(), wsrc)
        ms, mp = ref.move(scores, wsrc, wn), ref.move(pos, wsrc, wn)
        gs, gp = (ds, other) if which else (other, dp)
        assert np.array_equal(gs.cpu().numpy()[..., :keep], ms[..., :keep])
        assert np.array_equal(gp.cpu().numpy()[..., :keep], mp[..., :keep])


@pytest.mark.parametrize("n,keep", [(60000, 20000), (50001, 50000), (4097, 2000), (49152, 48000)])
def test_evict_long_heads(R, n, keep):
    """Heads whose keys fit the registers of sixteen waves, just do, and do not."""
    rng = np.random.default_rng(n)
    S = n + 5
    cache = make_cache(R, rng, 1, 2, S, 64)
    scores = np.exp(2 * rng.standard_normal((1, 2, S))).astype(np.float32)
    scores[0, 1] = np.round(scores[0, 1])                            # great ties, across waves
    pos = np.tile(np.arange(S, dtype=np.int32), (1, 2, 1))
    run_evict(R, cache, scores, pos, [n], [n], keep, 4, 30, False)


# ---- together ----

@pytest.mark.parametrize("layout", ["heads", "rows", "slots"])
def test_commit_moves_every_part(R, layout):
    rng = np.random.default_rng(50)
    B, H, S, D, N = 3, 2, 40, 128, 9
    cache = make_cache(R, rng, B, H, S, D, layout)
    old = arrays(cache)
    path = np.array([[0, 2, 5, 8], [0, 1, -1, -1], [0, 4, 7, -1]], np.int32)
    alen, prefix = [3, 1, -1], [10, 0, 5]
    n = R.kvq_commit(cache, ints(*prefix), dev(path), ints(*alen), N)
    assert n.tolist() == [14, 2, -1]
    for x0, x1 in zip(old, arrays(cache)):
        for b in range(2):
            p = path[b, :alen[b] + 1]
            x0[b][:, prefix[b]:prefix[b] + len(p)] = x0[b][:, prefix[b] + p].copy()
        assert np.array_equal(x0, x1)


def test_calls_on_two_streams_at_once(R):
    """Two caches attended and scored on two streams, each with its own workspace from the allocator: the bits of the
    calls made one after the other."""
    import torch
    rng = np.random.default_rng(51)
    jobs = []
    for i in range(2):
        cache = make_cache(R, rng, 2, 2, 6000, 128)
        q = queries(rng, 2, 40, 8, 128, "bf16")
        jobs.append((cache, q, ints(5000, 700 + i), torch.zeros((2, 2, 6000), device="cuda"),
                     torch.zeros((2, 2, 6000), dtype=torch.int32, device="cuda")))

    def work(cache, q, prefix, scores, pos):
        out, lse = R.kvq_attention(q, cache, prefix)
        scores.zero_()
        R.kvq_score(q, lse, cache, prefix, ints(39, 39), scores, pos, prefix)
        return out, lse, scores.clone()

    want = [work(*j) for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, j in zip(streams, jobs):
            with torch.cuda.stream(s):
                got.append(work(*j))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_one_query_for_all(R):
    """Queries broadcast over the batch and the tokens (strides of zero)."""
    rng = np.random.default_rng(52)
    cache = make_cache(R, rng, 3, 2, 200, 64)
    one = queries(rng, 1, 1, 4, 64, "bf16")
    q = one.expand(3, 5, 4, 64)
    out, lse = R.kvq_attention(q, cache, ints(100, 7, 190))
    check_attention(out, lse, q, cache, [100, 7, 190], None, None, 0.125)


def test_speculative_steps(R):
    """Three steps as a serving loop makes them: rerank a draft tree, append its rows, attend under its mask, verify
    greedily, commit the accepted path, score it, evict to a budget; each call's result against the 64-bit
    reference on the state before it."""
    import torch
    rng = np.random.default_rng(30)
    B, H, G, D, S, V, budget = 3, 2, 4, 128, 160, 64, 100
    m = 11
    N = m + 1
    cache = make_cache(R, rng, B, H, S, D)
    lens, seen = ints(90, 97, 60), ints(190, 97, 60)
    scores = dev(rng.random((B, H, S)).astype(np.float32))
    pos = dev(np.tile(np.arange(S, dtype=np.int32), (B, H, 1)))
    head = torch.from_numpy(rng.standard_normal((H * G * D, V)).astype(np.float32)).cuda()
    for step in range(3):
        par = np.array([[-1 if i < 4 else rng.integers(0, i) for i in range(30)] for _ in range(B)], np.int32)
        val = np.empty((B, 30), np.float32)
        for b in range(B):
            for i in range(30):
                val[b, i] = (1.0 if par[b, i] < 0 else val[b, par[b, i]]) * np.float32(rng.uniform(0.3, 0.95))
        nodes, ppos, mask = R.tree_rerank(dev(par), dev(val), m)
        k, v = (torch.from_numpy(rng.standard_normal((B, N, H, D)).astype(np.float32)).cuda().bfloat16() for _ in range(2))
        q = queries(rng, B, N, H * G, D, "bf16")
        prefix = lens.clone()
        R.kvq_append(cache, k, v, prefix)
        rk, _ = R.kvq_read(cache, prefix, N)
        assert np.array_equal(f64(rk), ref.quantise(f64(k))[0])
        out, lse = R.kvq_attention(q, cache, prefix, mask=mask)
        check_attention(out, lse, q, cache, prefix.tolist(), None, mask.cpu().numpy(), D ** -0.5)
        logits = (out.float().reshape(B, N, -1) @ head).contiguous()
        tree = torch.cat((torch.full((B, 1), -1, dtype=torch.int32, device="cuda"), ppos), 1)
        best = logits.argmax(-1).to(torch.int32)
        tokens = torch.from_numpy(rng.integers(0, V, (B, N)).astype(np.int32)).cuda()
        keep_some = torch.from_numpy(rng.random((B, N)) < 0.8).cuda()   # most nodes hold the token their parent wants
        tokens[:, 1:] = torch.where(keep_some[:, 1:], best.gather(1, ppos.long()), tokens[:, 1:])
        path, _, alen = R.verify_tree_greedy(logits, tokens, tree.contiguous())
        assert (alen >= 0).all()
        before = arrays(cache)
        lens = R.kvq_commit(cache, prefix, path, alen, N)
        assert (lens == prefix + alen + 1).all()
        for x0, x1 in zip(before, arrays(cache)):
            for b in range(B):
                n, p = int(prefix[b]), path[b, :int(alen[b]) + 1].cpu().numpy()
                x0[b, :, n:n + len(p)] = x0[b][:, n + p].copy()
            assert np.array_equal(x0, x1)
        s0, p0 = scores.cpu().numpy(), pos.cpu().numpy()
        R.kvq_score(q, lse, cache, prefix, alen, scores, pos, seen, path=path)
        want, wpos, tol = ref.score(f64(q), f64(lse), values(cache)[0], prefix.tolist(), path.cpu().numpy(),
                                    alen.cpu().numpy(), D ** -0.5, s0, p0, seen.cpu().numpy())
        assert (np.abs(f64(scores) - want) <= tol).all() and np.array_equal(pos.cpu().numpy(), wpos)
        seen = seen + alen + 1
        s0, p0, old = scores.cpu().numpy(), pos.cpu().numpy(), arrays(cache)
        wn, wsrc = ref.evict(s0, p0, lens.cpu().numpy(), seen.cpu().numpy(), budget, 4, 16)
        lens, src = R.kvq_evict(cache, scores, pos, lens, seen, budget, sink=4, recent=16)
        assert np.array_equal(lens.cpu().numpy(), wn) and np.array_equal(src.cpu().numpy(), wsrc)
        for x0, x1 in zip(old, arrays(cache)):
            assert np.array_equal(ref.move(x0, wsrc, wn), x1)


def test_graph_replays_and_streams(R):
    """Append, attention, score and eviction captured once and replayed with eager work between, and called on a
    side stream: the eager bits every time."""
    import torch
    rng = np.random.default_rng(31)
    B, N, H, G, D, S = 2, 5, 2, 4, 128, 3000
    cache = make_cache(R, rng, B, H, S, D)
    k, v = (torch.from_numpy(rng.standard_normal((B, N, H, D)).astype(np.float32)).cuda() for _ in range(2))
    q = queries(rng, B, N, H * G, D, "bf16")
    prefix, alen, seen = ints(2500, 900), ints(4, 2), ints(2500, 900)
    s0 = dev(rng.random((B, H, S)).astype(np.float32))
    p0 = torch.zeros((B, H, S), dtype=torch.int32, device="cuda")
    codes = [t.clone() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
    scores, pos = s0.clone(), p0.clone()

    def step():
        R.kvq_append(cache, k, v, prefix)
        out, lse = R.kvq_attention(q, cache, prefix)
        R.kvq_score(q, lse, cache, prefix, alen, scores, pos, seen)
        n, src = R.kvq_evict(cache, scores, pos, prefix + alen + 1, seen, 800, sink=1, recent=30)
        return out, lse, n, src

    def reset():
        for t, c in zip((cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales), codes):
            t.copy_(c)
        scores.copy_(s0)
        pos.copy_(p0)

    def state():
        return [t.clone() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, scores, pos)]

    want = [t.clone() for t in step()] + state()
    reset()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = list(step()) + state()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    reset()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for turn in range(4):
        reset()
        graph.replay()
        got = [t.clone() for t in held] + state()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), turn
        R.kvq_attention(q, cache, prefix)                # eager work between the replays


def test_binding_refusals(R):
    import torch
    rng = np.random.default_rng(40)
    cache = make_cache(R, rng, 2, 2, 16, 64)
    x = torch.zeros((2, 3, 2, 64), device="cuda")
    pre = ints(0, 0)
    with pytest.raises(ValueError):
        R.kvq_append(cache, x, x[:, :2], pre)
    with pytest.raises(TypeError):
        R.kvq_append(cache, x.half(), x.half(), pre)
    with pytest.raises(ValueError):
        R.kvq_append(cache, x, x, ints(0))
    with pytest.raises(TypeError):
        R.kvq_append(cache, x, x, pre.long())
    with pytest.raises(ValueError):
        R.kvq_append(cache, x, x, pre.cpu())
    with pytest.raises(R.SpecError):
        y = torch.zeros((2 * 3 * 2 * 64 + 1,), device="cuda")[1:].view(2, 3, 2, 64)      # 4 bytes off
        R.kvq_append(cache, y, y, pre)
    q = torch.zeros((2, 3, 4, 64), device="cuda")
    with pytest.raises(ValueError):
        R.kvq_attention(q[:, :, :3], cache, pre)
    with pytest.raises(ValueError):
        R.kvq_attention(q, cache, pre, mask=torch.zeros((3, 2), dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        R.kvq_attention(q, cache, pre, mask=torch.zeros((3, 3), dtype=torch.bool, device="cuda"))
    big = make_cache(R, rng, 1, 1, 4096, 64)
    assert R.kvq_attention_workspace_bytes(big, 3, 4, torch.float32) > 0
    with pytest.raises(ValueError):
        R.kvq_attention(q[:1], big, pre[:1], workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(R.SpecError):
        R.kvq_attention(q, cache, pre, scale=-1.0)
    with pytest.raises(ValueError):
        R.kvq_attention(q.transpose(2, 3).contiguous().transpose(2, 3), cache, pre)
    sc, po = torch.zeros((2, 2, 16), device="cuda"), torch.zeros((2, 2, 16), dtype=torch.int32, device="cuda")
    lse = torch.zeros((2, 3, 4), device="cuda")
    with pytest.raises(ValueError):
        R.kvq_score(q, lse[:, :2], cache, pre, pre, sc, po, pre)
    with pytest.raises(TypeError):
        R.kvq_score(q, lse, cache, pre, pre, sc.double(), po, pre)
    with pytest.raises(ValueError):
        R.kvq_evict(cache, sc, po, pre, pre, 17)
    with pytest.raises(ValueError):
        R.kvq_evict(cache, sc, po, pre, pre, 4, sink=-1)
    u = torch.zeros((2, 1, 16, 32), dtype=torch.uint8, device="cuda")
    s = torch.zeros((2, 2, 16, 2), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="share memory"):
        R.KVQCache(u.expand(2, 2, 16, 32), s, u.expand(2, 2, 16, 32), s)
