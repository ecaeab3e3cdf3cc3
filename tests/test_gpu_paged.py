"""The paged cache on the GPU against its definitions (paged_ref): pages of a step and rows in them (exact), attention
behind shared prefixes against float64, and a run of them together with a verification."""

import numpy as np
import pytest

import paged_ref as ref

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


def ints(v):
    return dev(np.asarray(v, np.int32))


def f64(t):
    return t.double().cpu().numpy()


# ---- pages ----

def make_pool(R, rng, T, width, P, fill=0.4, spare=0):
    """A pool in the middle of its life: rows of random lengths, free pages anywhere in the ring."""
    import torch
    held = np.minimum(rng.integers(0, max(1, int(width * fill)) + 1, T), width).astype(np.int32)
    pages = int(held.sum()) + spare + 1
    ids = rng.permutation(pages).astype(np.int32)
    tables = np.full((T, width + 3), -5, np.int32)
    at = 0
    for t in range(T):
        tables[t, :held[t]] = ids[at:at + held[t]]
        at += held[t]
    head, free = int(rng.integers(0, pages)), pages - at
    ring = np.full(pages, -9, np.int32)
    ring[(head + np.arange(free)) % pages] = ids[at:]
    t = dev(tables)[:, :width]                                # rows of a wider tensor
    return R.PagePool(t, ints(held), ints(ring), ints([head, free]), P)


def pool_arrays(pool):
    return [x.cpu().numpy().copy() for x in (pool.tables, pool.held, pool.ring, pool.state)]


@pytest.mark.parametrize("T,width,P,N,spare", [
    (1, 1, 16, 1, 0), (1, 40, 16, 600, 30), (3, 8, 64, 5, 0), (7, 5, 16, 16, 40), (300, 9, 32, 7, 500), (257, 70, 16, 1025, 9000),
    (700, 6, 128, 64, 300), (1500, 4, 16, 3, 100), (16, 300, 32, 8192, 4000),
])
@pytest.mark.parametrize("in_place", [True, False])
def test_page_step(R, T, width, P, N, spare, in_place):
    import torch
    rng = np.random.default_rng([T, width, N])
    pool = make_pool(R, rng, T, width, P, spare=spare)
    for step in range(5):
        tables, held, ring, state = pool_arrays(pool)
        lengths = np.maximum(held * P - rng.integers(0, 2 * P, T), 0).astype(np.int32)
        lengths[rng.random(T) < 0.2] = -1                     # ended
        back = rng.random(T) < 0.2
        lengths[back] = lengths[back] // 3                    # much was rejected
        counts = rng.integers(0, N + 1, T).astype(np.int32)
        if T > 4:                                             # numbers that make no sense
            counts[1], counts[2], lengths[3] = N + 1, -1, width * P
        use = None if step == 4 else counts
        want = ref.page_step(tables, held, ring, state, lengths, use, N, P)
        oh, os = (None, None) if in_place else (torch.full_like(pool.held, 77), torch.full_like(pool.state, 77))
        granted, slots = R.page_step(pool, ints(lengths), N, counts=None if use is None else ints(use), out_held=oh, out_state=os)
        got = (granted, slots, pool.tables, pool.held if in_place else oh, pool.ring, pool.state if in_place else os)
        for name, g, w in zip(("granted", "slots", "tables", "held", "ring", "state"), got, want):
            assert np.array_equal(g.cpu().numpy(), w), (name, step)
        assert (pool.tables.as_strided((T, 3), (width + 3, 1), width) == -5).all() and not pool._workspace.any()
        if not in_place:
            assert np.array_equal(pool.held.cpu().numpy(), held) and np.array_equal(pool.state.cpu().numpy(), state)
            pool.held.copy_(oh)
            pool.state.copy_(os)


def test_pages_run_out_in_the_order_of_the_rows(R):
    pool = R.new_page_pool(5, 4, 6, 16, "cuda")
    granted, slots = R.page_step(pool, ints([0, 0, 0, 0, 0]), 40, counts=ints([33, 16, 40, 0, 10]))
    assert granted.tolist() == [33, 16, -1, 0, -1]            # the third does not fit, so the fifth gets none either
    assert pool.held.tolist() == [3, 1, 0, 0, 0] and pool.state.tolist() == [4, 2]
    assert slots[1, :16].tolist() == list(range(48, 64)) and (slots[1, 16:] == -1).all() and (slots[2] == -1).all()
    # the first ends: its pages are free again, for the next call
    granted, _ = R.page_step(pool, ints([-1, 16, 0, 0, 0]), 40, counts=ints([7, 0, 40, 0, 32]))
    assert granted.tolist() == [0, 0, -1, 0, -1] and pool.state.tolist() == [4, 5]
    granted, slots = R.page_step(pool, ints([-1, 16, 0, 0, 0]), 40, counts=ints([0, 0, 40, 0, 32]))
    assert granted.tolist() == [0, 0, 40, 0, 32] and pool.state.tolist() == [3, 0]
    assert pool.tables[2, :3].tolist() == [4, 5, 0] and pool.tables[4, :2].tolist() == [1, 2]
    assert slots[4, :17].tolist() == list(range(16, 32)) + [32]


@pytest.mark.parametrize("state", [(-1, 3), (6, 3), (0, -1), (0, 7), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_a_ring_out_of_range_serves_nobody(R, state):
    pool = R.new_page_pool(2, 4, 6, 16, "cuda")
    pool.state.copy_(ints(state))
    granted, slots = R.page_step(pool, ints([0, -1]), 3)
    assert granted.tolist() == [-1, -1] and (slots == -1).all() and pool.held.tolist() == [0, 0]
    assert pool.state.tolist() == list(state) and (pool.tables == -1).all() and pool.ring.tolist() == list(range(6))


def test_more_pages_held_than_there_are(R):
    """Such a row's numbers make no sense: it is not served, and the ring keeps its other entries."""
    pool = R.new_page_pool(2, 40, 3, 16, "cuda")
    pool.held.copy_(ints([30, 0]))
    granted, slots = R.page_step(pool, ints([-1, 0]), 3)
    assert granted.tolist() == [-1, 3] and slots.tolist() == [[-1, -1, -1], [0, 1, 2]]
    assert pool.held.tolist() == [30, 1] and pool.state.tolist() == [1, 2] and pool.ring.tolist() == [0, 1, 2]


def test_pages_that_are_none_have_no_slots(R):
    pool = R.new_page_pool(1, 4, 3, 16, "cuda")
    pool.ring.copy_(ints([3, -1, 2]))
    granted, slots = R.page_step(pool, ints([0]), 48)
    assert granted.tolist() == [48] and (slots[0, :32] == -1).all() and slots[0, 32:].tolist() == list(range(32, 48))


# ---- rows ----

LAYOUTS = {"slots": (0, 1, 2), "heads": (0, 2, 1), "outer": (2, 0, 1), "inner": (1, 2, 0)}


def make_cache(R, rng, pages, P, H, D, layout="slots", fill=None):
    """Pages of normal rows (or one bit pattern), dimensions in any order of memory."""
    import torch
    order = LAYOUTS[layout]
    shape = [(pages, P, H)[i] for i in order]
    back = [order.index(i) for i in range(3)]
    out = []
    for _ in range(2):
        if fill is None:
            x = rng.standard_normal((*shape, D)).astype(np.float32)
            x[..., 3::29] *= 4.0
            t = torch.from_numpy(x).cuda().bfloat16()
        else:
            t = torch.full((*shape, D), fill, dtype=torch.int16, device="cuda").view(torch.bfloat16)
        out.append(t.permute(*back, 3))
    return R.PagedCache(*out)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "bf16"), (256, "bf16"), (64, "f32"), (128, "f32"), (256, "f32")])
def test_append(R, D, dtype, layout):
    import torch
    rng = np.random.default_rng(D)
    B, N, H, P, pages = 3, 21, 3, 16, 9
    cache = make_cache(R, rng, pages, P, H, D, layout)
    kv = torch.from_numpy(rng.standard_normal((B, N, 2, H, D)).astype(np.float32)).cuda()
    kv[0, 0, 0, 0, :3] = torch.tensor([float("nan"), float("inf"), -1e-45])
    kv = kv.bfloat16() if dtype == "bf16" else kv
    k, v = kv[:, :, 0], kv[:, :, 1]
    slots = rng.permutation(pages * P)[:B * N].reshape(B, N).astype(np.int32)
    slots[0, 5], slots[1, 6], slots[2, 7], slots[2, 8] = -1, pages * P, 2 ** 31 - 1, -2 ** 31
    want = [t.clone() for t in (cache.k_pages, cache.v_pages)]
    for b in range(B):
        for n in range(N):
            if 0 <= slots[b, n] < pages * P:
                for w, x in zip(want, (k, v)):
                    w[slots[b, n] // P, slots[b, n] % P] = x[b, n].bfloat16()
    wide = torch.full((B, N + 2), -1, dtype=torch.int32, device="cuda")
    wide[:, :N] = ints(slots)
    R.paged_append(cache, k, v, wide[:, :N])
    for got, w in zip((cache.k_pages, cache.v_pages), want):
        assert torch.equal(got.contiguous().view(torch.int16), w.contiguous().view(torch.int16))
    # an accepted path: rows 0, 2, 5, .. of the step again, in the first slots
    path = np.full((B, 4), -1, np.int32)
    path[0], path[1, :2], path[2] = [0, 2, 5, 20], [0, 3], [0, 1, -1, 30]
    alen = [3, 1, 3]
    for b in range(B):
        for i in range(alen[b] + 1):
            if 0 <= slots[b, i] < pages * P and 0 <= path[b, i] < N:
                for w, x in zip(want, (k, v)):
                    w[slots[b, i] // P, slots[b, i] % P] = x[b, path[b, i]].bfloat16()
    R.paged_append(cache, k, v, ints(slots), path=ints(path), accept_len=ints(alen))
    R.paged_append(cache, v, k, ints(slots), path=ints(path), accept_len=ints([-1, -1, 4]))     # nothing
    for got, w in zip((cache.k_pages, cache.v_pages), want):
        assert torch.equal(got.contiguous().view(torch.int16), w.contiguous().view(torch.int16))


# ---- attention ----

def tree_masks(rng, B, N):
    m = np.zeros((B, N, N), np.uint8)
    for b in range(B):
        for n in range(N):
            if n:
                m[b, n] = m[b, rng.integers(max(0, n - 5), n)]
            m[b, n, n] = 1
    return m


def queries(rng, B, N, Hq, D, dtype, size=1.5):
    import torch
    q = torch.from_numpy((size * rng.standard_normal((B, N, Hq, D))).astype(np.float32)).cuda()
    return q.bfloat16() if dtype == "bf16" else q


def make_tables(rng, pages, P, lens, N, B, width):
    """Tables of shuffled pages for rows of `lens` committed slots (N new ones behind those of the first B)."""
    ids = rng.permutation(pages)
    tables = np.full((len(lens), width), -1, np.int32)
    at = 0
    for t, n in enumerate(lens):
        k = -(-(max(n, 0) + (N if t < B else 0)) // P)
        tables[t, :min(k, width)] = ids[at:at + min(k, width)]
        at += k
    assert at <= pages
    return tables


def check(R, q, cache, tables, lens, B, counts=None, prefix_row=None, mask=None, scale=None, got=None):
    """Every output within the roundings that the arithmetic allows."""
    import torch
    N, Hq, D = q.shape[1:]
    if got is None:
        plan = R.paged_plan(cache, ints(tables), ints(lens), N, Hq, B=B, counts=None if counts is None else ints(counts),
                            prefix_row=None if prefix_row is None else ints(prefix_row))
        got = R.paged_attention(q, cache, plan, mask=None if mask is None else dev(mask), scale=scale)
    bf16 = q.dtype == torch.bfloat16
    scale = D ** -0.5 if scale is None else scale
    m = None if mask is None else np.broadcast_to(mask, (B, N, N))
    # a probability rounds to bf16 before it meets V with bf16 queries, and so does the output
    want, wlse, tol, ltol = ref.attend(f64(q), f64(cache.k_pages), f64(cache.v_pages), tables, lens, B, counts, prefix_row, m,
                                       scale, 2.0 ** -8 if bf16 else U)
    tol = tol + (2.0 ** -8 if bf16 else U) * 1.01 * np.abs(want)
    out, lse = f64(got[0]), f64(got[1])
    bad = ~(np.abs(out - want) <= tol + 1e-37)
    assert not bad.any(), (np.argwhere(bad)[:3], out[bad][:3], want[bad][:3], tol[bad][:3])
    assert np.array_equal(np.isneginf(lse), np.isneginf(wlse))
    live = ~np.isneginf(wlse)
    assert (np.abs(lse[live] - wlse[live]) <= ltol[live] + 1e-30).all()
    assert (out[~live] == 0).all()
    return got


CASES = [
    # B, N, H, G, D, P, lengths, prefixes (lengths), mask
    dict(B=1, N=1, H=1, G=1, D=64, P=16, lens=[0], pre=[]),
    dict(B=3, N=1, H=2, G=4, D=128, P=16, lens=[5, 0, 63], pre=[]),
    dict(B=4, N=1, H=8, G=4, D=128, P=16, lens=[100, 1, 64, 31], pre=[500]),
    dict(B=5, N=3, H=2, G=3, D=64, P=32, lens=[17, 200, 0, 64, 333], pre=[127, 128]),
    dict(B=6, N=8, H=2, G=4, D=128, P=64, lens=[70, 0, 129, 1000, 3, 5], pre=[1, 1023]),
    dict(B=4, N=27, H=2, G=5, D=128, P=16, lens=[70, 0, 129, 400], pre=[300], tree=True),
    dict(B=2, N=64, H=1, G=2, D=256, P=128, lens=[65, 1], pre=[70, 0], tree=True),
    dict(B=2, N=100, H=2, G=2, D=64, P=16, lens=[37, 0], pre=[200]),
    dict(B=2, N=193, H=1, G=3, D=128, P=16, lens=[0, 70], pre=[]),
    dict(B=1, N=2, H=2, G=2, D=256, P=1024, lens=[3000], pre=[2047]),
    dict(B=40, N=1, H=1, G=8, D=128, P=16, lens=[(37 * i) % 101 for i in range(40)], pre=[333, 64]),
    dict(B=2, N=5, H=16, G=1, D=64, P=16, lens=[5000, 77], pre=[]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(c[k]) for k in ("B", "N", "H", "G", "D", "P")))
def test_attention(R, case, dtype):
    rng = np.random.default_rng(case["D"] + case["N"])
    B, N, H, G, D, P = (case[k] for k in ("B", "N", "H", "G", "D", "P"))
    lens = case["lens"] + case["pre"]
    width = max(-(-(n + N) // P) for n in lens)
    pages = sum(-(-(n + N) // P) for n in lens) + 2
    cache = make_cache(R, rng, pages, P, H, D, list(LAYOUTS)[case["N"] % 4])
    tables = make_tables(rng, pages, P, lens, N, B, width)
    prefix = None
    if case["pre"]:
        prefix = np.array([B + b * len(case["pre"]) // B for b in range(B)])
        if B > 3:
            prefix[1] = -1                                    # one without, inside a run
    mask = tree_masks(rng, B, N) if case.get("tree") else None
    q = queries(rng, B, N, H * G, D, dtype)
    check(R, q, cache, tables, lens, B, prefix_row=prefix, mask=mask)
    counts = rng.integers(0, N + 1, B)
    check(R, q, cache, tables, lens, B, counts=counts, prefix_row=prefix, mask=mask, scale=0.3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_share_nothing_alternate_or_are_errors(R, dtype):
    rng = np.random.default_rng(9)
    B, N, H, G, D, P = 9, 2, 2, 2, 64, 16
    lens = [10, -1, 30, 161, 20, 0, 40, 50, 60, 100, 130, -3, 1000]
    width = 10
    pages = 200
    cache = make_cache(R, rng, pages, P, H, D)
    tables = rng.integers(0, pages, (13, width)).astype(np.int32)      # pages may be shared at will
    prefix = [9, 9, 10, 9, 13, 9, 11, 12, 0]                  # 13 is no row, 11 has no length, 12 too long; the last: batch row 0
    counts = [2, 2, 3, 2, 2, -1, 2, 2, 1]
    q = queries(rng, B, N, H * G, D, dtype)
    got = check(R, q, cache, tables, lens, B, counts=counts, prefix_row=prefix)
    assert (got[0][[1, 2, 3, 4, 5, 6, 7]] == 0).all()
    check(R, q, cache, tables, lens, B, prefix_row=prefix)
    check(R, q, cache, tables, lens, B, counts=counts)


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "bf16"), (256, "bf16"), (128, "f32")])
def test_what_is_not_seen_does_not_reach(R, D, dtype):
    """NaN and infinities behind the sequences' ends, in other pages, and in tokens a query's mask hides."""
    import torch
    rng = np.random.default_rng(D)
    B, N, H, G, P = 2, 6, 2, 3, 16
    lens, width, pages = [37, 5, 41], 4, 16
    cache = make_cache(R, rng, pages, P, H, D)
    tables = make_tables(rng, pages, P, lens, N, B, width)
    mask = np.repeat(np.eye(N, dtype=np.uint8)[None], B, 0)
    mask[:, :, 0] = 1
    mask[0, 4] = 0                                            # sees no new token
    used = torch.zeros(pages, P, dtype=torch.bool, device="cuda")
    for t, n in enumerate(lens):
        for s in range(n + (N if t < B else 0)):
            used[tables[t, s // P], s % P] = True
    for i, bad in enumerate((float("nan"), float("inf"), -float("inf"))):
        cache.k_pages[~used] = bad
        cache.v_pages[~used] = bad
        q = queries(rng, B, N, H * G, D, dtype)
        check(R, q, cache, tables, lens, B, prefix_row=[2, 2], mask=mask)
        # token 3's rows are bad: every other token's output is as it was
        clean = [t.clone() for t in (cache.k_pages, cache.v_pages)]
        plan = R.paged_plan(cache, ints(tables), ints(lens), N, H * G, B=B, prefix_row=ints([2, 2]))
        first = R.paged_attention(q, cache, plan, mask=dev(mask))
        for b in range(B):
            s = lens[b] + 3
            (cache.v_pages if i < 2 else cache.k_pages)[tables[b, s // P], s % P, :, 7] = bad
        second = R.paged_attention(q, cache, plan, mask=dev(mask))
        others = [0, 1, 2, 4, 5]
        assert torch.equal(first[0][:, others], second[0][:, others]) and torch.equal(first[1][:, others], second[1][:, others])
        assert torch.isfinite(first[0]).all()
        if i == 0:
            assert torch.isnan(second[0][:, 3]).any()
        cache.k_pages.copy_(clean[0])
        cache.v_pages.copy_(clean[1])


def test_pages_that_are_none(R):
    """A table that names a page outside the pool: the queries that see its slots answer NaN, the others what they did."""
    import torch
    rng = np.random.default_rng(2)
    B, N, H, G, D, P = 3, 2, 1, 2, 128, 16
    lens, width, pages = [40, 40, 200, 90], 16, 40
    cache = make_cache(R, rng, pages, P, H, D)
    tables = make_tables(rng, pages, P, lens, N, B, width)
    q = queries(rng, B, N, H * G, D, "bf16")
    args = dict(B=B, prefix_row=ints([3, -1, 3]))
    first = R.paged_attention(q, cache, R.paged_plan(cache, ints(tables), ints(lens), N, H * G, **args))
    for bad in (-1, pages, 2 ** 31 - 1, -2 ** 31):
        broken = tables.copy()
        broken[1, 1] = bad
        got = R.paged_attention(q, cache, R.paged_plan(cache, ints(broken), ints(lens), N, H * G, **args))
        assert torch.isnan(got[0][1]).all() and torch.isnan(got[1][1]).all()
        assert torch.equal(got[0][[0, 2]], first[0][[0, 2]]) and torch.equal(got[1][[0, 2]], first[1][[0, 2]])
        broken = tables.copy()
        broken[3, 5] = bad                                    # in the prefix of the other two
        got = R.paged_attention(q, cache, R.paged_plan(cache, ints(broken), ints(lens), N, H * G, **args))
        assert torch.isnan(got[0][[0, 2]]).all() and torch.equal(got[0][1], first[0][1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,H,G,D,shared,tail", [
    (1, 1, 8, 8, 128, None, 9000), (1, 1, 1, 1, 64, None, 20000), (4, 8, 2, 1, 256, 3000, 500), (32, 1, 2, 1, 64, 700, 900),
    (6, 1, 4, 5, 128, 1, 400), (3, 10, 2, 3, 128, None, 1500), (16, 2, 3, 1, 128, 5000, 1),
])
def test_small_calls_again_and_again(R, B, N, H, G, D, shared, tail, dtype):
    """Few rows, cut into many units: layer after layer on one plan the same bits; then other lengths."""
    import torch
    rng = np.random.default_rng(B + N + D)
    P = 16
    for again in range(2):
        lens = [tail if b == 0 else int(x) for b, x in enumerate(rng.integers(0, tail + 1, B))] + ([] if shared is None else [shared])
        width = -(-max(n + N for n in lens) // P)
        pages = sum(-(-(n + N) // P) for n in lens)
        cache = make_cache(R, rng, pages, P, H, D)
        tables = make_tables(rng, pages, P, lens, N, B, width)
        prefix = None if shared is None else [B if b != 1 else -1 for b in range(B)]
        counts = rng.integers(0, N + 1, B)
        counts[0] = N
        q = queries(rng, B, N, H * G, D, dtype)
        plan = R.paged_plan(cache, ints(tables), ints(lens), N, H * G, B=B, counts=ints(counts),
                            prefix_row=None if prefix is None else ints(prefix))
        first = R.paged_attention(q, cache, plan)
        check(R, q, cache, tables, lens, B, counts=counts, prefix_row=prefix, got=first)
        others = [queries(rng, B, N, H * G, D, dtype) for _ in range(3)]
        for k in range(20):
            R.paged_attention(others[k % 3], cache, plan)     # (its workspace has held other parts)
            out, lse = R.paged_attention(q, cache, plan)
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,H,G,D,P,shared,tail", [
    (24, 1, 8, 8, 128, 16, 9000, 300), (3, 8, 2, 4, 64, 64, 30011, 100), (1, 1, 1, 1, 128, 16, 70000, 3), (8, 20, 4, 4, 128, 16, 2500, 900),
])
def test_long_prefixes(R, B, N, H, G, D, P, shared, tail, dtype):
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(0, tail + 1, B)] + [shared]
    width = -(-max(shared, tail + N) // P)
    pages = sum(-(-(n + N) // P) for n in lens)
    cache = make_cache(R, rng, pages, P, H, D)
    tables = make_tables(rng, pages, P, lens, N, B, width)
    check(R, queries(rng, B, N, H * G, D, dtype), cache, tables, lens, B, prefix_row=[B] * B)


@pytest.mark.parametrize("B,N", [(1024, 2), (1300, 1), (2500, 3), (1030, 130)])
def test_many_rows(R, B, N):
    """More rows than the plan looks at at a time, runs of prefixes across its borders, windows of several tiles among them."""
    rng = np.random.default_rng(B)
    H, G, D, P, width = 1, 1, 64, 16, 12
    lens = rng.integers(0, 40, B).tolist() + [150, 0, 60]
    pages = 400
    cache = make_cache(R, rng, pages, P, H, D)
    tables = rng.integers(0, pages, (B + 3, width)).astype(np.int32)
    prefix = B + (np.arange(B) // 300) % 3
    prefix[rng.random(B) < 0.01] = -1
    counts = np.where(rng.random(B) < 0.03, N, rng.integers(0, min(N, 2) + 1, B))
    counts[[0, B - 1]] = N
    check(R, queries(rng, B, N, H * G, D, "bf16"), cache, tables, lens, B, counts=counts, prefix_row=prefix)


def test_a_plan_of_other_sizes_writes_nothing(R):
    import ctypes
    import torch
    rng = np.random.default_rng(1)
    cache = make_cache(R, rng, 8, 16, 2, 64)
    tables, lens = ints([[0, 1], [2, 3]]), ints([5, 9])
    plan = R.paged_plan(cache, tables, lens, 3, 4)
    other = R.paged_plan(cache, tables, lens, 2, 4)
    plan._buffer, plan._ptr = other._buffer, other._ptr       # as a C caller might mix them up
    out = (torch.full((2, 3, 4, 64), 7.0, device="cuda"), torch.full((2, 3, 4), 7.0, device="cuda"))
    q = queries(rng, 2, 3, 4, 64, "f32")
    R.paged_attention(q, cache, plan, out=out)
    assert (out[0] == 7).all() and (out[1] == 7).all()


def test_a_plan_of_other_heads_writes_nothing(R):
    """As many query rows a head, but the plan cuts them up by the number of heads."""
    import torch
    rng = np.random.default_rng(2)
    tables, lens = ints([[0, 1], [2, 3], [4, 5]]), ints([5, 9, 20])
    four, two = make_cache(R, rng, 8, 16, 4, 64), make_cache(R, rng, 8, 16, 2, 64)
    plan = R.paged_plan(four, tables, lens, 3, 8, B=2, prefix_row=ints([2, 2]))
    other = R.paged_plan(two, tables, lens, 3, 4, B=2, prefix_row=ints([2, 2]))
    assert other.bytes > plan.bytes
    plan._buffer, plan._ptr, plan.bytes = other._buffer, other._ptr, other.bytes
    out = (torch.full((2, 3, 8, 64), 7.0, device="cuda"), torch.full((2, 3, 8), 7.0, device="cuda"))
    R.paged_attention(queries(rng, 2, 3, 8, 64, "f32"), four, plan, out=out)
    assert (out[0] == 7).all() and (out[1] == 7).all()


@pytest.mark.parametrize("layout", ["slots", "outer"])
def test_offsets_past_32_bits(R, layout):
    """Pages all over a cache of more than 2^32 bytes (and 2^31 elements): what a small cache of the same rows gives."""
    import torch
    rng = np.random.default_rng(6)
    B, N, H, G, D, P = 3, 2, 8, 2, 128, 16
    lens, width = [300, 40, 700], 50
    few, many = 120, 140001
    shape = [(many, P, H)[i] for i in LAYOUTS[layout]] + [D]
    back = [LAYOUTS[layout].index(i) for i in range(3)] + [3]
    big = R.PagedCache(*(torch.empty(shape, dtype=torch.bfloat16, device="cuda").permute(*back) for _ in range(2)))
    small = make_cache(R, rng, few, P, H, D)
    at = np.append(rng.choice(many - 1, few - 1, replace=False), many - 1)       # where its pages lie in the big one
    for to, src in ((big.k_pages, small.k_pages), (big.v_pages, small.v_pages)):
        to[dev(at)] = src
    tables = make_tables(rng, few, P, lens, N, 2, width)
    tables[2][:3] = few - 1, tables[2][1], few - 1
    far = np.where(tables < 0, -1, at[tables])
    kv = torch.from_numpy(rng.standard_normal((2, 2, N, H, D)).astype(np.float32)).cuda()
    q = queries(rng, 2, N, H * G, D, "bf16")
    got = []
    for cache, t in ((small, tables), (big, far)):
        slots = np.array([[t[b, (lens[b] + n) // P] * P + (lens[b] + n) % P for n in range(N)] for b in range(2)])
        R.paged_append(cache, kv[:, 0], kv[:, 1], ints(slots))
        plan = R.paged_plan(cache, ints(t), ints(lens), N, H * G, B=2, prefix_row=ints([2, 2]))
        got.append(R.paged_attention(q, cache, plan))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1]) and torch.isfinite(got[0][0]).all()
    for a, b in ((small.k_pages, big.k_pages), (small.v_pages, big.v_pages)):
        assert torch.equal(a.contiguous(), b[dev(at)].contiguous())


def test_streams_and_graphs(R):
    """Captured together and replayed on new lengths, with eager calls between; and on a stream of its own."""
    import torch
    rng = np.random.default_rng(12)
    B, N, H, G, D, P = 6, 3, 2, 4, 128, 16
    pages, width = 200, 40
    cache = make_cache(R, rng, pages, P, H, D)
    pool = R.new_page_pool(B + 1, width, pages, P, "cuda")
    lengths, counts = ints([0] * (B + 1)), ints([0] * (B + 1))
    kv = torch.from_numpy(rng.standard_normal((B, 2, N, H, D)).astype(np.float32)).cuda().bfloat16()
    q = queries(rng, B, N, H * G, D, "bf16")
    prefix = ints([B] * B)

    def step(plan=None):
        granted, slots = R.page_step(pool, lengths, N, counts=counts)
        R.paged_append(cache, kv[:, 0], kv[:, 1], slots[:B])
        plan = R.paged_plan(cache, pool.tables, lengths, N, H * G, B=B, counts=granted[:B], prefix_row=prefix, out=plan)
        return (granted, slots, *R.paged_attention(q, cache, plan)), plan

    def reset(seed):
        g = np.random.default_rng(seed)
        new = R.new_page_pool(B + 1, width, pages, P, "cuda")
        for to, src in ((pool.tables, new.tables), (pool.held, new.held), (pool.ring, new.ring), (pool.state, new.state)):
            to.copy_(src)
        lens = g.integers(0, 130, B + 1)
        R.page_step(pool, ints([0] * (B + 1)), 300, counts=ints(lens))       # room for what is committed
        lengths.copy_(ints(lens))
        counts.copy_(ints(g.integers(0, N + 1, B + 1)))
        torch.cuda.synchronize()

    side = torch.cuda.Stream()
    reset(0)
    with torch.cuda.stream(side):
        _, plan = step()
    side.synchronize()
    reset(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = step(plan)
    for seed in range(1, 4):
        reset(seed)
        eager = [t.clone() for t in step()[0]]
        reset(seed)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert torch.equal(a, b)
        reset(seed)
        with torch.cuda.stream(side):
            other = step()[0]
        side.synchronize()
        for a, b in zip(other, eager):
            assert torch.equal(a, b)


@pytest.mark.parametrize("B,N", [(8, 2), (4, 2), (3, 1)])
def test_calls_at_once(R, B, N):
    """One plan, two streams, each with its own queries and workspace; and two pools at once."""
    import torch
    rng = np.random.default_rng(31)
    H, G, D, P = 2, 4, 128, 16
    lens = rng.integers(0, 900, B).tolist() + [3000]
    width, pages = 200, sum(-(-(n + N) // P) for n in lens)
    cache = make_cache(R, rng, pages, P, H, D)
    tables = ints(make_tables(rng, pages, P, lens, N, B, width))
    plan = R.paged_plan(cache, tables, ints(lens), N, H * G, B=B, prefix_row=ints([B] * B))
    qs = [queries(rng, B, N, H * G, D, "bf16") for _ in range(2)]
    need = R.paged_attention_workspace_bytes(plan, D) + 256
    work = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    want = [R.paged_attention(q, cache, plan) for q in qs]
    pools = [R.new_page_pool(64, 30, 700, 16, "cuda") for _ in range(2)]
    lengths = [ints(rng.integers(0, 100, 64)) for _ in range(2)]
    alone = [R.page_step(R.new_page_pool(64, 30, 700, 16, "cuda"), n, 40) for n in lengths]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got, steps = [[], []], [None, None]
    for k in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(R.paged_attention(qs[i], cache, plan, workspace=work[i]))
                if k == 0:
                    steps[i] = R.page_step(pools[i], lengths[i], 40)
    torch.cuda.synchronize()
    for i in range(2):
        for o, l in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])
        assert torch.equal(steps[i][0], alone[i][0]) and torch.equal(steps[i][1], alone[i][1])


def test_a_speculative_run(R):
    """Prompts into the pages, drafts behind them, verification, accepted rows in place, and log probabilities: three
    steps against attention over each sequence's own rows kept apart."""
    import torch
    rng = np.random.default_rng(21)
    B, N, H, G, D, P, V = 3, 7, 2, 2, 64, 16, 1000
    T, width, pages = B + 1, 8, 40
    cache = make_cache(R, rng, pages, P, H, D, fill=0x7fc0)   # NaN where nothing was written
    pool = R.new_page_pool(T, width, pages, P, "cuda")
    g = torch.Generator("cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")      # noqa: E731
    kept = [[[], []] for _ in range(T)]                       # K and V rows of every table row, as they should be

    lengths, counts = ints([0] * T), [30, 1, 17, 45]
    granted, slots = R.page_step(pool, lengths, 45, counts=ints(counts))
    k, v = rand(T, 45, H, D), rand(T, 45, H, D)
    R.paged_append(cache, k, v, slots)
    for t in range(T):
        kept[t][0].append(k[t, :counts[t]])
        kept[t][1].append(v[t, :counts[t]])
    lengths = ints(counts)
    prefix = ints([B, B, B])
    parents = [-1, 0, 0, 1, 1, 2, 3]
    mask = np.zeros((N, N), np.uint8)
    for n in range(N):
        mask[n, n] = 1
        if n:
            mask[n] |= mask[parents[n]]
    for step in range(3):
        granted, slots = R.page_step(pool, lengths, N, counts=ints([N] * B + [0]))
        assert granted.tolist() == [N] * B + [0]
        plan = R.paged_plan(cache, pool.tables, lengths, N, H * G, B=B, counts=granted[:B], prefix_row=prefix)
        k, v, q = rand(B, N, H, D), rand(B, N, H, D), rand(B, N, H * G, D)
        R.paged_append(cache, k, v, slots[:B])
        out, lse = R.paged_attention(q, cache, plan, mask=dev(mask))
        for b in range(B):
            K, W = (torch.cat(kept[B][i] + kept[b][i] + [x[b]]).bfloat16().double() for i, x in ((0, k), (1, v)))
            s = torch.stack([q[b, :, hq].double() @ K[:, hq // G].T for hq in range(H * G)]) / D ** 0.5
            s[:, :, -N:].masked_fill_(dev(mask) == 0, float("-inf"))
            want = torch.stack([s[hq].softmax(-1) @ W[:, hq // G] for hq in range(H * G)], 1)
            assert (out[b] - want).abs().max() < 1e-4 and (lse[b] - s.logsumexp(-1).T).abs().max() < 1e-4
        logits = 2 * rand(B, N, V)
        nodes = logits.argmax(-1).to(torch.int32)[:, [0 if p < 0 else p for p in parents]]
        nodes[:, 2] = 3                                       # some nodes are wrong
        nodes[1, 1] = 5
        path, tokens, alen = R.verify_tree_greedy(logits, nodes, parents)
        R.paged_append(cache, k, v, slots[:B], path=path, accept_len=alen)
        r = R.token_logprobs(logits.gather(1, path.clamp(min=0).long().unsqueeze(-1).expand(-1, -1, V)), tokens, top_n=1)
        for b in range(B):
            d = int(alen[b])
            at = path[b, :d + 1].long()
            kept[b][0].append(k[b, at])
            kept[b][1].append(v[b, at])
            rows = logits[b, at].double().log_softmax(-1)
            want = rows.gather(1, tokens[b, :d + 1].long().view(-1, 1)).view(-1)
            assert (r.logprobs[b, :d + 1] - want).abs().max() < 1e-5 and (r.logprobs[b, d + 1:] == 0).all()
            assert torch.equal(r.top_tokens[b, :d + 1, 0], tokens[b, :d + 1])      # greedy: the likeliest
        lengths = lengths + torch.cat((alen + 1, ints([0])))
    assert alen.max() > 0
    # one sequence ends, its pages are handed out again
    lengths[1] = -1
    free = int(pool.state[1])
    granted, _ = R.page_step(pool, lengths, 1, counts=ints([0, 0, 0, 0]))
    assert granted.tolist() == [0, 0, 0, 0] and pool.held[1] == 0 and int(pool.state[1]) > free


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,n", [(40, 16384), (40, 32768), (1, 32768), (8, 65536)])
@pytest.mark.parametrize("top", [16.5, 17.375, 18.0])
def test_one_key_of_weight_one(R, dtype, N, n, top):
    """And many of 2^-24 to 2^-26, each less than the sum's last place. Units that are not split (as many batch rows as that takes,
    all on the same pages), of 128 query rows and of 32. Scores are exact here: the queries have one element, the keys too.

    lse: m and the sum's logarithm meet near 25, in base two, off by half a step there (2^-20) and half a step of the product with
    ln 2 (2^-20); log2(e)/8 is off by 2^-25 of 25; the sum itself by a few 2^-24: 3e-6 in all.  An output of float32 queries: three
    parts of P, each eight keys' sum rounded to nearest at the output's size: six times the root of the sum of the squares."""
    import torch
    rng = np.random.default_rng(n + N)
    B, H, D, P = 64, 8, 64, 256
    cache = make_cache(R, rng, n // P + 1, P, H, D)
    cache.k_pages.zero_()
    cache.k_pages[0, 3, :, 0] = top
    tables = np.arange(n // P + 1, dtype=np.int32)[None].repeat(B, 0)
    q = torch.zeros(B, N, H, D, device="cuda")
    q[..., 0] = 8.0
    q = q.bfloat16() if dtype == "bf16" else q
    out, lse = R.paged_attention(q, cache, R.paged_plan(cache, ints(tables), ints([n] * B), N, H))
    others = n - 1 + np.arange(1, N + 1)
    w = np.exp(-top)
    assert np.abs(f64(lse) - (top + np.log1p(others * w))[None, :, None]).max() < 3e-6
    if dtype == "f32":
        v = f64(cache.v_pages).reshape(-1, H, D)
        rest = np.cumsum(v, 0)[n - 1 + np.arange(1, N + 1)] - v[3]
        want = (v[3] + w * rest) / (1 + others * w)[:, None, None]
        tol = 6 * np.sqrt(3 * (n + N) / 8 / 12) * 2.0 ** -22 * np.abs(want) + 2.0 ** -23
        assert (np.abs(f64(out) - want) < tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("N,n", [(3, 900), (50, 2100)])
@pytest.mark.parametrize("size", [2.0 ** 26, 2.0 ** 33, 2.0 ** 40, 2.0 ** 110])
def test_large_scores(R, dtype, D, N, n, size):
    """Scores whose product with log2(e)*scale rounds by more than a power of two: the largest key alone has weight, or those of the
    same score share it. Queries of one element, so that scores are exact, negative ones in every second row."""
    import torch
    rng = np.random.default_rng(N)
    B, H, G, P = 2, 2, 1, 16
    lens = [n, 5, 700]
    width = -(-(n + N) // P)
    pages = sum(-(-(x + N) // P) for x in lens)
    cache = make_cache(R, rng, pages, P, H, D)
    tables = make_tables(rng, pages, P, lens, N, B, width)
    cache.k_pages[..., 1:] = 0
    cache.k_pages[..., 0] = dev(rng.integers(1, 255, (pages, P, H)).astype(np.float32) / 128).bfloat16()       # ties among them
    q = torch.zeros(B, N, H * G, D, device="cuda")
    q[..., 0] = size
    q[:, 1::2] *= -1
    q = q.bfloat16() if dtype == "bf16" else q
    got = R.paged_attention(q, cache, R.paged_plan(cache, ints(tables), ints(lens), N, H * G, B=B, prefix_row=ints([2, 2])))
    assert torch.isfinite(got[0]).all() and torch.isfinite(got[1]).all()
    check(R, q, cache, tables, lens, B, prefix_row=[2, 2], got=got)


@pytest.mark.parametrize("B,heads,n", [(65536, 8, 2 ** 30 - 1), (65535, 16, 2 ** 30 - 1), (4096, 512, 2 ** 30 - 1), (65536, 8, 2 ** 29 + 77)])
def test_a_plan_of_the_longest_rows(R, B, heads, n):
    """More chunks in all than 2^31 a unit of the target: every job is one unit, and nothing is written behind the plan."""
    import ctypes
    import torch
    need = R.lib().spec_paged_plan_bytes(B, 1, heads, heads, 64, 1)
    plan = torch.full((need + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    off = -plan.data_ptr() % 256
    lengths, prefix = torch.full((B,), n, dtype=torch.int32, device="cuda"), torch.full((B,), -1, dtype=torch.int32, device="cuda")
    rc = R.lib().spec_paged_plan(B, 1, heads, heads, 64, B, 1 << 20, 1024, lengths.data_ptr(), None, prefix.data_ptr(),
                                 plan.data_ptr() + off, need, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    words = plan[off:off + need].view(torch.int32)
    assert words[0].item() == B
    units = words[64:64 + 12 * B].view(B, 12)                 # behind the sizes, 256 bytes: 48 a unit
    assert (units[:, 4] == 0).all() and (units[:, 5] == n + 1).all() and (units[:, 8] == -1).all()
    assert torch.equal(units[:, 0].sort().values, torch.arange(B, dtype=torch.int32, device="cuda"))
    assert (plan[off + need:] == 0x5a).all() and (plan[:off] == 0x5a).all()


@pytest.mark.parametrize("seed", range(12))
def test_plans_stay_within_their_sizes(R, seed):
    """Units and rows of parts of random batches: all there is room for, no part in two units, every key of every query row once."""
    import torch
    rng = np.random.default_rng(seed)
    for _ in range(12):
        B, N, G, H = int(rng.choice([1, 2, 3, 7, 30, 64, 500, 1500])), int(rng.choice([1, 2, 7, 27, 70])), int(rng.choice([1, 3, 8])), int(rng.choice([1, 2, 4, 8, 32]))
        D = int(rng.choice([64, 256]))
        if B * N > 20000:
            N = 1
        runs = int(rng.integers(1, 5))
        long = int(rng.choice([10, 600, 9000]))
        lens = np.concatenate((rng.integers(0, int(rng.choice([2, 300, 3000])), B), rng.integers(0, long, runs)))
        prefix = B + np.sort(rng.integers(0, runs, B))
        prefix[rng.random(B) < 0.1] = -1
        if rng.random() < 0.3:
            prefix = B + np.arange(B) % runs                  # no two neighbours alike
        P, width = 64, 200
        cache = make_cache(R, rng, 1, P, H, D)
        plan = R.paged_plan(cache, torch.zeros(B + runs, width, dtype=torch.int32, device="cuda"), ints(lens), N, H * G, B=B, prefix_row=ints(prefix))
        words = plan._buffer[plan._ptr - plan._buffer.data_ptr():][:plan.bytes].view(torch.int32).cpu().numpy()
        n, M = int(words[0]), N * G
        own_tiles = 1 if M <= 32 else -(-M // 128)
        target = -(-(256 if D == 256 else 512) // H)
        assert n <= 2 * B * own_tiles + target
        u = words[64:64 + 12 * n].reshape(n, 12)
        rows = (R.paged_attention_workspace_bytes(plan, D)) // (H * (D + 2) * 4)
        tile = np.where(u[:, 9] != 0, 128, 32)
        part = u[u[:, 8] >= 0]
        ends = part[:, 8] + tile[u[:, 8] >= 0]
        order = np.argsort(part[:, 8])
        assert ends.max(initial=0) <= rows and (ends[order][:-1] <= part[order][1:, 8]).all()
        seen = (u[:, 5] - u[:, 4]).astype(np.int64) * np.minimum(tile, u[:, 2] - u[:, 1])
        shared = np.where(prefix >= 0, lens[np.maximum(prefix, 0)], 0)
        least = (M * (shared + lens[:B])).sum()
        assert least <= seen.sum() <= least + M * N * B       # new tokens: those a tile looks at


@pytest.mark.parametrize("T,N", [(300, 5000), (1024, 1025), (1025, 1500), (9000, 1030)])
@pytest.mark.parametrize("in_place", [True, False])
def test_prompts_of_many_rows(R, T, N, in_place):
    """More rows than there are workgroups for each 1024 tokens of them."""
    import torch
    rng = np.random.default_rng(T)
    P, width = 128, -(-(N + 200) // 128)
    pool = make_pool(R, rng, T, width, P, fill=0.2, spare=int(0.4 * T * width))
    tables, held, ring, state = pool_arrays(pool)
    lengths = np.maximum(held * P - rng.integers(0, 2 * P, T), 0).astype(np.int32)
    lengths[rng.random(T) < 0.1] = -1
    counts = rng.integers(0, N + 1, T).astype(np.int32)
    want = ref.page_step(tables, held, ring, state, lengths, counts, N, P)
    oh, os = (None, None) if in_place else (torch.full_like(pool.held, 77), torch.full_like(pool.state, 77))
    granted, slots = R.page_step(pool, ints(lengths), N, counts=ints(counts), out_held=oh, out_state=os)
    got = (granted, slots, pool.tables, pool.held if in_place else oh, pool.ring, pool.state if in_place else os)
    for name, g, w in zip(("granted", "slots", "tables", "held", "ring", "state"), got, want):
        assert np.array_equal(g.cpu().numpy(), w), name
    assert (want[0] > 0).any() and not pool._workspace.any()


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "bf16"), (256, "bf16"), (64, "f32"), (128, "f32"), (256, "f32")])
@pytest.mark.parametrize("N", [1, 3, 40])
def test_pages_that_are_none_far_along(R, D, dtype, N):
    """In units that are not split, of 32 query rows and of 128: a bad page in any of the windows of 64 groups of keys that a wave
    holds the pages of, at their edges, and among the new tokens. Who sees it answers NaN, everyone else the same bits."""
    import torch
    rng = np.random.default_rng(D + N)
    B, H, P, n = 64, 8, 16, 4201
    width = -(-(n + N) // P)
    cache = make_cache(R, rng, width + 5, P, H, D)
    tables = np.stack([rng.permutation(width + 5)[:width] for _ in range(B)]).astype(np.int32)     # pages in common, in any order
    lens = np.full(B, n)
    lens[1::4] = 700                                          # one window alone
    q = queries(rng, B, N, H, D, dtype)
    first = R.paged_attention(q, cache, R.paged_plan(cache, ints(tables), ints(lens), N, H))
    few = [0, 1, 2, 3]                                        # (by the definition itself)
    check(R, q[few], cache, tables[few], lens[few], 4, got=[t[few] for t in first])
    for page in (0, 1, 31, 32, 43, 63, 64, 65, 127, 128, 191, 192, 255, 256, width - 2, width - 1):
        broken = tables.copy()
        hit = rng.random(B) < 0.4
        broken[hit, page] = rng.choice([-1, width + 5, 2 ** 31 - 1])
        got = R.paged_attention(q, cache, R.paged_plan(cache, ints(broken), ints(lens), N, H))
        sees = dev(hit[:, None] & (lens[:, None] + np.arange(N) >= page * P))
        assert torch.isnan(got[0][sees]).all() and torch.isnan(got[1][sees]).all(), page
        assert torch.equal(got[0][~sees], first[0][~sees]) and torch.equal(got[1][~sees], first[1][~sees]), page


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "f32"), (256, "bf16"), (256, "f32")])
def test_bad_pages_of_a_prefix(R, D, dtype):
    """Of several windows, read by tiles of 128 query rows: its own sequences answer NaN, those of the other prefix what they did."""
    import torch
    rng = np.random.default_rng(D)
    B, N, H, G, P, n = 24, 4, 32, 2, 16, 5003                 # 32 heads: 16 units a head, of some 600 keys and more
    lens = [5] * B + [n, n]
    width = -(-(n + N) // P)
    pages = 2 * width + B + 5
    cache = make_cache(R, rng, pages, P, H, D)
    tables = make_tables(rng, pages, P, lens, N, B, width)
    q = queries(rng, B, N, H * G, D, dtype)
    prefix = [B] * 12 + [B + 1] * 12
    first = R.paged_attention(q, cache, R.paged_plan(cache, ints(tables), ints(lens), N, H * G, B=B, prefix_row=ints(prefix)))
    for page in (0, 63, 64, 100, 128, 200, width - 1):
        for row in (0, 1):
            broken = tables.copy()
            broken[B + row, page] = -7
            got = R.paged_attention(q, cache, R.paged_plan(cache, ints(broken), ints(lens), N, H * G, B=B, prefix_row=ints(prefix)))
            bad, same = (slice(0, 12), slice(12, 24)) if row == 0 else (slice(12, 24), slice(0, 12))
            if page * P < n:
                assert torch.isnan(got[0][bad]).all() and torch.isnan(got[1][bad]).all()
            assert torch.equal(got[0][same], first[0][same]) and torch.equal(got[1][same], first[1][same])


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "bf16"), (256, "bf16"), (64, "f32"), (128, "f32"), (256, "f32")])
@pytest.mark.parametrize("N,G", [(50, 1), (27, 5), (64, 3)])
def test_hidden_new_tokens_in_large_windows(R, D, dtype, N, G):
    """More than 32 query rows: a new token of NaN or infinity reaches only those whose mask shows it."""
    import torch
    rng = np.random.default_rng(D + N)
    B, H, P = 3, 2, 16
    lens = [37, 1029, 0, 70]
    width = -(-(max(lens) + N) // P)
    pages = sum(-(-(x + N) // P) for x in lens)
    cache = make_cache(R, rng, pages, P, H, D)
    tables = make_tables(rng, pages, P, lens, N, B, width)
    mask = tree_masks(rng, B, N)
    q = queries(rng, B, N, H * G, D, dtype)
    plan = R.paged_plan(cache, ints(tables), ints(lens), N, H * G, B=B, prefix_row=ints([3, 3, -1]))
    first = check(R, q, cache, tables, lens, B, prefix_row=[3, 3, -1], mask=mask)
    for node in (0, 2, 15, 16, N - 1):
        for what, bad in (("k", float("inf")), ("v", float("nan")), ("v", -float("inf")), ("k", float("nan"))):
            t = cache.k_pages if what == "k" else cache.v_pages
            keep = t.clone()
            for b in range(B):
                s = lens[b] + node
                t[tables[b, s // P], s % P, :, 5] = bad
            got = R.paged_attention(q, cache, plan, mask=dev(mask))
            hidden = dev(mask[:, :, node] == 0)
            assert torch.equal(got[0][hidden], first[0][hidden]) and torch.equal(got[1][hidden], first[1][hidden]), (node, what, bad)
            t.copy_(keep)


@pytest.mark.parametrize("N,D,n,split", [(2, 64, 9000, True), (2, 128, 65536, True), (40, 128, 20000, True), (2, 64, 65536, False),
                                         (40, 64, 30000, False), (40, 256, 9000, False)])
def test_long_sums_of_float32(R, N, D, n, split):
    """Float32 queries behind many keys, with bounds that do not grow with the keys as a sum that adds them one by one would be off.

    A score goes through D/8 additions of each of three parts, half a step each in either direction: six times the root of the sum
    of their squares, sqrt(D/8) half steps of its size. The sum of the exponentials keeps what it rounds off, and lies in a few
    dozen parts; lse has a few roundings of its own. An output's additions, one for eight keys and each of three parts, likewise."""
    import torch
    rng = np.random.default_rng(n + N + D)
    H, P = 8, 64
    B = 2 if split else 64                                    # (of the same pages)
    cache = make_cache(R, rng, n // P + 2, P, H, D)
    tables = np.tile(rng.permutation(n // P + 2).astype(np.int32), (B, 1))
    q = queries(rng, B, N, H, D, "f32")
    out, lse = R.paged_attention(q, cache, R.paged_plan(cache, ints(tables), ints([n] * B), N, H))
    K, V = (t[dev(tables[0].astype(np.int64))].view(-1, H, D)[:n + N].double().transpose(0, 1).contiguous() for t in (cache.k_pages, cache.v_pages))
    for b in (0, B - 1):
        s = torch.matmul(q[b].double().transpose(0, 1).contiguous(), K.transpose(1, 2).contiguous()) * D ** -0.5          # [H, N, n + N]
        size = torch.matmul(q[b].double().abs().transpose(0, 1).contiguous(), K.abs().transpose(1, 2).contiguous()).amax(-1) * D ** -0.5
        s = s.masked_fill(torch.ones(N, n + N, dtype=torch.bool, device="cuda").tril(n) == 0, float("-inf"))
        want = s.logsumexp(-1)
        tol = U * (6 * (D / 8) ** 0.5 * size + 8 * want.abs() + 64)
        assert ((lse[b].T.double() - want).abs() <= tol).all(), ((lse[b].T.double() - want).abs() / tol).max()
        p = s.softmax(-1)
        spread = torch.matmul(p, V.abs())
        off = (out[b].transpose(0, 1).double() - torch.matmul(p, V)).abs()
        assert (off <= (2 * tol + 6 * (3 * n / 8 / 3) ** 0.5 * U).unsqueeze(-1) * spread).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,n", [(3, 900), (50, 2100)])
@pytest.mark.parametrize("far", [2.0 ** 13, 2.0 ** 20, -2.0 ** 20])
def test_weights_beside_large_scores(R, dtype, N, n, far):
    """Scores of one large number and a little, exact both, that rise along the keys: their weights go by the little, also between
    tiles and units with maxima of their own. Off by the exponents' two roundings (100 powers of two: 2^-17 each) and sums'."""
    import torch
    rng = np.random.default_rng(N)
    B, H, D, P = 2, 2, 64, 16
    lens = [n, 5, 700]
    width = -(-(n + N) // P)
    pages = sum(-(-(x + N) // P) for x in lens)
    cache = make_cache(R, rng, pages, P, H, D)
    tables = make_tables(rng, pages, P, lens, N, B, width)
    j = np.zeros((pages, P), np.float32)
    for t, x in enumerate(lens):                              # 0 .. 255 along each row's slots
        s = np.arange(x + (N if t < B else 0))
        j[tables[t][s // P], s % P] = s * 256 // (x + N)
    cache.k_pages.zero_()
    cache.k_pages[..., 0] = 1.0
    cache.k_pages[..., 1] = dev(j)[:, :, None].bfloat16()
    q = torch.zeros(B, N, H, D, device="cuda")
    q[..., 0], q[..., 1] = far, 1.0
    q = q.bfloat16() if dtype == "bf16" else q
    got = R.paged_attention(q, cache, R.paged_plan(cache, ints(tables), ints(lens), N, H, B=B, prefix_row=ints([2, 2])))
    want, wlse, _, _ = ref.attend(f64(q), f64(cache.k_pages), f64(cache.v_pages), tables, lens, B, None, [2, 2], None, D ** -0.5, 0.0)
    size = np.abs(f64(cache.v_pages)).max()
    p = 2.0 ** -8 if dtype == "bf16" else 0.0                 # P, and the output
    assert np.abs(f64(got[0]) - want).max() < size * (2 * np.log(2) * 2.0 ** -17 + 2.0 ** -18 + 2 * p)
    assert (np.abs(f64(got[1]) - wlse) < 4 * U * np.abs(wlse) + 2.0 ** -16).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,N,G,shared,tree", [(5, 1, 8, None, False), (3, 8, 4, None, False), (2, 6, 5, None, True), (4, 1, 4, 700, False), (2, 3, 5, 90, False)])
def test_few_query_rows_round_once(R, D, B, N, G, shared, tree):
    """bf16 queries, no more than 32 rows that meet the same slots: P is 2^-17 off, and what shows is the output's rounding."""
    import torch
    rng = np.random.default_rng(D + B)
    H, P = 2, 16
    lens = rng.integers(1, 1500, B).tolist() + ([] if shared is None else [shared])
    width = -(-(max(lens) + N) // P)
    pages = sum(-(-(x + N) // P) for x in lens)
    cache = make_cache(R, rng, pages, P, H, D)
    tables = make_tables(rng, pages, P, lens, N, B, width)
    prefix = None if shared is None else [B] * B
    mask = tree_masks(rng, B, N) if tree else None
    q = queries(rng, B, N, H * G, D, "bf16")
    plan = R.paged_plan(cache, ints(tables), ints(lens), N, H * G, B=B, prefix_row=None if prefix is None else ints(prefix))
    out, _ = R.paged_attention(q, cache, plan, mask=None if mask is None else dev(mask))
    want, _, tol, _ = ref.attend(f64(q), f64(cache.k_pages), f64(cache.v_pages), tables, lens, B, None, prefix, mask, D ** -0.5, 2.0 ** -16)
    assert (np.abs(f64(out) - want) <= tol + 2.0 ** -8 * 1.01 * np.abs(want) + 1e-37).all()
