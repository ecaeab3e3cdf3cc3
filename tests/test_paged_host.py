"""Arguments that the paged cache's calls refuse, on the host (no kernel is launched), and its reference by hand."""

import ctypes

import numpy as np
import pytest

import paged_ref as ref

EINVAL, EWORKSPACE, EUNSUPPORTED = -1, -2, -4
FAKE = 0x7F0000000000  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def L():
    import rejection_sampling_verify_10_amd as R
    return R.lib()


def cache(**kw):
    from rejection_sampling_verify_10_amd.paged import _CacheArgs
    H, D, P = kw.get("heads", 4), kw.get("head_dim", 128), kw.get("page_size", 32)
    a = dict(k=FAKE, v=FAKE, pages=100, page_size=P, heads=H, head_dim=D, page_stride=P * H * D, slot_stride=H * D, head_stride=D)
    a.update(kw)
    return _CacheArgs(**a)


def rows(data=FAKE, batch=4096, pos=1024, head=128):
    from rejection_sampling_verify_10_amd.kvq import _Rows
    return _Rows(data, batch, pos, head)


def ptr(s):
    return None if s is None else ctypes.byref(s)


def step(L, **kw):
    a = dict(tables=FAKE, stride=20, T=4, width=20, P=16, pages=50, held=FAKE, state=FAKE, ring=FAKE, lengths=FAKE, counts=None,
             N=3, oh=FAKE, os=FAKE, og=FAKE, sl=FAKE, ws=FAKE, wsb=256, stream=None)
    a.update(kw)
    return L.spec_page_step(*a.values())


def append(L, **kw):
    a = dict(c=cache(), k=rows(), v=rows(), dtype=1, B=2, N=3, source=3, slots=FAKE, stride=3, path=None, ps=0, alen=None, stream=None)
    a.update(kw)
    for n in ("c", "k", "v"):
        a[n] = ptr(a[n])
    return L.spec_paged_append(*a.values())


def plan(L, **kw):
    a = dict(B=2, N=3, Hq=8, H=4, D=128, T=3, width=20, P=32, lengths=FAKE, counts=None, prefix=FAKE, plan=FAKE, bytes=1 << 30, stream=None)
    a.update(kw)
    return L.spec_paged_plan(*a.values())


def attend(L, **kw):
    a = dict(q=rows(), dtype=1, B=2, N=3, Hq=8, c=cache(), tables=FAKE, stride=20, width=20, plan=FAKE, pbytes=1 << 30, pre=1,
             mask=None, mb=0, scale=0.1, out=FAKE, lse=None, ws=FAKE, wsb=0, stream=None)
    a.update(kw)
    for n in ("q", "c"):
        a[n] = ptr(a[n])
    return L.spec_paged_attention(*a.values())


@pytest.mark.parametrize("bad,code", [
    (dict(tables=None), EINVAL), (dict(T=0), EINVAL), (dict(width=0), EINVAL), (dict(stride=19), EINVAL), (dict(P=8), EINVAL),
    (dict(P=48), EINVAL), (dict(P=2048), EINVAL), (dict(pages=0), EINVAL), (dict(held=None), EINVAL), (dict(state=None), EINVAL),
    (dict(ring=None), EINVAL), (dict(lengths=None), EINVAL), (dict(counts=FAKE + 2), EINVAL), (dict(N=0), EINVAL),
    (dict(oh=None), EINVAL), (dict(os=None), EINVAL), (dict(og=None), EINVAL), (dict(sl=None), EINVAL), (dict(sl=FAKE + 1), EINVAL),
    (dict(T=65537), EUNSUPPORTED), (dict(N=65537), EUNSUPPORTED), (dict(pages=(1 << 26) + 1), EUNSUPPORTED),
    (dict(width=(1 << 26) + 1, stride=1 << 27), EUNSUPPORTED), (dict(ws=None), EWORKSPACE), (dict(ws=FAKE + 64), EWORKSPACE),
    (dict(wsb=255), EWORKSPACE),
])
def test_page_step_refuses(L, bad, code):
    assert step(L, **bad) == code


BAD_CACHES = [
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(k=FAKE + 8), EINVAL), (dict(pages=0), EINVAL), (dict(heads=0), EINVAL),
    (dict(head_dim=0), EINVAL), (dict(page_size=15), EINVAL), (dict(page_size=24), EINVAL), (dict(page_size=2048), EINVAL),
    (dict(slot_stride=120), EINVAL), (dict(slot_stride=0), EINVAL), (dict(slot_stride=132), EINVAL), (dict(page_stride=64), EINVAL),
    (dict(page_stride=-128), EINVAL), (dict(head_stride=0), EINVAL), (dict(head_stride=124), EINVAL),
    (dict(head_dim=96, head_stride=96), EUNSUPPORTED), (dict(pages=(1 << 25) + 1), EUNSUPPORTED), (dict(slot_stride=(1 << 20) + 8), EUNSUPPORTED),
    (dict(heads=65536), EUNSUPPORTED), (dict(page_stride=1 << 41), EUNSUPPORTED),
]


@pytest.mark.parametrize("bad,code", BAD_CACHES)
def test_caches_refused(L, bad, code):
    assert append(L, c=cache(**bad)) == code
    if "heads" not in bad:
        assert attend(L, c=cache(**bad)) == code


@pytest.mark.parametrize("bad,code", [
    (dict(c=None), EINVAL), (dict(k=None), EINVAL), (dict(v=rows(FAKE + 8)), EINVAL), (dict(k=rows(batch=4)), EINVAL), (dict(dtype=2), EINVAL),
    (dict(B=0), EINVAL), (dict(N=0), EINVAL), (dict(source=2), EINVAL), (dict(source=0), EINVAL), (dict(slots=None), EINVAL),
    (dict(slots=FAKE + 2), EINVAL), (dict(stride=2), EINVAL), (dict(path=FAKE, ps=3), EINVAL), (dict(path=FAKE, ps=2, alen=FAKE), EINVAL),
    (dict(path=FAKE + 1, ps=3, alen=FAKE), EINVAL), (dict(N=65537, source=65537, stride=65537), EUNSUPPORTED),
    (dict(B=60000, N=60000, source=60000, stride=60000), EUNSUPPORTED),
])
def test_append_refuses(L, bad, code):
    assert append(L, **bad) == code


@pytest.mark.parametrize("bad,code", [
    (dict(B=0), EINVAL), (dict(N=0), EINVAL), (dict(Hq=7), EINVAL), (dict(Hq=0), EINVAL), (dict(H=0), EINVAL), (dict(T=1), EINVAL),
    (dict(width=0), EINVAL), (dict(P=8), EINVAL), (dict(P=33), EINVAL), (dict(lengths=None), EINVAL), (dict(lengths=FAKE + 2), EINVAL),
    (dict(counts=FAKE + 1), EINVAL), (dict(prefix=FAKE + 2), EINVAL), (dict(N=65537), EUNSUPPORTED), (dict(width=1 << 26), EUNSUPPORTED),
    (dict(D=96), EUNSUPPORTED), (dict(B=1 << 20, T=1 << 20, N=1 << 16), EUNSUPPORTED), (dict(plan=None), EWORKSPACE), (dict(plan=FAKE + 4), EWORKSPACE),
    (dict(bytes=100), EWORKSPACE),
])
def test_plan_refuses(L, bad, code):
    assert plan(L, **bad) == code


@pytest.mark.parametrize("bad,code", [
    (dict(q=None), EINVAL), (dict(q=rows(FAKE + 8)), EINVAL), (dict(q=rows(pos=4)), EINVAL), (dict(dtype=2), EINVAL), (dict(dtype=-1), EINVAL),
    (dict(B=0), EINVAL), (dict(N=0), EINVAL), (dict(Hq=6), EINVAL), (dict(tables=None), EINVAL), (dict(tables=FAKE + 2), EINVAL),
    (dict(stride=19), EINVAL), (dict(width=0), EINVAL), (dict(out=None), EINVAL), (dict(out=FAKE + 8), EINVAL), (dict(lse=FAKE + 2), EINVAL),
    (dict(mask=FAKE, mb=-1), EINVAL), (dict(scale=0.0), EINVAL), (dict(scale=-1.0), EINVAL), (dict(scale=float("nan")), EINVAL),
    (dict(scale=3e38), EINVAL), (dict(mask=FAKE, N=65), EUNSUPPORTED), (dict(width=1 << 26, stride=1 << 26), EUNSUPPORTED),
    (dict(plan=None), EWORKSPACE), (dict(pbytes=64), EWORKSPACE), (dict(wsb=16), EWORKSPACE),
])
def test_attention_refuses(L, bad, code):
    assert attend(L, **bad) == code


def test_sizes_of_plans(L):
    assert L.spec_paged_plan_bytes(0, 1, 8, 4, 64, 0) == 0 and L.spec_paged_plan_bytes(2, 1, 9, 4, 64, 0) == 0
    assert 0 < L.spec_paged_plan_bytes(2, 1, 8, 4, 64, 0) <= L.spec_paged_plan_bytes(2, 1, 8, 4, 64, 1)
    assert L.spec_paged_plan_bytes(2, 1, 8, 4, 96, 0) == 0
    assert L.spec_paged_attention_workspace_bytes(2, 1, 8, 4, 96, 1) == 0
    # many rows of their own and no prefix: nothing is split, nothing joined
    assert L.spec_paged_attention_workspace_bytes(4096, 1, 8, 4, 128, 0) == 0


def test_reference_steps_by_hand():
    tables, held = np.full((2, 3), -1, np.int32), np.array([1, 0], np.int32)
    tables[0, 0] = 4
    ring = np.array([3, 9, 9, 0, 1], np.int32)                # three free, across the ring's end
    granted, slots, t, h, r, s = ref.page_step(tables, held, ring, [3, 3], [14, 0], [4, 20], 20, 16)
    assert granted.tolist() == [4, 20] and h.tolist() == [2, 2] and s.tolist() == [1, 0]
    assert t.tolist() == [[4, 0, -1], [1, 3, -1]]
    assert slots[0, :5].tolist() == [78, 79, 0, 1, -1] and slots[1, 15:20].tolist() == [31, 48, 49, 50, 51]
    granted, slots, t, h, r, s = ref.page_step(t, h, r, s, [-1, 5], None, 4, 16)
    assert granted.tolist() == [0, 4] and h.tolist() == [0, 1] and s.tolist() == [1, 3]
    assert r.tolist() == [3, 4, 0, 3, 1]                      # 4 and 0 of the first row, then 3 of the second


def test_reference_attention_by_hand():
    rng = np.random.default_rng(0)
    K, V = rng.standard_normal((3, 16, 1, 64)), rng.standard_normal((3, 16, 1, 64))
    q = rng.standard_normal((1, 2, 1, 64))
    out, lse, _, _ = ref.attend(q, K, V, np.array([[2], [0]]), [1, 2], 1, None, [1], None, 0.1, 0.0)
    k, v = np.concatenate((K[0, :2], K[2, :3]))[:, 0], np.concatenate((V[0, :2], V[2, :3]))[:, 0]
    for n in range(2):
        p = np.exp(0.1 * k[:4 + n] @ q[0, n, 0])
        assert np.allclose(out[0, n, 0], p @ v[:4 + n] / p.sum()) and np.isclose(lse[0, n, 0], np.log(p.sum()))


@pytest.mark.parametrize("B,N,Hq,H,D,most", [(2048, 1, 64, 8, 128, 600e6), (4, 1, 32, 8, 128, 10e6), (4, 1, 8, 8, 128, 10e6), (32, 8, 32, 8, 128, 62e6)])
def test_workspaces_hold_what_plans_need(L, B, N, Hq, H, D, most):
    """Parts of tiles as full as a batch's runs can make them, and of the split: not a tile of 128 rows for each batch row."""
    assert 0 < L.spec_paged_attention_workspace_bytes(B, N, Hq, H, D, 1) < most


def test_rows_of_runs_filled_up():
    """The bound of paged_plan_sizes on the query rows of runs, each filled up to tiles (32 for up to 32 rows, else 128), against
    every partition of a batch into runs, by dynamic programming; and of their tiles."""
    for M in (*range(1, 40), 63, 64, 100, 127, 128, 129, 135, 300):
        most, tiles = [0], [0]
        fewest = 32 // M + 1 if M <= 32 else 1
        for B in range(1, 30):
            pad = [32 if k * M <= 32 else -(-k * M // 128) * 128 for k in range(B + 1)]
            most.append(max(pad[k] + most[B - k] for k in range(1, B + 1)))
            tiles.append(max(max(-(-k * M // 128), 1) + tiles[B - k] for k in range(1, B + 1)))
            own = B * (1 if M <= 32 else -(-M // 128))
            bound = own * (32 if M <= 32 else 128) if M > 32 or B * M <= 32 else max(32 * B, -(-B * 128 // fewest))
            assert most[B] <= bound and tiles[B] <= own, (B, M)
