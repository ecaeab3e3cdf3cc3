"""Attention and scores at the limits of their forms: caches of 1024 and 1025 slots (one launch or a split key axis),
511 and 512 row tiles of the batch (split or not), rows of whole and broken tiles, lengths at the borders of the split's
chunks.  Compared with the definition in 64 bits, one batch row and head at a time on the GPU; the bounds are kvq_ref's."""

import numpy as np
import pytest

import kvq_ref as ref
from kvq_check import assert_within
from test_gpu_kvq import R, dev, f64, ints, make_cache, queries  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def decode(codes, scales):
    """One head's [S, D] float64 values, on the GPU."""
    import torch
    table = torch.tensor(list(ref.GRID) + [-v for v in ref.GRID], dtype=torch.float64, device=codes.device)
    c = codes.long()
    v = table[torch.stack((c & 15, c >> 4), -1).flatten(-2)]
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def check(R, cache, q, prefix, scale, dtype):
    """Every row of a chain's attention."""
    import torch
    out, lse = R.kvq_attention(q, cache, ints(*prefix), scale=scale)
    B, N, Hq, D = q.shape
    G = Hq // cache.heads
    for b in range(B):
        n = prefix[b] + N
        for h in range(cache.heads):
            K, V = decode(cache.k_codes[b, h, :n], cache.k_scales[b, h, :n]), decode(cache.v_codes[b, h, :n], cache.v_scales[b, h, :n])
            x = q[b, :, h * G:(h + 1) * G].double().reshape(N * G, D)
            s = scale * (x @ K.T)
            last = prefix[b] + torch.arange(N, device=x.device).repeat_interleave(G).view(-1, 1)
            sees = torch.arange(n, device=x.device) <= last
            s = torch.where(sees, s, -torch.inf)
            p = torch.softmax(s, -1)
            wlse = torch.logsumexp(s, -1)
            want, size_v = p @ V, p @ V.abs()
            top = torch.where(sees, scale * (x.abs() @ K.abs().T), 0.0).amax(-1)
            seen = torch.where(sees, s.abs(), 0.0).amax(-1)
            terms = (last.view(-1) + 1) + 4 * ((last.view(-1) + 1) / 32 + 16)
            rel = ((D * top + 8 * seen + 8 + terms) * U).view(-1, 1)
            step = 2.0 ** -8 if dtype == "bf16" else U       # of a probability before it meets V, and of the output
            tol = 2 * rel * size_v + step * size_v + step * want.abs() * 1.01 + 1e-37
            rows = slice(h * G, (h + 1) * G)
            assert_within(f64(out[b, :, rows].reshape(N * G, D)), f64(want), f64(tol))
            assert_within(f64(lse[b, :, rows].reshape(-1)), f64(wlse), f64(rel.view(-1) + 4 * U * wlse.abs()))


@pytest.mark.parametrize("S", [1024, 1025])
@pytest.mark.parametrize("N,G", [(1, 1), (1, 16), (1, 17), (4, 8), (11, 3)])     # 1, 16, 17, 32 and 33 rows a head
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "bf16"), (256, "bf16"), (64, "f32"), (128, "f32"), (256, "f32")])
def test_short_and_split_caches(R, S, N, G, D, dtype):
    rng = np.random.default_rng(S + N + G + D)
    cache = make_cache(R, rng, 2, 1, S, D)
    check(R, cache, queries(rng, 2, N, G, D, dtype), [S - N, 500], D ** -0.5, dtype)


@pytest.mark.parametrize("B,H", [(63, 8), (64, 8), (65, 8), (511, 1), (512, 1)])
def test_one_long_sequence_among_short_ones(R, B, H):
    """On both sides of the batch size from which the key axis is not split."""
    rng = np.random.default_rng(B + H)
    S = 5003
    cache = make_cache(R, rng, B, H, S, 64)
    prefix = rng.integers(0, 40, B)
    prefix[B // 2] = S - 1
    prefix[0] = 0
    check(R, cache, queries(rng, B, 1, 2 * H, 64, "bf16"), prefix.tolist(), 0.125, "bf16")


@pytest.mark.parametrize("n", [1, 31, 32, 33, 127, 128, 129, 255, 256, 257, 511, 513, 65535, 65537, 131071])
@pytest.mark.parametrize("S", [1100, 131080])
def test_lengths_at_the_borders_of_the_split(R, n, S):
    if n > S:
        n = S - n % 64
    rng = np.random.default_rng(n)
    cache = make_cache(R, rng, 2, 1, S, 128)
    check(R, cache, queries(rng, 2, 1, 4, 128, "bf16"), [n - 1, min(n + 300, S - 1)], 128 ** -0.5, "bf16")


@pytest.mark.parametrize("B,H,G,D,N,prefix,dtype", [
    (2, 2, 4, 128, 4, 900, "bf16"), (2, 2, 17, 128, 1, 900, "bf16"), (2, 1, 8, 256, 4, 70, "bf16"), (2, 1, 3, 64, 11, 3, "f32"),
    (2, 1, 1, 128, 256, 300, "bf16"), (2, 1, 1, 128, 257, 300, "bf16"), (1, 1, 4, 128, 64, 1, "bf16"),
    (1, 1, 5, 128, 51, 4000, "bf16"), (3, 1, 1, 256, 129, 77, "bf16"), (1, 2, 2, 64, 512, 0, "bf16"),
    (2, 1, 1, 128, 85, 31, "f32"), (2, 1, 1, 256, 33, 2000, "f32"), (1, 1, 2, 64, 171, 5, "f32")])
def test_scores_of_whole_and_broken_lots(R, B, H, G, D, N, prefix, dtype):
    """Rows that fill the registers or the shared lots exactly, and one more (accepted lengths shrink along the batch)."""
    import torch
    rng = np.random.default_rng(N + D)
    S = prefix + N + 2
    cache = make_cache(R, rng, B, H, S, D)
    q = queries(rng, B, N, H * G, D, dtype, size=0.5)
    lse = torch.from_numpy((4 + rng.standard_normal((B, N, H * G))).astype(np.float32)).cuda()
    alen = [N - 1 - b for b in range(B)]
    scores = torch.from_numpy(rng.random((B, H, S)).astype(np.float32)).cuda()
    before = scores.double()
    pos = torch.full((B, H, S), -3, dtype=torch.int32, device="cuda")
    R.kvq_score(q, lse, cache, ints(*[prefix] * B), ints(*alen), scores, pos, ints(*range(B)))
    slot = torch.arange(S, device="cuda")
    for b in range(B):
        T = alen[b] + 1
        sees = slot <= prefix + torch.arange(T, device="cuda").view(-1, 1)
        fresh = (slot >= prefix) & (slot < prefix + T)
        for h in range(H if T > 0 else 0):
            K = decode(cache.k_codes[b, h], cache.k_scales[b, h])
            w, err = torch.zeros(S, dtype=torch.float64, device="cuda"), torch.zeros(S, dtype=torch.float64, device="cuda")
            for g in range(G):
                x, z = q[b, :T, h * G + g].double(), lse[b, :T, h * G + g].double().view(-1, 1)
                s = (x @ K.T) * D ** -0.5
                e = torch.where(sees, torch.exp(s - z), 0.0)
                w += e.sum(0)
                err += (e * (D * (x.abs() @ K.abs().T) * D ** -0.5 + 8 * s.abs() + 8 * z.abs() + 8)).sum(0) * U
            err += w * (T * G + 24) * U
            want = torch.where(fresh, 0.0, before[b, h]) + w
            assert_within(f64(scores[b, h]), f64(want), f64(err + 2 * U * want.abs()))
        at = torch.where(fresh & (T > 0), b + slot - prefix, -3)
        assert torch.equal(pos[b], at.int().expand(H, S))
    if alen[-1] < 0:
        assert torch.equal(scores[-1].double(), before[-1])
