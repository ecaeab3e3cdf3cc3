"""The four-bit cache's operators from their definitions, in 64 bits (numpy), and how far float32 arithmetic may
be from them.  Shares nothing with the library."""

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def decode(codes, scales):
    """uint8 codes [..., D/2] and scales [..., D/32] -> float64 values [..., D]."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1)
    v = np.where(c & 8, -1.0, 1.0) * GRID[c & 7]
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return v * np.repeat(s, 32, -1)


def quantise(x):
    """float64 rows [..., D] (finite) -> values on the grid [..., D] and scale bytes [..., D/32]."""
    y = x.reshape(*x.shape[:-1], -1, 32)
    top = np.abs(y).max(-1)
    e = np.full(top.shape, -96.0)
    for _ in range(230):                                     # the smallest exponent that holds the block
        e = np.where(top > 7.0 * np.exp2(e), e + 1, e)
    step = np.exp2(e)[..., None]
    a = np.abs(y) / step
    d = np.abs(a[..., None] - GRID)
    best = d.min(-1, keepdims=True)
    tied = d == best                                         # one code, or two neighbours: then the even one
    code = np.where(tied.sum(-1) == 2, (tied * (np.arange(8) % 2 == 0)).argmax(-1), tied.argmax(-1))
    v = np.copysign(GRID[code], y) * step
    return v.reshape(x.shape), np.where(top == 0, 0, e + 127).astype(np.uint8)


def visible(pre, cnt, N, S, mask):
    """[N, S] of one batch row; no token sees anything where the row is an error row."""
    see = np.zeros((N, S), bool)
    if pre < 0 or cnt < 0 or cnt > N or pre + cnt > S:
        return see
    for n in range(cnt):
        see[n, :pre] = True
        see[n, pre:pre + cnt] = (np.arange(cnt) <= n) if mask is None else mask[n, :cnt] != 0
    return see


def attend(q, K, V, prefix, counts, mask, scale):
    """q [B, N, Hq, D], K, V [B, H, S, D] float64, mask [B, N, N] or None -> (out, lse, tolerances of both).

    The tolerances count roundings of float32 arithmetic, u = 2^-24 each: a score of D products is off by at most
    D*u*sum|q k| (scaled), its exponent by 4*u*|s| more, exp2 and log2 by 4*u, a sum of n terms with r rescalings by
    (n + 4r)*u; r is at most one a step of 32 keys and a few joins.  `p_round` is the relative rounding of a
    probability before it meets V, `o_round` that of the output.
    """
    B, N, Hq, D = q.shape
    H, S = K.shape[1:3]
    G = Hq // H
    out, lse = np.zeros((B, N, Hq, D)), np.full((B, N, Hq), -np.inf)
    tol_p, tol_l = np.zeros((B, N, Hq, D)), np.zeros((B, N, Hq))
    u = 2.0 ** -24
    for b in range(B):
        see = visible(prefix[b], counts[b], N, S, None if mask is None else mask[b])
        for hq in range(Hq):
            k, v = K[b, hq // G], V[b, hq // G]
            for n in range(N):
                at = np.flatnonzero(see[n])
                if not at.size:
                    continue
                x = q[b, n, hq]
                s = scale * (k[at] @ x)
                m = s.max()
                p = np.exp(s - m)
                l = p.sum()
                out[b, n, hq], lse[b, n, hq] = p @ v[at] / l, m + np.log(l)
                size = scale * (np.abs(k[at]) @ np.abs(x)).max()
                terms = at.size + 4 * (at.size / 32 + 16)
                rel = (D * size + 8 * np.abs(s).max() + 8 + terms) * u
                # o = sum p v / sum p: the relative error of p enters both
                tol_p[b, n, hq] = 2 * rel * (p @ np.abs(v[at])) / l
                tol_l[b, n, hq] = rel + 4 * u * abs(lse[b, n, hq])
    return out, lse, tol_p, tol_l


def attend_abs(q, K, V, prefix, counts, mask, scale):
    """sum p |v| / sum p of every output, what a relative rounding of p may move it by."""
    return attend(q, K, np.abs(V), prefix, counts, mask, scale)[0]


def score(q, lse, K, prefix, path, accept_len, scale, scores, positions, seen):
    """New (scores, positions) float64 / int, and the tolerance of the scores."""
    B, N, Hq, D = q.shape
    H, S = K.shape[1:3]
    G = Hq // H
    scores, positions = scores.astype(np.float64).copy(), positions.copy()
    tol = np.zeros_like(scores)
    u = 2.0 ** -24
    for b in range(B):
        d, pre = int(accept_len[b]), int(prefix[b])
        width = N if path is None else path.shape[1]
        p = np.arange(max(d, -1) + 1) if path is None else path[b, :max(d, -1) + 1]
        if d < 0 or d >= N or d >= width or pre < 0 or pre + d + 1 > S:
            continue
        if path is not None and (p[0] != 0 or (np.diff(p) <= 0).any() or (p >= N).any()):
            continue
        for h in range(H):
            w, err = np.zeros(S), np.zeros(S)
            for t in range(d + 1):
                for g in range(G):
                    x, z = q[b, p[t], h * G + g], float(lse[b, p[t], h * G + g])
                    if z == -np.inf:
                        continue
                    k = K[b, h, :pre + t + 1]
                    s = scale * (k @ x)
                    e = np.exp(s - z)
                    w[:pre + t + 1] += e
                    err[:pre + t + 1] += e * (D * scale * (np.abs(k) @ np.abs(x)) + 8 * np.abs(s) + 8 * abs(z) + 8) * u
            err += w * (d + 1) * G * u + w * 16 * u
            scores[b, h, pre:pre + d + 1] = 0
            scores[b, h] += w
            tol[b, h] = err + 2 * u * np.abs(scores[b, h])
            positions[b, h, pre:pre + d + 1] = seen[b] + np.arange(d + 1)
    return scores, positions, tol


def evict(scores, positions, lengths, seen, keep, sink, recent):
    """(new lengths [B], source [B, H, keep]) by the definition, one slot after another."""
    B, H, S = scores.shape
    new_len, source = np.full(B, -1, np.int32), np.full((B, H, keep), -1, np.int32)
    for b in range(B):
        n = int(lengths[b])
        if n < 0 or n > S:
            continue
        m = min(n, keep)
        new_len[b] = m
        for h in range(H):
            def order(s):
                p, x = int(positions[b, h, s]), float(scores[b, h, s])
                if p < sink or p >= int(seen[b]) - recent:
                    return (0, 0.0, s)
                return (2, 0.0, s) if np.isnan(x) else (1, -x, s)
            kept = sorted(sorted(range(n), key=order)[:m])
            movers = iter([s for s in kept if s >= m])
            there = set(kept)
            source[b, h, :m] = [s if s in there else next(movers) for s in range(m)]
    return new_len, source


def move(array, source, new_len):
    """array [B, H, S, ...] with the plan's rows moved."""
    out = array.copy()
    for b in range(array.shape[0]):
        if new_len[b] > 0:
            for h in range(array.shape[1]):
                out[b, h, :new_len[b]] = array[b, h, source[b, h, :new_len[b]]]
    return out
