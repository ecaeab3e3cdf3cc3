"""The paged cache by its definitions: pages of a step, one row after another, and attention in float64."""

import numpy as np

U = 2.0 ** -24


def page_step(tables, held, ring, state, lengths, counts, N, P):
    """-> granted, slots, and the new tables, held, ring, state."""
    tables, held, ring = tables.copy(), held.copy(), ring.copy()
    T, width = tables.shape
    pages = ring.size
    head, free = int(state[0]), int(state[1])
    granted, slots = np.full(T, -1, np.int32), np.full((T, N), -1, np.int32)
    if not (0 <= head < pages and 0 <= free <= pages):
        return granted, slots, tables, held, ring, np.array(state, np.int32)
    taken, asked, given = 0, 0, []
    for t in range(T):
        n, have = int(lengths[t]), int(held[t])
        c = N if counts is None else int(counts[t])
        if n < 0:
            c, need = 0, 0
        else:
            need = -(-(n + c) // P)
        if not 0 <= have <= min(width, pages) or not 0 <= c <= N or need > width:
            continue
        grow = max(need - have, 0)
        asked += grow
        if grow and asked > free:
            continue
        for j in range(have, need):
            tables[t, j] = ring[(head + taken) % pages]
            taken += 1
        given += [int(tables[t, j]) for j in range(need, have)]
        held[t], granted[t] = need, c
        for i in range(c):
            page = int(tables[t, (n + i) // P])
            if 0 <= page < pages:
                slots[t, i] = page * P + (n + i) % P
    for i, page in enumerate(given):
        ring[(head + free + i) % pages] = page
    return granted, slots, tables, held, ring, np.array([(head + taken) % pages, free - taken + len(given)], np.int32)


def attend(q, K, V, tables, lengths, B, counts, prefix_row, mask, scale, p_round):
    """K, V [pages, P, H, D], q [B, N, Hq, D] float64 -> out, lse and their tolerances (without the output's rounding).

    p_round: how far a probability is rounded, relative, before it meets V."""
    _, N, Hq, D = q.shape
    pages, P, H = K.shape[:3]
    T, width = tables.shape
    G = Hq // H
    out, lse = np.zeros(q.shape), np.full((B, N, Hq), -np.inf)
    tol, ltol = np.zeros(q.shape), np.zeros((B, N, Hq))

    def slots(row, n):
        s = np.arange(n)
        return tables[row][s // P], s % P

    for b in range(B):
        n, c = int(lengths[b]), N if counts is None else int(counts[b])
        pr = -1 if prefix_row is None else int(prefix_row[b])
        if n < 0 or not 0 <= c <= N or n + c > width * P or pr >= T:
            continue
        shared = int(lengths[pr]) if pr >= 0 else 0
        if not 0 <= shared <= width * P:
            continue
        pg, at = (np.concatenate(x) for x in zip(slots(pr, shared), slots(b, n + c)))
        sees = np.zeros((c, shared + n + c), bool)
        sees[:, :shared + n] = True
        sees[:, shared + n:] = np.tril(np.ones((c, c), bool)) if mask is None else mask[b][:c, :c] != 0
        for h in range(H):
            k, v = K[pg, at, h], V[pg, at, h]
            for g in range(G):
                x = q[b, :c, h * G + g]
                for t in range(c):                            # rows one by one where slots are hidden, to leave what they hold
                    live = np.flatnonzero(sees[t])
                    if not live.size:
                        continue
                    s = scale * (k[live] @ x[t])
                    m = s.max()
                    p = np.exp(s - m)
                    l = p.sum()
                    out[b, t, h * G + g], lse[b, t, h * G + g] = p @ v[live] / l, m + np.log(l)
                    size = scale * (np.abs(k[live]) @ np.abs(x[t])).max()
                    # products and sums of a score, its exponential; additions of a sum over keys, the joins
                    rel = (D * size + 8 * np.abs(s).max() + 8 + live.size + 4 * (live.size / 32 + 16)) * U
                    tol[b, t, h * G + g] = (2 * rel + p_round) * (p @ np.abs(v[live])) / l
                    ltol[b, t, h * G + g] = rel + 4 * U * abs(lse[b, t, h * G + g])
    return out, lse, tol, ltol
