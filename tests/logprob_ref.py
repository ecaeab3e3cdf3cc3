"""Token log probabilities, entropy and their gradient in float64, and what the float32 arithmetic may be off by."""

import numpy as np

U = 2.0 ** -24                      # half a step of float32, relative
HALF = {"bf16": 2.0 ** -8, "f32": U}
LN2 = np.log(2.0)
TERMS = 160                         # additions a sum goes through: 129 elements of a thread, 6 + 4 levels, 16 more slices


def rows(z, T):
    """One row's y and lse, both less the largest y, p and entropy (None for a row without them)."""
    z = z.astype(np.float64)
    if np.isnan(z).any() or (z == np.inf).any() or not (z > -np.inf).any():
        return None
    y = (z - z.max()) / T
    e = np.exp(y)
    lse = np.log(e.sum())
    p = e / e.sum()
    with np.errstate(invalid="ignore"):
        h = -np.where(p > 0, p * (y - lse), 0.0).sum()
    return y, lse, p, h


def forward(z, tokens, T, top_n):
    """z [R, V], tokens [R, M] -> per row (lp [M], entropy, top ids, top lp), and the tolerances of lp and entropy."""
    out = []
    for r in range(z.shape[0]):
        t = tokens[r]
        if t.size and (t < 0).all():
            out.append(dict(lp=np.zeros(t.size), h=0.0, top=np.full(top_n, -1), top_lp=np.full(top_n, -np.inf),
                            lp_tol=np.zeros(t.size), h_tol=0.0, top_tol=np.zeros(top_n)))
            continue
        d = rows(z[r], T)
        if d is None or (t >= z.shape[1]).any():
            nan = np.full(t.size, np.nan)
            out.append(dict(lp=nan, h=np.nan, top=np.full(top_n, -1), top_lp=np.full(top_n, np.nan), lp_tol=nan * 0,
                            h_tol=0.0, top_tol=np.zeros(top_n)))
            continue
        y, lse, p, h = d
        lp = np.where(t < 0, 0.0, y[np.maximum(t, 0)] - lse)
        order = np.argsort(-z[r].astype(np.float64), kind="stable")[:top_n]
        order = order[z[r][order] > -np.inf]
        top = np.full(top_n, -1)
        top_lp = np.full(top_n, -np.inf)
        top[:order.size] = order
        top_lp[:order.size] = y[order] - lse
        seen = p > 0
        x = (y[seen] - y.max()) / LN2                       # exponents in base two
        q = np.exp2(x)
        first, second = (q * -x).sum() / q.sum(), (q * x * x).sum() / q.sum()
        # an exponent is off by |x| (rounded product) + |x| (rounded constant) half steps, 2^x by two more, S by its additions
        s_tol = U * (2 + TERMS + 2 * LN2 * first)
        lp_tol = s_tol + 4 * U * np.abs(np.where(np.isfinite(lp), lp, 0.0))
        top_tol = s_tol + 4 * U * np.abs(np.where(np.isfinite(top_lp), top_lp, 0.0))
        h_tol = s_tol + LN2 * U * (TERMS * 2 * first + 2 * LN2 * second + 4 * first) + LN2 * first * s_tol + 2 * U * h
        out.append(dict(lp=lp, h=h, top=top, top_lp=top_lp, lp_tol=lp_tol, h_tol=h_tol, top_tol=top_tol))
    return out


def backward(z, tokens, g, gh, T, dtype):
    """-> the gradient [R, V] and its tolerance."""
    R, V = z.shape
    grad, tol = np.zeros((R, V)), np.zeros((R, V))
    for r in range(R):
        t = tokens[r]
        if (t < 0).all():
            continue
        d = rows(z[r], T)
        if d is None or (t >= V).any():
            grad[r] = np.nan
            continue
        y, lse, p, h = d
        live = t >= 0
        G, total = g[r][live].sum(), np.abs(g[r][live]).sum()
        with np.errstate(invalid="ignore"):
            logp = np.where(p > 0, y - lse, 0.0)
        one = np.zeros(V)
        np.add.at(one, t[live], g[r][live])
        mass = np.zeros(V)
        np.add.at(mass, t[live], np.abs(g[r][live]))
        w = gh[r] if gh is not None else 0.0
        grad[r] = (one - p * G - w * p * (logp + h)) / T
        # size of the two parts of p's factor; p is off by its exponent's roundings and those of the sum's logarithm
        size = (total + abs(w) * (np.abs(logp) + h)) / T
        l = abs(lse - y.max())
        p_rel = U * (4 + 4 * (np.abs(logp) + l) + 2 * l + 2 + TERMS + 2 * (h + l))
        h_off = U * (2 * h + 4 * TERMS * (1 + h + l))
        tol[r] = p * size * (p_rel + 80 * U) + p * abs(w) / T * h_off + mass / T * 80 * U + np.abs(grad[r]) * HALF[dtype]
        # the exponential gives no numbers below float32's normal ones: a p under 2^-126 is taken for 0, which is off by less
        # than 2^-126 times p's factor; and a result below the normal numbers is off by less than the smallest of them
        tol[r] += 2.0 ** -126 * (size + 1)
    return grad, tol
