"""The token losses from their definitions in 64 bits, one row after another
(numpy), with the gradients' formulas written out."""
import numpy as np


def softmax_row(x, T):
    """(z, log p, p, entropy) of one row, p log p = 0 where p = 0."""
    z = x / T
    m = z.max()
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        lse = m + np.log(np.exp(z - m).sum())
        lp = z - lse
        p = np.exp(lp)
        h = -np.where(p > 0, p * np.where(p > 0, lp, 0.0), p).sum()
    return z, lp, p, h


def log_probs(x, tokens, T, ignore, g_lp=None, g_h=None):
    rows, V = x.shape
    lp, h, dx = np.zeros(rows), np.zeros(rows), np.zeros((rows, V))
    for r, t in enumerate(tokens):
        if t == ignore or not 0 <= t < V:
            continue
        _, l, p, h[r] = softmax_row(x[r], T)
        lp[r] = l[t]
        if g_lp is not None:
            dx[r] = -p * g_lp[r]
            dx[r, t] += g_lp[r]
        if g_h is not None:
            dx[r] -= g_h[r] * p * (np.where(p > 0, l, 0.0) + h[r])
    return lp, h, dx / T


def policy(x, tokens, adv, old, ref, weight, lo, hi, kl_coef, ent_coef, T, ignore, scale, reduction):
    rows, V = x.shape
    lp, h, _ = log_probs(x, tokens, T, ignore)
    loss, slope, kl, clipped = np.zeros(rows), np.zeros(rows), np.zeros(rows), np.zeros(rows, bool)
    keep = np.array([t != ignore and 0 <= t < V for t in tokens], bool)
    w = np.ones(rows) if weight is None else weight
    for r in np.nonzero(keep)[0]:
        ratio = 1.0 if old is None else np.exp(lp[r] - old[r])
        a = adv[r]
        cut = min(max(ratio, 1 - lo), 1 + hi)
        loss[r] = -min(ratio * a, cut * a)
        clipped[r] = cut * a < ratio * a
        slope[r] = 0.0 if clipped[r] else -ratio * a
        if ref is not None:
            g = ref[r] - lp[r]
            kl[r] = np.expm1(g) - g
            loss[r] += kl_coef * kl[r]
            slope[r] -= kl_coef * np.expm1(g)
        loss[r] -= ent_coef * h[r]
    D = w[keep].sum() if reduction == "mean" else 1.0
    f = np.where(keep, scale * w / D if keep.any() else 0.0, 0.0)
    _, _, dx = log_probs(x, tokens, T, ignore, slope * f, -ent_coef * f * np.ones(rows))
    per = loss * f
    with np.errstate(invalid="ignore"):
        total = per if reduction == "none" else per.sum() if keep.any() or reduction == "sum" else np.nan
    return total, lp, h, kl, clipped, dx, (slope * f, -ent_coef * f)


def distill(x, teacher, index, lse, weight, T, scale, reduction):
    rows, V = x.shape
    loss, dx = np.zeros(rows), np.zeros((rows, V))
    keep = np.array([0 <= i[0] < V for i in index], bool)
    w = np.ones(rows) if weight is None else weight
    D = w[keep].sum() if reduction == "mean" else 1.0
    for r in np.nonzero(keep)[0]:
        _, lp, p, _ = softmax_row(x[r], T)
        ok = (index[r] >= 0) & (index[r] < V)
        j, v = index[r][ok], teacher[r][ok] / T
        if lse is None:
            lq = v - v.max()
            lq = lq - np.log(np.exp(lq).sum())
        else:
            lq = v - lse[r]
        q = np.exp(lq)
        some = q > 0
        with np.errstate(divide="ignore"):
            loss[r] = (q[some] * (lq[some] - lp[j][some])).sum()
        onto = np.zeros(V)
        np.add.at(onto, j, q)
        g = q.sum() * p - onto
        if lse is not None:
            rest = max(0.0, 1.0 - q.sum())
            others = np.ones(V, bool)
            others[j] = False
            left = p[others].sum()
            g = g + rest * p
            if left > 0:
                if rest > 0:
                    loss[r] += rest * (np.log(rest) - np.log(left))
                g = g - np.where(others, rest * p / left, 0.0)
        f = scale * w[r] / D
        loss[r] *= f
        dx[r] = g * f / T
    total = loss if reduction == "none" else loss.sum() if keep.any() or reduction == "sum" else np.nan
    return total, dx, keep


def preference(x, tokens, bounds, ref, kind, beta, margin, smoothing, average, ignore, scale, reduction):
    """bounds: (first row, last row + 1) of each of the 2 pairs sequences."""
    rows, V = x.shape
    pairs = len(bounds) // 2
    lp, _, _ = log_probs(x, tokens, 1.0, ignore)
    keep = np.array([t != ignore and 0 <= t < V for t in tokens], bool)
    n = np.array([max(1, keep[a:b].sum()) if average else 1 for a, b in bounds], float)
    s = np.array([lp[a:b][keep[a:b]].sum() for a, b in bounds]) / n
    ref = np.zeros(2 * pairs) if ref is None else ref
    d = (s[:pairs] - s[pairs:]) - (ref[:pairs] - ref[pairs:])
    if kind == "ipo":
        loss, slope = (d - 0.5 / beta) ** 2, 2 * (d - 0.5 / beta)
    else:
        u = beta * d - margin
        if kind == "hinge":
            loss, slope = np.maximum(0.0, 1.0 - u), np.where(u < 1, -beta, 0.0)
        else:
            loss = (1 - smoothing) * np.logaddexp(0, -u) + smoothing * np.logaddexp(0, u)
            slope = beta * (1 / (1 + np.exp(-u)) - (1 - smoothing))
    f = scale / (pairs if reduction == "mean" else 1)
    ds = np.concatenate([slope, -slope]) * f / n
    g = np.zeros(rows)
    for (a, b), v in zip(bounds, ds):
        g[a:b] = v
    g = np.where(keep, g, 0.0)
    _, _, dx = log_probs(x, tokens, 1.0, ignore, g)
    loss = loss * f
    total = loss if reduction == "none" else loss.sum() if pairs or reduction == "sum" else np.nan
    return total, s, dx, g
