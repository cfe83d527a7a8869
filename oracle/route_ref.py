"""Float64 oracle of routing by scores, a bias and groups (numpy, from the
formulas, one token after another).

    s = softmax(l) or sigmoid(l);  c = s + bias
    groups: the top_groups largest sums of their group_top largest c
    the k largest c of these, lower indexes first among equals
    (without a bias the logits stand for c, but in sums of several)
    w = scale * s / (sum of the chosen s, or 1)
"""
from __future__ import annotations

import numpy as np


def scores(logits, sigmoid):
    """s of float64 logits [E]; 0 where they are not finite."""
    ok = np.isfinite(logits)
    s = np.zeros(len(logits))
    x = logits[ok]
    with np.errstate(over="ignore"):
        if sigmoid:
            s[ok] = 1 / (1 + np.exp(-x))
        elif len(x):
            e = np.exp(x - x.max())
            s[ok] = e / e.sum()
    return s


def log_scores(logits, sigmoid):
    """log s, also where s itself is below float64's range."""
    x = np.where(np.isfinite(logits), logits, -np.inf)
    with np.errstate(over="ignore", invalid="ignore"):
        if sigmoid:
            return np.minimum(x, 0) - np.log1p(np.exp(-np.abs(x)))
        m = x.max()
        # (m + log would lose log where m is large: ulp(3e38) is 4e22)
        return (x - m) - np.log(np.exp(x - m).sum())


def order(c):
    """Indexes from the largest c down, equal ones from the lowest index."""
    return sorted(range(len(c)), key=lambda i: (-c[i], i))


def route(logits, bias, k, sigmoid, groups, top_groups, group_top, renorm,
          scale):
    """(idx, w) of logits [T, E] (float32 values)."""
    T, E = logits.shape
    idx, w = np.empty((T, k), dtype=np.int64), np.zeros((T, k))
    for t in range(T):
        x = logits[t].astype(np.float64)
        s = scores(x, sigmoid)
        c = s.copy()
        ok = np.isfinite(x)
        if bias is not None:
            b = bias.astype(np.float64)
            ok &= np.isfinite(b)
            c = np.where(ok, c + np.where(np.isfinite(b), b, 0.0), 0.0)
        c = np.where(ok, c, -np.inf)
        log = np.where(ok, log_scores(x, sigmoid), -np.inf)
        size = E // groups
        # without a bias experts rank by their logits, and so do groups by
        # that of their first
        by = np.where(ok, x, -np.inf) if bias is None else c
        by_sum = by if group_top == 1 else c
        sums = [sum(sorted(by_sum[g * size:(g + 1) * size])[::-1][:group_top])
                for g in range(groups)]
        kept = set(order(sums)[:top_groups])
        left = [e for e in order(by) if e // size in kept]
        idx[t] = left[:k]
        log = log[idx[t]]
        if renorm and np.isfinite(log.max()):
            log = log - log.max()
            log = log - np.log(np.exp(log).sum())
        w[t] = scale * np.exp(log)
    return idx, w


def route_backward(logits, idx, dw, sigmoid, renorm, scale):
    """dlogits of <dw, w> by the Jacobian, expert by expert."""
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        x = logits[t].astype(np.float64)
        s = scores(x, sigmoid)
        ds = np.zeros(E)
        ch = idx[t]
        if renorm:
            z = s[ch].sum()
            if z > 0:
                mean = (dw[t] * s[ch]).sum() / z
                np.add.at(ds, ch, scale * (dw[t] - mean) / z)
        else:
            np.add.at(ds, ch, scale * dw[t])
        if sigmoid:
            with np.errstate(over="ignore", invalid="ignore"):
                rest = 1 / (1 + np.exp(x))  # 1 - s would round to 0
            out[t] = np.where(np.isfinite(x), ds * s * rest, 0.0)
        else:
            out[t] = s * (ds - (ds * s).sum())
    return out
