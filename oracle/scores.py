"""Plain CPU reference of routing from logits (NumPy, fp64): selection, its
gradient and the balance loss.  Test infrastructure: it shares no code with the
HIP path."""
from __future__ import annotations

import numpy as np

F32_MAX = float(np.finfo(np.float32).max)


def _logits(z):
    z = np.array(z, dtype=np.float64)
    z[z == np.inf] = F32_MAX
    return z


def log_scores(z, score):
    """Logarithms of the scores of logits z [T, E]; -inf where z is."""
    z = _logits(z)
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return np.where(z == -np.inf, -np.inf,
                            np.minimum(z, 0) - np.log1p(np.exp(-np.abs(z))))
        top = np.where(np.isnan(z), -np.inf, z).max(1, keepdims=True)
        top = np.where(top > -np.inf, top, 0.0)
        return np.where(z == -np.inf, -np.inf,
                        z - top - np.log(np.exp(z - top).sum(1, keepdims=True)))


def scores(z, score):
    return np.exp(log_scores(z, score))


def select(z, *, score="softmax", sel_bias=None, num_groups=1, topk_groups=1, group_best=2, topk=8,
           renormalize=True):
    """(ids [T, k], weights [T, k]), token by token by the rule as it is written."""
    z = _logits(z)
    T, E = z.shape
    nan_rows = np.isnan(z).any(1)
    z = np.where(np.isnan(z), -np.inf, z)
    logs = log_scores(z, score)
    ids = np.full((T, topk), -1, dtype=np.int32)
    w = np.zeros((T, topk))
    size = E // num_groups
    for t in range(T):
        s = np.exp(logs[t])
        v = s if sel_bias is None else s + np.asarray(sel_bias, np.float64)
        order = z[t] if sel_bias is None else v
        some = (z[t] > -np.inf) & (v > -np.inf)  # False for a NaN
        totals = []
        for g in range(num_groups):
            mine = sorted((v[e] for e in range(g * size, (g + 1) * size) if some[e]), reverse=True)
            totals.append(sum(mine[:group_best]) if mine else -np.inf)
        kept = sorted(range(num_groups), key=lambda g: (-totals[g], g))[:topk_groups]
        best = sorted((e for e in range(E) if some[e] and e // size in kept),
                      key=lambda e: (-order[e], e))[:topk]
        if best:
            ids[t, :len(best)] = best
            l = logs[t][best]
            if renormalize:
                r = np.exp(l - l.max())
                w[t, :len(best)] = r / r.sum()
            else:
                w[t, :len(best)] = np.exp(l)
        if nan_rows[t]:
            w[t] = np.nan
    return ids, w


def _normalized(z, score):
    """Scores over their sum, by logarithms: rows of scores below 2^-1074 too."""
    l = log_scores(z, score)
    top = l.max(1, keepdims=True)
    r = np.exp(l - np.where(top > -np.inf, top, 0.0))
    total = r.sum(1, keepdims=True)
    return np.divide(r, total, out=np.zeros_like(r), where=~(total == 0))


def select_backward(z, ids, grad_w, *, score="softmax", renormalize=True, load=None, grad_loss=1.0):
    """Gradient [T, E], and the sum of the magnitudes of the terms that make it
    up (what a rounding in each of them is relative to)."""
    z = _logits(z)
    T, E = z.shape
    ids = np.asarray(ids)
    logs = log_scores(z, score)
    s = np.exp(logs)
    one_minus = np.exp(log_scores(-np.where(z == -np.inf, -1e300, z), "sigmoid")) \
        if score == "sigmoid" else np.ones_like(z)
    out, size = np.zeros((T, E)), np.zeros((T, E))
    q = _normalized(z, score)
    for t in range(T):
        slots = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        if not slots:
            continue
        e = ids[t, slots]
        if grad_w is not None:
            g = np.asarray(grad_w, np.float64)[t, slots]
            l = logs[t][e]
            if renormalize:
                w = np.exp(l - l.max()) if l.max() > -np.inf else np.zeros(len(e))
                w = w / w.sum() if w.sum() > 0 else w
                dot, mag = (g * w).sum(), np.abs(g * w).sum()
                for j, c in enumerate(e):
                    out[t, c] += w[j] * (g[j] - dot) * one_minus[t, c]
                    size[t, c] += w[j] * (abs(g[j]) + mag) * one_minus[t, c]
            else:
                each, mags = np.zeros(E), np.zeros(E)
                for j, c in enumerate(e):
                    each[c] += g[j]
                    mags[c] += abs(g[j])
                dot = (g * s[t][e]).sum() if score == "softmax" else 0.0
                mag = np.abs(g * s[t][e]).sum() if score == "softmax" else 0.0
                out[t] += s[t] * (each - dot) * one_minus[t]
                size[t] += s[t] * (mags + mag) * one_minus[t]
        if load is not None:
            c = np.asarray(load, np.float64)
            out[t] += grad_loss * q[t] * (c - (q[t] * c).sum()) * one_minus[t]
            size[t] += abs(grad_loss) * q[t] * (np.abs(c) + np.abs(q[t] * c).sum()) * one_minus[t]
        if np.isnan(z[t]).any():
            out[t] = np.nan
    return out, size


def balance_loss(z, ids, *, score="softmax", coef=1e-2):
    """(loss, load [E])."""
    z = _logits(z)
    ids = np.asarray(ids)
    T, E = z.shape
    on = (ids >= 0) & (ids < E)
    rows = on.any(1)
    count = np.bincount(ids[on], minlength=E).astype(np.float64)
    if not rows.any():
        return 0.0, np.zeros(E)
    f = E * count / count.sum()
    P = _normalized(z[rows], score).sum(0) / rows.sum()
    return coef * (f * P).sum(), coef * f / rows.sum()
