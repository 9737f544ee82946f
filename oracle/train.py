"""Plain CPU reference of the training calls (NumPy, fp64): rows sorted by
expert and back with their gradients, the router's gradient, AdamW.

Pair p = t*k + j is slot j of token t; perm_dst[p] is its row in the sorted
order, and anything outside [0, T*k) drops the pair.  Test infrastructure: it
shares no code with the HIP path."""
from __future__ import annotations

import numpy as np

from . import e4m3_decode


def _slots(perm_dst, T, k):
    d = np.asarray(perm_dst).reshape(T, k).astype(np.int64)
    return d, (d >= 0) & (d < T * k)


def dispatch(x, perm_dst, k, w=None, out=None):
    """out[perm_dst[p]] = w[p] * x[t]; other rows of out stay."""
    x = np.asarray(x, dtype=np.float64)
    T = x.shape[0]
    d, on = _slots(perm_dst, T, k)
    out = np.zeros((T * k, x.shape[1])) if out is None else np.array(out, dtype=np.float64)
    for j in range(k):
        t = np.nonzero(on[:, j])[0]
        out[d[t, j]] = x[t] if w is None else np.asarray(w, np.float64)[t, j, None] * x[t]
    return out


def combine(y, perm_dst, w, scale):
    """out[t] = scale * sum_j w[p] * y[perm_dst[p]]."""
    y, w = np.asarray(y, np.float64), np.asarray(w, np.float64)
    T, k = w.shape
    d, on = _slots(perm_dst, T, k)
    out = np.zeros((T, y.shape[1]))
    for j in range(k):
        t = np.nonzero(on[:, j])[0]
        out[t] += scale * w[t, j, None] * y[d[t, j]]
    return out


def dispatch_backward(g, perm_dst, k, x=None, w=None):
    """(grad x, grad w) of dispatch."""
    g = np.asarray(g, np.float64)
    T = g.shape[0] // k
    ones = np.ones((T, k)) if w is None else np.asarray(w, np.float64)
    gx = combine(g, perm_dst, ones, 1.0)
    if x is None:
        return gx, None
    return gx, _dots(np.asarray(x, np.float64), g, perm_dst, k)


def _dots(a, b, perm_dst, k):
    d, on = _slots(perm_dst, a.shape[0], k)
    out = np.zeros(d.shape)
    for j in range(k):
        t = np.nonzero(on[:, j])[0]
        out[t, j] = (a[t] * b[d[t, j]]).sum(1)
    return out


def combine_backward(g, y, perm_dst, w, scale, out=None):
    """(grad y, grad w) of combine; rows of grad y that no pair names stay."""
    g, w = np.asarray(g, np.float64), np.asarray(w, np.float64)
    gy = dispatch(g, perm_dst, w.shape[1], scale * w, out)
    return gy, scale * _dots(g, np.asarray(y, np.float64), perm_dst, w.shape[1])


def route_dz(logits, ids, g, renormalize, n_experts=256):
    """Gradient of the chosen logits from that of the combine weights g."""
    z, g, ids = np.asarray(logits, np.float64), np.asarray(g, np.float64), np.asarray(ids)
    on = (ids >= 0) & (ids < n_experts)
    log_s = np.where(on, np.minimum(z, 0) - np.log1p(np.exp(-np.abs(z))), -np.inf)
    rest = np.exp(np.minimum(-z, 0) - np.log1p(np.exp(-np.abs(z))))  # 1 - s
    if not renormalize:
        return np.where(on, np.exp(log_s) * rest * g, 0.0)
    top = log_s.max(1, keepdims=True)
    w = np.where(on, np.exp(log_s - np.where(np.isfinite(top), top, 0.0)), 0.0)
    total = w.sum(1, keepdims=True)
    w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    mean = (np.where(on, g, 0.0) * w).sum(1, keepdims=True)
    return np.where(on, w * rest * (g - mean), 0.0)


def route_backward(x, w_router, ids, logits, g, renormalize=True, add=None):
    """(grad w_router, grad x) of the router."""
    x, W, ids = np.asarray(x, np.float64), np.asarray(w_router, np.float64), np.asarray(ids)
    dz = route_dz(logits, ids, g, renormalize, W.shape[0])
    gw = np.zeros_like(W)
    gx = np.zeros_like(x) if add is None else np.array(add, np.float64)
    for j in range(ids.shape[1]):
        on = np.nonzero((ids[:, j] >= 0) & (ids[:, j] < W.shape[0]))[0]
        np.add.at(gw, ids[on, j], dz[on, j, None] * x[on])
        gx[on] += dz[on, j, None] * W[ids[on, j]]
    return gw, gx


# ---------------------------------------------------------------------------
# AdamW
def adamw(p, g, m, v, *, step, lr, beta1, beta2, eps, weight_decay, grad_scale=1.0):
    """(p, m, v) after one step, in fp64."""
    p, g, m, v = (np.asarray(a, np.float64) for a in (p, g, m, v))
    g = g * grad_scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    hat = (m / (1 - beta1 ** step)) / (np.sqrt(v / (1 - beta2 ** step)) + eps)
    return p - lr * weight_decay * p - lr * hat, m, v


def adamw_state_f32(g, m, v, *, beta1, beta2, grad_scale=1.0):
    """(m, v, sqrt v) after one step in fp32, every product and sum rounded by
    itself: the values whose 8-bit codes the library specifies."""
    f = np.float32
    g, m, v = (np.asarray(a, f) for a in (g, m, v))
    g = g * f(grad_scale)
    m = m * f(beta1) + g * f(1 - beta1)
    v = v * f(beta2) + (g * g) * f(1 - beta2)
    return m, v, np.sqrt(v)


def _mix(z):
    z = z & 0xFFFFFFFF
    z = ((z ^ (z >> 16)) * 0x7A3D5E4B) & 0xFFFFFFFF
    z = ((z ^ (z >> 15)) * 0xB5297A4D) & 0xFFFFFFFF
    return z ^ (z >> 16)


def rounding_bits(seed, step, place, n):
    """The 32 random bits of elements 0 .. n-1 of the list's tensor `place`
    (n below 2^32): the low 16 round m, the high 16 sqrt(v)."""
    key = _mix((seed * 0x9E3779B9 + step * 0x85157AF5 + place * 0x632BE5AB) & 0xFFFFFFFF)
    i = np.arange(n, dtype=np.uint64)
    return _mix(((i * np.uint64(0x9E3779B1)) & np.uint64(0xFFFFFFFF)) ^ np.uint64(key))


def block_scales(x):
    """E8M0 codes of the scales of 32-element blocks: the least power of two
    (at least 2^-126) by which the largest finite magnitude is at most 448."""
    x = np.abs(np.asarray(x, np.float64))
    x = np.where(np.isfinite(x), x, 0.0)
    x = np.concatenate([x, np.zeros(-len(x) % 32)]).reshape(-1, 32).max(1)
    e = np.ceil(np.log2(np.maximum(x, 2.0 ** -130) / 448.0))
    # log2 may be off by an ulp at the borders: settle them by comparing
    e = np.where(x <= 448.0 * 2.0 ** (e - 1), e - 1, e)
    e = np.where(x > 448.0 * 2.0 ** e, e + 1, e)
    return (np.maximum(e, -126) + 127).astype(np.uint8)


def encode_8bit(x, random, low):
    """(E4M3 codes, E8M0 scales) of x rounded by `random` (16 bits each)."""
    x = np.asarray(x, np.float64)
    scale = block_scales(x)
    y = x / 2.0 ** (np.repeat(scale.astype(np.float64), 32)[:len(x)] - 127)
    finite = np.isfinite(y)
    a = np.where(finite, np.abs(y), 0.0)
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6) - 3)
    units = np.floor(a / step + random.astype(np.float64) / 65536)
    q = units * step
    if low:
        q = np.where((a > 0) & (q == 0), 2.0 ** -9, q)
    table = np.array([e4m3_decode(np.array([c], np.uint8))[0] for c in range(127)])
    code = np.searchsorted(table, np.minimum(q, 448.0)).astype(np.uint8)
    assert np.all(table[code] == q)
    code = np.where(finite, code, 0x7F).astype(np.uint8)
    return np.where((y < 0) & finite, code | 0x80, code).astype(np.uint8), scale


def decode_8bit(code, scale):
    s = 2.0 ** (np.repeat(np.asarray(scale, np.float64), 32)[:len(code)] - 127)
    return e4m3_decode(np.asarray(code, np.uint8)).astype(np.float64) * s
