"""Plain NumPy oracle of a training step's operators, in 64 bits: the norms around a block with its gate and the
residual sum, the router's balance loss, the gradients' global norm."""
from __future__ import annotations

import numpy as np


def norm_stats(x, kind, eps):
    """[rows, 2]: mean (0 for "rms") and 1 / sqrt(mean square + eps)."""
    mean = x.mean(1) if kind == "layer" else np.zeros(len(x))
    c = x - mean[:, None]
    return np.stack([mean, 1 / np.sqrt((c * c).mean(1) + eps)], 1)


def normed(x, stats):
    return (x - stats[:, :1]) * stats[:, 1:]


def per_row(gate, rows, gate_rows):
    return np.ones((rows, 1)) if gate is None else np.repeat(gate, gate_rows, 0)[:rows]


def residual_norm_h(x, u, kind, w, b, gate, gate_rows, a, c, eps):
    """h before its rounding, and the post norm's statistics (None without one)."""
    if u is None:
        return a * x, None
    stats, v = None, u
    if kind != "none":
        stats = norm_stats(u, kind, eps)
        v = normed(u, stats) * w + b
    return a * x + c * per_row(gate, len(x), gate_rows) * v, stats


def norm_backward(dy, x, stats, w, kind):
    """Gradient at the norm's input; at its weight, at its bias."""
    n, rstd = normed(x, stats), stats[:, 1:]
    g = dy * w
    d = g - n * (g * n).mean(1, keepdims=True)
    if kind == "layer":
        d = d - g.mean(1, keepdims=True)
    return d * rstd, (dy * n).sum(0), dy.sum(0)


def residual_norm_backward(dz, dh, u, h, post, post_w, post_b, gate, gate_rows, pre, pre_w, post_stats, pre_stats, a, c):
    """dx, du and the gradients of post_w, post_b, gate, pre_w, pre_b."""
    dt = np.zeros_like(dz if dh is None else dh) if dh is None else dh
    gpw = gpb = gw = gb = gg = None
    if pre != "none":
        d, gpw, gpb = norm_backward(dz, h, pre_stats, pre_w, pre)
        dt = dt + d
    e = c * dt
    dv = e * per_row(gate, len(dt), gate_rows)
    du, v = dv, u
    if post != "none":
        du, gw, gb = norm_backward(dv, u, post_stats, post_w, post)
        v = normed(u, post_stats) * post_w + post_b
    if gate is not None:
        gg = np.stack([(e * v)[i:i + gate_rows].sum(0) for i in range(0, len(dt), gate_rows)])
    return a * dt, du, gw, gb, gg, gpw, gpb


def balance(logits, idx, offsets, mask, wb, wz, dloss=1.0, gates=None, dgates=None):
    """loss [3], counts [S, E], lse [T], dlogits [T, E]; token by token."""
    T, E = logits.shape
    k, S = idx.shape[1], len(offsets) - 1
    with np.errstate(divide="ignore"):
        m = logits.max(1, keepdims=True) if T else np.zeros((0, 1))
        m = np.where(np.isneginf(m), 0, m)
        q = np.exp(logits - m)
        lse = np.log(q.sum(1)) + m[:, 0]
    seq = np.full(T, -1)
    for s in range(S):
        seq[offsets[s]:offsets[s + 1]] = s
    live = (seq >= 0) & (mask != 0) & (q.sum(1) != 0)
    p = np.zeros((T, E))
    p[live] = q[live] / q[live].sum(1, keepdims=True)
    counts, n, ps = np.zeros((S, E), np.int64), np.zeros(S), np.zeros((S, E))
    for t in np.flatnonzero(live):
        n[seq[t]] += 1
        ps[seq[t]] += p[t]
        for e in idx[t]:
            if 0 <= e < E:
                counts[seq[t], e] += 1
    used, N = (n > 0).sum(), n.sum()
    slope = np.zeros((S, E))
    some = n > 0
    slope[some] = E * counts[some] / (k * n[some, None] ** 2)
    bal = (slope * ps).sum() / max(used, 1)
    z = (lse[live] ** 2).sum() / max(N, 1)
    d = np.zeros((T, E))
    for t in np.flatnonzero(live):
        a = slope[seq[t]] / used
        d[t] = dloss * p[t] * (wb * (a - (p[t] * a).sum()) + 2 * wz * lse[t] / N)
        if gates is not None:
            dot = (gates[t] * dgates[t]).sum()
            for e, g, dg in zip(idx[t], gates[t], dgates[t]):
                if 0 <= e < E:
                    d[t, e] += g * (dg - dot)
    return np.array([wb * bal + wz * z, bal, z]), counts, lse, d


def grad_norm(grads, max_norm, eps):
    """norm, scale."""
    big = max([np.abs(g).max() for g in grads if g.size] + [0.0])
    if not np.isfinite(big) or big == 0:
        norm = big if not any(np.isnan(g).any() for g in grads) else np.nan
    else:
        norm = big * np.sqrt(sum(((g / big) ** 2).sum() for g in grads))
    return norm, np.minimum(1.0, max_norm / (norm + eps))
