"""The balance loss of a choice of experts, gradient clipping and low-rank
adapters in 64 bits (numpy), with their gradients.

Beside a result that the library forms in FP32 stands ``err``: how far off an
evaluation in FP32 may be, in units of 2^-24, counted from its operations: the
hardware's exponential is within 2 + 1.173 |x| units in the last place (twice
that many of 2^-24), its quotient within 2, each product and each sum of a tree
within 1.
"""

from __future__ import annotations

import numpy as np

SUM_EPS = 1e-20


def shares(l: np.ndarray, score: str):
    """(p, rel, rest): each token's shares [T, E], their relative error in
    units of 2^-24, and what a share's derivative is formed with: 1 for softmax,
    1 - s for sigmoid scores.  Closed experts have p = 0, rows of them too."""
    l = np.asarray(l, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-l))
            total = s.sum(1, keepdims=True) + SUM_EPS
            rest, far = 1.0 / (1.0 + np.exp(l)), np.abs(l)
        else:
            m = l.max(1, keepdims=True)
            d = l - np.where(np.isneginf(m), 0.0, m)
            s = np.exp(d)
            total = s.sum(1, keepdims=True)
            total = np.where(total == 0, 1.0, total)
            rest, far = np.ones_like(l), np.abs(d)
        p = s / total
        # the score itself, and the sum's terms by their weight in it; the sum's
        # 16 terms a lane and 4 steps, quotients and products
        rel = 14.0 + 2.4 * np.where(p == 0, 0.0, far)
        rel = rel + (p * rel).sum(1, keepdims=True) + 32.0
    return p, np.where(p == 0, 0.0, rel), rest, total


def counted(T, offsets, mask):
    """The counted rows of each sequence."""
    offsets = [0, T] if offsets is None else np.clip(offsets, 0, T)
    for lo, hi in zip(offsets, offsets[1:]):
        rows = np.arange(lo, max(lo, hi))
        yield rows if mask is None else rows[np.asarray(mask, bool)[rows]]


def balance(l, ids, coefficient, score="softmax", offsets=None, mask=None):
    """(loss, err), counts [S, E], (slope, err)."""
    l = np.asarray(l, np.float64)
    T, E = l.shape
    K = ids.shape[1]
    runs = list(counted(T, offsets, mask))
    used = max(1, sum(r.size > 0 for r in runs))
    loss = err = 0.0
    counts, slope = np.zeros((len(runs), E), np.int64), np.zeros((len(runs), E))
    for s, rows in enumerate(runs):
        if not rows.size:
            continue
        p, rel, _, _ = shares(l[rows], score)
        i = ids[rows]
        counts[s] = np.bincount(i[(i >= 0) & (i < E)], minlength=E)
        n = rows.size
        slope[s] = coefficient * E * counts[s] / (K * n * n * used)
        loss += (slope[s] * p.sum(0)).sum()
        # (64: adds of a lane's rows, the warps and the runs; 16: of products,
        # of experts and sequences)
        err += (np.abs(slope[s]) * (p * (rel + 64.0)).sum(0)).sum() + 16.0 * np.abs(slope[s] * p.sum(0)).sum()
    return (loss, err), counts, (slope, 8.0 * np.abs(slope))


def balance_backward(l, slope, dloss, score="softmax", offsets=None, mask=None, add=None):
    """(dlogits, err)."""
    l = np.asarray(l, np.float64)
    out = np.zeros_like(l) if add is None else np.array(add, np.float64)
    err = np.abs(out)
    for s, rows in enumerate(counted(l.shape[0], offsets, mask)):
        if not rows.size:
            continue
        g = np.asarray(slope, np.float64)[s] * dloss
        p, rel, rest, total = shares(l[rows], score)
        mean = (p * g).sum(1, keepdims=True)
        off = (p * np.abs(g) * (rel + 24.0)).sum(1, keepdims=True)
        d = p * rest * (g - mean)
        out[rows] += d
        err[rows] += np.abs(d) * 2 + p * rest * ((rel + 14.0 + 2.4 * np.where(p == 0, 0.0, np.abs(l[rows])) *
                                                  (score == "sigmoid")) * np.abs(g - mean) + np.abs(g) * 2 + off)
    return out, err


def clip(grads, max_norm, eps):
    """norm, factor."""
    norm = np.sqrt(sum((np.asarray(g, np.float64) ** 2).sum() for g in grads))
    with np.errstate(invalid="ignore"):
        f = max_norm / (norm + eps)
    return norm, f if np.isnan(f) else min(1.0, f)


def adapters(x, ids, first, second, scales=None, base=None):
    """out [T, N], hidden [T, r], and the sums of the absolute values of the
    terms that each is formed from."""
    x = np.asarray(x, np.float64)
    T, L = x.shape[0], first.shape[0]
    h, hm = np.zeros((T, first.shape[1])), np.zeros((T, first.shape[1]))
    out = np.zeros((T, second.shape[2])) if base is None else np.array(base, np.float64)
    mag = np.abs(out)
    for a in range(L):
        rows = np.nonzero(ids == a)[0]
        s = 1.0 if scales is None else float(scales[a])
        h[rows] = s * (x[rows] @ first[a].T)
        hm[rows] = abs(s) * (np.abs(x[rows]) @ np.abs(first[a]).T)
        out[rows] += h[rows] @ second[a]
        mag[rows] += hm[rows] @ np.abs(second[a])
    return out, h, mag, hm


def adapters_backward(dout, x, hidden, ids, down, up, scales=None, base=None):
    """dx, ddown, dup and the sums of the absolute values of their terms."""
    dout, x, hidden = (np.asarray(v, np.float64) for v in (dout, x, hidden))
    dx, v, mx, vm = adapters(dout, ids, up, down, scales, base)
    dd, du = np.zeros(down.shape), np.zeros(up.shape)
    md, mu = np.zeros(down.shape), np.zeros(up.shape)
    for a in range(down.shape[0]):
        rows = np.nonzero(ids == a)[0]
        dd[a], md[a] = v[rows].T @ x[rows], vm[rows].T @ np.abs(x[rows])
        du[a], mu[a] = hidden[rows].T @ dout[rows], np.abs(hidden[rows]).T @ np.abs(dout[rows])
    return (dx, dd, du), (mx, md, mu)
