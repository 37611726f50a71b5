"""The operators around the expert layer in 64 bits (numpy): the choice of
experts and the norms before and after a block, with their gradients.

Beside each result stands ``mag``: the sum of the absolute values of the terms
the result is formed from, to which the error of an evaluation in fewer bits
is proportional.
"""

from __future__ import annotations

from typing import Optional

import numpy as np

SUM_EPS = 1e-20


def _sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


# ---- choice of experts ----

def scores(l: np.ndarray, score: str) -> np.ndarray:
    """Scores [T, E]; a row of -inf logits scores 0 everywhere."""
    if score == "sigmoid":
        return _sigmoid(l)
    m = l.max(axis=1, keepdims=True)
    e = np.exp(l - np.where(np.isneginf(m), 0.0, m))
    total = e.sum(axis=1, keepdims=True)
    return e / np.where(total == 0, 1.0, total)


def undefined_rows(l: np.ndarray, score: str) -> np.ndarray:
    return np.isnan(l).any(1) | (np.isposinf(l).any(1) & (score == "softmax"))


def route_choice(l: np.ndarray, score: str, bias, num_groups: int, top_groups: int, group_score: str):
    """What experts are chosen by, [T, E] (-inf: closed or outside the chosen
    groups), and the groups' scores [T, G] (None if no group is left out)."""
    T, E = l.shape
    size = E // num_groups
    v = np.where(undefined_rows(l, score)[:, None], -np.inf, l)
    if bias is not None or (num_groups > 1 and group_score == "top2"):
        with np.errstate(invalid="ignore"):
            v = np.where(np.isneginf(v), v, scores(v, score) + (0.0 if bias is None else np.asarray(bias, np.float64)))
    v[np.isnan(v)] = -np.inf
    if top_groups == num_groups:
        return v, None
    g = np.full((T, num_groups), -np.inf)
    for t in range(T):
        for i in range(num_groups):
            best = np.sort(v[t, i * size:(i + 1) * size])[::-1][:2 if group_score == "top2" else 1]
            best = best[best > -np.inf]
            if best.size:
                g[t, i] = best.sum()
        keep = np.lexsort((np.arange(num_groups), -g[t]))[:top_groups]
        v[t, ~np.isin(np.arange(E) // size, keep)] = -np.inf
    return v, g


def route(l: np.ndarray, K: int, score: str = "softmax", bias: Optional[np.ndarray] = None, num_groups: int = 1,
          top_groups: int = 1, group_score: str = "max", renormalize: bool = True, scale: float = 1.0):
    """(ids [T, K], weights [T, K]) from logits [T, E]."""
    l = np.asarray(l, dtype=np.float64)
    T, E = l.shape
    bad = undefined_rows(l, score)
    v, _ = route_choice(l, score, bias, num_groups, top_groups, group_score)
    s = scores(np.where(bad[:, None], 0.0, l), score)
    ids = np.stack([np.lexsort((np.arange(E), -v[t]))[:K] for t in range(T)]) if T else np.zeros((0, K), np.int64)
    w = np.where(np.take_along_axis(v, ids, 1) > -np.inf, np.take_along_axis(s, ids, 1), 0.0)
    if renormalize:
        w = w / (w.sum(axis=1, keepdims=True) + SUM_EPS)
    w[bad] = np.nan
    return ids, w * scale


def route_backward(l, ids, w, dw, score="softmax", renormalize=True, scale=1.0):
    """(dlogits [T, E], mag): slots of weight 0 or with an id outside [0, E)
    pass nothing."""
    l = np.asarray(l, dtype=np.float64)
    T, E = l.shape
    s = scores(l, score)
    live = (np.asarray(w) != 0) & (ids >= 0) & (ids < E)
    safe = np.where(live, ids, 0)
    sk = np.where(live, np.take_along_axis(s, safe, 1), 0.0)
    d = np.where(live, np.asarray(dw, np.float64) * scale, 0.0)
    mag = np.abs(d)
    if renormalize:
        total = sk.sum(axis=1, keepdims=True) + SUM_EPS
        mag = np.where(live, (np.abs(d) + (np.abs(d) * sk).sum(1, keepdims=True) / total) / total, 0.0)
        d = np.where(live, (d - (d * sk).sum(1, keepdims=True) / total) / total, 0.0)
    ds, ms = np.zeros_like(s), np.zeros_like(s)
    rows = np.arange(T)[:, None]
    np.add.at(ds, (rows, safe), d)
    np.add.at(ms, (rows, safe), mag)
    if score == "sigmoid":
        return ds * s * (1 - s), ms * s
    return s * (ds - (ds * s).sum(1, keepdims=True)), s * (ms + (ms * s).sum(1, keepdims=True))


# ---- norms around a block ----

def _norm(x, mag_x, w, kind, eps, offset):
    """n(x; w), its mag, and (xhat, mag of xhat, rstd)."""
    mean = x.mean(1, keepdims=True) if kind == "layer" else 0.0
    mag_d = mag_x + (mag_x.mean(1, keepdims=True) if kind == "layer" else 0.0)
    d = x - mean
    var = (d * d).mean(1, keepdims=True) + eps
    rstd = 1.0 / np.sqrt(var)
    xhat = d * rstd
    # (the statistic's own error: that of the squares, each d times its mag)
    mag_hat = mag_d * rstd + np.abs(xhat) * (1.0 + (np.abs(d) * mag_d).mean(1, keepdims=True) / var)
    wt = 1.0 if w is None else offset + w
    mag_w = 1.0 if w is None else np.abs(offset) + np.abs(w)
    return xhat * wt, mag_hat * mag_w, (xhat, mag_hat, rstd)


def _gate(gate, T, sigmoid):
    if gate is None:
        return 1.0
    g = np.asarray(gate, np.float64)
    if g.ndim == 1 and g.shape[0] != T:
        g = g[None, :]
    return _sigmoid(g) if sigmoid else g


def block_norm(r, y=None, gate=None, wp=None, wn=None, kind="rms", eps=1e-6, post=True, pre=True, gate_sigmoid=False,
               offset=0.0, scale=1.0):
    """((r', mag), (h, mag)); gate [1, H], [T, 1] or [T, H]."""
    r = np.asarray(r, np.float64)
    mag = np.abs(r)
    if y is not None:
        u = np.asarray(y, np.float64)
        mu = np.abs(u)
        if post:
            u, mu, _ = _norm(u, mu, wp, kind, eps, offset)
        g = _gate(gate, r.shape[0], gate_sigmoid)
        r = r + scale * g * u
        mag = mag + np.abs(scale * g) * mu
    if not pre:
        return (r, mag), None
    h, mh, _ = _norm(r, mag, wn, kind, eps, offset)
    return (r, mag), (h, mh)


def _norm_backward(dout, mag_out, x, w, kind, eps, offset):
    """((dx, mag), (dw, mag))."""
    _, _, (xhat, mh, rstd) = _norm(x, np.abs(x), w, kind, eps, offset)
    wt = 1.0 if w is None else offset + w
    mag_w = 1.0 if w is None else np.abs(offset) + np.abs(w)
    a, ma = dout * wt, mag_out * mag_w
    dx = a - xhat * (a * xhat).mean(1, keepdims=True)
    mx = ma + mh * (ma * mh).mean(1, keepdims=True)
    if kind == "layer":
        dx = dx - a.mean(1, keepdims=True)
        mx = mx + ma.mean(1, keepdims=True)
    # (rstd's own relative error, at most that of the whole of xhat)
    rel = 1.0 + (np.abs(xhat) * mh).mean(1, keepdims=True)
    return (dx * rstd, mx * rstd * rel), ((dout * xhat).sum(0), (mag_out * mh).sum(0))


def block_norm_backward(dr, dh, r_out, y=None, gate=None, wp=None, wn=None, kind="rms", eps=1e-6, post=True, pre=True,
                        gate_sigmoid=False, offset=0.0, scale=1.0):
    """{name: (gradient, mag)} of residual, y, gate, post_weight, pre_weight."""
    out = {}
    x = None if r_out is None else np.asarray(r_out, np.float64)
    d = np.zeros_like(x if dr is None else np.asarray(dr, np.float64)) if dr is None else np.asarray(dr, np.float64)
    md = np.abs(d)
    if pre:
        h = np.asarray(dh, np.float64)
        (dx, mx), out["pre_weight"] = _norm_backward(h, np.abs(h), x, wn, kind, eps, offset)
        d, md = d + dx, md + mx
    out["residual"] = (d, md)
    if y is None:
        return out
    y = np.asarray(y, np.float64)
    g = _gate(gate, y.shape[0], gate_sigmoid)
    e, me = scale * d, np.abs(scale) * md
    u, mu = y, np.abs(y)
    if post:
        u, mu, _ = _norm(y, mu, wp, kind, eps, offset)
    if gate is not None:
        f = g * (1 - g) if gate_sigmoid else 1.0
        mf = g if gate_sigmoid else 1.0
        dg, mg = e * u * f, me * mu * mf
        if g.shape[0] == 1 and y.shape[0] != 1 or np.ndim(gate) == 1:
            dg, mg = dg.sum(0), mg.sum(0)
        elif g.shape[1] == 1 and y.shape[1] != 1:
            dg, mg = dg.sum(1, keepdims=True), mg.sum(1, keepdims=True)
        out["gate"] = (dg, mg)
    b, mb = e * g, me * np.abs(g)
    if post:
        (b, mb), out["post_weight"] = _norm_backward(b, mb, y, wp, kind, eps, offset)
    out["y"] = (b, mb)
    return out
