"""The 64-bit oracle of the balance loss and the adapters against central
differences and hand-made cases."""

import numpy as np
import pytest

from oracle import training as ot


def _difference(f, x, way, h=1e-5):
    return (f(x + h * way) - f(x - h * way)) / (2 * h)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("offsets,masked", [(None, False), ([2, 9, 9, 20], True)])
def test_balance_gradient(score, offsets, masked):
    rng = np.random.default_rng(0)
    T, E, K = 23, 11, 3
    l = rng.standard_normal((T, E)) * 2
    l[4, :5] = -np.inf
    l[6] = -np.inf
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :K]
    mask = rng.random(T) < 0.7 if masked else None
    (loss, _), counts, (slope, _) = ot.balance(l, ids, 0.4, score, offsets, mask)
    d, _ = ot.balance_backward(l, slope, 1.0, score, offsets, mask)
    way = rng.standard_normal((T, E))
    num = _difference(lambda v: ot.balance(v, ids, 0.4, score, offsets, mask)[0][0], l, way)
    assert abs((d * way).sum() - num) < 1e-9
    assert np.isfinite(d).all() and not d[6].any()


def test_balance_by_hand():
    """Uniform scores: the loss is the coefficient; all on one of E experts with
    a share of 1: E times it."""
    l = np.zeros((4, 4))
    ids = np.array([[0], [1], [2], [3]])
    (loss, _), counts, _ = ot.balance(l, ids, 0.25)
    assert abs(loss - 0.25) < 1e-15 and (counts == 1).all()
    l[:, 0] = 800.0
    (loss, _), counts, _ = ot.balance(l, np.zeros((4, 1), int), 0.25)
    assert abs(loss - 1.0) < 1e-12 and counts[0, 0] == 4


def test_sequences_are_averaged():
    rng = np.random.default_rng(1)
    l, ids = rng.standard_normal((10, 6)), rng.integers(0, 6, (10, 2))
    one = [ot.balance(l[a:b], ids[a:b], 1.0)[0][0] for a, b in ((0, 3), (3, 10))]
    (loss, _), _, _ = ot.balance(l, ids, 1.0, offsets=[0, 3, 3, 10])
    assert abs(loss - sum(one) / 2) < 1e-14


def test_adapter_gradients():
    rng = np.random.default_rng(2)
    T, K, N, r, L = 12, 7, 5, 3, 4
    x, down, up = rng.standard_normal((T, K)), rng.standard_normal((L, r, K)), rng.standard_normal((L, r, N))
    ids, scales = rng.integers(-1, L + 1, T), rng.standard_normal(L)
    base, dout = rng.standard_normal((T, N)), rng.standard_normal((T, N))
    out, h, mag, _ = ot.adapters(x, ids, down, up, scales, base)
    none = (ids < 0) | (ids >= L)
    assert np.array_equal(out[none], base[none]) and (mag >= np.abs(out) - 1e-12).all()
    (dx, dd, du), _ = ot.adapters_backward(dout, x, h, ids, down, up, scales)
    for name, g in (("x", dx), ("down", dd), ("up", du)):
        a = dict(x=x, down=down, up=up)
        way = rng.standard_normal(a[name].shape)

        def f(v):
            b = dict(a)
            b[name] = v
            return (ot.adapters(b["x"], ids, b["down"], b["up"], scales, base)[0] * dout).sum()

        assert abs((g * way).sum() - _difference(f, a[name], way)) < 1e-7


def test_clip():
    n, f = ot.clip([np.array([3.0]), np.array([[4.0]])], 1.0, 1e-6)
    assert n == 5.0 and abs(f - 1.0 / 5.000001) < 1e-15
    assert ot.clip([np.array([3.0])], 4.0, 1e-6)[1] == 1.0
