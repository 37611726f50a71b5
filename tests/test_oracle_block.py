"""The 64-bit oracle of the operators around the layer, tied to things other
than itself: choices and weights by hand, the softmax top-k oracle of the
layer, torch's layer norm, and gradients against central differences."""

import numpy as np
import pytest
import torch

from oracle import block as ob


def test_route_by_hand():
    l = np.array([[0.0, 2.0, 1.0, 2.0]])
    ids, w = ob.route(l, 2, "sigmoid", renormalize=False)
    assert ids.tolist() == [[1, 3]]                       # equal logits: the lower id
    assert np.allclose(w, 1 / (1 + np.exp(-2.0)))
    ids, w = ob.route(l, 2, "sigmoid", bias=np.array([0.9, 0.0, 0.0, 0.0]), scale=3.0)
    s = 1 / (1 + np.exp(-np.array([0.0, 2.0])))
    assert ids.tolist() == [[0, 1]]                       # the bias moves the choice, not the weight
    assert np.allclose(w, 3 * s / s.sum())
    # two groups of two: {0, 2} and {1, 2}; the best two of the second win, the best one ties
    ids, _ = ob.route(l, 1, "sigmoid", num_groups=2, top_groups=1, group_score="max")
    assert ids.tolist() == [[1]]
    ids, _ = ob.route(l, 1, "sigmoid", num_groups=2, top_groups=1, group_score="top2")
    assert ids.tolist() == [[3]]


def test_route_closed_experts():
    inf = np.inf
    l = np.array([[-inf, -inf, 1.0, -inf], [-inf] * 4, [0.0, np.nan, 0.0, 0.0], [0.0, inf, 0.0, 0.0]])
    ids, w = ob.route(l, 3)
    assert ids.tolist() == [[2, 0, 1], [0, 1, 2], [0, 1, 2], [0, 1, 2]]
    assert w[0].tolist() == [1.0, 0.0, 0.0] and w[1].tolist() == [0.0] * 3
    assert np.isnan(w[2:]).all()
    ids, w = ob.route(l[3:], 2, "sigmoid", renormalize=False)
    assert ids.tolist() == [[1, 0]] and w.tolist() == [[1.0, 0.5]]


def test_route_is_the_layers_top_k():
    from oracle import moe as omoe

    rng = np.random.default_rng(0)
    l = rng.standard_normal((32, 24)).astype(np.float32)
    ids, w = ob.route(l, 5)
    ref = omoe.topk_route(l, 5)
    assert np.array_equal(ids, ref[0])
    assert np.allclose(w, ref[1], rtol=1e-6)


def test_norm_is_torchs():
    g = torch.Generator().manual_seed(0)
    x, w = torch.randn(5, 37, generator=g, dtype=torch.float64), torch.randn(37, generator=g, dtype=torch.float64)
    (_, _), (h, _) = ob.block_norm(x.numpy(), wn=w.numpy(), kind="layer", eps=1e-5)
    assert np.allclose(h, torch.nn.functional.layer_norm(x, (37,), w, None, 1e-5).numpy())
    (_, _), (h, _) = ob.block_norm(x.numpy(), wn=w.numpy(), offset=1.0, eps=1e-5)
    ref = x / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-5) * (1 + w)
    assert np.allclose(h, ref.numpy())


def _central(f, x, d, step=1e-5):
    return (f(x + step * d) - f(x - step * d)) / (2 * step)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(3)
    T, E, K = 6, 11, 4
    l = rng.standard_normal((T, E))
    ids, w = ob.route(l, K, score, renormalize=renorm, scale=1.7)
    dw, d = rng.standard_normal((T, K)), rng.standard_normal((T, E))

    def loss(x):
        s = np.take_along_axis(ob.scores(x, score), ids, 1)
        v = s / (s.sum(1, keepdims=True) + ob.SUM_EPS) if renorm else s
        return (v * 1.7 * dw).sum()

    dl, _ = ob.route_backward(l, ids, w, dw, score, renorm, 1.7)
    assert np.isclose((dl * d).sum(), _central(loss, l, d), rtol=1e-7)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("gate", [None, "channel", "token", "full"])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True)])
def test_norm_gradient_against_differences(kind, gate, post, pre):
    rng = np.random.default_rng(5)
    T, H = 4, 9
    shape = {"channel": (1, H), "token": (T, 1), "full": (T, H)}.get(gate)
    a = {"r": rng.standard_normal((T, H)), "y": rng.standard_normal((T, H)),
         "gate": None if shape is None else rng.standard_normal(shape),
         "wp": rng.standard_normal(H) if post else None, "wn": rng.standard_normal(H) if pre else None}
    kw = dict(kind=kind, post=post, pre=pre, gate_sigmoid=gate == "token", offset=0.5, scale=0.3, eps=1e-3)
    dr, dh = rng.standard_normal((T, H)), rng.standard_normal((T, H))

    def loss(**over):
        b = {**a, **over}
        (r, _), h = ob.block_norm(b["r"], b["y"], b["gate"], b["wp"], b["wn"], **kw)
        return (r * dr).sum() + ((h[0] * dh).sum() if pre else 0.0)

    r_out = ob.block_norm(a["r"], a["y"], a["gate"], a["wp"], a["wn"], **kw)[0][0]
    grads = ob.block_norm_backward(dr, dh, r_out, a["y"], a["gate"], a["wp"], a["wn"], **kw)
    for name, key in (("r", "residual"), ("y", "y"), ("gate", "gate"), ("wp", "post_weight"), ("wn", "pre_weight")):
        if a[name] is None:
            assert key not in grads
            continue
        d = rng.standard_normal(a[name].shape)
        got = (grads[key][0].reshape(a[name].shape) * d).sum()
        assert np.isclose(got, _central(lambda x: loss(**{name: x}), a[name], d), rtol=1e-6, atol=1e-9), key


def test_mag_bounds_its_value():
    rng = np.random.default_rng(7)
    r, y = rng.standard_normal((3, 20)), rng.standard_normal((3, 20))
    (ro, mr), (h, mh) = ob.block_norm(r, y, kind="layer")
    assert (np.abs(ro) <= mr).all() and (np.abs(h) <= mh).all()
    g = ob.block_norm_backward(r, y, ro, y, kind="layer")
    for v, m in g.values():
        assert (np.abs(v) <= m * (1 + 1e-12)).all()
