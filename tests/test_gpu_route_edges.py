"""The gradient of the choice where sigmoid scores are near 1.

Tolerance (set before the first run), with U = 2^-24: the factors but 1 - s
agree to 64 U of the sum of their terms' absolute values, as in
test_gpu_route_select.py.  A score taken from the weights is within 12 U (the
roundings of two weights, two quotients and a product, and the four of the
sigmoid), 16 U here, which 1 - s turns into 16 U s / (1 - s); from 1 - 1/64 on
(1 - 1/256 for the 16-bit types) 1 - s comes from the logit and has no such term.
An output of 16 bits adds half a unit in its last place and its smallest number.
"""

import numpy as np
import pytest
import torch

from tests.parity import built, gpu, needs_gpu

pytestmark = [gpu, needs_gpu]

U = 2.0 ** -24
UNIT = {torch.float32: (0.0, 0.0), torch.float16: (2.0 ** -11, 2.0 ** -25), torch.bfloat16: (2.0 ** -8, 2.0 ** -133)}


def _sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,K,pad", [(1, 8, 8, 0), (40, 64, 8, 0), (333, 97, 5, 3), (12000, 64, 6, 0),
                                       (12000, 250, 12, 1)])
def test_gradient_of_scores_near_one(T, E, K, pad, renormalize, dtype):
    from nvfp4_token_quantized_gb300 import ExpertRouter

    built()
    g = torch.Generator().manual_seed(T + E)
    wide = torch.zeros(T, E + pad)
    # logits from -4 to a row's largest, 2 to 40
    wide[:, :E] = torch.rand(T, E, generator=g) * (torch.rand(T, 1, generator=g) * 38 + 6) - 4
    l = wide.to(dtype).cuda()[:, :E]
    scale = 1.7
    r = ExpertRouter(E, K, score="sigmoid", renormalize=renormalize, scale=scale)
    ids, w = r.select(l)
    dw = torch.randn(T, K, generator=g).cuda()
    dl = r.select_backward(l, ids, w, dw)

    x = np.take_along_axis(l.double().cpu().numpy(), ids.cpu().numpy().astype(np.int64), 1)
    s, rest = _sigmoid(x), _sigmoid(-x)
    d = dw.double().cpu().numpy() * float(np.float32(scale))
    mag = np.abs(d)
    if renormalize:
        total = s.sum(1, keepdims=True)
        mag = (np.abs(d) + (np.abs(d) * s).sum(1, keepdims=True) / total) / total
        d = (d - (d * s).sum(1, keepdims=True) / total) / total
    ref = d * s * rest
    near = 64 if dtype == torch.float32 else 256
    from_weight = 16 * U * np.where(rest * near > 0.99, s / rest, 0.0)
    u, tiny = UNIT[dtype]
    got = np.take_along_axis(dl.double().cpu().numpy(), ids.cpu().numpy().astype(np.int64), 1)
    tol = mag * s * rest * (64 * U + from_weight) + u * np.abs(ref) + tiny + 1e-37
    assert (s > 0.999).any() and np.isfinite(got).all()
    assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) / tol).max())
    # what was not chosen gets none, and a second call gives the same bits
    rows = dl.double().cpu().numpy().copy()
    np.put_along_axis(rows, ids.cpu().numpy().astype(np.int64), 0.0, 1)
    assert (rows == 0).all()
    assert torch.equal(dl, r.select_backward(l, ids, w, dw))
    into = wide.to(dtype).cuda()[:, :E]
    assert torch.equal(dl, r.select_backward(into, ids, w, dw, dlogits=into))
