"""The operators together, as a tuning step of a sparse block uses them: adapters
beside the experts, the norms' and the adapters' gradients, the balance loss and
the clipping, each gradient against a 64-bit chain of the oracles.

A gradient here passes through three operators, each of which rounds its output
to bf16: it stays within the parity tolerance of tests/parity.py (2e-2 of the
rms, 5e-2 of the value); the FP32 ones, through two, too."""

import numpy as np
import pytest
import torch

import synthetic
from oracle import block as ob
from oracle import training as ot
from tests import parity
from tests.parity import built, gpu, needs_gpu

pytestmark = [gpu, needs_gpu]


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("T", [1, 48, 200])
def test_tuning_gradients(T):
    built()
    from examples import sparse_block as ex

    stack = ex.SparseStack(ex.SHAPE, 2, users=3)
    x = synthetic.make_activations(ex.SHAPE, T=T).cuda()
    user = (torch.arange(T, device="cuda") % 4 - 1).int()
    h, trace = stack.forward(x, user)
    s, i = trace[1], 1
    r_out, h2 = stack.norm.forward(s["residual"], s["y"], post_weight=stack.post[i], pre_weight=stack.pre[i + 1])
    assert torch.equal(h, h2)
    dh = torch.randn(T, ex.SHAPE.H, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    loss, counts, grads, norm = stack.tuning_gradients(s, r_out, dh, user, balance=0.5)

    eps = float(np.float32(1e-6))
    ref = ob.block_norm_backward(None, _np(dh), _np(r_out), _np(s["y"]), wp=_np(stack.post[i]), wn=_np(stack.pre[i + 1]),
                                 eps=eps)
    u = user.cpu().numpy()
    (_, dd, du), _ = ot.adapters_backward(ref["y"][0], _np(s["h"]), _np(s["hidden"]), u, _np(stack.down[i]),
                                          _np(stack.up[i]))
    ids = s["topk_ids"].cpu().numpy()
    (rl, _), rc, (rs, _) = ot.balance(_np(s["logits"]), ids, 0.5, "sigmoid")
    dl, _ = ot.balance_backward(_np(s["logits"]), rs, 1.0, "sigmoid")
    want = {"down": dd, "up": du, "post": ref["post_weight"][0], "pre": ref["pre_weight"][0],
            "gate": _np(s["h"]).T @ dl}
    assert np.array_equal(counts.cpu().numpy(), rc) and abs(loss.item() - rl) <= 1e-5 * abs(rl)
    total = np.sqrt(sum((g ** 2).sum() for g in want.values()))
    assert abs(norm.item() - total) <= 2e-2 * total
    factor = min(1.0, 1.0 / (norm.item() + 1e-6))
    assert factor < 1.0
    for name, g in want.items():
        parity.assert_close(_np(grads[name]), g * factor, what=name)


def test_adapters_are_the_users_own():
    """Rows without a user match the stack without adapters; a user's rows do not
    depend on who else is in the batch."""
    built()
    from examples import sparse_block as ex

    stack = ex.SparseStack(ex.SHAPE, 1, users=3)
    plain = ex.SparseStack(ex.SHAPE, 1)
    x = synthetic.make_activations(ex.SHAPE, T=60).cuda()
    none = torch.full((60,), -1, dtype=torch.int32, device="cuda")
    assert torch.equal(stack.forward(x, none)[0], plain.forward(x)[0])
    user = none.clone()
    user[10:20] = 1
    got = stack.forward(x, user)[0]
    rest = user < 0
    assert torch.equal(got[rest], plain.forward(x)[0][rest]) and not torch.equal(got[~rest], plain.forward(x)[0][~rest])


def test_steps_run():
    built()
    from examples import sparse_block as ex

    stack = ex.SparseStack(ex.SHAPE, 2, users=2)
    x = synthetic.make_activations(ex.SHAPE, T=100).cuda()
    user = (torch.arange(100, device="cuda") % 2).int()
    target = stack.forward(x, user)[0].roll(1, dims=1)
    for _ in range(3):
        values = stack.tuning_step(x, user, target, lr=1.0)
        assert all(torch.isfinite(v).all() for v in values)


def test_gradients_of_the_choice_and_the_balance_add_up():
    """One call's result goes on in the next: the choice's gradient, the balance
    loss's added in place, then clipped."""
    from nvfp4_token_quantized_gb300 import ExpertRouter, GradientClip

    built()
    g = torch.Generator().manual_seed(2)
    T, E, K = 300, 64, 4
    logits = torch.randn(T, E, generator=g).cuda()
    router = ExpertRouter(E, K, score="sigmoid", scale=2.5)
    ids, w = router.select(logits)
    dw = torch.randn(T, K, generator=g).cuda()
    loss, counts, slope = router.balance_loss(logits, ids, coefficient=3.0)
    d = router.select_backward(logits, ids, w, dw)
    router.balance_backward(logits, slope, add=d, dlogits=d)
    norm, (clipped,) = GradientClip(0.5).clip([d.clone()])
    a, _ = ob.route_backward(_np(logits), ids.cpu().numpy(), _np(w), _np(dw), "sigmoid", True, 2.5)
    (_, _), rc, (rs, _) = ot.balance(_np(logits), ids.cpu().numpy(), 3.0, "sigmoid")
    b, _ = ot.balance_backward(_np(logits), rs, 1.0, "sigmoid")
    want = a + b
    assert counts.sum().item() == T * K
    # (FP32 all through; the choice's own error is some 2^-20 of its terms)
    assert np.abs(_np(d) - want).max() <= 1e-5 * np.abs(want).max()
    f = 0.5 / (np.sqrt((want ** 2).sum()) + 1e-6)
    assert np.abs(_np(clipped) - want * f).max() <= 2e-5 * np.abs(want * f).max()
