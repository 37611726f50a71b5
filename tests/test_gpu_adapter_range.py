"""FP16 adapters whose hidden values differ by many powers of two, on the GPU
against 64 bits.

Tolerances (set before the first run).  The two parts of a hidden value keep it to
2^-22 of itself, or to 2^-39 of the largest value that shares its power of two,
whichever is more: the largest lies in [2^14, 2^15), and half of FP16's smallest
step is 2^-25.  Those that share it are a row's ranks in out and dx, and one rank's
rows of an adapter in the factors' gradients.  Tensor cores' sums as in
test_gpu_adapters: n / 16 + 40 steps of 2^-22 of the terms' absolute sum.  An output
is rounded once, 2^-11 of it or 2^-25."""

import numpy as np
import pytest
import torch

from tests.parity import built, gpu, needs_gpu

pytestmark = [gpu, needs_gpu]

F16 = torch.float16


def _adapters(K, N, r):
    from nvfp4_token_quantized_gb300 import LowRankAdapters

    built()
    return LowRankAdapters(K, N, r)


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _steps(n):
    return (n / 16 + 40) * 2.0 ** -22


def _near(got, want, tol, what):
    got = _np(got)
    assert np.isfinite(got).all(), what
    off = np.abs(got - want) / (tol + 2.0 ** -11 * (np.abs(want) + tol) + 2.0 ** -25)
    assert off.max() <= 1, f"{what}: {off.max()} times the tolerance at {np.unravel_index(off.argmax(), off.shape)}"


def _outer(hidden, x):
    """hidden^T x and what FP32 sums of two-part hidden may be off by."""
    parts = 2.0 ** -22 * np.abs(hidden) + 2.0 ** -39 * np.abs(hidden).max(0, keepdims=True)
    mag = np.abs(hidden).T @ np.abs(x)
    return hidden.T @ x, parts.T @ np.abs(x) + _steps(2 * len(x)) * mag, mag


POWERS = [0, -12, -16, -20, -24]


@pytest.mark.parametrize("T", [40, 700, 3000])
def test_factor_gradients_of_ranks_far_apart(T):
    """Each rank's gradient is as good as if it were the only one."""
    K, N, L = 136, 200, 2
    g = torch.Generator().manual_seed(T)
    r = len(POWERS)
    size = 2.0 ** torch.tensor(POWERS, dtype=torch.float32)
    ids = (torch.arange(T) % L).int()
    x = (torch.randn(T, K, generator=g) * 2.0 ** -5).to(F16)
    dout = (torch.randn(T, N, generator=g) * 64).to(F16)
    hidden = torch.randn(T, r, generator=g) * size * 0.5
    down = torch.randn(L, r, K, generator=g).to(F16)
    up = (torch.randn(L, r, N, generator=g) * size[None, :, None] * 8).to(F16)
    dev = [t.cuda() for t in (dout, x, hidden, ids, down, up)]
    _, dd, du = _adapters(K, N, r).backward(*dev)
    for a in range(L):
        rows = (ids == a).numpy()
        want, tol, _ = _outer(_np(hidden)[rows], _np(dout)[rows])
        _near(du[a], want, tol, f"dup of adapter {a}")
        v = _np(dout)[rows] @ _np(up[a]).T
        off = _steps(N) * (np.abs(_np(dout)[rows]) @ np.abs(_np(up[a])).T)  # of v itself
        want, tol, _ = _outer(v, _np(x)[rows])
        _near(dd[a], want, tol + off.T @ np.abs(_np(x)[rows]), f"ddown of adapter {a}")


@pytest.mark.parametrize("T", [40, 700, 3000])
def test_factor_gradients_beside_a_large_row(T):
    """A row far larger than the rest does nothing to columns in which it is 0."""
    K, N, r = 72, 80, 9
    g = torch.Generator().manual_seed(T)
    x, dout = torch.randn(T, K, generator=g).to(F16), torch.randn(T, N, generator=g).to(F16)
    hidden = torch.randn(T, r, generator=g)
    hidden[5] *= 2.0 ** 18
    dout[5] = 0
    dout[5, 0] = 1.0
    ids = torch.zeros(T, dtype=torch.int32)
    down, up = torch.randn(1, r, K, generator=g).to(F16), torch.randn(1, r, N, generator=g).to(F16)
    ad = _adapters(K, N, r)
    _, _, du = ad.backward(*(t.cuda() for t in (dout, x, hidden, ids, down, up)))
    want, tol, mag = _outer(_np(hidden), _np(dout))
    rest = 2.0 ** -39 * np.abs(_np(hidden)).max(0)[:, None] * np.abs(_np(dout)).sum(0)[None, :]
    assert (rest < 2.0 ** -13 * mag)[:, 1:].all()  # (so the bound means something)
    _near(du[0, :, 1:], want[:, 1:], tol[:, 1:], "dup")


@pytest.mark.parametrize("r", [5, 20, 40, 100])
def test_factor_gradients_in_large_sets(r):
    """Only adapters with rows are listed; one of several pieces, one of a row."""
    T, K, N, L = 1500, 40, 72, 300
    g = torch.Generator().manual_seed(r)
    sizes = {0: 1, 7: 700, 150: 97, 299: 300}
    ids = torch.full((T,), -1, dtype=torch.int32)
    ids[torch.randperm(T, generator=g)[:sum(sizes.values())]] = torch.cat(
        [torch.full((n,), a, dtype=torch.int32) for a, n in sizes.items()])
    power = 2.0 ** -(torch.arange(r) * 20 / r).floor()
    x, dout = torch.randn(T, K, generator=g).to(F16), torch.randn(T, N, generator=g).to(F16)
    hidden = torch.randn(T, r, generator=g) * power * 64
    down, up = torch.randn(L, r, K, generator=g).to(F16), torch.randn(L, r, N, generator=g).to(F16)
    _, _, du = _adapters(K, N, r).backward(*(t.cuda() for t in (dout, x, hidden, ids, down, up)))
    for a in range(L):
        rows = (ids == a).numpy()
        if not rows.any():
            assert not du[a].any()
            continue
        want, tol, _ = _outer(_np(hidden)[rows], _np(dout)[rows])
        _near(du[a], want, tol, f"dup of adapter {a}")


def test_an_infinite_hidden_leaves_the_other_ranks():
    """Of a rank that holds an infinity nothing finite is left; the others, above
    FP16's range, stay what they are."""
    T, K, N, r = 300, 64, 72, 4
    g = torch.Generator().manual_seed(1)
    x, dout = torch.randn(T, K, generator=g).to(F16), (torch.randn(T, N, generator=g) * 2.0 ** -10).to(F16)
    hidden = torch.randn(T, r, generator=g) * 2.0 ** 18
    hidden[7, 2] = float("inf")
    ids = torch.zeros(T, dtype=torch.int32)
    down, up = torch.randn(1, r, K, generator=g).to(F16), torch.randn(1, r, N, generator=g).to(F16)
    _, _, du = _adapters(K, N, r).backward(*(t.cuda() for t in (dout, x, hidden, ids, down, up)))
    assert not torch.isfinite(du[0, 2]).any()
    keep = [0, 1, 3]
    want, tol, _ = _outer(_np(hidden)[:, keep], _np(dout))
    _near(du[0, keep], want, tol, "dup")


@pytest.mark.parametrize("T", [6, 60, 300, 700])
def test_rows_whose_largest_rank_meets_zeros(T):
    """out and dx of ranks some 2^-16 of the row's largest, whose own second factor
    is 0 in half of the columns."""
    K, N, L = 64, 96, 2
    r = 4
    g = torch.Generator().manual_seed(T)
    x = (torch.randn(T, K, generator=g) * 2.0 ** 6).to(F16)
    down = torch.randn(L, r, K, generator=g) * 8
    down[:, 1:] = 2.0 ** -20 * torch.randint(1, 200, down[:, 1:].shape, generator=g)
    down = down.to(F16)
    up = torch.randn(L, r, N, generator=g).to(F16)
    up[:, 0, ::2] = 0
    ids = (torch.arange(T) % L).int()
    ad = _adapters(K, N, r)
    out, h = ad.forward(*(t.cuda() for t in (x, ids, down, up)), keep_hidden=True)
    swapped = _adapters(N, K, r)  # the same product as the gradient by x
    dx, _, _ = swapped.backward(x.cuda(), torch.zeros(T, N, dtype=F16, device="cuda"), h, ids.cuda(), up.cuda(),
                                down.cuda())
    for a in range(L):
        rows = (ids == a).numpy()
        d, u, xs = _np(down[a]), _np(up[a]), _np(x)[rows]
        hidden, own = xs @ d.T, _steps(K) * (np.abs(xs) @ np.abs(d).T)
        parts = own + 2.0 ** -22 * np.abs(hidden) + 2.0 ** -39 * (np.abs(hidden) + own).max(1, keepdims=True)
        tol = parts @ np.abs(u) + _steps(2 * r) * (np.abs(hidden) @ np.abs(u))
        assert (2.0 ** -25 * np.abs(hidden).max(1) > 2.0 ** -19 * np.abs(hidden[:, 1])).mean() > 0.5
        _near(out.cpu()[rows], hidden @ u, tol, f"out of adapter {a}")
        _near(dx.cpu()[rows], hidden @ u, tol, f"dx of adapter {a}")
