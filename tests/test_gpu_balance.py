"""The balance loss, its counts and its gradient on the GPU against the 64-bit
oracle, within the errors that oracle/training.py counts (set before the first
run); an output of fewer bits adds one rounding, half a step."""

import numpy as np
import pytest
import torch

from oracle import training as ot
from tests.parity import built, gpu, needs_gpu

pytestmark = [gpu, needs_gpu]

U = 2.0 ** -24
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
UNIT = {F32: (0.0, 2.0 ** -149), F16: (2.0 ** -11, 2.0 ** -25), BF16: (2.0 ** -8, 2.0 ** -133)}


def _router(E, K, score="softmax"):
    from nvfp4_token_quantized_gb300 import ExpertRouter

    built()
    return ExpertRouter(E, K, score=score)


def _np(t):
    return None if t is None else t.float().cpu().numpy().astype(np.float64)


def _close(got, val, err, what, dtype=F32):
    g = _np(got).reshape(np.shape(val))
    half, tiny = UNIT[dtype]
    tol = U * err + half * (np.abs(val) + U * err) + tiny + 1e-36
    assert np.isfinite(g).all(), what
    worst = np.max(np.abs(g - val) / tol) if g.size else 0.0
    assert worst <= 1, f"{what}: {worst} times the tolerance"


def _make(T, E, K, dtype=F32, S=0, mask=False, closed=0.0, pad=0, tail=0, seed=0):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, E, generator=g) * (0.5 + 2 * torch.rand(T, 1, generator=g))
    if closed:
        l = l.masked_fill(torch.rand(T, E, generator=g) < closed, -np.inf)
        l[::7] = -np.inf
    ids = torch.rand(T, E, generator=g).argsort(dim=1)[:, :K].int()
    ids[::5, 0] = -1
    ids[::11, -1] = E
    off = None
    if S:
        cuts = torch.randint(0, T - tail + 1, (S - 1,), generator=g).sort().values
        off = torch.cat([torch.tensor([min(2, T - tail)]) if S > 2 else torch.tensor([0]), cuts.clamp(min=min(2, T - tail)),
                         torch.tensor([T - tail])]).int()
    m = (torch.rand(T, generator=g) < 0.8) if mask else None
    wide = torch.full((T, E + pad), float("nan"))
    wide[:, :E] = l
    add = torch.randn(T, E, generator=g).to(dtype)
    return (wide.to(dtype).cuda()[:, :E], ids.cuda(), None if off is None else off.cuda(),
            None if m is None else m.cuda(), add.cuda())


def _check(T, E, K, dtype=F32, score="softmax", coefficient=0.3, S=0, mask=False, arrays=None, with_add=True, **kw):
    r = _router(E, K, score)
    l, ids, off, m, add = arrays or _make(T, E, K, dtype, S, mask, **kw)
    loss, counts, slope = r.balance_loss(l, ids, coefficient, off, m)
    ln, off_n, m_n = _np(l), None if off is None else off.cpu().numpy(), None if m is None else m.cpu().numpy()
    if m_n is not None:
        ln[~m_n.astype(bool)] = 0.0
    c32 = float(np.float32(coefficient))
    rl, rc, rs = ot.balance(ln, ids.cpu().numpy(), c32, score, off_n, m_n)
    assert loss.shape == () and counts.dtype == torch.int32
    assert np.array_equal(counts.cpu().numpy(), rc)
    _close(slope, *rs, "slope")
    _close(loss, *rl, "loss")
    dloss = torch.tensor(0.7, device="cuda")
    for a in ((None, add) if with_add else (None,)):
        d = r.balance_backward(l, slope, dloss, off, m, a)
        assert d.dtype == dtype and d.shape == (T, E)
        ref = ot.balance_backward(ln, _np(slope), float(np.float32(0.7)), score, off_n, m_n, _np(a))
        _close(d, *ref, "dlogits", dtype)
    return r, (l, ids, off, m, add), (loss, counts, slope)


@pytest.mark.parametrize("E", [1, 2, 7, 8, 31, 63, 64, 65, 97, 128, 160, 192, 250, 256, 260, 384, 500, 512])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_experts(E, score):
    _check(57, E, min(E, 4), score=score)
    _check(2500, E, min(E, 3), BF16, score=score, S=3, mask=True, closed=0.1)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_types_and_strides(dtype, score):
    for pad in (0, 1, 3, 4, 8):
        _check(300, 96, 5, dtype, score, pad=pad, mask=True)
        _check(300, 97, 5, dtype, score, pad=pad, S=4, closed=0.2)


@pytest.mark.parametrize("T", [0, 1, 2, 15, 16, 17, 33, 127, 1000, 4863, 4864, 4865, 10000])
def test_lengths(T):
    _check(T, 256, 8, score="sigmoid")
    if T:
        _check(T, 64, 2, S=min(T, 5), tail=T // 3, mask=True)


def test_many_short_sequences():
    _check(3000, 40, 3, S=1500, mask=True)
    _check(700, 16, 2, S=5000)  # (more sequences than rows: most are empty)


def test_one_sequence_by_offsets_equals_none():
    r, (l, ids, _, _, _), (loss, counts, slope) = _check(9000, 128, 8, score="sigmoid")
    off = torch.tensor([0, 9000], dtype=torch.int32, device="cuda")
    again = r.balance_loss(l, ids, 0.3, off)
    assert torch.equal(again[0], loss) and torch.equal(again[1], counts) and torch.equal(again[2], slope)


def test_nothing_counted():
    r = _router(32, 2)
    l, ids, _, _, add = _make(100, 32, 2)
    none = torch.zeros(100, dtype=torch.bool, device="cuda")
    off = torch.tensor([40, 40, 40], dtype=torch.int32, device="cuda")
    for o, m in ((None, none), (off, None)):
        loss, counts, slope = r.balance_loss(l, ids, 1.0, o, m)
        assert loss.item() == 0 and not counts.any() and not slope.any()
        assert not r.balance_backward(l, slope, None, o, m).any()
        assert torch.equal(r.balance_backward(l, slope, None, o, m, add), add)


def test_uncounted_rows_may_hold_anything():
    r = _router(64, 4, "softmax")
    l, ids, _, m, _ = _make(500, 64, 4, mask=True)
    want = r.balance_loss(l, ids, 1.0, None, m)
    dwant = r.balance_backward(l, want[2], None, None, m)
    bad = l.clone()
    bad[~m] = float("nan")
    ids2 = ids.clone()
    ids2[~m] = 3
    got = r.balance_loss(bad, ids2, 1.0, None, m)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(r.balance_backward(bad, got[2], None, None, m), dwant)
    # rows outside every sequence alike
    off = torch.tensor([100, 250, 400], dtype=torch.int32, device="cuda")
    want = r.balance_loss(l, ids, 1.0, off)
    bad = l.clone()
    bad[:100] = float("nan")
    bad[400:] = float("nan")
    got = r.balance_loss(bad, ids, 1.0, off)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    d = r.balance_backward(bad, got[2], None, off)
    assert not d[:100].any() and not d[400:].any() and torch.isfinite(d).all()


def test_undefined_logits_of_counted_rows_show():
    r = _router(64, 4)
    l, ids, _, _, _ = _make(40, 64, 4)
    l[7, 5] = float("nan")
    loss, counts, slope = r.balance_loss(l, ids)
    assert torch.isnan(loss) and torch.isfinite(slope).all()
    d = r.balance_backward(l, slope)
    assert torch.isnan(d[7]).all() and torch.isfinite(d[:7]).all() and torch.isfinite(d[8:]).all()


def test_large_logits():
    g = torch.Generator().manual_seed(3)
    l = (torch.randn(64, 48, generator=g) * 60).cuda()
    ids = torch.rand(64, 48, generator=g).argsort(dim=1)[:, :2].int().cuda()
    for score in ("softmax", "sigmoid"):
        _check(64, 48, 2, score=score, arrays=(l, ids, None, None, torch.zeros_like(l)))
    _, _, (loss, _, _) = _check(64, 48, 2, arrays=(l * 1e30, ids, None, None, torch.zeros_like(l)))
    assert torch.isfinite(loss)


def test_gradient_by_differences():
    """The loss itself, differenced in 64 bits on the host, along a direction."""
    T, E, K = 33, 24, 3
    for score in ("softmax", "sigmoid"):
        r = _router(E, K, score)
        l, ids, off, m, _ = _make(T, E, K, S=3, mask=True, seed=5)
        _, _, slope = r.balance_loss(l, ids, 1.0, off, m)
        d = _np(r.balance_backward(l, slope, None, off, m))
        way = np.random.default_rng(0).standard_normal((T, E))
        at = lambda e: ot.balance(_np(l) + e * way, ids.cpu().numpy(), 1.0, score, off.cpu().numpy(),  # noqa: E731
                                  m.cpu().numpy())[0][0]
        num = (at(1e-4) - at(-1e-4)) / 2e-4
        # (third differences: 1e-8 of the curvature; FP32 gradient: 2^-20 of its terms)
        assert abs((d * way).sum() - num) <= 1e-6 * np.abs(d * way).sum() + 1e-9


def test_in_place_and_repeated():
    r, (l, ids, off, m, add), (loss, counts, slope) = _check(5000, 160, 6, BF16, S=7, mask=True)
    want = r.balance_backward(l, slope, None, off, m, add)
    again = r.balance_loss(l, ids, 0.3, off, m)
    assert torch.equal(again[0], loss) and torch.equal(again[2], slope)
    into = add.clone()
    assert r.balance_backward(l, slope, None, off, m, into, dlogits=into) is into
    assert torch.equal(into, want)
    over = l.clone()
    r.balance_backward(over, slope, None, off, m, add, dlogits=over)
    assert torch.equal(over, want)


def test_captured_and_on_another_stream():
    r, (l, ids, off, m, add), (loss, counts, slope) = _check(2000, 64, 4, S=4, mask=True)
    d = r.balance_backward(l, slope, None, off, m, add)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = r.balance_loss(l, ids, 0.3, off, m, stream=side)
    gd = r.balance_backward(l, got[2], None, off, m, add, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], loss) and torch.equal(got[2], slope) and torch.equal(gd, d)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = r.balance_loss(l, ids, 0.3, off, m)
            od = r.balance_backward(l, out[2], None, off, m, add)
        graphs.append((graph, out, od))
    l2 = l.clone()
    l.mul_(0.5)
    want = r.balance_loss(l, ids, 0.3, off, m)
    wd = r.balance_backward(l, want[2], None, off, m, add)
    for graph, out, od in graphs:
        graph.replay()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, want)) and torch.equal(od, wd)
    l.copy_(l2)


def test_refusals():
    r = _router(32, 4)
    l, ids, _, m, add = _make(16, 32, 4)
    m = torch.ones(16, dtype=torch.bool, device="cuda")
    off = torch.tensor([0, 16], dtype=torch.int32, device="cuda")
    slope = torch.zeros(1, 32, device="cuda")
    for bad in (dict(ids=ids[:, :3]), dict(ids=ids.long()), dict(mask=m[:3]), dict(offsets=off.long()),
                dict(offsets=off[:1]), dict(coefficient=float("nan")), dict(logits=l.cpu()), dict(logits=l.double())):
        kw = dict(logits=l, ids=ids)
        kw.update(bad)
        with pytest.raises((ValueError, RuntimeError)):
            r.balance_loss(**kw)
    for bad in (dict(slope=slope[:, :8]), dict(slope=slope.double()), dict(offsets=torch.cat([off, off[1:]])),
                dict(add=add[:4]), dict(add=add.bfloat16()), dict(dlogits=add[:, :3]),
                dict(dloss=torch.zeros(2, device="cuda"))):
        kw = dict(logits=l, slope=slope)
        kw.update(bad)
        with pytest.raises((ValueError, RuntimeError)):
            r.balance_backward(**kw)
    both = torch.zeros(17, 32, device="cuda")
    with pytest.raises(RuntimeError, match="ALIAS"):
        r.balance_backward(both[:16], slope, dlogits=both[1:])
