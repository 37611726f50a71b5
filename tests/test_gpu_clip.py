"""The norm of many gradients and their clipping on the GPU against 64 bits.

Tolerances (set before the first run).  Norm: the squares (one rounding) are
summed over at most 64 values a thread and chunk (two chains) and then in FP32
over a thread's chunks, at most 16 here, the rest in FP64; the root halves a
relative error and rounds once: (1 + 64 + 16) / 2 + 1 < 48 units of 2^-24.
Clipped values: the factor carries the norm's error and three roundings, the
product is rounded once to FP32 and once (half a step) to the type."""

import numpy as np
import pytest
import torch

from tests.parity import built, gpu, needs_gpu

pytestmark = [gpu, needs_gpu]

U = 2.0 ** -24
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
UNIT = {F32: (U, 2.0 ** -149), F16: (2.0 ** -11, 2.0 ** -25), BF16: (2.0 ** -8, 2.0 ** -133)}


def _clip(max_norm=None, eps=1e-6):
    from nvfp4_token_quantized_gb300 import GradientClip

    built()
    return GradientClip(max_norm, eps=eps)


def _norm64(grads):
    return float(torch.stack([t.double().pow(2).sum() for t in grads]).sum().sqrt()) if grads else 0.0


def _check(grads, max_norm, out=None):
    c = _clip(max_norm)
    ref = _norm64(grads)
    before = [t.clone() for t in grads]
    n = c.norm(grads)
    assert n.shape == () and n.dtype == F32
    assert abs(n.item() - ref) <= 48 * U * ref + 2.0 ** -149
    norm, got = c.clip(grads, out=out)
    assert torch.equal(norm, n)
    m32, e32 = float(np.float32(max_norm)), float(np.float32(1e-6))
    f = min(1.0, m32 / (ref + e32))
    for t, b, g in zip(grads, before, got):
        assert g.dtype == b.dtype and g.shape == b.shape
        if out is not None:
            assert torch.equal(t, b)
        val = b.double() * f
        half, tiny = UNIT[b.dtype]
        tol = (54 * U * (f < 1) + half) * val.abs() + tiny
        assert bool(((g.double() - val).abs() <= tol).all())
        if f == 1.0:
            assert torch.equal(g, b)
    return norm, got


def _make(sizes, dtypes, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * scale * 10 ** (3 * torch.rand(1, generator=g) - 2)).to(dtypes[i % len(dtypes)])
            .cuda() for i, n in enumerate(sizes)]


@pytest.mark.parametrize("dtypes", [(F32,), (F16,), (BF16,), (F32, BF16, F16)])
def test_sizes(dtypes):
    for limit in (1e-2, 1e6):
        _check(_make([1], dtypes), limit)
        _check(_make([3, 0, 1, 17, 8, 4097, 16384, 16385, 40000, 255], dtypes), limit)  # one cluster
        _check(_make([1_000_003, 5, 65536, 777_777, 0, 1, 300_000], dtypes), limit)
        _check(_make([n % 37 for n in range(200)], dtypes), limit)                      # a long list
    _check(_make([1000] * 64, dtypes), 0.1)
    _check(_make([1000] * 65, dtypes), 0.1)


def test_more_tensors_than_one_launch_takes():
    for n in (1023, 1024, 1025, 2500):
        _check(_make([100 + i % 50 for i in range(n)], (F32, BF16), seed=n), 0.5)
        _check(_make([100 + i % 50 for i in range(n)], (F16,), seed=n), 1e9)


def test_empty_sets():
    for grads in ([], _make([0, 0], (F32,))):
        norm, got = _clip(1.0).clip(grads)
        assert norm.item() == 0 and len(got) == len(grads)
        assert _clip().norm(grads).item() == 0


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_every_offset_from_sixteen_bytes(dtype):
    g = torch.Generator().manual_seed(1)
    flat = torch.randn(100_000, generator=g).to(dtype).cuda()
    into = torch.empty_like(flat)
    for at in range(9):
        for n in (1, 2, 5, 8, 9, 31, 20_000):
            t, o = flat[at:at + n], into[at:at + n]
            into.fill_(7.0)
            _check([t], 0.01, out=[o])
            assert bool((into[:at] == 7).all()) and bool((into[at + n:] == 7).all())
            o2 = into[at + 3:at + 3 + n]  # (another offset than the data's)
            into.fill_(7.0)
            _check([t], 0.01, out=[o2])
            assert bool((into[:at + 3] == 7).all()) and bool((into[at + 3 + n:] == 7).all())


def test_views_of_one_buffer():
    flat = torch.randn(50_000, device="cuda")
    cuts = [0, 1, 4, 4, 1000, 20_001, 49_000, 50_000]
    _check([flat[a:b] for a, b in zip(cuts, cuts[1:])][::-1], 0.5)


def test_dense_in_any_order():
    t = torch.randn(6, 50, 70, device="cuda").permute(2, 0, 1)
    o = torch.empty(6, 50, 70, device="cuda").permute(2, 0, 1)
    want = t.clone()
    norm, (got,) = _clip(1.0).clip([t], out=[o])
    assert torch.allclose(got, want * min(1.0, 1.0 / (norm.item() + 1e-6)), rtol=1e-6, atol=0)


def test_magnitudes_past_the_squares_range():
    for size in (1e30, 3e37, 1e-30, 1e-38, 1e-44):
        for dtype in (F32, BF16):
            t = [(torch.rand(n, device="cuda") + 0.5).mul(size).to(dtype) for n in (10, 5000, 300_001)]
            ref = _norm64(t)
            got = _clip().norm(t).item()
            if ref < 3.4e38:
                assert abs(got - ref) <= 48 * U * ref + 2.0 ** -149, (size, dtype)
            else:
                assert np.isinf(got)
    # beside ordinary ones
    t = _make([50_000, 3], (F32,)) + [torch.full((40,), 1e25, device="cuda"), torch.zeros(100_000, device="cuda")]
    _check(t, 1.0)
    t = [torch.zeros(1_000_000, device="cuda"), torch.full((1,), 1e-30, device="cuda")]
    _check(t, 1.0)


def test_values_that_are_no_numbers():
    for value, small in ((float("inf"), True), (float("nan"), True), (float("-inf"), False), (float("nan"), False)):
        t = _make([100, 50] if small else [100, 3_000_000], (F32, BF16))
        t[0][7] = value
        norm, got = _clip(1.0).clip(t)
        if np.isnan(value):
            assert torch.isnan(norm) and torch.isnan(got[1]).all()
        else:
            assert torch.isinf(norm) and not got[1].any() and torch.isnan(got[0][7])


def test_limits():
    t = _make([5000], (F32,))
    norm, (g,) = _clip(0.0).clip([t[0].clone()])
    assert not g.any()
    n = _norm64(t)
    for limit in (n * 0.999, n * 1.001):
        _check([t[0].clone()], limit)


def test_the_norm_counts_a_tensor_twice():
    t = _make([5000, 100], (F32,))
    n = _clip().norm([t[0], t[1], t[0]]).item()
    ref = _norm64([t[0], t[1], t[0]])
    assert abs(n - ref) <= 48 * U * ref


def test_repeats_and_graphs_and_streams():
    grads = _make([4_000_000, 33, 1_000_000, 70], (BF16, F32))
    out = [torch.empty_like(t) for t in grads]
    c = _clip(0.5)
    norm, _ = c.clip(grads, out=out)
    want = [t.clone() for t in out]
    for _ in range(3):
        again, _ = c.clip(grads, out=out)
        assert torch.equal(again, norm) and all(torch.equal(a, b) for a, b in zip(out, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    n2, _ = c.clip(grads, out=out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(n2, norm)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gn, _ = c.clip(grads, out=out)
        graphs.append((graph, gn))
    grads[0].mul_(2.0)
    n3, _ = c.clip(grads, out=out)
    want = [t.clone() for t in out]
    for graph, gn in graphs:
        for o in out:
            o.zero_()
        graph.replay()
        graph.replay()
        assert torch.equal(gn, n3) and all(torch.equal(a, b) for a, b in zip(out, want))


def test_refusals():
    t = torch.zeros(64, device="cuda")
    with pytest.raises(ValueError):
        _clip().clip([t])
    for bad in (-1.0, float("inf"), float("nan")):
        with pytest.raises(ValueError):
            _clip(bad)
    with pytest.raises(ValueError):
        _clip(1.0, eps=0.0)
    for bad in ([t.double()], [t.cpu()], [torch.zeros(8, 8, device="cuda")[:, :3]], [t.view(8, 8)[::2]]):
        with pytest.raises(ValueError):
            _clip(1.0).clip(bad)
    with pytest.raises(TypeError):
        _clip(1.0).clip([None])
    for grads, out in (([t], [t, t]), ([t], [t[:3]]), ([t], [t.half()]), ([t.view(8, 8)], [t.view(8, 8).t()])):
        with pytest.raises(ValueError):
            _clip(1.0).clip(grads, out=out)
    big = torch.zeros(200, device="cuda")
    for grads, out in (([t, t], None), ([big[:100], big[50:150]], None), ([big[:100]], [big[50:150]]),
                       ([t, big[:64]], [big[64:128], big[100:164]]), ([t, big[:64]], [big[:64], big[64:128]])):
        with pytest.raises(RuntimeError, match="ALIAS"):
            _clip(1.0).clip(grads, out=out)
