"""Low-rank adapters and their gradients on the GPU against the 64-bit oracle.

Tolerances (set before the first run).  A sum of n products of 16-bit values in
the tensor cores takes n / 16 steps of at most 2^-22 of the terms' absolute sum
(products are exact, a step adds 16 of them to an FP32 sum and may truncate),
the parts of a split axis some 40 FP32 additions.  hidden enters the second
product as two 16-bit parts: 2^-17 of its terms, and with FP16, whose parts share
a power of two a row (or 64 rows), 2^-24 of the largest hidden beside it.  An
output is rounded once, half a step."""

import numpy as np
import pytest
import torch

from oracle import training as ot
from tests.parity import built, gpu, needs_gpu

pytestmark = [gpu, needs_gpu]

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
UNIT = {F16: (2.0 ** -11, 2.0 ** -25), BF16: (2.0 ** -8, 2.0 ** -133)}


def _adapters(K, N, r):
    from nvfp4_token_quantized_gb300 import LowRankAdapters

    built()
    return LowRankAdapters(K, N, r)


def _np(t):
    return None if t is None else t.float().cpu().numpy().astype(np.float64)


def _steps(n):
    return (n / 16 + 40) * 2.0 ** -22


def _close(got, val, tol, what, dtype):
    g = _np(got)
    assert g.shape == val.shape, what
    if dtype != F32:
        half, tiny = UNIT[dtype]
        tol = tol + half * (np.abs(val) + tol) + tiny
        # (a value past the type's largest number is rounded to infinity)
        big = np.isinf(g) & (np.abs(val) + tol >= torch.finfo(dtype).max) & (np.sign(g) == np.sign(val))
        g = np.where(big, val, g)
    assert np.isfinite(g).all(), what
    worst = np.max(np.abs(g - val) / (tol + 1e-37)) if g.size else 0.0
    assert worst <= 1, f"{what}: {worst} times the tolerance"
    # (the bounds above are worst cases; errors of many roundings add up to less)
    norm = np.linalg.norm(val)
    if norm > 0 and val.size > 64 and dtype == F32:
        assert np.linalg.norm(g - val) <= 2e-6 * norm, what


def _make(T, K, N, r, L, dtype, ids=None, pad=0, seed=0, size=1.0):
    g = torch.Generator().manual_seed(seed)

    def rows(w):
        wide = torch.full((T, w + pad), float("nan"))
        wide[:, :w] = torch.randn(T, w, generator=g) * torch.exp(torch.randn(T, 1, generator=g)) * size
        return wide.to(dtype).cuda()[:, :w]

    if ids is None:
        ids = torch.randint(-1, L + 1, (T,), generator=g)
    a = dict(x=rows(K), base=rows(N), dout=rows(N), dbase=rows(K), ids=ids.int().cuda(),
             down=(torch.randn(L, r, K, generator=g) / K ** 0.5).to(dtype).cuda(),
             up=(torch.randn(L, r, N, generator=g) / r ** 0.5).to(dtype).cuda(),
             scales=(torch.rand(L, generator=g) * 3 - 1).cuda())
    return a


def _apply_tol(x_mag, h, hm, up_by_row, n, r, dtype):
    extra = 0.0
    if dtype == F16:
        extra = 2.0 ** -24 * np.abs(h).max(1, initial=0.0, keepdims=True) * up_by_row
    return x_mag * (_steps(n) + _steps(2 * r) + 2.0 ** -17) + extra


def _sum_up(ids, factor):
    s = np.abs(factor).sum(1)
    out = np.zeros((ids.size, factor.shape[2]))
    ok = (ids >= 0) & (ids < factor.shape[0])
    out[ok] = s[ids[ok]]
    return out


def _check(T, K, N, r, L, dtype=BF16, base=True, scales=True, backward=True, arrays=None, **kw):
    ad = _adapters(K, N, r)
    a = arrays or _make(T, K, N, r, L, dtype, **kw)
    b = a["base"] if base else None
    s = a["scales"] if scales else None
    out, hidden = ad.forward(a["x"], a["ids"], a["down"], a["up"], scales=s, base=b, keep_hidden=True)
    assert out.dtype == dtype and hidden.dtype == F32
    ids, dn, un, sn = a["ids"].cpu().numpy(), _np(a["down"]), _np(a["up"]), _np(s)
    ref, h, mag, hm = ot.adapters(_np(a["x"]), ids, dn, un, sn, _np(b))
    _close(hidden, h, hm * _steps(K), "hidden", F32)
    _close(out, ref, _apply_tol(mag, h, hm, _sum_up(ids, un), K, r, dtype), "out", dtype)
    none = (ids < 0) | (ids >= L)
    assert np.array_equal(_np(out)[none], _np(b)[none] if base else np.zeros((none.sum(), N)))
    if not backward:
        return ad, a, out, hidden
    db = a["dbase"] if base else None
    got = ad.backward(a["dout"], a["x"], hidden, a["ids"], a["down"], a["up"], scales=s, base=db)
    (dx, dd, du), (mx, md, mu) = ot.adapters_backward(_np(a["dout"]), _np(a["x"]), _np(hidden), ids, dn, un, sn, _np(db))
    _, v, _, vm = ot.adapters(_np(a["dout"]), ids, un, dn, sn)
    _close(got[0], dx, _apply_tol(mx, v, vm, _sum_up(ids, dn), N, r, dtype), "dx", dtype)
    ed = eu = 0.0
    if dtype == F16:
        ed = 2.0 ** -24 * np.abs(v).max(initial=0.0) * np.abs(_np(a["x"])).sum(0)[None, None, :]
        eu = 2.0 ** -24 * np.abs(_np(hidden)).max(initial=0.0) * np.abs(_np(a["dout"])).sum(0)[None, None, :]
    _close(got[1], dd, md * (_steps(N) + _steps(2 * T) + 2.0 ** -17) + ed, "ddown", dtype)
    _close(got[2], du, mu * (_steps(2 * T) + 2.0 ** -17) + eu, "dup", dtype)
    for i in range(L):
        if not (ids == i).any():
            assert not got[1][i].any() and not got[2][i].any()
    return ad, a, out, hidden


@pytest.mark.parametrize("r", [1, 2, 7, 8, 9, 16, 17, 24, 31, 32, 40, 48, 50, 64, 65, 100, 128])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_ranks(r, dtype):
    _check(40, 256, 320, r, 3, dtype)
    _check(333, 264, 136, r, 4, dtype)
    _check(600, 264, 136, r, 4, dtype, backward=False)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 64, 65, 127, 128, 129, 256, 257, 300, 512, 513, 1000])
def test_lengths(T):
    for L in (1, 5, 40):
        _check(T, 512, 256, 16, L)


@pytest.mark.parametrize("K,N", [(1, 1), (1, 70), (7, 9), (8, 8), (31, 33), (32, 64), (100, 200), (513, 65), (1000, 1001),
                                 (2048, 768), (72, 4096)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_widths(K, N, dtype):
    _check(50, K, N, 8, 3, dtype)
    _check(200, K, N, 20, 3, dtype)
    _check(520, K, N, 20, 3, dtype, backward=False)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_strides(dtype):
    for pad in (1, 3, 8, 64):
        _check(77, 128, 192, 16, 4, dtype, pad=pad)
        _check(200, 129, 192, 16, 4, dtype, pad=pad)
        _check(520, 129, 192, 16, 4, dtype, pad=pad, backward=False)
        _check(530, 128, 192, 16, 4, dtype, pad=pad, backward=False)


def test_operands_that_may_be_absent():
    for base in (False, True):
        for scales in (False, True):
            _check(60, 256, 256, 16, 4, base=base, scales=scales)
            _check(260, 256, 256, 16, 4, F16, base=base, scales=scales)
            _check(530, 256, 256, 16, 4, F16, base=base, scales=scales, backward=False)


def test_who_has_which_adapter():
    T = 700
    one = torch.full((T,), 2)
    runs = torch.arange(T) * 6 // T
    for ids in (one, runs, torch.full((T,), -1), torch.full((T,), 1 << 30), runs.flip(0), torch.arange(T) % 5,
                torch.arange(T) - 300):
        _check(T, 256, 128, 16, 6, ids=ids)
        _check(90, 256, 128, 16, 6, F16, ids=ids[:90])
        for n in (48, 129, 300, 500):  # (tiles of one adapter, beside those that it does not fill)
            for L in (6, 300):
                _check(n, 256, 128, 16, L, ids=ids[:n], backward=False)
    _check(300, 64, 64, 4, 1000)  # more adapters than rows


def test_long_batches():
    _check(5000, 512, 640, 32, 7, ids=torch.randint(0, 7, (5000,)))
    _check(20000, 128, 64, 16, 3, F16, ids=torch.arange(20000) // 7000)
    _check(17000, 64, 72, 8, 40)


def test_wide_projections():
    _check(30, 20000, 10000, 16, 2)


def test_no_rows():
    ad = _adapters(64, 128, 8)
    a = _make(0, 64, 128, 8, 3, BF16)
    out, hidden = ad.forward(a["x"], a["ids"], a["down"], a["up"], base=a["base"], keep_hidden=True)
    assert out.shape == (0, 128) and hidden.shape == (0, 8)
    dx, dd, du = ad.backward(a["dout"], a["x"], hidden, a["ids"], a["down"], a["up"])
    assert dx.shape == (0, 64) and not dd.any() and not du.any()


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_hidden_past_the_types_range(dtype):
    """Large rows and factors: hidden near the end of FP16's range and far
    beyond it; and tiny ones."""
    for T, size in ((50, 30.0), (600, 200.0), (50, 200.0)):
        a = _make(T, 256, 128, 16, 2, dtype, size=size)
        a["down"] = (a["down"].float() * 300).to(dtype)
        a["up"] = (a["up"].float() * 1e-3).to(dtype)
        _, _, _, hidden = _check(T, 256, 128, 16, 2, dtype, arrays=a)
    assert hidden.abs().max() > 1e5
    a = _make(300, 256, 128, 16, 2, dtype, size=1e-3)
    a["down"] = (a["down"].float() * 1e-2).to(dtype)
    a["dout"] = (a["dout"].float() * 1e3).to(dtype)
    _check(300, 256, 128, 16, 2, dtype, arrays=a)


def test_rows_do_not_mix():
    """Values that are no numbers stay in their row and, for the factors'
    gradients, their adapter."""
    for T in (60, 400, 700):
        ad, a, out, hidden = _check(T, 256, 128, 16, 4, ids=torch.arange(T) % 5 - 1)
        bad = a["x"].clone()
        row = 7
        bad[row, 3] = float("nan")
        o2, h2 = ad.forward(bad, a["ids"], a["down"], a["up"], scales=a["scales"], base=a["base"], keep_hidden=True)
        keep = torch.arange(T, device="cuda") != row
        assert torch.equal(o2[keep], out[keep]) and torch.isnan(o2[row]).all() and torch.isnan(h2[row]).all()
        up = a["up"].clone()
        up[2, 0, 5] = float("inf")
        o3, _ = ad.forward(a["x"], a["ids"], a["down"], up, scales=a["scales"], base=a["base"])
        other = a["ids"] != 2
        assert torch.equal(o3[other], out[other]) and not torch.isfinite(o3[~other][:, 5]).any()
        want = ad.backward(a["dout"], a["x"], hidden, a["ids"], a["down"], a["up"])
        # a row without an adapter may hold anything
        bad = a["x"].clone()
        bad[a["ids"] < 0] = float("nan")
        got = ad.backward(a["dout"], bad, hidden, a["ids"], a["down"], a["up"])
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_in_place_and_repeated():
    for T, dtype in ((50, BF16), (300, BF16), (900, F16)):
        ad, a, out, hidden = _check(T, 256, 256, 16, 4, dtype)
        for _ in range(2):
            again, h2 = ad.forward(a["x"], a["ids"], a["down"], a["up"], scales=a["scales"], base=a["base"],
                                   keep_hidden=True)
            assert torch.equal(again, out) and torch.equal(h2, hidden)
        over = a["base"].clone()
        got, _ = ad.forward(a["x"], a["ids"], a["down"], a["up"], scales=a["scales"], base=over, out=over)
        assert got is over and torch.equal(over, out)
        want = ad.backward(a["dout"], a["x"], hidden, a["ids"], a["down"], a["up"], base=a["dbase"])
        over = a["dbase"].clone()
        got = ad.backward(a["dout"], a["x"], hidden, a["ids"], a["down"], a["up"], base=over, dx=over)
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_rows_behind_the_batch_are_left():
    ad = _adapters(64, 96, 8)
    a = _make(40, 64, 96, 8, 2, BF16)
    wide = torch.full((60, 128), 5.0, dtype=BF16, device="cuda")
    ad.forward(a["x"], a["ids"], a["down"], a["up"], out=wide[:40, :96])
    assert bool((wide[40:] == 5).all()) and bool((wide[:, 96:] == 5).all())


def test_captured_and_on_another_stream():
    for T in (64, 300, 1000):
        ad, a, out, hidden = _check(T, 256, 192, 16, 4)
        want = ad.backward(a["dout"], a["x"], hidden, a["ids"], a["down"], a["up"], scales=a["scales"])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        o, _ = ad.forward(a["x"], a["ids"], a["down"], a["up"], scales=a["scales"], base=a["base"], stream=side)
        b = ad.backward(a["dout"], a["x"], hidden, a["ids"], a["down"], a["up"], scales=a["scales"], stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(o, out) and all(torch.equal(p, q) for p, q in zip(b, want))
        ws = torch.empty(ad.workspace_bytes(T, 4, True), dtype=torch.uint8, device="cuda")  # shared by both graphs
        graphs = []
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                o, h = ad.forward(a["x"], a["ids"], a["down"], a["up"], scales=a["scales"], base=a["base"],
                                  keep_hidden=True, workspace=ws)
                b = ad.backward(a["dout"], a["x"], h, a["ids"], a["down"], a["up"], scales=a["scales"], workspace=ws)
            graphs.append((graph, o, b))
        a["ids"].copy_(a["ids"].flip(0))
        o2, h2 = ad.forward(a["x"], a["ids"], a["down"], a["up"], scales=a["scales"], base=a["base"], keep_hidden=True)
        b2 = ad.backward(a["dout"], a["x"], h2, a["ids"], a["down"], a["up"], scales=a["scales"])
        for graph, o, b in graphs:
            graph.replay()
            graph.replay()
            assert torch.equal(o, o2) and all(torch.equal(p, q) for p, q in zip(b, b2))


def test_refusals():
    ad = _adapters(64, 96, 8)
    a = _make(40, 64, 96, 8, 2, BF16)
    ok = dict(x=a["x"], ids=a["ids"], down=a["down"], up=a["up"], scales=a["scales"], base=a["base"])
    for bad in (dict(x=a["base"]), dict(x=a["x"].float()), dict(x=a["x"].cpu()), dict(ids=a["ids"].long()),
                dict(ids=a["ids"][:3]), dict(down=a["up"]), dict(down=a["down"][0]), dict(up=a["up"][:1]),
                dict(up=a["up"].half()), dict(down=a["down"].transpose(1, 2)), dict(scales=a["scales"][:1]),
                dict(base=a["x"]), dict(out=a["x"])):
        with pytest.raises((ValueError, RuntimeError, TypeError)):
            ad.forward(**{**ok, **bad})
    wide = torch.zeros(41, 96, dtype=BF16, device="cuda")
    for bad in (dict(out=a["up"].view(-1)[:40 * 96 - 0].view(-1)[:8 * 96].view(8, 96), x=a["x"][:8], ids=a["ids"][:8],
                     base=None), dict(base=wide[:40], out=wide[1:])):
        with pytest.raises(RuntimeError, match="ALIAS"):
            ad.forward(**{**ok, **bad})
    with pytest.raises(RuntimeError):
        _adapters(64, 96, 129)
    with pytest.raises(RuntimeError):
        _adapters(0, 96, 8)
    b = _make(600, 64, 96, 8, 2, BF16)
    with pytest.raises(ValueError, match="workspace"):
        ad.forward(b["x"], b["ids"], b["down"], b["up"], workspace=torch.zeros(2, device="cuda"))
    _, h = ad.forward(**ok, keep_hidden=True)
    okb = dict(dout=a["dout"], x=a["x"], hidden=h, ids=a["ids"], down=a["down"], up=a["up"])
    for bad in (dict(hidden=None), dict(hidden=h[:3]), dict(hidden=h.half()), dict(dout=a["x"]), dict(base=a["dout"]),
                dict(dx=a["dout"])):
        with pytest.raises((ValueError, RuntimeError)):
            ad.backward(**{**okb, **bad})
    with pytest.raises(RuntimeError, match="ALIAS"):
        ad.backward(**{**okb, "dx": a["x"]})
