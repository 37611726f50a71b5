"""The norms around a block and their gradient on the GPU against the 64-bit
oracle.

Tolerances (set before the first run): each result is formed in FP32 from
terms whose absolute values sum to ``mag`` (oracle/block.py), through sums
of at most 16 values a thread, 10 levels of trees, a root, a quotient and a
handful of products: within 48 * 2^-24 of mag.  Column sums add a run of rows
first; the row counts here keep them inside the same bound.  An output of
fewer bits adds one rounding (half a unit in the last place, and its smallest
number).
"""

import numpy as np
import pytest
import torch

from oracle import block as ob
from tests.parity import built, gpu, needs_gpu

pytestmark = [gpu, needs_gpu]

U = 2.0 ** -24
UNIT = {torch.float32: (U, 2.0 ** -149), torch.float16: (2.0 ** -11, 2.0 ** -25),
        torch.bfloat16: (2.0 ** -8, 2.0 ** -133)}
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def _norm(H, **kw):
    from nvfp4_token_quantized_gb300 import BlockNorm

    built()
    return BlockNorm(H, **kw)


def _np(t):
    return None if t is None else t.float().cpu().numpy().astype(np.float64)


def _close(got, ref, what, dtype=None):
    val, mag = ref
    dtype = got.dtype if dtype is None else dtype
    g = _np(got).reshape(val.shape)
    u, tiny = UNIT[dtype]
    tol = 48 * U * mag + (u * np.abs(val) if dtype != F32 else 0) + tiny + 1e-37
    assert np.isfinite(g).all(), what
    worst = np.max(np.abs(g - val) / tol)
    assert worst <= 1, f"{what}: {worst} times the tolerance"


def _make(T, H, dtype, rdtype, wdtype, gate, post, pre, pad=0, seed=0, zeros=True):
    g = torch.Generator().manual_seed(seed)

    def rows(dt, size=1.0):
        x = torch.randn(T, H, generator=g) * size * torch.exp(torch.randn(T, 1, generator=g))
        x[:, ::97] *= 10.0
        if zeros and T > 3:
            x[3] = 0.0
        wide = torch.full((T, H + pad), 77.0)
        wide[:, :H] = x
        return wide.to(dt).cuda()[:, :H]

    shape = {"channel": (H,), "token": (T, 1), "full": (T, H)}.get(gate)
    a = dict(residual=rows(rdtype), y=rows(dtype), dres=rows(rdtype, 0.5), dh=rows(dtype))
    a["gate"] = None if shape is None else torch.randn(*shape, generator=g).to(dtype).cuda()
    a["wp"] = (1 + 0.3 * torch.randn(H, generator=g)).to(wdtype).cuda() if post else None
    a["wn"] = (1 + 0.3 * torch.randn(H, generator=g)).to(wdtype).cuda() if pre else None
    return a


def _gate2d(gate, kind):
    g = _np(gate)
    return None if g is None else g[None, :] if kind == "channel" else g


def _check(T, H, dtype=BF16, rdtype=None, wdtype=None, kind="rms", gate=None, gate_sigmoid=False, post=True, pre=True,
           offset=0.0, scale=1.0, eps=1e-5, pad=0, seed=0, arrays=None, backward=True):
    rdtype, wdtype = rdtype or dtype, wdtype or dtype
    n = _norm(H, kind=kind, eps=eps, post=post, pre=pre, gate=gate, gate_sigmoid=gate_sigmoid, weight_offset=offset,
              branch_scale=scale)
    a = arrays or _make(T, H, dtype, rdtype, wdtype, gate, post, pre, pad, seed)
    eps32, off32, scale32 = (float(np.float32(v)) for v in (eps, offset, scale))
    kw = dict(kind=kind, eps=eps32, post=post, pre=pre, gate_sigmoid=gate_sigmoid, offset=off32, scale=scale32)
    out, h = n.forward(a["residual"], a["y"], gate=a["gate"], post_weight=a["wp"], pre_weight=a["wn"])
    assert out.dtype == rdtype and out.shape == (T, H) and (h is None) == (not pre)
    g2 = _gate2d(a["gate"], gate)
    ref, refh = ob.block_norm(_np(a["residual"]), _np(a["y"]), g2, _np(a["wp"]), _np(a["wn"]), **kw)
    _close(out, ref, "residual_out")
    if pre:
        assert h.dtype == dtype
        _close(h, refh, "h")
    if not backward:
        return n, a, out, h
    grads = n.backward(a["dres"], a["dh"] if pre else None, out, a["y"], gate=a["gate"], post_weight=a["wp"],
                       pre_weight=a["wn"])
    refg = ob.block_norm_backward(_np(a["dres"]), _np(a["dh"]), _np(out), _np(a["y"]), g2, _np(a["wp"]), _np(a["wn"]),
                                  **kw)
    _compare_grads(grads, refg, (rdtype, dtype, F32 if gate == "channel" else dtype, F32, F32))
    return n, a, out, h


NAMES = ("residual", "y", "gate", "post_weight", "pre_weight")


def _compare_grads(grads, refg, dtypes):
    for name, got, dt in zip(NAMES, grads, dtypes):
        assert (got is None) == (name not in refg), name
        if got is not None:
            assert got.dtype == dt, name
            _close(got, refg[name], "d" + name)


@pytest.mark.parametrize("dtype,rdtype,wdtype", [(BF16, BF16, BF16), (BF16, F32, F32), (F16, F16, F32), (F16, F32, F16),
                                                 (F32, F32, F32)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_types(dtype, rdtype, wdtype, kind):
    for gate in (None, "channel", "token", "full"):
        _check(9, 520, dtype, rdtype, wdtype, kind, gate, gate_sigmoid=gate == "token", offset=0.5, scale=0.22)


@pytest.mark.parametrize("H", [1, 2, 7, 8, 31, 64, 255, 256, 257, 1000, 2047, 2048, 4096, 4100, 7168, 8192, 8193, 8200,
                               11264, 16383, 16384])
def test_widths(H):
    _check(5, H)
    _check(5, H, kind="layer", gate="channel", rdtype=F32)


@pytest.mark.parametrize("T", [1, 2, 3, 64, 151, 305, 700])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_token_counts(T, kind):
    _check(T, 264, kind=kind, gate="channel")
    _check(T, 61, kind=kind, gate="full", dtype=F16)


@pytest.mark.parametrize("post,pre", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("gate,sig", [(None, False), ("channel", True), ("token", False), ("token", True),
                                      ("full", True)])
def test_parts(post, pre, gate, sig):
    for kind in ("rms", "layer"):
        _check(11, 136, kind=kind, gate=gate, gate_sigmoid=sig, post=post, pre=pre, scale=-1.5, offset=1.0)
        _check(11, 37, kind=kind, gate=gate, gate_sigmoid=sig, post=post, pre=pre, dtype=F32)


@pytest.mark.parametrize("pad", [1, 4, 8, 24])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides(pad, dtype):
    _check(6, 512, dtype, pad=pad, gate="token")
    _check(6, 512, dtype, rdtype=F32, pad=pad, kind="layer")


def test_full_gate_with_row_stride():
    a = _make(6, 128, BF16, BF16, BF16, "full", True, True)
    a["gate"] = torch.cat([a["gate"], a["gate"]], 1)[:, 64:192]
    _check(6, 128, gate="full", arrays=a)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("H", [96, 2048, 50])
def test_pre_norm_alone(kind, H):
    for dtype, hd in ((BF16, None), (F32, BF16), (F16, None), (F32, None)):
        n = _norm(H, kind=kind, eps=1e-5, post=True, pre=True, gate="token")
        a = _make(7, H, hd or dtype, dtype, hd or dtype, None, False, True)
        h_in = None if hd is None else torch.empty(7, H, dtype=hd, device="cuda")
        none, h = n.forward(a["residual"], pre_weight=a["wn"], h=h_in)
        assert none is None and (h_in is None or h is h_in)
        eps = float(np.float32(1e-5))
        _, ref = ob.block_norm(_np(a["residual"]), wn=_np(a["wn"]), kind=kind, eps=eps)
        _close(h, ref, "h")
        for dres in (a["dres"], None):
            grads = n.backward(dres, a["dh"], a["residual"], pre_weight=a["wn"])
            refg = ob.block_norm_backward(_np(dres), _np(a["dh"]), _np(a["residual"]), wn=_np(a["wn"]), kind=kind,
                                          eps=eps)
            _compare_grads(grads, refg, (dtype, None, None, None, F32))


def test_no_weights():
    n = _norm(200, kind="layer", eps=1e-5, weight_offset=3.0)
    a = _make(5, 200, BF16, F32, F32, None, False, False)
    out, h = n.forward(a["residual"], a["y"])
    kw = dict(kind="layer", eps=float(np.float32(1e-5)))
    ref, refh = ob.block_norm(_np(a["residual"]), _np(a["y"]), **kw)
    _close(out, ref, "residual_out")
    _close(h, refh, "h")
    grads = n.backward(a["dres"], a["dh"], out, a["y"])
    refg = ob.block_norm_backward(_np(a["dres"]), _np(a["dh"]), _np(out), _np(a["y"]), **kw)
    del refg["post_weight"], refg["pre_weight"]
    _compare_grads(grads, refg, (F32, BF16, None, None, None))


def test_far_off_centre():
    # a mean a thousand times the spread: statistics by differences of sums
    # would lose it all
    a = _make(6, 1024, F32, F32, F32, None, True, True, zeros=False)
    for k in ("residual", "y"):
        a[k] = a[k] + 1000.0
    _check(6, 1024, F32, kind="layer", arrays=a)
    a = _make(6, 1001, F32, F32, F32, None, True, True, zeros=False)
    a["y"] = a["y"] * 0.01 - 300.0
    _check(6, 1001, F32, kind="layer", arrays=a)


def test_tiny_and_huge_rows():
    for size in (1e-12, 1e12):
        a = _make(6, 512, F32, F32, F32, None, True, True)
        a["y"] = a["y"] * size
        _check(6, 512, F32, arrays=a, eps=1e-6)


def test_infinities_and_nan_stay_in_their_row():
    n = _norm(512)
    a = _make(6, 512, BF16, BF16, BF16, None, True, True)
    ref = n.forward(a["residual"], a["y"], post_weight=a["wp"], pre_weight=a["wn"])
    y = a["y"].clone()
    y[1, 5], y[4, 500] = float("nan"), float("inf")
    got = n.forward(a["residual"], y, post_weight=a["wp"], pre_weight=a["wn"])
    keep = [0, 2, 3, 5]
    for r, g in zip(ref, got):
        assert torch.equal(r[keep], g[keep])
        assert torch.isnan(g[1]).all() and not torch.isfinite(g[4].float()).all()


def test_in_place():
    n = _norm(512, gate="token")
    a = _make(40, 512, BF16, BF16, BF16, "token", True, True)
    w = dict(gate=a["gate"], post_weight=a["wp"], pre_weight=a["wn"])
    out, h = n.forward(a["residual"], a["y"], **w)
    r, y = a["residual"].clone(), a["y"].clone()
    o2, h2 = n.forward(r, y, residual_out=r, h=y, **w)
    assert o2 is r and h2 is y and torch.equal(o2, out) and torch.equal(h2, h)
    ref = n.backward(a["dres"], a["dh"], out, a["y"], **w)
    for over in ("dh", "y"):
        d = {k: a[k].clone() for k in ("dres", "dh", "y")}
        got = n.backward(d["dres"], d["dh"], out, d["y"], dresidual=d["dres"], dy=d[over], **w)
        for x, z in zip(ref, got):
            assert torch.equal(x, z)
    # outputs beside their inputs in one wider array
    wide = torch.empty(40, 1024, dtype=BF16, device="cuda")
    wide[:, :512] = a["residual"]
    o3, _ = n.forward(wide[:, :512], a["y"], residual_out=wide[:, 512:], **w)
    assert torch.equal(o3, out)


def test_repeats_bit_for_bit():
    for T, H, kind in ((1000, 512, "rms"), (333, 1001, "layer"), (500, 8192, "rms")):
        n = _norm(H, kind=kind, gate="channel")
        a = _make(T, H, BF16, F32, F32, "channel", True, True)
        w = dict(gate=a["gate"], post_weight=a["wp"], pre_weight=a["wn"])
        out, _ = n.forward(a["residual"], a["y"], **w)
        first = n.backward(a["dres"], a["dh"], out, a["y"], **w)
        for _ in range(3):
            for x, z in zip(first, n.backward(a["dres"], a["dh"], out, a["y"], **w)):
                assert torch.equal(x, z)


def test_rows_do_not_depend_on_the_batch():
    # one token alone gives the bits it gives in a batch
    for T, H in ((2000, 2048), (300, 8192), (500, 1000)):
        n = _norm(H)
        a = _make(T, H, BF16, BF16, BF16, None, True, True)
        out, h = n.forward(a["residual"], a["y"], post_weight=a["wp"], pre_weight=a["wn"])
        o1, h1 = n.forward(a["residual"][7:8], a["y"][7:8], post_weight=a["wp"], pre_weight=a["wn"])
        assert torch.equal(o1, out[7:8])
        err = (h1.float() - h[7:8].float()).abs()
        assert (err <= 2.0 ** -7 * h1.float().abs()).all()


def test_gradient_against_differences():
    for kind, gate in (("rms", "channel"), ("layer", "token")):
        T, H = 12, 200
        n, a, out, _ = _check(T, H, F32, kind=kind, gate=gate, gate_sigmoid=True, offset=1.0, scale=0.5)
        grads = n.backward(a["dres"], a["dh"], out, a["y"], gate=a["gate"], post_weight=a["wp"], pre_weight=a["wn"])
        kw = dict(kind=kind, eps=float(np.float32(1e-5)), gate_sigmoid=True, offset=1.0, scale=0.5)
        base = [_np(a["residual"]), _np(a["y"]), _gate2d(a["gate"], gate), _np(a["wp"]), _np(a["wn"])]
        rng = np.random.default_rng(1)

        def loss(x):
            (r, _), (h, _) = ob.block_norm(*x, **kw)
            return (r * _np(a["dres"])).sum() + (h * _np(a["dh"])).sum()

        for i, g in enumerate(grads):
            d = rng.standard_normal(base[i].shape) * np.abs(base[i])
            plus, minus = list(base), list(base)
            plus[i], minus[i] = base[i] + 1e-5 * d, base[i] - 1e-5 * d
            diff = (loss(plus) - loss(minus)) / 2e-5
            terms = _np(g).reshape(d.shape) * d
            assert abs(terms.sum() - diff) <= 1e-4 * np.abs(terms).sum(), NAMES[i]


def test_zero_tokens():
    n = _norm(64, gate="channel")
    e = torch.empty(0, 64, dtype=BF16, device="cuda")
    w = torch.ones(64, dtype=BF16, device="cuda")
    out, h = n.forward(e, e, gate=w, post_weight=w, pre_weight=w)
    assert out.shape == h.shape == (0, 64)
    grads = n.backward(e, e, out, e, gate=w, post_weight=w, pre_weight=w)
    assert grads[0].shape == (0, 64)
    for g in grads[2:]:
        assert (g == 0).all() and g.numel() == 64


def test_other_stream_and_graph():
    n = _norm(1024)
    a = _make(100, 1024, BF16, BF16, BF16, None, True, True)
    w = dict(post_weight=a["wp"], pre_weight=a["wn"])
    ref = n.forward(a["residual"], a["y"], **w)
    refg = n.backward(a["dres"], a["dh"], ref[0], a["y"], **w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = n.forward(a["residual"], a["y"], stream=s, **w)
    gotg = n.backward(a["dres"], a["dh"], got[0], a["y"], stream=s.cuda_stream, **w)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = n.forward(a["residual"], a["y"], **w)
        capg = n.backward(a["dres"], a["dh"], cap[0], a["y"], **w)
    g.replay()
    torch.cuda.synchronize()
    for x, z in zip(ref + refg, got + gotg):
        assert x is None and z is None or torch.equal(x, z)
    for x, z in zip(ref + refg, cap + capg):
        assert x is None and z is None or torch.equal(x, z)


def test_rows_past_32_bits():
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    T, H, ld = 3, 512, 1 << 30
    base = torch.empty(2 * ld + H, dtype=BF16, device="cuda")
    a = _make(T, H, BF16, BF16, BF16, None, True, True)
    far = base.as_strided((T, H), (ld, 1))
    far.copy_(a["y"])
    a["y"] = far
    _check(T, H, arrays=a)


def test_refusals():
    from nvfp4_token_quantized_gb300 import BlockNorm, MoEError

    built()
    for bad in (dict(hidden=0), dict(hidden=16392), dict(hidden=64, eps=0.0), dict(hidden=64, eps=float("nan")),
                dict(hidden=64, branch_scale=float("inf"))):
        with pytest.raises(MoEError):
            BlockNorm(**bad)
    for bad in (dict(kind="batch"), dict(gate="row")):
        with pytest.raises(ValueError):
            BlockNorm(64, **bad)
    n = _norm(64)
    r = torch.zeros(4, 64, dtype=BF16, device="cuda")
    w = torch.ones(64, dtype=BF16, device="cuda")
    for args, kw in (((r.cpu(), r), {}), ((r, r[:3]), {}), ((r, r[:, :60]), {}), ((r.half(), r), {}),
                     ((r.double(), r.double()), {}), ((r, r), dict(pre_weight=w[:63])),
                     ((r, r), dict(post_weight=w, pre_weight=w.float())), ((r, r), dict(pre_weight=w.half())),
                     ((r[0], r[0]), {})):
        with pytest.raises(ValueError):
            n.forward(*args, **kw)
    with pytest.raises(ValueError):
        _norm(64, pre=False).forward(r)
    with pytest.raises(TypeError):
        _norm(64, gate="full").forward(r, r)
    y = torch.zeros(4, 64, dtype=BF16, device="cuda")
    with pytest.raises(MoEError) as e:
        n.forward(r, y, residual_out=y)
    assert e.value.status == 5
    big = torch.zeros(5, 64, dtype=BF16, device="cuda")
    with pytest.raises(MoEError) as e:
        n.forward(big[:4], y, residual_out=big[1:])
    assert e.value.status == 5
    with pytest.raises(MoEError) as e:
        n.backward(r, y, big[:4], r.clone(), dresidual=big[:4])
    assert e.value.status == 5
    with pytest.raises(ValueError):
        n.backward(r, y, big[:4], r.clone(), post_weight=w, pre_weight=w,
                   workspace=torch.zeros(8, device="cuda"))


@pytest.mark.parametrize("H", [17, 250, 511, 700, 1023, 1535, 1801, 3001, 4095, 5001, 6143, 8191])
def test_odd_widths_over_many_rows(H):
    # rows that start anywhere in a 16-byte granule, more of them than CTAs
    T = 700
    _check(T, H, gate="full", rdtype=F32)
    _check(T, H, F16, kind="layer", gate="channel", pad=3, backward=H < 5000)
    if H < 2000:
        _check(T, H, F32, post=False, gate="token")


def test_views_at_every_offset():
    # rows of a view whose base is 2, 4, ... bytes into a granule
    for off in range(1, 9):
        a = _make(50, 264, BF16, BF16, BF16, None, True, True, pad=24)
        for k in ("residual", "y", "dres", "dh"):
            wide = torch.full((50, 300), 55.0, dtype=BF16, device="cuda")
            wide[:, off:off + 264] = a[k]
            a[k] = wide[:, off:off + 264]
        _check(50, 264, arrays=a)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("H", [64, 256, 264, 512, 1024, 2048, 4096, 6144])
def test_many_rows_a_cta(H, kind):
    # more rows than CTAs at every width, so that each CTA walks several
    T = 5000 if H <= 256 else 1500
    _check(T, H, kind=kind, gate="channel", rdtype=F32)
    _check(T, H, kind=kind, gate="token", post=H != 512, pre=H != 1024)
