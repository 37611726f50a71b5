"""The choice of experts and its gradient on the GPU against the 64-bit oracle.

Tolerances (set before the first run): ids are equal wherever the 64-bit
choice does not hang on a difference below 4e-6 between values that are not
equal (FP32 scores carry a few times 2^-24 of error); weights agree to
64 * 2^-24 relative, gradients to 64 * 2^-24 of the sum of their terms'
absolute values: exp(x - max) carries |x - max| 2^-24 <= 32 * 2^-24 for the
logits used here, the sums and quotients the rest.  A type of fewer bits adds
one rounding (half a unit in the last place, and its smallest number).
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
NEAR = 4e-6


def _router(E, K, **kw):
    from nvfp4_token_quantized_gb300 import ExpertRouter

    built()
    return ExpertRouter(E, K, **kw)


def _logits(T, E, dtype=torch.float32, seed=0, closed=0.0, pad=0):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, E, generator=g) * 2.0
    if closed:
        l[torch.rand(T, E, generator=g) < closed] = -float("inf")
        l[::7] = -float("inf")                       # rows with nothing open
    wide = torch.full((T, E + pad), 99.0)
    wide[:, :E] = l
    return wide.to(dtype).cuda()[:, :E]


def _bias(E, seed=1):
    g = torch.Generator().manual_seed(seed)
    return ((torch.randn(E, generator=g) * 100).round() / 1000).cuda()


def _unclear(l, K, score, bias, groups, top_groups, group_score):
    """Rows whose choice hangs on less than NEAR."""
    v, g = ob.route_choice(l, score, bias, groups, top_groups, group_score)
    by_score = bias is not None or (groups > 1 and group_score == "top2")
    bad = np.zeros(l.shape[0], bool)
    if not by_score:
        return bad
    with np.errstate(invalid="ignore"):
        top = -np.sort(-v, axis=1)[:, :K + 1]
        gap = top[:, :-1] - top[:, 1:]
        bad |= ((gap > 0) & (gap < NEAR)).any(1)
        if g is not None:
            order = -np.sort(-g, axis=1)
            gap = order[:, top_groups - 1] - order[:, top_groups]
            bad |= (gap > 0) & (gap < NEAR)
    return bad


def _check(T, E, K, dtype=torch.float32, biased=False, seed=0, closed=0.0, pad=0, logits=None, bias=None, **rule):
    l = _logits(T, E, dtype, seed, closed, pad) if logits is None else logits
    b = _bias(E, seed + 1) if biased else bias
    ids, w = _router(E, K, **rule).select(l, bias=b)
    assert ids.shape == w.shape == (l.shape[0], K) and ids.dtype == torch.int32 and w.dtype == torch.float32
    l64, b64 = l.float().cpu().numpy().astype(np.float64), None if b is None else b.cpu().numpy().astype(np.float64)
    score, groups = rule.get("score", "softmax"), rule.get("num_groups", 1)
    args = (groups, rule.get("top_groups", 1), rule.get("group_score", "max"))
    ref_ids, ref_w = ob.route(l64, K, score, b64, *args, rule.get("renormalize", True), rule.get("scale", 1.0))
    clear = ~_unclear(l64, K, score, b64, *args)
    assert clear.mean() > 0.9
    got_ids, got_w = ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    assert np.array_equal(got_ids[clear], ref_ids[clear])
    # every row: distinct ids in range
    assert ((got_ids >= 0) & (got_ids < E)).all()
    assert all(len(set(row)) == K for row in got_ids.tolist())
    err = np.abs(got_w[clear] - ref_w[clear])
    assert np.array_equal(np.isnan(got_w[clear]), np.isnan(ref_w[clear]))
    assert (np.nan_to_num(err) <= 64 * U * np.abs(np.nan_to_num(ref_w[clear])) + 1e-38).all()
    return ids, w


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("E,K", [(1, 1), (3, 2), (31, 5), (32, 32), (33, 8), (97, 7), (128, 8), (129, 1), (256, 8),
                                 (257, 16), (510, 32), (512, 10)])
def test_no_groups(E, K, dtype):
    for score in ("softmax", "sigmoid"):
        _check(37, E, K, dtype, score=score, renormalize=K > 1, scale=2.5)
        _check(37, E, K, dtype, score=score, biased=True, renormalize=False)


@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("E,G,top", [(8, 8, 3), (12, 4, 2), (60, 20, 7), (96, 6, 1), (160, 8, 3), (256, 8, 4),
                                     (255, 17, 5), (510, 17, 16), (512, 32, 9), (512, 2, 1), (64, 1, 1), (64, 4, 4)])
def test_groups(E, G, top, group_score):
    K = min(8, top * (E // G))
    for score in ("softmax", "sigmoid"):
        for biased in (False, True):
            _check(41, E, K, biased=biased, score=score, num_groups=G, top_groups=top, group_score=group_score)


@pytest.mark.parametrize("T", [0, 1, 2, 8, 63, 1000])
def test_token_counts(T):
    if T == 0:
        ids, w = _router(256, 8).select(_logits(1, 256)[:0])
        assert ids.shape == w.shape == (0, 8)
        return
    _check(T, 256, 8, biased=True, score="sigmoid", num_groups=8, top_groups=4, group_score="top2", scale=2.5)


@pytest.mark.parametrize("pad", [1, 2, 4, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides(pad, dtype):
    _check(33, 128, 8, dtype, pad=pad)
    _check(33, 100, 8, dtype, pad=pad, num_groups=5, top_groups=3)


def test_offset_rows_are_not_aligned():
    l = _logits(20, 131)
    for o in range(1, 4):
        _check(20, 128, 8, logits=l[:, o:o + 128])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups", [1, 8])
def test_closed_experts(score, biased, groups):
    # half the experts closed, some rows with none open, some with fewer than K
    _check(64, 64, 12, closed=0.5, biased=biased, score=score, num_groups=groups, top_groups=max(1, groups // 2),
           group_score="top2")
    _check(64, 64, 12, closed=0.9, biased=biased, score=score, num_groups=groups, top_groups=max(1, groups // 2))


def test_lowest_values_are_open():
    # a type's lowest number is a logit like any other, -inf alone closes
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        l = torch.full((3, 16), torch.finfo(dtype).min, dtype=dtype, device="cuda")
        l[1, 5] = 0.0
        l[2, ::2] = -float("inf")
        _check(3, 16, 4, logits=l)
        ids, w = _router(16, 4).select(l)
        assert ids.tolist()[0] == [0, 1, 2, 3] and w.tolist()[0] == [0.25] * 4
        assert ids.tolist()[2] == [1, 3, 5, 7]


def test_ties_go_to_the_lower_id():
    l = torch.zeros(5, 200, device="cuda")
    ids, _ = _check(5, 200, 32, logits=l)
    assert ids.tolist()[0] == list(range(32))
    l[:, 190] = 1.0
    ids, _ = _check(5, 200, 3, logits=l, num_groups=10, top_groups=2)
    assert ids.tolist()[0] == [190, 0, 1]
    # -0 and +0 are equal
    l = torch.zeros(1, 64, device="cuda")
    l[0, :32] = -0.0
    assert _check(1, 64, 4, logits=l)[0].tolist() == [[0, 1, 2, 3]]
    # two values a bf16 apart from many equal ones
    g = torch.Generator().manual_seed(4)
    l = (torch.randint(0, 4, (50, 256), generator=g) * 0.5).cuda()
    _check(50, 256, 16, logits=l)
    _check(50, 256, 16, logits=l, score="sigmoid", num_groups=8, top_groups=4, group_score="top2")


def test_many_equal_values_far_apart():
    # the k-th value shared by experts of every lane
    l = torch.zeros(4, 512, device="cuda")
    l[1, 3::16] = 1.0
    l[2, 500:] = 2.0
    l[3] = torch.arange(512, device="cuda") % 7
    for K in (1, 8, 32):
        _check(4, 512, K, logits=l)
        _check(4, 512, K, logits=l, bias=torch.zeros(512, device="cuda"), score="sigmoid")


def test_undefined_rows():
    l = _logits(6, 40)
    l[1, 7] = float("nan")
    l[2, 39] = float("inf")
    l[3, :] = float("nan")
    for score in ("softmax", "sigmoid"):
        ids, w = _check(6, 40, 4, logits=l, score=score)
        assert torch.isnan(w[1]).all() and ids[1].tolist() == [0, 1, 2, 3]
        assert torch.isnan(w[2]).all().item() == (score == "softmax")
    # a bias that closes or forces an expert
    b = torch.zeros(40, device="cuda")
    b[0], b[1], b[2] = -float("inf"), float("inf"), float("nan")
    ids, _ = _router(40, 8, score="sigmoid").select(_logits(30, 40), bias=b)
    assert (ids[:, 0] == 1).all() and not ((ids == 0) | (ids == 2)).any()


def test_extreme_logits():
    l = torch.tensor([[-200.0, -150.0, -100.0, -90.0], [200.0, 150.0, 100.0, 0.0], [88.0, -88.0, 0.0, 1e-30]],
                     device="cuda")
    for score in ("softmax", "sigmoid"):
        ids, w = _router(4, 3, score=score).select(l)
        ref_ids, ref_w = ob.route(l.cpu().numpy(), 3, score)
        assert np.array_equal(ids.cpu().numpy(), ref_ids)
        # scores below the smallest FP32 number are 0
        assert np.allclose(w.cpu().numpy(), ref_w, rtol=1e-5, atol=1e-18)


# ---- gradient ----

def _check_grad(T, E, K, dtype=torch.float32, score="softmax", renormalize=True, pad=0, closed=0.0, scale=2.5, seed=0,
                inplace=False):
    r = _router(E, K, score=score, renormalize=renormalize, scale=scale)
    l = _logits(T, E, dtype, seed, closed, pad)
    ids, w = r.select(l)
    dw = torch.randn(T, K, generator=torch.Generator().manual_seed(seed + 9)).cuda()
    l64 = l.float().cpu().numpy().astype(np.float64)
    dl = r.select_backward(l, ids, w, dw, dlogits=l if inplace else None)
    assert dl.dtype == dtype and dl.shape == (T, E)
    ref, mag = ob.route_backward(l64, ids.cpu().numpy().astype(np.int64), w.cpu().numpy(),
                                 dw.cpu().numpy().astype(np.float64), score, renormalize, scale)
    got = dl.float().cpu().numpy().astype(np.float64)
    u, tiny = UNIT[dtype]
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= 64 * U * mag + (u if dtype != torch.float32 else 0) * np.abs(ref) + tiny + 1e-37).all()
    return l64, ids, w, dw, got


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K", [(1, 1), (5, 5), (33, 3), (97, 5), (128, 8), (256, 8), (510, 32), (512, 10)])
def test_gradient(E, K, score, renormalize):
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        _check_grad(29, E, K, dtype, score, renormalize)
    _check_grad(29, E, K, torch.float32, score, renormalize, pad=3)
    _check_grad(1, E, K, torch.float32, score, renormalize, pad=4)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_of_closed_experts(score):
    for renorm in (True, False):
        _, ids, w, _, got = _check_grad(64, 48, 9, score=score, renormalize=renorm, closed=0.85)
        closed = w.cpu().numpy() == 0
        assert closed.any()
        assert (np.take_along_axis(got, ids.cpu().numpy().astype(np.int64), 1)[closed] == 0).all()
        assert (got[::7] == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_in_place_and_against_differences(score):
    l64, ids, w, dw, got = _check_grad(16, 40, 6, score=score, renormalize=True, inplace=True)
    _check_grad(16, 40, 6, score=score, renormalize=False, inplace=True)
    d = np.random.default_rng(0).standard_normal(l64.shape)
    idn, dwn = ids.cpu().numpy().astype(np.int64), dw.cpu().numpy().astype(np.float64)

    def loss(x):
        s = np.take_along_axis(ob.scores(x, score), idn, 1)
        return (s / s.sum(1, keepdims=True) * 2.5 * dwn).sum()

    step = 1e-5
    diff = (loss(l64 + step * d) - loss(l64 - step * d)) / (2 * step)
    assert abs((got * d).sum() - diff) <= 1e-4 * np.abs(got * d).sum()


def test_gradient_skips_ids_outside():
    r = _router(40, 4, score="sigmoid", renormalize=False)
    l = _logits(8, 40)
    ids, w = r.select(l)
    ids = ids.clone()
    ids[0, 0], ids[1, 1], ids[2, 2] = -1, 40, 2 ** 31 - 1
    dw = torch.ones_like(w)
    got = r.select_backward(l, ids, w, dw).cpu().numpy()
    ref, mag = ob.route_backward(l.cpu().numpy(), ids.cpu().numpy().astype(np.int64), w.cpu().numpy(),
                                 dw.cpu().numpy(), "sigmoid", False)
    assert (np.abs(got - ref) <= 64 * U * mag + 1e-37).all()


def test_other_stream():
    r = _router(256, 8, score="sigmoid")
    l = _logits(500, 256)
    ref = r.select(l)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = r.select(l, stream=s)
    also = r.select(l, stream=s.cuda_stream)
    s.synchronize()
    for a in (got, also):
        assert torch.equal(a[0], ref[0]) and torch.equal(a[1], ref[1])


def test_graph_capture_and_repeat():
    r = _router(256, 8, score="sigmoid", num_groups=8, top_groups=4, group_score="top2")
    l, b = _logits(300, 256), _bias(256)
    ids, w = r.select(l, bias=b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = r.select(l, bias=b)
    b.copy_(_bias(256, seed=8))
    g.replay()
    torch.cuda.synchronize()
    again = r.select(l, bias=b)
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])
    assert not torch.equal(out[0], ids)


def test_long_rows_past_32_bits():
    # row offsets beyond 2^31 elements, through a strided view
    T, E, ld = 3, 64, 1 << 30
    if torch.cuda.mem_get_info()[0] < 6 << 30:
        pytest.skip("needs 6 GB")
    base = torch.empty(2 * ld + E, dtype=torch.bfloat16, device="cuda")
    l = base.as_strided((T, E), (ld, 1))
    l.copy_(_logits(T, E, torch.bfloat16))
    _check(T, E, 5, logits=l)
    r = _router(E, 5)
    ids, w = r.select(l)
    dl = r.select_backward(l, ids, w, torch.ones_like(w))
    assert torch.equal(dl, r.select_backward(l.contiguous(), ids, w, torch.ones_like(w)))


def test_refusals():
    from nvfp4_token_quantized_gb300 import MoEError

    r = _router(64, 4)
    l = _logits(8, 64)
    for bad in (l.cpu(), l.double(), l[:, :63], l[0], l.t().contiguous().t()):
        with pytest.raises(ValueError):
            r.select(bad)
    with pytest.raises(TypeError):
        r.select(None)
    for bias in (torch.zeros(63, device="cuda"), torch.zeros(64), torch.zeros(64, device="cuda").half()):
        with pytest.raises(ValueError):
            r.select(l, bias=bias)
    with pytest.raises(ValueError):
        r.select(l, ids=torch.zeros(8, 5, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        r.select(l, weights=torch.zeros(8, 4, dtype=torch.float64, device="cuda"))
    ids, w = r.select(l)
    with pytest.raises(ValueError):
        r.select_backward(l, ids.long(), w, w)
    with pytest.raises(MoEError) as e:  # an output over the logits
        r.select(l, weights=l.view(-1)[:32].view(8, 4))
    assert e.value.status == 5
    with pytest.raises(MoEError) as e:  # a shifted in-place gradient
        wide = _logits(8, 65)
        r.select_backward(wide[:, :64], ids, w, w, dlogits=wide[:, 1:])
    assert e.value.status == 5


def test_values_next_to_each_other():
    # logits that differ in their last bit, denormal ones among them, and -0
    base = torch.tensor([0.0, 1e-45, 3e-45, 1e-40, -1e-45, -1e-40, 1.1754944e-38, -0.0, 1.0, 1.0000001, 0.99999994, -1.0,
                         -1.0000001, 3.4028235e38, -3.4028235e38, 1e-30], device="cuda")
    g = torch.Generator().manual_seed(2)
    rows = torch.stack([base[torch.randint(0, 16, (128,), generator=g).cuda()] for _ in range(3000)])
    for K in (1, 5, 8, 20):
        _check(3000, 128, K, logits=rows)
        _check(3000, 128, K, logits=rows, num_groups=8, top_groups=6)
    tiny = (torch.randint(0, 40, (3000, 64), generator=g) * 1e-45).float().cuda()
    _check(3000, 64, 6, logits=tiny, num_groups=4, top_groups=2)
    deep = (torch.rand(3000, 64, generator=g) * -20 - 70).cuda()        # scores down to 1e-39
    ids, _ = _router(64, 6, score="sigmoid", num_groups=4, top_groups=2, group_score="top2").select(deep)
    assert all(len(set(r)) == 6 for r in ids.tolist())


@pytest.mark.parametrize("E,G,top,K", [(128, 1, 1, 8), (256, 8, 4, 8), (160, 8, 3, 6), (64, 1, 1, 16), (255, 17, 5, 9),
                                       (512, 1, 1, 10), (512, 16, 4, 12), (97, 1, 1, 5)])
def test_many_rows_equal_few_rows(E, G, top, K):
    # rows taken several at a time give the bits that a row alone gives
    T = 12001
    for score in ("softmax", "sigmoid"):
        for dtype in (torch.float32, torch.bfloat16):
            r = _router(E, K, score=score, num_groups=G, top_groups=top, group_score="top2", scale=1.5)
            l, b = _logits(T, E, dtype, closed=0.02 if G == 1 else 0.0), _bias(E)
            for bias in (None, b):
                ids, w = r.select(l, bias=bias)
                for lo in (0, 5003, T - 900):
                    i2, w2 = r.select(l[lo:lo + 900], bias=bias)
                    assert torch.equal(ids[lo:lo + 900], i2) and torch.equal(w[lo:lo + 900], w2)
                dw = torch.randn(T, K, device="cuda")
                dl = r.select_backward(l, ids, w, dw)
                d2 = r.select_backward(l[5003:5903], ids[5003:5903], w[5003:5903], dw[5003:5903])
                assert torch.equal(dl[5003:5903], d2)


@pytest.mark.parametrize("E,G,top,K,pad", [(1, 1, 1, 1, 0), (6, 3, 2, 2, 0), (16, 16, 5, 1, 0), (32, 1, 1, 32, 0),
                                           (33, 1, 1, 4, 3), (60, 5, 4, 10, 3), (64, 8, 3, 6, 0), (120, 4, 2, 3, 8),
                                           (129, 3, 1, 32, 0), (328, 8, 4, 12, 0), (481, 13, 2, 9, 1),
                                           (512, 32, 7, 16, 0)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_large_batches_with_odd_rows_equal_few_rows(E, G, top, K, pad, score):
    # few open experts, rows without weights and equal values among many rows
    T = 12307
    b = _bias(E)
    if E > 40:
        b[3], b[5], b[7] = float("inf"), float("nan"), -float("inf")
    for dtype in (torch.float32, torch.float16):
        l = _logits(T, E, dtype, closed=0.6, pad=pad)
        l[1::11] = (l[1::11] * 2).round() / 2
        l[3::97, E // 2] = float("nan")
        l[5::89, E - 1] = float("inf")
        for renormalize in (True, False):
            for group_score in ("max", "top2"):
                r = _router(E, K, score=score, num_groups=G, top_groups=top, group_score=group_score,
                            renormalize=renormalize, scale=0.5)
                for bias in (None, _bias(E), b):
                    ids, w = r.select(l, bias=bias)
                    for lo in (0, 4001, T - 700):
                        i2, w2 = r.select(l[lo:lo + 700], bias=bias)
                        assert torch.equal(ids[lo:lo + 700], i2)
                        assert torch.equal(w[lo:lo + 700].view(torch.int32), w2.view(torch.int32))


@pytest.mark.parametrize("E,G,top", [(24, 1, 1), (100, 1, 1), (100, 5, 2), (256, 1, 1)])
@pytest.mark.parametrize("biased", [False, True])
def test_large_batches(E, G, top, biased):
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            _check(12200, E, 5, biased=biased, closed=0.1, pad=1, score=score, num_groups=G, top_groups=top,
                   group_score="top2", renormalize=renormalize)
