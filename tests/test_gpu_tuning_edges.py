"""Edges of the balance loss, gradient clipping and low-rank adapters: offsets past
32 bits, one short sequence inside a batch, gradients of one row, calls at the
same time on several streams."""

import numpy as np
import pytest
import torch

from oracle import training as ot
from tests.parity import built, gpu, needs_gpu

pytestmark = [gpu, needs_gpu]

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _lib():
    import nvfp4_token_quantized_gb300 as lib

    built()
    return lib


def test_gradients_past_32_bit_offsets():
    clip = _lib().GradientClip(1.0)
    n = (1 << 31) + 1000
    t = torch.zeros(n, dtype=BF16, device="cuda")
    t[5], t[n - 1], t[n - 700] = 3.0, 4.0, 12.0
    assert clip.norm([t]).item() == 13.0
    norm, _ = clip.clip([t])
    assert norm.item() == 13.0
    f = 1.0 / (13.0 + 1e-6)
    for at, v in ((5, 3.0), (n - 1, 4.0), (n - 700, 12.0)):
        assert abs(t[at].item() - v * f) <= 2.0 ** -8 * v * f
    assert torch.count_nonzero(t).item() == 3


def test_rows_past_32_bit_offsets():
    lib = _lib()
    T, K, N, r, L = 200, 128, 136, 8, 3
    g = torch.Generator().manual_seed(0)
    stride = (1 << 31) // 128 + 8  # rows from 128 on start behind 2^31 elements
    wide = torch.empty(T * stride, dtype=BF16, device="cuda")
    ids = torch.randint(0, L, (T,), generator=g).int().cuda()
    down = (torch.randn(L, r, K, generator=g) / 11).to(BF16).cuda()
    up = torch.randn(L, r, N, generator=g).to(BF16).cuda()
    x = torch.randn(T, K, generator=g).to(BF16).cuda()
    base = torch.randn(T, N, generator=g).to(BF16).cuda()
    ad = lib.LowRankAdapters(K, N, r)
    want, hidden = ad.forward(x, ids, down, up, base=base, keep_hidden=True)
    wantb = ad.backward(base, x, hidden, ids, down, up)
    xs = wide.as_strided((T, K), (stride, 1))
    xs.copy_(x)
    bs = wide.as_strided((T, N), (stride, 1), 256)
    bs.copy_(base)
    os = wide.as_strided((T, N), (stride, 1), 512)
    got, h = ad.forward(xs, ids, down, up, base=bs, out=os, keep_hidden=True)
    assert torch.equal(got, want) and torch.equal(h, hidden)
    gotb = ad.backward(bs, xs, h, ids, down, up)
    assert all(torch.equal(a, b) for a, b in zip(gotb, wantb))
    # logits alike
    E, k = 64, 4
    router = lib.ExpertRouter(E, k)
    l = torch.randn(T, E, generator=g).to(BF16).cuda()
    chosen = torch.rand(T, E, generator=g).argsort(dim=1)[:, :k].int().cuda()
    want = router.balance_loss(l, chosen)
    ls = wide.as_strided((T, E), (stride, 1), 1024)
    ls.copy_(l)
    got = router.balance_loss(ls, chosen)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ds = wide.as_strided((T, E), (stride, 1), 2048)
    router.balance_backward(ls, got[2], dlogits=ds)
    assert torch.equal(ds, router.balance_backward(l, want[2]))


def test_one_short_sequence_inside_a_batch():
    router = _lib().ExpertRouter(48, 3, score="sigmoid")
    g = torch.Generator().manual_seed(1)
    for T, lo, hi in ((100, 10, 53), (100, 0, 1), (100, 99, 100), (9, 4, 4), (9000, 4000, 4010)):
        l = torch.randn(T, 48, generator=g).cuda()
        ids = torch.rand(T, 48, generator=g).argsort(dim=1)[:, :3].int().cuda()
        off = torch.tensor([lo, hi], dtype=torch.int32, device="cuda")
        loss, counts, slope = router.balance_loss(l, ids, 0.5, off)
        (rl, err), rc, (rs, _) = ot.balance(_np(l), ids.cpu().numpy(), 0.5, "sigmoid", [lo, hi])
        assert np.array_equal(counts.cpu().numpy(), rc)
        assert abs(loss.item() - rl) <= 2.0 ** -24 * err + 1e-30
        assert np.allclose(_np(slope), rs, rtol=1e-6, atol=0)


def test_offsets_that_break_their_order_stay_inside():
    """The result is not defined, but nothing outside the outputs changes and
    the call after it is right."""
    router = _lib().ExpertRouter(32, 2)
    g = torch.Generator().manual_seed(2)
    l = torch.randn(6000, 32, generator=g).cuda()
    ids = torch.rand(6000, 32, generator=g).argsort(dim=1)[:, :2].int().cuda()
    good = torch.tensor([0, 3000, 6000], dtype=torch.int32, device="cuda")
    want = router.balance_loss(l, ids, 1.0, good)
    for bad in ([5000, 100, 4000], [-50, 9000, 2], [7000, 8000, 9000], [6000, 3000, 0]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        _, _, slope = router.balance_loss(l, ids, 1.0, off)
        router.balance_backward(l, slope, offsets=off)
    got = router.balance_loss(l, ids, 1.0, good)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_values_beyond_the_sets_adapters():
    """ids of every size stand for no adapter."""
    ad = _lib().LowRankAdapters(64, 64, 4)
    g = torch.Generator().manual_seed(3)
    down, up = (torch.randn(2, 4, 64, generator=g).to(F16).cuda() for _ in range(2))
    for T in (8, 300, 600):
        x = torch.randn(T, 64, generator=g).to(F16).cuda()
        ids = torch.tensor([-1, 2, -(1 << 31), (1 << 31) - 1] * (T // 4), dtype=torch.int32, device="cuda")
        out, h = ad.forward(x, ids, down, up, base=x.clone(), keep_hidden=True)
        assert torch.equal(out, x) and not h.any()


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_an_infinite_row_is_the_formulas(dtype):
    """Rank 1, filled up to whole fragments: an infinite x gives infinities of
    the factors' signs, not NaN; other rows stay as they are."""
    ad = _lib().LowRankAdapters(72, 80, 1)
    g = torch.Generator().manual_seed(5)
    down, up = torch.randn(2, 1, 72, generator=g).to(dtype).cuda(), torch.randn(2, 1, 80, generator=g).to(dtype).cuda()
    for T in (8, 300, 600):
        x = torch.randn(T, 72, generator=g).to(dtype).cuda()
        ids = (torch.arange(T, device="cuda") % 2).int()
        want, _ = ad.forward(x, ids, down, up)
        x[3, 5] = float("inf")
        out, h = ad.forward(x, ids, down, up, keep_hidden=True)
        assert torch.equal(out[3], torch.sign(down[1, 0, 5]) * torch.sign(up[1, 0]) * float("inf"))
        assert torch.isinf(h[3, 0])
        keep = torch.arange(T, device="cuda") != 3
        assert torch.equal(out[keep], want[keep])


def test_the_workspace_follows_the_rows():
    """A thousand adapters cost a batch of some rows no more than its sums, and
    groups of one, two and many pieces beside empty ones keep theirs apart."""
    ad = _lib().LowRankAdapters(256, 264, 16)
    assert ad.workspace_bytes(100, 1000, True) < 16 << 20
    T, L = 2600, 300
    g = torch.Generator().manual_seed(6)
    sizes = {3: 1, 4: 192, 5: 193, 120: 900, 121: 385, 250: 384, 299: 500}
    which = torch.cat([torch.full((n,), a) for a, n in sizes.items()])
    ids = torch.full((T,), -1)
    ids[torch.randperm(T, generator=g)[:which.numel()]] = which
    x, d = torch.randn(T, 256, generator=g).to(BF16).cuda(), torch.randn(T, 264, generator=g).to(BF16).cuda()
    down, up = (torch.randn(L, 16, n, generator=g).mul(0.1).to(BF16).cuda() for n in (256, 264))
    ids = ids.int().cuda()
    _, h = ad.forward(x, ids, down, up, keep_hidden=True)
    _, dd, du = ad.backward(d, x, h, ids, down, up)
    _, v, _, _ = ot.adapters(_np(d), ids.cpu().numpy(), _np(up), _np(down))
    for a in range(L):
        rows = (ids == a).cpu().numpy()
        for got, left, right in ((dd[a], v, _np(x)), (du[a], _np(h), _np(d))):
            want = left[rows].T @ right[rows]
            mag = np.abs(left[rows]).T @ np.abs(right[rows])
            # (half a step of bf16; FP32 sums and the two parts, of their terms)
            assert (np.abs(_np(got) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -13 * mag + 1e-37).all(), a


@pytest.mark.parametrize("L", [64, 255, 256, 257, 500, 65535])
def test_many_adapters(L):
    """Around the number of adapters from which only those with rows are listed,
    and the largest; the first and the last among those that have rows."""
    ad = _lib().LowRankAdapters(24, 40, 3)
    g = torch.Generator().manual_seed(7)
    down, up = (torch.randn(L, 3, n, generator=g).to(BF16).cuda() for n in (24, 40))
    for T in (1, 7, 100, 129, 700, 17000):
        ids = torch.randint(-2, L + 2, (T,), generator=g).int()
        ids[::3] = L - 1
        ids[::5] = 0
        ids[::7] = -1
        x, d = torch.randn(T, 24, generator=g).to(BF16).cuda(), torch.randn(T, 40, generator=g).to(BF16).cuda()
        which = ids.cuda()
        out, h = ad.forward(x, which, down, up, base=d, keep_hidden=True)
        has = (ids >= 0) & (ids < L)
        a = ids.clamp(0, L - 1).long()
        dn, un = down.cpu().double()[a], up.cpu().double()[a]
        hr = torch.einsum("tk,trk->tr", x.cpu().double(), dn) * has[:, None]
        want = d.cpu().double() + torch.einsum("tr,trn->tn", hr, un)
        mag = d.cpu().double().abs() + torch.einsum("tr,trn->tn", torch.einsum(
            "tk,trk->tr", x.cpu().double().abs(), dn.abs()), un.abs())
        # (FP32 sums of 24 and 3 products, two 16-bit parts; half a step of bf16)
        assert ((h.cpu().double() - hr).abs() <= 2.0 ** -16 * mag.amax(1, keepdim=True)).all()
        assert ((out.cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -15 * mag).all()
        _, dd, du = ad.backward(d, x, h, which, down, up)
        present = torch.zeros(L, dtype=torch.bool)
        present[a[has]] = True
        assert not dd.cpu()[~present].any() and not du.cpu()[~present].any()
        for i in (0, L - 1, L // 2):
            rows = ids == i
            r = h.cpu().double()[rows].t() @ d.cpu().double()[rows]
            m = h.cpu().double()[rows].abs().t() @ d.cpu().double()[rows].abs()
            assert ((du[i].cpu().double() - r).abs() <= 2.0 ** -8 * r.abs() + 2.0 ** -13 * m + 1e-37).all()


def test_calls_at_the_same_time():
    """Several streams at once, each with buffers of its own."""
    lib = _lib()
    g = torch.Generator().manual_seed(4)
    T, K, r, L = 3000, 512, 64, 5
    down = (torch.randn(L, r, K, generator=g) / 22).to(BF16).cuda()
    up = (torch.randn(L, r, K, generator=g) / 8).to(BF16).cuda()
    ids = torch.randint(-1, L, (T,), generator=g).int().cuda()
    xs = [torch.randn(T, K, generator=g).to(BF16).cuda() for _ in range(4)]
    ad, clip = lib.LowRankAdapters(K, K, r), lib.GradientClip(0.25)

    def step(x):
        y, h = ad.forward(x, ids, down, up, base=x, keep_hidden=True)
        grads = ad.backward(y, x, h, ids, down, up)
        norm, _ = clip.clip(grads[1:])
        return y, *grads, norm

    want = [step(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        got = []
        for x, s in zip(xs, streams):
            s.wait_stream(torch.cuda.default_stream())
            with torch.cuda.stream(s):
                got.append(step(x))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_another_device_is_refused_or_used():
    lib = _lib()
    clip, ad, router = lib.GradientClip(1.0), lib.LowRankAdapters(8, 8, 2), lib.ExpertRouter(8, 2)
    cpu = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        clip.norm([cpu])
    with pytest.raises(ValueError):
        ad.forward(cpu.half(), torch.zeros(4, dtype=torch.int32), torch.zeros(1, 2, 8).half(), torch.zeros(1, 2, 8).half())
    with pytest.raises(ValueError):
        router.balance_loss(cpu, torch.zeros(4, 2, dtype=torch.int32))
