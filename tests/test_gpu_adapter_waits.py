"""Low-rank adapters whose bounded waits run out: the first wait of a CTA is for a
barrier at which nothing arrives, and ends after a millisecond.  Nothing faults or
hangs: the calls return, and those after them are right."""

import pytest
import torch

from tests.parity import built, gpu, needs_gpu

pytestmark = [gpu, needs_gpu]

F16, BF16 = torch.float16, torch.bfloat16


class _Silent:
    """The library with the waiting tests' calls in the place of the usual ones."""

    def __init__(self, lib, silent):
        self._so, self._silent = lib, silent

    def __getattr__(self, name):
        return getattr(self._so, name)

    def moe_adapter_forward(self, cfg, io, rows, stream):
        return self._so.moe_debug_adapter_forward(cfg, io, rows, self._silent, stream)

    def moe_adapter_backward(self, cfg, io, rows, stream):
        return self._so.moe_debug_adapter_backward(cfg, io, rows, self._silent, stream)


def _make(T, K, N, r, L, dtype, pad=0):
    from nvfp4_token_quantized_gb300 import LowRankAdapters

    built()
    g = torch.Generator().manual_seed(T + r)

    def rows(w):
        return torch.randn(T, w + pad, generator=g).to(dtype).cuda()[:, :w]

    a = dict(x=rows(K), ids=(torch.arange(T) % (L + 1) - 1).int().cuda(),
             down=(torch.randn(L, r, K, generator=g) / K ** 0.5).to(dtype).cuda(),
             up=(torch.randn(L, r, N, generator=g) / r ** 0.5).to(dtype).cuda(), base=rows(N))
    return LowRankAdapters(K, N, r), LowRankAdapters(K, N, r), a, rows(N), rows(K)


# clusters of eight, four, two and one; rows that start anywhere; long axes of more
# stages than the ring has
CASES = [(600, 512, 512, 16, 3, BF16, 0), (600, 512, 512, 16, 3, F16, 1), (600, 200, 136, 128, 2, F16, 0),
         (6000, 512, 256, 32, 3, BF16, 0), (16000, 256, 192, 64, 3, BF16, 0), (40000, 256, 64, 16, 3, BF16, 0),
         (16000, 1024, 1024, 16, 3, BF16, 0), (16000, 1024, 1024, 16, 3, F16, 1)]


@pytest.mark.parametrize("T,K,N,r,L,dtype,pad", CASES)
def test_later_calls_are_right(T, K, N, r, L, dtype, pad):
    ad, lost, a, dout, dbase = _make(T, K, N, r, L, dtype, pad)
    out, hidden = ad.forward(**a, keep_hidden=True)
    back = dict(dout=dout, x=a["x"], hidden=hidden, ids=a["ids"], down=a["down"], up=a["up"], base=dbase)
    want = (out, hidden, *ad.backward(**back))
    for silent in (1, 2, 5, 8):
        lost._lib = _Silent(ad._lib, silent)
        for _ in range(2):
            lost.forward(**a, keep_hidden=True)
            lost.backward(**back)
            got = (*ad.forward(**a, keep_hidden=True), *ad.backward(**back))
            assert all(torch.equal(p, q) for p, q in zip(got, want))
    torch.cuda.synchronize()


def test_a_call_whose_wait_runs_out_beside_others():
    """On a stream of its own, while others form the same on theirs: tensor memory
    and shared memory of the same SMs."""
    ad, lost, a, dout, dbase = _make(3000, 512, 512, 32, 3, BF16)
    out, hidden = ad.forward(**a, keep_hidden=True)
    back = dict(dout=dout, x=a["x"], hidden=hidden, ids=a["ids"], down=a["down"], up=a["up"], base=dbase)
    want = (out, hidden, *ad.backward(**back))
    lost._lib = _Silent(ad._lib, 1)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(3):
        got = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                for _ in range(3):
                    which = lost if i == 0 else ad
                    y = (*which.forward(**a, keep_hidden=True), *which.backward(**back))
                    if i:
                        got.append(y)
        torch.cuda.synchronize()
        for y in got:
            assert all(torch.equal(p, q) for p, q in zip(y, want))


def test_nothing_waits_where_none_is_asked_to():
    """silent 0 is the call itself, and a negative one is refused."""
    ad, same, a, _, _ = _make(600, 256, 256, 16, 3, BF16)
    same._lib = _Silent(ad._lib, 0)
    assert torch.equal(same.forward(**a)[0], ad.forward(**a)[0])
    same._lib = _Silent(ad._lib, -1)
    with pytest.raises(RuntimeError):
        same.forward(**a)


@pytest.mark.parametrize("T,K,N,r,L,dtype,pad", CASES)
def test_rows_whose_wait_ran_out_are_no_numbers(T, K, N, r, L, dtype, pad):
    """Whole rows, whichever CTA of the cluster gave up, with their hidden, and from
    there the gradients; rows without an adapter are their base."""
    ad, lost, a, dout, dbase = _make(T, K, N, r, L, dtype, pad)
    _, hidden = ad.forward(**a, keep_hidden=True)
    has = a["ids"] >= 0
    back = dict(dout=dout, x=a["x"], hidden=hidden, ids=a["ids"], down=a["down"], up=a["up"], base=dbase)
    lost._lib = _Silent(ad._lib, 1)
    out, h = lost.forward(**a, keep_hidden=True)
    assert torch.isnan(out[has]).all() and torch.isnan(h[has]).all()
    assert torch.equal(out[~has], a["base"][~has]) and not h[~has].any()
    dx, dd, du = lost.backward(**back)
    assert torch.isnan(dx[has]).all() and torch.isnan(dd).all() and torch.isnan(du).all()
    assert torch.equal(dx[~has], dbase[~has])
    # what comes of such a hidden elsewhere
    _, dd, du = ad.backward(**{**back, "hidden": h})
    assert torch.isfinite(dd).all() and torch.isnan(du).all()


def test_another_cta_of_the_cluster():
    T, K, N, r, L = 600, 512, 512, 16, 3
    ad, lost, a, _, _ = _make(T, K, N, r, L, BF16)
    for silent in range(2, 9):
        lost._lib = _Silent(ad._lib, silent)
        out, h = lost.forward(**a, keep_hidden=True)
        assert torch.isnan(out[a["ids"] >= 0]).all() and torch.isnan(h[a["ids"] >= 0]).all()
