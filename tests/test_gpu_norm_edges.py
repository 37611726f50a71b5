"""The norms around a block at the edges of their arithmetic."""

import pytest
import torch

from tests.parity import built, gpu, needs_gpu

pytestmark = [gpu, needs_gpu]

BF16, F32 = torch.bfloat16, torch.float32
HUGE = 1e25  # squares past FP32


def _rows(T, H, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return {k: torch.randn(T, H, generator=g).to(dtype).cuda() for k in ("residual", "y", "dres", "dh")}


def _norm(H, **kw):
    from nvfp4_token_quantized_gb300 import BlockNorm

    built()
    return BlockNorm(H, **kw)


# a warp's row, one and two chunks a thread, four; and rows without 16-byte accesses
@pytest.mark.parametrize("H", [64, 1024, 8192, 12288, 37, 1001, 8209])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_rows_whose_squares_overflow(H, dtype, kind):
    # 1 / sqrt(inf) is 0: the normed row is 0, and no row else changes
    T, bad = 9, 4
    n, a = _norm(H, kind=kind), _rows(T, H, dtype)
    w = dict(post_weight=torch.ones(H, dtype=dtype, device="cuda"), pre_weight=torch.ones(H, dtype=dtype, device="cuda"))
    keep = [t for t in range(T) if t != bad]
    ref_out, ref_h = n.forward(a["residual"], a["y"], **w)
    # the block's output
    y = a["y"].clone()
    y[bad] *= HUGE
    out, h = n.forward(a["residual"], y, **w)
    assert torch.equal(out[bad], a["residual"][bad]) and torch.isfinite(h.float()).all()
    assert torch.equal(out[keep], ref_out[keep]) and torch.equal(h[keep], ref_h[keep])
    _, dy, _, dpost, _ = n.backward(a["dres"], a["dh"], out, y, **w)
    ref = n.backward(a["dres"][keep], a["dh"][keep], out[keep], y[keep], **w)
    assert (dy[bad] == 0).all() and torch.equal(dy[keep], ref[1])
    assert torch.isfinite(dpost).all() and torch.allclose(dpost, ref[3], rtol=1e-5, atol=1e-5)
    # the residual stream
    r = a["residual"].clone()
    r[bad] *= HUGE
    _, h = n.forward(r, pre_weight=w["pre_weight"])
    assert (h[bad] == 0).all() and torch.isfinite(h.float()).all()
    dr, _, _, _, dpre = n.backward(a["dres"], a["dh"], r, pre_weight=w["pre_weight"])
    ref = n.backward(a["dres"][keep], a["dh"][keep], r[keep], pre_weight=w["pre_weight"])
    assert torch.equal(dr[bad], a["dres"][bad]) and torch.equal(dr[keep], ref[0])
    assert torch.isfinite(dpre).all() and torch.allclose(dpre, ref[4], rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("T,H", [(2000, 2048), (300, 8192), (500, 1000), (700, 64), (40, 12288)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_one_row_alone_gives_every_bit_it_gives_in_a_batch(T, H, kind):
    n, a = _norm(H, kind=kind), _rows(T, H, BF16)
    w = dict(post_weight=torch.linspace(0.5, 1.5, H, device="cuda").to(BF16),
             pre_weight=torch.linspace(1.5, 0.5, H, device="cuda").to(BF16))
    out, h = n.forward(a["residual"], a["y"], **w)
    dr, dy = n.backward(a["dres"], a["dh"], out, a["y"], **w)[:2]
    for t in (0, 7, T - 1):
        one = slice(t, t + 1)
        o1, h1 = n.forward(a["residual"][one], a["y"][one], **w)
        assert torch.equal(o1, out[one]) and torch.equal(h1, h[one])
        r1, y1 = n.backward(a["dres"][one], a["dh"][one], out[one], a["y"][one], **w)[:2]
        assert torch.equal(r1, dr[one]) and torch.equal(y1, dy[one])
