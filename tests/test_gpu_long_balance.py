"""The balance loss of long batches of equal logits, whose FP32 roundings all go one
way, against what it is by arithmetic.

Tolerances in units of 2^-24 (set before the first run), each FP32 operation at most
one unit of what it gives."""

import pytest
import torch

from tests.parity import built, gpu, needs_gpu

pytestmark = [gpu, needs_gpu]

UNIT = 2.0 ** -24


def _lib():
    import nvfp4_token_quantized_gb300 as lib

    built()
    return lib


def _off_by(T, E, S, score, dtype=torch.float32):
    """The loss's distance from the coefficient, which equal shares give whoever is
    chosen, in units."""
    router = _lib().ExpertRouter(E, 1, score=score)
    l = torch.full((T, E), -0.25, dtype=dtype, device="cuda")
    ids = (torch.arange(T, device="cuda") % E).int()[:, None].contiguous()
    off = None
    if S > 1:
        off = (torch.arange(S + 1, device="cuda", dtype=torch.float64) * (T / S)).round().int()
    loss, counts, _ = router.balance_loss(l, ids, 0.75, off)
    assert counts.sum().item() == T
    del l, ids
    torch.cuda.empty_cache()
    return abs(loss.item() / 0.75 - 1) / UNIT


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,S", [(1 << 24, 3, 1), (1 << 23, 6, 1), (131072, 3, 1), (131072, 7, 1), (43000, 3, 1),
                                   (1 << 22, 7, 5), (300000, 3, 100000)])
def test_few_experts(T, E, S, score):
    """A share 6 (exponential, sum, quotient, the sum's own 1e-20), 32 rows of a lane 17
    in the mean, two halves 1, eight warps 5; the runs' join 12; slope 5, its product
    1, the sums over a CTA's experts and a cluster 6; sequences and the mean 3."""
    assert _off_by(T, E, S, score) <= 56


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E", [(1 << 24, 200), (1 << 22, 131)])
def test_many_experts(T, E, score):
    """As above, a share's sum of up to 16 experts a lane 16 more, and up to 32 such
    sums of 32 rows 17 in the mean."""
    assert _off_by(T, E, 1, score, torch.bfloat16) <= 56 + 33
