"""The norm of large sets of equal gradients, whose FP32 roundings all go one way,
against what it is by arithmetic.

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


@pytest.mark.parametrize("value", [1.1, 1.3, 0.7, 1.9])
def test_norm_of_hundreds_of_chunks_a_thread(value):
    """One element that is not 0 a thread and chunk (256 threads, 32 KB): a chunk's sum
    is its square, and those over the chunks are what is tested.

    Of the squares' sum: its terms' own rounding 1, the join of a thread's words 2,
    the tree over a CTA 13, FP64 behind it; half of that for the root, which with
    its own and the sum's rounding adds 2: 10."""
    lib = _lib()
    clip = lib.GradientClip(1.0)
    n = 1 << 26  # (256 MB; a list may name a tensor often where it is only read)
    t = torch.zeros(n, device="cuda")
    t.view(-1, 2048, 4)[:, :256, 0] = value
    count = (t != 0).sum().item()
    v = t[0].item()
    for times in (1, 4, 16, 64):
        want = v * (count * times) ** 0.5
        got = clip.norm([t] * times).item()
        assert abs(got / want - 1) <= 10 * UNIT, (times, (got / want - 1) / UNIT)


def test_clipping_by_a_long_norm():
    """The factor that the gradients get is the norm's."""
    lib = _lib()
    g = [torch.full((1 << 28,), 0.7, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    v, count = g[0][0].item(), 3 << 28
    want = v * count ** 0.5
    norm, _ = lib.GradientClip(want / 2).clip(g)
    # (a thread's 64 squares are 16-bit values: their sum is exact, as above)
    assert abs(norm.item() / want - 1) <= 10 * UNIT
    half = torch.tensor(v * 0.5)
    for t in g:
        # half a step of bf16, beside the factor's own FP32 roundings
        assert (t - half.cuda()).abs().max().item() <= (2.0 ** -9 + 2.0 ** -20) * v
