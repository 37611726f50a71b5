"""The balance loss of rows of up to 32 chosen experts, and calls whose offsets are
out of order inside buffers whose surroundings are watched."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import training as ot
from tests.parity import built, gpu, needs_gpu

pytestmark = [gpu, needs_gpu]

U = 2.0 ** -24


def _lib():
    import nvfp4_token_quantized_gb300 as lib

    built()
    return lib


@pytest.mark.parametrize("K", [15, 16, 17, 31, 32])
@pytest.mark.parametrize("T,E,S", [(1, 40, 1), (37, 64, 1), (37, 64, 3), (5000, 64, 1), (3001, 512, 4), (700, 33, 2)])
def test_many_slots(K, T, E, S):
    """Every slot counts; ids outside the experts and repeated ones, in the last
    slots too."""
    g = torch.Generator().manual_seed(K * 1000 + T)
    router = _lib().ExpertRouter(E, K)
    l = torch.randn(T, E, generator=g)
    ids = torch.rand(T, E, generator=g).argsort(dim=1)[:, :K].int()
    ids[::3, K - 1] = ids[::3, 0]
    ids[1::4, K - 1] = E
    ids[2::5, min(16, K - 1)] = -1
    mask = torch.rand(T, generator=g) < 0.9
    off = None if S == 1 else torch.linspace(0, T, S + 1).round().int()
    loss, counts, slope = router.balance_loss(l.cuda(), ids.cuda(), 0.5, None if off is None else off.cuda(), mask.cuda())
    (want, err), c, (sl, serr) = ot.balance(l.numpy(), ids.numpy(), 0.5, "softmax", None if off is None else off.tolist(),
                                            mask.numpy())
    assert np.array_equal(counts.cpu().numpy(), c)
    assert abs(loss.item() - want) <= U * (err + abs(want)) + 1e-36
    assert (np.abs(slope.cpu().numpy() - sl) <= U * (serr + np.abs(sl)) + 1e-36).all()


def test_offsets_out_of_order_write_nothing_else():
    """What the outputs hold is not defined then, but no byte around them, or around
    the workspace, changes."""
    lib = _lib()
    from nvfp4_token_quantized_gb300.binding import load_library, moe_balance_io, moe_route_config

    so = load_library()
    T, E, K, S = 6000, 32, 2, 3
    g = torch.Generator().manual_seed(3)
    l = torch.randn(T, E, generator=g).cuda()
    ids = torch.rand(T, E, generator=g).argsort(dim=1)[:, :K].int().cuda()
    router = lib.ExpertRouter(E, K)
    cfg = router._cfg
    need = int(so.moe_balance_workspace_bytes(cfg, T, S))
    table, row = S * E * 4, T * E * 4
    sizes = {"loss": 4, "counts": table, "slope": table, "workspace": need, "dlogits": row}
    guard, at, places = 4096, 4096, {}
    for name, n in sizes.items():
        places[name] = at
        at += (n + 15) // 16 * 16 + guard
    stream = torch.cuda.current_stream().cuda_stream
    for bad in ([5000, 100, 4000, 2], [-50, 9000, 2, 6000], [7000, 8000, 9000, 10], [6000, 3000, 0, 0],
                [0, 6000, 0, 6000], [1 << 30, -(1 << 31), (1 << 31) - 1, 5]):
        whole = torch.full((at,), 0xA5, dtype=torch.uint8, device="cuda")
        p = {k: whole.data_ptr() + v for k, v in places.items()}
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        io = moe_balance_io(l.data_ptr(), ids.data_ptr(), off.data_ptr(), None, E, S, 3)
        assert so.moe_balance_loss(cfg, ctypes.byref(io), 1.0, T, p["loss"], p["counts"], p["slope"], p["workspace"],
                                   stream) == 0
        assert so.moe_balance_loss_backward(cfg, ctypes.byref(io), p["slope"], None, None, 0, T, p["dlogits"], E,
                                            stream) == 0
        torch.cuda.synchronize()
        inside = torch.zeros(at, dtype=torch.bool, device="cuda")
        for name, n in sizes.items():
            inside[places[name]:places[name] + n] = True
        assert bool((whole[~inside] == 0xA5).all()), bad


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs a second GPU")
def test_tensors_of_another_device_are_refused():
    lib = _lib()
    far = torch.device("cuda:1")
    router, clip, ad = lib.ExpertRouter(8, 2), lib.GradientClip(1.0), lib.LowRankAdapters(8, 8, 2)
    l, ids = torch.zeros(4, 8, device=far), torch.zeros(4, 2, dtype=torch.int32, device=far)
    with torch.cuda.device(0):
        with pytest.raises(ValueError, match="current device"):
            router.balance_loss(l, ids)
        with pytest.raises(ValueError, match="cuda:0"):
            router.balance_loss(l.to("cuda:0"), ids)
        with pytest.raises(ValueError, match="cuda:0"):
            clip.norm([l])
        with pytest.raises(ValueError):
            ad.forward(l.half(), ids[:, 0].contiguous(), torch.zeros(1, 2, 8).half().cuda(), torch.zeros(1, 2, 8).half().cuda())
