"""Refusals of the balance loss and gradient clipping that need no device:
every call here returns a status before any CUDA work."""

import ctypes

import pytest

OK, INVALID, ALIAS, UNSUPPORTED = 0, 1, 5, 8
BF16, F16, F32 = 1, 2, 3
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from nvfp4_token_quantized_gb300 import build, load_library

    build()
    return load_library()


def _cfg(E=64, K=4, score=0):
    from nvfp4_token_quantized_gb300.binding import moe_route_config

    return ctypes.byref(moe_route_config(E, K, score, 1, 1, 0, 1, 1.0))


def _loss(lib, T=100, S=1, coefficient=1.0, loss=4 * MB, counts=5 * MB, slope=6 * MB, ws=7 * MB, cfg=None, **kw):
    from nvfp4_token_quantized_gb300.binding import moe_balance_io

    d = dict(logits=MB, topk_ids=2 * MB, offsets=None, mask=None, logits_stride=64, num_sequences=S, dtype=F32)
    d.update(kw)
    return lib.moe_balance_loss(cfg or _cfg(), ctypes.byref(moe_balance_io(**d)), coefficient, T, loss, counts, slope,
                                ws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), INVALID), (dict(topk_ids=None), INVALID), (dict(loss=None), INVALID),
    (dict(counts=None), INVALID), (dict(slope=None), INVALID), (dict(T=9999, ws=None), INVALID), (dict(ws=7 * MB + 8), INVALID),
    (dict(logits=MB + 2), INVALID), (dict(topk_ids=2 * MB + 2), INVALID), (dict(offsets=2), INVALID),
    (dict(logits_stride=63), INVALID), (dict(dtype=0), INVALID), (dict(dtype=4), INVALID), (dict(S=0), INVALID),
    (dict(S=2), INVALID), (dict(S=1 << 31, offsets=3 * MB), INVALID), (dict(T=-1), INVALID), (dict(T=1 << 30), INVALID),
    (dict(coefficient=float("inf")), INVALID), (dict(logits_stride=1 << 62), INVALID),
    (dict(loss=MB), ALIAS), (dict(counts=2 * MB), ALIAS), (dict(slope=5 * MB + 8), ALIAS), (dict(T=9999, ws=6 * MB + 16), ALIAS),
    (dict(loss=5 * MB + 4), ALIAS), (dict(mask=6 * MB + 10), ALIAS), (dict(offsets=4 * MB, S=3), ALIAS),
])
def test_balance_loss(lib, kw, status):
    assert _loss(lib, **kw) == status


def test_balance_configurations(lib):
    assert lib.moe_balance_loss(None, None, 1.0, 0, None, None, None, None, None) == INVALID
    assert lib.moe_balance_loss(_cfg(), None, 1.0, 0, None, None, None, None, None) == INVALID
    assert _loss(lib, cfg=_cfg(E=513)) == UNSUPPORTED and _loss(lib, cfg=_cfg(K=65)) == INVALID
    assert _loss(lib, cfg=_cfg(score=2)) == INVALID
    assert lib.moe_balance_workspace_bytes(_cfg(), 1000, 5) >= 5 * 129 * 4
    for T, S in ((-1, 1), (1000, 0), (1 << 30, 1)):
        assert lib.moe_balance_workspace_bytes(_cfg(), T, S) == 0
    assert lib.moe_balance_workspace_bytes(_cfg(E=0), 10, 1) == 0


def test_balance_gradient(lib):
    from nvfp4_token_quantized_gb300.binding import moe_balance_io

    def call(T=100, slope=2 * MB, dloss=None, add=None, la=64, dl=4 * MB, ldd=64, **kw):
        d = dict(logits=MB, topk_ids=None, offsets=None, mask=None, logits_stride=64, num_sequences=1, dtype=F32)
        d.update(kw)
        return lib.moe_balance_loss_backward(_cfg(), ctypes.byref(moe_balance_io(**d)), slope, dloss, add, la, T, dl,
                                             ldd, None)

    assert call(T=0, logits=None, slope=None, dl=None) == OK
    for bad in (dict(T=-1), dict(slope=None), dict(slope=2 * MB + 1), dict(dloss=3), dict(dl=None), dict(dl=4 * MB + 2),
                dict(ldd=63), dict(add=5 * MB, la=63), dict(add=5 * MB + 1), dict(num_sequences=2), dict(logits=None),
                dict(ldd=1 << 62)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dl=MB + 256), dict(dl=MB, ldd=65), dict(add=4 * MB + 256), dict(add=4 * MB, la=65),
                dict(slope=4 * MB), dict(dloss=4 * MB + 8), dict(mask=4 * MB), dict(offsets=4 * MB)):
        assert call(**bad) == ALIAS, bad


def _set(*tensors):
    from nvfp4_token_quantized_gb300.binding import moe_gradient

    return (moe_gradient * max(1, len(tensors)))(*[moe_gradient(*t) for t in tensors])


def _clip(lib, *tensors, limit=1.0, eps=1e-6, norm=64 * MB, ws=65 * MB, num=None):
    return lib.moe_clip_gradients(_set(*tensors), len(tensors) if num is None else num, limit, eps, norm, ws, None)


@pytest.mark.parametrize("t,status", [
    ((0, MB, 4, F32), INVALID), ((MB, 0, 4, F32), INVALID), ((MB, MB, -1, F32), INVALID), ((MB, MB, 4, 0), INVALID),
    ((MB, MB, 4, 4), INVALID), ((MB, MB, 4, F32 + (1 << 32)), INVALID), ((MB + 2, MB + 2, 4, F32), INVALID),
    ((MB + 1, MB + 1, 4, BF16), INVALID), ((MB, MB + 2, 4, F32), INVALID), ((MB, MB, 1 << 62, F16), INVALID),
    ((MB, MB + 4, 4, F32), ALIAS), ((MB, MB - 8, 8, BF16), ALIAS), ((64 * MB - 8, MB, 4, F32), ALIAS),
    ((MB, 65 * MB + 16, 4, F32), ALIAS),
])
def test_gradients(lib, t, status):
    assert _clip(lib, t) == status
    assert _clip(lib, (3 * MB, 3 * MB, 100, F32), t, (8 * MB, 9 * MB, 0, BF16)) == status


def test_sets_of_gradients(lib):
    a, b, c = (MB, MB, 100, F32), (MB + 400, MB + 400, 100, F32), (MB + 800, 2 * MB, 100, F32)
    for bad in ((a, a), (a, (MB + 396, MB + 396, 2, F32)), ((MB + 396, 9 * MB, 2, F32), a), (c, (2 * MB, 2 * MB, 1, BF16)),
                (c, (3 * MB, 2 * MB + 396, 100, F32)), (b, c, a, a)):
        assert _clip(lib, *bad) == ALIAS, bad
        assert _clip(lib, *bad[::-1]) == ALIAS, bad
    for kw in (dict(limit=-1.0), dict(limit=float("inf")), dict(limit=float("nan")), dict(eps=0.0),
               dict(eps=float("nan")), dict(norm=None), dict(norm=64 * MB + 2), dict(ws=None), dict(ws=65 * MB + 8),
               dict(num=-1)):
        assert _clip(lib, a, b, c, **kw) == INVALID, kw
    assert lib.moe_clip_gradients(None, 2, 1.0, 1e-6, 64 * MB, 65 * MB, None) == INVALID
    assert _clip(lib, a, norm=65 * MB) == ALIAS
    assert lib.moe_gradient_workspace_bytes() > 0


def test_gradient_norm(lib):
    def norm(*tensors, norm=64 * MB, ws=65 * MB):
        return lib.moe_gradient_norm(_set(*tensors), len(tensors), norm, ws, None)

    for bad in (dict(norm=None), dict(ws=None), dict(norm=64 * MB + 1), dict(ws=65 * MB + 4)):
        assert norm((MB, 0, 4, F32), **bad) == INVALID
    assert norm((0, 0, 4, F32)) == INVALID and norm((MB, 0, 4, 9)) == INVALID
    assert norm((64 * MB - 4, 0, 2, F32)) == ALIAS and norm((65 * MB + 8, 0, 1, BF16)) == ALIAS
    assert norm((MB, 0, 4, F32), norm=65 * MB) == ALIAS


def test_aligned_calls_reach_the_device_check(lib):
    import torch

    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    a, b = (MB, MB, 100, F32), (MB + 400, MB + 400, 100, F32)
    assert _clip(lib, b, a) == UNSUPPORTED and _clip(lib) == UNSUPPORTED
    assert _clip(lib, (MB, 3 * MB, 100, F32), (MB, 4 * MB, 100, F32)) == UNSUPPORTED  # (one source, read twice)
    assert _loss(lib) == UNSUPPORTED and _loss(lib, T=0, logits=None, topk_ids=None) == UNSUPPORTED


def _adapter_cfg(K=64, N=96, r=8, L=4, dtype=BF16):
    from nvfp4_token_quantized_gb300.binding import moe_adapter_config

    return ctypes.byref(moe_adapter_config(K, N, r, L, dtype))


@pytest.mark.parametrize("kw,status", [
    ({}, OK), (dict(r=128, dtype=F16), OK), (dict(K=1, N=1, r=1, L=1), OK), (dict(K=0), INVALID), (dict(N=-1), INVALID),
    (dict(r=0), INVALID), (dict(L=0), INVALID), (dict(dtype=F32), INVALID), (dict(dtype=0), INVALID),
    (dict(r=129), UNSUPPORTED), (dict(K=(1 << 20) + 1), UNSUPPORTED), (dict(N=(1 << 20) + 1), UNSUPPORTED),
    (dict(L=65536), UNSUPPORTED),
])
def test_adapter_configurations(lib, kw, status):
    from nvfp4_token_quantized_gb300.binding import moe_adapter_grad_io, moe_adapter_io

    cfg = _adapter_cfg(**kw)
    assert lib.moe_adapter_forward(cfg, ctypes.byref(moe_adapter_io()), 0, None) == status
    assert (lib.moe_adapter_workspace_bytes(cfg, 1000, 0) > 0) == (status == OK)
    assert lib.moe_adapter_workspace_bytes(cfg, 10, 1) >= lib.moe_adapter_workspace_bytes(cfg, 10, 0)
    assert lib.moe_adapter_workspace_bytes(cfg, -1, 0) == 0
    if status != OK:
        assert lib.moe_adapter_backward(cfg, ctypes.byref(moe_adapter_grad_io()), 4, None) == status


def test_adapter_operands(lib):
    from nvfp4_token_quantized_gb300.binding import moe_adapter_io

    def call(rows=600, **kw):
        d = dict(x=MB, base=2 * MB, down=3 * MB, up=4 * MB, ids=5 * MB, scales=6 * MB, out=7 * MB, hidden=8 * MB,
                 workspace=9 * MB, x_stride=64, base_stride=96, out_stride=96)
        d.update(kw)
        return lib.moe_adapter_forward(_adapter_cfg(), ctypes.byref(moe_adapter_io(**d)), rows, None)

    assert lib.moe_adapter_forward(None, None, 0, None) == INVALID
    assert lib.moe_adapter_forward(_adapter_cfg(), None, 0, None) == INVALID
    for bad in (dict(rows=-1), dict(rows=1 << 31), dict(x=None), dict(down=None), dict(up=None), dict(ids=None),
                dict(out=None), dict(workspace=None), dict(workspace=9 * MB + 8), dict(x=MB + 1), dict(base=2 * MB + 1),
                dict(down=3 * MB + 1), dict(ids=5 * MB + 2), dict(scales=6 * MB + 2), dict(hidden=8 * MB + 2),
                dict(x_stride=63), dict(out_stride=95), dict(base_stride=0), dict(x_stride=1 << 60)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(out=MB), dict(out=3 * MB), dict(out=4 * MB), dict(out=5 * MB), dict(out=6 * MB), dict(out=8 * MB),
                dict(out=9 * MB), dict(hidden=MB), dict(workspace=7 * MB), dict(out=2 * MB + 192),
                dict(out=2 * MB, out_stride=104)):
        assert call(**bad) == ALIAS, bad


def test_adapter_gradient_operands(lib):
    from nvfp4_token_quantized_gb300.binding import moe_adapter_grad_io

    def call(rows=200, **kw):
        d = dict(dout=MB, x=2 * MB, base=None, down=3 * MB, up=4 * MB, ids=5 * MB, scales=None, hidden=6 * MB, dx=7 * MB,
                 ddown=8 * MB, dup=9 * MB, workspace=10 * MB, dout_stride=96, x_stride=64, base_stride=64, dx_stride=64)
        d.update(kw)
        return lib.moe_adapter_backward(_adapter_cfg(), ctypes.byref(moe_adapter_grad_io(**d)), rows, None)

    assert lib.moe_adapter_backward(_adapter_cfg(), None, 0, None) == INVALID
    for bad in (dict(dout=None), dict(x=None), dict(down=None), dict(up=None), dict(ids=None), dict(hidden=None),
                dict(dx=None), dict(ddown=None), dict(dup=None), dict(workspace=None), dict(workspace=10 * MB + 4),
                dict(dx_stride=63), dict(rows=-1), dict(rows=0, ddown=None), dict(base=11 * MB, base_stride=60)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dx=2 * MB), dict(dx=MB), dict(ddown=3 * MB), dict(dup=4 * MB), dict(dup=8 * MB), dict(dx=6 * MB),
                dict(workspace=7 * MB), dict(base=7 * MB + 128), dict(base=7 * MB, base_stride=72)):
        assert call(**bad) == ALIAS, bad
