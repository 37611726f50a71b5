"""Refusals of the operators around the layer that need no device: every call
here returns a status before any CUDA work."""

import ctypes

import pytest

OK, INVALID, ALIAS, UNSUPPORTED = 0, 1, 5, 8
F32, BF16 = 3, 1


@pytest.fixture(scope="module")
def lib():
    from nvfp4_token_quantized_gb300 import build, load_library

    build()
    return load_library()


def _select(lib, E=64, K=4, score=0, groups=1, top=1, gscore=0, renorm=1, scale=1.0, dtype=F32, T=0, logits=None,
            stride=64, bias=None, ids=None, w=None):
    from nvfp4_token_quantized_gb300.binding import moe_route_config

    cfg = moe_route_config(E, K, score, groups, top, gscore, renorm, scale)
    return lib.moe_route_select(ctypes.byref(cfg), logits, dtype, stride, bias, T, ids, w, None)


@pytest.mark.parametrize("kw,status", [
    ({}, OK), (dict(E=512, K=32), OK), (dict(groups=32, top=2), OK), (dict(E=0), INVALID), (dict(K=0), INVALID),
    (dict(K=65), INVALID), (dict(groups=5), INVALID), (dict(groups=0), INVALID), (dict(groups=4, top=5), INVALID),
    (dict(groups=4, top=0), INVALID), (dict(groups=32, top=1), INVALID), (dict(score=2), INVALID),
    (dict(gscore=2), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=0.0), INVALID),
    (dict(dtype=4), INVALID), (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID), (dict(E=513), UNSUPPORTED),
    (dict(E=64, K=33), UNSUPPORTED), (dict(E=128, K=1, groups=64), UNSUPPORTED), (dict(T=1), INVALID),
    (dict(T=2, logits=4096, ids=65536, w=131072, stride=63), INVALID),
    (dict(T=2, logits=4098, ids=65536, w=131072), INVALID), (dict(T=2, logits=4096, ids=65537, w=131072), INVALID),
    (dict(T=2, logits=4096, ids=65536, w=131072, bias=2), INVALID),
    (dict(T=2, logits=4096, ids=4096, w=131072), ALIAS), (dict(T=2, logits=4096, ids=65536, w=65536), ALIAS),
    (dict(T=2, logits=4096, ids=65536, w=131072, bias=65536), ALIAS),
])
def test_route_select(lib, kw, status):
    assert _select(lib, **kw) == status


def test_route_select_needs_a_configuration(lib):
    assert lib.moe_route_select(None, None, F32, 0, None, 0, None, None, None) == INVALID
    assert lib.moe_route_select_backward(None, None, F32, 0, None, None, None, 0, None, 0, None) == INVALID
    assert lib.moe_set_routing(None, None, None, None) == INVALID


def test_route_select_backward(lib):
    from nvfp4_token_quantized_gb300.binding import moe_route_config

    cfg = ctypes.byref(moe_route_config(64, 4, 0, 1, 1, 0, 1, 1.0))

    def call(T=2, logits=4096, ld=64, ids=65536, w=131072, dw=196608, dl=262144, ldd=64, dtype=F32):
        return lib.moe_route_select_backward(cfg, logits, dtype, ld, ids, w, dw, T, dl, ldd, None)

    assert call(T=0, logits=None, ids=None, w=None, dw=None, dl=None) == OK
    for bad in (dict(dl=None), dict(dw=None), dict(ld=60), dict(ldd=60), dict(dl=262145), dict(dtype=0)):
        assert call(**bad) == INVALID
    for bad in (dict(dl=65536), dict(dl=131072), dict(dl=196608), dict(dl=4100), dict(dl=4096, ldd=65)):
        assert call(**bad) == ALIAS


def _norm_cfg(**kw):
    from nvfp4_token_quantized_gb300.binding import moe_norm_config

    d = dict(hidden=64, kind=0, branch=1, post=1, pre=1, gate=0, gate_sigmoid=0, dtype=BF16, residual_dtype=BF16,
             weight_dtype=BF16, eps=1e-5, weight_offset=0.0, branch_scale=1.0)
    d.update(kw)
    return moe_norm_config(**d)


@pytest.mark.parametrize("kw,status", [
    ({}, OK), (dict(hidden=16384), OK), (dict(residual_dtype=F32, weight_dtype=F32), OK), (dict(hidden=0), INVALID),
    (dict(kind=2), INVALID), (dict(gate=4), INVALID), (dict(gate=-1), INVALID), (dict(dtype=0), INVALID),
    (dict(residual_dtype=2), INVALID), (dict(weight_dtype=2), INVALID), (dict(dtype=F32), INVALID),
    (dict(branch=0), INVALID), (dict(branch=0, post=0), OK), (dict(branch=0, post=0, pre=0), INVALID),
    (dict(branch=0, post=0, gate=1), INVALID), (dict(eps=0.0), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(weight_offset=float("nan")), INVALID), (dict(branch_scale=float("inf")), INVALID),
    (dict(hidden=16385), UNSUPPORTED),
])
def test_norm_configurations(lib, kw, status):
    from nvfp4_token_quantized_gb300.binding import moe_norm_grad_io, moe_norm_io

    cfg = ctypes.byref(_norm_cfg(**kw))
    assert lib.moe_block_norm(cfg, ctypes.byref(moe_norm_io()), 0, None) == status
    assert (lib.moe_block_norm_workspace_bytes(cfg, 10) > 0) == (status == OK)
    if status != OK:
        assert lib.moe_block_norm_backward(cfg, ctypes.byref(moe_norm_grad_io()), 4, None) == status


def test_norm_operands(lib):
    from nvfp4_token_quantized_gb300.binding import moe_norm_io

    def call(rows=4, **kw):
        gate = kw.pop("gate_kind", 0)
        d = dict(y=1 << 20, residual=2 << 20, residual_out=3 << 20, h=4 << 20, post_weight=5 << 20,
                 pre_weight=6 << 20, y_stride=64, residual_stride=64, residual_out_stride=64, h_stride=64,
                 gate_stride=64)
        d.update(kw)
        return lib.moe_block_norm(ctypes.byref(_norm_cfg(gate=gate)), ctypes.byref(moe_norm_io(**d)), rows, None)

    assert lib.moe_block_norm(ctypes.byref(_norm_cfg()), None, 4, None) == INVALID
    for bad in (dict(rows=-1), dict(y=None), dict(residual=None), dict(residual_out=None), dict(h=None),
                dict(y=(1 << 20) + 1), dict(pre_weight=(6 << 20) + 1), dict(y_stride=63), dict(h_stride=0),
                dict(h_stride=1 << 62), dict(gate_kind=1), dict(gate_kind=3, gate=7 << 20, gate_stride=8)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(residual_out=1 << 20), dict(h=2 << 20), dict(h=3 << 20), dict(h=5 << 20),
                dict(residual_out=(2 << 20) + 2), dict(residual_out=2 << 20, residual_out_stride=72),
                dict(h=6 << 20), dict(gate_kind=2, gate=4 << 20)):
        assert call(**bad) == ALIAS, bad


def test_norm_gradient_operands(lib):
    from nvfp4_token_quantized_gb300.binding import moe_norm_grad_io

    def call(rows=4, **kw):
        d = dict(dresidual_out=1 << 20, dh=2 << 20, residual_out=3 << 20, y=4 << 20, post_weight=5 << 20,
                 pre_weight=6 << 20, dresidual=7 << 20, dy=8 << 20, dpost_weight=9 << 20, dpre_weight=10 << 20,
                 workspace=16 << 20)
        d.update({n: 64 for n in ("dresidual_out_stride", "dh_stride", "residual_out_stride", "y_stride",
                                  "dresidual_stride", "dy_stride")})
        d.update(kw)
        return lib.moe_block_norm_backward(ctypes.byref(_norm_cfg()), ctypes.byref(moe_norm_grad_io(**d)), rows, None)

    assert lib.moe_block_norm_backward(ctypes.byref(_norm_cfg()), None, 4, None) == INVALID
    for bad in (dict(rows=-1), dict(dh=None), dict(residual_out=None), dict(y=None), dict(dresidual=None),
                dict(dy=None), dict(workspace=None), dict(workspace=(16 << 20) + 8), dict(dy_stride=60)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dresidual=3 << 20), dict(dy=3 << 20), dict(dy=1 << 20), dict(dy=7 << 20),
                dict(dpre_weight=5 << 20), dict(dpre_weight=9 << 20), dict(workspace=8 << 20),
                dict(dy=(2 << 20) + 128, dy_stride=64)):
        assert call(**bad) == ALIAS, bad
