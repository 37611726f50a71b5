"""The adapters' calls for tests of their waits, without a GPU: the same refusals as the
usual calls, and one for a negative CTA."""

import ctypes

import pytest

INVALID_ARG, UNSUPPORTED = 1, 8


@pytest.fixture(scope="module")
def lib():
    from nvfp4_token_quantized_gb300 import build, load_library

    build()
    return load_library()


@pytest.mark.parametrize("silent", [0, 1, 8])
def test_refusals_are_those_of_the_call(lib, silent):
    from nvfp4_token_quantized_gb300.binding import moe_adapter_config, moe_adapter_grad_io, moe_adapter_io

    ok = moe_adapter_config(64, 64, 8, 2, 1)
    io, grad = moe_adapter_io(), moe_adapter_grad_io()
    for cfg in (None, moe_adapter_config(0, 64, 8, 2, 1), moe_adapter_config(64, 64, 129, 2, 1),
                moe_adapter_config(64, 64, 8, 2, 3), ok):
        c = None if cfg is None else ctypes.byref(cfg)
        for rows in (-1, 600):
            want = lib.moe_adapter_forward(c, ctypes.byref(io), rows, None)
            assert want in (INVALID_ARG, UNSUPPORTED)
            assert lib.moe_debug_adapter_forward(c, ctypes.byref(io), rows, silent, None) == want
            want = lib.moe_adapter_backward(c, ctypes.byref(grad), rows, None)
            assert want in (INVALID_ARG, UNSUPPORTED)
            assert lib.moe_debug_adapter_backward(c, ctypes.byref(grad), rows, silent, None) == want
    assert lib.moe_debug_adapter_forward(ctypes.byref(ok), ctypes.byref(io), 0, silent, None) == 0


def test_a_negative_cta_is_refused(lib):
    from nvfp4_token_quantized_gb300.binding import moe_adapter_config, moe_adapter_grad_io, moe_adapter_io

    ok = ctypes.byref(moe_adapter_config(64, 64, 8, 2, 1))
    assert lib.moe_debug_adapter_forward(ok, ctypes.byref(moe_adapter_io()), 0, -1, None) == INVALID_ARG
    assert lib.moe_debug_adapter_backward(ok, ctypes.byref(moe_adapter_grad_io()), 0, -1, None) == INVALID_ARG
