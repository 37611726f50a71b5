"""The norm of a set of gradients and their clipping (``moe_gradient_norm`` and
``moe_clip_gradients`` of ``include/moe_nvfp4.h``): argument checks and
marshalling only, as in ``operators``."""

from __future__ import annotations

import array
import math
from typing import List, Optional, Sequence, Tuple

import torch

from .binding import MoEError, MOE_OK, load_library
from .operators import _DTYPES, _OnStream, _current, _current_device, _new_scalar, _new_vector


def _dense(t) -> bool:
    """Whether the elements fill one run of memory, in any order of the
    dimensions."""
    if t.is_contiguous():
        return True
    run = 1
    for size, stride in sorted(zip(t.shape, t.stride()), key=lambda d: (d[1], d[0])):
        if size != 1:
            if stride != run:
                return t.numel() == 0
            run *= size
    return True


class GradientClip:
    """Clipping of gradients by the norm of all of them together: with norm the
    square root of the sum of every element's square, each gradient is
    multiplied by min(1, max_norm / (norm + eps)).

    The gradients are dense CUDA tensors of bfloat16, float16 or float32, in any
    mixture, on the current device.  max_norm None: only ``norm`` is called.
    """

    def __init__(self, max_norm: Optional[float] = None, eps: float = 1e-6):
        self.max_norm, self.eps = None if max_norm is None else float(max_norm), float(eps)
        if self.max_norm is not None and not (math.isfinite(self.max_norm) and self.max_norm >= 0.0):
            raise ValueError(f"max_norm must be finite and not negative, got {max_norm}")
        if not (math.isfinite(self.eps) and self.eps > 0.0):
            raise ValueError(f"eps must be finite and positive, got {eps}")
        self._lib = load_library()
        self._bytes = int(self._lib.moe_gradient_workspace_bytes())

    def norm(self, grads: Sequence[torch.Tensor], stream=None) -> torch.Tensor:
        """The norm of all of grads together, a float32 scalar."""
        if stream is not None:
            with _OnStream(stream, _current_device()) as on:
                return self._run(grads, None, False, on.handle)
        return self._run(grads, None, False, None)

    def clip(self, grads: Sequence[torch.Tensor], out: Optional[Sequence[torch.Tensor]] = None,
             stream=None) -> Tuple[torch.Tensor, List[torch.Tensor]]:
        """(norm, the clipped gradients): in place, or into the tensors of out
        (of the same types and sizes, their elements in the same order)."""
        if self.max_norm is None:
            raise ValueError("this GradientClip has no max_norm")
        if stream is not None:
            with _OnStream(stream, _current_device()) as on:
                return self._run(grads, out, True, on.handle), list(grads if out is None else out)
        return self._run(grads, out, True, None), list(grads if out is None else out)

    def _run(self, grads, out, clip, stream):
        dev = _current_device()
        if out is not None and len(out) != len(grads):
            raise ValueError(f"out holds {len(out)} tensors for {len(grads)} gradients")
        table, n = self._table(grads, grads if out is None else out, dev), len(grads)
        norm, ws = _new_scalar(), _new_vector(self._bytes, torch.uint8)
        where = table.buffer_info()[0] if n else None
        stream = _current(dev) if stream is None else stream
        if clip:
            st = self._lib.moe_clip_gradients(where, n, self.max_norm, self.eps, norm.data_ptr(), ws.data_ptr(), stream)
        else:
            st = self._lib.moe_gradient_norm(where, n, norm.data_ptr(), ws.data_ptr(), stream)
        if st != MOE_OK:
            raise MoEError(st, f"{'moe_clip_gradients' if clip else 'moe_gradient_norm'} of {n} tensors")
        return norm

    @staticmethod
    def _table(grads, out, dev):
        """moe_gradient of each tensor, as one array of integers (by torch's
        own calls and in as few as can be: long lists cost their number)."""
        try:
            return _in_place(grads, dev) if out is grads else _apart(grads, out, dev)
        except (AttributeError, TypeError):
            raise TypeError("gradients must be torch tensors") from None


_base = torch._C.TensorBase
_data_ptr, _numel, _get_device, _is_contiguous = _base.data_ptr, _base.numel, _base.get_device, _base.is_contiguous


def _in_place(grads, dev):
    n = len(grads)
    types = [_DTYPES.get(t.dtype) for t in grads]
    if None in types or (n and set(map(_get_device, grads)) != {dev}) or not all(map(_is_contiguous, grads)):
        for i, t in enumerate(grads):
            _check(i, t, dev)
    table = array.array("q", bytes(32 * n))
    table[0::4] = table[1::4] = array.array("q", list(map(_data_ptr, grads)))
    table[2::4] = array.array("q", list(map(_numel, grads)))
    table[3::4] = array.array("q", types)
    return table


def _apart(grads, out, dev):
    rows = []
    for i, (t, o) in enumerate(zip(grads, out)):
        dt, n = _DTYPES.get(t.dtype), _numel(t)
        if not (dt is not None and o.dtype is t.dtype and _numel(o) == n and _get_device(t) == dev
                and _get_device(o) == dev and _is_contiguous(t) and _is_contiguous(o)):
            dt = _check(i, t, dev)
            if o.dtype is not t.dtype or o.shape != t.shape or o.get_device() != dev or o.stride() != t.stride():
                raise ValueError(f"out {i} must be laid out as gradient {i}: {tuple(t.shape)} of {t.dtype}, strides "
                                 f"{t.stride()}, on cuda:{dev}")
        rows += (_data_ptr(t), _data_ptr(o), n, dt)
    return array.array("q", rows)


def _check(i, t, dev) -> int:
    """The type's code of a gradient that can be taken: contiguous, or dense in
    another order of its dimensions."""
    if t.dtype not in _DTYPES:
        raise ValueError(f"gradient {i} must be bfloat16, float16 or float32, not {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"gradient {i} must be on cuda:{dev}, the current device")
    if not _dense(t):
        raise ValueError(f"gradient {i}: the elements must lie next to each other")
    return _DTYPES[t.dtype]
