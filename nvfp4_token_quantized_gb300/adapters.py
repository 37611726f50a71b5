"""Low-rank adapters of many requests beside a projection, with their gradients
(``moe_adapter_forward`` and ``moe_adapter_backward`` of ``include/moe_nvfp4.h``):
argument checks and marshalling only, as in ``operators``."""

from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from .binding import (MOE_DTYPE_BF16, MOE_DTYPE_F16, MOE_OK, MoEError, load_library, moe_adapter_config,
                      moe_adapter_grad_io, moe_adapter_io)
from .operators import _OnStream, _current, _device, _empty_strided, _new_rows, _new_vector, _rows, _vector

# (forwards of so few rows need no workspace: not asked for, a call less)
_FEW_ROWS = 256
_HALVES = {torch.bfloat16: MOE_DTYPE_BF16, torch.float16: MOE_DTYPE_F16}


class LowRankAdapters:
    """Adapters of one rank beside a projection of ``in_features`` to
    ``out_features``: row t of a batch, with adapter a = ids[t], gets

        hidden = scales[a] * x down[a]^T,  out = base + hidden up[a].

    down [L, rank, in_features] and up [L, rank, out_features] hold L adapters
    (lower ranks: rows of zeros), bfloat16 or float16 as x; ids outside [0, L)
    stand for no adapter.
    """

    def __init__(self, in_features: int, out_features: int, rank: int):
        self.K, self.N, self.rank = int(in_features), int(out_features), int(rank)
        self._configs = {}
        self._lib = load_library()
        cfg = moe_adapter_config(self.K, self.N, self.rank, 1, MOE_DTYPE_BF16)
        # (no rows: only the configuration is looked at)
        st = self._lib.moe_adapter_forward(ctypes.byref(cfg), ctypes.byref(moe_adapter_io()), 0, None)
        if st != MOE_OK:
            raise MoEError(st, f"LowRankAdapters(in_features={in_features}, out_features={out_features}, rank={rank})")

    def _config(self, L: int, dtype):
        key = (L, dtype)
        cfg = self._configs.get(key)
        if cfg is None:
            if dtype not in _HALVES:
                raise ValueError(f"rows and factors must be bfloat16 or float16, not {dtype}")
            cfg = self._configs[key] = ctypes.byref(moe_adapter_config(self.K, self.N, self.rank, L, _HALVES[dtype]))
        return cfg

    def _factors(self, down, up, dtype, dev):
        """The number of adapters and the factors' addresses."""
        if not isinstance(down, torch.Tensor) or not isinstance(up, torch.Tensor):
            raise TypeError("down and up must be torch tensors")
        L = down.shape[0] if down.dim() == 3 else 0
        if L < 1 or down.shape != (L, self.rank, self.K):
            raise ValueError(f"down must be [adapters, {self.rank}, {self.K}], got {tuple(down.shape)}")
        if up.shape != (L, self.rank, self.N):
            raise ValueError(f"up must be [{L}, {self.rank}, {self.N}], got {tuple(up.shape)}")
        return (L, _vector(down, dtype, L * self.rank * self.K, "down", dev),
                _vector(up, dtype, L * self.rank * self.N, "up", dev))

    def workspace_bytes(self, rows: int, num_adapters: int, backward: bool = False) -> int:
        """Bytes of workspace a call of ``rows`` rows needs."""
        return int(self._lib.moe_adapter_workspace_bytes(self._config(num_adapters, torch.bfloat16), rows,
                                                         int(backward)))

    def _workspace(self, cfg, T, backward, workspace, dev):
        if T <= _FEW_ROWS and not backward:
            return None, None
        need = int(self._lib.moe_adapter_workspace_bytes(cfg, T, backward))
        if need == 0:
            return None, None
        if workspace is None:
            workspace = _new_vector(need, torch.uint8)
        elif workspace.get_device() != dev or not workspace.is_contiguous() or workspace.nbytes < need:
            raise ValueError(f"workspace must be a contiguous tensor of {need} bytes or more on cuda:{dev}")
        return workspace.data_ptr(), workspace

    @staticmethod
    def _batch(x, width, name):
        dev = _device(x, name)
        if len(x.shape) != 2:
            raise ValueError(f"{name} must be [num_tokens, {width}], got {tuple(x.shape)}")
        return dev, x.shape[0], _rows(x, x.dtype, x.shape[0], width, name, dev)

    def forward(self, x: torch.Tensor, ids: torch.Tensor, down: torch.Tensor, up: torch.Tensor,
                scales: Optional[torch.Tensor] = None, base: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, keep_hidden: bool = False,
                workspace: Optional[torch.Tensor] = None,
                stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
        """(out [T, out_features], hidden): x [T, in_features], ids int32 [T],
        scales float32 [L] (none: 1), base [T, out_features], the projection's
        own rows (none: zeros); out may be base.  hidden, float32 [T, rank], is
        what ``backward`` needs (None without keep_hidden)."""
        if stream is not None:
            with _OnStream(stream, _device(x, "x")) as on:
                return self._forward(x, ids, down, up, scales, base, out, keep_hidden, workspace, on.handle)
        return self._forward(x, ids, down, up, scales, base, out, keep_hidden, workspace, None)

    def _forward(self, x, ids, down, up, scales, base, out, keep_hidden, workspace, stream):
        dev, T, x_ld = self._batch(x, self.K, "x")
        dt = x.dtype
        L, pd, pu = self._factors(down, up, dt, dev)
        cfg = self._config(L, dt)
        pb, b_ld, o_ld = None, self.N, self.N
        if base is not None:
            b_ld = _rows(base, dt, T, self.N, "base", dev)
            pb = base.data_ptr()
        if out is None:
            out = _new_rows(T, self.N, dt)
        else:
            o_ld = _rows(out, dt, T, self.N, "out", dev)
        hidden = _new_rows(T, self.rank, torch.float32) if keep_hidden else None
        ws, _keep = self._workspace(cfg, T, 0, workspace, dev)
        io = moe_adapter_io(x.data_ptr(), pb, pd, pu, _vector(ids, torch.int32, T, "ids", dev),
                            None if scales is None else _vector(scales, torch.float32, L, "scales", dev),
                            out.data_ptr(), None if hidden is None else hidden.data_ptr(), ws, x_ld, b_ld, o_ld)
        st = self._lib.moe_adapter_forward(cfg, ctypes.byref(io), T, _current(dev) if stream is None else stream)
        if st != MOE_OK:
            raise MoEError(st, f"moe_adapter_forward(T={T}, in={self.K}, out={self.N}, rank={self.rank}, adapters={L})")
        return out, hidden

    def backward(self, dout: torch.Tensor, x: torch.Tensor, hidden: torch.Tensor, ids: torch.Tensor,
                 down: torch.Tensor, up: torch.Tensor, scales: Optional[torch.Tensor] = None,
                 base: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
        """(dx, ddown, dup) from dout [T, out_features], the forward's x, ids,
        factors and scales, and its hidden; base [T, in_features]: rows that dx
        is added to (dx may be base), such as the projection's own gradient."""
        args = (dout, x, hidden, ids, down, up, scales, base, dx, workspace)
        if stream is not None:
            with _OnStream(stream, _device(dout, "dout")) as on:
                return self._backward(*args, on.handle)
        return self._backward(*args, None)

    def _backward(self, dout, x, hidden, ids, down, up, scales, base, dx, workspace, stream):
        dev, T, g_ld = self._batch(dout, self.N, "dout")
        dt = dout.dtype
        L, pd, pu = self._factors(down, up, dt, dev)
        cfg = self._config(L, dt)
        x_ld = _rows(x, dt, T, self.K, "x", dev)
        if hidden is None or hidden.shape != (T, self.rank):
            raise ValueError(f"hidden must be [{T}, {self.rank}], as the forward gave it with keep_hidden")
        pb, b_ld, dx_ld = None, self.K, self.K
        if base is not None:
            b_ld = _rows(base, dt, T, self.K, "base", dev)
            pb = base.data_ptr()
        if dx is None:
            dx = _new_rows(T, self.K, dt)
        else:
            dx_ld = _rows(dx, dt, T, self.K, "dx", dev)
        ddown = _empty_strided((L, self.rank, self.K), (self.rank * self.K, self.K, 1), dt)
        dup = _empty_strided((L, self.rank, self.N), (self.rank * self.N, self.N, 1), dt)
        ws, _keep = self._workspace(cfg, T, 1, workspace, dev)
        io = moe_adapter_grad_io(dout.data_ptr(), x.data_ptr(), pb, pd, pu, _vector(ids, torch.int32, T, "ids", dev),
                                 None if scales is None else _vector(scales, torch.float32, L, "scales", dev),
                                 _vector(hidden, torch.float32, T * self.rank, "hidden", dev), dx.data_ptr(),
                                 ddown.data_ptr(), dup.data_ptr(), ws, g_ld, x_ld, b_ld, dx_ld)
        st = self._lib.moe_adapter_backward(cfg, ctypes.byref(io), T, _current(dev) if stream is None else stream)
        if st != MOE_OK:
            raise MoEError(st, f"moe_adapter_backward(T={T}, in={self.K}, out={self.N}, rank={self.rank}, "
                               f"adapters={L})")
        return dx, ddown, dup
