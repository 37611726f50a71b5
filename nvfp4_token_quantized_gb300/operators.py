"""The operators around the expert layer: the choice of experts and the norms
before and after a block, each with its gradient (``moe_route_select`` and
``moe_block_norm`` of ``include/moe_nvfp4.h``).

Argument checks and marshalling only, as in ``binding``.  Tensors live on the
current CUDA device; rows may be strided, their elements may not.  Results
that are not passed in are allocated here, on the stream the call runs on.
Nothing is recorded for autograd: results never require a gradient, and the
backward calls are the caller's to make.
"""

from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from .binding import (MOE_DTYPE_BF16, MOE_DTYPE_F16, MOE_DTYPE_F32, MOE_GATE_CHANNEL, MOE_GATE_FULL, MOE_GATE_NONE,
                      MOE_GATE_TOKEN, MOE_GROUP_MAX, MOE_GROUP_TOP2, MOE_NORM_LAYER, MOE_NORM_RMS, MOE_OK,
                      MOE_SCORE_SIGMOID, MOE_SCORE_SOFTMAX, MoEError, load_library, moe_norm_config,
                      moe_norm_grad_io, moe_norm_io, moe_route_config)

_DTYPES = {torch.bfloat16: MOE_DTYPE_BF16, torch.float16: MOE_DTYPE_F16, torch.float32: MOE_DTYPE_F32}
_SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}
_GROUP_SCORES = {"max": MOE_GROUP_MAX, "top2": MOE_GROUP_TOP2}
_KINDS = {"rms": MOE_NORM_RMS, "layer": MOE_NORM_LAYER}
_GATES = {None: MOE_GATE_NONE, "none": MOE_GATE_NONE, "channel": MOE_GATE_CHANNEL, "token": MOE_GATE_TOKEN,
          "full": MOE_GATE_FULL}


def _choice(table, key, name):
    if key not in table:
        raise ValueError(f"{name} must be one of {[k for k in table if k is not None]}, got {key!r}")
    return table[key]


def _device(t, name: str) -> int:
    """The CUDA ordinal of t, which must be the current device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev != _current_device():
        raise ValueError(f"{name} is on cuda:{dev} but the current device is cuda:{_current_device()}")
    return dev


def _rows(t, dtype, rows: int, width: int, name: str, dev: int) -> int:
    """Checks a [rows, width] tensor; returns its row stride."""
    try:
        if t.shape == (rows, width) and t.dtype is dtype and t.get_device() == dev:
            s0, s1 = t.stride()
            if s0 >= width and s1 == 1:
                return s0
    except AttributeError:
        raise TypeError(f"{name} must be a torch tensor") from None
    if t.shape != (rows, width):
        raise ValueError(f"{name} must be [{rows}, {width}], got {tuple(t.shape)}")
    if t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be a {dtype} tensor on cuda:{dev}")
    if s1 != 1 and width > 1:
        raise ValueError(f"{name}: the elements of a row must be next to each other")
    if rows > 1 and s0 < width:
        raise ValueError(f"{name}: rows overlap (row stride {s0}, width {width})")
    return max(s0, width)


def _vector(t, dtype, n: int, name: str, dev: int) -> int:
    """Checks a contiguous tensor of n elements; returns its address."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.numel() == n and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        raise TypeError(f"{name} must be a torch tensor") from None
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements on cuda:{dev}")


class _OnStream:
    """The stream of a call: its handle, and (inside ``with``) the stream that
    new tensors belong to."""

    def __init__(self, stream, dev: int):
        if isinstance(stream, torch.cuda.Stream):
            self.handle, self._ctx = stream.cuda_stream, torch.cuda.stream(stream)
        else:
            self.handle = int(stream)
            self._ctx = torch.cuda.stream(torch.cuda.ExternalStream(self.handle, device=dev))

    def __enter__(self):
        self._ctx.__enter__()
        return self

    def __exit__(self, *a):
        return self._ctx.__exit__(*a)


# The current stream's handle, the current device and new tensors on it, by
# torch's own cheap calls where it has them (a Stream object costs as much as a
# launch, torch.empty two thirds of one).
_current = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
try:
    _empty_strided = torch._C._dynamo.guards._empty_strided_cuda
except AttributeError:  # pragma: no cover
    def _empty_strided(size, stride, dtype):
        return torch.empty_strided(size, stride, dtype=dtype, device="cuda")


def _new_rows(rows: int, width: int, dtype):
    return _empty_strided((rows, width), (width, 1), dtype)


def _new_vector(n: int, dtype):
    return _empty_strided((n,), (1,), dtype)


def _ok(st: int, what: str) -> None:
    if st != MOE_OK:
        raise MoEError(st, what)


class ExpertRouter:
    """A rule that chooses ``top_k`` of ``num_experts`` experts a token.

    score: "softmax" or "sigmoid"; num_groups / top_groups: the experts form
    equal groups and only the best top_groups of them may be chosen, a group
    scoring its best expert ("max") or its best two ("top2"); renormalize: the
    chosen scores sum to one; scale: a factor on the weights.
    """

    def __init__(self, num_experts: int, top_k: int, score: str = "softmax", num_groups: int = 1,
                 top_groups: int = 1, group_score: str = "max", renormalize: bool = True, scale: float = 1.0):
        self.E, self.K = int(num_experts), int(top_k)
        self.config = moe_route_config(self.E, self.K, _choice(_SCORES, score, "score"), int(num_groups),
                                       int(top_groups), _choice(_GROUP_SCORES, group_score, "group_score"),
                                       int(bool(renormalize)), float(scale))
        self._cfg = ctypes.byref(self.config)
        self._lib = load_library()
        # (no tokens: only the configuration is looked at)
        _ok(self._lib.moe_route_select(self._cfg, None, MOE_DTYPE_F32, 0, None, 0, None, None, None),
            f"ExpertRouter(num_experts={num_experts}, top_k={top_k}, num_groups={num_groups}, "
            f"top_groups={top_groups}, scale={scale})")

    def _logits(self, logits):
        dev = _device(logits, "logits")
        dt = _DTYPES.get(logits.dtype)
        if dt is None:
            raise ValueError("logits must be bfloat16, float16 or float32")
        shape = logits.shape
        if len(shape) != 2:
            raise ValueError(f"logits must be [num_tokens, {self.E}], got {tuple(shape)}")
        return dev, dt, shape[0], _rows(logits, logits.dtype, shape[0], self.E, "logits", dev)

    def select(self, logits: torch.Tensor, bias: Optional[torch.Tensor] = None, ids: Optional[torch.Tensor] = None,
               weights: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """(ids int32 [T, K], weights float32 [T, K]) of logits [T, E]; bias:
        float32 [E], added to the scores for the choice only."""
        if stream is not None:
            with _OnStream(stream, _device(logits, "logits")) as on:
                return self._select(logits, bias, ids, weights, on.handle)
        return self._select(logits, bias, ids, weights, None)

    def _select(self, logits, bias, ids, weights, stream):
        dev, dt, T, ld = self._logits(logits)
        n = T * self.K
        b = None if bias is None else _vector(bias, torch.float32, self.E, "bias", dev)
        if ids is None:
            ids = _new_rows(T, self.K, torch.int32)
            pi = ids.data_ptr()
        elif ids.shape != (T, self.K):
            raise ValueError(f"ids must be [{T}, {self.K}], got {tuple(ids.shape)}")
        else:
            pi = _vector(ids, torch.int32, n, "ids", dev)
        if weights is None:
            weights = _new_rows(T, self.K, torch.float32)
            pw = weights.data_ptr()
        elif weights.shape != (T, self.K):
            raise ValueError(f"weights must be [{T}, {self.K}], got {tuple(weights.shape)}")
        else:
            pw = _vector(weights, torch.float32, n, "weights", dev)
        st = self._lib.moe_route_select(self._cfg, logits.data_ptr(), dt, ld, b, T, pi, pw,
                                        _current(dev) if stream is None else stream)
        if st != MOE_OK:
            raise MoEError(st, f"moe_route_select(T={T}, E={self.E}, K={self.K})")
        return ids, weights

    def select_backward(self, logits: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor,
                        dweights: torch.Tensor, dlogits: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Gradient of the logits from that of the weights (float32 [T, K]),
        the choice held fixed; logits, ids and weights as in ``select``."""
        if stream is not None:
            with _OnStream(stream, _device(logits, "logits")) as on:
                return self._select_backward(logits, ids, weights, dweights, dlogits, on.handle)
        return self._select_backward(logits, ids, weights, dweights, dlogits, None)

    def _select_backward(self, logits, ids, weights, dweights, dlogits, stream):
        dev, dt, T, ld = self._logits(logits)
        n = T * self.K
        if dlogits is None:
            dlogits, ldd = _new_rows(T, self.E, logits.dtype), self.E
        else:
            ldd = _rows(dlogits, logits.dtype, T, self.E, "dlogits", dev)
        st = self._lib.moe_route_select_backward(
            self._cfg, logits.data_ptr(), dt, ld, _vector(ids, torch.int32, n, "ids", dev),
            _vector(weights, torch.float32, n, "weights", dev), _vector(dweights, torch.float32, n, "dweights", dev),
            T, dlogits.data_ptr(), ldd, _current(dev) if stream is None else stream)
        if st != MOE_OK:
            raise MoEError(st, f"moe_route_select_backward(T={T}, E={self.E}, K={self.K})")
        return dlogits


class BlockNorm:
    """The norms on both sides of a block, its gate and its residual.

    post: norm the block's output y; pre: norm the new residual for the next
    block; kind: "rms" or "layer" (centred); gate: None, "channel" [H],
    "token" [T] or "full" [T, H], through a sigmoid first with gate_sigmoid;
    weight_offset: added to the stored weights; branch_scale: factor on the
    gated output.
    """

    def __init__(self, hidden: int, kind: str = "rms", eps: float = 1e-6, post: bool = True, pre: bool = True,
                 gate: Optional[str] = None, gate_sigmoid: bool = False, weight_offset: float = 0.0,
                 branch_scale: float = 1.0):
        self.H = int(hidden)
        self.kind, self.gate = _choice(_KINDS, kind, "kind"), _choice(_GATES, gate, "gate")
        self.post, self.pre, self.gate_sigmoid = bool(post), bool(pre), bool(gate_sigmoid)
        self.eps, self.weight_offset, self.branch_scale = float(eps), float(weight_offset), float(branch_scale)
        self._configs = {}
        self._lib = load_library()
        # (no rows: only the configuration is looked at)
        _ok(self._lib.moe_block_norm(self._config(True, torch.float32, torch.float32, torch.float32),
                                          ctypes.byref(moe_norm_io()), 0, None),
            f"BlockNorm(hidden={hidden}, eps={eps}, weight_offset={weight_offset}, branch_scale={branch_scale})")

    def _config(self, branch: bool, dtype, residual_dtype, weight_dtype):
        key = (branch, dtype, residual_dtype, weight_dtype)
        cfg = self._configs.get(key)
        if cfg is None:
            for name, t in (("y, gate and h", dtype), ("the residual", residual_dtype), ("weights", weight_dtype)):
                if t not in _DTYPES:
                    raise ValueError(f"{name} must be bfloat16, float16 or float32, not {t}")
            for name, t in (("the residual", residual_dtype), ("weights", weight_dtype)):
                if t not in (dtype, torch.float32):
                    raise ValueError(f"{name} must be {dtype} or float32, not {t}")
            if not branch and not self.pre:
                raise ValueError("without y there is only the pre-norm, which this BlockNorm leaves out")
            c = moe_norm_config(self.H, self.kind, int(branch), int(branch and self.post), int(self.pre),
                                self.gate if branch else MOE_GATE_NONE, int(self.gate_sigmoid), _DTYPES[dtype],
                                _DTYPES[residual_dtype], _DTYPES[weight_dtype], self.eps, self.weight_offset,
                                self.branch_scale)
            cfg = self._configs[key] = ctypes.byref(c)
        return cfg

    def _weights(self, branch, post_weight, pre_weight, dtype, dev):
        """Addresses of the weights in use (None: no weight) and their type."""
        post = post_weight if branch and self.post else None
        pre = pre_weight if self.pre else None
        w = post if post is not None else pre
        wt = dtype if w is None else w.dtype
        return (None if post is None else _vector(post, wt, self.H, "post_weight", dev),
                None if pre is None else _vector(pre, wt, self.H, "pre_weight", dev), wt)

    def _gate(self, branch, gate, dtype, T, dev):
        """Address and row stride of the gate."""
        if not branch or self.gate == MOE_GATE_NONE:
            return None, 0
        if self.gate == MOE_GATE_FULL:
            ld = _rows(gate, dtype, T, self.H, "gate", dev)
            return gate.data_ptr(), ld
        return _vector(gate, dtype, self.H if self.gate == MOE_GATE_CHANNEL else T, "gate", dev), 0

    def forward(self, residual: torch.Tensor, y: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                post_weight: Optional[torch.Tensor] = None, pre_weight: Optional[torch.Tensor] = None,
                residual_out: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
                stream=None) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
        """(residual_out, h) from the residual [T, H] and the block's output y
        [T, H]; without y, (None, h) with h the norm of the residual, in the
        type of a given h, else the residual's."""
        if stream is not None:
            with _OnStream(stream, _device(residual, "residual")) as on:
                return self._forward(residual, y, gate, post_weight, pre_weight, residual_out, h, on.handle)
        return self._forward(residual, y, gate, post_weight, pre_weight, residual_out, h, None)

    def _forward(self, residual, y, gate, post_weight, pre_weight, residual_out, h, stream):
        dev = _device(residual, "residual")
        shape = residual.shape
        if len(shape) != 2:
            raise ValueError(f"residual must be [num_tokens, {self.H}], got {tuple(shape)}")
        T, rt = shape[0], residual.dtype
        branch = y is not None
        dt = y.dtype if branch else rt if h is None else h.dtype
        r_ld = _rows(residual, rt, T, self.H, "residual", dev)
        wp, wn, wt = self._weights(branch, post_weight, pre_weight, dt, dev)
        cfg = self._config(branch, dt, rt, wt)
        g, g_ld = self._gate(branch, gate, dt, T, dev)
        py = po = ph = None
        y_ld = o_ld = h_ld = self.H
        if branch:
            y_ld = _rows(y, dt, T, self.H, "y", dev)
            py = y.data_ptr()
            if residual_out is None:
                residual_out = _new_rows(T, self.H, rt)
            else:
                o_ld = _rows(residual_out, rt, T, self.H, "residual_out", dev)
            po = residual_out.data_ptr()
        else:
            residual_out = None
        if self.pre:
            if h is None:
                h = _new_rows(T, self.H, dt)
            else:
                h_ld = _rows(h, dt, T, self.H, "h", dev)
            ph = h.data_ptr()
        else:
            h = None
        io = moe_norm_io(py, residual.data_ptr(), g, wp, wn, po, ph, y_ld, r_ld, g_ld, o_ld, h_ld)
        st = self._lib.moe_block_norm(cfg, ctypes.byref(io), T, _current(dev) if stream is None else stream)
        if st != MOE_OK:
            raise MoEError(st, f"moe_block_norm(T={T}, H={self.H})")
        return residual_out, h

    def backward(self, dresidual_out: Optional[torch.Tensor], dh: Optional[torch.Tensor],
                 residual_out: Optional[torch.Tensor], y: Optional[torch.Tensor] = None,
                 gate: Optional[torch.Tensor] = None, post_weight: Optional[torch.Tensor] = None,
                 pre_weight: Optional[torch.Tensor] = None, dresidual: Optional[torch.Tensor] = None,
                 dy: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
        """(dresidual, dy, dgate, dpost_weight, dpre_weight), None where the
        forward had no such operand.  residual_out: the forward's result (the
        residual itself without y); dresidual_out may be None (zero); the
        weights' and a channel gate's gradients are float32.  workspace: a
        CUDA tensor of at least ``workspace_bytes`` bytes to use instead of a
        new one."""
        args = (dresidual_out, dh, residual_out, y, gate, post_weight, pre_weight, dresidual, dy, workspace)
        if stream is not None:
            first = dh if dresidual_out is None else dresidual_out
            with _OnStream(stream, _device(first, "the incoming gradient")) as on:
                return self._backward(*args, on.handle)
        return self._backward(*args, None)

    def workspace_bytes(self, rows: int, branch: bool = True) -> int:
        """Bytes of workspace the gradient of ``rows`` rows needs."""
        cfg = self._config(branch, torch.float32, torch.float32, torch.float32)
        return int(self._lib.moe_block_norm_workspace_bytes(cfg, rows))

    def _backward(self, dresidual_out, dh, residual_out, y, gate, post_weight, pre_weight, dresidual, dy, workspace,
                  stream):
        H, lib = self.H, self._lib
        first = dh if dresidual_out is None else dresidual_out
        dev = _device(first, "the incoming gradient")
        if len(first.shape) != 2:
            raise ValueError(f"gradients must be [num_tokens, {H}], got {tuple(first.shape)}")
        T, branch = first.shape[0], y is not None
        rt = dresidual_out.dtype if residual_out is None else residual_out.dtype
        dt = y.dtype if branch else dh.dtype if dh is not None else rt
        wp, wn, wt = self._weights(branch, post_weight, pre_weight, dt, dev)
        cfg = self._config(branch, dt, rt, wt)
        g, g_ld = self._gate(branch, gate, dt, T, dev)
        p_in = ph = px = py = pdy = pdg = pdp = pdn = ws = None
        in_ld = h_ld = x_ld = y_ld = dr_ld = dy_ld = H
        if dresidual_out is not None:
            in_ld = _rows(dresidual_out, rt, T, H, "dresidual_out", dev)
            p_in = dresidual_out.data_ptr()
        if self.pre:
            h_ld = _rows(dh, dt, T, H, "dh", dev)
            x_ld = _rows(residual_out, rt, T, H, "residual_out", dev)
            ph, px = dh.data_ptr(), residual_out.data_ptr()
        if dresidual is None:
            dresidual = _new_rows(T, H, rt)
        else:
            dr_ld = _rows(dresidual, rt, T, H, "dresidual", dev)
        dgate = dpost = dpre = None
        if branch:
            y_ld = _rows(y, dt, T, H, "y", dev)
            py = y.data_ptr()
            if dy is None:
                dy = _new_rows(T, H, dt)
            else:
                dy_ld = _rows(dy, dt, T, H, "dy", dev)
            pdy = dy.data_ptr()
            if g is not None:
                dgate = (_new_rows(T, H, dt) if self.gate == MOE_GATE_FULL else
                         torch.empty_like(gate, dtype=torch.float32 if self.gate == MOE_GATE_CHANNEL else dt))
                pdg = dgate.data_ptr()
            if wp is not None:
                dpost = _new_vector(H, torch.float32)
                pdp = dpost.data_ptr()
        else:
            dy = None
        if wn is not None:
            dpre = _new_vector(H, torch.float32)
            pdn = dpre.data_ptr()
        need = int(lib.moe_block_norm_workspace_bytes(cfg, T))
        if need:
            if workspace is None:
                workspace = _new_vector(need, torch.uint8)
            elif workspace.get_device() != dev or not workspace.is_contiguous() or workspace.nbytes < need:
                raise ValueError(f"workspace must be a contiguous tensor of {need} bytes or more on cuda:{dev}")
            ws = workspace.data_ptr()
        io = moe_norm_grad_io(p_in, ph, px, py, g, wp, wn, dresidual.data_ptr(), pdy, pdg, pdp, pdn, ws, in_ld, h_ld,
                              x_ld, y_ld, g_ld, dr_ld, dy_ld, H)
        st = lib.moe_block_norm_backward(cfg, ctypes.byref(io), T, _current(dev) if stream is None else stream)
        if st != MOE_OK:
            raise MoEError(st, f"moe_block_norm_backward(T={T}, H={H})")
        return dresidual, dy, dgate, dpost, dpre
