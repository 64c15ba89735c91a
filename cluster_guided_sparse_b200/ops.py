"""Operators around the sparse attention of a transformer block: rotary
positions, the same behind a per-head RMS norm, with gradients.

Argument marshalling over libscope.so, as in the package's other entry points:
tensors are [B, H, N, D] device tensors of any layout with contiguous, 16-byte
aligned rows, all on one device (which need not be the current one).  A call
runs on `stream`, by default the current stream of that device; given a
stream, its outputs and workspace are allocated on it and its inputs are kept
from reuse until the stream has passed.  Outputs take the inputs' layout.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
from typing import Optional

import torch

from . import ScopeGrid, ScopeParams, ScopeTensor, ScopeError, _check, lib

SCOPE_F16 = 4
_DT = {torch.float32: 0, torch.bfloat16: 1, torch.float16: SCOPE_F16}
_I4 = ctypes.c_int64 * 4


class ScopePositions(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("B", ctypes.c_int64)]


class ScopeVector(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("dtype", ctypes.c_int)]


@functools.lru_cache(maxsize=None)
def _functions():
    """libscope.so with these operators' argument types set."""
    L, P, V, Z = lib(), ctypes.POINTER, ctypes.c_void_p, ctypes.c_size_t
    T, G, R, F = P(ScopeTensor), P(ScopeGrid), P(ScopeParams), ctypes.c_float
    L.scope_rope.argtypes = [T, G, R, P(ScopePositions), P(ScopeVector), F, ctypes.c_int, T, V]
    L.scope_rope_backward_workspace_bytes.argtypes = [T]
    L.scope_rope_backward_workspace_bytes.restype = Z
    L.scope_rope_backward.argtypes = [T, T, G, R, P(ScopePositions), P(ScopeVector), F, T, P(ScopeVector), V, Z, V]
    return L


def _tensor(x: torch.Tensor, name: str) -> ScopeTensor:
    if x.dim() != 4:
        raise ValueError(f"{name}: expected a [B, H, N, D] tensor")
    dt = _DT.get(x.dtype)
    if dt is None:
        raise ValueError(f"{name}: unsupported dtype {x.dtype}")
    return ScopeTensor(x.data_ptr(), dt, *x.shape, _I4(*x.stride()))


def _vector(x: torch.Tensor, D: int, name: str) -> ScopeVector:
    if x.dim() != 1 or x.shape[0] != D or x.stride(0) != 1:
        raise ValueError(f"{name}: expected a contiguous vector of {D}")
    dt = _DT.get(x.dtype)
    if dt is None:
        raise ValueError(f"{name}: unsupported dtype {x.dtype}")
    return ScopeVector(x.data_ptr(), dt)


def _device(*tensors) -> torch.device:
    dev = tensors[0].device
    if dev.type != "cuda":
        raise ValueError("expected CUDA tensors")
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors on {dev} and {t.device}")
    return dev


class _Launch:
    """Device, stream and allocations of one call."""

    def __init__(self, dev: torch.device, stream, *inputs):
        self.dev, self.stream = dev, stream
        if stream is None:
            self.raw = torch.cuda.current_stream(dev).cuda_stream
        else:
            if stream.device != dev:
                raise ValueError(f"stream of {stream.device} for tensors on {dev}")
            self.raw = stream.cuda_stream
            for t in inputs:
                if t is not None:
                    t.record_stream(stream)

    def on_stream(self):
        return contextlib.nullcontext() if self.stream is None else torch.cuda.stream(self.stream)

    def like(self, x: torch.Tensor, out: Optional[torch.Tensor]) -> torch.Tensor:
        if out is not None:
            return out
        with self.on_stream():
            return torch.empty_like(x)

    def empty(self, shape, dtype) -> torch.Tensor:
        with self.on_stream():
            return torch.empty(shape, dtype=dtype, device=self.dev)

    def workspace(self, given: Optional[torch.Tensor], need: int) -> torch.Tensor:
        if given is not None and given.numel() * given.element_size() >= need:
            return given
        return self.empty(need, torch.uint8)

    def __call__(self, fn, *args):
        if torch.cuda.current_device() == self.dev.index:
            st = fn(*args, self.raw)
        else:
            with torch.cuda.device(self.dev):
                st = fn(*args, self.raw)
        if st:
            _check(st)


def _positions(positions: Optional[torch.Tensor], x: torch.Tensor):
    if positions is None:
        return None
    if positions.dtype != torch.int32 or not positions.is_contiguous():
        raise ValueError("positions must be contiguous int32")
    N = x.shape[2]
    shape = tuple(positions.shape)
    if shape not in ((N, 3), (1, N, 3), (x.shape[0], N, 3)):
        raise ValueError(f"positions must be [N, 3], [1, N, 3] or [B, N, 3] (got {list(shape)})")
    return ctypes.byref(ScopePositions(positions.data_ptr(), shape[0] if len(shape) == 3 else 1))


def _grid(grid):
    return None if grid is None else ctypes.byref(grid)


def rope(x: torch.Tensor, params: ScopeParams, grid: Optional[ScopeGrid] = None, *,
         positions: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
         inverse: bool = False, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rotary positions of x ([B, H, N, D] f32, bf16 or f16) on the (t, h, w)
    axes of `params` (d_t, d_h, d_w, theta): tokens of a raster `grid`, or
    int32 `positions` [N, 3] or [B, N, 3].  With a `weight` [D], each row goes
    through an RMS norm first.  inverse=True (without a weight) turns back,
    which is the gradient of the plain rotation.  `out` may be x."""
    dev = _device(x, positions, weight, out)
    call = _Launch(dev, stream, x, positions, weight, out)
    tx = _tensor(x, "x")
    pos = _positions(positions, x)
    w = None if weight is None else ctypes.byref(_vector(weight, x.shape[-1], "weight"))
    y = call.like(x, out)
    call(_functions().scope_rope, ctypes.byref(tx), _grid(grid), ctypes.byref(params), pos, w, eps, int(inverse),
         ctypes.byref(_tensor(y, "out")))
    return y


def rope_backward(dy: torch.Tensor, x: torch.Tensor, params: ScopeParams, grid: Optional[ScopeGrid] = None, *,
                  weight: torch.Tensor, positions: Optional[torch.Tensor] = None, eps: float = 1e-6,
                  out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """(dx, dw) of rope(x, ..., weight=weight) for the gradient dy of its
    output; `out` (dx) may be x or dy.  Without a weight the gradient is
    rope(dy, ..., inverse=True)."""
    dev = _device(dy, x, positions, weight, out, workspace)
    call = _Launch(dev, stream, dy, x, positions, weight, out, workspace)
    tx = _tensor(x, "x")
    pos = _positions(positions, x)
    w = _vector(weight, x.shape[-1], "weight")
    L = _functions()
    need = L.scope_rope_backward_workspace_bytes(ctypes.byref(tx))
    if need == 0:
        raise ScopeError(1, L.scope_last_error().decode())
    ws = call.workspace(workspace, need)
    dx = call.like(x, out)
    dw = call.empty(weight.shape, weight.dtype)
    call(L.scope_rope_backward, ctypes.byref(_tensor(dy, "dy")), ctypes.byref(tx), _grid(grid), ctypes.byref(params),
         pos, ctypes.byref(w), eps, ctypes.byref(_tensor(dx, "out")), ctypes.byref(_vector(dw, x.shape[-1], "dw")),
         ws.data_ptr(), ws.numel() * ws.element_size())
    return dx, dw
