"""Operators around the sparse attention of a transformer block: rotary
positions, the same behind a per-head RMS norm, and cross attention to states
of another length, with gradients.

Argument marshalling over libscope.so, as in the package's other entry points:
tensors are [B, H, N, D] device tensors of any layout with contiguous, 16-byte
aligned rows, all on one device (which need not be the current one).  A call
runs on `stream`, by default the current stream of that device; given a
stream, its outputs and workspace are allocated on it and its inputs are kept
from reuse until the stream has passed.  Outputs take the inputs' layout.

As with the package's other calls, results carry no autograd graph, whether or not
inputs require gradients: those come from the _backward functions, which a caller's
own torch.autograd.Function may wrap.  (The gradient of a plain sum arrives there as
one expanded element; contiguous() makes the tensor that these calls take.)
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import Optional

import torch

from . import ScopeGrid, ScopeParams, ScopeTensor, ScopeError, _check, _strides, _whole, lib

SCOPE_F16 = 4
_DT = {torch.float32: 0, torch.bfloat16: 1, torch.float16: SCOPE_F16}
# The C structs as bytes: packing one takes 0.8 us, filling a ctypes structure 2 us, which
# counts where a call's kernel takes less than its arguments.
_TENSOR = struct.Struct("=Qi4x8q").pack     # scope_tensor
_VECTOR = struct.Struct("=Qi4x").pack       # scope_vector
_POSITIONS = struct.Struct("=Qq").pack      # scope_positions
_KEYS = struct.Struct("=QQq").pack          # scope_keys


class ScopePositions(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("B", ctypes.c_int64)]


class ScopeVector(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("dtype", ctypes.c_int)]


class ScopeKeys(ctypes.Structure):
    _fields_ = [("len", ctypes.c_void_p), ("mask", ctypes.c_void_p), ("mask_stride", ctypes.c_int64)]


@functools.lru_cache(maxsize=None)
def _functions():
    """libscope.so with these operators' argument types set."""
    P, L = ctypes.POINTER, lib()
    return _bind(L, P(ScopeTensor), P(ScopePositions), P(ScopeVector), P(ScopeKeys))


@functools.lru_cache(maxsize=None)
def _packed():
    """The same functions, taking tensors, positions, vectors and keys as bytes."""
    return _bind(ctypes.CDLL(lib()._name), *[ctypes.c_char_p] * 4)


def _bind(L, T, S, W, K):
    P, V, Z = ctypes.POINTER, ctypes.c_void_p, ctypes.c_size_t
    G, R, F = P(ScopeGrid), P(ScopeParams), ctypes.c_float
    L.scope_rope.argtypes = [T, G, R, S, W, F, ctypes.c_int, T, V]
    L.scope_rope_backward_workspace_bytes.argtypes = [T]
    L.scope_rope_backward_workspace_bytes.restype = Z
    L.scope_rope_backward.argtypes = [T, T, G, R, S, W, F, T, W, V, Z, V]
    L.scope_cross_attn_workspace_bytes.argtypes = [T, T, ctypes.c_int]
    L.scope_cross_attn_workspace_bytes.restype = Z
    L.scope_cross_attn.argtypes = [T, T, T, K, F, T, V, V, Z, V]
    L.scope_cross_attn_backward_workspace_bytes.argtypes = [T, T, ctypes.c_int]
    L.scope_cross_attn_backward_workspace_bytes.restype = Z
    L.scope_cross_attn_backward.argtypes = [T, T, T, T, T, V, K, F, T, T, T, V, Z, V]
    L.scope_ops_sync_status.argtypes = [V]
    L.scope_ops_selftest_wait_timeout.argtypes = [ctypes.c_int, ctypes.c_int64, V]
    L.scope_last_error.restype = ctypes.c_char_p
    return L


def _tensor(x: torch.Tensor, name: str) -> bytes:
    if x.dim() != 4:
        raise ValueError(f"{name}: expected a [B, H, N, D] tensor")
    dt = _DT.get(x.dtype)
    if dt is None:
        raise ValueError(f"{name}: unsupported dtype {x.dtype}")
    return _TENSOR(x.data_ptr(), dt, *x.shape, *_strides(x, name))


def _vector(x: torch.Tensor, D: int, name: str) -> bytes:
    if x.dim() != 1 or x.shape[0] != D or x.stride(0) != 1:
        raise ValueError(f"{name}: expected a contiguous vector of {D}")
    dt = _DT.get(x.dtype)
    if dt is None:
        raise ValueError(f"{name}: unsupported dtype {x.dtype}")
    return _VECTOR(x.data_ptr(), dt)


def _device(*tensors) -> int:
    """Index of the one CUDA device that all tensors are on."""
    if not tensors[0].is_cuda:
        raise ValueError("expected CUDA tensors")
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors on {tensors[0].device} and {t.device}")
    return dev


class _Launch:
    """Device, stream and allocations of one call."""

    __slots__ = ("dev", "stream", "raw")

    def __init__(self, stream, *tensors):
        self.dev, self.stream = _device(*tensors), stream
        if stream is None:
            self.raw = torch._C._cuda_getCurrentRawStream(self.dev)
        else:
            if stream.device.index != self.dev:
                raise ValueError(f"stream of {stream.device} for tensors on {tensors[0].device}")
            self.raw = stream.cuda_stream
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)

    def like(self, x: torch.Tensor, out: Optional[torch.Tensor]) -> torch.Tensor:
        if out is not None:
            return out
        if self.stream is None:
            return torch.empty_like(x)
        with torch.cuda.stream(self.stream):
            return torch.empty_like(x)

    def empty(self, x: torch.Tensor, shape, dtype) -> torch.Tensor:
        """On x's device."""
        if self.stream is None:
            return x.new_empty(shape, dtype=dtype)
        with torch.cuda.stream(self.stream):
            return x.new_empty(shape, dtype=dtype)

    def workspace(self, x: torch.Tensor, given: Optional[torch.Tensor], need: int) -> torch.Tensor:
        if given is not None and _whole(given).numel() * given.element_size() >= need:
            return given
        return self.empty(x, (need,), torch.uint8)

    def __call__(self, fn, *args):
        if torch._C._cuda_getDevice() == self.dev:
            st = fn(*args, self.raw)
        else:
            with torch.cuda.device(self.dev):
                st = fn(*args, self.raw)
        if st:
            _check(st)


def _positions(positions: Optional[torch.Tensor], x: torch.Tensor) -> Optional[bytes]:
    if positions is None:
        return None
    if positions.dtype != torch.int32 or not positions.is_contiguous():
        raise ValueError("positions must be contiguous int32")
    N = x.shape[2]
    shape = tuple(positions.shape)
    if shape not in ((N, 3), (1, N, 3), (x.shape[0], N, 3)):
        raise ValueError(f"positions must be [N, 3], [1, N, 3] or [B, N, 3] (got {list(shape)})")
    return _POSITIONS(positions.data_ptr(), shape[0] if len(shape) == 3 else 1)


def rope(x: torch.Tensor, params: ScopeParams, grid: Optional[ScopeGrid] = None, *,
         positions: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
         inverse: bool = False, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rotary positions of x ([B, H, N, D] f32, bf16 or f16) on the (t, h, w)
    axes of `params` (d_t, d_h, d_w, theta): tokens of a raster `grid`, or
    int32 `positions` [N, 3] or [B, N, 3].  With a `weight` [D], each row goes
    through an RMS norm first.  inverse=True (without a weight) turns back,
    which is the gradient of the plain rotation.  `out` may be x."""
    call = _Launch(stream, x, positions, weight, out)
    tx = _tensor(x, "x")
    pos = _positions(positions, x)
    w = None if weight is None else _vector(weight, x.shape[-1], "weight")
    y = call.like(x, out)
    call(_packed().scope_rope, tx, grid, params, pos, w, eps, int(inverse), _tensor(y, "out"))
    return y


def rope_backward(dy: torch.Tensor, x: torch.Tensor, params: ScopeParams, grid: Optional[ScopeGrid] = None, *,
                  weight: torch.Tensor, positions: Optional[torch.Tensor] = None, eps: float = 1e-6,
                  out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """(dx, dw) of rope(x, ..., weight=weight) for the gradient dy of its
    output; `out` (dx) may be x or dy.  Without a weight the gradient is
    rope(dy, ..., inverse=True)."""
    call = _Launch(stream, dy, x, positions, weight, out, workspace)
    tx = _tensor(x, "x")
    pos = _positions(positions, x)
    w = _vector(weight, x.shape[-1], "weight")
    L = _packed()
    need = L.scope_rope_backward_workspace_bytes(tx)
    if need == 0:
        raise ScopeError(1, L.scope_last_error().decode())
    ws = call.workspace(x, workspace, need)
    dx = call.like(x, out)
    dw = call.empty(weight, weight.shape, weight.dtype)
    call(L.scope_rope_backward, _tensor(dy, "dy"), tx, grid, params, pos, w, eps, _tensor(dx, "out"),
         _vector(dw, x.shape[-1], "dw"), ws.data_ptr(), ws.numel() * ws.element_size())
    return dx, dw


def _keys(k: torch.Tensor, kv_len: Optional[torch.Tensor], kv_mask: Optional[torch.Tensor]) -> Optional[bytes]:
    Bk, M = k.shape[0], k.shape[2]
    if kv_len is not None and (kv_len.dtype != torch.int32 or tuple(kv_len.shape) != (Bk,) or not kv_len.is_contiguous()):
        raise ValueError(f"kv_len must be contiguous int32 [{Bk}]")
    if kv_mask is None:
        return None if kv_len is None else _KEYS(kv_len.data_ptr(), 0, 0)
    if kv_mask.dtype not in (torch.bool, torch.uint8) or tuple(kv_mask.shape) != (Bk, M) or (M > 1 and kv_mask.stride(1) != 1):
        raise ValueError(f"kv_mask must be bool or uint8 [{Bk}, {M}] with contiguous rows")
    # a mask without keys has no memory: as a length of zero, any address serves
    return _KEYS(0 if kv_len is None else kv_len.data_ptr(), kv_mask.data_ptr() if M else 0, kv_mask.stride(0))


@functools.lru_cache(maxsize=4096)
def _cross_bytes(name: str, q_shape, k_shape, dtype: torch.dtype, masked: bool) -> int:
    """Workspace of a call with these shapes."""
    L, dt = _packed(), _DT[dtype]
    fake = 1 << 20  # sizes do not depend on addresses or strides
    q, k = (_TENSOR(fake, dt, *s, 0, 0, 0, 0) for s in (q_shape, k_shape))
    need = getattr(L, name)(q, k, int(masked))
    if need == 0:
        raise ScopeError(1, L.scope_last_error().decode())
    return need


def cross_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, kv_len: Optional[torch.Tensor] = None,
               kv_mask: Optional[torch.Tensor] = None, scale: Optional[float] = None, return_lse: bool = False,
               out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """softmax(scale q k^T) v of q [B, H, N, D] over k, v [Bk, Hk, M, D] (bf16 or
    f16): Bk is B, or 1 for states shared by the batch; Hk divides H.  Keys
    from kv_len (int32 [Bk]) on, or where kv_mask (bool [Bk, M]) is False, are
    not read.  scale: 1/sqrt(D).  return_lse: (o, lse) with lse f32 [B, H, N],
    which cross_attn_backward takes."""
    call = _Launch(stream, q, k, v, kv_len, kv_mask, out, workspace)
    tq, tk, tv = _tensor(q, "q"), _tensor(k, "k"), _tensor(v, "v")
    keys = _keys(k, kv_len, kv_mask)
    ws = call.workspace(q, workspace, _cross_bytes("scope_cross_attn_workspace_bytes", q.shape, k.shape, q.dtype,
                                                   kv_mask is not None))
    o = call.like(q, out)
    lse = call.empty(q, q.shape[:3], torch.float32) if return_lse else None
    call(_packed().scope_cross_attn, tq, tk, tv, keys, _scale(scale), _tensor(o, "out"),
         lse.data_ptr() if return_lse else None, ws.data_ptr(), ws.numel() * ws.element_size())
    return (o, lse) if return_lse else o


def cross_attn_backward(do: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                        lse: torch.Tensor, *, kv_len: Optional[torch.Tensor] = None,
                        kv_mask: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                        dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                        dv: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """(dq, dk, dv) of cross_attn(q, k, v, ...) for the gradient `do` of its
    output, from its results o and lse (return_lse=True) and the same masks and
    scale.  dk and dv have k's shape: summed over the query heads that read a
    key head and, for states shared by the batch, over the batch."""
    call = _Launch(stream, q, do, k, v, o, lse, kv_len, kv_mask, dq, dk, dv, workspace)
    tdo, tq, tk, tv, to = (_tensor(t, n) for t, n in ((do, "do"), (q, "q"), (k, "k"), (v, "v"), (o, "o")))
    if lse.dtype != torch.float32 or lse.shape != q.shape[:3] or not lse.is_contiguous():
        raise ValueError(f"lse must be contiguous float32 {list(q.shape[:3])}")
    keys = _keys(k, kv_len, kv_mask)
    ws = call.workspace(q, workspace, _cross_bytes("scope_cross_attn_backward_workspace_bytes", q.shape, k.shape,
                                                   q.dtype, kv_mask is not None))
    dq, dk, dv = call.like(q, dq), call.like(k, dk), call.like(v, dv)
    call(_packed().scope_cross_attn_backward, tdo, tq, tk, tv, to, lse.data_ptr(), keys, _scale(scale),
         _tensor(dq, "dq"), _tensor(dk, "dk"), _tensor(dv, "dv"), ws.data_ptr(), ws.numel() * ws.element_size())
    return dq, dk, dv


def _scale(scale: Optional[float]) -> float:
    if scale is None:
        return 0.0
    if not 1e-30 <= scale <= 1e30:
        raise ValueError(f"scale must be in [1e-30, 1e30] (got {scale})")
    return scale


def ops_sync_status(stream=None, device=None):
    """Synchronises the stream (by default the device's current one) and raises
    ScopeError if a bounded wait of the package's operators gave up since the
    last report."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    with torch.cuda.device(stream.device):
        _check(_functions().scope_ops_sync_status(stream.cuda_stream))


def ops_selftest_wait_timeout(cycles: int = 2_000_000, *, backward: bool = False, stream=None, device=None):
    """Enqueues the failure-handling self-test of ops_sync_status: a bounded wait
    on a barrier that nothing completes, recorded where the forward (or backward)
    kernels record theirs, so the next ops_sync_status raises ScopeError
    (SCOPE_ETIMEOUT)."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    with torch.cuda.device(stream.device):
        _check(_functions().scope_ops_selftest_wait_timeout(int(backward), int(cycles), stream.cuda_stream))
