"""Thin ctypes binding over libgla_mi355x.so (C ABI in include/gla.h).

Argument marshalling only: torch supplies device memory and the current
stream; every step of the forward runs in the library's HIP kernels. There is
no fallback: if the library is not built, or a call fails, this module raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
import weakref
from typing import Optional, Sequence, Union

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgla_mi355x.so")

L2R, R2L, T2B, B2T = 0, 1, 2, 3
F16, F32 = 0, 1
ACT_NONE, ACT_SILU, ACT_GELU, ACT_LOGSIGMOID = 0, 1, 2, 3
SCHED_AUTO, SCHED_SINGLE_PASS, SCHED_THREE_PHASE, SCHED_RUNS = 0, 1, 2, 3
CTRL_BYTES = 65536  # control words at the start of every workspace
OK, E_ARG, E_UNSUPPORTED, E_WORKSPACE, E_HIP, E_UNPREPARED = 0, -1, -2, -3, -4, -5
ERR_SPIN = 1  # sticky error bit: a single-pass wait ran out of its poll budget
ABI_VERSION = 5

# every symbol declared in include/gla.h
EXPORTS = ["gla_abi_version", "gla_fwd_workspace_bytes", "gla_workspace_layout", "gla_fwd",
           "gla_fwd_state", "gla_fwd_gated", "gla_fwd_schedule", "gla_auto_schedule", "gla_workspace_init",
           "gla_workspace_release", "gla_workspace_is_prepared", "gla_workspace_status",
           "gla_chunk_summaries", "gla_spatial_swiglu", "gla_state_scan", "gla_chunk_outputs", "gla_scan_perm",
           "gla_status_string", "gla_last_error_detail", "gla_fwd_noalloc",
           "gla_bwd_workspace_bytes", "gla_bwd", "gla_step", "gla_step_gated", "gla_add_rmsnorm",
           "gla_add_rmsnorm_q8", "gla_add_rmsnorm_bwd_workspace_bytes", "gla_add_rmsnorm_bwd",
           "gla_gate_bwd_workspace_bytes", "gla_gate_bwd",
           "gla_linear", "gla_linear_bwd_workspace_bytes", "gla_linear_bwd", "gla_gated_ff",
           "gla_gated_ff_bwd_workspace_bytes", "gla_gated_ff_bwd", "gla_gated_add_rmsnorm",
           "gla_gated_add_rmsnorm_bwd_workspace_bytes", "gla_gated_add_rmsnorm_bwd"]

# With check_errors(True), every forward call made through this module waits
# for its stream and raises if the workspace's sticky error word is set
# (skipped while the stream is being captured into a graph). Off by default:
# the check synchronises.
_check_errors = False


def check_errors(on: bool) -> None:
    global _check_errors
    _check_errors = bool(on)

_lib = None
_vp, _i32, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_i32p = ctypes.POINTER(ctypes.c_int32)
_i64, _f32 = ctypes.c_int64, ctypes.c_float


class GLAError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = load()
        msg = lib.gla_status_string(status).decode()
        detail = lib.gla_last_error_detail().decode()
        super().__init__(f"{where}: {msg}" + (f" ({detail})" if detail and status == E_HIP else ""))
        self.status = status


def load():
    """Load the library (once). Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"HIP library not built: {LIB_PATH} is missing; run "
                           "__graft_entry__.build() or recurrent_vision_token_gla_amd/build.py")
    lib = ctypes.CDLL(LIB_PATH)
    lib.gla_abi_version.restype = _i32
    lib.gla_fwd_workspace_bytes.restype = _sz
    lib.gla_fwd_workspace_bytes.argtypes = [_i32] * 7
    lib.gla_workspace_layout.restype = _i32
    lib.gla_workspace_layout.argtypes = [_i32] * 7 + [ctypes.POINTER(_sz)] * 5
    lib.gla_fwd.restype = _i32
    lib.gla_fwd.argtypes = [_vp] * 5 + [_i32] * 6 + [_i32p, _i32, _i32, _vp, _sz, _vp]
    lib.gla_fwd_noalloc.restype = _i32
    lib.gla_fwd_noalloc.argtypes = [_vp] * 5 + [_i32] * 6 + [_i32p, _i32, _i32, _vp]
    lib.gla_fwd_state.restype = _i32
    lib.gla_fwd_state.argtypes = ([_vp] * 5 + [_i32] * 6 + [_i32p, _i32, _i32, _vp, _vp, _vp, _sz,
                                                            _vp])
    lib.gla_fwd_gated.restype = _i32
    lib.gla_fwd_gated.argtypes = ([_vp] * 6 + [ctypes.c_float, _vp] + [_i32] * 6 +
                                  [_i32p, _i32, _i32, _vp, _vp, _vp, _sz, _vp])
    lib.gla_fwd_schedule.restype = _i32
    lib.gla_fwd_schedule.argtypes = ([_vp] * 5 + [_i32] * 6 + [_i32p, _i32, _i32, _vp, _vp, _i32,
                                                               _vp, _sz, _vp])
    lib.gla_auto_schedule.restype = _i32
    lib.gla_auto_schedule.argtypes = [_i32] * 7
    lib.gla_workspace_init.restype = _i32
    lib.gla_workspace_init.argtypes = [_vp, _sz, _vp]
    lib.gla_workspace_release.restype = _i32
    lib.gla_workspace_release.argtypes = [_vp]
    lib.gla_workspace_is_prepared.restype = _i32
    lib.gla_workspace_is_prepared.argtypes = [_vp]
    lib.gla_workspace_status.restype = _i32
    lib.gla_workspace_status.argtypes = [_vp, _sz, ctypes.POINTER(ctypes.c_uint32), _i32, _vp]
    lib.gla_chunk_summaries.restype = _i32
    lib.gla_chunk_summaries.argtypes = [_vp] * 3 + [_i32] * 6 + [_i32p, _i32, _i32, _vp, _sz, _vp]
    lib.gla_state_scan.restype = _i32
    lib.gla_state_scan.argtypes = [_i32] * 7 + [_vp, _vp, _vp, _sz, _vp]
    lib.gla_chunk_outputs.restype = _i32
    lib.gla_chunk_outputs.argtypes = [_vp] * 5 + [_i32] * 6 + [_i32p, _i32, _i32, _vp, _sz, _vp]
    lib.gla_scan_perm.restype = _i32
    lib.gla_scan_perm.argtypes = [_vp, _i32, _i32, _i32, _vp]
    lib.gla_spatial_swiglu.restype = _i32
    lib.gla_spatial_swiglu.argtypes = [_vp] * 5 + [_i32] * 5 + [_vp]
    lib.gla_bwd_workspace_bytes.restype = _sz
    lib.gla_bwd_workspace_bytes.argtypes = [_i32] * 6
    lib.gla_bwd.restype = _i32
    lib.gla_bwd.argtypes = [_vp] * 9 + [_i32] * 6 + [_i32p, _i32, _vp, _vp, _vp, _vp, _sz, _vp]
    lib.gla_step.restype = _i32
    lib.gla_step.argtypes = [_vp] * 5 + [_i32] * 5 + [_vp, _i64, _vp, _vp]
    lib.gla_step_gated.restype = _i32
    lib.gla_step_gated.argtypes = [_vp] * 6 + [_f32, _vp] + [_i32] * 5 + [_vp, _i64, _vp, _vp]
    lib.gla_add_rmsnorm.restype = _i32
    lib.gla_add_rmsnorm.argtypes = [_vp] * 3 + [_f32, _vp, _vp, _i64, _i32, _i32, _vp]
    lib.gla_add_rmsnorm_q8.restype = _i32
    lib.gla_add_rmsnorm_q8.argtypes = [_vp] * 3 + [_f32, _vp, _vp, _vp, _i64, _i32, _i32, _vp]
    lib.gla_add_rmsnorm_bwd_workspace_bytes.restype = _sz
    lib.gla_add_rmsnorm_bwd_workspace_bytes.argtypes = [_i64, _i32]
    lib.gla_add_rmsnorm_bwd.restype = _i32
    lib.gla_add_rmsnorm_bwd.argtypes = ([_vp, _vp, _f32] + [_vp] * 4 + [_i64, _i32, _i32, _vp, _sz,
                                                                        _vp])
    lib.gla_gate_bwd_workspace_bytes.restype = _sz
    lib.gla_gate_bwd_workspace_bytes.argtypes = [_i64, _i32]
    lib.gla_gate_bwd.restype = _i32
    lib.gla_gate_bwd.argtypes = [_vp, _vp, _vp, _f32] + [_vp] * 4 + [_i64, _i32, _i32, _vp, _sz, _vp]
    lib.gla_linear.restype = _i32
    lib.gla_linear.argtypes = [_vp] * 6 + [_i64, _i32, _i32, _i32, _f32, _i32, _vp]
    lib.gla_linear_bwd_workspace_bytes.restype = _sz
    lib.gla_linear_bwd_workspace_bytes.argtypes = [_i64] + [_i32] * 4
    lib.gla_linear_bwd.restype = _i32
    lib.gla_linear_bwd.argtypes = [_vp] * 7 + [_i64, _i32, _i32, _i32, _f32, _i32, _vp, _sz, _vp]
    lib.gla_gated_ff.restype = _i32
    lib.gla_gated_ff.argtypes = [_vp] * 6 + [_i64] + [_i32] * 4 + [_vp]
    lib.gla_gated_ff_bwd_workspace_bytes.restype = _sz
    lib.gla_gated_ff_bwd_workspace_bytes.argtypes = [_i64] + [_i32] * 3
    lib.gla_gated_ff_bwd.restype = _i32
    lib.gla_gated_ff_bwd.argtypes = [_vp] * 9 + [_i64] + [_i32] * 4 + [_vp, _sz, _vp]
    lib.gla_gated_add_rmsnorm.restype = _i32
    lib.gla_gated_add_rmsnorm.argtypes = ([_vp] * 4 + [_i64, _vp, _vp, _f32, _vp, _vp, _i64, _i32,
                                                       _i32, _vp])
    lib.gla_gated_add_rmsnorm_bwd_workspace_bytes.restype = _sz
    lib.gla_gated_add_rmsnorm_bwd_workspace_bytes.argtypes = [_i64, _i64, _i32]
    lib.gla_gated_add_rmsnorm_bwd.restype = _i32
    lib.gla_gated_add_rmsnorm_bwd.argtypes = ([_vp] * 4 + [_i64, _vp, _vp, _f32] + [_vp] * 8 +
                                              [_i64, _i32, _i32, _vp, _sz, _vp])
    lib.gla_status_string.restype = ctypes.c_char_p
    lib.gla_status_string.argtypes = [_i32]
    lib.gla_last_error_detail.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(status: int, where: str):
    if status != OK:
        raise GLAError(status, where)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float16:
        return F16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t.dtype}; use float16 or float32")


def _dirs(direction: Union[int, Sequence[int]], B: int):
    if isinstance(direction, int):
        vals = [direction] * B
    else:
        vals = [int(d) for d in direction]
        if len(vals) != B:
            raise ValueError(f"need one direction per batch element ({B}), got {len(vals)}")
    arr = (ctypes.c_int32 * max(1, B))(*vals)
    return arr


def _stream_ptr(stream: Optional[torch.cuda.Stream]) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def workspace_bytes(B, H, grid_h, grid_w, dk, dv, chunk=64) -> int:
    return int(load().gla_fwd_workspace_bytes(B, H, grid_h, grid_w, dk, dv, chunk))


def workspace_layout(B, H, grid_h, grid_w, dk, dv, chunk=64):
    """(off_U, off_a, off_S, off_scales, total) byte offsets inside the workspace."""
    vals = [_sz() for _ in range(5)]
    _check(load().gla_workspace_layout(B, H, grid_h, grid_w, dk, dv, chunk,
                                       *[ctypes.byref(x) for x in vals]), "gla_workspace_layout")
    return tuple(int(x.value) for x in vals)


def alloc_workspace(B, H, grid_h, grid_w, dk, dv, chunk=64, device=None,
                    prepare: bool = True) -> torch.Tensor:
    """A workspace for this problem. With prepare (the default) it is prepared
    for the single pass by workspace_init."""
    n = workspace_bytes(B, H, grid_h, grid_w, dk, dv, chunk)
    ws = torch.empty(max(n, CTRL_BYTES), dtype=torch.uint8, device=device or "cuda")
    if prepare:
        workspace_init(ws)
    return ws


def auto_schedule(B, H, grid_h, grid_w, dk, dv, chunk=64) -> int:
    """The schedule gla_fwd takes for this shape (SCHED_SINGLE_PASS or
    SCHED_THREE_PHASE)."""
    st = load().gla_auto_schedule(B, H, grid_h, grid_w, dk, dv, chunk)
    if st < 0:
        raise GLAError(st, "gla_auto_schedule")
    return st


def workspace_init(workspace: torch.Tensor, stream=None) -> None:
    """Prepare a workspace for the single pass: zero its control words (and
    the sticky error word) with a kernel and record it as prepared, until
    workspace_release or until its memory is freed."""
    ws, nws = _ws(workspace, workspace.device)
    with _on_device(workspace.device):
        st = load().gla_workspace_init(ws, nws, _stream_ptr(stream))
    _check(st, "gla_workspace_init")
    weakref.finalize(workspace.untyped_storage(), load().gla_workspace_release, ws)


def workspace_release(workspace: torch.Tensor) -> None:
    """Drop a workspace from the library's record of prepared workspaces."""
    _check(load().gla_workspace_release(workspace.data_ptr()), "gla_workspace_release")


def is_prepared(workspace: torch.Tensor) -> bool:
    return bool(load().gla_workspace_is_prepared(workspace.data_ptr()))


def workspace_error(workspace: torch.Tensor, clear: bool = False, stream=None) -> int:
    """The sticky error word (bit 0: a single-pass wait ran out), read after
    the work queued on the stream; optionally cleared. Synchronises."""
    ws, nws = _ws(workspace, workspace.device)
    bits = ctypes.c_uint32(0)
    with _on_device(workspace.device):
        st = load().gla_workspace_status(ws, nws, ctypes.byref(bits), int(clear),
                                         _stream_ptr(stream))
    _check(st, "gla_workspace_status")
    return int(bits.value)


def _after_call(workspace: torch.Tensor, stream) -> None:
    """With check_errors on: raise if the call left the sticky error word set
    (only a prepared workspace runs the single pass and has one)."""
    if not _check_errors or torch.cuda.is_current_stream_capturing() or not is_prepared(workspace):
        return
    bits = workspace_error(workspace, clear=True, stream=stream)
    if bits:
        raise GLAError(E_HIP, f"single-pass wait ran out (error bits {bits:#x})")


def _ws(workspace: torch.Tensor, device):
    """(pointer, size in bytes) of a workspace: a contiguous device tensor on
    the inputs' device, of any dtype."""
    if not workspace.is_cuda or workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _out(out: Optional[torch.Tensor], shape, dtype, device) -> torch.Tensor:
    """The caller's output tensor, checked (the kernels write all of it), or
    a new one."""
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if tuple(out.shape) != tuple(shape) or out.dtype != dtype or out.device != device or \
            not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return out


def _on_device(device):
    """Calls run on the inputs' device (its current stream unless one is given)."""
    return torch.cuda.device(device)


def _shapes(q, k, v, gk, grid_h, grid_w):
    for name, t in (("q", q), ("k", k), ("v", v), ("gk", gk)):
        if not t.is_cuda or t.device != q.device:
            raise ValueError(f"{name} must be a device tensor on q's device")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous [B, T, H, D]")
        if t.dim() != 4:
            raise ValueError(f"{name} must be 4-D [B, T, H, D]")
        if t.dtype != q.dtype:
            raise TypeError("q, k, v, gk must share one dtype")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if T != grid_h * grid_w:
        raise ValueError(f"T={T} but grid is {grid_h}x{grid_w}")
    if k.shape != q.shape or gk.shape != q.shape or v.shape[:3] != q.shape[:3]:
        raise ValueError("shape mismatch between q, k, gk [B,T,H,dk] and v [B,T,H,dv]")
    return B, T, H, dk, dv


def fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, gk: torch.Tensor,
        grid_h: int, grid_w: int, direction: Union[int, Sequence[int]] = L2R,
        chunk: int = 64, out: Optional[torch.Tensor] = None,
        workspace: Optional[torch.Tensor] = None,
        stream: Optional[torch.cuda.Stream] = None, schedule: int = SCHED_AUTO) -> torch.Tensor:
    """o = key-only GLA forward along `direction` (int, or one per batch element)."""
    B, T, H, dk, dv = _shapes(q, k, v, gk, grid_h, grid_w)
    out = _out(out, (B, T, H, dv), q.dtype, q.device)
    if workspace is None:
        workspace = alloc_workspace(B, H, grid_h, grid_w, dk, dv, chunk, q.device)
    if schedule == SCHED_AUTO:
        ws, nws = _ws(workspace, q.device)
        with _on_device(q.device):
            st = load().gla_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), gk.data_ptr(),
                                out.data_ptr(), B, H, grid_h, grid_w, dk, dv, _dirs(direction, B),
                                chunk, _dtype_code(q), ws, nws, _stream_ptr(stream))
        _check(st, "gla_fwd")
        _after_call(workspace, stream)
        return out
    return fwd_state(q, k, v, gk, grid_h, grid_w, direction, chunk, return_state=False, out=out,
                     workspace=workspace, stream=stream, schedule=schedule)


def fwd_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, gk: torch.Tensor,
                grid_h: int, grid_w: int, direction: Union[int, Sequence[int]] = L2R,
                chunk: int = 64, out: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The forward on the library's static scratch (gla_fwd_noalloc): no
    workspace is allocated; calls on one GPU must not overlap in time."""
    B, T, H, dk, dv = _shapes(q, k, v, gk, grid_h, grid_w)
    out = _out(out, (B, T, H, dv), q.dtype, q.device)
    with _on_device(q.device):
        st = load().gla_fwd_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), gk.data_ptr(),
                                    out.data_ptr(), B, H, grid_h, grid_w, dk, dv,
                                    _dirs(direction, B), chunk, _dtype_code(q), _stream_ptr(stream))
    _check(st, "gla_fwd_noalloc")
    return out


def _state_ptr(t: Optional[torch.Tensor], B, H, dk, dv, name, device=None) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda or t.dtype != torch.float32 or not t.is_contiguous() or \
            (device is not None and t.device != device):
        raise ValueError(f"{name} must be a contiguous float32 tensor on the inputs' device")
    if tuple(t.shape) != (B, H, dk, dv):
        raise ValueError(f"{name} must be [B, H, dk, dv] = {(B, H, dk, dv)}, got {tuple(t.shape)}")
    return t.data_ptr()


def fwd_state(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, gk: torch.Tensor,
              grid_h: int, grid_w: int, direction: Union[int, Sequence[int]] = L2R,
              chunk: int = 64, s0: Optional[torch.Tensor] = None,
              s_final: Optional[torch.Tensor] = None, return_state: bool = True,
              out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None, schedule: int = SCHED_AUTO):
    """Forward from the carried state s0 ([B, H, dk, dv] float32, None for
    zero); returns (o, S_T) with S_T written into s_final (allocated if None)
    when return_state, else o. schedule picks the kernel schedule."""
    B, T, H, dk, dv = _shapes(q, k, v, gk, grid_h, grid_w)
    out = _out(out, (B, T, H, dv), q.dtype, q.device)
    if return_state and s_final is None:
        s_final = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(B, H, grid_h, grid_w, dk, dv, chunk, q.device)
    ws, nws = _ws(workspace, q.device)
    p0 = _state_ptr(s0, B, H, dk, dv, "s0", q.device)
    pf = _state_ptr(s_final, B, H, dk, dv, "s_final", q.device)
    with _on_device(q.device):
        st = load().gla_fwd_schedule(q.data_ptr(), k.data_ptr(), v.data_ptr(), gk.data_ptr(),
                                     out.data_ptr(), B, H, grid_h, grid_w, dk, dv,
                                     _dirs(direction, B), chunk, _dtype_code(q), p0, pf, schedule,
                                     ws, nws, _stream_ptr(stream))
    _check(st, "gla_fwd_schedule")
    _after_call(workspace, stream)
    return (out, s_final) if return_state else out


def fwd_gated(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, gk: torch.Tensor,
              gate: torch.Tensor, norm_weight: torch.Tensor, eps: float, grid_h: int,
              grid_w: int, direction: Union[int, Sequence[int]] = L2R, chunk: int = 64,
              s0: Optional[torch.Tensor] = None, s_final: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """y = RMSNorm(o) * norm_weight * silu(gate) with o the forward (from s0,
    None for zero; S_T into s_final if given); gate [B, T, H, dv] in q's
    dtype, norm_weight [dv] float32."""
    B, T, H, dk, dv = _shapes(q, k, v, gk, grid_h, grid_w)
    if gate.shape != v.shape or gate.dtype != q.dtype or not gate.is_contiguous() or \
            gate.device != q.device:
        raise ValueError("gate must be a contiguous tensor shaped like v, in q's dtype and on its device")
    if norm_weight.dtype != torch.float32 or tuple(norm_weight.shape) != (dv,) or \
            norm_weight.device != q.device or not norm_weight.is_contiguous():
        raise ValueError("norm_weight must be a contiguous float32 [dv] tensor on q's device")
    out = _out(out, (B, T, H, dv), q.dtype, q.device)
    if workspace is None:
        workspace = alloc_workspace(B, H, grid_h, grid_w, dk, dv, chunk, q.device)
    ws, nws = _ws(workspace, q.device)
    p0 = _state_ptr(s0, B, H, dk, dv, "s0", q.device)
    pf = _state_ptr(s_final, B, H, dk, dv, "s_final", q.device)
    with _on_device(q.device):
        st = load().gla_fwd_gated(q.data_ptr(), k.data_ptr(), v.data_ptr(), gk.data_ptr(),
                                  gate.data_ptr(), norm_weight.data_ptr(), float(eps),
                                  out.data_ptr(), B, H, grid_h, grid_w, dk, dv,
                                  _dirs(direction, B), chunk, _dtype_code(q), p0, pf, ws, nws,
                                  _stream_ptr(stream))
    _check(st, "gla_fwd_gated")
    _after_call(workspace, stream)
    return out


def chunk_summaries(k, v, gk, grid_h, grid_w, direction=L2R, chunk=64, workspace=None,
                    stream=None) -> torch.Tensor:
    """Phase 1 only; returns the workspace holding U and a."""
    B, T, H, dk, dv = _shapes(k, k, v, gk, grid_h, grid_w)
    if workspace is None:
        workspace = alloc_workspace(B, H, grid_h, grid_w, dk, dv, chunk, k.device)
    ws, nws = _ws(workspace, k.device)
    with _on_device(k.device):
        st = load().gla_chunk_summaries(k.data_ptr(), v.data_ptr(), gk.data_ptr(), B, H, grid_h,
                                        grid_w, dk, dv, _dirs(direction, B), chunk, _dtype_code(k),
                                        ws, nws, _stream_ptr(stream))
    _check(st, "gla_chunk_summaries")
    return workspace


def state_scan(B, H, grid_h, grid_w, dk, dv, chunk, workspace, s0=None, s_final=None,
               stream=None) -> torch.Tensor:
    ws, nws = _ws(workspace, workspace.device)
    p0 = _state_ptr(s0, B, H, dk, dv, "s0", workspace.device)
    pf = _state_ptr(s_final, B, H, dk, dv, "s_final", workspace.device)
    with _on_device(workspace.device):
        st = load().gla_state_scan(B, H, grid_h, grid_w, dk, dv, chunk, p0, pf, ws, nws,
                                   _stream_ptr(stream))
    _check(st, "gla_state_scan")
    return workspace


def chunk_outputs(q, k, v, gk, grid_h, grid_w, direction=L2R, chunk=64, workspace=None,
                  out=None, stream=None) -> torch.Tensor:
    B, T, H, dk, dv = _shapes(q, k, v, gk, grid_h, grid_w)
    out = _out(out, (B, T, H, dv), q.dtype, q.device)
    if workspace is None:
        raise ValueError("chunk_outputs needs the workspace that holds the entering states")
    ws, nws = _ws(workspace, q.device)
    with _on_device(q.device):
        st = load().gla_chunk_outputs(q.data_ptr(), k.data_ptr(), v.data_ptr(), gk.data_ptr(),
                                      out.data_ptr(), B, H, grid_h, grid_w, dk, dv,
                                      _dirs(direction, B), chunk, _dtype_code(q), ws, nws,
                                      _stream_ptr(stream))
    _check(st, "gla_chunk_outputs")
    return out


def workspace_views(workspace: torch.Tensor, B, H, grid_h, grid_w, dk, dv, chunk=64):
    """Views of the stored arrays of the three phases: U [B,H,N,dk,dv] f16,
    a [B,H,N,dk] f32, S [B,H,N,dk,dv] f16, m [B,H,N,dk] f32 (the largest
    |U| of each row; a and m are the two halves of the stored (a, m) pairs)
    and the row scales sigS [B,H,N,dk] f32. The value of U row d is
    U[..., d, :] * row_scale(m[..., d]), that of S row d is
    S[..., d, :] * sigS[..., d]."""
    off_U, off_a, off_S, off_ss, _ = workspace_layout(B, H, grid_h, grid_w, dk, dv, chunk)
    N = -(-(grid_h * grid_w) // chunk)
    n_us = B * H * N * dk * dv
    n_a = B * H * N * dk
    U = workspace[off_U:off_U + 2 * n_us].view(torch.float16).view(B, H, N, dk, dv)
    pairs = workspace[off_a:off_a + 8 * n_a].view(torch.float32).view(B, H, N, dk, 2)
    S = workspace[off_S:off_S + 2 * n_us].view(torch.float16).view(B, H, N, dk, dv)
    sig_s = workspace[off_ss:off_ss + 4 * n_a].view(torch.float32).view(B, H, N, dk)
    return U, pairs[..., 0], S, pairs[..., 1], sig_s


def workspace_states(workspace: torch.Tensor, B, H, grid_h, grid_w, dk, dv, chunk=64):
    """(U, a, S) as float64 host arrays with the row scales applied."""
    U, a, S, m, ss = (x.double().cpu().numpy()
                      for x in workspace_views(workspace, B, H, grid_h, grid_w, dk, dv, chunk))
    return U * row_scale(m)[..., None], a, S * ss[..., None]


def row_scale(m):
    """The power-of-two scale a state row with largest magnitude m is stored
    divided by (the library's rule): 1 while m < 2^14, else the power of two
    that brings m into [2^13, 2^14)."""
    import numpy as np
    m = np.asarray(m, np.float32)
    e = ((m.view(np.uint32) >> 23) & 0xFF).astype(np.int64) - 140
    out = np.ldexp(np.float32(1), np.maximum(e, 0)).astype(np.float64)
    return np.where((e <= 0) | (e == 115), 1.0, out)


def scan_perm(grid_h: int, grid_w: int, direction: int, device="cuda", stream=None) -> torch.Tensor:
    """Device-computed scan order (raster index per scan position), int32."""
    perm = torch.empty(max(1, grid_h * grid_w), dtype=torch.int32, device=device)
    with _on_device(perm.device):
        st = load().gla_scan_perm(perm.data_ptr(), grid_h, grid_w, direction, _stream_ptr(stream))
    _check(st, "gla_scan_perm")
    return perm[:grid_h * grid_w]


def spatial_swiglu(a: torch.Tensor, u: torch.Tensor, weight: torch.Tensor,
                   bias: Optional[torch.Tensor], grid_h: int, grid_w: int,
                   out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """h = silu(a) * (3x3 depthwise conv of u on the grid + bias); a, u [B, T, F]
    (float16 or float32, contiguous), weight [F, 3, 3] and bias [F] float32."""
    for name, t in (("a", a), ("u", u)):
        if not t.is_cuda or t.device != u.device or not t.is_contiguous() or t.dim() != 3:
            raise ValueError(f"{name} must be a contiguous [B, T, F] device tensor on u's device")
    if a.shape != u.shape or a.dtype != u.dtype:
        raise ValueError("a and u must share shape and dtype")
    B, T, Fc = u.shape
    if T != grid_h * grid_w:
        raise ValueError(f"T={T} but grid is {grid_h}x{grid_w}")
    if weight.dtype != torch.float32 or tuple(weight.shape) != (Fc, 3, 3) or \
            not weight.is_contiguous() or weight.device != u.device:
        raise ValueError("weight must be a contiguous float32 [F, 3, 3] tensor on u's device")
    if bias is not None and (bias.dtype != torch.float32 or tuple(bias.shape) != (Fc,)
                             or bias.device != u.device or not bias.is_contiguous()):
        raise ValueError("bias must be a contiguous float32 [F] tensor on u's device")
    out = _out(out, tuple(u.shape), u.dtype, u.device)
    with _on_device(u.device):
        st = load().gla_spatial_swiglu(a.data_ptr(), u.data_ptr(), weight.data_ptr(),
                                       None if bias is None else bias.data_ptr(), out.data_ptr(),
                                       B, grid_h, grid_w, Fc, _dtype_code(u), _stream_ptr(stream))
    _check(st, "gla_spatial_swiglu")
    return out


# ---- gradients, single tokens and the norm before a mixer ---------------------

# the current stream of a device as a pointer, without building a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
# the current device, where a device tensor is at hand (so that the runtime is up)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


class _Here:
    """The current device and stream: nothing to switch, as in the small calls,
    which are bound by what the host does."""
    __slots__ = ("index",)

    def __init__(self, index: int):
        self.index = index

    def __enter__(self) -> int:
        return _raw_stream(self.index)

    def __exit__(self, *exc) -> None:
        pass


class _There:
    """Another device or a given stream. What the call allocates belongs to
    that stream, and the caller's tensors are not reused before its work is
    done (the caller orders the streams themselves)."""
    __slots__ = ("device", "stream", "inputs", "contexts")

    def __init__(self, device, stream, inputs):
        self.device, self.stream, self.inputs = device, stream, inputs

    def __enter__(self) -> int:
        with contextlib.ExitStack() as contexts:  # left again if anything below fails
            if self.stream is not None and self.stream.device != self.device:
                raise ValueError(f"stream is on {self.stream.device}, the tensors on {self.device}")
            contexts.enter_context(torch.cuda.device(self.device))
            if self.stream is None:
                ptr = _raw_stream(self.device.index)
            else:
                contexts.enter_context(torch.cuda.stream(self.stream))
                if not torch.cuda.is_current_stream_capturing():
                    for t in self.inputs:  # those elsewhere are refused by the call
                        if t is not None and t.device == self.device:
                            t.record_stream(self.stream)
                ptr = int(self.stream.cuda_stream)
            self.contexts = contexts.pop_all()
        return ptr

    def __exit__(self, *exc) -> None:
        self.contexts.__exit__(*exc)


def _launching(device, stream, *inputs):
    """Device and stream of a call, as a context with the raw stream pointer."""
    if stream is None and _current_device() == device.index:
        return _Here(device.index)
    return _There(device, stream, inputs)


def _like(t: torch.Tensor, shape, dtype, device, name: str) -> torch.Tensor:
    if t is None or t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t


def _alike(shape, dtype, device, names: str, *tensors) -> None:
    """_like for tensors of one shape."""
    for t in tensors:
        if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous():
            for name, u in zip(names.split(), tensors):
                _like(u, shape, dtype, device, name)


def _on_gpu(t: torch.Tensor, name: str) -> torch.device:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.device


def _out_like(out: Optional[torch.Tensor], t: torch.Tensor) -> torch.Tensor:
    """The caller's output tensor, checked against t, or a new one (t is
    contiguous, so is empty_like's)."""
    return torch.empty_like(t) if out is None else _out(out, t.shape, t.dtype, t.device)


@functools.lru_cache(maxsize=256)
def _norm_workspace_bytes(rows: int, F: int) -> int:
    return int(load().gla_add_rmsnorm_bwd_workspace_bytes(rows, F))


@functools.lru_cache(maxsize=256)
def _gate_workspace_bytes(rows: int, dv: int) -> int:
    return int(load().gla_gate_bwd_workspace_bytes(rows, dv))


def _scratch(workspace: Optional[torch.Tensor], need: int, device) -> torch.Tensor:
    """The caller's workspace or a new one (inside _launching). The gradients
    refuse memory with the control words of a workspace prepared for the
    forward; a new one is nobody's, even where a freed one was never released."""
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
        load().gla_workspace_release(workspace.data_ptr())
    return workspace


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=256)
def bwd_workspace_bytes(B, H, grid_h, grid_w, dk, dv) -> int:
    return int(load().gla_bwd_workspace_bytes(B, H, grid_h, grid_w, dk, dv))


def bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, gk: torch.Tensor, go: torch.Tensor,
        grid_h: int, grid_w: int, direction: Union[int, Sequence[int]] = L2R,
        s0: Optional[torch.Tensor] = None, gs_final: Optional[torch.Tensor] = None,
        return_gs0: bool = False, gs0: Optional[torch.Tensor] = None,
        out: Optional[Sequence[torch.Tensor]] = None, workspace: Optional[torch.Tensor] = None,
        stream: Optional[torch.cuda.Stream] = None):
    """Gradients (gq, gkey, gv, ggk) of the forward's q, k, v, gk from go =
    dL/do, along the same direction and from the same s0 (None for zero);
    gs_final [B, H, dk, dv] float32 is the gradient of the final state (None
    for zero). With return_gs0 the gradient of s0 follows (in gs0 if given,
    which may be gs_final). out: four tensors to write the gradients to."""
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, gk must be [B, T, H, dk] and v, go [B, T, H, dv]")
    B, T, H, dk = keys = q.shape
    dv, dev, dtype = v.shape[-1], _on_gpu(q, "q"), q.dtype
    values = (B, T, H, dv)
    if T != grid_h * grid_w:
        raise ValueError(f"T={T} but grid is {grid_h}x{grid_w}")
    _alike(keys, dtype, dev, "q k gk", q, k, gk)
    _alike(values, dtype, dev, "v go", v, go)
    p0 = _state_ptr(s0, B, H, dk, dv, "s0", dev)
    pf = _state_ptr(gs_final, B, H, dk, dv, "gs_final", dev)
    if gs0 is not None and not return_gs0:
        raise ValueError("gs0 is written with return_gs0 only")
    if out is not None and len(out) != 4:
        raise ValueError("out must be four tensors (gq, gkey, gv, ggk)")
    with _launching(dev, stream, q, k, v, gk, go, s0, gs_final, gs0, workspace, *(out or ())) as st_ptr:
        if out is None:
            outs = (torch.empty_like(q), torch.empty_like(q), torch.empty_like(v), torch.empty_like(q))
        else:
            outs = tuple(_out_like(o, t) for o, t in zip(out, (q, k, v, gk)))
        if return_gs0 and gs0 is None:
            gs0 = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
        pg = _state_ptr(gs0, B, H, dk, dv, "gs0", dev)
        if return_gs0 and T == 0 and gs0 is not gs_final:  # no token: the state passes through
            gs0.zero_() if gs_final is None else gs0.copy_(gs_final)
        workspace = _scratch(workspace, bwd_workspace_bytes(B, H, grid_h, grid_w, dk, dv), dev)
        ws, nws = _ws(workspace, dev)
        st = load().gla_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), gk.data_ptr(), go.data_ptr(),
                            outs[0].data_ptr(), outs[1].data_ptr(), outs[2].data_ptr(),
                            outs[3].data_ptr(), B, H, grid_h, grid_w, dk, dv, _dirs(direction, B),
                            _dtype_code(q), p0, pf, pg, ws, nws, st_ptr)
    _check(st, "gla_bwd")
    return outs + (gs0,) if return_gs0 else outs


def _step(q, k, v, gk, state, slots, out, stream, gated=False, gate=None, norm_weight=None, eps=0.0):
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k, gk must be [B, H, dk] and v [B, H, dv]")
    B, H, dk = keys = q.shape
    dv, dev, dtype = v.shape[-1], _on_gpu(q, "q"), q.dtype
    _alike(keys, dtype, dev, "q k gk", q, k, gk)
    _alike((B, H, dv), dtype, dev, "v", v)
    if state.dim() != 4:
        raise ValueError("state must be [n_slots, H, dk, dv]")
    n_slots = state.shape[0]
    _alike((n_slots, H, dk, dv), torch.float32, dev, "state", state)
    if slots is not None:
        _alike((B,), torch.int32, dev, "slots", slots)
    elif n_slots < B:
        raise ValueError(f"{B} rows without slots need as many states, got {n_slots}")
    if gated:
        _like(gate, (B, H, dv), dtype, dev, "gate")
        _like(norm_weight, (dv,), torch.float32, dev, "norm_weight")
    with _launching(dev, stream, q, k, v, gk, state, slots, out, gate, norm_weight) as st_ptr:
        out = _out_like(out, v)
        tail = (out.data_ptr(), B, H, dk, dv, _dtype_code(q), state.data_ptr(), n_slots,
                _ptr(slots), st_ptr)
        if not gated:
            st = load().gla_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), gk.data_ptr(), *tail)
        else:
            st = load().gla_step_gated(q.data_ptr(), k.data_ptr(), v.data_ptr(), gk.data_ptr(),
                                       gate.data_ptr(), norm_weight.data_ptr(), float(eps), *tail)
    _check(st, "gla_step_gated" if gated else "gla_step")
    return out


def step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, gk: torch.Tensor, state: torch.Tensor,
         slots: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
         stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One new token per row: state[slot] <- diag(exp(gk)) state[slot] + k^T v
    in place, o = q state[slot]; q, k, gk [B, H, dk], v [B, H, dv], state
    [n_slots, H, dk, dv] float32, slots [B] int32 (None: row b uses slot b).
    A slot outside the pool marks a padding row: its row of `out` is left as
    it was (unset in a new one). Rows of one slot are applied in row order."""
    return _step(q, k, v, gk, state, slots, out, stream)


def step_gated(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, gk: torch.Tensor,
               gate: torch.Tensor, norm_weight: torch.Tensor, eps: float, state: torch.Tensor,
               slots: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """step with the output gate, y = RMSNorm(o) * norm_weight * silu(gate);
    gate [B, H, dv] in q's dtype, norm_weight [dv] float32."""
    return _step(q, k, v, gk, state, slots, out, stream, True, gate, norm_weight, eps)


def _norm_args(x, residual, weight):
    dev = _on_gpu(x, "x")
    if not x.is_contiguous() or x.dim() < 1:
        raise ValueError("x must be a contiguous device tensor [..., F]")
    if residual is not None:
        _like(residual, x.shape, x.dtype, dev, "residual")
    F = x.shape[-1]
    _like(weight, (F,), torch.float32, dev, "weight")
    return (x.numel() // F if F else 0), F


def add_rmsnorm(x: torch.Tensor, residual: Optional[torch.Tensor], weight: torch.Tensor, eps: float,
                out: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None):
    """(y, s): s = x + residual (x if None) rounded to x's dtype, y =
    RMSNorm(s) * weight; x [..., F] float16 or float32, weight [F] float32, F
    a multiple of 8. out and sum_out may be x or residual (not the same one)."""
    rows, F = _norm_args(x, residual, weight)
    with _launching(x.device, stream, x, residual, weight, out, sum_out) as st_ptr:
        y = _out_like(out, x)
        s = _out_like(sum_out, x)
        st = load().gla_add_rmsnorm(x.data_ptr(), _ptr(residual), weight.data_ptr(), float(eps),
                                    s.data_ptr(), y.data_ptr(), rows, F, _dtype_code(x), st_ptr)
    _check(st, "gla_add_rmsnorm")
    return y, s


def add_rmsnorm_q8(x: torch.Tensor, residual: Optional[torch.Tensor], weight: torch.Tensor,
                   eps: float, out: Optional[torch.Tensor] = None,
                   scales: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None):
    """(y8, scales, s): add_rmsnorm with y in float8_e4m3fn and a float32
    scale per row (shape x.shape[:-1]): y8 * scale stands for y, the row's
    largest |y| for 448."""
    rows, F = _norm_args(x, residual, weight)
    with _launching(x.device, stream, x, residual, weight, out, scales, sum_out) as st_ptr:
        y8 = _out(out, x.shape, torch.float8_e4m3fn, x.device)
        sc = _out(scales, x.shape[:-1], torch.float32, x.device)
        s = _out_like(sum_out, x)
        st = load().gla_add_rmsnorm_q8(x.data_ptr(), _ptr(residual), weight.data_ptr(), float(eps),
                                       s.data_ptr(), y8.data_ptr(), sc.data_ptr(), rows, F,
                                       _dtype_code(x), st_ptr)
    _check(st, "gla_add_rmsnorm_q8")
    return y8, sc, s


def add_rmsnorm_bwd(s: torch.Tensor, weight: torch.Tensor, eps: float, gy: torch.Tensor,
                    gsum: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    gweight: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None):
    """(gx, gweight) of add_rmsnorm from its s and gy = dL/dy; gsum is the
    gradient that reaches s itself (None for none). gx is the gradient of x
    and of residual; out may be s, gy or gsum. gweight [F] float32."""
    rows, F = _norm_args(s, gsum, weight)
    _like(gy, s.shape, s.dtype, s.device, "gy")
    with _launching(s.device, stream, s, weight, gy, gsum, out, gweight, workspace) as st_ptr:
        gx = _out_like(out, s)
        gw = _out_like(gweight, weight)
        if rows == 0 and F > 0:  # no rows: a sum of nothing
            return gx, gw.zero_()
        workspace = _scratch(workspace, _norm_workspace_bytes(rows, F), s.device)
        ws, nws = _ws(workspace, s.device)
        st = load().gla_add_rmsnorm_bwd(s.data_ptr(), weight.data_ptr(), float(eps), gy.data_ptr(),
                                        _ptr(gsum), gx.data_ptr(), gw.data_ptr(), rows, F,
                                        _dtype_code(s), ws, nws, st_ptr)
    _check(st, "gla_add_rmsnorm_bwd")
    return gx, gw


def gate_bwd(o: torch.Tensor, gate: torch.Tensor, norm_weight: torch.Tensor, eps: float,
             gy: torch.Tensor, out: Optional[Sequence[torch.Tensor]] = None,
             gnorm_weight: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None):
    """(go, ggate, gnorm_weight) of the output gate y = RMSNorm(o) *
    norm_weight * silu(gate) (fwd_gated's, with o what fwd gives); o, gate, gy
    [..., dv]; norm_weight and its gradient [dv] float32. out: two tensors to
    write go and ggate to."""
    rows, dv = _norm_args(o, None, norm_weight)
    _like(gate, o.shape, o.dtype, o.device, "gate")
    _like(gy, o.shape, o.dtype, o.device, "gy")
    if out is not None and len(out) != 2:
        raise ValueError("out must be two tensors (go, ggate)")
    with _launching(o.device, stream, o, gate, norm_weight, gy, gnorm_weight, workspace,
                    *(out or ())) as st_ptr:
        go = _out_like(out[0] if out else None, o)
        gz = _out_like(out[1] if out else None, o)
        gw = _out_like(gnorm_weight, norm_weight)
        if rows == 0 and dv > 0:
            return go, gz, gw.zero_()
        workspace = _scratch(workspace, _gate_workspace_bytes(rows, dv), o.device)
        ws, nws = _ws(workspace, o.device)
        st = load().gla_gate_bwd(o.data_ptr(), gate.data_ptr(), norm_weight.data_ptr(), float(eps),
                                 gy.data_ptr(), go.data_ptr(), gz.data_ptr(), gw.data_ptr(), rows, dv,
                                 _dtype_code(o), ws, nws, st_ptr)
    _check(st, "gla_gate_bwd")
    return go, gz, gw


# ---- the products and norms between a block's mixers


def _rows_of(x: torch.Tensor, name: str):
    """(device, rows, width) of a contiguous device tensor [..., width]."""
    if not x.is_cuda or not x.is_contiguous() or x.dim() < 1:
        raise ValueError(f"{name} must be a contiguous device tensor [..., K]")
    K = x.shape[-1]
    return x.device, (x.numel() // K if K else math.prod(x.shape[:-1])), K


def _weight_of(weight: torch.Tensor, x: torch.Tensor, dev, K: int, name: str) -> int:
    """Rows of a weight [N, K] in x's dtype, on x's device."""
    shape = weight.shape
    if len(shape) != 2 or shape[1] != K or weight.dtype is not x.dtype or weight.device != dev or \
            not weight.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {x.dtype} tensor [N, {K}] on {dev}")
    return shape[0]


def _new(out: Optional[torch.Tensor], shape, like: torch.Tensor) -> torch.Tensor:
    """The caller's output tensor, checked, or a new one of like's dtype and device."""
    return like.new_empty(shape) if out is None else _out(out, shape, like.dtype, like.device)


@functools.lru_cache(maxsize=256)
def _linear_workspace_bytes(rows: int, K: int, N: int, act: int, dtype: int) -> int:
    return int(load().gla_linear_bwd_workspace_bytes(rows, K, N, act, dtype))


@functools.lru_cache(maxsize=256)
def _gated_ff_workspace_bytes(rows: int, K: int, F: int, dtype: int) -> int:
    return int(load().gla_gated_ff_bwd_workspace_bytes(rows, K, F, dtype))


@functools.lru_cache(maxsize=256)
def _gated_norm_workspace_bytes(rows: int, groups: int, F: int) -> int:
    return int(load().gla_gated_add_rmsnorm_bwd_workspace_bytes(rows, groups, F))


def linear(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
           act: int = ACT_NONE, alpha: float = 1.0, residual: Optional[torch.Tensor] = None,
           return_pre: bool = False, out: Optional[torch.Tensor] = None,
           pre: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """y = alpha * act(x weight^T + bias) + residual, or (y, pre) with
    return_pre, pre = x weight^T + bias for linear_bwd (written to `pre` if
    given). x [..., K], weight [N, K], residual, y and pre [..., N] in one
    dtype (float16 or float32), bias [N] float32; K and N multiples of 8. out
    may be residual."""
    dev, rows, K = _rows_of(x, "x")
    N = _weight_of(weight, x, dev, K, "weight")
    shape = (*x.shape[:-1], N)
    if bias is not None:
        _like(bias, (N,), torch.float32, dev, "bias")
    if residual is not None:
        _like(residual, shape, x.dtype, dev, "residual")
    if pre is not None and not return_pre:
        raise ValueError("pre is written with return_pre only")
    with _launching(dev, stream, x, weight, bias, residual, out, pre) as st_ptr:
        y = _new(out, shape, x)
        p = _new(pre, shape, x) if return_pre else None
        st = load().gla_linear(x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(residual), _ptr(p),
                               y.data_ptr(), rows, K, N, act, float(alpha), _dtype_code(x), st_ptr)
    _check(st, "gla_linear")
    return (y, p) if return_pre else y


def linear_bwd(x: torch.Tensor, weight: torch.Tensor, gy: torch.Tensor, act: int = ACT_NONE,
               alpha: float = 1.0, pre: Optional[torch.Tensor] = None, need_x: bool = True,
               need_weight: bool = True, need_bias: bool = True, gx: Optional[torch.Tensor] = None,
               gweight: Optional[torch.Tensor] = None, gbias: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """(gx, gweight, gbias) of linear from gy = dL/dy and the forward's pre
    (not needed for ACT_NONE); the residual's gradient is gy. None for those
    not needed. gx and gweight have x's dtype, gbias is float32."""
    dev, rows, K = _rows_of(x, "x")
    N = _weight_of(weight, x, dev, K, "weight")
    shape = (*x.shape[:-1], N)
    _like(gy, shape, x.dtype, dev, "gy")
    if act != ACT_NONE:
        _like(pre, shape, x.dtype, dev, "pre")
    with _launching(dev, stream, x, weight, gy, pre, gx, gweight, gbias, workspace) as st_ptr:
        gx = _out_like(gx, x) if need_x else None
        gw = _out_like(gweight, weight) if need_weight else None
        gb = _out(gbias, (N,), torch.float32, dev) if need_bias else None
        code = _dtype_code(x)
        if rows == 0 or N == 0:  # sums of nothing
            for g in (gx, gw, gb):
                if g is not None:
                    g.zero_()
            return gx, gw, gb
        workspace = _scratch(workspace, _linear_workspace_bytes(rows, K, N, act, code), dev)
        ws, nws = _ws(workspace, dev)
        st = load().gla_linear_bwd(x.data_ptr(), weight.data_ptr(),
                                   pre.data_ptr() if act != ACT_NONE else None, gy.data_ptr(), _ptr(gx),
                                   _ptr(gw), _ptr(gb), rows, K, N, act, float(alpha), code, ws, nws,
                                   st_ptr)
    _check(st, "gla_linear_bwd")
    return gx, gw, gb


def gated_ff(x: torch.Tensor, gate_weight: torch.Tensor, up_weight: torch.Tensor, act: int = ACT_SILU,
             return_parts: bool = False, out: Optional[torch.Tensor] = None,
             parts: Optional[Sequence[torch.Tensor]] = None,
             stream: Optional[torch.cuda.Stream] = None):
    """h = act(x gate_weight^T) * (x up_weight^T), or (h, a, u) with
    return_parts, the two products for gated_ff_bwd (written to `parts` if
    given). x [..., K], weights [F, K], h, a, u [..., F] in one dtype."""
    dev, rows, K = _rows_of(x, "x")
    F = _weight_of(gate_weight, x, dev, K, "gate_weight")
    if _weight_of(up_weight, x, dev, K, "up_weight") != F:
        raise ValueError(f"up_weight must be [{F}, {K}] as gate_weight is")
    if parts is not None and (not return_parts or len(parts) != 2):
        raise ValueError("parts must be two tensors (a, u), written with return_parts only")
    shape = (*x.shape[:-1], F)
    with _launching(dev, stream, x, gate_weight, up_weight, out, *(parts or ())) as st_ptr:
        h = _new(out, shape, x)
        a = u = None
        if return_parts:
            a, u = (_new(t, shape, x) for t in parts or (None, None))
        st = load().gla_gated_ff(x.data_ptr(), gate_weight.data_ptr(), up_weight.data_ptr(), _ptr(a),
                                 _ptr(u), h.data_ptr(), rows, K, F, act, _dtype_code(x), st_ptr)
    _check(st, "gla_gated_ff")
    return (h, a, u) if return_parts else h


def gated_ff_bwd(x: torch.Tensor, gate_weight: torch.Tensor, up_weight: torch.Tensor, a: torch.Tensor,
                 u: torch.Tensor, gh: torch.Tensor, act: int = ACT_SILU, need_x: bool = True,
                 need_weights: bool = True, gx: Optional[torch.Tensor] = None,
                 gweights: Optional[Sequence[torch.Tensor]] = None,
                 workspace: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None):
    """(gx, ggate_weight, gup_weight) of gated_ff from gh = dL/dh and the
    forward's a, u; None for those not needed. All in x's dtype."""
    dev, rows, K = _rows_of(x, "x")
    F = _weight_of(gate_weight, x, dev, K, "gate_weight")
    if _weight_of(up_weight, x, dev, K, "up_weight") != F:
        raise ValueError(f"up_weight must be [{F}, {K}] as gate_weight is")
    _alike((*x.shape[:-1], F), x.dtype, dev, "a u gh", a, u, gh)
    if gweights is not None and len(gweights) != 2:
        raise ValueError("gweights must be two tensors (ggate_weight, gup_weight)")
    with _launching(dev, stream, x, gate_weight, up_weight, a, u, gh, gx, workspace,
                    *(gweights or ())) as st_ptr:
        gx = _out_like(gx, x) if need_x else None
        gg = gu = None
        if need_weights:
            gg = _out_like(gweights[0] if gweights else None, gate_weight)
            gu = _out_like(gweights[1] if gweights else None, up_weight)
        code = _dtype_code(x)
        if rows == 0 or F == 0:  # sums of nothing
            for g in (gx, gg, gu):
                if g is not None:
                    g.zero_()
            return gx, gg, gu
        workspace = _scratch(workspace, _gated_ff_workspace_bytes(rows, K, F, code), dev)
        ws, nws = _ws(workspace, dev)
        st = load().gla_gated_ff_bwd(x.data_ptr(), gate_weight.data_ptr(), up_weight.data_ptr(),
                                     a.data_ptr(), u.data_ptr(), gh.data_ptr(), _ptr(gx), _ptr(gg),
                                     _ptr(gu), rows, K, F, act, code, ws, nws, st_ptr)
    _check(st, "gla_gated_ff_bwd")
    return gx, gg, gu


def _gated_norm_args(x, weight, post_weight, gate, scale):
    """(device, rows, F, groups) of the norms around a block."""
    dev, rows, F = _rows_of(x, "x")
    _like(weight, (F,), torch.float32, dev, "weight")
    if post_weight is not None:
        _like(post_weight, (F,), torch.float32, dev, "post_weight")
    if scale is not None:
        _like(scale, (F,), torch.float32, dev, "scale")
    groups = 1
    if gate is not None:
        _like(gate, gate.shape[:-1] + (F,), x.dtype, dev, "gate")
        groups = gate.numel() // F if F else 1
        if groups == 0 and rows == 0:  # an empty batch
            groups = 1
        if groups < 1 or rows % groups:
            raise ValueError(f"gate must have one row for each of equal groups of the {rows} rows, got {groups}")
    return dev, rows, F, groups


def gated_add_rmsnorm(x: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor, eps: float,
                      post_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                      scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                      sum_out: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None):
    """(y, s): s = residual + scale * gate * p rounded to x's dtype, with p =
    RMSNorm(x) * post_weight (x without it), and y = RMSNorm(s) * weight. x,
    residual [..., F]; gate [..., F] in x's dtype, one row for each of equal
    runs of x's rows; weight, post_weight, scale [F] float32; scale and gate
    count as 1 where None. out and sum_out may be x or residual."""
    dev, rows, F, groups = _gated_norm_args(x, weight, post_weight, gate, scale)
    _like(residual, x.shape, x.dtype, dev, "residual")
    with _launching(dev, stream, x, residual, weight, post_weight, gate, scale, out, sum_out) as st_ptr:
        y = _out_like(out, x)
        s = _out_like(sum_out, x)
        st = load().gla_gated_add_rmsnorm(x.data_ptr(), residual.data_ptr(), _ptr(post_weight), _ptr(gate),
                                          groups, _ptr(scale), weight.data_ptr(), float(eps), s.data_ptr(),
                                          y.data_ptr(), rows, F, _dtype_code(x), st_ptr)
    _check(st, "gla_gated_add_rmsnorm")
    return y, s


def gated_add_rmsnorm_bwd(x: torch.Tensor, s: torch.Tensor, weight: torch.Tensor, eps: float,
                          gy: torch.Tensor, post_weight: Optional[torch.Tensor] = None,
                          gate: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                          gsum: Optional[torch.Tensor] = None, gx: Optional[torch.Tensor] = None,
                          gresidual: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None,
                          stream: Optional[torch.cuda.Stream] = None):
    """(gx, gresidual, gweight, gpost_weight, ggate, gscale) of
    gated_add_rmsnorm from its x and s, gy = dL/dy and gsum, the gradient that
    reaches s itself (None for none); None for those without an input. gx and
    gresidual may be written to x, s, gy or gsum; ggate has gate's shape and
    dtype, the weights' gradients are float32."""
    dev, rows, F, groups = _gated_norm_args(x, weight, post_weight, gate, scale)
    _alike(x.shape, x.dtype, dev, "s gy", s, gy)
    if gsum is not None:
        _like(gsum, x.shape, x.dtype, dev, "gsum")
    with _launching(dev, stream, x, s, weight, gy, post_weight, gate, scale, gsum, gx, gresidual,
                    workspace) as st_ptr:
        gx = _out_like(gx, x)
        gr = _out_like(gresidual, x)
        gw = torch.empty_like(weight)
        gp = None if post_weight is None else torch.empty_like(post_weight)
        gg = None if gate is None else torch.empty_like(gate)
        gs = None if scale is None else torch.empty_like(scale)
        if rows == 0 and F > 0:  # sums of nothing
            for g in (gw, gp, gg, gs):
                if g is not None:
                    g.zero_()
            return gx, gr, gw, gp, gg, gs
        workspace = _scratch(workspace, _gated_norm_workspace_bytes(rows, groups, F), dev)
        ws, nws = _ws(workspace, dev)
        st = load().gla_gated_add_rmsnorm_bwd(x.data_ptr(), s.data_ptr(), _ptr(post_weight), _ptr(gate),
                                              groups, _ptr(scale), weight.data_ptr(), float(eps),
                                              gy.data_ptr(), _ptr(gsum), gx.data_ptr(), gr.data_ptr(),
                                              _ptr(gp), _ptr(gg), _ptr(gs), gw.data_ptr(), rows, F,
                                              _dtype_code(x), ws, nws, st_ptr)
    _check(st, "gla_gated_add_rmsnorm_bwd")
    return gx, gr, gw, gp, gg, gs
