"""Python binding of libssd (include/ssd.h): argument marshalling only.

Every step of the layer runs in the library's CUDA kernels; this module checks tensor
devices, dtypes and shapes, allocates outputs with torch when the caller passes none,
and forwards raw device pointers and the current CUDA stream through ctypes.  Importing
it loads libssd.so and raises if the library has not been built: there is no fallback.
"""
import ctypes
import functools
import os
from typing import Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libssd.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT = range(6)
F32, BF16 = 0, 1
_DTYPES = {torch.float32: F32, torch.bfloat16: BF16}


class SSDError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


class Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int64),
                ("headdim", ctypes.c_int64), ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64)]


class GlrDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("row_stride", ctypes.c_int64), ("grad_stride", ctypes.c_int64)]


class NormDims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("gate_stride", ctypes.c_int64), ("dgate_stride", ctypes.c_int64)]


# Every symbol include/ssd.h declares.
EXPORTS = ("ssd_status_string", "ssd_version", "ssd_prefill_workspace_size",
           "ssd_prefill_kernel_launches", "ssd_prefill", "ssd_prefill_ex", "ssd_prefill_timed",
           "ssd_prefill_kernel_name", "ssd_prefill_device_status", "ssd_prefill_noalloc",
           "ssd_prefill_noalloc_max_workspace", "ssd_prefill_noalloc_device_status", "ssd_decode_step",
           "ssd_frontend", "ssd_decode_window_step", "ssd_decode_window_flush", "ssd_wait_selftest",
           "ssd_prefill_host_buffer_size", "ssd_prefill_host", "ssd_glr_prefill", "ssd_glr_decode_step",
           "ssd_glr_wait_selftest", "ssd_glr_backward_workspace_size", "ssd_glr_backward", "ssd_residual_norm",
           "ssd_norm_backward_workspace_size", "ssd_residual_norm_backward", "ssd_gated_norm",
           "ssd_gated_norm_backward")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libssd.so is not built ({LIB_PATH}); run "
                          "`python -m selective_state_space_10_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, fp, i64, ci, sz = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    dp = ctypes.POINTER(Dims)
    lib.ssd_status_string.argtypes = [ci]
    lib.ssd_status_string.restype = ctypes.c_char_p
    lib.ssd_version.argtypes = []
    lib.ssd_version.restype = ci
    lib.ssd_prefill_workspace_size.argtypes = [dp, ci, ci]
    lib.ssd_prefill_workspace_size.restype = sz
    lib.ssd_prefill_kernel_launches.argtypes = [dp, ci, ci]
    lib.ssd_prefill_kernel_launches.restype = ci
    lib.ssd_prefill.argtypes = [dp, ci, vp, fp, fp, vp, vp, fp, ci, fp, fp, vp, sz, vp]
    lib.ssd_prefill.restype = ci
    lib.ssd_prefill_ex.argtypes = [dp, ci, vp, fp, fp, vp, vp, fp, ci, fp, fp, fp, fp, vp, sz, vp]
    lib.ssd_prefill_ex.restype = ci
    lib.ssd_prefill_timed.argtypes = [dp, ci, vp, fp, fp, vp, vp, fp, ci, fp, fp, vp, sz, vp,
                                      ctypes.POINTER(ctypes.c_void_p), ci]
    lib.ssd_prefill_timed.restype = ci
    lib.ssd_prefill_kernel_name.argtypes = [dp, ci, ci, ci]
    lib.ssd_prefill_kernel_name.restype = ctypes.c_char_p
    lib.ssd_prefill_device_status.argtypes = [vp, sz, vp]
    lib.ssd_prefill_device_status.restype = ci
    lib.ssd_prefill_noalloc.argtypes = [dp, ci, vp, fp, fp, vp, vp, fp, ci, fp, fp, vp]
    lib.ssd_prefill_noalloc.restype = ci
    lib.ssd_prefill_noalloc_max_workspace.argtypes = []
    lib.ssd_prefill_noalloc_max_workspace.restype = sz
    lib.ssd_prefill_noalloc_device_status.argtypes = [vp]
    lib.ssd_prefill_noalloc_device_status.restype = ci
    lib.ssd_prefill_host_buffer_size.argtypes = [dp, ci, ci]
    lib.ssd_prefill_host_buffer_size.restype = sz
    lib.ssd_prefill_host.argtypes = [dp, ci, vp, fp, fp, vp, vp, fp, ci, fp, fp, vp, sz, vp]
    lib.ssd_prefill_host.restype = ci
    lib.ssd_decode_step.argtypes = [dp, ci, fp, vp, fp, fp, vp, vp, fp, fp, vp]
    lib.ssd_decode_step.restype = ci
    lib.ssd_wait_selftest.argtypes = [vp, sz, ctypes.c_uint64, ci, vp]
    lib.ssd_wait_selftest.restype = ci
    lib.ssd_frontend.argtypes = [dp, ci, vp, fp, fp, fp, fp, fp, fp, vp, vp, vp, fp, vp]
    lib.ssd_frontend.restype = ci
    lib.ssd_decode_window_step.argtypes = [dp, ci, ci, ci, fp, vp, fp, vp, vp, fp, fp, vp, vp, fp, fp, vp]
    lib.ssd_decode_window_step.restype = ci
    lib.ssd_decode_window_flush.argtypes = [dp, ci, ci, ci, fp, vp, fp, vp, fp, vp]
    lib.ssd_decode_window_flush.restype = ci
    gp, np_, f32 = ctypes.POINTER(GlrDims), ctypes.POINTER(NormDims), ctypes.c_float
    for name, args in (("ssd_glr_prefill", [gp, ci] + [vp] * 8),
                       ("ssd_glr_decode_step", [gp, ci] + [vp] * 7),
                       ("ssd_glr_backward", [gp, ci] + [vp] * 14 + [sz, vp]),
                       ("ssd_residual_norm", [np_, ci, ci, vp, vp, vp, vp, f32, vp, vp, vp]),
                       ("ssd_residual_norm_backward", [np_, ci, ci, vp, vp, vp, vp, f32] + [vp] * 7 + [sz, vp]),
                       ("ssd_gated_norm", [np_, ci, ci, ci, vp, vp, vp, f32, vp, vp]),
                       ("ssd_gated_norm_backward", [np_, ci, ci, ci, vp, vp, vp, f32] + [vp] * 5 + [sz, vp])):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = ci
    lib.ssd_glr_wait_selftest.argtypes = [fp, sz, ci, ci, ci, ci, ctypes.c_uint64, ctypes.c_uint64, vp]
    lib.ssd_glr_wait_selftest.restype = ci
    lib.ssd_glr_backward_workspace_size.argtypes = [gp, ci]
    lib.ssd_glr_backward_workspace_size.restype = sz
    lib.ssd_norm_backward_workspace_size.argtypes = [np_]
    lib.ssd_norm_backward_workspace_size.restype = sz
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.ssd_status_string(int(status)).decode()


def version() -> int:
    return lib.ssd_version()


def _dims(batch, seqlen, nheads, headdim, dstate, ngroups) -> Dims:
    return Dims(int(batch), int(seqlen), int(nheads), int(headdim), int(dstate), int(ngroups))


def dims_of_prefill(x: torch.Tensor, B: torch.Tensor) -> Dims:
    b, L, H, P = x.shape
    return _dims(b, L, H, P, B.shape[3], B.shape[2])


def prefill_workspace_size(dims: Dims, dtype: int, chunk: int) -> int:
    return lib.ssd_prefill_workspace_size(ctypes.byref(dims), int(dtype), int(chunk))


def prefill_kernel_launches(dims: Dims, dtype: int, chunk: int) -> int:
    return lib.ssd_prefill_kernel_launches(ctypes.byref(dims), int(dtype), int(chunk))


def prefill_kernel_names(dims: Dims, dtype: int, chunk: int):
    n = prefill_kernel_launches(dims, dtype, chunk)
    return [lib.ssd_prefill_kernel_name(ctypes.byref(dims), int(dtype), int(chunk), i).decode()
            for i in range(max(n, 0))]


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(t: torch.Tensor, name: str, shape, dtype, device):
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _scratch_bytes(t: torch.Tensor, name: str) -> int:
    """The bytes of a scratch tensor.  A strided or expanded view has other memory between or behind its elements, which
    the call would write."""
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.numel() * t.element_size()


def prefill(x, dt, A, B, C, D, chunk: int = 256, y=None, final_state=None, workspace=None,
            stream=None, events=None, initial_state=None, chunk_states=None):
    """Chunked prefill.  Returns (y fp32 [b,L,H,P], final_state fp32 [b,H,P,N]).
    x, B, C are fp32 or bf16 (the same dtype); dt, A, D are fp32.

    `initial_state` (fp32 [b,H,P,N], optional): the state before the first token (zero if
    None); it may be `final_state` itself.  `chunk_states`: None, True (allocate), or an
    fp32 tensor [b, ceil(L/chunk), H, P, N] that receives the state after every chunk;
    when given, the return value is (y, final_state, chunk_states).  Either one routes the
    call through ssd_prefill_ex.

    `events`: optional list of torch.cuda.Event(enable_timing=True), at least
    prefill_kernel_launches() + 1 of them, already recorded once (so their handles
    exist); the call then goes through ssd_prefill_timed, which records events[i] before
    kernel i and events[-1] after the last kernel (not with initial_state/chunk_states)."""
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x must be [b,L,H,P] and B, C [b,L,G,N]")
    if x.dtype not in _DTYPES:
        raise ValueError(f"unsupported input dtype {x.dtype}")
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("libssd runs on CUDA tensors only")
    b, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    _check(x, "x", (b, L, H, P), x.dtype, dev)
    _check(dt, "dt", (b, L, H), torch.float32, dev)
    _check(A, "A", (H,), torch.float32, dev)
    _check(B, "B", (b, L, G, N), x.dtype, dev)
    _check(C, "C", (b, L, G, N), x.dtype, dev)
    _check(D, "D", (H,), torch.float32, dev)
    if y is None:
        y = torch.empty((b, L, H, P), dtype=torch.float32, device=dev)
    if final_state is None:
        final_state = torch.empty((b, H, P, N), dtype=torch.float32, device=dev)
    _check(y, "y", (b, L, H, P), torch.float32, dev)
    _check(final_state, "final_state", (b, H, P, N), torch.float32, dev)
    if initial_state is not None:
        _check(initial_state, "initial_state", (b, H, P, N), torch.float32, dev)
    want_cs = chunk_states is not None and chunk_states is not False
    if chunk_states is True:
        chunk_states = torch.empty((b, -(-L // int(chunk)) if chunk > 0 else 0, H, P, N), dtype=torch.float32,
                                   device=dev)
    if want_cs:
        _check(chunk_states, "chunk_states", (b, -(-L // int(chunk)) if chunk > 0 else 0, H, P, N),
               torch.float32, dev)
    extended = initial_state is not None or want_cs
    if extended and events is not None:
        raise ValueError("events cannot be combined with initial_state or chunk_states")
    dims = dims_of_prefill(x, B)
    dtype = _DTYPES[x.dtype]
    need = prefill_workspace_size(dims, dtype, chunk)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else _scratch_bytes(workspace, "workspace")
    if extended:
        st = lib.ssd_prefill_ex(ctypes.byref(dims), dtype, _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                int(chunk), _ptr(initial_state), _ptr(y), _ptr(final_state),
                                _ptr(chunk_states if want_cs else None), _ptr(workspace), ws_bytes, _stream(stream))
        if st != OK:
            raise SSDError(st, "ssd_prefill_ex")
        return (y, final_state, chunk_states) if want_cs else (y, final_state)
    args = (ctypes.byref(dims), dtype, _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
            int(chunk), _ptr(y), _ptr(final_state), _ptr(workspace), ws_bytes, _stream(stream))
    if events is None:
        st = lib.ssd_prefill(*args)
    else:
        handles = (ctypes.c_void_p * len(events))(*[ev.cuda_event for ev in events])
        st = lib.ssd_prefill_timed(*args, handles, len(events))
    if st != OK:
        raise SSDError(st, "ssd_prefill")
    return y, final_state


def prefill_host_buffer_size(dims: Dims, dtype: int, chunk: int) -> int:
    return int(lib.ssd_prefill_host_buffer_size(ctypes.byref(dims), int(dtype), int(chunk)))


def prefill_host(x, dt, A, B, C, D, chunk: int = 256, y=None, final_state=None, device_buffer=None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """ssd_prefill_host: the prefill end to end from host tensors (page-locked for
    asynchronous copies).  The library copies the inputs to `device_buffer` (a CUDA uint8
    tensor of at least prefill_host_buffer_size() bytes; allocated if None), runs the
    prefill, and copies y and final_state into host tensors, all on `stream`.  Returns the
    host (y, final_state); read them after synchronising the stream."""
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x must be [b,L,H,P] and B, C [b,L,G,N]")
    if x.dtype not in _DTYPES:
        raise ValueError(f"unsupported input dtype {x.dtype}")
    host = torch.device("cpu")
    b, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    for t, name, shape, dtype in ((x, "x", (b, L, H, P), x.dtype), (dt, "dt", (b, L, H), torch.float32),
                                  (A, "A", (H,), torch.float32), (B, "B", (b, L, G, N), x.dtype),
                                  (C, "C", (b, L, G, N), x.dtype), (D, "D", (H,), torch.float32)):
        _check(t, name, shape, dtype, host)
    pin = x.is_pinned()
    if y is None:
        y = torch.empty((b, L, H, P), dtype=torch.float32, pin_memory=pin)
    if final_state is None:
        final_state = torch.empty((b, H, P, N), dtype=torch.float32, pin_memory=pin)
    _check(y, "y", (b, L, H, P), torch.float32, host)
    _check(final_state, "final_state", (b, H, P, N), torch.float32, host)
    dims = dims_of_prefill(x, B)
    dtype = _DTYPES[x.dtype]
    need = prefill_host_buffer_size(dims, dtype, chunk)
    if device_buffer is None:
        device_buffer = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    if device_buffer.device.type != "cuda":
        raise ValueError("device_buffer must be a CUDA tensor")
    st = lib.ssd_prefill_host(ctypes.byref(dims), dtype, _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                              int(chunk), _ptr(y), _ptr(final_state), _ptr(device_buffer),
                              _scratch_bytes(device_buffer, "device_buffer"), _stream(stream))
    if st != OK:
        raise SSDError(st, "ssd_prefill_host")
    return y, final_state


def prefill_noalloc(x, dt, A, B, C, D, chunk: int = 256, y=None, final_state=None,
                    stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """ssd_prefill_noalloc: the same prefill, with no workspace argument.  For callers
    that cannot allocate device memory, the library takes its scratch from a fixed array
    of prefill_noalloc_max_workspace() bytes; calls that overlap on the GPU race on it.
    (Outputs are still allocated here when not given; pass y and final_state to avoid
    that.)"""
    b, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    dev = x.device
    for name, t, shape, dtype in (("dt", dt, (b, L, H), torch.float32), ("A", A, (H,), torch.float32),
                                  ("B", B, (b, L, G, N), x.dtype), ("C", C, (b, L, G, N), x.dtype),
                                  ("D", D, (H,), torch.float32)):
        _check(t, name, shape, dtype, dev)
    if x.dtype not in _DTYPES:
        raise ValueError(f"unsupported input dtype {x.dtype}")
    if y is None:
        y = torch.empty((b, L, H, P), dtype=torch.float32, device=dev)
    if final_state is None:
        final_state = torch.empty((b, H, P, N), dtype=torch.float32, device=dev)
    _check(y, "y", (b, L, H, P), torch.float32, dev)
    _check(final_state, "final_state", (b, H, P, N), torch.float32, dev)
    st = lib.ssd_prefill_noalloc(ctypes.byref(dims_of_prefill(x, B)), _DTYPES[x.dtype], _ptr(x), _ptr(dt),
                                 _ptr(A), _ptr(B), _ptr(C), _ptr(D), int(chunk), _ptr(y), _ptr(final_state),
                                 _stream(stream))
    if st != OK:
        raise SSDError(st, "ssd_prefill_noalloc")
    return y, final_state


def prefill_noalloc_max_workspace() -> int:
    return lib.ssd_prefill_noalloc_max_workspace()


def prefill_noalloc_device_status(stream=None) -> int:
    """ssd_prefill_noalloc_device_status: waits for the stream and returns OK or
    ERR_TIMEOUT from the error word of the library's scratch array."""
    return lib.ssd_prefill_noalloc_device_status(_stream(stream))


def prefill_device_status(workspace, stream=None) -> int:
    """Blocks until `stream` is idle, then returns the status word the prefill kernels
    left in `workspace` (OK, or ERR_TIMEOUT if a bounded device-side wait expired)."""
    return lib.ssd_prefill_device_status(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                         _stream(stream))


def decode_step(state, x, dt, A, B, C, D, y=None, stream=None) -> torch.Tensor:
    """One cached decode step: updates `state` [b,H,P,N] fp32 in place, returns y fp32
    [b,H,P].  x [b,H,P] and B, C [b,G,N] are fp32 or bf16; dt [b,H], A, D [H] fp32."""
    if x.dim() != 3 or B.dim() != 3 or state.dim() != 4:
        raise ValueError("state must be [b,H,P,N], x [b,H,P], B and C [b,G,N]")
    if x.dtype not in _DTYPES:
        raise ValueError(f"unsupported input dtype {x.dtype}")
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("libssd runs on CUDA tensors only")
    b, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    _check(state, "state", (b, H, P, N), torch.float32, dev)
    _check(dt, "dt", (b, H), torch.float32, dev)
    _check(A, "A", (H,), torch.float32, dev)
    _check(B, "B", (b, G, N), x.dtype, dev)
    _check(C, "C", (b, G, N), x.dtype, dev)
    _check(D, "D", (H,), torch.float32, dev)
    if y is None:
        y = torch.empty((b, H, P), dtype=torch.float32, device=dev)
    _check(y, "y", (b, H, P), torch.float32, dev)
    dims = _dims(b, 1, H, P, N, G)
    st = lib.ssd_decode_step(ctypes.byref(dims), _DTYPES[x.dtype], _ptr(state), _ptr(x), _ptr(dt),
                             _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(y), _stream(stream))
    if st != OK:
        raise SSDError(st, "ssd_decode_step")
    return y


def window_buffers(state: torch.Tensor, window: int, dtype=torch.bfloat16, ngroups: int = 1):
    """Device buffers for the windowed decode of a state [b,H,P,N]: (win_x [b,W,H,P],
    win_dt [b,W,H] fp32, win_B [b,W,G,N]), in the call's input dtype."""
    b, H, P, N = state.shape
    dev = state.device
    return (torch.empty((b, window, H, P), dtype=dtype, device=dev),
            torch.empty((b, window, H), dtype=torch.float32, device=dev),
            torch.empty((b, window, ngroups, N), dtype=dtype, device=dev))


def decode_window_step(state, buffers, pos: int, x, dt, A, B, C, D, y=None, stream=None) -> torch.Tensor:
    """ssd_decode_window_step: this token's y from the committed `state` (not modified) and
    the `pos` tokens buffered since the last flush; stores the token in slot `pos`."""
    win_x, win_dt, win_B = buffers
    b, H, P, N = state.shape
    G = B.shape[1]
    dev = state.device
    if x.dtype not in _DTYPES:
        raise ValueError(f"unsupported input dtype {x.dtype}")
    W = win_x.shape[1]
    _check(state, "state", (b, H, P, N), torch.float32, dev)
    _check(win_x, "win_x", (b, W, H, P), x.dtype, dev)
    _check(win_dt, "win_dt", (b, W, H), torch.float32, dev)
    _check(win_B, "win_B", (b, W, G, N), x.dtype, dev)
    for name, t, shape, dtype in (("x", x, (b, H, P), x.dtype), ("dt", dt, (b, H), torch.float32),
                                  ("A", A, (H,), torch.float32), ("B", B, (b, G, N), x.dtype),
                                  ("C", C, (b, G, N), x.dtype), ("D", D, (H,), torch.float32)):
        _check(t, name, shape, dtype, dev)
    if y is None:
        y = torch.empty((b, H, P), dtype=torch.float32, device=dev)
    _check(y, "y", (b, H, P), torch.float32, dev)
    st = lib.ssd_decode_window_step(ctypes.byref(_dims(b, 1, H, P, N, G)), _DTYPES[x.dtype], W, int(pos),
                                    _ptr(state), _ptr(win_x), _ptr(win_dt), _ptr(win_B), _ptr(x), _ptr(dt),
                                    _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(y), _stream(stream))
    if st != OK:
        raise SSDError(st, "ssd_decode_window_step")
    return y


def decode_window_flush(state, buffers, count: int, A, stream=None) -> torch.Tensor:
    """ssd_decode_window_flush: folds the first `count` buffered tokens into `state`."""
    win_x, win_dt, win_B = buffers
    b, H, P, N = state.shape
    W, G = win_x.shape[1], win_B.shape[2]
    if win_x.dtype not in _DTYPES:
        raise ValueError(f"unsupported input dtype {win_x.dtype}")
    st = lib.ssd_decode_window_flush(ctypes.byref(_dims(b, 1, H, P, N, G)), _DTYPES[win_x.dtype], W, int(count),
                                     _ptr(state), _ptr(win_x), _ptr(win_dt), _ptr(win_B), _ptr(A),
                                     _stream(stream))
    if st != OK:
        raise SSDError(st, "ssd_decode_window_flush")
    return state


def frontend(xbc, conv_w, dt_raw, dt_bias, nheads: int, headdim: int, ngroups: int, dstate: int, conv_b=None,
             conv_state_in=None, conv_state_out=None, x=None, B=None, C=None, dt=None, stream=None):
    """ssd_frontend: conv (width 4, causal, depthwise) + SiLU over xbc [b, L, H*P + 2*G*N],
    split into x [b,L,H,P], B and C [b,L,G,N] (xbc's dtype), and dt = softplus(dt_raw +
    dt_bias) [b,L,H] fp32.  conv_state_in / conv_state_out: fp32 [b, 3, channels] or None;
    they may be the same tensor.  Returns (x, B, C, dt)."""
    b, L, CH = xbc.shape
    H, P, G, N = int(nheads), int(headdim), int(ngroups), int(dstate)
    if CH != H * P + 2 * G * N:
        raise ValueError(f"xbc has {CH} channels, expected {H * P + 2 * G * N}")
    if xbc.dtype not in _DTYPES:
        raise ValueError(f"unsupported input dtype {xbc.dtype}")
    dev = xbc.device
    _check(xbc, "xbc", (b, L, CH), xbc.dtype, dev)
    _check(conv_w, "conv_w", (CH, 4), torch.float32, dev)
    _check(dt_raw, "dt_raw", (b, L, H), torch.float32, dev)
    _check(dt_bias, "dt_bias", (H,), torch.float32, dev)
    if conv_b is not None:
        _check(conv_b, "conv_b", (CH,), torch.float32, dev)
    for name, t in (("conv_state_in", conv_state_in), ("conv_state_out", conv_state_out)):
        if t is not None:
            _check(t, name, (b, 3, CH), torch.float32, dev)
    x = torch.empty((b, L, H, P), dtype=xbc.dtype, device=dev) if x is None else x
    B = torch.empty((b, L, G, N), dtype=xbc.dtype, device=dev) if B is None else B
    C = torch.empty((b, L, G, N), dtype=xbc.dtype, device=dev) if C is None else C
    dt = torch.empty((b, L, H), dtype=torch.float32, device=dev) if dt is None else dt
    st = lib.ssd_frontend(ctypes.byref(_dims(b, L, H, P, N, G)), _DTYPES[xbc.dtype], _ptr(xbc), _ptr(conv_w),
                          _ptr(conv_b), _ptr(conv_state_in), _ptr(conv_state_out), _ptr(dt_raw), _ptr(dt_bias),
                          _ptr(x), _ptr(B), _ptr(C), _ptr(dt), _stream(stream))
    if st != OK:
        raise SSDError(st, "ssd_frontend")
    return x, B, C, dt


def wait_selftest(workspace, limit_ns: int = 1_000_000, expire: bool = True, stream=None) -> int:
    """ssd_wait_selftest, then ssd_prefill_device_status: ERR_TIMEOUT when the bounded
    device wait ran out (expire=True), OK when it completed."""
    nbytes = workspace.numel() * workspace.element_size()
    st = lib.ssd_wait_selftest(_ptr(workspace), nbytes, int(limit_ns), 1 if expire else 0, _stream(stream))
    if st != OK:
        raise SSDError(st, "ssd_wait_selftest")
    return prefill_device_status(workspace, stream)


# The calls below are short next to a decode step's host work: the checks first compare what
# holds for every good call, and _check only words the refusal.  Like all calls here they are
# outside torch's autograd: the gradients are calls of their own.

def _cuda(t: torch.Tensor, name: str) -> int:
    """The tensor's CUDA device index."""
    if t.dtype not in _DTYPES:
        raise ValueError(f"unsupported {name} dtype {t.dtype}")
    if not t.is_cuda:
        raise ValueError("libssd runs on CUDA tensors only")
    return t.get_device()


def _ok(t: torch.Tensor, name: str, shape, dtype, dev: int) -> None:
    """A contiguous tensor of this shape and dtype on CUDA device `dev`."""
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous() or t.get_device() != dev:
        _check(t, name, shape, dtype, torch.device("cuda", dev))


def _ok_f32(tensors, shape, dev: int) -> None:
    for name, t in tensors:
        if t is not None and (t.shape != shape or t.dtype is not torch.float32 or not t.is_contiguous() or
                              t.get_device() != dev):
            _check(t, name, shape, torch.float32, torch.device("cuda", dev))


def _call(fn, dev: int, args) -> None:
    """fn(*args, stream) on the tensors' device and that device's current stream."""
    stream = torch._C._cuda_getCurrentRawStream(dev)  # torch.cuda.current_stream(dev) without its object
    if dev == torch._C._cuda_getDevice():
        st = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, stream)
    if st != OK:
        raise SSDError(st, fn.__name__)


def _on(stream, like: torch.Tensor, fn, *args):
    """fn(*args) with `stream` (a torch stream or a handle) current, so that what fn allocates
    is that stream's memory too: nothing of it is reused before the stream has passed the call."""
    if not like.is_cuda:
        raise ValueError("libssd runs on CUDA tensors only")
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=like.device)
    elif stream.device != like.device:
        raise ValueError(f"stream is on {stream.device}, expected {like.device}")
    with torch.cuda.stream(stream):
        return fn(*args)


def _address(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _row_stride(t: torch.Tensor, name: str, shape, dtype, dev: int) -> int:
    """Elements between consecutive rows of a [..., D] array whose rows may be slices of wider
    ones: unit stride within a row, one stride from row to row over all leading axes."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        _check(t, name, shape, dtype, torch.device("cuda", dev) if dev >= 0 else t.device)
    D = shape[-1]
    if t.is_contiguous():
        return D
    strides, row, n = t.stride(), None, 1
    for k in range(len(shape) - 2, -1, -1):
        if shape[k] == 1:
            continue
        if row is None:
            row = strides[k]
        elif strides[k] != row * n:
            raise ValueError(f"{name} has strides {tuple(strides)}: its rows must be evenly spaced")
        n *= shape[k]
    row = D if row is None or n == 0 else row
    if (D > 1 and strides[-1] != 1) or row < D:
        raise ValueError(f"{name} has strides {tuple(strides)}: its rows must be contiguous and not overlap")
    return row


def _same_stride(names, x, r, i, shape, dtype, dev: int) -> int:
    """The row stride that three arrays share (any of them where there is one row at most)."""
    row = _row_stride(x, names[0], shape, dtype, dev)
    strides = x.stride()
    if (r.stride() == strides and i.stride() == strides and r.shape == shape and i.shape == shape and
            r.dtype is dtype and i.dtype is dtype and r.get_device() == dev and i.get_device() == dev):
        return row
    for name, t in ((names[1], r), (names[2], i)):
        other = _row_stride(t, name, shape, dtype, dev)
        if other != row and shape[:-1].numel() > 1:
            raise ValueError(f"{', '.join(names)} must have the same row stride, got {row} and {other}")
    return row


_XRI, _GRADS = ("x", "r", "i"), ("dx", "dr", "di")


def _new(like: torch.Tensor, shape, dtype) -> torch.Tensor:
    """A contiguous tensor on like's device; empty_like is the quickest way to one."""
    if like.shape == shape:
        return torch.empty_like(like, dtype=dtype, memory_format=torch.contiguous_format)
    return like.new_empty(shape, dtype=dtype)


@functools.lru_cache(maxsize=256)  # sizes depend on these numbers alone
def _glr_workspace(b: int, L: int, D: int, dtype: int) -> int:
    return lib.ssd_glr_backward_workspace_size(ctypes.byref(GlrDims(b, L, D, D, D)), dtype)


@functools.lru_cache(maxsize=256)
def _norm_workspace(rows: int, D: int) -> int:
    return lib.ssd_norm_backward_workspace_size(ctypes.byref(NormDims(rows, D, 1, D, D)))


def _workspace(workspace, need: int, like: torch.Tensor):
    if workspace is None:
        return like.new_empty(need, dtype=torch.uint8), need
    if workspace.device != like.device:
        raise ValueError(f"workspace is on {workspace.device}, expected {like.device}")
    return workspace, _scratch_bytes(workspace, "workspace")


def glr_prefill(x, r, i, A, initial_state=None, h=None, final_state=None, stream=None):
    """ssd_glr_prefill: the gated linear recurrence h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t with
    a_t = exp(A sigmoid(r_t)), over x, r, i [b, L, D] (fp32 or bf16; they may be column slices of one array)
    and A [D] fp32 (<= 0), from initial_state [b, D] fp32 (None: zero).  Returns (h [b, L, D] in x's dtype,
    final_state [b, D] fp32); final_state may be initial_state."""
    if stream is not None:
        return _on(stream, x, glr_prefill, x, r, i, A, initial_state, h, final_state)
    if x.dim() != 3:
        raise ValueError("x, r and i must be [b,L,D]")
    dev = _cuda(x, "x")
    shape = x.shape
    b, L, D = shape
    row = _same_stride(_XRI, x, r, i, shape, x.dtype, dev)
    _ok(A, "A", (D,), torch.float32, dev)
    if h is None:
        h = _new(x, shape, x.dtype)
    else:
        _ok(h, "h", shape, x.dtype, dev)
    if final_state is None:
        final_state = _new(A if initial_state is None else initial_state, (b, D), torch.float32)
    _ok_f32((("initial_state", initial_state), ("final_state", final_state)), (b, D), dev)
    dims = GlrDims(b, L, D, row, D)
    _call(lib.ssd_glr_prefill, dev,
          (ctypes.byref(dims), _DTYPES[x.dtype], x.data_ptr(), r.data_ptr(), i.data_ptr(), A.data_ptr(),
           _address(initial_state), h.data_ptr(), final_state.data_ptr()))
    return h, final_state


def glr_decode_step(state, x, r, i, A, h=None, stream=None) -> torch.Tensor:
    """ssd_glr_decode_step: one token of every sequence.  Updates `state` [b, D] fp32 in place and returns h
    [b, D]; x, r, i [b, D] as for glr_prefill (their rows may be slices)."""
    if stream is not None:
        return _on(stream, x, glr_decode_step, state, x, r, i, A, h)
    if x.dim() != 2:
        raise ValueError("x, r and i must be [b,D]")
    dev = _cuda(x, "x")
    shape = x.shape
    b, D = shape
    row = _same_stride(_XRI, x, r, i, shape, x.dtype, dev)
    _ok(A, "A", (D,), torch.float32, dev)
    _ok(state, "state", shape, torch.float32, dev)
    if h is None:
        h = _new(x, shape, x.dtype)
    else:
        _ok(h, "h", shape, x.dtype, dev)
    dims = GlrDims(b, 1, D, row, D)
    _call(lib.ssd_glr_decode_step, dev,
          (ctypes.byref(dims), _DTYPES[x.dtype], state.data_ptr(), x.data_ptr(), r.data_ptr(), i.data_ptr(),
           A.data_ptr(), h.data_ptr()))
    return h


def glr_wait_selftest(ranks: int, tiles: int, late_rank: int = -1, late_tile: int = 0, delay_ns: int = 0,
                      limit_ns: int = 100_000_000, out=None, stream=None) -> torch.Tensor:
    """ssd_glr_wait_selftest: the state after every warp's update of 1, [tiles, ranks, 4, 64] fp32, from the scans'
    exchange alone, with a rank that is late at one round and a limit of the waits."""
    if out is None:
        out = torch.empty((tiles, ranks, 4, 64), dtype=torch.float32, device="cuda")
    if not out.is_cuda or out.dtype is not torch.float32 or not out.is_contiguous():
        raise ValueError("out must be a contiguous fp32 CUDA tensor")
    st = lib.ssd_glr_wait_selftest(_ptr(out), out.numel() * 4, int(ranks), int(tiles), int(late_rank), int(late_tile),
                                   int(delay_ns), int(limit_ns), _stream(stream))
    if st != OK:
        raise SSDError(st, "ssd_glr_wait_selftest")
    return out


def glr_backward(x, r, i, A, h, dh, initial_state=None, dfinal_state=None, dx=None, dr=None, di=None, dA=None,
                 dinitial_state=None, workspace=None, stream=None):
    """ssd_glr_backward: gradients of glr_prefill from its inputs, its output h, and the gradients dh of h
    and dfinal_state of the final state (None: zero).  Returns (dx, dr, di, dA, dinitial_state); dx, dr and di
    given by the caller may be column slices of one array."""
    if stream is not None:
        return _on(stream, x, glr_backward, x, r, i, A, h, dh, initial_state, dfinal_state, dx, dr, di, dA,
                   dinitial_state, workspace)
    if x.dim() != 3:
        raise ValueError("x, r and i must be [b,L,D]")
    dev = _cuda(x, "x")
    shape = x.shape
    b, L, D = shape
    row = _same_stride(_XRI, x, r, i, shape, x.dtype, dev)
    _ok(h, "h", shape, x.dtype, dev)
    _ok(dh, "dh", shape, x.dtype, dev)
    _ok_f32((("A", A), ("dA", dA)), (D,), dev)
    _ok_f32((("initial_state", initial_state), ("dfinal_state", dfinal_state), ("dinitial_state", dinitial_state)),
            (b, D), dev)
    if dx is None and dr is None and di is None:
        dx, dr, di, grad = torch.empty_like(h), torch.empty_like(h), torch.empty_like(h), D
    else:
        dx, dr, di = (torch.empty_like(h) if t is None else t for t in (dx, dr, di))
        grad = _same_stride(_GRADS, dx, dr, di, shape, x.dtype, dev)
    dA = torch.empty_like(A) if dA is None else dA
    if dinitial_state is None:
        dinitial_state = _new(A if dfinal_state is None else dfinal_state, (b, D), torch.float32)
    dims = GlrDims(b, L, D, row, grad)
    workspace, nbytes = _workspace(workspace, _glr_workspace(b, L, D, _DTYPES[x.dtype]), A)
    _call(lib.ssd_glr_backward, dev,
          (ctypes.byref(dims), _DTYPES[x.dtype], x.data_ptr(), r.data_ptr(), i.data_ptr(), A.data_ptr(),
           _address(initial_state), h.data_ptr(), dh.data_ptr(), _address(dfinal_state), dx.data_ptr(),
           dr.data_ptr(), di.data_ptr(), dA.data_ptr(), dinitial_state.data_ptr(), workspace.data_ptr(), nbytes))
    return dx, dr, di, dA, dinitial_state


def _norm_rows(t: torch.Tensor, name: str):
    if t.dim() < 1:
        raise ValueError(f"{name} must be [..., D]")
    D = t.shape[-1]
    if D < 1:
        raise ValueError(f"{name} has no channels")
    return t.numel() // D, D


def residual_norm(x, weight, residual=None, scale=None, residual_dtype=None, eps: float = 1e-5, residual_out=None,
                  out=None, stream=None):
    """ssd_residual_norm, before a block: s = residual + scale * x (residual None: 0; scale None: 1), out =
    s / sqrt(mean(s^2) + eps) * weight over the last axis.  x [..., D] fp32 or bf16; residual in x's dtype or
    fp32; weight, scale [D] fp32.  Returns (out in x's dtype, s in residual_dtype: residual's, else x's);
    residual_out may be residual."""
    if stream is not None:
        return _on(stream, x, residual_norm, x, weight, residual, scale, residual_dtype, eps, residual_out, out)
    dev = _cuda(x, "x")
    shape = x.shape
    rows, D = _norm_rows(x, "x")
    _ok(x, "x", shape, x.dtype, dev)
    if residual_dtype is None:
        residual_dtype = residual.dtype if residual is not None else \
            residual_out.dtype if residual_out is not None else x.dtype
    if residual_dtype not in _DTYPES:
        raise ValueError(f"unsupported residual dtype {residual_dtype}")
    _ok_f32((("weight", weight), ("scale", scale)), (D,), dev)
    if residual is not None:
        _ok(residual, "residual", shape, residual_dtype, dev)
    if residual_out is None:
        residual_out = _new(x if residual is None else residual, shape, residual_dtype)
    else:
        _ok(residual_out, "residual_out", shape, residual_dtype, dev)
    if out is None:
        out = torch.empty_like(x)
    else:
        _ok(out, "out", shape, x.dtype, dev)
    dims = NormDims(rows, D, 1, D, D)
    _call(lib.ssd_residual_norm, dev,
          (ctypes.byref(dims), _DTYPES[x.dtype], _DTYPES[residual_dtype], x.data_ptr(), _address(scale),
           _address(residual), weight.data_ptr(), eps, residual_out.data_ptr(), out.data_ptr()))
    return out, residual_out


def residual_norm_backward(dout, s, weight, x=None, scale=None, dresidual_out=None, eps: float = 1e-5, dx=None,
                           dresidual=None, dweight=None, dscale=None, workspace=None, stream=None):
    """ssd_residual_norm_backward: gradients of residual_norm from dout, the sum `s` it returned, and the
    gradient dresidual_out of that sum (None: zero); x is needed with a scale.  Returns (dx, dresidual,
    dweight, dscale), dscale None without a scale; dresidual may be dresidual_out."""
    if stream is not None:
        return _on(stream, dout, residual_norm_backward, dout, s, weight, x, scale, dresidual_out, eps, dx,
                   dresidual, dweight, dscale, workspace)
    dev = _cuda(dout, "dout")
    if s.dtype not in _DTYPES:
        raise ValueError(f"unsupported s dtype {s.dtype}")
    shape = dout.shape
    rows, D = _norm_rows(dout, "dout")
    _ok(dout, "dout", shape, dout.dtype, dev)
    _ok(s, "s", shape, s.dtype, dev)
    if dresidual_out is not None:
        _ok(dresidual_out, "dresidual_out", shape, s.dtype, dev)
    if scale is not None:
        if x is None:
            raise ValueError("the gradient of scale needs x")
        _ok(x, "x", shape, dout.dtype, dev)
        dscale = torch.empty_like(scale) if dscale is None else dscale
    elif dscale is not None:
        raise ValueError("dscale without a scale")
    if dx is None:
        dx = torch.empty_like(dout)
    else:
        _ok(dx, "dx", shape, dout.dtype, dev)
    if dresidual is None:
        dresidual = torch.empty_like(s)
    else:
        _ok(dresidual, "dresidual", shape, s.dtype, dev)
    _ok_f32((("weight", weight), ("scale", scale), ("dweight", dweight), ("dscale", dscale)), (D,), dev)
    dweight = torch.empty_like(weight) if dweight is None else dweight
    dims = NormDims(rows, D, 1, D, D)
    workspace, nbytes = _workspace(workspace, _norm_workspace(rows, D), weight)
    _call(lib.ssd_residual_norm_backward, dev,
          (ctypes.byref(dims), _DTYPES[dout.dtype], _DTYPES[s.dtype], _address(x if scale is not None else None),
           _address(scale), s.data_ptr(), weight.data_ptr(), eps, dout.data_ptr(), _address(dresidual_out),
           dx.data_ptr(), dresidual.data_ptr(), dweight.data_ptr(), _address(dscale), workspace.data_ptr(), nbytes))
    return dx, dresidual, dweight, dscale


def gated_norm(y, z, weight, ngroups: int = 1, gate_first: bool = True, eps: float = 1e-5, out=None,
               stream=None) -> torch.Tensor:
    """ssd_gated_norm, after a mixer: with silu(z) = z sigmoid(z) and the mean over each of ngroups runs of
    channels, v / sqrt(mean(v^2) + eps) * weight for v = y silu(z) (gate_first), or the norm of y times
    silu(z).  y [..., D] in z's dtype or fp32 (as ssd_prefill writes it; heads are flattened by the caller); z
    fp32 or bf16, its rows may be slices of a projection's; weight [D] fp32.  Returns out in z's dtype."""
    if stream is not None:
        return _on(stream, z, gated_norm, y, z, weight, ngroups, gate_first, eps, out)
    dev = _cuda(z, "z")
    if y.dtype not in _DTYPES:
        raise ValueError(f"unsupported y dtype {y.dtype}")
    shape = y.shape
    rows, D = _norm_rows(y, "y")
    _ok(y, "y", shape, y.dtype, dev)
    gate = _row_stride(z, "z", shape, z.dtype, dev)
    _ok(weight, "weight", (D,), torch.float32, dev)
    if out is None:
        out = _new(z, shape, z.dtype)
    else:
        _ok(out, "out", shape, z.dtype, dev)
    dims = NormDims(rows, D, int(ngroups), gate, D)
    _call(lib.ssd_gated_norm, dev,
          (ctypes.byref(dims), _DTYPES[z.dtype], _DTYPES[y.dtype], int(bool(gate_first)), y.data_ptr(), z.data_ptr(),
           weight.data_ptr(), eps, out.data_ptr()))
    return out


def gated_norm_backward(dout, y, z, weight, ngroups: int = 1, gate_first: bool = True, eps: float = 1e-5, dy=None,
                        dz=None, dweight=None, workspace=None, stream=None):
    """ssd_gated_norm_backward: gradients of gated_norm from dout (z's dtype).  Returns (dy, dz, dweight); a
    dz given by the caller may be a slice of the projection's gradient."""
    if stream is not None:
        return _on(stream, z, gated_norm_backward, dout, y, z, weight, ngroups, gate_first, eps, dy, dz,
                   dweight, workspace)
    dev = _cuda(z, "z")
    if y.dtype not in _DTYPES:
        raise ValueError(f"unsupported y dtype {y.dtype}")
    shape = y.shape
    rows, D = _norm_rows(y, "y")
    _ok(y, "y", shape, y.dtype, dev)
    gate = _row_stride(z, "z", shape, z.dtype, dev)
    _ok(dout, "dout", shape, z.dtype, dev)
    if dy is None:
        dy = torch.empty_like(y)
    else:
        _ok(dy, "dy", shape, y.dtype, dev)
    if dz is None:
        dz, dgate = torch.empty_like(dout), D
    else:
        dgate = _row_stride(dz, "dz", shape, z.dtype, dev)
    _ok_f32((("weight", weight), ("dweight", dweight)), (D,), dev)
    dweight = torch.empty_like(weight) if dweight is None else dweight
    dims = NormDims(rows, D, int(ngroups), gate, dgate)
    workspace, nbytes = _workspace(workspace, _norm_workspace(rows, D), weight)
    _call(lib.ssd_gated_norm_backward, dev,
          (ctypes.byref(dims), _DTYPES[z.dtype], _DTYPES[y.dtype], int(bool(gate_first)), y.data_ptr(), z.data_ptr(),
           weight.data_ptr(), eps, dout.data_ptr(), dy.data_ptr(), dz.data_ptr(), dweight.data_ptr(),
           workspace.data_ptr(), nbytes))
    return dy, dz, dweight
