"""Python binding of libkda (KDA recurrence hot path for B200 / sm_100a).

Argument marshalling only: every function hands raw device pointers, sizes
and the current CUDA stream of ``torch`` to the C ABI declared in
``include/kda.h`` and raises :class:`KdaError` on a non-OK status.  All work
runs in the library's CUDA kernels; there is no other implementation behind
these names, and importing fails loudly when ``libkda.so`` has not been built
(``python -m gated_delta_rule_prologue_b200.build``).  With the environment variable
``KDA_LIB=debug`` the bounds-checked build ``libkda_debug.so`` is loaded instead.

Tensor conventions (all contiguous, on the current CUDA device):
  q, k, v              [T, H, D]       float32, bfloat16 or float16
  o                    [T, H, D]       float32 (read-outs are always float32)
  g                    [T, H, Dk]      float32 (log-decay, alpha = exp(g))
  beta                 [T, H]          float32
  state                [N, H, Dv, Dk]  float32 (key index contiguous)
  x (projections)      [T, 3*H*D]      activation dtype, channel p*H*D + h*D + d
  conv_w               [3*H*D, 4]      float32
  conv cache           [N, 3, 3*H*D]   activation dtype, oldest row first
  cu_seqlens           [N+1]           int32

A call runs on torch's current stream, or on ``stream``.  Scratch and outputs that a call allocates come
from that stream's memory, as under ``torch.cuda.stream(stream)``: before another stream uses such an
output, it waits for ``stream``, and the output outlives that use or is given to ``record_stream``.

Gated delta rule with one decay per head (``kda_gdr_*``): q, k [T, HK, D], v, o [T, HV, D],
g and beta [T, HV] float32, states [N, HV, D, D] float32, HV a multiple of HK.
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "KdaError",
    "LIB_PATH",
    "lib",
    "kda_prologue",
    "kda_chunk_fwd",
    "kda_chunk_fwd_windowed_workspace_bytes",
    "kda_decode_step",
    "kda_prologue_chunk_fwd",
    "kda_gdr_recurrent",
    "kda_gdr_decode_step",
    "kda_gdr_chunk_fwd",
    "kda_gdr_chunk_fwd_workspace_bytes",
    "kda_gdr_chunk_bwd",
    "kda_gdr_chunk_bwd_workspace_bytes",
    "kda_prologue_bwd",
    "kda_prologue_bwd_workspace_bytes",
    "kda_output_epilogue_bwd",
    "kda_output_epilogue_bwd_workspace_bytes",
    "kda_get_device_status",
    "kda_selftest_wait_timeout",
    "kda_selftest_bounds",
    "kda_debug_build",
    "kda_version",
    "KDA_OK",
    "KDA_ERR_INVALID_ARG",
    "KDA_ERR_UNSUPPORTED",
    "KDA_ERR_CUDA",
    "KDA_ERR_DEVICE_TIMEOUT",
    "KDA_ERR_DEVICE_BOUNDS",
    "KDA_ERR_DEVICE_RANGE",
]

# KDA_LIB=debug selects the bounds-checked build (libkda_debug.so, built by
# ``python -m gated_delta_rule_prologue_b200.build --debug``); anything else, the release build.
_LIB_NAME = "libkda_debug.so" if os.environ.get("KDA_LIB") == "debug" else "libkda.so"
LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), _LIB_NAME)

KDA_OK = 0
KDA_ERR_INVALID_ARG = 1
KDA_ERR_UNSUPPORTED = 2
KDA_ERR_CUDA = 3
KDA_ERR_DEVICE_TIMEOUT = 4
KDA_ERR_DEVICE_BOUNDS = 5
KDA_ERR_DEVICE_RANGE = 6
_F32, _BF16, _F16 = 0, 1, 2


class KdaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"libkda status {status}: {message}")
        self.status = status


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with "
                      "`python -m gated_delta_rule_prologue_b200.build`")

lib = ctypes.CDLL(LIB_PATH)
_vp, _i, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
lib.kda_prologue.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp,
                             _vp]
lib.kda_chunk_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _f, _vp, _vp, _i, _i, _i, _i, _i, _i,
                              _i, _vp, _vp, _vp]
lib.kda_chunk_fwd_ws.argtypes = [_vp, _vp, _vp, _vp, _vp, _f, _vp, _vp, _i, _i, _i, _i, _i, _i,
                                 _i, _vp, _vp, _vp, ctypes.c_size_t, _vp]
lib.kda_chunk_fwd_static.argtypes = [_vp, _vp, _vp, _vp, _vp, _f, _vp, _vp, _i, _i, _i, _i, _i,
                                     _i, _i, _vp, _vp, _vp]
lib.kda_prologue_chunk_fwd_ws.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _f, _vp, _vp, _i, _i,
                                          _i, _i, _i, _vp, _vp, _vp, ctypes.c_size_t, _vp]
lib.kda_chunk_fwd_gated_ws.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _f, _vp, _f, _vp, _vp, _i,
                                       _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, ctypes.c_size_t,
                                       _vp]
lib.kda_prologue_chunk_fwd_gated_ws.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _f, _vp, _f,
                                                _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp,
                                                ctypes.c_size_t, _vp]
lib.kda_decode_step_gated.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _f, _vp, _f, _vp, _i, _i, _i,
                                      _i, _vp, _vp]
lib.kda_output_epilogue.argtypes = [_vp, _vp, _vp, _f, _i, _i, _i, _i, _vp, _vp]
lib.kda_chunk_fwd_workspace_bytes.argtypes = [_i, _i, _i, _i, _i, _i, _i]
lib.kda_chunk_fwd_workspace_bytes.restype = ctypes.c_size_t
lib.kda_chunk_fwd_segmented_workspace_bytes.argtypes = [_i, _i, _i, _i, _i, _i, _i, _i]
lib.kda_chunk_fwd_segmented_workspace_bytes.restype = ctypes.c_size_t
lib.kda_chunk_bwd_workspace_bytes.argtypes = [_i, _i, _i, _i, _i, _i, _i]
lib.kda_chunk_bwd_workspace_bytes.restype = ctypes.c_size_t
lib.kda_chunk_bwd_ws.argtypes = [_vp, _vp, _vp, _vp, _vp, _f, _vp, _vp, _i, _i, _i, _i, _i, _i, _i,
                                 _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t,
                                 _vp]
lib.kda_chunk_map_workspace_bytes.argtypes = [_i, _i, _i, _i, _i, _i, _i]
lib.kda_chunk_map_workspace_bytes.restype = ctypes.c_size_t
lib.kda_chunk_map_ws.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _vp,
                                 _vp, ctypes.c_size_t, _vp]
lib.kda_state_compose.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _vp]
lib.kda_chunk_fwd_segment_chunks.argtypes = [_i, _i, _i]
lib.kda_chunk_fwd_segment_chunks.restype = ctypes.c_int
lib.kda_chunk_fwd_segmented_ws.argtypes = [_vp, _vp, _vp, _vp, _vp, _f, _vp, _vp, _i, _i, _i, _i,
                                           _i, _i, _i, _vp, _vp, _i, _vp, ctypes.c_size_t, _vp]
lib.kda_chunk_fwd_windowed_ws.argtypes = [_vp, _vp, _vp, _vp, _vp, _f, _vp, _vp, _i, _i, _i, _i,
                                          _i, _i, _i, _vp, _vp, _i, _vp, ctypes.c_size_t, _vp]
lib.kda_chunk_fwd_windowed_workspace_bytes.argtypes = [_i, _i, _i, _i, _i, _i, _i, _i]
lib.kda_prologue_chunk_fwd_windowed_ws.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _f, _vp, _vp,
                                                   _i, _i, _i, _i, _i, _vp, _vp, _i, _vp,
                                                   ctypes.c_size_t, _vp]
lib.kda_chunk_fwd_windowed_workspace_bytes.restype = ctypes.c_size_t
lib.kda_decode_step.argtypes = [_vp, _vp, _vp, _vp, _vp, _f, _vp, _i, _i, _i, _i, _vp, _vp]
lib.kda_prologue_chunk_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _f, _vp, _vp, _i, _i, _i,
                                       _i, _i, _vp, _vp, _vp]
lib.kda_gdr_recurrent.argtypes = [_vp] * 5 + [_f, _vp, _vp] + [_i] * 6 + [_vp] * 3
lib.kda_gdr_decode_step.argtypes = [_vp] * 5 + [_f, _vp] + [_i] * 5 + [_vp] * 2
lib.kda_gdr_chunk_fwd_ws.argtypes = ([_vp] * 5 + [_f, _vp, _vp] + [_i] * 6
                                     + [_vp] * 3 + [ctypes.c_size_t, _vp])
lib.kda_gdr_chunk_bwd_ws.argtypes = ([_vp] * 5 + [_f, _vp, _vp] + [_i] * 6
                                     + [_vp] * 9 + [ctypes.c_size_t, _vp])
lib.kda_prologue_bwd.argtypes = [_vp] * 4 + [_i] * 6 + [_vp] * 7 + [ctypes.c_size_t, _vp]
lib.kda_output_epilogue_bwd.argtypes = ([_vp] * 3 + [_f, _vp] + [_i] * 4 + [_vp] * 4
                                        + [ctypes.c_size_t, _vp])
for _fn, _n in ((lib.kda_gdr_chunk_fwd_workspace_bytes, 6),
                (lib.kda_gdr_chunk_bwd_workspace_bytes, 6),
                (lib.kda_prologue_bwd_workspace_bytes, 5),
                (lib.kda_output_epilogue_bwd_workspace_bytes, 3)):
    _fn.argtypes = [_i] * _n
    _fn.restype = ctypes.c_size_t
lib.kda_get_device_status.argtypes = [ctypes.POINTER(ctypes.c_int)]
lib.kda_selftest_wait_timeout.argtypes = [ctypes.c_uint, _vp]
lib.kda_selftest_bounds.argtypes = [_i, _vp]
lib.kda_debug_build.argtypes = []
lib.kda_debug_build.restype = ctypes.c_int
for _fn in (lib.kda_prologue, lib.kda_chunk_fwd, lib.kda_chunk_fwd_ws, lib.kda_chunk_fwd_static,
            lib.kda_chunk_fwd_segmented_ws, lib.kda_chunk_fwd_windowed_ws,
            lib.kda_prologue_chunk_fwd_windowed_ws,
            lib.kda_chunk_bwd_ws, lib.kda_chunk_map_ws,
            lib.kda_state_compose,
            lib.kda_prologue_chunk_fwd_ws, lib.kda_decode_step, lib.kda_chunk_fwd_gated_ws,
            lib.kda_prologue_chunk_fwd_gated_ws, lib.kda_decode_step_gated,
            lib.kda_output_epilogue, lib.kda_gdr_recurrent, lib.kda_gdr_decode_step,
            lib.kda_gdr_chunk_fwd_ws, lib.kda_gdr_chunk_bwd_ws, lib.kda_prologue_bwd,
            lib.kda_output_epilogue_bwd,
            lib.kda_prologue_chunk_fwd, lib.kda_get_device_status,
            lib.kda_selftest_wait_timeout, lib.kda_selftest_bounds):
    _fn.restype = ctypes.c_int
lib.kda_last_error.restype = ctypes.c_char_p
lib.kda_last_error.argtypes = []
lib.kda_version.restype = ctypes.c_char_p
lib.kda_version.argtypes = []


def _check(status: int):
    if status != KDA_OK:
        raise KdaError(status, lib.kda_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _dtype(t) -> int:
    if t.dtype == torch.float32:
        return _F32
    if t.dtype == torch.bfloat16:
        return _BF16
    if t.dtype == torch.float16:
        return _F16
    raise TypeError(f"unsupported activation dtype {t.dtype}")


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t, name, dtype=None):
    if t is None:
        return
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


_STREAM = torch.cuda.Stream


def _new(shape, dtype, device, stream):
    """An uninitialised tensor for a call on ``stream`` (None: the current one), taken from that
    stream's memory.  torch's allocator orders a block's uses by the stream it was allocated on: a
    block of the current stream might still be in use there when the call begins, and would be
    given away there, once its tensor is gone, while the call still works in it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, _STREAM):  # another library's, by its handle
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def kda_version() -> str:
    return lib.kda_version().decode()


def kda_get_device_status() -> int:
    """Read and clear the current device's status word (0 = no fault)."""
    code = ctypes.c_int(0)
    _check(lib.kda_get_device_status(ctypes.byref(code)))
    return code.value


def kda_selftest_wait_timeout(limit_us: int = 1000, stream=None):
    """Launch one CTA whose bounded mbarrier wait runs out after ``limit_us``
    microseconds; it records KDA_ERR_DEVICE_TIMEOUT in the status word and
    returns without faulting (the failure path of every tensor-core kernel)."""
    _check(lib.kda_selftest_wait_timeout(int(limit_us), _stream(stream)))


def kda_debug_build() -> bool:
    """True when the loaded library is the bounds-checked build (KDA_LIB=debug)."""
    return bool(lib.kda_debug_build())


def kda_selftest_bounds(index: int, stream=None):
    """Debug build only: one checked write of a four-slot device probe at ``index``;
    outside [0, 4) it records KDA_ERR_DEVICE_BOUNDS and skips the write."""
    _check(lib.kda_selftest_bounds(int(index), _stream(stream)))


def kda_prologue(x, conv_w, q, k, v, *, H: int, D: int, cache_in=None, cache_out=None,
                 cu_seqlens=None, stream=None):
    """Short conv + SiLU + L2 on q/k: writes ``q, k, v`` [T, H, D] (and ``cache_out``).
    ``x`` and the caches share one dtype; ``q, k, v`` share another."""
    for t, n in ((x, "x"), (cache_in, "cache_in"), (cache_out, "cache_out")):
        _need(t, n, x.dtype)
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype)
    _need(conv_w, "conv_w", torch.float32)
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    T = x.shape[0]
    _check(lib.kda_prologue(_ptr(x), _ptr(conv_w), _ptr(cache_in), _ptr(cache_out),
                            _ptr(cu_seqlens), N, T, H, D, _dtype(x), _dtype(q), _ptr(q),
                            _ptr(k), _ptr(v), _stream(stream)))


def kda_chunk_fwd_workspace_bytes(N: int, T: int, H: int, Dk: int, Dv: int, chunk: int,
                                  dtype: torch.dtype) -> int:
    """Scratch bytes of the two-pass tensor-core prefill (0 if it does not apply)."""
    return int(lib.kda_chunk_fwd_workspace_bytes(N, T, H, Dk, Dv, chunk, _DTYPES[dtype]))


def kda_chunk_fwd_segment_chunks(N: int, T: int, H: int) -> int:
    """Segment length (in 64-token chunks) of the sequence-parallel state pass
    that the workspace entry points pick for these sizes (0: whole sequences)."""
    return int(lib.kda_chunk_fwd_segment_chunks(N, T, H))


def kda_chunk_fwd_segmented_workspace_bytes(N: int, T: int, H: int, Dk: int, Dv: int, chunk: int,
                                            dtype: torch.dtype, segment_chunks: int) -> int:
    """Scratch bytes of the two-pass prefill at an explicit segment length."""
    return int(lib.kda_chunk_fwd_segmented_workspace_bytes(N, T, H, Dk, Dv, chunk,
                                                           _DTYPES[dtype], segment_chunks))


def kda_chunk_fwd(q, k, v, g, beta, o, *, scale: float = 1.0, initial_state=None,
                  final_state=None, cu_seqlens=None, chunk: int = 64, workspace="auto",
                  segment_chunks=None, window_chunks=None, stream=None):
    """Chunkwise prefill: writes ``o`` [T, H, Dv] and optionally ``final_state``.

    ``workspace``: ``"auto"`` allocates the two-pass path's scratch from
    torch's caching allocator; a uint8 CUDA tensor is used as given (at least
    :func:`kda_chunk_fwd_workspace_bytes`); ``None`` runs the one-pass kernels.
    ``segment_chunks``: ``None`` lets the library pick the state pass's segment
    length; an int (0: whole sequences) calls ``kda_chunk_fwd_segmented_ws``
    with it (workspace sized by :func:`kda_chunk_fwd_segmented_workspace_bytes`).
    ``window_chunks``: an int >= 1 calls ``kda_chunk_fwd_windowed_ws``: the passes run
    one window of that many chunk numbers at a time, so the workspace (sized by
    :func:`kda_chunk_fwd_windowed_workspace_bytes`) does not grow with T.
    """
    if window_chunks is not None:
        return _chunk_fwd_windowed(q, k, v, g, beta, o, scale, initial_state, final_state,
                                   cu_seqlens, chunk, workspace, int(window_chunks), stream)
    if segment_chunks is not None:
        return _chunk_fwd_segmented(q, k, v, g, beta, o, scale, initial_state, final_state,
                                    cu_seqlens, chunk, workspace, int(segment_chunks), stream)
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype)
    for t, n in ((o, "o"), (g, "g"), (beta, "beta"), (initial_state, "initial_state"),
                 (final_state, "final_state")):
        _need(t, n, torch.float32)
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    T, H, Dk = q.shape
    Dv = v.shape[2]
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError(f"workspace must be 'auto', None or a tensor, not {workspace!r}")
        nbytes = kda_chunk_fwd_workspace_bytes(N, T, H, Dk, Dv, chunk, q.dtype)
        workspace = (_new(nbytes, torch.uint8, q.device, stream) if nbytes else None)
    if workspace is None:
        _check(lib.kda_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale),
                                 _ptr(initial_state), _ptr(cu_seqlens), N, T, H, Dk, Dv, chunk,
                                 _dtype(q), _ptr(o), _ptr(final_state), _stream(stream)))
        return
    _need(workspace, "workspace", torch.uint8)
    _check(lib.kda_chunk_fwd_ws(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale),
                                _ptr(initial_state), _ptr(cu_seqlens), N, T, H, Dk, Dv, chunk,
                                _dtype(q), _ptr(o), _ptr(final_state), _ptr(workspace),
                                workspace.numel(), _stream(stream)))


def kda_chunk_fwd_windowed_workspace_bytes(N, T, H, Dk, Dv, chunk, dtype, window_chunks) -> int:
    return int(lib.kda_chunk_fwd_windowed_workspace_bytes(N, T, H, Dk, Dv, chunk,
                                                          _DTYPES[dtype], window_chunks))


def _chunk_fwd_windowed(q, k, v, g, beta, o, scale, initial_state, final_state, cu_seqlens,
                        chunk, workspace, window_chunks, stream):
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype)
    for t, n in ((o, "o"), (g, "g"), (beta, "beta"), (initial_state, "initial_state"),
                 (final_state, "final_state")):
        _need(t, n, torch.float32)
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    T, H, Dk = q.shape
    Dv = v.shape[2]
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError(f"workspace must be 'auto' or a tensor, not {workspace!r}")
        nbytes = kda_chunk_fwd_windowed_workspace_bytes(N, T, H, Dk, Dv, chunk, q.dtype,
                                                        window_chunks)
        workspace = _new(max(nbytes, 1), torch.uint8, q.device, stream)
    _need(workspace, "workspace", torch.uint8)
    _check(lib.kda_chunk_fwd_windowed_ws(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                         float(scale), _ptr(initial_state), _ptr(cu_seqlens), N,
                                         T, H, Dk, Dv, chunk, _dtype(q), _ptr(o),
                                         _ptr(final_state), int(window_chunks), _ptr(workspace),
                                         workspace.numel(), _stream(stream)))


def _chunk_fwd_segmented(q, k, v, g, beta, o, scale, initial_state, final_state, cu_seqlens,
                         chunk, workspace, segment_chunks, stream):
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype)
    for t, n in ((o, "o"), (g, "g"), (beta, "beta"), (initial_state, "initial_state"),
                 (final_state, "final_state")):
        _need(t, n, torch.float32)
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    T, H, Dk = q.shape
    Dv = v.shape[2]
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError(f"workspace must be 'auto' or a tensor, not {workspace!r}")
        nbytes = kda_chunk_fwd_segmented_workspace_bytes(N, T, H, Dk, Dv, chunk, q.dtype,
                                                         segment_chunks)
        workspace = _new(max(nbytes, 1), torch.uint8, q.device, stream)
    _need(workspace, "workspace", torch.uint8)
    _check(lib.kda_chunk_fwd_segmented_ws(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                          float(scale), _ptr(initial_state), _ptr(cu_seqlens), N,
                                          T, H, Dk, Dv, chunk, _dtype(q), _ptr(o),
                                          _ptr(final_state), segment_chunks, _ptr(workspace),
                                          workspace.numel(), _stream(stream)))


def kda_chunk_bwd_workspace_bytes(N: int, T: int, H: int, Dk: int, Dv: int, chunk: int,
                                  dtype: torch.dtype) -> int:
    """Scratch bytes of :func:`kda_chunk_bwd` (0 off the tensor-core shapes)."""
    return int(lib.kda_chunk_bwd_workspace_bytes(N, T, H, Dk, Dv, chunk, _DTYPES[dtype]))


def kda_chunk_bwd(q, k, v, g, beta, d_o, *, scale: float = 1.0, initial_state=None,
                  d_final_state=None, cu_seqlens=None, chunk: int = 64, dq=None, dk=None,
                  dv=None, dg=None, dbeta=None, d_initial_state=None, want_d_initial_state=True,
                  workspace="auto", stream=None):
    """Gradients of :func:`kda_chunk_fwd` for L = sum(d_o * o) + sum(d_final_state *
    final_state).  Returns ``(dq, dk, dv, dg, dbeta, d_initial_state)`` (fp32; the
    last is None unless wanted); output tensors not given are allocated."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype)
    for t, n in ((g, "g"), (beta, "beta"), (d_o, "d_o"), (initial_state, "initial_state"),
                 (d_final_state, "d_final_state")):
        _need(t, n, torch.float32)
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    T, H, Dk = q.shape
    Dv = v.shape[2]
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    dev = q.device
    dq = _new((T, H, Dk), torch.float32, dev, stream) if dq is None else dq
    dk = _new((T, H, Dk), torch.float32, dev, stream) if dk is None else dk
    dv = _new((T, H, Dv), torch.float32, dev, stream) if dv is None else dv
    dg = _new((T, H, Dk), torch.float32, dev, stream) if dg is None else dg
    dbeta = _new((T, H), torch.float32, dev, stream) if dbeta is None else dbeta
    if d_initial_state is None and want_d_initial_state:
        d_initial_state = _new((N, H, Dv, Dk), torch.float32, dev, stream)
    for t, n in ((dq, "dq"), (dk, "dk"), (dv, "dv"), (dg, "dg"), (dbeta, "dbeta"),
                 (d_initial_state, "d_initial_state")):
        _need(t, n, torch.float32)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError(f"workspace must be 'auto' or a tensor, not {workspace!r}")
        nbytes = kda_chunk_bwd_workspace_bytes(N, T, H, Dk, Dv, chunk, q.dtype)
        workspace = _new(max(nbytes, 1), torch.uint8, dev, stream)
    _need(workspace, "workspace", torch.uint8)
    _check(lib.kda_chunk_bwd_ws(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale),
                                _ptr(initial_state), _ptr(cu_seqlens), N, T, H, Dk, Dv, chunk,
                                _dtype(q), _ptr(d_o), _ptr(d_final_state), _ptr(dq), _ptr(dk),
                                _ptr(dv), _ptr(dg), _ptr(dbeta), _ptr(d_initial_state),
                                _ptr(workspace), workspace.numel(), _stream(stream)))
    return dq, dk, dv, dg, dbeta, d_initial_state


def kda_chunk_map(q, k, v, g, beta, *, cu_seqlens=None, chunk: int = 64, M=None, B=None,
                  workspace="auto", stream=None):
    """Affine map of each sequence's prefill, final = M S0 + B: returns ``(M, B)``,
    both [N, H, D, D] fp32 stored like a state (column-major)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype)
    for t, n in ((g, "g"), (beta, "beta")):
        _need(t, n, torch.float32)
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    T, H, Dk = q.shape
    Dv = v.shape[2]
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    M = _new((N, H, Dk, Dk), torch.float32, q.device, stream) if M is None else M
    B = _new((N, H, Dv, Dk), torch.float32, q.device, stream) if B is None else B
    _need(M, "M", torch.float32)
    _need(B, "B", torch.float32)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError(f"workspace must be 'auto' or a tensor, not {workspace!r}")
        nbytes = int(lib.kda_chunk_map_workspace_bytes(N, T, H, Dk, Dv, chunk, _DTYPES[q.dtype]))
        workspace = _new(max(nbytes, 1), torch.uint8, q.device, stream)
    _need(workspace, "workspace", torch.uint8)
    _check(lib.kda_chunk_map_ws(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens), N,
                                T, H, Dk, Dv, chunk, _dtype(q), _ptr(M), _ptr(B), _ptr(workspace),
                                workspace.numel(), _stream(stream)))
    return M, B


def kda_state_compose(M, B, E_in, E_out=None, stream=None):
    """E_out = M E_in + B per (sequence, head) (E_in None: zero); returns E_out."""
    for t, n in ((M, "M"), (B, "B"), (E_in, "E_in")):
        _need(t, n, torch.float32)
    N, H, D = B.shape[0], B.shape[1], B.shape[2]
    E_out = _new(B.shape, B.dtype, B.device, stream) if E_out is None else E_out
    _need(E_out, "E_out", torch.float32)
    _check(lib.kda_state_compose(_ptr(M), _ptr(B), _ptr(E_in), _ptr(E_out), N, H, D,
                                 _stream(stream)))
    return E_out


# Size of the library's fixed scratch buffer (one per device) used by
# kda_chunk_fwd_static; equals KDA_CHUNK_STATIC_SCRATCH_BYTES in kda.h.
KDA_CHUNK_STATIC_SCRATCH_BYTES = 64 << 20


def kda_chunk_fwd_static(q, k, v, g, beta, o, *, scale: float = 1.0, initial_state=None,
                         final_state=None, cu_seqlens=None, chunk: int = 64, stream=None):
    """The two-pass prefill with the library's fixed scratch buffer instead of
    a workspace: allocates nothing.  Sizes needing more scratch than
    KDA_CHUNK_STATIC_SCRATCH_BYTES raise KdaError (KDA_ERR_UNSUPPORTED).  All
    calls on a device share the buffer, so calls that may overlap in time
    (different streams) race; calls in order on one stream are safe."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype)
    for t, n in ((o, "o"), (g, "g"), (beta, "beta"), (initial_state, "initial_state"),
                 (final_state, "final_state")):
        _need(t, n, torch.float32)
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    T, H, Dk = q.shape
    Dv = v.shape[2]
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    _check(lib.kda_chunk_fwd_static(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale),
                                    _ptr(initial_state), _ptr(cu_seqlens), N, T, H, Dk, Dv,
                                    chunk, _dtype(q), _ptr(o), _ptr(final_state),
                                    _stream(stream)))


def kda_prologue_chunk_fwd(x, conv_w, g, beta, o, *, H: int, D: int, scale: float = 1.0,
                           cache_in=None, cache_out=None, initial_state=None, final_state=None,
                           cu_seqlens=None, workspace="auto", window_chunks=None, stream=None):
    """Prologue fused into the chunkwise prefill (chunk 64): ``x`` [T, 3*H*D]
    bf16/fp16 projections in, ``o`` [T, H, D] float32 out; q, k, v stay on chip.

    ``workspace`` as in :func:`kda_chunk_fwd`: ``"auto"`` (two passes, scratch
    from torch's caching allocator), a uint8 CUDA tensor, or ``None`` (the
    one-pass kernel).  ``window_chunks``: an int >= 1 calls
    ``kda_prologue_chunk_fwd_windowed_ws`` (a workspace that does not grow with T)."""
    for t, n in ((x, "x"), (cache_in, "cache_in"), (cache_out, "cache_out")):
        _need(t, n, x.dtype)
    for t, n in ((conv_w, "conv_w"), (o, "o"), (g, "g"), (beta, "beta"),
                 (initial_state, "initial_state"), (final_state, "final_state")):
        _need(t, n, torch.float32)
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    T = x.shape[0]
    if window_chunks is not None:
        if isinstance(workspace, str):
            if workspace != "auto":
                raise ValueError(f"workspace must be 'auto' or a tensor, not {workspace!r}")
            nbytes = kda_chunk_fwd_windowed_workspace_bytes(N, T, H, D, D, 64, x.dtype,
                                                            int(window_chunks))
            workspace = _new(max(nbytes, 1), torch.uint8, x.device, stream)
        _need(workspace, "workspace", torch.uint8)
        _check(lib.kda_prologue_chunk_fwd_windowed_ws(
            _ptr(x), _ptr(conv_w), _ptr(cache_in), _ptr(cache_out), _ptr(g), _ptr(beta),
            float(scale), _ptr(initial_state), _ptr(cu_seqlens), N, T, H, D, _dtype(x), _ptr(o),
            _ptr(final_state), int(window_chunks), _ptr(workspace), workspace.numel(),
            _stream(stream)))
        return
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError(f"workspace must be 'auto', None or a tensor, not {workspace!r}")
        nbytes = kda_chunk_fwd_workspace_bytes(N, T, H, D, D, 64, x.dtype)
        workspace = (_new(nbytes, torch.uint8, x.device, stream) if nbytes else None)
    if workspace is None:
        _check(lib.kda_prologue_chunk_fwd(_ptr(x), _ptr(conv_w), _ptr(cache_in), _ptr(cache_out),
                                          _ptr(g), _ptr(beta), float(scale), _ptr(initial_state),
                                          _ptr(cu_seqlens), N, T, H, D, _dtype(x), _ptr(o),
                                          _ptr(final_state), _stream(stream)))
        return
    _need(workspace, "workspace", torch.uint8)
    _check(lib.kda_prologue_chunk_fwd_ws(_ptr(x), _ptr(conv_w), _ptr(cache_in), _ptr(cache_out),
                                         _ptr(g), _ptr(beta), float(scale), _ptr(initial_state),
                                         _ptr(cu_seqlens), N, T, H, D, _dtype(x), _ptr(o),
                                         _ptr(final_state), _ptr(workspace), workspace.numel(),
                                         _stream(stream)))


def kda_decode_step(x, conv_w, conv_cache, g, beta, state, o, *, H: int, D: int,
                    scale: float = 1.0, stream=None):
    """One decode token per sequence; updates ``state`` and ``conv_cache`` in place."""
    for t, n in ((x, "x"), (conv_cache, "conv_cache")):
        _need(t, n, x.dtype)
    for t, n in ((o, "o"), (conv_w, "conv_w"), (g, "g"), (beta, "beta"), (state, "state")):
        _need(t, n, torch.float32)
    N = x.shape[0]
    _check(lib.kda_decode_step(_ptr(x), _ptr(conv_w), _ptr(conv_cache), _ptr(g), _ptr(beta),
                               float(scale), _ptr(state), N, H, D, _dtype(x), _ptr(o),
                               _stream(stream)))


def _auto_workspace(workspace, N, T, H, D, dtype, device, stream):
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError(f"workspace must be 'auto' or a tensor, not {workspace!r}")
        nbytes = kda_chunk_fwd_workspace_bytes(N, T, H, D, D, 64, dtype)
        return _new(max(nbytes, 16), torch.uint8, device, stream)
    _need(workspace, "workspace", torch.uint8)
    return workspace


def kda_chunk_fwd_gated(q, k, v, g_raw, beta, o, *, A_log=None, dt_bias=None,
                        lower_bound: float = -5.0, scale: float = 1.0, initial_state=None,
                        final_state=None, cu_seqlens=None, chunk: int = 64, workspace="auto",
                        stream=None):
    """Two-pass prefill with the log-decay computed in the kernel from the gate
    pre-activations ``g_raw`` [T, H, Dk] (q's dtype):
    g = lower_bound * sigmoid(exp(A_log[h]) * (g_raw + dt_bias[h, :]))."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (g_raw, "g_raw")):
        _need(t, n, q.dtype)
    for t, n in ((o, "o"), (beta, "beta"), (A_log, "A_log"), (dt_bias, "dt_bias"),
                 (initial_state, "initial_state"), (final_state, "final_state")):
        _need(t, n, torch.float32)
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    T, H, Dk = q.shape
    Dv = v.shape[2]
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    workspace = _auto_workspace(workspace, N, T, H, Dk, q.dtype, q.device, stream)
    _check(lib.kda_chunk_fwd_gated_ws(_ptr(q), _ptr(k), _ptr(v), _ptr(g_raw), _ptr(A_log),
                                      _ptr(dt_bias), float(lower_bound), _ptr(beta), float(scale),
                                      _ptr(initial_state), _ptr(cu_seqlens), N, T, H, Dk, Dv,
                                      chunk, _dtype(q), _ptr(o), _ptr(final_state),
                                      _ptr(workspace), workspace.numel(), _stream(stream)))


def kda_prologue_chunk_fwd_gated(x, conv_w, g_raw, beta, o, *, H: int, D: int, A_log=None,
                                 dt_bias=None, lower_bound: float = -5.0, scale: float = 1.0,
                                 cache_in=None, cache_out=None, initial_state=None,
                                 final_state=None, cu_seqlens=None, workspace="auto",
                                 stream=None):
    """Fused two-pass prefill (prologue in the prep pass) with the in-kernel gate."""
    for t, n in ((x, "x"), (g_raw, "g_raw"), (cache_in, "cache_in"), (cache_out, "cache_out")):
        _need(t, n, x.dtype)
    for t, n in ((conv_w, "conv_w"), (o, "o"), (beta, "beta"), (A_log, "A_log"),
                 (dt_bias, "dt_bias"), (initial_state, "initial_state"),
                 (final_state, "final_state")):
        _need(t, n, torch.float32)
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    T = x.shape[0]
    workspace = _auto_workspace(workspace, N, T, H, D, x.dtype, x.device, stream)
    _check(lib.kda_prologue_chunk_fwd_gated_ws(_ptr(x), _ptr(conv_w), _ptr(cache_in),
                                               _ptr(cache_out), _ptr(g_raw), _ptr(A_log),
                                               _ptr(dt_bias), float(lower_bound), _ptr(beta),
                                               float(scale), _ptr(initial_state),
                                               _ptr(cu_seqlens), N, T, H, D, _dtype(x), _ptr(o),
                                               _ptr(final_state), _ptr(workspace),
                                               workspace.numel(), _stream(stream)))


def kda_decode_step_gated(x, conv_w, conv_cache, g_raw, beta, state, o, *, H: int, D: int,
                          A_log=None, dt_bias=None, lower_bound: float = -5.0,
                          scale: float = 1.0, stream=None):
    """Decode step with the in-kernel gate; ``g_raw`` [N, H, D] of x's dtype."""
    for t, n in ((x, "x"), (conv_cache, "conv_cache"), (g_raw, "g_raw")):
        _need(t, n, x.dtype)
    for t, n in ((o, "o"), (conv_w, "conv_w"), (beta, "beta"), (state, "state"),
                 (A_log, "A_log"), (dt_bias, "dt_bias")):
        _need(t, n, torch.float32)
    N = x.shape[0]
    _check(lib.kda_decode_step_gated(_ptr(x), _ptr(conv_w), _ptr(conv_cache), _ptr(g_raw),
                                     _ptr(A_log), _ptr(dt_bias), float(lower_bound), _ptr(beta),
                                     float(scale), _ptr(state), N, H, D, _dtype(x), _ptr(o),
                                     _stream(stream)))


def kda_output_epilogue(o, gate, weight, out, *, eps: float = 1e-5, stream=None):
    """Per-head RMSNorm of the read-out ``o`` [T, H, D] (f32) times the output
    gate: out = o / sqrt(mean(o^2) + eps) * weight * sigmoid(gate); ``gate`` and
    ``out`` share a dtype."""
    _need(o, "o", torch.float32)
    _need(weight, "weight", torch.float32)
    _need(gate, "gate", out.dtype)
    _need(out, "out", out.dtype)
    T, H, D = o.shape
    _check(lib.kda_output_epilogue(_ptr(o), _ptr(gate), _ptr(weight), float(eps), T, H, D,
                                   _dtype(out), _ptr(out), _stream(stream)))


# ---- gated delta rule with one decay per head; backward of prologue and epilogue ----------
# These functions check shapes as well: the kernels trust the sizes they are given.  A decode
# step's kernel takes three microseconds, so a call's checks are one expression that reads each
# attribute once; where it fails, _p looks at the tensors one by one and names what is wrong.

# None on a torch without CUDA, where no call gets past its checks.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _p(t, name, shape, dtype, device):
    """Address of a contiguous tensor of this shape and dtype on CUDA device number ``device``,
    the current one (None: None); anything else is an error that says why."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on the current device cuda:{device}, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _cuda_device(t):
    """Number of the current device, which the call's tensors must be on."""
    if not t.is_cuda:
        raise ValueError("tensors must be CUDA tensors")
    return _current_device()


def _stream_of(stream, device):
    return _raw_stream(device) if stream is None else stream.cuda_stream


def _scratch(workspace, nbytes, device, like, stream):
    """Address and bytes of a workspace ("auto": ``nbytes`` from torch's caching allocator); the
    third value keeps it alive until the call has been made."""
    if workspace is None:
        return None, 0, None
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError(f"workspace must be 'auto', None or a tensor, not {workspace!r}")
        if nbytes == 0:
            return None, 0, None
        workspace = _new(nbytes, torch.uint8, like.device, stream)
    n = workspace.numel()
    return _p(workspace, "workspace", (n,), torch.uint8, device), n, workspace


def _gdr_sizes(q, v, cu_seqlens):
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v have three dimensions: tokens, heads, channels")
    T, HK, D = q.shape
    return 1 if cu_seqlens is None else cu_seqlens.shape[0] - 1, T, HK, v.shape[1], D


def _gdr_forward(q, k, v, g, beta, o, initial_state, final_state, cu_seqlens, one_token=False):
    """Checks the tensors of a forward call and returns its addresses and sizes: (q, k, v, g, beta),
    initial_state, cu_seqlens, (N, T, HK, HV, D, dtype), o, final_state, device."""
    N, T, HK, HV, D = _gdr_sizes(q, v, cu_seqlens)
    if one_token:
        N = T
    dev, f32 = _cuda_device(q), torch.float32
    dt, qk, vo, heads, sq = q.dtype, q.shape, (T, HV, D), (T, HV), (N, HV, D, D)
    s0, sN, cu = initial_state, final_state, cu_seqlens
    if not (k.shape == qk and v.shape == vo and o.shape == vo and g.shape == heads
            and beta.shape == heads and k.dtype is dt and v.dtype is dt and g.dtype is f32
            and beta.dtype is f32 and o.dtype is f32 and q.is_contiguous() and k.is_contiguous()
            and v.is_contiguous() and g.is_contiguous() and beta.is_contiguous()
            and o.is_contiguous() and q.get_device() == dev and k.get_device() == dev
            and v.get_device() == dev and g.get_device() == dev and beta.get_device() == dev
            and o.get_device() == dev
            and (s0 is None or (s0.shape == sq and s0.dtype is f32 and s0.is_contiguous()
                                and s0.get_device() == dev))
            and (sN is None or sN is s0 or (sN.shape == sq and sN.dtype is f32 and sN.is_contiguous()
                                            and sN.get_device() == dev))
            and (cu is None or (cu.dim() == 1 and cu.dtype is torch.int32 and cu.is_contiguous()
                                and cu.get_device() == dev))):
        _gdr_inputs(q, k, v, g, beta, T, HK, HV, D, dev)
        _p(cu, "cu_seqlens", (N + 1,), torch.int32, dev)
        _p(o, "o", vo, f32, dev)
        _p(s0, "initial_state", sq, f32, dev)
        _p(sN, "final_state", sq, f32, dev)
    return ((q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr()),
            None if s0 is None else s0.data_ptr(), None if cu is None else cu.data_ptr(),
            (N, T, HK, HV, D, _dtype(q)), o.data_ptr(), None if sN is None else sN.data_ptr(), dev)


def _gdr_inputs(q, k, v, g, beta, T, HK, HV, D, dev):
    dt, qk, heads = q.dtype, (T, HK, D), (T, HV)
    return (_p(q, "q", qk, dt, dev), _p(k, "k", qk, dt, dev), _p(v, "v", (T, HV, D), dt, dev),
            _p(g, "g", heads, torch.float32, dev), _p(beta, "beta", heads, torch.float32, dev))


def kda_gdr_recurrent(q, k, v, g, beta, o, *, scale: float = 1.0, initial_state=None,
                      final_state=None, cu_seqlens=None, stream=None):
    """Gated delta rule with one decay per head, token by token: writes ``o`` [T, HV, D] and
    optionally ``final_state`` (which may be ``initial_state``)."""
    x, s0, cu, sizes, op, sN, dev = _gdr_forward(q, k, v, g, beta, o, initial_state, final_state,
                                                 cu_seqlens)
    _check(lib.kda_gdr_recurrent(*x, scale, s0, cu, *sizes, op, sN, _stream_of(stream, dev)))


def kda_gdr_decode_step(q, k, v, g, beta, state, o, *, scale: float = 1.0, stream=None):
    """One new token for each of N sequences (``q, k`` [N, HK, D], ``v, o`` [N, HV, D]);
    updates ``state`` [N, HV, D, D] in place."""
    x, s0, _, sizes, op, _, dev = _gdr_forward(q, k, v, g, beta, o, state, state, None, True)
    _check(lib.kda_gdr_decode_step(*x, scale, s0, sizes[0], *sizes[2:], op, _stream_of(stream, dev)))


def kda_gdr_chunk_fwd_workspace_bytes(N: int, T: int, HK: int, HV: int, D: int,
                                      dtype: torch.dtype) -> int:
    """Scratch bytes of the fastest form of :func:`kda_gdr_chunk_fwd` (0: it runs the recurrent
    form).  They do not grow with N and T, but a workspace for the largest N and T serves every
    smaller one, in the fastest form that fits."""
    return int(lib.kda_gdr_chunk_fwd_workspace_bytes(N, T, HK, HV, D, _DTYPES[dtype]))


def kda_gdr_chunk_fwd(q, k, v, g, beta, o, *, scale: float = 1.0, initial_state=None,
                      final_state=None, cu_seqlens=None, workspace="auto", stream=None):
    """Chunkwise prefill of the gated delta rule with one decay per head: writes ``o``
    [T, HV, D] and optionally ``final_state``.

    ``workspace``: ``"auto"`` takes the scratch from torch's caching allocator; a uint8 CUDA
    tensor of :func:`kda_gdr_chunk_fwd_workspace_bytes` is used as given; ``None`` runs
    :func:`kda_gdr_recurrent`.  fp32 inputs and D below 64 run the recurrent form."""
    x, s0, cu, sizes, op, sN, dev = _gdr_forward(q, k, v, g, beta, o, initial_state, final_state,
                                                 cu_seqlens)
    nbytes = 0
    if isinstance(workspace, str):
        nbytes = lib.kda_gdr_chunk_fwd_workspace_bytes(*sizes)
    ws, nbytes, _keep = _scratch(workspace, nbytes, dev, q, stream)
    _check(lib.kda_gdr_chunk_fwd_ws(*x, scale, s0, cu, *sizes, op, sN, ws, nbytes,
                                    _stream_of(stream, dev)))


def kda_gdr_chunk_bwd_workspace_bytes(N: int, T: int, HK: int, HV: int, D: int,
                                      dtype: torch.dtype) -> int:
    """Scratch bytes of :func:`kda_gdr_chunk_bwd` (0 for sizes and types it does not have)."""
    return int(lib.kda_gdr_chunk_bwd_workspace_bytes(N, T, HK, HV, D, _DTYPES[dtype]))


def kda_gdr_chunk_bwd(q, k, v, g, beta, d_o, *, scale: float = 1.0, initial_state=None,
                      d_final_state=None, cu_seqlens=None, dq=None, dk=None, dv=None, dg=None,
                      dbeta=None, d_initial_state=None, want_d_initial_state=True,
                      workspace="auto", stream=None):
    """Gradients of :func:`kda_gdr_chunk_fwd` for L = sum(d_o * o) + sum(d_final_state *
    final_state).  Returns ``(dq, dk, dv, dg, dbeta, d_initial_state)``: the first three of q's
    dtype, the others fp32, the last None unless wanted; outputs not given are allocated.  Rows of
    tokens outside every sequence are left as they are (undefined where allocated here)."""
    N, T, HK, HV, D = _gdr_sizes(q, v, cu_seqlens)
    dev, f32, sq, dt = _cuda_device(q), torch.float32, (N, HV, D, D), _dtype(q)
    heads, qk, vo, act = (T, HV), (T, HK, D), (T, HV, D), q.dtype
    dq = _new(qk, act, q.device, stream) if dq is None else dq
    dk = _new(qk, act, q.device, stream) if dk is None else dk
    dv = _new(vo, act, q.device, stream) if dv is None else dv
    dg = _new(heads, f32, q.device, stream) if dg is None else dg
    dbeta = _new(heads, f32, q.device, stream) if dbeta is None else dbeta
    if d_initial_state is None and want_d_initial_state:
        d_initial_state = _new(sq, f32, q.device, stream)
    nbytes = 0
    if workspace is not None and isinstance(workspace, str):
        nbytes = max(lib.kda_gdr_chunk_bwd_workspace_bytes(N, T, HK, HV, D, dt), 16)
    ws, nbytes, _keep = _scratch(workspace, nbytes, dev, q, stream)
    _check(lib.kda_gdr_chunk_bwd_ws(
        *_gdr_inputs(q, k, v, g, beta, T, HK, HV, D, dev), scale,
        _p(initial_state, "initial_state", sq, f32, dev),
        _p(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, dev), N, T, HK, HV, D, dt,
        _p(d_o, "d_o", vo, f32, dev), _p(d_final_state, "d_final_state", sq, f32, dev),
        _p(dq, "dq", qk, act, dev), _p(dk, "dk", qk, act, dev), _p(dv, "dv", vo, act, dev),
        _p(dg, "dg", heads, f32, dev), _p(dbeta, "dbeta", heads, f32, dev),
        _p(d_initial_state, "d_initial_state", sq, f32, dev), ws, nbytes, _stream_of(stream, dev)))
    return dq, dk, dv, dg, dbeta, d_initial_state


def kda_prologue_bwd_workspace_bytes(N: int, T: int, H: int, D: int, dtype: torch.dtype) -> int:
    """Scratch bytes of :func:`kda_prologue_bwd` (may be 0)."""
    return int(lib.kda_prologue_bwd_workspace_bytes(N, T, H, D, _DTYPES[dtype]))


def kda_prologue_bwd(x, conv_w, dq, dk, dv, dx, d_conv_w=None, *, H: int, D: int, cache_in=None,
                     d_cache_in=None, cu_seqlens=None, workspace="auto", stream=None):
    """Gradients of :func:`kda_prologue` for L = sum(dq * q) + sum(dk * k) + sum(dv * v):
    writes ``dx`` (x's dtype) and, where given, ``d_conv_w`` [3*H*D, 4] (fp32) and
    ``d_cache_in`` (x's dtype).  ``dq, dk, dv`` [T, H, D] share a dtype of their own."""
    T, C = x.shape[0], 3 * H * D
    N = 1 if cu_seqlens is None else cu_seqlens.shape[0] - 1
    dev, f32, act, gt = _cuda_device(x), torch.float32, x.dtype, dq.dtype
    tc, thd, wc = (T, C), (T, H, D), (C, 4)
    if not (x.shape == tc and dx.shape == tc and conv_w.shape == wc and dq.shape == thd
            and dk.shape == thd and dv.shape == thd and dx.dtype is act and conv_w.dtype is f32
            and dk.dtype is gt and dv.dtype is gt and x.is_contiguous() and dx.is_contiguous()
            and conv_w.is_contiguous() and dq.is_contiguous() and dk.is_contiguous()
            and dv.is_contiguous() and x.get_device() == dev and dx.get_device() == dev
            and conv_w.get_device() == dev and dq.get_device() == dev and dk.get_device() == dev
            and dv.get_device() == dev):
        for t, name, shape, kind in ((x, "x", tc, act), (conv_w, "conv_w", wc, f32),
                                     (dq, "dq", thd, gt), (dk, "dk", thd, gt), (dv, "dv", thd, gt),
                                     (dx, "dx", tc, act)):
            _p(t, name, shape, kind, dev)
    dt = _dtype(x)
    nbytes = 0
    if d_conv_w is not None and isinstance(workspace, str):
        nbytes = lib.kda_prologue_bwd_workspace_bytes(N, T, H, D, dt)
    ws, nbytes, _keep = _scratch(workspace, nbytes, dev, x, stream)
    _check(lib.kda_prologue_bwd(
        x.data_ptr(), conv_w.data_ptr(), _p(cache_in, "cache_in", (N, 3, C), act, dev),
        _p(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, dev), N, T, H, D, dt, _dtype(dq),
        dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dx.data_ptr(),
        _p(d_conv_w, "d_conv_w", wc, f32, dev), _p(d_cache_in, "d_cache_in", (N, 3, C), act, dev), ws,
        nbytes, _stream_of(stream, dev)))


def kda_output_epilogue_bwd_workspace_bytes(T: int, H: int, D: int) -> int:
    """Scratch bytes of :func:`kda_output_epilogue_bwd` (may be 0)."""
    return int(lib.kda_output_epilogue_bwd_workspace_bytes(T, H, D))


def kda_output_epilogue_bwd(o, gate, weight, d_out, d_o, d_gate, d_weight=None, *,
                            eps: float = 1e-5, workspace="auto", stream=None):
    """Gradients of :func:`kda_output_epilogue` for L = sum(d_out * out): writes ``d_o`` (fp32),
    ``d_gate`` (gate's dtype) and, where given, ``d_weight`` [D] (fp32)."""
    if o.dim() != 3:
        raise ValueError("o has three dimensions: tokens, heads, channels")
    thd = T, H, D = o.shape
    dev, f32, dt = _cuda_device(o), torch.float32, gate.dtype
    if not (gate.shape == thd and d_out.shape == thd and d_o.shape == thd and d_gate.shape == thd
            and weight.shape == (D,) and o.dtype is f32 and weight.dtype is f32 and d_o.dtype is f32
            and d_out.dtype is dt and d_gate.dtype is dt and o.is_contiguous()
            and gate.is_contiguous() and weight.is_contiguous() and d_out.is_contiguous()
            and d_o.is_contiguous() and d_gate.is_contiguous() and o.get_device() == dev
            and gate.get_device() == dev and weight.get_device() == dev
            and d_out.get_device() == dev and d_o.get_device() == dev and d_gate.get_device() == dev):
        for t, name, kind in ((o, "o", f32), (gate, "gate", dt), (d_out, "d_out", dt),
                              (d_o, "d_o", f32), (d_gate, "d_gate", dt)):
            _p(t, name, thd, kind, dev)
        _p(weight, "weight", (D,), f32, dev)
    nbytes = 0
    if d_weight is not None and isinstance(workspace, str):
        nbytes = lib.kda_output_epilogue_bwd_workspace_bytes(T, H, D)
    ws, nbytes, _keep = _scratch(workspace, nbytes, dev, o, stream)
    _check(lib.kda_output_epilogue_bwd(
        o.data_ptr(), gate.data_ptr(), weight.data_ptr(), eps, d_out.data_ptr(), T, H, D,
        _dtype(gate), d_o.data_ptr(), d_gate.data_ptr(), _p(d_weight, "d_weight", (D,), f32, dev), ws,
        nbytes, _stream_of(stream, dev)))
