"""ctypes binding of libssd (include/ssd.h) for torch tensors.

Argument marshalling only: every step of the scan and of the recurrent step
runs in the HIP kernels of libssd.so.  There is no fallback: if the library
is not built, loading it raises.

    out, final = ssd_scan_fwd(x, dt, dt_bias, A, B, C, D, init_state, chunk=256)
    y = ssd_step(state, x, dt, A, B, C, D)          # state updated in place

``stream`` is a HIP stream's handle (default: torch's current stream).  What a
call allocates itself, outputs that were not passed in and its workspace,
belongs to the stream it runs on, as under ``torch.cuda.stream``: the caller
lets that stream wait for the inputs, and other streams wait for it before
they use the results (and ``record_stream`` results that they outlive).
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import struct
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libssd.so")

SSD_F32, SSD_BF16, SSD_U8, SSD_I32, SSD_I64 = 0, 1, 2, 3, 4
SSD_GLR_SEGMENT = 64
SSD_ALGO_AUTO, SSD_ALGO_FUSED, SSD_ALGO_CHUNKED, SSD_ALGO_ROWS, SSD_ALGO_QUAD = 0, 1, 2, 3, 4
STATUS = {0: "SSD_OK", 1: "SSD_ERR_NULL", 2: "SSD_ERR_SHAPE", 3: "SSD_ERR_DTYPE",
          4: "SSD_ERR_LAYOUT", 5: "SSD_ERR_UNSUPPORTED", 6: "SSD_ERR_ALIAS",
          7: "SSD_ERR_NOMEM", 8: "SSD_ERR_HIP"}


class SsdTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("strides", ctypes.c_int64 * 4)]


class SsdError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("%s: %s" % (STATUS.get(status, status), message))
        self.status = status


_lib = None


def lib():
    """Load libssd.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libssd.so is not built (python -m mamba_ssd_scan_05_amd.build)")
        L = ctypes.CDLL(LIB_PATH)
        # tensor descriptors go in as addresses (ctypes pointers from
        # describe() are accepted too)
        P = ctypes.c_void_p
        L.ssd_scan_fwd.argtypes = [P] * 10 + [ctypes.c_int, ctypes.c_void_p]
        L.ssd_scan_fwd.restype = ctypes.c_int
        L.ssd_scan_fwd_algo.argtypes = [P] * 10 + [ctypes.c_int, ctypes.c_int, ctypes.c_void_p]
        L.ssd_scan_fwd_algo.restype = ctypes.c_int
        L.ssd_scan_fwd_rows.argtypes = [P] * 10 + [ctypes.c_int, ctypes.c_void_p]
        L.ssd_scan_fwd_rows.restype = ctypes.c_int
        L.ssd_scan_fwd_gated.argtypes = [P] * 11 + [ctypes.c_int, ctypes.c_int, ctypes.c_void_p]
        L.ssd_scan_fwd_gated.restype = ctypes.c_int
        L.ssd_selective_scan_fwd.argtypes = [P] * 10 + [ctypes.c_int, ctypes.c_void_p]
        L.ssd_selective_scan_fwd.restype = ctypes.c_int
        L.ssd_step.argtypes = [P] * 8 + [ctypes.c_void_p]
        L.ssd_scan_bwd.argtypes = [P] * 18 + [ctypes.c_void_p]
        L.ssd_scan_bwd.restype = ctypes.c_int
        L.ssd_scan_bwd_gated.argtypes = [P] * 20 + [ctypes.c_void_p]
        L.ssd_scan_bwd_gated.restype = ctypes.c_int
        L.ssd_step.restype = ctypes.c_int
        L.ssd_status_string.argtypes = [ctypes.c_int]
        L.ssd_status_string.restype = ctypes.c_char_p
        L.ssd_last_error.restype = ctypes.c_char_p
        L.ssd_version.restype = ctypes.c_int
        L.ssd_release_scratch.restype = ctypes.c_int
        L.ssd_release_scratch.argtypes = []
        L.ssd_scratch_stats.argtypes = [ctypes.POINTER(ctypes.c_int64)] * 2
        L.ssd_scratch_stats.restype = ctypes.c_int
        L.ssd_scan_fwd_noalloc.argtypes = [P] * 10 + [ctypes.c_int, ctypes.c_void_p]
        L.ssd_scan_fwd_noalloc.restype = ctypes.c_int
        L.ssd_fixed_scratch_bytes.argtypes = []
        L.ssd_fixed_scratch_bytes.restype = ctypes.c_int64
        L.ssd_scan_plan.argtypes = [ctypes.c_int64] * 6 + [ctypes.c_int, ctypes.c_int,
                                                            ctypes.POINTER(ctypes.c_int),
                                                            ctypes.POINTER(ctypes.c_int)]
        L.ssd_scan_plan.restype = ctypes.c_int
        I64 = ctypes.c_int64
        L.ssd_glr_workspace.argtypes = [I64] * 3 + [ctypes.c_int]
        L.ssd_glr_workspace.restype = I64
        L.ssd_glr_fwd.argtypes = [P] * 13 + [I64, P]
        L.ssd_glr_fwd.restype = ctypes.c_int
        L.ssd_glr_bwd.argtypes = [P] * 20 + [I64, P]
        L.ssd_glr_bwd.restype = ctypes.c_int
        L.ssd_glr_step.argtypes = [P] * 11
        L.ssd_glr_step.restype = ctypes.c_int
        L.ssd_norm_rotate_workspace.argtypes = [I64]
        L.ssd_norm_rotate_workspace.restype = I64
        L.ssd_norm_rotate_fwd.argtypes = [P] * 8 + [ctypes.c_float, ctypes.c_int, P]
        L.ssd_norm_rotate_fwd.restype = ctypes.c_int
        L.ssd_norm_rotate_bwd.argtypes = [P] * 12 + [ctypes.c_float, ctypes.c_int, P, I64, P]
        L.ssd_norm_rotate_bwd.restype = ctypes.c_int
        L.ssd_kv_append.argtypes = [P] * 10 + [ctypes.c_int, P]
        L.ssd_kv_append.restype = ctypes.c_int
        L.ssd_attn_workspace.argtypes = [I64] * 5
        L.ssd_attn_workspace.restype = I64
        L.ssd_attn_fwd.argtypes = [P] * 8 + [ctypes.c_float, I64, P, I64, P]
        L.ssd_attn_fwd.restype = ctypes.c_int
        L.ssd_attn_step.argtypes = [P] * 7 + [ctypes.c_float, I64, P, I64, P]
        L.ssd_attn_step.restype = ctypes.c_int
        _lib = L
    return _lib


_DTYPE_CODE = {torch.float32: SSD_F32, torch.bfloat16: SSD_BF16, torch.uint8: SSD_U8, torch.bool: SSD_U8,
               torch.int32: SSD_I32, torch.int64: SSD_I64}


def _dtype_code(t: torch.Tensor) -> int:
    return _DTYPE_CODE.get(t.dtype, 99)  # 99: rejected by the library as SSD_ERR_DTYPE


def describe(t: Optional[torch.Tensor]):
    """ssd_tensor descriptor of a torch tensor (None -> NULL pointer)."""
    if t is None:
        return None
    if t.dim() > 4:
        raise ValueError("ssd tensors have at most 4 dimensions")
    d = SsdTensor()
    d.data = t.data_ptr() if t.numel() else 0
    d.dtype = _dtype_code(t)
    d.ndim = t.dim()
    for i, (s, st) in enumerate(zip(t.shape, t.stride())):
        d.shape[i] = s
        d.strides[i] = st
    return ctypes.pointer(d)


# ssd_tensor as packed bytes: data, dtype, ndim, shape[4], strides[4]
_DESC = struct.Struct("<Qii4q4q")
assert _DESC.size == ctypes.sizeof(SsdTensor)


def _descs_py(*ts):
    """Descriptors of a call's tensors in one buffer: (buffer, addresses),
    None -> NULL.  Keep the buffer alive until the call returns."""
    buf = ctypes.create_string_buffer(_DESC.size * len(ts))
    base = ctypes.addressof(buf)
    addrs = []
    for i, t in enumerate(ts):
        if t is None:
            addrs.append(None)
            continue
        n = t.dim()
        if n > 4:
            raise ValueError("ssd tensors have at most 4 dimensions")
        pad = (0,) * (4 - n)
        _DESC.pack_into(buf, i * _DESC.size, t.data_ptr() if t.numel() else 0, _dtype_code(t), n,
                        *t.shape, *pad, *t.stride(), *pad)
        addrs.append(base + i * _DESC.size)
    return buf, addrs


def _descs_native(*ts):
    """_descs_py through the module _pydesc: the descriptors are bytes objects
    (ctypes passes their addresses), owned by the tuple."""
    d = _pydesc.pack(*ts)
    return d, d


# Same descriptors either way (a wheel of the plain sources has no _pydesc);
# the native module takes under 1 us for ten tensors, the Python one 7.
try:
    from . import _pydesc
    _descs = _descs_native
except ImportError:
    _descs = _descs_py


_NO_CONTEXT = contextlib.nullcontext()


def _on_device(t):
    """Make t's device current for the call (the library launches on the
    current device and refuses memory that device cannot address)."""
    if t is not None and t.is_cuda and t.get_device() != torch._C._cuda_getDevice():
        return torch.cuda.device(t.device)
    return _NO_CONTEXT


def _stream(stream, t):
    if stream is not None:
        return stream
    if t is not None and t.is_cuda:
        # torch.cuda.current_stream(t.device).cuda_stream without the Stream
        # object (1.9 us)
        return torch._C._cuda_getCurrentRawStream(t.get_device())
    return None


def _on_stream(stream, t):
    """Makes the call's stream torch's current one while the call's own tensors
    are allocated.  A block of another stream's pool may still be in use by
    that stream's earlier work, and may be handed out to its later work while
    this call is writing it."""
    if stream is None or t is None or not t.is_cuda or stream == torch._C._cuda_getCurrentRawStream(t.get_device()):
        return _NO_CONTEXT
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=t.device))


def _check(status: int):
    if status != 0:
        raise SsdError(status, lib().ssd_last_error().decode())


def ssd_scan_fwd(x, dt, dt_bias, A, B, C, D=None, init_state=None, out=None,
                 final_state=None, chunk: int = 256, stream=None,
                 algo: int = SSD_ALGO_AUTO, return_final_state: bool = True):
    """Forward SSD scan; returns (out, final_state or None)."""
    with _on_stream(stream, x):
        if out is None:
            out = torch.empty_like(x)
        if final_state is None and return_final_state:
            final_state = torch.empty((x.shape[0], x.shape[2], x.shape[3], B.shape[3]),
                                      dtype=torch.float32, device=x.device)
    keep, d = _descs(x, dt, dt_bias, A, B, C, D, init_state, out, final_state)
    with _on_device(x):
        st = _stream(stream, x)
        if algo == SSD_ALGO_AUTO:
            # the library's own plan: the plain entry point
            status = lib().ssd_scan_fwd(*d, int(chunk), st)
        else:
            status = lib().ssd_scan_fwd_algo(*d, int(chunk), int(algo), st)
    _check(status)
    return out, final_state


def ssd_scan_fwd_noalloc(x, dt, dt_bias, A, B, C, D=None, init_state=None, out=None,
                         final_state=None, chunk: int = 256, stream=None):
    """ssd_scan_fwd through the allocation-free entry point (scratch in the
    library's fixed device array).  out (and final_state, if wanted) should
    be passed in by callers that cannot allocate; returns (out, final_state)."""
    if out is None:
        with _on_stream(stream, x):
            out = torch.empty_like(x)
    with _on_device(x):
        st = _stream(stream, x)
        keep, d = _descs(x, dt, dt_bias, A, B, C, D, init_state, out, final_state)
        status = lib().ssd_scan_fwd_noalloc(*d, int(chunk), st)
    _check(status)
    return out, final_state


def ssd_fixed_scratch_bytes() -> int:
    return int(lib().ssd_fixed_scratch_bytes())


def ssd_scratch_stats():
    """(number of kept scratch buffers, their total bytes)."""
    n, t = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().ssd_scratch_stats(ctypes.byref(n), ctypes.byref(t)))
    return n.value, t.value


def ssd_scan_bwd(x, dt, dt_bias, A, B, C, D, init_state, dout, dfinal_state=None, *,
                 want_dt_bias: bool = True, want_D: bool = True, want_init: bool = True,
                 out: dict = None, stream=None):
    """Gradients of ssd_scan_fwd for the objective <dout, y> + <dfinal_state, final state>.

    Returns a dict of fp32 tensors: dx, ddt (at the raw dt), dA, dB, dC and,
    when asked for, ddt_bias, dD, dinit.  ``out`` may hold preallocated
    tensors under those names."""
    b, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    dev = x.device
    shapes = dict(dx=(b, L, H, P), ddt=(b, L, H), dA=(H,), dB=(b, L, G, N), dC=(b, L, G, N),
                  ddt_bias=(H,) if want_dt_bias else None, dD=(H,) if want_D else None,
                  dinit=(b, H, P, N) if want_init else None)
    g = dict(out or {})
    with _on_stream(stream, x):
        for k, shp in shapes.items():
            if shp is not None and g.get(k) is None:
                g[k] = torch.empty(shp, dtype=torch.float32, device=dev)
            elif shp is None:
                g[k] = None
    with _on_device(x):
        st = _stream(stream, x)
        keep, d = _descs(x, dt, dt_bias, A, B, C, D, init_state, dout, dfinal_state,
                         g["dx"], g["ddt"], g["ddt_bias"], g["dA"], g["dB"], g["dC"], g["dD"], g["dinit"])
        status = lib().ssd_scan_bwd(*d, st)
    _check(status)
    return g


def ssd_scan_bwd_gated(x, dt, dt_bias, A, B, C, z, D, init_state, dout, dfinal_state=None, *,
                       want_dt_bias: bool = True, want_D: bool = True, want_init: bool = True,
                       out: dict = None, stream=None):
    """Gradients of ssd_scan_fwd_gated (out = y * silu(z)); the dict of
    ssd_scan_bwd plus dz (fp32)."""
    b, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    dev = x.device
    shapes = dict(dx=(b, L, H, P), ddt=(b, L, H), dA=(H,), dB=(b, L, G, N), dC=(b, L, G, N),
                  ddt_bias=(H,) if want_dt_bias else None, dD=(H,) if want_D else None,
                  dinit=(b, H, P, N) if want_init else None, dz=(b, L, H, P))
    g = dict(out or {})
    with _on_stream(stream, x):
        for k, shp in shapes.items():
            if shp is not None and g.get(k) is None:
                g[k] = torch.empty(shp, dtype=torch.float32, device=dev)
            elif shp is None:
                g[k] = None
    with _on_device(x):
        st = _stream(stream, x)
        keep, d = _descs(x, dt, dt_bias, A, B, C, D, z, init_state, dout, dfinal_state,
                         g["dx"], g["ddt"], g["ddt_bias"], g["dA"], g["dB"], g["dC"], g["dD"], g["dz"],
                         g["dinit"])
        status = lib().ssd_scan_bwd_gated(*d, st)
    _check(status)
    return g


def ssd_scan_fwd_gated(x, dt, dt_bias, A, B, C, z, D=None, init_state=None, out=None,
                       final_state=None, chunk: int = 256, stream=None,
                       algo: int = SSD_ALGO_AUTO, return_final_state: bool = True):
    """Forward scan with the output gate: out = y * silu(z); returns
    (out, final_state or None)."""
    with _on_stream(stream, x):
        if out is None:
            out = torch.empty_like(x)
        if final_state is None and return_final_state:
            final_state = torch.empty((x.shape[0], x.shape[2], x.shape[3], B.shape[3]),
                                      dtype=torch.float32, device=x.device)
    with _on_device(x):
        st = _stream(stream, x)
        keep, d = _descs(x, dt, dt_bias, A, B, C, D, z, init_state, out, final_state)
        status = lib().ssd_scan_fwd_gated(*d, int(chunk), int(algo), st)
    _check(status)
    return out, final_state


def ssd_scan_fwd_rows(x, dt, dt_bias, A, B, C, D=None, init_state=None, out=None,
                      final_state=None, waves: int = 0, stream=None,
                      return_final_state: bool = True):
    """Row-sliced walk with `waves` waves per workgroup (0 = automatic)."""
    with _on_stream(stream, x):
        if out is None:
            out = torch.empty_like(x)
        if final_state is None and return_final_state:
            final_state = torch.empty((x.shape[0], x.shape[2], x.shape[3], B.shape[3]),
                                      dtype=torch.float32, device=x.device)
    with _on_device(x):
        st = _stream(stream, x)
        keep, d = _descs(x, dt, dt_bias, A, B, C, D, init_state, out, final_state)
        status = lib().ssd_scan_fwd_rows(*d, int(waves), st)
    _check(status)
    return out, final_state


def ssd_selective_scan_fwd(x, dt, dt_bias, A, B, C, D=None, init_state=None, out=None,
                           final_state=None, segments: int = 0, stream=None,
                           return_final_state: bool = True):
    """Selective scan with a diagonal A [D, N] per (channel, state index);
    x, dt [b, L, D]; returns (out, final_state or None)."""
    with _on_stream(stream, x):
        if out is None:
            out = torch.empty_like(x)
        if final_state is None and return_final_state:
            final_state = torch.empty((x.shape[0], x.shape[2], B.shape[3]), dtype=torch.float32,
                                      device=x.device)
    with _on_device(x):
        st = _stream(stream, x)
        keep, d = _descs(x, dt, dt_bias, A, B, C, D, init_state, out, final_state)
        status = lib().ssd_selective_scan_fwd(*d, int(segments), st)
    _check(status)
    return out, final_state


def ssd_step(state, x, dt, A, B, C, D=None, out=None, stream=None):
    """One recurrent step; ``state`` is updated in place; returns out."""
    if out is None:
        with _on_stream(stream, x):
            out = torch.empty_like(x)
    with _on_device(state):
        st = _stream(stream, state)
        keep, d = _descs(state, x, dt, A, B, C, D, out)
        status = lib().ssd_step(*d, st)
    _check(status)
    return out


def _workspace(nbytes: int, t):
    """Workspace of one call from torch's allocator, on the stream the call
    runs on (so that the memory is handed out again only behind the call;
    under graph capture it belongs to the graph).  Called under _on_stream."""
    return torch.empty(nbytes, dtype=torch.uint8, device=t.device) if nbytes > 0 else None


@functools.lru_cache(maxsize=1024)
def ssd_glr_workspace(b: int, L: int, D: int, backward: bool = False) -> int:
    """Workspace bytes of ssd_glr_fwd or ssd_glr_bwd (-1: a shape they refuse)."""
    return int(lib().ssd_glr_workspace(int(b), int(L), int(D), int(backward)))


def _glr_workspace(x, backward):
    if x.dim() != 3:
        return None  # refused by the call
    return _workspace(ssd_glr_workspace(*x.shape, backward), x)


def ssd_glr_states(x):
    """An uninitialised ``states`` tensor for ssd_glr_fwd on this x [b, L, D]."""
    b, L, D = x.shape
    return torch.empty((b, (L + SSD_GLR_SEGMENT - 1) // SSD_GLR_SEGMENT, D), dtype=torch.float32,
                       device=x.device)


def ssd_glr_fwd(x, r, i, A, r_bias=None, i_bias=None, *, reset=None, lengths=None, init_state=None,
                out=None, final_state=None, states=None, stream=None, return_final_state: bool = True):
    """Gated linear recurrence over whole sequences, per channel

        h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t + i_bias) x_t,
        a_t = exp(A sigmoid(r_t + r_bias)),

    x, r, i [b, L, D] (views allowed), reset [b, L] uint8 or bool, lengths [b]
    int32; ``states`` (see ssd_glr_states) is filled for ssd_glr_bwd.  Returns
    (out, final_state or None); tokens behind a row's length are not written."""
    with _on_stream(stream, x):
        if out is None:
            out = torch.empty_like(x, memory_format=torch.contiguous_format)
        if final_state is None and return_final_state:
            final_state = torch.empty((x.shape[0], x.shape[-1]), dtype=torch.float32, device=x.device)
        ws = _glr_workspace(x, False)
    with _on_device(x):
        st = _stream(stream, x)
        keep, d = _descs(x, r, i, A, r_bias, i_bias, reset, lengths, init_state, out, final_state, states)
        status = lib().ssd_glr_fwd(*d, ws.data_ptr() if ws is not None else None,
                                   ws.numel() if ws is not None else 0, st)
    _check(status)
    return out, final_state


def ssd_glr_bwd(x, r, i, A, r_bias=None, i_bias=None, *, reset=None, lengths=None, init_state=None,
                dout, dfinal_state=None, states=None, want_bias: bool = True, want_init: bool = True,
                out: dict = None, stream=None):
    """Gradients of ssd_glr_fwd for <dout, out> + <dfinal_state, final state>.

    ``dout`` in the dtype of x or fp32 (what ssd_scan_bwd returns).  Returns a
    dict: dx, dr, di (dtype of x), dA and, when asked for, dr_bias, di_bias,
    dinit (fp32).  ``states`` as filled by ssd_glr_fwd saves a pass
    over the inputs.  ``out`` may hold preallocated tensors under those names."""
    g = dict(out or {})
    with _on_stream(stream, x):
        for k in ("dx", "dr", "di"):
            if g.get(k) is None:
                g[k] = torch.empty_like(x, memory_format=torch.contiguous_format)
        for k, want in (("dA", True), ("dr_bias", want_bias), ("di_bias", want_bias)):
            if not want:
                g[k] = None
            elif g.get(k) is None:
                g[k] = torch.empty_like(A)  # cheaper than torch.empty
        if not want_init:
            g["dinit"] = None
        elif g.get("dinit") is None:
            g["dinit"] = (torch.empty((x.shape[0], x.shape[-1]), dtype=torch.float32, device=x.device)
                          if init_state is None else torch.empty_like(init_state))
        ws = _glr_workspace(x, True)
    with _on_device(x):
        st = _stream(stream, x)
        keep, d = _descs(x, r, i, A, r_bias, i_bias, reset, lengths, init_state, states, dout, dfinal_state,
                         g["dx"], g["dr"], g["di"], g["dA"], g["dr_bias"], g["di_bias"], g["dinit"])
        status = lib().ssd_glr_bwd(*d, ws.data_ptr() if ws is not None else None,
                                   ws.numel() if ws is not None else 0, st)
    _check(status)
    return g


def ssd_glr_step(state, x, r, i, A, r_bias=None, i_bias=None, *, reset=None, out=None, new_state=None,
                 stream=None):
    """One token of the gated linear recurrence for every row: state [b, D] is
    updated in place (or written to ``new_state``); returns out [b, D]."""
    if out is None:
        with _on_stream(stream, x):
            out = torch.empty_like(x, memory_format=torch.contiguous_format)
    with _on_device(state):
        st = _stream(stream, state)
        keep, d = _descs(state, x, r, i, A, r_bias, i_bias, reset,
                         state if new_state is None else new_state, out)
        status = lib().ssd_glr_step(*d, st)
    _check(status)
    return out


@functools.lru_cache(maxsize=64)
def ssd_norm_rotate_workspace(N: int) -> int:
    """Workspace bytes of ssd_norm_rotate_bwd (-1: an N it refuses)."""
    return int(lib().ssd_norm_rotate_workspace(int(N)))


def ssd_norm_rotate_fwd(q, k, q_weight=None, k_weight=None, freqs=None, positions=None, *,
                        eps: float = 1e-6, interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """Norm of queries q [b, L, Hq, N] and keys k [b, L, Hk, N] (C and B of the
    scan) for each head, then the rotation of their first 2 * len(freqs)
    elements by position * freqs; positions [b, L] int32 or int64 (default
    0..L-1).  Returns (q_out, k_out)."""
    with _on_stream(stream, q):
        if q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        if k_out is None:
            k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
    with _on_device(q):
        st = _stream(stream, q)
        keep, d = _descs(q, k, q_weight, k_weight, freqs, positions, q_out, k_out)
        status = lib().ssd_norm_rotate_fwd(*d, float(eps), int(interleaved), st)
    _check(status)
    return q_out, k_out


def ssd_norm_rotate_bwd(q, k, q_weight, k_weight, freqs, positions, dq_out, dk_out, *,
                        eps: float = 1e-6, interleaved: bool = False, want_weights: bool = True,
                        out: dict = None, stream=None):
    """Gradients of ssd_norm_rotate_fwd for <dq_out, q_out> + <dk_out, k_out>
    (both in the dtype of q, or both fp32 as ssd_scan_bwd returns them): a dict of
    dq, dk (dtype of q) and, when asked for, dq_weight, dk_weight
    (fp32).  ``out`` may hold preallocated tensors under those names."""
    g = dict(out or {})
    with _on_stream(stream, q):
        for n, t in (("dq", q), ("dk", k)):
            if g.get(n) is None:
                g[n] = torch.empty_like(t, memory_format=torch.contiguous_format)
        for n, w in (("dq_weight", q_weight), ("dk_weight", k_weight)):
            if not want_weights:
                g[n] = None
            elif g.get(n) is None:
                g[n] = (torch.empty_like(w) if w is not None else
                        torch.empty((q.shape[-1],), dtype=torch.float32, device=q.device))
        ws = (None if g["dq_weight"] is None and g["dk_weight"] is None else
              _workspace(ssd_norm_rotate_workspace(q.shape[-1]), q))
    with _on_device(q):
        st = _stream(stream, q)
        keep, d = _descs(q, k, q_weight, k_weight, freqs, positions, dq_out, dk_out, g["dq"], g["dk"],
                         g["dq_weight"], g["dk_weight"])
        status = lib().ssd_norm_rotate_bwd(*d, float(eps), int(interleaved),
                                           ws.data_ptr() if ws is not None else None,
                                           ws.numel() if ws is not None else 0, st)
    _check(status)
    return g


def ssd_kv_append(k, v, k_cache, v_cache, page_table, start, *, q=None, freqs=None, tokens=None,
                  interleaved: bool = False, q_out=None, stream=None):
    """Keys and values k, v [b, L, Hk, N] of new tokens into the paged caches
    [pages, page_size, Hk, N], the keys turned by their positions start[i] + t
    on the way, and queries q [b, L, Hq, N] turned in the same pass (``freqs`` as
    for ssd_norm_rotate_fwd, None: not turned).  page_table [b, width], start [b]
    and tokens [b] are int32; row i has tokens[i] of the L tokens (None: all).
    Returns q_out (None without q); tokens behind a row's are not written, so a
    q_out of this call's own holds anything there."""
    if q is not None and q_out is None:
        with _on_stream(stream, k):
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    with _on_device(k):
        st = _stream(stream, k)
        keep, d = _descs(q, k, v, freqs, page_table, start, tokens, q_out, k_cache, v_cache)
        status = lib().ssd_kv_append(*d, int(interleaved), st)
    _check(status)
    return q_out


@functools.lru_cache(maxsize=1024)
def ssd_attn_workspace(b: int, L: int, Hq: int, Hk: int, N: int) -> int:
    """Workspace bytes of ssd_attn_fwd, with L = 1 of ssd_attn_step (-1: sizes
    they refuse)."""
    return int(lib().ssd_attn_workspace(int(b), int(L), int(Hq), int(Hk), int(N)))


def _attn_scale(q, scale):
    if scale is not None:
        return float(scale)
    N = q.shape[-1] if q.dim() else 0
    return N ** -0.5 if N else 1.0  # refused by the call


def _attn_workspace(q, k_cache):
    if q.dim() not in (3, 4) or k_cache is None or k_cache.dim() != 4:
        return None  # refused by the call
    b, L = (q.shape[0], 1) if q.dim() == 3 else q.shape[:2]
    return _workspace(ssd_attn_workspace(b, L, q.shape[-2], k_cache.shape[2], q.shape[-1]), q)


def ssd_attn_fwd(q, k_cache, v_cache, page_table, start, *, tokens=None, scale: float = None, window: int = 0,
                 out=None, lse=None, return_lse: bool = True, stream=None):
    """Attention of the new tokens q [b, L, Hq, N], at positions start[i] + t, over
    the paged caches, which hold them already (see ssd_kv_append): each sees the
    keys up to its own position, with ``window`` the last ``window`` of them.
    tokens [b] int32: how many of the L tokens row i has (None: all).  scale: of the
    scores (default 1 / sqrt(N)).  Returns (out, lse or None), lse [b, L, Hq] the
    logarithm of the sum of e^score; tokens behind a row's are not written, so an
    out and lse of this call's own hold anything there."""
    with _on_stream(stream, q):
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        if lse is None and return_lse:
            lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
        ws = _attn_workspace(q, k_cache)
    with _on_device(q):
        st = _stream(stream, q)
        keep, d = _descs(q, k_cache, v_cache, page_table, start, tokens, out, lse)
        status = lib().ssd_attn_fwd(*d, _attn_scale(q, scale), int(window),
                                    ws.data_ptr() if ws is not None else None,
                                    ws.numel() if ws is not None else 0, st)
    _check(status)
    return out, lse


def ssd_attn_step(q, k_cache, v_cache, page_table, start, *, scale: float = None, window: int = 0, out=None,
                  lse=None, stream=None):
    """Attention of one new token for every row, q [b, Hq, N] at position
    start[i], over the paged caches (see ssd_attn_fwd); fills ``lse`` [b, Hq] if it is
    given; returns out."""
    with _on_stream(stream, q):
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        ws = _attn_workspace(q, k_cache)
    with _on_device(q):
        st = _stream(stream, q)
        keep, d = _descs(q, k_cache, v_cache, page_table, start, out, lse)
        status = lib().ssd_attn_step(*d, _attn_scale(q, scale), int(window),
                                     ws.data_ptr() if ws is not None else None,
                                     ws.numel() if ws is not None else 0, st)
    _check(status)
    return out


def ssd_scan_plan(b, L, H, P, G, N, dtype=torch.bfloat16, cus: int = 256):
    """(algo, seg_len) that SSD_ALGO_AUTO uses for this shape and input dtype."""
    algo, seg = ctypes.c_int(), ctypes.c_int()
    code = SSD_BF16 if dtype in (torch.bfloat16, SSD_BF16) else SSD_F32
    _check(lib().ssd_scan_plan(b, L, H, P, G, N, code, cus, ctypes.byref(algo), ctypes.byref(seg)))
    return algo.value, seg.value


def ssd_status_string(status: int) -> str:
    return lib().ssd_status_string(int(status)).decode()


def ssd_last_error() -> str:
    return lib().ssd_last_error().decode()


def ssd_version() -> int:
    return int(lib().ssd_version())


def ssd_release_scratch() -> None:
    """Frees the scratch buffers the library keeps between calls (waits for
    the queued work that uses them)."""
    _check(lib().ssd_release_scratch())
