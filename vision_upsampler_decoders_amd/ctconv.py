"""ctypes binding of libctconv (include/ctconv.h), plus torch-tensor helpers.

This module only marshals arguments: every step of the computation runs in
the HIP kernels of libctconv.so.  Importing it fails loudly when the library
has not been built; there is no CPU fallback.
"""

from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional, Sequence, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libctconv.so")

CTCONV_F32, CTCONV_BF16, CTCONV_F16 = 0, 1, 2
ROUTE_AUTO, ROUTE_POLYPHASE, ROUTE_GATHER = 0, 1, 2
# the two polyphase kernels, forced (cross-checks)
ROUTE_POLYPHASE_TILED, ROUTE_POLYPHASE_STREAM = 3, 4
STATUS = {0: "OK", 1: "ERR_NULL", 2: "ERR_SHAPE", 3: "ERR_PARAM", 4: "ERR_DTYPE",
          5: "ERR_ALIGN", 6: "ERR_HIP", 7: "ERR_WORKSPACE", 8: "ERR_SCRATCH"}

EXPORTED = (
    "ctconv_abi_version", "ctconv_status_string", "ctconv_output_shape", "ctconv_packed_bytes",
    "ctconv_prepack", "ctconv_forward", "ctconv_forward_route", "ctconv_forward_act",
    "ctconv_query_route", "ctconv_elu", "ctconv_stream_sizes", "ctconv_stream_step",
    "ctconv_stream_flush", "ctconv_istft_normalize", "ctconv_depthwise_forward",
    "ctconv_depthwise_forward_kernel", "ctconv_depthwise_query_kernel",
    "ctconv_workspace_bytes", "ctconv_forward_ws", "ctconv_forward_noalloc",
    "ctconv_scratch_bytes", "ctconv_clock_probe_bytes", "ctconv_clock_probe",
    "ctconv_cache_append", "ctconv_paged_attention_workspace_bytes", "ctconv_paged_attention",
    "ctconv_cache_evict", "ctconv_cross_attention_workspace_bytes", "ctconv_cross_attention",
    "ctconv_norm_residual", "ctconv_block_run",
)

DW_AUTO, DW_ROW, DW_ELEMENT = 0, 1, 2

ACT_NONE, ACT_ELU = 0, 1

NORM_NONE, NORM_RMS, NORM_LAYER = 0, 1, 2
GATE_NONE, GATE_LINEAR, GATE_SIGMOID, GATE_TANH = 0, 1, 2, 3


class CtconvError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS.get(status, status)} "
                         f"({_string(status) if _lib is not None else ''})")


_lib = None
_i64p = ctypes.POINTER(ctypes.c_int64)


def load(path: str = LIB_PATH):
    """Load libctconv.so and declare its prototypes."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with "
                          "`python -m vision_upsampler_decoders_amd.build`")
    lib = ctypes.CDLL(path)
    c_int, c_i64, c_vp = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p
    lib.ctconv_abi_version.argtypes = []
    lib.ctconv_abi_version.restype = c_int
    lib.ctconv_status_string.argtypes = [c_int]
    lib.ctconv_status_string.restype = ctypes.c_char_p
    lib.ctconv_output_shape.argtypes = [c_int] + [_i64p] * 7
    lib.ctconv_output_shape.restype = c_int
    lib.ctconv_packed_bytes.argtypes = [c_int, c_i64, c_i64, _i64p, _i64p, c_int,
                                        ctypes.POINTER(ctypes.c_size_t)]
    lib.ctconv_packed_bytes.restype = c_int
    lib.ctconv_prepack.argtypes = [c_vp, c_vp, c_int, c_i64, c_i64, _i64p, _i64p, c_int, c_vp]
    lib.ctconv_prepack.restype = c_int
    fwd = [c_vp, c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_int] + [_i64p] * 6 + [c_int]
    lib.ctconv_forward.argtypes = fwd + [c_vp]
    lib.ctconv_forward.restype = c_int
    lib.ctconv_forward_route.argtypes = fwd + [c_int, c_vp]
    lib.ctconv_forward_route.restype = c_int
    lib.ctconv_forward_act.argtypes = fwd + [c_int, c_int, c_vp]
    lib.ctconv_forward_act.restype = c_int
    lib.ctconv_query_route.argtypes = [c_i64, c_i64, c_i64, c_int] + [_i64p] * 6 + [
        c_int, ctypes.POINTER(c_int)]
    lib.ctconv_query_route.restype = c_int
    lib.ctconv_workspace_bytes.argtypes = [c_i64, c_i64, c_i64, c_int] + [_i64p] * 6 + [
        c_int, ctypes.POINTER(ctypes.c_size_t)]
    lib.ctconv_workspace_bytes.restype = c_int
    lib.ctconv_forward_ws.argtypes = fwd + [c_int, c_vp, ctypes.c_size_t, c_vp]
    lib.ctconv_forward_ws.restype = c_int
    lib.ctconv_forward_noalloc.argtypes = fwd + [c_int, c_vp]
    lib.ctconv_forward_noalloc.restype = c_int
    lib.ctconv_scratch_bytes.argtypes = []
    lib.ctconv_scratch_bytes.restype = ctypes.c_size_t
    lib.ctconv_clock_probe_bytes.argtypes = []
    lib.ctconv_clock_probe_bytes.restype = ctypes.c_size_t
    lib.ctconv_clock_probe.argtypes = [c_vp, ctypes.c_size_t, c_int, ctypes.POINTER(ctypes.c_double),
                                       ctypes.POINTER(ctypes.c_double), c_vp]
    lib.ctconv_clock_probe.restype = c_int
    lib.ctconv_depthwise_forward.argtypes = fwd + [c_int, c_vp]
    lib.ctconv_depthwise_forward.restype = c_int
    lib.ctconv_depthwise_forward_kernel.argtypes = fwd + [c_int, c_int, c_vp]
    lib.ctconv_depthwise_forward_kernel.restype = c_int
    lib.ctconv_depthwise_query_kernel.argtypes = [c_i64, c_i64, c_i64, c_int] + [_i64p] * 6 + [
        c_int, ctypes.POINTER(c_int)]
    lib.ctconv_depthwise_query_kernel.restype = c_int
    lib.ctconv_elu.argtypes = [c_vp, c_vp, c_i64, c_int, c_vp]
    lib.ctconv_elu.restype = c_int
    lib.ctconv_stream_sizes.argtypes = [c_i64, c_i64, c_i64, c_i64, c_i64, c_int, _i64p, _i64p,
                                        _i64p]
    lib.ctconv_stream_sizes.restype = c_int
    lib.ctconv_stream_step.argtypes = [c_vp] * 7 + [c_i64] * 6 + [c_int, c_int, c_vp]
    lib.ctconv_stream_step.restype = c_int
    lib.ctconv_stream_flush.argtypes = [c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_i64, c_int,
                                        c_int, c_vp]
    lib.ctconv_stream_flush.restype = c_int
    lib.ctconv_istft_normalize.argtypes = [c_vp, c_vp, c_vp, c_i64, c_i64, c_i64, c_i64, c_int,
                                           c_vp]
    lib.ctconv_istft_normalize.restype = c_int
    c_sz, c_f = ctypes.c_size_t, ctypes.c_float
    lib.ctconv_cache_append.argtypes = [c_vp] * 10 + [c_i64] * 7 + [_i64p, _i64p, c_i64, _i64p,
                                                                    c_int, c_vp]
    lib.ctconv_cache_append.restype = c_int
    lib.ctconv_paged_attention_workspace_bytes.argtypes = [c_i64] * 6 + [
        c_int, c_int, ctypes.POINTER(c_sz)]
    lib.ctconv_paged_attention_workspace_bytes.restype = c_int
    lib.ctconv_paged_attention.argtypes = [c_vp] * 8 + [c_i64] * 9 + [
        _i64p, _i64p, _i64p, c_i64, _i64p, c_f, c_int, c_vp, c_sz, c_vp]
    lib.ctconv_paged_attention.restype = c_int
    lib.ctconv_cache_evict.argtypes = [c_vp] * 11 + [c_i64] * 10 + [_i64p, c_i64, _i64p, _i64p,
                                                                    c_int, c_vp]
    lib.ctconv_cache_evict.restype = c_int
    lib.ctconv_cross_attention_workspace_bytes.argtypes = [c_i64] * 6 + [c_int,
                                                                         ctypes.POINTER(c_sz)]
    lib.ctconv_cross_attention_workspace_bytes.restype = c_int
    lib.ctconv_cross_attention.argtypes = [c_vp] * 7 + [c_i64] * 6 + [_i64p] * 4 + [
        c_i64, c_f, c_int, c_vp, c_sz, c_vp]
    lib.ctconv_cross_attention.restype = c_int
    lib.ctconv_norm_residual.argtypes = [c_vp] * 10 + [c_i64, c_i64, _i64p, c_i64, c_int, c_int,
                                                       c_int, c_f, c_int, c_vp]
    lib.ctconv_norm_residual.restype = c_int
    lib.ctconv_block_run.argtypes = [c_int, c_vp, c_vp, c_vp, c_sz, c_vp]
    lib.ctconv_block_run.restype = c_int
    _lib = lib
    return lib


def _string(status: int) -> str:
    return _lib.ctconv_status_string(status).decode()


def _arr(v: Sequence[int]):
    return (ctypes.c_int64 * len(v))(*[int(t) for t in v])


def per_dim(v, ndim: int) -> Tuple[int, ...]:
    """Broadcast a scalar to every spatial dimension (as parse_hw does for 2-D)."""
    if isinstance(v, int):
        return (v,) * ndim
    v = tuple(int(t) for t in v)
    if len(v) != ndim:
        raise ValueError(f"expected {ndim} values, got {v}")
    return v


def _check(fn: str, st: int):
    if st != 0:
        raise CtconvError(fn, st)


# ---------------------------------------------------------------------------
# Raw C-ABI calls with the same names (pointers and sizes only)
# ---------------------------------------------------------------------------


def ctconv_abi_version() -> int:
    return load().ctconv_abi_version()


def ctconv_status_string(status: int) -> str:
    load()
    return _string(status)


def ctconv_output_shape(in_spatial, kernel, stride, padding=0, output_padding=0, dilation=1):
    ndim = len(in_spatial)
    out = (ctypes.c_int64 * ndim)()
    st = load().ctconv_output_shape(ndim, _arr(in_spatial), _arr(per_dim(kernel, ndim)),
                                    _arr(per_dim(stride, ndim)), _arr(per_dim(padding, ndim)),
                                    _arr(per_dim(output_padding, ndim)),
                                    _arr(per_dim(dilation, ndim)), out)
    _check("ctconv_output_shape", st)
    return tuple(int(v) for v in out)


def ctconv_packed_bytes(ndim: int, C_in: int, C_out: int, kernel, stride, dtype: int) -> int:
    nb = ctypes.c_size_t(0)
    st = load().ctconv_packed_bytes(ndim, C_in, C_out, _arr(per_dim(kernel, ndim)),
                                    _arr(per_dim(stride, ndim)), dtype, ctypes.byref(nb))
    _check("ctconv_packed_bytes", st)
    return int(nb.value)


def ctconv_prepack(w_ptr: int, packed_ptr: int, ndim: int, C_in: int, C_out: int, kernel,
                   stride, dtype: int, stream: int) -> None:
    st = load().ctconv_prepack(w_ptr, packed_ptr, ndim, C_in, C_out,
                               _arr(per_dim(kernel, ndim)), _arr(per_dim(stride, ndim)), dtype,
                               stream)
    _check("ctconv_prepack", st)


def ctconv_forward_route(x_ptr: int, packed_ptr: int, bias_ptr: Optional[int], y_ptr: int, N: int,
                         C_in: int, C_out: int, in_spatial, kernel, stride, padding,
                         output_padding, dilation, dtype: int, route: int, stream: int) -> None:
    ndim = len(in_spatial)
    st = load().ctconv_forward_route(
        x_ptr, packed_ptr, bias_ptr, y_ptr, N, C_in, C_out, ndim, _arr(in_spatial),
        _arr(per_dim(kernel, ndim)), _arr(per_dim(stride, ndim)), _arr(per_dim(padding, ndim)),
        _arr(per_dim(output_padding, ndim)), _arr(per_dim(dilation, ndim)), dtype, route, stream)
    _check("ctconv_forward_route", st)


def ctconv_forward_act(x_ptr: int, packed_ptr: int, bias_ptr: Optional[int], y_ptr: int, N: int,
                       C_in: int, C_out: int, in_spatial, kernel, stride, padding,
                       output_padding, dilation, dtype: int, act: int, route: int,
                       stream: int) -> None:
    ndim = len(in_spatial)
    st = load().ctconv_forward_act(
        x_ptr, packed_ptr, bias_ptr, y_ptr, N, C_in, C_out, ndim, _arr(in_spatial),
        _arr(per_dim(kernel, ndim)), _arr(per_dim(stride, ndim)), _arr(per_dim(padding, ndim)),
        _arr(per_dim(output_padding, ndim)), _arr(per_dim(dilation, ndim)), dtype, act, route,
        stream)
    _check("ctconv_forward_act", st)


def ctconv_forward(x_ptr: int, packed_ptr: int, bias_ptr: Optional[int], y_ptr: int, N: int,
                   C_in: int, C_out: int, in_spatial, kernel, stride, padding, output_padding,
                   dilation, dtype: int, stream: int) -> None:
    ndim = len(in_spatial)
    st = load().ctconv_forward(
        x_ptr, packed_ptr, bias_ptr, y_ptr, N, C_in, C_out, ndim, _arr(in_spatial),
        _arr(per_dim(kernel, ndim)), _arr(per_dim(stride, ndim)), _arr(per_dim(padding, ndim)),
        _arr(per_dim(output_padding, ndim)), _arr(per_dim(dilation, ndim)), dtype, stream)
    _check("ctconv_forward", st)


def ctconv_workspace_bytes(N: int, C_in: int, C_out: int, in_spatial, kernel, stride, padding=0,
                           output_padding=0, dilation=1, dtype: int = CTCONV_F32) -> int:
    ndim = len(in_spatial)
    nb = ctypes.c_size_t(0)
    st = load().ctconv_workspace_bytes(
        N, C_in, C_out, ndim, _arr(in_spatial), _arr(per_dim(kernel, ndim)),
        _arr(per_dim(stride, ndim)), _arr(per_dim(padding, ndim)),
        _arr(per_dim(output_padding, ndim)), _arr(per_dim(dilation, ndim)), dtype,
        ctypes.byref(nb))
    _check("ctconv_workspace_bytes", st)
    return int(nb.value)


def ctconv_forward_ws(x_ptr: int, packed_ptr: int, bias_ptr: Optional[int], y_ptr: int, N: int,
                      C_in: int, C_out: int, in_spatial, kernel, stride, padding, output_padding,
                      dilation, dtype: int, act: int, ws_ptr: Optional[int], ws_bytes: int,
                      stream: int) -> None:
    ndim = len(in_spatial)
    st = load().ctconv_forward_ws(
        x_ptr, packed_ptr, bias_ptr, y_ptr, N, C_in, C_out, ndim, _arr(in_spatial),
        _arr(per_dim(kernel, ndim)), _arr(per_dim(stride, ndim)), _arr(per_dim(padding, ndim)),
        _arr(per_dim(output_padding, ndim)), _arr(per_dim(dilation, ndim)), dtype, act, ws_ptr,
        ws_bytes, stream)
    _check("ctconv_forward_ws", st)


def ctconv_forward_noalloc(x_ptr: int, packed_ptr: int, bias_ptr: Optional[int], y_ptr: int,
                           N: int, C_in: int, C_out: int, in_spatial, kernel, stride, padding,
                           output_padding, dilation, dtype: int, act: int, stream: int) -> None:
    ndim = len(in_spatial)
    st = load().ctconv_forward_noalloc(
        x_ptr, packed_ptr, bias_ptr, y_ptr, N, C_in, C_out, ndim, _arr(in_spatial),
        _arr(per_dim(kernel, ndim)), _arr(per_dim(stride, ndim)), _arr(per_dim(padding, ndim)),
        _arr(per_dim(output_padding, ndim)), _arr(per_dim(dilation, ndim)), dtype, act, stream)
    _check("ctconv_forward_noalloc", st)


def ctconv_scratch_bytes() -> int:
    return int(load().ctconv_scratch_bytes())


def ctconv_clock_probe_bytes() -> int:
    return int(load().ctconv_clock_probe_bytes())


def ctconv_clock_probe(ws_ptr: int, ws_bytes: int, iters: int, stream: int):
    """(sustained shader clock in MHz, the probe's bf16 MFMA TFLOP/s); synchronous."""
    mhz, tf = ctypes.c_double(), ctypes.c_double()
    st = load().ctconv_clock_probe(ws_ptr, ws_bytes, iters, ctypes.byref(mhz), ctypes.byref(tf),
                                   stream)
    _check("ctconv_clock_probe", st)
    return mhz.value, tf.value


def ctconv_query_route(N: int, C_in: int, C_out: int, in_spatial, kernel, stride, padding=0,
                       output_padding=0, dilation=1, dtype: int = CTCONV_F32) -> int:
    ndim = len(in_spatial)
    r = ctypes.c_int(-1)
    st = load().ctconv_query_route(
        N, C_in, C_out, ndim, _arr(in_spatial), _arr(per_dim(kernel, ndim)),
        _arr(per_dim(stride, ndim)), _arr(per_dim(padding, ndim)),
        _arr(per_dim(output_padding, ndim)), _arr(per_dim(dilation, ndim)), dtype,
        ctypes.byref(r))
    _check("ctconv_query_route", st)
    return r.value


def ctconv_depthwise_forward_kernel(x_ptr: int, w_ptr: int, bias_ptr: Optional[int], y_ptr: int,
                                    N: int, C_in: int, C_out: int, in_spatial, kernel, stride,
                                    padding, output_padding, dilation, dtype: int, act: int,
                                    which: int, stream: int) -> None:
    ndim = len(in_spatial)
    st = load().ctconv_depthwise_forward_kernel(
        x_ptr, w_ptr, bias_ptr, y_ptr, N, C_in, C_out, ndim, _arr(in_spatial),
        _arr(per_dim(kernel, ndim)), _arr(per_dim(stride, ndim)), _arr(per_dim(padding, ndim)),
        _arr(per_dim(output_padding, ndim)), _arr(per_dim(dilation, ndim)), dtype, act, which,
        stream)
    _check("ctconv_depthwise_forward_kernel", st)


def ctconv_depthwise_forward(x_ptr: int, w_ptr: int, bias_ptr: Optional[int], y_ptr: int, N: int,
                             C_in: int, C_out: int, in_spatial, kernel, stride, padding,
                             output_padding, dilation, dtype: int, act: int,
                             stream: int) -> None:
    ndim = len(in_spatial)
    st = load().ctconv_depthwise_forward(
        x_ptr, w_ptr, bias_ptr, y_ptr, N, C_in, C_out, ndim, _arr(in_spatial),
        _arr(per_dim(kernel, ndim)), _arr(per_dim(stride, ndim)), _arr(per_dim(padding, ndim)),
        _arr(per_dim(output_padding, ndim)), _arr(per_dim(dilation, ndim)), dtype, act, stream)
    _check("ctconv_depthwise_forward", st)


def ctconv_depthwise_query_kernel(N: int, C_in: int, C_out: int, in_spatial, kernel, stride,
                                  padding=0, output_padding=0, dilation=1,
                                  dtype: int = CTCONV_F32) -> int:
    ndim = len(in_spatial)
    r = ctypes.c_int(-1)
    st = load().ctconv_depthwise_query_kernel(
        N, C_in, C_out, ndim, _arr(in_spatial), _arr(per_dim(kernel, ndim)),
        _arr(per_dim(stride, ndim)), _arr(per_dim(padding, ndim)),
        _arr(per_dim(output_padding, ndim)), _arr(per_dim(dilation, ndim)), dtype,
        ctypes.byref(r))
    _check("ctconv_depthwise_query_kernel", st)
    return r.value


def ctconv_elu(x_ptr: int, y_ptr: int, n: int, dtype: int, stream: int) -> None:
    _check("ctconv_elu", load().ctconv_elu(x_ptr, y_ptr, n, dtype, stream))


def ctconv_stream_sizes(N: int, C_out: int, L_chunk: int, kernel: int, stride: int,
                        dtype: int) -> Tuple[int, int, int]:
    a, b, c = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    _check("ctconv_stream_sizes",
           load().ctconv_stream_sizes(N, C_out, L_chunk, kernel, stride, dtype, ctypes.byref(a),
                                      ctypes.byref(b), ctypes.byref(c)))
    return a.value, b.value, c.value


def ctconv_stream_step(x_ptr: int, packed_ptr: int, bias_ptr: Optional[int], y_ptr: int,
                       tail_in_ptr: Optional[int], tail_out_ptr: Optional[int], ws_ptr: int, N: int,
                       C_in: int, C_out: int, L_chunk: int, kernel: int, stride: int, dtype: int,
                       act: int, stream: int) -> None:
    _check("ctconv_stream_step",
           load().ctconv_stream_step(x_ptr, packed_ptr, bias_ptr, y_ptr, tail_in_ptr,
                                     tail_out_ptr, ws_ptr, N, C_in, C_out, L_chunk, kernel,
                                     stride, dtype, act, stream))


def ctconv_stream_flush(tail_in_ptr: Optional[int], bias_ptr: Optional[int], y_ptr: int, N: int,
                        C_out: int, kernel: int, stride: int, dtype: int, act: int,
                        stream: int) -> None:
    _check("ctconv_stream_flush",
           load().ctconv_stream_flush(tail_in_ptr, bias_ptr, y_ptr, N, C_out, kernel, stride,
                                      dtype, act, stream))


def ctconv_istft_normalize(y_ptr: int, env_ptr: int, out_ptr: int, rows: int, L_in: int,
                           trim: int, L_out: int, dtype: int, stream: int) -> None:
    _check("ctconv_istft_normalize",
           load().ctconv_istft_normalize(y_ptr, env_ptr, out_ptr, rows, L_in, trim, L_out, dtype,
                                         stream))


# ---------------------------------------------------------------------------
# torch helpers (device memory and streams only)
# ---------------------------------------------------------------------------


def _torch():
    import torch

    return torch


def dtype_code(t) -> int:
    torch = _torch()
    m = {torch.float32: CTCONV_F32, torch.bfloat16: CTCONV_BF16, torch.float16: CTCONV_F16}
    if t.dtype not in m:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return m[t.dtype]


def dtype_code_of(name: str) -> int:
    """"f32" / "bf16" / "f16" -> the ctconv_dtype code."""
    return {"f32": CTCONV_F32, "bf16": CTCONV_BF16, "f16": CTCONV_F16}[name]


def _stream(stream=None) -> int:
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _side_stream(stream, device):
    """The explicit stream when it differs from the current one (else None).
    Inputs made ready on the current stream (copies by .contiguous(), fresh
    allocations) must be visible to it, so it first waits for the current
    stream."""
    torch = _torch()
    if stream is None:
        return None
    cur = torch.cuda.current_stream(device)
    if int(stream.cuda_stream) == int(cur.cuda_stream):
        return None
    stream.wait_stream(cur)
    return stream


def _claim(side, *tensors):
    """Tell the caching allocator that these tensors are used on `side`, so
    their memory is not reused before the work queued there is done."""
    if side is None:
        return
    for t in tensors:
        if t is not None:
            t.record_stream(side)


def _check_tensor(name, t, dtype, device, shape=None, numel=None):
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")


def sustained_clock(iters: int = 4096, device=None, stream=None):
    """(MHz, TFLOP/s) of ctconv_clock_probe on `device` (a workspace is allocated here)."""
    torch = _torch()
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    nb = ctconv_clock_probe_bytes()
    ws = torch.empty(max(nb, 8), dtype=torch.uint8, device=dev)
    return ctconv_clock_probe(ws.data_ptr(), ws.numel(), iters, _stream(stream))


def prepack(w, stride, stream=None):
    """Packed phase-major copy of a ConvTranspose weight w [C_in, C_out, k...] (device)."""
    torch = _torch()
    if not w.is_cuda:
        raise ValueError("w must be a device tensor")
    w = w.contiguous()
    ndim = w.dim() - 2
    C_in, C_out = w.shape[0], w.shape[1]
    k = tuple(w.shape[2:])
    dt = dtype_code(w)
    nb = ctconv_packed_bytes(ndim, C_in, C_out, k, stride, dt)
    packed = torch.empty(nb // w.element_size(), dtype=w.dtype, device=w.device)
    side = _side_stream(stream, w.device)
    ctconv_prepack(w.data_ptr(), packed.data_ptr(), ndim, C_in, C_out, k, stride, dt,
                   _stream(stream))
    _claim(side, w, packed)
    return packed


def forward(x, packed, bias, C_out: int, kernel, stride, padding=0, output_padding=0,
            dilation=1, route: int = ROUTE_AUTO, out=None, stream=None, act: int = ACT_NONE,
            workspace=None):
    """y = act(ConvTranspose(x, w, bias)) with w given by its packed form (device tensors).

    packed must be the ctconv_prepack output for this C_in, C_out, kernel,
    stride and dtype: its byte size is checked against ctconv_packed_bytes.
    bias (or None) is [C_out] of x's dtype; out (or None) is the contiguous
    [N, C_out, out_spatial...] tensor of x's dtype to write.  workspace: None
    (ctconv_forward_act), True (ctconv_forward_ws with a workspace allocated
    here) or a device tensor of at least ctconv_workspace_bytes bytes
    (ctconv_forward_ws; route must be ROUTE_AUTO)."""
    torch = _torch()
    if not x.is_cuda:
        raise ValueError("x must be a device tensor")
    x = x.contiguous()
    ndim = x.dim() - 2
    if ndim not in (1, 2):
        raise ValueError("x must be [N, C_in, L] or [N, C_in, H, W]")
    N, C_in = x.shape[0], x.shape[1]
    sp = tuple(x.shape[2:])
    dt = dtype_code(x)
    kernel = per_dim(kernel, ndim)
    nb = ctconv_packed_bytes(ndim, C_in, C_out, kernel, stride, dt)
    _check_tensor("packed", packed, x.dtype, x.device)
    if not packed.is_contiguous() or packed.numel() * packed.element_size() != nb:
        raise ValueError(f"packed holds {packed.numel() * packed.element_size()} bytes; "
                         f"ctconv_packed_bytes gives {nb} for this weight shape, stride and "
                         f"dtype")
    osp = ctconv_output_shape(sp, kernel, stride, padding, output_padding, dilation)
    if bias is not None:
        _check_tensor("bias", bias, x.dtype, x.device, numel=C_out)
        bias = bias.contiguous()
    if out is not None:
        _check_tensor("out", out, x.dtype, x.device, shape=(N, C_out) + osp)
        if not out.is_contiguous():
            raise ValueError("out must be contiguous")
        y = out
    else:
        y = torch.empty((N, C_out) + osp, dtype=x.dtype, device=x.device)
    ws = None
    if workspace is not None:
        if route != ROUTE_AUTO:
            raise ValueError("a workspace call takes the automatic route")
        need = ctconv_workspace_bytes(N, C_in, C_out, sp, kernel, stride, padding,
                                      output_padding, dilation, dt)
        if workspace is True:
            ws = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
        else:
            ws = workspace
            if not ws.is_cuda or ws.device != x.device or not ws.is_contiguous():
                raise ValueError("workspace must be a contiguous tensor on x's device")
            if ws.numel() * ws.element_size() < need:
                raise ValueError(f"workspace holds {ws.numel() * ws.element_size()} bytes; "
                                 f"ctconv_workspace_bytes gives {need}")
    side = _side_stream(stream, x.device)
    bptr = None if bias is None else bias.data_ptr()
    if ws is None:
        ctconv_forward_act(x.data_ptr(), packed.data_ptr(), bptr, y.data_ptr(), N, C_in, C_out,
                           sp, kernel, stride, padding, output_padding, dilation, dt, act,
                           route, _stream(stream))
    else:
        ctconv_forward_ws(x.data_ptr(), packed.data_ptr(), bptr, y.data_ptr(), N, C_in, C_out, sp,
                          kernel, stride, padding, output_padding, dilation, dt, act,
                          ws.data_ptr(), ws.numel() * ws.element_size(), _stream(stream))
    _claim(side, x, packed, bias, y, ws)
    return y


def depthwise_forward(x, w, bias, stride, padding=0, output_padding=0, dilation=1,
                      act: int = ACT_NONE, which: int = DW_AUTO, out=None, stream=None):
    """y = act(ConvTranspose(x, w, bias, groups=C_in)) for w [C_in, M, k...] (device tensors)."""
    torch = _torch()
    if not x.is_cuda or not w.is_cuda:
        raise ValueError("x and w must be device tensors")
    x = x.contiguous()
    w = w.contiguous()
    ndim = x.dim() - 2
    if ndim not in (1, 2):
        raise ValueError("x must be [N, C_in, L] or [N, C_in, H, W]")
    N, C_in = x.shape[0], x.shape[1]
    if w.shape[0] != C_in or w.dim() != ndim + 2:
        raise ValueError("w must be [C_in, M, k...]")
    _check_tensor("w", w, x.dtype, x.device)
    C_out = C_in * w.shape[1]
    kernel = tuple(w.shape[2:])
    sp = tuple(x.shape[2:])
    osp = ctconv_output_shape(sp, kernel, stride, padding, output_padding, dilation)
    if bias is not None:
        _check_tensor("bias", bias, x.dtype, x.device, numel=C_out)
        bias = bias.contiguous()
    if out is not None:
        _check_tensor("out", out, x.dtype, x.device, shape=(N, C_out) + osp)
        if not out.is_contiguous():
            raise ValueError("out must be contiguous")
        y = out
    else:
        y = torch.empty((N, C_out) + osp, dtype=x.dtype, device=x.device)
    side = _side_stream(stream, x.device)
    bptr = None if bias is None else bias.data_ptr()
    ctconv_depthwise_forward_kernel(x.data_ptr(), w.data_ptr(), bptr, y.data_ptr(), N, C_in,
                                    C_out, sp, kernel, stride, padding, output_padding, dilation,
                                    dtype_code(x), act, which, _stream(stream))
    _claim(side, x, w, bias, y)
    return y


def elu(x, out=None, stream=None):
    torch = _torch()
    if not x.is_cuda:
        raise ValueError("x must be a device tensor")
    x = x.contiguous()
    if out is not None:
        _check_tensor("out", out, x.dtype, x.device, shape=tuple(x.shape))
        if not out.is_contiguous():
            raise ValueError("out must be contiguous")
        y = out
    else:
        y = torch.empty_like(x)
    side = _side_stream(stream, x.device)
    ctconv_elu(x.data_ptr(), y.data_ptr(), x.numel(), dtype_code(x), _stream(stream))
    _claim(side, x, y)
    return y


class Conv:
    """A transposed convolution with its arguments marshalled once.

    Holds the C arrays of one shape so that each call is a single foreign
    function call (no per-call Python-side shape work).  Buffers are passed as
    device tensors or raw pointers at call time.
    """

    def __init__(self, N: int, C_in: int, C_out: int, in_spatial, kernel, stride, padding=0,
                 output_padding=0, dilation=1, dtype: int = CTCONV_F32,
                 route: int = ROUTE_AUTO, act: int = ACT_NONE):
        nd = len(in_spatial)
        self.ndim = nd
        self.N, self.C_in, self.C_out = int(N), int(C_in), int(C_out)
        self.in_spatial = tuple(int(v) for v in in_spatial)
        self.kernel = per_dim(kernel, nd)
        self.stride = per_dim(stride, nd)
        self.padding = per_dim(padding, nd)
        self.output_padding = per_dim(output_padding, nd)
        self.dilation = per_dim(dilation, nd)
        self.dtype = dtype
        self.route = route
        self.act = act
        self.out_spatial = ctconv_output_shape(self.in_spatial, self.kernel, self.stride,
                                               self.padding, self.output_padding, self.dilation)
        self._args = [_arr(self.in_spatial), _arr(self.kernel), _arr(self.stride),
                      _arr(self.padding), _arr(self.output_padding), _arr(self.dilation)]
        self._fn = load().ctconv_forward_act

    def out_shape(self):
        return (self.N, self.C_out) + self.out_spatial

    def __call__(self, x_ptr: int, packed_ptr: int, bias_ptr, y_ptr: int, stream: int) -> None:
        st = self._fn(x_ptr, packed_ptr, bias_ptr, y_ptr, self.N, self.C_in, self.C_out,
                      self.ndim, *self._args, self.dtype, self.act, self.route, stream)
        if st != 0:
            raise CtconvError("ctconv_forward_act", st)


class DepthwiseConv(Conv):
    """A depthwise transposed convolution (groups = C_in) with its arguments
    marshalled once; called with the unpacked weight [C_in, C_out / C_in, k...]."""

    def __init__(self, *args, which: int = DW_AUTO, **kw):
        kw.pop("route", None)
        super().__init__(*args, **kw)
        self.which = which
        self._fn = load().ctconv_depthwise_forward_kernel

    def __call__(self, x_ptr: int, w_ptr: int, bias_ptr, y_ptr: int, stream: int) -> None:
        st = self._fn(x_ptr, w_ptr, bias_ptr, y_ptr, self.N, self.C_in, self.C_out,
                      self.ndim, *self._args, self.dtype, self.act, self.which, stream)
        if st != 0:
            raise CtconvError("ctconv_depthwise_forward_kernel", st)


class ConvWS(Conv):
    """A transposed convolution through ctconv_forward_ws (deterministic split
    of the reduction when the shape calls for one), arguments marshalled once;
    called with the workspace pointer and its size in bytes."""

    def __init__(self, *args, **kw):
        kw.pop("route", None)
        super().__init__(*args, **kw)
        self._fn = load().ctconv_forward_ws
        self.ws_bytes = ctconv_workspace_bytes(self.N, self.C_in, self.C_out, self.in_spatial,
                                               self.kernel, self.stride, self.padding,
                                               self.output_padding, self.dilation, self.dtype)

    def __call__(self, x_ptr: int, packed_ptr: int, bias_ptr, y_ptr: int, stream: int,
                 ws_ptr=None, ws_bytes: int = 0) -> None:
        st = self._fn(x_ptr, packed_ptr, bias_ptr, y_ptr, self.N, self.C_in, self.C_out,
                      self.ndim, *self._args, self.dtype, self.act, ws_ptr, ws_bytes, stream)
        if st != 0:
            raise CtconvError("ctconv_forward_ws", st)


# ---------------------------------------------------------------------------
# The transformer block of a streaming decoder: plans (arguments marshalled
# once, called with raw pointers, like Conv) and torch helpers.
# ---------------------------------------------------------------------------


OP_CACHE_APPEND, OP_PAGED_ATTENTION, OP_CACHE_EVICT = 0, 1, 2
OP_CROSS_ATTENTION, OP_NORM_RESIDUAL = 3, 4


def _strides(given, default):
    return tuple(int(v) for v in (default if given is None else given))


class _Plan:
    """A prepared ctconv_block_run: the sizes in one array, the call's pointers
    packed into another (a fresh one per call, so that threads can share a
    plan).  Against the functions themselves, whose arguments ctypes converts
    one by one, this takes about 1 us off a call of 5."""

    def _prepare(self, name: str, op: int, buffers: int, sizes):
        flat = []
        for v in sizes:
            flat.extend(v if isinstance(v, tuple) else (v,))
        as_int = [struct.unpack("q", struct.pack("d", v))[0] if isinstance(v, float) else int(v)
                  for v in flat]
        self._name, self._op = name, op
        self._sizes = _arr(as_int)
        self._sizes_ptr = ctypes.c_void_p(ctypes.addressof(self._sizes))
        self._pack = struct.Struct(f"{buffers}P").pack
        self._fn = load().ctconv_block_run


def _scale(scale, D: int) -> float:
    return float(D) ** -0.5 if scale is None else float(scale)


class _Paged(_Plan):
    """Sizes and strides of a paged cache.  Without strides: pages of
    [Hkv, page_size, D], a dense table, dense [B, Hkv, slots] slot arrays."""

    def _cache(self, B, Hkv, D, num_pages, page_size, max_pages, kv_strides, table_stride,
               slot_strides):
        self.B, self.Hkv, self.D = int(B), int(Hkv), int(D)
        self.num_pages, self.page_size = int(num_pages), int(page_size)
        self.max_pages = int(max_pages)
        self.slots = self.page_size * self.max_pages
        self._kv = _strides(kv_strides, (self.Hkv * self.page_size * self.D, self.D,
                                         self.page_size * self.D))
        self._table = self.max_pages if table_stride is None else int(table_stride)
        self._slot = _strides(slot_strides, (self.Hkv * self.slots, self.slots))


class CacheAppend(_Paged):
    """ctconv_cache_append for one shape: n new rows [B, n, Hkv, D] per sequence at most."""

    def __init__(self, B: int, n: int, Hkv: int, D: int, num_pages: int, page_size: int,
                 max_pages: int, dtype: int = CTCONV_F32, new_strides=None, kv_strides=None,
                 table_stride=None, slot_strides=None):
        self._cache(B, Hkv, D, num_pages, page_size, max_pages, kv_strides, table_stride,
                    slot_strides)
        self.n, self.dtype = int(n), dtype
        new = _strides(new_strides, (self.n * self.Hkv * self.D, self.Hkv * self.D, self.D))
        self._prepare("ctconv_cache_append", OP_CACHE_APPEND, 10,
                      (self.B, self.n, self.Hkv, self.D, self.num_pages, self.page_size,
                       self.max_pages, new, self._kv, self._table, self._slot, dtype))

    def __call__(self, k_new_ptr, v_new_ptr, k_ptr, v_ptr, table_ptr, lengths_ptr, counts_ptr,
                 now_ptr, positions_ptr, weight_ptr, stream: int) -> None:
        st = self._fn(
            self._op, self._sizes_ptr,
            self._pack(k_new_ptr or 0, v_new_ptr or 0, k_ptr or 0, v_ptr or 0, table_ptr or 0,
                       lengths_ptr or 0, counts_ptr or 0, now_ptr or 0, positions_ptr or 0,
                       weight_ptr or 0),
            None, 0, stream)
        if st != 0:
            raise CtconvError(self._name, st)


def ctconv_paged_attention_workspace_bytes(B: int, Hq: int, Hkv: int, D: int, max_length: int,
                                           window: int, weights: bool, dtype: int) -> int:
    nb = ctypes.c_size_t(0)
    _check("ctconv_paged_attention_workspace_bytes",
           load().ctconv_paged_attention_workspace_bytes(B, Hq, Hkv, D, max_length, window,
                                                         int(bool(weights)), dtype,
                                                         ctypes.byref(nb)))
    return int(nb.value)


class PagedAttention(_Paged):
    """ctconv_paged_attention for one shape.  weights: whether calls pass a
    weight_sum (the workspace then holds the scores).  scale: D ** -0.5."""

    def __init__(self, B: int, Hq: int, Hkv: int, D: int, num_pages: int, page_size: int,
                 max_pages: int, max_length=None, window: int = 0, scale=None,
                 weights: bool = False, dtype: int = CTCONV_F32, q_strides=None,
                 kv_strides=None, out_strides=None, table_stride=None, slot_strides=None):
        self._cache(B, Hkv, D, num_pages, page_size, max_pages, kv_strides, table_stride,
                    slot_strides)
        self.Hq, self.window, self.dtype = int(Hq), int(window), dtype
        self.max_length = self.slots if max_length is None else int(max_length)
        self.weights = bool(weights)
        dense = (self.Hq * self.D, self.D)
        self.workspace_bytes = ctconv_paged_attention_workspace_bytes(
            self.B, self.Hq, self.Hkv, self.D, self.max_length, self.window, self.weights, dtype)
        self._prepare("ctconv_paged_attention", OP_PAGED_ATTENTION, 8,
                      (self.B, self.Hq, self.Hkv, self.D, self.num_pages, self.page_size,
                       self.max_pages, self.max_length, self.window, _strides(q_strides, dense),
                       self._kv, _strides(out_strides, dense), self._table, self._slot,
                       _scale(scale, self.D), dtype))

    def __call__(self, q_ptr, k_ptr, v_ptr, table_ptr, lengths_ptr, out_ptr, lse_ptr, weight_ptr,
                 ws_ptr, ws_bytes: int, stream: int) -> None:
        st = self._fn(
            self._op, self._sizes_ptr,
            self._pack(q_ptr or 0, k_ptr or 0, v_ptr or 0, table_ptr or 0, lengths_ptr or 0,
                       out_ptr or 0, lse_ptr or 0, weight_ptr or 0),
            ws_ptr, ws_bytes, stream)
        if st != 0:
            raise CtconvError(self._name, st)


class CacheEvict(_Paged):
    """ctconv_cache_evict for one shape.  Without out_slot_strides the results
    are dense [B, Hkv, keep]; in place, pass slot_strides for both."""

    def __init__(self, B: int, Hkv: int, D: int, num_pages: int, page_size: int, max_pages: int,
                 keep: int, max_length=None, sink: int = 0, recent: int = 0,
                 dtype: int = CTCONV_F32, kv_strides=None, table_stride=None, slot_strides=None,
                 out_slot_strides=None):
        self._cache(B, Hkv, D, num_pages, page_size, max_pages, kv_strides, table_stride,
                    slot_strides)
        self.keep, self.sink, self.recent, self.dtype = int(keep), int(sink), int(recent), dtype
        self.max_length = self.slots if max_length is None else int(max_length)
        out = _strides(out_slot_strides, (self.Hkv * self.keep, self.keep))
        self._prepare("ctconv_cache_evict", OP_CACHE_EVICT, 11,
                      (self.B, self.Hkv, self.D, self.num_pages, self.page_size, self.max_pages,
                       self.max_length, self.keep, self.sink, self.recent, self._kv, self._table,
                       self._slot, out, dtype))

    def __call__(self, k_ptr, v_ptr, table_ptr, lengths_ptr, now_ptr, weight_ptr, positions_ptr,
                 weight_out_ptr, positions_out_ptr, lengths_out_ptr, source_ptr,
                 stream: int) -> None:
        st = self._fn(
            self._op, self._sizes_ptr,
            self._pack(k_ptr or 0, v_ptr or 0, table_ptr or 0, lengths_ptr or 0, now_ptr or 0,
                       weight_ptr or 0, positions_ptr or 0, weight_out_ptr or 0,
                       positions_out_ptr or 0, lengths_out_ptr or 0, source_ptr or 0),
            None, 0, stream)
        if st != 0:
            raise CtconvError(self._name, st)


def ctconv_cross_attention_workspace_bytes(B: int, Lq: int, Lk: int, Hq: int, Hkv: int, D: int,
                                           dtype: int) -> int:
    nb = ctypes.c_size_t(0)
    _check("ctconv_cross_attention_workspace_bytes",
           load().ctconv_cross_attention_workspace_bytes(B, Lq, Lk, Hq, Hkv, D, dtype,
                                                         ctypes.byref(nb)))
    return int(nb.value)


class CrossAttention(_Plan):
    """ctconv_cross_attention for one shape; dense [B, L, H, D] tensors without strides."""

    def __init__(self, B: int, Lq: int, Lk: int, Hq: int, Hkv: int, D: int, scale=None,
                 dtype: int = CTCONV_F32, q_strides=None, k_strides=None, v_strides=None,
                 out_strides=None, mask_stride=None):
        self.B, self.Lq, self.Lk, self.Hq = int(B), int(Lq), int(Lk), int(Hq)
        self.Hkv, self.D, self.dtype = int(Hkv), int(D), dtype
        q = (self.Lq * self.Hq * self.D, self.Hq * self.D, self.D)
        k = (self.Lk * self.Hkv * self.D, self.Hkv * self.D, self.D)
        self.workspace_bytes = ctconv_cross_attention_workspace_bytes(
            self.B, self.Lq, self.Lk, self.Hq, self.Hkv, self.D, dtype)
        self._prepare("ctconv_cross_attention", OP_CROSS_ATTENTION, 7,
                      (self.B, self.Lq, self.Lk, self.Hq, self.Hkv, self.D,
                       _strides(q_strides, q), _strides(k_strides, k), _strides(v_strides, k),
                       _strides(out_strides, q),
                       self.Lk if mask_stride is None else int(mask_stride),
                       _scale(scale, self.D), dtype))

    def __call__(self, q_ptr, k_ptr, v_ptr, lengths_ptr, mask_ptr, out_ptr, lse_ptr, ws_ptr,
                 ws_bytes: int, stream: int) -> None:
        st = self._fn(
            self._op, self._sizes_ptr,
            self._pack(q_ptr or 0, k_ptr or 0, v_ptr or 0, lengths_ptr or 0, mask_ptr or 0,
                       out_ptr or 0, lse_ptr or 0),
            ws_ptr, ws_bytes, stream)
        if st != 0:
            raise CtconvError(self._name, st)


class NormResidual(_Plan):
    """ctconv_norm_residual for one shape; dense rows without strides
    (strides: of x, h, gate, x_out, y)."""

    def __init__(self, rows: int, C: int, post: int = NORM_NONE, pre: int = NORM_LAYER,
                 gate: int = GATE_NONE, rows_per_gate: int = 1, eps: float = 1e-5,
                 dtype: int = CTCONV_F32, strides=None):
        self.rows, self.C, self.dtype = int(rows), int(C), dtype
        self.post, self.pre, self.gate = post, pre, gate
        self._prepare("ctconv_norm_residual", OP_NORM_RESIDUAL, 10,
                      (self.rows, self.C, _strides(strides, (self.C,) * 5), int(rows_per_gate),
                       post, pre, gate, float(eps), dtype))

    def __call__(self, x_ptr, h_ptr, post_weight_ptr, post_bias_ptr, scale_ptr, gate_ptr,
                 pre_weight_ptr, pre_bias_ptr, x_out_ptr, y_ptr, stream: int) -> None:
        st = self._fn(
            self._op, self._sizes_ptr,
            self._pack(x_ptr or 0, h_ptr or 0, post_weight_ptr or 0, post_bias_ptr or 0,
                       scale_ptr or 0, gate_ptr or 0, pre_weight_ptr or 0, pre_bias_ptr or 0,
                       x_out_ptr or 0, y_ptr or 0),
            None, 0, stream)
        if st != 0:
            raise CtconvError(self._name, st)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _rows_ready(name, t, dtype, device, dims: int):
    """t with a contiguous last dimension, unchanged otherwise (its strides are passed on)."""
    _check_tensor(name, t, dtype, device)
    if t.dim() != dims:
        raise ValueError(f"{name} has {t.dim()} dimensions, expected {dims}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return t


def _required(name, t):
    if t is None:
        raise ValueError(f"{name} is required")


def _index(name, t, device, shape, dtype=None):
    """An int32 (or `dtype`) array of `shape` whose last dimension is contiguous, or None."""
    if t is None:
        return None
    torch = _torch()
    _check_tensor(name, t, torch.int32 if dtype is None else dtype, device, shape=shape)
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return t


def _cache_tensors(k_cache, v_cache, page_table, dtype, device):
    """(num_pages, page_size, max_pages, Hkv, D, kv_strides) of a cache held as two
    [num_pages, Hkv, page_size, D] tensors of the same strides."""
    torch = _torch()
    _rows_ready("k_cache", k_cache, dtype, device, 4)
    _rows_ready("v_cache", v_cache, dtype, device, 4)
    if k_cache.shape != v_cache.shape or k_cache.stride() != v_cache.stride():
        raise ValueError("k_cache and v_cache must have the same shape and strides")
    _rows_ready("page_table", page_table, torch.int32, device, 2)
    num_pages, Hkv, page_size, D = k_cache.shape
    st = k_cache.stride()
    return num_pages, page_size, page_table.shape[1], Hkv, D, (st[0], st[2], st[1])


def _slot_arrays(arrays, B, Hkv, slots, device):
    """Strides shared by the given [B, Hkv, slots] arrays (name, tensor, dtype)."""
    strides = None
    for name, t, dtype in arrays:
        if t is None:
            continue
        _index(name, t, device, (B, Hkv, slots), dtype)
        if strides is not None and t.stride()[:2] != strides:
            raise ValueError(f"{name} must have the strides of the other slot arrays")
        strides = t.stride()[:2]
    return strides


def _workspace(workspace, need: int, device):
    torch = _torch()
    if need == 0:
        return None
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if not workspace.is_cuda or workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    if workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace holds {workspace.numel() * workspace.element_size()} bytes; "
                         f"the call needs {need}")
    return workspace


def _result(out, shape, dtype, device, name="out"):
    torch = _torch()
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _check_tensor(name, out, dtype, device, shape=shape)
    return _rows_ready(name, out, dtype, device, len(shape))


def cache_append(k_new, v_new, k_cache, v_cache, page_table, lengths, counts=None, now=None,
                 positions=None, weight_sum=None, stream=None) -> None:
    """Append k_new, v_new [B, n, Hkv, D] to the cache (see ctconv_cache_append).

    k_cache, v_cache [num_pages, Hkv, page_size, D] (any strides with a
    contiguous last dimension), page_table int32 [B, max_pages], lengths,
    counts, now int32 [B]; positions int32 and weight_sum fp32
    [B, Hkv, max_pages * page_size].  lengths already counts the new rows."""
    torch = _torch()
    dev, dt = k_new.device, k_new.dtype
    if not k_new.is_cuda:
        raise ValueError("k_new must be a device tensor")
    _rows_ready("k_new", k_new, dt, dev, 4)
    _rows_ready("v_new", v_new, dt, dev, 4)
    if v_new.shape != k_new.shape or v_new.stride() != k_new.stride():
        k_new, v_new = k_new.contiguous(), v_new.contiguous()
        if v_new.shape != k_new.shape:
            raise ValueError("k_new and v_new must have the same shape")
    B, n, Hkv, D = k_new.shape
    pages, size, cols, H, Dc, kv = _cache_tensors(k_cache, v_cache, page_table, dt, dev)
    if (H, Dc) != (Hkv, D) or page_table.shape[0] != B:
        raise ValueError("the cache's heads, width or table rows do not match k_new")
    _required("lengths", lengths)
    for name, t in (("lengths", lengths), ("counts", counts), ("now", now)):
        _index(name, t, dev, (B,))
    slots = _slot_arrays((("positions", positions, torch.int32),
                          ("weight_sum", weight_sum, torch.float32)), B, Hkv, cols * size, dev)
    plan = CacheAppend(B, n, Hkv, D, pages, size, cols, dtype_code(k_new), k_new.stride()[:3], kv,
                       page_table.stride(0), slots)
    side = _side_stream(stream, dev)
    plan(k_new.data_ptr(), v_new.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
         page_table.data_ptr(), lengths.data_ptr(), _ptr(counts), _ptr(now), _ptr(positions),
         _ptr(weight_sum), _stream(stream))
    _claim(side, k_new, v_new, k_cache, v_cache, page_table, lengths, counts, now, positions,
           weight_sum)


def paged_attention(q, k_cache, v_cache, page_table, lengths, max_length=None, window: int = 0,
                    scale=None, weight_sum=None, out=None, workspace=None, stream=None):
    """(out [B, Hq, D], lse fp32 [B, Hq]) of one new row per sequence over the
    paged cache (see ctconv_paged_attention); weight_sum fp32 [B, Hkv, slots]
    or None is added to.  max_length: a bound on lengths, default the table's
    capacity.  workspace: None (allocated here) or a device tensor."""
    torch = _torch()
    dev, dt = q.device, q.dtype
    if not q.is_cuda:
        raise ValueError("q must be a device tensor")
    _rows_ready("q", q, dt, dev, 3)
    B, Hq, D = q.shape
    pages, size, cols, Hkv, Dc, kv = _cache_tensors(k_cache, v_cache, page_table, dt, dev)
    if Dc != D or page_table.shape[0] != B:
        raise ValueError("the cache's width or table rows do not match q")
    _required("lengths", lengths)
    _index("lengths", lengths, dev, (B,))
    slots = _slot_arrays((("weight_sum", weight_sum, torch.float32),), B, Hkv, cols * size, dev)
    y = _result(out, (B, Hq, D), dt, dev)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=dev)
    plan = PagedAttention(B, Hq, Hkv, D, pages, size, cols, max_length, window, scale,
                          weight_sum is not None, dtype_code(q), q.stride()[:2], kv,
                          y.stride()[:2], page_table.stride(0), slots)
    ws = _workspace(workspace, plan.workspace_bytes, dev)
    side = _side_stream(stream, dev)
    plan(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(),
         lengths.data_ptr(), y.data_ptr(), lse.data_ptr(), _ptr(weight_sum), _ptr(ws),
         0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))
    _claim(side, q, k_cache, v_cache, page_table, lengths, y, lse, weight_sum, ws)
    return y, lse


def cache_evict(k_cache, v_cache, page_table, lengths, weight_sum, keep: int, positions=None,
                now=None, sink: int = 0, recent: int = 0, max_length=None, stream=None):
    """Cut the cache back to `keep` slots per head, in place (see
    ctconv_cache_evict): the rows move in k_cache and v_cache, and weight_sum,
    positions and lengths are updated.  Returns source int32 [B, Hkv, keep].
    weight_sum fp32 and positions int32 (or None) [B, Hkv, slots]."""
    torch = _torch()
    dev, dt = k_cache.device, k_cache.dtype
    if not k_cache.is_cuda:
        raise ValueError("k_cache must be a device tensor")
    pages, size, cols, Hkv, D, kv = _cache_tensors(k_cache, v_cache, page_table, dt, dev)
    B, slots = page_table.shape[0], cols * size
    _required("weight_sum", weight_sum)
    if not 1 <= keep <= slots:
        raise ValueError(f"keep must be between 1 and the table's {slots} slots")
    _required("lengths", lengths)
    for name, t in (("lengths", lengths), ("now", now)):
        _index(name, t, dev, (B,))
    st = _slot_arrays((("weight_sum", weight_sum, torch.float32),
                       ("positions", positions, torch.int32)), B, Hkv, slots, dev)
    source = torch.empty((B, Hkv, keep), dtype=torch.int32, device=dev)
    plan = CacheEvict(B, Hkv, D, pages, size, cols, keep, max_length, sink, recent,
                      dtype_code(k_cache), kv, page_table.stride(0), st, st)
    side = _side_stream(stream, dev)
    plan(k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(), lengths.data_ptr(),
         _ptr(now), weight_sum.data_ptr(), _ptr(positions), weight_sum.data_ptr(),
         _ptr(positions), lengths.data_ptr(), source.data_ptr(), _stream(stream))
    _claim(side, k_cache, v_cache, page_table, lengths, now, weight_sum, positions, source)
    return source


def cross_attention(q, k, v, lengths=None, mask=None, scale=None, out=None, workspace=None,
                    stream=None):
    """(out [B, Lq, Hq, D], lse fp32 [B, Hq, Lq]) of q [B, Lq, Hq, D] over
    k, v [B, Lk, Hkv, D] (see ctconv_cross_attention); lengths int32 [B] or
    None; mask bool or uint8 [B, Lk] or None (True: seen)."""
    torch = _torch()
    dev, dt = q.device, q.dtype
    if not q.is_cuda:
        raise ValueError("q must be a device tensor")
    for name, t in (("q", q), ("k", k), ("v", v)):
        _rows_ready(name, t, dt, dev, 4)
    B, Lq, Hq, D = q.shape
    Lk, Hkv = k.shape[1], k.shape[2]
    if tuple(k.shape) != (B, Lk, Hkv, D) or v.shape != k.shape:
        raise ValueError("k and v must be [B, Lk, Hkv, D] with q's batch and width")
    _index("lengths", lengths, dev, (B,))
    if mask is not None:
        if mask.dtype == torch.bool:
            mask = mask.view(torch.uint8)
        _index("mask", mask, dev, (B, Lk), torch.uint8)
    y = _result(out, (B, Lq, Hq, D), dt, dev)
    lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=dev)
    plan = CrossAttention(B, Lq, Lk, Hq, Hkv, D, scale, dtype_code(q), q.stride()[:3],
                          k.stride()[:3], v.stride()[:3], y.stride()[:3],
                          None if mask is None else mask.stride(0))
    ws = _workspace(workspace, plan.workspace_bytes, dev)
    side = _side_stream(stream, dev)
    plan(q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(lengths), _ptr(mask), y.data_ptr(),
         lse.data_ptr(), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
         _stream(stream))
    _claim(side, q, k, v, lengths, mask, y, lse, ws)
    return y, lse


def norm_residual(x, h, post: int = NORM_NONE, post_weight=None, post_bias=None, scale=None,
                  gate=None, gate_fn: int = GATE_NONE, rows_per_gate: int = 1,
                  pre: int = NORM_LAYER, pre_weight=None, pre_bias=None, eps: float = 1e-5,
                  x_out=None, y=None, stream=None):
    """(x + scale * g(gate) * post(h), pre of that) row by row (see
    ctconv_norm_residual); x, h [..., C], gate [ceil(rows / rows_per_gate), C],
    the rest [C].  The second result is None when pre is NORM_NONE.  x_out may
    be x and y may be h."""
    torch = _torch()
    dev, dt = x.device, x.dtype
    if not x.is_cuda:
        raise ValueError("x must be a device tensor")
    _check_tensor("h", h, dt, dev, shape=tuple(x.shape))
    C = x.shape[-1]
    rows = x.numel() // C if C else 0
    for name, t in (("x_out", x_out), ("y", y)):
        if t is not None:
            _check_tensor(name, t, dt, dev, shape=tuple(x.shape))
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
    x, h = x.contiguous(), h.contiguous()
    if (gate is None) != (gate_fn == GATE_NONE):
        raise ValueError("gate and gate_fn go together")
    if gate is not None:
        groups = -(-rows // rows_per_gate) if rows_per_gate > 0 else 0
        _check_tensor("gate", gate, dt, dev, numel=groups * C)
        gate = gate.contiguous()
    params = []
    for name, t in (("post_weight", post_weight), ("post_bias", post_bias), ("scale", scale),
                    ("pre_weight", pre_weight), ("pre_bias", pre_bias)):
        if t is not None:
            _check_tensor(name, t, dt, dev, numel=C)
            t = t.contiguous()
        params.append(t)
    pw, pb, sc, nw, nb = params
    xo = torch.empty_like(x) if x_out is None else x_out
    yo = None if pre == NORM_NONE else torch.empty_like(x) if y is None else y
    plan = NormResidual(rows, C, post, pre, gate_fn, rows_per_gate, eps, dtype_code(x))
    side = _side_stream(stream, dev)
    plan(x.data_ptr(), h.data_ptr(), _ptr(pw), _ptr(pb), _ptr(sc), _ptr(gate), _ptr(nw), _ptr(nb),
         xo.data_ptr(), _ptr(yo), _stream(stream))
    _claim(side, x, h, gate, pw, pb, sc, nw, nb, xo, yo)
    return xo, yo
