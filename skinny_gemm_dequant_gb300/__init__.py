"""Python binding of libqlinear.so, the GB300 quantized decode linear layer.

Argument marshalling only: every function passes device pointers, sizes and the current CUDA
stream to the C ABI declared in ``include/qlinear.h``; all computation runs in the library's
CUDA kernels.  PyTorch is used for device memory (outputs, workspace) and streams.

The library must have been built (``python -m skinny_gemm_dequant_gb300._build`` or
``__graft_entry__.build()``); importing this package without it raises ``ImportError`` -
there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading
from typing import NamedTuple

import torch

from ._build import LIB as _LIB_PATH

__all__ = [
    "lib", "QLError", "qlinear_int8_w8a8", "qlinear_fp8_block", "qlinear_mxfp4", "moe_mxfp4_grouped",
    "workspace_bytes", "Workspace", "read_device_status", "set_wait_limit",
    "OP_INT8_W8A8", "OP_FP8_BLOCK", "OP_MXFP4", "OP_MOE_MXFP4", "OP_BF16", "OP_FP8_CHANNEL", "qlinear_bf16",
    "qlinear_fp8", "FP8_E4M3", "FP8_E5M2", "ACT_BF16", "ACT_E4M3_1X128", "PATHS",
    "token_amax", "qlinear_int8_w8a8_partial", "qlinear_int8_epilogue", "qlinear_fp8_block_partial",
    "qlinear_mxfp4_partial", "finish_f32",
    "qlinear_int4", "gated_ffn_int4", "gated_ffn", "gated_ffn_backward", "FFNCheckpoint", "OP_GATED_FFN",
    "OP_GATED_FFN_BWD", "gated_ffn_plan", "FFNPlan",
    "quantize_int8", "qlinear_int8", "moe_bf16", "moe_int8", "moe_int4", "OP_INT8_CODES", "OP_MOE_FEW",
]

if not os.path.exists(_LIB_PATH):
    raise ImportError(f"libqlinear.so is not built ({_LIB_PATH}); run skinny_gemm_dequant_gb300._build.build()")

lib = ctypes.CDLL(_LIB_PATH)

_vp, _i64, _int, _u32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint32, ctypes.c_size_t
_ip = ctypes.POINTER(ctypes.c_int)

lib.ql_status_string.restype = ctypes.c_char_p
lib.ql_status_string.argtypes = [_int]
lib.ql_version.restype = _int
lib.ql_workspace_bytes.restype = _sz
lib.ql_workspace_bytes.argtypes = [_int, _i64, _i64, _i64, _int, _int]
lib.ql_workspace_init.restype = _int
lib.ql_workspace_init.argtypes = [_vp, _sz, _vp]
lib.ql_read_device_status.restype = _int
lib.ql_read_device_status.argtypes = [_vp, _vp, _int, ctypes.POINTER(_u32)]
lib.ql_capture_id.restype = ctypes.c_uint64
lib.ql_capture_id.argtypes = [_vp]
lib.ql_set_wait_limit.restype = None
lib.ql_set_wait_limit.argtypes = [_u32]
lib.qlinear_int8_w8a8.restype = _int
lib.qlinear_int8_w8a8.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _i64,
                                  _vp, _vp, _vp, _vp, _sz, _vp, _ip]
lib.qlinear_fp8_block.restype = _int
lib.qlinear_fp8_block.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _int, _int, _int, _vp, _vp,
                                  _i64, _vp, _vp, _vp, _sz, _vp, _ip]
lib.qlinear_bf16.restype = _int
lib.qlinear_bf16.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _sz, _vp,
                             ctypes.POINTER(_int)]
lib.qlinear_fp8.restype = _int
lib.qlinear_fp8.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _int, _vp, _i64, _vp, _vp, _i64, _vp, _sz,
                            _vp, _ip]
lib.qlinear_mxfp4.restype = _int
lib.qlinear_mxfp4.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _int, _vp, _vp, _i64,
                              _vp, _vp, _vp, _sz, _vp, _ip]
lib.moe_mxfp4_grouped.restype = _int
lib.moe_mxfp4_grouped.argtypes = [_vp, _i64, _i64, _vp, _vp, _vp, _int, _int, _int, _vp, _vp, _vp, _vp, _i64,
                                  ctypes.c_float, ctypes.c_float, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _ip]

lib.ql_token_amax.restype = _int
lib.ql_token_amax.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp]
lib.qlinear_int8_w8a8_partial.restype = _int
lib.qlinear_int8_w8a8_partial.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _sz, _vp, _ip]
lib.qlinear_int8_epilogue.restype = _int
lib.qlinear_int8_epilogue.argtypes = [_vp, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _i64, _vp]
lib.qlinear_fp8_block_partial.restype = _int
lib.qlinear_fp8_block_partial.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _int, _int, _vp, _i64, _vp,
                                          _sz, _vp, _ip]
lib.qlinear_mxfp4_partial.restype = _int
lib.qlinear_mxfp4_partial.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _sz, _vp,
                                      _ip]
lib.ql_finish_f32.restype = _int
lib.ql_finish_f32.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp]

lib.qlinear_int4.restype = _int
lib.qlinear_int4.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _int, _i64, _vp, _i64, _i64, _vp, _vp, _i64,
                             _vp, _ip]
lib.gated_ffn_int4.restype = _int
lib.gated_ffn_int4.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _int, _i64, _vp, _i64, _i64,
                               ctypes.c_float, ctypes.c_float, _vp, _i64, _vp, _ip]
lib.gated_ffn.restype = _int
lib.gated_ffn.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, _i64, ctypes.c_float, ctypes.c_float, _vp, _i64, _int,
                          _vp, _vp, _vp, _sz, _vp, _ip]
lib.gated_ffn_backward.restype = _int
lib.gated_ffn_backward.argtypes = [_vp, _i64, _vp, _i64, _i64, _i64, _vp, _i64, _i64, ctypes.c_float, ctypes.c_float,
                                   _int, _vp, _vp, _vp, _i64, _vp, _i64, _vp, _sz, _vp, _ip]

lib.ql_gated_ffn_plan.restype = _int
lib.ql_gated_ffn_plan.argtypes = [_int, _i64, _i64, _i64, _int, ctypes.POINTER(ctypes.c_int32)]

lib.quantize_int8.restype = _int
lib.quantize_int8.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _vp]
lib.qlinear_int8.restype = _int
lib.qlinear_int8.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _i64, _vp, _int, _vp, _i64, _vp, _sz,
                             _vp, _ip]
_MOE_HEAD = [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _int, _int, _int]
_MOE_TAIL = [_i64, ctypes.c_float, ctypes.c_float, _vp, _vp, _vp, _vp, _i64, _vp, _sz, _vp, _ip]
lib.moe_bf16.restype = _int
lib.moe_bf16.argtypes = _MOE_HEAD + 2 * [_vp, _i64, _i64] + _MOE_TAIL
lib.moe_int8.restype = _int
lib.moe_int8.argtypes = _MOE_HEAD + 2 * [_vp, _i64, _i64, _vp] + _MOE_TAIL
lib.moe_int4.restype = _int
lib.moe_int4.argtypes = _MOE_HEAD + 6 * [_vp, _i64, _i64] + [_int, _i64] + _MOE_TAIL

OP_INT8_W8A8, OP_FP8_BLOCK, OP_MXFP4, OP_MOE_MXFP4, OP_BF16, OP_FP8_CHANNEL = 1, 2, 3, 4, 5, 6
OP_GATED_FFN, OP_GATED_FFN_BWD, OP_INT8_CODES, OP_MOE_FEW = 7, 8, 9, 10
FP8_E4M3, FP8_E5M2 = 0, 1
SCALE_BF16, SCALE_FP16 = 0, 1
_SCALE_FORMATS = {torch.bfloat16: SCALE_BF16, torch.float16: SCALE_FP16}
SAVE_NONE, SAVE_BF16, SAVE_INT8 = 0, 1, 2
ACT_BF16, ACT_E4M3_1X128 = 0, 1
PATHS = {0: "none", 1: "int8_skinny", 2: "fp8_skinny", 3: "fp8_tcgen05", 4: "mxfp4_skinny",
         5: "mxfp4_tcgen05", 6: "moe_mxfp4", 7: "bf16_skinny", 8: "fp8_channel_skinny",
         9: "int8_tcgen05", 10: "moe_mxfp4_tcgen05", 11: "int4_skinny", 12: "gated_ffn_int4",
         13: "gated_ffn_skinny", 14: "gated_ffn_tcgen05", 15: "gated_ffn_backward",
         16: "int8_codes_skinny", 17: "int8_codes_tcgen05", 18: "moe_bf16", 19: "moe_int8", 20: "moe_int4"}


class QLError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {lib.ql_status_string(status).decode()} (status {status})")


def _check(status: int, where: str):
    if status != 0:
        raise QLError(status, where)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    # the current stream's handle without building a Stream object (2.9 us a call on the Arm host)
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def workspace_bytes(op: int, M: int, N: int, K: int, E: int = 0, topk: int = 0) -> int:
    return int(lib.ql_workspace_bytes(op, M, N, K, E, topk))


class Workspace:
    """Device scratch for the library calls; zeroed once when (re)allocated, as the C ABI
    requires.  Calls sharing one Workspace must be ordered (same stream)."""

    def __init__(self, device=None):
        self.device = torch.device(device if device is not None else "cuda")
        self.buf = None
        self.lock = threading.Lock()  # held from the choice of the buffer to a gated block call's last launch
        self._recorded = []  # buffers that graphs hold the addresses of: not freed by a larger call

    def get(self, nbytes: int, stream=None) -> torch.Tensor:
        if self.buf is None or self.buf.numel() < nbytes:
            self.buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.device)
            _check(lib.ql_workspace_init(_ptr(self.buf), self.buf.numel(), _stream(stream)), "ql_workspace_init")
        return self.buf


_default_ws: dict = {}


def _ws(device, nbytes, stream, workspace):
    if workspace is None:
        # keyed by the stream's handle: a Python object's id can be reused once it is collected
        key = (torch.device(device).index, None if stream is None else int(stream.cuda_stream))
        workspace = _default_ws.setdefault(key, Workspace(device))
    return workspace.get(nbytes, stream)


def read_device_status(ws: torch.Tensor | None = None, clear: bool = True, stream=None):
    """(status, flags) of a workspace's status word: of ws, or, without one, of all default workspaces
    on the current device together, whose work is waited for."""
    if ws is None:
        torch.cuda.synchronize()
        bufs = [w.buf for w in (*_default_ws.values(), *_ffn_workspaces.values()) if w.buf is not None]
        both = [read_device_status(b, clear, stream) for b in bufs if b.device.index == torch.cuda.current_device()]
        return max((st for st, _ in both), default=0), functools.reduce(int.__or__, (f for _, f in both), 0)
    flags = _u32(0)
    st = lib.ql_read_device_status(_ptr(ws), _stream(stream), int(clear), ctypes.byref(flags))
    return st, int(flags.value)


def set_wait_limit(polls: int):
    lib.ql_set_wait_limit(int(polls))


def _bf16(t, name):
    if t.dtype != torch.bfloat16 or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA bfloat16 tensor")
    return t


def qlinear_int8_w8a8(x, w, w_scale, bias=None, *, debug=False, out=None, workspace=None, stream=None):
    """y = bf16((acc * x_s) * w_s) (+ bias) with per-token dynamic INT8 activations.
    x: bf16 [M, K]; w: int8 [N, K] (row stride w.stride(0)); w_scale: fp32 [N] or [1].
    With debug=True returns (y, acc int32 [M,N], x_q int8 [M,K], x_s fp32 [M], path)."""
    _bf16(x, "x")
    M, K = x.shape
    N = w.shape[0]
    if w.dtype != torch.int8 or w.stride(1) != 1 or x.stride(1) != 1:
        raise TypeError("w must be int8 with unit inner stride; x must have unit inner stride")
    y = out if out is not None else torch.empty(M, N, dtype=torch.bfloat16, device=x.device)
    acc = xq = xs = None
    if debug:
        acc = torch.empty(M, N, dtype=torch.int32, device=x.device)
        xq = torch.empty(M, K, dtype=torch.int8, device=x.device)
        xs = torch.empty(M, dtype=torch.float32, device=x.device)
    nbytes = workspace_bytes(OP_INT8_W8A8, M, N, K)
    ws = _ws(x.device, nbytes, stream, workspace)
    path = ctypes.c_int(0)
    _check(lib.qlinear_int8_w8a8(_ptr(x), M, K, x.stride(0), _ptr(w), N, w.stride(0), _ptr(w_scale),
                                 w_scale.numel(), _ptr(bias), _ptr(y), y.stride(0), _ptr(acc), _ptr(xq), _ptr(xs),
                                 _ptr(ws), ws.numel(), _stream(stream), ctypes.byref(path)), "qlinear_int8_w8a8")
    if debug:
        return y, acc, xq, xs, PATHS[path.value]
    return y


def qlinear_fp8_block(x, w, w_scale, *, K=None, block_n=128, block_k=128, act_mode=ACT_BF16, bias=None,
                      debug=False, out=None, workspace=None, stream=None):
    """Block-scaled FP8 linear.  w: uint8 E4M3 codes [N, ldw] (first K columns used);
    w_scale: uint8 UE8M0 [ceil(N/block_n), ceil(K/block_k)].  debug=True returns
    (y, aq, as, path) where aq/as are the 1x128 activation codes/scales (act_mode 1)."""
    _bf16(x, "x")
    M, Kx = x.shape
    K = Kx if K is None else K
    N = w.shape[0]
    y = out if out is not None else torch.empty(M, N, dtype=torch.bfloat16, device=x.device)
    aq = as_ = None
    if debug and act_mode == ACT_E4M3_1X128:
        aq = torch.empty(M, K, dtype=torch.uint8, device=x.device)
        as_ = torch.empty(M, K // 128, dtype=torch.uint8, device=x.device)
    ws = _ws(x.device, workspace_bytes(OP_FP8_BLOCK, M, N, K), stream, workspace)
    path = ctypes.c_int(0)
    _check(lib.qlinear_fp8_block(_ptr(x), M, K, x.stride(0), _ptr(w), N, w.stride(0), _ptr(w_scale), block_n,
                                 block_k, act_mode, _ptr(bias), _ptr(y), y.stride(0), _ptr(aq), _ptr(as_), _ptr(ws),
                                 ws.numel(), _stream(stream), ctypes.byref(path)), "qlinear_fp8_block")
    if debug:
        return y, aq, as_, PATHS[path.value]
    return y


def qlinear_mxfp4(x, w, w_scale, *, act_mode=ACT_BF16, bias=None, debug=False, out=None, workspace=None,
                  stream=None):
    """MXFP4 linear.  w: packed E2M1 uint8 [N, >=K/2]; w_scale: UE8M0 uint8 [N, >=K/32]."""
    _bf16(x, "x")
    M, K = x.shape
    N = w.shape[0]
    y = out if out is not None else torch.empty(M, N, dtype=torch.bfloat16, device=x.device)
    aq = as_ = None
    if debug and act_mode == ACT_E4M3_1X128:
        aq = torch.empty(M, K, dtype=torch.uint8, device=x.device)
        as_ = torch.empty(M, K // 128, dtype=torch.uint8, device=x.device)
    ws = _ws(x.device, workspace_bytes(OP_MXFP4, M, N, K), stream, workspace)
    path = ctypes.c_int(0)
    _check(lib.qlinear_mxfp4(_ptr(x), M, K, x.stride(0), _ptr(w), N, w.stride(0), _ptr(w_scale), w_scale.stride(0),
                             act_mode, _ptr(bias), _ptr(y), y.stride(0), _ptr(aq), _ptr(as_), _ptr(ws), ws.numel(),
                             _stream(stream), ctypes.byref(path)), "qlinear_mxfp4")
    if debug:
        return y, aq, as_, PATHS[path.value]
    return y


def qlinear_bf16(x, w, bias=None, *, debug=False, out=None, workspace=None, stream=None):
    """BF16 linear on unquantised weights.  x: bf16 [M, K]; w: bf16 [N, >=K] (row stride
    w.stride(0)).  With debug=True returns (y, path)."""
    _bf16(x, "x")
    M, K = x.shape
    N = w.shape[0]
    if w.dtype != torch.bfloat16 or w.stride(1) != 1 or x.stride(1) != 1:
        raise TypeError("w must be bfloat16 with unit inner stride; x must have unit inner stride")
    y = out if out is not None else torch.empty(M, N, dtype=torch.bfloat16, device=x.device)
    ws = _ws(x.device, workspace_bytes(OP_BF16, M, N, K), stream, workspace)
    path = ctypes.c_int(0)
    _check(lib.qlinear_bf16(_ptr(x), M, K, x.stride(0), _ptr(w), N, w.stride(0), _ptr(bias), _ptr(y), y.stride(0),
                            _ptr(ws), ws.numel(), _stream(stream), ctypes.byref(path)), "qlinear_bf16")
    if debug:
        return y, PATHS[path.value]
    return y


def qlinear_fp8(x, w, w_scale, w_fmt="e4m3", bias=None, *, debug=False, out=None, workspace=None, stream=None):
    """y = bf16(w_scale[n or 0] * sum_k x w) (+ bias) on FP8 weight codes.  x: bf16 [M, K];
    w: uint8 FP8 codes [N, >=K] (row stride w.stride(0)); w_fmt: "e4m3" or "e5m2"; w_scale:
    fp32 [N] (per channel) or [1] (per tensor).  With debug=True returns (y, path)."""
    _bf16(x, "x")
    M, K = x.shape
    N = w.shape[0]
    if w.dtype != torch.uint8 or w.stride(1) != 1 or x.stride(1) != 1:
        raise TypeError("w must be uint8 FP8 codes with unit inner stride; x must have unit inner stride")
    if w_scale.dtype != torch.float32:
        raise TypeError("w_scale must be float32")
    fmt = {"e4m3": FP8_E4M3, "e5m2": FP8_E5M2}[w_fmt]
    y = out if out is not None else torch.empty(M, N, dtype=torch.bfloat16, device=x.device)
    ws = _ws(x.device, workspace_bytes(OP_FP8_CHANNEL, M, N, K), stream, workspace)
    path = ctypes.c_int(0)
    _check(lib.qlinear_fp8(_ptr(x), M, K, x.stride(0), _ptr(w), N, w.stride(0), fmt, _ptr(w_scale), w_scale.numel(),
                           _ptr(bias), _ptr(y), y.stride(0), _ptr(ws), ws.numel(), _stream(stream),
                           ctypes.byref(path)), "qlinear_fp8")
    if debug:
        return y, PATHS[path.value]
    return y


def moe_mxfp4_grouped(x, w13, s13, w2, s2, *, router_logits=None, topk_ids=None, topk_weights=None, topk=8,
                      renormalize=False, swiglu_alpha=1.0, swiglu_limit=None, debug=False, out=None, workspace=None,
                      stream=None):
    """MXFP4 MoE decode layer.  x: bf16 [M, H]; w13 [E, 2I, H/2], s13 [E, 2I, H/32],
    w2 [E, H, I/2], s2 [E, H, I/32] (uint8).  Either router_logits (bf16 [M, E]) or
    topk_ids/topk_weights.  Expert activation silu(alpha * min(g, limit)) * clamp(u, +-limit)
    (swiglu_limit None: plain silu(g) * u).  debug=True returns (y, ids, weights, h, path)."""
    _bf16(x, "x")
    M, H = x.shape
    E, twoI, _ = w13.shape
    I = twoI // 2
    if topk_ids is not None:
        topk = topk_ids.shape[1]
    y = out if out is not None else torch.empty(M, H, dtype=torch.bfloat16, device=x.device)
    ids = wts = h = None
    if debug:
        ids = torch.empty(M, topk, dtype=torch.int32, device=x.device)
        wts = torch.empty(M, topk, dtype=torch.float32, device=x.device)
        h = torch.empty(M * topk, I, dtype=torch.bfloat16, device=x.device)
    ws = _ws(x.device, workspace_bytes(OP_MOE_MXFP4, M, H, I, E, topk), stream, workspace)
    path = ctypes.c_int(0)
    _check(lib.moe_mxfp4_grouped(_ptr(x), M, H, _ptr(router_logits), _ptr(topk_ids), _ptr(topk_weights), E, topk,
                                 int(renormalize), _ptr(w13), _ptr(s13), _ptr(w2), _ptr(s2), I, float(swiglu_alpha),
                                 float("inf") if swiglu_limit is None else float(swiglu_limit), _ptr(ids), _ptr(wts),
                                 _ptr(h), _ptr(y), _ptr(ws), ws.numel(), _stream(stream), ctypes.byref(path)),
           "moe_mxfp4_grouped")
    if debug:
        return y, ids, wts, h, PATHS[path.value]
    return y


# ------------------------------------------------------------------ 4-bit group-scaled weights
# These calls take microseconds on the GPU, so their Python is kept short: shapes and strides are
# read once, and the dispatch marker is asked for only with debug=True.
def _inf(limit):
    return math.inf if limit is None else float(limit)


def _int4_weights(K, sx, w, w_scale, w_zero, group):
    """Checks packed codes [N, >=K/2] and scales and zero points [N, >=ceil(K/group)] against x
    [M, K] with strides sx; returns (N, row strides of w, w_scale and w_zero, scale format)."""
    (N, cols), (ldw, inner) = w.shape, w.stride()
    if w.dtype is not torch.uint8 or not w.is_cuda or inner != 1 or sx[1] != 1:
        raise TypeError("w must be packed uint8 CUDA codes with unit inner stride; x must have unit inner stride")
    fmt = _SCALE_FORMATS.get(w_scale.dtype)
    (rows, scols), (lds, inner) = w_scale.shape, w_scale.stride()
    if fmt is None or not w_scale.is_cuda or inner != 1:
        raise TypeError("w_scale must be a bfloat16 or float16 CUDA tensor with unit inner stride")
    if group < 1:
        raise ValueError("group must be positive")
    groups = -(-K // group)
    if cols * 2 < K or rows != N or scols < groups:
        raise ValueError("w must be [N, >=K/2] and w_scale [N, >=ceil(K/group)]")
    ldz = 0
    if w_zero is not None:
        (rows, zcols), (ldz, inner) = w_zero.shape, w_zero.stride()
        if w_zero.dtype is not torch.uint8 or not w_zero.is_cuda or inner != 1:
            raise TypeError("w_zero must be a uint8 CUDA tensor with unit inner stride")
        if rows != N or zcols < groups:
            raise ValueError("w_zero must be [N, >=ceil(K/group)]")
    return N, ldw, lds, ldz, fmt


def _empty(shape, dtype, x, stream):
    # an output belongs to the stream that writes it: memory of the current stream's pool may still
    # be in use there
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=x.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=x.device)


def _out(out, M, N, x, stream, name="out"):
    if out is None:
        return _empty((M, N), torch.bfloat16, x, stream)
    if out.dtype is not torch.bfloat16 or not out.is_cuda or out.shape != (M, N) or out.stride(1) != 1:
        raise TypeError(f"{name} must be a bfloat16 CUDA tensor [{M}, {N}] with unit inner stride")
    return out


def qlinear_int4(x, w, w_scale, w_zero=None, bias=None, *, group=128, debug=False, out=None, stream=None):
    """y = x W^T (+ bias after the bf16 cast) on 4-bit weights w[n,k] = (q - zero) * scale per group
    of K.  x: bf16 [M, K]; w: uint8 [N, >=K/2], element 2i in the low nibble of byte i; w_scale: bf16
    or fp16 [N, >=ceil(K/group)]; w_zero: uint8 [N, >=ceil(K/group)] or None: 8.
    group: a power of two >= 32.  With debug=True returns (y, path)."""
    _bf16(x, "x")
    (M, K), sx = x.shape, x.stride()
    N, ldw, lds, ldz, fmt = _int4_weights(K, sx, w, w_scale, w_zero, group)
    if bias is not None and (bias.dtype is not torch.bfloat16 or not bias.is_cuda or bias.shape != (N,)
                             or not bias.is_contiguous()):
        raise TypeError(f"bias must be a bfloat16 CUDA tensor [{N}]")
    y = _out(out, M, N, x, stream)
    path = ctypes.c_int(0) if debug else None
    st = lib.qlinear_int4(x.data_ptr(), M, K, sx[0], w.data_ptr(), N, ldw, w_scale.data_ptr(), fmt, lds, _ptr(w_zero),
                          ldz, group, _ptr(bias), y.data_ptr(), N if out is None else y.stride(0), _stream(stream),
                          path)
    if st:
        raise QLError(st, "qlinear_int4")
    return (y, PATHS[path.value]) if debug else y


def gated_ffn_int4(x, w13, w_scale, w_zero=None, *, group=128, swiglu_alpha=1.0, swiglu_limit=None, debug=False,
                   out=None, stream=None):
    """h = silu(alpha * min(g, limit)) * clamp(u, +-limit) with g, u = x W13^T on 4-bit weights (rows
    [0, I) gate, [I, 2I) up), stored as qlinear_int4's, in one launch.  x: bf16 [M, H]; w13: uint8
    [2I, >=H/2].  Returns bf16 [M, I]; with debug=True (h, path)."""
    _bf16(x, "x")
    (M, H), sx = x.shape, x.stride()
    N, ldw, lds, ldz, fmt = _int4_weights(H, sx, w13, w_scale, w_zero, group)
    if N & 1:
        raise ValueError("w13 must have an even number of rows (gate, then up)")
    I = N >> 1
    h = _out(out, M, I, x, stream)
    path = ctypes.c_int(0) if debug else None
    st = lib.gated_ffn_int4(x.data_ptr(), M, H, sx[0], w13.data_ptr(), I, ldw, w_scale.data_ptr(), fmt, lds,
                            _ptr(w_zero), ldz, group, swiglu_alpha, _inf(swiglu_limit), h.data_ptr(),
                            I if out is None else h.stride(0), _stream(stream), path)
    if st:
        raise QLError(st, "gated_ffn_int4")
    return (h, PATHS[path.value]) if debug else h


# ------------------------------------------------------------------ gated feed-forward block
class FFNCheckpoint(NamedTuple):
    """What gated_ffn keeps of g and u for gated_ffn_backward.  mode "bf16": data bf16 [M, 2, P];
    mode "int8": data int8 codes [M, 2, P] and scale fp32 [M, 2, P/128], value = code * scale; P = I
    rounded up to 128 (columns past I are undefined)."""
    mode: str
    data: torch.Tensor
    scale: torch.Tensor | None


_ffn_bytes = functools.lru_cache(maxsize=256)(workspace_bytes)
_ffn_workspaces: dict = {}
_ffn_captures: dict = {}  # of graphs being captured: (device, stream) -> _Captured
_ZERO_BYTES = 256 + (1 << 20)  # of a workspace's start: the status word and what is zero between calls


class _Captured:
    """The workspace of a graph's calls on one stream: memory of the graph's pool, zeroed once in the
    graph, before the first call that counts on it."""

    def __init__(self, capture, ws):
        self.capture, self.ws, self.zeroed = capture, ws, False


class _Scratch:
    """The workspace of a call of the gated block, of an 8-bit-code linear or of a few-token
    mixture-of-experts layer, locked while its launches are put on the stream:

        with _Scratch(...) as ws:  # the buffer

    The caller's Workspace, or one per device and stream (the current stream's handle if none is
    given), allocated from its stream's own pool.  A backward pass is two or three launches that hand
    [dg du] on in the workspace, a mixture-of-experts layer two that hand h on, and ctypes lets other
    threads run meanwhile: without the lock a thread's launches on the same stream could come between
    another's.

    While the stream is captured: a given Workspace that is large enough already, kept from then on
    for the graph's sake, or else memory of the graph's own, one piece for all of its calls on the
    stream: a Workspace that later calls use too would be zeroed by that graph alone and shared with
    every graph that is captured on the same stream.  cut() says whether the call counts on zeroed
    tickets."""

    __slots__ = ("ws", "nbytes", "stream", "recorded")

    def __init__(self, x, nbytes, stream, workspace, cut):
        self.nbytes, self.stream = nbytes, stream
        key = (x.device.index, _stream(stream))
        self.recorded = lib.ql_capture_id(key[1])
        if self.recorded:
            if workspace is None or workspace.buf is None or workspace.buf.numel() < self.nbytes:
                workspace = self.of_graph(key, x, cut)
        else:
            if _ffn_captures:
                _ffn_captures.clear()  # their graphs' pools keep the memory; one that goes on takes another piece
            if workspace is None:
                workspace = _ffn_workspaces.get(key)
                if workspace is None:
                    workspace = _ffn_workspaces.setdefault(key, Workspace(x.device))
        self.ws = workspace

    def of_graph(self, key, x, cut):
        mine = _ffn_captures.get(key)
        if mine is None or mine.capture != self.recorded or mine.ws.buf.numel() < self.nbytes:
            mine = _Captured(self.recorded, Workspace(x.device))
            mine.ws.buf = _empty((self.nbytes,), torch.uint8, x, self.stream)
            _ffn_captures[key] = mine
        if not mine.zeroed and cut():
            _check(lib.ql_workspace_init(_ptr(mine.ws.buf), _ZERO_BYTES, key[1]), "ql_workspace_init")
            mine.zeroed = True
        return mine.ws

    def __enter__(self):
        ws = self.ws
        ws.lock.acquire()
        try:
            if self.stream is None or (ws.buf is not None and ws.buf.numel() >= self.nbytes):
                buf = ws.get(self.nbytes, self.stream)
            else:
                with torch.cuda.stream(self.stream):
                    buf = ws.get(self.nbytes, self.stream)
            if self.recorded and not any(b is buf for b in ws._recorded):
                ws._recorded.append(buf)
            return buf
        except BaseException:
            ws.lock.release()
            raise

    def __exit__(self, *exc):
        self.ws.lock.release()


_SAVE = {None: SAVE_NONE, "bf16": SAVE_BF16, "int8": SAVE_INT8}


def _ffn_weights(x, w13):
    """Checks w13 [2I, H] against x [M, H]; returns (M, H, I, row strides of x and w13)."""
    (M, H), (ldx, ix) = x.shape, x.stride()
    (rows, cols), (ldw, iw) = w13.shape, w13.stride()
    if w13.dtype is not torch.bfloat16 or not w13.is_cuda or iw != 1 or ix != 1:
        raise TypeError("w13 must be a bfloat16 CUDA tensor with unit inner stride; x must have unit inner stride")
    if rows & 1 or cols != H:
        raise ValueError("w13 must be [2I, H] (gate rows, then up rows) for x [M, H]")
    return M, H, rows >> 1, ldx, ldw


def gated_ffn(x, w13, *, swiglu_alpha=1.0, swiglu_limit=None, save=None, debug=False, out=None, workspace=None,
              stream=None):
    """h = silu(alpha * min(g, limit)) * clamp(u, +-limit) with g, u = x W13^T, in one launch.  x: bf16
    [M, H]; w13: bf16 [2I, H], rows [0, I) gate and [I, 2I) up; H and I multiples of 8.  save: None,
    "bf16" or "int8" also returns an FFNCheckpoint of g and u: (h, checkpoint).  debug=True appends
    the path.  Without a workspace one is kept per device and stream; captured calls share a piece of
    their graph's own memory per stream.  As with every call here, autograd records nothing: the
    gradients are gated_ffn_backward's."""
    _bf16(x, "x")
    M, H, I, ldx, ldw = _ffn_weights(x, w13)
    if save not in _SAVE:
        raise ValueError('save must be None, "bf16" or "int8"')
    h = _out(out, M, I, x, stream)
    saved = data = scale = None
    if save is not None:
        P = -(-I // 128) * 128
        data = _empty((M, 2, P), torch.bfloat16 if save == "bf16" else torch.int8, x, stream)
        if save == "int8":
            scale = _empty((M, 2, P // 128), torch.float32, x, stream)
        saved = FFNCheckpoint(save, data, scale)
    path = ctypes.c_int(0) if debug else None
    with _Scratch(x, _ffn_bytes(OP_GATED_FFN, M, I, H), stream, workspace,
                  lambda: gated_ffn_plan("forward", M, I, H, save=save).cut) as ws:
        st = lib.gated_ffn(x.data_ptr(), M, H, ldx, w13.data_ptr(), I, ldw, swiglu_alpha, _inf(swiglu_limit),
                           h.data_ptr(), I if out is None else h.stride(0), _SAVE[save], _ptr(data), _ptr(scale),
                           ws.data_ptr(), ws.numel(), _stream(stream), path)
    if st:
        raise QLError(st, "gated_ffn")
    res = (h,) if saved is None else (h, saved)
    if debug:
        res += (PATHS[path.value],)
    return res[0] if len(res) == 1 else res


def gated_ffn_backward(dh, x, w13, saved, *, swiglu_alpha=1.0, swiglu_limit=None, need_dx=True, need_dw=True,
                       out_dx=None, out_dw=None, workspace=None, stream=None):
    """Gradients of gated_ffn from its checkpoint: (dx bf16 [M, H], dw13 bf16 [2I, H]) for dh bf16
    [M, I]; an output that is not needed is None and costs nothing.  swiglu_alpha and swiglu_limit
    as in the forward.  x is read for dw13 only and w13 for dx only: the other may be None
    (I is dh's width then)."""
    _bf16(dh, "dh")
    if (x is None and (need_dw or w13 is None)) or (w13 is None and need_dx):
        raise TypeError("x is needed for dw13, w13 for dx")
    # a row of the other operand stands in for the one that is not given: its shape is used, it is not read
    if x is None:
        x = w13[:1].expand(dh.shape[0], -1)
    if w13 is None:
        w13 = x[:1].expand(2 * dh.shape[1], -1)
    _bf16(x, "x")
    M, H, I, ldx, ldw = _ffn_weights(x, w13)
    if dh.shape != (M, I) or dh.stride(1) != 1:
        raise TypeError(f"dh must be [{M}, {I}] with unit inner stride")
    mode, data, scale = saved
    P = -(-I // 128) * 128
    if (mode not in ("bf16", "int8") or not data.is_cuda or data.shape != (M, 2, P) or not data.is_contiguous()
            or data.dtype is not (torch.bfloat16 if mode == "bf16" else torch.int8)):
        raise ValueError("saved must be the FFNCheckpoint of this x and w13")
    if mode == "int8" and (scale is None or not scale.is_cuda or scale.shape != (M, 2, P // 128) or not scale.is_contiguous()
                           or scale.dtype is not torch.float32):
        raise ValueError("saved must be the FFNCheckpoint of this x and w13")
    dx = _out(out_dx, M, H, x, stream, "out_dx") if need_dx else None
    dw = _out(out_dw, 2 * I, H, x, stream, "out_dw") if need_dw else None
    with _Scratch(x, _ffn_bytes(OP_GATED_FFN_BWD, M, I, H), stream, workspace, lambda: (
            (need_dx and gated_ffn_plan("dx", M, I, H, both=need_dw).cut)
            or (need_dw and gated_ffn_plan("dw", M, I, H, both=need_dx).cut))) as ws:
        st = lib.gated_ffn_backward(dh.data_ptr(), dh.stride(0), x.data_ptr(), M, H, ldx, w13.data_ptr(), I, ldw,
                                    swiglu_alpha, _inf(swiglu_limit), _SAVE[mode], data.data_ptr(), _ptr(scale), _ptr(dx),
                                    0 if dx is None else dx.stride(0), _ptr(dw), 0 if dw is None else dw.stride(0),
                                    ws.data_ptr(), ws.numel(), _stream(stream), None)
    if st:
        raise QLError(st, "gated_ffn_backward")
    return dx, dw


class FFNPlan(NamedTuple):
    """How one GEMM of the gated block is laid out: pairs of CTAs (0: the few-token kernel), columns of
    a tile, tiles taken whole, tiles cut along the summed dimension and parts of each, and the
    launches of the call's GEMMs."""
    pairs: int
    width: int
    whole: int
    cut: int
    parts: int
    launches: int


def gated_ffn_plan(gemm, M, I, H, *, save=None, both=True) -> FFNPlan:
    """gemm: "forward" (with save as in gated_ffn), "dx" or "dw" (both: the call computes the other
    gradient too).  Nothing is launched."""
    out = (ctypes.c_int32 * 6)()
    which = {"forward": 0, "dx": 1, "dw": 2}[gemm]
    _check(lib.ql_gated_ffn_plan(which, M, I, H, int(both) if which else _SAVE[save], out), "ql_gated_ffn_plan")
    return FFNPlan(*out)


# ------------------------------------------------------------------ 8-bit codes on both sides
# A few microseconds on the GPU: each tensor's shape, strides and device are read once.
_OUT_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _always():
    return True


def _device(x, name="x"):
    """x's device, the current one: launches go there."""
    dev = x.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError(f"{name} must be on the current CUDA device")
    return dev


def _codes(t, name, dev):
    """(shape, strides) of an int8 matrix."""
    shape, stride = t.shape, t.stride()
    if t.dtype is not torch.int8 or t.get_device() != dev or len(shape) != 2 or stride[1] != 1:
        raise TypeError(f"{name} must be a 2-d int8 tensor with unit inner stride on cuda:{dev}")
    return shape, stride


def _dense(t, name, shape, dtype, dev):
    """The address of a contiguous tensor of that shape."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {str(dtype)[6:]} tensor {list(shape)} on cuda:{dev}")
    return t.data_ptr()


def quantize_int8(x, *, out=None, out_scale=None, stream=None):
    """(codes int8 [M, K], scale fp32 [M]) of x bf16 [M, K], K a multiple of 8, by qlinear_int8_w8a8's
    rule: scale = max|x| / 127 of the row, codes = x / scale rounded half to even.  For projections
    that share their input: qlinear_int8 takes both."""
    dev = _device(x)
    _bf16(x, "x")
    (M, K), (ldx, inner) = x.shape, x.stride()
    if inner != 1:
        raise TypeError("x must have unit inner stride")
    if out is None:
        out = _empty((M, K), torch.int8, x, stream)
    else:
        _dense(out, "out", (M, K), torch.int8, dev)
    if out_scale is None:
        out_scale = _empty((M,), torch.float32, x, stream)
    else:
        _dense(out_scale, "out_scale", (M,), torch.float32, dev)
    _check(lib.quantize_int8(x.data_ptr(), M, K, ldx, out.data_ptr(), out_scale.data_ptr(), _stream(stream)),
           "quantize_int8")
    return out, out_scale


def qlinear_int8(x_q, x_scale, w, w_scale, bias=None, *, out_dtype=torch.bfloat16, debug=False, out=None,
                 workspace=None, stream=None):
    """y = (acc * x_scale) * w_scale (+ bias after the cast), acc = x_q w^T exact in int32.  x_q: int8
    [M, K], K a multiple of 16; x_scale: fp32 [M] (quantize_int8 gives both); w: int8 [N, K]; w_scale:
    fp32 [N] or [1]; bias: bf16 [N]; out_dtype: bfloat16, float16 or float32.  Without a workspace one
    is kept per device and stream; captured calls share a piece of their graph's own memory per stream.
    With debug=True returns (y, path)."""
    dev = _device(x_q, "x_q")
    (M, K), sx = _codes(x_q, "x_q", dev)
    (N, Kw), sw = _codes(w, "w", dev)
    if Kw != K:
        raise ValueError(f"w must be [N, {K}] for x_q [{M}, {K}]")
    xs = _dense(x_scale, "x_scale", (M,), torch.float32, dev)
    channels = w_scale.numel()
    ws = _dense(w_scale, "w_scale", (1 if channels == 1 else N,), torch.float32, dev)
    bias = None if bias is None else _dense(bias, "bias", (N,), torch.bfloat16, dev)
    if out is None:
        out = _empty((M, N), out_dtype, x_q, stream)
        ldy = N
    else:
        out_dtype, ldy = out.dtype, out.stride(0)
        if out.get_device() != dev or out.shape != (M, N) or out.stride(1) != 1:
            raise TypeError(f"out must be [{M}, {N}] with unit inner stride on cuda:{dev}")
    fmt = _OUT_TYPES.get(out_dtype)
    if fmt is None:
        raise TypeError("the output must be bfloat16, float16 or float32")
    path = ctypes.c_int(0) if debug else None
    with _Scratch(x_q, _ffn_bytes(OP_INT8_CODES, M, N, K), stream, workspace, _always) as buf:
        st = lib.qlinear_int8(x_q.data_ptr(), M, K, sx[0], xs, w.data_ptr(), N, sw[0], ws, channels, bias, fmt,
                              out.data_ptr(), ldy, buf.data_ptr(), buf.numel(), _stream(stream), path)
    if st:
        raise QLError(st, "qlinear_int8")
    return (out, PATHS[path.value]) if debug else out


# ------------------------------------------------------------------ mixture of experts, few tokens
def _experts(w, name, E, rows, cols, dtype, dev):
    """(address, row stride, expert stride) of [E, rows, >= cols] weights, scales or zero points."""
    shape, stride = w.shape, w.stride()
    if w.dtype is not dtype or w.get_device() != dev or len(shape) != 3 or stride[2] != 1:
        raise TypeError(f"{name} must be a 3-d {str(dtype)[6:]} tensor with unit inner stride on cuda:{dev}")
    if shape[0] != E or shape[1] != rows or shape[2] < cols:
        raise ValueError(f"{name} must be [{E}, {rows}, {cols}]")
    return w.data_ptr(), stride[1], stride[0]


def _moe(call, x, w13, mats, router_logits, topk_ids, topk_weights, topk, renormalize, swiglu_alpha, swiglu_limit, debug,
         out, workspace, stream):
    """mats(E, I, H, device): the weights' arguments of the C call, checked."""
    dev = _device(x)
    _bf16(x, "x")
    (M, H), sx, (E, rows, _) = x.shape, x.stride(), w13.shape
    if sx[1] != 1:
        raise TypeError("x must have unit inner stride")
    if rows & 1:
        raise ValueError("w13 must have an even number of rows (gate, then up)")
    I = rows >> 1
    logits = ids_in = w_in = None
    if topk_ids is None:
        if router_logits is None:
            raise ValueError("either router_logits or topk_ids and topk_weights must be given")
        logits = _dense(router_logits, "router_logits", (M, E), torch.bfloat16, dev)
    else:
        if router_logits is not None or topk_weights is None:
            raise ValueError("either router_logits or topk_ids and topk_weights must be given")
        topk = topk_ids.shape[-1]
        ids_in = _dense(topk_ids, "topk_ids", (M, topk), torch.int32, dev)
        w_in = _dense(topk_weights, "topk_weights", (M, topk), torch.float32, dev)
    args = mats(E, I, H, dev)
    if out is None:
        y, ldy = _empty((M, H), torch.bfloat16, x, stream), H
    else:
        y, ldy = _out(out, M, H, x, stream), out.stride(0)
        if out.get_device() != dev:
            raise TypeError(f"out must be on cuda:{dev}")
    ids = wts = h = path = None
    if debug:
        ids = _empty((M, topk), torch.int32, x, stream)
        wts = _empty((M, topk), torch.float32, x, stream)
        h = _empty((M * topk, I), torch.bfloat16, x, stream)
        path = ctypes.c_int(0)
    with _Scratch(x, _ffn_bytes(OP_MOE_FEW, M, H, I, E, topk), stream, workspace, _always) as buf:
        st = call(x.data_ptr(), M, H, sx[0], logits, ids_in, w_in, E, topk, renormalize, *args, I, swiglu_alpha,
                  _inf(swiglu_limit), _ptr(ids), _ptr(wts), _ptr(h), y.data_ptr(), ldy, buf.data_ptr(), buf.numel(),
                  _stream(stream), path)
    if st:
        raise QLError(st, call.__name__)
    return (y, ids, wts, h, PATHS[path.value]) if debug else y


def moe_bf16(x, w13, w2, *, router_logits=None, topk_ids=None, topk_weights=None, topk=8, renormalize=False,
             swiglu_alpha=1.0, swiglu_limit=None, debug=False, out=None, workspace=None, stream=None):
    """Mixture-of-experts layer for 1 to 64 tokens on bf16 weights, in two launches.  x: bf16 [M, H];
    w13: bf16 [E, 2I, H] (gate rows, then up rows), w2: bf16 [E, H, I]; H and I multiples of 8.  Routing,
    activation and debug=True's (y, ids, weights, h, path) are moe_mxfp4_grouped's; an id outside
    [0, E) is padding (debug=True: id -1 and a row of zeros in h), and a token without an expert gets
    zeros.  Workspaces as qlinear_int8's."""
    def mats(E, I, H, dev):
        return (*_experts(w13, "w13", E, 2 * I, H, torch.bfloat16, dev), *_experts(w2, "w2", E, H, I, torch.bfloat16, dev))
    return _moe(lib.moe_bf16, x, w13, mats, router_logits, topk_ids, topk_weights, topk, renormalize, swiglu_alpha,
                swiglu_limit, debug, out, workspace, stream)


def moe_int8(x, w13, s13, w2, s2, *, router_logits=None, topk_ids=None, topk_weights=None, topk=8, renormalize=False,
             swiglu_alpha=1.0, swiglu_limit=None, debug=False, out=None, workspace=None, stream=None):
    """moe_bf16's layer on 8-bit codes: w13 int8 [E, 2I, H] with s13 fp32 [E, 2I], w2 int8 [E, H, I]
    with s2 fp32 [E, H]; H and I multiples of 16.  x is quantised per token and h per (token, expert)
    inside, by quantize_int8's rule.  Sums of gate and up are exact, those of down over runs of at most
    1024 k of an expert, which are scaled and added in fp32."""
    def mats(E, I, H, dev):
        return (*_experts(w13, "w13", E, 2 * I, H, torch.int8, dev), _dense(s13, "s13", (E, 2 * I), torch.float32, dev),
                *_experts(w2, "w2", E, H, I, torch.int8, dev), _dense(s2, "s2", (E, H), torch.float32, dev))
    return _moe(lib.moe_int8, x, w13, mats, router_logits, topk_ids, topk_weights, topk, renormalize, swiglu_alpha,
                swiglu_limit, debug, out, workspace, stream)


_NO_ZEROS = (None, 0, 0)


def moe_int4(x, w13, s13, w2, s2, z13=None, z2=None, *, group=128, router_logits=None, topk_ids=None,
             topk_weights=None, topk=8, renormalize=False, swiglu_alpha=1.0, swiglu_limit=None, debug=False, out=None,
             workspace=None, stream=None):
    """moe_bf16's layer on 4-bit weights stored as qlinear_int4's: w13 uint8 [E, 2I, >=H/2], w2 uint8
    [E, H, >=I/2], scales bf16 or fp16 [E, rows, >=ceil(columns/group)], zero points uint8 of the same
    shape or None: 8; H and I multiples of 32, group a power of two >= 32."""
    def mats(E, I, H, dev):
        scale, u8 = s13.dtype, torch.uint8
        fmt = _SCALE_FORMATS.get(scale)
        if fmt is None:
            raise TypeError("s13 and s2 must both be bfloat16 or both float16")
        if group < 1:
            raise ValueError("group must be positive")
        g13, g2 = -(-H // group), -(-I // group)
        return (*_experts(w13, "w13", E, 2 * I, (H + 1) >> 1, u8, dev), *_experts(s13, "s13", E, 2 * I, g13, scale, dev),
                *(_NO_ZEROS if z13 is None else _experts(z13, "z13", E, 2 * I, g13, u8, dev)),
                *_experts(w2, "w2", E, H, (I + 1) >> 1, u8, dev), *_experts(s2, "s2", E, H, g2, scale, dev),
                *(_NO_ZEROS if z2 is None else _experts(z2, "z2", E, H, g2, u8, dev)), fmt, group)
    return _moe(lib.moe_int4, x, w13, mats, router_logits, topk_ids, topk_weights, topk, renormalize, swiglu_alpha,
                swiglu_limit, debug, out, workspace, stream)


# ------------------------------------------------------------------ sharded layers
def token_amax(x, *, out=None, stream=None):
    """Per-token max |x| of a K shard (fp32 [M]): the row-parallel INT8 layer's all-reduce MAX
    input."""
    _bf16(x, "x")
    M, K = x.shape
    amax = out if out is not None else torch.empty(M, dtype=torch.float32, device=x.device)
    _check(lib.ql_token_amax(_ptr(x), M, K, x.stride(0), _ptr(amax), _stream(stream)), "ql_token_amax")
    return amax


def qlinear_int8_w8a8_partial(x, w, amax, *, debug=False, out=None, workspace=None, stream=None):
    """A K shard of a row-parallel INT8 layer: exact int32 sums [M, N] over this shard's K, with
    x_s = amax / 127 (amax: the tokens' amax over the whole row).  debug=True also returns the
    codes and the path: (acc, x_q, path)."""
    _bf16(x, "x")
    M, K = x.shape
    N = w.shape[0]
    if w.dtype != torch.int8 or w.stride(1) != 1 or x.stride(1) != 1:
        raise TypeError("w must be int8 with unit inner stride; x must have unit inner stride")
    acc = out if out is not None else torch.empty(M, N, dtype=torch.int32, device=x.device)
    xq = torch.empty(M, K, dtype=torch.int8, device=x.device) if debug else None
    ws = _ws(x.device, workspace_bytes(OP_INT8_W8A8, M, N, K), stream, workspace)
    path = ctypes.c_int(0)
    _check(lib.qlinear_int8_w8a8_partial(_ptr(x), M, K, x.stride(0), _ptr(w), N, w.stride(0), _ptr(amax), _ptr(acc),
                                         _ptr(xq), _ptr(ws), ws.numel(), _stream(stream), ctypes.byref(path)),
           "qlinear_int8_w8a8_partial")
    if debug:
        return acc, xq, PATHS[path.value]
    return acc


def qlinear_int8_epilogue(acc, amax, w_scale, bias=None, *, out=None, stream=None):
    """y = bf16((acc * amax/127) * w_scale) (+ bias) on int32 sums added over the shards."""
    M, N = acc.shape
    y = out if out is not None else torch.empty(M, N, dtype=torch.bfloat16, device=acc.device)
    _check(lib.qlinear_int8_epilogue(_ptr(acc), M, N, _ptr(amax), _ptr(w_scale), w_scale.numel(), _ptr(bias), _ptr(y),
                                     y.stride(0), _stream(stream)), "qlinear_int8_epilogue")
    return y


def qlinear_fp8_block_partial(x, w, w_scale, *, K=None, block_n=128, block_k=128, out=None, workspace=None,
                              stream=None):
    """A K shard of a row-parallel FP8-block layer: fp32 partial sums [M, N] (no bias)."""
    _bf16(x, "x")
    M, Kx = x.shape
    K = Kx if K is None else K
    N = w.shape[0]
    y32 = out if out is not None else torch.empty(M, N, dtype=torch.float32, device=x.device)
    ws = _ws(x.device, workspace_bytes(OP_FP8_BLOCK, M, N, K), stream, workspace)
    path = ctypes.c_int(0)
    _check(lib.qlinear_fp8_block_partial(_ptr(x), M, K, x.stride(0), _ptr(w), N, w.stride(0), _ptr(w_scale), block_n,
                                         block_k, _ptr(y32), y32.stride(0), _ptr(ws), ws.numel(), _stream(stream),
                                         ctypes.byref(path)), "qlinear_fp8_block_partial")
    return y32


def qlinear_mxfp4_partial(x, w, w_scale, *, out=None, workspace=None, stream=None):
    """A K shard of a row-parallel MXFP4 layer: fp32 partial sums [M, N] (no bias)."""
    _bf16(x, "x")
    M, K = x.shape
    N = w.shape[0]
    y32 = out if out is not None else torch.empty(M, N, dtype=torch.float32, device=x.device)
    ws = _ws(x.device, workspace_bytes(OP_MXFP4, M, N, K), stream, workspace)
    path = ctypes.c_int(0)
    _check(lib.qlinear_mxfp4_partial(_ptr(x), M, K, x.stride(0), _ptr(w), N, w.stride(0), _ptr(w_scale),
                                     w_scale.stride(0), _ptr(y32), y32.stride(0), _ptr(ws), ws.numel(), _stream(stream),
                                     ctypes.byref(path)), "qlinear_mxfp4_partial")
    return y32


def finish_f32(y32, bias=None, *, out=None, stream=None):
    """bf16(y32) (+ bias after the cast): the one rounding of fp32 sums added over the shards."""
    M, N = y32.shape
    y = out if out is not None else torch.empty(M, N, dtype=torch.bfloat16, device=y32.device)
    _check(lib.ql_finish_f32(_ptr(y32), M, N, y32.stride(0), _ptr(bias), _ptr(y), y.stride(0), _stream(stream)),
           "ql_finish_f32")
    return y
