"""Python binding of libtsgemm (persistent bf16 GEMM with static / Cluster Launch
Control tile scheduling, the grid-stride int16 copy, and the mixture-of-experts
operators: routing, 8-bit quantisation and products, combine; a linear layer's
operators: fused product, gradients, orthogonalised updates) for one GB300.

This module only marshals arguments: torch tensors become device pointers and
sizes, the current torch stream becomes a cudaStream_t, and every computation
runs in the library's CUDA kernels.  There is no fallback: if the shared
library is missing or fails to load, importing this package raises.

The C entry points are declared in include/tsgemm.h; the functions here have
the same names.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libtsgemm.so")

TS_OK, TS_ERR_INVALID_ARG, TS_ERR_UNSUPPORTED, TS_ERR_CUDA, TS_ERR_TIMEOUT = range(5)
TS_SCHED_STATIC, TS_SCHED_CLC, TS_SCHED_NONPERSISTENT = 0, 1, 2
TS_OUT_BF16, TS_OUT_F32 = 0, 1
TS_TILE_AUTO, TS_TILE_128x128, TS_TILE_128x256, TS_TILE_256x256_2CTA = range(4)
PROTOCOL_LOG_ROLES = 20  # roles per CTA in a protocol log (ts_gemm_opts.protocol_log)

_SCHED = {"static": TS_SCHED_STATIC, "clc": TS_SCHED_CLC, "nonpersistent": TS_SCHED_NONPERSISTENT}
_TILE = {"auto": TS_TILE_AUTO, "128x128": TS_TILE_128x128, "128x256": TS_TILE_128x256,
         "256x256": TS_TILE_256x256_2CTA}
_OUT = {torch.bfloat16: TS_OUT_BF16, torch.float32: TS_OUT_F32}

EXPORTED = ("ts_gemm_bf16", "ts_gemm_bf16_ex", "ts_gemm_launch_info", "ts_gemm_bf16_checked_noalloc",
            "ts_copy_i16", "ts_spin",
            "ts_spin_wait_started", "ts_sync_and_check", "ts_num_sms", "ts_status_string",
            "ts_last_error_detail", "ts_gemm_fp8", "ts_gemm_fp8_grouped", "ts_quant_fp8", "ts_moe_route",
            "ts_moe_route_grad", "ts_moe_plan", "ts_moe_plan_workspace", "ts_moe_combine", "ts_moe_combine_grad",
            "ts_linear", "ts_linear_grad_input", "ts_linear_grad_weight", "ts_act_grad", "ts_orthogonalise",
            "ts_orthogonalise_workspace")


class TsError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{_status_name(status)}: {detail}")
        self.status = status
        self.detail = detail


class GemmOpts(ctypes.Structure):
    _fields_ = [("tile", ctypes.c_int32), ("max_workers", ctypes.c_int32), ("lda", ctypes.c_int64),
                ("ldb", ctypes.c_int64), ("ldd", ctypes.c_int64), ("timeout_s", ctypes.c_double),
                ("trace", ctypes.c_void_p), ("raster_group", ctypes.c_int32), ("split_tail", ctypes.c_int32),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64), ("skip_tiles", ctypes.c_void_p),
                ("row_sums", ctypes.c_void_p), ("epi_warps", ctypes.c_int32), ("merge", ctypes.c_int32),
                ("inputs_ready", ctypes.c_int32), ("protocol_log", ctypes.c_void_p),
                ("protocol_log_cap", ctypes.c_int32)]


class LaunchInfo(ctypes.Structure):
    _fields_ = [("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32), ("cluster", ctypes.c_int32),
                ("stages", ctypes.c_int32), ("tiles_m", ctypes.c_int64), ("tiles_n", ctypes.c_int64),
                ("num_tiles", ctypes.c_int64), ("grid_ctas", ctypes.c_int64), ("workers", ctypes.c_int64),
                ("smem_bytes", ctypes.c_int32), ("tma_store", ctypes.c_int32), ("num_units", ctypes.c_int64),
                ("split_tiles", ctypes.c_int64), ("split_parts", ctypes.c_int32), ("resident", ctypes.c_int32),
                ("workspace_bytes", ctypes.c_int64), ("epi_warps", ctypes.c_int32), ("merge", ctypes.c_int32),
                ("clc_lazy", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class RowsOpts(ctypes.Structure):
    _fields_ = [("tiles", ctypes.c_int64), ("rows_device", ctypes.c_void_p), ("skip_rows", ctypes.c_void_p),
                ("threads", ctypes.c_int32), ("max_workers", ctypes.c_int32), ("timeout_s", ctypes.c_double),
                ("trace", ctypes.c_void_p), ("chunk", ctypes.c_int64), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_int64), ("pack", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class Fp8Opts(ctypes.Structure):
    _fields_ = [("a_type", ctypes.c_int32), ("b_type", ctypes.c_int32), ("b_scale", ctypes.c_int32),
                ("trans_b", ctypes.c_int32), ("tile", ctypes.c_int32), ("max_workers", ctypes.c_int32),
                ("lda", ctypes.c_int64), ("ldb", ctypes.c_int64), ("ldd", ctypes.c_int64), ("b_group", ctypes.c_int64),
                ("sa_row", ctypes.c_int64), ("sa_blk", ctypes.c_int64), ("sb_row", ctypes.c_int64),
                ("sb_blk", ctypes.c_int64), ("sb_group", ctypes.c_int64), ("timeout_s", ctypes.c_double)]


class QuantOpts(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_void_p), ("out_rows", ctypes.c_int64), ("rows_div", ctypes.c_int32),
                ("transpose", ctypes.c_int32), ("ldx", ctypes.c_int64), ("ldq", ctypes.c_int64),
                ("s_row", ctypes.c_int64), ("s_blk", ctypes.c_int64)]


class RouteOpts(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("score", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("keep_groups", ctypes.c_int32), ("group_best", ctypes.c_int32), ("no_renorm", ctypes.c_int32),
                ("scale", ctypes.c_float), ("reserved", ctypes.c_int32), ("ldx", ctypes.c_int64),
                ("ldg", ctypes.c_int64)]


class LinearOpts(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("preact", ctypes.c_void_p),
                ("ldx", ctypes.c_int64), ("ldw", ctypes.c_int64), ("ldy", ctypes.c_int64),
                ("ld_residual", ctypes.c_int64), ("ld_preact", ctypes.c_int64), ("act", ctypes.c_int32),
                ("bias_type", ctypes.c_int32), ("tile", ctypes.c_int32), ("max_workers", ctypes.c_int32),
                ("timeout_s", ctypes.c_double)]


class LinearGradOpts(ctypes.Structure):
    _fields_ = [("aux", ctypes.c_void_p), ("ldg", ctypes.c_int64), ("ldb", ctypes.c_int64), ("ldd", ctypes.c_int64),
                ("ld_aux", ctypes.c_int64), ("act", ctypes.c_int32), ("tile", ctypes.c_int32),
                ("max_workers", ctypes.c_int32), ("reserved", ctypes.c_int32), ("timeout_s", ctypes.c_double)]


class OrthOpts(ctypes.Structure):
    _fields_ = [("steps", ctypes.c_int32), ("a", ctypes.c_float), ("b", ctypes.c_float), ("c", ctypes.c_float),
                ("eps", ctypes.c_float), ("reserved", ctypes.c_int32), ("ldg", ctypes.c_int64),
                ("ldo", ctypes.c_int64), ("g_matrix", ctypes.c_int64), ("o_matrix", ctypes.c_int64),
                ("timeout_s", ctypes.c_double)]


# The same layouts packed into bytes: a quarter of the time of filling a Structure, in calls of a few microseconds.
_PACK_FP8 = struct.Struct("6i9qd")
_PACK_QUANT = struct.Struct("Pqiiqqqq")
_PACK_ROUTE = struct.Struct("P5ifiqq")
_PACK_LINEAR = struct.Struct("3P5q4id")
_PACK_LINEAR_GRAD = struct.Struct("P4q4id")
_PACK_ORTH = struct.Struct("i4fi4qd")


class GemmProtocol(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "cluster", "stages", "tx_bytes", "full_arrivals", "empty_arrivals", "accumulators", "tmem_full_arrivals",
        "tmem_empty_arrivals", "clc_slots", "clc_full_arrivals", "clc_empty_arrivals", "clc_response_bytes",
        "epilogue_warps", "stage_bytes", "aux_empty_arrivals", "merge", "a_stage_bytes")]


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"libtsgemm.so not built ({path}); run python tile_scheduling_gb300/build.py")
    lib = ctypes.CDLL(path)
    P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.ts_gemm_bf16.argtypes = [P, P, P, I64, I64, I64, I32, I32, P]
    lib.ts_gemm_bf16_ex.argtypes = [P, P, P, I64, I64, I64, I32, I32, ctypes.POINTER(GemmOpts), P]
    lib.ts_gemm_bf16_host.argtypes = [P, P, P, P, P, P, I64, I64, I64, I32, I32, ctypes.POINTER(GemmOpts), P]
    lib.ts_gemm_launch_info.argtypes = [I64, I64, I64, I32, I32, ctypes.POINTER(GemmOpts),
                                        ctypes.POINTER(LaunchInfo)]
    lib.ts_gemm_bf16_checked_noalloc.argtypes = [P, P, P, I64, I64, I64, I32, I32, P, P]
    lib.ts_gemm_tile_coords.argtypes = [I64, I64, I64, I32, I32, ctypes.POINTER(GemmOpts), I64, I64, P, P]
    lib.ts_gemm_protocol_info.argtypes = [I32, I32, I32, I32, ctypes.POINTER(GemmProtocol)]
    lib.ts_protocol_check.argtypes = [I32, P, I32, I32, P, P, P, ctypes.c_char_p, I64, ctypes.POINTER(I64),
                                      ctypes.c_char_p, I32]
    lib.ts_protocol_check.restype = I32
    lib.ts_protocol_check_ex.argtypes = [I32, P, I32, I32, P, P, P, I32, P, ctypes.c_char_p, I64, ctypes.POINTER(I64),
                                         ctypes.c_char_p, I32]
    lib.ts_protocol_check_ex.restype = I32
    lib.ts_gemm_bf16_grouped.argtypes = [P, P, P, I64, I64, I64, P, I32, I32, ctypes.POINTER(GemmOpts), P]
    lib.ts_gemm_grouped_launch_info.argtypes = [I64, I64, I64, P, I32, I32, ctypes.POINTER(GemmOpts),
                                                ctypes.POINTER(LaunchInfo)]
    lib.ts_gemm_grouped_order.argtypes = [I64, P, P]
    lib.ts_copy_i16.argtypes = [P, P, I64, P]
    lib.ts_copy_i16_rows.argtypes = [P, P, I64, P, I64, I32, ctypes.POINTER(RowsOpts), P]
    lib.ts_copy_rows_launch_info.argtypes = [I64, I64, I32, ctypes.POINTER(RowsOpts), ctypes.POINTER(LaunchInfo)]
    lib.ts_spin.argtypes = [I32, I64, P, P]
    lib.ts_spin_wait_started.argtypes = [P, I32, ctypes.c_double]
    lib.ts_sync_and_check.argtypes = [P]
    lib.ts_num_sms.argtypes = []
    lib.ts_num_sms.restype = I32
    lib.ts_status_string.argtypes = [ctypes.c_int]
    lib.ts_status_string.restype = ctypes.c_char_p
    lib.ts_last_error_detail.argtypes = []
    lib.ts_last_error_detail.restype = ctypes.c_char_p
    F8, QO, RO = ctypes.POINTER(Fp8Opts), ctypes.POINTER(QuantOpts), ctypes.POINTER(RouteOpts)
    lib.ts_gemm_fp8.argtypes = [P, P, P, P, P, I64, I64, I64, I32, F8, P]
    lib.ts_gemm_fp8_grouped.argtypes = [P, P, P, P, P, P, I64, I64, I64, I64, I32, F8, P]
    lib.ts_quant_fp8.argtypes = [P, P, P, I64, I64, I32, I32, QO, P]
    lib.ts_moe_route.argtypes = [P, P, P, I64, I32, I32, I32, RO, P]
    lib.ts_moe_route_grad.argtypes = [P, P, P, P, I64, I32, I32, I32, RO, P]
    lib.ts_moe_plan.argtypes = [P, P, P, P, I64, I32, P, I64, P]
    lib.ts_moe_plan_workspace.argtypes = [I64, I32]
    lib.ts_moe_plan_workspace.restype = I64
    lib.ts_moe_combine.argtypes = [P, P, P, P, I64, I32, I64, I64, I32, I64, I64, P]
    lib.ts_moe_combine_grad.argtypes = [P, P, P, P, P, P, I64, I32, I64, I64, I32, I64, I64, I64, P]
    LO, LG, OO = ctypes.POINTER(LinearOpts), ctypes.POINTER(LinearGradOpts), ctypes.POINTER(OrthOpts)
    lib.ts_linear.argtypes = [P, P, P, I64, I64, I64, I32, LO, P]
    lib.ts_linear_grad_input.argtypes = [P, P, P, I64, I64, I64, I32, LG, P]
    lib.ts_linear_grad_weight.argtypes = [P, P, P, I64, I64, I64, I32, LG, P]
    lib.ts_act_grad.argtypes = [P, P, P, P, I64, I64, I32, I32, I64, I64, I64, P]
    lib.ts_orthogonalise.argtypes = [P, P, I64, I64, I64, I32, OO, P, I64, P]
    lib.ts_orthogonalise_workspace.argtypes = [I64, I64, I64, I32]
    lib.ts_orthogonalise_workspace.restype = I64
    for name in ("ts_linear", "ts_linear_grad_input", "ts_linear_grad_weight", "ts_act_grad", "ts_orthogonalise",
                 "ts_gemm_fp8", "ts_gemm_fp8_grouped", "ts_quant_fp8", "ts_moe_route", "ts_moe_route_grad",
                 "ts_moe_plan", "ts_moe_combine", "ts_moe_combine_grad", "ts_gemm_bf16", "ts_gemm_bf16_ex", "ts_gemm_launch_info", "ts_gemm_bf16_checked_noalloc",
                 "ts_gemm_tile_coords", "ts_gemm_protocol_info", "ts_gemm_bf16_grouped", "ts_gemm_grouped_launch_info",
                 "ts_gemm_grouped_order", "ts_copy_i16", "ts_copy_i16_rows", "ts_copy_rows_launch_info", "ts_spin",
                 "ts_spin_wait_started", "ts_sync_and_check"):
        getattr(lib, name).restype = ctypes.c_int
    for name in ("ts_gemm_fp8", "ts_gemm_fp8_grouped", "ts_quant_fp8", "ts_moe_route", "ts_moe_route_grad", "ts_linear",
                 "ts_linear_grad_input", "ts_linear_grad_weight", "ts_orthogonalise"):
        packed = lib[name]  # a handle of its own, whose options are packed bytes
        packed.argtypes = [P if t in (F8, QO, RO, LO, LG, OO) else t for t in getattr(lib, name).argtypes]
        packed.restype = ctypes.c_int
        setattr(lib, name + "_packed", packed)
    return lib


_lib = load_library()


def _status_name(s: int) -> str:
    return _lib.ts_status_string(s).decode()


def _check(status: int) -> None:
    if status != TS_OK:
        raise TsError(status, _lib.ts_last_error_detail().decode())


def _stream_handle(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _sched(s) -> int:
    return _SCHED[s] if isinstance(s, str) else int(s)


def _opts(tile="auto", max_workers=0, lda=0, ldb=0, ldd=0, timeout_s=0.0, trace=None, raster_group=0,
          split_tail=0, workspace=None, skip_tiles=None, row_sums=None, epi_warps=0, merge=0, inputs_ready=0,
          protocol_log=None):
    o = GemmOpts()
    o.epi_warps = int(epi_warps)
    o.merge = int(merge)
    o.inputs_ready = int(inputs_ready)
    if protocol_log is not None:
        if protocol_log.dtype != torch.int32 or not protocol_log.is_cuda or protocol_log.dim() != 3 or \
                not protocol_log.is_contiguous() or protocol_log.shape[1] != PROTOCOL_LOG_ROLES:
            raise TypeError(f"protocol_log must be a contiguous int32 CUDA tensor [CTAs][{PROTOCOL_LOG_ROLES}][cap + 1]")
        o.protocol_log = protocol_log.data_ptr()
        o.protocol_log_cap = protocol_log.shape[2] - 1
    if row_sums is not None:
        if row_sums.dtype != torch.float32 or not row_sums.is_cuda or not row_sums.is_contiguous():
            raise TypeError("row_sums must be a contiguous float32 CUDA tensor")
        o.row_sums = row_sums.data_ptr()
    if skip_tiles is not None:
        if skip_tiles.dtype not in (torch.uint8, torch.bool) or not skip_tiles.is_cuda or not skip_tiles.is_contiguous():
            raise TypeError("skip_tiles must be a contiguous uint8/bool CUDA tensor (one entry per tile)")
        o.skip_tiles = skip_tiles.data_ptr()
    o.split_tail = int(split_tail)
    if workspace is not None:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise TypeError("workspace must be a contiguous CUDA tensor")
        o.workspace = workspace.data_ptr()
        o.workspace_bytes = workspace.numel() * workspace.element_size()
    o.tile = _TILE[tile] if isinstance(tile, str) else int(tile)
    o.max_workers = int(max_workers)
    o.lda, o.ldb, o.ldd = int(lda), int(ldb), int(ldd)
    o.timeout_s = float(timeout_s)
    if trace is not None:
        if trace.dtype != torch.int64 or not trace.is_cuda or not trace.is_contiguous():
            raise TypeError("trace must be a contiguous int64 CUDA tensor")
        o.trace = trace.data_ptr()
    o.raster_group = int(raster_group)
    return o


def _matrix(t: torch.Tensor, name: str, dtype) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    if not t.is_cuda:
        raise TypeError(f"{name} must be on a CUDA device")
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be 2-D with unit column stride")
    return t.stride(0)


def _gemm_args(A, B, D):
    lda = _matrix(A, "A", torch.bfloat16)
    ldb = _matrix(B, "B", torch.bfloat16)
    if D.dtype not in _OUT:
        raise TypeError("D must be bfloat16 or float32")
    ldd = _matrix(D, "D", D.dtype)
    M, K = A.shape
    N, K2 = B.shape
    if K2 != K or tuple(D.shape) != (M, N):
        raise ValueError(f"shape mismatch: A {tuple(A.shape)}, B {tuple(B.shape)}, D {tuple(D.shape)}")
    return M, N, K, lda, ldb, ldd


_WORKSPACES: dict = {}


def workspace_for(nbytes: int, device=None, stream=None) -> torch.Tensor:
    """A zero-filled device workspace of at least ``nbytes``, cached per device and stream.

    The kernel leaves the workspace zeroed after every normal launch, so one
    buffer serves every call on a stream; calls on different streams, which may
    overlap on the GPU, get buffers of their own.  A buffer is allocated and
    zeroed on the stream it serves, so the zeroing is ordered before the
    launches that use it (``stream``: a torch stream or a raw handle; default
    the current stream)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    elif not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    key = (dev, stream.cuda_stream)
    ws = _WORKSPACES.get(key)
    if ws is None or ws.numel() < nbytes:
        with torch.cuda.stream(stream):
            ws = torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=dev)
        _WORKSPACES[key] = ws
    return ws


def ts_gemm_bf16_ex(A: torch.Tensor, B: torch.Tensor, D: torch.Tensor, sched="static", tile="auto",
                    max_workers=0, timeout_s=0.0, trace=None, raster_group=0, workspace="auto", split_tail=0,
                    skip_tiles=None, row_sums=None, epi_warps=0, merge=0, inputs_ready=0, protocol_log=None,
                    stream=None) -> None:
    """D = A @ B.T for bf16 A [M, K] and B [N, K]; D [M, N] is bf16 or fp32.

    Rows may be strided (the row stride becomes lda / ldb / ldd).  ``workspace``
    ("auto": a cached zero-filled buffer; None: no split tiles; or a CUDA tensor)
    lets the tiles that would leave the last wave partly empty be split along K.  ``epi_warps``: 4, 8,
    16 (256-column tiles) or 0 (automatic); ``merge``: 1 for the Merge barrier layout (A and B from
    separate producer warps); ``inputs_ready``: 1 when A, B and skip_tiles were final before the
    previous kernel in the stream began (their loads then overlap that kernel's tail);
    ``protocol_log``: a zeroed int32 CUDA tensor [CTAs][PROTOCOL_LOG_ROLES][cap + 1] that the
    protocol-logging build fills with every role's barrier operations (a test instrument).
    Asynchronous on ``stream`` (default: torch's current stream)."""
    M, N, K, lda, ldb, ldd = _gemm_args(A, B, D)
    lda, ldb, ldd = (lda if M > 1 else 0), (ldb if N > 1 else 0), (ldd if M > 1 else 0)
    workspace = _resolve_workspace(M, N, K, _OUT[D.dtype], sched, workspace,
                                   -1 if (skip_tiles is not None or row_sums is not None) else split_tail, tile=tile,
                                   max_workers=max_workers, lda=lda, ldb=ldb, ldd=ldd, stream=stream)
    o = _opts(tile, max_workers, lda, ldb, ldd, timeout_s, trace, raster_group, split_tail, workspace, skip_tiles,
              row_sums, epi_warps, merge, inputs_ready, protocol_log)
    _check(_lib.ts_gemm_bf16_ex(ctypes.c_void_p(A.data_ptr()), ctypes.c_void_p(B.data_ptr()),
                                ctypes.c_void_p(D.data_ptr()), M, N, K, _OUT[D.dtype], _sched(sched),
                                ctypes.byref(o), _stream_handle(stream)))


def ts_gemm_bf16_host(A_host: torch.Tensor, B_host: torch.Tensor, D_host: torch.Tensor, A: torch.Tensor,
                      B: torch.Tensor, D: torch.Tensor, sched="static", tile="auto", workspace="auto", epi_warps=0,
                      stream=None) -> None:
    """D_host = A_host @ B_host.T through the device buffers A, B, D: the copies in, the GEMM and the
    copy out are queued on ``stream`` (page-locked host tensors keep them asynchronous).  All six
    tensors are contiguous, each host tensor shaped and typed as its device one."""
    for h, d, name in ((A_host, A, "A"), (B_host, B, "B"), (D_host, D, "D")):
        if h.is_cuda or not h.is_contiguous() or not d.is_contiguous():
            raise TypeError(f"{name}_host must be a contiguous host tensor and {name} a contiguous CUDA tensor")
        if h.shape != d.shape or h.dtype != d.dtype:
            raise ValueError(f"{name}_host and {name} differ in shape or dtype")
    M, N, K, _, _, _ = _gemm_args(A, B, D)
    workspace = _resolve_workspace(M, N, K, _OUT[D.dtype], sched, workspace, 0, tile=tile, stream=stream)
    o = _opts(tile=tile, workspace=workspace, epi_warps=epi_warps)
    _check(_lib.ts_gemm_bf16_host(ctypes.c_void_p(A_host.data_ptr()), ctypes.c_void_p(B_host.data_ptr()),
                                  ctypes.c_void_p(D_host.data_ptr()), ctypes.c_void_p(A.data_ptr()),
                                  ctypes.c_void_p(B.data_ptr()), ctypes.c_void_p(D.data_ptr()), M, N, K,
                                  _OUT[D.dtype], _sched(sched), ctypes.byref(o), _stream_handle(stream)))


def ts_gemm_bf16(A: torch.Tensor, B: torch.Tensor, D: torch.Tensor, sched="static", stream=None) -> None:
    """D = A @ B.T with the default tile choice; all three tensors contiguous."""
    M, N, K, lda, ldb, ldd = _gemm_args(A, B, D)
    if (M > 1 and (lda != K or ldd != N)) or (N > 1 and ldb != K):
        raise ValueError("ts_gemm_bf16 takes dense rows; use ts_gemm_bf16_ex for strided ones")
    _check(_lib.ts_gemm_bf16(ctypes.c_void_p(A.data_ptr()), ctypes.c_void_p(B.data_ptr()),
                             ctypes.c_void_p(D.data_ptr()), M, N, K, _OUT[D.dtype], _sched(sched),
                             _stream_handle(stream)))


def ts_gemm_bf16_checked_noalloc(A: torch.Tensor, B: torch.Tensor, D: torch.Tensor, bad_tiles: torch.Tensor,
                                 sched="static", stream=None) -> None:
    """D = A @ B.T plus a tile-coverage check, without any device allocation.

    For callers that cannot call cudaMalloc: the per-tile trace lives in a
    fixed 2 MiB array inside the library (at most 65536 output tiles) rather
    than in caller memory.  ``bad_tiles`` (one int32 on the device) receives
    the number of tiles not computed exactly once.  Calls that overlap on the
    GPU share that array and race; the first call on a device should come
    before any stream capture."""
    M, N, K, lda, ldb, ldd = _gemm_args(A, B, D)
    if (M > 1 and (lda != K or ldd != N)) or (N > 1 and ldb != K):
        raise ValueError("dense rows required")
    if bad_tiles.dtype != torch.int32 or not bad_tiles.is_cuda or bad_tiles.numel() < 1:
        raise TypeError("bad_tiles must be an int32 CUDA tensor")
    _check(_lib.ts_gemm_bf16_checked_noalloc(ctypes.c_void_p(A.data_ptr()), ctypes.c_void_p(B.data_ptr()),
                                             ctypes.c_void_p(D.data_ptr()), M, N, K, _OUT[D.dtype], _sched(sched),
                                             ctypes.c_void_p(bad_tiles.data_ptr()), _stream_handle(stream)))


def ts_gemm_bf16_ptr(A: int, B: int, D: int, M: int, N: int, K: int, out: int, sched=0, stream=None,
                     **opts) -> int:  # no workspace unless one is passed
    """Raw-pointer call of ts_gemm_bf16_ex; returns the status without raising."""
    o = _opts(**opts)
    return _lib.ts_gemm_bf16_ex(ctypes.c_void_p(A), ctypes.c_void_p(B), ctypes.c_void_p(D), M, N, K, out,
                                _sched(sched), ctypes.byref(o), _stream_handle(stream))


def _launch_info_raw(M: int, N: int, K: int, out, sched, **opts) -> dict:
    o = _opts(**opts)
    info = LaunchInfo()
    _check(_lib.ts_gemm_launch_info(M, N, K, int(out), _sched(sched), ctypes.byref(o), ctypes.byref(info)))
    return {f: getattr(info, f) for f, _ in LaunchInfo._fields_}


def _resolve_workspace(M, N, K, out, sched, workspace, split_tail, stream=None, **opts):
    if not isinstance(workspace, str):
        return workspace
    if split_tail < 0:
        return None
    need = _launch_info_raw(M, N, K, out, sched, split_tail=split_tail, **opts)["workspace_bytes"]
    return workspace_for(need, stream=stream) if need > 0 else None


def ts_gemm_launch_info(M: int, N: int, K: int, out=TS_OUT_BF16, sched="static", workspace="auto", split_tail=0,
                        **opts) -> dict:
    """The launch ts_gemm_bf16_ex would make; ``workspace`` resolves as in that call."""
    ws = _resolve_workspace(M, N, K, out, sched, workspace, split_tail, **opts)
    return _launch_info_raw(M, N, K, out, sched, workspace=ws, split_tail=split_tail, **opts)


def ts_gemm_tile_coords(M: int, N: int, K: int, out=TS_OUT_BF16, sched="static", first=0, count=None, tile="auto",
                        raster_group=0):
    """(m_block, n_block) int32 arrays: the output tile that each tile id of the launch covers."""
    import numpy as np

    o = _opts(tile=tile, raster_group=raster_group)
    if count is None:
        if o.tile == TS_TILE_AUTO:  # the automatic choice depends on the device
            info = _launch_info_raw(M, N, K, out, sched, tile=tile, raster_group=raster_group)
            tiles = info["tiles_m"] * info["tiles_n"]
        else:
            bm = 256 if o.tile == TS_TILE_256x256_2CTA else 128
            bn = 128 if o.tile == TS_TILE_128x128 else 256
            tiles = -(-max(M, 0) // bm) * -(-max(N, 0) // bn)
        count = tiles - first
    mb = np.zeros(max(count, 0), dtype=np.int32)
    nb = np.zeros(max(count, 0), dtype=np.int32)
    _check(_lib.ts_gemm_tile_coords(M, N, K, int(out), _sched(sched), ctypes.byref(o), first, count,
                                    mb.ctypes.data, nb.ctypes.data))
    return mb, nb


def _offsets(k_offsets) -> "np.ndarray":
    import numpy as np

    off = np.ascontiguousarray(np.asarray(k_offsets, dtype=np.int64))
    if off.ndim != 1 or off.size < 2:
        raise ValueError("k_offsets must list groups + 1 offsets")
    return off


def ts_gemm_grouped_launch_info(M: int, N: int, k_offsets, out=TS_OUT_BF16, sched="static", **opts) -> dict:
    off = _offsets(k_offsets)
    o = _opts(**opts)
    info = LaunchInfo()
    _check(_lib.ts_gemm_grouped_launch_info(M, N, off.size - 1, off.ctypes.data, int(out), _sched(sched),
                                            ctypes.byref(o), ctypes.byref(info)))
    return {f: getattr(info, f) for f, _ in LaunchInfo._fields_}


def ts_gemm_grouped_order(k_offsets) -> "np.ndarray":
    """The order in which ts_gemm_bf16_grouped schedules the groups (longest K range first)."""
    import numpy as np

    off = _offsets(k_offsets)
    order = np.zeros(off.size - 1, dtype=np.int32)
    _check(_lib.ts_gemm_grouped_order(off.size - 1, off.ctypes.data, order.ctypes.data))
    return order


def ts_gemm_bf16_grouped(A: torch.Tensor, B: torch.Tensor, D: torch.Tensor, k_offsets, sched="static", tile="auto",
                         max_workers=0, timeout_s=0.0, trace=None, raster_group=0, skip_tiles=None,
                         row_sums=None, epi_warps=0, merge=0, inputs_ready=0, protocol_log=None,
                         stream=None) -> None:
    """D[g] = A[:, k_g:k_g+1] @ B[:, k_g:k_g+1].T for every group g (k_offsets: groups + 1 multiples of 64).

    A [M, >=K] and B [N, >=K] bf16 with unit column stride; D [groups, M, N]
    bf16 or fp32 whose groups are M * ldd elements apart."""
    off = _offsets(k_offsets)
    G = off.size - 1
    lda = _matrix(A, "A", torch.bfloat16)
    ldb = _matrix(B, "B", torch.bfloat16)
    if D.dtype not in _OUT or not D.is_cuda or D.dim() != 3 or D.stride(2) != 1:
        raise TypeError("D must be a [groups, M, N] bf16/fp32 CUDA tensor with unit column stride")
    M, N = A.shape[0], B.shape[0]
    if tuple(D.shape) != (G, M, N) or (G > 1 and D.stride(0) != M * D.stride(1)):
        raise ValueError(f"D must be [{G}, {M}, {N}] with groups M rows apart")
    if int(off[-1]) > min(A.shape[1], B.shape[1]):
        raise ValueError("k_offsets reach past the columns of A or B")
    o = _opts(tile, max_workers, lda if M > 1 else 0, ldb if N > 1 else 0, D.stride(1) if M > 1 else 0, timeout_s,
              trace, raster_group, skip_tiles=skip_tiles, row_sums=row_sums, epi_warps=epi_warps, merge=merge,
              inputs_ready=inputs_ready, protocol_log=protocol_log)
    _check(_lib.ts_gemm_bf16_grouped(ctypes.c_void_p(A.data_ptr()), ctypes.c_void_p(B.data_ptr()),
                                     ctypes.c_void_p(D.data_ptr()), M, N, G, off.ctypes.data, _OUT[D.dtype],
                                     _sched(sched), ctypes.byref(o), _stream_handle(stream)))


def ts_gemm_protocol_info(tile="256x256", out=TS_OUT_BF16, epi_warps=0, merge=0) -> dict:
    """Barrier layout and arrival counts of a kernel variant (no GPU needed)."""
    proto = GemmProtocol()
    _check(_lib.ts_gemm_protocol_info(_TILE[tile] if isinstance(tile, str) else int(tile), int(out), int(epi_warps),
                                      int(merge), ctypes.byref(proto)))
    return {f: getattr(proto, f) for f, _ in GemmProtocol._fields_}


def ts_copy_i16(src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
    """dst[i] = src[i] for contiguous int16 CUDA tensors of equal size."""
    for t, name in ((src, "src"), (dst, "dst")):
        if t.dtype != torch.int16 or not t.is_cuda or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous int16 CUDA tensor")
    if src.numel() != dst.numel():
        raise ValueError("src and dst differ in size")
    _check(_lib.ts_copy_i16(ctypes.c_void_p(src.data_ptr()), ctypes.c_void_p(dst.data_ptr()), src.numel(),
                            _stream_handle(stream)))


def ts_copy_i16_ptr(src: int, dst: int, n: int, stream=None) -> int:
    return _lib.ts_copy_i16(ctypes.c_void_p(src), ctypes.c_void_p(dst), n, _stream_handle(stream))


def _rows_opts(tiles=0, rows_device=None, skip_rows=None, threads=0, max_workers=0, timeout_s=0.0, trace=None,
               chunk=0, workspace=None, pack=0):
    o = RowsOpts()
    o.tiles = int(tiles)
    o.chunk = int(chunk)
    o.pack = int(pack)
    if workspace is not None:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise TypeError("workspace must be a contiguous CUDA tensor")
        o.workspace = workspace.data_ptr()
        o.workspace_bytes = workspace.numel() * workspace.element_size()
    o.threads = int(threads)
    o.max_workers = int(max_workers)
    o.timeout_s = float(timeout_s)
    for name, t, dtype in (("rows_device", rows_device, torch.int64), ("skip_rows", skip_rows, torch.uint8),
                           ("trace", trace, torch.int64)):
        if t is None:
            continue
        if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous {dtype} CUDA tensor")
        setattr(o, name, t.data_ptr())
    return o


def ts_copy_rows_launch_info(n: int, rows: int, sched="clc", **opts) -> dict:
    o = _rows_opts(**{k: v for k, v in opts.items() if k in ("tiles", "threads", "max_workers", "chunk", "pack")})
    info = LaunchInfo()
    _check(_lib.ts_copy_rows_launch_info(int(n), int(rows), _sched(sched), ctypes.byref(o), ctypes.byref(info)))
    return {f: getattr(info, f) for f, _ in LaunchInfo._fields_}


def ts_copy_i16_rows(src: torch.Tensor, dst: torch.Tensor, offsets: torch.Tensor, rows=None, sched="clc", tiles=0,
                     rows_device=None, skip_rows=None, threads=0, max_workers=0, timeout_s=0.0, trace=None,
                     chunk=0, workspace=None, pack=0, stream=None) -> None:
    """Copy rows [offsets[r], offsets[r+1]) of a jagged int16 array through a work queue.

    src and dst: contiguous int16 CUDA tensors of equal size n; offsets: int64
    CUDA tensor of rows + 1 entries (rows defaults to offsets.numel() - 1).
    Tiles past the row count (tiles > rows, or rows_device below rows) and rows
    marked in skip_rows copy nothing but still take part in the queue.
    chunk > 0 cuts rows into work tiles of at most chunk elements; with
    pack=1 the rows are laid end to end and every tile copies chunk of their
    elements.  The planning workspace is allocated here unless one is passed."""
    for t, name in ((src, "src"), (dst, "dst")):
        if t.dtype != torch.int16 or not t.is_cuda or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous int16 CUDA tensor")
    if src.numel() != dst.numel():
        raise ValueError("src and dst differ in size")
    if offsets.dtype != torch.int64 or not offsets.is_cuda or not offsets.is_contiguous():
        raise TypeError("offsets must be a contiguous int64 CUDA tensor")
    if rows is None:
        rows = max(offsets.numel() - 1, 0)
    if offsets.numel() < rows + 1:
        raise ValueError("offsets needs rows + 1 entries")
    if skip_rows is not None and skip_rows.numel() < rows:
        raise ValueError("skip_rows needs one byte per row")
    if chunk and workspace is None:
        need = ts_copy_rows_launch_info(src.numel(), rows, sched, tiles=tiles, chunk=chunk,
                                        pack=pack)["workspace_bytes"]
        workspace = torch.empty(need, dtype=torch.uint8, device=src.device)
    o = _rows_opts(tiles, rows_device, skip_rows, threads, max_workers, timeout_s, trace, chunk, workspace, pack)
    min_tiles = (0 if pack else int(rows)) + (-(-src.numel() // int(chunk)) if chunk else 0)
    if trace is not None and trace.numel() < 2 * max(int(tiles), min_tiles):
        raise ValueError("trace needs 2 * tiles entries")
    _check(_lib.ts_copy_i16_rows(ctypes.c_void_p(src.data_ptr()), ctypes.c_void_p(dst.data_ptr()), src.numel(),
                                 ctypes.c_void_p(offsets.data_ptr()), int(rows), _sched(sched), ctypes.byref(o),
                                 _stream_handle(stream)))


def ts_copy_i16_rows_ptr(src: int, dst: int, n: int, offsets: int, rows: int, sched=1, stream=None, **opts) -> int:
    """Raw-pointer call of ts_copy_i16_rows; returns the status without raising."""
    o = _rows_opts(**opts)
    return _lib.ts_copy_i16_rows(ctypes.c_void_p(src), ctypes.c_void_p(dst), int(n), ctypes.c_void_p(offsets),
                                 int(rows), _sched(sched), ctypes.byref(o), _stream_handle(stream))


TS_FP8_E4M3, TS_FP8_E5M2 = 0, 1
TS_SCALE_BLOCK, TS_SCALE_ROW = 0, 1
TS_SCORE_SOFTMAX, TS_SCORE_SIGMOID = 0, 1
_FP8 = {torch.float8_e4m3fn: TS_FP8_E4M3, torch.float8_e5m2: TS_FP8_E5M2}
_SCORE = {"softmax": TS_SCORE_SOFTMAX, "sigmoid": TS_SCORE_SIGMOID}


def _require(t, name: str, dtypes, dims: int) -> None:
    """Raise unless t is a CUDA tensor of one of ``dtypes`` with ``dims`` dimensions."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
        raise TypeError(f"{name} must be a tensor of {', '.join(str(d) for d in dtypes)}")
    if not t.is_cuda:
        raise TypeError(f"{name} must be on a CUDA device")
    if t.dim() != dims:
        raise ValueError(f"{name} must be {dims}-D")


_F32 = {torch.float32: 0}
_I32 = {torch.int32: 0}
_I64 = {torch.int64: 0}


def _matrix_of(t, name: str, dtypes, dims: int = 2):
    """(dtype code, shape, row stride) of a CUDA tensor with dense last dimension; the stride is 0, for
    the default, with a single row.  (Each attribute of a tensor costs some 0.1 us: no more are read than
    the checks need.)"""
    try:
        code, shape, stride, cuda = dtypes[t.dtype], t.shape, t.stride(), t.is_cuda
    except (AttributeError, KeyError, TypeError):
        cuda = False
    if not cuda or len(shape) != dims:
        _require(t, name, dtypes, dims)
    cols = shape[-1]
    if stride[-1] != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    if shape[-2] <= 1:
        return code, shape, 0
    pitch = stride[-2]
    if pitch == 0 and cols:
        raise ValueError(f"{name} has rows that share memory (an expanded tensor)")
    return code, shape, pitch


def _dense(t, name: str, dtypes, shape) -> int:
    """Address of a contiguous CUDA tensor of the given type and shape."""
    try:
        ok = t.dtype in dtypes and t.is_cuda
    except AttributeError:
        ok = False
    if not ok:
        _require(t, name, dtypes, len(shape))
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)}")
    return t.data_ptr()


def _scales(t, name: str, dims: int):
    """(shape, strides) of an fp32 scale tensor of any strides; an expanded one is broadcast along the
    dimension it is expanded in (both at once cannot be told from the default strides)."""
    try:
        ok = t.dtype is torch.float32 and t.is_cuda
        shape, stride = t.shape, t.stride()
    except (AttributeError, TypeError):
        ok = False
    if not ok or len(shape) != dims:
        _require(t, name, _F32, dims)
    if stride[-1] == 0 and stride[-2] == 0 and shape[-1] * shape[-2] > 1:
        raise ValueError(f"{name} is one scale expanded in both dimensions")
    return shape, stride


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream_of(stream) -> int:
    """The cudaStream_t of ``stream``, or of torch's current stream; the small operators below are called
    often enough that building a torch.cuda.Stream object for it each time would show."""
    if stream is None:
        if _raw_stream is not None and _raw_device is not None:
            return _raw_stream(_raw_device())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _fp8_opts(A, SA, B, SB, D, dims, trans_b, tile, max_workers, timeout_s):
    """Checks and options that the plain and the grouped 8-bit product share; returns (opts, M, N, K, out)."""
    a_type, (M, K), lda = _matrix_of(A, "A", _FP8)
    b_type, b_shape, ldb = _matrix_of(B, "B", _FP8, dims)
    out, d_shape, ldd = _matrix_of(D, "D", _OUT)
    sa_shape, sa_stride = _scales(SA, "SA", 2)
    sb_shape, sb_stride = _scales(SB, "SB", dims)
    R, C = b_shape[-2], b_shape[-1]
    N, depth = (C, R) if trans_b else (R, C)
    if depth != K or d_shape[0] != M or d_shape[1] != N:
        raise ValueError(f"shape mismatch: A {tuple(A.shape)}, B {tuple(B.shape)}, D {tuple(D.shape)}")
    kb = -(-K // 128)
    if sa_shape[0] != M or sa_shape[1] != kb:
        raise ValueError(f"SA must be [{M}, {kb}], not {tuple(SA.shape)}")
    b_scale = TS_SCALE_BLOCK
    if sb_shape[-2] != -(-R // 128) or sb_shape[-1] != -(-C // 128):
        if trans_b or dims != 2 or sb_shape[0] != N or sb_shape[1] != kb:
            raise ValueError(f"SB {tuple(SB.shape)} holds neither a scale for each 128 x 128 block of B "
                             f"{tuple(B.shape)} nor one for each row and 128 columns")
        b_scale = TS_SCALE_ROW
    b_group = sb_group = 0
    if dims == 3:
        if sb_shape[0] != b_shape[0]:
            raise ValueError(f"SB must hold the scales of {b_shape[0]} groups")
        if b_shape[0] > 1:
            b_group, sb_group = B.stride(0), sb_stride[0]
            if b_group == 0 or sb_group == 0:
                raise ValueError("groups of B or SB share memory (an expanded tensor)")
    o = _PACK_FP8.pack(a_type, b_type, b_scale, 1 if trans_b else 0,
                       _TILE[tile] if isinstance(tile, str) else int(tile), max_workers, lda, ldb, ldd, b_group,
                       sa_stride[0], sa_stride[1], sb_stride[-2], sb_stride[-1], sb_group, timeout_s)
    return o, M, N, K, out


def ts_gemm_fp8(A: torch.Tensor, SA: torch.Tensor, B: torch.Tensor, SB: torch.Tensor, D: torch.Tensor, trans_b=False,
                tile="auto", max_workers=0, timeout_s=0.0, stream=None) -> None:
    """D = (A * SA) @ (B * SB).T for 8-bit floating point A [M, K] and B [N, K]; D [M, N] is bf16 or fp32.

    SA [M, ceil(K / 128)] holds a scale for each row and 128 columns of A; SB one for each 128 x 128
    block of B ([ceil(N / 128), ceil(K / 128)]) or for each row and 128 columns ([N, ceil(K / 128)]).
    Where both shapes are the same (N = 1) the two mean the same.  Scales may have any strides; SA reads
    fastest with its rows contiguous (the transpose of a [ceil(K / 128), M] tensor).  ``trans_b``: B is
    [K, N] with block scales [ceil(K / 128), ceil(N / 128)].  Rows may be strided; rows of A and B start
    on 16-byte boundaries.  Asynchronous on ``stream`` (default: torch's current stream)."""
    o, M, N, K, out = _fp8_opts(A, SA, B, SB, D, 2, trans_b, tile, max_workers, timeout_s)
    st = _lib.ts_gemm_fp8_packed(A.data_ptr(), SA.data_ptr(), B.data_ptr(), SB.data_ptr(), D.data_ptr(), M, N, K, out,
                                 o, _stream_of(stream))
    if st:
        _check(st)


def ts_gemm_fp8_grouped(A: torch.Tensor, SA: torch.Tensor, B: torch.Tensor, SB: torch.Tensor, D: torch.Tensor,
                        offsets: torch.Tensor, trans_b=False, tile="auto", max_workers=0, timeout_s=0.0,
                        stream=None) -> None:
    """D[o_g:o_g+1] = (A * SA)[o_g:o_g+1] @ (B[g] * SB[g]).T for every group g, o = offsets (int64, on the device).

    B [groups, N, K] (``trans_b``: [groups, K, N]) with block scales SB of the same leading dimension;
    everything else as ts_gemm_fp8.  Rows outside every group are not written."""
    o, M, N, K, out = _fp8_opts(A, SA, B, SB, D, 3, trans_b, tile, max_workers, timeout_s)
    G = B.shape[0]
    st = _lib.ts_gemm_fp8_grouped_packed(A.data_ptr(), SA.data_ptr(), B.data_ptr(), SB.data_ptr(), D.data_ptr(),
                                         _dense(offsets, "offsets", _I64, (G + 1,)), G, M, N, K, out, o,
                                         _stream_of(stream))
    if st:
        _check(st)


def ts_quant_fp8(x: torch.Tensor, q: torch.Tensor, scales: torch.Tensor, rows=None, rows_div=1, transpose=False,
                 stream=None) -> None:
    """Quantise x [M, N] (bf16 or fp32) to 8-bit floating point q with one fp32 scale for each row and 128 columns of q.

    q is [M, N]; with ``rows`` (int32, on the device) [len(rows), N], row r taken from x's row
    rows[r] // rows_div (zeros for a negative entry); with ``transpose`` [N, M].  scales is
    [rows of q, ceil(columns of q / 128)] of any strides; with its rows contiguous it is what
    ts_gemm_fp8 reads fastest."""
    x_type, (M, N), ldx = _matrix_of(x, "x", _OUT)
    q_type, q_shape, ldq = _matrix_of(q, "q", _FP8)
    s_shape, s_stride = _scales(scales, "scales", 2)
    if 0 in s_stride and scales.numel() > 1:
        raise ValueError("scales share memory (an expanded tensor)")
    index, out_rows, want_r, want_c = 0, 0, M, N
    if rows is not None:
        if transpose:
            raise ValueError("rows and transpose cannot be combined")
        if rows_div < 1:
            raise ValueError("rows_div must be at least 1")
        index = _dense(rows, "rows", _I32, (rows.numel(),))
        out_rows = want_r = rows.shape[0]
    elif transpose:
        want_r, want_c = N, M
    blocks = -(-want_c // 128)
    if q_shape[0] != want_r or q_shape[1] != want_c or s_shape[0] != want_r or s_shape[1] != blocks:
        raise ValueError(f"q must be {(want_r, want_c)} and scales {(want_r, blocks)}, not {tuple(q.shape)} and "
                         f"{tuple(scales.shape)}")
    if want_r == 0:
        return
    o = _PACK_QUANT.pack(index, out_rows, int(rows_div), 1 if transpose else 0, ldx, ldq, s_stride[0], s_stride[1])
    st = _lib.ts_quant_fp8_packed(x.data_ptr(), q.data_ptr(), scales.data_ptr(), M, N, x_type, q_type, o,
                                  _stream_of(stream))
    if st:
        _check(st)


_SCALE_ZERO = 2.0 ** -150  # up to here a routing scale is 0 in fp32, as the options hold it, and 0 is the default


def _score(score) -> int:
    return _SCORE[score] if isinstance(score, str) else int(score)


def ts_moe_route(logits: torch.Tensor, experts: torch.Tensor, weights: torch.Tensor, bias=None, score="softmax",
                 groups=1, keep_groups=0, group_best=1, renorm=True, scale=1.0, stream=None) -> None:
    """Choose experts [T, k] (int32, best first) and their weights [T, k] (fp32) from logits [T, E] (bf16 or fp32).

    ``score``: "softmax" or "sigmoid"; ``bias`` [E] is added to the scores for the choice only; of
    ``groups`` equal groups of experts the ``keep_groups`` best (0: all) stay, by the sum of their
    ``group_best`` (1 or 2) best experts.  Equal values go to the lower index; an expert with logit -inf is
    never chosen, and slots without one hold -1 and weight 0.  ``renorm`` divides the weights by their sum."""
    if -_SCALE_ZERO <= scale <= _SCALE_ZERO:
        raise ValueError("scale must not be 0 in fp32")
    dtype, (T, E), ldx = _matrix_of(logits, "logits", _OUT)
    k = experts.shape[-1]
    o = _PACK_ROUTE.pack(_dense(bias, "bias", _F32, (E,)) if bias is not None else 0, _score(score), groups,
                         keep_groups, group_best, 0 if renorm else 1, scale, 0, ldx, 0)
    st = _lib.ts_moe_route_packed(logits.data_ptr(), _dense(experts, "experts", _I32, (T, k)),
                                  _dense(weights, "weights", _F32, (T, k)), T, E, k, dtype, o, _stream_of(stream))
    if st:
        _check(st)


def ts_moe_route_grad(logits: torch.Tensor, experts: torch.Tensor, grad_weights: torch.Tensor,
                      grad_logits: torch.Tensor, score="softmax", renorm=True, scale=1.0, stream=None) -> None:
    """grad_logits [T, E] (the logits' type) from grad_weights [T, k], for the experts that ts_moe_route chose."""
    if -_SCALE_ZERO <= scale <= _SCALE_ZERO:
        raise ValueError("scale must not be 0 in fp32")
    dtype, (T, E), ldx = _matrix_of(logits, "logits", _OUT)
    k = experts.shape[-1]
    g_dtype, g_shape, ldg = _matrix_of(grad_logits, "grad_logits", _OUT)
    if g_dtype != dtype:
        raise TypeError("grad_logits must have the logits' type")
    if g_shape[0] != T or g_shape[1] != E:
        raise ValueError(f"grad_logits must be {(T, E)}")
    o = _PACK_ROUTE.pack(0, _score(score), 1, 0, 1, 0 if renorm else 1, scale, 0, ldx, ldg)
    st = _lib.ts_moe_route_grad_packed(logits.data_ptr(), _dense(experts, "experts", _I32, (T, k)),
                                       _dense(grad_weights, "grad_weights", _F32, (T, k)), grad_logits.data_ptr(), T,
                                       E, k, dtype, o, _stream_of(stream))
    if st:
        _check(st)


def ts_moe_plan_workspace(slots: int, experts: int) -> int:
    """Bytes of workspace that ts_moe_plan needs for that many slots and experts."""
    return int(_lib.ts_moe_plan_workspace(int(slots), int(experts)))


@functools.lru_cache(maxsize=64)
def _plan_need(slots: int, experts: int) -> int:
    return _lib.ts_moe_plan_workspace(slots, experts)


class _Scratch(threading.local):
    def __init__(self):
        self.kept: dict = {}


_SCRATCH = _Scratch()


def _scratch_for(nbytes: int, device, stream, keep=True) -> torch.Tensor:
    """Uninitialised scratch of at least ``nbytes``, kept per device and stream and allocated on the stream
    it serves, so that calls on different streams never share one (nor do graphs, which may replay at once).
    Each thread keeps its own: a call launches several kernels that hand counts on through the scratch, and
    on a stream that threads share another's may come between them.  Without ``keep`` it is the call's own: once
    the caller drops it, torch's allocator hands it out again on the same stream, behind what was launched."""
    handle = _stream_of(stream)
    if stream is not None and handle != _stream_of(None):
        # as on that stream: whether it captures, and where memory that the call returns is used next
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(handle, device=device)
        with torch.cuda.stream(stream):
            return _scratch_for(nbytes, device, None, keep)
    if not keep or torch.cuda.is_current_stream_capturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=device)  # capturing: the graph's own
    key = (device, handle)
    ws = _SCRATCH.kept.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = _SCRATCH.kept[key] = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws


def ts_moe_plan(experts: torch.Tensor, offsets: torch.Tensor, order: torch.Tensor, position: torch.Tensor,
                workspace=None, stream=None) -> None:
    """Sort the slots of experts (int32, negative = dropped) by expert, stably.

    offsets [E + 1] (int64): the rows of each expert; order [slots] (int32): the slot of each row, -1 past
    the last; position (int32, experts' shape): the row of each slot, -1 if dropped.  The workspace that
    many slots need is one kept for each stream unless one is passed."""
    n = experts.numel()
    E = offsets.numel() - 1
    shape = experts.shape
    ptr = size = 0
    need = _plan_need(n, E)
    if need and workspace is None:
        workspace = _scratch_for(need, experts.device, stream)
    if workspace is not None:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise TypeError("workspace must be a contiguous CUDA tensor")
        ptr, size = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = _lib.ts_moe_plan(_dense(experts, "experts", _I32, shape), _dense(offsets, "offsets", _I64, (E + 1,)),
                          _dense(order, "order", _I32, (n,)), _dense(position, "position", _I32, shape), n, E, ptr,
                          size, _stream_of(stream))
    if st:
        _check(st)


def ts_moe_combine(y: torch.Tensor, position: torch.Tensor, out: torch.Tensor, weights=None, stream=None) -> None:
    """out[t] = sum_j weights[t, j] * y[position[t, j]] over the slots with position >= 0 (weights None: 1).

    y [R, N] and out [T, N] are both bf16 or both fp32; position [T, k] int32; weights [T, k] fp32."""
    dtype, (R, N), ldy = _matrix_of(y, "y", _OUT)
    o_dtype, o_shape, ldo = _matrix_of(out, "out", _OUT)
    if o_dtype != dtype:
        raise TypeError("out must have y's type")
    T, k = o_shape[0], position.shape[-1]
    if o_shape[1] != N:
        raise ValueError(f"out must be {(T, N)}")
    st = _lib.ts_moe_combine(y.data_ptr(), _dense(position, "position", _I32, (T, k)),
                             _dense(weights, "weights", _F32, (T, k)) if weights is not None else 0, out.data_ptr(), T,
                             k, N, R, dtype, ldy, ldo, _stream_of(stream))
    if st:
        _check(st)


def ts_moe_combine_grad(grad_out: torch.Tensor, y: torch.Tensor, position: torch.Tensor, weights, grad_y: torch.Tensor,
                        grad_weights=None, stream=None) -> None:
    """The gradient of ts_moe_combine: grad_y[position[t, j]] = weights[t, j] * grad_out[t] and
    grad_weights[t, j] = <grad_out[t], y[position[t, j]]>; rows of grad_y that no slot takes are not written."""
    dtype, (R, N), ldy = _matrix_of(y, "y", _OUT)
    o_dtype, o_shape, ldo = _matrix_of(grad_out, "grad_out", _OUT)
    g_dtype, g_shape, ldg = _matrix_of(grad_y, "grad_y", _OUT)
    if o_dtype != dtype or g_dtype != dtype:
        raise TypeError("grad_out and grad_y must have y's type")
    T, k = o_shape[0], position.shape[-1]
    if o_shape[1] != N or g_shape != y.shape:
        raise ValueError(f"grad_out must be {(T, N)} and grad_y {(R, N)}")
    st = _lib.ts_moe_combine_grad(grad_out.data_ptr(), y.data_ptr(), _dense(position, "position", _I32, (T, k)),
                                  _dense(weights, "weights", _F32, (T, k)) if weights is not None else 0,
                                  grad_y.data_ptr(),
                                  _dense(grad_weights, "grad_weights", _F32, (T, k)) if grad_weights is not None else 0,
                                  T, k, N, R, dtype, ldy, ldo, ldg, _stream_of(stream))
    if st:
        _check(st)


TS_ACT_NONE, TS_ACT_RELU, TS_ACT_GELU, TS_ACT_GELU_TANH, TS_ACT_SILU = range(5)
_ACT = {"none": TS_ACT_NONE, "relu": TS_ACT_RELU, "gelu": TS_ACT_GELU, "gelu_tanh": TS_ACT_GELU_TANH,
        "silu": TS_ACT_SILU}
_BF16 = {torch.bfloat16: TS_OUT_BF16}


def _device() -> int:
    """Index of the current device; on a machine without one a number that no tensor's device has."""
    try:
        return _raw_device() if _raw_device is not None else torch.cuda.current_device()
    except RuntimeError:
        return -2


def _elsewhere(t, name: str, device: int) -> None:
    if not t.is_cuda:
        raise TypeError(f"{name} must be on a CUDA device")
    raise ValueError(f"{name} lies on cuda:{t.get_device()} while the current device is cuda:{device}")


def _rows_of(t, name: str, dtypes, device: int, dims: int = 2):
    """As _matrix_of, for a tensor of the current device."""
    try:
        code, shape, stride, at = dtypes[t.dtype], t.shape, t.stride(), t.get_device()
    except (AttributeError, KeyError, TypeError):
        _require(t, name, dtypes, dims)
        raise
    if at != device:
        _elsewhere(t, name, device)
    if len(shape) != dims:
        _require(t, name, dtypes, dims)
    cols = shape[-1]
    if stride[-1] != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    if shape[-2] <= 1:
        return code, shape, 0
    pitch = stride[-2]
    if pitch == 0 and cols:
        raise ValueError(f"{name} has rows that share memory (an expanded tensor)")
    return code, shape, pitch


def _like(t, name: str, other: str, code: int, shape, device: int):
    """(address, row stride) of a matrix of the output's type and shape."""
    c, s, ld = _rows_of(t, name, _OUT, device)
    if c != code:
        raise TypeError(f"{name} must have the type of {other}")
    if s != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, not {tuple(s)}")
    return t.data_ptr(), ld


def _vector(t, name: str, dtypes, n: int, device: int) -> int:
    """Address of a dense vector of n values on the current device."""
    p = _dense(t, name, dtypes, (n,))
    if t.get_device() != device:
        _elsewhere(t, name, device)
    return p


def ts_linear(x: torch.Tensor, w: torch.Tensor, y: torch.Tensor, bias=None, act="none", residual=None, preact=None,
              tile="auto", max_workers=0, timeout_s=0.0, stream=None) -> None:
    """y = act(x @ w.T + bias) + residual for bf16 x [M, K] and w [N, K]; y [M, N] is bf16 or fp32.

    ``bias`` [N] is bf16 or fp32; ``act``: "none", "relu", "gelu", "gelu_tanh" or "silu"; ``residual``
    and ``preact`` are [M, N] of y's type, and preact receives x @ w.T + bias.  residual may be y
    itself.  Rows may be strided; rows of x and w start on 16-byte boundaries.  Asynchronous on
    ``stream`` (default: torch's current stream)."""
    device = _device()
    _, (M, K), ldx = _rows_of(x, "x", _BF16, device)
    _, (N, K2), ldw = _rows_of(w, "w", _BF16, device)
    out, shape, ldy = _rows_of(y, "y", _OUT, device)
    if K2 != K or shape[0] != M or shape[1] != N:
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, w {tuple(w.shape)}, y {tuple(y.shape)}")
    b = b_type = r = ldr = z = ldz = 0
    if bias is not None:
        b = _vector(bias, "bias", _OUT, N, device)
        b_type = _OUT[bias.dtype]
    if residual is not None:
        r, ldr = _like(residual, "residual", "y", out, shape, device)
    if preact is not None:
        z, ldz = _like(preact, "preact", "y", out, shape, device)
    o = _PACK_LINEAR.pack(b, r, z, ldx, ldw, ldy, ldr, ldz, _ACT[act] if isinstance(act, str) else int(act), b_type,
                          _TILE[tile] if isinstance(tile, str) else int(tile), max_workers, timeout_s)
    st = _lib.ts_linear_packed(x.data_ptr(), w.data_ptr(), y.data_ptr(), M, N, K, out, o, _stream_of(stream))
    if st:
        _check(st)


def ts_linear_grad_input(grad_z: torch.Tensor, w: torch.Tensor, grad_x: torch.Tensor, act="none", preact=None,
                         tile="auto", max_workers=0, timeout_s=0.0, stream=None) -> None:
    """grad_x = (grad_z @ w) * act'(preact) for bf16 grad_z [M, N] and w [N, K]; grad_x [M, K] is bf16 or fp32.

    ``act`` and ``preact`` ([M, K] of grad_x's type) are those of the layer that made this one's input;
    without them grad_x is the gradient by that input.  w is read in place."""
    device = _device()
    _, (M, N), ldg = _rows_of(grad_z, "grad_z", _BF16, device)
    _, (N2, K), ldw = _rows_of(w, "w", _BF16, device)
    out, shape, ldd = _rows_of(grad_x, "grad_x", _OUT, device)
    if N2 != N or shape[0] != M or shape[1] != K:
        raise ValueError(f"shape mismatch: grad_z {tuple(grad_z.shape)}, w {tuple(w.shape)}, grad_x {tuple(grad_x.shape)}")
    z, ldz = _like(preact, "preact", "grad_x", out, shape, device) if preact is not None else (0, 0)
    o = _PACK_LINEAR_GRAD.pack(z, ldg, ldw, ldd, ldz, _ACT[act] if isinstance(act, str) else int(act),
                               _TILE[tile] if isinstance(tile, str) else int(tile), max_workers, 0, timeout_s)
    st = _lib.ts_linear_grad_input_packed(grad_z.data_ptr(), w.data_ptr(), grad_x.data_ptr(), M, N, K, out, o,
                                          _stream_of(stream))
    if st:
        _check(st)


def ts_linear_grad_weight(grad_z: torch.Tensor, x: torch.Tensor, grad_w: torch.Tensor, base=None, tile="auto",
                          max_workers=0, timeout_s=0.0, stream=None) -> None:
    """grad_w = base + grad_z.T @ x for bf16 grad_z [M, N] and x [M, K]; grad_w [N, K] is bf16 or fp32.

    ``base`` ([N, K] of grad_w's type, which may be grad_w itself) is what has been accumulated so far."""
    device = _device()
    _, (M, N), ldg = _rows_of(grad_z, "grad_z", _BF16, device)
    _, (M2, K), ldx = _rows_of(x, "x", _BF16, device)
    out, shape, ldd = _rows_of(grad_w, "grad_w", _OUT, device)
    if M2 != M or shape[0] != N or shape[1] != K:
        raise ValueError(f"shape mismatch: grad_z {tuple(grad_z.shape)}, x {tuple(x.shape)}, grad_w {tuple(grad_w.shape)}")
    r, ldr = _like(base, "base", "grad_w", out, shape, device) if base is not None else (0, 0)
    o = _PACK_LINEAR_GRAD.pack(r, ldg, ldx, ldd, ldr, TS_ACT_NONE, _TILE[tile] if isinstance(tile, str) else int(tile),
                               max_workers, 0, timeout_s)
    st = _lib.ts_linear_grad_weight_packed(grad_z.data_ptr(), x.data_ptr(), grad_w.data_ptr(), M, N, K, out, o,
                                           _stream_of(stream))
    if st:
        _check(st)


def ts_act_grad(grad_y: torch.Tensor, preact, grad_z, grad_bias=None, act="none", stream=None) -> None:
    """grad_z = grad_y * act'(preact) and grad_bias = the sum of its rows (before rounding, fp32 [N]).

    grad_y, preact and grad_z are [M, N], all bf16 or all fp32.  preact is None with act "none"; grad_z
    may be None (the bias gradient alone), or grad_y or preact itself."""
    device = _device()
    dtype, shape, ldy = _rows_of(grad_y, "grad_y", _OUT, device)
    z, ldz = _like(preact, "preact", "grad_y", dtype, shape, device) if preact is not None else (0, 0)
    g, ldg = _like(grad_z, "grad_z", "grad_y", dtype, shape, device) if grad_z is not None else (0, 0)
    b = _vector(grad_bias, "grad_bias", _F32, shape[1], device) if grad_bias is not None else 0
    st = _lib.ts_act_grad(grad_y.data_ptr(), z, g, b, shape[0], shape[1], dtype,
                          _ACT[act] if isinstance(act, str) else int(act), ldy, ldz, ldg, _stream_of(stream))
    if st:
        _check(st)


def ts_orthogonalise_workspace(batch: int, R: int, C: int, steps: int = 5) -> int:
    """Bytes of workspace that ts_orthogonalise needs for ``batch`` matrices [R, C]."""
    return int(_lib.ts_orthogonalise_workspace(int(batch), int(R), int(C), int(steps)))


def ts_orthogonalise(g: torch.Tensor, out: torch.Tensor, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7,
                     workspace=None, timeout_s=0.0, stream=None) -> None:
    """out = the Newton-Schulz orthogonalisation of g [R, C], or of each matrix of g [batch, R, C].

    g is bf16 or fp32, out bf16 of the same shape; ``steps`` times X = a X + (b A + c A A) X with A = X X^T
    and (a, b, c) = ``coefficients``, from X = g / (norm(g) + eps).  The workspace is allocated for the call
    unless one is passed (ts_orthogonalise_workspace bytes, 256-byte aligned)."""
    dims = 3 if g.dim() == 3 else 2
    device = _device()
    g_type, shape, ldg = _rows_of(g, "g", _OUT, device, dims)
    _, o_shape, ldo = _rows_of(out, "out", _BF16, device, dims)
    if o_shape != shape:
        raise ValueError(f"out must be {tuple(shape)}, not {tuple(o_shape)}")
    steps = int(steps)
    if steps < 0:
        raise ValueError("steps must not be negative")
    if not eps > _SCALE_ZERO:
        raise ValueError("eps must be above 0 in fp32")
    a, b, c = coefficients
    if all(abs(v) <= _SCALE_ZERO for v in (a, b, c)):
        raise ValueError("the coefficients must not all be 0 in fp32")
    n, R, C = (1, *shape) if dims == 2 else shape
    gm = om = 0
    if n > 1:
        gm, om = g.stride(0), out.stride(0)
        if gm <= 0 or om <= 0:
            raise ValueError("matrices of g or out share memory (an expanded tensor)")
    need = _lib.ts_orthogonalise_workspace(n, R, C, steps)
    if need and workspace is None:
        workspace = _scratch_for(need, g.device, stream, keep=False)  # as large as some matrices, not some counts
    ptr = size = 0
    if workspace is not None:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise TypeError("workspace must be a contiguous CUDA tensor")
        if workspace.get_device() != device:
            _elsewhere(workspace, "workspace", device)
        ptr, size = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    o = _PACK_ORTH.pack(steps or -1, a, b, c, eps, 0, ldg, ldo, gm, om, timeout_s)
    st = _lib.ts_orthogonalise_packed(g.data_ptr(), out.data_ptr(), n, R, C, g_type, o, ptr, size, _stream_of(stream))
    if st:
        _check(st)


def ts_spin(ctas: int, duration_ns: int, started: torch.Tensor, stream=None) -> None:
    """Hold ``ctas`` SMs for ``duration_ns``; ``started`` is a pinned int32 host tensor."""
    if started.dtype != torch.int32 or started.is_cuda or not started.is_pinned():
        raise TypeError("started must be a pinned int32 CPU tensor")
    _check(_lib.ts_spin(int(ctas), int(duration_ns), ctypes.c_void_p(started.data_ptr()), _stream_handle(stream)))


def ts_spin_wait_started(started: torch.Tensor, expected: int, timeout_s: float = 5.0) -> None:
    _check(_lib.ts_spin_wait_started(ctypes.c_void_p(started.data_ptr()), int(expected), float(timeout_s)))


def ts_protocol_check(program, max_states: int = 20_000_000):
    """Explore a barrier-protocol program (see tile_scheduling_gb300.protocol)."""
    from .protocol import check

    return check(program, max_states)


def ts_protocol_check_ex(program, max_states: int = 20_000_000):
    """Explore a barrier-protocol program with global counters (the split tiles' handoff); the
    program's counters and their expected reductions travel with it."""
    from .protocol import check

    return check(program, max_states)


def ts_sync_and_check(stream=None) -> None:
    """Synchronise and raise TsError for a device-side timeout (or CUDA error).

    After a timeout the cached split-tile workspaces may hold partial counters,
    so they are zeroed again before the error is raised."""
    st = _lib.ts_sync_and_check(_stream_handle(stream))
    if st == TS_ERR_TIMEOUT:
        detail = _lib.ts_last_error_detail().decode()
        for ws in _WORKSPACES.values():
            ws.zero_()
        torch.cuda.synchronize()
        raise TsError(st, detail)
    _check(st)


def ts_num_sms() -> int:
    return int(_lib.ts_num_sms())


def ts_status_string(s: int) -> str:
    return _status_name(s)


def ts_last_error_detail() -> str:
    return _lib.ts_last_error_detail().decode()
