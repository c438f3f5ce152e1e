"""Thin ctypes binding over libtgemm.so (include/tgemm.h).

Argument marshalling only: every function checks tensor dtype/device/contiguity, passes
``data_ptr()`` values and the current CUDA stream to the C entry point of the same name,
and raises :class:`TgemmError` on a nonzero status.  All computation happens in the CUDA
kernels.  There is no fallback: if the shared library is missing or fails to load,
every call raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from typing import Optional

import torch

from . import build as _build

OK, EINVAL, EALIGN, ECUDA, EARCH, EWORKSPACE, ETOOLARGE = 0, -1, -2, -3, -4, -5, -6
NOALLOC_SCRATCH_BYTES = 40 * 1024 * 1024
OUT_F32, OUT_BF16 = 0, 1
OP_Q2, OP_Q2_LORA, OP_Q4 = 0, 1, 2
PATH_AUTO, PATH_SMALL_M, PATH_TENSOR, PATH_SMALL_M_PASS, PATH_SMALL_M_STREAM = 0, 1, 2, 3, 4
PACK_BAD_CODE, PACK_INEXACT, PACK_NONFINITE = 1, 2, 4
PACK_ZERO_MISMATCH, PACK_GROUP_MISMATCH = 8, 16
DEVERR_TIMEOUT = 1
ACT_NONE, ACT_SILU, ACT_GELU, ACT_GELU_TANH, ACT_RELU = range(5)
MAX_EXPERTS = 1024
KIND_TC_Q2, KIND_TC_Q2_LORA, KIND_TC_Q4, KIND_GEMV_Q2, KIND_GEMV_Q4, KIND_PREP = range(6)

_P = ctypes.c_void_p
_i = ctypes.c_int
_sz = ctypes.c_size_t

_SIGS = {
    "q2_pack": (_i, [_P, _P, _P, _P, _i, _i, _P, _P]),
    "q4_pack": (_i, [_P, _P, _P, _P, _P, _i, _i, _P, _P]),
    "q2_from_gemlite": (_i, [_P, _P, _P, _i, _i, _i, _P, _P, _P, _P]),
    "q2_dequant": (_i, [_P, _P, _P, _i, _i, _P]),
    "q4_dequant": (_i, [_P, _P, _P, _i, _i, _P]),
    "tgemm_selftest_wait_timeout": (_i, [_P]),
    "tgemm_selftest_bad_launch": (_i, [_P]),
    "tgemm_gemv_plan": (_i, [_i, _i, _i, _i, _i, _P]),
    "tgemm_mma_rate": (_i, [_i, _i, _i, _P, _i, _P]),
    "tgemm_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "tgemm_workspace_size_min": (_sz, [_i, _i, _i, _i, _i]),
    "tgemm_q2_dual_workspace_size": (_sz, [_i, _i, _i, _i]),
    "tgemm_q2_dual_workspace_size_min": (_sz, [_i, _i, _i, _i]),
    "tgemm_tc_plan": (_i, [_i, _i, _i, _i, _i, _i, _i, _P]),
    "tgemm_q2": (_i, [_P, _P, _P, _P, _i, _i, _i, _i, _P, _sz, _P]),
    "tgemm_q2_lora": (_i, [_P, _P, _P, _P, _P, _i, _P, _i, _i, _i, _i, _P, _sz, _P]),
    "tgemm_q2_lora_bt": (_i, [_P, _P, _P, _P, _P, _i, _P, _i, _i, _i, _i, _P, _sz, _P]),
    "tgemm_q4": (_i, [_P, _P, _P, _P, _i, _i, _i, _i, _P, _sz, _P]),
    "tgemm_q2_dual": (_i, [_P, _P, _P, _i, _P, _P, _P, _i, _P, _i, _i, _i, _P, _sz, _P]),
    "tgemm_q2_noalloc": (_i, [_P, _P, _P, _P, _i, _i, _i, _i, _P]),
    "tgemm_q2_ep": (_i, [_P, _P, _P, _P, _P, _i, _i, _i, _i, _P, _sz, _P]),
    "tgemm_q4_ep": (_i, [_P, _P, _P, _P, _P, _i, _i, _i, _i, _P, _sz, _P]),
    "tgemm_ep_workspace_size": (_sz, [_i, _i, _i, _i]),
    "tgemm_q2_grouped": (_i, [_P, _i, _P, _P, _P, _P, _P, _P, _i, _i, _i, _i, _i, _P, _sz, _P]),
    "tgemm_q4_grouped": (_i, [_P, _i, _P, _P, _P, _P, _P, _P, _i, _i, _i, _i, _i, _P, _sz, _P]),
    "tgemm_grouped_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "tgemm_expert_sort": (_i, [_P, _i, _i, _i, _P, _P, _P, _P, _sz, _P]),
    "tgemm_expert_sort_workspace_size": (_sz, [_i, _i, _i]),
    "tgemm_expert_combine": (_i, [_P, _i, _P, _P, _P, _i, _P, _i, _i, _i, _i, _i, _P]),
    "tgemm_strerror": (ctypes.c_char_p, [_i]),
    "tgemm_set_path": (_i, [_i]),
    "tgemm_device_error": (_i, [_P, _i]),
    "tgemm_version": (_i, []),
    "tgemm_profile_enable": (_i, [_i]),
    "tgemm_profile_read": (_i, [_i, _P, _P, _i]),
    "tgemm_launch_count": (ctypes.c_int64, []),
}


class TgemmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        try:
            msg = lib().tgemm_strerror(status).decode()
        except Exception:  # pragma: no cover - only if the library itself is unusable
            msg = "?"
        super().__init__(f"{where}: status {status} ({msg})")


_lib = None
_lock = threading.Lock()


def library_path() -> str:
    return _build.LIB


def lib():
    """Load libtgemm.so (building it first if the sources are newer)."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                path = _build.LIB
                if not os.path.exists(path) or _build.stale():
                    _build.build()
                handle = ctypes.CDLL(path)
                for name, (res, args) in _SIGS.items():
                    fn = getattr(handle, name)
                    fn.restype = res
                    fn.argtypes = args
                _lib = handle
    return _lib


def _check(status: int, where: str):
    if status != OK:
        raise TgemmError(status, where)


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, dtype, name: str):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# ---- packing ----------------------------------------------------------------------------

def q2_pack(codes: torch.Tensor, scale: torch.Tensor, status: Optional[torch.Tensor] = None):
    """codes uint8 [N, K], scale f32 [N, K/128] -> (wq uint8 [N, K/4], d f16 [N, K/128], status)."""
    _need(codes, torch.uint8, "codes")
    _need(scale, torch.float32, "scale")
    N, K = codes.shape
    wq = torch.empty((N, K // 4), dtype=torch.uint8, device=codes.device)
    d = torch.empty((N, K // 128), dtype=torch.float16, device=codes.device)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=codes.device)
    _check(lib().q2_pack(_ptr(codes), _ptr(scale), _ptr(wq), _ptr(d), N, K, _ptr(status),
                         _stream()), "q2_pack")
    return wq, d, status


def q2_from_gemlite(wq_g: torch.Tensor, scale: torch.Tensor, zero: torch.Tensor, g: int,
                    status: Optional[torch.Tensor] = None):
    """gemlite-int2 bytes uint8 [K/4, N], f32 scale and zero [N, K/g] -> Q2_0
    (wq uint8 [N, K/4], d f16 [N, K/128], status); see q2_from_gemlite in tgemm.h."""
    _need(wq_g, torch.uint8, "wq_g")
    _need(scale, torch.float32, "scale")
    _need(zero, torch.float32, "zero")
    K4, N = wq_g.shape
    K = 4 * K4
    if g < 1 or K % g or tuple(scale.shape) != (N, K // g) or tuple(zero.shape) != (N, K // g):
        raise ValueError("scale and zero must be [N, K/g]")
    wq = torch.empty((N, K4), dtype=torch.uint8, device=wq_g.device)
    d = torch.empty((N, K // 128), dtype=torch.float16, device=wq_g.device)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=wq_g.device)
    _check(lib().q2_from_gemlite(_ptr(wq_g), _ptr(scale), _ptr(zero), N, K, g, _ptr(wq), _ptr(d),
                                 _ptr(status), _stream()), "q2_from_gemlite")
    return wq, d, status


def q4_pack(codes: torch.Tensor, s: torch.Tensor, z: torch.Tensor,
            status: Optional[torch.Tensor] = None):
    """codes uint8 [N, K], s, z f32 [N, K/64] -> (wq uint8 [N, K/2], sz f16 [N, K/64, 2], status)."""
    _need(codes, torch.uint8, "codes")
    _need(s, torch.float32, "s")
    _need(z, torch.float32, "z")
    N, K = codes.shape
    wq = torch.empty((N, K // 2), dtype=torch.uint8, device=codes.device)
    sz = torch.empty((N, K // 64, 2), dtype=torch.float16, device=codes.device)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=codes.device)
    _check(lib().q4_pack(_ptr(codes), _ptr(s), _ptr(z), _ptr(wq), _ptr(sz), N, K, _ptr(status),
                         _stream()), "q4_pack")
    return wq, sz, status


def q2_dequant(wq: torch.Tensor, d: torch.Tensor) -> torch.Tensor:
    _need(wq, torch.uint8, "wq")
    _need(d, torch.float16, "d")
    N, K = wq.shape[0], wq.shape[1] * 4
    w = torch.empty((N, K), dtype=torch.float32, device=wq.device)
    _check(lib().q2_dequant(_ptr(wq), _ptr(d), _ptr(w), N, K, _stream()), "q2_dequant")
    return w


def q4_dequant(wq: torch.Tensor, sz: torch.Tensor) -> torch.Tensor:
    _need(wq, torch.uint8, "wq")
    _need(sz, torch.float16, "sz")
    N, K = wq.shape[0], wq.shape[1] * 2
    w = torch.empty((N, K), dtype=torch.float32, device=wq.device)
    _check(lib().q4_dequant(_ptr(wq), _ptr(sz), _ptr(w), N, K, _stream()), "q4_dequant")
    return w


# ---- matmuls --------------------------------------------------------------------------------

def selftest_wait_timeout() -> None:
    """Launch the failure-detection self test on the current stream: a wait that can never
    be satisfied gives up after the library's wait limit (1 s) and sets DEVERR_TIMEOUT."""
    _check(lib().tgemm_selftest_wait_timeout(_stream()), "tgemm_selftest_wait_timeout")


def workspace_size(op: int, M: int, N: int, K: int, r: int = 0) -> int:
    return int(lib().tgemm_workspace_size(op, M, N, K, r))


def workspace_size_min(op: int, M: int, N: int, K: int, r: int = 0) -> int:
    """Smallest accepted workspace (whole tiles per CTA); see tgemm_workspace_size_min."""
    return int(lib().tgemm_workspace_size_min(op, M, N, K, r))


TC_PLAN_KEYS = ("tiles_m", "num_tiles", "ksteps", "sk_t0", "upc", "dpc", "grid", "split")


def tc_plan(op: int, M: int, N: int, K: int, r: int = 0, K2: int = 0, sms: int = 148) -> dict:
    """The tensor-core kernel's schedule for these sizes on `sms` SMs (tgemm_tc_plan)."""
    out = (ctypes.c_int * len(TC_PLAN_KEYS))()
    _check(lib().tgemm_tc_plan(op, M, N, K, r, K2, sms, out), "tgemm_tc_plan")
    return dict(zip(TC_PLAN_KEYS, out))


GEMV_PLAN_KEYS = ("T", "kp", "passes", "grid", "S", "U", "j_max", "smem", "nbox", "xs_stride",
                  "off_x", "off_corr", "off_red", "off_acc", "off_sc", "off_ring", "off_bar")


def gemv_plan(fmt: int, M: int, N: int, K: int, sms: int = 148):
    """The small-M streaming kernel's launch plan (tgemm_gemv_plan), or None when no
    layout fits and the per-pass kernel serves the call."""
    out = (ctypes.c_int * len(GEMV_PLAN_KEYS))()
    st = lib().tgemm_gemv_plan(fmt, M, N, K, sms, out)
    if st == ETOOLARGE:
        return None
    _check(st, "tgemm_gemv_plan")
    return dict(zip(GEMV_PLAN_KEYS, out))


def mma_rate(mode: int, n: int = 16, iters: int = 4096) -> float:
    """Cycles per operation of tgemm_mma_rate's `mode` (averaged over the SMs)."""
    sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    out = torch.zeros(sms, dtype=torch.int64, device="cuda")
    _check(lib().tgemm_mma_rate(mode, n, iters, _ptr(out), sms, _stream()), "tgemm_mma_rate")
    torch.cuda.synchronize()
    return float(out.double().mean().item()) / iters


_ws_cache = {}


def _workspace(op, M, N, K, r, device, workspace):
    need = workspace_size(op, M, N, K, r)
    if need == 0:
        return None, 0
    if workspace is not None:
        _need(workspace, torch.uint8, "workspace")
        return workspace, workspace.numel()
    key = (device.index if device.index is not None else torch.cuda.current_device())
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < need:
        buf = torch.empty(need, dtype=torch.uint8, device=device)
        _ws_cache[key] = buf
    return buf, buf.numel()


def _out(y, M, N, out_dtype, device):
    dt = torch.float32 if out_dtype == OUT_F32 else torch.bfloat16
    if y is None:
        return torch.empty((M, N), dtype=dt, device=device)
    _need(y, dt, "y")
    if tuple(y.shape) != (M, N):
        raise ValueError(f"y must have shape {(M, N)}")
    return y


def gemm_q2(x: torch.Tensor, wq: torch.Tensor, d: torch.Tensor, *, out_dtype: int = OUT_BF16,
            y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """y = x . W^T, x bf16 [M, K], W packed Q2_0 (wq uint8 [N, K/4], d f16 [N, K/128])."""
    _need(x, torch.bfloat16, "x")
    _need(wq, torch.uint8, "wq")
    _need(d, torch.float16, "d")
    M, K = x.shape
    N = wq.shape[0]
    y = _out(y, M, N, out_dtype, x.device)
    ws, nbytes = _workspace(OP_Q2, M, N, K, 0, x.device, workspace)
    _check(lib().tgemm_q2(_ptr(x), _ptr(wq), _ptr(d), _ptr(y), M, N, K, out_dtype, _ptr(ws),
                          nbytes, _stream()), "tgemm_q2")
    return y


def gemm_q2_noalloc(x: torch.Tensor, wq: torch.Tensor, d: torch.Tensor, *,
                    out_dtype: int = OUT_BF16, y: Optional[torch.Tensor] = None):
    """gemm_q2 through tgemm_q2_noalloc: scratch comes from the library's built-in buffer.

    For callers that cannot allocate device memory (pass a preallocated ``y``).  Calls
    that overlap on the GPU share that buffer and race; see include/tgemm.h."""
    _need(x, torch.bfloat16, "x")
    _need(wq, torch.uint8, "wq")
    _need(d, torch.float16, "d")
    M, K = x.shape
    N = wq.shape[0]
    y = _out(y, M, N, out_dtype, x.device)
    _check(lib().tgemm_q2_noalloc(_ptr(x), _ptr(wq), _ptr(d), _ptr(y), M, N, K, out_dtype,
                                  _stream()), "tgemm_q2_noalloc")
    return y


def gemm_q2_lora(x, wq, d, a, b, *, out_dtype: int = OUT_BF16, y=None, workspace=None):
    """y = x . W^T + (x . A^T) . B^T with a bf16 [r, K], b bf16 [N, r]."""
    _need(x, torch.bfloat16, "x")
    _need(wq, torch.uint8, "wq")
    _need(d, torch.float16, "d")
    _need(a, torch.bfloat16, "a")
    _need(b, torch.bfloat16, "b")
    M, K = x.shape
    N = wq.shape[0]
    r = a.shape[0]
    if tuple(a.shape) != (r, K) or tuple(b.shape) != (N, r):
        raise ValueError(f"a must be [r, K] and b [N, r]; got {tuple(a.shape)}, {tuple(b.shape)}")
    y = _out(y, M, N, out_dtype, x.device)
    ws, nbytes = _workspace(OP_Q2_LORA, M, N, K, r, x.device, workspace)
    _check(lib().tgemm_q2_lora(_ptr(x), _ptr(wq), _ptr(d), _ptr(a), _ptr(b), r, _ptr(y), M, N,
                               K, out_dtype, _ptr(ws), nbytes, _stream()), "tgemm_q2_lora")
    return y


def gemm_q2_lora_bt(x, wq, d, a, bt, *, out_dtype: int = OUT_BF16, y=None, workspace=None):
    """gemm_q2_lora with B given transposed: bt bf16 [r, N] (see tgemm_q2_lora_bt)."""
    _need(x, torch.bfloat16, "x")
    _need(wq, torch.uint8, "wq")
    _need(d, torch.float16, "d")
    _need(a, torch.bfloat16, "a")
    _need(bt, torch.bfloat16, "bt")
    M, K = x.shape
    N = wq.shape[0]
    r = a.shape[0]
    if tuple(a.shape) != (r, K) or tuple(bt.shape) != (r, N):
        raise ValueError(f"a must be [r, K] and bt [r, N]; got {tuple(a.shape)}, {tuple(bt.shape)}")
    y = _out(y, M, N, out_dtype, x.device)
    ws, nbytes = _workspace(OP_Q2_LORA, M, N, K, r, x.device, workspace)
    _check(lib().tgemm_q2_lora_bt(_ptr(x), _ptr(wq), _ptr(d), _ptr(a), _ptr(bt), r, _ptr(y), M,
                                  N, K, out_dtype, _ptr(ws), nbytes, _stream()), "tgemm_q2_lora_bt")
    return y


def dual_workspace_size(M: int, N: int, K1: int, K2: int, minimum: bool = False) -> int:
    """Workspace bytes for gemm_q2_dual (fastest schedule, or the accepted minimum)."""
    fn = lib().tgemm_q2_dual_workspace_size_min if minimum else lib().tgemm_q2_dual_workspace_size
    return int(fn(M, N, K1, K2))


def gemm_q2_dual(x1, wq1, d1, x2, wq2, d2, *, out_dtype: int = OUT_BF16, y=None, workspace=None):
    """y = x1 . W1^T + x2 . W2^T: a projection split along its input axis, one kernel."""
    for t, dt, nm in ((x1, torch.bfloat16, "x1"), (wq1, torch.uint8, "wq1"), (d1, torch.float16, "d1"),
                      (x2, torch.bfloat16, "x2"), (wq2, torch.uint8, "wq2"), (d2, torch.float16, "d2")):
        _need(t, dt, nm)
    M, K1 = x1.shape
    K2 = x2.shape[1]
    N = wq1.shape[0]
    if x2.shape[0] != M or wq2.shape[0] != N:
        raise ValueError("x1/x2 must have the same tokens and W1/W2 the same rows")
    y = _out(y, M, N, out_dtype, x1.device)
    need = dual_workspace_size(M, N, K1, K2)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=x1.device)
    if workspace is not None:
        _need(workspace, torch.uint8, "workspace")
    nbytes = workspace.numel() if workspace is not None else 0
    _check(lib().tgemm_q2_dual(_ptr(x1), _ptr(wq1), _ptr(d1), K1, _ptr(x2), _ptr(wq2), _ptr(d2),
                               K2, _ptr(y), M, N, out_dtype, _ptr(workspace), nbytes, _stream()),
           "tgemm_q2_dual")
    return y


def gemm_q4(x, wq, sz, *, out_dtype: int = OUT_BF16, y=None, workspace=None):
    """y = x . W^T for 4-bit weights (wq uint8 [N, K/2], sz f16 [N, K/64, 2])."""
    _need(x, torch.bfloat16, "x")
    _need(wq, torch.uint8, "wq")
    _need(sz, torch.float16, "sz")
    M, K = x.shape
    N = wq.shape[0]
    y = _out(y, M, N, out_dtype, x.device)
    ws, nbytes = _workspace(OP_Q4, M, N, K, 0, x.device, workspace)
    _check(lib().tgemm_q4(_ptr(x), _ptr(wq), _ptr(sz), _ptr(y), M, N, K, out_dtype, _ptr(ws),
                          nbytes, _stream()), "tgemm_q4")
    return y


# ---- matmuls with an epilogue, and grouped by expert --------------------------------------------

class _Epilogue(ctypes.Structure):
    """tgemm_epilogue of tgemm.h."""
    _fields_ = [("bias", _P), ("gate", _P), ("residual", _P), ("bias_dtype", _i), ("act", _i),
                ("gate_rows", _i), ("residual_dtype", _i)]


_pack_epilogue = struct.Struct("@PPPiiii").pack  # _Epilogue's bytes
_bf16, _f16, _f32, _u8, _i32 = torch.bfloat16, torch.float16, torch.float32, torch.uint8, torch.int32
_empty_like = torch.empty_like
# a torch without CUDA has neither; every call has then refused its tensors before it needs them
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _on_device(index: int, call):
    """call() with `index` as the current device."""
    with torch.cuda.device(index):
        return call()


def _arg(t, dtype, name: str, index: int):
    """_need, and on CUDA device `index`; the pointer."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
        _need(t, dtype, name)
        raise ValueError(f"{name} must be on the same device as the first argument, got {t.device}")
    return t.data_ptr()


def _first(t, dtype, name: str) -> int:
    """_need for the argument whose device the call runs on; the device's index."""
    _need(t, dtype, name)
    return t.get_device()


def _out_code(t, name: str) -> int:
    dt = t.dtype if isinstance(t, torch.Tensor) else None
    if dt is torch.bfloat16:
        return OUT_BF16
    if dt is torch.float32:
        return OUT_F32
    raise TypeError(f"{name} must be a torch.float32 or torch.bfloat16 tensor, got {dt or type(t).__name__}")


def _c_ints(where: str, *sizes):
    """Refuses sizes that a C int does not hold (ctypes would pass their low 32 bits)."""
    if max(sizes) > 0x7FFFFFFF:
        raise TgemmError(ETOOLARGE, where)


def _shape(t: torch.Tensor, shape, name: str):
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _epilogue(bias, act, gate, residual, M, N, index, E=None):
    """Checks the epilogue's tensors; the C struct's bytes.  E is set for grouped calls."""
    pb = pg = pr = bias_dt = gate_rows = res_dt = 0
    if bias is not None:
        bias_dt = _out_code(bias, "bias")
        pb = _arg(bias, bias.dtype, "bias", index)
        _shape(bias, (N,) if E is None else (E, N), "bias")
    if gate is not None:
        pg = _arg(gate, _bf16, "gate", index)
        gate_rows = 0 if E is None and gate.dim() == 1 else 1
        _shape(gate, (M, N) if gate_rows else (N,), "gate")
    if residual is not None:
        res_dt = _out_code(residual, "residual")
        pr = _arg(residual, residual.dtype, "residual", index)
        _shape(residual, (M, N), "residual")
    return _pack_epilogue(pb, pg, pr, bias_dt, act, gate_rows, res_dt)


def _result(y, like, M, N, out_dtype, index, residual=None):
    """The output tensor (a new one, or the caller's y) and its pointer."""
    if out_dtype != OUT_BF16 and out_dtype != OUT_F32:
        raise ValueError(f"out_dtype must be OUT_F32 or OUT_BF16, got {out_dtype}")
    dt = _bf16 if out_dtype == OUT_BF16 else _f32
    if y is None:
        if residual is not None and residual.dtype is dt:  # contiguous, of y's shape
            y = _empty_like(residual)
        else:
            y = like.new_empty((M, N)) if like.dtype is dt else like.new_empty((M, N), dtype=dt)
        return y, y.data_ptr()
    ptr = _arg(y, dt, "y", index)
    _shape(y, (M, N), "y")
    return y, ptr


def _call_workspace(need: int, workspace, like, index):
    """The caller's workspace, or one of this call's own: the allocator gives it to no other
    stream or captured graph while this call may still use it.  (tensor, pointer, bytes)"""
    if workspace is not None:
        return workspace, _arg(workspace, torch.uint8, "workspace", index), workspace.numel()
    if need == 0:
        return None, None, 0
    ws = like.new_empty((need,), dtype=torch.uint8)
    return ws, ws.data_ptr(), need


def _gemm_ep(fn, op, x, wq, sc, per_byte, bias, act, gate, residual, out_dtype, y, workspace):
    index = _first(x, _bf16, "x")
    if _current_device() != index:
        return _on_device(index, lambda: _gemm_ep(fn, op, x, wq, sc, per_byte, bias, act, gate, residual, out_dtype,
                                                  y, workspace))
    pw = _arg(wq, _u8, "wq", index)
    ps = _arg(sc, _f16, "scales", index)
    if x.dim() != 2 or wq.dim() != 2:
        raise ValueError("x and wq must have two dimensions")
    M, K = x.shape
    N = wq.shape[0]
    _c_ints(fn, M, N, K)
    _shape(wq, (N, K // per_byte), "wq")
    _shape(sc, (N, K // 128) if per_byte == 4 else (N, K // 64, 2), "scales")
    ep = None
    if bias is not None or act or gate is not None or residual is not None:
        ep = _epilogue(bias, act, gate, residual, M, N, index)
    L = _lib or lib()
    y, py = _result(y, x, M, N, out_dtype, index, residual)
    if M == 0:
        return y
    ws, pws, nbytes = _call_workspace(L.tgemm_ep_workspace_size(op, M, N, K), workspace, x, index)
    st = getattr(L, fn)(x.data_ptr(), pw, ps, ep, py, M, N, K, out_dtype, pws, nbytes, _raw_stream(index))
    if st:
        raise TgemmError(st, fn)
    return y


def gemm_q2_ep(x, wq, d, *, bias=None, act: int = ACT_NONE, gate=None, residual=None,
               out_dtype: int = OUT_BF16, y=None, workspace=None):
    """y = residual + gate * act(x . W^T + bias), W packed Q2_0 (wq uint8 [N, K/4], d f16 [N, K/128]).

    bias f32 or bf16 [N]; act ACT_*; gate bf16 [N] or [M, N]; residual f32 or bf16 [M, N].  The
    epilogue is f32 with one rounding, at the store.  y may be the residual (of y's type) or a
    bf16 [M, N] gate.  An x of no rows gives an empty y.  See tgemm_epilogue in tgemm.h."""
    return _gemm_ep("tgemm_q2_ep", OP_Q2, x, wq, d, 4, bias, act, gate, residual, out_dtype, y, workspace)


def gemm_q4_ep(x, wq, sz, *, bias=None, act: int = ACT_NONE, gate=None, residual=None,
               out_dtype: int = OUT_BF16, y=None, workspace=None):
    """gemm_q2_ep for 4-bit weights (wq uint8 [N, K/2], sz f16 [N, K/64, 2])."""
    return _gemm_ep("tgemm_q4_ep", OP_Q4, x, wq, sz, 2, bias, act, gate, residual, out_dtype, y, workspace)


def _gemm_grouped(fn, op, x, wq, sc, per_byte, offsets, rows, bias, act, gate, residual, out_dtype, y, workspace):
    index = _first(x, _bf16, "x")
    if _current_device() != index:
        return _on_device(index, lambda: _gemm_grouped(fn, op, x, wq, sc, per_byte, offsets, rows, bias, act, gate,
                                                       residual, out_dtype, y, workspace))
    pw = _arg(wq, _u8, "wq", index)
    ps = _arg(sc, _f16, "scales", index)
    po = _arg(offsets, _i32, "offsets", index)
    if x.dim() != 2 or wq.dim() != 3:
        raise ValueError("x must have two dimensions and wq three")
    x_rows, K = x.shape
    E, N, kb = wq.shape
    _shape(wq, (E, N, K // per_byte), "wq")
    _shape(sc, (E, N, K // 128) if per_byte == 4 else (E, N, K // 64, 2), "scales")
    _shape(offsets, (E + 1,), "offsets")
    R, pr = x_rows, None
    if rows is not None:
        pr = _arg(rows, _i32, "rows", index)
        if rows.dim() != 1:
            raise ValueError("rows must have one dimension")
        R = rows.shape[0]
    _c_ints(fn, x_rows, R, E, N, K)
    ep = None
    if bias is not None or act or gate is not None or residual is not None:
        ep = _epilogue(bias, act, gate, residual, R, N, index, E)
    L = _lib or lib()
    y, py = _result(y, x, R, N, out_dtype, index, residual)
    if R == 0:
        return y
    ws, pws, nbytes = _call_workspace(L.tgemm_grouped_workspace_size(op, R, E, N, K), workspace, x, index)
    st = getattr(L, fn)(x.data_ptr(), x_rows, pw, ps, po, pr, ep, py, R, E, N, K, out_dtype, pws, nbytes,
                        _raw_stream(index))
    if st:
        raise TgemmError(st, fn)
    return y


def gemm_q2_grouped(x, wq, d, offsets, *, rows=None, bias=None, act: int = ACT_NONE, gate=None,
                    residual=None, out_dtype: int = OUT_BF16, y=None, workspace=None):
    """Matmul grouped by expert, Q2_0 weights: rows [offsets[e], offsets[e+1]) of y are
    residual + gate * act(xs . W_e^T + bias[e]), xs = x[rows] (or x).

    wq uint8 [E, N, K/4], d f16 [E, N, K/128], offsets int32 [E+1] on the device (as expert_sort
    gives them), rows int32 [R]; bias [E, N], gate bf16 [R, N], residual [R, N].  Rows of y behind
    the last group are left as they were; R = 0 gives an empty y.  See tgemm_q2_grouped in tgemm.h."""
    return _gemm_grouped("tgemm_q2_grouped", OP_Q2, x, wq, d, 4, offsets, rows, bias, act, gate, residual,
                         out_dtype, y, workspace)


def gemm_q4_grouped(x, wq, sz, offsets, *, rows=None, bias=None, act: int = ACT_NONE, gate=None,
                    residual=None, out_dtype: int = OUT_BF16, y=None, workspace=None):
    """gemm_q2_grouped for 4-bit weights (wq uint8 [E, N, K/2], sz f16 [E, N, K/64, 2])."""
    return _gemm_grouped("tgemm_q4_grouped", OP_Q4, x, wq, sz, 2, offsets, rows, bias, act, gate, residual,
                         out_dtype, y, workspace)


def expert_sort(ids: torch.Tensor, experts: int, *, workspace=None):
    """The plan of a grouped matmul from ids int32 [T, k] (the experts of each token).

    Returns (offsets int32 [experts+1], rows int32 [T*k], pos int32 [T, k]): expert e's sorted
    rows are [offsets[e], offsets[e+1]), rows[r] is the token of sorted row r (-1 behind the
    last), pos[t, j] the sorted row of pair (t, j) (-1 for an id outside [0, experts), whose pair
    is left out).  Pairs of one expert keep their order.  No tokens give a plan of no rows."""
    index = _first(ids, _i32, "ids")
    if _current_device() != index:
        return _on_device(index, lambda: expert_sort(ids, experts, workspace=workspace))
    if ids.dim() != 2:
        raise ValueError("ids must be [T, k]")
    if experts < 1 or experts > MAX_EXPERTS:
        raise ValueError(f"experts must be 1 to {MAX_EXPERTS}, got {experts}")
    T, k = ids.shape
    _c_ints("tgemm_expert_sort", T, k)
    L = _lib or lib()
    offsets = ids.new_empty((experts + 1,))
    rows = ids.new_empty((T * k,))
    pos = _empty_like(ids)
    if T == 0:
        return offsets.zero_(), rows, pos
    ws, pws, nbytes = _call_workspace(L.tgemm_expert_sort_workspace_size(T, k, experts), workspace, ids, index)
    _check(L.tgemm_expert_sort(ids.data_ptr(), T, k, experts, offsets.data_ptr(), rows.data_ptr(),
                               pos.data_ptr(), pws, nbytes, _raw_stream(index)), "tgemm_expert_sort")
    return offsets, rows, pos


def expert_combine(h: torch.Tensor, pos: torch.Tensor, weights: torch.Tensor, *, residual=None,
                   out_dtype: int = OUT_BF16, y=None):
    """y[t] = residual[t] + sum_j weights[t, j] * h[pos[t, j]] (pairs with pos outside [0, R) left
    out): h f32 or bf16 [R, N], pos int32 [T, k], weights f32 [T, k], residual f32 or bf16 [T, N].
    f32 sums in the order of j.  No tokens give an empty y."""
    hd = _out_code(h, "h")
    index = _first(h, h.dtype, "h")
    if _current_device() != index:
        return _on_device(index, lambda: expert_combine(h, pos, weights, residual=residual, out_dtype=out_dtype, y=y))
    pp = _arg(pos, torch.int32, "pos", index)
    pw = _arg(weights, torch.float32, "weights", index)
    if h.dim() != 2 or pos.dim() != 2:
        raise ValueError("h must be [R, N] and pos [T, k]")
    T, k = pos.shape
    R, N = h.shape
    _c_ints("tgemm_expert_combine", T, k, R, N)
    _shape(weights, (T, k), "weights")
    rd, pr = 0, None
    if residual is not None:
        rd = _out_code(residual, "residual")
        pr = _arg(residual, residual.dtype, "residual", index)
        _shape(residual, (T, N), "residual")
    y, py = _result(y, h, T, N, out_dtype, index, residual)
    if T == 0:
        return y
    _check(lib().tgemm_expert_combine(h.data_ptr(), hd, pp, pw, pr, rd, py, T, k, N, R, out_dtype,
                                      _raw_stream(index)), "tgemm_expert_combine")
    return y


# ---- control -------------------------------------------------------------------------------

def set_path(path: int) -> int:
    prev = lib().tgemm_set_path(path)
    if prev < 0:
        raise TgemmError(prev, "tgemm_set_path")
    return prev


def device_error(clear: bool = False) -> int:
    bits = ctypes.c_uint32(0)
    _check(lib().tgemm_device_error(ctypes.addressof(bits), 1 if clear else 0),
           "tgemm_device_error")
    return int(bits.value)


def version() -> int:
    return int(lib().tgemm_version())


PROFILE_ALL = (1 << 6) - 1


def profile_enable(kinds) -> int:
    """Record CUDA events around launches of the kernel kinds in the bit mask ``kinds``
    (``True`` = every kind, ``False`` = none; see tgemm_profile_enable).  Returns the
    previous mask."""
    if kinds is True:
        kinds = PROFILE_ALL
    elif kinds is False or kinds is None:
        kinds = 0
    return int(lib().tgemm_profile_enable(int(kinds)))


def profile_read(kind: int, reset: bool = True):
    """(total device ms, launches) recorded for kernel kind `kind` (KIND_*)."""
    ms = ctypes.c_double(0.0)
    n = ctypes.c_int64(0)
    _check(lib().tgemm_profile_read(kind, ctypes.addressof(ms), ctypes.addressof(n),
                                    1 if reset else 0), "tgemm_profile_read")
    return float(ms.value), int(n.value)


def launch_count() -> int:
    """Kernels launched by libtgemm.so since it was loaded."""
    return int(lib().tgemm_launch_count())
