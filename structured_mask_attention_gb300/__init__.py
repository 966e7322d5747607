"""Two-stream block-diffusion (BDLM) attention for GB300 (sm_103a).

Python binding of the C ABI in ``include/bdlm_attn.h``: every function here
has the name of the C entry point it calls and only marshals arguments
(tensor pointers, sizes, the current CUDA stream) and allocates outputs with
torch.  All computation runs in ``libbdlm_attn.so``; if the library is
missing or fails to load, every call raises.  There is no fallback path.

Layouts: Q, K, V, O, dO and gradients are ``[L, H, d]`` contiguous tensors per
stream (clean ``c``, corrupted ``n``); LSE and D are ``[H, L]`` float32.
"""
from __future__ import annotations

import ctypes
import math
import os
import re

__all__ = [
    "BdlmError", "load_library", "bdlm_workspace_size", "bdlm_attn_fwd", "bdlm_attn_fwd_shard",
    "bdlm_attn_fwd_shard_refmax", "bdlm_attn_fwd_shard_rows", "bdlm_attn_bwd_shard_rows",
    "bdlm_attn_fwd_rank", "bdlm_attn_bwd_rank",
    "bdlm_lse_merge", "bdlm_bwd_preprocess", "bdlm_attn_bwd", "bdlm_attn_bwd_noalloc", "bdlm_attn_bwd_shard",
    "bdlm_worklist", "bdlm_workspace_size_varlen", "bdlm_attn_fwd_varlen", "bdlm_attn_bwd_varlen",
    "bdlm_sync_status", "bdlm_watchdog_selftest", "bdlm_sync_status_noalloc", "bdlm_watchdog_selftest_noalloc",
    "BdlmCache", "bdlm_cache_workspace", "bdlm_workspace_size_cache", "bdlm_cache_append", "bdlm_attn_cached",
    "bdlm_cache_weights", "bdlm_cache_evict",
    "bdlm_tree_mask", "bdlm_attn_tree", "bdlm_tree_verify", "bdlm_verify_workspace", "bdlm_workspace_size_verify",
    "bdlm_cache_commit",
    "bdlm_kernel_launches", "bdlm_last_error",
    "bdlm_version", "bdlm_timing_enable", "bdlm_timing_report", "header_functions", "LIB_PATH",
    "HEADER_PATH",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libbdlm_attn.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "bdlm_attn.h")

STATUS = {0: "BDLM_OK", 1: "BDLM_ERR_INVALID_ARG", 2: "BDLM_ERR_SHAPE", 3: "BDLM_ERR_ALIGN",
          4: "BDLM_ERR_WORKSPACE", 5: "BDLM_ERR_CUDA", 6: "BDLM_ERR_UNSUPPORTED", 7: "BDLM_ERR_TIMEOUT"}
OP_FWD, OP_FWD_SHARD, OP_BWD, OP_BWD_SHARD = 0, 1, 2, 3
BF16, F32 = 0, 1


class BdlmError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


_lib = None

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I = ctypes.c_int
_F = ctypes.c_float
_SZ = ctypes.c_size_t

_SIGS = {
    "bdlm_workspace_size": (_SZ, [_I, _I64, _I64, _I, _I, _I, _I]),
    "bdlm_attn_fwd": (_I, [_P] * 6 + [_I64, _I64, _I, _I, _I, _F, _P, _P, _I, _P, _P, _P, _SZ, _P]),
    "bdlm_attn_fwd_shard": (_I, [_P] * 6 + [_I64, _I64, _I, _I, _I, _F, _I64, _I64, _I, _P, _P, _P, _P, _P,
                                            _SZ, _P]),
    "bdlm_attn_fwd_shard_refmax": (_I, [_P] * 6 + [_I64, _I64, _I, _I, _I, _F, _I64, _I64, _I, _P, _P, _P, _P, _P,
                                                   _P, _P, _SZ, _P]),
    "bdlm_lse_merge": (_I, [_I, _P, _P, _I64, _I, _I, _P, _I, _P, _P]),
    "bdlm_bwd_preprocess": (_I, [_P, _I, _P, _I64, _I, _I, _P, _P]),
    "bdlm_attn_bwd": (_I, [_P] * 12 + [_I64, _I64, _I, _I, _I, _F] + [_P] * 6 + [_I, _P, _SZ, _P]),
    "bdlm_attn_bwd_shard": (_I, [_P] * 12 + [_I64, _I64, _I, _I, _I, _F, _I64, _I64, _I] + [_P] * 6
                            + [_P, _SZ, _P]),
    "bdlm_attn_bwd_noalloc": (_I, [_P] * 12 + [_I64, _I64, _I, _I, _I, _F] + [_P] * 6 + [_I, _P]),
    "bdlm_attn_fwd_shard_rows": (_I, [_P] * 6 + [_I64, _I64, _I, _I, _I, _F, _I64, _I64, _I] + [_I64] * 4
                                 + [_P] * 5 + [_SZ, _P]),
    "bdlm_attn_bwd_shard_rows": (_I, [_P] * 12 + [_I64, _I64, _I, _I, _I, _F, _I64, _I64, _I] + [_I64] * 4
                                 + [_P] * 7 + [_SZ, _P]),
    "bdlm_attn_fwd_rank": (_I, [_P] * 6 + [_I64, _I64, _I, _I, _I, _F, _I64, _I64, _I] + [_I64] * 4
                           + [_P] * 5 + [_SZ, _P]),
    "bdlm_attn_bwd_rank": (_I, [_P] * 12 + [_I64, _I64, _I, _I, _I, _F, _I64, _I64, _I] + [_I64] * 4
                           + [_P] * 7 + [_SZ, _P]),
    "bdlm_worklist": (_I64, [_I64, _I64, _I, _I, _I, _I, _I64, _I64, _I, _P, _I64]),
    "bdlm_workspace_size_varlen": (_SZ, [_I, _P, _I, _I, _I, _I]),
    "bdlm_attn_fwd_varlen": (_I, [_P] * 6 + [_P, _I, _I64, _I, _I, _I, _F, _P, _P, _I, _P, _P, _P, _SZ, _P]),
    "bdlm_attn_bwd_varlen": (_I, [_P] * 12 + [_P, _I, _I64, _I, _I, _I, _F] + [_P] * 6 + [_I, _P, _SZ, _P]),
    "bdlm_workspace_size_cache": (_SZ, [_I, _I, _I, _I, _I64, _I64]),
    "bdlm_cache_append": (_I, [_P, _P, _P, _P, _I64, _I64, _P, _P, _SZ, _P]),
    "bdlm_attn_cached": (_I, [_P, _P, _P, _P, _P, _I64, _I64, _I, _F, _P, _I, _P, _P, _SZ, _P]),
    "bdlm_cache_weights": (_I, [_P, _P, _P, _P, _I64, _I64, _I, _F, _P, _P, _SZ, _P]),
    "bdlm_cache_evict": (_I, [_P, _P, _P, _I64, _I64, _I64, _P, _P, _P, _P, _SZ, _P]),
    "bdlm_tree_mask": (_I, [_P, _P, _P, _I64, _I64, _P, _I64, _P, _P, _SZ, _P]),
    "bdlm_attn_tree": (_I, [_P, _P, _P, _P, _I64, _P, _P, _I64, _I64, _I, _F, _P, _I, _P, _P, _SZ, _P]),
    "bdlm_workspace_size_verify": (_SZ, [_I, _I64, _I64]),
    "bdlm_tree_verify": (_I, [_P, _P, _P, _P, _I, _I64, _I64, _I64, _P, _P, _I, _P, _I64, _I64, _P, _I64, _P, _P, _P,
                              _SZ, _P]),
    "bdlm_cache_commit": (_I, [_P, _P, _P, _P, _I64, _P, _P, _I64, _I64, _P, _P, _SZ, _P]),
    "bdlm_sync_status": (_I, [_P, _P]),
    "bdlm_sync_status_noalloc": (_I, [_P]),
    "bdlm_watchdog_selftest_noalloc": (_I, [ctypes.c_uint32, _P]),
    "bdlm_watchdog_selftest": (_I, [_P, _SZ, ctypes.c_uint32, _P]),
    "bdlm_kernel_launches": (ctypes.c_uint64, []),
    "bdlm_timing_enable": (_I, [_I]),
    "bdlm_timing_report": (_I64, [ctypes.c_char_p, _I64, _I]),
    "bdlm_last_error": (ctypes.c_char_p, []),
    "bdlm_version": (ctypes.c_char_p, []),
}


def header_functions(path: str = HEADER_PATH):
    """Names of the functions declared in the C header."""
    with open(path) as fh:
        text = fh.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(bdlm_[a-z_0-9]+)\s*\(", text)))


def load_library(path: str = LIB_PATH):
    """Loads (once) and returns the native library; raises if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"native library {path} is missing; run __graft_entry__.build() "
                           "(structured_mask_attention_gb300.build.build())")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(status: int):
    if status != 0:
        raise BdlmError(status, bdlm_last_error())


def bdlm_last_error() -> str:
    return load_library().bdlm_last_error().decode()


def bdlm_version() -> str:
    return load_library().bdlm_version().decode()


def bdlm_kernel_launches() -> int:
    return int(load_library().bdlm_kernel_launches())


def bdlm_timing_enable(on: bool = True) -> None:
    """Turns per-kernel event timing (on the launching stream) on or off."""
    _check(load_library().bdlm_timing_enable(int(bool(on))))


def bdlm_timing_report(reset: bool = True) -> dict:
    """{kernel name: (launches, total_ms)} accumulated since the last reset."""
    lib = load_library()
    buf = ctypes.create_string_buffer(4096)
    n = lib.bdlm_timing_report(buf, len(buf), int(bool(reset)))
    if n < 0:
        raise BdlmError(5, "event timing failed")
    out = {}
    for line in buf.value.decode().splitlines():
        name, cnt, ms = line.split()
        out[name] = (int(cnt), float(ms))
    return out


def bdlm_workspace_size(op: int, L: int, B: int, Hq: int, Hkv: int, d: int, P: int = 1) -> int:
    return int(load_library().bdlm_workspace_size(op, L, B, Hq, Hkv, d, P))


# ----------------------------------------------------------------- torch side
def _torch():
    import torch
    return torch


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _shape(Qc, Kc):
    L, Hq, d = Qc.shape
    Hkv = Kc.shape[1]
    return L, Hq, Hkv, d


def _dt(dtype) -> int:
    torch = _torch()
    return F32 if dtype == torch.float32 else BF16


def _workspace(op, L, B, Hq, Hkv, d, device, ws):
    torch = _torch()
    need = bdlm_workspace_size(op, L, B, Hq, Hkv, d, 1)
    if ws is None:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    return ws


def _check_inputs(*ts):
    torch = _torch()
    for t in ts:
        if not t.is_cuda or not t.is_contiguous() or t.dtype != torch.bfloat16:
            raise ValueError("inputs must be contiguous bf16 CUDA tensors")


def bdlm_attn_fwd(Qc, Kc, Vc, Qn, Kn, Vn, B: int, scale: float | None = None, o_dtype=None,
                  out=None, workspace=None, stream=None):
    """O and LSE of both streams.  Returns (Oc, On, LSEc, LSEn)."""
    torch = _torch()
    _check_inputs(Qc, Kc, Vc, Qn, Kn, Vn)
    L, Hq, Hkv, d = _shape(Qc, Kc)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o_dtype = torch.bfloat16 if o_dtype is None else o_dtype
    if out is None:
        out = (torch.empty((L, Hq, d), dtype=o_dtype, device=Qc.device),
               torch.empty((L, Hq, d), dtype=o_dtype, device=Qc.device),
               torch.empty((Hq, L), dtype=torch.float32, device=Qc.device),
               torch.empty((Hq, L), dtype=torch.float32, device=Qc.device))
    Oc, On, LSEc, LSEn = out
    ws = _workspace(OP_FWD, L, B, Hq, Hkv, d, Qc.device, workspace)
    _check(load_library().bdlm_attn_fwd(
        _ptr(Qc), _ptr(Kc), _ptr(Vc), _ptr(Qn), _ptr(Kn), _ptr(Vn), L, B, Hq, Hkv, d, scale,
        _ptr(Oc), _ptr(On), _dt(Oc.dtype), _ptr(LSEc), _ptr(LSEn), _ptr(ws), ws.numel(), _stream(stream)))
    return Oc, On, LSEc, LSEn


def bdlm_attn_fwd_shard(Qc, Kc, Vc, Qn, Kn, Vn, B: int, kv_begin: int, kv_end: int, include_local: bool,
                        scale: float | None = None, out=None, workspace=None, stream=None):
    """fp32 partial (O_p, LSE_p) of both streams against clean keys
    [kv_begin, kv_end) (+ the corrupted own block if include_local).
    Returns (Op_c, Op_n, LSEp_c, LSEp_n)."""
    torch = _torch()
    _check_inputs(Qc, Kc, Vc, Qn, Kn, Vn)
    L, Hq, Hkv, d = _shape(Qc, Kc)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if out is None:
        out = (torch.empty((L, Hq, d), dtype=torch.float32, device=Qc.device),
               torch.empty((L, Hq, d), dtype=torch.float32, device=Qc.device),
               torch.empty((Hq, L), dtype=torch.float32, device=Qc.device),
               torch.empty((Hq, L), dtype=torch.float32, device=Qc.device))
    ws = _workspace(OP_FWD_SHARD, L, B, Hq, Hkv, d, Qc.device, workspace)
    _check(load_library().bdlm_attn_fwd_shard(
        _ptr(Qc), _ptr(Kc), _ptr(Vc), _ptr(Qn), _ptr(Kn), _ptr(Vn), L, B, Hq, Hkv, d, scale,
        kv_begin, kv_end, int(bool(include_local)), *[_ptr(t) for t in out], _ptr(ws), ws.numel(),
        _stream(stream)))
    return out


def bdlm_attn_fwd_shard_refmax(Qc, Kc, Vc, Qn, Kn, Vn, B: int, kv_begin: int, kv_end: int, include_local: bool,
                               Mref_c, Mref_n, scale: float | None = None, out=None, workspace=None, stream=None):
    """Verification mode of ``bdlm_attn_fwd_shard``: every row's probabilities
    are formed against the fixed reference ``Mref_c`` / ``Mref_n`` ([Hq, L]
    fp32, natural log, e.g. the unsharded forward's LSE) instead of its
    running maximum.  Returns (Op_c, Op_n, LSEp_c, LSEp_n), fp32."""
    torch = _torch()
    _check_inputs(Qc, Kc, Vc, Qn, Kn, Vn)
    L, Hq, Hkv, d = _shape(Qc, Kc)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    for t in (Mref_c, Mref_n):
        if not t.is_cuda or not t.is_contiguous() or t.dtype != torch.float32 or tuple(t.shape) != (Hq, L):
            raise ValueError("Mref must be a contiguous float32 CUDA tensor of shape [Hq, L]")
    if out is None:
        out = (torch.empty((L, Hq, d), dtype=torch.float32, device=Qc.device),
               torch.empty((L, Hq, d), dtype=torch.float32, device=Qc.device),
               torch.empty((Hq, L), dtype=torch.float32, device=Qc.device),
               torch.empty((Hq, L), dtype=torch.float32, device=Qc.device))
    ws = _workspace(OP_FWD_SHARD, L, B, Hq, Hkv, d, Qc.device, workspace)
    _check(load_library().bdlm_attn_fwd_shard_refmax(
        _ptr(Qc), _ptr(Kc), _ptr(Vc), _ptr(Qn), _ptr(Kn), _ptr(Vn), L, B, Hq, Hkv, d, scale,
        kv_begin, kv_end, int(bool(include_local)), _ptr(Mref_c), _ptr(Mref_n), *[_ptr(t) for t in out],
        _ptr(ws), ws.numel(), _stream(stream)))
    return out


def bdlm_lse_merge(O_parts, LSE_parts, o_dtype=None, out=None, lse_out=None, write_lse: bool = True,
                   stream=None):
    """Exact LSE merge of fp32 partials [rows, H, d] / [H, rows].
    Returns (O, LSE) (LSE is None when write_lse is False)."""
    torch = _torch()
    n = len(O_parts)
    rows, H, d = O_parts[0].shape
    o_dtype = torch.bfloat16 if o_dtype is None else o_dtype
    O = torch.empty((rows, H, d), dtype=o_dtype, device=O_parts[0].device) if out is None else out
    LSE = None
    if write_lse:
        LSE = torch.empty((H, rows), dtype=torch.float32, device=O_parts[0].device) if lse_out is None else lse_out
    arr_o = (ctypes.c_void_p * n)(*[t.data_ptr() for t in O_parts])
    arr_l = (ctypes.c_void_p * n)(*[t.data_ptr() for t in LSE_parts])
    _check(load_library().bdlm_lse_merge(n, ctypes.cast(arr_o, ctypes.c_void_p), ctypes.cast(arr_l, ctypes.c_void_p),
                                         rows, H, d, _ptr(O), _dt(O.dtype), _ptr(LSE), _stream(stream)))
    return O, LSE


def bdlm_bwd_preprocess(O, dO, out=None, stream=None):
    """D = rowsum(dO * O) as [H, rows] fp32."""
    torch = _torch()
    rows, H, d = O.shape
    D = torch.empty((H, rows), dtype=torch.float32, device=O.device) if out is None else out
    _check(load_library().bdlm_bwd_preprocess(_ptr(O), _dt(O.dtype), _ptr(dO), rows, H, d, _ptr(D), _stream(stream)))
    return D


def bdlm_attn_bwd(Qc, Kc, Vc, Qn, Kn, Vn, Oc, On, dOc, dOn, LSEc, LSEn, B: int, scale: float | None = None,
                  g_dtype=None, out=None, workspace=None, stream=None):
    """Gradients of both streams.  Returns (dQc, dKc, dVc, dQn, dKn, dVn)."""
    torch = _torch()
    _check_inputs(Qc, Kc, Vc, Qn, Kn, Vn, Oc, On, dOc, dOn)
    L, Hq, Hkv, d = _shape(Qc, Kc)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    g_dtype = torch.bfloat16 if g_dtype is None else g_dtype
    if out is None:
        mk = lambda H: torch.empty((L, H, d), dtype=g_dtype, device=Qc.device)
        out = (mk(Hq), mk(Hkv), mk(Hkv), mk(Hq), mk(Hkv), mk(Hkv))
    dQc, dKc, dVc, dQn, dKn, dVn = out
    ws = _workspace(OP_BWD, L, B, Hq, Hkv, d, Qc.device, workspace)
    _check(load_library().bdlm_attn_bwd(
        _ptr(Qc), _ptr(Kc), _ptr(Vc), _ptr(Qn), _ptr(Kn), _ptr(Vn), _ptr(Oc), _ptr(On), _ptr(dOc), _ptr(dOn),
        _ptr(LSEc), _ptr(LSEn), L, B, Hq, Hkv, d, scale, _ptr(dQc), _ptr(dKc), _ptr(dVc), _ptr(dQn), _ptr(dKn),
        _ptr(dVn), _dt(g_dtype), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def bdlm_attn_bwd_noalloc(Qc, Kc, Vc, Qn, Kn, Vn, Oc, On, dOc, dOn, LSEc, LSEn, B: int,
                          scale: float | None = None, g_dtype=None, out=None, stream=None,
                          check_status: bool = True):
    """bdlm_attn_bwd without a workspace argument, for callers that cannot
    allocate device memory: the library uses its own fixed-size device array
    (Hq * L <= 4194272).  With ``check_status`` (the default) the call waits
    for the stream and raises BdlmError(BDLM_ERR_TIMEOUT) if a kernel gave up
    on a device wait (``bdlm_sync_status_noalloc``); pass False to keep the
    call asynchronous and check later.  Returns (dQc, dKc, dVc, dQn, dKn, dVn)."""
    torch = _torch()
    _check_inputs(Qc, Kc, Vc, Qn, Kn, Vn, Oc, On, dOc, dOn)
    L, Hq, Hkv, d = _shape(Qc, Kc)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    g_dtype = torch.bfloat16 if g_dtype is None else g_dtype
    if out is None:
        mk = lambda H: torch.empty((L, H, d), dtype=g_dtype, device=Qc.device)
        out = (mk(Hq), mk(Hkv), mk(Hkv), mk(Hq), mk(Hkv), mk(Hkv))
    dQc, dKc, dVc, dQn, dKn, dVn = out
    _check(load_library().bdlm_attn_bwd_noalloc(
        _ptr(Qc), _ptr(Kc), _ptr(Vc), _ptr(Qn), _ptr(Kn), _ptr(Vn), _ptr(Oc), _ptr(On), _ptr(dOc), _ptr(dOn),
        _ptr(LSEc), _ptr(LSEn), L, B, Hq, Hkv, d, scale, _ptr(dQc), _ptr(dKc), _ptr(dVc), _ptr(dQn), _ptr(dKn),
        _ptr(dVn), _dt(g_dtype), _stream(stream)))
    if check_status:
        bdlm_sync_status_noalloc(stream)
    return out


def bdlm_attn_bwd_shard(Qc, Kc, Vc, Qn, Kn, Vn, dOc, dOn, LSEc, LSEn, Dc, Dn, B: int, kv_begin: int,
                        kv_end: int, include_local: bool, dQc_acc, dQn_acc, dKc, dVc, dKn, dVn,
                        scale: float | None = None, workspace=None, stream=None):
    """One shard's gradient contribution (fp32): writes dK/dV rows of the
    shard's keys, accumulates dQ into dQc_acc / dQn_acc."""
    _check_inputs(Qc, Kc, Vc, Qn, Kn, Vn, dOc, dOn)
    L, Hq, Hkv, d = _shape(Qc, Kc)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    ws = _workspace(OP_BWD_SHARD, L, B, Hq, Hkv, d, Qc.device, workspace)
    _check(load_library().bdlm_attn_bwd_shard(
        _ptr(Qc), _ptr(Kc), _ptr(Vc), _ptr(Qn), _ptr(Kn), _ptr(Vn), _ptr(dOc), _ptr(dOn), _ptr(LSEc), _ptr(LSEn),
        _ptr(Dc), _ptr(Dn), L, B, Hq, Hkv, d, scale, kv_begin, kv_end, int(bool(include_local)),
        _ptr(dQc_acc), _ptr(dQn_acc), _ptr(dKc), _ptr(dVc), _ptr(dKn), _ptr(dVn), _ptr(ws), ws.numel(),
        _stream(stream)))


def bdlm_attn_fwd_shard_rows(Qc, Kc, Vc, Qn, Kn, Vn, B: int, kv_begin: int, kv_end: int, include_local: bool,
                             rows_c, rows_n, scale: float | None = None, out=None, workspace=None, stream=None):
    """One rank's rows of the partial forward: clean rows ``rows_c`` =
    (begin, end) and corrupted rows ``rows_n``, against clean keys
    [kv_begin, kv_end) (+ the rows' own corrupted blocks if include_local).
    Only those rows of the fp32 outputs are written.  Returns
    (Op_c, Op_n, LSEp_c, LSEp_n)."""
    torch = _torch()
    _check_inputs(Qc, Kc, Vc, Qn, Kn, Vn)
    L, Hq, Hkv, d = _shape(Qc, Kc)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if out is None:
        out = (torch.zeros((L, Hq, d), dtype=torch.float32, device=Qc.device),
               torch.zeros((L, Hq, d), dtype=torch.float32, device=Qc.device),
               torch.full((Hq, L), float("-inf"), dtype=torch.float32, device=Qc.device),
               torch.full((Hq, L), float("-inf"), dtype=torch.float32, device=Qc.device))
    ws = _workspace(OP_FWD_SHARD, L, B, Hq, Hkv, d, Qc.device, workspace)
    _check(load_library().bdlm_attn_fwd_shard_rows(
        _ptr(Qc), _ptr(Kc), _ptr(Vc), _ptr(Qn), _ptr(Kn), _ptr(Vn), L, B, Hq, Hkv, d, scale,
        kv_begin, kv_end, int(bool(include_local)), int(rows_c[0]), int(rows_c[1]), int(rows_n[0]), int(rows_n[1]),
        *[_ptr(t) for t in out], _ptr(ws), ws.numel(), _stream(stream)))
    return out


def bdlm_attn_bwd_shard_rows(Qc, Kc, Vc, Qn, Kn, Vn, dOc, dOn, LSEc, LSEn, Dc, Dn, B: int, kv_begin: int,
                             kv_end: int, include_local: bool, rows_c, rows_n, dQc_acc, dQn_acc, dKc_acc, dVc_acc,
                             dKn_acc, dVn_acc, scale: float | None = None, workspace=None, stream=None):
    """One rank's rows of the sharded backward: adds the rows' dQ and their
    contributions to the call's keys' dK, dV into the fp32 accumulators."""
    _check_inputs(Qc, Kc, Vc, Qn, Kn, Vn, dOc, dOn)
    L, Hq, Hkv, d = _shape(Qc, Kc)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    ws = _workspace(OP_BWD_SHARD, L, B, Hq, Hkv, d, Qc.device, workspace)
    _check(load_library().bdlm_attn_bwd_shard_rows(
        _ptr(Qc), _ptr(Kc), _ptr(Vc), _ptr(Qn), _ptr(Kn), _ptr(Vn), _ptr(dOc), _ptr(dOn), _ptr(LSEc), _ptr(LSEn),
        _ptr(Dc), _ptr(Dn), L, B, Hq, Hkv, d, scale, kv_begin, kv_end, int(bool(include_local)),
        int(rows_c[0]), int(rows_c[1]), int(rows_n[0]), int(rows_n[1]),
        _ptr(dQc_acc), _ptr(dQn_acc), _ptr(dKc_acc), _ptr(dVc_acc), _ptr(dKn_acc), _ptr(dVn_acc),
        _ptr(ws), ws.numel(), _stream(stream)))


def _held(t, n, name):
    """A rank-local tensor must hold exactly n rows."""
    if t.shape[0] != n:
        raise ValueError(f"{name} holds {t.shape[0]} rows, the call's range has {n}")


def _ptr_held(t, spare):
    """A tensor with no rows is not read: a spare buffer stands in for its (null) address."""
    return _ptr(t) if t.numel() > 0 else _ptr(spare)


def bdlm_attn_fwd_rank(Qc, Kc, Vc, Qn, Kn, Vn, L: int, B: int, kv_begin: int, kv_end: int, include_local: bool,
                       rows_c, rows_n, scale: float | None = None, out=None, workspace=None, stream=None):
    """One rank's rows with rank-local tensors: Qc holds clean rows
    ``rows_c`` = (begin, end) only, Qn / Kn / Vn the corrupted rows
    ``rows_n`` only, Kc / Vc the clean keys [kv_begin, kv_end) only; L is the
    full length.  Returns the partial (Op_c, Op_n, LSEp_c, LSEp_n) of those
    rows (fp32, [rows, Hq, d] and [Hq, rows])."""
    torch = _torch()
    _check_inputs(Qc, Kc, Vc, Qn, Kn, Vn)
    nc, nn = rows_c[1] - rows_c[0], rows_n[1] - rows_n[0]
    for t, n, name in ((Qc, nc, "Qc"), (Qn, nn, "Qn"), (Kn, nn, "Kn"), (Vn, nn, "Vn"),
                       (Kc, kv_end - kv_begin, "Kc"), (Vc, kv_end - kv_begin, "Vc")):
        _held(t, n, name)
    Hq, d, Hkv = Qc.shape[1], Qc.shape[2], Kn.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    dev = Qc.device
    if out is None:
        out = (torch.zeros((nc, Hq, d), dtype=torch.float32, device=dev),
               torch.zeros((nn, Hq, d), dtype=torch.float32, device=dev),
               torch.full((Hq, nc), float("-inf"), dtype=torch.float32, device=dev),
               torch.full((Hq, nn), float("-inf"), dtype=torch.float32, device=dev))
    ws = _workspace(OP_FWD_SHARD, L, B, Hq, Hkv, d, dev, workspace)
    spare = torch.empty(256, dtype=torch.uint8, device=dev)
    _check(load_library().bdlm_attn_fwd_rank(
        *[_ptr_held(t, spare) for t in (Qc, Kc, Vc, Qn, Kn, Vn)], L, B, Hq, Hkv, d, scale, kv_begin, kv_end,
        int(bool(include_local)), int(rows_c[0]), int(rows_c[1]), int(rows_n[0]), int(rows_n[1]),
        *[_ptr_held(t, spare) for t in out], _ptr(ws), ws.numel(), _stream(stream)))
    return out


def bdlm_attn_bwd_rank(Qc, Kc, Vc, Qn, Kn, Vn, dOc, dOn, LSEc, LSEn, Dc, Dn, L: int, B: int, kv_begin: int,
                       kv_end: int, include_local: bool, rows_c, rows_n, dQc_acc, dQn_acc, dKc_acc, dVc_acc,
                       dKn_acc, dVn_acc, scale: float | None = None, workspace=None, stream=None):
    """One rank's rows of the backward with rank-local tensors (as
    bdlm_attn_fwd_rank; LSE, D of its rows as [Hq, rows]): adds the rows' dQ
    and their contributions to the call's keys' dK, dV into the fp32
    accumulators ([rows, Hq, d] for dQ, [keys, Hkv, d] for dK / dV)."""
    torch = _torch()
    _check_inputs(Qc, Kc, Vc, Qn, Kn, Vn, dOc, dOn)
    nc, nn, nk = rows_c[1] - rows_c[0], rows_n[1] - rows_n[0], kv_end - kv_begin
    for t, n, name in ((Qc, nc, "Qc"), (dOc, nc, "dOc"), (dQc_acc, nc, "dQc_acc"), (Qn, nn, "Qn"), (Kn, nn, "Kn"),
                       (Vn, nn, "Vn"), (dOn, nn, "dOn"), (dQn_acc, nn, "dQn_acc"), (dKn_acc, nn, "dKn_acc"),
                       (dVn_acc, nn, "dVn_acc"), (Kc, nk, "Kc"), (Vc, nk, "Vc"), (dKc_acc, nk, "dKc_acc"),
                       (dVc_acc, nk, "dVc_acc")):
        _held(t, n, name)
    Hq, d, Hkv = Qc.shape[1], Qc.shape[2], Kn.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    dev = Qc.device
    ws = _workspace(OP_BWD_SHARD, L, B, Hq, Hkv, d, dev, workspace)
    spare = torch.empty(256, dtype=torch.uint8, device=dev)
    ts = (Qc, Kc, Vc, Qn, Kn, Vn, dOc, dOn, LSEc, LSEn, Dc, Dn)
    acc = (dQc_acc, dQn_acc, dKc_acc, dVc_acc, dKn_acc, dVn_acc)
    _check(load_library().bdlm_attn_bwd_rank(
        *[_ptr_held(t, spare) for t in ts], L, B, Hq, Hkv, d, scale, kv_begin, kv_end, int(bool(include_local)),
        int(rows_c[0]), int(rows_c[1]), int(rows_n[0]), int(rows_n[1]), *[_ptr_held(t, spare) for t in acc],
        _ptr(ws), ws.numel(), _stream(stream)))


def bdlm_worklist(L: int, B: int, Hq: int, Hkv: int, tile_q: int = 256, tile_k: int = 128,
                  kv_begin: int = 0, kv_end: int | None = None, include_local: bool = True):
    """The forward work list as a list of 8-tuples (host only, no GPU)."""
    kv_end = L if kv_end is None else kv_end
    lib = load_library()
    n = lib.bdlm_worklist(L, B, Hq, Hkv, tile_q, tile_k, kv_begin, kv_end, int(include_local), None, 0)
    if n < 0:
        raise BdlmError(2, "invalid work-list shape")
    buf = (ctypes.c_int32 * (8 * n))()
    lib.bdlm_worklist(L, B, Hq, Hkv, tile_q, tile_k, kv_begin, kv_end, int(include_local),
                      ctypes.cast(buf, ctypes.c_void_p), n)
    return [tuple(buf[8 * i:8 * i + 8]) for i in range(n)]


def _offsets(seq_lens):
    """Host int64 array of the n + 1 row offsets of packed sequences."""
    lens = [int(x) for x in seq_lens]
    arr = (ctypes.c_int64 * (len(lens) + 1))()
    acc = 0
    for i, n in enumerate(lens):
        arr[i] = acc
        acc += n
    arr[len(lens)] = acc
    return arr, len(lens), acc


def bdlm_workspace_size_varlen(op: int, seq_lens, Hq: int, Hkv: int, d: int) -> int:
    arr, n, _ = _offsets(seq_lens)
    return load_library().bdlm_workspace_size_varlen(op, ctypes.cast(arr, ctypes.c_void_p), n, Hq, Hkv, d)


def _workspace_varlen(op, seq_lens, Hq, Hkv, d, device, ws):
    torch = _torch()
    need = bdlm_workspace_size_varlen(op, seq_lens, Hq, Hkv, d)
    if ws is None:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    return ws


def bdlm_attn_fwd_varlen(Qc, Kc, Vc, Qn, Kn, Vn, seq_lens, B: int, scale: float | None = None, o_dtype=None,
                         out=None, workspace=None, stream=None):
    """Packed batch: sequences of the given lengths stored back to back along
    the token dimension ([T, H, d], T = sum of the lengths).  Returns
    (Oc, On, LSEc, LSEn) with LSE as [Hq, T]."""
    torch = _torch()
    _check_inputs(Qc, Kc, Vc, Qn, Kn, Vn)
    T, Hq, Hkv, d = _shape(Qc, Kc)
    arr, n, tot = _offsets(seq_lens)
    if tot != T:
        raise ValueError(f"sequence lengths sum to {tot}, tensors hold {T} rows")
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o_dtype = torch.bfloat16 if o_dtype is None else o_dtype
    if out is None:
        out = (torch.empty((T, Hq, d), dtype=o_dtype, device=Qc.device),
               torch.empty((T, Hq, d), dtype=o_dtype, device=Qc.device),
               torch.empty((Hq, T), dtype=torch.float32, device=Qc.device),
               torch.empty((Hq, T), dtype=torch.float32, device=Qc.device))
    Oc, On, LSEc, LSEn = out
    ws = _workspace_varlen(OP_FWD, seq_lens, Hq, Hkv, d, Qc.device, workspace)
    _check(load_library().bdlm_attn_fwd_varlen(
        _ptr(Qc), _ptr(Kc), _ptr(Vc), _ptr(Qn), _ptr(Kn), _ptr(Vn), ctypes.cast(arr, ctypes.c_void_p), n, B,
        Hq, Hkv, d, scale, _ptr(Oc), _ptr(On), _dt(Oc.dtype), _ptr(LSEc), _ptr(LSEn), _ptr(ws), ws.numel(),
        _stream(stream)))
    return Oc, On, LSEc, LSEn


def bdlm_attn_bwd_varlen(Qc, Kc, Vc, Qn, Kn, Vn, Oc, On, dOc, dOn, LSEc, LSEn, seq_lens, B: int,
                         scale: float | None = None, g_dtype=None, out=None, workspace=None, stream=None):
    """Gradients of a packed batch.  Returns (dQc, dKc, dVc, dQn, dKn, dVn)."""
    torch = _torch()
    _check_inputs(Qc, Kc, Vc, Qn, Kn, Vn, dOc, dOn)
    T, Hq, Hkv, d = _shape(Qc, Kc)
    arr, n, tot = _offsets(seq_lens)
    if tot != T:
        raise ValueError(f"sequence lengths sum to {tot}, tensors hold {T} rows")
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    g_dtype = torch.bfloat16 if g_dtype is None else g_dtype
    if out is None:
        mk = lambda H: torch.empty((T, H, d), dtype=g_dtype, device=Qc.device)
        out = (mk(Hq), mk(Hkv), mk(Hkv), mk(Hq), mk(Hkv), mk(Hkv))
    dQc, dKc, dVc, dQn, dKn, dVn = out
    ws = _workspace_varlen(OP_BWD, seq_lens, Hq, Hkv, d, Qc.device, workspace)
    _check(load_library().bdlm_attn_bwd_varlen(
        _ptr(Qc), _ptr(Kc), _ptr(Vc), _ptr(Qn), _ptr(Kn), _ptr(Vn), _ptr(Oc), _ptr(On), _ptr(dOc), _ptr(dOn),
        _ptr(LSEc), _ptr(LSEn), ctypes.cast(arr, ctypes.c_void_p), n, B, Hq, Hkv, d, scale,
        _ptr(dQc), _ptr(dKc), _ptr(dVc), _ptr(dQn), _ptr(dKn), _ptr(dVn), _dt(dQc.dtype), _ptr(ws), ws.numel(),
        _stream(stream)))
    return out


# ------------------------------------------------------------ 8-bit cache
class _CacheStruct(ctypes.Structure):
    _fields_ = [("k8", _P), ("v8", _P), ("k_scale", _P), ("v_scale", _P), ("page_table", _P), ("lens", _P),
                ("n_pages", _I64), ("n_seqs", _I), ("max_pages", _I), ("page", _I), ("Hkv", _I), ("d", _I)]


class BdlmCache:
    """A paged 8-bit cache over the caller's tensors, checked once here:

    ``k8``, ``v8`` [n_pages, Hkv, page, d] torch.float8_e4m3fn (codes);
    ``k_scale``, ``v_scale`` [n_pages, Hkv] float32 (value = code * scale);
    ``page_table`` [n_seqs, max_pages] int32; ``lens`` [n_seqs] int32.

    The handle keeps the tensors; update ``page_table`` and ``lens`` in place
    (``copy_``), or make a new handle for other tensors.

    The calls on it share these arguments:

    ``row_offsets`` [n_seqs + 1] int32 on the device (sequence s owns rows
    ``row_offsets[s]`` to ``row_offsets[s + 1]``), or None: equally many rows each.
    ``max_rows``: the most rows of any sequence.  Give it with ``row_offsets``: the
    host does not read them and would take all rows for it, which is right but
    slow (64 single tokens then run in the kernels for long blocks).
    ``workspace`` from ``bdlm_cache_workspace``; without one the call makes its own
    and drops it, and with it what ``bdlm_sync_status`` would report: expired waits
    and page ids, lengths or offsets out of range.
    ``stream`` (default: the current one of the cache's device): tensors that the
    call makes are ordered behind the current stream; inputs, given outputs and a
    given workspace are the caller's to order and to keep alive."""
    __slots__ = ("k8", "v8", "k_scale", "v_scale", "page_table", "lens", "device", "n_pages", "n_seqs", "max_pages",
                 "page", "Hkv", "d", "_struct", "_ref")

    def __init__(self, k8, v8, k_scale, v_scale, page_table, lens):
        torch = _torch()
        if k8.dim() != 4 or page_table.dim() != 2:
            raise ValueError("k8 must be [n_pages, Hkv, page, d], page_table [n_seqs, max_pages]")
        n_pages, Hkv, page, d = k8.shape
        n_seqs, max_pages = page_table.shape
        for name, t, dtype, shape in (("k8", k8, torch.float8_e4m3fn, (n_pages, Hkv, page, d)),
                                      ("v8", v8, torch.float8_e4m3fn, (n_pages, Hkv, page, d)),
                                      ("k_scale", k_scale, torch.float32, (n_pages, Hkv)),
                                      ("v_scale", v_scale, torch.float32, (n_pages, Hkv)),
                                      ("page_table", page_table, torch.int32, (n_seqs, max_pages)),
                                      ("lens", lens, torch.int32, (n_seqs,))):
            _check_tensor(name, t, dtype, shape, k8.device)
            object.__setattr__(self, name, t)
        set_ = lambda name, v: object.__setattr__(self, name, v)
        for name, v in (("device", k8.device), ("n_pages", n_pages), ("n_seqs", n_seqs), ("max_pages", max_pages),
                        ("page", page), ("Hkv", Hkv), ("d", d)):
            set_(name, v)
        set_("_struct", _CacheStruct(*(t.data_ptr() for t in (k8, v8, k_scale, v_scale, page_table, lens)),
                                     n_pages, n_seqs, max_pages, page, Hkv, d))
        set_("_ref", ctypes.cast(ctypes.pointer(self._struct), _P))

    def __setattr__(self, name, value):
        raise AttributeError("a BdlmCache is fixed: update its tensors in place or make a new handle")


def _check_tensor(name, t, dtype, shape, device):
    if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)} on {device} (a CUDA "
                         f"device), not {t.dtype} {list(t.shape)} on {t.device}"
                         f"{'' if t.is_contiguous() else ', not contiguous'}")


def _cache_rows(cache, row_offsets, max_rows, T):
    """(row_offsets pointer, max_rows) of a call on T packed rows."""
    if row_offsets is None:
        if max_rows is None:
            if T % cache.n_seqs:
                raise ValueError(f"{T} rows are not a multiple of n_seqs = {cache.n_seqs}: give row_offsets")
            max_rows = T // cache.n_seqs
        return None, max_rows
    _check_tensor("row_offsets", row_offsets, _torch().int32, (cache.n_seqs + 1,), cache.device)
    return row_offsets.data_ptr(), max(T, 1) if max_rows is None else max_rows


def _cache_call(fn, cache, stream, args, tensors=()):
    """Calls an entry point with the current (or given) stream of the cache's device appended; `tensors` made by this
    call are marked as used on a given stream."""
    torch = _torch()
    cuda = torch.cuda
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(cache.device.index)  # (torch.cuda.current_stream costs 2 us a call)
    else:
        if stream.device != cache.device:
            raise ValueError(f"the stream is on {stream.device}, the cache on {cache.device}")
        raw = stream.cuda_stream
        if tensors:
            # made on the current stream, where their memory may have had other users: the call waits for those
            stream.wait_stream(cuda.current_stream(cache.device))
            for t in tensors:
                t.record_stream(stream)
    if cuda.current_device() == cache.device.index:
        status = fn(*args, raw)
    else:
        with cuda.device(cache.device):
            status = fn(*args, raw)
    if status:
        _check(status)


def bdlm_workspace_size_cache(n_seqs: int, Hq: int, Hkv: int, d: int, max_rows: int, keep: int = 0) -> int:
    return int(load_library().bdlm_workspace_size_cache(n_seqs, Hq, Hkv, d, max_rows, keep))


def bdlm_cache_workspace(cache, Hq: int = 0, max_rows: int = 0, keep: int = 0):
    """A zeroed workspace for every call on ``cache``: attention of at most
    ``max_rows`` new rows per sequence with ``Hq`` query heads, evictions to at
    most ``keep`` tokens.  One call at a time uses it; make one per stream and
    one per captured graph that may run beside others."""
    torch = _torch()
    n = bdlm_workspace_size_cache(cache.n_seqs, Hq, cache.Hkv, cache.d, max_rows, keep)
    if not n:
        raise ValueError(f"no workspace for Hq={Hq}, max_rows={max_rows}, keep={keep} on this cache")
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=cache.device)


def _cache_workspace(cache, ws, made, need):
    if ws is None:
        # the kernels' part is written before it is read; only the header has to be zero
        ws = _torch().empty(need, dtype=_torch().uint8, device=cache.device)
        ws[:256].zero_()
        made.append(ws)
    elif ws.device != cache.device:
        raise ValueError(f"the workspace is on {ws.device}, the cache on {cache.device}")
    elif not ws.is_contiguous():  # (a view's elements may be more than its memory)
        raise ValueError("the workspace must be contiguous")
    return ws


def bdlm_cache_append(cache, K, V, row_offsets=None, max_rows: int | None = None, lens_out=None, workspace=None,
                      stream=None):
    """Quantises the new tokens' K, V [rows, Hkv, d] (bf16) into the pages of
    their sequences, behind ``cache.lens`` tokens (which stays as it is).
    Returns ``lens_out`` [n_seqs] int32 = lens + rows; copy it into
    ``cache.lens`` once the sequences have grown."""
    torch = _torch()
    T = K.shape[0]
    _check_tensor("K", K, torch.bfloat16, (T, cache.Hkv, cache.d), cache.device)
    _check_tensor("V", V, torch.bfloat16, (T, cache.Hkv, cache.d), cache.device)
    off, max_rows = _cache_rows(cache, row_offsets, max_rows, T)
    made = []
    if lens_out is None:
        lens_out = torch.empty(cache.n_seqs, dtype=torch.int32, device=cache.device)
        made.append(lens_out)
    else:
        _check_tensor("lens_out", lens_out, torch.int32, (cache.n_seqs,), cache.device)
    ws = _cache_workspace(cache, workspace, made, 256)
    _cache_call(load_library().bdlm_cache_append, cache, stream,
                (K.data_ptr(), V.data_ptr(), cache._ref, off, T, max_rows, lens_out.data_ptr(), ws.data_ptr(),
                 ws.nbytes), made)
    return lens_out


def bdlm_attn_cached(Qn, Kn, Vn, cache, row_offsets=None, max_rows: int | None = None, scale: float | None = None,
                     o_dtype=None, out=None, workspace=None, stream=None):
    """Attention of packed new rows (Qn [rows, Hq, d]; Kn, Vn [rows, Hkv, d],
    or both None for the cached tokens alone) to their sequence's cached
    tokens and their own block.  Returns (O [rows, Hq, d], LSE [Hq, rows])."""
    if (Kn is None) != (Vn is None):
        raise ValueError("Kn and Vn: give both or neither")
    return _cached_attention(load_library().bdlm_attn_cached, Qn, Kn, Vn, (), cache, row_offsets, max_rows, scale, o_dtype,
                             out, workspace, stream)


def _cached_attention(fn, Qn, Kn, Vn, mask, cache, row_offsets, max_rows, scale, o_dtype, out, workspace, stream):
    """What bdlm_attn_cached and bdlm_attn_tree share; ``mask``: what the call takes behind Vn."""
    torch = _torch()
    T, Hq, d = Qn.shape
    _check_tensor("Qn", Qn, torch.bfloat16, (T, Hq, cache.d), cache.device)
    if Kn is not None:
        _check_tensor("Kn", Kn, torch.bfloat16, (T, cache.Hkv, cache.d), cache.device)
        _check_tensor("Vn", Vn, torch.bfloat16, (T, cache.Hkv, cache.d), cache.device)
    off, max_rows = _cache_rows(cache, row_offsets, max_rows, T)
    made = []
    if out is None:
        # (torch.empty costs about half of Tensor.new_empty, 1.6 against 2.8 us: a token's call is bound by its host time)
        O = torch.empty((T, Hq, d), dtype=torch.bfloat16 if o_dtype is None else o_dtype, device=cache.device)
        LSE = torch.empty((Hq, T), dtype=torch.float32, device=cache.device)
        made += [O, LSE]
    else:
        O, LSE = out
        _check_tensor("O", O, O.dtype if o_dtype is None else o_dtype, (T, Hq, d), cache.device)
        _check_tensor("LSE", LSE, torch.float32, (Hq, T), cache.device)
    if O.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"O must be bfloat16 or float32, not {O.dtype}")
    ws = _cache_workspace(cache, workspace, made,
                          max(bdlm_workspace_size_cache(cache.n_seqs, Hq, cache.Hkv, d, max_rows), 256)
                          if workspace is None else 0)
    _cache_call(fn, cache, stream,
                (Qn.data_ptr(), None if Kn is None else Kn.data_ptr(), None if Vn is None else Vn.data_ptr(), *mask, cache._ref,
                 off, T, max_rows, Hq, 1.0 / math.sqrt(d) if scale is None else scale, O.data_ptr(),
                 F32 if O.dtype == torch.float32 else BF16, LSE.data_ptr(), ws.data_ptr(), ws.nbytes), made)
    return O, LSE


def bdlm_cache_weights(Qn, LSE, cache, weights, row_offsets=None, max_rows: int | None = None,
                       scale: float | None = None, workspace=None, stream=None):
    """Adds to ``weights`` [n_seqs, Hkv, max_pages * page] float32 the attention
    weight that every cached token receives from the rows (their LSE [Hq,
    rows] from ``bdlm_attn_cached``).  Returns ``weights``."""
    torch = _torch()
    T, Hq, d = Qn.shape
    _check_tensor("Qn", Qn, torch.bfloat16, (T, Hq, cache.d), cache.device)
    _check_tensor("LSE", LSE, torch.float32, (Hq, T), cache.device)
    _check_tensor("weights", weights, torch.float32, (cache.n_seqs, cache.Hkv, cache.max_pages * cache.page),
                  cache.device)
    off, max_rows = _cache_rows(cache, row_offsets, max_rows, T)
    made = []
    ws = _cache_workspace(cache, workspace, made, 256)
    _cache_call(load_library().bdlm_cache_weights, cache, stream,
                (Qn.data_ptr(), LSE.data_ptr(), cache._ref, off, T, max_rows, Hq,
                 1.0 / math.sqrt(d) if scale is None else scale, weights.data_ptr(), ws.data_ptr(), ws.nbytes), made)
    return weights


def bdlm_cache_evict(cache, weights, dst_table, keep: int, sinks: int = 0, recent: int = 0, lens_out=None,
                     weights_out=None, kept=None, workspace=None, stream=None):
    """Cuts every sequence back to at most ``keep`` tokens per KV head (the
    first ``sinks``, the last ``recent``, and those of largest weight), moved
    to the pages of ``dst_table`` [n_seqs, max_pages].  Returns (lens_out,
    weights_out, kept); kept [n_seqs, Hkv, keep] int32 holds the old
    positions, -1 behind the last."""
    torch = _torch()
    shape = (cache.n_seqs, cache.Hkv, cache.max_pages * cache.page)
    _check_tensor("weights", weights, torch.float32, shape, cache.device)
    _check_tensor("dst_table", dst_table, torch.int32, (cache.n_seqs, cache.max_pages), cache.device)
    made = []
    new = lambda s, dt: made.append(torch.empty(s, dtype=dt, device=cache.device)) or made[-1]
    lens_out = new((cache.n_seqs,), torch.int32) if lens_out is None else lens_out
    weights_out = new(shape, torch.float32) if weights_out is None else weights_out
    if kept is None:
        kept = new((cache.n_seqs, cache.Hkv, max(int(keep), 0)), torch.int32)
    _check_tensor("lens_out", lens_out, torch.int32, (cache.n_seqs,), cache.device)
    _check_tensor("weights_out", weights_out, torch.float32, shape, cache.device)
    _check_tensor("kept", kept, torch.int32, (cache.n_seqs, cache.Hkv, max(int(keep), 0)), cache.device)
    ws = _cache_workspace(cache, workspace, made, 256)
    _cache_call(load_library().bdlm_cache_evict, cache, stream,
                (cache._ref, weights.data_ptr(), dst_table.data_ptr(), keep, sinks, recent, lens_out.data_ptr(),
                 weights_out.data_ptr(), kept.data_ptr() or None, ws.data_ptr(), ws.nbytes), made)
    return lens_out, weights_out, kept


# --------------------------------------------------------- drafted tokens
def _tree_words(visible, T, device):
    if visible.dim() != 2:
        raise ValueError(f"visible must be [rows, words], not {list(visible.shape)}")
    _check_tensor("visible", visible, _torch().int32, (T, visible.shape[1]), device)
    return visible.shape[1]


def bdlm_tree_mask(cache, parents, row_offsets=None, max_rows: int | None = None, out=None, workspace=None, stream=None):
    """What the rows of drafted trees see.  ``parents`` [rows] int32: the row of
    its own sequence that a row follows, one before it, or -1.  Returns (visible
    [rows, ceil(max_rows / 32)] int32, bit j % 32 of word j / 32: the row sees row j
    of its sequence, an ancestor or itself; positions [rows] int32, ``cache.lens`` plus
    the number of ancestors).  A tree has at most 4096 rows: give ``max_rows`` where
    there are more in all (and to keep the words few)."""
    torch = _torch()
    T = parents.shape[0]
    _check_tensor("parents", parents, torch.int32, (T,), cache.device)
    off, max_rows = _cache_rows(cache, row_offsets, max_rows, T)
    made = []
    if out is None:
        visible = torch.empty((T, max(1, (max_rows + 31) // 32)), dtype=torch.int32, device=cache.device)
        positions = torch.empty(T, dtype=torch.int32, device=cache.device)
        made += [visible, positions]
    else:
        visible, positions = out
        _check_tensor("positions", positions, torch.int32, (T,), cache.device)
    words = _tree_words(visible, T, cache.device)
    ws = _cache_workspace(cache, workspace, made, 256)
    _cache_call(load_library().bdlm_tree_mask, cache, stream,
                (parents.data_ptr(), cache._ref, off, T, max_rows, visible.data_ptr(), words, positions.data_ptr(),
                 ws.data_ptr(), ws.nbytes), made)
    return visible, positions


def bdlm_attn_tree(Qn, Kn, Vn, visible, cache, row_offsets=None, max_rows: int | None = None,
                   scale: float | None = None, o_dtype=None, out=None, workspace=None, stream=None):
    """``bdlm_attn_cached`` with own rows that see only those of their sequence whose
    bit is set in ``visible`` [rows, words] int32 (from ``bdlm_tree_mask``, or any other
    pattern), and all its cached tokens.  Returns (O [rows, Hq, d], LSE [Hq, rows])."""
    if Kn is None or Vn is None:
        raise ValueError("Kn and Vn: a tree's rows see themselves, give both")
    words = _tree_words(visible, Qn.shape[0], cache.device)
    return _cached_attention(load_library().bdlm_attn_tree, Qn, Kn, Vn, (visible.data_ptr(), words), cache, row_offsets,
                             max_rows, scale, o_dtype, out, workspace, stream)


def bdlm_workspace_size_verify(n_seqs: int, max_rows: int, V: int) -> int:
    return int(load_library().bdlm_workspace_size_verify(n_seqs, max_rows, V))


def bdlm_verify_workspace(n_seqs: int, max_rows: int, V: int, device="cuda"):
    """A zeroed workspace for ``bdlm_tree_verify``; one call at a time uses it."""
    n = bdlm_workspace_size_verify(n_seqs, max_rows, V)
    if not n:
        raise ValueError(f"no workspace for n_seqs={n_seqs}, max_rows={max_rows}, V={V}")
    return _torch().zeros(n, dtype=_torch().uint8, device=device)


def _check_probs(name, t, dtype, shape, device):
    """The row stride of a [rows, V] tensor whose rows lie apart, each side by side."""
    if t.shape == shape and t.dtype is dtype and t.device == device and t.is_cuda:
        row, one = t.stride()
        if (one == 1 or shape[1] == 1) and (row >= shape[1] or shape[0] < 2):
            return row if shape[0] > 1 else shape[1]
    raise ValueError(f"{name} must be a {dtype} tensor of shape {list(shape)} on {device} (a CUDA device) with rows that lie "
                     f"apart and values side by side, not {t.dtype} {list(t.shape)} of strides {list(t.stride())} on {t.device}")


def bdlm_tree_verify(parents, tokens, target, draft, uniforms, sample, row_offsets=None, max_rows: int | None = None,
                     max_path: int | None = None, out=None, workspace=None, stream=None):
    """Tests drafted trees against the target's probabilities, from given random numbers.

    ``parents``, ``tokens`` [rows] int32; ``target`` [rows, V] float32 or bfloat16: row i
    the target's probabilities of the token behind row i (a row's values side by side, rows
    any stride apart); ``draft`` of the same type and shape: the drafter's probabilities
    that the children of row i were drawn from, or None: they were chosen, not drawn;
    ``uniforms`` [rows] and ``sample`` [n_seqs] float32 in [0, 1).  Row 0 of a sequence is
    its last token.  ``max_path``: the most rows of a path (default: max_rows).

    Returns (path [n_seqs, max_path] int32, the accepted rows of each sequence and -1
    behind them; accepted [n_seqs] int32, how many; next_token [n_seqs] int32, drawn so
    that the tokens follow the target's distribution).  ``row_offsets``, ``max_rows``,
    ``workspace`` (from ``bdlm_verify_workspace``) and ``stream`` as in the calls on a cache."""
    torch = _torch()
    T, n, device, dtype = parents.shape[0], sample.shape[0], target.device, target.dtype
    if dtype is not torch.float32 and dtype is not torch.bfloat16:
        raise ValueError(f"target must be float32 or bfloat16, not {dtype}")
    if target.dim() != 2:
        raise ValueError(f"target must be [rows, V], not {list(target.shape)}")
    shape = (T, target.shape[1])
    row_t = row_d = _check_probs("target", target, dtype, shape, device)
    if draft is not None:
        row_d = _check_probs("draft", draft, dtype, shape, device)
    _check_tensor("parents", parents, torch.int32, (T,), device)
    _check_tensor("tokens", tokens, torch.int32, (T,), device)
    _check_tensor("uniforms", uniforms, torch.float32, (T,), device)
    _check_tensor("sample", sample, torch.float32, (n,), device)
    like = _Batch(n, device)
    off, max_rows = _cache_rows(like, row_offsets, max_rows, T)
    made = []
    if out is None:
        path = torch.empty((n, max_rows if max_path is None else max_path), dtype=torch.int32, device=device)
        accepted = torch.empty(n, dtype=torch.int32, device=device)
        token = torch.empty(n, dtype=torch.int32, device=device)
        made += [path, accepted, token]
    else:
        path, accepted, token = out
        if max_path is not None and path.shape[-1] != max_path:
            raise ValueError(f"path has {path.shape[-1]} columns, max_path is {max_path}")
        _check_tensor("path", path, torch.int32, (n, path.shape[-1]), device)
        _check_tensor("accepted", accepted, torch.int32, (n,), device)
        _check_tensor("next_token", token, torch.int32, (n,), device)
    ws = _cache_workspace(like, workspace, made, 256)
    _cache_call(load_library().bdlm_tree_verify, like, stream,
                (parents.data_ptr(), tokens.data_ptr(), target.data_ptr(), None if draft is None else draft.data_ptr(),
                 F32 if dtype is torch.float32 else BF16, shape[1], row_t, row_d, uniforms.data_ptr(),
                 sample.data_ptr(), n, off, T, max_rows, path.data_ptr(), path.shape[1], accepted.data_ptr(),
                 token.data_ptr(), ws.data_ptr(), ws.nbytes), made)
    return path, accepted, token


class _Batch:
    """What the shared checks of the calls on a cache need of one that has none."""
    __slots__ = ("n_seqs", "device")

    def __init__(self, n_seqs, device):
        self.n_seqs, self.device = n_seqs, device


def bdlm_cache_commit(cache, K, V, path, accepted, row_offsets=None, max_rows: int | None = None, lens_out=None,
                      workspace=None, stream=None):
    """``bdlm_cache_append`` of the rows that ``bdlm_tree_verify`` accepted: of each
    sequence rows ``path[s, :accepted[s]]`` (counted from its first row), in this order.
    Returns ``lens_out`` [n_seqs] int32 = lens + accepted; copy it into ``cache.lens`` once
    every layer's cache has them."""
    torch = _torch()
    if path.dim() != 2:
        raise ValueError(f"path must be [n_seqs, max_path], not {list(path.shape)}")
    T = K.shape[0]
    _check_tensor("K", K, torch.bfloat16, (T, cache.Hkv, cache.d), cache.device)
    _check_tensor("V", V, torch.bfloat16, (T, cache.Hkv, cache.d), cache.device)
    _check_tensor("path", path, torch.int32, (cache.n_seqs, path.shape[1]), cache.device)
    _check_tensor("accepted", accepted, torch.int32, (cache.n_seqs,), cache.device)
    off, max_rows = _cache_rows(cache, row_offsets, max_rows, T)
    made = []
    if lens_out is None:
        lens_out = torch.empty(cache.n_seqs, dtype=torch.int32, device=cache.device)
        made.append(lens_out)
    else:
        _check_tensor("lens_out", lens_out, torch.int32, (cache.n_seqs,), cache.device)
    ws = _cache_workspace(cache, workspace, made, 256)
    _cache_call(load_library().bdlm_cache_commit, cache, stream,
                (K.data_ptr(), V.data_ptr(), cache._ref, path.data_ptr(), path.shape[1], accepted.data_ptr(), off, T,
                 max_rows, lens_out.data_ptr(), ws.data_ptr(), ws.nbytes), made)
    return lens_out


def bdlm_sync_status(workspace, stream=None):
    """Synchronises and raises BdlmError(BDLM_ERR_TIMEOUT) if a kernel's
    bounded wait expired since the last call on this workspace, or
    BdlmError(BDLM_ERR_INVALID_ARG) if a cache call met contents out of range."""
    _check(load_library().bdlm_sync_status(_ptr(workspace), _stream(stream)))


def bdlm_sync_status_noalloc(stream=None):
    """Synchronises and raises BdlmError(BDLM_ERR_TIMEOUT) if a kernel of an
    allocation-free call gave up on a device wait since the last check."""
    _check(load_library().bdlm_sync_status_noalloc(_stream(stream)))


def bdlm_watchdog_selftest_noalloc(limit_us: int = 20000, stream=None) -> int:
    """The watchdog self-test on the allocation-free array's status word;
    returns the status code (7 = the wait ran out and was reported)."""
    return int(load_library().bdlm_watchdog_selftest_noalloc(limit_us, _stream(stream)))


def bdlm_watchdog_selftest(workspace, limit_us: int = 20000, stream=None) -> int:
    """Runs the watchdog self-test; returns the status code (7 = the bounded
    wait expired and was reported, the expected outcome)."""
    return int(load_library().bdlm_watchdog_selftest(_ptr(workspace), workspace.numel(), limit_us,
                                                      _stream(stream)))
