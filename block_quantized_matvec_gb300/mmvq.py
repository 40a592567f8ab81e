"""Thin Python binding of libmmvq.so (include/mmvq.h).

Argument marshalling only: every step of the path runs in the library's
CUDA kernels.  Tensors are torch CUDA tensors; each call runs on the current
torch stream (or the one passed in).  If the library is missing the first
call raises; there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmmvq.so")

TYPE_Q4_K = 12
TYPE_Q6_K = 14
TYPE_Q6_K_PLANAR = 1014
TYPE_Q4_K_PLANAR = 1012
TYPE_Q5_K = 13
TYPE_Q5_K_PLANAR = 1013
BLOCK_BYTES = {TYPE_Q4_K: 144, TYPE_Q6_K: 210, TYPE_Q6_K_PLANAR: 210, TYPE_Q4_K_PLANAR: 144,
               TYPE_Q5_K: 176, TYPE_Q5_K_PLANAR: 176}
Q8_1_BYTES = 36
MAX_COLS = 8

OK = 0
FLAG_XQ_STABLE = 1
FLAG_TENSOR_CORE = 2
ERR_TYPE, ERR_SHAPE, ERR_NCOLS, ERR_NULL, ERR_ALIGN, ERR_ROUTING, ERR_CUDA = -1, -2, -3, -4, -5, -6, -7
ERR_SCRATCH = -8
ERR_VALUE = -9
NOALLOC_SCRATCH_BYTES = 2 << 20  # MMVQ_NOALLOC_SCRATCH_BYTES

# name -> (restype, argtypes); mirrors include/mmvq.h
_P, _I, _I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
SIGNATURES = {
    "mmvq_version": (_I, []),
    "mmvq_strerror": (ctypes.c_char_p, [_I]),
    "mmvq_quantize_q8_1": (_I, [_P, _I, _I, _I64, _P, _P]),
    "mmvq_gemv": (_I, [_I, _P, _I64, _I, _P, _I, _P, _P]),
    "mmvq_gemv_ex": (_I, [_I, _P, _I64, _I, _P, _I, _P, ctypes.c_uint, _P]),
    "mmvq_debug_block_sums": (_I, [_I, _P, _I64, _I, _P, _I, _P, _P, _P]),
    "mmvq_debug_block_sums_ex": (_I, [_I, _P, _I64, _I, _P, _I, _P, _P, ctypes.c_uint, _P]),
    "mmvq_gemv_f32": (_I, [_I, _P, _I64, _I, _P, _I64, _I, _P, _P, ctypes.c_uint, _P]),
    "mmvq_gemv_f32_fused": (_I, [_I, _I64, _I, _I, _P]),
    "mmvq_grouped": (_I, [_I, _P, _I, _I64, _I, _P, _P, _I, _P, _P, _I, _P, _P, _P]),
    "mmvq_route_groups": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "mmvq_quantize_route_groups": (_I, [_P, _I, _I, _I64, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "mmvq_silu_mul_quantize_q8_1": (_I, [_P, _I, _I, _P, _P, _P]),
    "mmvq_planar_bytes": (_I64, [_I, _I64, _I]),
    "mmvq_repack_planar": (_I, [_I, _P, _I64, _I, _P, _P]),
    "mmvq_gather_planar_rows": (_I, [_P, _I64, _I, _P, _I, _P, _P, _P]),
    "mmvq_read_device_fault": (_I, [_P, _P]),
    "mmvq_selftest_wait_timeout": (_I, [ctypes.c_uint, _P]),
    "mmvq_rmsnorm_quantize_q8_1": (_I, [_P, _P, ctypes.c_float, _I, _I, _I64, _P, _P, _P]),
    "mmvq_launch_shape": (_I, [_I, _I64, _I, _I, _P]),
    "mmvq_launch_shape_ex": (_I, [_I, _I64, _I, _I, _P, _I]),
    "mmvq_expert_ffn": (_I, [_I, _P, _P, _I, _I, _I, _P, _I64, _I, _P, _I, _P, _P, _P, _P, _P,
                             _P, _P, _P, _P, _P, _P]),
    "mmvq_expert_ffn_noalloc": (_I, [_I, _P, _P, _I, _I, _I, _P, _I64, _I, _P, _I, _P, _P, _P,
                                     _P, _P, _P, _P]),
    "mmvq_expert_ffn_shape": (_I, [_I, _I, _I, _I, _I, _I, _P]),
    "mmvq_selftest_grid_barrier_timeout": (_I, [_P, ctypes.c_uint, _P]),
    "mmvq_kv4_page_bytes": (_I64, [_I, _I, _I]),
    "mmvq_kv4_append": (_I, [_I, _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I, _I, _I, _P, _I64,
                             _P, _P, _I, _I, _P, _P]),
    "mmvq_kv4_read": (_I, [_I, _P, _P, _P, _I64, _I, _I, _I, _P, _I64, _P, _P, _I, _I, _P, _P]),
    "mmvq_kv4_attention": (_I, [_I, _P, _I64, _I64, _I, ctypes.c_float, _I, _I, _P, _P, _P, _I64,
                                _I, _I, _I, _P, _I64, _P, _P, _I, _I, _P, _P, _P]),
    "mmvq_kv4_attention_workspace_bytes": (_I64, [_I]),
    "mmvq_norm_rope": (_I, [_I, _P, _I64, _I64, _I, _P, _I64, _I64, _I, _I, _I, _P, _I64, _I, _P, _I,
                            _P, _P, ctypes.c_float, ctypes.c_uint, _P, _I64, _I64, _P, _I64, _I64,
                            _P, _P]),
    "mmvq_route_topk": (_I, [_I, _P, _I64, _I, _I, _I, _I, _P, _I, _I, _I, ctypes.c_float, _P, _P,
                             _P, _P]),
    "mmvq_combine_experts": (_I, [_I, _P, _I64, _I, _P, _P, _I, _I, _P, _I, _P, _P, _I64, _P, _I64,
                                  _P, _P, _I64, _P, _P]),
    "mmvq_token_logprobs": (_I, [_I, _P, _I64, _I, _I, ctypes.c_float, _P, _I, _I, _P, _P, _P, _P,
                                 _P, _P, _P]),
}


class MMVQError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {strerror(code)} (code {code})")


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """The loaded C-ABI library.  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(
                    f"{LIB_PATH} is missing: build it with "
                    "`python -m block_quantized_matvec_gb300.build` (nvcc, sm_103a)")
            l = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                f = getattr(l, name)
                f.restype = res
                f.argtypes = args
            _lib = l
    return _lib


def strerror(code: int) -> str:
    return lib().mmvq_strerror(code).decode()


def _check(rc: int, what: str):
    if rc != OK:
        raise MMVQError(rc, what)


def _ptr(t):
    return None if t is None else t.data_ptr()


# The current stream's handle without building a torch Stream object (about
# 3 us a call otherwise); torch's own raw accessor where it exists.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _made(stream, make, *args, **kw):
    """A tensor that a call makes itself, on the stream that the call runs on: its zeroing and its
    memory's earlier uses come before the kernel, and its memory is used again only after it."""
    if stream is None:
        return make(*args, **kw)
    with torch.cuda.stream(stream):
        return make(*args, **kw)


def _dev(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# ------------------------------------------------------------- entry points --

def quantize_q8_1(x: torch.Tensor, K: int | None = None, out: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """fp32 x [ncols, ldx] -> Q8_1 bytes [ncols, K/32, 36] (uint8)."""
    _dev(x, "x")
    if x.dtype != torch.float32:
        raise ValueError("x must be float32")
    x2 = x if x.dim() == 2 else x.view(1, -1)
    ncols, ldx = x2.shape
    K = ldx if K is None else K
    if out is None:
        out = _made(stream, torch.empty, (ncols, K // 32, Q8_1_BYTES), dtype=torch.uint8, device=x.device)
    _check(lib().mmvq_quantize_q8_1(_ptr(x2), K, ncols, ldx, _ptr(out), _stream(stream)),
           "mmvq_quantize_q8_1")
    return out


def gemv(type_: int, W: torch.Tensor, rows: int, K: int, xq: torch.Tensor, ncols: int,
         out: torch.Tensor | None = None, stream=None, flags: int = 0) -> torch.Tensor:
    """y [ncols, rows] fp32 = W (rows x K, block type ``type_``) times ncols Q8_1 columns.
    flags: FLAG_XQ_STABLE when no still-running kernel writes xq, FLAG_TENSOR_CORE for
    the tensor-core consumer (mmvq_gemv_ex)."""
    _dev(W, "W")
    _dev(xq, "xq")
    if out is None:
        out = _made(stream, torch.empty, (ncols, rows), dtype=torch.float32, device=W.device)
    if flags:
        _check(lib().mmvq_gemv_ex(type_, _ptr(W), rows, K, _ptr(xq), ncols, _ptr(out), flags,
                                  _stream(stream)), "mmvq_gemv_ex")
    else:
        _check(lib().mmvq_gemv(type_, _ptr(W), rows, K, _ptr(xq), ncols, _ptr(out),
                               _stream(stream)), "mmvq_gemv")
    return out


def gemv_f32(type_: int, W: torch.Tensor, rows: int, K: int, x: torch.Tensor, ncols: int | None = None,
             xq: torch.Tensor | None = None, out: torch.Tensor | None = None, flags: int = 0,
             stream=None):
    """fp32 x [ncols, ldx] -> (y [ncols, rows], xq [ncols, K/32, 36]): Q8_1 of x and the
    product, in one launch where the columns are small enough."""
    _dev(W, "W")
    if x.dim() == 1:
        x = x.view(1, -1)
    if not x.is_cuda or x.dtype != torch.float32 or x.stride(1) != 1:
        raise ValueError("x must be a CUDA float32 tensor with unit column stride")
    ncols = x.shape[0] if ncols is None else ncols
    if xq is None:
        xq = _made(stream, torch.empty, (ncols, K // 32, Q8_1_BYTES), dtype=torch.uint8, device=x.device)
    if out is None:
        out = _made(stream, torch.empty, (ncols, rows), dtype=torch.float32, device=x.device)
    _check(lib().mmvq_gemv_f32(type_, _ptr(W), rows, K, _ptr(x), x.stride(0), ncols, _ptr(xq),
                               _ptr(out), flags, _stream(stream)), "mmvq_gemv_f32")
    return out, xq


def gemv_f32_fused(type_: int, rows: int, K: int, ncols: int) -> bool:
    """Whether gemv_f32 runs this call as one launch (host-only)."""
    f = ctypes.c_int32(0)
    _check(lib().mmvq_gemv_f32_fused(type_, rows, K, ncols, ctypes.byref(f)), "mmvq_gemv_f32_fused")
    return bool(f.value)


def debug_block_sums(type_: int, W: torch.Tensor, rows: int, K: int, xq: torch.Tensor, ncols: int,
                     stream=None, flags: int = 0):
    """(sumi [ncols, rows, K/32] int32, y [ncols, rows]) from the gemv kernel itself."""
    _dev(W, "W")
    _dev(xq, "xq")
    sumi = _made(stream, torch.empty, (ncols, rows, K // 32), dtype=torch.int32, device=W.device)
    y = _made(stream, torch.empty, (ncols, rows), dtype=torch.float32, device=W.device)
    if flags:
        _check(lib().mmvq_debug_block_sums_ex(type_, _ptr(W), rows, K, _ptr(xq), ncols,
                                              _ptr(sumi), _ptr(y), flags, _stream(stream)),
               "mmvq_debug_block_sums_ex")
    else:
        _check(lib().mmvq_debug_block_sums(type_, _ptr(W), rows, K, _ptr(xq), ncols, _ptr(sumi),
                                           _ptr(y), _stream(stream)), "mmvq_debug_block_sums")
    return sumi, y


def grouped(type_: int, W_experts: torch.Tensor, n_experts: int, rows: int, K: int,
            expert_ids: torch.Tensor, offsets: torch.Tensor, act_index: torch.Tensor | None,
            xq: torch.Tensor, n_xq_cols: int, n_positions: int, out: torch.Tensor | None = None,
            status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [n_positions, rows]: row p = expert of p's group times xq column act_index[p]."""
    for t, n in ((W_experts, "W_experts"), (expert_ids, "expert_ids"), (offsets, "offsets"),
                 (xq, "xq")):
        _dev(t, n)
    if out is None:
        out = _made(stream, torch.empty, (max(n_positions, 1), rows), dtype=torch.float32, device=xq.device)
    _check(lib().mmvq_grouped(type_, _ptr(W_experts), n_experts, rows, K, _ptr(expert_ids),
                              _ptr(offsets), expert_ids.numel(), _ptr(act_index), _ptr(xq),
                              n_xq_cols, _ptr(out), _ptr(status), _stream(stream)), "mmvq_grouped")
    return out


def quantize_route_groups(x: torch.Tensor, topk: torch.Tensor, n_experts: int,
                          xq: torch.Tensor | None = None, stream=None):
    """One launch: Q8_1 of x [ncols, K] and the per-expert lists of topk [T, k]
    -> (xq, expert_ids, offsets, act_index, slot_of, status)."""
    _dev(x, "x")
    _dev(topk, "topk")
    if x.dim() == 1:
        x = x.view(1, -1)
    ncols, K = x.shape
    T, k = topk.shape
    dev = x.device
    if xq is None:
        xq = _made(stream, torch.empty, (ncols, K // 32, Q8_1_BYTES), dtype=torch.uint8, device=dev)
    eids = _made(stream, torch.empty, n_experts, dtype=torch.int32, device=dev)
    offs = _made(stream, torch.empty, n_experts + 1, dtype=torch.int32, device=dev)
    act = _made(stream, torch.empty, max(T * k, 1), dtype=torch.int32, device=dev)
    slot = _made(stream, torch.empty, max(T * k, 1), dtype=torch.int32, device=dev)
    status = _made(stream, torch.zeros, 1, dtype=torch.int32, device=dev)
    _check(lib().mmvq_quantize_route_groups(_ptr(x), K, ncols, K, _ptr(xq),
                                            _ptr(topk) if T else None, T, k, n_experts,
                                            _ptr(eids), _ptr(offs), _ptr(act), _ptr(slot),
                                            _ptr(status), _stream(stream)),
           "mmvq_quantize_route_groups")
    return xq, eids, offs, act, slot, status


def expert_ffn_workspace(device) -> torch.Tensor:
    """A zeroed grid-barrier word for expert_ffn (one per concurrently running launch)."""
    return torch.zeros(4, dtype=torch.int32, device=device)


def expert_ffn(type_: int, W_gate_up: torch.Tensor, W_down: torch.Tensor, n_experts: int,
               H: int, F: int, x: torch.Tensor, topk: torch.Tensor, *,
               gu: torch.Tensor | None = None, hq: torch.Tensor | None = None,
               y: torch.Tensor | None = None, lists: bool = True, xq: torch.Tensor | None = None,
               status: torch.Tensor | None = None, sync: torch.Tensor | None = None,
               stream=None) -> dict:
    """The routed-expert FFN of one MoE layer in one launch: x [T, H] fp32 (T <= 8),
    topk [T, k] int32, planar experts W_gate_up (2F x H each) and W_down (H x F
    each).  Returns a dict with xq [T, H/32, 36], gu [T*k, 2F], hq [T*k, F/32, 36],
    y [T*k, H] and, with lists=True, expert_ids, offsets, act_index, slot_of."""
    for t, n in ((W_gate_up, "W_gate_up"), (W_down, "W_down"), (x, "x"), (topk, "topk")):
        _dev(t, n)
    if x.dim() == 1:
        x = x.view(1, -1)
    T, k = topk.shape
    n = T * k
    dev = x.device
    if gu is None:
        gu = _made(stream, torch.empty, (n, 2 * F), dtype=torch.float32, device=dev)
    if hq is None:
        hq = _made(stream, torch.empty, (n, F // 32, Q8_1_BYTES), dtype=torch.uint8, device=dev)
    if y is None:
        y = _made(stream, torch.empty, (n, H), dtype=torch.float32, device=dev)
    out = {"gu": gu, "hq": hq, "y": y}
    if lists:
        out.update(expert_ids=_made(stream, torch.empty, n_experts, dtype=torch.int32, device=dev),
                   offsets=_made(stream, torch.empty, n_experts + 1, dtype=torch.int32, device=dev),
                   act_index=_made(stream, torch.empty, max(n, 1), dtype=torch.int32, device=dev),
                   slot_of=_made(stream, torch.empty, max(n, 1), dtype=torch.int32, device=dev))
    if xq is None:
        xq = _made(stream, torch.empty, (T, H // 32, Q8_1_BYTES), dtype=torch.uint8, device=dev)
    out["xq"] = xq
    if status is not None:
        out["status"] = status
    if sync is None:
        sync = _made(stream, expert_ffn_workspace, dev)
    _check(lib().mmvq_expert_ffn(type_, _ptr(W_gate_up), _ptr(W_down), n_experts, H, F, _ptr(x),
                                 x.stride(0), T, _ptr(topk), k, _ptr(gu), _ptr(hq), _ptr(y),
                                 _ptr(out.get("expert_ids")), _ptr(out.get("offsets")),
                                 _ptr(out.get("act_index")), _ptr(out.get("slot_of")),
                                 _ptr(xq), _ptr(status), _ptr(sync), _stream(stream)),
           "mmvq_expert_ffn")
    return out


def expert_ffn_noalloc(type_: int, W_gate_up: torch.Tensor, W_down: torch.Tensor,
                       n_experts: int, H: int, F: int, x: torch.Tensor, topk: torch.Tensor, *,
                       y: torch.Tensor | None = None, lists: bool = True,
                       status: torch.Tensor | None = None, stream=None) -> dict:
    """expert_ffn with its intermediates (xq, gu, hq, barrier word) in the library's
    fixed device array: for callers that cannot allocate.  Pass y (and the list
    outputs) preallocated to allocate nothing here either.  Returns y and, with
    lists=True, expert_ids, offsets, act_index, slot_of."""
    for t, n in ((W_gate_up, "W_gate_up"), (W_down, "W_down"), (x, "x"), (topk, "topk")):
        _dev(t, n)
    if x.dim() == 1:
        x = x.view(1, -1)
    T, k = topk.shape
    n = T * k
    dev = x.device
    if y is None:
        y = _made(stream, torch.empty, (n, H), dtype=torch.float32, device=dev)
    out = {"y": y}
    if lists:
        out.update(expert_ids=_made(stream, torch.empty, n_experts, dtype=torch.int32, device=dev),
                   offsets=_made(stream, torch.empty, n_experts + 1, dtype=torch.int32, device=dev),
                   act_index=_made(stream, torch.empty, max(n, 1), dtype=torch.int32, device=dev),
                   slot_of=_made(stream, torch.empty, max(n, 1), dtype=torch.int32, device=dev))
    if status is not None:
        out["status"] = status
    _check(lib().mmvq_expert_ffn_noalloc(type_, _ptr(W_gate_up), _ptr(W_down), n_experts, H, F,
                                         _ptr(x), x.stride(0), T, _ptr(topk), k, _ptr(y),
                                         _ptr(out.get("expert_ids")), _ptr(out.get("offsets")),
                                         _ptr(out.get("act_index")), _ptr(out.get("slot_of")),
                                         _ptr(status), _stream(stream)),
           "mmvq_expert_ffn_noalloc")
    return out


def expert_ffn_shape(type_: int, n_experts: int, H: int, F: int, T: int, k: int) -> dict:
    """The launch shape mmvq_expert_ffn picks (host-only)."""
    info = (ctypes.c_int32 * 8)()
    _check(lib().mmvq_expert_ffn_shape(type_, n_experts, H, F, T, k, info),
           "mmvq_expert_ffn_shape")
    keys = ("grid", "threads", "smem", "stages", "G_gate_up", "P_gate_up", "G_down", "P_down")
    return dict(zip(keys, list(info)))


def selftest_grid_barrier_timeout(sync: torch.Tensor, limit_us: int = 2000, stream=None) -> None:
    """Run the expert FFN's grid barrier to expiry on its own word (sets bit 2 of the fault word)."""
    _dev(sync, "sync")
    _check(lib().mmvq_selftest_grid_barrier_timeout(_ptr(sync), limit_us, _stream(stream)),
           "mmvq_selftest_grid_barrier_timeout")


def route_groups(topk: torch.Tensor, n_experts: int, stream=None):
    """topk [T, k] int32 -> (expert_ids [E], offsets [E+1], act_index [T*k], slot_of [T*k], status)."""
    _dev(topk, "topk")
    T, k = topk.shape
    dev = topk.device
    eids = _made(stream, torch.empty, n_experts, dtype=torch.int32, device=dev)
    offs = _made(stream, torch.empty, n_experts + 1, dtype=torch.int32, device=dev)
    act = _made(stream, torch.empty, max(T * k, 1), dtype=torch.int32, device=dev)
    slot = _made(stream, torch.empty, max(T * k, 1), dtype=torch.int32, device=dev)
    status = _made(stream, torch.zeros, 1, dtype=torch.int32, device=dev)
    _check(lib().mmvq_route_groups(_ptr(topk) if T else None, T, k, n_experts, _ptr(eids),
                                   _ptr(offs), _ptr(act), _ptr(slot), _ptr(status),
                                   _stream(stream)), "mmvq_route_groups")
    return eids, offs, act, slot, status


def silu_mul_quantize_q8_1(gu: torch.Tensor, F: int, out: torch.Tensor | None = None,
                           h_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """gu [n, 2F] = [gate | up] -> Q8_1 of silu(gate)*up, [n, F/32, 36]."""
    _dev(gu, "gu")
    n = gu.shape[0]
    if out is None:
        out = _made(stream, torch.empty, (n, F // 32, Q8_1_BYTES), dtype=torch.uint8, device=gu.device)
    _check(lib().mmvq_silu_mul_quantize_q8_1(_ptr(gu), F, n, _ptr(out), _ptr(h_out),
                                             _stream(stream)), "mmvq_silu_mul_quantize_q8_1")
    return out


def launch_shape(type_: int, rows: int, K: int, ncols: int) -> dict:
    """The launch shape mmvq_gemv picks (host-only query)."""
    info = (ctypes.c_int32 * 7)()
    _check(lib().mmvq_launch_shape_ex(type_, rows, K, ncols, info, 7), "mmvq_launch_shape_ex")
    keys = (["grid", "threads", "smem", "G", "P", "stages", "cluster"]
            if type_ in (TYPE_Q6_K_PLANAR, TYPE_Q4_K_PLANAR, TYPE_Q5_K_PLANAR)
            else ["grid", "threads", "smem", "WR", "WK", "unused", "cluster"])
    return dict(zip(keys, list(info)))


def read_device_fault(stream=None) -> int:
    """Synchronise the stream, return and clear the device fault word (0 = none)."""
    v = ctypes.c_int(0)
    _check(lib().mmvq_read_device_fault(ctypes.byref(v), _stream(stream)), "mmvq_read_device_fault")
    return v.value


def rmsnorm_quantize_q8_1(x: torch.Tensor, w: torch.Tensor, eps: float,
                          out: torch.Tensor | None = None, y_out: torch.Tensor | None = None,
                          stream=None) -> torch.Tensor:
    """x [ncols, K] fp32 (rows may be strided), w [K] fp32 -> Q8_1 of RMSNorm(x) * w,
    [ncols, K/32, 36]."""
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    _dev(w, "w")
    if x.dim() == 1:
        x = x.view(1, -1)
    ncols, K = x.shape
    if x.dtype != torch.float32 or w.dtype != torch.float32 or x.stride(1) != 1 or \
            not w.is_contiguous() or w.numel() != K:
        raise ValueError("x [ncols, K] with unit inner stride and w [K], both float32")
    if out is None:
        out = _made(stream, torch.empty, (ncols, K // 32, Q8_1_BYTES), dtype=torch.uint8, device=x.device)
    _check(lib().mmvq_rmsnorm_quantize_q8_1(_ptr(x), _ptr(w), eps, K, ncols, x.stride(0),
                                            _ptr(out), _ptr(y_out), _stream(stream)),
           "mmvq_rmsnorm_quantize_q8_1")
    return out


def selftest_wait_timeout(limit_us: int = 2000, stream=None) -> None:
    """Run one bounded barrier wait to expiry (sets bit 1 of the fault word)."""
    _check(lib().mmvq_selftest_wait_timeout(limit_us, _stream(stream)),
           "mmvq_selftest_wait_timeout")


def planar_bytes(rows: int, K: int, type_: int = TYPE_Q6_K) -> int:
    n = lib().mmvq_planar_bytes(type_, rows, K)
    if n < 0:
        raise MMVQError(ERR_SHAPE, "mmvq_planar_bytes")
    return int(n)


def repack_planar(W_gguf: torch.Tensor, rows: int, K: int, out: torch.Tensor | None = None,
                  stream=None, type_: int = TYPE_Q6_K) -> torch.Tensor:
    """GGUF Q6_K (or Q4_K) bytes -> planar tiles (uint8, planar_bytes(rows, K, type_))."""
    _dev(W_gguf, "W_gguf")
    if out is None:
        out = _made(stream, torch.empty, planar_bytes(rows, K, type_), dtype=torch.uint8, device=W_gguf.device)
    _check(lib().mmvq_repack_planar(type_, _ptr(W_gguf), rows, K, _ptr(out), _stream(stream)),
           "mmvq_repack_planar")
    return out


def gather_planar_rows(W_planar: torch.Tensor, rows: int, K: int, row_ids: torch.Tensor,
                       out: torch.Tensor | None = None, stream=None):
    """Planar matrix of len(row_ids) rows, row k = row row_ids[k] of W_planar; returns (out, status)."""
    _dev(W_planar, "W_planar")
    _dev(row_ids, "row_ids")
    n = row_ids.numel()
    if out is None:
        out = _made(stream, torch.empty, planar_bytes(n, K), dtype=torch.uint8, device=W_planar.device)
    status = _made(stream, torch.zeros, 1, dtype=torch.int32, device=W_planar.device)
    _check(lib().mmvq_gather_planar_rows(_ptr(W_planar), rows, K, _ptr(row_ids), n, _ptr(out),
                                         _ptr(status), _stream(stream)), "mmvq_gather_planar_rows")
    return out, status


# ---------------------------------------------------- 4-bit key/value cache --

KV4_TILE = 16  # tokens of a cache tile
KV4_MAX_NEW = 8  # query tokens of a sequence in kv4_attention
_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 30}  # mmvq_dtype


def kv4_page_bytes(n_kv_heads: int, head_dim: int, page_tokens: int) -> int:
    n = lib().mmvq_kv4_page_bytes(n_kv_heads, head_dim, page_tokens)
    if n < 0:
        raise MMVQError(ERR_SHAPE, "mmvq_kv4_page_bytes")
    return n


def kv4_cache(n_pages: int, n_kv_heads: int, head_dim: int, page_tokens: int,
              device) -> torch.Tensor:
    """An empty 4-bit key/value cache: uint8 [n_pages, n_kv_heads, page_tokens/16, 20*head_dim]
    (16-token tiles; the layout is in include/mmvq.h)."""
    kv4_page_bytes(n_kv_heads, head_dim, page_tokens)
    return torch.zeros((n_pages, n_kv_heads, page_tokens // KV4_TILE, 20 * head_dim),
                       dtype=torch.uint8, device=device)


def _kv4_where(cache, page_table, offsets, lens, status):
    """Checks the tensors of a batch: its device's number, and the cache's and the batch's arguments of
    the C calls."""
    n_pages, n_kv, tiles, tile_bytes = cache.shape
    n_seqs, ld = page_table.shape
    dev = cache.get_device()  # -1: the host's
    if cache.dtype is not torch.uint8 or dev < 0 or not cache.is_contiguous() or tile_bytes % 20:
        raise ValueError("cache must be a contiguous CUDA uint8 tensor [pages, kv heads, "
                         "page_tokens/16, 20*head_dim] (kv4_cache)")
    i32 = torch.int32
    if page_table.dtype is not i32 or page_table.get_device() != dev or \
            not page_table.is_contiguous():
        raise ValueError("page_table must be a contiguous int32 tensor on the cache's device")
    if offsets.dtype is not i32 or offsets.get_device() != dev or not offsets.is_contiguous() or \
            offsets.numel() != n_seqs + 1:
        raise ValueError(f"offsets must be a contiguous int32 tensor of {n_seqs + 1} values on the "
                         "cache's device")
    if lens.dtype is not i32 or lens.get_device() != dev or not lens.is_contiguous() or \
            lens.numel() != n_seqs:
        raise ValueError(f"lens must be a contiguous int32 tensor of {n_seqs} values on the cache's "
                         "device")
    if status is not None and (status.dtype is not i32 or status.get_device() != dev or
                               status.numel() < 1):
        raise ValueError("status must be an int32 tensor on the cache's device")
    return dev, (cache.data_ptr(), n_pages, tiles * KV4_TILE, n_kv, tile_bytes // 20,
                 page_table.data_ptr(), ld, offsets.data_ptr(), lens.data_ptr(), n_seqs)


def _kv4_rows(t, heads, dim, dev, name):
    """A [n, heads, dim] tensor with unit inner stride: its type's number, tokens, and the token and
    head strides."""
    n, h, d = t.shape
    ld, hs, one = t.stride()
    dtype = _DTYPES.get(t.dtype)
    if dtype is None or t.get_device() != dev or (heads and h != heads) or d != dim or \
            (one != 1 and n):
        raise ValueError(f"{name} must be a float32, float16 or bfloat16 tensor [tokens, "
                         f"{heads or 'heads'}, {dim}] with unit inner stride on the cache's device")
    return dtype, n, h, ld, hs


def kv4_append(k: torch.Tensor, v: torch.Tensor, cache: torch.Tensor, page_table: torch.Tensor,
               offsets: torch.Tensor, lens: torch.Tensor, status: torch.Tensor | None = None,
               stream=None) -> None:
    """Quantises keys and values [n, kv heads, head_dim] into the cache: rows
    offsets[b]..offsets[b+1]-1 are the last tokens of sequence b, whose length with them is
    lens[b]; position p of it lies in page page_table[b, p // page_tokens].  (mmvq_kv4_append)"""
    dev, where = _kv4_where(cache, page_table, offsets, lens, status)
    dtype, n, _, ldk, hk = _kv4_rows(k, where[3], where[4], dev, "k")
    dtype_v, n_v, _, ldv, hv = _kv4_rows(v, where[3], where[4], dev, "v")
    if n_v != n or dtype_v != dtype:
        raise ValueError("k and v must have the same tokens and type")
    _check(lib().mmvq_kv4_append(dtype, k.data_ptr(), ldk, hk, v.data_ptr(), ldv, hv, *where, n,
                                 _ptr(status), _stream(stream)), "mmvq_kv4_append")


def kv4_read(cache: torch.Tensor, page_table: torch.Tensor, offsets: torch.Tensor,
             lens: torch.Tensor, n_tokens: int, dtype: torch.dtype = torch.float32,
             out: tuple[torch.Tensor, torch.Tensor] | None = None,
             status: torch.Tensor | None = None, stream=None):
    """(k, v), each [n_tokens, kv heads, head_dim] of dtype: the cached values of the last
    offsets[b+1]-offsets[b] of the first lens[b] tokens of each sequence b.  (mmvq_kv4_read)"""
    dev, where = _kv4_where(cache, page_table, offsets, lens, status)
    number = _DTYPES.get(dtype)
    if number is None:
        raise ValueError("dtype must be float32, float16 or bfloat16")
    shape = (n_tokens, where[3], where[4])
    if out is None:
        k = _made(stream, torch.empty, shape, dtype=dtype, device=cache.device)
        v = _made(stream, torch.empty_like, k)
    else:
        k, v = out
        for t in out:
            if t.shape != shape or t.dtype != dtype or t.get_device() != dev or \
                    not t.is_contiguous():
                raise ValueError(f"out must be two contiguous tensors {list(shape)} of {dtype} on the "
                                 "cache's device")
    _check(lib().mmvq_kv4_read(number, k.data_ptr(), v.data_ptr(), *where, n_tokens,
                               _ptr(status), _stream(stream)), "mmvq_kv4_read")
    return k, v


_workspace_bytes = {}  # by head_dim: a constant of the library


def kv4_attention_workspace_bytes(head_dim: int) -> int:
    n = _workspace_bytes.get(head_dim)
    if n is None:
        n = lib().mmvq_kv4_attention_workspace_bytes(head_dim)
        if n < 0:
            raise MMVQError(ERR_SHAPE, "mmvq_kv4_attention_workspace_bytes")
        _workspace_bytes[head_dim] = n
    return n


def kv4_attention_workspace(head_dim: int, device) -> torch.Tensor:
    """A zeroed workspace for kv4_attention (one per concurrently running call)."""
    return torch.zeros(kv4_attention_workspace_bytes(head_dim), dtype=torch.uint8, device=device)


def kv4_attention(q: torch.Tensor, cache: torch.Tensor, page_table: torch.Tensor,
                  offsets: torch.Tensor, lens: torch.Tensor, *, scale: float | None = None,
                  window: int = 0, sinks: int = 0, out: torch.Tensor | None = None,
                  lse: torch.Tensor | None = None, with_lse: bool = False,
                  workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
                  stream=None):
    """Attention of q [n, heads, head_dim] (1-8 query tokens a sequence, the batch as in
    kv4_append) over the cache -> y [n, heads, head_dim], or (y, lse [n, heads] fp32) with
    with_lse or lse.  A query sees the tokens up to its own position; with window > 0 only the
    last `window` of them and the first `sinks` of the sequence.  scale defaults to
    head_dim**-0.5; workspace: kv4_attention_workspace, zeroed before this call on its stream
    (a temporary one otherwise).  (mmvq_kv4_attention)"""
    dev, where = _kv4_where(cache, page_table, offsets, lens, status)
    dim = where[4]
    dtype, n, heads, ldq, hq = _kv4_rows(q, 0, dim, dev, "q")
    if out is None:
        out = _made(stream, torch.empty_like, q, memory_format=torch.contiguous_format)
    elif out.shape != q.shape or out.dtype != q.dtype or out.get_device() != dev or \
            not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor of q's shape and type on its device")
    if lse is None and with_lse:
        lse = _made(stream, q.new_empty, (n, heads), dtype=torch.float32)
    elif lse is not None and (lse.shape != (n, heads) or lse.dtype != torch.float32 or
                              lse.get_device() != dev or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 tensor [tokens, heads] on q's device")
    if workspace is None:
        workspace = _made(stream, kv4_attention_workspace, dim, q.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous() or \
            workspace.nbytes < kv4_attention_workspace_bytes(dim):
        raise ValueError("workspace is too small or on another device: "
                         "kv4_attention_workspace(head_dim, device)")
    _check(lib().mmvq_kv4_attention(dtype, q.data_ptr(), ldq, hq, heads,
                                    dim ** -0.5 if scale is None else scale, window, sinks,
                                    out.data_ptr(), _ptr(lse), *where, n, workspace.data_ptr(),
                                    _ptr(status), _stream(stream)), "mmvq_kv4_attention")
    return out if lse is None else (out, lse)


# ------------------------------------- the layer's steps between the products

ROPE_INTERLEAVED = 1
ROPE_NO_NORM = 2
_SCORING = {"softmax": 0, "sigmoid": 1}  # mmvq_scoring


_F32, _I32 = torch.float32, torch.int32
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on(t: torch.Tensor, stream):
    """The number of a tensor's device, which has to be the current one (a launch elsewhere fails)
    and the stream's, and the stream's handle."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("the tensors must be CUDA tensors")
    if stream is not None and dev != stream.device_index:
        raise ValueError("the tensors are on another device than the call's stream")
    if dev != _current_device():
        raise ValueError("the tensors are on another device than the current one (torch.cuda.device)")
    if stream is None and _raw_stream is not None:
        return dev, _raw_stream(dev)
    return dev, _stream(stream)


def _plain(t, dtype, shape, dev, name):
    """A contiguous tensor of this type and shape on the device (None passes): its address."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on the call's device")
    return t.data_ptr()


def _list(t, dtype, n, dev, name):
    """A contiguous tensor [n] of this type on the device (None passes): its address."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != n or t.dim() != 1 or t.get_device() != dev or \
            not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor [{n}] on the call's device")
    return t.data_ptr()


def _layer_status(status, dev):
    if status is None:
        return None
    if status.dtype is not _I32 or status.get_device() != dev or status.numel() < 1:
        raise ValueError("status must be an int32 tensor on the call's device")
    return status.data_ptr()


def _rows(t, dtype, shape, dev, name):
    """A [rows, n] tensor with unit inner stride (None passes): its address and row stride."""
    if t is None:
        return None, 0
    n, m = shape
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
        ld, one = t.stride()
        if (one == 1 or m == 1) and (ld >= m or n <= 1):
            return t.data_ptr(), ld if ld >= m else m
    raise ValueError(f"{name} must be a {dtype} tensor {list(shape)} with unit inner stride and rows "
                     "that do not overlap, on the call's device")


def _heads(x, y, dim, dev, name):
    """Heads [n, heads, dim] and a tensor like them, both with unit inner stride: the shape, and the
    addresses with their token and head strides."""
    shape, dtype = x.shape, x.dtype
    ld, h, one = x.stride()
    ldy, hy, one_y = y.stride()
    if y.shape != shape or shape[2] != dim or y.dtype is not dtype or x.get_device() != dev or \
            y.get_device() != dev or ((one != 1 or one_y != 1) and shape[0]):
        raise ValueError(f"{name} and its out must be [tokens, heads, {dim}] tensors of one type with unit "
                         "inner stride on the call's device")
    return shape, (x.data_ptr(), ld, h), (y.data_ptr(), ldy, hy)


def _inverse_two_pi(bits: int) -> int:
    """2^bits / (2 pi), rounded down; pi by Machin's formula in whole numbers."""
    one = 1 << (bits + 32)

    def arctan_of_inverse(n):
        term = one // n
        total, i, sign = term, 1, 1
        while term:
            term //= n * n
            i, sign = i + 2, -sign
            total += sign * (term // i)
        return total
    pi = 4 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239))
    return (one << bits) // (2 * pi)


def rope_table(inv_freq, sections=None, axis_of=None, device="cuda") -> torch.Tensor:
    """The table of norm_rope, int64 [2, rot_dim/2], made once and kept: inv_freq, the angle of
    each pair per position in radians (numbers or a tensor, taken as 64-bit floats), and the axis
    whose position turns it: axis_of, a number for each pair, or sections, the pairs of axis 0, 1,
    ... one after another (neither: axis 0)."""
    freq = [float(f) for f in (inv_freq.double().tolist() if isinstance(inv_freq, torch.Tensor)
                               else inv_freq)]
    if not freq or not all(abs(f) < 2.0 ** 64 for f in freq):
        raise ValueError("inv_freq must be numbers below 2^64")
    if sections is not None and axis_of is not None:
        raise ValueError("sections or axis_of, not both")
    if sections is not None:
        axis_of = [a for a, n in enumerate(sections) for _ in range(n)]
    axis_of = [0] * len(freq) if axis_of is None else [int(a) for a in axis_of]
    if len(axis_of) != len(freq) or not all(0 <= a < 4 for a in axis_of):
        raise ValueError("an axis (0-3) for each of inv_freq")
    bits = 1300  # 64 of the fraction and, for the smallest doubles, their 1074 behind it
    inv = _inverse_two_pi(bits)
    steps = []
    for f in freq:
        num, den = f.as_integer_ratio()  # den is a power of two
        step = ((num * inv << 64) // den + (1 << (bits - 1)) >> bits) % (1 << 64)
        steps.append(step - (1 << 64) if step >= 1 << 63 else step)
    return torch.tensor([steps, axis_of], dtype=torch.int64, device=device)


def norm_rope(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor,
              table: torch.Tensor, *, q_weight: torch.Tensor | None = None,
              k_weight: torch.Tensor | None = None, eps: float | None = 1e-6,
              interleaved: bool = False, out: tuple | None = None,
              status: torch.Tensor | None = None, stream=None):
    """RMS norm of every head of q [n, heads, head_dim] and k [n, kv heads, head_dim] (None:
    queries alone), times q_weight and k_weight [head_dim] fp32 (None: ones), then the rotation by
    the token's position -> (q, k), contiguous or written to out (which may be q and k themselves).
    positions: int32 [n], or [axes, n]; table: rope_table; eps=None leaves the norm and the weights out;
    interleaved pairs neighbours instead of halves.  (mmvq_norm_rope)"""
    dev, on = _on(q, stream)
    n, heads, dim = q.shape
    number = _DTYPES.get(q.dtype)
    if number is None:
        raise ValueError("q must be float32, float16 or bfloat16")
    if out is None:
        yq = _made(stream, torch.empty_like, q, memory_format=torch.contiguous_format)
        yk = None if k is None else _made(stream, torch.empty_like, k,
                                          memory_format=torch.contiguous_format)
    else:
        yq, yk = out
    _, q_at, yq_at = _heads(q, yq, dim, dev, "q")
    kv, k_at, yk_at = 0, (None, 0, 0), (None, 0, 0)
    if k is not None:
        if yk is None:
            raise ValueError("out must be (q, k)")
        shape, k_at, yk_at = _heads(k, yk, dim, dev, "k")
        if shape[0] != n or k.dtype is not q.dtype:
            raise ValueError("k must have the tokens and type of q")
        kv = shape[1]
    elif yk is not None:
        raise ValueError("out must be (q, None) where k is None")
    shape, strides = positions.shape, positions.stride()
    axes, ld_pos = (1, 0) if len(shape) == 1 else (shape[0], strides[0])
    if positions.dtype is not torch.int32 or positions.get_device() != dev or shape[-1] != n or \
            len(shape) > 2 or (strides[-1] != 1 and n > 1):
        raise ValueError(f"positions must be an int32 tensor [{n}] or [axes, {n}] with unit inner "
                         "stride on the call's device")
    two, half = table.shape
    if table.dtype is not torch.int64 or two != 2 or table.get_device() != dev or \
            not table.is_contiguous():
        raise ValueError("table must be a rope_table on the call's device")
    flags = (ROPE_INTERLEAVED if interleaved else 0) | (ROPE_NO_NORM if eps is None else 0)
    _check(lib().mmvq_norm_rope(number, *q_at, heads, *k_at, kv, dim, n, positions.data_ptr(),
                                ld_pos, axes, table.data_ptr(), 2 * half,
                                _list(q_weight, _F32, dim, dev, "q_weight"),
                                _list(k_weight, _F32, dim, dev, "k_weight"),
                                0.0 if eps is None else eps, flags, *yq_at, *yk_at,
                                _layer_status(status, dev), on), "mmvq_norm_rope")
    return yq, yk


def route_topk(logits: torch.Tensor, k: int, *, scoring: str = "softmax",
               bias: torch.Tensor | None = None, n_groups: int = 1, top_groups: int | None = None,
               renormalize: bool = True, scale: float = 1.0, out: tuple | None = None,
               status: torch.Tensor | None = None, stream=None):
    """Router logits [n, experts] -> (topk [n, k] int32, weights [n, k] fp32): the k experts of the
    largest score (softmax or sigmoid of the logits) + bias [experts] fp32, among the top_groups
    (all by default) of n_groups runs of experts whose two best add up to most; weights are their
    scores, renormalised to sum to 1 before scale.  What route_groups, expert_ffn and
    combine_experts take.  (mmvq_route_topk)"""
    dev, on = _on(logits, stream)
    n, experts = logits.shape
    dtype = _DTYPES.get(logits.dtype)
    if dtype is None or scoring not in _SCORING:
        raise ValueError("logits must be float32, float16 or bfloat16, scoring softmax or sigmoid")
    address, ld = _rows(logits, logits.dtype, (n, experts), dev, "logits")
    if out is None:
        out = (_made(stream, torch.empty, (n, k), dtype=torch.int32, device=logits.device),
               _made(stream, torch.empty, (n, k), dtype=torch.float32, device=logits.device))
    topk, weights = out
    _check(lib().mmvq_route_topk(dtype, address, ld, n, experts, k, _SCORING[scoring],
                                 _list(bias, _F32, experts, dev, "bias"), n_groups,
                                 n_groups if top_groups is None else top_groups,
                                 1 if renormalize else 0, scale,
                                 _plain(topk, _I32, (n, k), dev, "out[0]"),
                                 _plain(weights, _F32, (n, k), dev, "out[1]"),
                                 _layer_status(status, dev), on), "mmvq_route_topk")
    return topk, weights


def combine_experts(y: torch.Tensor, topk: torch.Tensor, weights: torch.Tensor,
                    offsets: torch.Tensor, slot_of: torch.Tensor, *,
                    residual: torch.Tensor | None = None, shared: torch.Tensor | None = None,
                    shared_gate: torch.Tensor | None = None, dtype: torch.dtype | None = None,
                    out: torch.Tensor | None = None, status: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """out [n, H] = residual + sigmoid(shared_gate) * shared + the experts' rows y [positions, H]
    fp32 times weights [n, k], where offsets and slot_of are the lists of topk [n, k] (route_groups,
    expert_ffn).  residual and shared [n, H] (either may be missing) have out's type: dtype, theirs,
    or float32.  shared_gate: fp32 [n], None for a weight of 1.  (mmvq_combine_experts)"""
    dev, on = _on(y, stream)
    n, k = topk.shape
    positions, H = y.shape
    if dtype is None:
        dtype = next((t.dtype for t in (out, residual, shared) if t is not None), torch.float32)
    number = _DTYPES.get(dtype)
    if number is None:
        raise ValueError("dtype must be float32, float16 or bfloat16")
    if out is None:
        out = _made(stream, torch.empty, (n, H), dtype=dtype, device=y.device)
    residual_at, ldr = _rows(residual, dtype, (n, H), dev, "residual")
    shared_at, lds = _rows(shared, dtype, (n, H), dev, "shared")
    out_at, ldo = _rows(out, dtype, (n, H), dev, "out")
    experts, slots = offsets.numel() - 1, slot_of.numel()
    if slots < n * k:
        raise ValueError(f"slot_of must hold {n * k} slots")
    _check(lib().mmvq_combine_experts(number, _plain(y, _F32, (positions, H), dev, "y"), positions,
                                      H, _plain(topk, _I32, (n, k), dev, "topk"),
                                      _plain(weights, _F32, (n, k), dev, "weights"), n, k,
                                      _list(offsets, _I32, experts + 1, dev, "offsets"), experts,
                                      _list(slot_of, _I32, slots, dev, "slot_of"),
                                      residual_at, ldr, shared_at, lds,
                                      _list(shared_gate, _F32, n, dev, "shared_gate"), out_at,
                                      ldo, _layer_status(status, dev), on),
           "mmvq_combine_experts")
    return out


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor | None = None, *, top: int = 0,
                   scale: float = 1.0, out: dict | None = None,
                   status: torch.Tensor | None = None, stream=None) -> dict:
    """Of the softmax of scale * logits [n, vocab]: a dict of lse [n], entropy [n], logprobs [n, m]
    of the given tokens [n, m] int32, and the `top` likeliest tokens, top_ids [n, top] int32 and
    top_logprobs [n, top].  out: such a dict to write to; lse and entropy may be missing in it.
    (mmvq_token_logprobs)"""
    dev, on = _on(logits, stream)
    n, vocab = logits.shape
    dtype = _DTYPES.get(logits.dtype)
    if dtype is None:
        raise ValueError("logits must be float32, float16 or bfloat16")
    address, ld = _rows(logits, logits.dtype, (n, vocab), dev, "logits")
    m = 0 if tokens is None else tokens.shape[1]
    if out is None:
        make = lambda shape, kind: _made(stream, torch.empty, shape, dtype=kind,  # noqa: E731
                                         device=logits.device)
        out = dict(lse=make((n,), _F32), entropy=make((n,), _F32), logprobs=make((n, m), _F32),
                   top_ids=make((n, top), _I32), top_logprobs=make((n, top), _F32))
    get = out.get
    _check(lib().mmvq_token_logprobs(dtype, address, ld, n, vocab, scale,
                                     _plain(tokens, _I32, (n, m), dev, "tokens"), m, top,
                                     _list(get("lse"), _F32, n, dev, "lse"),
                                     _list(get("entropy"), _F32, n, dev, "entropy"),
                                     _plain(get("logprobs"), _F32, (n, m), dev, "logprobs"),
                                     _plain(get("top_ids"), _I32, (n, top), dev, "top_ids"),
                                     _plain(get("top_logprobs"), _F32, (n, top), dev,
                                            "top_logprobs"),
                                     _layer_status(status, dev), on),
           "mmvq_token_logprobs")
    return out
