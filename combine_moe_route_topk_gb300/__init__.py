"""Python binding of libmoe_route.so (GB300 MoE token routing).

Argument marshalling only: every step runs in the library's CUDA kernels.
Tensors are PyTorch CUDA tensors (device memory and streams come from
PyTorch); they are checked for device, contiguity and size before their raw
pointers are handed to the C ABI declared in ``include/moe_route.h``.

The library is built in-tree by ``combine_moe_route_topk_gb300._build``
(``__graft_entry__.build()``); importing an op without it raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import workloads  # noqa: F401  (re-exported for convenience)

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_route.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED = -2
MOE_ERR_CUDA = -3
MOE_ERR_CAPACITY = -4
MOE_ERR_TIMEOUT = -5

MOE_BF16, MOE_F32, MOE_FP8E4M3_BLK128 = 0, 1, 2
MOE_SOFTMAX, MOE_SIGMOID = 0, 1
MOE_EXPERT_LINEAR, MOE_EXPERT_SWIGLU = 0, 1  # include/moe_expert.h
MOE_BIAS_SELECT_ONLY = 0x10  # OR into score_fn: the bias enters the selection key only

STATUS_NAMES = {0: "MOE_OK", -1: "MOE_ERR_INVALID_ARG", -2: "MOE_ERR_UNSUPPORTED",
                -3: "MOE_ERR_CUDA", -4: "MOE_ERR_CAPACITY", -5: "MOE_ERR_TIMEOUT"}

_TORCH_DTYPE = {MOE_BF16: torch.bfloat16, MOE_F32: torch.float32, MOE_FP8E4M3_BLK128: torch.uint8}


class MoeError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(code, code)}: {msg}")
        self.code = code


class MoeDims(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("T", ctypes.c_int32), ("E", ctypes.c_int32),
                ("R", ctypes.c_int32), ("H", ctypes.c_int32), ("x_dtype", ctypes.c_int32),
                ("y_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("cap_rows", ctypes.c_int64)]


_SIZE_FIELDS = ["bound_rows", "cap_rows", "total_pairs", "logits_bytes", "topk_idx_bytes",
                "topk_w_bytes", "pos_bytes", "expert_counts_bytes", "expert_offsets_bytes",
                "rank_counts_bytes", "rank_offsets_bytes", "send_counts_bytes", "x_bytes",
                "x_scales_bytes", "packed_x_bytes", "packed_scales_bytes", "packed_src_bytes",
                "y_bytes", "out_bytes", "status_bytes", "partial_slots", "partial_bytes",
                "slot_rank_bytes", "fused_workspace_bytes"]


class MoeSizes(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int64) for f in _SIZE_FIELDS]

    def as_dict(self) -> dict:
        return {f: int(getattr(self, f)) for f in _SIZE_FIELDS}


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """Load libmoe_route.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; "
                    f"g.build()'` (needs nvcc); there is no fallback implementation")
            L = ctypes.CDLL(LIB_PATH)
            P, i32 = ctypes.c_void_p, ctypes.c_int
            D = ctypes.POINTER(MoeDims)
            L.moe_buffer_sizes.argtypes = [D, ctypes.POINTER(MoeSizes)]
            L.moe_route_topk.argtypes = [D, P, P, i32, i32, P, P, P]
            L.moe_dispatch_count.argtypes = [D, P, P, P, P, P, P, P, P, P]
            L.moe_dispatch_pack.argtypes = [D, P, P, P, P, P, P, P]
            L.moe_combine.argtypes = [D, P, P, P, P, P]
            L.moe_dispatch_pack_quant.argtypes = [D, P, P, P, P, P, P]
            L.moe_dispatch_pack_rank.argtypes = [D, i32, P, P, P, P, P, P, P]
            L.moe_dispatch_fused.argtypes = [D, P, P, i32, i32, P, P, P, P, P, P, P, P, P, P, P,
                                             P, P, P, P, P]
            L.moe_dispatch_fused_static.argtypes = [D, P, P, i32, i32, P, P, P, P, P, P, P, P, P,
                                                    P, P, P, P, P, P]
            L.moe_dispatch_fused_quant.argtypes = [D, P, P, i32, i32, P, P, P, P, P, P, P, P, P, P,
                                                   P, P, P, P, P]
            L.moe_combine_rank.argtypes = [D, i32, P, P, P, P, P]
            L.moe_combine_partials.argtypes = [D, P, P, P, P, P, P]
            L.moe_combine_reduce_partials.argtypes = [D, P, P, P, P]
            L.moe_expert_gemm.argtypes = [D, i32, i32, i32, P, P, P, P, P, P]
            L.moe_expert_gemm_dgrad.argtypes = [D, i32, i32, P, P, P, P, P]
            L.moe_expert_gemm_wgrad.argtypes = [D, i32, i32, P, P, P, P, i32, P]
            L.moe_expert_swiglu_grad.argtypes = [D, i32, P, P, P, P, P]
            L.moe_expert_gemm_fp8.argtypes = [D, i32, i32, i32, P, P, P, P, P, P, P, P]
            L.moe_expert_gemm_w4.argtypes = [D, i32, i32, i32, i32, P, P, P, P, P, P, P]
            L.moe_combine_grad.argtypes = [D, P, P, P, P, P, P, P]
            L.moe_dispatch_grad.argtypes = [D, P, P, P, P, P]
            L.moe_route_grad.argtypes = [D, P, P, i32, i32, P, P, P, P, P, P]
            L.moe_read_status.argtypes = [P, P]
            L.moe_take_device_error.argtypes = [P]
            L.moe_selftest_bounded_wait.argtypes = [P, ctypes.c_int64, P]
            L.moe_last_error.restype = ctypes.c_char_p
            L.moe_last_error.argtypes = []
            L.moe_version.restype = i32
            for fn in ("moe_buffer_sizes", "moe_route_topk", "moe_dispatch_count",
                       "moe_dispatch_pack", "moe_dispatch_pack_quant", "moe_dispatch_pack_rank",
                       "moe_dispatch_fused", "moe_dispatch_fused_static", "moe_dispatch_fused_quant",
                       "moe_combine", "moe_combine_rank", "moe_combine_partials",
                       "moe_combine_reduce_partials", "moe_expert_gemm", "moe_expert_gemm_dgrad",
                       "moe_expert_gemm_wgrad", "moe_expert_swiglu_grad", "moe_expert_gemm_fp8",
                       "moe_expert_gemm_w4", "moe_combine_grad", "moe_dispatch_grad", "moe_route_grad",
                       "moe_read_status",
                       "moe_take_device_error", "moe_selftest_bounded_wait"):
                getattr(L, fn).restype = i32
            _lib = L
    return _lib


def _check(rc: int) -> None:
    if rc != MOE_OK:
        raise MoeError(rc, lib().moe_last_error().decode())


def make_dims(N, T, E, R, H, x_dtype=MOE_BF16, y_dtype=MOE_BF16, cap_rows=0) -> MoeDims:
    return MoeDims(N, T, E, R, H, x_dtype, y_dtype, 0, cap_rows)


def dims_of(w) -> MoeDims:
    """MoeDims of a ``workloads.Workload``."""
    return make_dims(w.N, w.T, w.E, w.R, w.H, w.x_dtype, w.y_dtype, w.cap_rows)


_sizes_cache: dict = {}


def buffer_sizes(dims: MoeDims) -> dict:
    """Buffer sizes for ``dims`` (memoised: the query is pure host arithmetic)."""
    key = bytes(dims)
    hit = _sizes_cache.get(key)
    if hit is not None:
        return hit
    s = MoeSizes()
    _check(lib().moe_buffer_sizes(ctypes.byref(dims), ctypes.byref(s)))
    d = s.as_dict()
    if len(_sizes_cache) < 256:
        _sizes_cache[key] = d
    return d


# torch.cuda.current_device() without its check for lazy initialisation (0.2 us an argument): asked
# once a CUDA tensor is at hand
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream) -> int:
    """The stream's handle (None: the current one), as an integer for a void* argument."""
    if stream is None:  # the handle without a torch.cuda.Stream object, which costs 3 us
        return torch._C._cuda_getCurrentRawStream(_current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t: torch.Tensor | None, nbytes: int, name: str, dtype=None, optional=False):
    """t's address, as an integer for a void* argument, once t is seen to fit."""
    if (t is not None and t.is_cuda and t.get_device() == _current_device() and t.is_contiguous()
            and (dtype is None or t.dtype is dtype) and t.nbytes >= nbytes):
        return t.data_ptr()
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (got {t.device})")
    if t.get_device() != _current_device():
        raise ValueError(f"{name} is on {t.device}, not the current device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    raise ValueError(f"{name} holds {t.nbytes} bytes, needs {nbytes}")


def route_topk(dims: MoeDims, logits, bias, score_fn, renormalize, topk_idx, topk_w, stream=None):
    s = buffer_sizes(dims)
    _check(lib().moe_route_topk(
        ctypes.byref(dims), _ptr(logits, s["logits_bytes"], "logits", torch.float32),
        _ptr(bias, dims.E * 4, "bias", torch.float32, optional=True), int(score_fn),
        int(bool(renormalize)), _ptr(topk_idx, s["topk_idx_bytes"], "topk_idx", torch.int32),
        _ptr(topk_w, s["topk_w_bytes"], "topk_w", torch.float32), _stream(stream)))


def dispatch_count(dims: MoeDims, topk_idx, expert_counts, expert_offsets, rank_counts,
                   rank_offsets, send_counts, pos, status, stream=None):
    s = buffer_sizes(dims)
    i32 = torch.int32
    _check(lib().moe_dispatch_count(
        ctypes.byref(dims), _ptr(topk_idx, s["topk_idx_bytes"], "topk_idx", i32),
        _ptr(expert_counts, s["expert_counts_bytes"], "expert_counts", i32),
        _ptr(expert_offsets, s["expert_offsets_bytes"], "expert_offsets", i32),
        _ptr(rank_counts, s["rank_counts_bytes"], "rank_counts", i32),
        _ptr(rank_offsets, s["rank_offsets_bytes"], "rank_offsets", i32),
        _ptr(send_counts, s["send_counts_bytes"], "send_counts", i32),
        _ptr(pos, s["pos_bytes"], "pos", i32), _ptr(status, 4, "status", i32), _stream(stream)))


def dispatch_pack(dims: MoeDims, x, x_scales, pos, packed_x, packed_scales, packed_src,
                  stream=None):
    s = buffer_sizes(dims)
    fp8 = dims.x_dtype == MOE_FP8E4M3_BLK128
    _check(lib().moe_dispatch_pack(
        ctypes.byref(dims), _ptr(x, s["x_bytes"], "x", _TORCH_DTYPE[dims.x_dtype]),
        _ptr(x_scales, s["x_scales_bytes"], "x_scales", torch.float32, optional=not fp8),
        _ptr(pos, s["pos_bytes"], "pos", torch.int32),
        _ptr(packed_x, s["packed_x_bytes"], "packed_x", _TORCH_DTYPE[dims.x_dtype]),
        _ptr(packed_scales, s["packed_scales_bytes"], "packed_scales", torch.float32,
             optional=not fp8),
        _ptr(packed_src, s["packed_src_bytes"], "packed_src", torch.int32), _stream(stream)))


def dispatch_fused(dims: MoeDims, logits, bias, score_fn, renormalize, x, x_scales, topk_idx,
                   topk_w, expert_counts, expert_offsets, rank_counts, rank_offsets, send_counts,
                   pos, status, packed_x, packed_scales, packed_src, workspace, stream=None):
    """Route + count + pack in one launch (decode batches)."""
    s = buffer_sizes(dims)
    i32, f32 = torch.int32, torch.float32
    fp8 = dims.x_dtype == MOE_FP8E4M3_BLK128
    _check(lib().moe_dispatch_fused(
        ctypes.byref(dims), _ptr(logits, s["logits_bytes"], "logits", f32),
        _ptr(bias, dims.E * 4, "bias", f32, optional=True), int(score_fn), int(bool(renormalize)),
        _ptr(x, s["x_bytes"], "x", _TORCH_DTYPE[dims.x_dtype]),
        _ptr(x_scales, s["x_scales_bytes"], "x_scales", f32, optional=not fp8),
        _ptr(topk_idx, s["topk_idx_bytes"], "topk_idx", i32),
        _ptr(topk_w, s["topk_w_bytes"], "topk_w", f32),
        _ptr(expert_counts, s["expert_counts_bytes"], "expert_counts", i32),
        _ptr(expert_offsets, s["expert_offsets_bytes"], "expert_offsets", i32),
        _ptr(rank_counts, s["rank_counts_bytes"], "rank_counts", i32),
        _ptr(rank_offsets, s["rank_offsets_bytes"], "rank_offsets", i32),
        _ptr(send_counts, s["send_counts_bytes"], "send_counts", i32),
        _ptr(pos, s["pos_bytes"], "pos", i32), _ptr(status, 4, "status", i32),
        _ptr(packed_x, s["packed_x_bytes"], "packed_x", _TORCH_DTYPE[dims.x_dtype]),
        _ptr(packed_scales, s["packed_scales_bytes"], "packed_scales", f32, optional=not fp8),
        _ptr(packed_src, s["packed_src_bytes"], "packed_src", i32),
        _ptr(workspace, s["fused_workspace_bytes"], "workspace", optional=dims.N * dims.T == 0),
        _stream(stream)))


def dispatch_fused_static(dims: MoeDims, logits, bias, score_fn, renormalize, x, x_scales,
                          topk_idx, topk_w, expert_counts, expert_offsets, rank_counts,
                          rank_offsets, send_counts, pos, status, packed_x, packed_scales,
                          packed_src, stream=None):
    """moe_dispatch_fused with the library's own static scratch: nothing is
    allocated by the call (for callers that cannot allocate device memory
    when they dispatch).  Calls that overlap on the GPU race on the scratch."""
    s = buffer_sizes(dims)
    i32, f32 = torch.int32, torch.float32
    fp8 = dims.x_dtype == MOE_FP8E4M3_BLK128
    _check(lib().moe_dispatch_fused_static(
        ctypes.byref(dims), _ptr(logits, s["logits_bytes"], "logits", f32),
        _ptr(bias, dims.E * 4, "bias", f32, optional=True), int(score_fn), int(bool(renormalize)),
        _ptr(x, s["x_bytes"], "x", _TORCH_DTYPE[dims.x_dtype]),
        _ptr(x_scales, s["x_scales_bytes"], "x_scales", f32, optional=not fp8),
        _ptr(topk_idx, s["topk_idx_bytes"], "topk_idx", i32),
        _ptr(topk_w, s["topk_w_bytes"], "topk_w", f32),
        _ptr(expert_counts, s["expert_counts_bytes"], "expert_counts", i32),
        _ptr(expert_offsets, s["expert_offsets_bytes"], "expert_offsets", i32),
        _ptr(rank_counts, s["rank_counts_bytes"], "rank_counts", i32),
        _ptr(rank_offsets, s["rank_offsets_bytes"], "rank_offsets", i32),
        _ptr(send_counts, s["send_counts_bytes"], "send_counts", i32),
        _ptr(pos, s["pos_bytes"], "pos", i32), _ptr(status, 4, "status", i32),
        _ptr(packed_x, s["packed_x_bytes"], "packed_x", _TORCH_DTYPE[dims.x_dtype]),
        _ptr(packed_scales, s["packed_scales_bytes"], "packed_scales", f32, optional=not fp8),
        _ptr(packed_src, s["packed_src_bytes"], "packed_src", i32), _stream(stream)))


def fp8_dims(dims: MoeDims) -> MoeDims:
    """The same problem with fp8 block-scaled rows (sizes of quantised buffers)."""
    return make_dims(dims.N, dims.T, dims.E, dims.R, dims.H, MOE_FP8E4M3_BLK128, dims.y_dtype,
                     dims.cap_rows)


def dispatch_pack_quant(dims: MoeDims, x, pos, packed_q, packed_scales, packed_src,
                        stream=None):
    """Pack bf16 rows as e4m3 codes + one f32 scale per 128 elements."""
    s = buffer_sizes(dims)
    q = buffer_sizes(fp8_dims(dims))
    _check(lib().moe_dispatch_pack_quant(
        ctypes.byref(dims), _ptr(x, s["x_bytes"], "x", torch.bfloat16),
        _ptr(pos, s["pos_bytes"], "pos", torch.int32),
        _ptr(packed_q, q["packed_x_bytes"], "packed_q", torch.uint8),
        _ptr(packed_scales, q["packed_scales_bytes"], "packed_scales", torch.float32),
        _ptr(packed_src, s["packed_src_bytes"], "packed_src", torch.int32), _stream(stream)))


def dispatch_fused_quant(dims: MoeDims, logits, bias, score_fn, renormalize, x, topk_idx, topk_w,
                         expert_counts, expert_offsets, rank_counts, rank_offsets, send_counts, pos,
                         status, packed_q, packed_scales, packed_src, workspace, stream=None):
    """Route + count + fp8-quantising pack in one call (decode batches; bf16 rows
    in, e4m3 codes + one f32 scale per 128 elements out)."""
    s = buffer_sizes(dims)
    q = buffer_sizes(fp8_dims(dims))
    i32, f32 = torch.int32, torch.float32
    _check(lib().moe_dispatch_fused_quant(
        ctypes.byref(dims), _ptr(logits, s["logits_bytes"], "logits", f32),
        _ptr(bias, dims.E * 4, "bias", f32, optional=True), int(score_fn), int(bool(renormalize)),
        _ptr(x, s["x_bytes"], "x", torch.bfloat16),
        _ptr(topk_idx, s["topk_idx_bytes"], "topk_idx", i32),
        _ptr(topk_w, s["topk_w_bytes"], "topk_w", f32),
        _ptr(expert_counts, s["expert_counts_bytes"], "expert_counts", i32),
        _ptr(expert_offsets, s["expert_offsets_bytes"], "expert_offsets", i32),
        _ptr(rank_counts, s["rank_counts_bytes"], "rank_counts", i32),
        _ptr(rank_offsets, s["rank_offsets_bytes"], "rank_offsets", i32),
        _ptr(send_counts, s["send_counts_bytes"], "send_counts", i32),
        _ptr(pos, s["pos_bytes"], "pos", i32), _ptr(status, 4, "status", i32),
        _ptr(packed_q, q["packed_x_bytes"], "packed_q", torch.uint8),
        _ptr(packed_scales, q["packed_scales_bytes"], "packed_scales", f32),
        _ptr(packed_src, s["packed_src_bytes"], "packed_src", i32),
        _ptr(workspace, s["fused_workspace_bytes"], "workspace", optional=dims.N * dims.T == 0),
        _stream(stream)))


def _place(stream):
    """(current device, stream handle) of a call."""
    try:
        dev = _current_device()
    except RuntimeError:  # no driver: every tensor is refused by _on
        return None, None
    return dev, torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _expert_call(dims: MoeDims, stream):
    """(rows of the receive buffers, current device, stream handle) of a call."""
    return dims.N * buffer_sizes(dims)["cap_rows"], *_place(stream)


def _on(dev, t, nbytes: int, name: str, dtype):
    """_ptr for a call that has asked for its device once (0.4 us an argument instead of 0.6)."""
    if t is not None and t.get_device() == dev and t.dtype is dtype and t.is_contiguous() and t.nbytes >= nbytes:
        return t.data_ptr()
    return _ptr(t, nbytes, name, dtype)


def expert_gemm(dims: MoeDims, K: int, F: int, act: int, x, w, expert_offsets, y, pre=None,
                stream=None):
    """Each expert's rows times its matrix in bf16: y = x w^T (MOE_EXPERT_LINEAR, y of
    dims.y_dtype) or silu(g) * u of the gate and up halves (MOE_EXPERT_SWIGLU, y bf16,
    g and u kept in `pre` where given)."""
    (rows, dev, st), bf16 = _expert_call(dims, stream), torch.bfloat16
    gated = int(act) == MOE_EXPERT_SWIGLU
    yt = bf16 if gated else _TORCH_DTYPE[dims.y_dtype]
    _check(lib().moe_expert_gemm(
        ctypes.byref(dims), int(K), int(F), int(act), _on(dev, x, rows * K * 2, "x", bf16),
        _on(dev, w, dims.E * F * K * (4 if gated else 2), "w", bf16),
        _on(dev, expert_offsets, (dims.E + 1) * 4, "expert_offsets", torch.int32),
        _on(dev, y, rows * F * yt.itemsize, "y", yt),
        None if pre is None else _on(dev, pre, rows * F * 4, "pre", bf16), st))


def expert_gemm_dgrad(dims: MoeDims, K: int, F: int, dy, w, expert_offsets, dx, stream=None):
    """dx = dy w of each expert's rows (bf16)."""
    (rows, dev, st), bf16 = _expert_call(dims, stream), torch.bfloat16
    _check(lib().moe_expert_gemm_dgrad(
        ctypes.byref(dims), int(K), int(F), _on(dev, dy, rows * F * 2, "dy", bf16),
        _on(dev, w, dims.E * F * K * 2, "w", bf16),
        _on(dev, expert_offsets, (dims.E + 1) * 4, "expert_offsets", torch.int32),
        _on(dev, dx, rows * K * 2, "dx", bf16), st))


def expert_gemm_wgrad(dims: MoeDims, K: int, F: int, dy, x, expert_offsets, dw, stream=None):
    """dw[e] = dy^T x over e's rows, 0 without any (dw bf16 or f32, written whole)."""
    (rows, dev, st), bf16 = _expert_call(dims, stream), torch.bfloat16
    if dw is not None and dw.dtype not in (bf16, torch.float32):
        raise ValueError(f"dw must be {bf16} or {torch.float32} (got {dw.dtype})")
    f32 = dw is not None and dw.dtype == torch.float32
    _check(lib().moe_expert_gemm_wgrad(
        ctypes.byref(dims), int(K), int(F), _on(dev, dy, rows * F * 2, "dy", bf16),
        _on(dev, x, rows * K * 2, "x", bf16),
        _on(dev, expert_offsets, (dims.E + 1) * 4, "expert_offsets", torch.int32),
        _on(dev, dw, dims.E * F * K * (4 if f32 else 2), "dw", torch.float32 if f32 else bf16), MOE_F32 if f32 else MOE_BF16,
        st))


def expert_swiglu_grad(dims: MoeDims, F: int, pre, dh, expert_offsets, dpre, stream=None):
    """Gradient of silu(g) * u: dpre = (dg, du) from pre = (g, u) and dh (bf16)."""
    (rows, dev, st), bf16 = _expert_call(dims, stream), torch.bfloat16
    _check(lib().moe_expert_swiglu_grad(
        ctypes.byref(dims), int(F), _on(dev, pre, rows * F * 4, "pre", bf16),
        _on(dev, dh, rows * F * 2, "dh", bf16),
        _on(dev, expert_offsets, (dims.E + 1) * 4, "expert_offsets", torch.int32),
        _on(dev, dpre, rows * F * 4, "dpre", bf16), st))


def expert_gemm_fp8(dims: MoeDims, K: int, F: int, act: int, xq, x_scales, wq, w_scales,
                    expert_offsets, y, y_scales=None, stream=None):
    """Each expert's rows times its matrix in e4m3 with block scales (1 x 128 for the rows,
    128 x 128 for the matrices): y of dims.y_dtype (MOE_EXPERT_LINEAR), or silu(g) * u
    quantised again into codes y and scales y_scales (MOE_EXPERT_SWIGLU)."""
    (rows, dev, st), f32, u8 = _expert_call(dims, stream), torch.float32, torch.uint8
    gated = int(act) == MOE_EXPERT_SWIGLU
    W = F * (2 if gated else 1)
    yt = u8 if gated else _TORCH_DTYPE[dims.y_dtype]
    _check(lib().moe_expert_gemm_fp8(
        ctypes.byref(dims), int(K), int(F), int(act), _on(dev, xq, rows * K, "xq", u8),
        _on(dev, x_scales, rows * (K // 128) * 4, "x_scales", f32), _on(dev, wq, dims.E * W * K, "wq", u8),
        _on(dev, w_scales, dims.E * -(-W // 128) * (K // 128) * 4, "w_scales", f32),
        _on(dev, expert_offsets, (dims.E + 1) * 4, "expert_offsets", torch.int32),
        _on(dev, y, rows * F * yt.itemsize, "y", yt),
        None if y_scales is None and not gated else
        _on(dev, y_scales, rows * (F // 128) * 4, "y_scales", f32), st))


def pack_w4(q: torch.Tensor) -> torch.Tensor:
    """Whole numbers in [-8, 7] (integers [..., K], K % 8 == 0) as expert_gemm_w4's words, int32
    [..., K/8]: element 2j of eight at bit 4j, element 2j + 1 at bit 16 + 4j.  On q's device."""
    if q.shape[-1] % 8 != 0 or q.dtype.is_floating_point:
        raise ValueError(f"q must be integers, a multiple of 8 in a row (got {q.dtype} {tuple(q.shape)})")
    if q.numel() and (int(q.min()) < -8 or int(q.max()) > 7):
        raise ValueError("q must lie in [-8, 7]")
    q = q.unflatten(-1, (-1, 8))
    words = torch.zeros(q.shape[:-1], dtype=torch.int32, device=q.device)
    for i in range(8):
        words |= (q[..., i].to(torch.int32) & 15) << (4 * (i // 2) + 16 * (i % 2))
    return words


def quantize_w4(w: torch.Tensor, group: int):
    """Matrices [E][W][K] (of finite values) in expert_gemm_w4's form: (wq int32 [E][W][K/8],
    group_scales e4m3 as uint8 [E][K/group][W], row_scales f32 [E][W]).  A group's scale makes its
    largest magnitude 7; the row's scale makes the largest group's 448, e4m3's largest."""
    if w.dim() != 3 or group not in (32, 64, 128) or w.shape[-1] % group != 0:
        raise ValueError(f"w must be [E][W][K] with K a multiple of group 32, 64 or 128 (got {tuple(w.shape)}, {group})")
    E, W, K = w.shape
    wq = torch.empty(E, W, K // 8, dtype=torch.int32, device=w.device)
    group_scales = torch.empty(E, K // group, W, dtype=torch.uint8, device=w.device)
    row_scales = torch.empty(E, W, dtype=torch.float32, device=w.device)
    for e in range(E):  # one matrix at a time: what it needs on the way is four times its size
        m = w[e].float().view(W, K // group, group)
        want = m.abs().amax(dim=2) / 7.0
        row = want.amax(dim=1) / 448.0
        row = torch.where(row > 0, row, torch.ones_like(row))
        s = (want / row.unsqueeze(1)).clamp(max=448.0).to(torch.float8_e4m3fn)
        step = s.float() * row.unsqueeze(1)
        q = (m / torch.where(step > 0, step, torch.ones_like(step)).unsqueeze(2)).round_().clamp_(-8.0, 7.0)
        wq[e] = pack_w4(torch.where((step > 0).unsqueeze(2), q, 0.0).to(torch.int8).view(W, K))
        group_scales[e] = s.t().contiguous().view(torch.uint8)
        row_scales[e] = row
    return wq, group_scales, row_scales


_w4_sizes_cache: dict = {}


def _w4_sizes(dims: MoeDims, K: int, F: int, gated: bool, group: int):
    """(bytes of x, wq, group_scales, row_scales, expert_offsets and y, y's type) of a call (memoised like
    buffer_sizes: host arithmetic that took 0.8 us of a call's 9)."""
    key = (bytes(dims), K, F, gated, group)
    hit = _w4_sizes_cache.get(key)
    if hit is None:
        rows, E, W = dims.N * buffer_sizes(dims)["cap_rows"], dims.E, F * (2 if gated else 1)
        yt = torch.bfloat16 if gated else _TORCH_DTYPE[dims.y_dtype]
        hit = (rows * K * 2, E * W * K // 2, E * W * K // group if group in (32, 64, 128) else 0, E * W * 4,
               (E + 1) * 4, rows * F * yt.itemsize, yt)
        if len(_w4_sizes_cache) < 256:
            _w4_sizes_cache[key] = hit
    return hit


def expert_gemm_w4(dims: MoeDims, K: int, F: int, act: int, group: int, x, wq, group_scales, row_scales,
                   expert_offsets, y, stream=None):
    """Each expert's rows (bf16) times its matrix of 4-bit weights with group scales: y of
    dims.y_dtype (MOE_EXPERT_LINEAR), or silu(g) * u of the gate and up halves (MOE_EXPERT_SWIGLU,
    y bf16).  Weights as from quantize_w4; group_scales may be uint8 or float8_e4m3fn."""
    K, F, act, group = int(K), int(F), int(act), int(group)
    nx, nq, ng, nr, no, ny, yt = _w4_sizes(dims, K, F, act == MOE_EXPERT_SWIGLU, group)
    (dev, st), i32 = _place(stream), torch.int32
    e4m3 = torch.float8_e4m3fn
    st8 = e4m3 if group_scales is not None and group_scales.dtype is e4m3 else torch.uint8
    _check(lib().moe_expert_gemm_w4(
        ctypes.byref(dims), K, F, act, group, _on(dev, x, nx, "x", torch.bfloat16), _on(dev, wq, nq, "wq", i32),
        _on(dev, group_scales, ng, "group_scales", st8), _on(dev, row_scales, nr, "row_scales", torch.float32),
        _on(dev, expert_offsets, no, "expert_offsets", i32), _on(dev, y, ny, "y", yt), st))


def combine_grad(dims: MoeDims, dout, y, pos, topk_w, dy, dtopk_w, stream=None):
    """Gradient of combine: rows dy[pos] = topk_w * dout and dtopk_w = <dout, y[pos]>."""
    s = buffer_sizes(dims)
    yt = _TORCH_DTYPE[dims.y_dtype]
    (dev, st), f32 = _place(stream), torch.float32
    _check(lib().moe_combine_grad(
        ctypes.byref(dims), _on(dev, dout, s["out_bytes"], "dout", yt), _on(dev, y, s["y_bytes"], "y", yt),
        _on(dev, pos, s["pos_bytes"], "pos", torch.int32), _on(dev, topk_w, s["topk_w_bytes"], "topk_w", f32),
        _on(dev, dy, s["y_bytes"], "dy", yt), _on(dev, dtopk_w, s["topk_w_bytes"], "dtopk_w", f32), st))


def dispatch_grad(dims: MoeDims, dpacked, pos, dx, add=None, stream=None):
    """Gradient of dispatch_pack: dx = add + the sum of a token's rows of dpacked (add may be
    None, or dx itself)."""
    s = buffer_sizes(dims)
    xt = _TORCH_DTYPE[dims.x_dtype]
    dev, st = _place(stream)
    _check(lib().moe_dispatch_grad(
        ctypes.byref(dims), _on(dev, dpacked, s["packed_x_bytes"], "dpacked", xt),
        _on(dev, pos, s["pos_bytes"], "pos", torch.int32),
        None if add is None else _on(dev, add, s["x_bytes"], "add", xt), _on(dev, dx, s["x_bytes"], "dx", xt), st))


def route_grad(dims: MoeDims, logits, bias, score_fn, renormalize, topk_idx, topk_w, dtopk_w, dlogits,
               dbias=None, stream=None):
    """Gradient of route_topk's weights: dlogits, and their sum over the tokens as the gradient of
    a bias that is added to the logits."""
    s = buffer_sizes(dims)
    (dev, st), f32 = _place(stream), torch.float32
    _check(lib().moe_route_grad(
        ctypes.byref(dims), _on(dev, logits, s["logits_bytes"], "logits", f32),
        None if bias is None else _on(dev, bias, dims.E * 4, "bias", f32), int(score_fn), int(bool(renormalize)),
        _on(dev, topk_idx, s["topk_idx_bytes"], "topk_idx", torch.int32),
        _on(dev, topk_w, s["topk_w_bytes"], "topk_w", f32), _on(dev, dtopk_w, s["topk_w_bytes"], "dtopk_w", f32),
        _on(dev, dlogits, s["logits_bytes"], "dlogits", f32),
        None if dbias is None else _on(dev, dbias, dims.E * 4, "dbias", f32), st))


def combine(dims: MoeDims, y, pos, topk_w, out, stream=None):
    s = buffer_sizes(dims)
    yt = _TORCH_DTYPE[dims.y_dtype]
    _check(lib().moe_combine(
        ctypes.byref(dims), _ptr(y, s["y_bytes"], "y", yt),
        _ptr(pos, s["pos_bytes"], "pos", torch.int32),
        _ptr(topk_w, s["topk_w_bytes"], "topk_w", torch.float32),
        _ptr(out, s["out_bytes"], "out", yt), _stream(stream)))


def dispatch_pack_rank(dims: MoeDims, rank: int, x, x_scales, pos, packed_x, packed_scales,
                       packed_src, stream=None):
    """moe_dispatch_pack restricted to the pairs routed to rank `rank`."""
    s = buffer_sizes(dims)
    fp8 = dims.x_dtype == MOE_FP8E4M3_BLK128
    _check(lib().moe_dispatch_pack_rank(
        ctypes.byref(dims), int(rank), _ptr(x, s["x_bytes"], "x", _TORCH_DTYPE[dims.x_dtype]),
        _ptr(x_scales, s["x_scales_bytes"], "x_scales", torch.float32, optional=not fp8),
        _ptr(pos, s["pos_bytes"], "pos", torch.int32),
        _ptr(packed_x, s["packed_x_bytes"], "packed_x", _TORCH_DTYPE[dims.x_dtype]),
        _ptr(packed_scales, s["packed_scales_bytes"], "packed_scales", torch.float32,
             optional=not fp8),
        _ptr(packed_src, s["packed_src_bytes"], "packed_src", torch.int32), _stream(stream)))


def combine_rank(dims: MoeDims, rank: int, y, pos, topk_w, out, stream=None):
    """Local accumulation of rank `rank` (dense [N*T][H])."""
    s = buffer_sizes(dims)
    yt = _TORCH_DTYPE[dims.y_dtype]
    _check(lib().moe_combine_rank(
        ctypes.byref(dims), int(rank), _ptr(y, s["y_bytes"], "y", yt),
        _ptr(pos, s["pos_bytes"], "pos", torch.int32),
        _ptr(topk_w, s["topk_w_bytes"], "topk_w", torch.float32),
        _ptr(out, s["out_bytes"], "out", yt), _stream(stream)))


def combine_partials(dims: MoeDims, y, pos, topk_w, partial, slot_rank, stream=None):
    """Per (token, destination rank) partial rows and their ranks."""
    s = buffer_sizes(dims)
    yt = _TORCH_DTYPE[dims.y_dtype]
    _check(lib().moe_combine_partials(
        ctypes.byref(dims), _ptr(y, s["y_bytes"], "y", yt),
        _ptr(pos, s["pos_bytes"], "pos", torch.int32),
        _ptr(topk_w, s["topk_w_bytes"], "topk_w", torch.float32),
        _ptr(partial, s["partial_bytes"], "partial", yt),
        _ptr(slot_rank, s["slot_rank_bytes"], "slot_rank", torch.int32), _stream(stream)))


def combine_reduce_partials(dims: MoeDims, partial, slot_rank, out, stream=None):
    """out[g] = sum of token g's used partial rows."""
    s = buffer_sizes(dims)
    yt = _TORCH_DTYPE[dims.y_dtype]
    _check(lib().moe_combine_reduce_partials(
        ctypes.byref(dims), _ptr(partial, s["partial_bytes"], "partial", yt),
        _ptr(slot_rank, s["slot_rank_bytes"], "slot_rank", torch.int32),
        _ptr(out, s["out_bytes"], "out", yt), _stream(stream)))


def read_status(status, stream=None) -> int:
    """Wait for the stream and return the device status word of dispatch_count."""
    rc = lib().moe_read_status(_ptr(status, 4, "status", torch.int32), _stream(stream))
    if rc == MOE_ERR_CUDA:
        raise MoeError(rc, lib().moe_last_error().decode())
    return rc


def take_device_error(stream=None) -> int:
    """Wait for the stream; return and clear the library's device error word
    (MOE_OK, or MOE_ERR_TIMEOUT if a bounded wait in a kernel gave up)."""
    rc = lib().moe_take_device_error(_stream(stream))
    if rc == MOE_ERR_CUDA:
        raise MoeError(rc, lib().moe_last_error().decode())
    return rc


def selftest_bounded_wait(status, polls: int, stream=None) -> None:
    """Enqueue the bounded-wait self-test: status[0] becomes MOE_OK if
    status[1] turned nonzero within `polls` polls, else MOE_ERR_TIMEOUT."""
    _check(lib().moe_selftest_bounded_wait(_ptr(status, 8, "status", torch.int32), int(polls),
                                           _stream(stream)))


class Buffers:
    """Device buffers for one problem size, allocated with PyTorch.

    ``y`` aliases ``packed_x`` when the expert op keeps the dtype (the
    harness applies it in place); otherwise it is its own allocation.
    """

    def __init__(self, dims: MoeDims, device="cuda", separate_y: bool | None = None):
        self.dims = dims
        s = self.sizes = buffer_sizes(dims)
        N, T, E, R, H = dims.N, dims.T, dims.E, dims.R, dims.H
        NT, cap = N * T, s["cap_rows"]
        i32, f32 = torch.int32, torch.float32
        kw = dict(device=device)
        self.topk_idx = torch.empty(NT, R, dtype=i32, **kw)
        self.topk_w = torch.empty(NT, R, dtype=f32, **kw)
        self.pos = torch.empty(NT, R, dtype=i32, **kw)
        self.expert_counts = torch.empty(E, dtype=i32, **kw)
        self.expert_offsets = torch.empty(E + 1, dtype=i32, **kw)
        self.rank_counts = torch.empty(N, dtype=i32, **kw)
        self.rank_offsets = torch.empty(N + 1, dtype=i32, **kw)
        self.send_counts = torch.empty(N, N, dtype=i32, **kw)
        self.status = torch.zeros(1, dtype=i32, **kw)
        xt = _TORCH_DTYPE[dims.x_dtype]
        self.packed_x = torch.empty(N * cap, H, dtype=xt, **kw)
        spr = H // 128 if dims.x_dtype == MOE_FP8E4M3_BLK128 else 0
        self.packed_scales = torch.empty(N * cap, spr, dtype=f32, **kw) if spr else None
        self.packed_src = torch.empty(N * cap, dtype=i32, **kw)
        if separate_y is None:
            separate_y = dims.x_dtype != dims.y_dtype
        yt = _TORCH_DTYPE[dims.y_dtype]
        self.y = torch.empty(N * cap, H, dtype=yt, **kw) if separate_y else self.packed_x
        self.out = torch.empty(NT, H, dtype=yt, **kw)
