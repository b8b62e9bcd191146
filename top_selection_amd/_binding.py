"""ctypes binding of libdstopk.so (include/dstopk.h). Argument marshalling only.

Every step of top-k runs in the HIP kernels behind the C ABI; torch is used here for
device memory and streams only. There is no fallback: if the library is not built or
cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct
import threading
from typing import Dict, NamedTuple, Optional, Tuple

import numpy as np

BF16 = 0
FP32 = 1
E4M3 = 2
E5M2 = 3

DS_OK = 0
DS_ERR_INVALID_ARG = -1
DS_ERR_UNSUPPORTED = -2
DS_ERR_ALIGNMENT = -3
DS_ERR_WORKSPACE = -4
DS_ERR_LAUNCH = -5
DS_ERR_DEVICE = -6
DS_MAX_K = 4096
DS_NOALLOC_SCRATCH_BYTES = 8 << 20
PRESAMPLE_AUTO, PRESAMPLE_OFF, PRESAMPLE_ON = 0, 1, 2
MERGE_AUTO, MERGE_LISTS, MERGE_SELECT = 0, 1, 2
SCHEDULE_AUTO, SCHEDULE_FREE, SCHEDULE_LOCKSTEP = 0, 1, 2
OUTPUT_UNSORTED, OUTPUT_INDEX_INT64 = 1, 2
SHARE_AUTO, SHARE_OFF, SHARE_ON = 0, 1, 2
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
DS_MAX_EXPERTS = 1024
DS_MAX_ROUTE_K = 64
DS_MAX_ROUTE_GROUPS = 64
DS_MAX_DRAFTS = 64
DS_BLOCK = 128
DS_MAX_EXPERT_ALIGN = 1024
BLOCK_ROW, BLOCK_COLUMN, BLOCK_TILE = 0, 1, 2
GROUP_NONE, GROUP_ROWS, GROUP_INNER = 0, 1, 2
DS_EXACT_SUMS = 256

_HERE = os.path.dirname(os.path.abspath(__file__))
# DS_LIBRARY names another build of the library (e.g. one with host-side sanitizers)
LIB_PATH = os.environ.get("DS_LIBRARY") or os.path.join(_HERE, "libdstopk.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "dstopk.h")


class DSError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {ds_status_string(status)} ({status})")


class ds_config(ctypes.Structure):
    _fields_ = [("block", ctypes.c_int32), ("slack", ctypes.c_int32), ("slices", ctypes.c_int32),
                ("waves", ctypes.c_int32), ("presample", ctypes.c_int32), ("order_group", ctypes.c_int32),
                ("merge", ctypes.c_int32), ("schedule", ctypes.c_int32),
                ("depth", ctypes.c_int32), ("output", ctypes.c_int32), ("warmup", ctypes.c_int32),
                ("share", ctypes.c_int32)]


class ds_route_config(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32),
                ("group_top", ctypes.c_int32), ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float)]


class ds_expert_plan(ctypes.Structure):
    _fields_ = [("place", ctypes.c_void_p), ("order", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("capacity", ctypes.c_int64), ("k", ctypes.c_int32),
                ("experts", ctypes.c_int32), ("align", ctypes.c_int32)]


class ds_block_operand(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("stride", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("scale_rows", ctypes.c_int32)]


STATS_FIELDS = ["appended", "compactions", "work", "max_len", "reads", "index_sum", "monotone", "slice_lo",
                "slice_len", "block", "slack", "t_total_ns", "t_compact_ns", "t_sync_ns", "t_final_ns", "passes"]
STATS_DTYPE = np.dtype([(f, np.uint64) for f in STATS_FIELDS])

_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it is not built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() first")
            L = ctypes.CDLL(LIB_PATH)
            vp, i64, i32, u64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint64, ctypes.c_int
            cfgp = ctypes.POINTER(ds_config)
            L.ds_topk.argtypes = [vp, i64, i64, i64, ci, ci, u64, vp, vp, vp]
            L.ds_topk.restype = ci
            L.ds_topk_ex.argtypes = [vp, vp, i64, i64, i64, ci, ci, u64, vp, vp, vp, ctypes.c_size_t, cfgp, vp, vp]
            L.ds_topk_ex.restype = ci
            L.ds_topk_noalloc.argtypes = [vp, i64, i64, i64, ci, ci, u64, vp, vp, vp]
            L.ds_topk_noalloc.restype = ci
            L.ds_topk_slices.argtypes = [vp, vp, i64, i64, i64, ci, ci, u64, vp, vp, vp, ctypes.c_size_t, cfgp,
                                         vp, vp]
            L.ds_topk_slices.restype = ci
            L.ds_topk_merge.argtypes = [vp, i64, i64, ci, ci, u64, vp, vp, vp, ctypes.c_size_t, cfgp, vp]
            L.ds_topk_merge.restype = ci
            L.ds_topk_plan.argtypes = [i64, i64, ci, ci, cfgp, cfgp]
            L.ds_topk_plan.restype = ci
            L.ds_topk_workspace_size.argtypes = [i64, i64, ci, ci, cfgp, ctypes.POINTER(ctypes.c_size_t)]
            L.ds_topk_workspace_size.restype = ci
            L.ds_probe_read.argtypes = [vp, i64, vp, vp]
            L.ds_probe_read.restype = ci
            L.ds_probe_sink_words.argtypes = [i64]
            L.ds_probe_sink_words.restype = i64
            L.ds_probe_copy.argtypes = [vp, vp, i64, vp]
            L.ds_probe_copy.restype = ci
            rcp, szp, sz = ctypes.POINTER(ds_route_config), ctypes.POINTER(ctypes.c_size_t), ctypes.c_size_t
            L.ds_route.argtypes = [vp, i64, i64, i64, ci, ci, vp, rcp, vp, vp, vp, vp]
            L.ds_route.restype = ci
            L.ds_route_grad.argtypes = [vp, i64, i64, i64, ci, ci, rcp, vp, vp, vp, i64, vp]
            L.ds_route_grad.restype = ci
            L.ds_softmax.argtypes = [vp, i64, i64, i64, ci, vp, vp, i64, ci, vp, sz, vp]
            L.ds_softmax.restype = ci
            L.ds_softmax_workspace_size.argtypes = [i64, i64, ci, szp]
            L.ds_softmax_workspace_size.restype = ci
            L.ds_topk_softmax.argtypes = [vp, vp, i64, ci, ci, vp, vp, vp, i64, vp, i64, ci, vp, vp]
            L.ds_topk_softmax.restype = ci
            L.ds_verify.argtypes = [vp, i64, vp, i64, vp, vp, vp, vp, i64, ci, i64, ci, vp, vp, vp, sz, vp]
            L.ds_verify.restype = ci
            L.ds_verify_workspace_size.argtypes = [i64, i64, ci, szp]
            L.ds_verify_workspace_size.restype = ci
            plp, opp = vp, vp  # (a structure by reference, or its bytes)
            L.ds_expert_capacity.argtypes = [i64, ci, ci, ci, ctypes.POINTER(i64)]
            L.ds_expert_capacity.restype = ci
            L.ds_expert_sort.argtypes = [vp, plp, vp, sz, vp]
            L.ds_expert_sort.restype = ci
            L.ds_expert_sort_workspace_size.argtypes = [i64, ci, ci, szp]
            L.ds_expert_sort_workspace_size.restype = ci
            L.ds_expert_gather.argtypes = [vp, i64, i64, ci, plp, vp, i64, vp]
            L.ds_expert_gather.restype = ci
            L.ds_expert_combine.argtypes = [vp, i64, i64, ci, plp, vp, vp, i64, vp]
            L.ds_expert_combine.restype = ci
            L.ds_expert_combine_grad.argtypes = [vp, i64, vp, i64, i64, ci, plp, vp, vp, i64, vp, vp]
            L.ds_expert_combine_grad.restype = ci
            L.ds_block_quantize.argtypes = [vp, i64, i64, i64, ci, ci, plp, vp, i64, ci, vp, vp]
            L.ds_block_quantize.restype = ci
            L.ds_block_product.argtypes = [opp, opp, i64, i64, i64, ci, ci, vp, vp, i64, ci, vp]
            L.ds_block_product.restype = ci
            L.ds_status_string.argtypes = [ci]
            L.ds_status_string.restype = ctypes.c_char_p
            _lib = L
    return _lib


def header_functions() -> list:
    """Names of the functions include/dstopk.h declares."""
    text = open(HEADER_PATH).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[\w]+\s*\*?\s*(ds_\w+)\s*\(", text, flags=re.M)))


def ds_status_string(status: int) -> str:
    return lib().ds_status_string(int(status)).decode()


def _cfg(cfg: Optional[Dict[str, int]]):
    if cfg is None:
        return None
    c = ds_config(int(cfg.get("block", 0)), int(cfg.get("slack", 0)), int(cfg.get("slices", 0)),
                  int(cfg.get("waves", 0)), int(cfg.get("presample", 0)), int(cfg.get("order_group", 0)),
                  int(cfg.get("merge", 0)), int(cfg.get("schedule", 0)), 0, int(cfg.get("output", 0)),
                  int(cfg.get("warmup", 0)), int(cfg.get("share", 0)))
    return ctypes.pointer(c)


def ds_topk_plan(rows: int, n: int, k: int, dtype: int, cfg: Optional[Dict[str, int]] = None) -> Dict[str, int]:
    out = ds_config()
    st = lib().ds_topk_plan(rows, n, k, dtype, _cfg(cfg), ctypes.byref(out))
    if st != DS_OK:
        raise DSError(st, "ds_topk_plan")
    return {"block": out.block, "slack": out.slack, "slices": out.slices, "waves": out.waves,
            "presample": out.presample, "order_group": out.order_group, "merge": out.merge,
            "schedule": out.schedule, "depth": out.depth, "output": out.output, "warmup": out.warmup,
            "share": out.share}


def ds_topk_workspace_size(rows: int, n: int, k: int, dtype: int, cfg: Optional[Dict[str, int]] = None) -> int:
    b = ctypes.c_size_t(0)
    st = lib().ds_topk_workspace_size(rows, n, k, dtype, _cfg(cfg), ctypes.byref(b))
    if st != DS_OK:
        raise DSError(st, "ds_topk_workspace_size")
    return int(b.value)


# ----------------------------------------------------------------------------- torch-facing calls
def _torch():
    import torch  # noqa: WPS433 (device memory and streams only)
    return torch


def dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return FP32
    raise TypeError(f"unsupported dtype {t.dtype}; expected torch.bfloat16 or torch.float32")


def _stream_handle(stream, device=None) -> Optional[int]:
    """The hipStream_t of `stream`, or of torch's current stream on `device` (read without
    building a Stream object when torch offers the raw accessor)."""
    if stream is not None:
        return stream.cuda_stream
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        index = device.index if device is not None and device.index is not None else torch.cuda.current_device()
        return raw(index)
    return torch.cuda.current_stream().cuda_stream


def _prep(x, k: int, values: bool, indices: bool, out_vals, out_idx, idx64: bool = False):
    torch = _torch()
    if x.dim() != 2:
        raise ValueError("x must be 2-D [rows, N]")
    if not x.is_cuda:
        raise ValueError("x must be a device tensor")
    if x.shape[0] > 0 and x.stride(1) != 1:
        raise ValueError("rows of x must be contiguous (stride(1) == 1)")
    rows, n = x.shape
    dt = dtype_code(x)
    if values and out_vals is None:
        out_vals = torch.empty((rows, k), dtype=x.dtype, device=x.device)
    idt = torch.int64 if idx64 else torch.int32
    if indices and out_idx is None:
        out_idx = torch.empty((rows, k), dtype=idt, device=x.device)
    for o, want in ((out_vals, x.dtype), (out_idx, idt)):
        if o is not None and (o.dtype != want or not o.is_contiguous() or tuple(o.shape) != (rows, k)):
            raise ValueError("outputs must be contiguous [rows, k] of the input dtype / the index type")
    row_stride = x.stride(0) if rows > 0 else n
    return rows, n, row_stride, dt, out_vals, out_idx


def ds_topk(x, k: int, seed: int = 0, values: bool = True, indices: bool = True, out_vals=None, out_idx=None,
            stream=None) -> Tuple[Optional[object], Optional[object]]:
    """Top-k of every row of the 2-D device tensor x (bf16 or fp32); see include/dstopk.h.

    Returns (values [rows,k] of x's dtype, indices [rows,k] int32), sorted by value
    descending (+0 before -0), ties by smaller index. Enqueued on `stream` (default: the
    current torch stream); no synchronisation.
    """
    rows, n, rs, dt, out_vals, out_idx = _prep(x, k, values, indices, out_vals, out_idx)
    st = lib().ds_topk(x.data_ptr() if rows else None, rows, n, rs, k, dt, seed & 0xFFFFFFFFFFFFFFFF,
                       out_vals.data_ptr() if out_vals is not None else None,
                       out_idx.data_ptr() if out_idx is not None else None, _stream_handle(stream, x.device))
    if st != DS_OK:
        raise DSError(st, "ds_topk")
    return out_vals, out_idx


def ds_topk_noalloc(x, k: int, seed: int = 0, values: bool = True, indices: bool = True, out_vals=None,
                    out_idx=None, stream=None) -> Tuple[Optional[object], Optional[object]]:
    """ds_topk whose workspace is the library's fixed per-GPU device array (no device
    allocation by the library; outputs not given are allocated here by torch). Raises
    DSError(DS_ERR_WORKSPACE) when the plan needs more than DS_NOALLOC_SCRATCH_BYTES."""
    rows, n, rs, dt, out_vals, out_idx = _prep(x, k, values, indices, out_vals, out_idx)
    st = lib().ds_topk_noalloc(x.data_ptr() if rows else None, rows, n, rs, k, dt, seed & 0xFFFFFFFFFFFFFFFF,
                               out_vals.data_ptr() if out_vals is not None else None,
                               out_idx.data_ptr() if out_idx is not None else None, _stream_handle(stream, x.device))
    if st != DS_OK:
        raise DSError(st, "ds_topk_noalloc")
    return out_vals, out_idx


def _idx64(cfg) -> bool:
    return bool(cfg and int(cfg.get("output", 0)) & OUTPUT_INDEX_INT64)


def _lens_ptr(lens, rows: int):
    if lens is None:
        return None
    torch = _torch()
    if not lens.is_cuda or lens.dtype != torch.int32 or not lens.is_contiguous() or lens.numel() != rows:
        raise ValueError("lens must be a contiguous device int32 tensor of one length per row")
    return lens.data_ptr()


def ds_topk_ex(x, k: int, seed: int = 0, workspace=None, cfg: Optional[Dict[str, int]] = None, stats=None,
               values: bool = True, indices: bool = True, out_vals=None, out_idx=None, stream=None, lens=None):
    """ds_topk with a caller workspace (a device tensor), forced config (including the output
    flags), optional stats (a device uint8 tensor of rows*slices*128 bytes) and optional
    per-row lengths (a device int32 tensor [rows]). Allocates nothing itself beyond the
    outputs it is not given."""
    rows, n, rs, dt, out_vals, out_idx = _prep(x, k, values, indices, out_vals, out_idx, _idx64(cfg))
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(),
                                                            workspace.numel() * workspace.element_size())
    st = lib().ds_topk_ex(x.data_ptr() if rows else None, _lens_ptr(lens, rows), rows, n, rs, k, dt,
                          seed & 0xFFFFFFFFFFFFFFFF,
                          out_vals.data_ptr() if out_vals is not None else None,
                          out_idx.data_ptr() if out_idx is not None else None, ws_ptr, ws_bytes, _cfg(cfg),
                          stats.data_ptr() if stats is not None else None, _stream_handle(stream, x.device))
    if st != DS_OK:
        raise DSError(st, "ds_topk_ex")
    return out_vals, out_idx


def ds_topk_slices(x, k: int, seed: int = 0, workspace=None, cfg: Optional[Dict[str, int]] = None, stats=None,
                   out_vals=None, out_idx=None, values: bool = True, indices: bool = True, stream=None, lens=None):
    """First launch of ds_topk_ex (the select kernel); returns the outputs it may fill."""
    rows, n, rs, dt, out_vals, out_idx = _prep(x, k, values, indices, out_vals, out_idx, _idx64(cfg))
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(),
                                                            workspace.numel() * workspace.element_size())
    st = lib().ds_topk_slices(x.data_ptr() if rows else None, _lens_ptr(lens, rows), rows, n, rs, k, dt,
                              seed & 0xFFFFFFFFFFFFFFFF,
                              out_vals.data_ptr() if out_vals is not None else None,
                              out_idx.data_ptr() if out_idx is not None else None, ws_ptr, ws_bytes, _cfg(cfg),
                              stats.data_ptr() if stats is not None else None, _stream_handle(stream, x.device))
    if st != DS_OK:
        raise DSError(st, "ds_topk_slices")
    return out_vals, out_idx


def ds_topk_merge(rows: int, n: int, k: int, dtype: int, seed: int = 0, workspace=None,
                  cfg: Optional[Dict[str, int]] = None, out_vals=None, out_idx=None, stream=None, lens=None):
    """Second launch of ds_topk_ex (the merge kernel) into the given output tensors."""
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(),
                                                            workspace.numel() * workspace.element_size())
    st = lib().ds_topk_merge(_lens_ptr(lens, rows), rows, n, k, dtype, seed & 0xFFFFFFFFFFFFFFFF,
                             out_vals.data_ptr() if out_vals is not None else None,
                             out_idx.data_ptr() if out_idx is not None else None, ws_ptr, ws_bytes, _cfg(cfg),
                             _stream_handle(stream, out_vals.device if out_vals is not None else
                                            (out_idx.device if out_idx is not None else None)))
    if st != DS_OK:
        raise DSError(st, "ds_topk_merge")
    return out_vals, out_idx


# ------------------------------------------------------- the operators beside the selection
# These calls are short (small batches of a serving loop), so their checks read each property
# once and the C functions are looked up once.
_functions: Dict[str, object] = {}
_sizes: Dict[tuple, int] = {}
_codes: Dict[object, int] = {}  # torch dtypes, once one was asked for


def _function(name: str):
    f = _functions.get(name)
    if f is None:
        f = _functions[name] = getattr(lib(), name)
    return f


def _code(dtype) -> int:
    """The element type's code (dtype_code of a tensor's dtype)."""
    code = _codes.get(dtype)
    if code is None:
        torch = _torch()
        _codes.update({torch.bfloat16: BF16, torch.float32: FP32})
        code = _codes.get(dtype)
        if code is None:
            raise TypeError(f"unsupported dtype {dtype}; expected torch.bfloat16 or torch.float32")
    return code


def _matrix(x, what: str):
    """rows, n, row stride of a 2-D device tensor with contiguous rows."""
    if x.dim() != 2:
        raise ValueError(f"{what} must be 2-D")
    if not x.is_cuda:
        raise ValueError(f"{what} must be a device tensor")
    rows, n = x.shape
    stride, one = x.stride()
    if one != 1 and n > 1:
        raise ValueError(f"rows of {what} must be contiguous (stride(-1) == 1)")
    return rows, n, stride if rows > 1 else max(n, 1)


def _batch_rows(x, what: str):
    """batch, rows per sequence, n, row stride of a 3-D device tensor whose rows lie evenly apart."""
    if x.dim() != 3:
        raise ValueError(f"{what} must be 3-D")
    if not x.is_cuda:
        raise ValueError(f"{what} must be a device tensor")
    b, m, n = x.shape
    of_b, of_m, one = x.stride()
    if one != 1 and n > 1:
        raise ValueError(f"rows of {what} must be contiguous (stride(-1) == 1)")
    if m > 1:
        if b > 1 and of_b != m * of_m:
            raise ValueError(f"rows of {what} must lie evenly apart (stride(0) == shape[1] * stride(1))")
        return b, m, n, of_m
    return b, m, n, of_b if b > 1 else max(n, 1)


def _operand(t, what: str, dtype, shape, device):
    """The address of an optional contiguous device tensor of the given type, shape and device."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t.data_ptr()


def _call(name: str, device, stream, *args) -> None:
    """Calls the C entry with the stream last, with `device` current (the stream is the given
    one, or torch's current stream on that device)."""
    f = _functions.get(name) or _function(name)
    torch = _torch()
    index = device.index
    if index == torch._C._cuda_getDevice():
        st = f(*args, torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(device):
            st = f(*args, _stream_handle(stream, device))
    if st != DS_OK:
        raise DSError(st, name)


def _workspace_size(name: str, rows: int, n: int, dtype: int) -> int:
    key = (name, rows, n, dtype)
    size = _sizes.get(key)
    if size is None:
        b = ctypes.c_size_t(0)
        st = _function(name)(rows, n, dtype, ctypes.byref(b))
        if st != DS_OK:
            raise DSError(st, name)
        if len(_sizes) >= 4096:
            _sizes.clear()
        size = _sizes[key] = int(b.value)
    return size


def ds_softmax_workspace_size(rows: int, n: int, dtype: int) -> int:
    return _workspace_size("ds_softmax_workspace_size", rows, n, dtype)


def ds_verify_workspace_size(batch: int, n: int, dtype: int) -> int:
    return _workspace_size("ds_verify_workspace_size", batch, n, dtype)


def _empty(shape, dtype, device, stream):
    """A new tensor for work on `stream` (torch's current one if None): memory that torch's allocator
    hands out is free for the stream it is asked for on, and for no other."""
    torch = _torch()
    steps = (1,) if len(shape) == 1 else (shape[1], 1)
    if stream is None:  # (with its strides given the allocation takes 1.25 us in place of 1.6)
        return torch.empty_strided(shape, steps, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty_strided(shape, steps, dtype=dtype, device=device)


def _scratch(need: int, workspace, device, stream):
    """The call's workspace (to be kept until the call has been made), its address and its bytes:
    the one given, or a new one of the needed size."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = _empty((need,), _torch().uint8, device, stream)
        return workspace, workspace.data_ptr(), need
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def ds_route(x, k: int, bias=None, score: int = SCORE_SOFTMAX, groups: int = 1, topk_groups: int = 0,
             group_top: int = 1, renormalize: bool = False, scale: float = 1.0, counts=None, weights: bool = True,
             out_weights=None, out_idx=None, stream=None):
    """The k experts of every row of the logits x [rows, experts] (bf16 or fp32) and their
    weights; see include/dstopk.h.

    Returns (weights [rows, k] fp32 or None, indices [rows, k] int32). bias: fp32 [experts],
    moves the choice only. counts: int32 [experts], gets the rows that chose each expert added.
    Outside torch's autograd, as every call here: an x that requires a gradient gets it from
    ds_route_grad, which the caller's backward pass calls.
    """
    torch = _torch()
    rows, n, rs = _matrix(x, "x")
    dt, dev, shape = _code(x.dtype), x.device, (rows, k)
    if out_weights is not None:
        wp = _operand(out_weights, "out_weights", torch.float32, shape, dev)
    elif weights:
        out_weights = _empty(shape, torch.float32, dev, stream)
        wp = out_weights.data_ptr()
    else:
        wp = None
    if out_idx is not None:
        ip = _operand(out_idx, "out_idx", torch.int32, shape, dev)
    else:
        out_idx = _empty(shape, torch.int32, dev, stream)
        ip = out_idx.data_ptr()
    cfg = ds_route_config(score, groups, topk_groups, group_top, 1 if renormalize else 0, scale)
    _call("ds_route", dev, stream, x.data_ptr(), rows, n, rs, k, dt,
          None if bias is None else _operand(bias, "bias", torch.float32, (n,), dev), ctypes.byref(cfg), wp, ip,
          None if counts is None else _operand(counts, "counts", torch.int32, (n,), dev))
    return out_weights, out_idx


def ds_route_grad(x, idx, grad_weights, score: int = SCORE_SOFTMAX, renormalize: bool = False, scale: float = 1.0,
                  out=None, stream=None):
    """The gradient of ds_route's weights to its logits x, for the chosen experts idx [rows, k]
    int32 and the weights' gradient [rows, k] fp32; [rows, experts] of x's dtype. out may be x."""
    torch = _torch()
    rows, n, rs = _matrix(x, "x")
    dt, dev = _code(x.dtype), x.device
    if idx.dim() != 2:
        raise ValueError("idx must be 2-D [rows, k]")
    shape = (rows, idx.shape[1])
    if out is None:
        out, os = _empty((rows, n), x.dtype, dev, stream), n
    else:
        _, _, os = _matrix(out, "out")
        if out.dtype != x.dtype or out.shape != (rows, n) or out.device != dev:
            raise ValueError("out must be [rows, experts] of x's dtype on x's device")
    cfg = ds_route_config(score, 1, 1, 1, 1 if renormalize else 0, scale)
    _call("ds_route_grad", dev, stream, x.data_ptr(), rows, n, rs, shape[1], dt, ctypes.byref(cfg),
          _operand(idx, "idx", torch.int32, shape, dev),
          _operand(grad_weights, "grad_weights", torch.float32, shape, dev), out.data_ptr(), os)
    return out


def _out_rows(out, out_dtype, rows: int, n: int, dev, stream):
    torch = _torch()
    if out is None:
        return _empty((rows, n), out_dtype or torch.float32, dev, stream), n
    _, _, os = _matrix(out, "out")
    if out.shape != (rows, n) or out.device != dev or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError("out must be [rows, n] of out_dtype on the inputs' device")
    return out, os


def ds_softmax(x, temperature=None, out_dtype=None, out=None, workspace=None, stream=None):
    """Probabilities [rows, n] (fp32, or out_dtype / out's type) of the logits x [rows, n] (bf16
    or fp32) at a temperature per row (fp32 [rows] on the device; not above 0: one-hot at the
    first maximum); see include/dstopk.h. out shares no memory with x."""
    torch = _torch()
    rows, n, rs = _matrix(x, "x")
    dt, dev = _code(x.dtype), x.device
    out, os = _out_rows(out, out_dtype, rows, n, dev, stream)
    keep, ws, ws_bytes = _scratch(ds_softmax_workspace_size(rows, n, dt), workspace, dev, stream)
    _call("ds_softmax", dev, stream, x.data_ptr(), rows, n, rs, dt,
          None if temperature is None else _operand(temperature, "temperature", torch.float32, (rows,), dev),
          out.data_ptr(), os, _code(out.dtype), ws, ws_bytes)
    return out


def ds_topk_softmax(vals, idx, n: int, ks=None, temperature=None, top_p=None, out_dtype=None, out=None,
                    out_list=None, rows_out: bool = True, stream=None):
    """Probabilities of the rows' top-k lists (vals, idx) [rows, k] as ds_topk returns them, as
    whole rows [rows, n] (zeros elsewhere): the first ks[r] entries (int32 [rows]) at
    temperature[r], cut to the shortest prefix that holds top_p[r] of their mass (both fp32
    [rows]). out_list: an fp32 [rows, k] tensor that gets the entries' probabilities too.
    rows_out=False: only the list is written. Returns the whole rows, or out_list."""
    torch = _torch()
    if vals.dim() != 2 or not vals.is_cuda or not vals.is_contiguous():
        raise ValueError("vals must be a contiguous 2-D device tensor [rows, k]")
    rows, k = shape = vals.shape
    dt, dev, f32 = _code(vals.dtype), vals.device, torch.float32
    if rows_out:
        out, os = _out_rows(out, out_dtype, rows, n, dev, stream)
        op, odt = out.data_ptr(), _code(out.dtype)
    else:
        op, os, odt = None, n, FP32
        if out_list is None:
            out_list = _empty(shape, f32, dev, stream)
    per_row = (rows,)
    _call("ds_topk_softmax", dev, stream, vals.data_ptr(), _operand(idx, "idx", torch.int32, shape, dev), rows, k, dt,
          None if ks is None else _operand(ks, "ks", torch.int32, per_row, dev),
          None if temperature is None else _operand(temperature, "temperature", f32, per_row, dev),
          None if top_p is None else _operand(top_p, "top_p", f32, per_row, dev), n, op, os, odt,
          None if out_list is None else _operand(out_list, "out_list", f32, shape, dev))
    return out if rows_out else out_list


def ds_verify(target, draft, draft_tokens, accept_u, sample_u, draft_lens=None, out_tokens=None, out_accepted=None,
              workspace=None, stream=None):
    """Verification of drafted tokens: target [batch, drafts + 1, n] and draft [batch, drafts, n]
    (or None: certain drafts) probabilities, bf16 or fp32; draft_tokens int32 and accept_u fp32
    [batch, drafts]; sample_u fp32 [batch]; draft_lens int32 [batch]. See include/dstopk.h.

    Returns (tokens [batch, drafts + 1] int32: the accepted drafts, the drawn token, then -1;
    accepted [batch] int32).
    """
    torch = _torch()
    batch, m, n, ts = _batch_rows(target, "target")
    dt, dev, K = _code(target.dtype), target.device, m - 1
    if K < 0:
        raise ValueError("target must hold at least one row per sequence")
    if sample_u is None or (K > 0 and (draft_tokens is None or accept_u is None)):
        raise ValueError("draft_tokens, accept_u and sample_u are needed")
    dp, dstride = None, n
    if draft is not None and K > 0:
        b2, k2, n2, dstride = _batch_rows(draft, "draft")
        if (b2, k2, n2) != (batch, K, n) or draft.dtype != target.dtype or draft.device != dev:
            raise ValueError("draft must be [batch, drafts, n] of target's dtype on its device")
        dp = draft.data_ptr()
    i32, f32, each, per_seq = torch.int32, torch.float32, (batch, K), (batch,)
    if out_tokens is None:
        out_tokens = _empty((batch, m), i32, dev, stream)
        tp = out_tokens.data_ptr()
    else:
        tp = _operand(out_tokens, "out_tokens", i32, (batch, m), dev)
    if out_accepted is None:
        out_accepted = _empty(per_seq, i32, dev, stream)
        ap = out_accepted.data_ptr()
    else:
        ap = _operand(out_accepted, "out_accepted", i32, per_seq, dev)
    keep, ws, ws_bytes = _scratch(ds_verify_workspace_size(batch, n, dt), workspace, dev, stream)
    _call("ds_verify", dev, stream, target.data_ptr(), ts, dp, dstride,
          _operand(draft_tokens, "draft_tokens", i32, each, dev),
          None if draft_lens is None else _operand(draft_lens, "draft_lens", i32, per_seq, dev),
          _operand(accept_u, "accept_u", f32, each, dev), _operand(sample_u, "sample_u", f32, per_seq, dev),
          batch, K, n, dt, tp, ap, ws, ws_bytes)
    return out_tokens, out_accepted


# ------------------------------------------------------------------------- behind a router
class ExpertPlan(NamedTuple):
    """Where the slots of rows [rows, k] lie when sorted by expert (see include/dstopk.h): int32
    device tensors place [rows, k] (a slot's position, or -1), order [capacity] (a position's slot, or
    -1) and offsets [experts + 1]; every expert's segment is a multiple of align long."""
    place: object
    order: object
    offsets: object
    align: int = 1


# ds_expert_plan and ds_block_operand as bytes: a third of the time of filling a ctypes structure
_pack_plan = struct.Struct("@PPPqqiiii").pack
_pack_operand = struct.Struct("@PPqii").pack


def _plan(plan: ExpertPlan, device):
    """The plan as the C entries take it (the bytes of a ds_expert_plan), its rows and its capacity."""
    i32, at = _torch().int32, device.index
    place, order, offsets, align = plan
    if not (place.dtype is i32 and order.dtype is i32 and offsets.dtype is i32 and place.get_device() == at
            and order.get_device() == at and offsets.get_device() == at and place.is_contiguous()
            and order.is_contiguous() and offsets.is_contiguous()):
        raise ValueError(f"a plan's tensors must be contiguous int32 tensors on {device}")
    try:
        rows, k = place.shape
        capacity, = order.shape
        ends, = offsets.shape
    except ValueError:
        raise ValueError("a plan's place must be 2-D, order and offsets 1-D") from None
    return _pack_plan(place.data_ptr(), order.data_ptr(), offsets.data_ptr(), rows, capacity, k, ends - 1, align,
                      0), rows, capacity


def ds_expert_capacity(rows: int, k: int, experts: int, align: int = 1) -> int:
    """The length of a plan's order: positions that hold every choice of experts."""
    key = ("ds_expert_capacity", rows, k, experts, align)
    size = _sizes.get(key)
    if size is None:
        c = ctypes.c_int64(0)
        st = _function("ds_expert_capacity")(rows, k, experts, align, ctypes.byref(c))
        if st != DS_OK:
            raise DSError(st, "ds_expert_capacity")
        if len(_sizes) >= 4096:
            _sizes.clear()
        size = _sizes[key] = int(c.value)
    return size


def ds_expert_sort_workspace_size(rows: int, k: int, experts: int) -> int:
    return _workspace_size("ds_expert_sort_workspace_size", rows, k, experts)


def ds_expert_sort(idx, experts: int, align: int = 1, out: Optional[ExpertPlan] = None, workspace=None,
                   stream=None) -> ExpertPlan:
    """The slots of idx [rows, k] (int32, as ds_route returns them) sorted by expert; entries outside
    [0, experts) are slots without an expert. out: a plan of the same sizes whose tensors are written."""
    torch = _torch()
    if idx.dim() != 2 or idx.dtype != torch.int32 or not idx.is_cuda or not idx.is_contiguous():
        raise ValueError("idx must be a contiguous 2-D int32 device tensor [rows, k]")
    shape, dev, i32 = idx.shape, idx.device, torch.int32
    rows, k = shape
    if out is None:
        capacity = ds_expert_capacity(rows, k, experts, align)
        place, order = _empty(shape, i32, dev, stream), _empty((capacity,), i32, dev, stream)
        offsets = _empty((experts + 1,), i32, dev, stream)
        out = ExpertPlan(place, order, offsets, align)
        plan = _pack_plan(place.data_ptr(), order.data_ptr(), offsets.data_ptr(), rows, capacity, k, experts, align, 0)
    elif out.place.shape != shape or out.offsets.shape != (experts + 1,) or out.align != align:
        raise ValueError("out must be a plan of idx's shape, of the experts and of the alignment")
    else:
        plan, _, _ = _plan(out, dev)
    keep, ws, ws_bytes = _scratch(ds_expert_sort_workspace_size(rows, k, experts), workspace, dev, stream)
    _call("ds_expert_sort", dev, stream, idx.data_ptr(), plan, ws, ws_bytes)
    return out


def _rows_out(out, rows: int, n: int, dtype, dev, stream, what: str = "out"):
    """An output matrix and its row stride: the one given, or a new one."""
    if out is None:
        return _empty((rows, n), dtype, dev, stream), n
    _, _, stride = _matrix(out, what)
    if out.shape != (rows, n) or out.dtype != dtype or out.device != dev:
        raise ValueError(f"{what} must be a [{rows}, {n}] tensor of {dtype} on {dev}")
    return out, stride


def ds_expert_gather(x, plan: ExpertPlan, out=None, stream=None):
    """Every row of x [rows, n] (bf16 or fp32) at its slots' positions: [capacity, n], zeros in the
    segments' padding, and from the plan's end on what out held (uninitialised in a new tensor). Its
    gradient is ds_expert_combine without weights."""
    rows, n, rs = _matrix(x, "x")
    dt, dev = _code(x.dtype), x.device
    c, plan_rows, capacity = _plan(plan, dev)
    if plan_rows != rows:
        raise ValueError("x must have the plan's rows")
    out, os = _rows_out(out, capacity, n, x.dtype, dev, stream)
    _call("ds_expert_gather", dev, stream, x.data_ptr(), n, rs, dt, c, out.data_ptr(), os)
    return out


def ds_expert_combine(y, plan: ExpertPlan, weights=None, out=None, stream=None):
    """The rows back: [rows, n], row r the sum of weights[r, j] (fp32; None: 1) times y's row at slot
    (r, j)'s position, y [capacity, n] (bf16 or fp32). The gradient is ds_expert_combine_grad."""
    capacity, n, ys = _matrix(y, "y")
    dt, dev = _code(y.dtype), y.device
    c, rows, plan_capacity = _plan(plan, dev)
    if plan_capacity != capacity:
        raise ValueError("y must have the plan's capacity of rows")
    out, os = _rows_out(out, rows, n, y.dtype, dev, stream)
    _call("ds_expert_combine", dev, stream, y.data_ptr(), n, ys, dt, c,
          None if weights is None else _operand(weights, "weights", _torch().float32, plan.place.shape, dev),
          out.data_ptr(), os)
    return out


def ds_expert_combine_grad(grad, y, plan: ExpertPlan, weights=None, grad_y: bool = True, grad_weights: bool = True,
                           out_y=None, out_weights=None, stream=None):
    """The gradients of ds_expert_combine for grad [rows, n], the gradient of its result: (grad_y
    [capacity, n] or None, grad_weights [rows, k] fp32 or None). From the plan's end on grad_y holds what
    out_y held. out_y may be y itself. y may be None when grad_weights is False."""
    torch = _torch()
    rows, n, gs = _matrix(grad, "grad")
    dt, dev = _code(grad.dtype), grad.device
    c, plan_rows, capacity = _plan(plan, dev)
    if plan_rows != rows:
        raise ValueError("grad must have the plan's rows")
    yp, ys, op, os, wp = None, n, None, n, None
    if grad_weights:
        if y is None:
            raise ValueError("y is needed for the weights' gradient")
        _, _, ys = _matrix(y, "y")
        if y.shape != (capacity, n) or y.dtype != grad.dtype or y.device != dev:
            raise ValueError("y must be [capacity, n] of grad's dtype on its device")
        yp = y.data_ptr()
        if out_weights is None:
            out_weights = _empty(plan.place.shape, torch.float32, dev, stream)
        wp = _operand(out_weights, "out_weights", torch.float32, plan.place.shape, dev)
    if grad_y:
        out_y, os = _rows_out(out_y, capacity, n, grad.dtype, dev, stream, "out_y")
        op = out_y.data_ptr()
    _call("ds_expert_combine_grad", dev, stream, grad.data_ptr(), gs, yp, ys, n, dt, c,
          None if weights is None else _operand(weights, "weights", torch.float32, plan.place.shape, dev), op, os, wp)
    return out_y if grad_y else None, out_weights if grad_weights else None


_codes8: Dict[object, int] = {}


def _code8(dtype) -> int:
    code = _codes8.get(dtype)
    if code is None:
        torch = _torch()
        _codes8.update({torch.float8_e4m3fn: E4M3, torch.float8_e5m2: E5M2})
        code = _codes8.get(dtype)
        if code is None:
            raise TypeError(f"unsupported dtype {dtype}; expected torch.float8_e4m3fn or torch.float8_e5m2")
    return code


def ds_block_quantize(x, layout: int = BLOCK_ROW, dtype=None, plan: Optional[ExpertPlan] = None, out=None,
                      out_scales=None, stream=None):
    """x [rows, n] (bf16 or fp32) in blocks of 128 as 8-bit floats (torch.float8_e4m3fn, or
    float8_e5m2) and fp32 scales; see include/dstopk.h for the layouts and a plan's part. Returns (q,
    scales): BLOCK_ROW q [P, n up to 16s], scales [P, ceil(n / 128)]; BLOCK_COLUMN (transposed)
    q [n, P up to 16s], scales [n, ceil(P / 128)]; BLOCK_TILE q [rows, n up to 16s], scales
    [ceil(rows / 128), ceil(n / 128)], P the plan's capacity or the rows. What lies behind the plan's
    end is what the outputs held. Rows already at a plan's positions are quantised without a plan, whole.
    BLOCK_TILE takes a stack x [groups, rows, n] too (experts' weights): one launch if rows is a multiple of
    128, else one for each matrix."""
    torch = _torch()
    dtype = dtype or torch.float8_e4m3fn
    if x.dim() == 3:
        return _quantize_stack(x, layout, dtype, plan, out, out_scales, stream)
    rows, n, rs = _matrix(x, "x")
    dt, qt, dev = _code(x.dtype), _code8(dtype), x.device
    c, positions = None, rows
    if plan is not None:
        c, plan_rows, positions = _plan(plan, dev)
        if plan_rows != rows:
            raise ValueError("x must have the plan's rows")
    if layout == BLOCK_COLUMN:
        q_rows, cols, shape = n, positions, (n, -(-positions // DS_BLOCK))
    else:
        q_rows, cols = positions, n
        shape = (-(-positions // DS_BLOCK) if layout == BLOCK_TILE else positions, -(-n // DS_BLOCK))
    out, qs = _rows_out(out, q_rows, -(-cols // 16) * 16, dtype, dev, stream)
    if out_scales is None:
        out_scales = _empty(shape, torch.float32, dev, stream)
    _call("ds_block_quantize", dev, stream, x.data_ptr(), rows, n, rs, dt, layout, c, out.data_ptr(), qs, qt,
          _operand(out_scales, "out_scales", torch.float32, shape, dev))
    return out, out_scales


def _quantize_stack(x, layout, dtype, plan, out, out_scales, stream):
    """ds_block_quantize of each matrix of a contiguous stack (one call where tiles do not cross them: 64 of 4096 x
    4096 bf16 570 us; else one for each: 64 of 1000 x 1024 339 us, five a matrix, where the bytes take 39)."""
    torch = _torch()
    if layout != BLOCK_TILE or plan is not None:
        raise ValueError("a stack of matrices is quantised in tiles, without a plan")
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError("a stack of matrices must be a contiguous device tensor")
    G, rows, n = x.shape
    wide, tiles = -(-n // 16) * 16, (-(-rows // DS_BLOCK), -(-n // DS_BLOCK))
    if out is None:
        out = _empty((G * rows, wide), dtype, x.device, stream).view(G, rows, wide)
    if out_scales is None:
        out_scales = _empty((G * tiles[0], tiles[1]), torch.float32, x.device, stream).view(G, *tiles)
    if out.shape != (G, rows, wide) or out.dtype != dtype or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous [{G}, {rows}, {wide}] tensor of {dtype}")
    if out_scales.shape != (G, *tiles) or out_scales.dtype != torch.float32 or not out_scales.is_contiguous():
        raise ValueError(f"out_scales must be a contiguous {(G, *tiles)} fp32 tensor")
    if rows % DS_BLOCK == 0:
        ds_block_quantize(x.view(G * rows, n), layout, dtype, None, out.view(G * rows, wide),
                          out_scales.view(G * tiles[0], tiles[1]), stream)
    else:
        for g in range(G):
            ds_block_quantize(x[g], layout, dtype, None, out[g], out_scales[g], stream)
    return out, out_scales


def ds_block_product(a, a_scales, b, b_scales, offsets=None, inner: bool = False, out=None, out_dtype=None,
                     stream=None, exact: bool = False):
    """a b^T of 8-bit operands with a scale for each 128 along the inner axis (ds_block_quantize's);
    bf16 (or out_dtype / out's type: bf16 or fp32). a [m, k] with scales [m, ceil(k / 128)].
      offsets None   b [n, k]; [m, n].
      offsets        int32 [groups + 1], the segments of a's rows (a plan's offsets), b [groups, n, k];
                     [m, n], rows outside the segments hold what out held.
      inner=True     offsets are segments of the inner axis, at multiples of 128; b [n, k] with scales
                     [n, ceil(k / 128)]; [groups, m, n].
    b is e4m3, with scales [.., n, ceil(k / 128)] or, in tiles, [.., ceil(n / 128), ceil(k / 128)]; a is e4m3
    or e5m2. k is a multiple of 16. The gradients are products of the same kind (include/dstopk.h).
    exact=True: bf16 results of exact products and fp32 sums, as fp32 results always are; without it large calls
    leave the sums of blocks to the 8-bit matrix unit (up to twice the rate, errors a hundredth of bf16's rounding), so
    that a row's bits may depend on the number of rows."""
    torch = _torch()
    m, k, a_stride = _matrix(a, "a")
    a_type, dev = _code8(a.dtype), a.device
    stacked = offsets is not None and not inner
    if stacked:
        groups_b, n, kb, b_stride = _batch_rows(b, "b")
    else:
        n, kb, b_stride = _matrix(b, "b")
        groups_b = 1
    if kb != k or b.device != dev:
        raise ValueError("b must have a's inner length and device")
    b_type, blocks, group, groups, op = _code8(b.dtype), -(-k // DS_BLOCK), GROUP_NONE, 1, None
    if offsets is not None:
        group, groups = (GROUP_INNER if inner else GROUP_ROWS), offsets.shape[0] - 1
        if offsets.dim() != 1 or groups < 1 or (stacked and groups != groups_b):
            raise ValueError("offsets must be 1-D, one more than the groups")
        op = _operand(offsets, "offsets", torch.int32, (groups + 1,), dev)
    elif inner:
        raise ValueError("inner needs offsets")
    shape = (groups, m, n) if inner else (m, n)
    if out is None:
        out = _empty((groups * m, n) if inner else shape, out_dtype or torch.bfloat16, dev, stream)
        stride = n
        if inner:
            out = out.view(shape)
    else:
        if out.shape != shape or out.device != dev or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError(f"out must be {shape} of out_dtype on {dev}")
        stride = _batch_rows(out, "out")[3] if inner else _matrix(out, "out")[2]
    scale_rows = 1
    if not inner and b_scales.dim() == b.dim() and b_scales.shape[-2] != n:
        scale_rows = DS_BLOCK
    lead = (groups_b,) if stacked else ()
    sp = _operand(b_scales, "b_scales", torch.float32, (*lead, n if scale_rows == 1 else -(-n // DS_BLOCK), blocks), dev)
    of_a = _pack_operand(a.data_ptr(), _operand(a_scales, "a_scales", torch.float32, (m, blocks), dev), a_stride,
                         a_type, 1)
    of_b = _pack_operand(b.data_ptr(), sp, b_stride, b_type, scale_rows)
    _call("ds_block_product", dev, stream, of_a, of_b, m, n, k, group, groups, op,
          out.data_ptr(), stride, _code(out.dtype) | (DS_EXACT_SUMS if exact else 0))
    return out


def stats_buffer(rows: int, slices: int, device):
    torch = _torch()
    return torch.zeros(rows * slices * STATS_DTYPE.itemsize, dtype=torch.uint8, device=device)


def decode_stats(buf) -> np.ndarray:
    return buf.cpu().numpy().view(STATS_DTYPE)


def ds_probe_read(src, sink=None, stream=None):
    """Stream all bytes of the device tensor src through the scan's 16-byte loads."""
    torch = _torch()
    nbytes = src.numel() * src.element_size()
    words = int(lib().ds_probe_sink_words(nbytes))
    if sink is None:
        sink = torch.empty(words, dtype=torch.int32, device=src.device)
    st = lib().ds_probe_read(src.data_ptr(), nbytes, sink.data_ptr(), _stream_handle(stream, src.device))
    if st != DS_OK:
        raise DSError(st, "ds_probe_read")
    return sink


def ds_probe_copy(dst, src, stream=None):
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() < nbytes:
        raise ValueError("dst too small")
    st = lib().ds_probe_copy(dst.data_ptr(), src.data_ptr(), nbytes, _stream_handle(stream, src.device))
    if st != DS_OK:
        raise DSError(st, "ds_probe_copy")
    return dst
