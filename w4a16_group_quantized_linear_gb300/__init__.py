"""W4A16 group-quantized linear layer for GB300 (sm_103a).

y = x W^T with int4-symmetric weights (nibble q+8, even k in the low nibble),
one fp16 scale per group of 32/64/128 input features and fp16 activations
(LLM170 page, introduction: "W4A16 (int4 sym g128, f16 activations)").

Around the layer: the routed experts' dispatch, GGUF block formats, and the
attention that sits between a decoder's projections (rotary positions, a paged
key/value cache and attention over it, fp16 or bf16).

This module is a thin ctypes binding over the C ABI of ``libw4a16.so``
(declared in ``include/w4a16.h``): it checks tensor dtypes and shapes,
allocates outputs with PyTorch and passes raw device pointers and the current
CUDA stream. Every step of the computation runs in the library's CUDA
kernels; there is no fallback. If the library is missing, every call raises.

Calls that split work across thread blocks join it in a workspace that this
module keeps for each stream. A CUDA graph goes on using the workspace of the
stream that it was captured on, whatever is called on that stream afterwards; graphs
captured on one stream must therefore be replayed one after another, and not at
the same time as other calls on that stream. A graph captured on a stream on
which nothing was called before has a workspace of its own.

Build it with ``python -m w4a16_group_quantized_linear_gb300.build`` (or
``__graft_entry__.build()``).
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
import threading

import torch

__all__ = ["pack", "unpack", "linear", "linear_gated", "grouped_linear", "grouped_linear_gather", "moe_route",
           "moe_dispatch", "moe_combine", "blocks_row_bytes", "blocks_linear", "blocks_dequant", "BLOCK_FORMATS",
           "rope_table", "rope", "kv_append", "paged_attention",
           "workspace_bytes", "device_status", "STATIC_WEIGHTS",
           "W4A16Error", "lib", "LIB_PATH", "EXPORTS", "STATUS"]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libw4a16.so")

STATUS = {0: "W4A16_OK", 1: "W4A16_ERR_INVALID_ARG", 2: "W4A16_ERR_UNSUPPORTED", 3: "W4A16_ERR_MISALIGNED",
          4: "W4A16_ERR_CUDA", 5: "W4A16_ERR_TIMEOUT", 6: "W4A16_ERR_BAD_OFFSETS", 7: "W4A16_ERR_WORKSPACE",
          8: "W4A16_ERR_BAD_ROUTING", 9: "W4A16_ERR_BAD_CACHE"}

TIMEOUT = 5  # of STATUS: a bounded wait on the device gave up

_P, _I64, _I32, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t


class _Rotary(ctypes.Structure):
    """w4a16_rotary"""
    _fields_ = [("table", _P), ("rows", _I64), ("rotary_dim", _I32), ("interleaved", _I32), ("positions", _P),
                ("axes", _I32), ("pair_axes", ctypes.c_char_p)]


class _PagedCache(ctypes.Structure):
    """w4a16_paged_cache"""
    _fields_ = [("k", _P), ("v", _P), ("pages", _I64), ("page_stride", _I64), ("slot_stride", _I64),
                ("head_stride", _I64), ("page_table", _P), ("page_table_stride", _I64), ("max_pages", _I32),
                ("page_size", _I32), ("q_offsets", _P), ("kv_lens", _P), ("batch", _I32), ("kv_heads", _I32),
                ("head_dim", _I32), ("dtype", _I32)]


# name -> (restype, argtypes); mirrors include/w4a16.h
EXPORTS = {
    "w4a16_pack": (_I32, [_P, _I64, _I64, _I32, _P, _P, _P]),
    "w4a16_unpack": (_I32, [_P, _I64, _I64, _P, _P]),
    "w4a16_linear": (_I32, [_P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _SZ, _P]),
    "w4a16_linear_ex": (_I32, [_P, _P, _P, _P, _I64, _I64, _I64, _I32, ctypes.c_uint32, _P, _SZ, _P]),
    "w4a16_linear_noalloc": (_I32, [_P, _P, _P, _P, _I64, _I64, _I64, _I32, _P]),
    "w4a16_linear_gated": (_I32, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _SZ, _P]),
    "w4a16_linear_gated_ex": (_I32, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, ctypes.c_uint32, _P, _SZ,
                                     _P]),
    "w4a16_linear_gated_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I32]),
    "w4a16_grouped_linear": (_I32, [_P, _P, _P, _P, _P, _I32, _I64, _I64, _I64, _I32, _P, _SZ, _P]),
    "w4a16_grouped_linear_gather": (_I32, [_P, _I64, _P, _P, _P, _P, _P, _I32, _I64, _I64, _I64, _I32, _P]),
    "w4a16_moe_route": (_I32, [_P, _I64, _I32, _I32, _I32, _P, _P, _P]),
    "w4a16_moe_dispatch_workspace_bytes": (_SZ, [_I64, _I32, _I32]),
    "w4a16_moe_dispatch": (_I32, [_P, _I64, _I32, _I32, _P, _I64, _P, _P, _P, _P, _P, _SZ, _P]),
    "w4a16_moe_combine": (_I32, [_P, _I64, _P, _P, _I64, _I32, _I64, _P, _P]),
    "w4a16_blocks_row_bytes": (_I64, [_I32, _I64]),
    "w4a16_blocks_linear": (_I32, [_I32, _P, _P, _P, _I64, _I64, _I64, _P]),
    "w4a16_blocks_dequant": (_I32, [_I32, _P, _I64, _I64, _P, _P]),
    "w4a16_rope": (_I32, [_I32, _P, _I64, _I64, _P, _I64, _I64, _I64, _I32, _I32, _P, _P]),
    "w4a16_kv_append": (_I32, [_P, _I64, _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _I32, _P, _P, _P]),
    "w4a16_paged_attention": (_I32, [_P, _I64, _P, _I64, _I64, _I32, _I64, ctypes.c_uint32, _I32, ctypes.c_float,
                                     _P, _P, _P, _SZ, _P]),
    "w4a16_paged_attention_workspace_bytes": (_SZ, [_I64, _I32, _I32, _I32, _I32, _I64]),
    "w4a16_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I32, _I32]),
    "w4a16_workspace_init": (_I32, [_P, _SZ, _P]),
    "w4a16_stream_capture_id": (_I32, [_P, _P]),
    "w4a16_device_status": (_I32, [_P]),
    "w4a16_status_string": (ctypes.c_char_p, [_I32]),
    "w4a16_version": (_I32, []),
    "w4a16_last_cuda_error": (ctypes.c_char_p, []),
}


# flags of w4a16_linear_ex / w4a16_linear_gated_ex (include/w4a16.h)
STATIC_WEIGHTS = 1

# flag of w4a16_paged_attention
CAUSAL = 1

# element types of the attention operators (W4A16_DTYPE_* in include/w4a16.h)
_DTYPES = {torch.float16: 1, torch.bfloat16: 2}

# GGUF block formats (W4A16_FORMAT_* in include/w4a16.h)
BLOCK_FORMATS = {"q4_k": 1, "q5_1": 2}


class W4A16Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = ""
        if status == 4 and _lib is not None:
            detail = " (" + _lib.w4a16_last_cuda_error().decode(errors="replace") + ")"
        super().__init__(f"{where}: {STATUS.get(status, status)}{detail}")


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"libw4a16.so not built ({LIB_PATH}); run "
                                   "python -m w4a16_group_quantized_linear_gb300.build")
            h = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in EXPORTS.items():
                f = getattr(h, name)
                f.restype, f.argtypes = res, args
            _lib = h
    return _lib


def _check(status: int, where: str):
    if status != 0:
        raise W4A16Error(status, where)


def _on_current_device(index):
    """The library launches on the current device, and sizes workspaces for it."""
    current = torch._C._cuda_getDevice()
    if index is not None and index != current:
        raise ValueError(f"the tensors are on cuda:{index} and the current device is cuda:{current}: make the call "
                         "under torch.cuda.device(tensor.device)")


def _stream(dev: torch.device):
    _on_current_device(dev.index)
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _ptr(t: torch.Tensor):
    return ctypes.c_void_p(t.data_ptr())


def _need(t: torch.Tensor, name: str, dtype, dim: int):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.dim() != dim or not t.is_cuda:
        raise ValueError(f"{name}: expected a {dim}-d {dtype} CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _out(out, shape, device: torch.device, K: int):
    """The output of a dense layer: new on x's device, or the caller's tensor,
    which may be on x's device or in pinned host memory (the kernels then store
    to it directly through unified addressing: no separate copy)."""
    if out is None:
        return torch.empty(shape, dtype=torch.float16, device=device)
    if not isinstance(out, torch.Tensor) or out.dtype != torch.float16 or out.dim() != 2:
        raise ValueError("out: expected a 2-d torch.float16 tensor")
    if not out.is_contiguous():
        raise ValueError("out: must be contiguous")
    if tuple(out.shape) != tuple(shape):
        raise ValueError("out must be [M, N]")
    if out.is_cuda:
        if out.device != device:
            raise ValueError("out must be on x's device")
    elif not out.is_pinned() or K == 0:
        raise ValueError("out must be a CUDA tensor, or pinned host memory (K > 0)")
    return out


# One zero-initialised workspace per (device, stream, kind of call), grown on
# demand. A buffer that a larger one takes the place of is kept: a captured
# graph may hold its address. Each is at least twice the one before it, so
# all that are kept are together no larger than the newest.
_ws: dict = {}
_replaced: list = []
# The same for calls under capture on a stream that has no workspace of its own
# yet: (capture id, buffer). Such a buffer is the graph's (its memory comes
# from the graph's pool, its zero-fill is one of the graph's nodes), so no
# call outside that capture may use it.
_captured: dict = {}


def _capture_id(stream) -> int:
    """Of the capture that `stream` is part of; 0: none."""
    n = ctypes.c_uint64(0)
    _check(lib().w4a16_stream_capture_id(stream, ctypes.byref(n)), "w4a16_stream_capture_id")
    return n.value


def _workspace(dev: torch.device, stream, nbytes: int, kind: str = "linear"):
    if nbytes == 0:
        return None
    key = (dev.index, stream.value or 0, kind)
    buf = _ws.get(key)
    if buf is not None and buf.numel() >= nbytes:
        return buf
    capture = _capture_id(stream)
    if capture:
        of, own = _captured.get(key, (0, None))
        if of == capture and own.numel() >= nbytes:
            return own
    new = torch.empty(max(nbytes, 1 << 20, 0 if capture or buf is None else 2 * buf.numel()), dtype=torch.uint8,
                      device=dev)
    _check(lib().w4a16_workspace_init(_ptr(new), new.numel(), stream), "w4a16_workspace_init")
    if capture:
        _captured[key] = (capture, new)
        return new
    if buf is not None:
        _replaced.append(buf)
    _ws[key] = new
    return new


def workspace_bytes(M: int, N: int, K: int, group: int, E: int = 1) -> int:
    return int(lib().w4a16_workspace_bytes(M, N, K, group, E))


def pack(w: torch.Tensor, group: int = 128):
    """fp32 [N, K] -> (qweight uint8 [N, K/2], scales fp16 [N, K/group])."""
    _need(w, "w", torch.float32, 2)
    N, K = w.shape
    qw = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    s = torch.empty((N, K // group if group else 0), dtype=torch.float16, device=w.device)
    _check(lib().w4a16_pack(_ptr(w), N, K, group, _ptr(qw), _ptr(s), _stream(w.device)), "w4a16_pack")
    return qw, s


def unpack(qw: torch.Tensor, K: int) -> torch.Tensor:
    """uint8 [N, K/2] -> int8 q [N, K] in [-8, 7]."""
    _need(qw, "qweight", torch.uint8, 2)
    N = qw.shape[0]
    if qw.shape[1] * 2 != K:
        raise ValueError("qweight must be [N, K/2]")
    q = torch.empty((N, K), dtype=torch.int8, device=qw.device)
    _check(lib().w4a16_unpack(_ptr(qw), N, K, _ptr(q), _stream(qw.device)), "w4a16_unpack")
    return q


def linear(x: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor, group: int = 128,
           out: torch.Tensor | None = None, static_weights: bool = False) -> torch.Tensor:
    """y = x W^T for x fp16 [M, K], qweight uint8 [N, K/2], scales fp16 [N, K/group].
    ``out`` may be a CUDA tensor on x's device or pinned host memory (K > 0).

    ``static_weights=True`` passes W4A16_STATIC_WEIGHTS: the caller promises
    that no work still pending on the stream writes qweight or scales (the
    weights of a decode loop), so the decode GEMV may stream them before the
    previous kernel on the stream completes. Results are identical."""
    _need(x, "x", torch.float16, 2)
    _need(qweight, "qweight", torch.uint8, 2)
    _need(scales, "scales", torch.float16, 2)
    M, K = x.shape
    N = qweight.shape[0]
    if qweight.shape[1] * 2 != K or (group and tuple(scales.shape) != (N, K // group)):
        raise ValueError("shape mismatch between x, qweight and scales")
    out = _out(out, (M, N), x.device, K)
    st = _stream(x.device)
    nb = workspace_bytes(M, N, K, group, 1)
    ws = _workspace(x.device, st, nb)
    _check(lib().w4a16_linear_ex(_ptr(x), _ptr(qweight), _ptr(scales), _ptr(out), M, N, K, group,
                                 STATIC_WEIGHTS if static_weights else 0,
                                 _ptr(ws) if ws is not None else None, ws.numel() if ws is not None else 0, st),
           "w4a16_linear")
    return out


def _format(fmt) -> int:
    if isinstance(fmt, str):
        if fmt not in BLOCK_FORMATS:
            raise ValueError(f"unknown block format {fmt!r}")
        return BLOCK_FORMATS[fmt]
    return int(fmt)


def blocks_row_bytes(fmt, K: int) -> int:
    """Bytes of one row of K weights in a GGUF block format (-1: not whole blocks)."""
    return int(lib().w4a16_blocks_row_bytes(_format(fmt), K))


def blocks_linear(fmt, x: torch.Tensor, blocks: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """y = x W^T for x fp16 [M, K] and GGUF block-format weights ("q4_k" or
    "q5_1"), blocks uint8 [N, blocks_row_bytes(fmt, K)]."""
    _need(x, "x", torch.float16, 2)
    _need(blocks, "blocks", torch.uint8, 2)
    M, K = x.shape
    N = blocks.shape[0]
    f = _format(fmt)
    if blocks.shape[1] != blocks_row_bytes(f, K):
        raise ValueError("blocks: expected [N, blocks_row_bytes(fmt, K)] bytes")
    out = _out(out, (M, N), x.device, K)
    _check(lib().w4a16_blocks_linear(f, _ptr(x), _ptr(blocks), _ptr(out), M, N, K, _stream(x.device)),
           "w4a16_blocks_linear")
    return out


def blocks_dequant(fmt, blocks: torch.Tensor, K: int) -> torch.Tensor:
    """W^ fp32 [N, K] from GGUF block-format weights uint8 [N, row_bytes]."""
    _need(blocks, "blocks", torch.uint8, 2)
    f = _format(fmt)
    N = blocks.shape[0]
    if blocks.shape[1] != blocks_row_bytes(f, K):
        raise ValueError("blocks: expected [N, blocks_row_bytes(fmt, K)] bytes")
    w = torch.empty((N, K), dtype=torch.float32, device=blocks.device)
    _check(lib().w4a16_blocks_dequant(f, _ptr(blocks), N, K, _ptr(w), _stream(blocks.device)),
           "w4a16_blocks_dequant")
    return w


def linear_gated(x: torch.Tensor, qweight_gate: torch.Tensor, scales_gate: torch.Tensor,
                 qweight_up: torch.Tensor, scales_up: torch.Tensor, group: int = 128,
                 out: torch.Tensor | None = None, static_weights: bool = False) -> torch.Tensor:
    """y = silu(x Wg^T) * (x Wu^T) in one launch (the decode GEMV for M <= 16,
    the tensor-core GEMM above); both weight matrices uint8 [N, K/2] with fp16
    scales [N, K/group]. ``static_weights`` as in :func:`linear`."""
    _need(x, "x", torch.float16, 2)
    for t, name in ((qweight_gate, "qweight_gate"), (qweight_up, "qweight_up")):
        _need(t, name, torch.uint8, 2)
    for t, name in ((scales_gate, "scales_gate"), (scales_up, "scales_up")):
        _need(t, name, torch.float16, 2)
    M, K = x.shape
    N = qweight_gate.shape[0]
    if (qweight_gate.shape[1] * 2 != K or tuple(qweight_up.shape) != tuple(qweight_gate.shape)
            or tuple(scales_gate.shape) != (N, K // group) or tuple(scales_up.shape) != (N, K // group)):
        raise ValueError("shape mismatch between x, the weights and the scales")
    out = _out(out, (M, N), x.device, K)
    st = _stream(x.device)
    nb = int(lib().w4a16_linear_gated_workspace_bytes(M, N, K, group))
    ws = _workspace(x.device, st, nb)
    _check(lib().w4a16_linear_gated_ex(_ptr(x), _ptr(qweight_gate), _ptr(scales_gate), _ptr(qweight_up),
                                       _ptr(scales_up), _ptr(out), M, N, K, group,
                                       STATIC_WEIGHTS if static_weights else 0,
                                       _ptr(ws) if ws is not None else None, ws.numel() if ws is not None else 0,
                                       st), "w4a16_linear_gated")
    return out


def grouped_linear(x_sorted: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor,
                   expert_offsets: torch.Tensor, group: int = 32,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """Routed experts: x_sorted fp16 [R, K] (rows sorted by expert), qweight uint8
    [E, N, K/2], scales fp16 [E, N, K/group], expert_offsets int32 [E+1] on the device."""
    _need(x_sorted, "x_sorted", torch.float16, 2)
    _need(qweight, "qweight", torch.uint8, 3)
    _need(scales, "scales", torch.float16, 3)
    _need(expert_offsets, "expert_offsets", torch.int32, 1)
    R, K = x_sorted.shape
    E, N = qweight.shape[0], qweight.shape[1]
    if qweight.shape[2] * 2 != K or tuple(scales.shape) != (E, N, K // group) or expert_offsets.numel() != E + 1:
        raise ValueError("shape mismatch between x_sorted, qweight, scales and expert_offsets")
    if out is None:
        out = torch.empty((R, N), dtype=torch.float16, device=x_sorted.device)
    else:
        _need(out, "out", torch.float16, 2)
    st = _stream(x_sorted.device)
    nb = workspace_bytes(R, N, K, group, E)
    ws = _workspace(x_sorted.device, st, nb)
    _check(lib().w4a16_grouped_linear(_ptr(x_sorted), _ptr(qweight), _ptr(scales), _ptr(expert_offsets),
                                      _ptr(out), E, R, N, K, group,
                                      _ptr(ws) if ws is not None else None, ws.numel() if ws is not None else 0,
                                      st), "w4a16_grouped_linear")
    return out


def grouped_linear_gather(x: torch.Tensor, token_of_row: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor,
                          expert_offsets: torch.Tensor, group: int = 32,
                          out: torch.Tensor | None = None) -> torch.Tensor:
    """Routed experts reading their rows straight from the token-major x:
    y_sorted[r] = x[token_of_row[r]] W_e^T for the expert e of row r. x fp16
    [T, K]; token_of_row int32 [R] (from moe_dispatch); qweight uint8
    [E, N, K/2]; scales fp16 [E, N, K/group] (group 32); expert_offsets int32
    [E+1]. The same bits as grouped_linear on the gathered rows."""
    _need(x, "x", torch.float16, 2)
    _need(token_of_row, "token_of_row", torch.int32, 1)
    _need(qweight, "qweight", torch.uint8, 3)
    _need(scales, "scales", torch.float16, 3)
    _need(expert_offsets, "expert_offsets", torch.int32, 1)
    T, K = x.shape
    R = token_of_row.shape[0]
    E, N = qweight.shape[0], qweight.shape[1]
    if qweight.shape[2] * 2 != K or tuple(scales.shape) != (E, N, K // group) or expert_offsets.numel() != E + 1:
        raise ValueError("shape mismatch between x, qweight, scales and expert_offsets")
    if out is None:
        out = torch.empty((R, N), dtype=torch.float16, device=x.device)
    else:
        _need(out, "out", torch.float16, 2)
        if tuple(out.shape) != (R, N):
            raise ValueError("out must be [R, N]")
    _check(lib().w4a16_grouped_linear_gather(_ptr(x), T, _ptr(token_of_row), _ptr(qweight), _ptr(scales),
                                             _ptr(expert_offsets), _ptr(out), E, R, N, K, group,
                                             _stream(x.device)), "w4a16_grouped_linear_gather")
    return out


def moe_route(logits: torch.Tensor, top_k: int, renormalize: bool = True):
    """Softmax top-k router: logits fp32 [T, E] -> (topk_ids int32 [T, top_k],
    topk_weights fp32 [T, top_k])."""
    _need(logits, "logits", torch.float32, 2)
    T, E = logits.shape
    ids = torch.empty((T, top_k), dtype=torch.int32, device=logits.device)
    w = torch.empty((T, top_k), dtype=torch.float32, device=logits.device)
    _check(lib().w4a16_moe_route(_ptr(logits), T, E, top_k, 1 if renormalize else 0, _ptr(ids), _ptr(w),
                                 _stream(logits.device)), "w4a16_moe_route")
    return ids, w


def moe_dispatch(topk_ids: torch.Tensor, E: int, x: torch.Tensor | None = None):
    """Expert-major order of the (token, slot) pairs: returns (expert_offsets int32
    [E+1], row_of int32 [T, top_k], token_of_row int32 [T*top_k], x_sorted fp16
    [T*top_k, K] or None when x is None)."""
    _need(topk_ids, "topk_ids", torch.int32, 2)
    T, k = topk_ids.shape
    dev = topk_ids.device
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    row_of = torch.empty((T, k), dtype=torch.int32, device=dev)
    token_of_row = torch.empty(T * k, dtype=torch.int32, device=dev)
    x_sorted, K = None, 0
    if x is not None:
        _need(x, "x", torch.float16, 2)
        if x.shape[0] != T:
            raise ValueError("x must have one row per token")
        K = x.shape[1]
        x_sorted = torch.empty((T * k, K), dtype=torch.float16, device=dev)
    nb = int(lib().w4a16_moe_dispatch_workspace_bytes(T, k, E))
    ws = torch.empty(nb, dtype=torch.uint8, device=dev) if nb else None
    _check(lib().w4a16_moe_dispatch(_ptr(topk_ids), T, k, E, _ptr(x) if x is not None else None, K,
                                    _ptr(offsets), _ptr(row_of), _ptr(token_of_row),
                                    _ptr(x_sorted) if x_sorted is not None else None,
                                    _ptr(ws) if ws is not None else None, nb, _stream(dev)), "w4a16_moe_dispatch")
    return offsets, row_of, token_of_row, x_sorted


def moe_combine(y_sorted: torch.Tensor, row_of: torch.Tensor, topk_weights: torch.Tensor,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """y[t] = sum_j topk_weights[t, j] * y_sorted[row_of[t, j]] (fp32 sum, fp16 result)."""
    _need(y_sorted, "y_sorted", torch.float16, 2)
    _need(row_of, "row_of", torch.int32, 2)
    _need(topk_weights, "topk_weights", torch.float32, 2)
    if tuple(topk_weights.shape) != tuple(row_of.shape):
        raise ValueError("row_of and topk_weights must both be [T, top_k]")
    T, k = row_of.shape
    R, N = y_sorted.shape
    if out is None:
        out = torch.empty((T, N), dtype=torch.float16, device=y_sorted.device)
    else:
        _need(out, "out", torch.float16, 2)
        if tuple(out.shape) != (T, N):
            raise ValueError("out must be [T, N]")
    _check(lib().w4a16_moe_combine(_ptr(y_sorted), R, _ptr(row_of), _ptr(topk_weights), T, k, N, _ptr(out),
                                   _stream(y_sorted.device)), "w4a16_moe_combine")
    return out


@functools.lru_cache(maxsize=1024)
def _attention_workspace_bytes(index: int, T: int, B: int, H: int, G: int, D: int, max_q_len: int) -> int:
    return int(lib().w4a16_paged_attention_workspace_bytes(T, B, H, G, D, max_q_len))


def rope_table(rows: int, rotary_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """The angles of :func:`rope` and :func:`kv_append`: fp32 [rows, rotary_dim],
    cos(p * base^(-2i / rotary_dim)) for pair i in the first half of row p and
    the sine in the second, formed in 64 bits and rounded once. A table of any
    other frequencies in the same layout serves as well."""
    pair = torch.arange(0, rotary_dim, 2, dtype=torch.float64, device=device)
    angle = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * base ** (-pair / rotary_dim)
    return torch.cat((angle.cos(), angle.sin()), dim=1).float()


def _packer(c_type) -> struct.Struct:
    """Packs the fields of a ctypes structure, in native alignment: several times faster than making one."""
    code = {_P: "P", ctypes.c_char_p: "P", _I64: "q", _I32: "i"}
    return struct.Struct("".join(code[t] for _, t in c_type._fields_))


# The calls below are made once per layer and token, so their checks ask each
# tensor for little: its device index (-1 off the GPU), type, shape and strides.
_CACHE, _ROTARY = _packer(_PagedCache), _packer(_Rotary)


def _raw_stream(index: int) -> int:
    _on_current_device(index)
    return torch._C._cuda_getCurrentRawStream(index)


def _rows(t: torch.Tensor, name: str, dtype=None, index: int = -1):
    """(shape, strides) of a [tokens, heads, head_dim] tensor whose heads' rows are contiguous."""
    if not isinstance(t, torch.Tensor) or t.ndim != 3:
        raise ValueError(f"{name}: expected a 3-d torch.float16 or torch.bfloat16 CUDA tensor")
    if dtype is None:
        if t.dtype not in _DTYPES or not t.is_cuda:
            raise ValueError(f"{name}: expected a 3-d torch.float16 or torch.bfloat16 CUDA tensor")
    elif t.dtype != dtype or t.get_device() != index:
        raise ValueError(f"{name}: expected the type and device of the other tensors")
    shape, stride = t.shape, t.stride()
    if stride[2] != 1 and shape[2] != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return shape, stride


def _rows_out(out, x: torch.Tensor, shape, name: str, index: int):
    """A contiguous result of x's shape: new, or the caller's."""
    if out is None:
        return torch.empty(shape, dtype=x.dtype, device=x.device)
    if _rows(out, name, x.dtype, index)[0] != shape or not out.is_contiguous():
        raise ValueError(f"{name}: must be contiguous and of the input's shape")
    return out


def _int32(t: torch.Tensor, name: str, dim: int, index: int):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.ndim != dim or t.get_device() != index:
        raise ValueError(f"{name}: expected a {dim}-d torch.int32 tensor on the other tensors' device")
    shape, stride = t.shape, t.stride()
    if stride[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return shape, stride


def _rotary(table, positions, pair_axes, interleaved: bool, T: int, index: int):
    """(packed w4a16_rotary, what it points to)"""
    if not isinstance(table, torch.Tensor) or table.dtype != torch.float32 or table.ndim != 2 \
            or table.get_device() != index or not table.is_contiguous():
        raise ValueError("table: expected a contiguous 2-d torch.float32 tensor on the other tensors' device")
    rows, dim = table.shape
    axes, at, axis_of, axis_ptr = 1, 0, None, 0
    if positions is not None:
        if isinstance(positions, torch.Tensor) and positions.ndim == 1:
            positions = positions[None]
        shape, stride = _int32(positions, "positions", 2, index)
        axes = shape[0]
        if shape[1] != T or (axes > 1 and T > 0 and stride[0] != T):
            raise ValueError("positions: expected contiguous [T] or [axes, T]")
        at = positions.data_ptr()
    if pair_axes is not None:
        axis_of = bytes(pair_axes)
        if 2 * len(axis_of) != dim:
            raise ValueError("pair_axes: expected one axis per pair, rotary_dim / 2 of them")
        axis_ptr = ctypes.cast(axis_of, _P).value
    return _ROTARY.pack(table.data_ptr(), rows, dim, 1 if interleaved else 0, at, axes, axis_ptr), axis_of


def rope(x: torch.Tensor, positions: torch.Tensor, table: torch.Tensor, pair_axes=None, interleaved: bool = False,
         out: torch.Tensor | None = None) -> torch.Tensor:
    """x turned by its tokens' positions: x fp16 or bf16 [T, heads, head_dim]
    (a view of a fused projection will do), positions int32 [T] or [axes, T],
    table fp32 [rows, rotary_dim] (:func:`rope_table`); elements past rotary_dim
    are copied. Pair i is elements (i, i + rotary_dim / 2), or (2i, 2i + 1) with
    ``interleaved``. ``pair_axes`` gives the axis (0 to 3) whose position turns
    each pair (time, height and width of a video's patches, say); without it
    axis 0 turns all. ``out`` may be x itself."""
    shape, sx = _rows(x, "x")
    index = x.get_device()
    T, H, D = shape
    if positions is None:
        raise ValueError("positions: expected contiguous [T] or [axes, T]")
    r, keep = _rotary(table, positions, pair_axes, interleaved, T, index)
    if out is None:
        out, so = torch.empty(shape, dtype=x.dtype, device=x.device), (H * D, D)
    else:
        out_shape, so = _rows(out, "out", x.dtype, index)
        if out_shape != shape:
            raise ValueError("out: must have x's shape")
    status = (_lib or lib()).w4a16_rope(_DTYPES[x.dtype], x.data_ptr(), sx[0], sx[1], out.data_ptr(), so[0], so[1], T,
                                        H, D, r, _raw_stream(index))
    if status:
        raise W4A16Error(status, "w4a16_rope")
    return out


def _packed_cache(k_cache, v_cache, page_table, q_offsets, kv_lens, dtype, index: int):
    """(packed w4a16_paged_cache, batch, kv_heads, head_dim)"""
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if not isinstance(t, torch.Tensor) or t.ndim != 4 or t.dtype != dtype or t.get_device() != index:
            raise ValueError(f"{name}: expected a 4-d tensor of the other tensors' type and device")
    shape, stride = k_cache.shape, k_cache.stride()
    if v_cache.shape != shape or v_cache.stride() != stride:
        raise ValueError("k_cache and v_cache must have the same shape and strides")
    if stride[3] != 1:
        raise ValueError("k_cache, v_cache: the last dimension must be contiguous")
    table_shape, table_stride = _int32(page_table, "page_table", 2, index)
    B = _int32(kv_lens, "kv_lens", 1, index)[0][0]
    if table_shape[0] != B or _int32(q_offsets, "q_offsets", 1, index)[0][0] != B + 1:
        raise ValueError("page_table [B, max_pages], q_offsets [B + 1] and kv_lens [B] must agree")
    pages, size, G, D = shape
    return _CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), pages, stride[0], stride[1], stride[2],
                       page_table.data_ptr(), table_stride[0], table_shape[1], size, q_offsets.data_ptr(),
                       kv_lens.data_ptr(), B, G, D, _DTYPES[dtype]), B, G, D


def _cache(k_cache, v_cache, page_table, q_offsets, kv_lens, like: torch.Tensor) -> _PagedCache:
    """The checked arguments as the C structure, for callers of the C ABI."""
    return _PagedCache.from_buffer_copy(
        _packed_cache(k_cache, v_cache, page_table, q_offsets, kv_lens, like.dtype, like.get_device())[0])


def kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              page_table: torch.Tensor, q_offsets: torch.Tensor, kv_lens: torch.Tensor,
              q: torch.Tensor | None = None, table: torch.Tensor | None = None,
              positions: torch.Tensor | None = None, pair_axes=None, interleaved: bool = False,
              q_out: torch.Tensor | None = None):
    """Stores the new tokens' k and v (fp16 or bf16 [T, kv_heads, head_dim]) into
    the paged cache and, with ``table``, turns k and q by their rotary positions
    on the way (``positions`` and the rest as in :func:`rope`; without
    ``positions`` each token's place in its sequence). Returns the turned q
    [T, heads, head_dim] (contiguous; ``q_out`` if given), or None without q.

    The cache is [pages, page_size, kv_heads, head_dim] in any strides with
    contiguous rows (page_size a multiple of 16, head_dim 64 or 128). Sequence
    b's new tokens are rows q_offsets[b] to q_offsets[b + 1] of k, v and q;
    kv_lens[b] counts its cached tokens with these among them; its place p lives in
    slot p % page_size of page page_table[b, p // page_size]. All three are int32
    on the device: a captured graph follows their values."""
    shape, sk = _rows(k, "k")
    index, dtype = k.get_device(), k.dtype
    v_shape, sv = _rows(v, "v", dtype, index)
    if v_shape != shape:
        raise ValueError("k and v must have the same shape")
    T, G, D = shape
    c, _, cache_heads, cache_dim = _packed_cache(k_cache, v_cache, page_table, q_offsets, kv_lens, dtype, index)
    if cache_heads != G or cache_dim != D:
        raise ValueError("the cache must have k's heads and head_dim")
    H, sq, q_ptr, out_ptr = 0, (0, 0), 0, 0
    if q is not None:
        q_shape, sq = _rows(q, "q", dtype, index)
        if q_shape[0] != T or q_shape[2] != D:
            raise ValueError("q must be [T, heads, head_dim]")
        H = q_shape[1]
        q_out = _rows_out(q_out, q, q_shape, "q_out", index)
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    r = keep = None
    if table is not None:
        r, keep = _rotary(table, positions, pair_axes, interleaved, T, index)
    elif positions is not None or pair_axes is not None:
        raise ValueError("positions and pair_axes need table")
    status = (_lib or lib()).w4a16_kv_append(c, T, k.data_ptr(), sk[0], sk[1], v.data_ptr(), sv[0], sv[1], q_ptr,
                                             sq[0], sq[1], H, out_ptr, r, _raw_stream(index))
    if status:
        raise W4A16Error(status, "w4a16_kv_append")
    return q_out


def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                    q_offsets: torch.Tensor, kv_lens: torch.Tensor, max_q_len: int, causal: bool = True,
                    window: int = 0, scale: float | None = None, out: torch.Tensor | None = None,
                    return_lse: bool = False):
    """Attention of the new tokens' queries (fp16 or bf16 [T, heads, head_dim])
    over the paged cache of :func:`kv_append`: softmax(scale q k^T) v per row,
    heads in groups of heads / kv_heads sharing a cached head. A row sees its sequence's
    places up to its own (all of them with ``causal=False``), the last ``window``
    of them where that is not 0. ``max_q_len`` is at least the longest sequence's number
    of new tokens (it chooses the kernels, so one that is larger than need be costs time and
    some accuracy; the lengths themselves stay on the device). ``scale`` defaults to head_dim^-1/2. A row that sees nothing gets 0.

    Returns out [T, heads, head_dim], or (out, lse) with ``return_lse``: lse
    fp32 [T, heads] is the natural logarithm of the softmax's sum."""
    shape, sq = _rows(q, "q")
    index = q.get_device()
    T, H, D = shape
    c, B, G, cache_dim = _packed_cache(k_cache, v_cache, page_table, q_offsets, kv_lens, q.dtype, index)
    if cache_dim != D or G == 0 or H % G != 0:
        raise ValueError("the cache must have q's head_dim, and heads must be a multiple of its heads")
    out = _rows_out(out, q, shape, "out", index)
    lse = torch.empty((T, H), dtype=torch.float32, device=q.device) if return_lse else None
    st = _raw_stream(index)
    h = _lib or lib()
    need = _attention_workspace_bytes(index, T, B, H, G, D, max_q_len)
    ws = _ws.get((index, st, "attention"))
    if need and (ws is None or ws.numel() < need):
        ws = _workspace(q.device, ctypes.c_void_p(st), need, "attention")
    status = h.w4a16_paged_attention(c, T, q.data_ptr(), sq[0], sq[1], H, max_q_len, CAUSAL if causal else 0, window,
                                     D ** -0.5 if scale is None else scale, out.data_ptr(),
                                     lse.data_ptr() if return_lse else 0, ws.data_ptr() if need else 0,
                                     ws.numel() if need else 0, st)
    if status:
        raise W4A16Error(status, "w4a16_paged_attention")
    return (out, lse) if return_lse else out


def device_status(raise_on_error: bool = True) -> int:
    """Synchronizes the current stream and reads/clears the device error word.
    After a timeout the workspaces kept here are made ready again (the whole
    device is synchronized): the call that gave up left its counters set."""
    index = torch.cuda.current_device()
    st = _stream(torch.device("cuda", index))
    status = int(lib().w4a16_device_status(st))
    if status == TIMEOUT:
        torch.cuda.synchronize(index)
        for buf in [*_ws.values(), *_replaced, *(own for _, own in _captured.values())]:
            if buf.get_device() == index:
                _check(lib().w4a16_workspace_init(_ptr(buf), buf.numel(), st), "w4a16_workspace_init")
        torch.cuda.synchronize(index)
    if raise_on_error:
        _check(status, "device")
    return status
