"""Thin ctypes binding over libmoe_layout.so (argument marshalling only).

Every function has the name of its C entry point and forwards raw device
pointers, sizes and the current CUDA stream; all computation happens in the
library's CUDA kernels.  There is no CPU fallback: if the library is missing
or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os
import re
import threading

import torch

from . import build as _build

MOE_OK = 0
MOE_DEV_ERR_EXPERT_RANGE = 1
MOE_DEV_ERR_DUPLICATE = 2
MOE_DEV_ERR_REGION_OVERFLOW = 4
MOE_DEV_ERR_TIMEOUT = 8

_lock = threading.Lock()
_lib = None


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {moe_status_string(status)} (status {status})")


def library_path() -> str:
    return _build.LIB_PATH


def load(path: str | None = None):
    """Load the CUDA library (built beforehand by build.build())."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            p = path or _build.LIB_PATH
            if not os.path.exists(p):
                raise RuntimeError(
                    f"{p} is missing: build it with "
                    "combine_moe_layout_05_gb300.build.build()")
            lib = ctypes.CDLL(p)
            P, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
            lib.moe_status_string.argtypes = [ctypes.c_int]
            lib.moe_status_string.restype = ctypes.c_char_p
            lib.moe_layout_workspace_bytes.argtypes = [i32, i32, i32]
            lib.moe_layout_workspace_bytes.restype = sz
            lib.moe_layout.argtypes = [P, i32, i32, i32, i32, P, P, P, P, P, P,
                                       P, sz, P]
            lib.moe_layout.restype = ctypes.c_int
            lib.moe_dispatch.argtypes = [P, i32, i32, i32, P, i32, P, P, P]
            lib.moe_dispatch.restype = ctypes.c_int
            lib.moe_combine.argtypes = [P, P, P, i32, i32, i32, P, P]
            lib.moe_combine.restype = ctypes.c_int
            lib.moe_layout_dispatch.argtypes = [P, P, i32, i32, i32, i32, i32, i32,
                                                P, P, P, P, P, P, P, P, P, sz, P]
            lib.moe_layout_dispatch.restype = ctypes.c_int
            lib.moe_layout_dispatch_kernels.argtypes = [i32, i32, i32, i32, i32]
            lib.moe_layout_dispatch_kernels.restype = i32
            lib.moe_layout_kernels.argtypes = [i32, i32, i32]
            lib.moe_layout_kernels.restype = i32
            lib.moe_combine_fp8.argtypes = [P, P, P, P, i32, i32, i32, P, P]
            lib.moe_combine_fp8.restype = ctypes.c_int
            lib.moe_combine_rank_partial.argtypes = [P, P, P, P, i32, i32, i32, i32, i32, P, P]
            lib.moe_combine_rank_partial.restype = ctypes.c_int
            lib.moe_dispatch_send.argtypes = [P, i32, i32, i32, i32, i32, P, P, P, i32, i32,
                                              P, P, i32, P, P, P, P]
            lib.moe_dispatch_send.restype = ctypes.c_int
            lib.moe_dispatch_recv.argtypes = [P, P, i32, P, P, i32, P, i32, i32, i32, i32,
                                              i32, P, P, P]
            lib.moe_dispatch_recv.restype = ctypes.c_int
            lib.moe_layout_static.argtypes = [P, i32, i32, i32, i32, P, P, P, P, P, P, P]
            lib.moe_layout_static.restype = ctypes.c_int
            f32 = ctypes.c_float
            lib.moe_route_workspace_bytes.argtypes = [i32, i32]
            lib.moe_route_workspace_bytes.restype = sz
            lib.moe_route.argtypes = [P, i32, i32, i32, i32, i32, f32, P, P, P, P, P, P, P, sz, P]
            lib.moe_route.restype = ctypes.c_int
            lib.moe_route_backward.argtypes = [P, i32, i32, i32, i32, i32, f32, P, P, P, P, P, P, P]
            lib.moe_route_backward.restype = ctypes.c_int
            lib.moe_dispatch_int8.argtypes = [P, i32, i32, i32, P, P, P, P]
            lib.moe_dispatch_int8.restype = ctypes.c_int
            lib.moe_expert_matmul_int8.argtypes = [P, P, P, P, P, i32, i32, i32, i32, P, P, P]
            lib.moe_expert_matmul_int8.restype = ctypes.c_int
            _lib = lib
    return _lib


def declared_functions(header: str | None = None) -> list[str]:
    """Names of the functions the public header declares."""
    header = header or os.path.join(_build.INCLUDE, "moe_layout.h")
    text = open(header).read()
    return sorted(set(re.findall(r"MOE_API\s+[\w\s\*]*?\b(moe_\w+)\s*\(", text)))


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()          # 0 for an empty tensor


# The current stream's handle without a Stream object, at a tenth of its cost.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_get_device = getattr(torch._C, "_cuda_getDevice", None)
if _raw_stream is None or _get_device is None:
    def _current_stream() -> int:
        return torch.cuda.current_stream().cuda_stream
else:
    def _current_stream() -> int:
        return _raw_stream(_get_device())


def _stream(stream) -> int | None:
    if stream is None:
        return _current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(name: str, t, dtype, device=None):
    if t is None or (t.dtype is dtype and t.is_cuda and t.is_contiguous()):
        return
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def _raise(fn: str, status: int):
    if status != MOE_OK:
        raise MoeError(fn, status)


def moe_status_string(status: int) -> str:
    return load().moe_status_string(int(status)).decode()


def moe_layout_workspace_bytes(T: int, K: int, E: int) -> int:
    return int(load().moe_layout_workspace_bytes(T, K, E))


def moe_layout_dispatch_kernels(T: int, H: int, K: int, E: int, fp8: bool) -> int:
    return int(load().moe_layout_dispatch_kernels(T, H, K, E, int(bool(fp8))))


def moe_layout_kernels(T: int, K: int, E: int) -> int:
    return int(load().moe_layout_kernels(T, K, E))


def moe_layout(topk_ids, E: int, R: int, expert_counts, expert_offsets,
               rank_offsets, src_token, dst_row, dev_error=None,
               workspace=None, stream=None) -> None:
    """Routing histogram, scan and stable slot map (see include/moe_layout.h)."""
    T, K = topk_ids.shape
    _check("topk_ids", topk_ids, torch.int32)
    for n, t in (("expert_counts", expert_counts), ("expert_offsets", expert_offsets),
                 ("rank_offsets", rank_offsets), ("src_token", src_token),
                 ("dst_row", dst_row)):
        _check(n, t, torch.int32)
    if expert_counts.numel() < E or expert_offsets.numel() < E + 1 or rank_offsets.numel() < R + 1:
        raise ValueError("moe_layout: output arrays too small")
    if src_token.numel() < T * K or dst_row.numel() < T * K:
        raise ValueError("moe_layout: src_token/dst_row too small")
    if dev_error is not None:
        _check("dev_error", dev_error, torch.int32)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load().moe_layout(_ptr(topk_ids), T, K, E, R, _ptr(expert_counts),
                           _ptr(expert_offsets), _ptr(rank_offsets),
                           _ptr(src_token), _ptr(dst_row), _ptr(dev_error),
                           _ptr(workspace), ws_bytes, _stream(stream))
    _raise("moe_layout", st)


def moe_dispatch(tokens, dst_row, packed, scales=None, fp8: bool = False,
                 stream=None) -> None:
    """Pack token rows into their K slots, bf16 or block-scaled e4m3."""
    T, H = tokens.shape
    K = dst_row.shape[1] if dst_row.dim() == 2 else 1
    _check("tokens", tokens, torch.bfloat16)
    _check("dst_row", dst_row, torch.int32)
    if fp8:
        _check("packed", packed, torch.float8_e4m3fn)
        _check("scales", scales, torch.float32)
        if scales is None or scales.numel() < T * K * (H // 128):
            raise ValueError("moe_dispatch: scales missing or too small")
    else:
        _check("packed", packed, torch.bfloat16)
    if dst_row.numel() != T * K or packed.numel() < T * K * H:
        raise ValueError("moe_dispatch: dst_row/packed have the wrong size")
    st = load().moe_dispatch(_ptr(tokens), T, H, K, _ptr(dst_row), int(bool(fp8)),
                             _ptr(packed), _ptr(scales) if fp8 else None,
                             _stream(stream))
    _raise("moe_dispatch", st)


def moe_layout_dispatch(topk_ids, tokens, E: int, R: int, expert_counts,
                        expert_offsets, rank_offsets, src_token, dst_row, packed,
                        scales=None, fp8: bool = False, dev_error=None,
                        workspace=None, stream=None) -> None:
    """moe_layout then moe_dispatch in one call (one kernel for small batches)."""
    T, K = topk_ids.shape
    H = tokens.shape[1]
    if tokens.shape[0] != T:
        raise ValueError("moe_layout_dispatch: tokens and topk_ids disagree on T")
    _check("topk_ids", topk_ids, torch.int32)
    _check("tokens", tokens, torch.bfloat16)
    for n, t in (("expert_counts", expert_counts), ("expert_offsets", expert_offsets),
                 ("rank_offsets", rank_offsets), ("src_token", src_token),
                 ("dst_row", dst_row)):
        _check(n, t, torch.int32)
    if expert_counts.numel() < E or expert_offsets.numel() < E + 1 or rank_offsets.numel() < R + 1:
        raise ValueError("moe_layout_dispatch: output arrays too small")
    if src_token.numel() < T * K or dst_row.numel() < T * K or packed.numel() < T * K * H:
        raise ValueError("moe_layout_dispatch: src_token/dst_row/packed too small")
    if fp8:
        _check("packed", packed, torch.float8_e4m3fn)
        _check("scales", scales, torch.float32)
        if scales is None or scales.numel() < T * K * (H // 128):
            raise ValueError("moe_layout_dispatch: scales missing or too small")
    else:
        _check("packed", packed, torch.bfloat16)
    if dev_error is not None:
        _check("dev_error", dev_error, torch.int32)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load().moe_layout_dispatch(
        _ptr(topk_ids), _ptr(tokens), T, H, K, E, R, int(bool(fp8)), _ptr(expert_counts),
        _ptr(expert_offsets), _ptr(rank_offsets), _ptr(src_token), _ptr(dst_row),
        _ptr(dev_error), _ptr(packed), _ptr(scales) if fp8 else None,
        _ptr(workspace), ws_bytes, _stream(stream))
    _raise("moe_layout_dispatch", st)


def moe_combine(expert_out, topk_weights, dst_row, out, stream=None) -> None:
    """Routing-weighted fp32 sum of each token's K expert rows, rounded to bf16."""
    T, K = topk_weights.shape
    H = out.shape[1]
    _check("expert_out", expert_out, torch.bfloat16)
    _check("topk_weights", topk_weights, torch.float32)
    _check("dst_row", dst_row, torch.int32)
    _check("out", out, torch.bfloat16)
    if dst_row.numel() != T * K or out.shape[0] != T or expert_out.numel() < T * K * H:
        raise ValueError("moe_combine: argument sizes disagree")
    st = load().moe_combine(_ptr(expert_out), _ptr(topk_weights), _ptr(dst_row),
                            T, H, K, _ptr(out), _stream(stream))
    _raise("moe_combine", st)


def moe_combine_rank_partial(expert_out, topk_weights, topk_ids, dst_row, E: int,
                             R: int, out, stream=None) -> None:
    """Combine with sender-side per-rank partial sums (bf16 partials)."""
    T, K = topk_weights.shape
    H = out.shape[1]
    _check("expert_out", expert_out, torch.bfloat16)
    _check("topk_weights", topk_weights, torch.float32)
    _check("topk_ids", topk_ids, torch.int32)
    _check("dst_row", dst_row, torch.int32)
    _check("out", out, torch.bfloat16)
    if dst_row.numel() != T * K or topk_ids.numel() != T * K or out.shape[0] != T \
            or expert_out.numel() < T * K * H:
        raise ValueError("moe_combine_rank_partial: argument sizes disagree")
    st = load().moe_combine_rank_partial(_ptr(expert_out), _ptr(topk_weights), _ptr(topk_ids),
                                         _ptr(dst_row), T, H, K, E, R, _ptr(out),
                                         _stream(stream))
    _raise("moe_combine_rank_partial", st)


def moe_dispatch_send(tokens, topk_ids, dst_row, rank_offsets, E: int, R: int,
                      priv, bulk, priv_scales=None, bulk_scales=None, fp8: bool = False,
                      dev_error=None, stream=None) -> None:
    """Dispatch into per-rank regions: priv [R,P,H] for each rank's first P
    rows, bulk [R,C,H] for the rest (bf16, or e4m3 codes + block scales)."""
    T, H = tokens.shape
    K = topk_ids.shape[1]
    R_, P = priv.shape[0], priv.shape[1]
    C = bulk.shape[1]
    if R_ != R or bulk.shape[0] != R:
        raise ValueError("moe_dispatch_send: region buffers must have R rows of regions")
    _check("tokens", tokens, torch.bfloat16)
    for n, t in (("topk_ids", topk_ids), ("dst_row", dst_row), ("rank_offsets", rank_offsets)):
        _check(n, t, torch.int32)
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    _check("priv", priv, dt)
    _check("bulk", bulk, dt)
    if fp8:
        _check("priv_scales", priv_scales, torch.float32)
        _check("bulk_scales", bulk_scales, torch.float32)
    st = load().moe_dispatch_send(_ptr(tokens), T, H, K, E, R, _ptr(topk_ids), _ptr(dst_row),
                                  _ptr(rank_offsets), int(bool(fp8)), P, _ptr(priv),
                                  _ptr(priv_scales) if fp8 else None, C, _ptr(bulk),
                                  _ptr(bulk_scales) if fp8 else None, _ptr(dev_error),
                                  _stream(stream))
    _raise("moe_dispatch_send", st)


def moe_dispatch_recv(priv, bulk, rank_offsets, T: int, K: int, packed,
                      priv_scales=None, bulk_scales=None, scales=None, fp8: bool = False,
                      stream=None) -> None:
    """Region rows back to slot order (the grouped-GEMM input)."""
    R, P = priv.shape[0], priv.shape[1]
    C = bulk.shape[1]
    H = packed.shape[1]
    _check("rank_offsets", rank_offsets, torch.int32)
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    for n, t in (("priv", priv), ("bulk", bulk), ("packed", packed)):
        _check(n, t, dt)
    st = load().moe_dispatch_recv(_ptr(priv), _ptr(priv_scales) if fp8 else None, P,
                                  _ptr(bulk), _ptr(bulk_scales) if fp8 else None, C,
                                  _ptr(rank_offsets), R, T, H, K, int(bool(fp8)), _ptr(packed),
                                  _ptr(scales) if fp8 else None, _stream(stream))
    _raise("moe_dispatch_recv", st)


def moe_layout_static(topk_ids, E: int, R: int, expert_counts, expert_offsets,
                      rank_offsets, src_token, dst_row, dev_error=None,
                      stream=None) -> None:
    """moe_layout for callers that cannot allocate: the large-batch scratch is
    a fixed array inside the library (see include/moe_layout.h)."""
    T, K = topk_ids.shape
    _check("topk_ids", topk_ids, torch.int32)
    for n, t in (("expert_counts", expert_counts), ("expert_offsets", expert_offsets),
                 ("rank_offsets", rank_offsets), ("src_token", src_token),
                 ("dst_row", dst_row)):
        _check(n, t, torch.int32)
    if expert_counts.numel() < E or expert_offsets.numel() < E + 1 or rank_offsets.numel() < R + 1:
        raise ValueError("moe_layout_static: output arrays too small")
    if src_token.numel() < T * K or dst_row.numel() < T * K:
        raise ValueError("moe_layout_static: src_token/dst_row too small")
    if dev_error is not None:
        _check("dev_error", dev_error, torch.int32)
    st = load().moe_layout_static(_ptr(topk_ids), T, K, E, R, _ptr(expert_counts),
                                  _ptr(expert_offsets), _ptr(rank_offsets),
                                  _ptr(src_token), _ptr(dst_row), _ptr(dev_error),
                                  _stream(stream))
    _raise("moe_layout_static", st)


def moe_combine_fp8(expert_out, expert_scales, topk_weights, dst_row, out,
                    stream=None) -> None:
    """Routing-weighted sum of e4m3 expert rows (value = code * block scale)."""
    T, K = topk_weights.shape
    H = out.shape[1]
    _check("expert_out", expert_out, torch.float8_e4m3fn)
    _check("expert_scales", expert_scales, torch.float32)
    _check("topk_weights", topk_weights, torch.float32)
    _check("dst_row", dst_row, torch.int32)
    _check("out", out, torch.bfloat16)
    if dst_row.numel() != T * K or out.shape[0] != T or expert_out.numel() < T * K * H \
            or expert_scales.numel() < T * K * (H // 128):
        raise ValueError("moe_combine_fp8: argument sizes disagree")
    st = load().moe_combine_fp8(_ptr(expert_out), _ptr(expert_scales), _ptr(topk_weights),
                                _ptr(dst_row), T, H, K, _ptr(out), _stream(stream))
    _raise("moe_combine_fp8", st)


# The calls below test their tensors in place: a function call for each would
# cost as much as the tests, and a small call waits for its host side.
_bf16, _f32, _i32, _i8 = torch.bfloat16, torch.float32, torch.int32, torch.int8


def _check_all(pairs) -> None:
    """The error of the first (name, tensor, dtype) that does not fit."""
    for name, t, dtype in pairs:
        _check(name, t, dtype)


def moe_dispatch_int8(tokens, dst_row, packed, scales, stream=None) -> None:
    """Pack token rows into their K slots as int8 codes with one scale a row."""
    T, H = tokens.shape
    K = dst_row.shape[1] if dst_row.dim() == 2 else 1
    if not (tokens.dtype is _bf16 and tokens.is_cuda and tokens.is_contiguous()
            and dst_row.dtype is _i32 and dst_row.is_cuda and dst_row.is_contiguous()
            and packed.dtype is _i8 and packed.is_cuda and packed.is_contiguous()
            and scales.dtype is _f32 and scales.is_cuda and scales.is_contiguous()):
        _check_all((("tokens", tokens, torch.bfloat16), ("dst_row", dst_row, torch.int32),
                    ("packed", packed, torch.int8), ("scales", scales, torch.float32)))
    rows = T * K
    if dst_row.numel() != rows or packed.numel() < rows * H or scales.numel() < rows:
        raise ValueError("moe_dispatch_int8: dst_row/packed/scales have the wrong size")
    st = (_lib or load()).moe_dispatch_int8(
        tokens.data_ptr(), T, H, K, dst_row.data_ptr(), packed.data_ptr(), scales.data_ptr(),
        _current_stream() if stream is None else _stream(stream))
    if st:
        _raise("moe_dispatch_int8", st)


def moe_expert_matmul_int8(x, x_scales, weights, w_scales, expert_offsets, out,
                           dev_error=None, stream=None) -> None:
    """Packed int8 rows times their experts' int8 weights (see include/moe_layout.h)."""
    rows, H = x.shape
    E, N = weights.shape[0], weights.shape[1]
    if not (x.dtype is _i8 and x.is_cuda and x.is_contiguous()
            and x_scales.dtype is _f32 and x_scales.is_cuda and x_scales.is_contiguous()
            and weights.dtype is _i8 and weights.is_cuda and weights.is_contiguous()
            and w_scales.dtype is _f32 and w_scales.is_cuda and w_scales.is_contiguous()
            and expert_offsets.dtype is _i32 and expert_offsets.is_cuda and expert_offsets.is_contiguous()
            and out.dtype is _bf16 and out.is_cuda and out.is_contiguous()):
        _check_all((("x", x, torch.int8), ("x_scales", x_scales, torch.float32),
                    ("weights", weights, torch.int8), ("w_scales", w_scales, torch.float32),
                    ("expert_offsets", expert_offsets, torch.int32), ("out", out, torch.bfloat16)))
    _check("dev_error", dev_error, torch.int32)
    if weights.dim() != 3 or weights.shape[2] != H or w_scales.numel() != E * N \
            or x_scales.numel() < rows or expert_offsets.numel() < E + 1 \
            or out.numel() < rows * N or out.shape[-1] != N:
        raise ValueError("moe_expert_matmul_int8: argument sizes disagree")
    st = (_lib or load()).moe_expert_matmul_int8(
        x.data_ptr(), x_scales.data_ptr(), weights.data_ptr(), w_scales.data_ptr(),
        expert_offsets.data_ptr(), rows, H, N, E, out.data_ptr(), _ptr(dev_error),
        _current_stream() if stream is None else _stream(stream))
    if st:
        _raise("moe_expert_matmul_int8", st)


def moe_route_workspace_bytes(T: int, E: int) -> int:
    return int(load().moe_route_workspace_bytes(T, E))


def _logits_type(fn: str, logits) -> int:
    if logits.dtype is _f32:
        return 0
    if logits.dtype is not _bf16:
        raise TypeError(f"{fn}: logits must be float32 or bfloat16, got {logits.dtype}")
    return 1


def moe_route(logits, topk_ids, topk_weights, expert_counts, routed_tokens, loss,
              renormalize: bool = True, loss_coef: float = 1.0, token_mask=None,
              workspace=None, stream=None) -> None:
    """Router logits to top-k ids, weights, counts and the balance loss (see
    include/moe_layout.h)."""
    T, E = logits.shape
    K = topk_ids.shape[1]
    bf16 = _logits_type("moe_route", logits)
    if not (logits.is_cuda and logits.is_contiguous()
            and topk_ids.dtype is _i32 and topk_ids.is_cuda and topk_ids.is_contiguous()
            and topk_weights.dtype is _f32 and topk_weights.is_cuda and topk_weights.is_contiguous()
            and expert_counts.dtype is _i32 and expert_counts.is_cuda and expert_counts.is_contiguous()
            and routed_tokens.dtype is _i32 and routed_tokens.is_cuda and routed_tokens.is_contiguous()
            and loss.dtype is _f32 and loss.is_cuda and loss.is_contiguous()):
        _check_all((("logits", logits, logits.dtype), ("topk_ids", topk_ids, torch.int32),
                    ("topk_weights", topk_weights, torch.float32),
                    ("expert_counts", expert_counts, torch.int32),
                    ("routed_tokens", routed_tokens, torch.int32), ("loss", loss, torch.float32)))
    if token_mask is not None:
        _check("token_mask", token_mask, torch.bool)
        if token_mask.numel() != T:
            raise ValueError("moe_route: token_mask has the wrong size")
    if topk_ids.numel() != T * K or topk_weights.numel() != T * K or expert_counts.numel() < E \
            or routed_tokens.numel() < 1 or loss.numel() < 1:
        raise ValueError("moe_route: output arrays have the wrong size")
    if workspace is not None and not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("moe_route: workspace must be a contiguous CUDA tensor")
    st = (_lib or load()).moe_route(
        logits.data_ptr(), bf16, T, E, K, 1 if renormalize else 0, loss_coef, _ptr(token_mask),
        topk_ids.data_ptr(), topk_weights.data_ptr(), expert_counts.data_ptr(),
        routed_tokens.data_ptr(), loss.data_ptr(), _ptr(workspace),
        0 if workspace is None else workspace.nbytes,
        _current_stream() if stream is None else _stream(stream))
    if st:
        _raise("moe_route", st)


def moe_route_backward(logits, topk_ids, expert_counts, routed_tokens, grad_weights, grad_loss,
                       grad_logits, renormalize: bool = True, loss_coef: float = 1.0,
                       stream=None) -> None:
    """Gradient of moe_route's weights and loss to the logits; grad_weights or
    grad_loss may be None (zero)."""
    T, E = logits.shape
    K = topk_ids.shape[1]
    bf16 = _logits_type("moe_route_backward", logits)
    if not (logits.is_cuda and logits.is_contiguous()
            and grad_logits.dtype is logits.dtype and grad_logits.is_cuda and grad_logits.is_contiguous()
            and topk_ids.dtype is _i32 and topk_ids.is_cuda and topk_ids.is_contiguous()
            and expert_counts.dtype is _i32 and expert_counts.is_cuda and expert_counts.is_contiguous()
            and routed_tokens.dtype is _i32 and routed_tokens.is_cuda and routed_tokens.is_contiguous()):
        _check_all((("logits", logits, logits.dtype), ("grad_logits", grad_logits, logits.dtype),
                    ("topk_ids", topk_ids, torch.int32),
                    ("expert_counts", expert_counts, torch.int32),
                    ("routed_tokens", routed_tokens, torch.int32)))
    _check("grad_weights", grad_weights, torch.float32)
    _check("grad_loss", grad_loss, torch.float32)
    if topk_ids.numel() != T * K or expert_counts.numel() < E or routed_tokens.numel() < 1 \
            or grad_logits.numel() != T * E \
            or (grad_weights is not None and grad_weights.numel() != T * K) \
            or (grad_loss is not None and grad_loss.numel() != 1):
        raise ValueError("moe_route_backward: argument sizes disagree")
    st = (_lib or load()).moe_route_backward(
        logits.data_ptr(), bf16, T, E, K, 1 if renormalize else 0, loss_coef, topk_ids.data_ptr(),
        expert_counts.data_ptr(), routed_tokens.data_ptr(), _ptr(grad_weights), _ptr(grad_loss),
        grad_logits.data_ptr(), _current_stream() if stream is None else _stream(stream))
    if st:
        _raise("moe_route_backward", st)


class RouteBuffers:
    """Device buffers for routing T tokens over E experts, K a token (allocated by torch)."""

    def __init__(self, T: int, K: int, E: int, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        self.T, self.K, self.E = T, K, E
        self.topk_ids = torch.empty((T, K), **i32)
        self.topk_weights = torch.empty((T, K), dtype=torch.float32, device=device)
        self.expert_counts = torch.empty(E, **i32)
        self.routed_tokens = torch.empty(1, **i32)
        self.loss = torch.empty(1, dtype=torch.float32, device=device)
        self.workspace = torch.empty(moe_route_workspace_bytes(T, E), dtype=torch.uint8,
                                     device=device)

    def run(self, logits, renormalize: bool = True, loss_coef: float = 1.0, token_mask=None,
            stream=None) -> "RouteBuffers":
        moe_route(logits, self.topk_ids, self.topk_weights, self.expert_counts,
                  self.routed_tokens, self.loss, renormalize, loss_coef, token_mask,
                  self.workspace, stream)
        return self

    def backward(self, logits, grad_weights, grad_loss, grad_logits, renormalize: bool = True,
                 loss_coef: float = 1.0, stream=None) -> None:
        """Gradient to the logits of the run() before it."""
        moe_route_backward(logits, self.topk_ids, self.expert_counts, self.routed_tokens,
                           grad_weights, grad_loss, grad_logits, renormalize, loss_coef, stream)


class LayoutBuffers:
    """Device buffers for one layout of T x K entries (allocated by torch)."""

    def __init__(self, T: int, K: int, E: int, R: int, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        self.T, self.K, self.E, self.R = T, K, E, R
        self.expert_counts = torch.empty(E, **i32)
        self.expert_offsets = torch.empty(E + 1, **i32)
        self.rank_offsets = torch.empty(R + 1, **i32)
        self.src_token = torch.empty(T * K, **i32)
        self.dst_row = torch.empty((T, K), **i32)
        self.dev_error = torch.empty(1, **i32)
        ws = moe_layout_workspace_bytes(T, K, E)
        self.workspace = torch.empty(ws, dtype=torch.uint8, device=device) if ws else None

    def run(self, topk_ids, stream=None) -> "LayoutBuffers":
        moe_layout(topk_ids, self.E, self.R, self.expert_counts,
                   self.expert_offsets, self.rank_offsets, self.src_token,
                   self.dst_row, self.dev_error, self.workspace, stream)
        return self

    def run_dispatch(self, topk_ids, tokens, packed, scales=None, fp8=False,
                     stream=None) -> "LayoutBuffers":
        """Layout and dispatch together (moe_layout_dispatch)."""
        moe_layout_dispatch(topk_ids, tokens, self.E, self.R, self.expert_counts,
                            self.expert_offsets, self.rank_offsets, self.src_token,
                            self.dst_row, packed, scales, fp8, self.dev_error,
                            self.workspace, stream)
        return self
