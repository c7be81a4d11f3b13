"""Thin Python binding over libpe's C ABI (include/pe.h).

Argument marshalling only: every step of the packed-attention path runs in the
library's CUDA kernels. PyTorch provides device memory (outputs and
workspaces are torch tensors) and the current CUDA stream. There is no CPU
fallback: if libpe.so is missing or the device is not sm_103a the calls raise.
"""

from __future__ import annotations

import ctypes
import math
import os

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpe.so")

PE_BF16 = 0
PE_FP32 = 1

EXPORTED = (
    "pe_status_string", "pe_abi_version", "pe_pack_workspace_size", "pe_pack_sequences",
    "pe_gather_packed", "pe_scatter_padded", "pe_attention_workspace_size",
    "pe_packed_attention_fwd", "pe_packed_attention_bwd", "pe_packed_attention_fwd_local",
    "pe_packed_attention_bwd_local", "pe_read_device_status", "pe_attention_kernel",
    "pe_rows_workspace_size", "pe_pack_document_ids", "pe_flatten_packed_metadata",
    "pe_packed_positions", "pe_rope_packed", "pe_layernorm", "pe_geglu", "pe_upload_packed",
    "pe_download_padded", "pe_packed_attention_fwd_noalloc", "pe_read_noalloc_status",
    "pe_set_wait_limit_ns", "pe_attention_kernel_local", "pe_rmsnorm", "pe_rmsnorm_fp8",
    "pe_rmsnorm_bwd_workspace_size", "pe_rmsnorm_bwd", "pe_quantize_fp8",
    "pe_matmul_fp8_workspace_size", "pe_matmul_fp8", "pe_read_matmul_status",
)

_lib = None


class PackedAttentionError(RuntimeError):
    def __init__(self, call: str, status: int, text: str):
        super().__init__(f"{call} failed with status {status}: {text}")
        self.status = status


def load_library(path: str = LIB_PATH):
    """Loads libpe.so and declares its signatures. Raises if it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"libpe.so not found at {path}; build it with "
            "`python -c 'import __graft_entry__ as g; g.build()'` (needs nvcc)")
    lib = ctypes.CDLL(path)
    c = ctypes
    i32, i64, vp, sz = c.c_int32, c.c_int64, c.c_void_p, c.c_size_t
    lib.pe_status_string.argtypes = [c.c_int]
    lib.pe_status_string.restype = c.c_char_p
    lib.pe_abi_version.argtypes = []
    lib.pe_abi_version.restype = c.c_int
    lib.pe_pack_workspace_size.argtypes = [i32]
    lib.pe_pack_workspace_size.restype = sz
    lib.pe_pack_sequences.argtypes = [vp, i32, i32, vp, vp, c.POINTER(i64), vp, sz, vp]
    lib.pe_pack_sequences.restype = c.c_int
    lib.pe_gather_packed.argtypes = [vp, vp, i64, i64, vp, vp]
    lib.pe_gather_packed.restype = c.c_int
    lib.pe_scatter_padded.argtypes = [vp, vp, i32, i32, i64, vp, vp]
    lib.pe_scatter_padded.restype = c.c_int
    lib.pe_attention_workspace_size.argtypes = [c.c_int, i32, i64, i32, i32, i32, c.c_int, c.c_int]
    lib.pe_attention_workspace_size.restype = sz
    lib.pe_packed_attention_fwd.argtypes = [c.c_int, i32, i64, i32, i32, i32, vp, vp, vp, vp,
                                            c.c_float, c.c_int, vp, vp, vp, sz, vp]
    lib.pe_packed_attention_fwd.restype = c.c_int
    lib.pe_packed_attention_bwd.argtypes = [c.c_int, i32, i64, i32, i32, i32, vp, vp, vp, vp,
                                            c.c_float, c.c_int, vp, vp, vp, vp, vp, vp, vp, sz,
                                            vp]
    lib.pe_packed_attention_bwd.restype = c.c_int
    lib.pe_packed_attention_fwd_local.argtypes = [c.c_int, i32, i64, i32, i32, i32, vp, vp, vp,
                                                  vp, c.c_float, i32, i32, c.c_int, vp, vp, vp,
                                                  sz, vp]
    lib.pe_packed_attention_fwd_local.restype = c.c_int
    lib.pe_packed_attention_bwd_local.argtypes = [c.c_int, i32, i64, i32, i32, i32, vp, vp, vp,
                                                  vp, c.c_float, i32, i32, c.c_int, vp, vp, vp,
                                                  vp, vp, vp, vp, sz, vp]
    lib.pe_packed_attention_bwd_local.restype = c.c_int
    lib.pe_rows_workspace_size.argtypes = [i32]
    lib.pe_rows_workspace_size.restype = sz
    lib.pe_pack_document_ids.argtypes = [vp, i32, i32, vp, vp, c.POINTER(i64), c.POINTER(i32),
                                         vp, sz, vp]
    lib.pe_pack_document_ids.restype = c.c_int
    lib.pe_flatten_packed_metadata.argtypes = [vp, vp, i32, i32, i32, vp, vp, c.POINTER(i64),
                                               c.POINTER(i32), vp, sz, vp]
    lib.pe_flatten_packed_metadata.restype = c.c_int
    lib.pe_upload_packed.argtypes = [vp, vp, i32, i32, i64, vp, vp]
    lib.pe_upload_packed.restype = c.c_int
    lib.pe_download_padded.argtypes = [vp, vp, i32, i32, i64, vp, vp]
    lib.pe_download_padded.restype = c.c_int
    lib.pe_packed_positions.argtypes = [vp, i32, i64, vp, vp]
    lib.pe_packed_positions.restype = c.c_int
    lib.pe_rope_packed.argtypes = [c.c_int, vp, i32, vp, i32, vp, i64, i32, c.c_double, vp]
    lib.pe_rope_packed.restype = c.c_int
    lib.pe_layernorm.argtypes = [c.c_int, vp, vp, vp, vp, i64, i32, c.c_float, vp, vp, vp]
    lib.pe_layernorm.restype = c.c_int
    lib.pe_geglu.argtypes = [c.c_int, vp, i64, i32, vp, vp]
    lib.pe_geglu.restype = c.c_int
    lib.pe_attention_kernel.argtypes = [c.c_int, i32, c.c_int, c.c_int]
    lib.pe_attention_kernel.restype = c.c_char_p
    lib.pe_attention_kernel_local.argtypes = [c.c_int, i32, i32, i32, i32, c.c_int, c.c_int]
    lib.pe_attention_kernel_local.restype = c.c_char_p
    lib.pe_read_device_status.argtypes = [vp, vp]
    lib.pe_read_device_status.restype = c.c_int
    lib.pe_read_noalloc_status.argtypes = [vp]
    lib.pe_read_noalloc_status.restype = c.c_int
    lib.pe_set_wait_limit_ns.argtypes = [c.c_uint64]
    lib.pe_set_wait_limit_ns.restype = c.c_uint64
    lib.pe_packed_attention_fwd_noalloc.argtypes = [c.c_int, i32, i64, i32, i32, i32, vp, vp, vp,
                                                    vp, c.c_float, c.c_int, vp, vp, vp]
    lib.pe_packed_attention_fwd_noalloc.restype = c.c_int
    lib.pe_rmsnorm.argtypes = [c.c_int, vp, vp, vp, i64, i32, c.c_float, vp, vp, vp]
    lib.pe_rmsnorm.restype = c.c_int
    lib.pe_rmsnorm_fp8.argtypes = [c.c_int, c.c_int, vp, vp, vp, i64, i32, c.c_float, vp, i64, vp,
                                   vp, vp, vp]
    lib.pe_rmsnorm_fp8.restype = c.c_int
    lib.pe_rmsnorm_bwd_workspace_size.argtypes = [i32]
    lib.pe_rmsnorm_bwd_workspace_size.restype = sz
    lib.pe_rmsnorm_bwd.argtypes = [c.c_int, vp, vp, vp, vp, i64, i32, c.c_float, vp, vp, vp, sz,
                                   vp]
    lib.pe_rmsnorm_bwd.restype = c.c_int
    lib.pe_quantize_fp8.argtypes = [c.c_int, c.c_int, vp, i64, i64, i32, vp, i64, vp, vp, i64, vp,
                                    vp]
    lib.pe_quantize_fp8.restype = c.c_int
    lib.pe_matmul_fp8_workspace_size.argtypes = [i64, i64, i64]
    lib.pe_matmul_fp8_workspace_size.restype = sz
    lib.pe_matmul_fp8.argtypes = [c.c_int, vp, i64, vp, c.c_int, vp, i64, vp, i64, i64, i64,
                                  c.c_int, vp, vp, sz, vp]
    lib.pe_matmul_fp8.restype = c.c_int
    lib.pe_read_matmul_status.argtypes = [vp]
    lib.pe_read_matmul_status.restype = c.c_int
    _lib = lib
    return lib


def _check(call: str, status: int):
    if status != 0:
        text = load_library().pe_status_string(status).decode()
        raise PackedAttentionError(call, status, text)


# The handle of a device's current stream without a Stream object around it
# (2 us a call on the GPU's host); the public way where torch lacks it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(device: torch.device) -> int:
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _dtype_code(dtype: torch.dtype) -> int:
    if dtype == torch.bfloat16:
        return PE_BF16
    if dtype == torch.float32:
        return PE_FP32
    raise TypeError(f"unsupported dtype {dtype}: bfloat16 or float32 only")


def _cuda(t: torch.Tensor, name: str) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
    return t.contiguous()


def _cuda_or_pinned(t: torch.Tensor, name: str) -> torch.Tensor:
    """A CUDA tensor, or a pinned host tensor that kernels address directly."""
    if not (t.is_cuda or t.is_pinned()):
        raise ValueError(f"{name} must be a CUDA tensor or pinned host memory")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def pe_pack_sequences(lengths: torch.Tensor, max_seq_len: int):
    """Returns (flat_index int64 [N], cu_seqlens int32 [B+1], N) for device lengths."""
    lib = load_library()
    lengths = _cuda(lengths, "lengths").to(torch.int32)
    b = int(lengths.numel())
    dev = lengths.device
    flat = torch.empty(max(b * int(max_seq_len), 1), dtype=torch.int64, device=dev)
    cu = torch.empty(b + 1, dtype=torch.int32, device=dev)
    ws = _workspace(lib.pe_pack_workspace_size(b), dev)
    n = ctypes.c_int64(0)
    _check("pe_pack_sequences",
           lib.pe_pack_sequences(_ptr(lengths), b, int(max_seq_len), _ptr(flat), _ptr(cu),
                                 ctypes.byref(n), _ptr(ws), ws.numel(), _stream(dev)))
    return flat[: n.value], cu, int(n.value)


def pe_pack_document_ids(document_ids: torch.Tensor):
    """Indexed packing mask [B, S] (document i of a row marked i, 0 = padding)
    -> (flat_index int64 [N] into the [B, S] layout, cu_seqlens int32 [D+1], N)."""
    lib = load_library()
    ids = _cuda(document_ids, "document_ids").to(torch.int32)
    b, s = (int(x) for x in ids.shape)
    dev = ids.device
    flat = torch.empty(max(b * s, 1), dtype=torch.int64, device=dev)
    cu = torch.empty(b * s + 1, dtype=torch.int32, device=dev)
    ws = _workspace(lib.pe_rows_workspace_size(b), dev)
    n, d = ctypes.c_int64(0), ctypes.c_int32(0)
    _check("pe_pack_document_ids",
           lib.pe_pack_document_ids(_ptr(ids), b, s, _ptr(flat), _ptr(cu), ctypes.byref(n),
                                    ctypes.byref(d), _ptr(ws), ws.numel(), _stream(dev)))
    return flat[: n.value], cu[: d.value + 1], int(n.value)


def pe_flatten_packed_metadata(token_indices: torch.Tensor, row_cu_seqlens: torch.Tensor):
    """Row-local token indices [B, S] and row-local cumulative lengths [B, M+1]
    (both -1 padded) -> (flat_index int64 [N], cu_seqlens int32 [D+1], N)."""
    lib = load_library()
    tok = _cuda(token_indices, "token_indices").to(torch.int64)
    rcu = _cuda(row_cu_seqlens, "row_cu_seqlens").to(torch.int32)
    b, s = (int(x) for x in tok.shape)
    m1 = int(rcu.shape[1])
    if int(rcu.shape[0]) != b:
        raise ValueError("token_indices and row_cu_seqlens disagree on the number of rows")
    dev = tok.device
    flat = torch.empty(max(b * s, 1), dtype=torch.int64, device=dev)
    cu = torch.empty(b * max(m1 - 1, 0) + 1, dtype=torch.int32, device=dev)
    ws = _workspace(lib.pe_rows_workspace_size(b), dev)
    n, d = ctypes.c_int64(0), ctypes.c_int32(0)
    _check("pe_flatten_packed_metadata",
           lib.pe_flatten_packed_metadata(_ptr(tok), _ptr(rcu), b, s, m1, _ptr(flat), _ptr(cu),
                                          ctypes.byref(n), ctypes.byref(d), _ptr(ws), ws.numel(),
                                          _stream(dev)))
    return flat[: n.value], cu[: d.value + 1], int(n.value)


def pe_gather_packed(padded: torch.Tensor, flat_index: torch.Tensor, num_tokens: int | None = None,
                     out: torch.Tensor | None = None):
    """packed[t] = padded.flatten(0, 1)[flat_index[t]] for a [B, S, ...] grid.
    The grid may be pinned host memory: only the real rows cross the host link."""
    lib = load_library()
    padded = _cuda_or_pinned(padded, "padded")
    flat_index = _cuda(flat_index, "flat_index")
    dev = flat_index.device
    n = int(flat_index.numel()) if num_tokens is None else int(num_tokens)
    row_shape = tuple(padded.shape[2:])
    packed = (torch.empty((n,) + row_shape, dtype=padded.dtype, device=dev) if out is None
              else out)
    row_bytes = padded.element_size() * math.prod(row_shape)
    _check("pe_gather_packed",
           lib.pe_gather_packed(_ptr(padded), _ptr(flat_index), n, row_bytes, _ptr(packed),
                                _stream(dev)))
    return packed


def pe_upload_packed(padded_host: torch.Tensor, lengths_host, out: torch.Tensor) -> torch.Tensor:
    """Copies the real rows of a host [B, S, ...] grid into the packed device
    buffer `out` [sum L, ...] with one asynchronous copy per sequence on the
    current stream of out's device (pinned host memory for asynchrony)."""
    lib = load_library()
    if padded_host.is_cuda or not padded_host.is_contiguous():
        raise ValueError("padded_host must be a contiguous host tensor")
    lengths = np.ascontiguousarray(np.asarray(lengths_host, dtype=np.int32))
    b, s = int(padded_host.shape[0]), int(padded_host.shape[1])
    if lengths.shape != (b,):
        raise ValueError("one length per grid row")
    row_bytes = padded_host.element_size() * math.prod(tuple(padded_host.shape[2:]))
    # Checked before anything is enqueued: every copy writes L_i rows into out.
    if out.dtype != padded_host.dtype or not out.is_contiguous() or out.numel() != int(
            lengths.sum()) * (row_bytes // padded_host.element_size()):
        raise ValueError("out must be contiguous and hold sum(L) rows of the grid's row shape "
                         "and dtype")
    out = _cuda(out, "out")
    _check("pe_upload_packed",
           lib.pe_upload_packed(_ptr(padded_host), lengths.ctypes.data, b, s, row_bytes,
                                _ptr(out), _stream(out.device)))
    return out


def pe_download_padded(packed: torch.Tensor, lengths_host, out_host: torch.Tensor) -> torch.Tensor:
    """Copies the packed device rows [sum L, ...] into the real rows of the host
    [B, S, ...] grid `out_host` with one asynchronous copy per sequence on the
    current stream of packed's device (pinned host memory for asynchrony). Pad
    rows of out_host are not written: allocate it zeroed for to_dense_batch's
    zero fill."""
    lib = load_library()
    if out_host.is_cuda or not out_host.is_contiguous():
        raise ValueError("out_host must be a contiguous host tensor")
    lengths = np.ascontiguousarray(np.asarray(lengths_host, dtype=np.int32))
    b, s = int(out_host.shape[0]), int(out_host.shape[1])
    if lengths.shape != (b,):
        raise ValueError("one length per grid row")
    row_bytes = out_host.element_size() * math.prod(tuple(out_host.shape[2:]))
    if packed.dtype != out_host.dtype or not packed.is_contiguous() or packed.numel() != int(
            lengths.sum()) * (row_bytes // out_host.element_size()):
        raise ValueError("packed must be contiguous and hold sum(L) rows of the grid's row "
                         "shape and dtype")
    packed = _cuda(packed, "packed")
    _check("pe_download_padded",
           lib.pe_download_padded(_ptr(packed), lengths.ctypes.data, b, s, row_bytes,
                                  _ptr(out_host), _stream(packed.device)))
    return out_host


def pe_scatter_padded(packed: torch.Tensor, cu_seqlens: torch.Tensor, max_seq_len: int,
                      out: torch.Tensor | None = None):
    """Returns the zero-padded [B, S, ...] grid of a packed [N, ...] buffer; `out`
    may be pinned host memory (the rows are then written across the host link)."""
    lib = load_library()
    packed = _cuda(packed, "packed")
    if out is not None:
        out = _cuda_or_pinned(out, "out")
    cu_seqlens = _cuda(cu_seqlens, "cu_seqlens")
    b = int(cu_seqlens.numel()) - 1
    row_shape = tuple(packed.shape[1:])
    if out is None:
        out = torch.empty((b, int(max_seq_len)) + row_shape, dtype=packed.dtype,
                          device=packed.device)
    row_bytes = packed.element_size() * math.prod(row_shape)
    _check("pe_scatter_padded",
           lib.pe_scatter_padded(_ptr(packed), _ptr(cu_seqlens), b, int(max_seq_len), row_bytes,
                                 _ptr(out), _stream(packed.device)))
    return out


def attention_workspace_bytes(dtype, num_sequences, num_tokens, num_heads, head_dim,
                              max_seq_len, query_is_first_token=False, backward=False) -> int:
    return int(load_library().pe_attention_workspace_size(
        _dtype_code(dtype), int(num_sequences), int(num_tokens), int(num_heads), int(head_dim),
        int(max_seq_len), int(bool(query_is_first_token)), int(bool(backward))))


def pe_packed_attention_fwd(q, k, v, cu_seqlens, max_seq_len: int, scale: float | None = None,
                            query_is_first_token: bool = False, need_lse: bool = False,
                            out=None, lse=None, workspace=None):
    """Packed attention forward. Returns (out, lse or None)."""
    return _forward(None, q, k, v, cu_seqlens, max_seq_len, scale, query_is_first_token,
                    need_lse, out, lse, workspace)


def pe_packed_attention_fwd_local(q, k, v, cu_seqlens, max_seq_len: int, window_left: int,
                                  window_right: int, scale: float | None = None,
                                  query_is_first_token: bool = False, need_lse: bool = False,
                                  out=None, lse=None, workspace=None):
    """Local (sliding-window) packed attention forward: the query at position r
    sees keys r - window_left .. r + window_right of its own sequence (a negative
    bound is unbounded). Returns (out, lse or None)."""
    return _forward((int(window_left), int(window_right)), q, k, v, cu_seqlens, max_seq_len,
                    scale, query_is_first_token, need_lse, out, lse, workspace)


def _forward(window, q, k, v, cu_seqlens, max_seq_len, scale, query_is_first_token, need_lse,
             out, lse, workspace):
    lib = load_library()
    q, k, v = _cuda(q, "q"), _cuda(k, "k"), _cuda(v, "v")
    cu_seqlens = _cuda(cu_seqlens, "cu_seqlens")
    n, h, d = k.shape
    b = int(cu_seqlens.numel()) - 1
    nq = b if query_is_first_token else n
    if tuple(q.shape) != (nq, h, d) or v.shape != k.shape or q.dtype != k.dtype:
        raise ValueError(f"shape/dtype mismatch: q {tuple(q.shape)} k {tuple(k.shape)}")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if out is None:
        out = torch.empty_like(q)
    if need_lse and lse is None:
        lse = torch.empty((h, nq), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = _workspace(attention_workspace_bytes(q.dtype, b, n, h, d, max_seq_len,
                                                         query_is_first_token, False), q.device)
    head = (_dtype_code(q.dtype), b, n, h, d, int(max_seq_len), _ptr(q), _ptr(k), _ptr(v),
            _ptr(cu_seqlens), scale)
    tail = (int(bool(query_is_first_token)), _ptr(out), _ptr(lse), _ptr(workspace),
            workspace.numel(), _stream(q.device))
    if window is None:
        _check("pe_packed_attention_fwd", lib.pe_packed_attention_fwd(*head, *tail))
    else:
        _check("pe_packed_attention_fwd_local",
               lib.pe_packed_attention_fwd_local(*head, window[0], window[1], *tail))
    return out, lse


def pe_packed_attention_bwd(dout, q, k, v, out, lse, cu_seqlens, max_seq_len: int,
                            scale: float | None = None, query_is_first_token: bool = False,
                            workspace=None):
    """Packed attention backward. Returns (dq, dk, dv)."""
    return _backward(None, dout, q, k, v, out, lse, cu_seqlens, max_seq_len, scale,
                     query_is_first_token, workspace)


def pe_packed_attention_bwd_local(dout, q, k, v, out, lse, cu_seqlens, max_seq_len: int,
                                  window_left: int, window_right: int,
                                  scale: float | None = None, query_is_first_token: bool = False,
                                  workspace=None):
    """Local (sliding-window) packed attention backward; out and lse come from
    pe_packed_attention_fwd_local with the same window. Returns (dq, dk, dv)."""
    return _backward((int(window_left), int(window_right)), dout, q, k, v, out, lse, cu_seqlens,
                     max_seq_len, scale, query_is_first_token, workspace)


def _backward(window, dout, q, k, v, out, lse, cu_seqlens, max_seq_len, scale,
              query_is_first_token, workspace):
    lib = load_library()
    q, k, v = _cuda(q, "q"), _cuda(k, "k"), _cuda(v, "v")
    out, dout, lse = _cuda(out, "out"), _cuda(dout, "dout"), _cuda(lse, "lse")
    cu_seqlens = _cuda(cu_seqlens, "cu_seqlens")
    n, h, d = k.shape
    b = int(cu_seqlens.numel()) - 1
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if workspace is None:
        workspace = _workspace(attention_workspace_bytes(q.dtype, b, n, h, d, max_seq_len,
                                                         query_is_first_token, True), q.device)
    head = (_dtype_code(q.dtype), b, n, h, d, int(max_seq_len), _ptr(q), _ptr(k), _ptr(v),
            _ptr(cu_seqlens), scale)
    tail = (int(bool(query_is_first_token)), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq),
            _ptr(dk), _ptr(dv), _ptr(workspace), workspace.numel(), _stream(q.device))
    if window is None:
        _check("pe_packed_attention_bwd", lib.pe_packed_attention_bwd(*head, *tail))
    else:
        _check("pe_packed_attention_bwd_local",
               lib.pe_packed_attention_bwd_local(*head, window[0], window[1], *tail))
    return dq, dk, dv


def pe_attention_kernel(dtype: torch.dtype, head_dim: int, query_is_first_token: bool = False,
                        backward: bool = False, window=None, max_seq_len: int | None = None) -> str:
    """Kernel family the forward (or backward) dispatches to for these arguments;
    with window = (left, right) and max_seq_len, that of the local calls."""
    lib = load_library()
    if window is None:
        return lib.pe_attention_kernel(
            _dtype_code(dtype), int(head_dim), int(bool(query_is_first_token)),
            int(bool(backward))).decode()
    if max_seq_len is None:
        raise ValueError("a window needs max_seq_len")
    return lib.pe_attention_kernel_local(
        _dtype_code(dtype), int(head_dim), int(max_seq_len), int(window[0]), int(window[1]),
        int(bool(query_is_first_token)), int(bool(backward))).decode()


def pe_read_device_status(workspace: torch.Tensor) -> int:
    """Device-side status left in an attention workspace (0 = the layout passed
    its check and every pipeline wait completed)."""
    lib = load_library()
    return int(lib.pe_read_device_status(_ptr(workspace), _stream(workspace.device)))


def pe_set_wait_limit_ns(ns: int) -> int:
    """Process-wide limit of the kernels' bounded pipeline waits (0 = the
    default 2 s); returns the previous limit."""
    return int(load_library().pe_set_wait_limit_ns(int(ns)))


def pe_packed_attention_fwd_noalloc(q, k, v, cu_seqlens, max_seq_len: int,
                                    scale: float | None = None,
                                    query_is_first_token: bool = False, need_lse: bool = False,
                                    out=None, lse=None):
    """The forward without a workspace: the library's static device array holds
    its scratch. Returns (out, lse or None)."""
    lib = load_library()
    q, k, v = _cuda(q, "q"), _cuda(k, "k"), _cuda(v, "v")
    cu_seqlens = _cuda(cu_seqlens, "cu_seqlens")
    n, h, d = k.shape
    b = int(cu_seqlens.numel()) - 1
    nq = b if query_is_first_token else n
    if tuple(q.shape) != (nq, h, d) or v.shape != k.shape or q.dtype != k.dtype:
        raise ValueError(f"shape/dtype mismatch: q {tuple(q.shape)} k {tuple(k.shape)}")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if out is None:
        out = torch.empty_like(q)
    if need_lse and lse is None:
        lse = torch.empty((h, nq), dtype=torch.float32, device=q.device)
    _check("pe_packed_attention_fwd_noalloc",
           lib.pe_packed_attention_fwd_noalloc(
               _dtype_code(q.dtype), b, n, h, d, int(max_seq_len), _ptr(q), _ptr(k), _ptr(v),
               _ptr(cu_seqlens), scale, int(bool(query_is_first_token)), _ptr(out), _ptr(lse),
               _stream(q.device)))
    return out, lse


def pe_read_noalloc_status(device=None) -> int:
    """Device-side status of the last allocation-free forward on the device."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    return int(load_library().pe_read_noalloc_status(_stream(dev)))


# --------------------------------------------------------------------------- layer tail

def pe_packed_positions(cu_seqlens: torch.Tensor, num_tokens: int, out=None) -> torch.Tensor:
    """Position of every token inside its own sequence (int32 [num_tokens])."""
    lib = load_library()
    cu = _cuda(cu_seqlens, "cu_seqlens")
    if out is None:
        out = torch.empty(int(num_tokens), dtype=torch.int32, device=cu.device)
    _check("pe_packed_positions",
           lib.pe_packed_positions(_ptr(cu), int(cu.numel()) - 1, int(num_tokens), _ptr(out),
                                   _stream(cu.device)))
    return out


def pe_rope_packed(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor,
                   theta: float) -> None:
    """Split-half rotary embedding, in place, on q [N, Hq, D] and k [N, Hk, D]."""
    lib = load_library()
    if not (q.is_cuda and q.is_contiguous()) or (k is not None and not k.is_contiguous()):
        raise ValueError("q and k must be contiguous CUDA tensors (rotated in place)")
    positions = _cuda(positions, "positions").to(torch.int32)
    n, hq, d = q.shape
    hk = 0 if k is None else int(k.shape[1])
    _check("pe_rope_packed",
           lib.pe_rope_packed(_dtype_code(q.dtype), _ptr(q), hq, _ptr(k), hk, _ptr(positions), n,
                              d, float(theta), _stream(q.device)))


def pe_layernorm(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
                 eps: float = 1e-5, residual: torch.Tensor | None = None, out=None):
    """LayerNorm over the last dim of x [N, C]; with a residual, of h = x + residual
    (rounded to x's dtype), returning (y, h). Otherwise returns y."""
    lib = load_library()
    x = _cuda(x, "x")
    n, c = x.shape
    weight = _cuda(weight, "weight").to(x.dtype)
    bias = None if bias is None else _cuda(bias, "bias").to(x.dtype)
    residual = None if residual is None else _cuda(residual, "residual")
    y = torch.empty_like(x) if out is None else out
    h = torch.empty_like(x) if residual is not None else None
    _check("pe_layernorm",
           lib.pe_layernorm(_dtype_code(x.dtype), _ptr(x), _ptr(residual), _ptr(weight),
                            _ptr(bias), n, c, float(eps), _ptr(y), _ptr(h), _stream(x.device)))
    return (y, h) if residual is not None else y


def pe_geglu(x: torch.Tensor, out=None) -> torch.Tensor:
    """gelu(x[:, :F]) * x[:, F:] for x [N, 2F] (exact GELU)."""
    lib = load_library()
    x = _cuda(x, "x")
    n, f2 = x.shape
    y = torch.empty((n, f2 // 2), dtype=x.dtype, device=x.device) if out is None else out
    _check("pe_geglu", lib.pe_geglu(_dtype_code(x.dtype), _ptr(x), n, f2 // 2, _ptr(y),
                                    _stream(x.device)))
    return y


# --------------------------------------------------------------------------- 8-bit layer

_FP8_CODES = {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}


def _fp8_code(dtype: torch.dtype) -> int:
    code = _FP8_CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}: float8_e4m3fn or float8_e5m2 only")
    return code


def _call(name: str, device: torch.device, *args) -> None:
    """Runs one entry point on `device` and its current stream."""
    fn = getattr(_lib or load_library(), name)
    if device.index == _current_device():
        status = fn(*args, _stream(device))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _stream(device))
    if status:
        _check(name, status)


def _input(t: torch.Tensor, name: str, like: torch.Tensor | None = None,
           shape=None) -> torch.Tensor:
    """A contiguous CUDA tensor on the device and in the dtype of `like`."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
    if like is not None and (t.dtype is not like.dtype or t.get_device() != like.get_device()):
        raise ValueError(f"{name} must be {like.dtype} on {like.device}, got {t.dtype} on {t.device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t if t.is_contiguous() else t.contiguous()


def _output(t: torch.Tensor | None, name: str, shape, dtype, device) -> torch.Tensor:
    """The caller's contiguous output tensor after a check, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if t.shape != shape or t.dtype != dtype or t.device != device or not (
            t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on "
                         f"{device}")
    return t


def _two_dims(t: torch.Tensor, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, got shape {tuple(t.shape)}")
    return t.shape


def _round16(n: int) -> int:
    return (n + 15) // 16 * 16


def _fp8_rows_ok(t: torch.Tensor) -> bool:
    """Rows of adjacent bytes that start at multiples of 16."""
    rows, cols = t.shape
    ld, step = t.stride()
    return (t.data_ptr() % 16 == 0 and (cols <= 1 or step == 1)
            and (rows <= 1 or (ld % 16 == 0 and ld >= cols)))


def _fp8_ld(t: torch.Tensor) -> int:
    return t.stride(0) if t.shape[0] > 1 else _round16(t.shape[1])


def _fp8_empty(rows: int, cols: int, dtype, device) -> torch.Tensor:
    """An 8-bit matrix whose rows start at multiples of 16 bytes."""
    return torch.empty_strided((rows, cols), (_round16(cols), 1), dtype=dtype, device=device)


def _fp8_output(t: torch.Tensor | None, name: str, rows: int, cols: int, dtype, device):
    if t is None:
        return _fp8_empty(rows, cols, dtype, device)
    if t.shape != (rows, cols) or t.dtype != dtype or t.device != device or not _fp8_rows_ok(t):
        raise ValueError(f"{name} must be a {dtype} matrix of shape {(rows, cols)} on {device} "
                         "whose rows start at multiples of 16 bytes")
    return t


def _fp8_operand(t: torch.Tensor, name: str) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
    _two_dims(t, name)
    if _fp8_rows_ok(t):
        return t
    return _fp8_empty(t.shape[0], t.shape[1], t.dtype, t.device).copy_(t)


def _workspace_for(t: torch.Tensor | None, need: int, device) -> tuple[torch.Tensor, int]:
    """The caller's workspace after a check (kernels write there), or a new one, and
    its bytes."""
    if t is None:
        t = _workspace(need, device)
    elif t.device != device or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return t, t.numel() * t.element_size()


def _norm_weight(weight, rows, c) -> torch.Tensor:
    """The weight in the rows' dtype: another one is refused, since a cast here would
    round it without the caller's knowledge."""
    if weight.dtype is not rows.dtype:
        _dtype_code(rows.dtype)
        raise ValueError(f"weight must be {rows.dtype} like the rows, got {weight.dtype}")
    return _input(weight, "weight", rows, (c,))


def _norm_inputs(x, weight, residual):
    x = _input(x, "x")
    _, c = _two_dims(x, "x")
    weight = _norm_weight(weight, x, c)
    if residual is not None:
        residual = _input(residual, "residual", x, x.shape)
    return x, weight, residual


def pe_rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5,
               residual: torch.Tensor | None = None, out=None, residual_out=None):
    """RMSNorm over the last dim of x [N, C]; with a residual, of h = x + residual
    (rounded to x's dtype), returning (y, h). Otherwise returns y. weight [C] and
    residual are in x's dtype."""
    x, weight, residual = _norm_inputs(x, weight, residual)
    n, c = x.shape
    y = _output(out, "out", x.shape, x.dtype, x.device)
    if residual is None and residual_out is not None:
        raise ValueError("residual_out needs a residual")
    h = None if residual is None else _output(residual_out, "residual_out", x.shape, x.dtype,
                                              x.device)
    _call("pe_rmsnorm", x.device, _dtype_code(x.dtype), x.data_ptr(), _ptr(residual),
          weight.data_ptr(), n, c, float(eps), y.data_ptr(), _ptr(h))
    return y if residual is None else (y, h)


def pe_rmsnorm_fp8(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5,
                   residual: torch.Tensor | None = None, dtype=torch.float8_e4m3fn, out=None,
                   y=None, residual_out=None):
    """RMSNorm with an 8-bit output: returns (q [N, C], scales fp32
    [ceil(C / 128), N]), and also h = x + residual with a residual. q's rows
    start at multiples of 16 bytes (its stride is C rounded up to a multiple of
    16). With `y` (a tensor like x) the norm is also written there in x's dtype.
    weight [C] and residual are in x's dtype."""
    x, weight, residual = _norm_inputs(x, weight, residual)
    n, c = x.shape
    code = _fp8_code(dtype)
    q = _fp8_output(out, "out", n, c, dtype, x.device)
    scales = torch.empty(((c + 127) // 128, n), dtype=torch.float32, device=x.device)
    if y is not None:
        y = _output(y, "y", x.shape, x.dtype, x.device)
    if residual is None and residual_out is not None:
        raise ValueError("residual_out needs a residual")
    h = None if residual is None else _output(residual_out, "residual_out", x.shape, x.dtype,
                                              x.device)
    _call("pe_rmsnorm_fp8", x.device, _dtype_code(x.dtype), code, x.data_ptr(), _ptr(residual),
          weight.data_ptr(), n, c, float(eps), q.data_ptr(), _fp8_ld(q), scales.data_ptr(),
          _ptr(y), _ptr(h))
    return (q, scales) if residual is None else (q, scales, h)


def pe_rmsnorm_bwd(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5,
                   dresidual: torch.Tensor | None = None, out=None, workspace=None):
    """RMSNorm backward for the stored norm input h [N, C]; dresidual is the
    gradient that reaches h by other ways; dy, weight and dresidual are in h's dtype.
    Returns (dx, dweight): dx (of x and of residual alike) in h's dtype, dweight fp32
    [C]."""
    lib = load_library()
    h = _input(h, "h")
    n, c = _two_dims(h, "h")
    dy = _input(dy, "dy", h, h.shape)
    weight = _norm_weight(weight, h, c)
    if dresidual is not None:
        dresidual = _input(dresidual, "dresidual", h, h.shape)
    dx = _output(out, "out", h.shape, h.dtype, h.device)
    dweight = torch.empty(c, dtype=torch.float32, device=h.device)
    ws, ws_bytes = _workspace_for(workspace, lib.pe_rmsnorm_bwd_workspace_size(c), h.device)
    _call("pe_rmsnorm_bwd", h.device, _dtype_code(h.dtype), dy.data_ptr(), h.data_ptr(),
          weight.data_ptr(), _ptr(dresidual), n, c, float(eps), dx.data_ptr(),
          dweight.data_ptr(), ws.data_ptr(), ws_bytes)
    return dx, dweight


def pe_quantize_fp8(x: torch.Tensor, block_rows: int = 1, dtype=torch.float8_e4m3fn,
                    plain: bool = True, transposed: bool = False):
    """x [R, C] in 8 bits with one fp32 scale for each block of block_rows (1 or
    128) x 128: (q [R, C], scales [ceil(C / 128), ceil(R / block_rows)]) when
    `plain`, and the same of x's transpose when `transposed` (both: four
    tensors). Rows of q start at multiples of 16 bytes."""
    x = _input(x, "x")
    r, c = _two_dims(x, "x")
    code = _fp8_code(dtype)
    if block_rows not in (1, 128):
        raise ValueError(f"block_rows must be 1 or 128, got {block_rows}")
    if not (plain or transposed):
        raise ValueError("neither the matrix nor its transpose is wanted")

    def outputs(rows, cols):
        return (_fp8_empty(rows, cols, dtype, x.device),
                torch.empty(((cols + 127) // 128, -(-rows // block_rows)), dtype=torch.float32,
                            device=x.device))

    q, s = outputs(r, c) if plain else (None, None)
    qt, st = outputs(c, r) if transposed else (None, None)
    _call("pe_quantize_fp8", x.device, _dtype_code(x.dtype), code, x.data_ptr(), r, c,
          block_rows, _ptr(q), _fp8_ld(q) if plain else 0, _ptr(s), _ptr(qt),
          _fp8_ld(qt) if transposed else 0, _ptr(st))
    return ((q, s) if plain else ()) + ((qt, st) if transposed else ())


def pe_matmul_fp8(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor,
                  b_scales: torch.Tensor, dtype=torch.bfloat16, out=None, workspace=None):
    """a [M, K] times the transpose of b [N, K], both in 8 bits: a with scales of
    1 x 128 blocks [ceil(K / 128), M], b with scales of 128 x 128 blocks
    [ceil(K / 128), ceil(N / 128)]. Returns [M, N] in `dtype` (bfloat16 or
    float32), or in out and its dtype."""
    lib = load_library()
    a, b = _fp8_operand(a, "a"), _fp8_operand(b, "b")
    a_code, b_code = _fp8_code(a.dtype), _fp8_code(b.dtype)
    m, k = a.shape
    n = b.shape[0]
    dev = a.device
    if b.shape[1] != k or b.device != dev:
        raise ValueError(f"a is {tuple(a.shape)} on {dev}, b is {tuple(b.shape)} on {b.device}")
    kb = (k + 127) // 128
    for name, s, shape in (("a_scales", a_scales, (kb, m)),
                           ("b_scales", b_scales, (kb, (n + 127) // 128))):
        if s.shape != shape or s.dtype != torch.float32 or s.device != dev:
            raise ValueError(f"{name} must be float32 of shape {shape} on {dev}")
    a_scales, b_scales = a_scales.contiguous(), b_scales.contiguous()
    out = _output(out, "out", (m, n), dtype if out is None else out.dtype, dev)
    need = lib.pe_matmul_fp8_workspace_size(m, n, k)
    ws, ws_bytes = _workspace_for(workspace, need, dev) if need else (None, 0)
    _call("pe_matmul_fp8", dev, a_code, a.data_ptr(), _fp8_ld(a), a_scales.data_ptr(), b_code,
          b.data_ptr(), _fp8_ld(b), b_scales.data_ptr(), m, n, k, _dtype_code(out.dtype),
          out.data_ptr(), _ptr(ws), ws_bytes)
    return out


def pe_read_matmul_status(device=None) -> int:
    """Status of the 8-bit matrix products on the device since the last read (0:
    every pipeline wait completed); waits for the current stream and clears it."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else (
        torch.device(device))
    with torch.cuda.device(dev):
        return int(load_library().pe_read_matmul_status(_stream(dev)))
