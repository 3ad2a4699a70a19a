"""Thin Python binding of the C ABI in include/fa.h (argument marshalling only).

Every step of the attention forward pass runs in the CUDA library
``libfa.so``; this module only checks tensor metadata, passes raw device
pointers and the current CUDA stream, and turns status codes into
exceptions. There is no fallback: if the library is missing, every call
raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfa.so")

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_CUDA = 3
FA_ERR_TIMEOUT = 4

#: every symbol include/fa.h declares
EXPORTED = ("fa_fwd", "fa_get_device_status", "fa_status_string", "fa_last_cuda_error", "fa_fwd_fault_test",
            "fa_naive_fwd", "fa_naive_workspace_bytes", "fa_naive_fwd_noalloc", "fa_bwd", "fa_bwd_workspace_bytes",
            "fa_bwd_fault_test", "fa_fwd_kv", "fa_fwd_kv_num_splits", "fa_fwd_kv_workspace_bytes",
            "fa_fwd_kv_fault_test", "fa_merge_partials", "fa_fwd_host", "fa_fwd_host_workspace_bytes",
            "fa_fwd_kv_f32", "fa_fwd_kv_f32_workspace_bytes", "fa_fwd_launch_shape",
            "fa_fwd_varlen", "fa_fwd_varlen_workspace_bytes", "fa_fwd_varlen_fault_test",
            "fa_bwd_varlen", "fa_bwd_varlen_workspace_bytes", "fa_bwd_varlen_fault_test",
            "fa_fwd_prefix", "fa_fwd_prefix_workspace_bytes", "fa_fwd_prefix_fault_test",
            "fa_rope_frequencies", "fa_rope", "fa_kv_append", "fa_fwd_paged", "fa_fwd_paged_workspace_bytes",
            "fa_fwd_paged_fault_test")

_lib = None


class Strides(ctypes.Structure):
    """fa_strides_t: element strides of a packed tensor [T, heads, d]."""
    _fields_ = [("token", ctypes.c_longlong), ("head", ctypes.c_longlong)]


class BatchStrides(ctypes.Structure):
    """fa_batch_strides_t: element strides of a tensor [B, heads, N, d]."""
    _fields_ = [("batch", ctypes.c_longlong), ("head", ctypes.c_longlong), ("row", ctypes.c_longlong)]


class PageStrides(ctypes.Structure):
    """fa_page_strides_t: byte strides of 8-bit pages [num_pages, H_kv, page_size, d]."""
    _fields_ = [("page", ctypes.c_longlong), ("head", ctypes.c_longlong), ("row", ctypes.c_longlong)]


class FaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {fa_status_string(status)}"
        if status == FA_ERR_CUDA:
            msg += f" (cudaError {fa_last_cuda_error()})"
        super().__init__(msg)


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libfa.so (once). Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with exact_io_aware_34_gb300.build.build()")
    lib = ctypes.CDLL(path)
    vp, i, f, u64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_ulonglong
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, vp]
    lib.fa_fwd.restype = i
    lib.fa_fwd_host.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, ctypes.c_size_t, vp]
    lib.fa_fwd_host.restype = i
    lib.fa_fwd_host_workspace_bytes.argtypes = [i, i, i, i]
    lib.fa_fwd_host_workspace_bytes.restype = ctypes.c_size_t
    lib.fa_fwd_fault_test.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, u64, vp]
    lib.fa_fwd_fault_test.restype = i
    lib.fa_get_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint)]
    lib.fa_get_device_status.restype = i
    lib.fa_status_string.argtypes = [i]
    lib.fa_status_string.restype = ctypes.c_char_p
    lib.fa_last_cuda_error.argtypes = []
    lib.fa_last_cuda_error.restype = i
    lib.fa_naive_workspace_bytes.argtypes = [i, i, i]
    lib.fa_naive_workspace_bytes.restype = ctypes.c_size_t
    lib.fa_naive_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, vp, ctypes.c_size_t, vp]
    lib.fa_naive_fwd.restype = i
    lib.fa_naive_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, vp]
    lib.fa_naive_fwd_noalloc.restype = i
    lib.fa_bwd_workspace_bytes.argtypes = [i, i, i]
    lib.fa_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, vp, ctypes.c_size_t, vp]
    lib.fa_bwd.restype = i
    lib.fa_bwd_fault_test.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, vp, ctypes.c_size_t, i, u64,
                                      vp]
    lib.fa_bwd_fault_test.restype = i
    lib.fa_fwd_kv.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp, ctypes.c_size_t, vp]
    lib.fa_fwd_kv.restype = i
    lib.fa_fwd_kv_fault_test.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp, ctypes.c_size_t, i, u64, vp]
    lib.fa_fwd_kv_fault_test.restype = i
    lib.fa_fwd_kv_num_splits.argtypes = [i, i, i, i, i, i]
    lib.fa_fwd_kv_num_splits.restype = i
    lib.fa_fwd_kv_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
    lib.fa_fwd_kv_workspace_bytes.restype = ctypes.c_size_t
    lib.fa_fwd_kv_f32.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp, ctypes.c_size_t, vp]
    lib.fa_fwd_kv_f32.restype = i
    lib.fa_fwd_kv_f32_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
    lib.fa_fwd_kv_f32_workspace_bytes.restype = ctypes.c_size_t
    ip = ctypes.POINTER(ctypes.c_int)
    lib.fa_fwd_launch_shape.argtypes = [i, i, i, i, ip, ip, ip]
    lib.fa_fwd_launch_shape.restype = i
    lib.fa_merge_partials.argtypes = [vp, vp, vp, vp, i, ctypes.c_longlong, i, vp]
    lib.fa_merge_partials.restype = i
    sz = ctypes.c_size_t
    lib.fa_fwd_varlen_workspace_bytes.argtypes = [i, i, i, i, i, i]
    lib.fa_fwd_varlen_workspace_bytes.restype = sz
    lib.fa_fwd_varlen.argtypes = [vp] * 7 + [i] * 6 + [vp, f, i, vp, sz, vp]
    lib.fa_fwd_varlen.restype = i
    lib.fa_fwd_varlen_fault_test.argtypes = [vp] * 7 + [i] * 6 + [f, i, vp, sz, i, u64, vp]
    lib.fa_fwd_varlen_fault_test.restype = i
    lib.fa_bwd_varlen_workspace_bytes.argtypes = [i, i, i, i, i]
    lib.fa_bwd_varlen_workspace_bytes.restype = sz
    lib.fa_bwd_varlen.argtypes = [vp] * 11 + [i] * 6 + [vp, f, i, vp, sz, vp]
    lib.fa_bwd_varlen.restype = i
    lib.fa_bwd_varlen_fault_test.argtypes = [vp] * 11 + [i] * 6 + [f, i, vp, sz, i, u64, vp]
    lib.fa_bwd_varlen_fault_test.restype = i
    lib.fa_fwd_prefix_workspace_bytes.argtypes = [i] * 7
    lib.fa_fwd_prefix_workspace_bytes.restype = sz
    lib.fa_fwd_prefix.argtypes = [vp] * 8 + [i] * 7 + [vp, f, i, vp, sz, vp]
    lib.fa_fwd_prefix.restype = i
    lib.fa_fwd_prefix_fault_test.argtypes = [vp] * 8 + [i] * 7 + [f, i, vp, sz, i, u64, vp]
    lib.fa_fwd_prefix_fault_test.restype = i
    dbl = ctypes.c_double
    lib.fa_rope_frequencies.argtypes = [vp, i, dbl, i, dbl, dbl, dbl, dbl]
    lib.fa_rope_frequencies.restype = i
    lib.fa_rope.argtypes = [vp, vp, i, vp, vp, i, vp, vp, i, i, i, vp, i, i, f, vp]
    lib.fa_rope.restype = i
    lib.fa_kv_append.argtypes = [vp] * 13 + [i] * 9 + [vp, vp, i, f, vp]
    lib.fa_kv_append.restype = i
    lib.fa_fwd_paged_workspace_bytes.argtypes = [i] * 8
    lib.fa_fwd_paged_workspace_bytes.restype = sz
    lib.fa_fwd_paged.argtypes = [vp] * 10 + [i] * 8 + [vp, vp, f, i, vp, sz, vp]
    lib.fa_fwd_paged.restype = i
    lib.fa_fwd_paged_fault_test.argtypes = [vp] * 10 + [i] * 8 + [f, i, vp, sz, i, u64, vp]
    lib.fa_fwd_paged_fault_test.restype = i
    _lib = lib
    return lib


def fa_status_string(status: int) -> str:
    return load_library().fa_status_string(int(status)).decode()


def fa_last_cuda_error() -> int:
    return int(load_library().fa_last_cuda_error())


def _stream_handle(stream, device) -> int:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _on_stream(stream, device):
    """Context in which ``device`` is current and allocations belong to
    ``stream`` (None: torch's current stream of that device)."""
    if stream is None:
        return torch.cuda.device(device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device) if int(stream) \
            else torch.cuda.default_stream(device)
    if stream.device != device:
        raise ValueError(f"stream belongs to {stream.device}, the tensors to {device}")
    return torch.cuda.stream(stream)


#: index of the current device (torch.cuda.current_device without its initialisation, which a CUDA tensor has seen;
#: a torch built without CUDA lacks it)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _launch(fn, stream, device):
    """fn() with ``device`` current and ``stream`` torch's current stream: what
    fn allocates and enqueues belongs to it. (The usual case enters no context;
    small calls are bound by the host.)"""
    if stream is None and _current_device() == device.index:
        return fn()
    with _on_stream(stream, device):
        return fn()


def _check_qkv(q, k, v):
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype != torch.bfloat16:
            raise ValueError(f"{name} must be bfloat16, got {t.dtype}")
        if t.dim() != 4:
            raise ValueError(f"{name} must be [B, H, N, d]")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if not (q.shape == k.shape == v.shape):
        raise ValueError(f"q, k, v shapes differ: {tuple(q.shape)} {tuple(k.shape)} {tuple(v.shape)}")
    if not (q.device == k.device == v.device):
        raise ValueError("q, k, v must be on the same device")


def fa_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor | None = None,
           lse: torch.Tensor | None = None, scale: float | None = None, stream=None):
    """O = softmax(scale * q k^T) v and LSE, by one launch of the fused kernel.

    q, k, v: bf16 CUDA tensors [B, H, N, d], contiguous. ``o`` (bf16 [B,H,N,d])
    and ``lse`` (float32 [B,H,N]) are allocated with torch when not given.
    ``scale`` defaults to 1/sqrt(d). Enqueued on ``stream`` (default: torch's
    current stream for q's device). Returns (o, lse).
    """
    _check_qkv(q, k, v)
    B, H, N, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if o.dtype != torch.bfloat16 or o.shape != q.shape or not o.is_contiguous() or o.device != q.device:
        raise ValueError("o must be a contiguous bf16 tensor shaped like q on q's device")
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N) or not lse.is_contiguous() \
            or lse.device != q.device:
        raise ValueError("lse must be a contiguous float32 [B, H, N] tensor on q's device")
    lib = load_library()
    with torch.cuda.device(q.device):
        st = lib.fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                        B, H, N, d, float(scale), _stream_handle(stream, q.device))
    if st != FA_OK:
        raise FaError(st, "fa_fwd")
    return o, lse


def fa_fwd_host_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(load_library().fa_fwd_host_workspace_bytes(int(B), int(H), int(N), int(d)))


def fa_fwd_host(qh: torch.Tensor, kh: torch.Tensor, vh: torch.Tensor, oh: torch.Tensor | None = None,
                lseh: torch.Tensor | None = None, scale: float | None = None, num_chunks: int = 0, workspace=None,
                device=None, stream=None):
    """fa_fwd on host tensors, end to end (upload, kernel, download, pipelined
    over head groups by the library).

    qh, kh, vh: bf16 CPU tensors [B, H, N, d], contiguous (pinned for full copy
    bandwidth). ``oh`` / ``lseh`` (CPU, allocated pinned when not given) receive
    O and LSE. ``workspace``: a CUDA uint8 tensor of at least
    fa_fwd_host_workspace_bytes(B, H, N, d) bytes on ``device`` (default: the
    current CUDA device), allocated with torch when None. The call is
    asynchronous on ``stream``: synchronise it before reading ``oh`` and
    ``lseh``. Returns (oh, lseh).
    """
    for x in (qh, kh, vh):
        if x.device.type != "cpu" or x.dtype != torch.bfloat16 or not x.is_contiguous() or x.dim() != 4:
            raise ValueError("qh, kh, vh must be contiguous bf16 CPU tensors [B, H, N, d]")
    if not (qh.shape == kh.shape == vh.shape):
        raise ValueError("qh, kh, vh must have the same shape")
    B, H, N, d = qh.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if oh is None:
        oh = torch.empty(qh.shape, dtype=torch.bfloat16).pin_memory()
    if lseh is None:
        lseh = torch.empty((B, H, N), dtype=torch.float32).pin_memory()
    if oh.device.type != "cpu" or oh.dtype != torch.bfloat16 or oh.shape != qh.shape or not oh.is_contiguous():
        raise ValueError("oh must be a contiguous bf16 CPU tensor shaped like qh")
    if lseh.device.type != "cpu" or lseh.dtype != torch.float32 or tuple(lseh.shape) != (B, H, N) \
            or not lseh.is_contiguous():
        raise ValueError("lseh must be a contiguous float32 CPU tensor [B, H, N]")
    need = fa_fwd_host_workspace_bytes(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    lib = load_library()
    with torch.cuda.device(dev):
        st = lib.fa_fwd_host(qh.data_ptr(), kh.data_ptr(), vh.data_ptr(), oh.data_ptr(), lseh.data_ptr(), B, H, N, d,
                             float(scale), int(num_chunks), workspace.data_ptr(),
                             workspace.numel() * workspace.element_size(), _stream_handle(stream, dev))
    if st != FA_OK:
        raise FaError(st, "fa_fwd_host")
    return oh, lseh


def fa_naive_workspace_bytes(B: int, H: int, N: int) -> int:
    return int(load_library().fa_naive_workspace_bytes(int(B), int(H), int(N)))


def fa_naive_fwd(q, k, v, o=None, lse=None, scale: float | None = None, workspace=None, stream=None):
    """Standard attention with S and P materialised in ``workspace`` (the
    comparator of the fused kernel). ``workspace`` is a CUDA tensor of at least
    fa_naive_workspace_bytes(B, H, N) bytes; allocated with torch when None.
    Returns (o, lse)."""
    _check_qkv(q, k, v)
    B, H, N, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    need = fa_naive_workspace_bytes(B, H, N)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    lib = load_library()
    with torch.cuda.device(q.device):
        st = lib.fa_naive_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, N, d,
                              float(scale), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                              _stream_handle(stream, q.device))
    if st != FA_OK:
        raise FaError(st, "fa_naive_fwd")
    return o, lse


def fa_fwd_launch_shape(B: int, H: int, N: int, d: int) -> tuple:
    """(grid, cluster, whole_units) of the launch fa_fwd makes for these sizes
    on the current device: cluster is 1, or 2 when CTA pairs share the units
    of the last, partial round."""
    grid, cluster, whole = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    st = load_library().fa_fwd_launch_shape(int(B), int(H), int(N), int(d), ctypes.byref(grid),
                                            ctypes.byref(cluster), ctypes.byref(whole))
    if st != FA_OK:
        raise FaError(st, "fa_fwd_launch_shape")
    return grid.value, cluster.value, whole.value


def fa_fwd_kv_num_splits(B: int, H: int, H_kv: int, N_q: int, N_kv: int, d: int) -> int:
    return int(load_library().fa_fwd_kv_num_splits(int(B), int(H), int(H_kv), int(N_q), int(N_kv), int(d)))


def fa_fwd_kv_workspace_bytes(B: int, H: int, H_kv: int, N_q: int, N_kv: int, d: int, num_splits: int = 0) -> int:
    return int(load_library().fa_fwd_kv_workspace_bytes(int(B), int(H), int(H_kv), int(N_q), int(N_kv), int(d),
                                                         int(num_splits)))


def _check_kv(q, k, v):
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.bfloat16 or t.dim() != 4 \
                or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor [B, heads, N, d]")
    if k.shape != v.shape or q.shape[0] != k.shape[0] or q.shape[3] != k.shape[3]:
        raise ValueError(f"shapes do not match: q {tuple(q.shape)} k {tuple(k.shape)} v {tuple(v.shape)}")
    if not (q.device == k.device == v.device):
        raise ValueError("q, k, v must be on the same device")


def fa_fwd_kv(q, k, v, o=None, lse=None, scale: float | None = None, num_splits: int = 0, workspace=None,
              stream=None):
    """O = softmax(scale q k^T) v with shared K/V heads and any N_q, N_kv.

    q: bf16 [B, H, N_q, d]; k, v: bf16 [B, H_kv, N_kv, d] with H a multiple of
    H_kv (query head h uses K/V head h // (H // H_kv)). Returns (o, lse).
    ``num_splits`` = 0 lets the library choose the key split (none when the
    fused forward kernel fills the device; see :func:`fa_fwd_kv_num_splits`),
    1 forbids one; the workspace is allocated with torch when needed and not
    given.
    """
    _check_kv(q, k, v)
    B, H, N_q, d = q.shape
    H_kv, N_kv = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N_q), dtype=torch.float32, device=q.device)
    need = fa_fwd_kv_workspace_bytes(B, H, H_kv, N_q, N_kv, d, num_splits)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    lib = load_library()
    with torch.cuda.device(q.device):
        st = lib.fa_fwd_kv(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, H_kv, N_q,
                           N_kv, d, float(scale), int(num_splits), ws_ptr, ws_bytes, _stream_handle(stream, q.device))
    if st != FA_OK:
        raise FaError(st, "fa_fwd_kv")
    return o, lse


def fa_fwd_kv_f32_workspace_bytes(B: int, H: int, H_kv: int, N_q: int, N_kv: int, d: int,
                                  num_splits: int = 0) -> int:
    return int(load_library().fa_fwd_kv_f32_workspace_bytes(int(B), int(H), int(H_kv), int(N_q), int(N_kv), int(d),
                                                             int(num_splits)))


def fa_fwd_kv_f32(q, k, v, o=None, lse=None, scale: float | None = None, num_splits: int = 0, workspace=None,
                  stream=None):
    """:func:`fa_fwd_kv` with o returned in float32 (normalised, not rounded):
    the partial result of one key shard that a sequence split exchanges.
    Returns (o float32 [B, H, N_q, d], lse float32 [B, H, N_q])."""
    _check_kv(q, k, v)
    B, H, N_q, d = q.shape
    H_kv, N_kv = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if o is None:
        o = torch.empty((B, H, N_q, d), dtype=torch.float32, device=q.device)
    if o.dtype != torch.float32 or tuple(o.shape) != (B, H, N_q, d) or not o.is_contiguous():
        raise ValueError("o must be a contiguous float32 [B, H, N_q, d] tensor")
    if lse is None:
        lse = torch.empty((B, H, N_q), dtype=torch.float32, device=q.device)
    need = fa_fwd_kv_f32_workspace_bytes(B, H, H_kv, N_q, N_kv, d, num_splits)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    lib = load_library()
    with torch.cuda.device(q.device):
        st = lib.fa_fwd_kv_f32(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, H_kv,
                               N_q, N_kv, d, float(scale), int(num_splits), ws_ptr, ws_bytes,
                               _stream_handle(stream, q.device))
    if st != FA_OK:
        raise FaError(st, "fa_fwd_kv_f32")
    return o, lse


def fa_fwd_kv_fault_test(q, k, v, o, lse, scale: float, num_splits: int, workspace, drop_load: int,
                         timeout_ns: int, stream=None) -> int:
    """Test hook of the C ABI (see include/fa.h): returns the raw status code."""
    _check_kv(q, k, v)
    B, H, N_q, d = q.shape
    lib = load_library()
    with torch.cuda.device(q.device):
        return int(lib.fa_fwd_kv_fault_test(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, k.shape[1], N_q, k.shape[2],
            d, float(scale), int(num_splits), workspace.data_ptr() if workspace is not None else None,
            workspace.numel() * workspace.element_size() if workspace is not None else 0, int(drop_load),
            int(timeout_ns), _stream_handle(stream, q.device)))


def fa_merge_partials(o_parts: torch.Tensor, lse_parts: torch.Tensor, o=None, lse=None, stream=None):
    """Merge partial results over disjoint key sets (see include/fa.h).

    o_parts: float32 CUDA [P, ..., d]; lse_parts: float32 CUDA [P, ...] with the
    same leading shape. Returns (o bf16 [..., d], lse float32 [...]).
    """
    for name, t in (("o_parts", o_parts), ("lse_parts", lse_parts)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.float32 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 CUDA tensor")
    if o_parts.shape[:-1] != lse_parts.shape or o_parts.dim() < 3:
        raise ValueError(f"shapes do not match: {tuple(o_parts.shape)} vs {tuple(lse_parts.shape)}")
    P, d = o_parts.shape[0], o_parts.shape[-1]
    out_shape = tuple(o_parts.shape[1:])
    rows = int(lse_parts[0].numel())
    if o is None:
        o = torch.empty(out_shape, dtype=torch.bfloat16, device=o_parts.device)
    if lse is None:
        lse = torch.empty(out_shape[:-1], dtype=torch.float32, device=o_parts.device)
    lib = load_library()
    with torch.cuda.device(o_parts.device):
        st = lib.fa_merge_partials(o_parts.data_ptr(), lse_parts.data_ptr(), o.data_ptr(), lse.data_ptr(), int(P), rows,
                                   int(d), _stream_handle(stream, o_parts.device))
    if st != FA_OK:
        raise FaError(st, "fa_merge_partials")
    return o, lse


def fa_bwd_workspace_bytes(B: int, H: int, N: int) -> int:
    return int(load_library().fa_bwd_workspace_bytes(int(B), int(H), int(N)))


def fa_bwd(q, k, v, o, do, lse, dq=None, dk=None, dv=None, scale: float | None = None, workspace=None,
           stream=None):
    """Gradients (dq, dk, dv) of <do, o> for o = softmax(scale * q k^T) v, with
    the probabilities rebuilt from the forward's ``lse`` and ``o``.

    q, k, v, o, do: bf16 CUDA tensors [B, H, N, d], contiguous; lse: float32
    [B, H, N]. Outputs (bf16, shaped like q) and the workspace (at least
    fa_bwd_workspace_bytes(B, H, N) bytes) are allocated with torch when not
    given. ``scale`` defaults to 1/sqrt(d). Returns (dq, dk, dv).
    """
    _check_qkv(q, k, v)
    B, H, N, d = q.shape
    for name, t in (("o", o), ("do", do)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or t.shape != q.shape \
                or not t.is_contiguous() or t.device != q.device:
            raise ValueError(f"{name} must be a contiguous bf16 tensor shaped like q on q's device")
    if not isinstance(lse, torch.Tensor) or lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N) \
            or not lse.is_contiguous() or lse.device != q.device:
        raise ValueError("lse must be a contiguous float32 [B, H, N] tensor on q's device")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    outs = []
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        if t is None:
            t = torch.empty_like(q)
        elif t.dtype != torch.bfloat16 or t.shape != q.shape or not t.is_contiguous() or t.device != q.device:
            raise ValueError(f"{name} must be a contiguous bf16 tensor shaped like q on q's device")
        outs.append(t)
    need = fa_bwd_workspace_bytes(B, H, N)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    lib = load_library()
    with torch.cuda.device(q.device):
        st = lib.fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(),
                        outs[0].data_ptr(), outs[1].data_ptr(), outs[2].data_ptr(), B, H, N, d, float(scale),
                        workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                        _stream_handle(stream, q.device))
    if st != FA_OK:
        raise FaError(st, "fa_bwd")
    return tuple(outs)


def _bf16(name, t, device, shape):
    """Checks a bf16 tensor of this shape on this device whose last dimension is
    contiguous; whether it is contiguous as a whole."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or t.shape != shape or t.device != device:
        raise ValueError(f"{name} must be a bf16 tensor of shape {tuple(shape)} on {device}")
    if t.is_contiguous():
        return True
    if t.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return False


#: arrays of strides for the C ABI by the tensors' strides, and workspace sizes
#: by (function, device, sizes); small calls are bound by the host
_strides_of: dict = {}
_need_of: dict = {}


def _strides(dense, *tensors):
    """The C ABI's array of strides, or None (all contiguous). None among the
    tensors: a prefix that is not there; a prefix has no batch stride."""
    if dense:
        return None
    key = tuple([None if t is None else t.stride() for t in tensors])
    array = _strides_of.get(key)
    if array is None:
        flat = []
        for st in key:
            if st is None:
                flat += (0, 0, 0)
            else:
                if len(st) == 3 and len(key[0]) == 4:
                    flat.append(0)
                flat += st[:-1]
        if len(_strides_of) > 4096:
            _strides_of.clear()
        array = _strides_of[key] = (ctypes.c_longlong * len(flat))(*flat)
    return array


def _leading(name, t, dims):
    """Shape of a CUDA tensor that others are checked against."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != dims:
        raise ValueError(f"{name} must be a CUDA tensor of {dims} dimensions")
    return t.shape


def _int32(name, t, device, n):
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or t.shape != (n,) or t.device != device \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor [{n}] on {device}")


def _out_lse(lse, shape, device):
    if lse is None:
        return torch.empty(shape, dtype=torch.float32, device=device)
    if not isinstance(lse, torch.Tensor) or lse.dtype is not torch.float32 or lse.shape != shape \
            or lse.device != device or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 tensor {list(shape)} on {device}")
    return lse


def _out_bf16(name, t, device, shape, like=None):
    """(tensor, whether it is contiguous) of an output, allocated when not given
    (like a contiguous tensor of its shape, which is quicker)."""
    if t is None:
        if like is not None and like.is_contiguous():
            return torch.empty_like(like), True
        return torch.empty(shape, dtype=torch.bfloat16, device=device), True
    return t, _bf16(name, t, device, shape)


def _need(name, device, *sizes):
    key = (name, device.index, *sizes)
    need = _need_of.get(key)
    if need is None:
        if len(_need_of) > 4096:
            _need_of.clear()
        need = _need_of[key] = getattr(load_library(), name)(*sizes)
    return need


def _workspace(workspace, need, device):
    """(tensor, pointer, bytes) of the caller's workspace, or of a new one if any is needed."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        return workspace, workspace.data_ptr(), need
    if not isinstance(workspace, torch.Tensor) or workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _raw_stream(device) -> int:
    """Handle of torch's current stream of a device."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _packed_sizes(q, k, cu_q):
    """(device, T_q, H, T_kv, H_kv, d, B) of packed tensors, from q, k and cu_q."""
    T_q, H, d = _leading("q", q, 3)
    T_kv, H_kv, _ = _leading("k", k, 3)
    if not isinstance(cu_q, torch.Tensor) or cu_q.dim() != 1 or cu_q.shape[0] < 2:
        raise ValueError("cu_q must hold B + 1 offsets")
    return q.device, T_q, H, T_kv, H_kv, d, cu_q.shape[0] - 1


def fa_fwd_varlen_workspace_bytes(B: int, H: int, H_kv: int, T_q: int, T_kv: int, d: int) -> int:
    return int(load_library().fa_fwd_varlen_workspace_bytes(int(B), int(H), int(H_kv), int(T_q), int(T_kv), int(d)))


def fa_fwd_varlen(q, k, v, cu_q, cu_kv, o=None, lse=None, scale: float | None = None, causal: bool = True,
                  workspace=None, stream=None):
    """Attention over packed sequences of different lengths with shared K/V heads.

    q: bf16 [T_q, H, d]; k, v: bf16 [T_kv, H_kv, d], H a multiple of H_kv. Only
    d has to be contiguous: slices of one projection's output need no copy.
    cu_q, cu_kv: int32 CUDA [B + 1]; sequence b has the query rows
    [cu_q[b], cu_q[b+1]) and the keys [cu_kv[b], cu_kv[b+1]). With ``causal`` row
    i of a sequence sees its keys j <= i + n_kv - n_q, else all of them; a row
    that sees none gets o = 0 and lse = -inf. Rows of no sequence are not written.
    The offsets stay on the device; with ones outside the buffers nothing is
    written and :func:`fa_get_device_status` says so. Returns (o bf16 [T_q, H, d], lse float32 [H, T_q]).
    """
    device, T_q, H, T_kv, H_kv, d, B = _packed_sizes(q, k, cu_q)
    rows, keys = (T_q, H, d), (T_kv, H_kv, d)
    dense = _bf16("q", q, device, rows) & _bf16("k", k, device, keys) & _bf16("v", v, device, keys)
    _int32("cu_q", cu_q, device, B + 1)
    _int32("cu_kv", cu_kv, device, B + 1)

    def run():
        out, out_dense = _out_bf16("o", o, device, rows, q)
        out_lse = _out_lse(lse, (H, T_q), device)
        need = _need("fa_fwd_varlen_workspace_bytes", device, B, H, H_kv, T_q, T_kv, d)
        ws, ws_ptr, ws_bytes = _workspace(workspace, need, device)
        st = load_library().fa_fwd_varlen(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), out_lse.data_ptr(), cu_q.data_ptr(),
            cu_kv.data_ptr(), B, H, H_kv, T_q, T_kv, d, _strides(dense and out_dense, q, k, v, out),
            d ** -0.5 if scale is None else float(scale), bool(causal), ws_ptr, ws_bytes, _raw_stream(device))
        if st != FA_OK:
            raise FaError(st, "fa_fwd_varlen")
        return out, out_lse

    return _launch(run, stream, device)


def fa_fwd_varlen_fault_test(q, k, v, o, lse, cu_q, cu_kv, scale: float, causal: bool, workspace, drop_load: int,
                             timeout_ns: int, stream=None) -> int:
    """Test hook of the C ABI (see include/fa.h): returns the raw status code."""
    T_q, H, d = q.shape
    lib = load_library()
    with torch.cuda.device(q.device):
        return int(lib.fa_fwd_varlen_fault_test(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), cu_q.data_ptr(), cu_kv.data_ptr(),
            cu_q.shape[0] - 1, H, k.shape[1], T_q, k.shape[0], d, float(scale), bool(causal), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), int(drop_load), int(timeout_ns),
            _stream_handle(stream, q.device)))


def fa_bwd_varlen_workspace_bytes(B: int, H: int, H_kv: int, T_q: int, T_kv: int) -> int:
    return int(load_library().fa_bwd_varlen_workspace_bytes(int(B), int(H), int(H_kv), int(T_q), int(T_kv)))


def fa_bwd_varlen(q, k, v, o, do, lse, cu_q, cu_kv, dq=None, dk=None, dv=None, scale: float | None = None,
                  causal: bool = True, workspace=None, stream=None):
    """Gradients (dq, dk, dv) of <do, o> for :func:`fa_fwd_varlen`'s ``o``, from
    its outputs ``o`` and ``lse``. do, dq: bf16 [T_q, H, d]; dk, dv: bf16
    [T_kv, H_kv, d], summed over the query heads of a K/V head. Other arguments
    as for the forward. Rows and keys of no sequence are not written."""
    device, T_q, H, T_kv, H_kv, d, B = _packed_sizes(q, k, cu_q)
    rows, keys = (T_q, H, d), (T_kv, H_kv, d)
    dense = (_bf16("q", q, device, rows) & _bf16("k", k, device, keys) & _bf16("v", v, device, keys)
             & _bf16("o", o, device, rows) & _bf16("do", do, device, rows))
    if not isinstance(lse, torch.Tensor):
        raise ValueError("lse must be a tensor")
    _out_lse(lse, (H, T_q), device)
    _int32("cu_q", cu_q, device, B + 1)
    _int32("cu_kv", cu_kv, device, B + 1)

    def run():
        gq, q_dense = _out_bf16("dq", dq, device, rows, o)
        gk, k_dense = _out_bf16("dk", dk, device, keys, k)
        gv, v_dense = _out_bf16("dv", dv, device, keys, v)
        need = _need("fa_bwd_varlen_workspace_bytes", device, B, H, H_kv, T_q, T_kv)
        ws, ws_ptr, ws_bytes = _workspace(workspace, need, device)
        st = load_library().fa_bwd_varlen(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(), gq.data_ptr(),
            gk.data_ptr(), gv.data_ptr(), cu_q.data_ptr(), cu_kv.data_ptr(), B, H, H_kv, T_q, T_kv, d,
            _strides(dense and q_dense and k_dense and v_dense, q, k, v, o, do, gq, gk, gv),
            d ** -0.5 if scale is None else float(scale), bool(causal), ws_ptr, ws_bytes, _raw_stream(device))
        if st != FA_OK:
            raise FaError(st, "fa_bwd_varlen")
        return gq, gk, gv

    return _launch(run, stream, device)


def fa_bwd_varlen_fault_test(q, k, v, o, do, lse, cu_q, cu_kv, dq, dk, dv, scale: float, causal: bool, workspace,
                             drop_load: int, timeout_ns: int, stream=None) -> int:
    """Test hook of the C ABI (see include/fa.h): returns the raw status code."""
    T_q, H, d = q.shape
    lib = load_library()
    with torch.cuda.device(q.device):
        return int(lib.fa_bwd_varlen_fault_test(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(), dq.data_ptr(),
            dk.data_ptr(), dv.data_ptr(), cu_q.data_ptr(), cu_kv.data_ptr(), cu_q.shape[0] - 1, H, k.shape[1], T_q,
            k.shape[0], d, float(scale), bool(causal), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), int(drop_load), int(timeout_ns),
            _stream_handle(stream, q.device)))


def fa_fwd_prefix_workspace_bytes(B: int, H: int, H_kv: int, N_q: int, N_prefix: int, N_own: int, d: int) -> int:
    return int(load_library().fa_fwd_prefix_workspace_bytes(int(B), int(H), int(H_kv), int(N_q), int(N_prefix),
                                                             int(N_own), int(d)))


def fa_fwd_prefix(q, k_prefix, v_prefix, k, v, seq_lens, o=None, lse=None, scale: float | None = None,
                  causal: bool = False, workspace=None, stream=None):
    """Attention of a few new tokens per sequence over a prefix that the batch
    shares and each sequence's own cache.

    q: bf16 [B, H, N_q, d], N_q <= 128; k_prefix, v_prefix: bf16
    [H_kv, N_prefix, d], or None when nothing is shared; k, v: bf16
    [B, H_kv, N_own, d], of which the first seq_lens[b] rows count (int32 CUDA
    [B], read on the device). Only d has to be contiguous. With ``causal`` the
    N_q new tokens are the last of the own cache and row i sees its keys
    j < seq_lens[b] - (N_q - 1 - i). A row that sees no key gets o = 0 and
    lse = -inf. Returns (o bf16 [B, H, N_q, d], lse float32 [B, H, N_q]).
    """
    rows = _leading("q", q, 4)
    B, H, N_q, d = rows
    _, H_kv, N_own, _ = _leading("k", k, 4)
    device, cache = q.device, (B, H_kv, N_own, d)
    dense = _bf16("q", q, device, rows) & _bf16("k", k, device, cache) & _bf16("v", v, device, cache)
    if (k_prefix is None) != (v_prefix is None):
        raise ValueError("k_prefix and v_prefix come together")
    N_prefix, p_ptr = 0, (None, None)
    if k_prefix is not None:
        N_prefix = _leading("k_prefix", k_prefix, 3)[1]
        shared = (H_kv, N_prefix, d)
        dense &= _bf16("k_prefix", k_prefix, device, shared) & _bf16("v_prefix", v_prefix, device, shared)
        p_ptr = k_prefix.data_ptr(), v_prefix.data_ptr()
    _int32("seq_lens", seq_lens, device, B)

    def run():
        out, out_dense = _out_bf16("o", o, device, rows, q)
        out_lse = _out_lse(lse, (B, H, N_q), device)
        need = _need("fa_fwd_prefix_workspace_bytes", device, B, H, H_kv, N_q, N_prefix, N_own, d)
        ws, ws_ptr, ws_bytes = _workspace(workspace, need, device)
        st = load_library().fa_fwd_prefix(
            q.data_ptr(), *p_ptr, k.data_ptr(), v.data_ptr(), seq_lens.data_ptr(), out.data_ptr(), out_lse.data_ptr(),
            B, H, H_kv, N_q, N_prefix, N_own, d, _strides(dense and out_dense, q, k_prefix, v_prefix, k, v, out),
            d ** -0.5 if scale is None else float(scale), bool(causal), ws_ptr, ws_bytes, _raw_stream(device))
        if st != FA_OK:
            raise FaError(st, "fa_fwd_prefix")
        return out, out_lse

    return _launch(run, stream, device)


def fa_fwd_prefix_fault_test(q, k_prefix, v_prefix, k, v, seq_lens, o, lse, scale: float, causal: bool, workspace,
                             drop_load: int, timeout_ns: int, stream=None) -> int:
    """Test hook of the C ABI (see include/fa.h): returns the raw status code."""
    B, H, N_q, d = q.shape
    lib = load_library()
    with torch.cuda.device(q.device):
        return int(lib.fa_fwd_prefix_fault_test(
            q.data_ptr(), k_prefix.data_ptr(), v_prefix.data_ptr(), k.data_ptr(), v.data_ptr(), seq_lens.data_ptr(),
            o.data_ptr(), lse.data_ptr(), B, H, k.shape[1], N_q, k_prefix.shape[1], k.shape[2], d, float(scale),
            bool(causal), workspace.data_ptr(), workspace.numel() * workspace.element_size(), int(drop_load),
            int(timeout_ns), _stream_handle(stream, q.device)))


#: how fa_rope_frequencies slows frequencies down for long contexts
_RAMPS = {None: 0, "linear": 0, "turns": 1, "log_turns": 2}


def fa_rope_frequencies(rot: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                        low_turns: float = 1.0, high_turns: float = 32.0, original: float = 4096.0, device=None):
    """Radians per position of the rot / 2 pairs of a rotated head, float64, for
    :func:`fa_rope` and :func:`fa_kv_append`: base^(-2 j / rot), and for contexts
    longer than ``original``

    "linear": every frequency divided by ``factor``;
    "turns", "log_turns": a pair that turns ``high_turns`` times or more over the
    original context keeps its frequency, one that turns ``low_turns`` times or less
    has it divided by ``factor``, and between them both are mixed by where its
    turns (their logarithm) lie. (The limits are not moved to whole pairs.)
    """
    if scaling not in _RAMPS:
        raise ValueError(f"scaling must be one of {[k for k in _RAMPS]}")
    out = torch.empty(max(0, int(rot)) // 2, dtype=torch.float64)
    st = load_library().fa_rope_frequencies(out.data_ptr(), int(rot), float(base), _RAMPS[scaling],
                                            float(factor) if scaling else 1.0, float(low_turns), float(high_turns),
                                            float(original))
    if st != FA_OK:
        raise FaError(st, "fa_rope_frequencies")
    return out if device is None else out.to(device)


def _frequencies(inv_freq, device):
    """Columns that these frequencies rotate."""
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dtype is not torch.float64 or inv_freq.dim() != 1 \
            or inv_freq.device != device or not inv_freq.is_contiguous():
        raise ValueError(f"inv_freq must be a contiguous float64 tensor [rot / 2] on {device}")
    return 2 * inv_freq.shape[0]


def fa_rope(x, positions, inv_freq, y=None, out=None, out_y=None, interleaved: bool = False, transpose: bool = False,
            factor: float = 1.0, stream=None):
    """Rotary positions of x (and y, as queries and keys) in one launch, or the
    gradient of that.

    x: bf16 [T, heads, d], y: bf16 [T, heads_y, d] or None; only d has to be
    contiguous. positions: int32 [T]; inv_freq: float64 [rot / 2], radians per
    position (:func:`fa_rope_frequencies`). Pairs are the columns j and
    j + rot / 2, or with ``interleaved`` 2 j and 2 j + 1; columns from rot on are
    copied. ``factor`` multiplies cos and sin. With ``transpose`` the transposed
    rotation: given the gradient of the outputs it returns that of the inputs.
    out, out_y: where the results go, x and y themselves for a rotation in place.
    Returns out, or (out, out_y) with y.
    """
    T, heads, d = rows = _leading("x", x, 3)
    device = x.device
    dense = _bf16("x", x, device, rows)
    heads_y, rows_y, y_ptr = 0, None, None
    if y is not None:
        heads_y = _leading("y", y, 3)[1]
        rows_y = (T, heads_y, d)
        dense &= _bf16("y", y, device, rows_y)
        y_ptr = y.data_ptr()
    elif out_y is not None:
        raise ValueError("out_y comes with y")
    _int32("positions", positions, device, T)
    rot = _frequencies(inv_freq, device)

    def run():
        o, all_dense = _out_bf16("out", out, device, rows, x)
        all_dense &= dense
        oy = oy_ptr = None
        if y is not None:
            oy, oy_dense = _out_bf16("out_y", out_y, device, rows_y, y)
            all_dense &= oy_dense
            oy_ptr = oy.data_ptr()
        strides = None
        if not all_dense:
            strides = _strides(False, x, o) if y is None else _strides(False, x, o, y, oy)
        st = (_lib or load_library()).fa_rope(
            x.data_ptr(), o.data_ptr(), heads, y_ptr, oy_ptr, heads_y, positions.data_ptr(), inv_freq.data_ptr(), T, d,
            rot, strides, bool(interleaved), bool(transpose), float(factor), _raw_stream(device))
        if st != FA_OK:
            raise FaError(st, "fa_rope")
        return o if y is None else (o, oy)

    return _launch(run, stream, device)


def _pages(name, t, device, shape):
    """As _bf16, for a cache in pages of 8 bits."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.float8_e4m3fn or t.shape != shape or t.device != device:
        raise ValueError(f"{name} must be a float8_e4m3fn tensor of shape {tuple(shape)} on {device}")
    if t.is_contiguous():
        return True
    if t.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return False


def _cache(k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, device, B):
    """(pages' shape, entries of a sequence in the table, whether the pages are contiguous)."""
    shape = _leading("k_cache", k_cache, 4)
    dense = _pages("k_cache", k_cache, device, shape) & _pages("v_cache", v_cache, device, shape)
    scales = shape[:2]
    for t in (k_scale, v_scale):
        if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32 or t.shape != scales or t.device != device \
                or not t.is_contiguous():
            raise ValueError(f"k_scale and v_scale must be contiguous float32 tensors {list(scales)} on {device}")
    if not isinstance(page_table, torch.Tensor) or page_table.dtype is not torch.int32 or page_table.dim() != 2 \
            or page_table.device != device or not page_table.is_contiguous():
        raise ValueError(f"page_table must be a contiguous int32 tensor [{B}, max_pages] on {device}")
    sequences, max_pages = page_table.shape
    if sequences != B:
        raise ValueError(f"page_table must have a row for each of {B} sequences")
    _int32("seq_lens", seq_lens, device, B)
    return shape, max_pages, dense


def _sequences(name, cu, device):
    """Number of sequences that these offsets separate."""
    if not isinstance(cu, torch.Tensor) or cu.dtype is not torch.int32 or cu.dim() != 1 or cu.device != device \
            or not cu.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor [B + 1] on {device}")
    n = len(cu) - 1
    if n < 1:
        raise ValueError(f"{name} must hold B + 1 offsets")
    return n


def fa_kv_append(k, v, cu_new, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, q=None, q_out=None,
                 inv_freq=None, positions=None, interleaved: bool = False, factor: float = 1.0, stream=None):
    """New keys and values into the pages of an 8-bit cache, the keys rotated to
    their positions on the way, and the queries beside them; one launch.

    k, v: bf16 [T, H_kv, d], packed: sequence b has the rows [cu_new[b],
    cu_new[b+1]) (int32 CUDA [B + 1]), the last ones of its seq_lens[b] (int32 [B],
    with the new tokens). k_cache, v_cache: float8_e4m3fn [num_pages, H_kv,
    page_size, d]; k_scale, v_scale: float32 [num_pages, H_kv], the scale of each
    page and head; page_table: int32 [B, max_pages]. All four are updated in place.
    Only d has to be contiguous in q, k, v and the pages. q: bf16 [T, H, d],
    rotated into q_out (q itself for a rotation in place). inv_freq, interleaved,
    factor: as for :func:`fa_rope`; without inv_freq nothing is rotated.
    positions: int32 [T], else a token's place in its sequence. See include/fa.h
    for how scales are chosen. Lengths, offsets and pages that do not fit are left out and
    reported by :func:`fa_get_device_status`. Returns the rotated q (q itself
    without inv_freq), or None without q.
    """
    T, H_kv, d = rows = _leading("k", k, 3)
    device = k.device
    dense = _bf16("k", k, device, rows) & _bf16("v", v, device, rows)
    B = _sequences("cu_new", cu_new, device)
    (num_pages, heads, page, d_cache), max_pages, dense_cache = _cache(k_cache, v_cache, k_scale, v_scale, page_table,
                                                                       seq_lens, device, B)
    if heads != H_kv or d_cache != d:
        raise ValueError(f"the cache holds {heads} heads of {d_cache}, k has {H_kv} of {d}")
    rot = 0 if inv_freq is None else _frequencies(inv_freq, device)
    if positions is not None:
        _int32("positions", positions, device, T)
    H, rows_q = 0, None
    if q is not None:
        H = _leading("q", q, 3)[1]
        rows_q = (T, H, d)
        dense &= _bf16("q", q, device, rows_q)
    if q_out is not None and (q is None or not rot):
        raise ValueError("q_out comes with q and inv_freq")
    turn = q is not None and rot > 0

    def run():
        o = q_ptr = o_ptr = None
        all_dense = dense
        if turn:
            o, o_dense = _out_bf16("q_out", q_out, device, rows_q, q)
            all_dense &= o_dense
            q_ptr, o_ptr = q.data_ptr(), o.data_ptr()
        strides = None
        if not all_dense:
            strides = _strides(False, k, v, q, o) if turn else _strides(False, k, v)
        st = (_lib or load_library()).fa_kv_append(
            k.data_ptr(), v.data_ptr(), cu_new.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
            v_scale.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(), q_ptr, o_ptr,
            inv_freq.data_ptr() if rot else None, None if positions is None else positions.data_ptr(), B, H, H_kv, T, d,
            num_pages, page, max_pages, rot, strides, None if dense_cache else _strides(False, k_cache, v_cache),
            bool(interleaved), float(factor), _raw_stream(device))
        if st != FA_OK:
            raise FaError(st, "fa_kv_append")
        return o if turn else q

    return _launch(run, stream, device)


def fa_fwd_paged_workspace_bytes(B: int, H: int, H_kv: int, T_q: int, d: int, num_pages: int, page_size: int,
                                 max_pages: int) -> int:
    return int(load_library().fa_fwd_paged_workspace_bytes(int(B), int(H), int(H_kv), int(T_q), int(d), int(num_pages),
                                                           int(page_size), int(max_pages)))


def fa_fwd_paged(q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, cu_q, o=None, lse=None,
                 scale: float | None = None, causal: bool = True, workspace=None, stream=None):
    """Attention of new tokens over a paged 8-bit cache that holds their keys too
    (:func:`fa_kv_append`): single tokens, drafted tokens and pieces of prompts in
    any mixture.

    q: bf16 [T_q, H, d], packed by cu_q (int32 CUDA [B + 1]). k_cache, v_cache:
    float8_e4m3fn [num_pages, H_kv, page_size, d], H a multiple of H_kv; k_scale,
    v_scale: float32 [num_pages, H_kv]; page_table: int32 [B, max_pages];
    seq_lens: int32 [B]. Only d has to be contiguous in q and the pages. With
    ``causal`` row i of n_q sees the keys j <= i + seq_lens[b] - n_q, else all
    seq_lens[b]; a row that sees none gets o = 0 and lse = -inf. Rows of no
    sequence are not written. A long piece of a prompt among many single tokens is
    better off in a call of its own (see include/fa.h). Returns (o bf16 [T_q, H, d], lse float32 [H, T_q]).
    """
    T_q, H, d = rows = _leading("q", q, 3)
    device = q.device
    dense = _bf16("q", q, device, rows)
    B = _sequences("cu_q", cu_q, device)
    (num_pages, H_kv, page, d_cache), max_pages, dense_cache = _cache(k_cache, v_cache, k_scale, v_scale, page_table,
                                                                      seq_lens, device, B)
    if d_cache != d:
        raise ValueError(f"the cache holds heads of {d_cache}, q of {d}")

    def run():
        out, out_dense = _out_bf16("o", o, device, rows, q)
        out_lse = _out_lse(lse, (H, T_q), device)
        need = _need("fa_fwd_paged_workspace_bytes", device, B, H, H_kv, T_q, d, num_pages, page, max_pages)
        ws, ws_ptr, ws_bytes = _workspace(workspace, need, device)
        st = (_lib or load_library()).fa_fwd_paged(
            q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
            page_table.data_ptr(), seq_lens.data_ptr(), cu_q.data_ptr(), out.data_ptr(), out_lse.data_ptr(), B, H,
            H_kv, T_q, d, num_pages, page, max_pages, None if dense and out_dense else _strides(False, q, out),
            None if dense_cache else _strides(False, k_cache, v_cache), d ** -0.5 if scale is None else float(scale),
            bool(causal), ws_ptr, ws_bytes, _raw_stream(device))
        if st != FA_OK:
            raise FaError(st, "fa_fwd_paged")
        return out, out_lse

    return _launch(run, stream, device)


def fa_fwd_paged_fault_test(q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, cu_q, o, lse, scale: float,
                            causal: bool, workspace, drop_load: int, timeout_ns: int, stream=None) -> int:
    """Test hook of the C ABI (see include/fa.h): returns the raw status code."""
    T_q, H, d = q.shape
    num_pages, H_kv, page, _ = k_cache.shape
    lib = load_library()
    with torch.cuda.device(q.device):
        return int(lib.fa_fwd_paged_fault_test(
            q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
            page_table.data_ptr(), seq_lens.data_ptr(), cu_q.data_ptr(), o.data_ptr(), lse.data_ptr(),
            cu_q.shape[0] - 1, H, H_kv, T_q, d, num_pages, page, page_table.shape[1], float(scale), bool(causal),
            workspace.data_ptr(), workspace.numel() * workspace.element_size(), int(drop_load), int(timeout_ns),
            _stream_handle(stream, q.device)))


def fa_bwd_fault_test(q, k, v, o, do, lse, dq, dk, dv, scale: float, workspace, drop_load: int, timeout_ns: int,
                      stream=None) -> int:
    """Test hook of the C ABI (see include/fa.h): returns the raw status code."""
    _check_qkv(q, k, v)
    B, H, N, d = q.shape
    lib = load_library()
    with torch.cuda.device(q.device):
        return int(lib.fa_bwd_fault_test(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(),
                                         lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, N, d,
                                         float(scale), workspace.data_ptr(),
                                         workspace.numel() * workspace.element_size(), int(drop_load),
                                         int(timeout_ns), _stream_handle(stream, q.device)))


def fa_fwd_fault_test(q, k, v, o, lse, scale: float, drop_load: int, timeout_ns: int, stream=None) -> int:
    """Test hook of the C ABI (see include/fa.h): returns the raw status code."""
    _check_qkv(q, k, v)
    B, H, N, d = q.shape
    lib = load_library()
    with torch.cuda.device(q.device):
        return int(lib.fa_fwd_fault_test(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                         B, H, N, d, float(scale), int(drop_load), int(timeout_ns),
                                         _stream_handle(stream, q.device)))


def fa_get_device_status(stream=None, device=None):
    """Synchronise the stream and read/clear the device status word: (status, info[4])."""
    lib = load_library()
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    info = (ctypes.c_uint * 4)()
    with torch.cuda.device(device):
        st = lib.fa_get_device_status(_stream_handle(stream, device), info)
    return int(st), [int(x) for x in info]
