"""Thin Python binding of libkdt.so (ctypes). Argument marshalling only.

Every computation runs in the library's CUDA kernels; this module passes device
pointers (``tensor.data_ptr()``) and the current CUDA stream, and allocates
output and workspace tensors with torch when the caller does not pass them.
Functions that take ``stream`` run on that torch stream instead, which must have
waited for the current one; what they allocate is recorded on it.
There is no CPU fallback: if libkdt.so is missing, importing the library raises.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libkdt.so")

(KDT_OK, KDT_ERR_NULL_ARG, KDT_ERR_BAD_SHAPE, KDT_ERR_UNSUPPORTED, KDT_ERR_WORKSPACE, KDT_ERR_CUDA,
 KDT_ERR_NOT_DEVICE) = range(7)
KDT_F32, KDT_BF16 = 0, 1
IMPLS = {"auto": 0, "simt": 1, "tcgen05": 2, "simt_small": 3, "q8_rows": 4}
IMPL_NAMES = {v: k for k, v in IMPLS.items()}
DEFAULT_SCALE = 1.0 / math.sqrt(192.0)

# Names the header declares (checked by the CPU test suite against include/kdt.h).
EXPORTS = ("kdt_status_str", "kdt_version", "kdt_build_visibility", "kdt_verify_attn",
           "kdt_verify_attn_workspace_size", "kdt_verify_attn_plan", "kdt_merge_attn_states",
           "kdt_verify_attn_noalloc", "kdt_rope_neox", "kdt_tree_accept", "kdt_kv_compact", "kdt_tree_build",
           "kdt_verify_attn_host", "kdt_verify_attn_host_buffer_size", "kdt_vc_up_proj",
           "kdt_test_verify_attn_wait_expiry", "kdt_latent_write_q8", "kdt_latent_read_q8", "kdt_kv_compact_q8",
           "kdt_verify_attn_q8", "kdt_verify_attn_q8_workspace_size", "kdt_verify_attn_q8_plan",
           "kdt_tree_sample", "kdt_page_assign", "kdt_latent_write_paged", "kdt_kv_compact_paged",
           "kdt_verify_attn_paged", "kdt_verify_attn_paged_workspace_size", "kdt_verify_attn_paged_plan",
           "kdt_sample")


class KdtError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_str(status)} (status {status})")


class VerifyArgs(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
        ("D_c", ctypes.c_int), ("D_r", ctypes.c_int), ("dtype", ctypes.c_int),
        ("q_nope", ctypes.c_void_p), ("q_pe", ctypes.c_void_p),
        ("c_kv", ctypes.c_void_p), ("k_pe", ctypes.c_void_p),
        ("kv_row_stride", ctypes.c_int64),
        ("prefix_len", ctypes.c_void_p),
        ("max_kv_len", ctypes.c_int),
        ("parent", ctypes.c_void_p), ("vis", ctypes.c_void_p),
        ("scale", ctypes.c_float),
        ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("err", ctypes.c_void_p),
        ("impl", ctypes.c_int), ("num_splits", ctypes.c_int),
        ("q_nope_row_stride", ctypes.c_int64), ("q_pe_row_stride", ctypes.c_int64),
    ]


class RopeArgs(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int), ("D_r", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("q", ctypes.c_void_p), ("q_row_stride", ctypes.c_int64),
        ("k_pe", ctypes.c_void_p), ("kv_row_stride", ctypes.c_int64),
        ("prefix_len", ctypes.c_void_p), ("pos", ctypes.c_void_p),
        ("base", ctypes.c_double),
    ]


class LatentWriteArgs(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int), ("T", ctypes.c_int), ("D_c", ctypes.c_int), ("D_r", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("c", ctypes.c_void_p), ("c_row_stride", ctypes.c_int64),
        ("k", ctypes.c_void_p), ("k_row_stride", ctypes.c_int64),
        ("gamma", ctypes.c_void_p), ("eps", ctypes.c_float),
        ("pos", ctypes.c_void_p), ("base", ctypes.c_double),
        ("prefix_len", ctypes.c_void_p), ("n_rows", ctypes.c_void_p),
        ("c_q8", ctypes.c_void_p), ("c_scale", ctypes.c_void_p), ("k_pe", ctypes.c_void_p),
        ("kv_row_stride", ctypes.c_int64),
    ]


class VerifyQ8Args(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int), ("D_c", ctypes.c_int), ("D_r", ctypes.c_int),
        ("q_nope", ctypes.c_void_p), ("q_nope_row_stride", ctypes.c_int64),
        ("q_pe", ctypes.c_void_p), ("q_pe_row_stride", ctypes.c_int64),
        ("c_q8", ctypes.c_void_p), ("c_scale", ctypes.c_void_p), ("k_pe", ctypes.c_void_p),
        ("kv_row_stride", ctypes.c_int64),
        ("prefix_len", ctypes.c_void_p), ("max_kv_len", ctypes.c_int),
        ("parent", ctypes.c_void_p), ("vis", ctypes.c_void_p),
        ("scale", ctypes.c_float),
        ("out", ctypes.c_void_p), ("out_dtype", ctypes.c_int), ("lse", ctypes.c_void_p), ("err", ctypes.c_void_p),
        ("impl", ctypes.c_int), ("num_splits", ctypes.c_int),
    ]


class PageArgs(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int), ("W", ctypes.c_int),
        ("table", ctypes.c_void_p), ("table_row_stride", ctypes.c_int64),
        ("held", ctypes.c_void_p), ("free_pages", ctypes.c_void_p), ("n_free", ctypes.c_void_p),
        ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int),
        ("new_len", ctypes.c_void_p), ("start", ctypes.c_void_p), ("T", ctypes.c_int),
        ("slots", ctypes.c_void_p), ("err", ctypes.c_void_p),
    ]


class LatentWritePagedArgs(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int), ("D_c", ctypes.c_int), ("D_r", ctypes.c_int), ("dtype", ctypes.c_int),
        ("c", ctypes.c_void_p), ("c_row_stride", ctypes.c_int64),
        ("k", ctypes.c_void_p), ("k_row_stride", ctypes.c_int64),
        ("gamma", ctypes.c_void_p), ("eps", ctypes.c_float),
        ("pos", ctypes.c_void_p), ("base", ctypes.c_double),
        ("slots", ctypes.c_void_p), ("c_kv", ctypes.c_void_p), ("k_pe", ctypes.c_void_p), ("n_slots", ctypes.c_int),
    ]


class VerifyPagedArgs(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int), ("D_c", ctypes.c_int), ("D_r", ctypes.c_int),
        ("q_nope", ctypes.c_void_p), ("q_nope_row_stride", ctypes.c_int64),
        ("q_pe", ctypes.c_void_p), ("q_pe_row_stride", ctypes.c_int64),
        ("c_kv", ctypes.c_void_p), ("k_pe", ctypes.c_void_p),
        ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int),
        ("table", ctypes.c_void_p), ("table_width", ctypes.c_int), ("table_row_stride", ctypes.c_int64),
        ("prefix_len", ctypes.c_void_p), ("n_rows", ctypes.c_void_p), ("max_kv_len", ctypes.c_int),
        ("parent", ctypes.c_void_p), ("vis", ctypes.c_void_p),
        ("scale", ctypes.c_float),
        ("out", ctypes.c_void_p), ("out_dtype", ctypes.c_int), ("lse", ctypes.c_void_p), ("err", ctypes.c_void_p),
        ("num_splits", ctypes.c_int),
    ]


class SampleArgs(ctypes.Structure):
    _fields_ = [
        ("R", ctypes.c_int), ("V", ctypes.c_int),
        ("logits", ctypes.c_void_p), ("dtype", ctypes.c_int), ("row_stride", ctypes.c_int64),
        ("u", ctypes.c_void_p),
        ("temperature", ctypes.c_void_p), ("temperature_all", ctypes.c_double),
        ("top_k", ctypes.c_void_p), ("top_k_all", ctypes.c_int),
        ("top_p", ctypes.c_void_p), ("top_p_all", ctypes.c_double),
        ("min_p", ctypes.c_void_p), ("min_p_all", ctypes.c_double),
        ("token", ctypes.c_void_p), ("logp", ctypes.c_void_p), ("err", ctypes.c_void_p),
    ]


class Plan(ctypes.Structure):
    _fields_ = [("impl", ctypes.c_int), ("num_splits", ctypes.c_int), ("num_launches", ctypes.c_int),
                ("ctas", ctypes.c_int), ("workspace_bytes", ctypes.c_size_t)]


_lib = None


def lib():
    """The loaded libkdt.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libkdt.so not found at {LIB_PATH}: build it with "
                              "`python -m speculative_decoding_tree_absorb_gb300.build_lib` "
                              "(there is no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        vp = ctypes.c_void_p
        L.kdt_status_str.argtypes = [ctypes.c_int]
        L.kdt_status_str.restype = ctypes.c_char_p
        L.kdt_version.argtypes = []
        L.kdt_version.restype = ctypes.c_int
        L.kdt_build_visibility.argtypes = [vp, ctypes.c_int, ctypes.c_int, vp, vp, vp]
        L.kdt_build_visibility.restype = ctypes.c_int
        L.kdt_verify_attn.argtypes = [ctypes.POINTER(VerifyArgs), vp, ctypes.c_size_t, vp]
        L.kdt_verify_attn.restype = ctypes.c_int
        L.kdt_verify_attn_workspace_size.argtypes = [ctypes.POINTER(VerifyArgs)]
        L.kdt_verify_attn_workspace_size.restype = ctypes.c_size_t
        L.kdt_verify_attn_plan.argtypes = [ctypes.POINTER(VerifyArgs), ctypes.POINTER(Plan)]
        L.kdt_verify_attn_plan.restype = ctypes.c_int
        L.kdt_merge_attn_states.argtypes = [vp, vp, vp, vp, ctypes.c_int64, ctypes.c_int, vp, vp, vp]
        L.kdt_merge_attn_states.restype = ctypes.c_int
        L.kdt_verify_attn_host.argtypes = [ctypes.POINTER(VerifyArgs), ctypes.c_int, vp, ctypes.c_size_t, vp, vp, vp]
        L.kdt_verify_attn_host.restype = ctypes.c_int
        L.kdt_verify_attn_host_buffer_size.argtypes = [ctypes.POINTER(VerifyArgs), ctypes.c_int]
        L.kdt_verify_attn_host_buffer_size.restype = ctypes.c_size_t
        L.kdt_vc_up_proj.argtypes = [vp, vp, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                     vp, vp, vp]
        L.kdt_vc_up_proj.restype = ctypes.c_int
        L.kdt_test_verify_attn_wait_expiry.argtypes = [ctypes.POINTER(VerifyArgs), vp, ctypes.c_size_t,
                                                       ctypes.c_uint32, vp]
        L.kdt_test_verify_attn_wait_expiry.restype = ctypes.c_int
        L.kdt_verify_attn_noalloc.argtypes = [ctypes.POINTER(VerifyArgs), vp]
        L.kdt_verify_attn_noalloc.restype = ctypes.c_int
        L.kdt_rope_neox.argtypes = [ctypes.POINTER(RopeArgs), vp]
        L.kdt_rope_neox.restype = ctypes.c_int
        L.kdt_tree_accept.argtypes = [vp, vp, vp, ctypes.c_int, ctypes.c_int, vp, vp, vp, vp, vp]
        L.kdt_tree_accept.restype = ctypes.c_int
        L.kdt_kv_compact.argtypes = [vp, vp, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                     ctypes.c_int64, vp, vp, vp, ctypes.c_int, vp]
        L.kdt_kv_compact.restype = ctypes.c_int
        L.kdt_tree_build.argtypes = [vp, vp, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, vp, vp, vp, vp,
                                     vp, vp]
        L.kdt_tree_build.restype = ctypes.c_int
        L.kdt_latent_write_q8.argtypes = [ctypes.POINTER(LatentWriteArgs), vp]
        L.kdt_latent_write_q8.restype = ctypes.c_int
        L.kdt_latent_read_q8.argtypes = [vp, vp, vp, ctypes.c_int64, ctypes.c_int, ctypes.c_int, vp, vp, ctypes.c_int,
                                         vp, vp, vp]
        L.kdt_latent_read_q8.restype = ctypes.c_int
        L.kdt_kv_compact_q8.argtypes = [vp, vp, vp, ctypes.c_int, ctypes.c_int, ctypes.c_int64, vp, vp, vp,
                                        ctypes.c_int, vp]
        L.kdt_kv_compact_q8.restype = ctypes.c_int
        L.kdt_verify_attn_q8.argtypes = [ctypes.POINTER(VerifyQ8Args), vp, ctypes.c_size_t, vp]
        L.kdt_verify_attn_q8.restype = ctypes.c_int
        L.kdt_verify_attn_q8_workspace_size.argtypes = [ctypes.POINTER(VerifyQ8Args)]
        L.kdt_verify_attn_q8_workspace_size.restype = ctypes.c_size_t
        L.kdt_verify_attn_q8_plan.argtypes = [ctypes.POINTER(VerifyQ8Args), ctypes.POINTER(Plan)]
        L.kdt_verify_attn_q8_plan.restype = ctypes.c_int
        L.kdt_tree_sample.argtypes = [vp, vp, vp, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int64,
                                      ctypes.c_double, vp, vp, vp, vp, vp, vp, vp, vp]
        L.kdt_tree_sample.restype = ctypes.c_int
        L.kdt_page_assign.argtypes = [ctypes.POINTER(PageArgs), vp]
        L.kdt_page_assign.restype = ctypes.c_int
        L.kdt_latent_write_paged.argtypes = [ctypes.POINTER(LatentWritePagedArgs), vp]
        L.kdt_latent_write_paged.restype = ctypes.c_int
        L.kdt_kv_compact_paged.argtypes = [vp, vp, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, vp,
                                           ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int, vp, vp, vp,
                                           ctypes.c_int, vp]
        L.kdt_kv_compact_paged.restype = ctypes.c_int
        L.kdt_verify_attn_paged.argtypes = [ctypes.POINTER(VerifyPagedArgs), vp, ctypes.c_size_t, vp]
        L.kdt_verify_attn_paged.restype = ctypes.c_int
        L.kdt_verify_attn_paged_workspace_size.argtypes = [ctypes.POINTER(VerifyPagedArgs)]
        L.kdt_verify_attn_paged_workspace_size.restype = ctypes.c_size_t
        L.kdt_verify_attn_paged_plan.argtypes = [ctypes.POINTER(VerifyPagedArgs), ctypes.POINTER(Plan)]
        L.kdt_verify_attn_paged_plan.restype = ctypes.c_int
        L.kdt_sample.argtypes = [ctypes.POINTER(SampleArgs), vp]
        L.kdt_sample.restype = ctypes.c_int
        _lib = L
    return _lib


def status_str(status: int) -> str:
    return lib().kdt_status_str(int(status)).decode()


def _check(status: int, where: str):
    if status != KDT_OK:
        raise KdtError(status, where)


def _stream_ptr(stream):
    import torch
    if stream is None:      # the current stream's handle without building a Stream object (3 us of a 20 us call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _i32(v, name) -> int:
    """A whole number that goes to the library as a C int (ctypes would drop its upper bits)."""
    v = int(v)
    if not -2 ** 31 <= v < 2 ** 31:
        raise ValueError(f"{name} must fit 32 bits, got {v}")
    return v


def _kept(t, stream):
    """A new tensor that a call uses on ``stream`` (None: the current one): its memory belongs to the current
    stream, which must not hand it out again while another one still uses it."""
    if stream is not None:
        t.record_stream(stream)
    return t


def _empty(shape, dtype, device, stream):
    import torch
    return _kept(torch.empty(shape, dtype=dtype, device=device), stream)


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return KDT_F32
    if t.dtype == torch.bfloat16:
        return KDT_BF16
    raise TypeError(f"inputs must be float32 or bfloat16, got {t.dtype}")


def make_args(q_nope, q_pe, c_kv, k_pe, prefix_len, *, parent=None, vis=None, max_kv_len=None,
              scale=DEFAULT_SCALE, out=None, lse=None, err=None, impl="auto", num_splits=0) -> VerifyArgs:
    """Fill the C argument struct from tensors (no checks beyond what the library does)."""
    B, T, H = q_nope.shape[0], q_nope.shape[1], q_nope.shape[2]
    L = c_kv.shape[1]
    a = VerifyArgs()
    a.B, a.T, a.H = B, T, H
    a.D_c, a.D_r = q_nope.shape[3], q_pe.shape[3]
    a.dtype = _dtype_code(q_nope)
    a.q_nope, a.q_pe, a.c_kv, a.k_pe = (t.data_ptr() for t in (q_nope, q_pe, c_kv, k_pe))
    a.kv_row_stride = L
    a.prefix_len = prefix_len.data_ptr()
    a.max_kv_len = _i32(L if max_kv_len is None else max_kv_len, "max_kv_len")
    a.parent = None if parent is None else parent.data_ptr()
    a.vis = None if vis is None else vis.data_ptr()
    a.scale = float(scale)
    a.out = None if out is None else out.data_ptr()
    a.lse = None if lse is None else lse.data_ptr()
    a.err = None if err is None else err.data_ptr()
    a.impl = IMPLS[impl] if isinstance(impl, str) else int(impl)
    a.num_splits = _i32(num_splits, "num_splits")
    a.q_nope_row_stride = _row_stride(q_nope)
    a.q_pe_row_stride = _row_stride(q_pe)
    return a


def _row_stride(q):
    """0 for a contiguous [B,T,H,d] tensor; else the element stride between (b,i,h) rows
    of a view with a contiguous last dim and equally spaced rows (e.g. a slice of a
    combined [B,T,H,576] query buffer)."""
    if q.is_contiguous():
        return 0
    s, n = q.stride(), q.shape
    # (rows of an expanded view have stride 0, which the library takes for "contiguous")
    if s[3] != 1 or s[2] < n[3] or s[2] * n[2] != s[1] or s[1] * n[1] != s[0]:
        raise ValueError("query views must have a contiguous last dim and equally spaced (b,i,h) rows that do not overlap")
    return s[2]


def plan(args: VerifyArgs) -> dict:
    p = Plan()
    _check(lib().kdt_verify_attn_plan(ctypes.byref(args), ctypes.byref(p)), "kdt_verify_attn_plan")
    return dict(impl=IMPL_NAMES.get(p.impl, p.impl), num_splits=p.num_splits, num_launches=p.num_launches,
                ctas=p.ctas, workspace_bytes=int(p.workspace_bytes))


def workspace_size(args: VerifyArgs) -> int:
    return int(lib().kdt_verify_attn_workspace_size(ctypes.byref(args)))


def build_visibility(parent, err=None, stream=None):
    """parent int32 [B,T] (cuda) -> packed bits uint32-as-int32 tensor [B,T,ceil(T/32)]."""
    import torch
    B, T = parent.shape
    vis = _empty((B, T, (T + 31) // 32), torch.int32, parent.device, stream)
    _check(lib().kdt_build_visibility(_ptr(parent), B, T, _ptr(vis), _ptr(err), _stream_ptr(stream)),
           "kdt_build_visibility")
    return vis


def verify_attn(q_nope, q_pe, c_kv, k_pe, prefix_len, *, parent=None, vis=None, max_kv_len=None,
                scale=DEFAULT_SCALE, out=None, lse=None, err=None, impl="auto", num_splits=0,
                workspace=None, stream=None, want_lse=True):
    """Tree-verify MLA-absorb attention. Returns (out [B,T,H,512] fp32, lse [B,T,H] fp32 or None).

    ``max_kv_len`` defaults to the cache row stride (c_kv.shape[1]), a valid host
    bound that needs no device->host read of prefix_len.
    """
    import torch
    B, T, H = q_nope.shape[:3]
    dev = q_nope.device
    if out is None:
        out = _empty((B, T, H, q_nope.shape[3]), torch.float32, dev, stream)
    if lse is None and want_lse:
        lse = _empty((B, T, H), torch.float32, dev, stream)
    a = make_args(q_nope, q_pe, c_kv, k_pe, prefix_len, parent=parent, vis=vis, max_kv_len=max_kv_len,
                  scale=scale, out=out, lse=lse, err=err, impl=impl, num_splits=num_splits)
    need = workspace_size(a)
    if workspace is None and need > 0:
        workspace = _empty(need, torch.uint8, dev, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().kdt_verify_attn(ctypes.byref(a), _ptr(workspace), ws_bytes, _stream_ptr(stream)),
           "kdt_verify_attn")
    return out, lse


def host_buffer_size(args: VerifyArgs, n_chunks=0) -> int:
    return int(lib().kdt_verify_attn_host_buffer_size(ctypes.byref(args), _i32(n_chunks, "n_chunks")))


def verify_attn_host(q_nope, q_pe, c_kv, k_pe, prefix_len, *, parent=None, vis=None, max_kv_len=None,
                     scale=DEFAULT_SCALE, out=None, lse=None, err=None, impl="auto", num_splits=0, n_chunks=0,
                     dev_buf=None, streams=None, want_lse=True, device=None):
    """kdt_verify_attn_host: host (CPU, ideally pinned) tensors in, host out and lse back.

    ``streams`` = (compute, copy in, copy out) torch streams (default: the current
    stream and two new ones); ``dev_buf`` a device uint8 tensor of at least
    host_buffer_size() bytes (allocated here if None). The result is complete once
    the compute stream is synchronised. ``err`` is a device int32 word."""
    import torch
    B, T, H = q_nope.shape[:3]
    dev = torch.device("cuda") if device is None else torch.device(device)
    if out is None:
        out = torch.empty((B, T, H, q_nope.shape[3]), dtype=torch.float32, pin_memory=True)
    if lse is None and want_lse:
        lse = torch.empty((B, T, H), dtype=torch.float32, pin_memory=True)
    a = make_args(q_nope, q_pe, c_kv, k_pe, prefix_len, parent=parent, vis=vis, max_kv_len=max_kv_len,
                  scale=scale, out=out, lse=lse, err=err, impl=impl, num_splits=num_splits)
    need = host_buffer_size(a, n_chunks)
    if dev_buf is None and need > 0:
        dev_buf = _empty(need, torch.uint8, dev, None if streams is None else streams[0])   # (where all of it ends)
    nbytes = 0 if dev_buf is None else dev_buf.numel() * dev_buf.element_size()
    if streams is None:
        streams = (torch.cuda.current_stream(dev), torch.cuda.Stream(dev), torch.cuda.Stream(dev))
    s, s_in, s_out = (ctypes.c_void_p(x.cuda_stream) for x in streams)
    _check(lib().kdt_verify_attn_host(ctypes.byref(a), _i32(n_chunks, "n_chunks"), _ptr(dev_buf), nbytes, s, s_in, s_out),
           "kdt_verify_attn_host")
    return out, lse


def merge_attn_states(o_a, lse_a, o_b, lse_b, out=None, lse=None, stream=None):
    """Log-sum-exp merge of two attention states over disjoint key sets."""
    import torch
    D = o_a.shape[-1]
    rows = lse_a.numel()
    if out is None:
        out = _kept(torch.empty_like(o_a), stream)
    if lse is None:
        lse = _kept(torch.empty_like(lse_a), stream)
    _check(lib().kdt_merge_attn_states(_ptr(o_a), _ptr(lse_a), _ptr(o_b), _ptr(lse_b), rows, D, _ptr(out),
                                       _ptr(lse), _stream_ptr(stream)), "kdt_merge_attn_states")
    return out, lse


def vc_up_proj(o, w_vc, out=None, err=None, stream=None):
    """Per-head value up-projection (kdt_vc_up_proj): o fp32 [..., H, 512] (e.g. the
    verify output [B,T,H,512]), w_vc bf16 [H, 512, D_v] -> fp32 [..., H, D_v]."""
    import torch
    H, D_c = o.shape[-2], o.shape[-1]
    D_v = w_vc.shape[-1]
    if tuple(w_vc.shape[:2]) != (H, D_c):
        raise ValueError("w_vc must be [H, D_c, D_v] matching o [..., H, D_c]")
    R = o.numel() // (H * D_c) if o.numel() else 0
    if out is None:
        out = _empty(tuple(o.shape[:-1]) + (D_v,), torch.float32, o.device, stream)
    _check(lib().kdt_vc_up_proj(_ptr(o), _ptr(w_vc), _dtype_code(w_vc), R, H, D_c, D_v, _ptr(out), _ptr(err),
                                _stream_ptr(stream)), "kdt_vc_up_proj")
    return out


def verify_attn_noalloc(q_nope, q_pe, c_kv, k_pe, prefix_len, *, out, lse=None, parent=None, vis=None,
                        max_kv_len=None, scale=DEFAULT_SCALE, err=None, impl="auto", num_splits=0, stream=None):
    """kdt_verify_attn_noalloc: the same attention with the library's fixed scratch array.

    For callers that must not allocate device memory at call time: the caller passes
    every input and output (``out`` is required); the library neither allocates nor
    asks for a workspace. Calls on one device share the scratch array, so calls
    that overlap on the GPU race; see include/kdt.h.
    """
    a = make_args(q_nope, q_pe, c_kv, k_pe, prefix_len, parent=parent, vis=vis, max_kv_len=max_kv_len,
                  scale=scale, out=out, lse=lse, err=err, impl=impl, num_splits=num_splits)
    _check(lib().kdt_verify_attn_noalloc(ctypes.byref(a), _stream_ptr(stream)), "kdt_verify_attn_noalloc")
    return out, lse


def rope_neox(pos, *, q=None, k_pe=None, prefix_len=None, base=10000.0, stream=None):
    """NeoX rotary embedding in place (kdt_rope_neox).

    ``q``: a [B,T,H,d] view whose last dim is contiguous -- e.g. the rope slice
    ``q_comb[..., 512:]`` of a combined [B,T,H,576] query buffer (its row stride is
    taken from the view). ``k_pe``: the [B,L,d] key cache; rows prefix_len[b] + i are
    rotated. ``pos`` int32 [B,T]. Returns nothing: the tensors are updated in place.
    """
    a = RopeArgs()
    a.B, a.T = pos.shape
    ref = q if q is not None else k_pe
    a.dtype = _dtype_code(ref)
    if q is not None:
        if q.stride(3) != 1 or q.stride(2) * q.shape[2] != q.stride(1) or q.stride(1) * q.shape[1] != q.stride(0):
            raise ValueError("q must be a [B,T,H,d] view with equally spaced (b,i,h) rows and a contiguous last dim")
        a.H, a.D_r = q.shape[2], q.shape[3]
        a.q, a.q_row_stride = q.data_ptr(), q.stride(2)
    else:
        a.H, a.D_r = 1, k_pe.shape[2]
    if k_pe is not None:
        a.k_pe, a.kv_row_stride = k_pe.data_ptr(), k_pe.shape[1]
        a.prefix_len = None if prefix_len is None else prefix_len.data_ptr()
    a.pos = pos.data_ptr()
    a.base = float(base)
    _check(lib().kdt_rope_neox(ctypes.byref(a), _stream_ptr(stream)), "kdt_rope_neox")


def tree_accept(parent, tok, target, err=None, stream=None):
    """Greedy accept walk (kdt_tree_accept). Returns (acc_nodes [B,T], n_acc [B], bonus [B]) int32."""
    import torch
    B, T = parent.shape
    dev = parent.device
    acc = _empty((B, T), torch.int32, dev, stream)
    n = _empty(B, torch.int32, dev, stream)
    bonus = _empty(B, torch.int32, dev, stream)
    _check(lib().kdt_tree_accept(_ptr(parent), _ptr(tok), _ptr(target), B, T, _ptr(acc), _ptr(n), _ptr(bonus),
                                 _ptr(err), _stream_ptr(stream)), "kdt_tree_accept")
    return acc, n, bonus


def kv_compact(c_kv, k_pe, prefix_len, acc_nodes, n_acc, update_prefix=True, stream=None):
    """Move the accepted path's cache rows to prefix_len + k, in place (kdt_kv_compact)."""
    B, T = acc_nodes.shape
    _check(lib().kdt_kv_compact(_ptr(c_kv), _ptr(k_pe), _dtype_code(c_kv), c_kv.shape[2], k_pe.shape[2], B, T,
                                c_kv.shape[1], _ptr(prefix_len), _ptr(acc_nodes), _ptr(n_acc),
                                1 if update_prefix else 0, _stream_ptr(stream)), "kdt_kv_compact")


def tree_build(cand_tok, cand_lp, N, root_tok=None, stream=None):
    """Best-first draft tree (kdt_tree_build). cand_tok int32 / cand_lp float32 [B,D,K].
    Returns (parent, tok, depth) int32 [B,N+1] and score float32 [B,N+1]."""
    import torch
    B, D, K = cand_lp.shape
    dev = cand_lp.device
    parent, tok, depth = (_empty((B, N + 1), torch.int32, dev, stream) for _ in range(3))
    score = _empty((B, N + 1), torch.float32, dev, stream)
    _check(lib().kdt_tree_build(_ptr(cand_tok), _ptr(cand_lp), B, D, K, _i32(N, "N"), _ptr(root_tok), _ptr(parent),
                                _ptr(tok), _ptr(depth), _ptr(score), _stream_ptr(stream)), "kdt_tree_build")
    return parent, tok, depth, score


def _row_stride3(t, name):
    """Element stride between the (b,i) rows of a [B,T,d] view with a contiguous last dim and
    equally spaced rows (e.g. a slice of a combined [B,T,576] buffer). Rows that overlap are
    refused: an expanded view's stride of 0 means "contiguous" to the library."""
    s, n = t.stride(), t.shape
    stride = s[1] if n[1] > 1 else (s[0] if n[0] > 1 else n[2])
    if s[2] != 1 or stride < n[2] or (n[0] > 1 and n[1] > 1 and s[0] != s[1] * n[1]):
        raise ValueError(f"{name} must be a [B,T,d] view with a contiguous last dim and equally spaced (b,i) rows "
                         "that do not overlap")
    return stride


def _check_q8_cache(c_q8, c_scale, k_pe):
    """The three arrays of an 8-bit cache: [B,L,512] and [B,L,16] bytes (uint8 or the float8
    types of the same width), [B,L,64] bf16, contiguous. Returns (B, L)."""
    import torch
    B, L, D = c_q8.shape
    if (D != 512 or c_scale.shape != (B, L, 16) or k_pe.shape != (B, L, 64) or c_q8.element_size() != 1 or c_scale.element_size() != 1 or k_pe.dtype != torch.bfloat16):
        raise ValueError("an 8-bit cache is c_q8 [B,L,512] and c_scale [B,L,16] of one byte an element and "
                         "k_pe [B,L,64] bf16")
    if not (c_q8.is_contiguous() and c_scale.is_contiguous() and k_pe.is_contiguous()):
        raise ValueError("the arrays of an 8-bit cache must be contiguous")
    return B, L


def _int32_of(t, n, name):
    import torch
    if t is not None and (t.dtype != torch.int32 or t.numel() != n or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous int32 tensor of {n} elements")
    return t


def _err_of(t):
    """Address of an error word: four bytes are written there."""
    if t is None:
        return None
    if t.element_size() != 4 or t.numel() < 1:
        raise ValueError("err must be an int32 tensor of at least one element")
    return t.data_ptr()


def latent_write_q8(c, k, c_q8, c_scale, k_pe, prefix_len, *, gamma=None, eps=1e-6, pos=None, base=10000.0,
                    n_rows=None, stream=None):
    """Norm, rotate, quantise and store new rows of an 8-bit cache (kdt_latent_write_q8).

    ``c`` [B,T,512] and ``k`` [B,T,64] (float32 or bf16) may be slices of one combined
    [B,T,576] buffer; row (b,i) goes to cache row prefix_len[b] + i. ``gamma`` [512] is the
    RMS norm's weight (None: no norm), ``pos`` int32 [B,T] the rotary positions (None: k as
    it is), ``n_rows`` int32 [B] the rows of each sequence of a padded batch. The cache
    (``c_q8`` [B,L,512], ``c_scale`` [B,L,16] bytes, ``k_pe`` [B,L,64] bf16) is updated in place.
    """
    B, L = _check_q8_cache(c_q8, c_scale, k_pe)
    T = c.shape[1]
    if c.shape != (B, T, 512) or k.shape != (B, T, 64) or k.dtype != c.dtype:
        raise ValueError("c must be [B,T,512] and k [B,T,64] of the same type, B as in the cache")
    if gamma is not None and (gamma.numel() != 512 or gamma.dtype != c.dtype or not gamma.is_contiguous()):
        raise ValueError("gamma must be a contiguous [512] tensor of c's type")
    _int32_of(prefix_len, B, "prefix_len"), _int32_of(n_rows, B, "n_rows"), _int32_of(pos, B * T, "pos")
    a = LatentWriteArgs(B, T, 512, 64, _dtype_code(c), c.data_ptr(), _row_stride3(c, "c"), k.data_ptr(),
                        _row_stride3(k, "k"), None if gamma is None else gamma.data_ptr(), float(eps),
                        None if pos is None else pos.data_ptr(), float(base), prefix_len.data_ptr(),
                        None if n_rows is None else n_rows.data_ptr(), c_q8.data_ptr(), c_scale.data_ptr(),
                        k_pe.data_ptr(), L)
    _check(lib().kdt_latent_write_q8(ctypes.byref(a), _stream_ptr(stream)), "kdt_latent_write_q8")


def latent_read_q8(c_q8, c_scale, k_pe, start, R, *, n_rows=None, dtype=None, out_c=None, out_k=None, stream=None):
    """Rows start[b] .. start[b] + R of an 8-bit cache as (c [B,R,512], k [B,R,64]) in bf16 (the
    default) or float32 (kdt_latent_read_q8); ``start`` int32 [B] or None for 0. With ``n_rows``
    int32 [B] the rows of c and k behind it are not written."""
    import torch
    B, L = _check_q8_cache(c_q8, c_scale, k_pe)
    R = _i32(R, "R")
    dtype = dtype or (out_c.dtype if out_c is not None else torch.bfloat16)
    _int32_of(start, B, "start"), _int32_of(n_rows, B, "n_rows")
    if out_c is None:
        out_c = _empty((B, R, 512), dtype, c_q8.device, stream)
    if out_k is None:
        out_k = _empty((B, R, 64), dtype, c_q8.device, stream)
    for t, d in ((out_c, 512), (out_k, 64)):
        if t.shape != (B, R, d) or t.dtype != dtype or not t.is_contiguous():
            raise ValueError("out_c and out_k must be contiguous [B,R,512] and [B,R,64] tensors of dtype")
    _check(lib().kdt_latent_read_q8(_ptr(c_q8), _ptr(c_scale), _ptr(k_pe), L, B, R, _ptr(start), _ptr(n_rows),
                                    _dtype_code(out_c), _ptr(out_c), _ptr(out_k), _stream_ptr(stream)),
           "kdt_latent_read_q8")
    return out_c, out_k


def kv_compact_q8(c_q8, c_scale, k_pe, prefix_len, acc_nodes, n_acc, update_prefix=True, stream=None):
    """Move the accepted path's rows of an 8-bit cache to prefix_len + k, in place (kdt_kv_compact_q8)."""
    B, L = _check_q8_cache(c_q8, c_scale, k_pe)
    T = acc_nodes.shape[1]
    _int32_of(prefix_len, B, "prefix_len"), _int32_of(acc_nodes, B * T, "acc_nodes"), _int32_of(n_acc, B, "n_acc")
    _check(lib().kdt_kv_compact_q8(_ptr(c_q8), _ptr(c_scale), _ptr(k_pe), B, T, L, _ptr(prefix_len), _ptr(acc_nodes),
                                   _ptr(n_acc), 1 if update_prefix else 0, _stream_ptr(stream)), "kdt_kv_compact_q8")


def _q8_size_args(B, T, H, max_kv_len, out_dtype, bits, impl, num_splits) -> VerifyQ8Args:
    """Arguments with the sizes filled in and placeholder pointers: enough for a plan."""
    import torch
    fake = 1 << 12
    a = VerifyQ8Args(B, T, H, 512, 64, fake, 0, fake, 0, fake, fake, fake, _i32(max_kv_len, "max_kv_len"), fake, int(max_kv_len),
                     None if bits else fake, fake if bits else None, 1.0, fake,
                     KDT_BF16 if out_dtype == torch.bfloat16 else KDT_F32, None, None, IMPLS[impl], _i32(num_splits, "num_splits"))
    return a


def verify_attn_q8_plan(B, T, H, max_kv_len, *, out_dtype=None, bits=False, impl="auto", num_splits=0) -> dict:
    """What verify_attn_q8 launches for these sizes (``bits``: visibility given as bits, not parents)."""
    p = Plan()
    a = _q8_size_args(B, T, H, max_kv_len, out_dtype, bits, impl, num_splits)
    _check(lib().kdt_verify_attn_q8_plan(ctypes.byref(a), ctypes.byref(p)), "kdt_verify_attn_q8_plan")
    return dict(impl=IMPL_NAMES.get(p.impl, p.impl), num_splits=p.num_splits, num_launches=p.num_launches,
                ctas=p.ctas, workspace_bytes=int(p.workspace_bytes))


def verify_attn_q8_workspace_size(B, T, H, max_kv_len, *, out_dtype=None, bits=False, impl="auto", num_splits=0) -> int:
    """Bytes of workspace verify_attn_q8 needs for these sizes."""
    return verify_attn_q8_plan(B, T, H, max_kv_len, out_dtype=out_dtype, bits=bits, impl=impl,
                               num_splits=num_splits)["workspace_bytes"]


def verify_attn_q8(q_nope, q_pe, c_q8, c_scale, k_pe, prefix_len, *, parent=None, vis=None, max_kv_len=None,
                   scale=DEFAULT_SCALE, out=None, out_dtype=None, lse=None, err=None, impl="auto", num_splits=0,
                   workspace=None, stream=None, want_lse=True):
    """Tree-verify attention over an 8-bit latent cache (kdt_verify_attn_q8).

    ``q_nope`` [B,T,H,512] and ``q_pe`` [B,T,H,64] are bf16 (slices of a combined [B,T,H,576]
    buffer are taken where they lie); the cache is c_q8 [B,L,512], c_scale [B,L,16], k_pe
    [B,L,64]. Returns (out [B,T,H,512], lse [B,T,H] fp32 or None); ``out_dtype`` is float32 (the
    default) or bfloat16. ``max_kv_len`` defaults to L.
    """
    import torch
    B, L = _check_q8_cache(c_q8, c_scale, k_pe)
    shape = q_nope.shape
    T, H = shape[1], shape[2]
    if shape != (B, T, H, 512) or q_pe.shape != (B, T, H, 64):
        raise ValueError("q_nope must be [B,T,H,512] and q_pe [B,T,H,64], B as in the cache")
    if q_nope.dtype != torch.bfloat16 or q_pe.dtype != torch.bfloat16:
        raise TypeError("queries must be bfloat16")
    _int32_of(prefix_len, B, "prefix_len"), _int32_of(parent, B * T, "parent")
    if vis is not None and (vis.numel() != B * T * ((T + 31) // 32) or vis.element_size() != 4 or not vis.is_contiguous()):
        raise ValueError("vis must be a contiguous 32-bit [B,T,ceil(T/32)] tensor")
    if out is None:
        out = _empty((B, T, H, 512), out_dtype or torch.float32, q_nope.device, stream)
    elif out.shape != (B, T, H, 512) or not out.is_contiguous() or (out_dtype or out.dtype) != out.dtype:
        raise ValueError("out must be a contiguous [B,T,H,512] tensor of out_dtype")
    if lse is None and want_lse:
        lse = _empty((B, T, H), torch.float32, q_nope.device, stream)
    elif lse is not None and (lse.numel() != B * T * H or lse.dtype != torch.float32 or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [B,T,H] tensor")
    a = VerifyQ8Args(B, T, H, 512, 64, q_nope.data_ptr(), _row_stride(q_nope), q_pe.data_ptr(), _row_stride(q_pe),
                     c_q8.data_ptr(), c_scale.data_ptr(), k_pe.data_ptr(), L, prefix_len.data_ptr(),
                     L if max_kv_len is None else _i32(max_kv_len, "max_kv_len"), None if parent is None else parent.data_ptr(),
                     None if vis is None else vis.data_ptr(), float(scale), out.data_ptr(), _dtype_code(out),
                     None if lse is None else lse.data_ptr(), _err_of(err),
                     IMPLS[impl] if isinstance(impl, str) else int(impl), _i32(num_splits, "num_splits"))
    if workspace is None:
        need = int(lib().kdt_verify_attn_q8_workspace_size(ctypes.byref(a)))
        workspace = _empty(need, torch.uint8, q_nope.device, stream) if need else None
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().kdt_verify_attn_q8(ctypes.byref(a), _ptr(workspace), ws_bytes, _stream_ptr(stream)),
           "kdt_verify_attn_q8")
    return out, lse


def tree_sample(parent, tok, logits, u_node, u_bonus, *, temperature=1.0, err=None, want_logp=True, stream=None):
    """Sampled verification of a drafted tree (kdt_tree_sample). ``logits`` [B,T,V] float32 or bf16 (equally
    spaced rows, a contiguous last dim), ``u_node`` [B,T] and ``u_bonus`` [B] float32 random numbers in
    [0, 1). Returns (acc_nodes [B,T], n_acc [B], bonus [B]) int32 and logp [B,T] float32 (or None)."""
    import torch
    B, T = parent.shape
    V = logits.shape[2]
    if logits.shape != (B, T, V):
        raise ValueError("logits must be [B,T,V], B and T as in parent")
    row_stride = _row_stride3(logits, "logits")
    _int32_of(parent, B * T, "parent"), _int32_of(tok, B * T, "tok")
    for t, n, name in ((u_node, B * T, "u_node"), (u_bonus, B, "u_bonus")):
        if t.dtype != torch.float32 or t.numel() != n or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 tensor of {n} elements")
    dev = logits.device
    acc = _empty((B, T), torch.int32, dev, stream)
    n = _empty(B, torch.int32, dev, stream)
    bonus = _empty(B, torch.int32, dev, stream)
    logp = _empty((B, T), torch.float32, dev, stream) if want_logp else None
    _check(lib().kdt_tree_sample(_ptr(parent), _ptr(tok), _ptr(logits), _dtype_code(logits), B, T, V, row_stride,
                                 float(temperature), _ptr(u_node), _ptr(u_bonus), _ptr(acc), _ptr(n), _ptr(bonus),
                                 _ptr(logp), _err_of(err), _stream_ptr(stream)), "kdt_tree_sample")
    return acc, n, bonus, logp


def _check_paged_cache(c_kv, k_pe):
    """The two arrays of a paged cache: [n_pages, page, 512] and [n_pages, page, 64] bf16, contiguous.
    Returns (n_pages, page)."""
    import torch
    n, page, D = c_kv.shape
    if D != 512 or k_pe.shape != (n, page, 64) or c_kv.dtype != torch.bfloat16 or k_pe.dtype != torch.bfloat16:
        raise ValueError("a paged cache is c_kv [n_pages,page,512] and k_pe [n_pages,page,64], both bf16")
    if not (c_kv.is_contiguous() and k_pe.is_contiguous()):
        raise ValueError("the arrays of a paged cache must be contiguous")
    return n, page


def _check_table(table, B):
    """A page table int32 [B,W], its rows contiguous, at equal distances and not overlapping. Returns (W, row stride)."""
    import torch
    W = table.shape[1]
    stride = table.stride(0) if B > 1 else W
    if table.shape[0] != B or table.dtype != torch.int32 or (W > 1 and table.stride(1) != 1) or stride < W:
        raise ValueError("table must be an int32 [B,W] tensor whose rows are contiguous and do not overlap")
    return W, stride


def page_assign(table, held, free_pages, n_free, new_len, page_size, *, start=None, T=0, slots=None, err=None,
                stream=None):
    """Pages for requests' new lengths, and the slots of their rows (kdt_page_assign).

    ``table`` int32 [B,W], ``held`` int32 [B], ``free_pages`` int32 [n_pages] (a stack) and ``n_free``
    int32 [1] are updated in place; ``new_len`` int32 [B] is what each request is to have room for. With
    ``T`` > 0, returns int32 [B,T]: the cache row of row start[b] + i, -1 at or beyond new_len[b]; else None.
    """
    import torch
    B = table.shape[0]
    W, stride = _check_table(table, B)
    _int32_of(held, B, "held"), _int32_of(new_len, B, "new_len"), _int32_of(n_free, 1, "n_free")
    _int32_of(free_pages, free_pages.numel(), "free_pages"), _int32_of(start, B, "start")
    T, page_size = _i32(T, "T"), _i32(page_size, "page_size")
    if T > 0:
        if start is None:
            raise ValueError("start is needed for slots")
        if slots is None:
            slots = _empty((B, T), torch.int32, table.device, stream)
        _int32_of(slots, B * T, "slots")
    else:
        slots = None
    a = PageArgs(B, W, table.data_ptr(), stride, held.data_ptr(), free_pages.data_ptr(), n_free.data_ptr(),
                 free_pages.numel(), page_size, new_len.data_ptr(), _ptr(start), T, _ptr(slots), _err_of(err))
    _check(lib().kdt_page_assign(ctypes.byref(a), _stream_ptr(stream)), "kdt_page_assign")
    return slots


def latent_write_paged(c, k, c_kv, k_pe, slots, *, gamma=None, eps=1e-6, pos=None, base=10000.0, stream=None):
    """Norm, rotate and store new rows of a paged cache at their slots (kdt_latent_write_paged).

    ``c`` [B,T,512] and ``k`` [B,T,64] (float32 or bf16) may be slices of one combined [B,T,576] buffer;
    row (b,i) goes to cache row slots[b,i] (int32 [B,T], e.g. of page_assign; one outside the cache is not
    written). ``gamma`` [512] is the RMS norm's weight (None: no norm), ``pos`` int32 [B,T] the rotary
    positions (None: k as it is). The cache (bf16 [n_pages,page,512] and [n_pages,page,64]) is updated in place.
    """
    n, page = _check_paged_cache(c_kv, k_pe)
    B, T = c.shape[:2]
    if c.shape != (B, T, 512) or k.shape != (B, T, 64) or k.dtype != c.dtype:
        raise ValueError("c must be [B,T,512] and k [B,T,64] of the same type")
    if gamma is not None and (gamma.numel() != 512 or gamma.dtype != c.dtype or not gamma.is_contiguous()):
        raise ValueError("gamma must be a contiguous [512] tensor of c's type")
    if slots is None:
        raise ValueError("slots is needed")
    _int32_of(slots, B * T, "slots"), _int32_of(pos, B * T, "pos")
    a = LatentWritePagedArgs(B * T, 512, 64, _dtype_code(c), c.data_ptr(), _row_stride3(c, "c"), k.data_ptr(),
                             _row_stride3(k, "k"), _ptr(gamma), float(eps), _ptr(pos), float(base), slots.data_ptr(),
                             c_kv.data_ptr(), k_pe.data_ptr(), n * page)
    _check(lib().kdt_latent_write_paged(ctypes.byref(a), _stream_ptr(stream)), "kdt_latent_write_paged")


def kv_compact_paged(c_kv, k_pe, table, prefix_len, acc_nodes, n_acc, update_prefix=True, stream=None):
    """Move the accepted path's rows of a paged cache to prefix_len + k, in place (kdt_kv_compact_paged)."""
    n, page = c_kv.shape[:2]
    B, T = acc_nodes.shape
    if k_pe.shape[:2] != (n, page) or k_pe.dtype != c_kv.dtype or not (c_kv.is_contiguous() and k_pe.is_contiguous()):
        raise ValueError("the arrays of a paged cache must be contiguous [n_pages,page,.] tensors of one type")
    W, stride = _check_table(table, B)
    _int32_of(prefix_len, B, "prefix_len"), _int32_of(acc_nodes, B * T, "acc_nodes"), _int32_of(n_acc, B, "n_acc")
    _check(lib().kdt_kv_compact_paged(_ptr(c_kv), _ptr(k_pe), _dtype_code(c_kv), c_kv.shape[2], k_pe.shape[2], n, page,
                                      _ptr(table), W, stride, B, T, _ptr(prefix_len), _ptr(acc_nodes), _ptr(n_acc),
                                      1 if update_prefix else 0, _stream_ptr(stream)), "kdt_kv_compact_paged")


def verify_attn_paged_plan(B, T, H, max_kv_len, page_size, *, out_dtype=None, bits=False, num_splits=0) -> dict:
    """What verify_attn_paged launches for these sizes (``bits``: visibility given as bits, not parents; with
    T = 1, neither)."""
    import torch
    fake = 1 << 12
    B, T, H, max_kv_len, page_size = (_i32(v, n) for v, n in ((B, "B"), (T, "T"), (H, "H"), (max_kv_len, "max_kv_len"),
                                                              (page_size, "page_size")))
    W = -(-max_kv_len // page_size) if page_size > 0 else 1
    a = VerifyPagedArgs(B, T, H, 512, 64, fake, 0, fake, 0, fake, fake, 1, page_size, fake, max(W, 1), 0, fake, None,
                        max_kv_len, None if bits or T == 1 else fake, fake if bits else None, 1.0, fake,
                        KDT_BF16 if out_dtype == torch.bfloat16 else KDT_F32, None, None, _i32(num_splits, "num_splits"))
    p = Plan()
    _check(lib().kdt_verify_attn_paged_plan(ctypes.byref(a), ctypes.byref(p)), "kdt_verify_attn_paged_plan")
    return dict(impl=IMPL_NAMES.get(p.impl, p.impl), num_splits=p.num_splits, num_launches=p.num_launches,
                ctas=p.ctas, workspace_bytes=int(p.workspace_bytes))


def verify_attn_paged_workspace_size(B, T, H, max_kv_len, page_size, *, out_dtype=None, bits=False, num_splits=0) -> int:
    """Bytes of workspace verify_attn_paged needs for these sizes."""
    return verify_attn_paged_plan(B, T, H, max_kv_len, page_size, out_dtype=out_dtype, bits=bits,
                                  num_splits=num_splits)["workspace_bytes"]


def verify_attn_paged(q_nope, q_pe, c_kv, k_pe, table, prefix_len, *, n_rows=None, parent=None, vis=None, max_kv_len=None,
                      scale=DEFAULT_SCALE, out=None, out_dtype=None, lse=None, err=None, num_splits=0, workspace=None,
                      stream=None, want_lse=True):
    """Tree-verify attention over a paged latent cache (kdt_verify_attn_paged); T = 1 is plain decoding.

    ``q_nope`` [B,T,H,512] and ``q_pe`` [B,T,H,64] are bf16 (slices of a combined [B,T,H,576] buffer are
    taken where they lie); the cache is c_kv [n_pages,page,512] and k_pe [n_pages,page,64] bf16, ``table``
    int32 [B,W] names each sequence's pages. ``parent`` int32 [B,T] or ``vis`` gives the tree (neither is
    needed with T = 1); ``n_rows`` int32 [B] the nodes of each sequence of a padded batch. Returns
    (out [B,T,H,512], lse [B,T,H] fp32 or None); ``out_dtype`` is float32 (the default) or bfloat16.
    ``max_kv_len`` defaults to the table's width in rows.
    """
    import torch
    n, page = _check_paged_cache(c_kv, k_pe)
    B, T, H = q_nope.shape[:3]
    W, stride = _check_table(table, B)
    if q_nope.shape != (B, T, H, 512) or q_pe.shape != (B, T, H, 64):
        raise ValueError("q_nope must be [B,T,H,512] and q_pe [B,T,H,64]")
    if q_nope.dtype != torch.bfloat16 or q_pe.dtype != torch.bfloat16:
        raise TypeError("queries must be bfloat16")
    _int32_of(prefix_len, B, "prefix_len"), _int32_of(n_rows, B, "n_rows"), _int32_of(parent, B * T, "parent")
    if vis is not None and (vis.numel() != B * T * ((T + 31) // 32) or vis.element_size() != 4 or not vis.is_contiguous()):
        raise ValueError("vis must be a contiguous 32-bit [B,T,ceil(T/32)] tensor")
    if out is None:
        out = _empty((B, T, H, 512), out_dtype or torch.float32, q_nope.device, stream)
    elif out.shape != (B, T, H, 512) or not out.is_contiguous() or (out_dtype or out.dtype) != out.dtype:
        raise ValueError("out must be a contiguous [B,T,H,512] tensor of out_dtype")
    if lse is None and want_lse:
        lse = _empty((B, T, H), torch.float32, q_nope.device, stream)
    elif lse is not None and (lse.numel() != B * T * H or lse.dtype != torch.float32 or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [B,T,H] tensor")
    a = VerifyPagedArgs(B, T, H, 512, 64, q_nope.data_ptr(), _row_stride(q_nope), q_pe.data_ptr(), _row_stride(q_pe),
                        c_kv.data_ptr(), k_pe.data_ptr(), n, page, table.data_ptr(), W, stride, prefix_len.data_ptr(),
                        _ptr(n_rows), min(W * page, 2 ** 31 - 257) if max_kv_len is None else _i32(max_kv_len, "max_kv_len"),
                        _ptr(parent), _ptr(vis), float(scale), out.data_ptr(), _dtype_code(out), _ptr(lse), _err_of(err),
                        _i32(num_splits, "num_splits"))
    if workspace is None:
        need = int(lib().kdt_verify_attn_paged_workspace_size(ctypes.byref(a)))
        workspace = _empty(need, torch.uint8, q_nope.device, stream) if need else None
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().kdt_verify_attn_paged(ctypes.byref(a), _ptr(workspace), ws_bytes, _stream_ptr(stream)),
           "kdt_verify_attn_paged")
    return out, lse


def _setting(v, R, dtype, name, off):
    """A sampling setting as (address of an array of one a row or None, one number for all rows)."""
    import torch
    if v is None:
        return None, off
    if torch.is_tensor(v):
        if v.dtype != dtype or v.numel() != R or not v.is_contiguous():
            raise ValueError(f"{name} must be a number or a contiguous {dtype} tensor of {R} elements")
        return v.data_ptr(), off
    if type(off) is int:        # a number of tokens: any that passes 32 bits keeps all of them, as the largest that fits
        return None, max(-1, min(int(v), 2 ** 31 - 1))
    return None, float(v)


def sample(logits, u, *, temperature=1.0, top_k=None, top_p=None, min_p=None, err=None, want_logp=True, stream=None):
    """One token a row under temperature, top-k, top-p and min-p (kdt_sample). ``logits`` [R,V] float32 or bf16
    (equally spaced rows, a contiguous last dim), ``u`` float32 [R] random numbers in [0, 1). A setting is a
    number, or a tensor of one a row (float32; top_k int32); None leaves a filter out; temperature 0 is greedy.
    Returns token [R] int32 and logp [R] float32 (or None)."""
    import torch
    R, V = logits.shape
    stride = logits.stride(0) if R > 1 else V
    if (V > 1 and logits.stride(1) != 1) or stride < V:
        raise ValueError("logits must be [R,V] with a contiguous last dim and rows that do not overlap")
    if u.dtype != torch.float32 or u.numel() != R or not u.is_contiguous():
        raise ValueError(f"u must be a contiguous float32 tensor of {R} elements")
    temp = _setting(temperature, R, torch.float32, "temperature", 1.0)
    k, p, low = (_setting(top_k, R, torch.int32, "top_k", 0), _setting(top_p, R, torch.float32, "top_p", 1.0),
                 _setting(min_p, R, torch.float32, "min_p", 0.0))
    token = _empty(R, torch.int32, logits.device, stream)
    logp = _empty(R, torch.float32, logits.device, stream) if want_logp else None
    a = SampleArgs(R, V, logits.data_ptr(), _dtype_code(logits), stride, u.data_ptr(), *temp, *k, *p, *low,
                   token.data_ptr(), _ptr(logp), _err_of(err))
    _check(lib().kdt_sample(ctypes.byref(a), _stream_ptr(stream)), "kdt_sample")
    return token, logp
