"""Thin ctypes binding of libgdn_dual.so (the C ABI in include/gdn_dual.h).

Argument marshalling only: every step of the forward runs in the library's CUDA kernels.
PyTorch supplies device memory and the current stream.  There is no fallback: if the
library is missing or cannot load, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgdn_dual.so")

GDN_OK, GDN_ERR_INVALID_ARG, GDN_ERR_ALIGNMENT, GDN_ERR_UNSUPPORTED, GDN_ERR_CUDA, GDN_ERR_TIMEOUT, GDN_ERR_BOUNDS = range(7)
GDN_BF16, GDN_FP32 = 0, 1
ALGO_AUTO, ALGO_SEQUENTIAL, ALGO_CHUNKED, ALGO_ROUTE1, ALGO_PIPELINED = 0, 1, 2, 3, 4
EXPORTED = ("gdn_dual_forward", "gdn_dual_workspace_size", "gdn_dual_read_device_status",
            "gdn_status_string", "gdn_dual_version", "gdn_dual_select_algo",
            "gdn_decode_replay", "gdn_decode_verify", "gdn_decode_commit", "gdn_dual_workspace_size_route1",
            "gdn_attn_forward", "gdn_attn_workspace_size", "gdn_dual_backward",
            "gdn_dual_backward_workspace_size", "gdn_dual_forward_noalloc",
            "gdn_dual_noalloc_read_device_status", "gdn_dual_forward_test_wait_limit",
            "gdn_dual_read_device_status_where", "gdn_attn_forward_test_wait_limit",
            "gdn_dual_backward_conv", "gdn_dual_backward_conv_workspace_size",
            "gdn_dual_forward_host", "gdn_dual_host_staging_size", "gdn_dual_host_read_device_status",
            "gdn_rotary_frequencies", "gdn_rotary_forward", "gdn_rotary_backward", "gdn_rotary_append",
            "gdn_kv_extend", "gdn_prefix_attn", "gdn_prefix_attn_workspace_size", "gdn_prefix_attn_test_wait_limit")
ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "ramp": 3}


class GdnError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


class Desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_docs", "num_heads", "d_k", "d_v", "num_views",
                                               "block_size", "dtype", "conv_width", "algo", "reserved")]


class DecodeDesc(ctypes.Structure):
    """gdn_decode_desc of include/gdn_decode.h."""
    _fields_ = [(n, ctypes.c_int32) for n in ("num_seqs", "num_heads", "d_k", "d_v", "num_tokens",
                                               "pool_slots", "dtype", "reserved")]


class AttnDesc(ctypes.Structure):
    """gdn_attn_desc of include/gdn_attention.h."""
    _fields_ = [(n, ctypes.c_int32) for n in ("num_docs", "num_heads", "num_kv_heads", "head_dim", "num_views",
                                               "block_size", "dtype", "reserved")]


class RotaryDesc(ctypes.Structure):
    """gdn_rotary_desc of include/gdn_rotary.h."""
    _fields_ = ([(n, ctypes.c_int32) for n in ("num_rows", "num_positions", "num_heads", "num_kv_heads", "head_dim",
                                                "rot_dim", "interleaved", "dtype")]
                + [("scale", ctypes.c_float), ("reserved", ctypes.c_int32)]
                + [(n, ctypes.c_int64) for n in ("q_row_stride", "q_head_stride", "k_row_stride", "k_head_stride",
                                                 "q_out_row_stride", "q_out_head_stride", "k_out_row_stride",
                                                 "k_out_head_stride")])


class AppendDesc(ctypes.Structure):
    """gdn_append_desc of include/gdn_kvcache.h."""
    _fields_ = ([(n, ctypes.c_int32) for n in ("num_rows", "num_heads", "num_kv_heads", "head_dim", "rot_dim",
                                                "interleaved", "page_size", "num_pages", "dtype")]
                + [("scale", ctypes.c_float)]
                + [(n, ctypes.c_int64) for n in ("q_row_stride", "q_head_stride", "k_row_stride", "k_head_stride",
                                                 "v_row_stride", "v_head_stride", "q_out_row_stride",
                                                 "q_out_head_stride")])


class KvExtendDesc(ctypes.Structure):
    """gdn_kv_extend_desc of include/gdn_kvcache.h."""
    _fields_ = [(n, ctypes.c_int32) for n in ("num_seqs", "table_width", "page_size", "num_free", "max_new_tokens",
                                               "prefix_len", "reserved0", "reserved1")]


class PrefixAttnDesc(ctypes.Structure):
    """gdn_prefix_attn_desc of include/gdn_kvcache.h."""
    _fields_ = [(n, ctypes.c_int32) for n in ("num_seqs", "num_tokens", "num_heads", "num_kv_heads", "head_dim",
                                               "page_size", "num_pages", "table_width", "prefix_len", "causal",
                                               "dtype")] + [("scale", ctypes.c_float)]


_lock = threading.Lock()
_lib = None


def load_library(path: str = LIB_PATH):
    """Load the CUDA library (raises OSError if it is missing; nothing falls back)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise OSError(f"{path} not found: build it with `python -m gated_deltanet_dual_b200.build`")
            lib = ctypes.CDLL(path)
            vp, fp, ip = ctypes.c_void_p, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_int32)
            lib.gdn_dual_forward.restype = ctypes.c_int
            lib.gdn_dual_forward.argtypes = [ctypes.POINTER(Desc), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                             ip, ip, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
            lib.gdn_dual_workspace_size.restype = ctypes.c_size_t
            lib.gdn_dual_workspace_size.argtypes = [ctypes.POINTER(Desc), ip]
            lib.gdn_dual_workspace_size_route1.restype = ctypes.c_size_t
            lib.gdn_dual_workspace_size_route1.argtypes = [ctypes.POINTER(Desc), ip, ip]
            lib.gdn_dual_read_device_status.restype = ctypes.c_int
            lib.gdn_dual_read_device_status.argtypes = [vp, vp]
            lib.gdn_status_string.restype = ctypes.c_char_p
            lib.gdn_status_string.argtypes = [ctypes.c_int]
            lib.gdn_dual_version.restype = ctypes.c_int32
            lib.gdn_dual_select_algo.restype = ctypes.c_int32
            lib.gdn_dual_select_algo.argtypes = [ctypes.POINTER(Desc)]
            dd = ctypes.POINTER(DecodeDesc)
            for name in ("gdn_decode_replay", "gdn_decode_verify", "gdn_decode_commit"):
                getattr(lib, name).restype = ctypes.c_int
            lib.gdn_decode_replay.argtypes = [dd, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
            lib.gdn_decode_verify.argtypes = [dd, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
            lib.gdn_decode_commit.argtypes = [dd, vp, vp, vp, vp, vp, vp]
            lib.gdn_dual_backward_workspace_size.restype = ctypes.c_size_t
            lib.gdn_dual_backward_workspace_size.argtypes = [ctypes.POINTER(Desc), ip]
            lib.gdn_dual_backward.restype = ctypes.c_int
            lib.gdn_dual_backward.argtypes = ([ctypes.POINTER(Desc)] + [vp] * 10 + [ip, ip] + [vp] * 3 + [vp] * 10
                                              + [vp, ctypes.c_size_t, vp])
            ad = ctypes.POINTER(AttnDesc)
            lib.gdn_attn_workspace_size.restype = ctypes.c_size_t
            lib.gdn_attn_workspace_size.argtypes = [ad, ip, ip]
            lib.gdn_attn_forward.restype = ctypes.c_int
            lib.gdn_attn_forward.argtypes = [ad, vp, vp, vp, vp, vp, vp, ip, ip, vp, vp, vp, ctypes.c_size_t, vp]
            lib.gdn_dual_host_staging_size.restype = ctypes.c_size_t
            lib.gdn_dual_host_staging_size.argtypes = [ctypes.POINTER(Desc), ip, ip, ctypes.c_int32]
            lib.gdn_dual_forward_host.restype = ctypes.c_int
            lib.gdn_dual_forward_host.argtypes = ([ctypes.POINTER(Desc)] + [vp] * 10 + [ip, ip, vp, vp, vp, vp, vp,
                                                  ctypes.c_size_t, ctypes.c_int32, vp])
            lib.gdn_dual_host_read_device_status.restype = ctypes.c_int
            lib.gdn_dual_host_read_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_int32), vp]
            for name in ("gdn_rotary_frequencies", "gdn_rotary_forward", "gdn_rotary_backward", "gdn_rotary_append",
                         "gdn_kv_extend", "gdn_prefix_attn"):
                getattr(lib, name).restype = ctypes.c_int
            dbl = ctypes.c_double
            lib.gdn_rotary_frequencies.argtypes = [ctypes.c_int32, dbl, ctypes.c_int32, dbl, dbl, dbl, dbl, vp]
            for name in ("gdn_rotary_forward", "gdn_rotary_backward"):
                getattr(lib, name).argtypes = [ctypes.POINTER(RotaryDesc)] + [vp] * 7
            lib.gdn_rotary_append.argtypes = [ctypes.POINTER(AppendDesc)] + [vp] * 11
            lib.gdn_kv_extend.argtypes = [ctypes.POINTER(KvExtendDesc)] + [vp] * 12
            lib.gdn_prefix_attn_workspace_size.restype = ctypes.c_size_t
            lib.gdn_prefix_attn_workspace_size.argtypes = [ctypes.POINTER(PrefixAttnDesc)]
            lib.gdn_prefix_attn.argtypes = [ctypes.POINTER(PrefixAttnDesc)] + [vp] * 8 + [ctypes.c_size_t, vp]
            _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load_library().gdn_status_string(int(status)).decode()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    if t.dtype == torch.float32:
        return GDN_FP32
    raise TypeError(f"unsupported I/O dtype {t.dtype}")


def make_desc(num_docs, num_heads, d_k, d_v, num_views, block_size, dtype_code, conv_width=0, algo=ALGO_AUTO):
    return Desc(num_docs, num_heads, d_k, d_v, num_views, block_size, dtype_code, conv_width, algo, 0)


def _host_i32(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def workspace_size(desc: Desc, doc_offsets) -> int:
    offs = _host_i32(doc_offsets)
    return int(load_library().gdn_dual_workspace_size(ctypes.byref(desc),
                                                      offs.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))))


def workspace_size_route1(desc: Desc, doc_offsets, prompt_len) -> int:
    """Workspace bytes for ALGO_ROUTE1 (header plus the materialised block-boundary states)."""
    offs, pl = _host_i32(doc_offsets), _host_i32(prompt_len)
    ip = ctypes.POINTER(ctypes.c_int32)
    return int(load_library().gdn_dual_workspace_size_route1(ctypes.byref(desc), offs.ctypes.data_as(ip),
                                                             pl.ctypes.data_as(ip)))


def select_algo(desc: Desc) -> int:
    return int(load_library().gdn_dual_select_algo(ctypes.byref(desc)))


def forward_raw(desc: Desc, q, k, v, g, beta, qn, kn, vn, gn, betan, doc_offsets, prompt_len, conv_w,
                out, out_noisy, final_state, workspace, stream=None) -> int:
    """Direct C-ABI call with tensors (or None) for every pointer; returns the status code."""
    lib = load_library()
    offs = _host_i32(doc_offsets)
    pl = _host_i32(prompt_len)
    ip = ctypes.POINTER(ctypes.c_int32)
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else 0
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return int(lib.gdn_dual_forward(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                    _ptr(qn), _ptr(kn), _ptr(vn), _ptr(gn), _ptr(betan),
                                    offs.ctypes.data_as(ip), pl.ctypes.data_as(ip), _ptr(conv_w),
                                    _ptr(out), _ptr(out_noisy), _ptr(final_state),
                                    _ptr(workspace), ctypes.c_size_t(ws_bytes), ctypes.c_void_p(stream)))


def forward_test_wait_limit_raw(desc: Desc, q, k, v, g, beta, qn, kn, vn, gn, betan, doc_offsets, prompt_len,
                                conv_w, out, out_noisy, final_state, workspace, wait_iters: int, stream=None) -> int:
    """C-ABI call of gdn_dual_forward_test_wait_limit (tests of the bounded-wait error path only:
    every device-side wait is bounded by `wait_iters` try-waits).  Returns the status code."""
    lib = load_library()
    fn = lib.gdn_dual_forward_test_wait_limit
    vp, ip = ctypes.c_void_p, ctypes.POINTER(ctypes.c_int32)
    fn.restype = ctypes.c_int
    fn.argtypes = [ctypes.POINTER(Desc)] + [vp] * 10 + [ip, ip] + [vp] * 5 + [ctypes.c_size_t, ctypes.c_uint32, vp]
    offs = _host_i32(doc_offsets)
    pl = _host_i32(prompt_len)
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    ws_bytes = workspace.numel() * workspace.element_size()
    return int(fn(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(qn), _ptr(kn), _ptr(vn),
                  _ptr(gn), _ptr(betan), offs.ctypes.data_as(ip), pl.ctypes.data_as(ip), _ptr(conv_w),
                  _ptr(out), _ptr(out_noisy), _ptr(final_state), _ptr(workspace), ctypes.c_size_t(ws_bytes),
                  ctypes.c_uint32(wait_iters), ctypes.c_void_p(stream)))


def read_device_status_where(workspace_tensor, stream=None):
    """(status, where): the device-side status word of a workspace and the diagnostic code of the
    wait that gave up (0 when none did).  Synchronises the stream."""
    lib = load_library()
    fn = lib.gdn_dual_read_device_status_where
    fn.restype = ctypes.c_int
    fn.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_int32), ctypes.c_void_p]
    where = ctypes.c_int32(0)
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    st = int(fn(_ptr(workspace_tensor), ctypes.byref(where), ctypes.c_void_p(stream)))
    return st, int(where.value)


class Workspace:
    """Caller-owned device scratch for gdn_dual_forward (allocated by torch, reused)."""

    def __init__(self, nbytes: int, device="cuda"):
        self.tensor = torch.zeros(max(256, (nbytes + 255) // 256 * 256), dtype=torch.uint8, device=device)


def _check(t: Optional[torch.Tensor], name: str, shape, dtype, device):
    if t is None:
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype} != {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def forward(q, k, v, g, beta, qn, kn, vn, gn, betan, doc_offsets, prompt_len, block_size,
            conv_w=None, *, algo: int = ALGO_AUTO, out=None, out_noisy=None, final_state=None,
            workspace: Optional[Workspace] = None, stream=None):
    """Dual-stream Gated DeltaNet forward on the GPU.

    Shapes: q, k [T,H,d]; v [T,H,d]; g, beta [T,H] fp32; qn, kn, vn [V,T_R,H,d]; gn, betan
    [V,T_R,H] fp32; conv_w [3,H*d,4] fp32 or None; doc_offsets [N+1], prompt_len [N] host ints.
    Returns (out [T,H,d], out_noisy [V,T_R,H,d], final_state [N,H,d,d] fp32)."""
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    T, H, dk = q.shape
    dv = v.shape[2]
    V, TR = qn.shape[0], qn.shape[1]
    offs = _host_i32(doc_offsets)
    pl = _host_i32(prompt_len)
    N = offs.shape[0] - 1
    io = q.dtype
    f32 = torch.float32
    if offs.ndim != 1 or pl.shape != (N,):
        raise ValueError("doc_offsets must be [N+1] and prompt_len [N]")
    if N >= 1 and int(offs[-1]) != T:
        raise ValueError(f"doc_offsets[-1] = {int(offs[-1])} but q has {T} tokens")
    if N >= 1 and int((np.diff(offs.astype(np.int64)) - pl).sum()) != TR:
        raise ValueError(f"noisy tensors have {TR} rows but the documents have "
                         f"{int((np.diff(offs.astype(np.int64)) - pl).sum())} response tokens")
    for t, name, shape, dt in ((q, "q", (T, H, dk), io), (k, "k", (T, H, dk), io), (v, "v", (T, H, dv), io),
                               (g, "g", (T, H), f32), (beta, "beta", (T, H), f32),
                               (qn, "qn", (V, TR, H, dk), io), (kn, "kn", (V, TR, H, dk), io),
                               (vn, "vn", (V, TR, H, dv), io), (gn, "gn", (V, TR, H), f32),
                               (betan, "betan", (V, TR, H), f32)):
        _check(t, name, shape, dt, dev)
    conv_width = 0
    if conv_w is not None:
        conv_width = int(conv_w.shape[-1])
        _check(conv_w, "conv_w", (3, H * dk, conv_width), f32, dev)
    if out is None:
        out = torch.empty(T, H, dv, dtype=io, device=dev)
    if out_noisy is None:
        out_noisy = torch.empty(V, TR, H, dv, dtype=io, device=dev)
    if final_state is None:
        final_state = torch.empty(N, H, dk, dv, dtype=f32, device=dev)
    _check(out, "out", (T, H, dv), io, dev)
    _check(out_noisy, "out_noisy", (V, TR, H, dv), io, dev)
    _check(final_state, "final_state", (N, H, dk, dv), f32, dev)
    desc = make_desc(N, H, dk, dv, V, int(block_size), _dtype_code(q), conv_width, algo)
    ws_tensor = workspace.tensor if workspace is not None else None
    if workspace is None:
        nbytes = workspace_size_route1(desc, offs, pl) if algo == ALGO_ROUTE1 else workspace_size(desc, offs)
        # size 0: the descriptor or the layout is invalid; the library's own validation below
        # then returns the status (nothing launches)
        if nbytes:
            ws_tensor = Workspace(nbytes, device=dev).tensor
    st = forward_raw(desc, q, k, v, g, beta, qn, kn, vn, gn, betan, offs, pl, conv_w,
                     out, out_noisy, final_state, ws_tensor, stream=stream)
    if st != GDN_OK:
        raise GdnError(st, f"gdn_dual_forward failed: {status_string(st)}")
    return out, out_noisy, final_state


def read_device_status(workspace: Workspace, stream=None) -> int:
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    return int(load_library().gdn_dual_read_device_status(_ptr(workspace.tensor), ctypes.c_void_p(stream)))


def host_staging_size(desc: Desc, doc_offsets, prompt_len, groups: int) -> int:
    """Device staging bytes gdn_dual_forward_host needs (0: invalid descriptor or layout)."""
    offs, pl = _host_i32(doc_offsets), _host_i32(prompt_len)
    ip = ctypes.POINTER(ctypes.c_int32)
    return int(load_library().gdn_dual_host_staging_size(ctypes.byref(desc), offs.ctypes.data_as(ip),
                                                         pl.ctypes.data_as(ip), int(groups)))


def forward_host_raw(desc: Desc, q, k, v, g, beta, qn, kn, vn, gn, betan, doc_offsets, prompt_len, conv_w,
                     out, out_noisy, final_state, staging: torch.Tensor, groups: int, stream=None) -> int:
    """C-ABI call of gdn_dual_forward_host: every tensor argument is a (pinned) CPU tensor, `staging`
    a CUDA byte tensor of host_staging_size() bytes.  Returns the status code; the outputs are in
    host memory once `stream` is synchronised."""
    lib = load_library()
    offs, pl = _host_i32(doc_offsets), _host_i32(prompt_len)
    ip = ctypes.POINTER(ctypes.c_int32)
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    return int(lib.gdn_dual_forward_host(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                         _ptr(qn), _ptr(kn), _ptr(vn), _ptr(gn), _ptr(betan),
                                         offs.ctypes.data_as(ip), pl.ctypes.data_as(ip), _ptr(conv_w),
                                         _ptr(out), _ptr(out_noisy), _ptr(final_state), _ptr(staging),
                                         ctypes.c_size_t(staging.numel()), int(groups), ctypes.c_void_p(stream)))


def read_host_device_status(staging: torch.Tensor, stream=None):
    """(status, where) recorded by the groups of the last gdn_dual_forward_host on `staging`."""
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    where = ctypes.c_int32(0)
    st = int(load_library().gdn_dual_host_read_device_status(_ptr(staging), ctypes.byref(where),
                                                             ctypes.c_void_p(stream)))
    return st, int(where.value)


def forward_problem(prob, **kw):
    """Run the forward on a synthetic problem whose tensors live on the GPU."""
    return forward(prob.q, prob.k, prob.v, prob.g, prob.beta, prob.qn, prob.kn, prob.vn, prob.gn,
                   prob.betan, prob.doc_offsets, prob.prompt_len, prob.block_size, conv_w=prob.conv_w, **kw)


def forward_noalloc_raw(desc: Desc, q, k, v, g, beta, qn, kn, vn, gn, betan, doc_offsets, prompt_len, conv_w,
                        out, out_noisy, final_state, stream=None) -> int:
    """C-ABI call of gdn_dual_forward_noalloc (no workspace: the library's fixed device scratch
    is used, for callers that cannot allocate).  Returns the status code."""
    lib = load_library()
    fn = lib.gdn_dual_forward_noalloc
    vp, ip = ctypes.c_void_p, ctypes.POINTER(ctypes.c_int32)
    fn.restype = ctypes.c_int
    fn.argtypes = [ctypes.POINTER(Desc), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ip, ip, vp, vp, vp, vp, vp]
    offs = _host_i32(doc_offsets)
    pl = _host_i32(prompt_len)
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    return int(fn(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(qn), _ptr(kn), _ptr(vn),
                  _ptr(gn), _ptr(betan), offs.ctypes.data_as(ip), pl.ctypes.data_as(ip), _ptr(conv_w),
                  _ptr(out), _ptr(out_noisy), _ptr(final_state), ctypes.c_void_p(stream)))


def noalloc_read_device_status(stream=None) -> int:
    """C-ABI call of gdn_dual_noalloc_read_device_status: the device-side status of the last
    gdn_dual_forward_noalloc on the current device (synchronises the stream)."""
    lib = load_library()
    fn = lib.gdn_dual_noalloc_read_device_status
    fn.restype = ctypes.c_int
    fn.argtypes = [ctypes.c_void_p]
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    return int(fn(ctypes.c_void_p(stream)))


# ----------------------------------------------------------------------------- decode side
def make_decode_desc(num_seqs, num_heads, d_k, d_v, num_tokens, pool_slots, dtype_code) -> DecodeDesc:
    return DecodeDesc(num_seqs, num_heads, d_k, d_v, num_tokens, pool_slots, dtype_code, 0)


def _decode_args(state_pool, slots, q, k, v, g, beta):
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    N, L, H, dk = q.shape
    dv = v.shape[3]
    P = state_pool.shape[0]
    io, f32 = q.dtype, torch.float32
    for t, name, shape, dt in ((state_pool, "state_pool", (P, H, dk, dv), f32), (slots, "slots", (N,), torch.int32),
                               (q, "q", (N, L, H, dk), io), (k, "k", (N, L, H, dk), io), (v, "v", (N, L, H, dv), io),
                               (g, "g", (N, L, H), f32), (beta, "beta", (N, L, H), f32)):
        _check(t, name, shape, dt, dev)
    return make_decode_desc(N, H, dk, dv, L, P, _dtype_code(q)), dev, (N, L, H, dk, dv)


def _stream(stream):
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream if stream is None else stream)


def decode_replay(state_pool, slots, q, k, v, g, beta, *, out=None, device_status=None, stream=None):
    """Causal replay of a committed block (gdn_decode_replay): runs the L tokens of every sequence
    from its pooled state, writes the outputs and the final state back into state_pool[slots]."""
    desc, dev, (N, L, H, dk, dv) = _decode_args(state_pool, slots, q, k, v, g, beta)
    if out is None:
        out = torch.empty(N, L, H, dv, dtype=q.dtype, device=dev)
    _check(out, "out", (N, L, H, dv), q.dtype, dev)
    st = load_library().gdn_decode_replay(ctypes.byref(desc), _ptr(state_pool), _ptr(slots), _ptr(q), _ptr(k),
                                          _ptr(v), _ptr(g), _ptr(beta), _ptr(out), _ptr(device_status),
                                          _stream(stream))
    if st != GDN_OK:
        raise GdnError(st, f"gdn_decode_replay failed: {status_string(st)}")
    return out


def decode_verify(state_pool, slots, q, k, v, g, beta, *, out=None, state_cache=None, device_status=None,
                  stream=None):
    """Verify forward with state cache (gdn_decode_verify): outputs of the L candidates and the
    state after each step in state_cache [N, L, H, d_k, d_v]; the pool is only read."""
    desc, dev, (N, L, H, dk, dv) = _decode_args(state_pool, slots, q, k, v, g, beta)
    if out is None:
        out = torch.empty(N, L, H, dv, dtype=q.dtype, device=dev)
    if state_cache is None:
        state_cache = torch.empty(N, L, H, dk, dv, dtype=torch.float32, device=dev)
    _check(out, "out", (N, L, H, dv), q.dtype, dev)
    _check(state_cache, "state_cache", (N, L, H, dk, dv), torch.float32, dev)
    st = load_library().gdn_decode_verify(ctypes.byref(desc), _ptr(state_pool), _ptr(slots), _ptr(q), _ptr(k),
                                          _ptr(v), _ptr(g), _ptr(beta), _ptr(out), _ptr(state_cache),
                                          _ptr(device_status), _stream(stream))
    if st != GDN_OK:
        raise GdnError(st, f"gdn_decode_verify failed: {status_string(st)}")
    return out, state_cache


def decode_commit(state_pool, slots, state_cache, accepted, *, device_status=None, stream=None):
    """Commit the accepted prefix (gdn_decode_commit): state_pool[slots[n]] := state_cache[n, r-1]
    for r = accepted[n] >= 1."""
    dev = state_pool.device
    N, L, H, dk, dv = state_cache.shape
    P = state_pool.shape[0]
    for t, name, shape, dt in ((state_pool, "state_pool", (P, H, dk, dv), torch.float32),
                               (slots, "slots", (N,), torch.int32), (accepted, "accepted", (N,), torch.int32),
                               (state_cache, "state_cache", (N, L, H, dk, dv), torch.float32)):
        _check(t, name, shape, dt, dev)
    desc = make_decode_desc(N, H, dk, dv, L, P, GDN_FP32)
    st = load_library().gdn_decode_commit(ctypes.byref(desc), _ptr(state_pool), _ptr(slots), _ptr(state_cache),
                                          _ptr(accepted), _ptr(device_status), _stream(stream))
    if st != GDN_OK:
        raise GdnError(st, f"gdn_decode_commit failed: {status_string(st)}")
    return state_pool


# ----------------------------------------------------------------------------- softmax attention
def make_attn_desc(num_docs, num_heads, num_kv_heads, head_dim, num_views, block_size, dtype_code) -> AttnDesc:
    return AttnDesc(num_docs, num_heads, num_kv_heads, head_dim, num_views, block_size, dtype_code, 0)


def attn_workspace_size(desc: AttnDesc, doc_offsets, prompt_len) -> int:
    offs = np.ascontiguousarray(doc_offsets, dtype=np.int32)
    pl = np.ascontiguousarray(prompt_len, dtype=np.int32)
    ip = ctypes.POINTER(ctypes.c_int32)
    return int(load_library().gdn_attn_workspace_size(ctypes.byref(desc), offs.ctypes.data_as(ip),
                                                      pl.ctypes.data_as(ip)))


def attention_forward(q, k, v, qn, kn, vn, doc_offsets, prompt_len, block_size, *, out=None, out_noisy=None,
                      workspace=None, stream=None):
    """Dual-stream softmax attention with the document-blocked causal / block-bidirectional mask
    (gdn_attn_forward).  q [T, H, d], k and v [T, H_kv, d]; qn [V, T_R, H, d], kn and vn
    [V, T_R, H_kv, d]; doc_offsets [N+1] and prompt_len [N] on the host.  Returns (out, out_noisy)."""
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    T, H, d = q.shape
    Hkv = k.shape[1]
    V, TR = qn.shape[0], qn.shape[1]
    offs = np.ascontiguousarray(doc_offsets, dtype=np.int32)
    pl = np.ascontiguousarray(prompt_len, dtype=np.int32)
    N = len(pl)
    if offs.ndim != 1 or offs.shape[0] != N + 1:
        raise ValueError("doc_offsets must be [N+1] and prompt_len [N]")
    if N >= 1 and int(offs[-1]) != T:
        raise ValueError(f"doc_offsets[-1] = {int(offs[-1])} but q has {T} tokens")
    if N >= 1 and int((np.diff(offs.astype(np.int64)) - pl).sum()) != TR:
        raise ValueError(f"noisy tensors have {TR} rows but the documents have "
                         f"{int((np.diff(offs.astype(np.int64)) - pl).sum())} response tokens")
    io = q.dtype
    for t, name, shape in ((q, "q", (T, H, d)), (k, "k", (T, Hkv, d)), (v, "v", (T, Hkv, d)),
                           (qn, "qn", (V, TR, H, d)), (kn, "kn", (V, TR, Hkv, d)), (vn, "vn", (V, TR, Hkv, d))):
        _check(t, name, shape, io, dev)
    if out is None:
        out = torch.empty(T, H, d, dtype=io, device=dev)
    if out_noisy is None:
        out_noisy = torch.empty(V, TR, H, d, dtype=io, device=dev)
    _check(out, "out", (T, H, d), io, dev)
    _check(out_noisy, "out_noisy", (V, TR, H, d), io, dev)
    desc = make_attn_desc(N, H, Hkv, d, V, int(block_size), _dtype_code(q))
    ws = workspace
    if ws is None:
        nbytes = attn_workspace_size(desc, offs, pl)
        if nbytes:
            ws = Workspace(nbytes, device=dev).tensor
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    ip = ctypes.POINTER(ctypes.c_int32)
    noisy = V > 0 and TR > 0
    st = load_library().gdn_attn_forward(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v),
                                         _ptr(qn) if noisy else None, _ptr(kn) if noisy else None,
                                         _ptr(vn) if noisy else None, offs.ctypes.data_as(ip), pl.ctypes.data_as(ip),
                                         _ptr(out), _ptr(out_noisy) if noisy else None, _ptr(ws),
                                         ctypes.c_size_t(ws_bytes), _stream(stream))
    if st != GDN_OK:
        raise GdnError(st, f"gdn_attn_forward failed: {status_string(st)}")
    return out, out_noisy


def attention_forward_test_wait_limit_raw(desc, q, k, v, qn, kn, vn, doc_offsets, prompt_len, out, out_noisy,
                                          workspace, wait_iters: int, stream=None) -> int:
    """C-ABI call of gdn_attn_forward_test_wait_limit (tests of the bounded-wait error path only).
    Returns the status code."""
    lib = load_library()
    fn = lib.gdn_attn_forward_test_wait_limit
    vp, ip = ctypes.c_void_p, ctypes.POINTER(ctypes.c_int32)
    fn.restype = ctypes.c_int
    fn.argtypes = [ctypes.POINTER(AttnDesc)] + [vp] * 6 + [ip, ip] + [vp] * 3 + [ctypes.c_size_t, ctypes.c_uint32, vp]
    offs = np.ascontiguousarray(doc_offsets, dtype=np.int32)
    pl = np.ascontiguousarray(prompt_len, dtype=np.int32)
    ws_bytes = workspace.numel() * workspace.element_size()
    return int(fn(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(qn), _ptr(kn), _ptr(vn),
                  offs.ctypes.data_as(ip), pl.ctypes.data_as(ip), _ptr(out), _ptr(out_noisy), _ptr(workspace),
                  ctypes.c_size_t(ws_bytes), ctypes.c_uint32(wait_iters), _stream(stream)))


# ----------------------------------------------------------------------------- backward
def backward_workspace_size(desc: Desc, doc_offsets) -> int:
    offs = np.ascontiguousarray(doc_offsets, dtype=np.int32)
    return int(load_library().gdn_dual_backward_workspace_size(ctypes.byref(desc),
                                                                offs.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))))


def backward(q, k, v, g, beta, qn, kn, vn, gn, betan, doc_offsets, prompt_len, block_size, d_out, d_out_noisy,
             d_final_state=None, *, conv_w=None, workspace=None, stream=None):
    """Gradients of <d_out, out> + <d_out_noisy, out_noisy> + <d_final_state, final_state> with
    respect to every input of the dual-stream forward, fp32 (gdn_dual_backward; with conv_w, the
    width-4 ShortConv prologue: gdn_dual_backward_conv, gradients of the raw inputs plus dconv_w).
    Returns a dict dq, dk, dv, dg, dbeta, dqn, dkn, dvn, dgn, dbetan (and dconv_w)."""
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    T, H, dk_ = q.shape
    dv_ = v.shape[2]
    V, TR = qn.shape[0], qn.shape[1]
    offs = np.ascontiguousarray(doc_offsets, dtype=np.int32)
    pl = np.ascontiguousarray(prompt_len, dtype=np.int32)
    N = len(pl)
    if offs.shape != (N + 1,) or (N >= 1 and int(offs[-1]) != T):
        raise ValueError("doc_offsets must be [N+1] and end at T")
    if N >= 1 and int((np.diff(offs.astype(np.int64)) - pl).sum()) != TR:
        raise ValueError("noisy tensors do not match the documents' response tokens")
    io, f32 = q.dtype, torch.float32
    for t, name, shape, dt in ((q, "q", (T, H, dk_), io), (k, "k", (T, H, dk_), io), (v, "v", (T, H, dv_), io),
                               (g, "g", (T, H), f32), (beta, "beta", (T, H), f32),
                               (qn, "qn", (V, TR, H, dk_), io), (kn, "kn", (V, TR, H, dk_), io),
                               (vn, "vn", (V, TR, H, dv_), io), (gn, "gn", (V, TR, H), f32),
                               (betan, "betan", (V, TR, H), f32), (d_out, "d_out", (T, H, dv_), io),
                               (d_out_noisy, "d_out_noisy", (V, TR, H, dv_), io),
                               (d_final_state, "d_final_state", (N, H, dk_, dv_), f32)):
        _check(t, name, shape, dt, dev)
    conv_width = 0
    if conv_w is not None:
        conv_width = int(conv_w.shape[-1])
        _check(conv_w, "conv_w", (3, H * dk_, conv_width), f32, dev)
    out = {n: torch.empty(x.shape, dtype=f32, device=dev) for n, x in (("dq", q), ("dk", k), ("dv", v), ("dg", g),
                                                                         ("dbeta", beta), ("dqn", qn), ("dkn", kn),
                                                                         ("dvn", vn), ("dgn", gn), ("dbetan", betan))}
    desc = make_desc(N, H, dk_, dv_, V, int(block_size), _dtype_code(q), conv_width)
    lib = load_library()
    ws = workspace
    if ws is None:
        nbytes = backward_workspace_size(desc, offs) if conv_w is None else backward_conv_workspace_size(desc, offs)
        if nbytes:
            ws = Workspace(nbytes, device=dev).tensor
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    noisy = V > 0 and TR > 0
    nz = lambda t: _ptr(t) if noisy else None
    ip = ctypes.POINTER(ctypes.c_int32)
    head = [ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), nz(qn), nz(kn), nz(vn), nz(gn),
            nz(betan), offs.ctypes.data_as(ip), pl.ctypes.data_as(ip)]
    grads = [_ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dg"]), _ptr(out["dbeta"]),
             nz(out["dqn"]), nz(out["dkn"]), nz(out["dvn"]), nz(out["dgn"]), nz(out["dbetan"])]
    ups = [_ptr(d_out), nz(d_out_noisy), _ptr(d_final_state)]
    if conv_w is None:
        st = lib.gdn_dual_backward(*head, *ups, *grads, _ptr(ws), ctypes.c_size_t(ws_bytes), _stream(stream))
        name = "gdn_dual_backward"
    else:
        out["dconv_w"] = torch.empty_like(conv_w)
        fn = lib.gdn_dual_backward_conv
        fn.restype = ctypes.c_int
        vp = ctypes.c_void_p
        fn.argtypes = [ctypes.POINTER(Desc)] + [vp] * 10 + [ip, ip] + [vp] * 4 + [vp] * 10 + [vp, vp, ctypes.c_size_t, vp]
        st = fn(*head, _ptr(conv_w), *ups, *grads, _ptr(out["dconv_w"]), _ptr(ws), ctypes.c_size_t(ws_bytes),
                _stream(stream))
        name = "gdn_dual_backward_conv"
    if st != GDN_OK:
        raise GdnError(st, f"{name} failed: {status_string(st)}")
    return out


def backward_conv_workspace_size(desc: Desc, doc_offsets) -> int:
    offs = np.ascontiguousarray(doc_offsets, dtype=np.int32)
    fn = load_library().gdn_dual_backward_conv_workspace_size
    fn.restype = ctypes.c_size_t
    fn.argtypes = [ctypes.POINTER(Desc), ctypes.POINTER(ctypes.c_int32)]
    return int(fn(ctypes.byref(desc), offs.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))))


# ----------------------------------------------------------------------------- serving calls
# The calls below are made once per layer and decode step, where a few microseconds on the host count: all
# properties are tested in one expression, and only a call that fails it goes through the checks that
# name what is wrong.
def _want(t: torch.Tensor, name: str, shape, dtype, index: int):
    """t is a contiguous CUDA tensor of this shape and dtype on device `index`, or raises."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        _check(t, name, shape, dtype, torch.device("cuda", index))
        raise ValueError(f"{name} must be a contiguous CUDA tensor")


def _rows(t: Optional[torch.Tensor], name: str, shape, dtype, index: int):
    """(row stride, head stride) in elements of [..., rows, heads, d] with contiguous heads."""
    if t is None:
        return 0, 0
    st = t.stride()
    if t.shape == shape and t.dtype is dtype and st[-1] == 1 and len(st) == 3 and t.get_device() == index:
        return st[0], st[1]
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype} != {dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    if len(shape) == 4 and shape[1] == 1:      # a row a view: the views are the rows
        return st[0], st[2]
    if len(shape) == 4 and shape[0] > 1 and st[0] != shape[1] * st[1]:
        raise ValueError(f"{name}: the views must lie {shape[1]} rows apart")
    return st[-3], st[-2]


def _cuda_index(t: torch.Tensor) -> int:
    index = t.get_device()
    if index < 0:
        raise ValueError("inputs must be CUDA tensors")
    return index


_PAST = 1 << 31                 # a size from here on does not fit the descriptors' int32; so for their bits together


def _int32(**values):
    """Raises when a value does not fit the descriptors' int32 (ctypes would drop its upper bits)."""
    for name, x in values.items():
        if not -1 << 31 <= x < 1 << 31:
            raise ValueError(f"{name}: {x} does not fit 32 bits")


def _fresh(like: torch.Tensor, shape, stream, dtype=None) -> torch.Tensor:
    """A new tensor for a call on `stream`.  It is allocated there: memory that the current stream has freed may still
    be written by work queued on it.  The current stream, where the caller may use it, is on its record too."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    index = like.get_device()
    current = torch.cuda.current_stream(index)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=index)):
        t = like.new_empty(shape, dtype=dtype)
    if stream != current.cuda_stream:
        t.record_stream(current)
    return t


def _call(name: str, index: int, stream, *args):
    """Calls the library on device `index` and raises on an error."""
    fn = getattr(_lib or load_library(), name)
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, torch._C._cuda_getCurrentRawStream(index) if stream is None else stream)
    else:
        with torch.cuda.device(index):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(index) if stream is None else stream)
    if st != GDN_OK:
        raise GdnError(st, f"{name} failed: {status_string(st)}")


# ----------------------------------------------------------------------------- rotary positions
class RotaryTable:
    """The frequencies of a rotary embedding on the device (made by rotary_table, kept by the caller)."""

    def __init__(self, turns: torch.Tensor, rot_dim: int, interleaved: bool, scale: float):
        if turns.dtype != torch.int64 or tuple(turns.shape) != (rot_dim // 2,) or not turns.is_contiguous():
            raise ValueError("turns must be a contiguous int64 tensor of rot_dim / 2 entries")
        self._turns, self._index, self._ptr = turns, turns.get_device(), turns.data_ptr()
        self._args = int(rot_dim), int(bool(interleaved)), float(scale)

    turns = property(lambda self: self._turns)
    rot_dim = property(lambda self: self._args[0])
    interleaved = property(lambda self: bool(self._args[1]))
    scale = property(lambda self: self._args[2])

    def _on(self, index: int):
        if self._index != index:
            raise ValueError(f"the rotary table is on {self._turns.device}, expected cuda:{index}")
        if self._turns.data_ptr() != self._ptr:
            raise ValueError("the rotary table's tensor was resized or replaced")
        return self._ptr


def rotary_frequencies(rot_dim, *, base=10000.0, scaling="none", factor=1.0, original_len=0, beta_fast=32.0,
                       beta_slow=1.0) -> np.ndarray:
    """gdn_rotary_frequencies: the pairs' fractions of a turn per position, uint64 fixed point (host)."""
    if scaling not in ROPE_SCALING:
        raise ValueError(f"scaling: {scaling!r} is none of {sorted(ROPE_SCALING)}")
    _int32(rot_dim=rot_dim)
    turns = np.zeros(max(1, int(rot_dim) // 2), dtype=np.uint64)
    st = load_library().gdn_rotary_frequencies(int(rot_dim), float(base), ROPE_SCALING[scaling], float(factor),
                                               float(original_len), float(beta_fast), float(beta_slow), turns.ctypes.data)
    if st != GDN_OK:
        raise GdnError(st, f"gdn_rotary_frequencies failed: {status_string(st)}")
    return turns[:int(rot_dim) // 2]


def rotary_table(rot_dim, *, interleaved=False, base=10000.0, scaling="none", factor=1.0, original_len=0,
                 beta_fast=32.0, beta_slow=1.0, attn_scale=None, device="cuda") -> RotaryTable:
    """Frequencies of the first rot_dim elements of a head (scaling: "none", "linear", "ntk" or "ramp", as
    include/gdn_rotary.h defines them).  attn_scale multiplies the rotated part; None means 1, and
    0.1 ln(factor) + 1 for "ramp"."""
    turns = rotary_frequencies(rot_dim, base=base, scaling=scaling, factor=factor, original_len=original_len,
                               beta_fast=beta_fast, beta_slow=beta_slow)
    if attn_scale is None:
        attn_scale = 0.1 * float(np.log(factor)) + 1.0 if scaling == "ramp" else 1.0
    return RotaryTable(torch.from_numpy(turns.view(np.int64).copy()).to(device), int(rot_dim), interleaved, attn_scale)


def _rotary(name, q, k, positions, table, q_out, k_out, stream):
    lead = q if q is not None else k
    if lead is None:
        raise ValueError("q and k are both None")
    index, io, shape = _cuda_index(lead), lead.dtype, lead.shape
    if len(shape) not in (3, 4):
        raise ValueError("q and k must be [T, H, d] or [V, T, H, d]")
    front, d = shape[:-2], shape[-1]
    T = front[-1]
    rows = T if len(front) == 1 else T * front[0]
    H = q.shape[-2] if q is not None else 0
    Hkv = k.shape[-2] if k is not None else 0
    q_shape, k_shape = front + (H, d), front + (Hkv, d)
    strides = _rows(q, "q", q_shape, io, index) + _rows(k, "k", k_shape, io, index)
    for given, out, label, want in ((q, q_out, "q_out", q_shape), (k, k_out, "k_out", k_shape)):
        if given is None:
            strides += 0, 0
        elif out is None:
            strides += want[-2] * d, d         # of a new tensor
        else:
            strides += _rows(out, label, want, io, index)
    if q is not None and q_out is None:
        q_out = _fresh(q, q_shape, stream)
    if k is not None and k_out is None:
        k_out = _fresh(k, k_shape, stream)
    _want(positions, "positions", (T,), torch.int32, index)
    turns = table._on(index)
    if rows | H | Hkv | d >= _PAST:
        _int32(rows=rows, num_heads=H, num_kv_heads=Hkv, head_dim=d)
    if rows and H + Hkv:
        desc = RotaryDesc(rows, T, H, Hkv, d, table._args[0], table._args[1], _dtype_code(lead), table._args[2], 0, *strides)
        _call(name, index, stream, ctypes.byref(desc), turns, positions.data_ptr(), q.data_ptr() if H else None,
              k.data_ptr() if Hkv else None, q_out.data_ptr() if H else None, k_out.data_ptr() if Hkv else None)
    return q_out if q is not None else None, k_out if k is not None else None


def rotary_forward(q, k, positions, table: RotaryTable, *, q_out=None, k_out=None, stream=None):
    """Rotary positions on q [T, H, d] and k [T, H_kv, d] (gdn_rotary_forward), or on the noisy twins
    [V, T, H, d], whose views share the positions [T] int32.  Rows and heads may be strided (slices of
    one projection's output); either of q and k may be None; q_out may be q.  Returns (q_out, k_out)."""
    return _rotary("gdn_rotary_forward", q, k, positions, table, q_out, k_out, stream)


def rotary_backward(dq, dk, positions, table: RotaryTable, *, dq_out=None, dk_out=None, stream=None):
    """Gradients of rotary_forward's inputs from those of its outputs (gdn_rotary_backward)."""
    return _rotary("gdn_rotary_backward", dq, dk, positions, table, dq_out, dk_out, stream)


# ----------------------------------------------------------------------------- paged key/value cache
class KvTables:
    """What kv_extend writes for a step of num_seqs sequences and at most max_new_tokens packed rows:
    slot_map, positions [max_new_tokens], cu_new [num_seqs + 1], seq_lens [num_seqs], free_left [1], all int32."""

    def __init__(self, num_seqs: int, max_new_tokens: int, device="cuda"):
        sizes = (max_new_tokens, max_new_tokens, num_seqs + 1, num_seqs, 1)
        self._tensors = tuple(torch.empty(n, dtype=torch.int32, device=device) for n in sizes)
        self._index = self._tensors[4].get_device()
        self._sizes = int(num_seqs), int(max_new_tokens)
        self._ptrs = tuple(t.data_ptr() for t in self._tensors)

    def _where(self):
        """The tensors' addresses (0 where there are no rows); their memory is still that of the sizes they were made for."""
        a, b, c, d, e = self._tensors
        if (a.data_ptr(), b.data_ptr(), c.data_ptr(), d.data_ptr(), e.data_ptr()) != self._ptrs:
            raise ValueError("a tensor of the tables was resized or replaced")
        return self._ptrs

    slot_map = property(lambda self: self._tensors[0])
    positions = property(lambda self: self._tensors[1])
    cu_new = property(lambda self: self._tensors[2])
    seq_lens = property(lambda self: self._tensors[3])
    free_left = property(lambda self: self._tensors[4])


def kv_extend(block_table, seq_lens, new_lens, free_pages, free_count, page_size, tables: KvTables, *, prefix_len=0,
              device_status=None, stream=None) -> KvTables:
    """Block tables, slots and positions of a step's new tokens (gdn_kv_extend): block_table [N, W] is
    extended in place with pages from the top of free_pages [F] (free_count [1] of them are free),
    tables receives the rest.  The next step takes tables.seq_lens and tables.free_left as its
    seq_lens and free_count (from another KvTables: outputs must not overlap inputs)."""
    index, i32 = _cuda_index(block_table), torch.int32
    if block_table.ndim != 2:
        raise ValueError("block_table must be [N, W]")
    N, W = block_table.shape
    F, M = free_pages.numel(), tables._sizes[1]
    if not (tables._sizes[0] == N and tables._index == index and seq_lens.shape == new_lens.shape == (N,)
            and free_pages.shape == (F,) and free_count.shape == (1,) and block_table.dtype is i32
            and seq_lens.dtype is i32 and new_lens.dtype is i32 and free_pages.dtype is i32 and free_count.dtype is i32
            and seq_lens.get_device() == new_lens.get_device() == free_pages.get_device() == free_count.get_device() == index
            and block_table.is_contiguous() and seq_lens.is_contiguous() and new_lens.is_contiguous()
            and free_pages.is_contiguous()):
        for t, name, shape in ((block_table, "block_table", (N, W)), (seq_lens, "seq_lens", (N,)), (new_lens, "new_lens", (N,)),
                               (free_pages, "free_pages", (F,)), (free_count, "free_count", (1,))):
            _want(t, name, shape, i32, index)
        raise ValueError(f"tables are made for {tables._sizes[0]} sequences on {tables.free_left.device}, not for {N} on cuda:{index}")
    if device_status is not None:
        _want(device_status, "device_status", (1,), i32, index)
    if not 0 <= page_size | prefix_len | N | W | F | M < _PAST:
        _int32(page_size=page_size, prefix_len=prefix_len, num_seqs=N, table_width=W, num_free=F, max_new_tokens=M)
    desc = KvExtendDesc(N, W, page_size, F, M, prefix_len, 0, 0)
    _call("gdn_kv_extend", index, stream, ctypes.byref(desc), block_table.data_ptr(), seq_lens.data_ptr(),
          new_lens.data_ptr(), free_pages.data_ptr(), free_count.data_ptr(), *tables._where(),
          None if device_status is None else device_status.data_ptr())
    return tables


def rotary_append(q, k, v, positions, slot_map, table: RotaryTable, k_cache, v_cache, *, q_out=None,
                  device_status=None, stream=None):
    """Rotary positions fused with the append to the cache (gdn_rotary_append): q [R, H, d] rotated into
    q_out, k [R, H_kv, d] rotated into k_cache [P, p, H_kv, d] and v copied into v_cache, at slot_map [R]
    int32, each slot at most once.  Rows with slot -1 are padding and are left as they were.  Returns q_out."""
    index, io = _cuda_index(q), q.dtype
    if q.ndim != 3 or k.ndim != 3 or v.ndim != 3 or k_cache.ndim != 4 or (q_out is not None and q_out.ndim != 3):
        raise ValueError("q, k, v and q_out must be [R, heads, d] and the caches [P, p, H_kv, d]")
    R, H, d = q.shape
    Hkv, (P, page) = k.shape[1], k_cache.shape[:2]
    if R | H | Hkv | d | P | page >= _PAST:
        _int32(num_rows=R, num_heads=H, num_kv_heads=Hkv, head_dim=d, num_pages=P, page_size=page)
    if q_out is None:
        q_out = _fresh(q, (R, H, d), stream)
    (qr, qh, q1), (kr, kh, k1), (vr, vh, v1), (outr, outh, out1) = q.stride(), k.stride(), v.stride(), q_out.stride()
    if not (q1 == k1 == v1 == out1 == 1 and k.shape[0] == R and k.shape[2] == d and v.shape == k.shape
            and q_out.shape == q.shape and k_cache.shape == v_cache.shape == (P, page, Hkv, d) and k.dtype is io
            and v.dtype is io and q_out.dtype is io and k_cache.dtype is io and v_cache.dtype is io
            and positions.dtype is torch.int32 and slot_map.dtype is torch.int32
            and positions.shape == slot_map.shape == (R,) and k_cache.is_contiguous() and v_cache.is_contiguous()
            and positions.is_contiguous() and slot_map.is_contiguous()
            and k.get_device() == v.get_device() == q_out.get_device() == k_cache.get_device() == v_cache.get_device()
            == positions.get_device() == slot_map.get_device() == index):
        for t, name, heads in ((q, "q", H), (k, "k", Hkv), (v, "v", Hkv), (q_out, "q_out", H)):
            _rows(t, name, (R, heads, d), io, index)
        _want(k_cache, "k_cache", (P, page, Hkv, d), io, index)
        _want(v_cache, "v_cache", (P, page, Hkv, d), io, index)
        _want(positions, "positions", (R,), torch.int32, index)
        _want(slot_map, "slot_map", (R,), torch.int32, index)
    if device_status is not None:
        _want(device_status, "device_status", (1,), torch.int32, index)
    desc = AppendDesc(R, H, Hkv, d, table._args[0], table._args[1], page, P, _dtype_code(q), table._args[2],
                      qr, qh, kr, kh, vr, vh, outr, outh)
    _call("gdn_rotary_append", index, stream, ctypes.byref(desc), table._on(index), positions.data_ptr(),
          slot_map.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(), k_cache.data_ptr(),
          v_cache.data_ptr(), None if device_status is None else device_status.data_ptr())
    return q_out


def make_prefix_attn_desc(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim, page_size, num_pages, table_width,
                          prefix_len, causal, scale=None, dtype_code=GDN_BF16) -> PrefixAttnDesc:
    """gdn_prefix_attn_desc; scale None is 1 / sqrt(head_dim)."""
    return PrefixAttnDesc(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim, page_size, num_pages, table_width,
                          prefix_len, 1 if causal else 0, dtype_code, 0.0 if scale is None else scale)


def prefix_attn_workspace_size(desc: PrefixAttnDesc) -> int:
    """Workspace bytes of gdn_prefix_attn (0: invalid or unsupported descriptor)."""
    return int(load_library().gdn_prefix_attn_workspace_size(ctypes.byref(desc)))


def prefix_attention(q, k_cache, v_cache, prefix_pages, prefix_len, block_table, seq_lens, *, causal=True, scale=None,
                     out=None, workspace: Optional[Workspace] = None, device_status=None, stream=None):
    """Attention of the L newest tokens of N sequences, q [N, L, H, d] bf16, over a shared prefix (the
    first prefix_len tokens on the pages prefix_pages) and each sequence's own seq_lens[n] keys through
    block_table [N, W], in caches [P, p, H_kv, d] (gdn_prefix_attn).  causal=False lets the L tokens see
    one another (a denoised block).  scale None is 1 / sqrt(d).  A workspace (Workspace, of
    prefix_attn_workspace_size bytes) belongs to one call at a time; None allocates one.  What is found wrong on the
    device (a length or page id out of range, a wait that gave up) is in device_status [1] int32 once the call is
    done, and in the workspace; the rows of a length out of range stay as they were, in a new out unset.  Returns
    out [N, L, H, d]."""
    index, io = _cuda_index(q), q.dtype
    if q.ndim != 4 or k_cache.ndim != 4 or block_table.ndim != 2:
        raise ValueError("q must be [N, L, H, d], the caches [P, p, H_kv, d] and block_table [N, W]")
    N, L, H, d = shape = q.shape
    P, page, Hkv = k_cache.shape[:3]
    W = block_table.shape[1]
    i32 = torch.int32
    if not (k_cache.dtype is io and v_cache.dtype is io and block_table.dtype is i32 and seq_lens.dtype is i32
            and k_cache.shape[3] == d and v_cache.shape == k_cache.shape and block_table.shape[0] == N
            and seq_lens.shape == (N,) and q.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous()
            and block_table.is_contiguous() and seq_lens.is_contiguous()
            and k_cache.get_device() == v_cache.get_device() == block_table.get_device() == seq_lens.get_device() == index):
        _want(q, "q", shape, io, index)
        _want(k_cache, "k_cache", (P, page, Hkv, d), io, index)
        _want(v_cache, "v_cache", (P, page, Hkv, d), io, index)
        _want(block_table, "block_table", (N, W), i32, index)
        _want(seq_lens, "seq_lens", (N,), i32, index)
    if scale is not None and not ctypes.c_float(scale).value > 0:      # what fp32 makes zero would mean 1 / sqrt(d)
        raise ValueError("scale must be positive in fp32")
    if prefix_len:
        if prefix_pages is None:
            raise ValueError("prefix_len needs prefix_pages")
        _want(prefix_pages, "prefix_pages", (prefix_pages.numel(),), torch.int32, index)
        if prefix_len < 0 or prefix_pages.numel() < -(-prefix_len // page):
            raise ValueError(f"prefix_pages holds {prefix_pages.numel()} pages of {page} for {prefix_len} tokens")
    if N | L | H | Hkv | d | page | P | W | prefix_len >= _PAST:
        _int32(num_seqs=N, num_tokens=L, num_heads=H, num_kv_heads=Hkv, head_dim=d, page_size=page, num_pages=P,
               table_width=W, prefix_len=prefix_len)
    if out is None:
        out = _fresh(q, shape, stream)
    else:
        _want(out, "out", shape, io, index)
    if device_status is not None:
        _want(device_status, "device_status", (1,), i32, index)
        at = device_status.data_ptr()
        for t in (q, k_cache, v_cache, prefix_pages, block_table, seq_lens, out, workspace and workspace.tensor):
            if t is not None and t.data_ptr() < at + 4 and at < t.data_ptr() + t.numel() * t.element_size():
                raise ValueError("device_status overlaps another tensor of the call")
    desc = PrefixAttnDesc(N, L, H, Hkv, d, page, P, W, prefix_len, 1 if causal else 0, _dtype_code(q),
                          0.0 if scale is None else scale)
    if workspace is None:
        ws = _fresh(q, (max(256, prefix_attn_workspace_size(desc)),), stream, torch.uint8)
    else:
        ws = workspace.tensor
        if ws.get_device() != index:
            raise ValueError(f"workspace is on {ws.device}, expected cuda:{index}")
    _call("gdn_prefix_attn", index, stream, ctypes.byref(desc), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
          prefix_pages.data_ptr() if prefix_len else None, block_table.data_ptr() if W else None, seq_lens.data_ptr(),
          out.data_ptr(), ws.data_ptr(), ws.numel())
    if device_status is not None:              # behind the call, on its stream
        found = ws[:4].view(i32)
        if stream is None:
            device_status.copy_(found)
        else:
            with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=index)):
                device_status.copy_(found)
    return out


def prefix_attention_test_wait_limit_raw(desc: PrefixAttnDesc, q, k_cache, v_cache, prefix_pages, block_table, seq_lens,
                                         out, workspace, wait_iters: int, stream=None) -> int:
    """C-ABI call of gdn_prefix_attn_test_wait_limit (tests of the bounded-wait error path only).
    Returns the status code."""
    fn = load_library().gdn_prefix_attn_test_wait_limit
    vp = ctypes.c_void_p
    fn.restype = ctypes.c_int
    fn.argtypes = [ctypes.POINTER(PrefixAttnDesc)] + [vp] * 8 + [ctypes.c_size_t, ctypes.c_uint32, vp]
    return int(fn(ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(prefix_pages), _ptr(block_table),
                  _ptr(seq_lens), _ptr(out), _ptr(workspace), ctypes.c_size_t(workspace.numel()),
                  ctypes.c_uint32(wait_iters), _stream(stream)))
