"""Python binding of libneattn (causal GQA + RoPE flash attention for sm_103a).

Argument marshalling only: every function checks dtypes, shapes and devices, then
calls the C ABI declared in include/neattn.h with raw device pointers and the
current torch CUDA stream.  All arithmetic runs in the library's CUDA kernels.  There
is no CPU fallback: if libneattn.so is missing or no sm_103 device is present the
calls raise.

Layouts: q, o, dO, dq are [B, T, Hq, D]; k, v, dk, dv are [B, T, Hkv, D]; lse is
[B, Hq, T] fp32.  bf16 tensors run on bf16 tensor cores, fp32 tensors on TF32.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import torch

from . import synthetic  # noqa: F401  (seeded inputs; no attention arithmetic)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libneattn.so")
_lock = threading.Lock()
_lib = None

NE_OK, NE_ERR_INVALID_ARG, NE_ERR_UNSUPPORTED, NE_ERR_CUDA, NE_ERR_DEVICE_TIMEOUT, NE_ERR_NO_DEVICE = range(6)

# Every symbol include/neattn.h declares (checked by the tests).
EXPORTS = (
    "ne_rope_table", "ne_attn_fwd", "ne_attn_fwd_f32", "ne_attn_bwd_workspace_size", "ne_attn_bwd",
    "ne_attn_bwd_f32", "ne_status_string", "ne_last_error", "ne_get_device_error",
    "ne_set_wait_timeout_ms", "ne_selftest_wait_timeout", "ne_shutdown", "ne_attn_bwd_noalloc",
    "ne_profile_enable", "ne_profile_totals", "ne_attn_decode_workspace_size", "ne_attn_decode",
    "ne_attn_decode_f32", "ne_noalloc_get_device_error", "ne_attn_fwd_varlen", "ne_attn_fwd_varlen_f32",
    "ne_attn_bwd_varlen", "ne_attn_bwd_varlen_f32", "ne_qkv_prologue", "ne_attn_fwd_train",
    "ne_attn_fwd_train_f32", "ne_attn_bwd_train", "ne_attn_bwd_train_f32", "ne_qkv_prologue_workspace_size",
    "ne_rope_spec_init", "ne_paged_append", "ne_paged_append_f32", "ne_paged_attn_workspace_size", "ne_paged_attn",
    "ne_paged_attn_f32", "ne_pages_workspace_size", "ne_pages_fork", "ne_pages_resize", "ne_pages_compact",
)


class PagedCache(ctypes.Structure):
    """ne_paged_cache of include/neattn.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("elem_bytes", ctypes.c_int), ("layers", ctypes.c_int),
                ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int),
                ("layer_stride", ctypes.c_int64), ("page_stride", ctypes.c_int64), ("tok_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class RopeSpec(ctypes.Structure):
    """ne_rope_spec of include/neattn.h (made by rope_spec)."""
    _fields_ = [("D", ctypes.c_int), ("rot_dim", ctypes.c_int), ("layout", ctypes.c_int), ("mscale", ctypes.c_float),
                ("turns", ctypes.c_uint64 * 64)]


class NeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{msg} [status {status}]")
        self.status = status


def load(path: str | None = None):
    """Load libneattn.so (built by ``_build.build()``).  Raises if it is missing."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise ImportError(f"libneattn.so not found at {p}; run __graft_entry__.build() first")
        lib = ctypes.CDLL(p)
        vp, i, d, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_double, ctypes.c_size_t
        lib.ne_rope_table.argtypes = [vp, vp, i, i, d, vp]
        lib.ne_attn_fwd.argtypes = [vp] * 5 + [i] * 5 + [d, vp]
        lib.ne_attn_fwd_f32.argtypes = lib.ne_attn_fwd.argtypes
        lib.ne_attn_bwd_workspace_size.argtypes = [i] * 5
        lib.ne_attn_bwd_workspace_size.restype = sz
        lib.ne_attn_bwd.argtypes = [vp] * 9 + [i] * 5 + [d, vp, sz, vp]
        lib.ne_attn_bwd_f32.argtypes = lib.ne_attn_bwd.argtypes
        lib.ne_status_string.argtypes = [i]
        lib.ne_status_string.restype = ctypes.c_char_p
        lib.ne_last_error.argtypes = []
        lib.ne_last_error.restype = ctypes.c_char_p
        lib.ne_get_device_error.argtypes = [vp]
        lib.ne_set_wait_timeout_ms.argtypes = [ctypes.c_uint32]
        lib.ne_set_wait_timeout_ms.restype = None
        lib.ne_selftest_wait_timeout.argtypes = [ctypes.c_uint32, vp]
        lib.ne_attn_bwd_noalloc.argtypes = [vp] * 9 + [i] * 5 + [d, vp]
        lib.ne_attn_fwd_varlen.argtypes = [vp] * 6 + [i] * 5 + [d, vp]
        lib.ne_attn_fwd_varlen_f32.argtypes = lib.ne_attn_fwd_varlen.argtypes
        lib.ne_attn_bwd_varlen.argtypes = [vp] * 10 + [i] * 5 + [d, vp, sz, vp]
        lib.ne_attn_bwd_varlen_f32.argtypes = lib.ne_attn_bwd_varlen.argtypes
        lib.ne_qkv_prologue.argtypes = [vp] * 6 + [i] * 6 + [d, d, i, vp, sz, vp]
        lib.ne_qkv_prologue_workspace_size.argtypes = [i] * 6
        lib.ne_qkv_prologue_workspace_size.restype = sz
        lib.ne_attn_fwd_train.argtypes = [vp] * 6 + [sz] + [i] * 5 + [d, vp]
        lib.ne_attn_fwd_train_f32.argtypes = lib.ne_attn_fwd_train.argtypes
        lib.ne_attn_bwd_train.argtypes = lib.ne_attn_bwd.argtypes
        lib.ne_attn_bwd_train_f32.argtypes = lib.ne_attn_bwd.argtypes
        lib.ne_noalloc_get_device_error.argtypes = [vp]
        lib.ne_profile_enable.argtypes = [i]
        lib.ne_profile_enable.restype = None
        lib.ne_profile_totals.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int)]
        lib.ne_profile_totals.restype = i
        lib.ne_shutdown.argtypes = []
        lib.ne_shutdown.restype = None
        lib.ne_attn_decode_workspace_size.argtypes = [i] * 5
        lib.ne_attn_decode_workspace_size.restype = sz
        lib.ne_attn_decode.argtypes = [vp] * 6 + [i] * 5 + [d, vp, sz, vp]
        lib.ne_attn_decode_f32.argtypes = lib.ne_attn_decode.argtypes
        i64 = ctypes.c_int64
        lib.ne_rope_spec_init.argtypes = [vp, i, i, i, d, i, d, i, d, d, d]
        lib.ne_paged_append.argtypes = [vp] * 8 + [i, vp] + [i64] * 4 + [i] * 4 + [vp]
        lib.ne_paged_append_f32.argtypes = lib.ne_paged_append.argtypes
        lib.ne_paged_attn_workspace_size.argtypes = [i] * 5
        lib.ne_paged_attn_workspace_size.restype = sz
        lib.ne_paged_attn.argtypes = [vp] * 7 + [i64] + [i] * 5 + [vp, sz, vp]
        lib.ne_paged_attn_f32.argtypes = lib.ne_paged_attn.argtypes
        lib.ne_pages_workspace_size.argtypes = [i, i, i]
        lib.ne_pages_workspace_size.restype = sz
        lib.ne_pages_fork.argtypes = [vp] * 5 + [i] + [vp] * 4 + [i] * 3 + [vp, sz, vp]
        lib.ne_pages_resize.argtypes = [vp] * 8 + [i] * 2 + [vp, sz, vp]
        lib.ne_pages_compact.argtypes = [vp] * 7 + [i] * 2 + [vp, sz, vp]
        for f in ("ne_rope_table", "ne_attn_fwd", "ne_attn_fwd_f32", "ne_attn_bwd", "ne_attn_bwd_f32",
                  "ne_get_device_error", "ne_selftest_wait_timeout", "ne_attn_bwd_noalloc", "ne_attn_decode",
                  "ne_noalloc_get_device_error", "ne_attn_fwd_varlen", "ne_attn_fwd_varlen_f32",
                  "ne_attn_bwd_varlen", "ne_attn_bwd_varlen_f32", "ne_qkv_prologue",
                  "ne_attn_decode_f32", "ne_rope_spec_init", "ne_paged_append", "ne_paged_append_f32", "ne_paged_attn",
                  "ne_paged_attn_f32", "ne_pages_fork", "ne_pages_resize", "ne_pages_compact"):
            getattr(lib, f).restype = i
        _lib = lib
    return _lib


def _check(status: int):
    if status != NE_OK:
        lib = load()
        raise NeError(status, f"{lib.ne_status_string(status).decode()}: {lib.ne_last_error().decode()}")


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _dims(q, k, v):
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [B, T, H, D]")
    B, T, Hq, D = q.shape
    Hkv = k.shape[2]
    if tuple(k.shape) != (B, T, Hkv, D) or tuple(v.shape) != (B, T, Hkv, D):
        raise ValueError(f"k, v must be [B, T, Hkv, D]; got {tuple(k.shape)}, {tuple(v.shape)}")
    for t in (q, k, v):
        if not t.is_cuda or not t.is_contiguous() or t.dtype != q.dtype:
            raise ValueError("q, k, v must be contiguous CUDA tensors of one dtype")
    if q.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("dtype must be bfloat16 or float32")
    return B, T, Hq, Hkv, D


def rope_table(T: int, D: int, theta: float = 10000.0, device="cuda"):
    """cos, sin [T, D/2] fp32 on ``device`` (ne_rope_table)."""
    lib = load()
    c = torch.empty((T, D // 2), dtype=torch.float32, device=device)
    s = torch.empty_like(c)
    _check(lib.ne_rope_table(_ptr(c), _ptr(s), T, D, float(theta), _stream(c)))
    return c, s


def attn_fwd(q, k, v, theta: float = 10000.0, o=None, lse=None):
    """Forward: returns (o [B,T,Hq,D], lse [B,Hq,T] fp32)."""
    lib = load()
    B, T, Hq, Hkv, D = _dims(q, k, v)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, T), dtype=torch.float32, device=q.device)
    fn = lib.ne_attn_fwd if q.dtype == torch.bfloat16 else lib.ne_attn_fwd_f32
    _check(fn(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, T, Hq, Hkv, D, float(theta), _stream(q)))
    return o, lse


def _check_lens(seq_lens, B, device):
    if seq_lens.dtype != torch.int32 or tuple(seq_lens.shape) != (B,) or not seq_lens.is_cuda \
            or not seq_lens.is_contiguous() or seq_lens.device != device:
        raise ValueError("seq_lens must be a contiguous int32 CUDA tensor [B] on the tensors' device")


def attn_fwd_varlen(q, k, v, seq_lens, theta: float = 10000.0, o=None, lse=None):
    """Forward over a padded batch of sequences of lengths seq_lens (int32 [B] on the
    device): returns (o, lse); padding rows get o = 0 and lse = -inf."""
    lib = load()
    B, T, Hq, Hkv, D = _dims(q, k, v)
    _check_lens(seq_lens, B, q.device)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, T), dtype=torch.float32, device=q.device)
    fn = lib.ne_attn_fwd_varlen if q.dtype == torch.bfloat16 else lib.ne_attn_fwd_varlen_f32
    _check(fn(_ptr(q), _ptr(k), _ptr(v), _ptr(seq_lens), _ptr(o), _ptr(lse), B, T, Hq, Hkv, D, float(theta),
              _stream(q)))
    return o, lse


def workspace_size(B, T, Hq, Hkv, D) -> int:
    return int(load().ne_attn_bwd_workspace_size(B, T, Hq, Hkv, D))


def alloc_workspace(B, T, Hq, Hkv, D, device="cuda"):
    n = workspace_size(B, T, Hq, Hkv, D)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def attn_bwd(q, k, v, o, lse, dO, theta: float = 10000.0, workspace=None, dq=None, dk=None, dv=None):
    """Backward: returns (dq, dk, dv) in the input dtype."""
    lib = load()
    B, T, Hq, Hkv, D = _dims(q, k, v)
    for t in (o, dO):
        if tuple(t.shape) != tuple(q.shape) or t.dtype != q.dtype or not t.is_contiguous():
            raise ValueError("o and dO must match q")
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, Hq, T) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [B, Hq, T]")
    if workspace is None:
        workspace = alloc_workspace(B, T, Hq, Hkv, D, q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    fn = lib.ne_attn_bwd if q.dtype == torch.bfloat16 else lib.ne_attn_bwd_f32
    _check(fn(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq), _ptr(dk), _ptr(dv),
              B, T, Hq, Hkv, D, float(theta), _ptr(workspace), workspace.numel() * workspace.element_size(),
              _stream(q)))
    return dq, dk, dv


def attn_fwd_train(q, k, v, workspace, theta: float = 10000.0, o=None, lse=None):
    """Training forward: what attn_fwd returns, and (bf16, head_dim 32/64) the backward
    workspace filled for attn_bwd_train of the same layer (see include/neattn.h)."""
    lib = load()
    B, T, Hq, Hkv, D = _dims(q, k, v)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, T), dtype=torch.float32, device=q.device)
    fn = lib.ne_attn_fwd_train if q.dtype == torch.bfloat16 else lib.ne_attn_fwd_train_f32
    _check(fn(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(workspace),
              workspace.numel() * workspace.element_size(), B, T, Hq, Hkv, D, float(theta), _stream(q)))
    return o, lse


def attn_bwd_train(q, k, v, o, lse, dO, workspace, theta: float = 10000.0, dq=None, dk=None, dv=None):
    """Backward after attn_fwd_train on the same workspace: returns (dq, dk, dv)."""
    lib = load()
    B, T, Hq, Hkv, D = _dims(q, k, v)
    for t in (o, dO):
        if tuple(t.shape) != tuple(q.shape) or t.dtype != q.dtype or not t.is_contiguous():
            raise ValueError("o and dO must match q")
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, Hq, T) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [B, Hq, T]")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    fn = lib.ne_attn_bwd_train if q.dtype == torch.bfloat16 else lib.ne_attn_bwd_train_f32
    _check(fn(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq), _ptr(dk), _ptr(dv),
              B, T, Hq, Hkv, D, float(theta), _ptr(workspace), workspace.numel() * workspace.element_size(),
              _stream(q)))
    return dq, dk, dv


def attn_bwd_varlen(q, k, v, o, lse, dO, seq_lens, theta: float = 10000.0, workspace=None, dq=None, dk=None,
                    dv=None):
    """Backward over a padded batch (see attn_fwd_varlen): returns (dq, dk, dv); padding
    positions get zero gradients."""
    lib = load()
    B, T, Hq, Hkv, D = _dims(q, k, v)
    _check_lens(seq_lens, B, q.device)
    for t in (o, dO):
        if tuple(t.shape) != tuple(q.shape) or t.dtype != q.dtype or not t.is_contiguous():
            raise ValueError("o and dO must match q")
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, Hq, T) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [B, Hq, T]")
    if workspace is None:
        workspace = alloc_workspace(B, T, Hq, Hkv, D, q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    fn = lib.ne_attn_bwd_varlen if q.dtype == torch.bfloat16 else lib.ne_attn_bwd_varlen_f32
    _check(fn(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(seq_lens), _ptr(dq), _ptr(dk), _ptr(dv),
              B, T, Hq, Hkv, D, float(theta), _ptr(workspace), workspace.numel() * workspace.element_size(),
              _stream(q)))
    return dq, dk, dv


def qkv_prologue(x, gamma, w, Hq: int, Hkv: int, D: int, eps: float = 1e-5, theta: float = 10000.0,
                 rotate: bool = False, q=None, k=None, v=None, workspace=None):
    """RMSNorm (gain gamma) -> projection w [(Hq + 2 Hkv) D, dim] -> q, k, v heads, RoPE
    on q and k when `rotate` (the attention calls take the unrotated form).  x [B, T, dim]
    bf16; returns q [B, T, Hq, D], k and v [B, T, Hkv, D] bf16."""
    lib = load()
    if x.dim() != 3:
        raise ValueError("x must be [B, T, dim]")
    B, T, dim = x.shape
    N = (Hq + 2 * Hkv) * D
    for t in (x, gamma, w):
        if not t.is_cuda or not t.is_contiguous() or t.dtype != torch.bfloat16 or t.device != x.device:
            raise ValueError("x, gamma and w must be contiguous bf16 CUDA tensors on one device")
    if tuple(gamma.shape) != (dim,) or tuple(w.shape) != (N, dim):
        raise ValueError(f"gamma must be [dim] and w [(Hq + 2 Hkv) D, dim] = [{N}, {dim}]")
    q = torch.empty((B, T, Hq, D), dtype=torch.bfloat16, device=x.device) if q is None else q
    k = torch.empty((B, T, Hkv, D), dtype=torch.bfloat16, device=x.device) if k is None else k
    v = torch.empty((B, T, Hkv, D), dtype=torch.bfloat16, device=x.device) if v is None else v
    if workspace is None:
        n = int(lib.ne_qkv_prologue_workspace_size(B, T, dim, Hq, Hkv, D))
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=x.device)
    _check(lib.ne_qkv_prologue(_ptr(x), _ptr(gamma), _ptr(w), _ptr(q), _ptr(k), _ptr(v), B, T, dim, Hq, Hkv, D,
                               float(eps), float(theta), 1 if rotate else 0, _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream(x)))
    return q, k, v


def decode_workspace_size(B, T_max, Hq, Hkv, D) -> int:
    return int(load().ne_attn_decode_workspace_size(B, T_max, Hq, Hkv, D))


def attn_decode(q, k_cache, v_cache, seq_lens, theta: float = 10000.0, o=None, lse=None, workspace=None):
    """Decode step: q [B, Hq, D] is the newest token of each sequence (unrotated),
    k_cache / v_cache [B, T_max, Hkv, D] hold positions 0 .. seq_lens[b] - 1 (the newest
    token's key and value included), seq_lens int32 [B] on the device.  Returns
    (o [B, Hq, D], lse [B, Hq] fp32): row seq_lens[b] - 1 of the causal attention."""
    lib = load()
    if q.dim() != 3 or k_cache.dim() != 4 or v_cache.dim() != 4:
        raise ValueError("q must be [B, Hq, D] and the caches [B, T_max, Hkv, D]")
    B, Hq, D = q.shape
    T_max, Hkv = k_cache.shape[1], k_cache.shape[2]
    if tuple(k_cache.shape) != (B, T_max, Hkv, D) or tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError(f"caches must be [B, T_max, Hkv, D]; got {tuple(k_cache.shape)}, {tuple(v_cache.shape)}")
    for t in (q, k_cache, v_cache):
        if not t.is_cuda or not t.is_contiguous() or t.dtype != q.dtype:
            raise ValueError("q and the caches must be contiguous CUDA tensors of one dtype")
    if q.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("dtype must be bfloat16 or float32")
    if seq_lens.dtype != torch.int32 or tuple(seq_lens.shape) != (B,) or not seq_lens.is_cuda \
            or not seq_lens.is_contiguous():
        raise ValueError("seq_lens must be a contiguous int32 CUDA tensor [B]")
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device) if lse is None else lse
    need = decode_workspace_size(B, T_max, Hq, Hkv, D)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    fn = lib.ne_attn_decode if q.dtype == torch.bfloat16 else lib.ne_attn_decode_f32
    _check(fn(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seq_lens), _ptr(o), _ptr(lse), B, T_max, Hq, Hkv, D,
              float(theta), _ptr(workspace), ws_bytes, _stream(q)))
    return o, lse


# ---------------------------------------------------------------- paged cache

ROPE_LAYOUTS = {"interleaved": 0, "half": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "parts": 3}


_INT_MAX = 2 ** 31 - 1


def _c_ints(**values):
    """Refuses what a C int does not hold: ctypes passes on the low 32 bits of any int."""
    for name, x in values.items():
        if not -_INT_MAX <= x <= _INT_MAX:
            raise ValueError(f"{name} = {x} does not fit into 32 bits")


def rope_spec(D: int, rot_dim: int | None = None, theta: float = 10000.0, layout: str = "interleaved",
              scaling: str = "none", factor: float = 1.0, orig_len: int = 0, beta_fast: float = 32.0,
              beta_slow: float = 1.0, mscale: float = 1.0) -> RopeSpec:
    """Rotary positions for paged_append (see ne_rope_spec in include/neattn.h): `layout`
    interleaved (pairs 2i, 2i+1) or half (pairs i, i + rot_dim/2), the first `rot_dim`
    elements of a head, `scaling` none, linear, base or parts for contexts `factor` times
    longer than trained.  A host value: make it once and keep it."""
    if layout not in ROPE_LAYOUTS or scaling not in ROPE_SCALINGS:
        raise ValueError(f"layout must be one of {tuple(ROPE_LAYOUTS)}, scaling one of {tuple(ROPE_SCALINGS)}")
    rot_dim = D if rot_dim is None else rot_dim
    _c_ints(D=D, rot_dim=rot_dim, orig_len=orig_len)
    out = RopeSpec()
    _check(load().ne_rope_spec_init(ctypes.byref(out), D, rot_dim, ROPE_LAYOUTS[layout],
                                    float(theta), ROPE_SCALINGS[scaling], float(factor), orig_len, float(beta_fast),
                                    float(beta_slow), float(mscale)))
    return out


# A generation step is a few small kernels, so these bindings keep the host's share low:
# plain comparisons, devices by index, addresses as integers, and no stream object (the
# current stream's handle is all the C calls take).

_I32, _BF16, _F32 = torch.int32, torch.bfloat16, torch.float32
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)


def _launch(fn, index, *args):
    """Calls fn with the device's current stream as last argument, on that device."""
    if _current_device() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status != NE_OK:
        _check(status)


_CACHE = struct.Struct("=QQ6i4q")                            # the fields of PagedCache in order
assert _CACHE.size == ctypes.sizeof(PagedCache)


def _paged_cache(k_pages, v_pages, layers: bool):
    """The pools [P, page_size, Hkv, D] ([L, P, page_size, Hkv, D] with `layers`) as the C
    struct (bytes), their device index, dtype, pages, heads and head_dim.  Any strides in
    multiples of 16 bytes with D dense (head-major pages are a transposed view), the same
    for both."""
    shape, st, dt, dev = k_pages.shape, k_pages.stride(), k_pages.dtype, k_pages.get_device()
    nd = len(shape)
    if nd == 4:
        P, ps, H, D = shape
        sp, stk, sh, sd = st
        L, ls = 1, 0
    elif nd == 5 and layers:
        L, P, ps, H, D = shape
        ls, sp, stk, sh, sd = st
    else:
        nd = 0
    if nd == 0 or v_pages.shape != shape:
        raise ValueError(f"k_pages and v_pages must be [{'L, ' if layers else ''}P, page_size, Hkv, D]; got "
                         f"{tuple(shape)}, {tuple(v_pages.shape)}")
    if dev < 0 or v_pages.get_device() != dev:
        raise ValueError("k_pages and v_pages must be CUDA tensors on one device")
    if (dt is not _BF16 and dt is not _F32) or v_pages.dtype is not dt:
        raise ValueError("k_pages and v_pages must both be bfloat16 or float32")
    if sd != 1 or v_pages.stride() != st:
        raise ValueError("k_pages and v_pages must have the same strides, D dense")
    return _CACHE.pack(k_pages.data_ptr(), v_pages.data_ptr(), 2 if dt is _BF16 else 4, L, P, ps, H, D, ls, sp, stk,
                       sh), dev, dt, P, H, D


def _ws(t, dev):
    """Address and bytes of a workspace."""
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the pages' device")
    return t.data_ptr(), t.nbytes


def _ints(t, shape, dev, name):
    """Address of an int32 tensor of that shape."""
    if t.dtype is _I32 and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous int32 CUDA tensor {list(shape)} on the pages' device")


def _paged_batch(page_table, seq_lens, cu_new, N, dev):
    """B, max_pages and the addresses of page_table, seq_lens and cu_new (0: one row each)."""
    shape = page_table.shape
    if len(shape) != 2:
        raise ValueError("page_table must be [B, max_pages]")
    B, W = shape
    if (B | W | N) > _INT_MAX:
        _c_ints(sequences=B, max_pages=W, rows=N)
    if cu_new is None and N != B:
        raise ValueError(f"without cu_new every sequence has one row: {N} rows for {B} sequences")
    return (B, W, _ints(page_table, shape, dev, "page_table"), _ints(seq_lens, (B,), dev, "seq_lens"),
            0 if cu_new is None else _ints(cu_new, (B + 1,), dev, "cu_new"))


def _rows(t, name, N, heads, D, dtype, dev):
    """Row stride of a [N, heads, D] tensor whose rows are dense."""
    if t.shape != (N, heads, D) or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be a {[N, heads, D]} {dtype} tensor on the pages' device; got "
                         f"{tuple(t.shape)} {t.dtype}")
    s0, s1, s2 = t.stride()
    if s2 != 1 or (heads > 1 and s1 != D):
        raise ValueError(f"{name}: the heads of a row must be dense")
    return s0 if N > 1 else heads * D


def paged_append(k, v, k_pages, v_pages, page_table, seq_lens, cu_new=None, rope=None, pos_offset: int = 0, q=None,
                 q_out=None):
    """New tokens into the paged cache (ne_paged_append): k, v [N, Hkv, D] packed rows
    cu_new[b] .. cu_new[b+1]-1 of sequence b (None: one row each) go to positions
    seq_lens[b] - n_b .. seq_lens[b] - 1 of its pages, k rotated by `rope` (a rope_spec, None:
    not).  With q [N, Hq, D] the query rows are rotated into q_out (which may be q), returned.
    Row slices of one fused projection are taken as they are."""
    if not 0 <= pos_offset <= _INT_MAX:
        _c_ints(pos_offset=pos_offset)
    lib = _lib or load()
    c, dev, dt, _, Hkv, D = _paged_cache(k_pages, v_pages, False)
    N = k.shape[0]
    B, W, pt, ln, cu = _paged_batch(page_table, seq_lens, cu_new, N, dev)
    k_ld, v_ld = _rows(k, "k", N, Hkv, D, dt, dev), _rows(v, "v", N, Hkv, D, dt, dev)
    Hq = q_ld = qo_ld = qp = qop = 0
    if q is not None:
        Hq = q.shape[1]
        q_ld = _rows(q, "q", N, Hq, D, dt, dev)
        if q_out is None:                                  # (without cu_new every row is written)
            q_out = q.new_empty((N, Hq, D)) if cu_new is None else q.new_zeros((N, Hq, D))
        qo_ld = _rows(q_out, "q_out", N, Hq, D, dt, dev)
        qp, qop = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out needs q")
    _launch(lib.ne_paged_append if dt is _BF16 else lib.ne_paged_append_f32, dev, qp, k.data_ptr(), v.data_ptr(),
            c, pt, ln, cu, ctypes.byref(rope) if rope is not None else None, pos_offset, qop, q_ld, k_ld, v_ld,
            qo_ld, B, N, Hq, W)
    return q_out


def paged_workspace_size(B, N, Hq, Hkv, D) -> int:
    _c_ints(B=B, N=N, Hq=Hq, Hkv=Hkv, D=D)
    return int(load().ne_paged_attn_workspace_size(B, N, Hq, Hkv, D))


def alloc_paged_workspace(B, N, Hq, Hkv, D, device="cuda"):
    """Workspace of paged_attn calls of this shape that run one after another."""
    return torch.empty(max(paged_workspace_size(B, N, Hq, Hkv, D), 256), dtype=torch.uint8, device=device)


def paged_attn(q, k_pages, v_pages, page_table, seq_lens, cu_new=None, max_new: int | None = None, o=None, lse=None,
               workspace=None):
    """Attention of the new tokens over the paged cache (ne_paged_attn): q [N, Hq, D]
    rotated rows, packed as in paged_append; row i of sequence b attends to its first
    seq_lens[b] - n_b + i + 1 positions.  Returns (o [N, Hq, D], lse [N, Hq] fp32); rows
    outside the sequences are not written (zeros in a fresh o and lse).  max_new: the most
    new tokens of a sequence, if known (a choice of kernel, not of results)."""
    if max_new is not None and not 1 <= max_new <= _INT_MAX:
        _c_ints(max_new=max_new)
    lib = _lib or load()
    c, dev, dt, _, Hkv, D = _paged_cache(k_pages, v_pages, False)
    N, Hq = q.shape[:2]
    B, W, pt, ln, cu = _paged_batch(page_table, seq_lens, cu_new, N, dev)
    q_ld = _rows(q, "q", N, Hq, D, dt, dev)
    new = q.new_empty if cu_new is None else q.new_zeros   # (without cu_new every row is written)
    if o is None:
        o = new((N, Hq, D))
    elif o.shape != q.shape or o.dtype is not dt or o.get_device() != dev or not o.is_contiguous():
        raise ValueError("o must be contiguous and match q")
    if lse is None:
        lse = new((N, Hq), dtype=_F32)
    elif lse.shape != (N, Hq) or lse.dtype is not torch.float32 or lse.get_device() != dev or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [N, Hq]")
    if workspace is None:
        workspace = alloc_paged_workspace(B, N, Hq, Hkv, D, k_pages.device)
    _launch(lib.ne_paged_attn if dt is _BF16 else lib.ne_paged_attn_f32, dev, q.data_ptr(), c, pt,
            ln, cu, o.data_ptr(), lse.data_ptr(), q_ld, B, N, Hq, W, max(1, N) if max_new is None else max_new,
            *_ws(workspace, dev))
    return o, lse


def alloc_pages_workspace(n_pages: int, n: int, max_pages: int, device="cuda"):
    """Workspace of pages_* calls over a pool of n_pages and tables of n sequences (a fork: children)."""
    _c_ints(n_pages=n_pages, n=n, max_pages=max_pages)
    return torch.empty(max(int(load().ne_pages_workspace_size(n_pages, n, max_pages)), 256), dtype=torch.uint8,
                       device=device)


def _out_ints(t, shape, dev, name, like):
    """An int32 output and its address: the caller's, or a new one beside `like` (int32)."""
    if t is None:
        t = like.new_empty(shape)
        return t, t.data_ptr()
    return t, _ints(t, shape, dev, name)


def pages_fork(refcount, page_table, seq_lens, parents, k_pages, v_pages, deep: bool = False, refcount_out=None,
               child_table=None, child_lens=None, short=None, workspace=None):
    """Children continue sequences parents[c] (int32 [C], -1: empty): whole pages shared and
    the partly filled last one copied, or (deep) every page copied, over all layers of
    k_pages, v_pages [L, P, page_size, Hkv, D].  Returns (refcount_out [P], child_table
    [C, max_pages], child_lens [C], short [1]); short > 0: that many pages were missing and
    nothing changed.  refcount_out may be refcount."""
    lib = _lib or load()
    c, dev, _, n_pages, _, _ = _paged_cache(k_pages, v_pages, True)
    P = (n_pages,)
    if page_table.dim() != 2 or parents.dim() != 1:
        raise ValueError("page_table must be [B, max_pages] and parents [C]")
    B, W = page_table.shape
    C = parents.shape[0]
    if (B | W | C) > _INT_MAX:
        _c_ints(sequences=B, max_pages=W, children=C)
    refcount_out, ro = _out_ints(refcount_out, P, dev, "refcount_out", refcount)
    child_table, ct = _out_ints(child_table, (C, W), dev, "child_table", refcount)
    child_lens, cl = _out_ints(child_lens, (C,), dev, "child_lens", refcount)
    short, sh = _out_ints(short, (1,), dev, "short", refcount)
    workspace = alloc_pages_workspace(n_pages, C, W, k_pages.device) if workspace is None else workspace
    _launch(lib.ne_pages_fork, dev, c, _ints(refcount, P, dev, "refcount"),
            _ints(page_table, (B, W), dev, "page_table"), _ints(seq_lens, (B,), dev, "seq_lens"),
            _ints(parents, (C,), dev, "parents"), 1 if deep else 0, ro, ct, cl, sh, B, C, W, *_ws(workspace, dev))
    return refcount_out, child_table, child_lens, short


def pages_resize(refcount, page_table, seq_lens, new_lens, k_pages, v_pages, refcount_out=None, table_out=None, short=None,
                 workspace=None):
    """Sequences go from seq_lens to new_lens positions (0: freed): pages behind the new
    lengths are given back, a shared page that would be written is copied, new pages are
    taken, lowest free ids first.  Returns (refcount_out, table_out, short [1]); short > 0:
    that many pages were missing and nothing changed.  Both outputs may be the inputs."""
    lib = _lib or load()
    c, dev, _, n_pages, _, _ = _paged_cache(k_pages, v_pages, True)
    P, T = (n_pages,), page_table.shape
    if len(T) != 2:
        raise ValueError("page_table must be [B, max_pages]")
    B, W = T
    if (B | W) > _INT_MAX:
        _c_ints(sequences=B, max_pages=W)
    refcount_out, ro = _out_ints(refcount_out, P, dev, "refcount_out", refcount)
    table_out, to = _out_ints(table_out, T, dev, "table_out", refcount)
    short, sh = _out_ints(short, (1,), dev, "short", refcount)
    workspace = alloc_pages_workspace(n_pages, B, W, k_pages.device) if workspace is None else workspace
    _launch(lib.ne_pages_resize, dev, c, _ints(refcount, P, dev, "refcount"),
            _ints(page_table, T, dev, "page_table"), _ints(seq_lens, (B,), dev, "seq_lens"),
            _ints(new_lens, (B,), dev, "new_lens"), ro, to, sh, B, W,
            *_ws(workspace, dev))
    return refcount_out, table_out, short


def pages_compact(refcount, page_table, k_pages, v_pages, refcount_out=None, table_out=None, remap=None, n_live=None,
                  workspace=None):
    """Moves the live pages of the pool into 0 .. n_live - 1.  Returns (refcount_out,
    table_out, remap [P]: new id of every live page, -1 for free ones, n_live [1]).  Both
    outputs may be the inputs; further tables go through remap."""
    lib = _lib or load()
    c, dev, _, n_pages, _, _ = _paged_cache(k_pages, v_pages, True)
    P, T = (n_pages,), page_table.shape
    if len(T) != 2:
        raise ValueError("page_table must be [B, max_pages]")
    B, W = T
    if (B | W) > _INT_MAX:
        _c_ints(sequences=B, max_pages=W)
    refcount_out, ro = _out_ints(refcount_out, P, dev, "refcount_out", refcount)
    table_out, to = _out_ints(table_out, T, dev, "table_out", refcount)
    remap, rm = _out_ints(remap, P, dev, "remap", refcount)
    n_live, nl = _out_ints(n_live, (1,), dev, "n_live", refcount)
    workspace = alloc_pages_workspace(n_pages, B, W, k_pages.device) if workspace is None else workspace
    _launch(lib.ne_pages_compact, dev, c, _ints(refcount, P, dev, "refcount"),
            _ints(page_table, T, dev, "page_table"), ro, to, rm, nl, B, W,
            *_ws(workspace, dev))
    return refcount_out, table_out, remap, n_live


def get_device_error(device=None) -> int:
    """Synchronise the current stream and return (and clear) the device error status."""
    lib = load()
    s = torch.cuda.current_stream(device).cuda_stream
    return int(lib.ne_get_device_error(ctypes.c_void_p(s)))


def set_wait_timeout_ms(ms: int):
    load().ne_set_wait_timeout_ms(int(ms))


def selftest_wait_timeout(timeout_ms: int = 50):
    lib = load()
    _check(lib.ne_selftest_wait_timeout(int(timeout_ms), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)))


PHASES = ("attn_fwd", "bwd_pre", "attn_bwd", "bwd_post")


def profile_enable(on: bool = True):
    """Diagnostic: record CUDA events around every kernel the calls launch."""
    load().ne_profile_enable(1 if on else 0)


def profile_totals() -> dict:
    """{phase: (total_ms, launches)} since profile_enable(True); synchronises."""
    lib = load()
    ms = (ctypes.c_double * 4)()
    n = (ctypes.c_int * 4)()
    _check(lib.ne_profile_totals(ms, n))
    return {PHASES[i]: (float(ms[i]), int(n[i])) for i in range(4)}


def last_error() -> str:
    return load().ne_last_error().decode()


def shutdown():
    load().ne_shutdown()
