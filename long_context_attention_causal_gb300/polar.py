"""Thin Python binding of libpolarattn.so (the C ABI in include/polar_attn.h).

Argument marshalling only: torch tensors provide device memory and the
current CUDA stream; every step of the computation runs in the library's
CUDA kernels.  There is no fallback: if the library is missing or the
device is not an sm_103 GPU, the calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpolarattn.so")

POLAR_F32 = 0
POLAR_BF16 = 1

_lib = None
_lock = threading.Lock()


class PolarError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = ""
        if status == 5:
            try:
                detail = " - " + lib().polar_attn_last_error().decode()
            except Exception:
                pass
        super().__init__(f"{where}: status {status} ({strerror(status)}){detail}")


class Consts(ctypes.Structure):
    """polar_consts_t: log_t0, kappa, sigma_k, eps (fp32), floor_order."""
    _fields_ = [("log_t0", ctypes.c_float), ("kappa", ctypes.c_float),
                ("sigma_k", ctypes.c_float), ("eps", ctypes.c_float),
                ("floor_order", ctypes.c_int)]


def default_consts(floor_order: int = 1) -> Consts:
    return Consts(math.log(2048.0), math.log(2048.0), 1.0, 1e-6, floor_order)


def lib() -> ctypes.CDLL:
    """Load libpolarattn.so (build it first with __graft_entry__.build())."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(
                    f"{LIB_PATH} is missing: build the CUDA library first "
                    "(python -c 'import __graft_entry__ as g; g.build()')")
            L = ctypes.CDLL(LIB_PATH)
            vp, fp = ctypes.c_void_p, ctypes.POINTER(ctypes.c_float)
            ci, cs = ctypes.c_int, ctypes.c_size_t
            cp = ctypes.POINTER(Consts)
            L.polar_attn_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, ci, ci,
                                         ci, ci, ci, cp, vp]
            L.polar_attn_decode.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, ci,
                                            ci, ci, ci, ci, cp, ci, vp, cs, vp]
            L.polar_attn_combine.argtypes = [vp, ci, vp, vp, vp, vp, vp, vp, ci,
                                             ci, ci, ci, ci, cp, vp]
            L.polar_attn_decode_workspace_bytes.argtypes = [ci, ci, ci, ci, ci]
            L.polar_attn_decode_workspace_bytes.restype = cs
            L.polar_attn_decode_num_splits.argtypes = [ci, ci, ci, ci]
            L.polar_attn_strerror.argtypes = [ci]
            L.polar_attn_strerror.restype = ctypes.c_char_p
            L.polar_attn_device_status.argtypes = [ci]
            L.polar_attn_selftest_wait_timeout.argtypes = [ci, vp]
            L.polar_attn_default_consts.argtypes = [cp]
            L.polar_attn_decode_static_scratch.argtypes = [
                vp, vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, cp, ci, vp]
            L.polar_attn_decode_static_scratch.restype = ci
            L.polar_attn_decode_paged.argtypes = [
                vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, ci, ci,
                ci, cp, ci, vp, cs, vp]
            L.polar_attn_decode_paged.restype = ci
            L.polar_attn_decode_paged_num_splits.argtypes = [ci, ci, ci, ci]
            L.polar_attn_decode_paged_num_splits.restype = ci
            L.polar_attn_decode_paged_workspace_bytes.argtypes = [ci, ci, ci, ci, ci, ci]
            L.polar_attn_decode_paged_workspace_bytes.restype = cs
            L.polar_memory_step.argtypes = [vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci,
                                            ci, ctypes.c_float, vp]
            L.polar_memory_step.restype = ci
            L.polar_attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, ci, ci, ci,
                                         ci, ci, cp, vp, cs, vp]
            L.polar_attn_bwd.restype = ci
            L.polar_attn_fwd_stats.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, ci, ci,
                                               ci, ci, ci, cp, vp]
            L.polar_attn_fwd_stats.restype = ci
            L.polar_attn_bwd_stats.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                               vp, vp, vp, ci, ci, ci, ci, ci, cp, vp, cs, vp]
            L.polar_attn_bwd_stats.restype = ci
            L.polar_attn_bwd_workspace_bytes.argtypes = [ci, ci, ci, ci]
            L.polar_attn_bwd_workspace_bytes.restype = cs
            L.polar_attn_fwd_host.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, ci, ci, ci,
                                              ci, ci, cp, ci, vp, cs, vp]
            L.polar_attn_fwd_host.restype = ci
            L.polar_attn_fwd_host_workspace_bytes.argtypes = [ci, ci, ci, ci, ci]
            L.polar_attn_fwd_host_workspace_bytes.restype = cs
            cf = ctypes.c_float
            L.polar_linear_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci,
                                           cf, vp, cs, vp]
            L.polar_linear_step.argtypes = [vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, cf, vp]
            L.polar_linear_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ci,
                                           ci, ci, ci, ci, cf, vp, cs, vp]
            for f in ("polar_linear_workspace_bytes", "polar_linear_bwd_workspace_bytes"):
                getattr(L, f).argtypes = [ci, ci, ci, ci, ci]
                getattr(L, f).restype = cs
            L.polar_attn_decode_paged_weights.argtypes = [
                vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, ci, ci, ci,
                ci, cp, ci, vp, cs, vp]
            L.polar_attn_decode_paged_weights_workspace_bytes.argtypes = [ci, ci, ci, ci, ci, ci]
            L.polar_attn_decode_paged_weights_workspace_bytes.restype = cs
            L.polar_attn_decode_paged_weights_num_splits.argtypes = [ci, ci, ci, ci]
            L.polar_attn_decode_paged_weights_num_splits.restype = ci
            L.polar_cache_evict.argtypes = [vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci,
                                            ci, ci, ci, ci, ci, vp, cs, vp]
            L.polar_cache_evict_workspace_bytes.argtypes = [ci, ci, ci, ci]
            L.polar_cache_evict_workspace_bytes.restype = cs
            L.polar_attn_last_error.argtypes = []
            L.polar_attn_last_error.restype = ctypes.c_char_p
            for f in ("polar_attn_fwd", "polar_attn_decode", "polar_attn_combine",
                      "polar_attn_decode_num_splits", "polar_attn_device_status",
                      "polar_attn_selftest_wait_timeout", "polar_attn_version",
                      "polar_attn_default_consts", "polar_linear_fwd", "polar_linear_step",
                      "polar_linear_bwd", "polar_attn_decode_paged_weights",
                      "polar_cache_evict"):
                getattr(L, f).restype = ci
            _lib = L
    return _lib


def strerror(status: int) -> str:
    try:
        return lib().polar_attn_strerror(int(status)).decode()
    except ImportError:
        return "library not loaded"


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return POLAR_F32
    if t.dtype == torch.bfloat16:
        return POLAR_BF16
    raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _dev(t, name, dtype=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def _shape(t, name, shape):
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")


def _dec_outputs(q, out, n_eff, conf, bh):
    _dev(out, "out", q.dtype)
    _dev(n_eff, "n_eff", torch.float32)
    _dev(conf, "conf", torch.float32)
    _shape(out, "out", q.shape)
    _shape(n_eff, "n_eff", bh)
    _shape(conf, "conf", bh)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(st, where):
    if st != 0:
        raise PolarError(st, where)


def fwd(q, k, v, mem, w_count, out=None, n_eff=None, conf=None, consts=None,
        want_conf=False, stream=None):
    """Causal prefill: q, k, v, mem [B, H, T, d] (bf16 or fp32, same dtype),
    w_count [H, d] fp32.  Returns (out, n_eff, conf or None)."""
    _dev(q, "q")
    dt = q.dtype
    for name, t in (("k", k), ("v", v), ("mem", mem)):
        _dev(t, name, dt)
    _dev(w_count, "w_count", torch.float32)
    B, H, T, d = q.shape
    if k.shape != q.shape or v.shape != q.shape or mem.shape != q.shape:
        raise ValueError("q, k, v, mem must share the shape [B, H, T, d]")
    if tuple(w_count.shape) != (H, d):
        raise ValueError("w_count must be [H, d]")
    if out is None:
        out = torch.empty_like(q)
    if n_eff is None:
        n_eff = torch.empty((B, H, T), device=q.device, dtype=torch.float32)
    if conf is None and want_conf:
        conf = torch.empty((B, H, T), device=q.device, dtype=torch.float32)
    _dev(out, "out", dt)
    _dev(n_eff, "n_eff", torch.float32)
    _dev(conf, "conf", torch.float32)
    _shape(out, "out", q.shape)
    _shape(n_eff, "n_eff", (B, H, T))
    _shape(conf, "conf", (B, H, T))
    c = consts or default_consts()
    st = lib().polar_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(mem), _ptr(w_count),
                              _ptr(out), _ptr(n_eff), _ptr(conf), B, H, T, d,
                              _dtype_code(q), ctypes.byref(c), _stream(stream))
    _check(st, "polar_attn_fwd")
    return out, n_eff, conf


def fwd_stats(q, k, v, mem, w_count, consts=None, stream=None):
    """Causal prefill (bf16) that also keeps the backward's row statistics.
    Returns (out, n_eff, conf, stats [B, H, T, 2] = logsumexp, |a|)."""
    _dev(q, "q", torch.bfloat16)
    for name, t in (("k", k), ("v", v), ("mem", mem)):
        _dev(t, name, torch.bfloat16)
    _dev(w_count, "w_count", torch.float32)
    if q.dim() != 4:
        raise ValueError("q must be [B, H, T, d]")
    B, H, T, d = q.shape
    for name, t in (("k", k), ("v", v), ("mem", mem)):
        _shape(t, name, q.shape)
    _shape(w_count, "w_count", (H, d))
    out = torch.empty_like(q)
    n_eff = torch.empty((B, H, T), device=q.device, dtype=torch.float32)
    conf = torch.empty_like(n_eff)
    stats = torch.empty((B, H, T, 2), device=q.device, dtype=torch.float32)
    c = consts or default_consts()
    st = lib().polar_attn_fwd_stats(_ptr(q), _ptr(k), _ptr(v), _ptr(mem), _ptr(w_count),
                                    _ptr(out), _ptr(n_eff), _ptr(conf), _ptr(stats), B, H, T,
                                    d, _dtype_code(q), ctypes.byref(c), _stream(stream))
    _check(st, "polar_attn_fwd_stats")
    return out, n_eff, conf, stats


def _host(t, name, dtype=None):
    if not isinstance(t, torch.Tensor) or t.device.type != "cpu":
        raise TypeError(f"{name} must be a CPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def fwd_host_workspace_bytes(B, H, T, d, dtype=torch.bfloat16) -> int:
    code = 1 if dtype == torch.bfloat16 else 0
    return int(lib().polar_attn_fwd_host_workspace_bytes(B, H, T, d, code))


def fwd_host(q, k, v, mem, w_count, out=None, n_eff=None, conf=None, want_conf=False,
             num_pieces=0, workspace=None, consts=None, stream=None, synchronize=True):
    """Causal prefill from host (CPU) tensors: copies in, kernels and copies
    out overlap piece by piece inside the library.  Pinned tensors
    (pin_memory()) let the copies run asynchronously.  workspace: a CUDA
    uint8 tensor of fwd_host_workspace_bytes(...) bytes (allocated here if
    None).  With synchronize=False the CPU outputs are valid only after the
    stream has been synchronised.  Returns (out, n_eff, conf or None) on the
    CPU."""
    _host(q, "q")
    dt = q.dtype
    if dt not in (torch.bfloat16, torch.float32):
        raise TypeError("q must be bf16 or fp32")
    for name, t in (("k", k), ("v", v), ("mem", mem)):
        _host(t, name, dt)
    _host(w_count, "w_count", torch.float32)
    if q.dim() != 4:
        raise ValueError("q must be [B, H, T, d]")
    B, H, T, d = q.shape
    for name, t in (("k", k), ("v", v), ("mem", mem)):
        _shape(t, name, q.shape)
    _shape(w_count, "w_count", (H, d))
    pin = q.is_pinned()
    if out is None:
        out = torch.empty(q.shape, dtype=dt, pin_memory=pin)
    if n_eff is None:
        n_eff = torch.empty((B, H, T), dtype=torch.float32, pin_memory=pin)
    if conf is None and want_conf:
        conf = torch.empty((B, H, T), dtype=torch.float32, pin_memory=pin)
    _host(out, "out", dt)
    _host(n_eff, "n_eff", torch.float32)
    _shape(out, "out", q.shape)
    _shape(n_eff, "n_eff", (B, H, T))
    if conf is not None:
        _host(conf, "conf", torch.float32)
        _shape(conf, "conf", (B, H, T))
    need = fwd_host_workspace_bytes(B, H, T, d, dt)
    if workspace is None:
        workspace = torch.empty(max(need, 256), device="cuda", dtype=torch.uint8)
    _dev(workspace, "workspace", torch.uint8)
    c = consts or default_consts()
    st = lib().polar_attn_fwd_host(
        _ptr(q), _ptr(k), _ptr(v), _ptr(mem), _ptr(w_count), _ptr(out), _ptr(n_eff),
        _ptr(conf), B, H, T, d, _dtype_code(q), ctypes.byref(c), int(num_pieces),
        _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "polar_attn_fwd_host")
    if synchronize:
        (stream or torch.cuda.current_stream()).synchronize()
    return out, n_eff, conf


def decode_num_splits(B, H, Tkv, d) -> int:
    return int(lib().polar_attn_decode_num_splits(B, H, Tkv, d))


def decode_workspace_bytes(B, H, Tkv, d, num_splits=0) -> int:
    return int(lib().polar_attn_decode_workspace_bytes(B, H, Tkv, d, num_splits))


def decode(q, k_cache, v_cache, mem, w_count, num_splits=0, workspace=None,
           out=None, n_eff=None, conf=None, consts=None, want_conf=False,
           stream=None):
    """Split-KV decode: q, mem [B, H, d]; k_cache, v_cache [B, H, Tkv, d];
    w_count [H, d] fp32.  workspace: a CUDA uint8 tensor (allocated here if
    None).  Returns (out, n_eff, conf or None)."""
    _dev(q, "q")
    dt = q.dtype
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache), ("mem", mem)):
        _dev(t, name, dt)
    _dev(w_count, "w_count", torch.float32)
    B, H, Tkv, d = k_cache.shape
    if tuple(q.shape) != (B, H, d) or tuple(mem.shape) != (B, H, d):
        raise ValueError("q and mem must be [B, H, d]")
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must share a shape")
    _shape(w_count, "w_count", (H, d))
    need = decode_workspace_bytes(B, H, Tkv, d, num_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=q.device, dtype=torch.uint8)
    _dev(workspace, "workspace")
    if out is None:
        out = torch.empty_like(q)
    if n_eff is None:
        n_eff = torch.empty((B, H), device=q.device, dtype=torch.float32)
    if conf is None and want_conf:
        conf = torch.empty((B, H), device=q.device, dtype=torch.float32)
    _dec_outputs(q, out, n_eff, conf, (B, H))
    c = consts or default_consts()
    st = lib().polar_attn_decode(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(mem), _ptr(w_count), _ptr(out),
        _ptr(n_eff), _ptr(conf), B, H, Tkv, d, _dtype_code(q), ctypes.byref(c),
        int(num_splits), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream))
    _check(st, "polar_attn_decode")
    return out, n_eff, conf


def decode_static_scratch(q, k_cache, v_cache, mem, w_count, num_splits=0,
                          out=None, n_eff=None, conf=None, consts=None,
                          want_conf=False, stream=None):
    """Split-KV decode that allocates nothing: the split partials live in
    the library's fixed device array (see polar_attn_decode_static_scratch).
    For callers that cannot allocate device memory when they decode.  Calls
    that overlap on the GPU share that array and must be serialised."""
    _dev(q, "q")
    dt = q.dtype
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache), ("mem", mem)):
        _dev(t, name, dt)
    _dev(w_count, "w_count", torch.float32)
    B, H, Tkv, d = k_cache.shape
    if tuple(q.shape) != (B, H, d) or tuple(mem.shape) != (B, H, d):
        raise ValueError("q and mem must be [B, H, d]")
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must share a shape")
    _shape(w_count, "w_count", (H, d))
    if out is None:
        out = torch.empty_like(q)
    if n_eff is None:
        n_eff = torch.empty((B, H), device=q.device, dtype=torch.float32)
    if conf is None and want_conf:
        conf = torch.empty((B, H), device=q.device, dtype=torch.float32)
    _dec_outputs(q, out, n_eff, conf, (B, H))
    c = consts or default_consts()
    st = lib().polar_attn_decode_static_scratch(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(mem), _ptr(w_count), _ptr(out),
        _ptr(n_eff), _ptr(conf), B, H, Tkv, d, _dtype_code(q), ctypes.byref(c),
        int(num_splits), _stream(stream))
    if st == 4:
        raise PolarError(st, "polar_attn_decode_static_scratch: "
                         + lib().polar_attn_last_error().decode())
    _check(st, "polar_attn_decode_static_scratch")
    return out, n_eff, conf


def decode_paged_workspace_bytes(B, Hq, Hkv, max_seq_len, d, num_splits=0) -> int:
    return int(lib().polar_attn_decode_paged_workspace_bytes(B, Hq, Hkv, max_seq_len, d,
                                                             num_splits))


def decode_paged(q, k_pages, v_pages, block_table, seq_lens, mem, w_count,
                 max_seq_len=None, num_splits=0, workspace=None, out=None, n_eff=None,
                 conf=None, consts=None, want_conf=False, stream=None):
    """Decode against a paged cache with grouped-query heads.

    q, mem [B, Hq, d]; k_pages, v_pages [num_pages, Hkv, page, d];
    block_table [B, max_pages] int32; seq_lens [B] int32 (device);
    w_count [Hq, d] fp32.  max_seq_len bounds seq_lens (default: the
    table's capacity max_pages * page).  Returns (out, n_eff, conf)."""
    _dev(q, "q")
    dt = q.dtype
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages), ("mem", mem)):
        _dev(t, name, dt)
    _dev(block_table, "block_table", torch.int32)
    _dev(seq_lens, "seq_lens", torch.int32)
    _dev(w_count, "w_count", torch.float32)
    B, Hq, d = q.shape
    num_pages, Hkv, page, d2 = k_pages.shape
    if d2 != d or v_pages.shape != k_pages.shape or tuple(mem.shape) != (B, Hq, d):
        raise ValueError("shape mismatch between q, mem and the pages")
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_pages]")
    _shape(seq_lens, "seq_lens", (B,))
    _shape(w_count, "w_count", (Hq, d))
    max_pages = block_table.shape[1]
    if max_seq_len is None:
        max_seq_len = max_pages * page
    need = decode_paged_workspace_bytes(B, Hq, Hkv, max_seq_len, d, num_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=q.device, dtype=torch.uint8)
    if out is None:
        out = torch.empty_like(q)
    if n_eff is None:
        n_eff = torch.empty((B, Hq), device=q.device, dtype=torch.float32)
    if conf is None and want_conf:
        conf = torch.empty((B, Hq), device=q.device, dtype=torch.float32)
    _dec_outputs(q, out, n_eff, conf, (B, Hq))
    c = consts or default_consts()
    st = lib().polar_attn_decode_paged(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(block_table), _ptr(seq_lens),
        _ptr(mem), _ptr(w_count), _ptr(out), _ptr(n_eff), _ptr(conf), B, Hq, Hkv, d,
        page, num_pages, max_pages, int(max_seq_len), _dtype_code(q), ctypes.byref(c),
        int(num_splits), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream))
    _check(st, "polar_attn_decode_paged")
    return out, n_eff, conf


def memory_step(state, q, k, v, alpha, beta, mem=None, eps=1e-6, stream=None):
    """Gated-delta memory over T tokens, state updated in place.

    state [B, H, d, d] fp32 (modified); q, k, v [B, H, T, d] (bf16 or fp32);
    alpha, beta [B, H, T] fp32.  Returns mem [B, H, T, d] (the memory
    stream)."""
    _dev(state, "state", torch.float32)
    _dev(q, "q")
    for name, t in (("k", k), ("v", v)):
        _dev(t, name, q.dtype)
    _dev(alpha, "alpha", torch.float32)
    _dev(beta, "beta", torch.float32)
    B, H, T, d = q.shape
    if tuple(state.shape) != (B, H, d, d) or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("state [B,H,d,d] and q, k, v [B,H,T,d] shapes disagree")
    if tuple(alpha.shape) != (B, H, T) or tuple(beta.shape) != (B, H, T):
        raise ValueError("alpha and beta must be [B, H, T]")
    if mem is None:
        mem = torch.empty_like(q)
    _dev(mem, "mem", q.dtype)
    st = lib().polar_memory_step(_ptr(state), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                                 _ptr(beta), _ptr(mem), B, H, T, d, _dtype_code(q),
                                 float(eps), _stream(stream))
    _check(st, "polar_memory_step")
    return mem


# The calls below are made once a token and layer, where the host's time
# counts: an argument is checked in one expression, and only one that fails
# goes through the checks that name what is wrong.

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _fail(t, name, dtype, shape, dev):
    _dev(t, name, dtype)
    _shape(t, name, shape)
    raise ValueError(f"{name} must be on cuda:{dev}, like the first tensor, got {t.device}")


def _in(t, name, dtype, shape, dev):
    """Address of a tensor argument after its checks (0 for None)."""
    if t is None:
        return 0
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == dev and t.is_contiguous()):
        _fail(t, name, dtype, shape, dev)
    return t.data_ptr()


def _need(t, name):
    if t is None:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t


def _call(dev, where, f, *args):
    """f(*args, stream) on `dev` and its current stream."""
    if _raw_stream is not None:
        raw = _raw_stream(dev)
    else:
        raw = torch.cuda.current_stream(dev).cuda_stream
    if dev == torch.cuda.current_device():
        st = f(*args, raw)
    else:
        with torch.cuda.device(dev):
            st = f(*args, raw)
    if st != 0:
        raise PolarError(st, where)


def _on_stream(f):
    """Adds the argument `stream`: the call, and what it allocates, belong to
    that stream then."""
    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        first = args[0] if args else next(iter(kw.values()), None)
        if isinstance(first, torch.Tensor) and first.is_cuda and first.device != stream.device:
            raise ValueError(f"the tensors are on {first.device}, the stream on {stream.device}")
        with torch.cuda.stream(stream):
            return f(*args, **kw)
    return call


@functools.lru_cache(maxsize=1024)
def _bytes(name, dev, *sizes):
    """Workspace bytes of a call on device `dev` (None: the current one)."""
    if dev is None or dev == torch.cuda.current_device():
        return int(getattr(lib(), name)(*sizes))
    with torch.cuda.device(dev):
        return int(getattr(lib(), name)(*sizes))


def _scratch(workspace, need, dev):
    """(address, bytes, tensor to keep) of the caller's workspace or a new one."""
    if workspace is None:
        workspace = torch.empty(need if need > 16 else 16, device=torch.device("cuda", dev),
                                dtype=torch.uint8)
        return workspace.data_ptr(), need, workspace
    _dev(workspace, "workspace")
    if workspace.get_device() != dev:
        raise ValueError(f"workspace must be on cuda:{dev}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def linear_workspace_bytes(B, H, T, d, dtype=torch.bfloat16) -> int:
    code = 1 if dtype == torch.bfloat16 else 0
    return int(lib().polar_linear_workspace_bytes(B, H, T, d, code))


def linear_bwd_workspace_bytes(B, H, T, d, dtype=torch.bfloat16) -> int:
    code = 1 if dtype == torch.bfloat16 else 0
    return int(lib().polar_linear_bwd_workspace_bytes(B, H, T, d, code))


@_on_stream
def linear_fwd(q, k, v, log_decay, state=None, lengths=None, scale=None, mem=None,
               state_out=None, want_state=False, workspace=None):
    """Decayed linear attention over a prompt (a memory stream whose decay is
    one number per head): q, k, v [B, H, T, d] (bf16 or fp32); log_decay [H]
    fp32, <= 0; state [B, H, d, d] fp32 or None (zero); lengths [B] int32 or
    None (all T): tokens of a padded batch.  scale defaults to d ** -0.5.
    Returns (mem [B, H, T, d], state after the last token or None); rows of
    mem past a length are zero.  state_out may be state."""
    _dev(_need(q, "q"), "q")
    if q.dim() != 4:
        raise ValueError("q must be [B, H, T, d]")
    B, H, T, d = shape = q.shape
    dt, dev, code = q.dtype, q.get_device(), _dtype_code(q)
    if mem is None:
        mem = torch.empty_like(q)
    square = (B, H, d, d)
    if state_out is None and want_state:
        state_out = torch.empty(square, device=q.device, dtype=torch.float32)
    f32 = torch.float32
    need = _bytes("polar_linear_workspace_bytes", dev, B, H, T, d, code)
    ws, size, _ = _scratch(workspace, need, dev) if need or workspace is not None else (0, 0, None)
    _call(dev, "polar_linear_fwd", lib().polar_linear_fwd, q.data_ptr(),
          _in(_need(k, "k"), "k", dt, shape, dev), _in(_need(v, "v"), "v", dt, shape, dev),
          _in(_need(log_decay, "log_decay"), "log_decay", f32, (H,), dev),
          _in(lengths, "lengths", torch.int32, (B,), dev), _in(state, "state", f32, square, dev),
          _in(mem, "mem", dt, shape, dev), _in(state_out, "state_out", f32, square, dev),
          B, H, T, d, code, d ** -0.5 if scale is None else float(scale), ws, size)
    return mem, state_out


@_on_stream
def linear_step(state, q, k, v, log_decay, scale=None, mem=None):
    """One token of the decayed linear attention, the state updated in place:
    state [B, H, d, d] fp32; q, k, v [B, H, d] (bf16 or fp32); log_decay [H]
    fp32.  Returns mem [B, H, d]."""
    _dev(_need(q, "q"), "q")
    if q.dim() != 3:
        raise ValueError("q must be [B, H, d]")
    B, H, d = shape = q.shape
    dt, dev = q.dtype, q.get_device()
    if mem is None:
        mem = torch.empty_like(q)
    _call(dev, "polar_linear_step", lib().polar_linear_step,
          _in(_need(state, "state"), "state", torch.float32, (B, H, d, d), dev), q.data_ptr(),
          _in(_need(k, "k"), "k", dt, shape, dev), _in(_need(v, "v"), "v", dt, shape, dev),
          _in(_need(log_decay, "log_decay"), "log_decay", torch.float32, (H,), dev),
          _in(mem, "mem", dt, shape, dev), B, H, d, _dtype_code(q),
          d ** -0.5 if scale is None else float(scale))
    return mem


@_on_stream
def linear_bwd(q, k, v, log_decay, dmem, state=None, dstate_out=None, lengths=None, scale=None,
               dq=None, dk=None, dv=None, dstate=None, want_dstate=False, workspace=None):
    """Gradients of linear_fwd: dmem [B, H, T, d] in q's type and dstate_out
    [B, H, d, d] fp32 (None: zero) are the gradients of its two results.
    Returns (dq, dk, dv in q's type, dstate fp32 or None).  The decay is a
    constant and gets none."""
    _dev(_need(q, "q"), "q")
    if q.dim() != 4:
        raise ValueError("q must be [B, H, T, d]")
    B, H, T, d = shape = q.shape
    dt, dev, code = q.dtype, q.get_device(), _dtype_code(q)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    square = (B, H, d, d)
    if dstate is None and want_dstate:
        dstate = torch.empty(square, device=q.device, dtype=torch.float32)
    f32 = torch.float32
    need = _bytes("polar_linear_bwd_workspace_bytes", dev, B, H, T, d, code)
    ws, size, _ = _scratch(workspace, need, dev) if need or workspace is not None else (0, 0, None)
    _call(dev, "polar_linear_bwd", lib().polar_linear_bwd, q.data_ptr(),
          _in(_need(k, "k"), "k", dt, shape, dev), _in(_need(v, "v"), "v", dt, shape, dev),
          _in(_need(log_decay, "log_decay"), "log_decay", f32, (H,), dev),
          _in(lengths, "lengths", torch.int32, (B,), dev), _in(state, "state", f32, square, dev),
          _in(_need(dmem, "dmem"), "dmem", dt, shape, dev),
          _in(dstate_out, "dstate_out", f32, square, dev), _in(dq, "dq", dt, shape, dev),
          _in(dk, "dk", dt, shape, dev), _in(dv, "dv", dt, shape, dev),
          _in(dstate, "dstate", f32, square, dev), B, H, T, d, code,
          d ** -0.5 if scale is None else float(scale), ws, size)
    return dq, dk, dv, dstate


def decode_paged_weights_workspace_bytes(B, Hq, Hkv, max_seq_len, d, num_splits=0) -> int:
    return int(lib().polar_attn_decode_paged_weights_workspace_bytes(B, Hq, Hkv, max_seq_len, d,
                                                                     num_splits))


def decode_paged_weights_num_splits(B, Hkv, max_seq_len, d) -> int:
    return int(lib().polar_attn_decode_paged_weights_num_splits(B, Hkv, max_seq_len, d))


_DEFAULT_CONSTS = default_consts()


@_on_stream
def decode_paged_weights(q, k_pages, v_pages, block_table, seq_lens, mem, w_count, weights,
                         max_seq_len=None, num_splits=0, workspace=None, out=None, n_eff=None,
                         conf=None, consts=None, want_conf=False):
    """decode_paged that also adds every cache row's attention weight, summed
    over the query heads of its group, to weights [B, Hkv, stride] fp32
    (stride >= max_seq_len).  max_seq_len defaults to the smaller of the
    table's capacity and the stride; the workspace holds one fp32 value per
    query head and row up to it, so with a generous table give the longest
    length.  Returns (out, n_eff, conf)."""
    for name, t in (("q", q), ("k_pages", k_pages), ("block_table", block_table),
                    ("weights", weights)):
        _dev(_need(t, name), name)
    if q.dim() != 3 or k_pages.dim() != 4 or block_table.dim() != 2 or weights.dim() != 3:
        raise ValueError("q must be [B, Hq, d], the pages [num_pages, Hkv, page, d], block_table "
                         "[B, max_pages], weights [B, Hkv, stride]")
    B, Hq, d = shape = q.shape
    num_pages, Hkv, page, _ = k_pages.shape
    max_pages, stride = block_table.shape[1], weights.shape[2]
    dt, dev, f32, i32 = q.dtype, q.get_device(), torch.float32, torch.int32
    if max_seq_len is None:
        max_seq_len = min(max_pages * page, stride)
    if out is None:
        out = torch.empty_like(q)
    if n_eff is None:
        n_eff = torch.empty((B, Hq), device=q.device, dtype=f32)
    if conf is None and want_conf:
        conf = torch.empty((B, Hq), device=q.device, dtype=f32)
    pages = (num_pages, Hkv, page, d)
    need = _bytes("polar_attn_decode_paged_weights_workspace_bytes", dev, B, Hq, Hkv,
                  int(max_seq_len), d, int(num_splits))
    ws, size, _ = _scratch(workspace, need, dev)
    c = _DEFAULT_CONSTS if consts is None else consts
    _call(dev, "polar_attn_decode_paged_weights", lib().polar_attn_decode_paged_weights,
          q.data_ptr(), _in(k_pages, "k_pages", dt, pages, dev),
          _in(_need(v_pages, "v_pages"), "v_pages", dt, pages, dev),
          _in(block_table, "block_table", i32, (B, max_pages), dev),
          _in(_need(seq_lens, "seq_lens"), "seq_lens", i32, (B,), dev),
          _in(_need(mem, "mem"), "mem", dt, shape, dev),
          _in(_need(w_count, "w_count"), "w_count", f32, (Hq, d), dev),
          _in(out, "out", dt, shape, dev), _in(n_eff, "n_eff", f32, (B, Hq), dev),
          _in(conf, "conf", f32, (B, Hq), dev),
          _in(weights, "weights", f32, (B, Hkv, stride), dev), stride, B, Hq, Hkv, d, page,
          num_pages, max_pages, int(max_seq_len), _dtype_code(q), ctypes.byref(c),
          int(num_splits), ws, size)
    return out, n_eff, conf


def cache_evict_workspace_bytes(B, Hkv, max_seq_len, keep) -> int:
    return int(lib().polar_cache_evict_workspace_bytes(B, Hkv, max_seq_len, keep))


@_on_stream
def cache_evict(k_pages, v_pages, block_table, seq_lens, weights, positions, keep, recent=0,
                max_seq_len=None, new_lens=None, workspace=None):
    """Cuts every sequence of more than `keep` rows to `keep`, per KV head and
    in place: the rows of the newest `recent` tokens stay, then those of
    largest accumulated weight.

    k_pages, v_pages [num_pages, Hkv, page, d]; block_table [B, max_pages]
    and seq_lens [B] int32; weights [B, Hkv, stride] fp32 and positions [B,
    Hkv, stride] int32 move with the rows.  Returns the new lengths [B] int32
    (written into new_lens when given, which may be seq_lens)."""
    for name, t in (("k_pages", k_pages), ("block_table", block_table), ("weights", weights)):
        _dev(_need(t, name), name)
    if k_pages.dim() != 4 or block_table.dim() != 2 or weights.dim() != 3:
        raise ValueError("the pages must be [num_pages, Hkv, page, d], block_table [B, "
                         "max_pages], weights [B, Hkv, stride]")
    num_pages, Hkv, page, d = pages = k_pages.shape
    B, max_pages = block_table.shape
    stride = weights.shape[2]
    dt, dev, i32 = k_pages.dtype, k_pages.get_device(), torch.int32
    if max_seq_len is None:
        max_seq_len = min(max_pages * page, stride)
    if new_lens is None:
        new_lens = torch.empty((B,), device=k_pages.device, dtype=i32)
    need = _bytes("polar_cache_evict_workspace_bytes", dev, B, Hkv, int(max_seq_len), int(keep))
    ws, size, _ = _scratch(workspace, need, dev)
    slots = (B, Hkv, stride)
    _call(dev, "polar_cache_evict", lib().polar_cache_evict, k_pages.data_ptr(),
          _in(_need(v_pages, "v_pages"), "v_pages", dt, pages, dev),
          _in(block_table, "block_table", i32, (B, max_pages), dev),
          _in(_need(seq_lens, "seq_lens"), "seq_lens", i32, (B,), dev),
          _in(weights, "weights", torch.float32, slots, dev),
          _in(_need(positions, "positions"), "positions", i32, slots, dev),
          _in(new_lens, "new_lens", i32, (B,), dev), B, Hkv, d, page, num_pages, max_pages,
          int(max_seq_len), stride, _dtype_code(k_pages), int(keep), int(recent), ws, size)
    return new_lens


def bwd_workspace_bytes(B, H, T, d) -> int:
    return int(lib().polar_attn_bwd_workspace_bytes(B, H, T, d))


def bwd(q, k, v, w_count, dout, consts=None, workspace=None, stream=None):
    """Gradients of the causal prefill output: returns (dq, dk, dv, dw_count)
    in fp32; d out / d mem is dout itself."""
    _dev(q, "q")
    for name, t in (("k", k), ("v", v), ("dout", dout)):
        _dev(t, name, q.dtype)
    _dev(w_count, "w_count", torch.float32)
    if q.dim() != 4:
        raise ValueError("q must be [B, H, T, d]")
    B, H, T, d = q.shape
    for name, t in (("k", k), ("v", v), ("dout", dout)):
        _shape(t, name, q.shape)
    _shape(w_count, "w_count", (H, d))
    dq = torch.empty(q.shape, device=q.device, dtype=torch.float32)
    dk = torch.empty_like(dq)
    dv = torch.empty_like(dq)
    dw = torch.empty((H, d), device=q.device, dtype=torch.float32)
    need = int(lib().polar_attn_bwd_workspace_bytes(B, H, T, d))
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=q.device, dtype=torch.uint8)
    c = consts or default_consts()
    st = lib().polar_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(w_count), _ptr(dout), _ptr(dq),
                              _ptr(dk), _ptr(dv), _ptr(dw), B, H, T, d, _dtype_code(q),
                              ctypes.byref(c), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "polar_attn_bwd")
    return dq, dk, dv, dw


def bwd_stats(q, k, v, mem, w_count, out, n_eff, conf, stats, dout, consts=None,
              workspace=None, stream=None, dq=None, dk=None, dv=None, dw=None):
    """Gradients (bf16) from the outputs of fwd_stats: returns (dq, dk, dv,
    dw_count) in fp32 (written into dq, dk, dv, dw when given); d out / d mem
    is dout itself."""
    _dev(q, "q", torch.bfloat16)
    for name, t in (("k", k), ("v", v), ("mem", mem), ("out", out), ("dout", dout)):
        _dev(t, name, torch.bfloat16)
    for name, t in (("w_count", w_count), ("n_eff", n_eff), ("conf", conf), ("stats", stats)):
        _dev(t, name, torch.float32)
    if q.dim() != 4:
        raise ValueError("q must be [B, H, T, d]")
    B, H, T, d = q.shape
    for name, t in (("k", k), ("v", v), ("mem", mem), ("out", out), ("dout", dout)):
        _shape(t, name, q.shape)
    _shape(w_count, "w_count", (H, d))
    _shape(n_eff, "n_eff", (B, H, T))
    _shape(conf, "conf", (B, H, T))
    _shape(stats, "stats", (B, H, T, 2))
    if dq is None:
        dq = torch.empty(q.shape, device=q.device, dtype=torch.float32)
    if dk is None:
        dk = torch.empty(q.shape, device=q.device, dtype=torch.float32)
    if dv is None:
        dv = torch.empty(q.shape, device=q.device, dtype=torch.float32)
    if dw is None:
        dw = torch.empty((H, d), device=q.device, dtype=torch.float32)
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv), ("dw", dw)):
        _dev(t, name, torch.float32)
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _shape(t, name, q.shape)
    _shape(dw, "dw", (H, d))
    need = int(lib().polar_attn_bwd_workspace_bytes(B, H, T, d))
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=q.device, dtype=torch.uint8)
    c = consts or default_consts()
    st = lib().polar_attn_bwd_stats(
        _ptr(q), _ptr(k), _ptr(v), _ptr(mem), _ptr(w_count), _ptr(out), _ptr(n_eff), _ptr(conf),
        _ptr(stats), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dw), B, H, T, d,
        _dtype_code(q), ctypes.byref(c), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "polar_attn_bwd_stats")
    return dq, dk, dv, dw


def combine(partials, q, mem, w_count, Tkv, out=None, n_eff=None, conf=None,
            consts=None, want_conf=False, stream=None):
    """Merge split partials [B, H, S, d + 4] fp32 and apply the epilogue."""
    _dev(partials, "partials", torch.float32)
    _dev(q, "q")
    _dev(mem, "mem", q.dtype)
    _dev(w_count, "w_count", torch.float32)
    if partials.dim() != 4:
        raise ValueError("partials must be [B, H, S, d + 4]")
    B, H, S, d4 = partials.shape
    d = d4 - 4
    _shape(q, "q", (B, H, d))
    _shape(mem, "mem", (B, H, d))
    _shape(w_count, "w_count", (H, d))
    if out is None:
        out = torch.empty_like(q)
    if n_eff is None:
        n_eff = torch.empty((B, H), device=q.device, dtype=torch.float32)
    if conf is None and want_conf:
        conf = torch.empty((B, H), device=q.device, dtype=torch.float32)
    _dec_outputs(q, out, n_eff, conf, (B, H))
    c = consts or default_consts()
    st = lib().polar_attn_combine(_ptr(partials), S, _ptr(q), _ptr(mem), _ptr(w_count),
                                  _ptr(out), _ptr(n_eff), _ptr(conf), B, H, int(Tkv), d,
                                  _dtype_code(q), ctypes.byref(c), _stream(stream))
    _check(st, "polar_attn_combine")
    return out, n_eff, conf


def device_status(reset: bool = False) -> int:
    """Kernel-side status word (0 = no wait ran out).  Synchronises."""
    return int(lib().polar_attn_device_status(1 if reset else 0))


def selftest_wait_timeout(limit_us: int = 1000, stream=None) -> None:
    _check(lib().polar_attn_selftest_wait_timeout(int(limit_us), _stream(stream)),
           "polar_attn_selftest_wait_timeout")


def version() -> int:
    return int(lib().polar_attn_version())
