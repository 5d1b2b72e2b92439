"""ctypes binding of libpolar_attn.so, the C ABI of include/polar_attn.h,
include/polar_gdelta.h and include/polar_cache.h.

Argument marshalling only: torch tensors supply device memory and streams, and
every step of the computation runs in the library's CUDA kernels.  There is no
CPU or PyTorch fallback; a missing or unloadable library raises at once.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpolar_attn.so")

POLAR_BF16, POLAR_FP32 = 0, 1
IMPLS = {"auto": 0, "simt": 1, "tc": 2}
STATUS = {0: "POLAR_OK", 1: "POLAR_ERR_INVALID_ARG", 2: "POLAR_ERR_UNSUPPORTED",
          3: "POLAR_ERR_WORKSPACE", 4: "POLAR_ERR_BAD_PAGE", 5: "POLAR_ERR_TIMEOUT",
          6: "POLAR_ERR_CUDA", 7: "POLAR_ERR_BAD_SEQLEN", 8: "POLAR_ERR_BAD_SLOT",
          9: "POLAR_ERR_NO_PAGES"}

# Every entry point that the headers under include/ declare.
EXPORTS = ["polar_attn_default_params", "polar_attn_fwd_workspace_size", "polar_attn_fwd",
           "polar_attn_fwd_ws",
           "polar_attn_fwd_staging_size",
           "polar_attn_fwd_host", "polar_attn_decode_workspace_size", "polar_attn_decode_paged",
           "polar_attn_decode_staging_size", "polar_attn_decode_paged_host",
           "polar_attn_get_status", "polar_attn_status_string", "polar_attn_launch_count",
           "polar_attn_decode_paged_noalloc", "polar_attn_selftest_exp2",
           "polar_attn_decode_chunk_workspace_size", "polar_attn_decode_paged_chunk",
           "polar_attn_bwd_workspace_size", "polar_attn_bwd",
           "polar_gdelta_prefill_workspace_size", "polar_gdelta_prefill", "polar_gdelta_step",
           "polar_attn_selftest_timeout", "polar_attn_selftest_decode_per_head",
           "polar_attn_fwd_state_size", "polar_attn_fwd_train", "polar_attn_bwd_from_state",
           "polar_attn_selftest_fwd_host_segments", "polar_attn_selftest_tree_copies",
           "polar_attn_decode_tree_workspace_size", "polar_attn_decode_paged_tree",
           "polar_attn_decode_sparse_workspace_size", "polar_attn_decode_paged_sparse",
           "polar_attn_cache_workspace_size", "polar_attn_cache_reserve",
           "polar_attn_cache_append", "polar_attn_cache_fork", "polar_attn_cache_free",
           "polar_attn_cache_compact"]


class PolarError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)} ({status_string(code)})")


class Params(ctypes.Structure):
    """polar_params_t."""
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("Hq", ctypes.c_int),
                ("Hkv", ctypes.c_int), ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int),
                ("logit_scale", ctypes.c_float), ("alpha", ctypes.c_float),
                ("L_train", ctypes.c_int), ("beta", ctypes.c_float), ("causal", ctypes.c_int),
                ("impl", ctypes.c_int), ("window", ctypes.c_int)]


class GdeltaParams(ctypes.Structure):
    """polar_gdelta_params_t."""
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int), ("zero_init", ctypes.c_int),
                ("accumulate", ctypes.c_int)]


class Cache(ctypes.Structure):
    """polar_cache_t."""
    _fields_ = [("kv_pages", ctypes.c_void_p), ("bounds", ctypes.c_void_p),
                ("refs", ctypes.c_void_p), ("num_pages", ctypes.c_int), ("Hkv", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int)]


_lib = None
_lock = threading.Lock()


def lib() -> ctypes.CDLL:
    """Loads libpolar_attn.so (build it with ``python -m polar_attention_b200.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build the CUDA library with "
                                   "`python -m polar_attention_b200.build` (no fallback exists)")
            L = ctypes.CDLL(LIB_PATH)
            P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
            PP = ctypes.POINTER(Params)
            L.polar_attn_default_params.argtypes = [PP, I, I, I, I, I]
            L.polar_attn_default_params.restype = None
            L.polar_attn_fwd_workspace_size.argtypes = [PP]
            L.polar_attn_fwd_workspace_size.restype = Z
            L.polar_attn_fwd.argtypes = [P, P, P, P, PP, P, P, P]
            L.polar_attn_fwd_ws.argtypes = [P, P, P, P, PP, P, P, P, Z, P]
            L.polar_attn_bwd_workspace_size.argtypes = [PP]
            L.polar_attn_bwd_workspace_size.restype = Z
            L.polar_attn_bwd.argtypes = [P, P, P, P, P, PP, P, P, P, P, P, Z, P]
            L.polar_attn_fwd_state_size.argtypes = [PP]
            L.polar_attn_fwd_state_size.restype = Z
            L.polar_attn_fwd_train.argtypes = [P, P, P, P, PP, P, P, P, P]
            L.polar_attn_bwd_from_state.argtypes = [P, P, P, P, P, P, P, PP, P, P, P, P, P, Z, P]
            L.polar_attn_fwd_staging_size.argtypes = [PP]
            L.polar_attn_fwd_staging_size.restype = Z
            L.polar_attn_fwd_host.argtypes = [P, P, P, P, PP, P, P, P, Z, P]
            L.polar_attn_decode_workspace_size.argtypes = [I, I, PP]
            L.polar_attn_decode_workspace_size.restype = Z
            L.polar_attn_decode_paged.argtypes = [P, P, I, P, I, P, I, P, PP, P, P, P, Z, P]
            L.polar_attn_decode_chunk_workspace_size.argtypes = [I, I, I, PP]
            L.polar_attn_decode_chunk_workspace_size.restype = Z
            L.polar_attn_decode_paged_chunk.argtypes = [P, P, I, P, I, P, I, I, P, PP, P, P, P, Z, P]
            L.polar_attn_decode_staging_size.argtypes = [I, I, PP]
            L.polar_attn_decode_staging_size.restype = Z
            L.polar_attn_decode_paged_host.argtypes = [P, P, I, P, I, P, I, P, PP, P, P, P, Z, P]
            L.polar_attn_decode_paged_noalloc.argtypes = [P, P, I, P, I, P, I, P, PP, P, P, P]
            L.polar_attn_selftest_exp2.argtypes = [P, P, P, I, P]
            L.polar_attn_selftest_timeout.argtypes = [P]
            L.polar_attn_selftest_decode_per_head.argtypes = [P, P, I, P, I, P, I, P, PP, P, P, P,
                                                              Z, P]
            IP = ctypes.POINTER(ctypes.c_int)
            L.polar_attn_selftest_fwd_host_segments.argtypes = [I, IP, IP, I]
            L.polar_attn_selftest_fwd_host_segments.restype = I
            L.polar_attn_selftest_tree_copies.argtypes = [IP, I, I, IP]
            L.polar_attn_selftest_tree_copies.restype = I
            GP = ctypes.POINTER(GdeltaParams)
            L.polar_gdelta_prefill_workspace_size.argtypes = [GP]
            L.polar_gdelta_prefill_workspace_size.restype = Z
            L.polar_gdelta_prefill.argtypes = [P, P, P, P, P, P, GP, P, P, Z, P]
            L.polar_gdelta_step.argtypes = [P, P, P, P, P, P, I, P, I, GP, P, P]
            CP = ctypes.POINTER(Cache)
            L.polar_attn_decode_tree_workspace_size.argtypes = [I, I, I, PP]
            L.polar_attn_decode_tree_workspace_size.restype = Z
            L.polar_attn_decode_paged_tree.argtypes = [P, P, P, P, P, I, P, I, P, I, P, I, P, PP,
                                                       P, P, P, Z, P]
            L.polar_attn_decode_sparse_workspace_size.argtypes = [I, I, I, PP]
            L.polar_attn_decode_sparse_workspace_size.restype = Z
            L.polar_attn_decode_paged_sparse.argtypes = [P, P, P, I, P, I, P, I, I, P, PP, P, P, P,
                                                         P, Z, P]
            L.polar_attn_cache_workspace_size.argtypes = [CP, I]
            L.polar_attn_cache_workspace_size.restype = Z
            L.polar_attn_cache_reserve.argtypes = [CP, P, I, P, P, I, P, P, Z, P]
            L.polar_attn_cache_append.argtypes = [CP, P, P, I, P, I, P, P, I, P, I, P]
            L.polar_attn_cache_fork.argtypes = [CP, P, P, I, P, I, P, P, I, P]
            L.polar_attn_cache_free.argtypes = [CP, P, I, P, P, I, P]
            L.polar_attn_cache_compact.argtypes = [CP, P, I, P, I, P, P, Z, P]
            L.polar_attn_get_status.argtypes = [P]
            L.polar_attn_status_string.argtypes = [I]
            L.polar_attn_status_string.restype = ctypes.c_char_p
            L.polar_attn_launch_count.restype = ctypes.c_uint64
            for name in ("polar_attn_fwd", "polar_attn_fwd_ws", "polar_attn_fwd_host", "polar_attn_decode_paged",
                         "polar_attn_decode_paged_host", "polar_attn_get_status",
                         "polar_attn_decode_paged_noalloc", "polar_attn_selftest_exp2",
                         "polar_attn_decode_paged_chunk", "polar_attn_bwd",
                         "polar_gdelta_prefill", "polar_gdelta_step",
                         "polar_attn_selftest_timeout", "polar_attn_selftest_decode_per_head",
                         "polar_attn_fwd_train", "polar_attn_bwd_from_state",
                         "polar_attn_decode_paged_tree", "polar_attn_decode_paged_sparse",
                         "polar_attn_cache_reserve", "polar_attn_cache_append",
                         "polar_attn_cache_fork", "polar_attn_cache_free",
                         "polar_attn_cache_compact"):
                getattr(L, name).restype = I
            _lib = L
    return _lib


def fwd_host_segments(T: int, cap: int = 64):
    """The row segments polar_attn_fwd_host sends for a tensor-core prefill of
    T rows, in order: a list of (lo, hi) (host logic; no device work)."""
    lo = (ctypes.c_int * max(cap, 1))()
    hi = (ctypes.c_int * max(cap, 1))()
    n = lib().polar_attn_selftest_fwd_host_segments(int(T), lo, hi, int(cap))
    if n < 0:
        raise ValueError(f"polar_attn_selftest_fwd_host_segments: bad arguments (T={T}, cap={cap})")
    return [(lo[i], hi[i]) for i in range(n)]


def tree_copies(steps, fail_at: int = -1):
    """The copying thread of the drafted trees' tensor-core kernel on counters, for
    tiles of these numbers of steps, with its wait number fail_at running out
    (host logic; no device work).  Returns (barriers left before their last copy
    has landed, waits on the way)."""
    waits = ctypes.c_int()
    n = lib().polar_attn_selftest_tree_copies((ctypes.c_int * max(len(steps), 1))(*steps),
                                              len(steps), int(fail_at), ctypes.byref(waits))
    if n < 0:
        raise ValueError(f"polar_attn_selftest_tree_copies: bad arguments (steps={steps})")
    return n, waits.value


def status_string(code: int) -> str:
    try:
        return lib().polar_attn_status_string(int(code)).decode()
    except Exception:  # the library may be what failed
        return "?"


def make_params(B=0, T=0, Hq=16, Hkv=4, dtype=POLAR_BF16, s=8.0, alpha=0.3, L=2048, beta=1.0,
                impl="auto", window=0) -> Params:
    p = Params()
    lib().polar_attn_default_params(ctypes.byref(p), B, T, Hq, Hkv, dtype)
    p.logit_scale, p.alpha, p.L_train, p.beta = s, alpha, L, beta
    p.window = int(window)
    p.impl = IMPLS[impl] if isinstance(impl, str) else int(impl)
    return p


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return POLAR_BF16
    if t.dtype == torch.float32:
        return POLAR_FP32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(code: int, where: str):
    if code != 0:
        raise PolarError(code, where)


def fwd_workspace_size(B: int, T: int, Hq: int, Hkv: int) -> int:
    p = make_params(B, T, Hq, Hkv, POLAR_BF16)
    return int(lib().polar_attn_fwd_workspace_size(ctypes.byref(p)))


def fwd(q, k, v, u, out=None, neff=None, workspace=None, *, s=8.0, alpha=0.3, L=2048, beta=1.0,
        impl="auto", stream=None, want_neff=True, moments=True, window=0):
    """Causal prefill.  q [B,T,Hq,64], k/v [B,T,Hkv,64] (bf16 or fp32, CUDA,
    contiguous), u [Hq,64] fp32.  Returns (out [B,T,Hq,64], neff [B,Hq,T]).
    moments=True calls polar_attn_fwd_ws with a workspace for the key-moment
    pre-pass (allocated here when `workspace` is None); moments=False calls
    polar_attn_fwd, which takes none."""
    B, T, Hq, D = q.shape
    Hkv = k.shape[2]
    for t in (q, k, v, u):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("inputs must be contiguous CUDA tensors")
    if u.dtype != torch.float32:
        raise TypeError("u must be float32")
    if out is None:
        out = torch.empty_like(q)
    if neff is None and want_neff:
        neff = torch.empty((B, Hq, T), device=q.device, dtype=torch.float32)
    p = make_params(B, T, Hq, Hkv, _dt(q), s, alpha, L, beta, impl, window)
    p.head_dim = D
    if not moments:
        _check(lib().polar_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(u), ctypes.byref(p),
                                    _ptr(out), _ptr(neff), _stream(stream)), "polar_attn_fwd")
        return out, neff
    ws_bytes = int(lib().polar_attn_fwd_workspace_size(ctypes.byref(p)))
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), device=q.device, dtype=torch.uint8)
    else:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().polar_attn_fwd_ws(_ptr(q), _ptr(k), _ptr(v), _ptr(u), ctypes.byref(p),
                                   _ptr(out), _ptr(neff), _ptr(workspace), ws_bytes,
                                   _stream(stream)), "polar_attn_fwd_ws")
    return out, neff


def bwd_workspace_size(B: int, T: int, Hq: int, Hkv: int) -> int:
    p = make_params(B, T, Hq, Hkv, POLAR_BF16)
    return int(lib().polar_attn_bwd_workspace_size(ctypes.byref(p)))


def bwd(q, k, v, u, dout, dq=None, dk=None, dv=None, du=None, workspace=None, *, s=8.0,
        alpha=0.3, L=2048, beta=1.0, window=0, stream=None):
    """Backward of the causal prefill.  q, dout [B,T,Hq,64] and k, v [B,T,Hkv,64]
    (bf16 or fp32, CUDA, contiguous), u [Hq,64] fp32.  Returns fp32
    (dq, dk, dv, du) shaped like q, k, v, u."""
    B, T, Hq, D = q.shape
    Hkv = k.shape[2]
    for t in (q, k, v, u, dout):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("inputs must be contiguous CUDA tensors")
    if dout.dtype != q.dtype:
        raise TypeError("dout must have the dtype of q")
    p = make_params(B, T, Hq, Hkv, _dt(q), s, alpha, L, beta, "auto", window)
    p.head_dim = D
    f32 = torch.float32
    dq = torch.empty(q.shape, device=q.device, dtype=f32) if dq is None else dq
    dk = torch.empty(k.shape, device=q.device, dtype=f32) if dk is None else dk
    dv = torch.empty(v.shape, device=q.device, dtype=f32) if dv is None else dv
    du = torch.empty(u.shape, device=q.device, dtype=f32) if du is None else du
    need = int(lib().polar_attn_bwd_workspace_size(ctypes.byref(p)))
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=q.device, dtype=torch.uint8)
    _check(lib().polar_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(u), _ptr(dout), ctypes.byref(p),
                                _ptr(dq), _ptr(dk), _ptr(dv), _ptr(du), _ptr(workspace),
                                workspace.numel(), _stream(stream)), "polar_attn_bwd")
    return dq, dk, dv, du


def fwd_state_size(B: int, T: int, Hq: int, Hkv: int) -> int:
    p = make_params(B, T, Hq, Hkv, POLAR_BF16)
    return int(lib().polar_attn_fwd_state_size(ctypes.byref(p)))


def fwd_train(q, k, v, u, out=None, neff=None, state=None, *, s=8.0, alpha=0.3, L=2048, beta=1.0,
              impl="auto", window=0, stream=None, want_neff=True):
    """Training forward: as fwd, plus each row's saved state for
    bwd_from_state.  Returns (out, neff, state); state is a float32
    [B, Hq, T, 8] tensor (left untouched where the state path does not
    apply)."""
    B, T, Hq, D = q.shape
    Hkv = k.shape[2]
    for t in (q, k, v, u):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("inputs must be contiguous CUDA tensors")
    if u.dtype != torch.float32:
        raise TypeError("u must be float32")
    if out is None:
        out = torch.empty_like(q)
    if neff is None and want_neff:
        neff = torch.empty((B, Hq, T), device=q.device, dtype=torch.float32)
    if state is None:
        state = torch.empty((B, Hq, T, 8), device=q.device, dtype=torch.float32)
    p = make_params(B, T, Hq, Hkv, _dt(q), s, alpha, L, beta, impl, window)
    p.head_dim = D
    _check(lib().polar_attn_fwd_train(_ptr(q), _ptr(k), _ptr(v), _ptr(u), ctypes.byref(p),
                                      _ptr(out), _ptr(neff), _ptr(state), _stream(stream)),
           "polar_attn_fwd_train")
    return out, neff, state


def bwd_from_state(q, k, v, u, out, state, dout, dq=None, dk=None, dv=None, du=None,
                   workspace=None, *, s=8.0, alpha=0.3, L=2048, beta=1.0, impl="auto", window=0,
                   stream=None):
    """Backward from a training forward's out and saved state (fwd_train with
    the same arguments).  Returns fp32 (dq, dk, dv, du) as bwd."""
    B, T, Hq, D = q.shape
    Hkv = k.shape[2]
    for t in (q, k, v, u, out, state, dout):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("inputs must be contiguous CUDA tensors")
    if dout.dtype != q.dtype or out.dtype != q.dtype:
        raise TypeError("out and dout must have the dtype of q")
    p = make_params(B, T, Hq, Hkv, _dt(q), s, alpha, L, beta, impl, window)
    p.head_dim = D
    f32 = torch.float32
    dq = torch.empty(q.shape, device=q.device, dtype=f32) if dq is None else dq
    dk = torch.empty(k.shape, device=q.device, dtype=f32) if dk is None else dk
    dv = torch.empty(v.shape, device=q.device, dtype=f32) if dv is None else dv
    du = torch.empty(u.shape, device=q.device, dtype=f32) if du is None else du
    need = int(lib().polar_attn_bwd_workspace_size(ctypes.byref(p)))
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=q.device, dtype=torch.uint8)
    _check(lib().polar_attn_bwd_from_state(_ptr(q), _ptr(k), _ptr(v), _ptr(u), _ptr(out),
                                           _ptr(state), _ptr(dout), ctypes.byref(p), _ptr(dq),
                                           _ptr(dk), _ptr(dv), _ptr(du), _ptr(workspace),
                                           workspace.numel(), _stream(stream)),
           "polar_attn_bwd_from_state")
    return dq, dk, dv, du


def decode_workspace_size(num_seqs: int, max_pages: int, Hq: int, Hkv: int) -> int:
    p = make_params(0, 0, Hq, Hkv, POLAR_BF16)
    return int(lib().polar_attn_decode_workspace_size(num_seqs, max_pages, ctypes.byref(p)))


def decode_paged(q, kv_pages, page_table, seqlens, u, out=None, neff=None, workspace=None, *,
                 s=8.0, alpha=0.3, L=2048, beta=1.0, stream=None, want_neff=True, window=0):
    """Paged GQA decode.  q [N,Hq,64] bf16; kv_pages [P,2,Hkv,64,64] bf16;
    page_table [N,max_pages] int32; seqlens [N] int32; u [Hq,64] fp32.
    Returns (out [N,Hq,64], neff [N,Hq])."""
    N, Hq, D = q.shape
    P_, _, Hkv, _, _ = kv_pages.shape
    max_pages = page_table.shape[1]
    if page_table.dtype != torch.int32 or seqlens.dtype != torch.int32:
        raise TypeError("page_table and seqlens must be int32")
    p = make_params(0, 0, Hq, Hkv, _dt(q), s, alpha, L, beta, window=window)
    p.head_dim = D
    ws_need = int(lib().polar_attn_decode_workspace_size(N, max_pages, ctypes.byref(p)))
    if workspace is None:
        workspace = torch.empty(max(ws_need, 16), device=q.device, dtype=torch.uint8)
    if out is None:
        out = torch.empty_like(q)
    if neff is None and want_neff:
        neff = torch.empty((N, Hq), device=q.device, dtype=torch.float32)
    _check(lib().polar_attn_decode_paged(
        _ptr(q), _ptr(kv_pages), P_, _ptr(page_table), max_pages, _ptr(seqlens), N, _ptr(u),
        ctypes.byref(p), _ptr(out), _ptr(neff), _ptr(workspace), workspace.numel(),
        _stream(stream)), "polar_attn_decode_paged")
    return out, neff


def decode_chunk_workspace_size(num_seqs: int, max_pages: int, chunk: int, Hq: int,
                                Hkv: int) -> int:
    p = make_params(0, 0, Hq, Hkv, POLAR_BF16)
    return int(lib().polar_attn_decode_chunk_workspace_size(num_seqs, max_pages, chunk,
                                                            ctypes.byref(p)))


def decode_paged_chunk(q, kv_pages, page_table, seqlens, u, out=None, neff=None, workspace=None,
                       *, s=8.0, alpha=0.3, L=2048, beta=1.0, stream=None, want_neff=True,
                       window=0):
    """Multi-token paged decode.  q [N,C,Hq,64] bf16: token t of sequence n is
    the query at cache position seqlens[n] - C + t.  Returns (out [N,C,Hq,64],
    neff [N,C,Hq])."""
    N, C, Hq, D = q.shape
    P_, _, Hkv, _, _ = kv_pages.shape
    max_pages = page_table.shape[1]
    if page_table.dtype != torch.int32 or seqlens.dtype != torch.int32:
        raise TypeError("page_table and seqlens must be int32")
    p = make_params(0, 0, Hq, Hkv, _dt(q), s, alpha, L, beta, window=window)
    p.head_dim = D
    ws_need = int(lib().polar_attn_decode_chunk_workspace_size(N, max_pages, C, ctypes.byref(p)))
    if workspace is None:
        workspace = torch.empty(max(ws_need, 16), device=q.device, dtype=torch.uint8)
    if out is None:
        out = torch.empty_like(q)
    if neff is None and want_neff:
        neff = torch.empty((N, C, Hq), device=q.device, dtype=torch.float32)
    _check(lib().polar_attn_decode_paged_chunk(
        _ptr(q), _ptr(kv_pages), P_, _ptr(page_table), max_pages, _ptr(seqlens), N, C, _ptr(u),
        ctypes.byref(p), _ptr(out), _ptr(neff), _ptr(workspace), workspace.numel(),
        _stream(stream)), "polar_attn_decode_paged_chunk")
    return out, neff


# Bytes of the fixed device scratch behind decode_paged_noalloc (POLAR_NOALLOC_SCRATCH_BYTES).
NOALLOC_SCRATCH_BYTES = 16 << 20


def decode_paged_noalloc(q, kv_pages, page_table, seqlens, u, out, neff=None, *, s=8.0,
                         alpha=0.3, L=2048, beta=1.0, stream=None, window=0):
    """polar_attn_decode_paged_noalloc: the paged decode with no workspace, for
    callers that cannot allocate device memory.  out (and neff, if given) must
    be preallocated by the caller; this wrapper allocates nothing."""
    N, Hq, D = q.shape
    P_, _, Hkv, _, _ = kv_pages.shape
    p = make_params(0, 0, Hq, Hkv, _dt(q), s, alpha, L, beta, window=window)
    p.head_dim = D
    _check(lib().polar_attn_decode_paged_noalloc(
        _ptr(q), _ptr(kv_pages), P_, _ptr(page_table), page_table.shape[1], _ptr(seqlens), N,
        _ptr(u), ctypes.byref(p), _ptr(out), _ptr(neff), _stream(stream)),
        "polar_attn_decode_paged_noalloc")
    return out, neff


def fwd_staging_size(B, T, Hq, Hkv, dtype=POLAR_BF16) -> int:
    p = make_params(B, T, Hq, Hkv, dtype)
    return int(lib().polar_attn_fwd_staging_size(ctypes.byref(p)))


def fwd_host(q_h, k_h, v_h, u_h, out_h, neff_h, staging, *, s=8.0, alpha=0.3, L=2048, beta=1.0,
             impl="auto", stream=None, window=0):
    """polar_attn_fwd_host on (pinned) host tensors; staging is a CUDA uint8
    tensor of at least fwd_staging_size bytes.  Synchronises the stream."""
    B, T, Hq, D = q_h.shape
    p = make_params(B, T, Hq, k_h.shape[2], _dt(q_h), s, alpha, L, beta, impl, window)
    p.head_dim = D
    _check(lib().polar_attn_fwd_host(_ptr(q_h), _ptr(k_h), _ptr(v_h), _ptr(u_h), ctypes.byref(p),
                                     _ptr(out_h), _ptr(neff_h), _ptr(staging), staging.numel(),
                                     _stream(stream)), "polar_attn_fwd_host")


def decode_staging_size(num_seqs, max_pages, Hq, Hkv) -> int:
    p = make_params(0, 0, Hq, Hkv, POLAR_BF16)
    return int(lib().polar_attn_decode_staging_size(num_seqs, max_pages, ctypes.byref(p)))


def decode_paged_host(q_h, kv_pages, page_table_h, seqlens_h, u_h, out_h, neff_h, staging, *,
                      s=8.0, alpha=0.3, L=2048, beta=1.0, stream=None, window=0):
    """polar_attn_decode_paged_host: per-step inputs and outputs in (pinned)
    host memory, the KV pool resident on the device.  Synchronises the stream."""
    N, Hq, D = q_h.shape
    P_, _, Hkv, _, _ = kv_pages.shape
    p = make_params(0, 0, Hq, Hkv, _dt(q_h), s, alpha, L, beta, window=window)
    p.head_dim = D
    _check(lib().polar_attn_decode_paged_host(
        _ptr(q_h), _ptr(kv_pages), P_, _ptr(page_table_h), page_table_h.shape[1], _ptr(seqlens_h),
        N, _ptr(u_h), ctypes.byref(p), _ptr(out_h), _ptr(neff_h), _ptr(staging), staging.numel(),
        _stream(stream)), "polar_attn_decode_paged_host")


def selftest_exp2(x, stream=None):
    """The prefill kernel's FMA-pipe 2^x and MUFU ex2.approx on a CUDA fp32
    tensor x (even length).  Returns (poly, mufu)."""
    poly, mufu = torch.empty_like(x), torch.empty_like(x)
    _check(lib().polar_attn_selftest_exp2(_ptr(x), _ptr(poly), _ptr(mufu), x.numel(),
                                          _stream(stream)), "polar_attn_selftest_exp2")
    return poly, mufu


def _gd_params(B, T, H, dtype, zero_init, accumulate) -> GdeltaParams:
    return GdeltaParams(int(B), int(T), int(H), 64, int(dtype), int(bool(zero_init)),
                        int(bool(accumulate)))


def gdelta_workspace_size(B: int, T: int, H: int) -> int:
    p = _gd_params(B, T, H, POLAR_BF16, 0, 0)
    return int(lib().polar_gdelta_prefill_workspace_size(ctypes.byref(p)))


def gdelta_prefill(q, k, v, alpha, beta, state=None, out=None, workspace=None, *,
                   accumulate=False, stream=None):
    """Memory channel over whole sequences.  q, k, v [B,T,H,64] (bf16 or fp32,
    CUDA, contiguous), alpha, beta [B,T,H] fp32.  ``state`` [B,H,64,64] fp32 is
    updated in place (S_0 in, final state out); None starts from zero and
    returns a fresh final-state tensor.  With accumulate, ``out`` (required)
    gets the memory read added to it.  Returns (out, state)."""
    B, T, H, D = q.shape
    for t in (q, k, v, alpha, beta):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("inputs must be contiguous CUDA tensors")
    zero_init = state is None
    if state is None:
        state = torch.empty((B, H, D, D), device=q.device, dtype=torch.float32)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs the output tensor to add into")
        out = torch.empty_like(q)
    p = _gd_params(B, T, H, _dt(q), zero_init, accumulate)
    p.head_dim = D
    need = int(lib().polar_gdelta_prefill_workspace_size(ctypes.byref(p)))
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=q.device, dtype=torch.uint8)
    _check(lib().polar_gdelta_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                      _ptr(state), ctypes.byref(p), _ptr(out), _ptr(workspace),
                                      workspace.numel(), _stream(stream)), "polar_gdelta_prefill")
    return out, state


def gdelta_step(q, k, v, alpha, beta, state_pool, slots, out=None, *, accumulate=False,
                stream=None):
    """One decode token per sequence with the states updated in place in their
    pool slots.  q, k, v [N,H,64]; alpha, beta [N,H] fp32; state_pool
    [num_slots,H,64,64] fp32; slots [N] int32 (negative: skip).  Returns out."""
    N, H, D = q.shape
    for t in (q, k, v, alpha, beta, state_pool, slots):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("inputs must be contiguous CUDA tensors")
    if slots.dtype != torch.int32:
        raise TypeError("slots must be int32")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs the output tensor to add into")
        out = torch.empty_like(q)
    p = _gd_params(0, 0, H, _dt(q), 0, accumulate)
    p.head_dim = D
    _check(lib().polar_gdelta_step(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                   _ptr(state_pool), state_pool.shape[0], _ptr(slots), N,
                                   ctypes.byref(p), _ptr(out), _stream(stream)),
           "polar_gdelta_step")
    return out


@functools.lru_cache(maxsize=64)
def _decode_params(Hq, Hkv, D, dtype, s, alpha, L, beta):
    """A polar_params_t of these values, and its pointer; never changed after."""
    p = make_params(0, 0, Hq, Hkv, dtype, s, alpha, L, beta)
    p.head_dim = D
    return p, ctypes.pointer(p)


def _current(dev):
    """Whether this is the current CUDA device's index."""
    return dev >= 0 and dev == torch._C._cuda_getDevice()


class _Scope:
    """The device of `tensor` and `stream` (None: the device's current stream)
    made current: what a call in it allocates belongs to that device and
    stream."""
    __slots__ = ("tensor", "given", "stack")

    def __init__(self, tensor, stream):
        self.tensor, self.given, self.stack = tensor, stream, None

    def __enter__(self):
        index = self.tensor.get_device()
        if index < 0:
            raise ValueError("inputs must be contiguous CUDA tensors")
        if self.given is not None and self.given.device.index != index:
            raise ValueError(f"stream of {self.given.device} for tensors on cuda:{index}")
        self.stack = [torch.cuda.device(index)]
        if self.given is not None:
            self.stack.append(torch.cuda.stream(self.given))
        for c in self.stack:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self.stack):
            c.__exit__(*exc)


def _need(name, t, dtype, shape, dev):
    """t's address, once it is a contiguous tensor of this type and shape on the
    CUDA device of this index."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on cuda:{dev}, the others' device")
    raise ValueError(f"{name} must have the shape {shape}, not {tuple(t.shape)}")


def _scratch(workspace, need, dev):
    """The workspace, its address and its size; a fresh one of `need` bytes where
    the caller gave none."""
    if workspace is None:
        need = max(need, 16)
        workspace = torch.empty(need, device=dev, dtype=torch.uint8)
        return workspace, workspace.data_ptr(), need
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _pool_shape(kv_pages, D):
    if kv_pages.dim() != 5 or kv_pages.shape[1] != 2 or tuple(kv_pages.shape[3:]) != (64, D):
        raise ValueError(f"kv_pages must be [pages, 2, Hkv, 64, {D}], not {tuple(kv_pages.shape)}")
    return kv_pages.shape[0], kv_pages.shape[2]


@functools.lru_cache(maxsize=64)
def _untouched(dev, need):
    """A workspace that no kernel reads or writes: one for all calls."""
    return torch.empty(need, device=dev, dtype=torch.uint8)


@functools.lru_cache(maxsize=256)
def decode_tree_workspace_size(num_seqs: int, max_pages: int, tree: int, Hq: int, Hkv: int) -> int:
    _, pp = _decode_params(Hq, Hkv, 64, POLAR_BF16, 8.0, 0.3, 2048, 1.0)
    return int(lib().polar_attn_decode_tree_workspace_size(num_seqs, max_pages, tree, pp))


def decode_paged_tree(q, k, v, tree_mask, kv_pages, page_table, seqlens, u, out=None, neff=None,
                      workspace=None, *, tree_lens=None, s=8.0, alpha=0.3, L=2048, beta=1.0,
                      stream=None, want_neff=True):
    """Decode for a tree of drafted tokens.  q [N,M,Hq,64], k and v [N,M,Hkv,64]
    bf16: the drafted nodes, which are not in the cache; tree_mask [N,M] int64:
    bit j of word t: node t sees node j; tree_lens [N] int32 (None: M nodes
    each); kv_pages, page_table, u as decode_paged; seqlens [N] int32: cached
    tokens, 0 and up.  Returns (out [N,M,Hq,64], neff [N,M,Hq]); rows at or past
    a sequence's nodes are left as they are (unset where out is allocated
    here)."""
    N, M, Hq, D = q.shape
    P_, Hkv = _pool_shape(kv_pages, D)
    bf16, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    max_pages = page_table.shape[1]
    dev = q.get_device()
    if stream is not None or not _current(dev):
        with _Scope(q, stream):
            return decode_paged_tree(q, k, v, tree_mask, kv_pages, page_table, seqlens, u, out,
                                     neff, workspace, tree_lens=tree_lens, s=s, alpha=alpha, L=L,
                                     beta=beta, want_neff=want_neff)
    st = torch._C._cuda_getCurrentRawStream(dev)
    ptr = (_need("q", q, bf16, (N, M, Hq, D), dev), _need("k", k, bf16, (N, M, Hkv, D), dev),
           _need("v", v, bf16, (N, M, Hkv, D), dev),
           _need("tree_mask", tree_mask, torch.int64, (N, M), dev),
           None if tree_lens is None else _need("tree_lens", tree_lens, i32, (N,), dev), M,
           _need("kv_pages", kv_pages, bf16, (P_, 2, Hkv, 64, D), dev), P_,
           _need("page_table", page_table, i32, (N, max_pages), dev), max_pages,
           _need("seqlens", seqlens, i32, (N,), dev), N, _need("u", u, f32, (Hq, D), dev))
    _, pp = _decode_params(Hq, Hkv, D, POLAR_BF16, s, alpha, L, beta)
    if out is None:
        out = torch.empty_like(q)
    if neff is None and want_neff:
        neff = torch.empty((N, M, Hq), device=dev, dtype=f32)
    need = decode_tree_workspace_size(N, max_pages, M, Hq, Hkv)
    if workspace is None and need == 16:  # nothing is split
        workspace = _untouched(dev, need)
    workspace, wp, wb = _scratch(workspace, need, dev)
    _check(lib().polar_attn_decode_paged_tree(
        *ptr, pp, _need("out", out, bf16, (N, M, Hq, D), dev),
        None if neff is None else _need("neff", neff, f32, (N, M, Hq), dev), wp, wb, st),
        "polar_attn_decode_paged_tree")
    return out, neff


@functools.lru_cache(maxsize=256)
def decode_sparse_workspace_size(num_seqs: int, max_pages: int, keep: int, Hq: int,
                                 Hkv: int) -> int:
    _, pp = _decode_params(Hq, Hkv, 64, POLAR_BF16, 8.0, 0.3, 2048, 1.0)
    return int(lib().polar_attn_decode_sparse_workspace_size(num_seqs, max_pages, keep, pp))


def decode_paged_sparse(q, kv_pages, bounds, page_table, seqlens, u, keep, out=None, neff=None,
                        selected=None, workspace=None, *, s=8.0, alpha=0.3, L=2048, beta=1.0,
                        stream=None, want_neff=True, want_selected=True):
    """Decode over at most `keep` pages per (sequence, kv head), chosen by a
    score on the pages' key bounds [P,Hkv,2,64] bf16 (smallest and largest key;
    cache_append keeps them).  A row is that of a sequence of the selected pages
    alone: their number of positions is n in the length temperature and the null
    floor (include/polar_attn.h says how far that is from the whole sequence's
    row).  Other arguments as decode_paged.  Returns (out
    [N,Hq,64], neff [N,Hq], selected [N,Hkv,keep] int32: the logical pages
    read, ascending, then -1)."""
    N, Hq, D = q.shape
    P_, Hkv = _pool_shape(kv_pages, D)
    keep = int(keep)
    bf16, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    max_pages = page_table.shape[1]
    dev = q.get_device()
    if stream is not None or not _current(dev):
        with _Scope(q, stream):
            return decode_paged_sparse(q, kv_pages, bounds, page_table, seqlens, u, keep, out, neff,
                                       selected, workspace, s=s, alpha=alpha, L=L, beta=beta,
                                       want_neff=want_neff, want_selected=want_selected)
    st = torch._C._cuda_getCurrentRawStream(dev)
    ptr = (_need("q", q, bf16, (N, Hq, D), dev),
           _need("kv_pages", kv_pages, bf16, (P_, 2, Hkv, 64, D), dev),
           _need("bounds", bounds, bf16, (P_, Hkv, 2, D), dev), P_,
           _need("page_table", page_table, i32, (N, max_pages), dev), max_pages,
           _need("seqlens", seqlens, i32, (N,), dev), N, keep,
           _need("u", u, f32, (Hq, D), dev))
    _, pp = _decode_params(Hq, Hkv, D, POLAR_BF16, s, alpha, L, beta)
    if out is None:
        out = torch.empty_like(q)
    if neff is None and want_neff:
        neff = torch.empty((N, Hq), device=dev, dtype=f32)
    if selected is None and want_selected:
        selected = torch.empty((N, Hkv, max(keep, 0)), device=dev, dtype=i32)
    need = decode_sparse_workspace_size(N, max_pages, keep, Hq, Hkv)
    if workspace is None and selected is not None and need <= (N * Hkv * keep * 4 + 15) // 16 * 16:
        workspace = _untouched(dev, max(need, 16))  # of the list alone, which `selected` takes
    workspace, wp, wb = _scratch(workspace, need, dev)
    _check(lib().polar_attn_decode_paged_sparse(
        *ptr, pp, _need("out", out, bf16, (N, Hq, D), dev),
        None if neff is None else _need("neff", neff, f32, (N, Hq), dev),
        None if selected is None else _need("selected", selected, i32, (N, Hkv, keep), dev), wp,
        wb, st), "polar_attn_decode_paged_sparse")
    return out, neff, selected


class PageCache:
    """A paged KV cache: the pool kv_pages [P,2,Hkv,64,64] bf16, the references
    refs [P] int32 (page-table entries that name a page; 0: free; None for a
    caller with an allocator of its own, who then only appends) and the pages'
    key bounds [P,Hkv,2,64] bf16 (None: not kept).  Holds the tensors, whose
    contents may change but which stay the same three: another pool, or a smaller
    one after a compaction, is another PageCache.  Page tables and lengths are
    arguments of each call."""
    __slots__ = ("_tensors", "_c", "_p", "_dev", "_pages", "_heads")

    def __init__(self, kv_pages, refs=None, bounds=None):
        P_, Hkv = _pool_shape(kv_pages, 64)
        dev, bf16 = kv_pages.get_device(), torch.bfloat16
        if dev < 0:
            raise ValueError("inputs must be contiguous CUDA tensors")
        self._tensors = (kv_pages, refs, bounds)
        self._c = Cache(
            _need("kv_pages", kv_pages, bf16, (P_, 2, Hkv, 64, 64), dev),
            None if bounds is None else _need("bounds", bounds, bf16, (P_, Hkv, 2, 64), dev),
            None if refs is None else _need("refs", refs, torch.int32, (P_,), dev), P_, Hkv, 64,
            POLAR_BF16)
        self._p, self._dev, self._pages, self._heads = ctypes.byref(self._c), dev, P_, Hkv

    # Read only: the calls use the addresses that were checked above.
    kv_pages = property(lambda self: self._tensors[0])
    refs = property(lambda self: self._tensors[1])
    bounds = property(lambda self: self._tensors[2])


@functools.lru_cache(maxsize=256)
def _cache_workspace(num_pages, Hkv, num_seqs):
    c = Cache(None, None, None, num_pages, Hkv, 64, POLAR_BF16)
    return int(lib().polar_attn_cache_workspace_size(ctypes.byref(c), num_seqs))


def cache_workspace_size(cache: PageCache, num_seqs: int) -> int:
    return _cache_workspace(cache._pages, cache._heads, num_seqs)


def _rows(cache, page_table, seqlens):
    """(addresses and sizes of a page table and its lengths), rows, pages a row."""
    dev, i32 = cache._dev, torch.int32
    N, max_pages = page_table.shape
    return (_need("page_table", page_table, i32, (N, max_pages), dev),
            _need("seqlens", seqlens, i32, (N,), dev), N, max_pages)


def cache_reserve(cache: PageCache, page_table, seqlens, grow, granted=None, workspace=None, *,
                  stream=None):
    """Room for grow [N] int32 more tokens in each row: takes free pages (and
    copies a shared last page) and grows page_table [N,max_pages] and seqlens
    [N] (int32) in place.  Returns granted [N] int32: grow, or 0 from the first
    row on that the pool cannot serve."""
    dev, i32 = cache._dev, torch.int32
    if stream is not None or not _current(dev):
        with _Scope(cache.kv_pages, stream):
            return cache_reserve(cache, page_table, seqlens, grow, granted, workspace)
    st = torch._C._cuda_getCurrentRawStream(dev)
    table, lens, N, max_pages = _rows(cache, page_table, seqlens)
    g = _need("grow", grow, i32, (N,), dev)
    if granted is None:
        granted = torch.empty_like(grow)
    workspace, wp, wb = _scratch(
        workspace, _cache_workspace(cache._pages, cache._heads, N), dev)
    _check(lib().polar_attn_cache_reserve(cache._p, table, max_pages, lens, g, N,
                                          _need("granted", granted, i32, (N,), dev), wp, wb,
                                          st), "polar_attn_cache_reserve")
    return granted


def cache_append(cache: PageCache, k, v, page_table, seqlens, counts=None, pick=None, *,
                 stream=None):
    """Writes the newest tokens of each row: token t < counts[n] (None: all) of
    row n, from k, v [N,T,Hkv,64] row t (pick [N,C] int32: row pick[n,t]), to
    position seqlens[n] - counts[n] + t; the touched pages' bounds are kept."""
    dev, bf16, i32 = cache._dev, torch.bfloat16, torch.int32
    if stream is not None or not _current(dev):
        with _Scope(cache.kv_pages, stream):
            return cache_append(cache, k, v, page_table, seqlens, counts, pick)
    st = torch._C._cuda_getCurrentRawStream(dev)
    table, lens, N, max_pages = _rows(cache, page_table, seqlens)
    if k.dim() != 4:
        raise ValueError(f"k must be [N, T, Hkv, 64], not {tuple(k.shape)}")
    T, Hkv = k.shape[1], cache._heads
    C = T if pick is None else pick.shape[1]
    _check(lib().polar_attn_cache_append(
        cache._p, _need("k", k, bf16, (N, T, Hkv, 64), dev),
        _need("v", v, bf16, (N, T, Hkv, 64), dev), T,
        None if pick is None else _need("pick", pick, i32, (N, C), dev), C,
        None if counts is None else _need("counts", counts, i32, (N,), dev), table, max_pages,
        lens, N, st), "polar_attn_cache_append")


def cache_fork(cache: PageCache, src_table, src_lens, src_rows, dst_table, dst_lens, *,
               stream=None):
    """Row i of dst_table, dst_lens becomes a copy of row src_rows[i] (int32) of
    src_table, src_lens that shares its pages; a negative source leaves the row
    alone.  The two tables may not overlap."""
    dev, i32 = cache._dev, torch.int32
    if stream is not None or not _current(dev):
        with _Scope(cache.kv_pages, stream):
            return cache_fork(cache, src_table, src_lens, src_rows, dst_table, dst_lens)
    st = torch._C._cuda_getCurrentRawStream(dev)
    src, slens, S, width = _rows(cache, src_table, src_lens)
    dst, dlens, N, max_pages = _rows(cache, dst_table, dst_lens)
    if width != max_pages:
        raise ValueError("src_table and dst_table must be equally wide")
    _check(lib().polar_attn_cache_fork(cache._p, src, slens, S,
                                       _need("src_rows", src_rows, i32, (N,), dev), N, dst,
                                       dlens, max_pages, st), "polar_attn_cache_fork")


def cache_free(cache: PageCache, page_table, seqlens, keep=None, *, stream=None):
    """Cuts each row to its first keep [N] int32 tokens (None: none; negative:
    the row is left alone) and gives the pages behind them back, in place."""
    dev = cache._dev
    if stream is not None or not _current(dev):
        with _Scope(cache.kv_pages, stream):
            return cache_free(cache, page_table, seqlens, keep)
    st = torch._C._cuda_getCurrentRawStream(dev)
    table, lens, N, max_pages = _rows(cache, page_table, seqlens)
    _check(lib().polar_attn_cache_free(
        cache._p, table, max_pages, lens,
        None if keep is None else _need("keep", keep, torch.int32, (N,), dev), N, st),
        "polar_attn_cache_free")


def cache_compact(cache: PageCache, page_table, seqlens, used=None, workspace=None, *,
                  stream=None):
    """Moves the live pages to the front of the pool and rewrites page_table (all
    rows that name pages of this pool) in place.  Returns used [1] int32: the
    number of live pages, which are pages 0 .. used - 1 afterwards."""
    dev, i32 = cache._dev, torch.int32
    if stream is not None or not _current(dev):
        with _Scope(cache.kv_pages, stream):
            return cache_compact(cache, page_table, seqlens, used, workspace)
    st = torch._C._cuda_getCurrentRawStream(dev)
    table, lens, N, max_pages = _rows(cache, page_table, seqlens)
    if used is None:
        used = torch.empty(1, device=dev, dtype=i32)
    workspace, wp, wb = _scratch(
        workspace, _cache_workspace(cache._pages, cache._heads, N), dev)
    _check(lib().polar_attn_cache_compact(cache._p, table, max_pages, lens, N,
                                          _need("used", used, i32, (1,), dev), wp, wb, st),
           "polar_attn_cache_compact")
    return used


def selftest_decode_per_head(q, kv_pages, page_table, seqlens, u, out=None, neff=None,
                             workspace=None, *, s=8.0, alpha=0.3, L=2048, beta=1.0, stream=None,
                             window=0):
    """polar_attn_selftest_decode_per_head: decode_paged with one query head per
    CTA (pages read once per query head).  Returns (out, neff)."""
    N, Hq, D = q.shape
    P_, _, Hkv, _, _ = kv_pages.shape
    max_pages = page_table.shape[1]
    p = make_params(0, 0, Hq, Hkv, _dt(q), s, alpha, L, beta, window=window)
    p.head_dim = D
    ws_need = int(lib().polar_attn_decode_workspace_size(N, max_pages, ctypes.byref(p)))
    if workspace is None:
        workspace = torch.empty(max(ws_need, 16), device=q.device, dtype=torch.uint8)
    if out is None:
        out = torch.empty_like(q)
    if neff is None:
        neff = torch.empty((N, Hq), device=q.device, dtype=torch.float32)
    _check(lib().polar_attn_selftest_decode_per_head(
        _ptr(q), _ptr(kv_pages), P_, _ptr(page_table), max_pages, _ptr(seqlens), N, _ptr(u),
        ctypes.byref(p), _ptr(out), _ptr(neff), _ptr(workspace), workspace.numel(),
        _stream(stream)), "polar_attn_selftest_decode_per_head")
    return out, neff


def selftest_timeout(stream=None):
    """Launches one bounded wait that can never complete; afterwards
    get_status() returns POLAR_ERR_TIMEOUT (5)."""
    _check(lib().polar_attn_selftest_timeout(_stream(stream)), "polar_attn_selftest_timeout")


def get_status(stream=None) -> int:
    """Synchronises the stream; returns and clears the device status word."""
    return int(lib().polar_attn_get_status(_stream(stream)))


def launch_count() -> int:
    return int(lib().polar_attn_launch_count())
