"""Python binding of the C ABI in include/fmha.h (argument marshalling only).

Every step of the computation runs in libfmha.so's CUDA kernels; this module
only turns torch tensors into pointers and the current torch stream into a
cudaStream_t.  If the library has not been built it raises: there is no
fallback of any kind.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import Optional, Tuple

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfmha.so")

F16, BF16, E4M3 = 0, 1, 2
MASK_NONE, MASK_RESIDUAL, MASK_CAUSAL = 0, 1, 2
ROPE_HALF, ROPE_PAIRS = 0, 1
CAUSAL_QBEGIN, CAUSAL_QEND = 0, 1
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT = 0, -1, -2, -3, -4

_TORCH_DTYPE = {torch.float16: F16, torch.bfloat16: BF16, torch.float8_e4m3fn: E4M3}
_MASKS = {"none": MASK_NONE, "residual": MASK_RESIDUAL, "causal": MASK_CAUSAL}
_CAUSAL = {"qbegin": CAUSAL_QBEGIN, "qend": CAUSAL_QEND}

EXPORTED = ("fmha_fwd", "fmha_fwd_simt", "fmha_fwd_splitkv", "fmha_fwd_splitkv_workspace_size",
            "fmha_fwd_splitkv_noalloc",
            "fmha_status_string", "fmha_device_status", "fmha_kv_tile_range")


class fmha_tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int)]


class FmhaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{msg} (status {status})")
        self.status = status


_lib = None


def library_path() -> str:
    return _LIB_PATH


def lib():
    """Load libfmha.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build it with __graft_entry__.build()")
        L = ctypes.CDLL(_LIB_PATH)
        fwd_args = [fmha_tensor, fmha_tensor, fmha_tensor, fmha_tensor, ctypes.c_void_p,
                    ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                    ctypes.c_int, ctypes.c_float, ctypes.c_float, ctypes.c_int, ctypes.c_int,
                    ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                    ctypes.c_void_p]
        for name in ("fmha_fwd", "fmha_fwd_simt"):
            f = getattr(L, name)
            f.restype = ctypes.c_int
            f.argtypes = fwd_args
        L.fmha_fwd_splitkv.restype = ctypes.c_int
        L.fmha_fwd_splitkv.argtypes = fwd_args[:-1] + [ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t,
                                                       ctypes.c_void_p]
        L.fmha_fwd_splitkv_noalloc.restype = ctypes.c_int
        L.fmha_fwd_splitkv_noalloc.argtypes = fwd_args[:-1] + [ctypes.c_int, ctypes.c_void_p]
        L.fmha_fwd_splitkv_workspace_size.restype = ctypes.c_size_t
        L.fmha_fwd_splitkv_workspace_size.argtypes = [ctypes.c_int] * 5 + [ctypes.c_int64]
        L.fmha_gen_fwd.restype = ctypes.c_int
        L.fmha_gen_fwd.argtypes = [fmha_tensor] * 6 + [ctypes.c_void_p] + [ctypes.c_int] * 6 + [
            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float, ctypes.c_float, ctypes.c_void_p,
            ctypes.c_size_t, ctypes.c_void_p]
        L.fmha_gen_workspace_size.restype = ctypes.c_size_t
        L.fmha_gen_workspace_size.argtypes = [ctypes.c_int] * 5
        L.fmha_tree_fwd.restype = ctypes.c_int
        L.fmha_tree_fwd.argtypes = [fmha_tensor] * 6 + [ctypes.c_void_p] + [ctypes.c_int] * 7 + [
            ctypes.c_void_p] * 4 + [ctypes.c_int64, ctypes.c_float, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t,
                                    ctypes.c_void_p]
        L.fmha_tree_workspace_size.restype = ctypes.c_size_t
        L.fmha_tree_workspace_size.argtypes = [ctypes.c_int] * 6
        L.fmha_tree_commit.restype = ctypes.c_int
        L.fmha_tree_commit.argtypes = [fmha_tensor] * 4 + [ctypes.c_int] * 7 + [ctypes.c_void_p] * 5
        L.fmha_cache_weights.restype = ctypes.c_int
        L.fmha_cache_weights.argtypes = [fmha_tensor] * 2 + [ctypes.c_void_p] * 3 + [ctypes.c_int] * 7 + [
            ctypes.c_void_p] * 3 + [ctypes.c_float, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        L.fmha_cache_weights_workspace_size.restype = ctypes.c_size_t
        L.fmha_cache_weights_workspace_size.argtypes = []
        L.fmha_cache_evict.restype = ctypes.c_int
        L.fmha_cache_evict.argtypes = [fmha_tensor] * 2 + [ctypes.c_void_p] + [fmha_tensor] * 2 + [
            ctypes.c_void_p] + [ctypes.c_int] * 7 + [ctypes.c_void_p] * 3 + [ctypes.c_int] * 2 + [ctypes.c_void_p] * 3
        L.fmha_page_plan.restype = ctypes.c_int
        L.fmha_page_plan.argtypes = [ctypes.c_void_p] * 11 + [ctypes.c_int] * 6 + [ctypes.c_void_p]
        L.fmha_page_write.restype = ctypes.c_int
        L.fmha_page_write.argtypes = ([fmha_tensor] + [ctypes.c_int64] * 2) * 2 + [ctypes.c_void_p] * 5 + [
            ctypes.c_int] * 5 + [ctypes.c_void_p]
        L.fmha_page_fwd.restype = ctypes.c_int
        L.fmha_page_fwd.argtypes = [fmha_tensor] + [ctypes.c_void_p] * 4 + [fmha_tensor, ctypes.c_void_p] + [
            ctypes.c_int] * 10 + [ctypes.c_void_p] * 4 + [ctypes.c_float, ctypes.c_float, ctypes.c_int, ctypes.c_void_p,
                                                          ctypes.c_size_t, ctypes.c_void_p]
        L.fmha_page_workspace_size.restype = ctypes.c_size_t
        L.fmha_page_workspace_size.argtypes = [ctypes.c_int] * 3
        L.fmha_rope.restype = ctypes.c_int
        L.fmha_rope.argtypes = ([fmha_tensor] + [ctypes.c_int64] * 3) * 4 + [ctypes.c_int] * 6 + [ctypes.c_void_p] * 2 + [
            ctypes.c_float] + [ctypes.c_int] * 2 + [ctypes.c_void_p]
        L.fmha_bwd.restype = ctypes.c_int
        L.fmha_bwd.argtypes = [fmha_tensor] * 5 + [ctypes.c_void_p] + [fmha_tensor] * 3 + [ctypes.c_int] * 5 + [
            ctypes.c_float, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        L.fmha_bwd_workspace_size.restype = ctypes.c_size_t
        L.fmha_bwd_workspace_size.argtypes = [ctypes.c_int] * 3
        L.fmha_bwd_workspace_size_ex.restype = ctypes.c_size_t
        L.fmha_bwd_workspace_size_ex.argtypes = [ctypes.c_int] * 6
        L.fmha_status_string.restype = ctypes.c_char_p
        L.fmha_status_string.argtypes = [ctypes.c_int]
        L.fmha_device_status.restype = ctypes.c_int
        L.fmha_device_status.argtypes = [ctypes.c_int]
        L.fmha_set_wait_limit_ns.restype = ctypes.c_int
        L.fmha_set_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
        L.fmha_set_test_gate.restype = ctypes.c_int
        L.fmha_set_test_gate.argtypes = [ctypes.c_int]
        L.fmha_kv_tile_range.restype = ctypes.c_int
        L.fmha_kv_tile_range.argtypes = [ctypes.c_int] * 7 + [ctypes.POINTER(ctypes.c_int)] * 2
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().fmha_status_string(int(status)).decode()


def device_status(reset: bool = False) -> int:
    return lib().fmha_device_status(1 if reset else 0)


def set_wait_limit_ns(ns: int) -> int:
    """Test hook (see fmha_set_wait_limit_ns): the kernels' bounded waits
    give up after ns nanoseconds; 0 restores the default."""
    return lib().fmha_set_wait_limit_ns(int(ns))


def set_test_gate(on: bool) -> int:
    """Test hook (see fmha_set_test_gate): the kernels' producers first wait for
    a flag that nothing sets."""
    return lib().fmha_set_test_gate(1 if on else 0)


def kv_tile_range(q_row0: int, q_rows: int, Sq: int, Sk: int, mask: int, causal_type: int,
                  tile_n: int) -> Tuple[int, int]:
    a, b = ctypes.c_int(), ctypes.c_int()
    rc = lib().fmha_kv_tile_range(q_row0, q_rows, Sq, Sk, mask, causal_type, tile_n,
                                  ctypes.byref(a), ctypes.byref(b))
    if rc != OK:
        raise FmhaError(rc, status_string(rc))
    return a.value, b.value


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _tensor(t, dtype: Optional[int] = None) -> fmha_tensor:
    if t is None:
        return fmha_tensor(None, BF16 if dtype is None else dtype)
    if isinstance(t, torch.Tensor):
        return fmha_tensor(t.data_ptr(), _TORCH_DTYPE[t.dtype] if dtype is None else dtype)
    return fmha_tensor(int(t), dtype)


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _call(name, q, k, v, o, lse, B, H, H_k, Sq, Sk, D, scale, out_scale, mask, causal_type,
          cu_seqlens_q, cu_seqlens_k, max_len, total_length, stream) -> int:
    f = getattr(lib(), name)
    return f(_tensor(q), _tensor(k), _tensor(v), _tensor(o), _ptr(lse), int(B), int(H), int(H_k),
             int(Sq), int(Sk), int(D), float(scale), float(out_scale), int(mask), int(causal_type),
             _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), int(max_len), int(total_length),
             _stream(stream))


def fmha_fwd(q, k, v, o, lse, B, H, H_k, Sq, Sk, D, scale, out_scale, mask, causal_type,
             cu_seqlens_q=None, cu_seqlens_k=None, max_len=0, total_length=0, stream=None) -> int:
    """Same arguments, order and status codes as the C function fmha_fwd.

    Tensors are passed as torch tensors (or raw device addresses); ``stream``
    defaults to torch's current stream.  Returns the C status code."""
    return _call("fmha_fwd", q, k, v, o, lse, B, H, H_k, Sq, Sk, D, scale, out_scale, mask,
                 causal_type, cu_seqlens_q, cu_seqlens_k, max_len, total_length, stream)


def fmha_fwd_simt(q, k, v, o, lse, B, H, H_k, Sq, Sk, D, scale, out_scale, mask, causal_type,
                  cu_seqlens_q=None, cu_seqlens_k=None, max_len=0, total_length=0,
                  stream=None) -> int:
    """The CUDA-core cross-check kernel; same contract as fmha_fwd."""
    return _call("fmha_fwd_simt", q, k, v, o, lse, B, H, H_k, Sq, Sk, D, scale, out_scale, mask,
                 causal_type, cu_seqlens_q, cu_seqlens_k, max_len, total_length, stream)


def fmha_fwd_splitkv(q, k, v, o, lse, B, H, H_k, Sq, Sk, D, scale, out_scale, mask, causal_type,
                     cu_seqlens_q=None, cu_seqlens_k=None, max_len=0, total_length=0,
                     num_splits=1, workspace=None, workspace_bytes=None, stream=None) -> int:
    """Same arguments, order and status codes as the C function fmha_fwd_splitkv."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    return lib().fmha_fwd_splitkv(
        _tensor(q), _tensor(k), _tensor(v), _tensor(o), _ptr(lse), int(B), int(H), int(H_k), int(Sq),
        int(Sk), int(D), float(scale), float(out_scale), int(mask), int(causal_type),
        _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), int(max_len), int(total_length), int(num_splits),
        _ptr(workspace), int(workspace_bytes), _stream(stream))


def fmha_fwd_splitkv_noalloc(q, k, v, o, lse, B, H, H_k, Sq, Sk, D, scale, out_scale, mask,
                             causal_type, cu_seqlens_q=None, cu_seqlens_k=None, max_len=0,
                             total_length=0, num_splits=1, stream=None) -> int:
    """Same arguments, order and status codes as the C function
    fmha_fwd_splitkv_noalloc: split-KV with the library's built-in scratch,
    for callers that must not allocate device memory while they run."""
    return lib().fmha_fwd_splitkv_noalloc(
        _tensor(q), _tensor(k), _tensor(v), _tensor(o), _ptr(lse), int(B), int(H), int(H_k), int(Sq),
        int(Sk), int(D), float(scale), float(out_scale), int(mask), int(causal_type),
        _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), int(max_len), int(total_length), int(num_splits),
        _stream(stream))


def fmha_fwd_splitkv_workspace_size(B, H, Sq, D, num_splits, total_length=0) -> int:
    return int(lib().fmha_fwd_splitkv_workspace_size(int(B), int(H), int(Sq), int(D), int(num_splits),
                                                     int(total_length)))


def fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, scale: Optional[float] = None,
        out_scale: float = 1.0, mask: str = "none", causal_type: str = "qbegin",
        cu_seqlens_q: Optional[torch.Tensor] = None, cu_seqlens_k: Optional[torch.Tensor] = None,
        max_len: Optional[int] = None, total_length: Optional[int] = None,
        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
        return_lse: bool = True, impl: str = "tc", num_splits: Optional[int] = None, stream=None):
    """Attention forward on device tensors; allocates O (and LSE) if not given.

    Fixed length: q [B,Sq,H,D], k/v [B,Sk,H_k,D].  Varlen: q [T,H,D], k/v
    [T,H_k,D] with int32 device cumulative lengths.  ``num_splits`` selects
    the split-KV entry point (a workspace is allocated with torch).
    Returns (O, LSE)."""
    varlen = cu_seqlens_q is not None
    D = q.shape[-1]
    if varlen:
        T = q.shape[0] if total_length is None else int(total_length)
        B = cu_seqlens_q.numel() - 1
        H, H_k = q.shape[1], k.shape[1]
        Sq = Sk = 0
        if max_len is None:
            raise ValueError("varlen needs max_len")
        lse_shape = (H, T)
    else:
        B, Sq, H = q.shape[0], q.shape[1], q.shape[2]
        Sk, H_k = k.shape[1], k.shape[2]
        T = 0
        lse_shape = (B, H, Sq)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty(lse_shape, dtype=torch.float32, device=q.device)
    sc = 1.0 / math.sqrt(D) if scale is None else scale
    if num_splits is not None:
        nbytes = fmha_fwd_splitkv_workspace_size(B, H, Sq, D, num_splits, T)
        ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
        rc = fmha_fwd_splitkv(q, k, v, out, lse, B, H, H_k, Sq, Sk, D, sc, out_scale, _MASKS[mask],
                              _CAUSAL[causal_type], cu_seqlens_q, cu_seqlens_k, max_len or 0, T,
                              num_splits, ws, nbytes, stream)
        if rc != OK:
            raise FmhaError(rc, status_string(rc))
        return out, lse
    name = "fmha_fwd" if impl == "tc" else "fmha_fwd_simt"
    rc = _call(name, q, k, v, out, lse, B, H, H_k, Sq, Sk, D, sc, out_scale, _MASKS[mask],
               _CAUSAL[causal_type], cu_seqlens_q, cu_seqlens_k, max_len or 0, T, stream)
    if rc != OK:
        raise FmhaError(rc, status_string(rc))
    return out, lse


def fmha_gen_fwd(q, k_cache, v_cache, k_new, v_new, o, lse, B, H, H_k, D, B_cache, S_max, seqlen,
                 batch_idx, scale, out_scale, workspace, workspace_bytes, stream=None) -> int:
    """Same arguments, order and status codes as the C function fmha_gen_fwd."""
    dt = _TORCH_DTYPE[q.dtype] if isinstance(q, torch.Tensor) else None
    return lib().fmha_gen_fwd(
        _tensor(q), _tensor(k_cache), _tensor(v_cache), _tensor(k_new, dt), _tensor(v_new, dt), _tensor(o),
        _ptr(lse), int(B), int(H), int(H_k), int(D), int(B_cache), int(S_max), _ptr(seqlen),
        _ptr(batch_idx), float(scale), float(out_scale), _ptr(workspace), int(workspace_bytes),
        _stream(stream))


def fmha_gen_workspace_size(B, H, H_k, D, S_max) -> int:
    return int(lib().fmha_gen_workspace_size(int(B), int(H), int(H_k), int(D), int(S_max)))


def gen_fwd(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, seqlen: torch.Tensor, *,
            k_new: Optional[torch.Tensor] = None, v_new: Optional[torch.Tensor] = None,
            batch_idx: Optional[torch.Tensor] = None, scale: Optional[float] = None,
            out_scale: float = 1.0, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
            return_lse: bool = True, workspace: Optional[torch.Tensor] = None, stream=None):
    """Generation-phase attention on device tensors (see fmha_gen_fwd).

    q [B, H, 128]; k_cache / v_cache [B_cache, S_max, H_k, 128]; seqlen int32
    [B]; k_new / v_new [B, H_k, 128] (insert mode) or None (cache-only);
    batch_idx int32 [B] or None.  Allocates O, LSE and the workspace with torch
    when not given.  Returns (O, LSE)."""
    B, H, D = q.shape
    B_cache, S_max, H_k = k_cache.shape[0], k_cache.shape[1], k_cache.shape[2]
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    nbytes = fmha_gen_workspace_size(B, H, H_k, D, S_max) if B > 0 else 0
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    sc = 1.0 / math.sqrt(D) if scale is None else scale
    rc = fmha_gen_fwd(q, k_cache, v_cache, k_new, v_new, out, lse, B, H, H_k, D, B_cache, S_max, seqlen,
                      batch_idx, sc, out_scale, workspace, max(nbytes, workspace.numel()), stream)
    if rc != OK:
        raise FmhaError(rc, status_string(rc))
    return out, lse


def fmha_tree_fwd(q, k_cache, v_cache, k_new, v_new, o, lse, B, T, H, H_k, D, B_cache, S_max, seqlen, batch_idx,
                  n_draft, tree_mask, mask_batch_stride, scale, out_scale, workspace, workspace_bytes,
                  stream=None) -> int:
    """Same arguments, order and status codes as the C function fmha_tree_fwd."""
    return lib().fmha_tree_fwd(
        _tensor(q), _tensor(k_cache), _tensor(v_cache), _tensor(k_new), _tensor(v_new), _tensor(o), _ptr(lse), int(B),
        int(T), int(H), int(H_k), int(D), int(B_cache), int(S_max), _ptr(seqlen), _ptr(batch_idx), _ptr(n_draft),
        _ptr(tree_mask), int(mask_batch_stride), float(scale), float(out_scale), _ptr(workspace),
        int(workspace_bytes), _stream(stream))


def fmha_tree_workspace_size(B, T, H, H_k, D, S_max) -> int:
    return int(lib().fmha_tree_workspace_size(int(B), int(T), int(H), int(H_k), int(D), int(S_max)))


def fmha_tree_commit(k_cache, v_cache, k_new, v_new, B, T, P, H_k, D, B_cache, S_max, seqlen, batch_idx, path,
                     n_accept, stream=None) -> int:
    """Same arguments, order and status codes as the C function fmha_tree_commit."""
    return lib().fmha_tree_commit(_tensor(k_cache), _tensor(v_cache), _tensor(k_new), _tensor(v_new), int(B), int(T),
                                  int(P), int(H_k), int(D), int(B_cache), int(S_max), _ptr(seqlen), _ptr(batch_idx),
                                  _ptr(path), _ptr(n_accept), _stream(stream))


# The operators below are called once a layer and token, where a call's Python
# steps outlast its kernels.  So tensors are looked at once, a group at a time
# (_check only names what did not fit), the C function is called directly, and
# scratch comes from torch's allocator without a tensor around it, which alone
# took 6 us (tree_fwd: 41 -> 24 -> 19 us, weights 20 -> 14 to enqueue).
_current_device, _raw_stream, _alloc, _free = (
    getattr(torch._C, name, None) for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream",
                                               "_cuda_cudaCachingAllocator_raw_alloc",
                                               "_cuda_cudaCachingAllocator_raw_delete"))


def _fit(index: int, dtype, shape: tuple, *tensors) -> bool:
    """Would the library, which takes only addresses, read these tensors right?"""
    for t in tensors:
        if t is not None and not (t.dtype is dtype and t.shape == shape and t.get_device() == index
                                  and t.is_contiguous()):
            return False
    return True


def _check(index: int, dtype, shape: tuple, **tensors) -> None:
    """Refuse the first of the tensors that the library would misread."""
    for name, t in tensors.items():
        if _fit(index, dtype, shape, t):
            continue
        if t.get_device() != index:
            raise ValueError(f"{name} is on {t.device}, not on the call's device cuda:{index}")
        if t.dtype is not dtype:
            raise ValueError(f"{name} has dtype {t.dtype}, not {dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
        raise ValueError(f"{name} is not contiguous")


def _device_and_code(t: torch.Tensor) -> Tuple[int, int]:
    """CUDA device index and element type code of a call's first tensor."""
    index, code = t.get_device(), _TORCH_DTYPE.get(t.dtype)
    if index < 0:
        raise ValueError(f"the tensors are on {t.device}, not on a CUDA device")
    if code is None:
        raise FmhaError(ERR_UNSUPPORTED, f"dtype {t.dtype}: {status_string(ERR_UNSUPPORTED)}")
    return index, code


def _on(stream, index: int):
    """The call's device and stream made torch's current ones: what the call
    allocates and fills then belongs to its stream, and torch hands none of it
    out again before the stream is past it."""
    if stream is None:
        return torch.cuda.device(index)
    if not isinstance(stream, torch.cuda.Stream):
        # torch takes a handle of 0, the default stream's, for none given, and makes a new stream
        stream = torch.cuda.ExternalStream(int(stream), device=index) if int(stream) else torch.cuda.default_stream(index)
    if stream.device.index != index:
        raise ValueError(f"the stream is of {stream.device}, not of the tensors' cuda:{index}")
    return torch.cuda.stream(stream)


def _given(workspace: torch.Tensor, index: int) -> Tuple[int, int]:
    """Address and bytes of a caller's workspace."""
    if workspace.get_device() != index:
        raise ValueError(f"workspace is on {workspace.device}, not on cuda:{index}")
    if not workspace.is_contiguous():
        raise ValueError("workspace is not contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _raise(rc: int) -> None:
    if rc != OK:
        raise FmhaError(rc, status_string(rc))


_tree_workspace_size = functools.lru_cache(maxsize=256)(fmha_tree_workspace_size)


def tree_fwd(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
             seqlen: torch.Tensor, *, tree_mask: Optional[torch.Tensor] = None,
             n_draft: Optional[torch.Tensor] = None, batch_idx: Optional[torch.Tensor] = None,
             scale: Optional[float] = None, out_scale: float = 1.0, out: Optional[torch.Tensor] = None,
             lse: Optional[torch.Tensor] = None, return_lse: bool = True,
             workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of drafted tokens over a K/V cache (see fmha_tree_fwd).

    q [B, T, H, 128]; k_cache / v_cache [B_cache, S_max, H_k, 128]; k_new /
    v_new [B, T, H_k, 128]; seqlen, n_draft, batch_idx int32 [B]; tree_mask
    bool or uint8 [B, T, T], or [T, T] for every sequence, true where draft
    row sees draft column (None: a chain).  Allocates O, LSE [B, H, T] and the
    workspace with torch when not given; rows of drafts at or past n_draft[b]
    are not written.  Returns (O, LSE)."""
    index, code = _device_and_code(q)
    if stream is not None or _current_device() != index:
        with _on(stream, index):
            return tree_fwd(q, k_cache, v_cache, k_new, v_new, seqlen, tree_mask=tree_mask, n_draft=n_draft,
                            batch_idx=batch_idx, scale=scale, out_scale=out_scale, out=out, lse=lse,
                            return_lse=return_lse, workspace=workspace)
    if q.dim() != 4 or k_cache.dim() != 4:
        raise ValueError("q is [B, T, H, 128] and the caches are [B_cache, S_max, H_k, 128]")
    (B, T, H, D), (B_cache, S_max, H_k, _) = q.shape, k_cache.shape
    dt, cache, new, per_seq = q.dtype, (B_cache, S_max, H_k, D), (B, T, H_k, D), (B,)
    if not (_fit(index, dt, cache, k_cache, v_cache) and _fit(index, dt, new, k_new, v_new)
            and _fit(index, torch.int32, per_seq, seqlen, n_draft, batch_idx)):
        _check(index, dt, cache, k_cache=k_cache, v_cache=v_cache)
        _check(index, dt, new, k_new=k_new, v_new=v_new)
        _check(index, torch.int32, per_seq, seqlen=seqlen, n_draft=n_draft, batch_idx=batch_idx)
    stride = 0
    if tree_mask is not None:
        if tree_mask.dtype not in (torch.bool, torch.uint8):
            raise ValueError(f"tree_mask has dtype {tree_mask.dtype}, not bool or uint8")
        each = tree_mask.dim() == 3
        stride = T * T if each else 0
        if not _fit(index, tree_mask.dtype, (B, T, T) if each else (T, T), tree_mask):
            _check(index, tree_mask.dtype, (B, T, T) if each else (T, T), tree_mask=tree_mask)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((B, H, T), dtype=torch.float32, device=q.device)
    if not (_fit(index, dt, q.shape, q, out) and _fit(index, torch.float32, (B, H, T), lse)):
        _check(index, dt, q.shape, q=q, out=out)
        _check(index, torch.float32, (B, H, T), lse=lse)
    raw = _raw_stream(index)
    if workspace is None:
        nbytes = _tree_workspace_size(B, T, H, H_k, D, S_max)
        ws = _alloc(nbytes or 1, raw)
    else:
        ws, nbytes = _given(workspace, index)
    try:
        rc = lib().fmha_tree_fwd(
            fmha_tensor(q.data_ptr(), code), fmha_tensor(k_cache.data_ptr(), code),
            fmha_tensor(v_cache.data_ptr(), code), fmha_tensor(k_new.data_ptr(), code),
            fmha_tensor(v_new.data_ptr(), code), fmha_tensor(out.data_ptr(), code), _ptr(lse), B, T, H, H_k, D, B_cache,
            S_max, seqlen.data_ptr(), _ptr(batch_idx), _ptr(n_draft), _ptr(tree_mask), stride,
            1.0 / math.sqrt(D) if scale is None else scale, out_scale, ws, nbytes, raw)
    finally:
        if workspace is None:
            _free(ws)                       # for what this stream runs next
    _raise(rc)
    return out, lse


def tree_commit(k_cache: torch.Tensor, v_cache: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                seqlen: torch.Tensor, path: torch.Tensor, n_accept: torch.Tensor, *,
                batch_idx: Optional[torch.Tensor] = None, stream=None) -> None:
    """Write the accepted drafts into the cache (see fmha_tree_commit): rows
    path[b, i], i < n_accept[b], of k_new / v_new [B, T, H_k, 128] become rows
    seqlen[b] + i of sequence b's entry.  path int32 [B, P]; n_accept, seqlen,
    batch_idx int32 [B].  seqlen is not changed."""
    index, code = _device_and_code(k_cache)
    if stream is not None or _current_device() != index:
        with _on(stream, index):
            return tree_commit(k_cache, v_cache, k_new, v_new, seqlen, path, n_accept, batch_idx=batch_idx)
    if k_cache.dim() != 4 or k_new.dim() != 4 or path.dim() != 2:
        raise ValueError("the caches are [B_cache, S_max, H_k, 128], k_new is [B, T, H_k, 128] and path is [B, P]")
    (B_cache, S_max, H_k, D), (B, T, _, _), P = k_cache.shape, k_new.shape, path.shape[1]
    dt, cache, new, per_seq = k_cache.dtype, (B_cache, S_max, H_k, D), (B, T, H_k, D), (B,)
    if not (_fit(index, dt, cache, k_cache, v_cache) and _fit(index, dt, new, k_new, v_new)
            and _fit(index, torch.int32, per_seq, seqlen, n_accept, batch_idx)
            and _fit(index, torch.int32, (B, P), path)):
        _check(index, dt, cache, k_cache=k_cache, v_cache=v_cache)
        _check(index, dt, new, k_new=k_new, v_new=v_new)
        _check(index, torch.int32, per_seq, seqlen=seqlen, n_accept=n_accept, batch_idx=batch_idx)
        _check(index, torch.int32, (B, P), path=path)
    _raise(lib().fmha_tree_commit(
        fmha_tensor(k_cache.data_ptr(), code), fmha_tensor(v_cache.data_ptr(), code),
        fmha_tensor(k_new.data_ptr(), code), fmha_tensor(v_new.data_ptr(), code), B, T, P, H_k, D, B_cache, S_max,
        seqlen.data_ptr(), _ptr(batch_idx), path.data_ptr(), n_accept.data_ptr(), _raw_stream(index)))


def fmha_cache_weights(q, k_cache, lse, acc_in, acc_out, B, Sq, H, H_k, D, B_cache, S_max, seqlen, batch_idx, n_query,
                       scale, mask, workspace, workspace_bytes, stream=None) -> int:
    """Same arguments, order and status codes as the C function fmha_cache_weights."""
    return lib().fmha_cache_weights(
        _tensor(q), _tensor(k_cache), _ptr(lse), _ptr(acc_in), _ptr(acc_out), int(B), int(Sq), int(H), int(H_k), int(D),
        int(B_cache), int(S_max), _ptr(seqlen), _ptr(batch_idx), _ptr(n_query), float(scale), int(mask),
        _ptr(workspace), int(workspace_bytes), _stream(stream))


def fmha_cache_weights_workspace_size() -> int:
    return int(lib().fmha_cache_weights_workspace_size())


def fmha_cache_evict(k_cache, v_cache, acc, k_out, v_out, acc_out, B, H_k, D, B_cache, S_max, B_out, S_out, seqlen,
                     batch_idx, out_idx, budget, recent, kept, new_seqlen, stream=None) -> int:
    """Same arguments, order and status codes as the C function fmha_cache_evict."""
    return lib().fmha_cache_evict(
        _tensor(k_cache), _tensor(v_cache), _ptr(acc), _tensor(k_out), _tensor(v_out), _ptr(acc_out), int(B), int(H_k),
        int(D), int(B_cache), int(S_max), int(B_out), int(S_out), _ptr(seqlen), _ptr(batch_idx), _ptr(out_idx),
        int(budget), int(recent), _ptr(kept), _ptr(new_seqlen), _stream(stream))


_weights_workspace_size = functools.lru_cache(maxsize=1)(fmha_cache_weights_workspace_size)


def cache_weights(q: torch.Tensor, k_cache: torch.Tensor, lse: torch.Tensor, seqlen: torch.Tensor, *,
                  acc: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  n_query: Optional[torch.Tensor] = None, batch_idx: Optional[torch.Tensor] = None,
                  mask: str = "none", scale: Optional[float] = None, workspace: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """Add the attention weight of every cached key to a running score (see
    fmha_cache_weights).

    q [B, Sq, H, 128], or [B, H, 128] of a generation step; k_cache [B_cache,
    S_max, H_k, 128]; lse [B, H, Sq], or [B, H], as the attention call returned
    it; acc float [B_cache, H_k, S_max], None: start from nothing; mask "none"
    or "causal" (q-end).  Updates acc in place unless ``out`` is given; with
    neither, returns a new array that is zero past every length."""
    index, code = _device_and_code(q)
    if stream is not None or _current_device() != index:
        with _on(stream, index):
            return cache_weights(q, k_cache, lse, seqlen, acc=acc, out=out, n_query=n_query, batch_idx=batch_idx,
                                 mask=mask, scale=scale, workspace=workspace)
    if q.dim() == 3:
        q, lse = q.unsqueeze(1), lse.unsqueeze(-1)
    if q.dim() != 4 or k_cache.dim() != 4:
        raise ValueError("q is [B, Sq, H, 128] or [B, H, 128] and the cache is [B_cache, S_max, H_k, 128]")
    if mask not in ("none", "causal"):
        raise ValueError(f"mask is none or causal, not {mask!r}")
    (B, Sq, H, D), (B_cache, S_max, H_k, _) = q.shape, k_cache.shape
    dt, scores, per_seq = q.dtype, (B_cache, H_k, S_max), (B,)
    if not (_fit(index, dt, q.shape, q) and _fit(index, dt, (B_cache, S_max, H_k, D), k_cache)
            and _fit(index, torch.float32, (B, H, Sq), lse)
            and _fit(index, torch.int32, per_seq, seqlen, n_query, batch_idx)):
        _check(index, dt, q.shape, q=q)
        _check(index, dt, (B_cache, S_max, H_k, D), k_cache=k_cache)
        _check(index, torch.float32, (B, H, Sq), lse=lse)
        _check(index, torch.int32, per_seq, seqlen=seqlen, n_query=n_query, batch_idx=batch_idx)
    if out is None:
        out = torch.zeros(scores, dtype=torch.float32, device=q.device) if acc is None else acc
    if not _fit(index, torch.float32, scores, acc, out):
        _check(index, torch.float32, scores, acc=acc, out=out)
    raw = _raw_stream(index)
    if workspace is None:
        nbytes = _weights_workspace_size()
        ws = _alloc(nbytes, raw)
    else:
        ws, nbytes = _given(workspace, index)
    try:
        rc = lib().fmha_cache_weights(
            fmha_tensor(q.data_ptr(), code), fmha_tensor(k_cache.data_ptr(), code), lse.data_ptr(), _ptr(acc),
            out.data_ptr(), B, Sq, H, H_k, D, B_cache, S_max, seqlen.data_ptr(), _ptr(batch_idx), _ptr(n_query),
            1.0 / math.sqrt(D) if scale is None else scale, _MASKS[mask], ws, nbytes, raw)
    finally:
        if workspace is None:
            _free(ws)                       # for what this stream runs next
    _raise(rc)
    return out


def cache_evict(k_cache: torch.Tensor, v_cache: torch.Tensor, acc: torch.Tensor, seqlen: torch.Tensor, budget: int, *,
                recent: int = 0, batch_idx: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                v_out: Optional[torch.Tensor] = None, acc_out: Optional[torch.Tensor] = None,
                out_idx: Optional[torch.Tensor] = None, kept: Optional[torch.Tensor] = None,
                new_seqlen: Optional[torch.Tensor] = None, stream=None):
    """Shrink sequences to ``budget`` cached rows by score (see fmha_cache_evict).

    k_cache / v_cache [B_cache, S_max, H_k, 128], acc float [B_cache, H_k,
    S_max], seqlen int32 [B].  In place unless k_out / v_out [B_out, S_out,
    H_k, 128] and acc_out [B_out, H_k, S_out] are given (out_idx: their
    entries).  Returns (kept int32 [B, H_k, budget], new_seqlen int32 [B])."""
    index, code = _device_and_code(k_cache)
    if stream is not None or _current_device() != index:
        with _on(stream, index):
            return cache_evict(k_cache, v_cache, acc, seqlen, budget, recent=recent, batch_idx=batch_idx, k_out=k_out,
                               v_out=v_out, acc_out=acc_out, out_idx=out_idx, kept=kept, new_seqlen=new_seqlen)
    given = (k_out is not None) + (v_out is not None) + (acc_out is not None)
    if given not in (0, 3) or (given == 0 and out_idx is not None):
        raise ValueError("k_out, v_out and acc_out come together, and out_idx only with them")
    if given == 0:
        k_out, v_out, acc_out, out_idx = k_cache, v_cache, acc, batch_idx
    if k_cache.dim() != 4 or k_out.dim() != 4 or seqlen.dim() != 1:
        raise ValueError("the caches are [B_cache, S_max, H_k, 128] and seqlen is [B]")
    (B_cache, S_max, H_k, D), (B_out, S_out), B = k_cache.shape, k_out.shape[:2], seqlen.shape[0]
    dt, cache, moved, per_seq = k_cache.dtype, (B_cache, S_max, H_k, D), (B_out, S_out, H_k, D), (B,)
    if kept is None:
        kept = torch.empty((B, H_k, max(budget, 0)), dtype=torch.int32, device=k_cache.device)
    if new_seqlen is None:
        new_seqlen = torch.empty(per_seq, dtype=torch.int32, device=k_cache.device)
    if not (_fit(index, dt, cache, k_cache, v_cache) and _fit(index, torch.float32, (B_cache, H_k, S_max), acc)
            and _fit(index, dt, moved, k_out, v_out) and _fit(index, torch.float32, (B_out, H_k, S_out), acc_out)
            and _fit(index, torch.int32, per_seq, seqlen, batch_idx, out_idx, new_seqlen)
            and _fit(index, torch.int32, (B, H_k, max(budget, 0)), kept)):
        _check(index, dt, cache, k_cache=k_cache, v_cache=v_cache)
        _check(index, torch.float32, (B_cache, H_k, S_max), acc=acc)
        _check(index, dt, moved, k_out=k_out, v_out=v_out)
        _check(index, torch.float32, (B_out, H_k, S_out), acc_out=acc_out)
        _check(index, torch.int32, per_seq, seqlen=seqlen, batch_idx=batch_idx, out_idx=out_idx, new_seqlen=new_seqlen)
        _check(index, torch.int32, (B, H_k, max(budget, 0)), kept=kept)
    _raise(lib().fmha_cache_evict(
        fmha_tensor(k_cache.data_ptr(), code), fmha_tensor(v_cache.data_ptr(), code), acc.data_ptr(),
        fmha_tensor(k_out.data_ptr(), code), fmha_tensor(v_out.data_ptr(), code), acc_out.data_ptr(), B, H_k, D,
        B_cache, S_max, B_out, S_out, seqlen.data_ptr(), _ptr(batch_idx), _ptr(out_idx), budget, recent,
        kept.data_ptr(), new_seqlen.data_ptr(), _raw_stream(index)))
    return kept, new_seqlen


# ---------------------------------------------------------------------------
# Paged caches of e4m3 codes, and rotary positions
# ---------------------------------------------------------------------------

def fmha_page_plan(seqlen, n_new, batch_idx, table, free_list, n_free, n_free_out, slots, positions, cu_new, new_seqlen,
                   B, N, B_table, max_pages, n_pages, page_size, stream=None) -> int:
    """Same arguments, order and status codes as the C function fmha_page_plan."""
    return lib().fmha_page_plan(
        _ptr(seqlen), _ptr(n_new), _ptr(batch_idx), _ptr(table), _ptr(free_list), _ptr(n_free), _ptr(n_free_out),
        _ptr(slots), _ptr(positions), _ptr(cu_new), _ptr(new_seqlen), int(B), int(N), int(B_table), int(max_pages),
        int(n_pages), int(page_size), _stream(stream))


def page_plan(seqlen: torch.Tensor, n_new: torch.Tensor, table: torch.Tensor, free_list: torch.Tensor,
              n_free: torch.Tensor, *, page_size: int, max_tokens: Optional[int] = None,
              batch_idx: Optional[torch.Tensor] = None, slots: Optional[torch.Tensor] = None,
              positions: Optional[torch.Tensor] = None, cu_new: Optional[torch.Tensor] = None,
              new_seqlen: Optional[torch.Tensor] = None, n_free_out: Optional[torch.Tensor] = None, stream=None):
    """Block tables and slot maps of a step from request lengths (see
    fmha_page_plan).

    seqlen, n_new, batch_idx int32 [B]; table int32 [B_table, max_pages] and
    free_list int32 [n_pages], both changed in place; n_free int32 [1], changed
    in place unless ``n_free_out`` is given.  The step's tensors have
    ``max_tokens`` rows (or as many as ``slots``).  Returns (slots, positions,
    cu_new [B + 1], new_seqlen [B]), all int32; ``new_seqlen`` may be seqlen.
    Without sequences (an idle step) every row is told that it has none."""
    index = n_free.get_device()
    if index < 0:
        raise ValueError(f"the tensors are on {n_free.device}, not on a CUDA device")
    if stream is not None or _current_device() != index:
        with _on(stream, index):
            return page_plan(seqlen, n_new, table, free_list, n_free, page_size=page_size, max_tokens=max_tokens,
                             batch_idx=batch_idx, slots=slots, positions=positions, cu_new=cu_new,
                             new_seqlen=new_seqlen, n_free_out=n_free_out)
    if table.dim() != 2 or seqlen.dim() != 1 or free_list.dim() != 1:
        raise ValueError("seqlen is [B], the table is [B_table, max_pages] and free_list is [n_pages]")
    if slots is None and positions is None and max_tokens is None:
        raise ValueError("max_tokens, slots or positions say how many rows the step has")
    N = max_tokens if max_tokens is not None else (slots if slots is not None else positions).shape[0]
    i32, B = torch.int32, seqlen.shape[0]
    new = lambda n: torch.empty((n,), dtype=i32, device=n_free.device)
    slots = new(N) if slots is None else slots
    positions = new(N) if positions is None else positions
    cu_new = new(B + 1) if cu_new is None else cu_new
    new_seqlen = new(B) if new_seqlen is None else new_seqlen
    n_free_out = n_free if n_free_out is None else n_free_out
    per_seq, rows = (B,), (N,)
    given = ((seqlen, n_new, new_seqlen, slots, positions, cu_new, table, free_list, n_free)
             + (() if batch_idx is None else (batch_idx,)) + (() if n_free_out is n_free else (n_free_out,)))
    ok = (n_new.shape == per_seq and new_seqlen.shape == per_seq and slots.shape == rows and positions.shape == rows
          and cu_new.shape == (B + 1,) and n_free.shape == (1,) and n_free_out.shape == (1,)
          and (batch_idx is None or batch_idx.shape == per_seq))
    for t in given:
        ok = ok and t.dtype is i32 and t.get_device() == index and t.is_contiguous()
    if not ok:
        _check(index, i32, per_seq, seqlen=seqlen, n_new=n_new, batch_idx=batch_idx, new_seqlen=new_seqlen)
        _check(index, i32, rows, slots=slots, positions=positions)
        _check(index, i32, (B + 1,), cu_new=cu_new)
        _check(index, i32, (1,), n_free=n_free, n_free_out=n_free_out)
        _check(index, i32, table.shape, table=table)
        _check(index, i32, free_list.shape, free_list=free_list)
    if B == 0:                              # the C function has nothing to do, or refuses rows without sequences
        cu_new.zero_()
        slots.fill_(-1)
        positions.fill_(-1)
        if n_free_out is not n_free:
            n_free_out.copy_(n_free)
        return slots, positions, cu_new, new_seqlen
    _raise(lib().fmha_page_plan(
        seqlen.data_ptr(), n_new.data_ptr(), _ptr(batch_idx), table.data_ptr(), free_list.data_ptr(), n_free.data_ptr(),
        n_free_out.data_ptr(), slots.data_ptr(), positions.data_ptr(), cu_new.data_ptr(), new_seqlen.data_ptr(), B, N,
        table.shape[0], table.shape[1], free_list.shape[0], page_size, _raw_stream(index)))
    return slots, positions, cu_new, new_seqlen


def fmha_page_write(k_new, k_token_stride, k_head_stride, v_new, v_token_stride, v_head_stride, slots, k_pages, v_pages,
                    k_scale, v_scale, N, H_k, D, n_pages, page_size, stream=None) -> int:
    """Same arguments, order and status codes as the C function fmha_page_write."""
    return lib().fmha_page_write(
        _tensor(k_new), int(k_token_stride), int(k_head_stride), _tensor(v_new), int(v_token_stride), int(v_head_stride),
        _ptr(slots), _ptr(k_pages), _ptr(v_pages), _ptr(k_scale), _ptr(v_scale), int(N), int(H_k), int(D),
        int(n_pages), int(page_size), _stream(stream))


def _fit_strided(index: int, dtype, shape: tuple, t) -> bool:
    """As _fit, for a tensor of which the last dimension alone has to be contiguous."""
    return t.dtype is dtype and t.shape == shape and t.get_device() == index and (t.shape[-1] <= 1 or t.stride(-1) == 1)


def _check_strided(index: int, dtype, shape: tuple, **tensors) -> None:
    for name, t in tensors.items():
        if t is None or _fit_strided(index, dtype, shape, t):
            continue
        if t.get_device() == index and t.dtype is dtype and t.shape == shape:
            raise ValueError(f"{name}'s last dimension is not contiguous")
        _check(index, dtype, shape, **{name: t})


def _fit_pages(index: int, k_pages, v_pages, k_scale, v_scale) -> Tuple[int, int, int, int]:
    """(n_pages, H_k, page_size, D) of a paged cache, once its arrays are looked at."""
    if k_pages.dim() != 4:
        raise ValueError("the pages are [n_pages, H_k, page_size, 128]")
    shape, e4m3, f32 = k_pages.shape, torch.float8_e4m3fn, torch.float32
    if not (k_pages.dtype is e4m3 and k_pages.get_device() == index and k_pages.is_contiguous()
            and v_pages.dtype is e4m3 and v_pages.get_device() == index and v_pages.is_contiguous() and v_pages.shape == shape
            and k_scale.dtype is f32 and k_scale.get_device() == index and k_scale.is_contiguous()
            and v_scale.dtype is f32 and v_scale.get_device() == index and v_scale.is_contiguous()
            and k_scale.shape == shape[:2] and v_scale.shape == shape[:2]):
        _check(index, e4m3, shape, k_pages=k_pages, v_pages=v_pages)
        _check(index, f32, shape[:2], k_scale=k_scale, v_scale=v_scale)
    return shape


def page_write(k_new: torch.Tensor, v_new: torch.Tensor, slots: torch.Tensor, k_pages: torch.Tensor,
               v_pages: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor, *, stream=None) -> None:
    """Write new keys and values into a paged cache at their slots (see
    fmha_page_write).

    k_new, v_new bf16 or f16 [N, H_k, 128], of any strides that are multiples
    of 8 (pieces of a projection's rows); slots int32 [N], negative: not
    written; k_pages, v_pages e4m3 [n_pages, H_k, page_size, 128]; k_scale,
    v_scale float [n_pages, H_k]."""
    index, code = _device_and_code(k_new)
    if stream is not None or _current_device() != index:
        with _on(stream, index):
            return page_write(k_new, v_new, slots, k_pages, v_pages, k_scale, v_scale)
    if k_new.dim() != 3:
        raise ValueError("k_new and v_new are [N, H_k, 128]")
    n_pages, H_k, P, D = _fit_pages(index, k_pages, v_pages, k_scale, v_scale)
    new, dt, N = k_new.shape, k_new.dtype, k_new.shape[0]
    if not (new == (N, H_k, D) and v_new.shape == new and v_new.dtype is dt and v_new.get_device() == index
            and k_new.stride(2) == 1 and v_new.stride(2) == 1 and _fit(index, torch.int32, (N,), slots)):
        _check_strided(index, dt, (N, H_k, D), k_new=k_new, v_new=v_new)
        _check(index, torch.int32, (N,), slots=slots)
    (kt, kh, _), (vt, vh, _) = k_new.stride(), v_new.stride()
    _raise(lib().fmha_page_write(
        fmha_tensor(k_new.data_ptr(), code), kt, kh, fmha_tensor(v_new.data_ptr(), code), vt, vh, slots.data_ptr(),
        k_pages.data_ptr(), v_pages.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), N, H_k, D, n_pages, P, _raw_stream(index)))


def fmha_page_fwd(q, k_pages, v_pages, k_scale, v_scale, o, lse, B, N, max_q, H, H_k, D, n_pages, page_size, B_table,
                  max_pages, table, seqlen, batch_idx, cu_q, scale, out_scale, mask, workspace, workspace_bytes,
                  stream=None) -> int:
    """Same arguments, order and status codes as the C function fmha_page_fwd."""
    return lib().fmha_page_fwd(
        _tensor(q), _ptr(k_pages), _ptr(v_pages), _ptr(k_scale), _ptr(v_scale), _tensor(o), _ptr(lse), int(B), int(N),
        int(max_q), int(H), int(H_k), int(D), int(n_pages), int(page_size), int(B_table), int(max_pages), _ptr(table),
        _ptr(seqlen), _ptr(batch_idx), _ptr(cu_q), float(scale), float(out_scale), int(mask), _ptr(workspace),
        int(workspace_bytes), _stream(stream))


def fmha_page_workspace_size(max_q, H, H_k) -> int:
    return int(lib().fmha_page_workspace_size(int(max_q), int(H), int(H_k)))


_page_workspace_size = functools.lru_cache(maxsize=256)(fmha_page_workspace_size)


def page_fwd(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, k_scale: torch.Tensor,
             v_scale: torch.Tensor, table: torch.Tensor, seqlen: torch.Tensor, *, cu_q: Optional[torch.Tensor] = None,
             max_q: Optional[int] = None, batch_idx: Optional[torch.Tensor] = None, mask: str = "causal",
             scale: Optional[float] = None, out_scale: float = 1.0, out: Optional[torch.Tensor] = None,
             lse: Optional[torch.Tensor] = None, return_lse: bool = True, workspace: Optional[torch.Tensor] = None,
             stream=None):
    """Attention over a paged e4m3 cache (see fmha_page_fwd).

    q bf16 or f16 [N, H, 128], the rows of all sequences behind one another as
    cu_q int32 [B + 1] says, at most max_q (None: N) of one sequence; cu_q None: one row a
    sequence.  k_pages, v_pages e4m3 [n_pages, H_k, page_size, 128]; k_scale,
    v_scale float [n_pages, H_k]; table int32 [B_table, max_pages]; seqlen,
    batch_idx int32 [B].  mask "causal" (q-end) or "none".  Allocates O, LSE
    [N, H] and the workspace with torch when not given; rows behind the last
    sequence are not written.  Returns (O, LSE)."""
    index, dt = q.get_device(), q.dtype
    code = _TORCH_DTYPE.get(dt)
    if index < 0 or code is None:
        _device_and_code(q)
    if stream is not None or _current_device() != index:
        with _on(stream, index):
            return page_fwd(q, k_pages, v_pages, k_scale, v_scale, table, seqlen, cu_q=cu_q, max_q=max_q,
                            batch_idx=batch_idx, mask=mask, scale=scale, out_scale=out_scale, out=out, lse=lse,
                            return_lse=return_lse, workspace=workspace)
    if q.dim() != 3 or table.dim() != 2 or seqlen.dim() != 1:
        raise ValueError("q is [N, H, 128], the table is [B_table, max_pages] and seqlen is [B]")
    if mask not in ("none", "causal"):
        raise ValueError(f"mask is none or causal, not {mask!r}")
    n_pages, H_k, P, D = _fit_pages(index, k_pages, v_pages, k_scale, v_scale)
    (N, H, _), (B_table, width), B = q.shape, table.shape, seqlen.shape[0]
    if cu_q is None and N != B:
        raise ValueError(f"{N} rows of q for {B} sequences need cu_q")
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((N, H), dtype=torch.float32, device=q.device)
    i32, shape = torch.int32, q.shape
    if not (shape[2] == D and q.is_contiguous() and out.shape == shape and out.dtype is dt and out.get_device() == index
            and out.is_contiguous() and seqlen.dtype is i32 and seqlen.get_device() == index and seqlen.is_contiguous()
            and table.dtype is i32 and table.get_device() == index and table.is_contiguous()
            and (lse is None or _fit(index, torch.float32, (N, H), lse))
            and (batch_idx is None or _fit(index, i32, (B,), batch_idx)) and (cu_q is None or _fit(index, i32, (B + 1,), cu_q))):
        _check(index, dt, (N, H, D), q=q, out=out)
        _check(index, torch.float32, (N, H), lse=lse)
        _check(index, torch.int32, (B,), seqlen=seqlen, batch_idx=batch_idx)
        _check(index, torch.int32, (B + 1,), cu_q=cu_q)
        _check(index, torch.int32, (B_table, width), table=table)
    most = 1 if cu_q is None else N if max_q is None else max_q
    raw = _raw_stream(index)
    if workspace is None:
        nbytes = _page_workspace_size(most, H, H_k)
        ws = _alloc(nbytes or 1, raw)
    else:
        ws, nbytes = _given(workspace, index)
    try:
        rc = lib().fmha_page_fwd(
            fmha_tensor(q.data_ptr(), code), k_pages.data_ptr(), v_pages.data_ptr(), k_scale.data_ptr(),
            v_scale.data_ptr(), fmha_tensor(out.data_ptr(), code), None if lse is None else lse.data_ptr(), B, N, most, H, H_k, D,
            n_pages, P, B_table, width, table.data_ptr(), seqlen.data_ptr(),
            None if batch_idx is None else batch_idx.data_ptr(), None if cu_q is None else cu_q.data_ptr(),
            1.0 / math.sqrt(D) if scale is None else scale, out_scale, _MASKS[mask], ws, nbytes, raw)
    finally:
        if workspace is None:
            _free(ws)                       # for what this stream runs next
    _raise(rc)
    return out, lse


def fmha_rope(q, q_strides, k, k_strides, q_out, q_out_strides, k_out, k_out_strides, B, S, H, H_k, D, rot, positions,
              inv_freq, magnitude, layout, transpose, stream=None) -> int:
    """Same arguments, order and status codes as the C function fmha_rope;
    strides as (batch, token, head) in elements."""
    return lib().fmha_rope(
        _tensor(q), *map(int, q_strides), _tensor(k), *map(int, k_strides), _tensor(q_out), *map(int, q_out_strides),
        _tensor(k_out), *map(int, k_out_strides), int(B), int(S), int(H), int(H_k), int(D), int(rot), _ptr(positions),
        _ptr(inv_freq), float(magnitude), int(layout), int(transpose), _stream(stream))


def rope_frequencies(rot: int, *, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     trained: Optional[int] = None, slow: float = 1.0, fast: float = 32.0, device=None):
    """Rotary frequencies for fmha_rope, and the magnitude that goes with them:
    (inv_freq float64 [rot / 2], magnitude).

    ``scaling`` for contexts ``factor`` times as long as the model was trained on:
      "none"      inv_freq[i] = base ** (-2 i / rot)
      "linear"    all of them divided by factor
      "ntk"       a larger base, base * factor ** (rot / (rot - 2)): the first
                  pair turns as before, the last factor times slower
      "by_parts"  pairs that turn at least ``fast`` times within ``trained``
                  positions as before, those that turn ``slow`` times at most
                  factor times slower, a linear blend between; the magnitude
                  is 0.1 ln(factor) + 1
    """
    if rot <= 0 or rot % 2:
        raise ValueError(f"rot is even and positive, not {rot}")
    if not (base > 0 and factor >= 1):
        raise ValueError("base is positive and factor at least 1")
    i2 = torch.arange(0, rot, 2, dtype=torch.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2)) if rot > 2 else base
    inv_freq, magnitude = base ** (-i2 / rot), 1.0
    if scaling == "linear":
        inv_freq = inv_freq / factor
    elif scaling == "by_parts":
        if trained is None or not fast > slow:
            raise ValueError("by_parts needs trained, the positions the model was trained on, and fast above slow")
        turns = trained * inv_freq / (2 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0, 1)
        inv_freq, magnitude = inv_freq * (keep + (1 - keep) / factor), 0.1 * math.log(factor) + 1
    elif scaling not in ("none", "ntk"):
        raise ValueError(f"scaling is none, linear, ntk or by_parts, not {scaling!r}")
    return inv_freq.to(device) if device is not None else inv_freq, magnitude


_NO_TENSOR = fmha_tensor(None, BF16)


def _rope(q, k, inv_freq, positions, interleaved, magnitude, q_out, k_out, out_dtype, stream, transpose):
    index, dt = q.get_device(), q.dtype
    code = _TORCH_DTYPE.get(dt)
    if index < 0 or code is None:
        _device_and_code(q)
    if stream is not None or _current_device() != index:
        with _on(stream, index):
            return _rope(q, k, inv_freq, positions, interleaved, magnitude, q_out, k_out, out_dtype, None, transpose)
    shape, qs = q.shape, q.stride()
    if len(shape) == 4:
        (B, S, H, D), qb = shape, qs[0]
    elif len(shape) == 3:
        (S, H, D), B, qb = shape, 1, 0
    else:
        raise ValueError("q is [B, S, H, D] or [N, H, D], and k alike")
    lead, H_k, kt, kot = shape[:-2], 0, _NO_TENSOR, _NO_TENSOR
    kb = k_t = k_h = kob = ko_t = ko_h = 0
    odt = out_dtype or (dt if q_out is None else q_out.dtype)
    ocode = code if odt is dt else _TORCH_DTYPE.get(odt)
    if ocode is None:
        raise FmhaError(ERR_UNSUPPORTED, f"dtype {odt}: {status_string(ERR_UNSUPPORTED)}")
    if q_out is None:
        q_out = torch.empty(shape, dtype=odt, device=q.device)
    qos = q_out.stride()
    ok = (q_out.shape == shape and q_out.dtype is odt and q_out.get_device() == index
          and (D == 1 or (qs[-1] == 1 and qos[-1] == 1)))
    if k is not None:
        H_k = k.shape[-2] if k.dim() > 1 else 0
        k_shape, ks = (*lead, H_k, D), k.stride()
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=odt, device=q.device)
        kos = k_out.stride()
        ok = ok and (k.shape == k_shape and k_out.shape == k_shape and k.dtype is dt and k_out.dtype is odt
                     and k.get_device() == index and k_out.get_device() == index
                     and (D == 1 or (ks[-1] == 1 and kos[-1] == 1)))
        if ok:
            kt, kot = fmha_tensor(k.data_ptr(), code), fmha_tensor(k_out.data_ptr(), ocode)
            (k_t, k_h), (ko_t, ko_h) = ks[-3:-1], kos[-3:-1]
            kb, kob = (ks[0], kos[0]) if len(shape) == 4 else (0, 0)
    elif k_out is not None:
        raise ValueError("k_out comes with k")
    if not (ok and inv_freq.dtype is torch.float64 and inv_freq.dim() == 1 and inv_freq.get_device() == index
            and inv_freq.is_contiguous() and _fit(index, torch.int32, lead, positions)):
        _check_strided(index, dt, shape, q=q)
        _check_strided(index, odt, shape, q_out=q_out)
        if k is not None:
            _check_strided(index, dt, k_shape, k=k)
            _check_strided(index, odt, k_shape, k_out=k_out)
        _check(index, torch.int32, lead, positions=positions)
        _check(index, torch.float64, (inv_freq.numel(),), inv_freq=inv_freq)
    _raise(lib().fmha_rope(
        fmha_tensor(q.data_ptr(), code), qb, qs[-3], qs[-2], kt, kb, k_t, k_h, fmha_tensor(q_out.data_ptr(), ocode),
        qos[0] if len(shape) == 4 else 0, qos[-3], qos[-2], kot, kob, ko_t, ko_h, B, S, H, H_k, D, 2 * inv_freq.shape[0],
        None if positions is None else positions.data_ptr(), inv_freq.data_ptr(), magnitude,
        ROPE_PAIRS if interleaved else ROPE_HALF, transpose, _raw_stream(index)))
    return q_out, k_out


def rope(q: torch.Tensor, k: Optional[torch.Tensor], inv_freq: torch.Tensor, *,
         positions: Optional[torch.Tensor] = None, interleaved: bool = False, magnitude: float = 1.0,
         q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None, out_dtype=None, stream=None):
    """Rotary positions of queries and keys (see fmha_rope).

    q [B, S, H, D] or packed [N, H, D], k alike with H_k heads, or None, bf16
    or f16, of any strides with a contiguous last dimension; inv_freq float64
    [rot / 2] on the device (see rope_frequencies), rot at most D; positions
    int32 [B, S] or [N], None: 0, 1, ... in every sequence.  Pairs are elements
    i and i + rot / 2, or with ``interleaved`` 2 i and 2 i + 1.  Allocates the
    outputs, of the inputs' type or ``out_dtype`` (e4m3), unless given; in place
    with q_out=q and k_out=k.  Returns (q_out, k_out)."""
    return _rope(q, k, inv_freq, positions, interleaved, magnitude, q_out, k_out, out_dtype, stream, 0)


def rope_bwd(dq: torch.Tensor, dk: Optional[torch.Tensor], inv_freq: torch.Tensor, *,
             positions: Optional[torch.Tensor] = None, interleaved: bool = False, magnitude: float = 1.0,
             q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None, stream=None):
    """Gradients of rope's inputs from those of its outputs; arguments as rope."""
    return _rope(dq, dk, inv_freq, positions, interleaved, magnitude, q_out, k_out, None, stream, 1)


def fmha_bwd(q, k, v, o, dout, lse, dq, dk, dv, B, H, Sq, Sk, D, scale, mask, causal_type, workspace,
             workspace_bytes, stream=None) -> int:
    """Same arguments, order and status codes as the C function fmha_bwd."""
    return lib().fmha_bwd(_tensor(q), _tensor(k), _tensor(v), _tensor(o), _tensor(dout), _ptr(lse), _tensor(dq),
                          _tensor(dk), _tensor(dv), int(B), int(H), int(Sq), int(Sk), int(D), float(scale),
                          int(mask), int(causal_type), _ptr(workspace), int(workspace_bytes), _stream(stream))


def fmha_bwd_workspace_size(B, H, Sq) -> int:
    return int(lib().fmha_bwd_workspace_size(int(B), int(H), int(Sq)))


def fmha_bwd_workspace_size_ex(B, H, Sq, Sk, D, dtype) -> int:
    return int(lib().fmha_bwd_workspace_size_ex(int(B), int(H), int(Sq), int(Sk), int(D), int(dtype)))


def bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, dout: torch.Tensor,
        lse: torch.Tensor, *, scale: Optional[float] = None, mask: str = "none", causal_type: str = "qbegin",
        dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None, dv: Optional[torch.Tensor] = None,
        workspace: Optional[torch.Tensor] = None, stream=None):
    """Backward of fwd (see fmha_bwd): q, o, dout [B,Sq,H,D]; k, v [B,Sk,H,D];
    lse [B,H,Sq] from fwd.  Allocates the gradients (bf16 for e4m3 inputs, else
    the inputs' type) and the workspace with torch when not given.  Returns
    (dq, dk, dv)."""
    B, Sq, H, D = q.shape
    Sk = k.shape[1]
    gdt = torch.bfloat16 if q.dtype == torch.float8_e4m3fn else q.dtype
    dq = torch.empty(q.shape, dtype=gdt, device=q.device) if dq is None else dq
    dk = torch.empty(k.shape, dtype=gdt, device=k.device) if dk is None else dk
    dv = torch.empty(v.shape, dtype=gdt, device=v.device) if dv is None else dv
    nbytes = fmha_bwd_workspace_size_ex(B, H, Sq, Sk, D, _TORCH_DTYPE[q.dtype])
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    sc = 1.0 / math.sqrt(D) if scale is None else scale
    rc = fmha_bwd(q, k, v, o, dout, lse, dq, dk, dv, B, H, Sq, Sk, D, sc, _MASKS[mask], _CAUSAL[causal_type],
                  workspace, max(nbytes, workspace.numel()), stream)
    if rc != OK:
        raise FmhaError(rc, status_string(rc))
    return dq, dk, dv
