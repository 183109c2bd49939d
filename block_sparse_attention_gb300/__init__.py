"""Python binding of the bsattn C ABI (block-sparse attention for GB300 / sm_103a).

Argument marshalling only: every function passes tensor data pointers, shapes and the
current CUDA stream to the same-named C entry point of libbsattn.so and raises on a
non-zero status.  torch supplies device memory (outputs, workspaces) and streams; no step of
the computation runs in Python, and there is no CPU fallback: if the library is missing
the calls raise.

    bsattn_prefill(q, k, v, block_mask, is_causal)                      -> out
    bsattn_decode_varlen(q, k, v, cache_seqlens, block_indices, num_splits=0) -> out
    bsattn_mask_from_topk(scores, topk, use_dense_for_last_block, apply_tril)  -> mask
    bsattn_mask_from_threshold(scores, thr, use_dense_for_last_block, apply_tril) -> mask
    bsattn_num_splits_heuristic(...)                                     -> int

Around them, for a paged serving loop:

    bsattn_paged_plan(cached_lens, new_lens, free_pages, free_count, block_table, page_size, max_tokens)
                                                  -> (slots, starts, seqlens, free_left)
    bsattn_kv4_cache(num_pages, Hkv, page_size, d)                       -> Kv4Cache (4-bit pages)
    bsattn_kv4_append(k, v, slots, cache)         bsattn_kv4_gather(slots, cache, dtype) -> (k, v)
    bsattn_decode_paged_kv4(q, cache, cache_seqlens, block_table, block_indices=None, window=0) -> out
    bsattn_prefill_window(q, k, v, window, sinks)                        -> out
    bsattn_decode_window(q, k, v, cache_seqlens, window, sinks)          -> out
    bsattn_decode_window_paged(q, k_pages, v_pages, cache_seqlens, block_table, window, sinks) -> out
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import NamedTuple

import torch

from . import build as _build

__all__ = [
    "BSATTN_OK", "BSATTN_ERR_INVALID_ARG", "BSATTN_ERR_UNSUPPORTED", "BSATTN_ERR_CUDA",
    "BSATTN_ERR_TIMEOUT", "BSATTN_ERR_BAD_INDEX", "BsattnError", "library_path", "load",
    "bsattn_prefill", "bsattn_prefill_bs", "bsattn_prefill_workspace_size", "bsattn_decode_varlen",
    "bsattn_decode_workspace_size", "bsattn_decode_default_splits", "bsattn_num_splits_heuristic",
    "bsattn_mask_from_topk", "bsattn_mask_from_threshold", "bsattn_get_device_status",
    "bsattn_set_wait_budget_ns", "bsattn_status_string", "bsattn_version", "workspace",
    "bsattn_decode_varlen_mask", "bsattn_decode_paged", "bsattn_mask_from_cumulative_threshold",
    "bsattn_decode_varlen_noalloc", "bsattn_decode_noalloc_status",
    "BSATTN_ERR_NO_SPACE", "Kv4Cache", "bsattn_kv4_cache", "bsattn_kv4_append", "bsattn_kv4_gather",
    "bsattn_decode_paged_kv4", "bsattn_decode_kv4_workspace_size", "bsattn_paged_plan",
    "bsattn_prefill_window", "bsattn_decode_window", "bsattn_decode_window_paged",
    "bsattn_decode_window_workspace_size", "call_workspace", "status_workspace", "bsattn_set_status_word",
]

BSATTN_OK = 0
BSATTN_ERR_INVALID_ARG = 1
BSATTN_ERR_UNSUPPORTED = 2
BSATTN_ERR_CUDA = 4
BSATTN_ERR_TIMEOUT = 8
BSATTN_ERR_BAD_INDEX = 16
BSATTN_ERR_NO_SPACE = 32

_F16, _BF16 = 0, 1
_lock = threading.Lock()
_lib = None


class BsattnError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {bsattn_status_string(status)} ({status})")
        self.status = status


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Loads libbsattn.so (building it with nvcc first if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = _build.LIB
            if not os.path.exists(path):
                if not build_if_missing:
                    raise OSError(f"{path} is not built; run block_sparse_attention_gb300.build")
                _build.build()
            lib = ctypes.CDLL(path)
            P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
            L, F = ctypes.c_longlong, ctypes.c_float
            sig = {
                "bsattn_status_string": ([I], ctypes.c_char_p),
                "bsattn_version": ([], ctypes.c_char_p),
                "bsattn_prefill": ([P, P, P, P, I, P, I, I, I, I, I, I, P, Z, P], I),
                "bsattn_prefill_bs": ([P, P, P, P, I, I, P, I, I, I, I, I, I, P, Z, P], I),
                "bsattn_prefill_workspace_size": ([I, I, I, I], Z),
                "bsattn_decode_varlen": ([P, P, P, P, P, I, P, I, I, I, I, I, I, I, P, Z, P], I),
                "bsattn_decode_workspace_size": ([I, I, I, I, I, I], Z),
                "bsattn_decode_default_splits": ([I, I, I, I, I], I),
                "bsattn_num_splits_heuristic": ([I, I, I, I, ctypes.c_longlong, I, I], I),
                "bsattn_mask_from_topk": ([P, I, I, I, I, I, I, I, P], I),
                "bsattn_mask_from_threshold": ([P, I, I, I, I, ctypes.c_float, I, I, P], I),
                "bsattn_get_device_status": ([P, P], I),
                "bsattn_decode_varlen_mask": ([P, P, P, P, P, I, P, I, I, I, I, I, I, I, P, Z, P], I),
                "bsattn_decode_paged": ([P, P, P, P, P, P, I, P, I, I, I, I, I, I, I, I, I, P, Z, P], I),
                "bsattn_mask_from_cumulative_threshold": ([P, I, I, I, I, ctypes.c_double, I, P], I),
                "bsattn_set_wait_budget_ns": ([ctypes.c_ulonglong], None),
                "bsattn_set_status_word": ([P], I),
                "bsattn_decode_varlen_noalloc": ([P, P, P, P, P, I, P, I, I, I, I, I, I, I, P], I),
                "bsattn_decode_noalloc_status": ([P], I),
                "bsattn_paged_plan": ([P] * 9 + [I] * 5 + [P, Z, P], I),
                "bsattn_kv4_append": ([P, P, L, L, L, L, P, P, P, P, P, F, F, I, I, I, I, I, I, P, Z, P], I),
                "bsattn_kv4_gather": ([P, P, P, P, P, F, F, P, P, I, I, I, I, I, I, P, Z, P], I),
                "bsattn_decode_paged_kv4": ([P, P, P, P, P, F, F, P, P, P, I, I, P, I, I, I, I, I, I, I, I, I,
                                             P, Z, P], I),
                "bsattn_decode_kv4_workspace_size": ([I, I, I], Z),
                "bsattn_prefill_window": ([P, P, P, I, I, P, I, I, I, I, I, I, P, I, P, Z, P], I),
                "bsattn_decode_window": ([P, P, P, P, I, I, P, I, I, I, I, I, I, P, Z, P], I),
                "bsattn_decode_window_paged": ([P, P, P, P, P, I, I, P, I, I, I, I, I, I, I, I, P, Z, P], I),
                "bsattn_decode_window_workspace_size": ([I, I, I], Z),
            }
            for name, (args, res) in sig.items():
                f = getattr(lib, name)
                f.argtypes = args
                f.restype = res
            _lib = lib
    return _lib


def _check(fn: str, rc: int):
    if rc != BSATTN_OK:
        raise BsattnError(fn, rc)


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float16:
        return _F16
    if t.dtype == torch.bfloat16:
        return _BF16
    raise TypeError(f"bsattn takes fp16 or bf16 tensors, got {t.dtype}")


def _cuda_contig(name: str, t: torch.Tensor) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


# zero-filled workspaces, one per (device, purpose); the kernels leave them zeroed
_ws_cache: dict = {}


def workspace(device, purpose: str, nbytes: int) -> torch.Tensor:
    """The zero-filled workspace this binding passes for `purpose` on `device`."""
    device = torch.device(device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    key = (device.index, purpose)
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)
        _ws_cache[key] = buf
    return buf


def bsattn_status_string(status: int) -> str:
    return load().bsattn_status_string(int(status)).decode()


def bsattn_version() -> str:
    return load().bsattn_version().decode()


def bsattn_prefill_workspace_size(B: int, H: int, Sq: int, Sk: int) -> int:
    return int(load().bsattn_prefill_workspace_size(B, H, Sq, Sk))


def bsattn_prefill(q, k, v, block_mask, is_causal: bool, out=None, ws=None, block_size: int = 64):
    """Block-sparse attention forward.  q [B,H,Sq,d], k/v [B,H,Sk,d] fp16|bf16 CUDA;
    block_mask [B,H,ceil(Sq/bs),ceil(Sk/bs)] uint8/bool CUDA, bs = block_size (64 or 128)."""
    lib = load()
    for name, t in (("q", q), ("k", k), ("v", v), ("block_mask", block_mask)):
        _cuda_contig(name, t)
    B, H, Sq, d = q.shape
    Sk = k.shape[2]
    if block_mask.dtype == torch.bool:
        block_mask = block_mask.view(torch.uint8)
    if block_mask.dtype not in (torch.uint8, torch.int8):
        raise TypeError("block_mask must be uint8, int8 or bool")
    if tuple(block_mask.shape) != (B, H, -(-Sq // block_size), -(-Sk // block_size)):
        raise ValueError(f"block_mask shape {tuple(block_mask.shape)} does not match q/k")
    if k.shape != v.shape or k.shape[:2] != q.shape[:2] or k.shape[3] != d:
        raise ValueError("q, k, v shapes disagree")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k, v must share a dtype")
    if out is None:
        out = torch.empty_like(q)
    if ws is None:
        ws = workspace(q.device, "prefill", bsattn_prefill_workspace_size(B, H, Sq, Sk))
    if block_size == 64:
        rc = lib.bsattn_prefill(q.data_ptr(), k.data_ptr(), v.data_ptr(), block_mask.data_ptr(),
                                int(bool(is_causal)), out.data_ptr(), B, H, Sq, Sk, d, _dtype_code(q),
                                ws.data_ptr(), ws.numel(), _stream(q.device))
    else:
        rc = lib.bsattn_prefill_bs(q.data_ptr(), k.data_ptr(), v.data_ptr(), block_mask.data_ptr(),
                                   int(block_size), int(bool(is_causal)), out.data_ptr(), B, H, Sq,
                                   Sk, d, _dtype_code(q), ws.data_ptr(), ws.numel(), _stream(q.device))
    _check("bsattn_prefill", rc)
    return out


def bsattn_decode_default_splits(B: int, Hkv: int, max_sel: int, d: int = 128,
                                 num_sms: int = 0) -> int:
    return int(load().bsattn_decode_default_splits(B, Hkv, max_sel, d, num_sms))


def bsattn_decode_workspace_size(B, Hq, Hkv, d, max_sel, num_splits=0) -> int:
    return int(load().bsattn_decode_workspace_size(B, Hq, Hkv, d, max_sel, num_splits))


def bsattn_decode_varlen(q, k, v, cache_seqlens, block_indices, num_splits: int = 0, out=None,
                         ws=None):
    """GQA varlen sparse decode.  q [B,Hq,d]; k/v [B,Smax,Hkv,d] fp16|bf16 CUDA;
    cache_seqlens int32 [B]; block_indices int32 [B,Hkv,max_sel] (-1 = empty)."""
    lib = load()
    for name, t in (("q", q), ("k", k), ("v", v), ("cache_seqlens", cache_seqlens),
                    ("block_indices", block_indices)):
        _cuda_contig(name, t)
    if cache_seqlens.dtype != torch.int32 or block_indices.dtype != torch.int32:
        raise TypeError("cache_seqlens and block_indices must be int32")
    B, Hq, d = q.shape
    _, Smax, Hkv, _ = k.shape
    max_sel = block_indices.shape[2]
    if tuple(block_indices.shape[:2]) != (B, Hkv) or k.shape != v.shape:
        raise ValueError("decode shapes disagree")
    if out is None:
        out = torch.empty_like(q)
    if ws is None:
        ws = workspace(q.device, "decode",
                       bsattn_decode_workspace_size(B, Hq, Hkv, d, max_sel, num_splits))
    rc = lib.bsattn_decode_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                  cache_seqlens.data_ptr(), block_indices.data_ptr(),
                                  int(num_splits), out.data_ptr(), B, Hq, Hkv, Smax, d, max_sel,
                                  _dtype_code(q), ws.data_ptr(), ws.numel(), _stream(q.device))
    _check("bsattn_decode_varlen", rc)
    return out


def bsattn_decode_varlen_noalloc(q, k, v, cache_seqlens, block_indices, num_splits: int = 0, out=None):
    """bsattn_decode_varlen on the library's own fixed scratch array (no workspace argument, no
    device allocation by the library; `out` is allocated here when not given)."""
    lib = load()
    for name, t in (("q", q), ("k", k), ("v", v), ("cache_seqlens", cache_seqlens),
                    ("block_indices", block_indices)):
        _cuda_contig(name, t)
    if cache_seqlens.dtype != torch.int32 or block_indices.dtype != torch.int32:
        raise TypeError("cache_seqlens and block_indices must be int32")
    B, Hq, d = q.shape
    _, Smax, Hkv, _ = k.shape
    max_sel = block_indices.shape[2]
    if tuple(block_indices.shape[:2]) != (B, Hkv) or k.shape != v.shape:
        raise ValueError("decode shapes disagree")
    if out is None:
        out = torch.empty_like(q)
    rc = lib.bsattn_decode_varlen_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                          cache_seqlens.data_ptr(), block_indices.data_ptr(),
                                          int(num_splits), out.data_ptr(), B, Hq, Hkv, Smax, d,
                                          max_sel, _dtype_code(q), _stream(q.device))
    _check("bsattn_decode_varlen_noalloc", rc)
    return out


def bsattn_decode_noalloc_status(device=None) -> int:
    """Reads and clears the status word of the allocation-free decode on `device` (default: the
    current one); syncs that device's current stream."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return int(load().bsattn_decode_noalloc_status(_stream(dev)))


def bsattn_decode_varlen_mask(q, k, v, cache_seqlens, block_mask, num_splits: int = 0, out=None,
                              ws=None):
    """GQA varlen sparse decode, block-mask form.  block_mask [B,Hkv,num_blocks] uint8/bool."""
    lib = load()
    for name, t in (("q", q), ("k", k), ("v", v), ("cache_seqlens", cache_seqlens),
                    ("block_mask", block_mask)):
        _cuda_contig(name, t)
    if block_mask.dtype == torch.bool:
        block_mask = block_mask.view(torch.uint8)
    if cache_seqlens.dtype != torch.int32 or block_mask.dtype != torch.uint8:
        raise TypeError("cache_seqlens must be int32 and block_mask uint8/bool")
    B, Hq, d = q.shape
    _, Smax, Hkv, _ = k.shape
    nb = block_mask.shape[2]
    if tuple(block_mask.shape[:2]) != (B, Hkv) or k.shape != v.shape:
        raise ValueError("decode shapes disagree")
    if out is None:
        out = torch.empty_like(q)
    if ws is None:
        ws = workspace(q.device, "decode", bsattn_decode_workspace_size(B, Hq, Hkv, d, nb, num_splits))
    rc = lib.bsattn_decode_varlen_mask(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                       cache_seqlens.data_ptr(), block_mask.data_ptr(),
                                       int(num_splits), out.data_ptr(), B, Hq, Hkv, Smax, d, nb,
                                       _dtype_code(q), ws.data_ptr(), ws.numel(), _stream(q.device))
    _check("bsattn_decode_varlen_mask", rc)
    return out


def bsattn_decode_paged(q, k_pages, v_pages, cache_seqlens, block_indices, block_table,
                        num_splits: int = 0, out=None, ws=None):
    """GQA varlen sparse decode over a paged KV cache.  k_pages/v_pages
    [num_pages, page_size, Hkv, d]; block_table int32 [B, max_pages_per_seq]."""
    lib = load()
    for name, t in (("q", q), ("k_pages", k_pages), ("v_pages", v_pages),
                    ("cache_seqlens", cache_seqlens), ("block_indices", block_indices),
                    ("block_table", block_table)):
        _cuda_contig(name, t)
    if (cache_seqlens.dtype, block_indices.dtype, block_table.dtype) != (torch.int32,) * 3:
        raise TypeError("cache_seqlens, block_indices and block_table must be int32")
    B, Hq, d = q.shape
    num_pages, page_size, Hkv, _ = k_pages.shape
    max_sel = block_indices.shape[2]
    if k_pages.shape != v_pages.shape or tuple(block_indices.shape[:2]) != (B, Hkv):
        raise ValueError("paged decode shapes disagree")
    if out is None:
        out = torch.empty_like(q)
    if ws is None:
        ws = workspace(q.device, "decode", bsattn_decode_workspace_size(B, Hq, Hkv, d, max_sel, num_splits))
    rc = lib.bsattn_decode_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                 cache_seqlens.data_ptr(), block_indices.data_ptr(),
                                 block_table.data_ptr(), int(num_splits), out.data_ptr(), B, Hq,
                                 Hkv, num_pages, page_size, block_table.shape[1], d, max_sel,
                                 _dtype_code(q), ws.data_ptr(), ws.numel(), _stream(q.device))
    _check("bsattn_decode_paged", rc)
    return out


def bsattn_mask_from_cumulative_threshold(attn_sum, threshold: float, causal: bool = True):
    """Host-side XAttention cumulative-threshold block mask; CPU uint8 tensor."""
    s = _host_scores(attn_sum)
    B, H, nq, nk = s.shape
    out = torch.empty(s.shape, dtype=torch.uint8)
    rc = load().bsattn_mask_from_cumulative_threshold(s.data_ptr(), B, H, nq, nk, float(threshold),
                                                      int(bool(causal)), out.data_ptr())
    _check("bsattn_mask_from_cumulative_threshold", rc)
    return out


def bsattn_num_splits_heuristic(total_mblocks, num_SMs, num_n_blocks, num_m_blocks,
                                size_one_kv_head, is_causal_or_local, max_splits) -> int:
    return int(load().bsattn_num_splits_heuristic(int(total_mblocks), int(num_SMs),
                                                  int(num_n_blocks), int(num_m_blocks),
                                                  int(size_one_kv_head),
                                                  int(bool(is_causal_or_local)), int(max_splits)))


def _host_scores(scores) -> torch.Tensor:
    s = torch.as_tensor(scores)
    if s.dim() != 4:
        raise ValueError("scores must be [B, H, nq, nk]")
    return s.detach().to("cpu", torch.float32).contiguous()


def bsattn_mask_from_topk(scores, topk: int, use_dense_for_last_block: bool = False,
                          apply_tril: bool = True) -> torch.Tensor:
    """Host-side top-k block mask; returns a CPU uint8 tensor of the scores' shape."""
    s = _host_scores(scores)
    B, H, nq, nk = s.shape
    out = torch.empty(s.shape, dtype=torch.uint8)
    rc = load().bsattn_mask_from_topk(s.data_ptr(), B, H, nq, nk, int(topk),
                                      int(bool(use_dense_for_last_block)), int(bool(apply_tril)),
                                      out.data_ptr())
    _check("bsattn_mask_from_topk", rc)
    return out


def bsattn_mask_from_threshold(scores, threshold: float, use_dense_for_last_block: bool = False,
                               apply_tril: bool = True) -> torch.Tensor:
    """Host-side threshold block mask (score > threshold); CPU uint8 tensor."""
    s = _host_scores(scores)
    B, H, nq, nk = s.shape
    out = torch.empty(s.shape, dtype=torch.uint8)
    rc = load().bsattn_mask_from_threshold(s.data_ptr(), B, H, nq, nk, float(threshold),
                                           int(bool(use_dense_for_last_block)),
                                           int(bool(apply_tril)), out.data_ptr())
    _check("bsattn_mask_from_threshold", rc)
    return out


def bsattn_get_device_status(ws: torch.Tensor) -> int:
    """Reads and clears the device status word of a workspace (syncs its stream)."""
    with torch.cuda.device(ws.device):
        return int(load().bsattn_get_device_status(ws.data_ptr(), _stream(ws.device)))


def bsattn_set_wait_budget_ns(ns: int) -> None:
    load().bsattn_set_wait_budget_ns(int(ns))


def bsattn_set_status_word(ws) -> None:
    """Makes this thread's paged-serving calls record what they find in the first word of `ws` and not in
    their workspaces; None ends that."""
    if ws is not None and not (ws.is_cuda and ws.is_contiguous() and ws.numel() * ws.element_size() >= 4):
        raise ValueError("ws must be a contiguous CUDA tensor of 4 bytes or more")
    _check("bsattn_set_status_word", load().bsattn_set_status_word(None if ws is None else ws.data_ptr()))
    _own_word.ws = ws                              # kept alive


# ----------------------------------------------------------------- paged serving
#
# A step of a server makes these calls back to back with kernels of a few microseconds, so what the
# binding itself takes counts.  Each call tests its arguments in one expression; only if that fails does
# it go through them one by one for the error that says which is wrong.

_STREAM_HEADER = 256 + 4 * 1024          # status word and tickets: all that has to start at zero
# the calls behind torch.cuda's own (absent from a CPU-only torch, which has no CUDA tensors to pass)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None)
_I32, _I64, _U8 = torch.int32, torch.int64, torch.uint8
_CODES = {torch.float16: _F16, torch.bfloat16: _BF16}


def _device_index(device) -> int:
    if isinstance(device, int):
        return device
    device = torch.device(device)
    return torch.cuda.current_device() if device.index is None else device.index


def call_workspace(device, purpose: str, nbytes: int) -> torch.Tensor:
    """A workspace for the stream decodes that no other call in flight uses: one per (stream, purpose),
    "decode_kv4" or "decode_window", and a new one for every call captured into a CUDA graph (graphs may be
    replayed side by side).  With nbytes 0 outside a capture, the one that such calls on the current stream
    use, for bsattn_get_device_status; what captured calls find is in status_workspace(device)."""
    return _call_workspace(_device_index(device), purpose, nbytes, _capturing())


def _call_workspace(index, purpose, nbytes, capturing):
    key = (index, purpose, _raw_stream(index))
    buf = None if capturing else _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.empty(max(nbytes, _STREAM_HEADER), dtype=_U8, device=torch.device("cuda", index))
        buf[:_STREAM_HEADER].zero_()
        if not capturing:
            _ws_cache[key] = buf
            status_workspace(index)                 # there by the time that a warmed-up call is captured
    return buf


def _to_status_workspace(f, index):
    """f, recording in the device's status word: a captured call's own workspace goes back to the graph's
    pool, where nobody can read it after a replay."""
    def call(*args):
        lib = load()
        lib.bsattn_set_status_word(status_workspace(index).data_ptr())
        try:
            return f(*args)
        finally:
            lib.bsattn_set_status_word(None)
    return f if getattr(_own_word, "ws", None) is not None else call


_status_ws: dict = {}
_own_word = threading.local()                      # .ws: what the thread has set with bsattn_set_status_word


def status_workspace(device) -> torch.Tensor:
    """The 256-byte workspace of the calls that keep only a status word in it.  They set bits of it and
    read nothing, so all of a device's streams and graphs share it; bsattn_get_device_status of it returns
    what any of them has found.  It is made by the first such call, decode or call of this function on the
    device; a call captured before that records in a word of its own that cannot be read."""
    index = _device_index(device)
    buf = _status_ws.get(index)
    if buf is None:
        buf = torch.zeros(256, dtype=_U8, device=torch.device("cuda", index))
        if not _capturing():
            torch.cuda.current_stream(index).synchronize()
            _status_ws[index] = buf
    return buf


def _refuse(*tensors):
    """Raises for the first of (name, tensor, dtype, dims, shape or None) that is not as it should be."""
    index = tensors[0][1].get_device()
    for name, t, dtype, dims, shape in tensors:
        if t.get_device() < 0:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.get_device() != index:
            raise ValueError(f"{name} is on {t.device}, {tensors[0][0]} on {tensors[0][1].device}")
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.dim() != dims:
            raise ValueError(f"{name} must have {dims} dimensions, not {t.dim()}")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    raise ValueError("the arguments' shapes disagree")


_INT_MAX = 2 ** 31 - 1


def _int(v) -> int:
    """v as a C int (ctypes would cut larger values off)."""
    v = int(v)
    if not -_INT_MAX <= v <= _INT_MAX:
        raise ValueError(f"{v} does not fit 32 bits")
    return v


def _span(window, sinks):
    """A window and sinks as C ints: past 2^31 - 1 tokens there is nothing more to see."""
    if type(window) is int and type(sinks) is int and 0 <= window <= _INT_MAX and 0 <= sinks <= _INT_MAX:
        return window, sinks
    return max(min(int(window), _INT_MAX), -1), max(min(int(sinks), _INT_MAX), -1)


def _check_out(out, q, contiguous):
    if out.get_device() != q.get_device() or out.dtype is not q.dtype or out.shape != q.shape:
        raise ValueError("out must have the queries' device, dtype and shape")
    if contiguous and not out.is_contiguous():
        raise ValueError("out must be contiguous")


def _check_ws(ws, index):
    if ws.get_device() != index or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous tensor on the device of the call's other tensors")


def bsattn_paged_plan(cached_lens, new_lens, free_pages, free_count, block_table, page_size: int,
                      max_tokens: int, ws=None):
    """Block-table rows and slot map for `new_lens` tokens on top of `cached_lens`, both int32 [B].
    free_pages int32 [n] is the free list, free_count int32 [1] how many of it are free (taken from the
    end); block_table int32 [B, max_pages] gets the new pages.  Returns (slots int64 [max_tokens], -1
    where there is no token; starts int32 [B + 1]; seqlens int32 [B]; free_left int32 [1])."""
    i = cached_lens.get_device()
    B = cached_lens.numel()
    if not (i >= 0 and new_lens.get_device() == i and free_pages.get_device() == i
            and free_count.get_device() == i and block_table.get_device() == i
            and cached_lens.dtype is _I32 and new_lens.dtype is _I32 and free_pages.dtype is _I32
            and free_count.dtype is _I32 and block_table.dtype is _I32
            and cached_lens.dim() == 1 and new_lens.shape == cached_lens.shape and free_pages.dim() == 1
            and free_count.numel() == 1 and block_table.dim() == 2 and block_table.shape[0] == B
            and cached_lens.is_contiguous() and new_lens.is_contiguous() and free_pages.is_contiguous()
            and block_table.is_contiguous()):
        _refuse(("cached_lens", cached_lens, _I32, 1, None), ("new_lens", new_lens, _I32, 1, (B,)),
                ("free_pages", free_pages, _I32, 1, None), ("free_count", free_count, _I32, 1, (1,)),
                ("block_table", block_table, _I32, 2, (B, *block_table.shape[1:])))
    if _current_device() != i:
        with torch.cuda.device(i):
            return bsattn_paged_plan(cached_lens, new_lens, free_pages, free_count, block_table, page_size,
                                     max_tokens, ws)
    page_size, max_tokens = _int(page_size), _int(max_tokens)
    device = cached_lens.device
    slots = torch.empty(max(max_tokens, 0), dtype=_I64, device=device)
    starts = torch.empty(B + 1, dtype=_I32, device=device)
    seqlens, left = torch.empty_like(cached_lens), torch.empty_like(free_count)
    if ws is None:
        ws = status_workspace(i)
    else:
        _check_ws(ws, i)
    rc = load().bsattn_paged_plan(cached_lens.data_ptr(), new_lens.data_ptr(), free_pages.data_ptr(),
                                  free_count.data_ptr(), block_table.data_ptr(), slots.data_ptr(),
                                  starts.data_ptr(), seqlens.data_ptr(), left.data_ptr(), B, page_size,
                                  block_table.shape[1], free_pages.numel(), max_tokens, ws.data_ptr(),
                                  ws.numel(), _raw_stream(i))
    if rc:
        _check("bsattn_paged_plan", rc)
    return slots, starts, seqlens, left


class Kv4Cache(NamedTuple):
    """A paged 4-bit cache: e2m1 codes [pages, Hkv, page_size, d/2] and e4m3 scales
    [pages, Hkv, page_size, d/16] of keys and values, all uint8."""
    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: torch.Tensor
    v_scales: torch.Tensor


def bsattn_kv4_cache(num_pages: int, Hkv: int, page_size: int, d: int, device="cuda") -> Kv4Cache:
    """A zeroed paged 4-bit cache."""
    def make(n):
        return torch.zeros(num_pages, Hkv, page_size, n, dtype=_U8, device=device)
    return Kv4Cache(make(d // 2), make(d // 16), make(d // 2), make(d // 16))


def _kv4(cache, i):
    """The shape (pages, Hkv, page_size, d / 2) of a 4-bit cache on device i, or an error."""
    kc, ks, vc, vs = cache
    shape = kc.shape
    scales = ks.shape
    if not (i >= 0 and kc.get_device() == i and ks.get_device() == i and vc.get_device() == i
            and vs.get_device() == i and kc.dtype is _U8 and ks.dtype is _U8 and vc.dtype is _U8 and vs.dtype is _U8
            and len(shape) == 4 and vc.shape == shape and vs.shape == scales and scales[:3] == shape[:3]
            and len(scales) == 4 and 8 * scales[3] == shape[3] and kc.is_contiguous() and ks.is_contiguous()
            and vc.is_contiguous() and vs.is_contiguous()):
        small = (*shape[:3], shape[-1] // 8)
        _refuse(("k_codes", kc, _U8, 4, None), ("k_scales", ks, _U8, 4, small), ("v_codes", vc, _U8, 4, shape),
                ("v_scales", vs, _U8, 4, small))
    return shape


def _row_strides(name, t):
    st = t.stride()
    if st[2] != 1 and t.numel():
        raise ValueError(f"{name}'s channels must be contiguous")
    # the stride of a dimension of one entry is never used
    return (st[0] if t.shape[0] > 1 else 0), (st[1] if t.shape[1] > 1 else 0)


def bsattn_kv4_append(k, v, slots, cache, k_scale: float = 1.0, v_scale: float = 1.0, ws=None) -> None:
    """Rounds k and v [T, Hkv, d] fp16|bf16 (channels contiguous, any 16-byte aligned token and head
    strides) into the rows that slots int64 [T] names (negative: skipped; all others distinct)."""
    i = k.get_device()
    pages, hkv, page, half = _kv4(cache, i)
    T = slots.numel()
    dtype = _dtype_code(k)
    if not (v.get_device() == i and slots.get_device() == i and v.dtype is k.dtype and slots.dtype is _I64
            and slots.dim() == 1 and slots.is_contiguous() and k.shape == (T, hkv, 2 * half) and v.shape == k.shape):
        _refuse(("slots", slots, _I64, 1, None), ("k", k.contiguous(), k.dtype, 3, (T, hkv, 2 * half)),
                ("v", v.contiguous(), k.dtype, 3, (T, hkv, 2 * half)))
    if _current_device() != i:
        with torch.cuda.device(i):
            return bsattn_kv4_append(k, v, slots, cache, k_scale, v_scale, ws)
    kt, kh = _row_strides("k", k)
    vt, vh = _row_strides("v", v)
    if ws is None:
        ws = status_workspace(i)
    else:
        _check_ws(ws, i)
    kc, ks, vc, vs = cache
    rc = load().bsattn_kv4_append(k.data_ptr(), v.data_ptr(), kt, kh, vt, vh, slots.data_ptr(), kc.data_ptr(),
                                  ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), float(k_scale), float(v_scale), T, hkv,
                                  pages, page, 2 * half, dtype, ws.data_ptr(), ws.numel(), _raw_stream(i))
    if rc:
        _check("bsattn_kv4_append", rc)


def bsattn_kv4_gather(slots, cache, dtype, k_scale: float = 1.0, v_scale: float = 1.0, ws=None):
    """The rows that slots int64 [T] names, as (k, v) [T, Hkv, d] of `dtype` (negative slots: zeros)."""
    i = slots.get_device()
    pages, hkv, page, half = _kv4(cache, i)
    if not (slots.dtype is _I64 and slots.dim() == 1 and slots.is_contiguous()):
        _refuse(("slots", slots, _I64, 1, None))
    if dtype not in _CODES:
        raise TypeError(f"bsattn gives fp16 or bf16 rows, not {dtype}")
    if _current_device() != i:
        with torch.cuda.device(i):
            return bsattn_kv4_gather(slots, cache, dtype, k_scale, v_scale, ws)
    T = slots.numel()
    k = torch.empty((T, hkv, 2 * half), dtype=dtype, device=slots.device)
    v = torch.empty_like(k)
    if ws is None:
        ws = status_workspace(i)
    else:
        _check_ws(ws, i)
    kc, ks, vc, vs = cache
    rc = load().bsattn_kv4_gather(slots.data_ptr(), kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(),
                                  float(k_scale), float(v_scale), k.data_ptr(), v.data_ptr(), T, hkv, pages, page, 2 * half,
                                  _CODES[dtype], ws.data_ptr(), ws.numel(), _raw_stream(i))
    if rc:
        _check("bsattn_kv4_gather", rc)
    return k, v


def bsattn_decode_window_workspace_size(Hq: int, Hkv: int, d: int) -> int:
    return int(load().bsattn_decode_window_workspace_size(Hq, Hkv, d))


def bsattn_decode_kv4_workspace_size(Hq: int, Hkv: int, d: int) -> int:
    return int(load().bsattn_decode_kv4_workspace_size(Hq, Hkv, d))


_stream_sizes: dict = {}


def _stream_workspace(f, index, purpose, size, Hq, hkv, d):
    """(workspace, f as to be called with it) of a call that is given none."""
    key = (index, purpose, Hq, hkv, d)
    n = _stream_sizes.get(key)
    if n is None:
        n = _stream_sizes[key] = size(Hq, hkv, d)
    capturing = _capturing()
    return _call_workspace(index, purpose, n, capturing), _to_status_workspace(f, index) if capturing else f


def bsattn_decode_paged_kv4(q, cache, cache_seqlens, block_table, block_indices=None, window: int = 0,
                            sinks: int = 0, k_scale: float = 1.0, v_scale: float = 1.0, out=None, ws=None):
    """One query token per sequence over a paged 4-bit cache.  q [B,Hq,d] fp16|bf16; cache_seqlens int32
    [B]; block_table int32 [B,max_pages]; block_indices int32 [B,Hkv,max_sel] (-1 = empty) limits each kv
    head to chosen 64-token blocks, window > 0 to the last `window` tokens and the first `sinks`."""
    i = q.get_device()
    pages, hkv, page, half = _kv4(cache, i)
    d = 2 * half
    dtype = _dtype_code(q)
    qs = q.shape
    if not (len(qs) == 3 and qs[2] == d and q.is_contiguous() and cache_seqlens.get_device() == i
            and block_table.get_device() == i and cache_seqlens.dtype is _I32 and block_table.dtype is _I32
            and cache_seqlens.shape == qs[:1] and block_table.dim() == 2 and block_table.shape[0] == qs[0]
            and cache_seqlens.is_contiguous() and block_table.is_contiguous()):
        _refuse(("q", q, q.dtype, 3, (*qs[:2], d)), ("cache_seqlens", cache_seqlens, _I32, 1, qs[:1]),
                ("block_table", block_table, _I32, 2, (qs[0], *block_table.shape[1:])))
    B, Hq, _ = qs
    window, sinks = _span(window, sinks)
    max_sel, chosen = 0, None
    if block_indices is not None:
        max_sel, chosen = block_indices.shape[-1], block_indices.data_ptr()
        if not (block_indices.get_device() == i and block_indices.dtype is _I32 and block_indices.is_contiguous()
                and block_indices.shape == (B, hkv, max_sel) and max_sel > 0):
            _refuse(("q", q, q.dtype, 3, None), ("block_indices", block_indices, _I32, 3, (B, hkv, max(max_sel, 1))))
    if _current_device() != i:
        with torch.cuda.device(i):
            return bsattn_decode_paged_kv4(q, cache, cache_seqlens, block_table, block_indices, window, sinks,
                                           k_scale, v_scale, out, ws)
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_out(out, q, True)
    f = load().bsattn_decode_paged_kv4
    if ws is None:
        ws, f = _stream_workspace(f, i, "decode_kv4", bsattn_decode_kv4_workspace_size, Hq, hkv, d)
    else:
        _check_ws(ws, i)
    kc, ks, vc, vs = cache
    rc = f(q.data_ptr(), kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), float(k_scale), float(v_scale),
           cache_seqlens.data_ptr(), chosen, block_table.data_ptr(), window, sinks, out.data_ptr(), B, Hq, hkv, pages,
           page, block_table.shape[1], d, max_sel, dtype, ws.data_ptr(), ws.numel(), _raw_stream(i))
    if rc:
        _check("bsattn_decode_paged_kv4", rc)
    return out


def _window_args(q, k, v, cache_seqlens):
    """Checks shared by the two window decodes; (device, dtype code)."""
    i = q.get_device()
    dtype = _dtype_code(q)
    qs, ks = q.shape, k.shape
    if not (i >= 0 and k.get_device() == i and v.get_device() == i and cache_seqlens.get_device() == i
            and k.dtype is q.dtype and v.dtype is q.dtype and cache_seqlens.dtype is _I32 and len(qs) == 3
            and len(ks) == 4 and v.shape == ks and qs[2] == ks[3] and cache_seqlens.shape == qs[:1]
            and q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and cache_seqlens.is_contiguous()):
        _refuse(("q", q, q.dtype, 3, None), ("k", k, q.dtype, 4, (*ks[:3], qs[-1])), ("v", v, q.dtype, 4, ks),
                ("cache_seqlens", cache_seqlens, _I32, 1, qs[:1]))
    return i, dtype


def bsattn_decode_window(q, k, v, cache_seqlens, window: int, sinks: int = 0, out=None, ws=None):
    """One query token per sequence over the last `window` tokens and the first `sinks` of a contiguous
    cache.  q [B,Hq,d]; k/v [B,Smax,Hkv,d] fp16|bf16 CUDA; cache_seqlens int32 [B]."""
    i, dtype = _window_args(q, k, v, cache_seqlens)
    B, Hq, d = q.shape
    if k.shape[0] != B:
        raise ValueError("k and v must be [B, Smax, Hkv, d]")
    if _current_device() != i:
        with torch.cuda.device(i):
            return bsattn_decode_window(q, k, v, cache_seqlens, window, sinks, out, ws)
    _, Smax, hkv, _ = k.shape
    window, sinks = _span(window, sinks)
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_out(out, q, True)
    f = load().bsattn_decode_window
    if ws is None:
        ws, f = _stream_workspace(f, i, "decode_window", bsattn_decode_window_workspace_size, Hq, hkv, d)
    else:
        _check_ws(ws, i)
    rc = f(q.data_ptr(), k.data_ptr(), v.data_ptr(), cache_seqlens.data_ptr(), window, sinks, out.data_ptr(), B, Hq, hkv,
           Smax, d, dtype, ws.data_ptr(), ws.numel(), _raw_stream(i))
    if rc:
        _check("bsattn_decode_window", rc)
    return out


def bsattn_decode_window_paged(q, k_pages, v_pages, cache_seqlens, block_table, window: int, sinks: int = 0,
                               out=None, ws=None):
    """bsattn_decode_window over a paged cache: k_pages/v_pages [num_pages,page_size,Hkv,d]; block_table
    int32 [B,max_pages]."""
    i, dtype = _window_args(q, k_pages, v_pages, cache_seqlens)
    B, Hq, d = q.shape
    if not (block_table.get_device() == i and block_table.dtype is _I32 and block_table.dim() == 2
            and block_table.shape[0] == B and block_table.is_contiguous()):
        _refuse(("q", q, q.dtype, 3, None), ("block_table", block_table, _I32, 2, (B, *block_table.shape[1:])))
    if _current_device() != i:
        with torch.cuda.device(i):
            return bsattn_decode_window_paged(q, k_pages, v_pages, cache_seqlens, block_table, window, sinks, out, ws)
    pages, page, hkv, _ = k_pages.shape
    window, sinks = _span(window, sinks)
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_out(out, q, True)
    f = load().bsattn_decode_window_paged
    if ws is None:
        ws, f = _stream_workspace(f, i, "decode_window", bsattn_decode_window_workspace_size, Hq, hkv, d)
    else:
        _check_ws(ws, i)
    rc = f(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), cache_seqlens.data_ptr(), block_table.data_ptr(),
           window, sinks, out.data_ptr(), B, Hq, hkv, pages, page, block_table.shape[1], d, dtype, ws.data_ptr(),
           ws.numel(), _raw_stream(i))
    if rc:
        _check("bsattn_decode_window_paged", rc)
    return out


_Strides = ctypes.c_int64 * 12


def bsattn_prefill_window(q, k, v, window: int, sinks: int = 0, out=None, ws=None):
    """Causal attention with a sliding window and sinks: query row i (position p = i + Sk - Sq) sees key j
    iff j <= p and (j < sinks or j > p - window).  q [B,Hq,Sq,d], k/v [B,Hkv,Sk,d] fp16|bf16 CUDA views
    with contiguous channels and 16-byte aligned strides; out: laid out as q is, unless given."""
    i = q.get_device()
    dtype = _dtype_code(q)
    if not (i >= 0 and k.get_device() == i and v.get_device() == i and k.dtype is q.dtype and v.dtype is q.dtype
            and q.dim() == 4 and k.dim() == 4 and v.shape == k.shape and q.shape[0] == k.shape[0]
            and q.shape[3] == k.shape[3]):
        _refuse(("q", q.contiguous(), q.dtype, 4, None),
                ("k", k.contiguous(), q.dtype, 4, (q.shape[0], *k.shape[1:-1], q.shape[-1])),
                ("v", v.contiguous(), q.dtype, 4, k.shape))
    if _current_device() != i:
        with torch.cuda.device(i):
            return bsattn_prefill_window(q, k, v, window, sinks, out, ws)
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_out(out, q, False)
    B, Hq, Sq, d = q.shape
    _, hkv, Sk, _ = k.shape
    window, sinks = _span(window, sinks)
    strides = None
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and out.is_contiguous()):
        qs, ks, vs, os_ = q.stride(), k.stride(), v.stride(), out.stride()
        if (qs[3] != 1 or os_[3] != 1) and q.numel() or (ks[3] != 1 or vs[3] != 1) and k.numel():
            raise ValueError("channels (the last dimension) must be contiguous")
        strides = _Strides(*qs[:3], *ks[:3], *vs[:3], *os_[:3])
    if ws is None:
        ws = status_workspace(i)
    else:
        _check_ws(ws, i)
    rc = load().bsattn_prefill_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), window, sinks, out.data_ptr(), B,
                                      Hq, hkv, Sq, Sk, d, strides, dtype, ws.data_ptr(), ws.numel(), _raw_stream(i))
    if rc:
        _check("bsattn_prefill_window", rc)
    return out
