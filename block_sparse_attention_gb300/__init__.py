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
    "bsattn_decode_window_workspace_size", "call_workspace", "status_workspace",
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
    return int(load().bsattn_get_device_status(ws.data_ptr(), _stream(ws.device)))


def bsattn_set_wait_budget_ns(ns: int) -> None:
    load().bsattn_set_wait_budget_ns(int(ns))


# ----------------------------------------------------------------- paged serving

_STREAM_HEADER = 256 + 4 * 1024          # status word and tickets: all that has to start at zero


def call_workspace(device, purpose: str, nbytes: int) -> torch.Tensor:
    """A workspace for the stream decodes that no other call in flight uses: one per (stream, purpose),
    and a new one for every call captured into a CUDA graph (graphs may be replayed side by side)."""
    device = torch.device(device)
    capturing = torch.cuda.is_current_stream_capturing()
    key = (device.index, purpose, _stream(device))
    buf = None if capturing else _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        buf[:_STREAM_HEADER].zero_()
        if not capturing:
            _ws_cache[key] = buf
    return buf


_status_ws: dict = {}


def status_workspace(device) -> torch.Tensor:
    """The 256-byte workspace of the calls that keep only a status word in it.  They set bits of it and
    read nothing, so all of a device's streams and graphs share it."""
    device = torch.device(device)
    buf = _status_ws.get(device.index)
    if buf is None:
        buf = torch.zeros(256, dtype=torch.uint8, device=device)
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(device).synchronize()
            _status_ws[device.index] = buf
    return buf


def _same_device(**tensors):
    dev = None
    for name, t in tensors.items():
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if dev is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the other tensors on {dev}")
        dev = t.device
    return dev


def _contiguous(**tensors):
    for name, t in tensors.items():
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _dtypes(dtype, **tensors):
    for name, t in tensors.items():
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _shape(name, t, want):
    if tuple(t.shape) != tuple(want):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(want)}")


def _out(out, like):
    if out is None:
        return torch.empty(like.shape, dtype=like.dtype, device=like.device)
    if out.device != like.device or out.dtype != like.dtype:
        raise ValueError("out must have the queries' device and dtype")
    _shape("out", out, like.shape)
    return out


def bsattn_paged_plan(cached_lens, new_lens, free_pages, free_count, block_table, page_size: int,
                      max_tokens: int, ws=None):
    """Block-table rows and slot map for `new_lens` tokens on top of `cached_lens`, both int32 [B].
    free_pages int32 [n] is the free list, free_count int32 [1] how many of it are free (taken from the
    end); block_table int32 [B, max_pages] gets the new pages.  Returns (slots int64 [max_tokens], -1
    where there is no token; starts int32 [B + 1]; seqlens int32 [B]; free_left int32 [1])."""
    lib = load()
    dev = _same_device(cached_lens=cached_lens, new_lens=new_lens, free_pages=free_pages,
                       free_count=free_count, block_table=block_table)
    _contiguous(cached_lens=cached_lens, new_lens=new_lens, free_pages=free_pages, free_count=free_count,
                block_table=block_table)
    _dtypes(torch.int32, cached_lens=cached_lens, new_lens=new_lens, free_pages=free_pages,
            free_count=free_count, block_table=block_table)
    B = cached_lens.numel()
    _shape("new_lens", new_lens, cached_lens.shape)
    if cached_lens.dim() != 1 or block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("cached_lens must be [B] and block_table [B, max_pages]")
    if free_count.numel() != 1:
        raise ValueError("free_count must have one element")
    with torch.cuda.device(dev):
        slots = torch.empty(int(max_tokens), dtype=torch.int64, device=dev)
        ints = torch.empty(2 * B + 2, dtype=torch.int32, device=dev)
        starts, seqlens, left = ints[:B + 1], ints[B + 1:2 * B + 1], ints[2 * B + 1:]
        if ws is None:
            ws = status_workspace(dev)
        rc = lib.bsattn_paged_plan(cached_lens.data_ptr(), new_lens.data_ptr(), free_pages.data_ptr(),
                                   free_count.data_ptr(), block_table.data_ptr(), slots.data_ptr(),
                                   starts.data_ptr(), seqlens.data_ptr(), left.data_ptr(), B,
                                   int(page_size), block_table.shape[1], free_pages.numel(),
                                   int(max_tokens), ws.data_ptr(), ws.numel(), _stream(dev))
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
        return torch.zeros(num_pages, Hkv, page_size, n, dtype=torch.uint8, device=device)
    return Kv4Cache(make(d // 2), make(d // 16), make(d // 2), make(d // 16))


def _kv4(cache):
    c = Kv4Cache(*cache)
    _contiguous(**c._asdict())
    _dtypes(torch.uint8, **c._asdict())
    if c.k_codes.dim() != 4:
        raise ValueError("a 4-bit cache's tensors are [pages, Hkv, page_size, ...]")
    pages, hkv, page, half = c.k_codes.shape
    _shape("v_codes", c.v_codes, c.k_codes.shape)
    for name in ("k_scales", "v_scales"):
        _shape(name, getattr(c, name), (pages, hkv, page, half // 8))
    return c, pages, hkv, page, 2 * half


def bsattn_kv4_append(k, v, slots, cache, k_scale: float = 1.0, v_scale: float = 1.0, ws=None) -> None:
    """Rounds k and v [T, Hkv, d] fp16|bf16 (channels contiguous, any 16-byte aligned token and head
    strides) into the rows that slots int64 [T] names (negative: skipped; all others distinct)."""
    lib = load()
    c, pages, hkv, page, d = _kv4(cache)
    dev = _same_device(k=k, v=v, slots=slots, **c._asdict())
    _dtypes(torch.int64, slots=slots)
    _contiguous(slots=slots)
    if k.dim() != 3 or v.dtype != k.dtype:
        raise ValueError("k and v must be [T, Hkv, d] of one dtype")
    T = k.shape[0]
    _shape("k", k, (T, hkv, d))
    _shape("v", v, (T, hkv, d))
    _shape("slots", slots, (T,))
    for name, t in (("k", k), ("v", v)):
        if T and t.stride(2) != 1:
            raise ValueError(f"{name}'s channels must be contiguous")
    # the stride of a dimension of one entry is never used
    st = [t.stride(i) if t.shape[i] > 1 else 0 for t in (k, v) for i in (0, 1)]
    with torch.cuda.device(dev):
        if ws is None:
            ws = status_workspace(dev)
        rc = lib.bsattn_kv4_append(k.data_ptr(), v.data_ptr(), *st, slots.data_ptr(), *(t.data_ptr() for t in c),
                                   float(k_scale), float(v_scale), T, hkv, pages, page, d, _dtype_code(k),
                                   ws.data_ptr(), ws.numel(), _stream(dev))
    _check("bsattn_kv4_append", rc)


def bsattn_kv4_gather(slots, cache, dtype, k_scale: float = 1.0, v_scale: float = 1.0, ws=None):
    """The rows that slots int64 [T] names, as (k, v) [T, Hkv, d] of `dtype` (negative slots: zeros)."""
    lib = load()
    c, pages, hkv, page, d = _kv4(cache)
    dev = _same_device(slots=slots, **c._asdict())
    _dtypes(torch.int64, slots=slots)
    _contiguous(slots=slots)
    if slots.dim() != 1:
        raise ValueError("slots must be [T]")
    with torch.cuda.device(dev):
        k = torch.empty(slots.numel(), hkv, d, dtype=dtype, device=dev)
        v = torch.empty_like(k)
        if ws is None:
            ws = status_workspace(dev)
        rc = lib.bsattn_kv4_gather(slots.data_ptr(), *(t.data_ptr() for t in c), float(k_scale), float(v_scale),
                                   k.data_ptr(), v.data_ptr(), slots.numel(), hkv, pages, page, d,
                                   _dtype_code(k), ws.data_ptr(), ws.numel(), _stream(dev))
    _check("bsattn_kv4_gather", rc)
    return k, v


def bsattn_decode_window_workspace_size(Hq: int, Hkv: int, d: int) -> int:
    return int(load().bsattn_decode_window_workspace_size(Hq, Hkv, d))


def bsattn_decode_kv4_workspace_size(Hq: int, Hkv: int, d: int) -> int:
    return int(load().bsattn_decode_kv4_workspace_size(Hq, Hkv, d))


def _decode_args(q, cache_seqlens, block_table, hkv, d):
    if q.dim() != 3 or q.shape[2] != d:
        raise ValueError(f"q must be [B, Hq, {d}]")
    _contiguous(q=q, cache_seqlens=cache_seqlens)
    _dtypes(torch.int32, cache_seqlens=cache_seqlens)
    _shape("cache_seqlens", cache_seqlens, (q.shape[0],))
    if block_table is not None:
        _contiguous(block_table=block_table)
        _dtypes(torch.int32, block_table=block_table)
        if block_table.dim() != 2 or block_table.shape[0] != q.shape[0]:
            raise ValueError("block_table must be [B, max_pages]")


def bsattn_decode_paged_kv4(q, cache, cache_seqlens, block_table, block_indices=None, window: int = 0,
                            sinks: int = 0, k_scale: float = 1.0, v_scale: float = 1.0, out=None, ws=None):
    """One query token per sequence over a paged 4-bit cache.  q [B,Hq,d] fp16|bf16; cache_seqlens int32
    [B]; block_table int32 [B,max_pages]; block_indices int32 [B,Hkv,max_sel] (-1 = empty) limits each kv
    head to chosen 64-token blocks, window > 0 to the last `window` tokens and the first `sinks`."""
    lib = load()
    c, pages, hkv, page, d = _kv4(cache)
    dev = _same_device(q=q, cache_seqlens=cache_seqlens, block_table=block_table, **c._asdict())
    _decode_args(q, cache_seqlens, block_table, hkv, d)
    B, Hq, _ = q.shape
    max_sel, chosen = 0, None
    if block_indices is not None:
        _same_device(q=q, block_indices=block_indices)
        _contiguous(block_indices=block_indices)
        _dtypes(torch.int32, block_indices=block_indices)
        if block_indices.dim() != 3 or tuple(block_indices.shape[:2]) != (B, hkv):
            raise ValueError("block_indices must be [B, Hkv, max_sel]")
        max_sel, chosen = block_indices.shape[2], block_indices.data_ptr()
        if max_sel == 0:
            raise ValueError("block_indices has no slots")
    with torch.cuda.device(dev):
        out = _out(out, q)
        _contiguous(out=out)
        if ws is None:
            ws = call_workspace(dev, "decode_kv4", bsattn_decode_kv4_workspace_size(Hq, hkv, d))
        rc = lib.bsattn_decode_paged_kv4(q.data_ptr(), *(t.data_ptr() for t in c), float(k_scale), float(v_scale),
                                         cache_seqlens.data_ptr(), chosen, block_table.data_ptr(), int(window),
                                         int(sinks), out.data_ptr(), B, Hq, hkv, pages, page,
                                         block_table.shape[1], d, max_sel, _dtype_code(q), ws.data_ptr(),
                                         ws.numel(), _stream(dev))
    _check("bsattn_decode_paged_kv4", rc)
    return out


def bsattn_decode_window(q, k, v, cache_seqlens, window: int, sinks: int = 0, out=None, ws=None):
    """One query token per sequence over the last `window` tokens and the first `sinks` of a contiguous
    cache.  q [B,Hq,d]; k/v [B,Smax,Hkv,d] fp16|bf16 CUDA; cache_seqlens int32 [B]."""
    lib = load()
    dev = _same_device(q=q, k=k, v=v, cache_seqlens=cache_seqlens)
    _contiguous(k=k, v=v)
    if k.dim() != 4 or k.shape[0] != q.shape[0] or k.shape != v.shape:
        raise ValueError("k and v must be [B, Smax, Hkv, d]")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k, v must share a dtype")
    _, Smax, hkv, d = k.shape
    _decode_args(q, cache_seqlens, None, hkv, d)
    B, Hq, _ = q.shape
    with torch.cuda.device(dev):
        out = _out(out, q)
        _contiguous(out=out)
        if ws is None:
            ws = call_workspace(dev, "decode_window", bsattn_decode_window_workspace_size(Hq, hkv, d))
        rc = lib.bsattn_decode_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), cache_seqlens.data_ptr(),
                                      int(window), int(sinks), out.data_ptr(), B, Hq, hkv, Smax, d,
                                      _dtype_code(q), ws.data_ptr(), ws.numel(), _stream(dev))
    _check("bsattn_decode_window", rc)
    return out


def bsattn_decode_window_paged(q, k_pages, v_pages, cache_seqlens, block_table, window: int, sinks: int = 0,
                               out=None, ws=None):
    """bsattn_decode_window over a paged cache: k_pages/v_pages [num_pages,page_size,Hkv,d]; block_table
    int32 [B,max_pages]."""
    lib = load()
    dev = _same_device(q=q, k_pages=k_pages, v_pages=v_pages, cache_seqlens=cache_seqlens,
                       block_table=block_table)
    _contiguous(k_pages=k_pages, v_pages=v_pages)
    if k_pages.dim() != 4 or k_pages.shape != v_pages.shape:
        raise ValueError("k_pages and v_pages must be [num_pages, page_size, Hkv, d]")
    if not (q.dtype == k_pages.dtype == v_pages.dtype):
        raise TypeError("q, k_pages, v_pages must share a dtype")
    pages, page, hkv, d = k_pages.shape
    _decode_args(q, cache_seqlens, block_table, hkv, d)
    B, Hq, _ = q.shape
    with torch.cuda.device(dev):
        out = _out(out, q)
        _contiguous(out=out)
        if ws is None:
            ws = call_workspace(dev, "decode_window", bsattn_decode_window_workspace_size(Hq, hkv, d))
        rc = lib.bsattn_decode_window_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                            cache_seqlens.data_ptr(), block_table.data_ptr(), int(window),
                                            int(sinks), out.data_ptr(), B, Hq, hkv, pages, page,
                                            block_table.shape[1], d, _dtype_code(q), ws.data_ptr(), ws.numel(),
                                            _stream(dev))
    _check("bsattn_decode_window_paged", rc)
    return out


def bsattn_prefill_window(q, k, v, window: int, sinks: int = 0, out=None, ws=None):
    """Causal attention with a sliding window and sinks: query row i (position p = i + Sk - Sq) sees key j
    iff j <= p and (j < sinks or j > p - window).  q [B,Hq,Sq,d], k/v [B,Hkv,Sk,d] fp16|bf16 CUDA views
    with contiguous channels and 16-byte aligned strides; out: as q laid out, unless given."""
    lib = load()
    dev = _same_device(q=q, k=k, v=v)
    if q.dim() != 4 or k.dim() != 4 or k.shape != v.shape or q.shape[0] != k.shape[0] or q.shape[3] != k.shape[3]:
        raise ValueError("q must be [B, Hq, Sq, d], k and v [B, Hkv, Sk, d]")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k, v must share a dtype")
    B, Hq, Sq, d = q.shape
    hkv, Sk = k.shape[1], k.shape[2]
    with torch.cuda.device(dev):
        if out is None:
            out = torch.empty_like(q)
        out = _out(out, q)
        for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
            if t.numel() and t.stride(3) != 1:
                raise ValueError(f"{name}'s channels must be contiguous")
        strides = (ctypes.c_int64 * 12)(*(s for t in (q, k, v, out) for s in t.stride()[:3]))
        if ws is None:
            ws = status_workspace(dev)
        rc = lib.bsattn_prefill_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), int(window), int(sinks),
                                       out.data_ptr(), B, Hq, hkv, Sq, Sk, d, strides, _dtype_code(q),
                                       ws.data_ptr(), ws.numel(), _stream(dev))
    _check("bsattn_prefill_window", rc)
    return out
