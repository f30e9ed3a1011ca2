"""Python binding of libpagedattn (ctypes): argument marshalling only.

Every function here checks tensor devices, dtypes and shapes, then calls the
C ABI declared in ``include/pagedattn.h`` and ``include/pagedattn/`` with raw
device pointers and the current torch CUDA stream. All computation happens in the library's CUDA
kernels; there is no fallback. If the shared library has not been built, the
first call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

PA_OK, PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_WORKSPACE, PA_ERR_CUDA = range(5)

# every entry point the headers declare, with its ctypes signature
_P, _I32, _I64, _F32, _F64, _SZ = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                                   ctypes.c_double, ctypes.c_size_t)
SIGNATURES = {
    "pa_status_string": ([_I32], ctypes.c_char_p),
    "pa_store_kvcache": ([_P, _P, _P, _P, _P, _I64, _I32, _I32, _I32, _I64, _P], _I32),
    "pa_decode_workspace_size": ([_I32, _I32, _I32, _I32], _SZ),
    "pa_decode": ([_P, _P, _P, _P, _I32, _P, _F32, _P, _I32, _I32, _I32, _I32, _I32, _I64,
                   _P, _SZ, _P], _I32),
    "pa_decode_splitk": ([_P, _P, _P, _P, _I32, _P, _F32, _P, _I32, _I32, _I32, _I32, _I32,
                          _I64, _P, _SZ, _I32, _P], _I32),
    "pa_decode_noalloc": ([_P, _P, _P, _P, _I32, _P, _F32, _P, _I32, _I32, _I32, _I32, _I32,
                           _I64, _P], _I32),
    "pa_decode_multi_workspace_size": ([_I32, _I32, _I32, _I32], _SZ),
    "pa_prefill": ([_P, _P, _P, _P, _I32, _P, _P, _I32, _F32, _P, _I32, _I32, _I32, _I32, _I32,
                    _I32, _I64, _P], _I32),
    "pa_take_device_error": ([_P, _P], _I32),
    "pa_debug_prefill_fault": ([_I32], _I32),
    "pa_debug_kernel_variant": ([_I32], _I32),
    "pa_prefill_layout": ([_P, _P, _P, _P, _I32, _P, _P, _I32, _F32, _P, _I32, _I32, _I32, _I32,
                           _I32, _I32, _I64, _I32, _P], _I32),
    "pa_store_kvcache_layout": ([_P, _P, _P, _P, _P, _I64, _I32, _I32, _I32, _I64, _I32, _P],
                                _I32),
    "pa_decode_layout": ([_P, _P, _P, _P, _I32, _P, _F32, _P, _I32, _I32, _I32, _I32, _I32, _I64,
                          _I32, _P, _SZ, _I32, _P], _I32),
    "pa_decode_multi": ([_P, _P, _P, _P, _I32, _P, _I32, _F32, _P, _I32, _I32, _I32, _I32, _I32,
                         _I64, _P, _SZ, _P], _I32),
    "pa_decode_step": ([_P, _P, _P, _I64, _P, _P, _P, _P, _I32, _P, _F32, _P, _I32, _I32, _I32,
                        _I32, _I32, _I64, _I32, _P, _SZ, _P], _I32),
    "pa_decode_shared_workspace_size": ([_I32, _I32, _I32, _I32, _I32], _SZ),
    "pa_decode_shared": ([_P, _P, _P, _P, _I32, _P, _P, _P, _I32, _F32, _P, _I32, _I32, _I32, _I32,
                          _I32, _I64, _I32, _P, _SZ, _P], _I32),
    "pa_copy_blocks": ([_P, _I32, _P, _I64, _I32, _I32, _I32, _I64, _P], _I32),
    "pa_blocks_workspace_size": ([_I32, _I64], _SZ),
    "pa_fork_blocks": ([_P, _I32, _P, _I32, _P, _I32, _P, _P, _P, _I32, _I32, _I32, _I32, _I64,
                        _I32, _P, _SZ, _P], _I32),
    "pa_free_blocks": ([_P, _I32, _P, _I32, _P, _P, _I32, _I32, _I64, _P], _I32),
    "pa_compact_blocks": ([_P, _I32, _P, _I32, _P, _I32, _P, _P, _P, _I32, _I32, _I32, _I64, _P,
                           _SZ, _P], _I32),
    "pa_decode_tree_workspace_size": ([_I32, _I32, _I32], _SZ),
    "pa_decode_tree": ([_P, _P, _P, _P, _I32, _P, _P, _P, _I32, _F32, _P, _I32, _I32, _I32, _I32, _I32, _I32, _I64,
                        _I32, _P, _SZ, _P], _I32),
    "pa_keep_tokens": ([_P, _I32, _P, _I32, _P, _P, _P, _I32, _I32, _P, _I32, _I32, _I32, _I64, _I32, _P], _I32),
    "pa_rotary_init": ([_P, _I32, _I32, _F64, _I32, _F64, _F64, _F64, _F64, _F64], _I32),
    "pa_rotary_init_frequencies": ([_P, _I32, _I32, _P, _F64], _I32),
    "pa_rotate": ([_P, _I64, _I64, _P, _I64, _I64, _I32, _P, _I64, _I64, _P, _I64, _I64, _I32, _I32, _P, _I64, _P,
                   _P, _P, _F32, _P], _I32),
    "pa_append_kvcache": ([_P, _I64, _I64, _P, _I64, _I64, _I32, _P, _I64, _I64, _P, _I64, _I64, _I32, _I32, _P, _P,
                           _P, _I32, _I64, _I32, _P, _I64, _P, _P, _P, _F32, _P], _I32),
    "pa_decode_multi_layout": ([_P, _P, _P, _P, _I32, _P, _I32, _F32, _P, _I32, _I32, _I32, _I32,
                                _I32, _I64, _I32, _P, _SZ, _P], _I32),
}

_lock = threading.Lock()
_lib = None
_workspaces = {}


class PagedAttnError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")


def library_path() -> str:
    return _build.LIB_PATH


def lib() -> ctypes.CDLL:
    """The loaded libpagedattn; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.LIB_PATH
            if not os.path.exists(path):
                raise RuntimeError(
                    f"libpagedattn is not built ({path} missing): run "
                    "paged_kv_cache_255_gb300.build.build() first")
            handle = ctypes.CDLL(path)
            for name, (args, res) in SIGNATURES.items():
                fn = getattr(handle, name)
                fn.argtypes = args
                fn.restype = res
            _lib = handle
    return _lib


def status_string(status: int) -> str:
    return lib().pa_status_string(int(status)).decode()


def _check(fn: str, status: int):
    if status != PA_OK:
        raise PagedAttnError(fn, status)


def _stream_ptr(stream, device) -> int:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return int(stream.cuda_stream)


def _cuda(t: torch.Tensor, name: str, dtype, device=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def store_kvcache(k, v, k_cache, v_cache, slot_mapping, stream=None, head_major=False):
    """Write row i of k/v to cache slot slot_mapping[i] (-1 rows skipped).

    k, v: bf16 [N, Hkv, D]; k_cache, v_cache: bf16 [NB, bs, Hkv, D], or
    [NB, Hkv, bs, D] with ``head_major``; slot_mapping: int64 [N]. Runs on the
    current stream (or ``stream``).
    """
    dev = k_cache.device
    for t, n, dt in ((k, "k", torch.bfloat16), (v, "v", torch.bfloat16),
                     (k_cache, "k_cache", torch.bfloat16), (v_cache, "v_cache", torch.bfloat16),
                     (slot_mapping, "slot_mapping", torch.int64)):
        _cuda(t, n, dt, dev)
    if head_major:
        NB, Hkv, bs, D = k_cache.shape
    else:
        NB, bs, Hkv, D = k_cache.shape
    N = slot_mapping.shape[0]
    if v_cache.shape != k_cache.shape or k.shape != (N, Hkv, D) or v.shape != (N, Hkv, D):
        raise ValueError("shape mismatch between k, v, caches and slot_mapping")
    with torch.cuda.device(dev):
        st = lib().pa_store_kvcache_layout(k.data_ptr(), v.data_ptr(), k_cache.data_ptr(),
                                           v_cache.data_ptr(), slot_mapping.data_ptr(), N, Hkv,
                                           D, bs, NB, 1 if head_major else 0,
                                           _stream_ptr(stream, dev))
    _check("pa_store_kvcache", st)


def decode_step(k_new, v_new, slot_mapping, q, k_cache, v_cache, block_tables, context_lens,
                scale, out=None, workspace=None, stream=None, head_major=False):
    """One decode step through pa_decode_step: store the step's new K/V rows
    (``k_new``, ``v_new`` bf16 [N, Hkv, D] at ``slot_mapping`` int64 [N]),
    then single-token decode over the updated cache; returns ``out``. Same
    results as store_kvcache followed by decode; the decode plans its work
    split while the store runs."""
    dev = q.device
    for t, n, dt in ((k_new, "k_new", torch.bfloat16), (v_new, "v_new", torch.bfloat16),
                     (slot_mapping, "slot_mapping", torch.int64), (q, "q", torch.bfloat16),
                     (k_cache, "k_cache", torch.bfloat16), (v_cache, "v_cache", torch.bfloat16),
                     (block_tables, "block_tables", torch.int32),
                     (context_lens, "context_lens", torch.int32)):
        _cuda(t, n, dt, dev)
    S, Hq, D = q.shape
    if head_major:
        NB, Hkv, bs, D2 = k_cache.shape
    else:
        NB, bs, Hkv, D2 = k_cache.shape
    N = slot_mapping.shape[0]
    if v_cache.shape != k_cache.shape or D2 != D or block_tables.dim() != 2 \
            or block_tables.shape[0] != S or context_lens.shape != (S,) \
            or k_new.shape != (N, Hkv, D) or v_new.shape != (N, Hkv, D):
        raise ValueError("shape mismatch between the step's tensors")
    if out is None:
        out = torch.empty_like(q)
    else:
        _cuda(out, "out", torch.bfloat16, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if workspace is None:
        workspace = workspace_for(Hq, Hkv, D, 0, dev)
    else:
        _cuda(workspace, "workspace", workspace.dtype, dev)
    with torch.cuda.device(dev):
        st = lib().pa_decode_step(k_new.data_ptr(), v_new.data_ptr(), slot_mapping.data_ptr(), N,
                                  q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                  block_tables.data_ptr(), block_tables.shape[1],
                                  context_lens.data_ptr(), float(scale), out.data_ptr(), S, Hq,
                                  Hkv, D, bs, NB, 1 if head_major else 0, workspace.data_ptr(),
                                  workspace.numel() * workspace.element_size(),
                                  _stream_ptr(stream, dev))
    _check("pa_decode_step", st)
    return out


def decode_workspace_size(num_q_heads: int, num_kv_heads: int, head_dim: int = 128,
                          num_partitions: int = 0, device=None) -> int:
    """Workspace bytes pa_decode needs on ``device`` (default: current)."""
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        n = lib().pa_decode_workspace_size(num_q_heads, num_kv_heads, head_dim, num_partitions)
    if n == 0:
        raise ValueError("unsupported head configuration")
    return int(n)


def workspace_for(num_q_heads, num_kv_heads, head_dim=128, num_partitions=0, device=None):
    """A cached uint8 workspace tensor big enough for these heads on ``device``."""
    device = torch.device(device if device is not None else f"cuda:{torch.cuda.current_device()}")
    n = decode_workspace_size(num_q_heads, num_kv_heads, head_dim, num_partitions, device)
    key = (device, n)
    ws = _workspaces.get(key)
    if ws is None:
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


def decode(q, k_cache, v_cache, block_tables, context_lens, scale, out=None, workspace=None,
           num_partitions: int = 0, stream=None, head_major=False):
    """Single-token paged decode attention; returns ``out`` (bf16 [S, Hq, D]).

    q: bf16 [S, Hq, D]; caches: bf16 [NB, bs, Hkv, D] ([NB, Hkv, bs, D] with
    ``head_major``); block_tables: int32 [S, max_blocks]; context_lens: int32
    [S]. ``num_partitions`` > 0 forces the split-K share count
    (pa_decode_splitk).
    """
    dev = q.device
    for t, n, dt in ((q, "q", torch.bfloat16), (k_cache, "k_cache", torch.bfloat16),
                     (v_cache, "v_cache", torch.bfloat16), (block_tables, "block_tables", torch.int32),
                     (context_lens, "context_lens", torch.int32)):
        _cuda(t, n, dt, dev)
    S, Hq, D = q.shape
    if head_major:
        NB, Hkv, bs, D2 = k_cache.shape
    else:
        NB, bs, Hkv, D2 = k_cache.shape
    if v_cache.shape != k_cache.shape or D2 != D or block_tables.dim() != 2 \
            or block_tables.shape[0] != S or context_lens.shape != (S,):
        raise ValueError("shape mismatch between q, caches, block_tables and context_lens")
    if out is None:
        out = torch.empty_like(q)
    else:
        _cuda(out, "out", torch.bfloat16, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if workspace is None:
        workspace = workspace_for(Hq, Hkv, D, num_partitions, dev)
    else:
        _cuda(workspace, "workspace", workspace.dtype, dev)
    ws_bytes = workspace.numel() * workspace.element_size()
    args = (q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
            block_tables.shape[1], context_lens.data_ptr(), float(scale), out.data_ptr(), S, Hq,
            Hkv, D, bs, NB, workspace.data_ptr(), ws_bytes)
    with torch.cuda.device(dev):
        if head_major:
            st = lib().pa_decode_layout(*args[:14], 1, *args[14:], int(num_partitions),
                                        _stream_ptr(stream, dev))
        elif num_partitions:
            st = lib().pa_decode_splitk(*args, int(num_partitions), _stream_ptr(stream, dev))
        else:
            st = lib().pa_decode(*args, _stream_ptr(stream, dev))
    _check("pa_decode", st)
    return out


def decode_multi(q, k_cache, v_cache, block_tables, context_lens, scale, out=None,
                 workspace=None, stream=None, head_major=False):
    """Decode of Q new tokens per sequence (speculative verification): q is
    bf16 [S, Q, Hq, D]; query token i attends to keys t <= L - Q + i, with
    L = context_lens[s] counting all Q new tokens. The pool is
    [NB, bs, Hkv, D], or [NB, Hkv, bs, D] with head_major=True. Returns out
    [S, Q, Hq, D]."""
    dev = q.device
    for t, n, dt in ((q, "q", torch.bfloat16), (k_cache, "k_cache", torch.bfloat16),
                     (v_cache, "v_cache", torch.bfloat16), (block_tables, "block_tables", torch.int32),
                     (context_lens, "context_lens", torch.int32)):
        _cuda(t, n, dt, dev)
    S, Q, Hq, D = q.shape
    if head_major:
        NB, Hkv, bs, D2 = k_cache.shape
    else:
        NB, bs, Hkv, D2 = k_cache.shape
    if v_cache.shape != k_cache.shape or D2 != D or block_tables.dim() != 2 \
            or block_tables.shape[0] != S or context_lens.shape != (S,):
        raise ValueError("shape mismatch between q, caches, block_tables and context_lens")
    if out is None:
        out = torch.empty_like(q)
    else:
        _cuda(out, "out", torch.bfloat16, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if workspace is None:
        with torch.cuda.device(dev):
            n = lib().pa_decode_multi_workspace_size(Q, Hq, Hkv, D)
        if n == 0:
            raise ValueError("unsupported query-token / head configuration")
        key = (dev, "multi", n)
        workspace = _workspaces.get(key)
        if workspace is None:
            workspace = torch.zeros(n, dtype=torch.uint8, device=dev)
            _workspaces[key] = workspace
    else:
        _cuda(workspace, "workspace", workspace.dtype, dev)
    ws_bytes = workspace.numel() * workspace.element_size()
    with torch.cuda.device(dev):
        st = lib().pa_decode_multi_layout(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                          block_tables.data_ptr(), block_tables.shape[1],
                                          context_lens.data_ptr(), Q, float(scale),
                                          out.data_ptr(), S, Hq, Hkv, D, bs, NB,
                                          1 if head_major else 0,
                                          workspace.data_ptr(), ws_bytes, _stream_ptr(stream, dev))
    _check("pa_decode_multi_layout", st)
    return out


def decode_shared(q, k_cache, v_cache, block_tables, context_lens, group_starts, prefix_blocks, scale,
                  out=None, workspace=None, stream=None, head_major=False):
    """Single-token decode for sequences in groups that share their first
    blocks; returns ``out`` (bf16 [S, Hq, D]).

    group_starts: int32 [G + 1]; group g is sequences group_starts[g] ..
    group_starts[g + 1] - 1, whose first prefix_blocks[g] (int32 [G]) table
    entries are the same. The prefix is read once per group, as far as the group's
    shortest non-empty sequence reaches; the results are decode's, but for the
    order of the sums. Rows of ``out`` outside all groups are left as they were.
    The other arguments are decode's."""
    dev = q.device
    if not _fits(dev.index, torch.bfloat16, q, k_cache, v_cache):
        _explain(dev, torch.bfloat16, q=q, k_cache=k_cache, v_cache=v_cache)
    if not _fits(dev.index, torch.int32, block_tables, context_lens, group_starts, prefix_blocks):
        _explain(dev, torch.int32, block_tables=block_tables, context_lens=context_lens,
                 group_starts=group_starts, prefix_blocks=prefix_blocks)
    S, Hq, D = q.shape
    if head_major:
        NB, Hkv, bs, D2 = k_cache.shape
    else:
        NB, bs, Hkv, D2 = k_cache.shape
    G = prefix_blocks.shape[0]
    if v_cache.shape != k_cache.shape or D2 != D or block_tables.dim() != 2 \
            or block_tables.shape[0] != S or context_lens.shape != (S,) \
            or prefix_blocks.dim() != 1 or group_starts.shape != (G + 1,):
        raise ValueError("shape mismatch between q, caches, block_tables, context_lens and groups")
    if out is None:
        out = _new(q.shape, q.dtype, dev, stream)
    else:
        _cuda(out, "out", torch.bfloat16, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if workspace is None:
        workspace = _scratch("shared", decode_shared_workspace_size(S, G, Hq, Hkv, D, dev), dev, stream)
    else:
        _cuda(workspace, "workspace", workspace.dtype, dev)
    _call("pa_decode_shared", dev, stream, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
          block_tables.data_ptr(), block_tables.shape[1], context_lens.data_ptr(),
          group_starts.data_ptr(), prefix_blocks.data_ptr(), G, float(scale), out.data_ptr(), S, Hq, Hkv,
          D, bs, NB, 1 if head_major else 0, workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return out


def decode_shared_workspace_size(num_seqs: int, num_groups: int, num_q_heads: int, num_kv_heads: int,
                                 head_dim: int = 128, device=None) -> int:
    """Workspace bytes pa_decode_shared needs on ``device`` (default: current)."""
    index = None if device is None else torch.device(device).index
    if index is None:       # no device, or "cuda": the current one
        index = torch.cuda.current_device()
    n = _size("pa_decode_shared_workspace_size", index, num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim)
    if n == 0:
        raise ValueError("unsupported head configuration or number of groups")
    return n


def prefill(q, k_cache, v_cache, block_tables, context_lens, query_start_loc, scale,
            max_query_len=None, out=None, stream=None, head_major=False):
    """Paged prefill: q is bf16 [total_q, Hq, D], rows packed per sequence by
    query_start_loc (int32 [S + 1]); row i of sequence s sits at position
    context_lens[s] - n_s + i and attends causally to the sequence's cached
    tokens. The pool is [NB, bs, Hkv, D], or [NB, Hkv, bs, D] with
    head_major=True. Returns out [total_q, Hq, D]."""
    dev = q.device
    for t, n, dt in ((q, "q", torch.bfloat16), (k_cache, "k_cache", torch.bfloat16),
                     (v_cache, "v_cache", torch.bfloat16), (block_tables, "block_tables", torch.int32),
                     (context_lens, "context_lens", torch.int32),
                     (query_start_loc, "query_start_loc", torch.int32)):
        _cuda(t, n, dt, dev)
    T, Hq, D = q.shape
    if head_major:
        NB, Hkv, bs, D2 = k_cache.shape
    else:
        NB, bs, Hkv, D2 = k_cache.shape
    S = context_lens.shape[0]
    if v_cache.shape != k_cache.shape or D2 != D or block_tables.dim() != 2 \
            or block_tables.shape[0] != S or query_start_loc.shape != (S + 1,):
        raise ValueError("shape mismatch between q, caches, block_tables and query_start_loc")
    if max_query_len is None:
        max_query_len = int((query_start_loc[1:] - query_start_loc[:-1]).max().item()) if S else 0
    if out is None:
        out = torch.empty_like(q)
    else:
        _cuda(out, "out", torch.bfloat16, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    with torch.cuda.device(dev):
        st = lib().pa_prefill_layout(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                     block_tables.data_ptr(), block_tables.shape[1],
                                     context_lens.data_ptr(), query_start_loc.data_ptr(),
                                     int(max_query_len), float(scale), out.data_ptr(), S, T, Hq,
                                     Hkv, D, bs, NB, 1 if head_major else 0,
                                     _stream_ptr(stream, dev))
    _check("pa_prefill_layout", st)
    return out


class CachePools:
    """The pools that share one set of block ids, normally the K and the V pool
    of every layer: bf16 [NB, bs, Hkv, 128], or [NB, Hkv, bs, 128] with
    ``head_major``, all of one shape on one device. Made once for the life of
    the pools (checked here, not at every call); keeps them alive."""

    def __init__(self, caches, head_major=False):
        caches = list(caches)
        if not caches:
            raise ValueError("no pools")
        dev, shape = caches[0].device, caches[0].shape
        for c in caches:
            _cuda(c, "cache", torch.bfloat16, dev)
            if c.shape != shape or c.dim() != 4:
                raise ValueError("the pools must be 4-D tensors of one shape")
        if len({c.data_ptr() for c in caches}) != len(caches):
            raise ValueError("a pool is listed twice")
        self.caches, self.device, self.head_major = caches, dev, bool(head_major)
        self.num_blocks = shape[0]
        self.num_kv_heads, self.block_size = (shape[1], shape[2]) if head_major else (shape[2], shape[1])
        self.head_dim = shape[3]
        self._ptrs = (ctypes.c_void_p * len(caches))(*(c.data_ptr() for c in caches))
        self._args = (ctypes.addressof(self._ptrs), len(caches))
        self._shape = (self.num_kv_heads, self.head_dim, self.block_size, self.num_blocks)


_raw_stream = torch._C._cuda_getCurrentRawStream


def _fits(index, dtype, *tensors):
    """Whether every tensor is a contiguous one of this dtype on CUDA device
    ``index``. The calls below cost a few microseconds on the GPU, less than
    _cuda takes for each argument in turn; it is asked only for the message."""
    try:
        for t in tensors:
            if t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
                return False
    except (AttributeError, TypeError):
        return False
    return True


def _explain(dev, dtype, **tensors):
    """Raise for the first tensor that is why _fits said no."""
    for n, t in tensors.items():
        _cuda(t, n, dtype, dev)


def _check_table_shapes(block_tables, context_lens, ref_counts):
    if block_tables.dim() != 2 or context_lens.shape != block_tables.shape[:1] or ref_counts.dim() != 1:
        raise ValueError("shape mismatch between block_tables, context_lens and ref_counts")


def _call(fn, dev, stream, *args):
    """One library call on ``dev`` and ``stream`` (None: the current one)."""
    index = dev.index
    st = _raw_stream(index) if stream is None else stream.cuda_stream
    f = getattr(_lib or lib(), fn)
    if torch._C._cuda_getDevice() == index:
        status = f(*args, st)
    else:
        with torch.cuda.device(dev):
            status = f(*args, st)
    if status != PA_OK:
        raise PagedAttnError(fn, status)


def _new(shape, dtype, dev, stream):
    """An output or workspace of a call on ``stream`` (None: the current one).
    For another stream it comes from that stream's memory: what the current
    stream has freed may still be in use there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=dev)
    t.record_stream(torch.cuda.current_stream(dev))     # the caller may use it there, too
    return t


_kept = threading.local()


def _scratch(kind, nbytes, dev, stream):
    """Workspace of one call. Calls of one kind from one thread on its current
    stream run one after the other and share a buffer that is kept (an
    allocation costs as much as the rest of a short call); a call on another
    stream, and every captured call, gets one of its own from torch's allocator,
    so calls that may run at the same time never share. The largest of a kind is
    kept until the thread ends (for decode_shared tens of MB and more:
    decode_shared_workspace_size); a caller that passes a workspace keeps none here."""
    if stream is not None or torch._C._cuda_isCurrentStreamCapturing():
        return _new(nbytes, torch.uint8, dev, stream)
    key = (kind, dev.index, _raw_stream(dev.index))
    ws = _kept.__dict__.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = _kept.__dict__[key] = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    return ws


_sizes = {}
_MOST_SIZES = 4096


def _size(fn, index, *args):
    """The library's answer to a workspace size question, asked once for the
    same sizes on the same device (0, for sizes it does not take or after an
    error of the driver, every time). A serving loop asks for many sizes: the
    answers kept are thrown away when there are _MOST_SIZES."""
    key = (fn, index, args)
    n = _sizes.get(key)
    if n is None:
        with torch.cuda.device(index):
            n = int(getattr(lib(), fn)(*args))
        if n:
            if len(_sizes) >= _MOST_SIZES:
                _sizes.clear()
            _sizes[key] = n
    return n


def copy_blocks(pools: CachePools, block_pairs, stream=None):
    """Block ``block_pairs[i, 1]`` becomes a copy of block ``block_pairs[i, 0]``
    in every pool (int32 [n, 2]; pairs holding -1 are skipped). A block one
    pair writes must not stand in another pair."""
    dev = pools.device
    if not _fits(dev.index, torch.int32, block_pairs):
        _explain(dev, torch.int32, block_pairs=block_pairs)
    if block_pairs.dim() != 2 or block_pairs.shape[1] != 2:
        raise ValueError("block_pairs must be [n, 2]")
    _call("pa_copy_blocks", dev, stream, *pools._args, block_pairs.data_ptr(),
          block_pairs.shape[0], *pools._shape)


def fork_blocks(pools: CachePools, block_tables, context_lens, ref_counts, parents, children,
                workspace=None, stream=None):
    """Row ``children[i]`` becomes a second sequence with the tokens of row
    ``parents[i]`` (int32 [n]): full blocks are shared (their counts go up), a
    partly filled last block is copied into the lowest free block. Changes
    block_tables, context_lens, ref_counts and the pools in place. The child
    rows must be empty; forks that cannot be made change nothing and are
    recorded (take_device_error: 6)."""
    dev = pools.device
    if not _fits(dev.index, torch.int32, block_tables, context_lens, ref_counts, parents, children):
        _explain(dev, torch.int32, block_tables=block_tables, context_lens=context_lens,
                 ref_counts=ref_counts, parents=parents, children=children)
    _check_table_shapes(block_tables, context_lens, ref_counts)
    if parents.dim() != 1 or children.shape != parents.shape:
        raise ValueError("parents and children must be [n]")
    n, (rows, width) = parents.shape[0], block_tables.shape
    if ref_counts.shape[0] != pools.num_blocks:
        raise ValueError("ref_counts must have one entry per block")
    if n > rows:
        raise ValueError("more forks than rows")
    if workspace is None:
        workspace = _scratch("blocks", _size("pa_blocks_workspace_size", dev.index, rows, pools.num_blocks), dev,
                             stream)
    else:
        _cuda(workspace, "workspace", workspace.dtype, dev)
    _call("pa_fork_blocks", dev, stream, *pools._args, block_tables.data_ptr(), width,
          context_lens.data_ptr(), rows, ref_counts.data_ptr(), parents.data_ptr(),
          children.data_ptr(), n, *pools._shape, 1 if pools.head_major else 0,
          workspace.data_ptr(), workspace.numel() * workspace.element_size())


def free_blocks(block_tables, context_lens, ref_counts, rows, block_size: int, stream=None):
    """The listed rows (int32 [n]; -1 is skipped) give up their blocks: counts
    go down by one per entry, entries and lengths become 0."""
    dev = block_tables.device
    if not _fits(dev.index, torch.int32, block_tables, context_lens, ref_counts, rows):
        _explain(dev, torch.int32, block_tables=block_tables, context_lens=context_lens,
                 ref_counts=ref_counts, rows=rows)
    _check_table_shapes(block_tables, context_lens, ref_counts)
    if rows.dim() != 1:
        raise ValueError("rows must be [n]")
    _call("pa_free_blocks", dev, stream, block_tables.data_ptr(), block_tables.shape[1],
          context_lens.data_ptr(), block_tables.shape[0], ref_counts.data_ptr(), rows.data_ptr(),
          rows.shape[0], int(block_size), ref_counts.shape[0])


def compact_blocks(pools: CachePools, block_tables, context_lens, ref_counts, remap=None,
                   num_live=None, workspace=None, stream=None):
    """The live blocks move to ids 1 .. n in every pool with the fewest moves;
    block_tables and ref_counts follow. Returns (remap, num_live): int32 [NB],
    the new id of every live block and 0 for the others, and int32 [1], n."""
    dev = pools.device
    if not _fits(dev.index, torch.int32, block_tables, context_lens, ref_counts):
        _explain(dev, torch.int32, block_tables=block_tables, context_lens=context_lens, ref_counts=ref_counts)
    _check_table_shapes(block_tables, context_lens, ref_counts)
    NB, (rows, width) = pools.num_blocks, block_tables.shape
    if ref_counts.shape[0] != NB:
        raise ValueError("ref_counts must have one entry per block")
    if remap is None:
        remap = _new(NB, torch.int32, dev, stream)
    elif not _fits(dev.index, torch.int32, remap) or remap.shape != (NB,):
        _explain(dev, torch.int32, remap=remap)
        raise ValueError("remap must be [num_blocks]")
    if num_live is None:
        num_live = _new(1, torch.int32, dev, stream)
    elif not _fits(dev.index, torch.int32, num_live) or num_live.shape != (1,):
        _explain(dev, torch.int32, num_live=num_live)
        raise ValueError("num_live must be [1]")
    if workspace is None:
        workspace = _scratch("blocks", _size("pa_blocks_workspace_size", dev.index, rows, NB), dev, stream)
    else:
        _cuda(workspace, "workspace", workspace.dtype, dev)
    _call("pa_compact_blocks", dev, stream, *pools._args, block_tables.data_ptr(), width,
          context_lens.data_ptr(), rows, ref_counts.data_ptr(), remap.data_ptr(),
          num_live.data_ptr(), *pools._shape, workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return remap, num_live


def decode_tree_workspace_size(num_q_heads: int, num_kv_heads: int, head_dim: int = 128, device=None) -> int:
    """Workspace bytes pa_decode_tree needs on ``device`` (default: current)."""
    index = None if device is None else torch.device(device).index
    if index is None:       # no device, or "cuda": the current one
        index = torch.cuda.current_device()
    n = _size("pa_decode_tree_workspace_size", index, num_q_heads, num_kv_heads, head_dim)
    if n == 0:
        raise ValueError("unsupported head configuration")
    return n


def decode_tree(q, k_cache, v_cache, block_tables, context_lens, query_start_loc, tree_mask, scale, out=None,
                workspace=None, stream=None, head_major=False):
    """Decode of a tree of drafted tokens per sequence; returns ``out``. q is bf16
    [total_q, Hq, D], the nodes packed per sequence by query_start_loc (int32 [S + 1]);
    a sequence's n nodes are the last n of its context_lens[s] cached tokens. A row sees
    every token before them, and node j where bit j % 64 of tree_mask[row, j // 64]
    (int64 [total_q, words], at most 16 words) is set: its ancestors and itself. The other
    arguments are decode's. Rows of ``out`` outside all sequences are left as they were."""
    dev = q.device
    if not _fits(dev.index, torch.bfloat16, q, k_cache, v_cache):
        _explain(dev, torch.bfloat16, q=q, k_cache=k_cache, v_cache=v_cache)
    if not _fits(dev.index, torch.int32, block_tables, context_lens, query_start_loc):
        _explain(dev, torch.int32, block_tables=block_tables, context_lens=context_lens, query_start_loc=query_start_loc)
    if not _fits(dev.index, torch.int64, tree_mask):
        _explain(dev, torch.int64, tree_mask=tree_mask)
    T, Hq, D = q.shape
    if head_major:
        NB, Hkv, bs, D2 = k_cache.shape
    else:
        NB, bs, Hkv, D2 = k_cache.shape
    S = context_lens.shape[0]
    if v_cache.shape != k_cache.shape or D2 != D or block_tables.dim() != 2 or block_tables.shape[0] != S \
            or context_lens.dim() != 1 or query_start_loc.shape != (S + 1,):
        raise ValueError("shape mismatch between q, caches, block_tables, context_lens and query_start_loc")
    if tree_mask.dim() != 2 or tree_mask.shape[0] != T:
        raise ValueError("tree_mask must be [total_q, words]")
    if out is None:
        out = _new(q.shape, q.dtype, dev, stream)
    else:
        _cuda(out, "out", torch.bfloat16, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if workspace is None:
        workspace = _scratch("tree", decode_tree_workspace_size(Hq, Hkv, D, dev), dev, stream)
    else:
        _cuda(workspace, "workspace", workspace.dtype, dev)
    _call("pa_decode_tree", dev, stream, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
          block_tables.shape[1], context_lens.data_ptr(), query_start_loc.data_ptr(), tree_mask.data_ptr(),
          tree_mask.shape[1], float(scale), out.data_ptr(), S, T, Hq, Hkv, D, bs, NB, 1 if head_major else 0,
          workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out


def keep_tokens(pools: CachePools, block_tables, context_lens, query_start_loc, kept, ref_counts=None, stream=None):
    """Keep the accepted nodes of every sequence's draft (the last n of its tokens, n from
    query_start_loc, int32 [S + 1]): kept is int32 [S, m], a row's nodes in ascending order
    up to the first -1. Their rows move to consecutive places behind the context in every
    pool and context_lens becomes the shorter length, in place; with ref_counts
    (fork_blocks) the blocks no longer needed are given back."""
    dev = pools.device
    if not _fits(dev.index, torch.int32, block_tables, context_lens, query_start_loc, kept):
        _explain(dev, torch.int32, block_tables=block_tables, context_lens=context_lens,
                 query_start_loc=query_start_loc, kept=kept)
    S = context_lens.shape[0]
    if block_tables.dim() != 2 or block_tables.shape[0] != S or context_lens.dim() != 1 \
            or query_start_loc.shape != (S + 1,) or kept.dim() != 2 or kept.shape[0] != S:
        raise ValueError("shape mismatch between block_tables, context_lens, query_start_loc and kept")
    refs = None
    if ref_counts is not None:
        if not _fits(dev.index, torch.int32, ref_counts):
            _explain(dev, torch.int32, ref_counts=ref_counts)
        if ref_counts.shape != (pools.num_blocks,):
            raise ValueError("ref_counts must have one entry per block")
        refs = ref_counts.data_ptr()
    _call("pa_keep_tokens", dev, stream, *pools._args, block_tables.data_ptr(), block_tables.shape[1],
          context_lens.data_ptr(), query_start_loc.data_ptr(), kept.data_ptr(), kept.shape[1], S, refs, *pools._shape,
          1 if pools.head_major else 0)


class _RotaryStruct(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("amplitude", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("turns", ctypes.c_uint64 * 64)]


class Rotary:
    """The rotation of a head's first ``rot_dim`` of 128 dims by its position:
    neighbouring pairs (``interleaved``) or pairs half of ``rot_dim`` apart, at
    base^(-2 i / rot_dim) radians a token. Made once for a model.

    ``scaling`` for contexts longer than the model was trained on
    (``original_context`` tokens): "linear", "ntk", "yarn" or "banded", by
    ``factor``; ``low`` and ``high`` are the turns in original_context between
    which yarn (1, 32) and banded (1, 4) mix. ``amplitude`` multiplies the result;
    None is the scaling's own. ``frequencies`` (rot_dim / 2 numbers, radians a
    token) replace all of these."""

    SCALINGS = (None, "linear", "ntk", "yarn", "banded")

    def __init__(self, rot_dim: int = 128, base: float = 10000.0, interleaved: bool = False, scaling=None,
                 factor: float = 1.0, original_context: float = 0.0, low=None, high=None, amplitude=None,
                 frequencies=None):
        self._struct = _RotaryStruct()
        self._addr = ctypes.addressof(self._struct)
        if frequencies is not None:
            f = [float(x) for x in frequencies]
            if len(f) != int(rot_dim) // 2:
                raise ValueError("frequencies must be rot_dim / 2 numbers")
            data = (ctypes.c_double * max(1, len(f)))(*f)
            _check("pa_rotary_init_frequencies", lib().pa_rotary_init_frequencies(
                self._addr, int(rot_dim), int(bool(interleaved)), ctypes.addressof(data),
                1.0 if amplitude is None else float(amplitude)))
            return
        if scaling not in self.SCALINGS:
            raise ValueError(f"scaling must be one of {self.SCALINGS}")
        if amplitude is not None and float(amplitude) == 0.0:
            raise ValueError("amplitude must not be 0")
        low = 1.0 if low is None else float(low)
        high = (32.0 if scaling == "yarn" else 4.0) if high is None else float(high)
        _check("pa_rotary_init", lib().pa_rotary_init(
            self._addr, int(rot_dim), int(bool(interleaved)), float(base), self.SCALINGS.index(scaling),
            float(factor), float(original_context), low, high, 0.0 if amplitude is None else float(amplitude)))

    # a copy has a struct of its own, and its address
    def __getstate__(self):
        return bytes(self._struct)

    def __setstate__(self, state):
        self._struct = _RotaryStruct.from_buffer_copy(state)
        self._addr = ctypes.addressof(self._struct)

    rot_dim = property(lambda self: self._struct.rot_dim)
    interleaved = property(lambda self: bool(self._struct.interleaved))
    amplitude = property(lambda self: self._struct.amplitude)


def _heads(t, name, index, tokens):
    """(address, token stride, head stride, heads) of rows [tokens, heads, 128]."""
    try:
        shape, (ts, hs, ds) = t.shape, t.stride()
        if t.dtype is torch.bfloat16 and t.get_device() == index and shape[0] == tokens and shape[2] == 128 \
                and ds == 1:
            return t.data_ptr(), ts, hs, shape[1]
    except (AttributeError, TypeError, ValueError):
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.get_device() != index:
        raise ValueError(f"{name} must be a tensor on CUDA device {index}")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    raise ValueError(f"{name} must be [{tokens}, heads, 128] with the dims of a head contiguous, got "
                     f"{list(t.shape)} with strides {list(t.stride())}")


_NO_HEADS = (None, 0, 0, 0)


def _weight(w, name, dev):
    if w is None:
        return None
    if not _fits(dev.index, torch.bfloat16, w) or w.shape != (128,):
        _explain(dev, torch.bfloat16, **{name: w})
        raise ValueError(f"{name} must be [128]")
    return w.data_ptr()


def _positions(positions, rotary, tokens, dev):
    """(address of the rotation, address of the positions)"""
    if rotary is None:
        return None, None
    if not _fits(dev.index, torch.int32, positions) or positions.shape != (tokens,):
        _explain(dev, torch.int32, positions=positions)
        raise ValueError("positions must be [tokens]")
    return rotary._addr, positions.data_ptr()


def _out_heads(x, out, name, rows, dev, tokens, stream):
    """An output for the rows x ([T, H, 128], ``rows`` of _heads), and its own."""
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format) if stream is None \
            else _new(x.shape, x.dtype, dev, stream)
        return out, (out.data_ptr(), rows[3] * 128, 128)
    o = _heads(out, name, dev.index, tokens)
    if o[3] != rows[3]:
        raise ValueError(f"{name} must have its input's shape")
    return out, o[:3]


def rotate(q, k, positions, rotary, q_weight=None, k_weight=None, eps: float = 1e-6, q_out=None, k_out=None,
           stream=None):
    """The heads of queries and keys (bf16 [T, H, 128], any token and head stride
    that is a multiple of 8) rotated by their tokens' positions (int32 [T]) after
    the norm of each head's row where a weight (bf16 [128]) is given. Returns (q_out,
    k_out); an output may be its input. q or k may be None, and so may ``rotary`` (a
    Rotary; None: norms only, positions are not read)."""
    x = q if q is not None else k
    if not isinstance(x, torch.Tensor):
        raise ValueError("q or k must be a CUDA tensor")
    dev, T = x.device, x.shape[0]
    index = dev.index
    qr = _heads(q, "q", index, T) if q is not None else _NO_HEADS
    kr = _heads(k, "k", index, T) if k is not None else _NO_HEADS
    rot, pos = _positions(positions, rotary, T, dev)
    qo = ko = _NO_HEADS[:3]
    if q is not None:
        q_out, qo = _out_heads(q, q_out, "q_out", qr, dev, T, stream)
    if k is not None:
        k_out, ko = _out_heads(k, k_out, "k_out", kr, dev, T, stream)
    _call("pa_rotate", dev, stream, qr[0], qr[1], qr[2], *qo, qr[3], kr[0], kr[1], kr[2], *ko, kr[3], 128, pos, T, rot,
          _weight(q_weight, "q_weight", dev), _weight(k_weight, "k_weight", dev), float(eps))
    return q_out, k_out


def append_kvcache(q, k, v, k_cache, v_cache, slot_mapping, positions, rotary, q_weight=None, k_weight=None,
                   eps: float = 1e-6, q_out=None, stream=None, head_major=False):
    """A step's keys, rotated and normed as by rotate, and its values as they are,
    into the slots of the pools (int64 [T], -1 rows skipped) as by store_kvcache; and
    the queries, rotated and normed, into ``q_out``, which is returned. q, k, v may
    be strided parts of one projection; q may be None."""
    dev, T = k_cache.device, slot_mapping.shape[0]
    index = dev.index
    if not _fits(index, torch.bfloat16, k_cache, v_cache):
        _explain(dev, torch.bfloat16, k_cache=k_cache, v_cache=v_cache)
    if not _fits(index, torch.int64, slot_mapping):
        _explain(dev, torch.int64, slot_mapping=slot_mapping)
    qr = _heads(q, "q", index, T) if q is not None else _NO_HEADS
    kr, vr = _heads(k, "k", index, T), _heads(v, "v", index, T)
    if head_major:
        NB, Hkv, bs, D = k_cache.shape
    else:
        NB, bs, Hkv, D = k_cache.shape
    if v_cache.shape != k_cache.shape or kr[3] != Hkv or vr[3] != Hkv or D != 128 or slot_mapping.dim() != 1:
        raise ValueError("shape mismatch between k, v, caches and slot_mapping")
    rot, pos = _positions(positions, rotary, T, dev)
    qo = _NO_HEADS[:3]
    if q is not None:
        q_out, qo = _out_heads(q, q_out, "q_out", qr, dev, T, stream)
    _call("pa_append_kvcache", dev, stream, qr[0], qr[1], qr[2], *qo, qr[3], kr[0], kr[1], kr[2], vr[0], vr[1], vr[2],
          Hkv, 128, k_cache.data_ptr(), v_cache.data_ptr(), slot_mapping.data_ptr(), bs, NB, 1 if head_major else 0,
          pos, T, rot, _weight(q_weight, "q_weight", dev), _weight(k_weight, "k_weight", dev), float(eps))
    return q_out


def take_device_error(stream=None, device=None) -> int:
    """Synchronize the stream and return (and clear) the smallest device-side
    error code recorded so far: 0 none, 1 shared memory misaligned, 2 a wait
    ran out, 3 a bad slot, 4 a bad block id, 5 a bad row or block in a block
    operation (or a path that is none in keep_tokens), 6 a fork refused."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    code = ctypes.c_int32(0)
    with torch.cuda.device(dev):
        st = lib().pa_take_device_error(ctypes.addressof(code), _stream_ptr(stream, dev))
    _check("pa_take_device_error", st)
    return int(code.value)


def debug_prefill_fault(mode: int) -> None:
    """Test hook (off by default): mode 1 makes later prefill launches, the
    prefix kernel of later decode_shared calls and the kernel of later
    decode_tree calls hold back one barrier arrival so that a bounded wait runs out and code 2 is recorded; mode 0 turns it off."""
    _check("pa_debug_prefill_fault", lib().pa_debug_prefill_fault(int(mode)))


VARIANT_DECODE_SIMT, VARIANT_PREFILL_MMA = 1, 2


def debug_kernel_variant(flags: int) -> None:
    """Test hook (off by default): run the comparison kernels kept for tests
    (VARIANT_DECODE_SIMT: CUDA-core decode tiles; VARIANT_PREFILL_MMA: the
    mma.sync prefill kernel) instead of the product kernels; 0 restores them."""
    _check("pa_debug_kernel_variant", lib().pa_debug_kernel_variant(int(flags)))


class DecodeStepGraph:
    """One decode step (store of the new K/V rows, then decode, through
    pa_decode_step) captured into a CUDA graph and replayed with one launch
    per step.

    The tensors passed in are the graph's fixed buffers: update their contents
    in place (q, k_new, v_new, slot_mapping, block_tables, context_lens) and
    call replay(); the result lands in ``out``. With ``host_stage`` (a pinned
    uint8 tensor) and ``device_stage`` (a device uint8 tensor of the same size
    whose slices back the input tensors), the host-to-device copy of the step's
    inputs is captured too, and with ``host_out`` (pinned) the read-back of
    ``out``: one replay is then the whole step from host buffers to host
    buffers. The decode is the automatic-partition pa_decode; its workspace is
    allocated once here, before capture.
    """

    def __init__(self, q, k_cache, v_cache, block_tables, context_lens, scale, k_new=None,
                 v_new=None, slot_mapping=None, out=None, host_stage=None, device_stage=None,
                 host_out=None, head_major=False):
        dev = q.device
        S, Hq, D = q.shape
        Hkv = k_cache.shape[1] if head_major else k_cache.shape[2]
        self.out = out if out is not None else torch.empty_like(q)
        self.workspace = workspace_for(Hq, Hkv, D, 0, dev)
        has_store = slot_mapping is not None and slot_mapping.shape[0] > 0

        def body():
            if host_stage is not None:
                device_stage.copy_(host_stage, non_blocking=True)
            if has_store:
                decode_step(k_new, v_new, slot_mapping, q, k_cache, v_cache, block_tables,
                            context_lens, scale, out=self.out, workspace=self.workspace,
                            head_major=head_major)
            else:
                decode(q, k_cache, v_cache, block_tables, context_lens, scale, out=self.out,
                       workspace=self.workspace, head_major=head_major)
            if host_out is not None:
                host_out.copy_(self.out, non_blocking=True)

        # one eager run first: library set-up calls happen outside the capture
        side = torch.cuda.Stream(dev)
        side.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(side):
            body()
        torch.cuda.current_stream(dev).wait_stream(side)
        torch.cuda.synchronize(dev)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            body()

    def replay(self):
        self.graph.replay()
        return self.out
