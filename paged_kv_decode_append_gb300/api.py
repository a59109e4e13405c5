"""Python binding of the C ABI (``include/pkv.h``): same names, torch tensors
in, argument marshalling only.  Every step of the computation runs in the
library's CUDA kernels; there is no Python or CPU fallback, and a missing or
unloadable library raises.
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import _lib
from ._lib import CacheDesc

NHD = 0
HND = 1

OK, EINVAL, EUNSUPPORTED, ECUDA, ENOPAGES, EWORKSPACE, ETOOBIG = range(7)
DECODE_OVERLAP_PROLOGUE = 1  # pkv_decode_attn_ex flags (see include/pkv.h)
DECODE_EARLY_KV = 2
DECODE_MAKE_PLAN = 4
DECODE_USE_PLAN = 8
ERR_PAGE, ERR_OVERFLOW, ERR_TIMEOUT, ERR_QLEN, ERR_PLAN, ERR_POOL, ERR_TREE = 1, 2, 4, 8, 16, 32, 64


class PkvError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = _lib.load().pkv_status_str(status).decode()
        super().__init__(f"{what}: {msg} (status {status})")


def _check(status: int, what: str) -> None:
    if status != OK:
        raise PkvError(status, what)


def cache_desc(k_cache: torch.Tensor, layout: int = NHD) -> CacheDesc:
    """Descriptor of a pool tensor: NHD ``[pages, P, Hkv, D]`` or HND
    ``[pages, Hkv, P, D]``."""
    if k_cache.dim() != 4:
        raise ValueError("cache must be 4-D")
    if layout == NHD:
        n, p, h, d = k_cache.shape
    else:
        n, h, p, d = k_cache.shape
    return CacheDesc(n, p, h, d, layout)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _bf16(t, name):
    if t is None:
        return
    if t.dtype != torch.bfloat16 or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name}: expected a contiguous CUDA bfloat16 tensor")


def _i32(t, name):
    if t is None:
        return
    if t.dtype != torch.int32 or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name}: expected a contiguous CUDA int32 tensor")


def pkv_decode_workspace_size(batch: int, max_blocks: int, num_q_heads: int, desc: CacheDesc) -> int:
    return int(_lib.load().pkv_decode_workspace_size(batch, max_blocks, num_q_heads, ctypes.byref(desc)))


def decode_workspace(batch: int, max_blocks: int, num_q_heads: int, desc: CacheDesc, device) -> torch.Tensor:
    """A zero-filled workspace for pkv_decode_attn (reusable across calls)."""
    n = pkv_decode_workspace_size(batch, max_blocks, num_q_heads, desc)
    if n == 0:
        raise PkvError(EUNSUPPORTED, "pkv_decode_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def pkv_append(k_cache, v_cache, k_new, v_new, block_table, cache_seqlens, append_indptr=None, err_flag=None,
               layout: int = NHD) -> None:
    """Bit-copy ``k_new``/``v_new`` ``[T, Hkv, D]`` into their page slots."""
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache"), (k_new, "k_new"), (v_new, "v_new")):
        _bf16(t, n)
    for t, n in ((block_table, "block_table"), (cache_seqlens, "cache_seqlens"), (append_indptr, "append_indptr"),
                 (err_flag, "err_flag")):
        _i32(t, n)
    desc = cache_desc(k_cache, layout)
    st = _lib.load().pkv_append(ctypes.byref(desc), _ptr(k_cache), _ptr(v_cache), _ptr(k_new), _ptr(v_new),
                                k_new.shape[0], _ptr(append_indptr), _ptr(block_table), block_table.shape[1],
                                _ptr(cache_seqlens), cache_seqlens.shape[0], _ptr(err_flag),
                                _stream(k_cache.device))
    _check(st, "pkv_append")


def pkv_decode_attn(k_cache, v_cache, q, k_new, v_new, block_table, cache_seqlens, softmax_scale: float,
                    out=None, lse=None, workspace=None, err_flag=None, layout: int = NHD,
                    flags: int = 0) -> torch.Tensor:
    """Fused append + decode attention; returns ``out`` ``[B, Hq, D]`` bf16.
    ``flags`` (e.g. DECODE_OVERLAP_PROLOGUE) selects ``pkv_decode_attn_ex``."""
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache"), (q, "q"), (k_new, "k_new"), (v_new, "v_new"),
                 (out, "out")):
        _bf16(t, n)
    for t, n in ((block_table, "block_table"), (cache_seqlens, "cache_seqlens"), (err_flag, "err_flag")):
        _i32(t, n)
    if lse is not None and (lse.dtype != torch.float32 or not lse.is_contiguous()):
        raise ValueError("lse: expected contiguous float32")
    desc = cache_desc(k_cache, layout)
    B, Hq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = decode_workspace(B, block_table.shape[1], Hq, desc, q.device)
    args = (ctypes.byref(desc), _ptr(k_cache), _ptr(v_cache), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(block_table),
            block_table.shape[1], _ptr(cache_seqlens), B, Hq, float(softmax_scale), _ptr(out), _ptr(lse),
            _ptr(workspace), workspace.numel(), _ptr(err_flag), _stream(q.device))
    if flags:
        _check(_lib.load().pkv_decode_attn_ex(*args, int(flags)), "pkv_decode_attn_ex")
    else:
        _check(_lib.load().pkv_decode_attn(*args), "pkv_decode_attn")
    return out


def pkv_decode_attn_noalloc(k_cache, v_cache, q, k_new, v_new, block_table, cache_seqlens, softmax_scale: float,
                            out=None, lse=None, err_flag=None, layout: int = NHD) -> torch.Tensor:
    """pkv_decode_attn for callers that cannot allocate device memory: no
    workspace argument, the library's built-in scratch is used instead (see
    include/pkv.h for its size limit and sharing rules).  Pass ``out`` to
    avoid the allocation of a fresh output tensor here."""
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache"), (q, "q"), (k_new, "k_new"), (v_new, "v_new"),
                 (out, "out")):
        _bf16(t, n)
    for t, n in ((block_table, "block_table"), (cache_seqlens, "cache_seqlens"), (err_flag, "err_flag")):
        _i32(t, n)
    if lse is not None and (lse.dtype != torch.float32 or not lse.is_contiguous()):
        raise ValueError("lse: expected contiguous float32")
    desc = cache_desc(k_cache, layout)
    B, Hq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    st = _lib.load().pkv_decode_attn_noalloc(
        ctypes.byref(desc), _ptr(k_cache), _ptr(v_cache), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(block_table),
        block_table.shape[1], _ptr(cache_seqlens), B, Hq, float(softmax_scale), _ptr(out), _ptr(lse), _ptr(err_flag),
        _stream(q.device))
    _check(st, "pkv_decode_attn_noalloc")
    return out


def pkv_decode_bucket(batch: int) -> int:
    """Graph batch size serving ``batch`` rows (0 if out of range)."""
    return int(_lib.load().pkv_decode_bucket(batch))


class DecodeStep:
    """``pkv_decode_step_*``: every layer's fused append + decode of one step
    captured once as a CUDA graph.  The tensors given here are baked in:
    write each step's inputs (``q``, ``k_new``, ``v_new``, ``cache_seqlens``)
    into them, then call :meth:`launch`."""

    def __init__(self, k_caches, v_caches, q, k_new, v_new, block_table, cache_seqlens, softmax_scale: float, out,
                 lse=None, workspace=None, err_flag=None, layout: int = NHD, flags: int = 0):
        layers = len(k_caches)
        if not (len(v_caches) == len(q) == len(out) == layers) or layers < 1:
            raise ValueError("one k / v cache, q and out per layer")
        for lst, n in ((k_caches, "k_caches"), (v_caches, "v_caches"), (q, "q"), (out, "out"),
                       (k_new or [], "k_new"), (v_new or [], "v_new")):
            for t in lst:
                _bf16(t, n)
        for t, n in ((block_table, "block_table"), (cache_seqlens, "cache_seqlens"), (err_flag, "err_flag")):
            _i32(t, n)
        desc = cache_desc(k_caches[0], layout)
        B, Hq, D = q[0].shape
        if workspace is None:
            workspace = decode_workspace(B, block_table.shape[1], Hq, desc, q[0].device)
        arr = ctypes.c_void_p * layers

        def ptrs(lst):
            return None if lst is None else arr(*[t.data_ptr() if t is not None else None for t in lst])

        self._keep = (k_caches, v_caches, q, k_new, v_new, block_table, cache_seqlens, out, lse, workspace, err_flag)
        self._lib = _lib.load()
        handle = ctypes.c_void_p()
        st = self._lib.pkv_decode_step_create(
            ctypes.byref(desc), layers, ptrs(k_caches), ptrs(v_caches), ptrs(q), ptrs(k_new), ptrs(v_new),
            _ptr(block_table), block_table.shape[1], _ptr(cache_seqlens), B, Hq, float(softmax_scale), ptrs(out),
            ptrs(lse), _ptr(workspace), workspace.numel(), _ptr(err_flag), int(flags), ctypes.byref(handle))
        _check(st, "pkv_decode_step_create")
        self._h = handle
        self.device = q[0].device

    def launch(self) -> None:
        _check(self._lib.pkv_decode_step_launch(self._h, _stream(self.device)), "pkv_decode_step_launch")

    def __del__(self):
        if getattr(self, "_h", None):
            self._lib.pkv_decode_step_destroy(self._h)
            self._h = None


def pkv_prefill_workspace_size(batch: int, total_q: int, num_q_heads: int, desc: CacheDesc) -> int:
    return int(_lib.load().pkv_prefill_workspace_size(batch, total_q, num_q_heads, ctypes.byref(desc)))


def prefill_workspace(batch: int, total_q: int, num_q_heads: int, desc: CacheDesc, device) -> torch.Tensor:
    """A workspace for pkv_prefill_attn (needs no initialisation)."""
    n = pkv_prefill_workspace_size(batch, total_q, num_q_heads, desc)
    if n == 0:
        raise PkvError(EUNSUPPORTED, "pkv_prefill_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def pkv_prefill_attn(k_cache, v_cache, q, qo_indptr, kv_lens, block_table, softmax_scale: float, out=None,
                     lse=None, workspace=None, err_flag=None, layout: int = NHD) -> torch.Tensor:
    """Ragged end-aligned causal prefill over the paged cache; ``q`` is
    ``[total_q, Hq, D]``, request b owns rows ``qo_indptr[b]:qo_indptr[b+1]``
    and sees ``kv_lens[b]`` keys.  Returns ``out`` ``[total_q, Hq, D]`` bf16."""
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache"), (q, "q"), (out, "out")):
        _bf16(t, n)
    for t, n in ((qo_indptr, "qo_indptr"), (kv_lens, "kv_lens"), (block_table, "block_table"),
                 (err_flag, "err_flag")):
        _i32(t, n)
    if lse is not None and (lse.dtype != torch.float32 or not lse.is_contiguous()):
        raise ValueError("lse: expected contiguous float32")
    desc = cache_desc(k_cache, layout)
    total_q, Hq, D = q.shape
    B = kv_lens.shape[0]
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = prefill_workspace(B, total_q, Hq, desc, q.device)
    st = _lib.load().pkv_prefill_attn(
        ctypes.byref(desc), _ptr(k_cache), _ptr(v_cache), _ptr(q), _ptr(qo_indptr), _ptr(kv_lens),
        _ptr(block_table), block_table.shape[1], B, Hq, total_q, float(softmax_scale), _ptr(out), _ptr(lse),
        _ptr(workspace), workspace.numel(), _ptr(err_flag), _stream(q.device))
    _check(st, "pkv_prefill_attn")
    return out


def pkv_mixed_workspace_size(batch: int, total_q: int, max_blocks: int, num_q_heads: int, max_qlen: int,
                             decode_max_qlen: int, desc: CacheDesc) -> int:
    return int(_lib.load().pkv_mixed_workspace_size(batch, total_q, max_blocks, num_q_heads, max_qlen,
                                                    decode_max_qlen, ctypes.byref(desc)))


def default_decode_max_qlen(num_q_heads: int, num_kv_heads: int) -> int:
    """Longest row the decode kernel takes by default in a mixed step: up to
    16 (query, head) columns of a kv head (two decode units)."""
    return max(1, 16 // max(1, num_q_heads // num_kv_heads))


def mixed_workspace(batch: int, total_q: int, max_blocks: int, num_q_heads: int, max_qlen: int,
                    decode_max_qlen: int, desc: CacheDesc, device) -> torch.Tensor:
    """A zero-filled workspace for pkv_mixed_attn (reusable across calls)."""
    n = pkv_mixed_workspace_size(batch, total_q, max_blocks, num_q_heads, max_qlen, decode_max_qlen, desc)
    if n == 0:
        raise PkvError(EUNSUPPORTED, "pkv_mixed_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def pkv_mixed_attn(k_cache, v_cache, q, k_new, v_new, qo_indptr, block_table, cache_seqlens, softmax_scale: float,
                   max_qlen: int, decode_max_qlen: int | None = None, out=None, lse=None, workspace=None,
                   err_flag=None, layout: int = NHD) -> torch.Tensor:
    """One step of a mixed batch: row b appends its ``qo_indptr[b+1] -
    qo_indptr[b]`` new tokens (``k_new``/``v_new`` ``[total_q, Hkv, D]``, or
    both None when already appended) after its ``cache_seqlens[b]`` cached
    ones, then its query i attends keys ``0 .. kv_b - q_b + i``.  Rows of up
    to ``decode_max_qlen`` queries run on the decode kernel, longer ones on
    the prefill kernel.  Returns ``out`` ``[total_q, Hq, D]`` bf16."""
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache"), (q, "q"), (k_new, "k_new"), (v_new, "v_new"),
                 (out, "out")):
        _bf16(t, n)
    for t, n in ((qo_indptr, "qo_indptr"), (block_table, "block_table"), (cache_seqlens, "cache_seqlens"),
                 (err_flag, "err_flag")):
        _i32(t, n)
    if lse is not None and (lse.dtype != torch.float32 or not lse.is_contiguous()):
        raise ValueError("lse: expected contiguous float32")
    desc = cache_desc(k_cache, layout)
    total_q, Hq, D = q.shape
    B = cache_seqlens.shape[0]
    if decode_max_qlen is None:
        decode_max_qlen = default_decode_max_qlen(Hq, desc.num_kv_heads)
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = mixed_workspace(B, total_q, block_table.shape[1], Hq, max_qlen, decode_max_qlen, desc,
                                    q.device)
    st = _lib.load().pkv_mixed_attn(
        ctypes.byref(desc), _ptr(k_cache), _ptr(v_cache), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(qo_indptr),
        _ptr(block_table), block_table.shape[1], _ptr(cache_seqlens), B, Hq, total_q, int(max_qlen),
        int(decode_max_qlen), float(softmax_scale), _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(),
        _ptr(err_flag), _stream(q.device))
    _check(st, "pkv_mixed_attn")
    return out


POOL_HEADER = 16  # int32 words before the ring of a device pool

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(dev: int) -> int:
    """The current stream of device ``dev`` as an integer."""
    return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream


def _at(dev: int, name: str, t, dtype, *shape):
    """Address of ``t`` (None for None) once it is a contiguous tensor of
    ``dtype`` and ``shape`` (if given) on CUDA device ``dev``."""
    if t is None:
        return None
    if t.dtype is not dtype or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor on cuda:{dev}")
    if shape and t.shape != shape:
        raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")
    return t.data_ptr()


def _device_of(t, name: str) -> int:
    """The device a call runs on: its first tensor's, which has to be the
    current one (the library launches on the current device)."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if dev != torch.cuda.current_device():
        raise ValueError(f"{name} is on cuda:{dev}, which is not the current device")
    return dev


_I32, _I64, _BF16, _F32, _U8 = torch.int32, torch.int64, torch.bfloat16, torch.float32, torch.uint8


def device_pool(num_pages: int, device="cuda") -> torch.Tensor:
    """A pool of pages ``1 .. num_pages - 1`` in device memory
    (``pkv_device_pool_init``), as an int32 tensor; every page is free."""
    n = int(_lib.load().pkv_device_pool_bytes(num_pages))
    if n == 0:
        raise PkvError(EINVAL, "pkv_device_pool_bytes")
    pool = torch.empty(n // 4, dtype=torch.int32, device=device)
    dev = _device_of(pool, "pool")
    _check(_lib.load().pkv_device_pool_init(pool.data_ptr(), n, num_pages, _stream_of(dev)), "pkv_device_pool_init")
    return pool


def pkv_table_update(pool, block_table, held_blocks, cache_seqlens, new_tokens, page_size: int, indptr=None,
                     slot_map=None, positions=None, err_flag=None) -> None:
    """Makes every row's ``block_table`` entry list cover ``cache_seqlens[b] +
    new_tokens[b]`` tokens (none for an inactive row) from the device ``pool``,
    and writes the new tokens' ``indptr`` ``[B + 1]``, ``slot_map`` (int64) and
    ``positions`` ``[max_tokens]`` where given."""
    dev = _device_of(pool, "pool")
    B, width = block_table.shape
    tokens = 0
    if slot_map is not None:
        tokens = slot_map.numel()
    elif positions is not None:
        tokens = positions.numel()
    st = _lib.load().pkv_table_update(
        _at(dev, "pool", pool, _I32), pool.numel() - POOL_HEADER + 1, page_size,
        _at(dev, "block_table", block_table, _I32), width, _at(dev, "held_blocks", held_blocks, _I32, B),
        _at(dev, "cache_seqlens", cache_seqlens, _I32, B), _at(dev, "new_tokens", new_tokens, _I32, B), B,
        _at(dev, "indptr", indptr, _I32, B + 1), _at(dev, "slot_map", slot_map, _I64, tokens),
        _at(dev, "positions", positions, _I32, tokens), tokens, _at(dev, "err_flag", err_flag, _I32), _stream_of(dev))
    if st:
        _check(st, "pkv_table_update")


def pkv_tree_build(parents, qo_indptr, cache_seqlens, max_nodes: int, mask=None, positions=None, err_flag=None):
    """Ancestor masks (int32 words, bit j of node i: j is i or an ancestor)
    and positions ``cache_seqlens[b] + depth`` of drafted trees; ``parents``
    ``[total_q]`` holds the parent's index within the row, or -1.  Returns
    ``(mask, positions)``."""
    dev = _device_of(parents, "parents")
    T, B = parents.numel(), cache_seqlens.numel()
    if mask is None:
        mask = torch.empty(T, (max_nodes + 31) // 32, dtype=torch.int32, device=parents.device)
    if positions is None:
        positions = torch.empty(T, dtype=torch.int32, device=parents.device)
    words = mask.size(-1)
    st = _lib.load().pkv_tree_build(
        _at(dev, "parents", parents, _I32, T), _at(dev, "qo_indptr", qo_indptr, _I32, B + 1),
        _at(dev, "cache_seqlens", cache_seqlens, _I32, B), B, T, max_nodes, _at(dev, "mask", mask, _I32, T, words), words,
        _at(dev, "positions", positions, _I32, T), _at(dev, "err_flag", err_flag, _I32), _stream_of(dev))
    if st:
        _check(st, "pkv_tree_build")
    return mask, positions


def pkv_tree_workspace_size(batch: int, total_q: int, max_blocks: int, num_q_heads: int, max_nodes: int,
                            desc: CacheDesc) -> int:
    return int(_lib.load().pkv_tree_workspace_size(batch, total_q, max_blocks, num_q_heads, max_nodes,
                                                   ctypes.byref(desc)))


def tree_workspace(batch: int, total_q: int, max_blocks: int, num_q_heads: int, max_nodes: int, desc: CacheDesc,
                   device) -> torch.Tensor:
    """A workspace for pkv_tree_attn (needs no initialisation)."""
    n = pkv_tree_workspace_size(batch, total_q, max_blocks, num_q_heads, max_nodes, desc)
    if n == 0:
        raise PkvError(EUNSUPPORTED, "pkv_tree_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def pkv_tree_attn(k_cache, v_cache, q, k_new, v_new, qo_indptr, tree_mask, block_table, cache_seqlens,
                  softmax_scale: float, max_nodes: int, out=None, lse=None, workspace=None, err_flag=None,
                  layout: int = NHD) -> torch.Tensor:
    """Append of every row's drafted tokens (``k_new``/``v_new`` ``[total_q,
    Hkv, D]``, or both None when cached already), then attention of every node
    over its row's ``cache_seqlens[b]`` cached keys and the drafted ones whose
    bit ``tree_mask`` ``[total_q, words]`` sets.  Returns ``out`` ``[total_q,
    Hq, D]`` bf16."""
    dev = _device_of(q, "q")
    desc = cache_desc(k_cache, layout)
    T, Hq, D = q.shape
    B, width = block_table.shape
    words = tree_mask.size(-1)
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = tree_workspace(B, T, width, Hq, max_nodes, desc, q.device)
    if D != desc.head_dim:
        raise ValueError("q: head_dim differs from the cache's")
    K = desc.num_kv_heads
    st = _lib.load().pkv_tree_attn(
        ctypes.byref(desc), _at(dev, "k_cache", k_cache, _BF16), _at(dev, "v_cache", v_cache, _BF16, *k_cache.shape),
        _at(dev, "q", q, _BF16), _at(dev, "k_new", k_new, _BF16, T, K, D), _at(dev, "v_new", v_new, _BF16, T, K, D),
        _at(dev, "qo_indptr", qo_indptr, _I32, B + 1), _at(dev, "tree_mask", tree_mask, _I32, T, words), words,
        _at(dev, "block_table", block_table, _I32), width, _at(dev, "cache_seqlens", cache_seqlens, _I32, B), B, Hq, T,
        max_nodes, softmax_scale, _at(dev, "out", out, _BF16, T, Hq, D), _at(dev, "lse", lse, _F32, T, Hq),
        _at(dev, "workspace", workspace, _U8), workspace.numel(), _at(dev, "err_flag", err_flag, _I32), _stream_of(dev))
    if st:
        _check(st, "pkv_tree_attn")
    return out


def pkv_tree_accept(parents, draft_tokens, target_tokens, root_targets, qo_indptr, cache_seqlens, max_nodes: int,
                    path=None, path_len=None, next_token=None, seqlens_out=None, err_flag=None):
    """The path of drafted tokens that the target model chose itself.  Returns
    ``(path [B, max_path], path_len [B], next_token [B], seqlens_out [B])``;
    ``root_targets`` None accepts each row's first root unseen."""
    dev = _device_of(parents, "parents")
    T, B = parents.numel(), cache_seqlens.numel()
    if path is None:
        path = torch.empty(B, max_nodes, dtype=torch.int32, device=parents.device)
    if path_len is None:
        path_len = torch.empty(B, dtype=torch.int32, device=parents.device)
    if next_token is None:
        next_token = torch.empty(B, dtype=torch.int32, device=parents.device)
    if seqlens_out is None:
        seqlens_out = torch.empty(B, dtype=torch.int32, device=parents.device)
    width = path.size(-1)
    st = _lib.load().pkv_tree_accept(
        _at(dev, "parents", parents, _I32, T), _at(dev, "draft_tokens", draft_tokens, _I32, T),
        _at(dev, "target_tokens", target_tokens, _I32, T), _at(dev, "root_targets", root_targets, _I32, B),
        _at(dev, "qo_indptr", qo_indptr, _I32, B + 1), _at(dev, "cache_seqlens", cache_seqlens, _I32, B), B, T, max_nodes,
        _at(dev, "path", path, _I32, B, width), width, _at(dev, "path_len", path_len, _I32, B),
        _at(dev, "next_token", next_token, _I32, B), _at(dev, "seqlens_out", seqlens_out, _I32, B),
        _at(dev, "err_flag", err_flag, _I32), _stream_of(dev))
    if st:
        _check(st, "pkv_tree_accept")
    return path, path_len, next_token, seqlens_out


class LayerCaches:
    """The K and V pools of a model's layers, which share one block table, as
    :func:`pkv_tree_commit` takes them (keeps the tensors alive)."""

    def __init__(self, k_caches, v_caches, layout: int = NHD):
        if len(k_caches) != len(v_caches) or len(k_caches) < 1:
            raise ValueError("one k and one v cache per layer")
        self.device = _device_of(k_caches[0], "k_caches")
        self._keep = (list(k_caches), list(v_caches))
        shape = k_caches[0].shape
        arr = ctypes.c_void_p * len(k_caches)
        self.k_ptrs, self.v_ptrs = (arr(*[_at(self.device, "caches", t, _BF16, *shape) for t in side])
                                    for side in self._keep)
        self.num_layers = len(k_caches)
        self.desc = cache_desc(k_caches[0], layout)


def pkv_tree_commit(layers: LayerCaches, path, path_len, block_table, cache_seqlens, err_flag=None) -> None:
    """Moves the K/V of each row's accepted nodes ``path[b, :path_len[b]]``
    from position ``cache_seqlens[b] + path[b, i]`` to ``cache_seqlens[b] +
    i`` in every layer (``cache_seqlens`` without the accepted tokens)."""
    dev = _device_of(path, "path")
    if dev != layers.device:
        raise ValueError("path and caches on different devices")
    B, width = block_table.shape
    steps = path.size(-1)
    st = _lib.load().pkv_tree_commit(
        ctypes.byref(layers.desc), layers.num_layers, layers.k_ptrs, layers.v_ptrs,
        _at(dev, "path", path, _I32, B, steps), steps, _at(dev, "path_len", path_len, _I32, B),
        _at(dev, "block_table", block_table, _I32), width, _at(dev, "cache_seqlens", cache_seqlens, _I32, B), B,
        _at(dev, "err_flag", err_flag, _I32), _stream_of(dev))
    if st:
        _check(st, "pkv_tree_commit")


def pkv_pool_bytes(desc: CacheDesc) -> int:
    return int(_lib.load().pkv_pool_bytes(ctypes.byref(desc)))


def pkv_validate_host(desc: CacheDesc, block_table: np.ndarray, seqlens: np.ndarray, extra_tokens: int):
    """Host check of a block table; returns (status, first bad row or -1)."""
    bt = np.ascontiguousarray(block_table, dtype=np.int32)
    sl = np.ascontiguousarray(seqlens, dtype=np.int32)
    bad = ctypes.c_int32(-1)
    st = _lib.load().pkv_validate_host(ctypes.byref(desc), bt.ctypes.data_as(_lib.I32P), bt.shape[1],
                                       sl.ctypes.data_as(_lib.I32P), sl.shape[0], extra_tokens, ctypes.byref(bad))
    return st, bad.value


class PagePool:
    """Host page pool (``pkv_pool_*``): pages 1..num_pages-1, page 0 never
    handed out; a fresh pool hands pages out in ascending order."""

    def __init__(self, num_pages: int):
        self._lib = _lib.load()
        self._p = self._lib.pkv_pool_create(num_pages)
        if not self._p:
            raise PkvError(EINVAL, "pkv_pool_create")

    def __del__(self):
        if getattr(self, "_p", None):
            self._lib.pkv_pool_destroy(self._p)
            self._p = None

    @property
    def num_free(self) -> int:
        return int(self._lib.pkv_pool_num_free(self._p))

    def alloc(self, n: int) -> np.ndarray:
        out = np.zeros(max(n, 0), np.int32)
        _check(self._lib.pkv_pool_alloc(self._p, n, out.ctypes.data_as(_lib.I32P)), "pkv_pool_alloc")
        return out

    def free(self, pages) -> None:
        pages = np.ascontiguousarray(pages, dtype=np.int32)
        _check(self._lib.pkv_pool_free(self._p, pages.ctypes.data_as(_lib.I32P), pages.size), "pkv_pool_free")

    def shuffle(self, seed: int) -> None:
        _check(self._lib.pkv_pool_shuffle(self._p, seed), "pkv_pool_shuffle")

    def reserve(self, row: np.ndarray, page_size: int, cur_len: int, new_len: int) -> None:
        """Extend one block-table row (an int32 numpy view) from cur_len to new_len tokens."""
        assert row.dtype == np.int32 and row.flags.c_contiguous
        _check(self._lib.pkv_table_reserve(self._p, row.ctypes.data_as(_lib.I32P), row.size, page_size, cur_len,
                                           new_len), "pkv_table_reserve")

    def release(self, row: np.ndarray, page_size: int, length: int) -> None:
        assert row.dtype == np.int32 and row.flags.c_contiguous
        _check(self._lib.pkv_table_release(self._p, row.ctypes.data_as(_lib.I32P), row.size, page_size, length),
               "pkv_table_release")
