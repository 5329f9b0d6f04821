"""The attention that reads the paged KV cache, the cache's writer and its page
calls: argument marshalling for the entry points of ``include/dsaidx.h`` that
take a ``DsaKv`` or ``DsaPages``.

Tensors are on the current CUDA device. Results and scratch are allocated with
torch when the caller does not pass them, with ``stream`` given as that
stream's memory. Every call is asynchronous.
"""
from __future__ import annotations

import ctypes

import torch

from .binding import (DsaAttnC, DsaCacheDescC, DsaError, DsaKvC, DsaPagesC, _check, _ptr, load)

BLOCK_SIZE = 64
_DTYPES = {torch.bfloat16: 0, torch.float16: 1}


def new_kv_cache(num_blocks: int, num_kv_heads: int, head_dim: int, dtype=torch.bfloat16, device=None):
    """A zeroed pair of K and V caches [num_blocks, 64, num_kv_heads, head_dim]."""
    if dtype not in _DTYPES or head_dim not in (64, 128) or num_blocks < 1 or num_kv_heads < 1:
        raise DsaError("a KV cache has bf16 or fp16 rows of 64 or 128, at least one page and one head")
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    shape = (int(num_blocks), BLOCK_SIZE, int(num_kv_heads), int(head_dim))
    return torch.zeros(shape, dtype=dtype, device=dev), torch.zeros(shape, dtype=dtype, device=dev)


# ---------------------------------------------------------------- arguments

def _here(t, what, dtype=None):
    """A CUDA tensor of the current device (and of dtype)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise DsaError(f"{what} must be a CUDA tensor")
    if t.device.index != torch.cuda.current_device():
        raise DsaError(f"{what} is on {t.device}, the current device is {torch.cuda.current_device()}")
    if dtype is not None and t.dtype != dtype:
        raise DsaError(f"{what} must be {dtype}, got {t.dtype}")
    return t


def _dense(t, what, dtype):
    if not _here(t, what, dtype).is_contiguous():
        raise DsaError(f"{what} must be contiguous")
    return t


def _err(dev_err):
    if dev_err is not None:
        _dense(dev_err, "dev_err", torch.int32)
    return _ptr(dev_err)


def _strides(t, axes, what):
    """Strides of the named axes; an axis of one element gets the row's length,
    since torch leaves such a stride arbitrary."""
    if t.stride(-1) != 1:
        raise DsaError(f"{what} must have a contiguous last axis")
    return [t.stride(a) if t.shape[a] > 1 else int(t.shape[-1]) for a in axes]


def _kv(k_cache, v_cache, packed=False):
    """The C description of a cache [num_blocks, 64, heads, head_dim], or of
    packed rows [rows, heads, head_dim]; any strides with a contiguous last axis."""
    dims = 3 if packed else 4
    for t, what in ((k_cache, "k"), (v_cache, "v")):
        _here(t, what)
        if t.dtype not in _DTYPES:
            raise DsaError(f"{what} must be bf16 or fp16, got {t.dtype}")
        if t.dim() != dims or (not packed and t.shape[1] != BLOCK_SIZE):
            raise DsaError(f"{what} must be " + ("[rows, heads, head_dim]" if packed else
                                                 "[num_blocks, 64, heads, head_dim]"))
    if k_cache.shape != v_cache.shape or k_cache.dtype != v_cache.dtype:
        raise DsaError("k and v must have one shape and one type")
    n, heads, d = int(k_cache.shape[0]), int(k_cache.shape[-2]), int(k_cache.shape[-1])
    if packed:
        ks, vs = ([d] + _strides(t, (0, 1), w) for t, w in ((k_cache, "k"), (v_cache, "v")))
    else:
        ks, vs = (_strides(t, (0, 1, 2), w) for t, w in ((k_cache, "k"), (v_cache, "v")))
    return DsaKvC(k_cache.data_ptr(), v_cache.data_ptr(), _DTYPES[k_cache.dtype], heads, d, n, *ks, *vs)


def _made(stream, shape, dtype, device, covered):
    """A result made here, for the stream it is written on; zeros where the call
    does not write every row."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _made(None, shape, dtype, device, covered)
    return (torch.empty if covered else torch.zeros)(shape, dtype=dtype, device=device)


def _attn(q, out, lse, kv, dtype, scale, first, rows, stream):
    """The C description of q, out and lse for a call that writes rows [first,
    rows), allocating what is missing."""
    _here(q, "q", dtype)
    if q.dim() != 3 or q.shape[2] != kv.head_dim:
        raise DsaError(f"q must be [tokens, heads, {kv.head_dim}]")
    if q.shape[0] < rows:
        raise DsaError(f"q has {q.shape[0]} rows, the call needs {rows}")
    heads = int(q.shape[1])
    if heads == 0 or heads % kv.num_kv_heads:
        raise DsaError(f"{heads} query heads cannot share {kv.num_kv_heads} KV heads")
    if out is None:
        out = _made(stream, q.shape, dtype, q.device, first == 0 and rows == q.shape[0])
    elif _here(out, "out", dtype).shape != q.shape:
        raise DsaError("out must have q's shape")
    if lse is None:
        lse = _made(stream, q.shape[:2], torch.float32, q.device, first == 0 and rows == q.shape[0])
    elif _dense(lse, "lse", torch.float32).shape != q.shape[:2]:
        raise DsaError("lse must be [tokens, heads]")
    qs, os = _strides(q, (0, 1), "q"), _strides(out, (0, 1), "out")
    return DsaAttnC(q.data_ptr(), *qs, out.data_ptr(), *os, lse.data_ptr(), heads, float(scale)), out, lse


def _on(stream):
    return stream if stream is not None else torch.cuda.current_stream()


def _scratch(ws, nbytes, device, stream):
    """The caller's scratch, checked, or a new one that belongs to the stream it is used on."""
    if ws is not None:
        return _dense(ws, "ws", torch.uint8)
    if stream is None:
        return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------- entry points

def kv_write(k, v, slot_mapping, k_cache, v_cache, dev_err=None, stream=None):
    """Write the rows k and v [tokens, heads, head_dim] at their slots (int64,
    -1 = padding) of the caches [num_blocks, 64, heads, head_dim]."""
    kv = _kv(k_cache, v_cache)
    _dense(slot_mapping, "slot_mapping", torch.int64)
    n = int(slot_mapping.shape[0])
    for t, what in ((k, "k"), (v, "v")):
        _here(t, what, k_cache.dtype)
        if t.dim() != 3 or tuple(t.shape[1:]) != (kv.num_kv_heads, kv.head_dim) or t.shape[0] != n:
            raise DsaError(f"{what} must be [{n}, {kv.num_kv_heads}, {kv.head_dim}]")
    if n == 0:
        return
    ks, vs = _strides(k, (0, 1), "k"), _strides(v, (0, 1), "v")
    st = load().dsa_kv_write(k.data_ptr(), *ks, v.data_ptr(), *vs, n, slot_mapping.data_ptr(), ctypes.byref(kv),
                             _err(dev_err), _on(stream).cuda_stream)
    _check(st, "dsa_kv_write")


def attn_decode_workspace_size(batch, num_heads: int, num_kv_heads: int, head_dim: int) -> int:
    return int(load().dsa_attn_decode_workspace_size(ctypes.byref(batch.c), int(num_heads), int(num_kv_heads),
                                                     int(head_dim)))


def attn_decode(batch, q, k_cache, v_cache, scale: float = 0.0, out=None, lse=None, ws=None, dev_err=None,
                stream=None):
    """Attention of the batch's decode tokens, rows [0, num_decode_tokens) of q
    [tokens, heads, head_dim], over their requests' pages. Returns (out, lse);
    the other rows of a passed ``out`` and ``lse`` stay as they were."""
    kv = _kv(k_cache, v_cache)
    at, o, l = _attn(q, out, lse, kv, k_cache.dtype, scale, 0, batch.num_decode_tokens, stream)
    ws = _scratch(ws, attn_decode_workspace_size(batch, at.num_heads, kv.num_kv_heads, kv.head_dim)
                  if ws is None else 0, q.device, stream)
    st = load().dsa_attn_decode(ctypes.byref(batch.c), ctypes.byref(kv), ctypes.byref(at), ws.data_ptr(), ws.numel(),
                                _err(dev_err), _on(stream).cuda_stream)
    _check(st, "dsa_attn_decode")
    return o, l


def attn_selected_workspace_size(n_tokens: int, topk: int, num_heads: int, num_kv_heads: int, head_dim: int) -> int:
    return int(load().dsa_attn_selected_workspace_size(int(n_tokens), int(topk), int(num_heads), int(num_kv_heads),
                                                       int(head_dim)))


def attn_selected(q, k_cache, v_cache, physical, scale: float = 0.0, out=None, lse=None, ws=None, dev_err=None,
                  stream=None):
    """Attention of each row of q [tokens, heads, head_dim] over the slots
    physical [tokens, topk] (int32, -1 = none) selects for it. Returns (out, lse)."""
    kv = _kv(k_cache, v_cache)
    _dense(physical, "physical", torch.int32)
    if physical.dim() != 2 or physical.shape[1] < 1:
        raise DsaError("physical must be [tokens, topk]")
    n, topk = (int(x) for x in physical.shape)
    at, o, l = _attn(q, out, lse, kv, k_cache.dtype, scale, 0, n, stream)
    if q.shape[0] != n:
        raise DsaError(f"q has {q.shape[0]} rows, physical {n}")
    ws = _scratch(ws, attn_selected_workspace_size(n, topk, at.num_heads, kv.num_kv_heads, kv.head_dim)
                  if ws is None else 0, q.device, stream)
    st = load().dsa_attn_selected(ctypes.byref(kv), ctypes.byref(at), physical.data_ptr(), n, topk, ws.data_ptr(),
                                  ws.numel(), _err(dev_err), _on(stream).cuda_stream)
    _check(st, "dsa_attn_selected")
    return o, l


def attn_prompt(batch, q, k, v, scale: float = 0.0, kv_start=None, out=None, lse=None, dev_err=None, stream=None):
    """Causal attention of the batch's prefill tokens, rows [num_decode_tokens,
    num_tokens) of q [tokens, heads, head_dim]. k and v are the paged caches, or
    with ``kv_start`` (int32 [num_reqs]) packed rows [rows, heads, head_dim]
    where key s of request r is row kv_start[r] + s. Returns (out, lse); the
    other rows of a passed ``out`` and ``lse`` stay as they were."""
    kv = _kv(k, v, packed=kv_start is not None)
    if kv_start is not None and _dense(kv_start, "kv_start", torch.int32).numel() < batch.num_reqs:
        raise DsaError("kv_start needs an entry per request")
    at, o, l = _attn(q, out, lse, kv, k.dtype, scale, batch.num_decode_tokens, batch.num_tokens, stream)
    st = load().dsa_attn_prompt(ctypes.byref(batch.c), ctypes.byref(kv), _ptr(kv_start), ctypes.byref(at),
                                _err(dev_err), _on(stream).cuda_stream)
    _check(st, "dsa_attn_prompt")
    return o, l


# ---------------------------------------------------------------- pages

def _caches(caches, num_blocks):
    """The C array for caches whose first axis is the page."""
    arr = (DsaCacheDescC * max(len(caches), 1))()
    for i, t in enumerate(caches):
        _here(t, f"caches[{i}]")
        if t.dim() < 2 or t.shape[0] != num_blocks:
            raise DsaError(f"caches[{i}] must have {num_blocks} pages as its first axis")
        if not t[0].is_contiguous():
            raise DsaError(f"caches[{i}] must have contiguous pages")
        size = t[0].numel() * t.element_size()
        arr[i] = DsaCacheDescC(t.data_ptr(), size, t.stride(0) * t.element_size() if num_blocks > 1 else size)
    return arr, len(caches)


def _pool(refs, block_table, seq_lens):
    _dense(refs, "refs", torch.int32)
    _dense(block_table, "block_table", torch.int32)
    if refs.dim() != 1 or block_table.dim() != 2 or block_table.shape[1] < 1:
        raise DsaError("refs must be [num_blocks], block_table [rows, entries]")
    rows = int(block_table.shape[0])
    if seq_lens is not None and (_dense(seq_lens, "seq_lens", torch.int32).dim() != 1 or seq_lens.shape[0] != rows):
        raise DsaError("seq_lens needs an entry per row of block_table")
    return DsaPagesC(refs.data_ptr(), int(refs.shape[0]), block_table.data_ptr(), int(block_table.shape[1]), rows,
                     seq_lens.data_ptr() if seq_lens is not None else None)


def _list(t, what, n=None):
    if _dense(t, what, torch.int32).dim() != 1 or (n is not None and t.shape[0] != n):
        raise DsaError(f"{what} must be a list" + (f" of {n}" if n is not None else ""))
    return int(t.shape[0])


def pages_workspace_size(num_blocks: int, n: int) -> int:
    return int(load().dsa_pages_workspace_size(int(num_blocks), int(n)))


def pages_copy(caches, src, dst, ws=None, dev_err=None, stream=None):
    """Page src[i] over page dst[i] in every cache [num_blocks, ...] (int32
    lists; -1 = padding). A page is the destination of one pair at most and
    then no source; other pairs are skipped and flagged."""
    if not caches:
        raise DsaError("pages_copy needs a cache")
    n = _list(src, "src")
    _list(dst, "dst", n)
    blocks = int(caches[0].shape[0])
    arr, m = _caches(caches, blocks)
    ws = _scratch(ws, pages_workspace_size(blocks, n) if ws is None else 0, src.device, stream)
    st = load().dsa_pages_copy(arr, m, blocks, src.data_ptr(), dst.data_ptr(), n, ws.data_ptr(), ws.numel(),
                               _err(dev_err), _on(stream).cuda_stream)
    _check(st, "dsa_pages_copy")


def pages_fork(refs, block_table, seq_lens, parents, children, caches=(), ws=None, dev_err=None, stream=None):
    """Make rows ``children`` copies of rows ``parents``: full pages shared
    (counts up), a part-filled last page copied to a fresh page in every cache."""
    g = _pool(refs, block_table, seq_lens)
    n = _list(parents, "parents")
    _list(children, "children", n)
    arr, m = _caches(caches, g.num_blocks)
    ws = _scratch(ws, pages_workspace_size(g.num_blocks, n) if ws is None else 0, refs.device, stream)
    st = load().dsa_pages_fork(ctypes.byref(g), parents.data_ptr(), children.data_ptr(), n, arr, m, ws.data_ptr(),
                               ws.numel(), _err(dev_err), _on(stream).cuda_stream)
    _check(st, "dsa_pages_fork")


def pages_free(refs, block_table, seq_lens, rows, dev_err=None, stream=None):
    """End the sequences of these rows: their pages' counts go down, their
    entries become -1, their lengths 0."""
    g = _pool(refs, block_table, seq_lens)
    st = load().dsa_pages_free(ctypes.byref(g), rows.data_ptr(), _list(rows, "rows"), _err(dev_err),
                               _on(stream).cuda_stream)
    _check(st, "dsa_pages_free")


def pages_compact(refs, block_table, caches=(), ws=None, dev_err=None, stream=None):
    """Move the pool's used pages to its front: counts, block-table entries and
    every cache's bytes follow."""
    g = _pool(refs, block_table, None)
    arr, m = _caches(caches, g.num_blocks)
    ws = _scratch(ws, pages_workspace_size(g.num_blocks, 0) if ws is None else 0, refs.device, stream)
    st = load().dsa_pages_compact(ctypes.byref(g), arr, m, ws.data_ptr(), ws.numel(), _err(dev_err),
                                  _on(stream).cuda_stream)
    _check(st, "dsa_pages_compact")
