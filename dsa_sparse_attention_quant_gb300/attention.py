"""The attention that reads the paged KV cache, the cache's writer and its page
calls: argument marshalling for the entry points of ``include/dsaidx.h`` that
take a ``DsaKv`` or ``DsaPages``.

Tensors are on the current CUDA device. Results and scratch are allocated with
torch when the caller does not pass them, with ``stream`` given as that
stream's memory. Every call is asynchronous.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from .binding import DsaAttnC, DsaCacheDescC, DsaError, DsaKvC, DsaPagesC, _check, load

BLOCK_SIZE = 64
_DTYPES = {torch.bfloat16: 0, torch.float16: 1}
# torch.cuda.current_device() without its check that CUDA is up: asked only once a CUDA tensor is at hand
_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def new_kv_cache(num_blocks: int, num_kv_heads: int, head_dim: int, dtype=torch.bfloat16, device=None):
    """A zeroed pair of K and V caches [num_blocks, 64, num_kv_heads, head_dim]."""
    if dtype not in _DTYPES or head_dim not in (64, 128) or num_blocks < 1 or num_kv_heads < 1:
        raise DsaError("a KV cache has bf16 or fp16 rows of 64 or 128, at least one page and one head")
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    shape = (int(num_blocks), BLOCK_SIZE, int(num_kv_heads), int(head_dim))
    return torch.zeros(shape, dtype=dtype, device=dev), torch.zeros(shape, dtype=dtype, device=dev)


# ---------------------------------------------------------------- arguments
# A decode step makes these calls once per layer, so their host time counts: the
# C structs are packed with ``struct`` (their layout is checked against ctypes
# below) and every check is one or two cheap tensor queries.

_KV = struct.Struct("PPiii4xq6q")         # DsaKv
_ATTN = struct.Struct("PqqPqqPif")        # DsaAttn
_PAGES = struct.Struct("PqPqi4xP")        # DsaPages
assert (_KV.size, _ATTN.size, _PAGES.size) == tuple(ctypes.sizeof(c) for c in (DsaKvC, DsaAttnC, DsaPagesC))


def _here(t, what, dtype=None):
    """A CUDA tensor of the current device (and of dtype)."""
    at = t.get_device() if isinstance(t, torch.Tensor) else -1
    if at < 0:
        raise DsaError(f"{what} must be a CUDA tensor")
    if at != _device():
        raise DsaError(f"{what} is on cuda:{at}, the current device is cuda:{_device()}")
    if dtype is not None and t.dtype is not dtype:
        raise DsaError(f"{what} must be {dtype}, got {t.dtype}")
    return t


def _dense(t, what, dtype):
    if not _here(t, what, dtype).is_contiguous():
        raise DsaError(f"{what} must be contiguous")
    return t


def _err(dev_err):
    return None if dev_err is None else _dense(dev_err, "dev_err", torch.int32).data_ptr()


def _kv(k, v, packed=False):
    """(C description, heads, head_dim, dtype) of a cache [num_blocks, 64, heads,
    head_dim], or of packed rows [rows, heads, head_dim]; any strides with a
    contiguous last axis."""
    _here(k, "k")
    shape, dtype = k.shape, k.dtype
    code = _DTYPES.get(dtype)
    if code is None:
        raise DsaError(f"k must be bf16 or fp16, got {dtype}")
    if not isinstance(v, torch.Tensor) or v.get_device() != k.get_device() or v.dtype is not dtype or v.shape != shape:
        _here(v, "v", dtype)
        raise DsaError("k and v must have one shape")
    ks, vs = k.stride(), v.stride()
    if ks[-1] != 1 or vs[-1] != 1:
        raise DsaError("k and v must have a contiguous last axis")
    if packed:
        if len(shape) != 3:
            raise DsaError("k and v must be [rows, heads, head_dim]")
        n, heads, d = shape
        return _KV.pack(k.data_ptr(), v.data_ptr(), code, heads, d, n, d, ks[0], ks[1], d, vs[0], vs[1]), heads, d, dtype
    if len(shape) != 4 or shape[1] != BLOCK_SIZE:
        raise DsaError("k and v must be [num_blocks, 64, heads, head_dim]")
    n, _, heads, d = shape
    return _KV.pack(k.data_ptr(), v.data_ptr(), code, heads, d, n, *ks[:3], *vs[:3]), heads, d, dtype


def _made(stream, shape, dtype, device, rest):
    """A result made here, for the stream it is written on; ``rest`` fills the
    rows that the call does not write (None: it writes every row)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _made(None, shape, dtype, device, rest)
    if rest is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return torch.full(shape, rest, dtype=dtype, device=device)


def _attn(q, out, lse, kv_heads, d, dtype, scale, rows, every, stream):
    """(C description, out, lse, heads) for a call that reaches rows [0, rows)
    and writes every row or only some, allocating what is missing: rows that are
    not written are empty ones (0, -infinity)."""
    shape = _here(q, "q", dtype).shape
    if len(shape) != 3 or shape[2] != d:
        raise DsaError(f"q must be [tokens, heads, {d}]")
    n, heads, _ = shape
    if n < rows:
        raise DsaError(f"q has {n} rows, the call needs {rows}")
    if heads == 0 or kv_heads == 0 or heads % kv_heads:
        raise DsaError(f"{heads} query heads cannot share {kv_heads} KV heads")
    if out is None:
        out = _made(stream, shape, dtype, q.device, None if every else 0.0)
    elif not isinstance(out, torch.Tensor) or out.get_device() != q.get_device() or out.dtype is not dtype \
            or out.shape != shape:
        _here(out, "out", dtype)
        raise DsaError("out must have q's shape")
    if lse is None:
        lse = _made(stream, shape[:2], torch.float32, q.device, None if every else -math.inf)
    elif _dense(lse, "lse", torch.float32).shape != shape[:2]:
        raise DsaError("lse must be [tokens, heads]")
    qs, os = q.stride(), out.stride()
    if qs[2] != 1 or os[2] != 1:
        raise DsaError("q and out must have a contiguous last axis")
    return (_ATTN.pack(q.data_ptr(), qs[0], qs[1], out.data_ptr(), os[0], os[1], lse.data_ptr(), heads, scale), out,
            lse, heads)


def _on(stream):
    """The C stream: the given one, or the current device's current one."""
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(_device())


def _scratch(ws, nbytes, device, stream):
    """A scratch of nbytes() bytes that belongs to the stream it is used on, or
    the caller's, checked."""
    if ws is not None:
        return _dense(ws, "ws", torch.uint8)
    size = max(int(nbytes()), 16)
    if stream is None:
        return torch.empty(size, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(size, dtype=torch.uint8, device=device)


# ---------------------------------------------------------------- entry points

def kv_write(k, v, slot_mapping, k_cache, v_cache, dev_err=None, stream=None):
    """Write the rows k and v [tokens, heads, head_dim] at their slots (int64,
    -1 = padding) of the caches [num_blocks, 64, heads, head_dim]."""
    kv, heads, d, dtype = _kv(k_cache, v_cache)
    n = _dense(slot_mapping, "slot_mapping", torch.int64).numel()
    want = (n, heads, d)
    for t, what in ((k, "k rows"), (v, "v rows")):
        if _here(t, what, dtype).shape != want:
            raise DsaError(f"{what} must be [{n}, {heads}, {d}]")
        if t.stride(2) != 1:
            raise DsaError(f"{what} must have a contiguous last axis")
    if n == 0:
        return
    st = load().dsa_kv_write(k.data_ptr(), *k.stride()[:2], v.data_ptr(), *v.stride()[:2], n, slot_mapping.data_ptr(),
                             kv, _err(dev_err), _on(stream))
    _check(st, "dsa_kv_write")


def attn_decode_workspace_size(batch, num_heads: int, num_kv_heads: int, head_dim: int) -> int:
    return int(load().dsa_attn_decode_workspace_size(ctypes.byref(batch.c), int(num_heads), int(num_kv_heads),
                                                     int(head_dim)))


def attn_decode(batch, q, k_cache, v_cache, scale: float = 0.0, out=None, lse=None, ws=None, dev_err=None,
                stream=None):
    """Attention of the batch's decode tokens, rows [0, num_decode_tokens) of q
    [tokens, heads, head_dim], over their requests' pages. Returns (out, lse);
    the other rows of a passed ``out`` and ``lse`` stay as they were, of one made
    here they are 0 and -infinity."""
    kv, kv_heads, d, dtype = _kv(k_cache, v_cache)
    _here(batch.seq_lens, "the batch")
    n = batch.num_decode_tokens
    at, out, lse, heads = _attn(q, out, lse, kv_heads, d, dtype, scale, n, n == q.shape[0], stream)
    ws = _scratch(ws, lambda: attn_decode_workspace_size(batch, heads, kv_heads, d), q.device, stream)
    st = load().dsa_attn_decode(ctypes.byref(batch.c), kv, at, ws.data_ptr(), ws.numel(), _err(dev_err), _on(stream))
    _check(st, "dsa_attn_decode")
    return out, lse


def attn_selected_workspace_size(n_tokens: int, topk: int, num_heads: int, num_kv_heads: int, head_dim: int) -> int:
    return int(load().dsa_attn_selected_workspace_size(int(n_tokens), int(topk), int(num_heads), int(num_kv_heads),
                                                       int(head_dim)))


def attn_selected(q, k_cache, v_cache, physical, scale: float = 0.0, out=None, lse=None, ws=None, dev_err=None,
                  stream=None):
    """Attention of each row of q [tokens, heads, head_dim] over the slots
    physical [tokens, topk] (int32, -1 = none) selects for it. Returns (out, lse)."""
    kv, kv_heads, d, dtype = _kv(k_cache, v_cache)
    shape = _dense(physical, "physical", torch.int32).shape
    if len(shape) != 2 or shape[1] < 1:
        raise DsaError("physical must be [tokens, topk]")
    n, topk = shape
    at, out, lse, heads = _attn(q, out, lse, kv_heads, d, dtype, scale, n, True, stream)
    if q.shape[0] != n:
        raise DsaError(f"q has {q.shape[0]} rows, physical {n}")
    ws = _scratch(ws, lambda: attn_selected_workspace_size(n, topk, heads, kv_heads, d), q.device, stream)
    st = load().dsa_attn_selected(kv, at, physical.data_ptr(), n, topk, ws.data_ptr(), ws.numel(), _err(dev_err),
                                  _on(stream))
    _check(st, "dsa_attn_selected")
    return out, lse


def attn_prompt(batch, q, k, v, scale: float = 0.0, kv_start=None, out=None, lse=None, dev_err=None, stream=None):
    """Causal attention of the batch's prefill tokens, rows [num_decode_tokens,
    num_tokens) of q [tokens, heads, head_dim]. k and v are the paged caches, or
    with ``kv_start`` (int32 [num_reqs]) packed rows [rows, heads, head_dim]
    where key s of request r is row kv_start[r] + s. Returns (out, lse); the
    other rows, and those that are no request's (behind query_start_loc's end, of
    a request that is refused), stay as they were in a passed ``out`` and
    ``lse``. Which they are is known on the GPU alone, so results made here are
    filled with 0 and -infinity first: passing both saves that."""
    kv, kv_heads, d, dtype = _kv(k, v, packed=kv_start is not None)
    _here(batch.seq_lens, "the batch")
    start = None
    if kv_start is not None:
        start = _dense(kv_start, "kv_start", torch.int32).data_ptr()
        if kv_start.numel() < batch.num_reqs:
            raise DsaError("kv_start needs an entry per request")
    at, out, lse, _ = _attn(q, out, lse, kv_heads, d, dtype, scale, batch.num_tokens, False, stream)
    st = load().dsa_attn_prompt(ctypes.byref(batch.c), kv, start, at, _err(dev_err), _on(stream))
    _check(st, "dsa_attn_prompt")
    return out, lse


# ---------------------------------------------------------------- pages

def _caches(caches, num_blocks):
    """The C array for caches whose first axis is the page."""
    flat, like, dev, size = [], None, -1, 0
    for t in caches:
        if not isinstance(t, torch.Tensor) or t.get_device() != dev or dev < 0:
            dev = _here(t, "a cache").get_device()
        kind = t.shape, t.dtype
        if kind != like:   # a model's caches are mostly alike
            if t.dim() < 2 or t.size(0) != num_blocks:
                raise DsaError(f"a cache must have {num_blocks} pages as its first axis")
            like, size = kind, t.nbytes // max(num_blocks, 1)
        stride = size
        if not t.is_contiguous():
            if not t[0].is_contiguous():
                raise DsaError("a cache must have contiguous pages")
            if num_blocks > 1:
                stride = t.stride(0) * t.element_size()
        flat += (t.data_ptr(), size, stride)
    return struct.pack(f"{len(flat)}q", *flat), len(caches)


assert ctypes.sizeof(DsaCacheDescC) == struct.calcsize("3q")


def _pool(refs, block_table, seq_lens):
    _dense(refs, "refs", torch.int32)
    shape = _dense(block_table, "block_table", torch.int32).shape
    if refs.dim() != 1 or len(shape) != 2 or shape[1] < 1:
        raise DsaError("refs must be [num_blocks], block_table [rows, entries]")
    if seq_lens is not None and _dense(seq_lens, "seq_lens", torch.int32).shape != shape[:1]:
        raise DsaError("seq_lens needs an entry per row of block_table")
    n = refs.numel()
    return _PAGES.pack(refs.data_ptr(), n, block_table.data_ptr(), shape[1], shape[0],
                       seq_lens.data_ptr() if seq_lens is not None else 0), n


def _list(t, what, n=None):
    if _dense(t, what, torch.int32).dim() != 1 or (n is not None and t.numel() != n):
        raise DsaError(f"{what} must be a list" + (f" of {n}" if n is not None else ""))
    return t.numel()


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
    ws = _scratch(ws, lambda: pages_workspace_size(blocks, n), src.device, stream)
    st = load().dsa_pages_copy(arr, m, blocks, src.data_ptr(), dst.data_ptr(), n, ws.data_ptr(), ws.numel(),
                               _err(dev_err), _on(stream))
    _check(st, "dsa_pages_copy")


def pages_fork(refs, block_table, seq_lens, parents, children, caches=(), ws=None, dev_err=None, stream=None):
    """Make rows ``children`` copies of rows ``parents``: full pages shared
    (counts up), a part-filled last page copied to a fresh page in every cache."""
    if seq_lens is None:
        raise DsaError("pages_fork needs seq_lens")
    pool, blocks = _pool(refs, block_table, seq_lens)
    n = _list(parents, "parents")
    _list(children, "children", n)
    arr, m = _caches(caches, blocks)
    ws = _scratch(ws, lambda: pages_workspace_size(blocks, n), refs.device, stream)
    st = load().dsa_pages_fork(pool, parents.data_ptr(), children.data_ptr(), n, arr, m, ws.data_ptr(), ws.numel(),
                               _err(dev_err), _on(stream))
    _check(st, "dsa_pages_fork")


def pages_free(refs, block_table, seq_lens, rows, dev_err=None, stream=None):
    """End the sequences of these rows: their pages' counts go down, their
    entries become -1, their lengths 0."""
    if seq_lens is None:
        raise DsaError("pages_free needs seq_lens")
    pool, _ = _pool(refs, block_table, seq_lens)
    st = load().dsa_pages_free(pool, rows.data_ptr(), _list(rows, "rows"), _err(dev_err), _on(stream))
    _check(st, "dsa_pages_free")


def pages_compact(refs, block_table, caches=(), ws=None, dev_err=None, stream=None):
    """Move the pool's used pages to its front: counts, block-table entries and
    every cache's bytes follow."""
    pool, blocks = _pool(refs, block_table, None)
    arr, m = _caches(caches, blocks)
    ws = _scratch(ws, lambda: pages_workspace_size(blocks, 0), refs.device, stream)
    st = load().dsa_pages_compact(pool, arr, m, ws.data_ptr(), ws.numel(), _err(dev_err), _on(stream))
    _check(st, "dsa_pages_compact")
