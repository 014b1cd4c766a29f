"""Attention-layer operators on torch tensors: head norms with rotation, the
paged key/value cache, and attention over it.

Owners and argument checks only; the work runs in libdg.so (the dg_qk_norm_rope
and dg_cache_* calls of include/dg.h). Calls run on torch's current stream of
the tensors' device, allocate their outputs and scratch with torch, and can be
captured into a CUDA graph. They are for inference: results carry no gradient.
A given out or lse shares no memory with an input.
"""
from __future__ import annotations

import ctypes

import torch

from . import (DG_BF16, DG_F32, DG_KV_BF16, DG_KV_E4M3, DG_MASK_CAUSAL, DG_MASK_FULL, DG_MASK_TREE,
               DgError, dg_cache_attention, dg_cache_attention_scratch_bytes, dg_cache_read,
               dg_cache_write, dg_kv_batch, dg_kv_cache, dg_qk_norm_rope)

# the current stream's handle without a Stream object around it: a tenth of the time
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch.cuda.current_device
_empty_like, _contiguous = torch.empty_like, torch.contiguous_format
_KEPT_SIZES = 64            # scratch sizes a cache remembers (one per shape of call)
_DTYPES = {torch.bfloat16: DG_BF16, torch.float32: DG_F32}


def _call(index: int, fn, *args) -> None:
    """fn(*args, stream) on torch's current stream of device `index`, that device current."""
    if _current_device() == index:
        fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            fn(*args, _raw_stream(index))


def _dtype(t) -> int:
    try:
        return _DTYPES[t]
    except KeyError:
        raise ValueError(f"dtype must be bfloat16 or float32, not {t}") from None


def _rows(name, t, heads, head_dim, index, tokens=None):
    """Check a [tokens, heads, head_dim] argument; returns its (token, head) strides."""
    shape = t.shape
    if len(shape) != 3 or t.get_device() != index or (tokens is not None and shape[0] != tokens) \
            or (heads is not None and shape[1] != heads) or shape[2] != head_dim:
        raise ValueError(f"{name} must be [{'tokens' if tokens is None else tokens}, "
                         f"{'heads' if heads is None else heads}, {head_dim}] on cuda:{index}, got "
                         f"{tuple(shape)} on {t.device}")
    st, sh, sd = t.stride()
    if sd != 1 and head_dim > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    # a stride over a dimension of one element is never taken
    return (st if shape[0] > 1 else 0), (sh if shape[1] > 1 else 0)


def _vector(name, t, dtype, index, n):
    if t.dtype is not dtype or t.get_device() != index or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} vector of {n} on cuda:{index}")
    return t.data_ptr()


def rope_frequencies(rot_dim: int, base: float = 10000.0, device="cuda"):
    """inv_freq for qk_norm_rope: base^(-2i / rot_dim), i < rot_dim / 2, in fp64."""
    i = torch.arange(rot_dim // 2, dtype=torch.float64, device=device)
    return base ** (-2.0 * i / rot_dim)


def qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, *, interleaved: bool = False,
                 eps: float = 1e-6, weight_offset: float = 0.0):
    """RMS-norm every head of q [tokens, q_heads, D] and k [tokens, k_heads, D], then rotate the
    first 2 * len(inv_freq) elements by positions (see dg_qk_norm_rope). Returns new (q, k).

    weights: [D] of q's dtype, or None for ones; positions int32 [tokens]; inv_freq float64.
    """
    dt = q.dtype
    code = _dtype(dt)
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    if k.dtype is not dt:
        raise ValueError("q and k must have one dtype")
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [tokens, heads, head_dim]")
    index = q.get_device()
    tokens, hq, d = q.shape
    hk, half = k.shape[1], inv_freq.shape[0]
    qs, ks = _rows("q", q, None, d, index), _rows("k", k, None, d, index, tokens)
    wq = _vector("q_weight", q_weight, dt, index, d) if q_weight is not None else None
    wk = _vector("k_weight", k_weight, dt, index, d) if k_weight is not None else None
    pos = _vector("positions", positions, torch.int32, index, tokens)
    freq = _vector("inv_freq", inv_freq, torch.float64, index, half)
    qo, ko = _empty_like(q, memory_format=_contiguous), _empty_like(k, memory_format=_contiguous)
    _call(index, dg_qk_norm_rope, tokens, hq, hk, d, 2 * half, interleaved, code, q.data_ptr(), *qs,
          k.data_ptr(), *ks, wq, wk, weight_offset, eps, pos, freq, qo.data_ptr(), ko.data_ptr())
    return qo, ko


class KVBatch:
    """Which tokens a cache call is about: sequence b has rows first[b] .. first[b+1]-1 at the
    positions past[b], past[b]+1, ... of the pages page_table[b] (int32 CUDA tensors, kept by
    reference: a captured graph replays with whatever they hold then). tokens: rows of q, k, v;
    rows from first[-1] on are padding."""

    def __init__(self, page_table, first, past, tokens: int):
        dev = page_table.device
        if not page_table.is_cuda or page_table.dtype != torch.int32 or page_table.dim() != 2 \
                or not page_table.is_contiguous():
            raise ValueError("page_table must be a contiguous int32 CUDA tensor [batch, pages]")
        n, index = page_table.shape[0], page_table.get_device()
        _vector("first", first, torch.int32, index, n + 1)
        _vector("past", past, torch.int32, index, n)
        self.page_table, self.first, self.past, self.tokens = page_table, first, past, int(tokens)
        self.device, self.index = dev, index
        self.c = dg_kv_batch(page_table=page_table.data_ptr(), first=first.data_ptr(),
                             past=past.data_ptr(), batch=n, table_stride=page_table.shape[1],
                             tokens=self.tokens)


class KVCache:
    """A paged cache over caller-made tensors: k, v [pages, kv_heads, page_size, head_dim], bf16, or
    float8_e4m3fn with k_exp, v_exp uint8 [pages, kv_heads, page_size]."""

    def __init__(self, k, v, k_exp=None, v_exp=None):
        dev = k.device
        if k.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise ValueError("cache pages must be bfloat16 or float8_e4m3fn")
        for name, t, shape, dt in (("k", k, k.shape, k.dtype), ("v", v, k.shape, k.dtype)) + (
                (("k_exp", k_exp, k.shape[:3], torch.uint8), ("v_exp", v_exp, k.shape[:3], torch.uint8))
                if k.dtype != torch.bfloat16 else ()):
            if t is None or not t.is_cuda or t.device != dev or t.dim() != len(shape) or len(k.shape) != 4 \
                    or t.shape != shape or t.dtype != dt or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {dt} CUDA tensor {tuple(shape)}, pages "
                                 "[pages, kv_heads, page_size, head_dim] on one device")
        self.k, self.v, self.k_exp, self.v_exp, self.device, self.index = k, v, k_exp, v_exp, dev, k.get_device()
        self._scratch = {}                  # bytes by (tokens, batch, q_heads)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        f8 = k.dtype != torch.bfloat16
        self.c = dg_kv_cache(k=k.data_ptr(), v=v.data_ptr(), k_exp=k_exp.data_ptr() if f8 else None,
                             v_exp=v_exp.data_ptr() if f8 else None, status=self.status.data_ptr(),
                             pages=k.shape[0], page_size=k.shape[2], kv_heads=k.shape[1],
                             head_dim=k.shape[3], format=DG_KV_E4M3 if f8 else DG_KV_BF16)

    @classmethod
    def empty(cls, pages: int, page_size: int, kv_heads: int, head_dim: int,
              fmt: int = DG_KV_BF16, device="cuda"):
        """A cache with pages of its own, zeroed."""
        shape = (pages, kv_heads, page_size, head_dim)
        if fmt == DG_KV_BF16:
            return cls(*(torch.zeros(shape, dtype=torch.bfloat16, device=device) for _ in "kv"))
        kv = (torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in "kv")
        return cls(*kv, *(torch.zeros(shape[:3], dtype=torch.uint8, device=device) for _ in "kv"))

    def check(self) -> None:
        """Raise DgError if a call met a bad page or a wait ran out. Waits for the whole device: calls
        may have run on any of its streams. The first error stays until status is set to zero."""
        torch.cuda.synchronize(self.index)
        code = int(self.status.item())
        if code:
            raise DgError(code, "a cache call met a page or position outside the cache, or a wait ran out")

    def _batch(self, batch):
        if batch.index != self.index:
            raise ValueError(f"the batch is on {batch.device}, the cache on {self.device}")

    def write(self, k, v, batch: KVBatch) -> None:
        """Write k, v [tokens, kv_heads, head_dim] (bf16 or fp32) at the batch's positions."""
        self._batch(batch)
        c, index, tokens = self.c, self.index, batch.tokens
        code = _dtype(k.dtype)
        if v.dtype is not k.dtype:
            raise ValueError("k and v must have one dtype")
        h, d = c.kv_heads, c.head_dim
        ks, vs = _rows("k", k, h, d, index, tokens), _rows("v", v, h, d, index, tokens)
        _call(index, dg_cache_write, c, batch.c, code, k.data_ptr(), *ks, v.data_ptr(), *vs)

    def read(self, batch: KVBatch, dtype=torch.bfloat16, out=None):
        """The batch's rows as (k, v) [tokens, kv_heads, head_dim]; padding rows are not written."""
        self._batch(batch)
        c, index = self.c, self.index
        code = _dtype(dtype)
        if out is None:
            shape = (batch.tokens, c.kv_heads, c.head_dim)
            k, v = self.k.new_empty(shape, dtype=dtype), self.k.new_empty(shape, dtype=dtype)
        else:
            k, v = out
            for t in (k, v):
                _rows("out", t, c.kv_heads, c.head_dim, index, batch.tokens)
                if t.dtype is not dtype or not t.is_contiguous():
                    raise ValueError(f"out must be contiguous {dtype}")
        _call(index, dg_cache_read, c, batch.c, code, k.data_ptr(), v.data_ptr())
        return k, v

    def attend(self, q, batch: KVBatch, mask: int, *, tree=None, scale: float | None = None, out=None,
               lse=None):
        """Attention of q [tokens, q_heads, head_dim] (bf16) over the cache; returns (out, lse).

        mask: DG_MASK_FULL, DG_MASK_CAUSAL, or DG_MASK_TREE with tree int32 [tokens, words] (bit j of
        a row: this token sees new token j of its sequence). scale defaults to head_dim ** -0.5.
        The keys and values of the new tokens are in the cache already (write). out and lse may be
        given; padding rows are not written.
        """
        self._batch(batch)
        c, index, tokens = self.c, self.index, batch.tokens
        if q.dtype is not torch.bfloat16:
            raise ValueError("q must be bfloat16")
        qs = _rows("q", q, None, c.head_dim, index, tokens)
        hq, words, tree_ptr = q.shape[1], 0, None
        if mask == DG_MASK_TREE:
            if tree is None or tree.dtype is not torch.int32 or tree.get_device() != index or tree.dim() != 2 \
                    or tree.shape[0] != tokens or not tree.is_contiguous():
                raise ValueError(f"tree must be a contiguous int32 tensor [{tokens}, words] on {self.device}")
            words, tree_ptr = tree.shape[1], tree.data_ptr()
        elif tree is not None:
            raise ValueError("tree goes with DG_MASK_TREE")
        if out is None:
            out = _empty_like(q, memory_format=_contiguous)
        elif out.dtype is not torch.bfloat16 or out.shape != q.shape or not out.is_contiguous() \
                or out.get_device() != index:
            raise ValueError("out must be contiguous bfloat16 of q's shape")
        if lse is None:
            lse = q.new_empty((tokens, hq), dtype=torch.float32)
        elif lse.dtype is not torch.float32 or lse.shape != q.shape[:2] or not lse.is_contiguous() \
                or lse.get_device() != index:
            raise ValueError("lse must be contiguous float32 [tokens, q_heads]")
        key = (tokens, batch.c.batch, hq)
        n = self._scratch.get(key)
        if n is None:
            n = dg_cache_attention_scratch_bytes(c, batch.c, hq)
            if n:                           # 0: the call below is refused, for reasons the key lacks
                if len(self._scratch) == _KEPT_SIZES:
                    self._scratch.clear()
                self._scratch[key] = n
        scratch = self.status.new_empty((n // 4,))
        _call(index, dg_cache_attention, c, batch.c, hq, q.data_ptr(), *qs,
              c.head_dim ** -0.5 if scale is None else scale, mask, tree_ptr, words, out.data_ptr(),
              lse.data_ptr(), scratch.data_ptr(), n)
        return out, lse
