"""Attention-layer operators on torch tensors: head norms with rotation, the
paged key/value cache, and attention over it.

Owners and argument checks only; the work runs in libdg.so (the dg_qk_norm_rope
and dg_cache_* calls of include/dg.h). Calls run on torch's current stream of
the tensors' device, allocate their outputs and scratch with torch, and can be
captured into a CUDA graph.
"""
from __future__ import annotations

import ctypes

import torch

from . import (DG_BF16, DG_F32, DG_KV_BF16, DG_KV_E4M3, DG_MASK_CAUSAL, DG_MASK_FULL, DG_MASK_TREE,
               DgError, dg_cache_attention, dg_cache_attention_scratch_bytes, dg_cache_read,
               dg_cache_write, dg_kv_batch, dg_kv_cache, dg_qk_norm_rope)

_DTYPES = {torch.bfloat16: DG_BF16, torch.float32: DG_F32}


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _dtype(t) -> int:
    try:
        return _DTYPES[t if isinstance(t, torch.dtype) else t.dtype]
    except KeyError:
        raise ValueError(f"dtype must be bfloat16 or float32, not {t}") from None


def _rows(name, t, heads, head_dim, device, tokens=None):
    """Check a [tokens, heads, head_dim] argument; returns its (token, head) strides."""
    if t.dim() != 3 or t.device != device or (tokens is not None and t.shape[0] != tokens) \
            or (heads is not None and t.shape[1] != heads) or t.shape[2] != head_dim:
        raise ValueError(f"{name} must be [{'tokens' if tokens is None else tokens}, "
                         f"{'heads' if heads is None else heads}, {head_dim}] on {device}, got "
                         f"{tuple(t.shape)} on {t.device}")
    st, sh, sd = t.stride()
    if sd != 1 and head_dim > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    # a stride over a dimension of one element is never taken
    return (st if t.shape[0] > 1 else 0), (sh if t.shape[1] > 1 else 0)


def _vector(name, t, dtype, device, n):
    if t.dtype != dtype or t.device != device or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} vector of {n} on {device}")
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
    dt, dev = _dtype(q), q.device
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    if k.dtype != q.dtype:
        raise ValueError("q and k must have one dtype")
    tokens, hq, d = q.shape if q.dim() == 3 else (0, 0, 0)
    qs = _rows("q", q, None, d, dev)
    ks = _rows("k", k, None, d, dev, tokens)
    hk, rot = k.shape[1], 2 * inv_freq.shape[0]
    wq = _vector("q_weight", q_weight, q.dtype, dev, d) if q_weight is not None else 0
    wk = _vector("k_weight", k_weight, q.dtype, dev, d) if k_weight is not None else 0
    pos = _vector("positions", positions, torch.int32, dev, tokens)
    freq = _vector("inv_freq", inv_freq, torch.float64, dev, rot // 2)
    with torch.cuda.device(dev):
        qo, ko = q.new_empty((tokens, hq, d)), k.new_empty((tokens, hk, d))
        dg_qk_norm_rope(tokens, hq, hk, d, rot, interleaved, dt, q.data_ptr(), *qs, k.data_ptr(), *ks,
                        wq, wk, weight_offset, eps, pos, freq, qo.data_ptr(), ko.data_ptr(),
                        _stream(dev))
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
        n = page_table.shape[0]
        _vector("first", first, torch.int32, dev, n + 1)
        _vector("past", past, torch.int32, dev, n)
        self.page_table, self.first, self.past, self.tokens, self.device = page_table, first, past, int(tokens), dev
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
        self.k, self.v, self.k_exp, self.v_exp, self.device = k, v, k_exp, v_exp, dev
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
        """Raise DgError if a call met a bad page or a wait ran out (synchronises)."""
        code = int(self.status.item())
        if code:
            raise DgError(code, "a cache call met a page or position outside the cache, or a wait ran out")

    def _batch(self, batch):
        if batch.device != self.device:
            raise ValueError(f"the batch is on {batch.device}, the cache on {self.device}")

    def write(self, k, v, batch: KVBatch) -> None:
        """Write k, v [tokens, kv_heads, head_dim] (bf16 or fp32) at the batch's positions."""
        self._batch(batch)
        c = self.c
        dt = _dtype(k)
        if v.dtype != k.dtype:
            raise ValueError("k and v must have one dtype")
        ks = _rows("k", k, c.kv_heads, c.head_dim, self.device, batch.tokens)
        vs = _rows("v", v, c.kv_heads, c.head_dim, self.device, batch.tokens)
        with torch.cuda.device(self.device):
            dg_cache_write(c, batch.c, dt, k.data_ptr(), *ks, v.data_ptr(), *vs, _stream(self.device))

    def read(self, batch: KVBatch, dtype=torch.bfloat16, out=None):
        """The batch's rows as (k, v) [tokens, kv_heads, head_dim]; padding rows are not written."""
        self._batch(batch)
        c = self.c
        dt = _dtype(dtype)
        with torch.cuda.device(self.device):
            if out is None:
                shape = (batch.tokens, c.kv_heads, c.head_dim)
                out = tuple(torch.empty(shape, dtype=dtype, device=self.device) for _ in "kv")
            for t in out:
                _rows("out", t, c.kv_heads, c.head_dim, self.device, batch.tokens)
                if t.dtype != dtype or not t.is_contiguous():
                    raise ValueError(f"out must be contiguous {dtype}")
            dg_cache_read(c, batch.c, dt, out[0].data_ptr(), out[1].data_ptr(), _stream(self.device))
        return out

    def attend(self, q, batch: KVBatch, mask: int, *, tree=None, scale: float | None = None, out=None,
               lse=None):
        """Attention of q [tokens, q_heads, head_dim] (bf16) over the cache; returns (out, lse).

        mask: DG_MASK_FULL, DG_MASK_CAUSAL, or DG_MASK_TREE with tree int32 [tokens, words] (bit j of
        a row: this token sees new token j of its sequence). scale defaults to head_dim ** -0.5.
        The keys and values of the new tokens are in the cache already (write). out and lse may be
        given; padding rows are not written.
        """
        self._batch(batch)
        c, dev = self.c, self.device
        if q.dtype != torch.bfloat16:
            raise ValueError("q must be bfloat16")
        qs = _rows("q", q, None, c.head_dim, dev, batch.tokens)
        hq, words, tree_ptr = q.shape[1], 0, 0
        if mask == DG_MASK_TREE:
            if tree is None or tree.dtype != torch.int32 or tree.device != dev or tree.dim() != 2 \
                    or tree.shape[0] != batch.tokens or not tree.is_contiguous():
                raise ValueError(f"tree must be a contiguous int32 tensor [{batch.tokens}, words] on {dev}")
            words, tree_ptr = tree.shape[1], tree.data_ptr()
        elif tree is not None:
            raise ValueError("tree goes with DG_MASK_TREE")
        with torch.cuda.device(dev):
            if out is None:
                out = torch.empty((batch.tokens, hq, c.head_dim), dtype=torch.bfloat16, device=dev)
            if lse is None:
                lse = torch.empty((batch.tokens, hq), dtype=torch.float32, device=dev)
            if out.dtype != torch.bfloat16 or out.shape != q.shape or not out.is_contiguous() \
                    or lse.dtype != torch.float32 or lse.shape != q.shape[:2] or not lse.is_contiguous() \
                    or out.device != dev or lse.device != dev:
                raise ValueError("out must be contiguous bfloat16 of q's shape, lse float32 [tokens, q_heads]")
            n = dg_cache_attention_scratch_bytes(c, batch.c, hq)
            scratch = torch.empty(n, dtype=torch.uint8, device=dev)
            dg_cache_attention(c, batch.c, hq, q.data_ptr(), *qs,
                               c.head_dim ** -0.5 if scale is None else scale, mask, tree_ptr, words,
                               out.data_ptr(), lse.data_ptr(), scratch.data_ptr(), n, _stream(dev))
        return out, lse
