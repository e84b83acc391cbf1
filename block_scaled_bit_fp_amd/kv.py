"""A paged key/value cache held in 4 bits: tables, writes and attention.

    cache = empty_kv_cache(NVFP4, pages, kv_heads, head_dim, page_size=64, k_scale=gk, v_scale=gv)
    batch = kv_plan(past_lens, q_lens, block_table, free_pages, free_begin, tokens, page_size=64)
    kv_append(cache, k, v, batch.slots)          # quantize the new rows into their pages
    out = kv_attention(q, cache, batch)          # [tokens, heads, head_dim] bf16
    past_lens.copy_(batch.next_lens)             # what each request has in the cache now
    free_begin.copy_(batch.state[:1])

One plan serves every layer of a step; each layer has a cache of its own.
"""
from __future__ import annotations

import ctypes as C
import math
from dataclasses import dataclass
from typing import Optional, Tuple, Union

import torch

from . import (AFFINE, GROUP, MXFP4, NVFP4, QTensorDesc, QuantizedTensor, _check, _stream,
               empty_quantized, lib)

PAGE_SIZES = (16, 32, 64, 128, 256)
HEAD_DIMS = (64, 128, 256)


class KvCacheDesc(C.Structure):
    """Mirror of bsfp_kv_cache."""
    _fields_ = [("k", C.POINTER(QTensorDesc)), ("v", C.POINTER(QTensorDesc)),
                ("pages", C.c_int64), ("kv_heads", C.c_int32), ("page_size", C.c_int32)]


@dataclass
class KvCache:
    """One layer's cache: two quantized tensors of [pages * kv_heads * page_size, head_dim]
    (see include/bsfp.h).  dequantize(cache.k) reads it whole."""
    k: QuantizedTensor
    v: QuantizedTensor
    kv_heads: int
    page_size: int

    def __post_init__(self):
        if self.page_size not in PAGE_SIZES:
            raise ValueError(f"page_size={self.page_size} is not one of {PAGE_SIZES}")
        if self.kv_heads < 1 or self.k.rows % (self.kv_heads * self.page_size):
            raise ValueError(f"{self.k.rows} rows are not whole pages of {self.kv_heads} heads x "
                             f"{self.page_size} tokens")
        if (self.k.mode, self.k.rows, self.k.cols) != (self.v.mode, self.v.rows, self.v.cols):
            raise ValueError("K and V differ in format or shape")
        for t in (self.k, self.v):
            g = t.global_scale
            if g is not None and (g.dtype != torch.float32 or g.numel() != 1):
                raise ValueError("a global scale is one fp32 value")
            for buf in (t.codes, t.scales, t.biases, g):
                if buf is not None and buf.device != self.device:
                    raise ValueError(f"the cache's tensors are on {self.device} and {buf.device}")
            G, words = t.group_size, t.cols * t.nbits // 32
            want = [(t.codes, t.rows * words * 4), (t.scales, t.rows * (t.cols // G) *
                                                    (2 if t.mode == AFFINE else 1))]
            if t.mode == AFFINE:
                want.append((t.biases, t.rows * (t.cols // G) * 2))
            for buf, need in want:
                if buf is None or not buf.is_contiguous() or buf.numel() * buf.element_size() != need:
                    raise ValueError("a cache tensor's codes, scales or biases do not fit its shape")

    @property
    def head_dim(self) -> int:
        return self.k.cols

    @property
    def pages(self) -> int:
        return self.k.rows // (self.kv_heads * self.page_size)

    @property
    def device(self) -> torch.device:
        return self.k.codes.device

    def desc(self):
        """The C descriptor, by reference; rebuilt when a field or a tensor's descriptor changed."""
        kd, vd = self.k.desc(), self.v.desc()
        heads, page = self.kv_heads, self.page_size
        cached = self.__dict__.get("_kv_desc")
        if (cached is None or cached[0] is not kd or cached[1] is not vd or cached[2] != heads
                or cached[3] != page):
            self.__post_init__()
            d = KvCacheDesc(C.pointer(kd), C.pointer(vd), self.pages, heads, page)
            self.__dict__["_kv_desc"] = cached = (kd, vd, heads, page, C.byref(d))
        return cached[4]


def empty_kv_cache(mode: int, pages: int, kv_heads: int, head_dim: int, page_size: int = 64,
                   device="cuda", k_scale: Optional[torch.Tensor] = None,
                   v_scale: Optional[torch.Tensor] = None) -> KvCache:
    """A cache of `pages` pages in NVFP4, MXFP4 or AFFINE (group 64).  k_scale and v_scale: the
    NVFP4 global scales (fp32 [1] on the device, e.g. amax/2688 of a calibration run), or None."""
    if mode not in (AFFINE, MXFP4, NVFP4):
        raise ValueError("a cache holds NVFP4, MXFP4 or AFFINE")
    if mode != NVFP4 and (k_scale is not None or v_scale is not None):
        raise ValueError("only NVFP4 tensors have a global scale")
    if head_dim not in HEAD_DIMS:
        raise ValueError(f"head_dim={head_dim} is not one of {HEAD_DIMS}")
    out = []
    for g in (k_scale, v_scale):
        if g is not None and (g.dtype != torch.float32 or g.numel() != 1 or not g.is_cuda):
            raise ValueError("a global scale is one fp32 value on the GPU")
        t = empty_quantized(mode, pages * kv_heads * page_size, head_dim, device, global_scale=False)
        t.global_scale = g
        out.append(t)
    return KvCache(out[0], out[1], kv_heads, page_size)


@dataclass
class KvBatch:
    """The tables of one step.  kv_attention needs the first three (int32, on the GPU)."""
    block_table: torch.Tensor                  # [requests, max_pages]
    kv_lens: torch.Tensor                      # [requests]
    q_starts: torch.Tensor                     # [requests + 1]
    slots: Optional[torch.Tensor] = None       # int64 [tokens]
    positions: Optional[torch.Tensor] = None   # int32 [tokens]
    state: Optional[torch.Tensor] = None       # int32 [2]: next free begin, refused requests
    # int32 [requests]: the next step's past_lens (kv_lens is 0 for a refused request, this is not)
    next_lens: Optional[torch.Tensor] = None


def _vector(t: torch.Tensor, dtype, shape, what: str, device) -> torch.Tensor:
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{what} must be {dtype} of shape {tuple(shape)}, got {t.dtype} "
                         f"{tuple(t.shape)}")
    if not t.is_cuda or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous tensor on the call's GPU ({device})")
    return t


def kv_plan(past_lens: torch.Tensor, q_lens: torch.Tensor, block_table: torch.Tensor,
            free_pages: torch.Tensor, free_begin: torch.Tensor, tokens: int,
            page_size: int = 64, out: Optional[KvBatch] = None) -> KvBatch:
    """The step's tables from the request lengths, in one launch (bsfp_kv_plan): new pages from
    free_pages[free_begin:] into block_table (in place), and the kv_lens, q_starts, slots,
    positions, state and next_lens of the returned KvBatch.  `tokens` bounds the sum of q_lens;
    rows past the sum get slot and position -1.  The next step's past_lens is next_lens, its
    free_begin state[:1].  out: a KvBatch of earlier outputs to write into; they must not be this
    call's inputs (out.next_lens is not past_lens: copy it there after the call)."""
    if past_lens.dim() != 1:
        raise ValueError("past_lens must be one-dimensional")
    R, device = past_lens.shape[0], past_lens.device
    i32 = torch.int32
    _vector(past_lens, i32, (R,), "past_lens", device)
    _vector(q_lens, i32, (R,), "q_lens", device)
    if block_table.dim() != 2 or block_table.shape[0] != R:
        raise ValueError(f"block_table must have {R} rows")
    _vector(block_table, i32, block_table.shape, "block_table", device)
    _vector(free_pages, i32, (free_pages.numel(),), "free_pages", device)
    _vector(free_begin, i32, (1,), "free_begin", device)
    if tokens < 0:
        raise ValueError("tokens must not be negative")
    if out is None:
        lens, starts, positions, state, after = torch.split_with_sizes(
            past_lens.new_empty(3 * R + tokens + 3), (R, R + 1, tokens, 2, R))
        out = KvBatch(block_table, lens, starts, past_lens.new_empty(tokens, dtype=torch.int64),
                      positions, state, after)
    else:
        if out.block_table is not block_table:
            raise ValueError("out belongs to another block_table")
        _vector(out.kv_lens, i32, (R,), "out.kv_lens", device)
        _vector(out.q_starts, i32, (R + 1,), "out.q_starts", device)
        _vector(out.slots, torch.int64, (tokens,), "out.slots", device)
        _vector(out.positions, i32, (tokens,), "out.positions", device)
        _vector(out.state, i32, (2,), "out.state", device)
        if out.next_lens is None:
            out.next_lens = past_lens.new_empty(R)
        _vector(out.next_lens, i32, (R,), "out.next_lens", device)
    _check(lib().bsfp_kv_plan_carry(past_lens.data_ptr(), q_lens.data_ptr(), R, page_size,
                                    block_table.data_ptr(), block_table.shape[1],
                                    free_pages.data_ptr(), free_pages.numel(),
                                    free_begin.data_ptr(), tokens, out.kv_lens.data_ptr(),
                                    out.q_starts.data_ptr(), out.slots.data_ptr(),
                                    out.positions.data_ptr(), out.state.data_ptr(),
                                    out.next_lens.data_ptr(), _stream()))
    return out


def _int32(n: int) -> int:
    """A bound on lengths, which are 32-bit: no larger one says more (ctypes would wrap it)."""
    return min(max(n, -1), 0x7fffffff)


def _rows(t: torch.Tensor, heads: Optional[int], cache: KvCache, what: str) -> int:
    """Checks bf16 rows [tokens, heads, head_dim] with contiguous heads and columns; returns the
    token stride in elements."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{what}: expected bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{what}: expected a tensor on the GPU")
    if t.device != cache.device:
        raise ValueError(f"{what} is on {t.device}, the cache on {cache.device}")
    shape, head_dim = t.shape, cache.head_dim
    if len(shape) != 3 or shape[2] != head_dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{what} must be [tokens, {'heads' if heads is None else heads}, "
                         f"{head_dim}], got {tuple(shape)}")
    stride = t.stride()
    if shape[0] and (stride[2] != 1 or (stride[1] != head_dim and shape[1] > 1)):
        raise ValueError(f"{what}: heads and columns must be contiguous")
    return stride[0] if shape[0] > 1 else shape[1] * head_dim


def kv_append(cache: KvCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor) -> None:
    """Quantizes the rows k, v [tokens, kv_heads, head_dim] into the cache at `slots`
    (bsfp_kv_append); rows whose slot is negative are skipped.  k and v may be columns of one
    fused projection's output (any token stride that is a multiple of 8)."""
    ks = _rows(k, cache.kv_heads, cache, "k")
    vs = _rows(v, cache.kv_heads, cache, "v")
    if v.shape[0] != k.shape[0]:
        raise ValueError(f"k has {k.shape[0]} rows, v has {v.shape[0]}")
    _vector(slots, torch.int64, (k.shape[0],), "slots", k.device)
    _check(lib().bsfp_kv_append(k.data_ptr(), ks, v.data_ptr(), vs, k.shape[0], slots.data_ptr(),
                                cache.desc(), _stream()))


def kv_attention_workspace_bytes(tokens: int, heads: int, kv_heads: int, head_dim: int,
                                 requests: int) -> int:
    return int(lib().bsfp_kv_attention_workspace_bytes(tokens, heads, kv_heads, head_dim, requests))


def kv_attention_workspace(tokens: int, heads: int, cache: KvCache, requests: int,
                           max_q: Optional[int] = None) -> torch.Tensor:
    """A workspace for kv_attention calls of at most these sizes, to keep between calls.  With
    max_q it is for calls that give no larger one (a decode step's is far smaller)."""
    rows = tokens if max_q is None else min(tokens, max_q)
    need = kv_attention_workspace_bytes(rows, heads, cache.kv_heads, cache.head_dim, requests)
    return torch.empty(need, dtype=torch.uint8, device=cache.device)


def kv_attention(q: torch.Tensor, cache: KvCache, batch: KvBatch, scale: Optional[float] = None,
                 window: int = 0, max_q: Optional[int] = None,
                 out: Optional[torch.Tensor] = None, return_lse: bool = False,
                 lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
                 ) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
    """Causal attention of the step's queries q [tokens, heads, head_dim] over the cache
    (bsfp_kv_attention).  scale: 1/sqrt(head_dim) by default; window > 0: only that many keys
    up to the row's own; max_q: an upper bound on the batch's q_lens if the host knows one (1 in
    a decode step).  Returns out, or (out, lse) with return_lse."""
    stride = _rows(q, None, cache, "q")
    T, H, D = q.shape
    device = q.device
    table, lens, starts = batch.block_table, batch.kv_lens, batch.q_starts
    R, M = table.shape
    _vector(table, torch.int32, (R, M), "block_table", device)
    _vector(lens, torch.int32, (R,), "kv_lens", device)
    _vector(starts, torch.int32, (R + 1,), "q_starts", device)
    if out is None:
        out = q.new_empty((T, H, D))
    else:
        _vector(out, torch.bfloat16, (T, H, D), "out", device)
    if lse is not None:
        _vector(lse, torch.float32, (T, H), "lse", device)
    elif return_lse:
        lse = q.new_empty((T, H), dtype=torch.float32)
    if workspace is None:
        workspace = kv_attention_workspace(T, H, cache, R, max_q)
    elif not workspace.is_cuda or workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    _check(lib().bsfp_kv_attention(
        q.data_ptr(), stride, T, H, cache.desc(), table.data_ptr(), M, lens.data_ptr(),
        starts.data_ptr(), R, max(T, 1) if max_q is None else _int32(max_q),
        1.0 / math.sqrt(D) if scale is None else scale, _int32(window), out.data_ptr(),
        None if lse is None else lse.data_ptr(), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream()))
    return (out, lse) if return_lse else out
