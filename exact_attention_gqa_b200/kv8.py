"""The 8-bit paged KV cache with block scales: torch front end of its entry points.

A serving step, none of which waits for the host:

    t = gqa_attn_kv_tables(cached_lens, new_lens, free_pages, block_table,
                           page_size=64, max_tokens=T)
    gqa_attn_kv8_append(k, v, t.slot_map, k8, v8, k_scale, v_scale)
    out, lse = gqa_attn_kv8_decode(q, k8, v8, k_scale, v_scale, block_table, t.seqlens_k)

The cache is a pool of pages: k8, v8 [num_pages, page_size, Hkv, D] (float8_e4m3fn or uint8
codes) and k_scale, v_scale fp32 [num_pages, page_size / scale_block, Hkv]; a stored value
is code * scale.  Outputs and workspaces come from torch's allocator on the current stream,
one for each call.
"""
from __future__ import annotations

import math

from . import _capi
from ._capi import GqaError

__all__ = ["KvTables", "gqa_attn_kv_tables", "gqa_attn_kv8_append", "gqa_attn_kv8_gather",
           "gqa_attn_kv8_decode"]


class KvTables:
    """One step's device tables (gqa_attn_kv_tables), all int32: slot_map [max_tokens],
    seqlens_k [B], cu_seqlens_q and cu_seqlens_k [B + 1], free_end [1]."""

    def __init__(self, slot_map, seqlens_k, cu_seqlens_q, cu_seqlens_k, free_end):
        self.slot_map, self.seqlens_k = slot_map, seqlens_k
        self.cu_seqlens_q, self.cu_seqlens_k = cu_seqlens_q, cu_seqlens_k
        self.free_end = free_end


def _check(device, **tensors):
    for name, t in tensors.items():
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
        if t.device != device:
            raise ValueError(f"{name} must be on the same device as the other tensors")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _int32(torch, **tensors):
    for name, t in tensors.items():
        if t.dtype != torch.int32:
            raise ValueError(f"{name} must be int32")


def _call(torch, name, device, *args):
    """The C entry point on the current stream of `device`, which is made current."""
    stream = torch.cuda.current_stream(device).cuda_stream
    fn = getattr(_capi.load(), name)
    if device.index == torch.cuda.current_device():
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, stream)
    if rc != 0:
        raise GqaError(name, rc)


def _pool(torch, k8, v8, k_scale, v_scale):
    """(num_pages, page_size, scale_block, Hkv, D) of a cache."""
    codes = (torch.uint8, torch.float8_e4m3fn)
    if k8.dtype not in codes or v8.dtype not in codes:
        raise ValueError("k8 and v8 must hold e4m3 codes (uint8 or float8_e4m3fn)")
    if k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32:
        raise ValueError("k_scale and v_scale must be fp32")
    if k8.dim() != 4 or v8.shape != k8.shape:
        raise ValueError("k8 and v8 are [num_pages, page_size, Hkv, D] and alike")
    pages, page, Hkv, D = k8.shape
    if k_scale.dim() != 3 or v_scale.shape != k_scale.shape or k_scale.shape[0] != pages or \
            k_scale.shape[2] != Hkv or k_scale.shape[1] < 1 or page % k_scale.shape[1]:
        raise ValueError("k_scale and v_scale are [num_pages, page_size / scale_block, Hkv]")
    _check(k8.device, k8=k8, v8=v8, k_scale=k_scale, v_scale=v_scale)
    return pages, page, page // k_scale.shape[1], Hkv, D


def _table(torch, block_table, B, device):
    _check(device, block_table=block_table)
    _int32(torch, block_table=block_table)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_pages]")


def gqa_attn_kv_tables(cached_lens, new_lens, free_pages, block_table, *, page_size: int,
                       max_tokens: int, free_start=None) -> KvTables:
    """Pages, slots and prefix sums of one step from the requests' lengths.

    cached_lens, new_lens int32 [B]: tokens in the cache and tokens to come; free_pages
    int32 [n]: pages to hand out, from entry free_start (int32 [1] on the GPU; None: 0);
    block_table int32 [B, max_pages]: each request's row is completed in place with the
    pages of its new tokens.  max_tokens: the slot map's length, at least the number of
    new tokens (slots past them are -1).  Returns KvTables; its free_end is the next
    step's free_start."""
    import torch

    device = block_table.device
    if cached_lens.dim() != 1 or new_lens.shape != cached_lens.shape or free_pages.dim() != 1:
        raise ValueError("cached_lens and new_lens are [B], free_pages is [n]")
    B = cached_lens.shape[0]
    _table(torch, block_table, B, device)
    _check(device, cached_lens=cached_lens, new_lens=new_lens, free_pages=free_pages)
    _int32(torch, cached_lens=cached_lens, new_lens=new_lens, free_pages=free_pages)
    if free_start is not None:
        _check(device, free_start=free_start)
        _int32(torch, free_start=free_start)
        if free_start.numel() != 1:
            raise ValueError("free_start must hold one number")
    if not 0 <= max_tokens < 2 ** 31:
        raise ValueError("max_tokens must be in [0, 2^31)")
    # one allocation, cut into the five tables
    buf = torch.empty(max_tokens + 3 * B + 3, dtype=torch.int32, device=device)
    t = KvTables(*buf.split([max_tokens, B, B + 1, B + 1, 1]))
    p = buf.data_ptr()
    at = [p, p + 4 * max_tokens]
    at += [at[1] + 4 * B]
    at += [at[2] + 4 * (B + 1)]
    at += [at[3] + 4 * (B + 1)]
    _call(torch, "gqa_attn_kv_tables", device, cached_lens.data_ptr(), new_lens.data_ptr(),
          free_pages.data_ptr(), None if free_start is None else free_start.data_ptr(),
          block_table.data_ptr(), *at, B, free_pages.shape[0], block_table.shape[1],
          page_size, max_tokens)
    return t


def gqa_attn_kv8_append(k, v, slot_map, k8, v8, k_scale, v_scale) -> None:
    """Write new tokens' keys and values into the cache, in place (gqa_attn_kv8_append).

    k, v bf16 [T, Hkv, D] (a view whose heads are contiguous will do, as a slice of a
    fused projection); slot_map int32 [T] as gqa_attn_kv_tables made it, -1 for rows to
    leave out.  Codes and scales of every scale block that receives tokens are updated."""
    import torch

    pages, page, block, Hkv, D = _pool(torch, k8, v8, k_scale, v_scale)
    if k.dim() != 3 or v.shape != k.shape or k.shape[1:] != (Hkv, D):
        raise ValueError("k and v are [T, Hkv, D], with the cache's heads")
    T = k.shape[0]
    if slot_map.shape != (T,):
        raise ValueError("slot_map must be [T]")
    for name, t in (("k", k), ("v", v)):
        if not t.is_cuda or t.device != k8.device:
            raise ValueError(f"{name} must be a CUDA tensor on the cache's device")
        if t.dtype != torch.bfloat16:
            raise ValueError(f"{name} must be bf16")
        if t.stride(2) != 1 or (Hkv > 1 and t.stride(1) != D):
            raise ValueError(f"the heads of a token of {name} must be contiguous")
    _check(k8.device, slot_map=slot_map)
    _int32(torch, slot_map=slot_map)
    row = Hkv * D  # of one token alone a view's stride says nothing
    _call(torch, "gqa_attn_kv8_append", k8.device, k.data_ptr(), v.data_ptr(),
          slot_map.data_ptr(), k8.data_ptr(), v8.data_ptr(), k_scale.data_ptr(),
          v_scale.data_ptr(), T, Hkv, D, k.stride(0) if T > 1 else row,
          v.stride(0) if T > 1 else row, pages, page, block)


def gqa_attn_kv8_gather(k8, v8, k_scale, v_scale, block_table, cu_seqlens_k, *, total: int,
                        k=None, v=None):
    """The cache's values as packed bf16 rows k, v [total, Hkv, D] (gqa_attn_kv8_gather):
    row cu_seqlens_k[b] + j is position j of sequence b.  cu_seqlens_k int32 [B + 1] on the
    GPU; total: its last entry, or more (rows past it stay as they are)."""
    import torch

    pages, page, block, Hkv, D = _pool(torch, k8, v8, k_scale, v_scale)
    device = k8.device
    if cu_seqlens_k.dim() != 1 or cu_seqlens_k.shape[0] < 1:
        raise ValueError("cu_seqlens_k must be [B + 1]")
    B = cu_seqlens_k.shape[0] - 1
    _table(torch, block_table, B, device)
    _check(device, cu_seqlens_k=cu_seqlens_k)
    _int32(torch, cu_seqlens_k=cu_seqlens_k)
    if not 0 <= total < 2 ** 31:
        raise ValueError("total must be in [0, 2^31)")
    out = []
    for name, t in (("k", k), ("v", v)):
        if t is None:
            t = torch.empty((total, Hkv, D), dtype=torch.bfloat16, device=device)
        else:
            _check(device, **{name: t})
            if t.dtype != torch.bfloat16 or t.shape != (total, Hkv, D):
                raise ValueError(f"{name} must be bf16 [total, Hkv, D]")
        out.append(t)
    _call(torch, "gqa_attn_kv8_gather", device, k8.data_ptr(), v8.data_ptr(),
          k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(),
          cu_seqlens_k.data_ptr(), out[0].data_ptr(), out[1].data_ptr(), B, total, Hkv, D,
          pages, page, block_table.shape[1], block)
    return out[0], out[1]


def gqa_attn_kv8_decode(q, k8, v8, k_scale, v_scale, block_table, seqlens_k, *,
                        cu_seqlens_q=None, max_seqlen_q: int | None = None, window: int = 0,
                        scale: float | None = None, out=None, lse=None):
    """Attention of each sequence's newest positions over the cache (gqa_attn_kv8_decode).

    q bf16 [B, Sq, Hq, D]: the last Sq positions of each sequence (1: decode; more:
    drafted tokens, causal among themselves), their keys and values being in the cache.
    Or packed q [total_q, Hq, D] with cu_seqlens_q int32 [B + 1] and max_seqlen_q, the
    most queries of one sequence.  block_table int32 [B, max_pages], seqlens_k int32 [B].
    window > 0: each query sees its `window` most recent keys.
    Returns (out like q, lse fp32 [B, Hq, Sq], or packed [Hq, total_q])."""
    import torch

    pages, page, block, Hkv, D = _pool(torch, k8, v8, k_scale, v_scale)
    device = k8.device
    if q.dtype != torch.bfloat16:
        raise ValueError("q must be bf16")
    packed = cu_seqlens_q is not None
    if packed:
        if q.dim() != 3 or max_seqlen_q is None:
            raise ValueError("packed q is [total_q, Hq, D], with max_seqlen_q")
        if cu_seqlens_q.dim() != 1 or cu_seqlens_q.shape[0] < 1:
            raise ValueError("cu_seqlens_q must be [B + 1]")
        _check(device, cu_seqlens_q=cu_seqlens_q)
        _int32(torch, cu_seqlens_q=cu_seqlens_q)
        B, Sq, total_q, Hq = cu_seqlens_q.shape[0] - 1, int(max_seqlen_q), q.shape[0], q.shape[1]
        lse_shape = (Hq, total_q)
    else:
        if q.dim() != 4:
            raise ValueError("q is [B, Sq, Hq, D]")
        B, Sq, Hq, _ = q.shape
        total_q = B * Sq
        lse_shape = (B, Hq, Sq)
    if q.shape[-1] != D:
        raise ValueError("q's head dimension must be the cache's")
    _check(device, q=q, seqlens_k=seqlens_k)
    _table(torch, block_table, B, device)
    _int32(torch, seqlens_k=seqlens_k)
    if seqlens_k.shape != (B,):
        raise ValueError("seqlens_k must be [B]")
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(lse_shape, dtype=torch.float32, device=device)
    _check(device, out=out, lse=lse)
    if out.shape != q.shape or out.dtype != q.dtype or lse.shape != lse_shape or \
            lse.dtype != torch.float32:
        raise ValueError(f"out must be like q and lse fp32 {lse_shape}")
    need = _capi.load().gqa_attn_kv8_decode_workspace_bytes(B, Sq, Hq, Hkv, D)
    ws = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _call(torch, "gqa_attn_kv8_decode", device, q.data_ptr(), k8.data_ptr(), v8.data_ptr(),
          k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(), seqlens_k.data_ptr(),
          cu_seqlens_q.data_ptr() if packed else None, out.data_ptr(), lse.data_ptr(),
          ws.data_ptr() if need else None, need, B, Sq, total_q, Hq, Hkv, D, pages, page,
          block_table.shape[1], block,
          1.0 / math.sqrt(D) if scale is None else float(scale),
          min(int(window), 2 ** 31 - 1))
    return out, lse
