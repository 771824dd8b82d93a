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


# The checks below run before every launch of a few microseconds, so each looks at a tensor
# as few times as it can and words its refusal only when there is one.
def _check(dev, dtype, **tensors):
    """Contiguous tensors of one type on the GPU of index dev."""
    for name, t in tensors.items():
        if t.get_device() != dev or t.dtype is not dtype or not t.is_contiguous():
            _refuse(dev, dtype, name, t)


def _refuse(dev, dtype, name, t):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the same device as the other tensors")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}")
    raise ValueError(f"{name} must be contiguous")


def _check_int(**numbers):
    """Of 31 bits: ctypes would cut a larger one down to 32 bits without a word."""
    for name, x in numbers.items():
        if not 0 <= x < 2 ** 31:
            raise ValueError(f"{name} must be in [0, 2^31)")


def _call(torch, name, dev, *args):
    """The C entry point on the current stream of GPU dev, which is made current."""
    fn = getattr(_capi.load(), name)
    if dev == torch.cuda.current_device():
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if rc != 0:
        raise GqaError(name, rc)


def _pool(torch, k8, v8, k_scale, v_scale):
    """(device index, num_pages, page_size, scale_block, Hkv, D) of a cache."""
    kind, shape, scales = k8.dtype, k8.shape, k_scale.shape
    if kind is not torch.float8_e4m3fn and kind is not torch.uint8:
        raise ValueError("k8 and v8 must hold e4m3 codes (uint8 or float8_e4m3fn)")
    if len(shape) != 4 or v8.shape != shape:
        raise ValueError("k8 and v8 are [num_pages, page_size, Hkv, D] and alike")
    pages, page, Hkv, D = shape
    if len(scales) != 3 or v_scale.shape != scales or scales[0] != pages or \
            scales[2] != Hkv or scales[1] < 1 or page % scales[1]:
        raise ValueError("k_scale and v_scale are [num_pages, page_size / scale_block, Hkv]")
    dev = k8.get_device()
    if dev < 0:
        _refuse(dev, kind, "k8", k8)
    _check(dev, kind, k8=k8, v8=v8)
    _check(dev, torch.float32, k_scale=k_scale, v_scale=v_scale)
    return dev, pages, page, page // scales[1], Hkv, D


def _is_table(block_table, B):
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_pages]")
    return block_table.shape[1]


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

    _check_int(max_tokens=max_tokens, page_size=page_size)
    dev, i32 = block_table.get_device(), torch.int32
    if dev < 0:
        _refuse(dev, i32, "block_table", block_table)
    if cached_lens.dim() != 1 or new_lens.shape != cached_lens.shape or free_pages.dim() != 1:
        raise ValueError("cached_lens and new_lens are [B], free_pages is [n]")
    B = cached_lens.shape[0]
    max_pages = _is_table(block_table, B)
    _check(dev, i32, block_table=block_table, cached_lens=cached_lens, new_lens=new_lens,
           free_pages=free_pages)
    if free_start is not None:
        _check(dev, i32, free_start=free_start)
        if free_start.numel() != 1:
            raise ValueError("free_start must hold one number")
    # one allocation, cut into the five tables
    sizes = (max_tokens, B, B + 1, B + 1, 1)
    buf = block_table.new_empty(sum(sizes))
    p, at = buf.data_ptr(), []
    for n in sizes:
        at.append(p)
        p += 4 * n
    _call(torch, "gqa_attn_kv_tables", dev, cached_lens.data_ptr(), new_lens.data_ptr(),
          free_pages.data_ptr(), None if free_start is None else free_start.data_ptr(),
          block_table.data_ptr(), *at, B, free_pages.shape[0], max_pages, page_size,
          max_tokens)
    return KvTables(*buf.split_with_sizes(sizes))


def gqa_attn_kv8_append(k, v, slot_map, k8, v8, k_scale, v_scale) -> None:
    """Write new tokens' keys and values into the cache, in place (gqa_attn_kv8_append).

    k, v bf16 [T, Hkv, D] (a view whose heads are contiguous will do, as a slice of a
    fused projection); slot_map int32 [T] as gqa_attn_kv_tables made it, -1 for rows to
    leave out.  Codes and scales of every scale block that receives tokens are updated."""
    import torch

    dev, pages, page, block, Hkv, D = _pool(torch, k8, v8, k_scale, v_scale)
    if k.dim() != 3 or v.shape != k.shape or k.shape[1:] != (Hkv, D):
        raise ValueError("k and v are [T, Hkv, D], with the cache's heads")
    T, row = k.shape[0], Hkv * D
    if slot_map.shape != (T,):
        raise ValueError("slot_map must be [T]")
    strides = []
    for name, t in (("k", k), ("v", v)):
        if t.get_device() != dev:
            raise ValueError(f"{name} must be a CUDA tensor on the cache's device")
        if t.dtype is not torch.bfloat16:
            raise ValueError(f"{name} must be bf16")
        s0, s1, s2 = t.stride()
        if s2 != 1 or (Hkv > 1 and s1 != D):
            raise ValueError(f"the heads of a token of {name} must be contiguous")
        strides.append(s0 if T > 1 else row)  # of one token alone it says nothing
    _check(dev, torch.int32, slot_map=slot_map)
    _call(torch, "gqa_attn_kv8_append", dev, k.data_ptr(), v.data_ptr(), slot_map.data_ptr(),
          k8.data_ptr(), v8.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), T, Hkv, D,
          strides[0], strides[1], pages, page, block)


def gqa_attn_kv8_gather(k8, v8, k_scale, v_scale, block_table, cu_seqlens_k, *, total: int,
                        k=None, v=None):
    """The cache's values as packed bf16 rows k, v [total, Hkv, D] (gqa_attn_kv8_gather):
    row cu_seqlens_k[b] + j is position j of sequence b.  cu_seqlens_k int32 [B + 1] on the
    GPU; total: its last entry, or more (rows past it stay as they are)."""
    import torch

    _check_int(total=total)
    dev, pages, page, block, Hkv, D = _pool(torch, k8, v8, k_scale, v_scale)
    if cu_seqlens_k.dim() != 1 or cu_seqlens_k.shape[0] < 1:
        raise ValueError("cu_seqlens_k must be [B + 1]")
    B = cu_seqlens_k.shape[0] - 1
    max_pages = _is_table(block_table, B)
    _check(dev, torch.int32, block_table=block_table, cu_seqlens_k=cu_seqlens_k)
    bf16, shape, out = torch.bfloat16, (total, Hkv, D), []
    for name, t in (("k", k), ("v", v)):
        if t is None:
            t = torch.empty(total, Hkv, D, dtype=bf16, device=k8.device)
        else:
            _check(dev, bf16, **{name: t})
            if t.shape != shape:
                raise ValueError(f"{name} must be [total, Hkv, D]")
        out.append(t)
    k, v = out
    _call(torch, "gqa_attn_kv8_gather", dev, k8.data_ptr(), v8.data_ptr(), k_scale.data_ptr(),
          v_scale.data_ptr(), block_table.data_ptr(), cu_seqlens_k.data_ptr(), k.data_ptr(),
          v.data_ptr(), B, total, Hkv, D, pages, page, max_pages, block)
    return k, v


_ws_bytes = {}  # workspace size of each problem shape seen


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

    if max_seqlen_q is not None:
        _check_int(max_seqlen_q=max_seqlen_q)
    dev, pages, page, block, Hkv, D = _pool(torch, k8, v8, k_scale, v_scale)
    i32 = torch.int32
    _check(dev, torch.bfloat16, q=q)
    shape = q.shape
    if cu_seqlens_q is not None:
        if len(shape) != 3 or max_seqlen_q is None:
            raise ValueError("packed q is [total_q, Hq, D], with max_seqlen_q")
        if cu_seqlens_q.dim() != 1 or cu_seqlens_q.shape[0] < 1:
            raise ValueError("cu_seqlens_q must be [B + 1]")
        _check(dev, i32, cu_seqlens_q=cu_seqlens_q)
        B, Sq, total_q, Hq = cu_seqlens_q.shape[0] - 1, int(max_seqlen_q), shape[0], shape[1]
        lse_shape = (Hq, total_q)
    else:
        if len(shape) != 4:
            raise ValueError("q is [B, Sq, Hq, D]")
        B, Sq, Hq, _ = shape
        total_q = B * Sq
        lse_shape = (B, Hq, Sq)
    if shape[-1] != D:
        raise ValueError("q's head dimension must be the cache's")
    max_pages = _is_table(block_table, B)
    _check(dev, i32, block_table=block_table, seqlens_k=seqlens_k)
    if seqlens_k.shape != (B,):
        raise ValueError("seqlens_k must be [B]")
    if out is None:
        out = torch.empty_like(q)
    else:
        _check(dev, torch.bfloat16, out=out)
        if out.shape != shape:
            raise ValueError("out must be shaped like q")
    if lse is None:
        lse = k_scale.new_empty(lse_shape)
    else:
        _check(dev, torch.float32, lse=lse)
        if lse.shape != lse_shape:
            raise ValueError(f"lse must be {lse_shape}")
    key = (B, Sq, Hq, Hkv, D)
    need = _ws_bytes.get(key)
    if need is None:
        need = _ws_bytes[key] = _capi.load().gqa_attn_kv8_decode_workspace_bytes(*key)
    ws = k_scale.new_empty(need // 4)  # of this call alone (the size is a multiple of 16)
    _call(torch, "gqa_attn_kv8_decode", dev, q.data_ptr(), k8.data_ptr(), v8.data_ptr(),
          k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(), seqlens_k.data_ptr(),
          None if cu_seqlens_q is None else cu_seqlens_q.data_ptr(), out.data_ptr(),
          lse.data_ptr(), ws.data_ptr(), need, B, Sq, total_q, Hq, Hkv, D, pages, page,
          max_pages, block, 1.0 / math.sqrt(D) if scale is None else float(scale),
          max(min(int(window), 2 ** 31 - 1), -1))
    return out, lse
