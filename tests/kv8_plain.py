"""Plain 64-bit forms of the 8-bit paged cache's operators, for the tests: loops over
requests, blocks and heads, from the definitions in include/gqa_attn.h."""
import math

import numpy as np
import torch

BF16_MAX = float(torch.finfo(torch.bfloat16).max)


def e4m3_values():
    """The 256 codes' values in float64 (NaN at 0x7f and 0xff), from the format."""
    t = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        t[c] = math.nan if (c & 0x7f) == 0x7f else (-v if s else v)
    return t


VALUES = e4m3_values()
_POS = VALUES[:0x7f]  # ascending


def e4m3_encode(x):
    """Codes of float64 x: nearest, ties to the even code, saturating, NaN to a NaN code."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    a0 = np.where(np.isnan(a), 0.0, a)
    hi = np.clip(np.searchsorted(_POS, a0), 0, 0x7e)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = a0 - _POS[lo], _POS[hi] - a0
    c = np.where((dlo < dhi) | ((dlo == dhi) & (lo % 2 == 0)), lo, hi)
    c = np.where(a0 == _POS[hi], hi, c)
    c = np.where(np.isnan(x), 0x7f, c).astype(np.uint8)
    return (c | (np.signbit(x).astype(np.uint8) << 7)).astype(np.uint8)


def pow2_scale(a):
    """The smallest power of two s >= 2^-126 with a <= 448 s."""
    if a == 0:
        return 2.0 ** -126
    e = math.frexp(a)[1] - 10
    while a > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** max(e, -126)


def tables(cached, new, free, start, table, page, max_tokens):
    """(block_table, slot_map, seqlens_k, cu_q, cu_k, free_end) as Python lists."""
    table = [list(r) for r in table]
    slot, lens, cu_q, cu_k, f = [], [], [0], [0], start
    for b, (c, n) in enumerate(zip(cached, new)):
        for p in range(-(-c // page), -(-(c + n) // page)):
            table[b][p] = free[f] if f < len(free) else -1
            f += 1
        for pos in range(c, c + n):
            pg = table[b][pos // page]
            slot.append(pg * page + pos % page if pg >= 0 else -1)
        lens.append(c + n)
        cu_q.append(cu_q[-1] + n)
        cu_k.append(cu_k[-1] + c + n)
    slot = (slot + [-1] * max_tokens)[:max_tokens]
    return table, slot, lens, cu_q, cu_k, f


def append(x, slots, codes, scale, block):
    """x [T, H, D] float64, slots list, codes uint8 [slots, H, D], scale float64 [blocks, H];
    returns the updated (codes, scale)."""
    codes, scale = codes.copy(), scale.copy()
    H = x.shape[1]
    t = 0
    while t < len(slots):
        if slots[t] < 0 or slots[t] >= len(codes):
            t += 1
            continue
        blk, t1 = slots[t] // block, t
        while t1 < len(slots) and slots[t1] >= 0 and slots[t1] // block == blk:
            t1 += 1
        mine = {slots[i] % block: i for i in range(t, t1)}
        for h in range(H):
            rows = np.minimum(np.abs(x[t:t1, h]), BF16_MAX)
            s = pow2_scale(np.nanmax(rows) if not np.all(np.isnan(rows)) else 0.0)
            old = scale[blk, h]
            if 0 not in mine and math.isfinite(old) and old > 0:
                m, e = math.frexp(old)
                s = max(s, 2.0 ** min(max(e - 1 if m == 0.5 else e, -126), 127))
                if s != old:
                    for i in range(block):
                        if i not in mine:
                            c = codes[blk * block + i, h]
                            codes[blk * block + i, h] = e4m3_encode(VALUES[c] * (old / s))
            scale[blk, h] = s
            for i, src in mine.items():
                codes[blk * block + i, h] = e4m3_encode(x[src, h] / s)
        t = t1
    return codes, scale


def gather(codes, scale, table, length, page, block):
    """float64 values [length, H, D] of one sequence (table: its row)."""
    pos = np.arange(length)
    slot = np.asarray(table, dtype=np.int64)[pos // page] * page + pos % page if length else pos
    return VALUES[codes[slot]] * scale[slot // block][:, :, None]


def coarse(codes, scale, table, length, page, block, tile=128):
    """|code| times the largest scale of its tile of keys, [length, H, D]: what a weight's
    absolute error is multiplied with (see check_decode)."""
    pos = np.arange(length)
    slot = np.asarray(table, dtype=np.int64)[pos // page] * page + pos % page if length else pos
    s = scale[slot // block]
    top = np.stack([s[t // tile * tile:t // tile * tile + tile].max(0) for t in pos]) \
        if length else s
    return np.abs(VALUES[codes[slot]]) * top[:, :, None]


def decode(q, k, v, n, scale, window, G, v_coarse):
    """One sequence: q [n, Hq, D], k and v [L, Hkv, D] float64.  Returns out, lse, and per
    output the weighted |v| and the largest weight times the sum of v_coarse, and per
    query the largest |q|_inf |k|_1."""
    L, Hq, D = len(k), q.shape[1], q.shape[2]
    out, absout, floor = (np.zeros((n, Hq, D)) for _ in range(3))
    lse, norm = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    for i in range(n):
        hi = max(L - n + i + 1, 0)
        lo = max(hi - window, 0) if window else 0
        if hi <= lo:
            continue
        for h in range(Hq):
            kk, vv = k[lo:hi, h // G], v[lo:hi, h // G]
            s = scale * (kk @ q[i, h])
            m = s.max()
            p = np.exp(s - m)
            lse[i, h] = m + math.log(p.sum())
            p /= p.sum()
            out[i, h] = p @ vv
            absout[i, h] = p @ np.abs(vv)
            floor[i, h] = p.max() * v_coarse[lo:hi, h // G].sum(0)
            norm[i, h] = np.abs(q[i, h]).max() * np.abs(kk).sum(1).max()
    return out, lse, absout, floor, norm


def check_decode(out, lse, ref, scale):
    """The bounds the kernel's arithmetic gives.

    Logits: q enters as two e4m3 terms of a power-of-two scale, off by at most 2^-21 of
    the row's largest |q| in each element; the products are exact and their fp32 sum of
    D terms is off by a few 2^-22 of sum |q k|: together within 2^-19 |q|_inf |k|_1 times
    the softmax scale.  L adds fp32 exponentials and a logarithm: 2^-19 of its size or 1.
    Weights: two e4m3 terms of a half step of 2^-4 each, 2^-8 relative, and a logit's
    error moves a weight by as much, its normaliser too.  Small weights: the second term's
    subnormal step is 2^-9 / 32, its half 2^-15, where a weight of 32 stands for the row's
    reference, at most the largest weight: 2^-20 of that, times the code and the largest
    scale of its 128 keys
    (the weight carries its own scale over that).  The output's rounding to bf16: half a
    step, 2^-8 relative, at least half a subnormal.  fp32 sums of the weights: 2^-16 of
    sum p |v|.
    """
    o_ref, l_ref, a_ref, floor, norm = ref
    out, lse = np.asarray(out, np.float64), np.asarray(lse, np.float64)
    ds = scale * norm * 2.0 ** -19
    dead = np.isneginf(l_ref)
    assert np.array_equal(np.isneginf(lse), dead)
    lerr = np.abs(np.where(dead, 0, lse) - np.where(dead, 0, l_ref))
    lbar = ds + 2.0 ** -19 * np.maximum(1, np.abs(np.where(dead, 0, l_ref)))
    assert np.all(lerr <= lbar), (lerr - lbar).max()
    err = np.abs(out - o_ref)
    bar = (2.0 ** -8 + 2.0 ** -16 + 3 * ds[..., None]) * a_ref + \
        2.0 ** -8 * np.abs(o_ref) * 1.01 + 2.0 ** -20 * floor + 2.0 ** -134
    assert np.all(np.isfinite(out))
    assert np.all(err <= bar), (err / np.maximum(bar, 1e-300)).max()
    return ((err / np.maximum(bar, 1e-300)).max(initial=0.0), (lerr / lbar).max(initial=0.0))
