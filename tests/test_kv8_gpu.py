"""The 8-bit paged cache with block scales on the GPU, against plain 64-bit forms: tables,
append and gather to the bit, decode within the bounds of its arithmetic."""
import math

import numpy as np
import pytest
import torch

import exact_attention_gqa_b200 as G
import kv8_plain as P
from exact_attention_gqa_b200 import build, gqa_attn_get_device_error

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    yield
    torch.cuda.synchronize()
    assert gqa_attn_get_device_error() == 0


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ----------------------------------------------------------------------------- tables
def run_tables(cached, new, page, seed, spare=4, max_pages=None, slack=3, start=0):
    need = [-(-(c + n) // page) for c, n in zip(cached, new)]
    had = [-(-c // page) for c in cached]
    g = torch.Generator().manual_seed(seed)
    perm = torch.randperm(sum(need) + start + max(spare, 0), generator=g).tolist()
    width = max_pages or max(need + [1])
    table, at = [], 0
    for h in had:
        table.append(perm[at:at + h] + [-7] * (width - h))
        at += h
    free = perm[at:]
    if spare < 0:
        free = free[:spare]
    max_tokens = sum(new) + slack
    bt = i32(table).reshape(len(cached), width)
    fs = i32([start]) if start else None
    t = G.gqa_attn_kv_tables(i32(cached), i32(new), i32(free), bt, page_size=page,
                             max_tokens=max_tokens, free_start=fs)
    torch.cuda.synchronize()
    ref = P.tables(cached, new, free, start, table, page, max_tokens)
    got = (bt.tolist(), t.slot_map.tolist(), t.seqlens_k.tolist(), t.cu_seqlens_q.tolist(),
           t.cu_seqlens_k.tolist(), t.free_end.tolist()[0])
    for x, y, what in zip(got, ref, ("table", "slots", "lens", "cu_q", "cu_k", "free_end")):
        assert x == y, what


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("cached,new", [
    ([0], [1]), ([15, 16, 17], [1, 1, 1]), ([0, 5, 0, 300, 31], [0, 0, 0, 0, 0]),
    ([0, 1000, 16, 255, 256], [257, 1, 0, 16, 17]), ([0], [5000]),
])
def test_tables(cached, new, page):
    run_tables(cached, new, page, seed=page)
    run_tables(cached, new, page, seed=page + 1, start=3, max_pages=500)


@pytest.mark.parametrize("B", [511, 512, 513, 2000])
def test_tables_of_many_requests(B):
    rng = np.random.default_rng(B)
    run_tables(rng.integers(0, 100, B).tolist(), rng.integers(0, 40, B).tolist(), 16, seed=B)


def test_tables_largest_batch_and_none():
    run_tables([7] * 16384, [1] * 16384, 16, seed=1)
    run_tables([], [], 16, seed=1, max_pages=1)


def test_tables_report_what_does_not_fit():
    run_tables([16, 16, 3], [20, 1, 100], 16, seed=5, spare=-2)      # two pages short
    assert gqa_attn_get_device_error() == 4
    run_tables([3, 4], [5, 6], 16, seed=6, slack=-2)                 # two slots short
    assert gqa_attn_get_device_error() == 4
    bt = torch.full((2, 2), -1, dtype=torch.int32, device=DEV)       # past the row, negative
    t = G.gqa_attn_kv_tables(i32([0, -5]), i32([40, 3]), i32([9, 8, 7, 6]), bt, page_size=16,
                             max_tokens=50)
    torch.cuda.synchronize()
    assert gqa_attn_get_device_error() == 4
    assert t.seqlens_k.tolist() == [32, 3] and bt.tolist() == [[9, 8], [7, -1]]
    assert t.slot_map.tolist() == list(range(144, 160)) + list(range(128, 144)) + \
        [112, 113, 114] + [-1] * 15


# ----------------------------------------------------------------------------- append
def make_pool(pages, page, block, H, D, seed, garbage=False):
    """Codes (uint8 torch) and fp32 scales; garbage: every code, NaN among them."""
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(0, 256, (pages, page, H, D), generator=g, dtype=torch.int32)
    if not garbage:
        c = torch.where((c & 0x7f) >= 0x78, c & 0x87, c)  # magnitudes below 256
    e = torch.randint(-9, 2, (pages, page // block, H), generator=g)
    return c.to(torch.uint8), torch.exp2(e.float())


def run_append(k, v, slots, page, block, H, D, pages, seed, garbage=False, scales=None,
               k_dev=None, v_dev=None):
    k8, ks = make_pool(pages, page, block, H, D, seed, garbage)
    v8, vs = make_pool(pages, page, block, H, D, seed + 1, garbage)
    if scales is not None:
        ks.copy_(scales), vs.copy_(scales)
    d8 = [t.to(DEV) for t in (k8, v8, ks, vs)]
    G.gqa_attn_kv8_append(k.to(DEV) if k_dev is None else k_dev,
                          v.to(DEV) if v_dev is None else v_dev, i32(slots), *d8)
    torch.cuda.synchronize()
    for x, c0, s0, c1, s1 in ((k, k8, ks, d8[0], d8[2]), (v, v8, vs, d8[1], d8[3])):
        c, s = P.append(x.double().numpy(), slots, c0.numpy().reshape(-1, H, D),
                        s0.double().numpy().reshape(-1, H), block)
        assert np.array_equal(s1.cpu().double().numpy().reshape(-1, H), s, equal_nan=True)
        got = c1.cpu().numpy().reshape(-1, H, D)
        nan = np.isnan(P.VALUES[c])  # a NaN keeps no sign
        assert np.array_equal(np.isnan(P.VALUES[got]), nan)
        assert np.array_equal(got[~nan], c[~nan])


def draw_kv(T, H, D, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    mag = torch.exp(spread * torch.randn(T, H, 1, generator=g))
    return tuple((torch.randn(T, H, D, generator=g) * mag).bfloat16() for _ in range(2))


@pytest.mark.parametrize("H,D", [(8, 128), (3, 64), (1, 128), (1, 64), (12, 64)])
@pytest.mark.parametrize("page,block", [(16, 16), (64, 16), (64, 64), (256, 256), (128, 32)])
def test_append_runs(H, D, page, block):
    # whole blocks, a run into a filled block, one that crosses two, single tokens, gaps
    pages = 6
    n = pages * page
    slots = (list(range(2 * page, 3 * page)) + [-1] + list(range(block // 2, block)) + [-1, -1] +
             list(range(3 * page + block - 3, min(3 * page + block + 5, n))) +
             [5 * page + 7] + [n - 1])
    k, v = draw_kv(len(slots), H, D, seed=page + block + H)
    run_append(k, v, slots, page, block, H, D, pages, seed=H + D)


@pytest.mark.parametrize("T", [1, 2, 33])
def test_append_single_tokens_of_requests(T):
    H, D, page, block = 8, 128, 32, 16
    slots = [i * page + (i * 7) % page for i in range(T)]
    k, v = draw_kv(T, H, D, seed=T)
    run_append(k, v, slots, page, block, H, D, T, seed=T)


def test_append_any_order_within_a_block():
    slots = [35, 33, 47, 32, 40, 7, 3, 12]
    k, v = draw_kv(8, 2, 64, seed=3)
    run_append(k, v, slots, 16, 16, 2, 64, 4, seed=9)


def test_append_over_garbage_scales_and_extreme_values():
    H, D, page, block = 2, 64, 32, 16
    scales = torch.tensor([math.nan, -1.0, 0.0, math.inf, 3.0, 2.0 ** -126, 2.0 ** 127, 0.75])
    scales = scales.view(4, 2, 1).expand(4, 2, 2).contiguous()
    slots = [5, 6, 21, 37, 38, 53, 70, 71, 85, 101, 117]
    k, v = draw_kv(len(slots), H, D, seed=4)
    k[0] = 0
    k[1, 0, 3] = math.inf
    k[2, 0, 5] = -math.inf
    k[3] = math.nan
    k[4, 1, 0] = math.nan
    v[2] = 2.0 ** -130          # subnormal
    v[3] = torch.finfo(torch.bfloat16).max
    v[6, 0] = 448.0             # the border of a scale, and the next value
    v[6, 1] = 450.0
    run_append(k, v, slots, page, block, H, D, 4, seed=11, garbage=True, scales=scales)


def test_append_from_a_slice_of_a_fused_projection():
    Hq, H, D, T = 8, 2, 128, 40
    g = torch.Generator().manual_seed(8)
    qkv = torch.randn(T, Hq + 2 * H, D, generator=g).bfloat16()
    dev = qkv.to(DEV)
    slots = list(range(16, 16 + T))
    run_append(qkv[:, Hq:Hq + H], qkv[:, Hq + H:], slots, 64, 32, H, D, 2, seed=2,
               k_dev=dev[:, Hq:Hq + H], v_dev=dev[:, Hq + H:])


def test_append_reports_slots_outside_the_pool():
    k, v = draw_kv(4, 2, 64, seed=5)
    run_append(k, v, [3, 64, -5, 20], 16, 16, 2, 64, 4, seed=3)
    assert gqa_attn_get_device_error() == 3


def test_append_token_by_token_equals_the_definition_and_keeps_precision():
    """A block filled one token at a time: every step to the bit, and at the end each
    value within half a step of its own size plus the block's subnormal step."""
    H, D, block = 2, 64, 16
    k, v = draw_kv(block, H, D, seed=6, spread=1.0)
    k8 = torch.zeros(1, block, H, D, dtype=torch.uint8, device=DEV)
    v8, ks = k8.clone(), torch.full((1, 1, H), math.nan, device=DEV)
    vs = ks.clone()
    for i in range(block):
        G.gqa_attn_kv8_append(k[i:i + 1].to(DEV), v[i:i + 1].to(DEV), i32([i]), k8, v8, ks, vs)
    got = P.VALUES[k8.cpu().numpy()][0] * ks.cpu().double().numpy()[0, 0][:, None]
    x = k.double().numpy()
    s = ks.cpu().double().numpy()[0, 0][:, None]
    # at most one rounding per growth of the scale below the normal range: 16 half steps
    assert np.all(np.abs(got - x) <= np.abs(x) * 2.0 ** -4 + 16 * s * 2.0 ** -10)


# ----------------------------------------------------------------------------- gather
def build_cache(lens, page, block, H, D, seed, spare=2, garbage_rest=True, max_pages=None):
    """A pool whose pages hold the sequences in shuffled order.  Rows that no sequence
    holds carry every code, NaN among them, and their blocks wild scales; table entries
    past a sequence are -1."""
    used = [-(-int(n) // page) for n in lens]
    pages = sum(used) + spare
    g = torch.Generator().manual_seed(seed)
    perm = torch.randperm(pages, generator=g).tolist()
    k8, ks = make_pool(pages, page, block, H, D, seed)
    v8, vs = make_pool(pages, page, block, H, D, seed + 1)
    ks /= 32  # keys of about unit size
    gk, _ = make_pool(pages, page, block, H, D, seed + 2, garbage=True)
    live = torch.zeros(pages, page, dtype=torch.bool)
    table = torch.full((len(lens), max_pages or max(used + [1])), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        for p in range(used[b]):
            table[b, p] = perm[at]
            live[perm[at], : min(page, n - p * page)] = True
            at += 1
    if garbage_rest:
        k8[~live], v8[~live] = gk[~live], gk[~live]
        dead = ~live.view(pages, page // block, block).any(2)
        ks[dead], vs[dead] = math.nan, math.inf
    return k8, v8, ks, vs, table


def cache_np(k8, v8, ks, vs, H, D):
    return (k8.numpy().reshape(-1, H, D), ks.double().numpy().reshape(-1, H),
            v8.numpy().reshape(-1, H, D), vs.double().numpy().reshape(-1, H))


@pytest.mark.parametrize("H,D", [(8, 128), (1, 64), (3, 64)])
@pytest.mark.parametrize("page,block", [(16, 16), (256, 32), (64, 64)])
def test_gather(H, D, page, block):
    lens = [1, 0, 257, 16, 15, 700]
    cache = build_cache(lens, page, block, H, D, seed=page + D)
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    total = cu[-1] + 5
    out = [torch.full((total, H, D), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    d = [t.to(DEV) for t in cache]
    G.gqa_attn_kv8_gather(*d, i32(cu), total=total, k=out[0], v=out[1])
    torch.cuda.synchronize()
    kc, ks, vc, vs = cache_np(*cache[:4], H, D)
    for o, c, s in ((out[0], kc, ks), (out[1], vc, vs)):
        ref = np.concatenate([P.gather(c, s, cache[4][b].tolist(), n, page, block)
                              for b, n in enumerate(lens)])
        assert torch.equal(o[:cu[-1]].cpu(), torch.from_numpy(ref).bfloat16())
        assert bool((o[cu[-1]:] == 7.0).all())   # rows behind the last sequence


# ----------------------------------------------------------------------------- decode
def run_decode(lens, Hq, H, D, page, block, n=1, window=0, seed=0, cu=None, q_mult=1.5,
               scale=None, cache=None, max_pages=None, free_scales=False, total_extra=0):
    cache = cache or build_cache(lens, page, block, H, D, seed, max_pages=max_pages)
    if free_scales:  # any positive fp32, not only powers of two
        g = torch.Generator().manual_seed(seed + 9)
        for t in cache[2:4]:
            t.mul_(torch.rand(t.shape, generator=g) + 0.5)
    B = len(lens)
    g = torch.Generator().manual_seed(seed + 5)
    scale = scale or 1 / math.sqrt(D)
    d = [t.to(DEV) for t in cache]
    if cu is None:
        q = (q_mult * torch.randn(B, n, Hq, D, generator=g)).bfloat16()
        out, lse = G.gqa_attn_kv8_decode(q.to(DEV), *d, i32(lens), window=window, scale=scale)
        qs = [q[b] for b in range(B)]
        outs = [out[b] for b in range(B)]
        lses = [lse[b].T for b in range(B)]
    else:
        rows = cu[-1] + total_extra
        q = (q_mult * torch.randn(rows, Hq, D, generator=g)).bfloat16()
        out = torch.full_like(q, 5.0, device=DEV)
        lse = torch.full((Hq, rows), 5.0, device=DEV)
        G.gqa_attn_kv8_decode(q.to(DEV), *d, i32(lens), cu_seqlens_q=i32(cu), max_seqlen_q=n,
                              window=window, scale=scale, out=out, lse=lse)
        qs = [q[cu[b]:cu[b + 1]] for b in range(B)]
        outs = [out[cu[b]:cu[b + 1]] for b in range(B)]
        lses = [lse[:, cu[b]:cu[b + 1]].T for b in range(B)]
        assert bool((out[cu[-1]:] == 5.0).all()) and bool((lse[:, cu[-1]:] == 5.0).all())
    torch.cuda.synchronize()
    kc, ks, vc, vs = cache_np(*cache[:4], H, D)
    worst = (0.0, 0.0)
    for b in range(B):
        row = cache[4][b].tolist()
        k = P.gather(kc, ks, row, lens[b], page, block)
        v = P.gather(vc, vs, row, lens[b], page, block)
        coarse = P.coarse(vc, vs, row, lens[b], page, block)
        ref = P.decode(qs[b].double().numpy(), k, v, len(qs[b]), scale, window, Hq // H, coarse)
        got = P.check_decode(outs[b].float().cpu().numpy(), lses[b].cpu().numpy(), ref, scale)
        worst = tuple(max(x, y) for x, y in zip(worst, got))
    print("worst share of the bound: out %.3f, lse %.3f" % worst)


LENS = [1, 0, 127, 128, 129, 1000, 31, 2049]


@pytest.mark.parametrize("Hq,H,D", [(32, 8, 128), (4, 1, 128), (8, 8, 128), (12, 4, 64),
                                    (6, 3, 64), (1, 1, 64), (16, 2, 128), (40, 2, 64),
                                    (71, 1, 128), (64, 1, 64)])
@pytest.mark.parametrize("page,block", [(16, 16), (64, 32), (256, 256)])
def test_decode(Hq, H, D, page, block):
    run_decode(LENS, Hq, H, D, page, block, seed=Hq + page)


@pytest.mark.parametrize("Hq,H,D", [(24, 24, 128), (34, 17, 128), (33, 33, 64), (64, 32, 64),
                                    (20, 20, 64)])
def test_decode_head_counts(Hq, H, D):
    """Head groups that fill teams of 12, 1, 1, 16 and 10 CTAs."""
    run_decode(LENS, Hq, H, D, 32, 16, seed=Hq)


def test_decode_nothing_to_see():
    run_decode([0, 0, 0], 8, 2, 128, 16, 16, seed=1)
    run_decode([0, 0, 0], 4, 2, 64, 16, 16, n=3, seed=1)
    run_decode([2, 0, 1], 8, 2, 128, 16, 16, n=5, seed=1)    # more queries than keys


def test_decode_many_sequences_of_any_length():
    lens = np.random.default_rng(3).integers(0, 400, 77).tolist()
    run_decode(lens, 4, 2, 64, 16, 16, n=2, seed=5)
    run_decode(lens, 8, 2, 128, 16, 16, seed=6)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,window", [(1, 1), (1, 100), (1, 5000), (2, 0), (3, 17), (5, 128),
                                      (8, 0), (20, 0), (40, 300)])
def test_decode_drafted_tokens_and_windows(n, window, D):
    # lengths below n leave the first queries without a key
    run_decode(LENS, 16, 4, D, 32, 16, n=n, window=window, seed=n + window)


def test_decode_packed_queries():
    n = [3, 0, 1, 8, 0, 2, 1, 5]
    cu = np.concatenate([[0], np.cumsum(n)]).tolist()
    run_decode(LENS, 8, 2, 128, 64, 16, n=8, cu=cu, seed=3, total_extra=4)


@pytest.mark.parametrize("B,L", [(1, 1), (1, 40000), (3, 12345), (300, 90)])
def test_decode_split_and_whole_sequences(B, L):
    """Few long sequences (each cut into many parts) and many short ones."""
    run_decode([L] * B, 8, 2, 128, 128, 64, seed=B, max_pages=-(-L // 128) + 3)


def test_decode_free_scales():
    run_decode(LENS, 8, 2, 128, 64, 16, seed=21, free_scales=True)


def test_decode_large_logits():
    run_decode(LENS, 8, 2, 128, 64, 16, seed=22, q_mult=30.0)


def test_decode_wild_scales_of_neighbouring_blocks():
    """A block of zeros (scale 2^-126) beside ordinary ones, and values of 2^60."""
    lens = [300, 64, 17]
    cache = build_cache(lens, 64, 16, 2, 128, seed=30)
    k8, v8, ks, vs, table = cache
    for page in table[0].tolist()[::2]:
        v8[page, 16:32] = 0
        vs[page, 1] = 2.0 ** -126
        k8[page, 16:32] = 0
        ks[page, 1] = 2.0 ** -126
    vs[table[1, 0]] = 2.0 ** 60
    vs[table[2, 0]] = 2.0 ** -100
    run_decode(lens, 8, 2, 128, 64, 16, seed=31, cache=cache)


def check_decode_nan(got, lse, ref, scale):
    """NaN exactly where the formula has it, the rest within check_decode's bounds."""
    assert np.array_equal(np.isnan(got), np.isnan(ref[0]))
    assert np.array_equal(np.isnan(lse), np.isnan(ref[1]))
    clean = [np.where(np.isnan(x), 0.0, x) for x in ref]
    P.check_decode(np.where(np.isnan(got), 0.0, got), np.where(np.isnan(lse), 0.0, lse),
                   clean, scale)


@pytest.mark.parametrize("Hq,H,D", [(2, 2, 64), (4, 4, 64), (8, 4, 64), (12, 3, 64), (16, 2, 64),
                                    (32, 2, 64), (32, 8, 128)])
def test_decode_nan_key_of_one_head(Hq, H, D):
    """It spoils the rows of that head only, at D = 64 not its neighbour's either."""
    page, block, lens = 16, 16, [300, 129, 5]
    cache = build_cache(lens, page, block, H, D, 5)
    kf, table = cache[0].view(-1, H, D), cache[4]
    for b, pos, h in ((0, 299, H - 1), (1, 0, 0), (2, 4, H // 2)):
        kf[table[b, pos // page].item() * page + pos % page, h, 3] = 0x7f
    q = torch.randn(3, 1, Hq, D, generator=torch.Generator().manual_seed(2)).bfloat16()
    out, lse = G.gqa_attn_kv8_decode(q.to(DEV), *[t.to(DEV) for t in cache], i32(lens))
    torch.cuda.synchronize()
    kc, ks, vc, vs = cache_np(*cache[:4], H, D)
    for b, n in enumerate(lens):
        row = table[b].tolist()
        k, v = P.gather(kc, ks, row, n, page, block), P.gather(vc, vs, row, n, page, block)
        coarse = P.coarse(vc, vs, row, n, page, block)
        ref = P.decode(q[b].double().numpy(), k, v, 1, 1 / math.sqrt(D), 0, Hq // H, coarse)
        check_decode_nan(out[b].float().cpu().numpy(), lse[b].T.cpu().numpy(), ref,
                         1 / math.sqrt(D))


@pytest.mark.parametrize("Hq,H,D", [(8, 2, 128), (4, 4, 64), (8, 4, 64), (12, 3, 64), (16, 2, 64),
                                    (32, 2, 64), (32, 1, 128)])
@pytest.mark.parametrize("n,window", [(1, 0), (1, 100), (4, 0), (5, 130)])
def test_decode_nan_codes_reach_only_who_sees_them(Hq, H, D, n, window):
    """NaN in keys of one head, and in single dimensions of values: at keys that all queries
    see, only some do, or none (before a window, and not yet for the earlier drafts)."""
    page, block, lens = 32, 16, [700, 300, 5, 129]
    cache = build_cache(lens, page, block, H, D, 3)
    k8, v8, ks, vs, table = cache
    def at(b, pos):
        return table[b, pos // page].item() * page + pos % page
    kf, vf = k8.view(-1, H, D), v8.view(-1, H, D)   # views of the pool
    nan = 0x7f
    kf[at(0, 699), H - 1, 5] = nan                # the newest key, one head
    vf[at(0, 698), 0, 7] = nan                    # a value the first drafts do not see
    vf[at(0, 699), H - 1, D - 1] = 0xff
    vf[at(1, 299 - n), 0, 0] = nan                # a value that all see
    vf[at(1, 180), 0, 33] = nan                   # at a window's edge, or well inside
    vf[at(1, 299 - 100 + 1), H - 1, 34] = nan
    vf[at(1, 299 - 130), H - 1, 35] = nan         # seen by the first queries of a window
    kf[at(2, 4), 0, :] = nan
    vf[at(2, 3), H - 1, 1:9] = nan
    g = torch.Generator().manual_seed(11)
    q = torch.randn(4, n, Hq, D, generator=g).bfloat16()
    out, lse = G.gqa_attn_kv8_decode(q.to(DEV), *[t.to(DEV) for t in cache], i32(lens),
                                     window=window)
    torch.cuda.synchronize()
    kc, ksn, vc, vsn = cache_np(*cache[:4], H, D)
    scale = 1 / math.sqrt(D)
    for b in range(4):
        row = table[b].tolist()
        k = P.gather(kc, ksn, row, lens[b], page, block)
        v = P.gather(vc, vsn, row, lens[b], page, block)
        coarse = np.nan_to_num(P.coarse(vc, vsn, row, lens[b], page, block))
        ref = P.decode(q[b].double().numpy(), k, v, n, scale, window, Hq // H, coarse)
        check_decode_nan(out[b].float().cpu().numpy(), lse[b].T.cpu().numpy(), ref, scale)


@pytest.mark.parametrize("Hq,H,D", [(4, 2, 128), (8, 2, 64)])
def test_decode_nan_codes_in_many_short_sequences(Hq, H, D):
    """The same where a CTA takes several sequences, one after the other, each whole."""
    page, block, n, B = 16, 16, 3, 640
    lens = [(37 * b) % 150 + 3 for b in range(B)]
    cache = build_cache(lens, page, block, H, D, 8)
    vf, table = cache[1].view(-1, H, D), cache[4]
    for b in range(0, B, 3):  # the newest value, in a dimension of the sequence's own
        pos = lens[b] - 1
        vf[table[b, pos // page].item() * page + pos % page, b % H, b % D] = 0x7f
    q = torch.randn(B, n, Hq, D, generator=torch.Generator().manual_seed(4)).bfloat16()
    out, lse = G.gqa_attn_kv8_decode(q.to(DEV), *[t.to(DEV) for t in cache], i32(lens))
    torch.cuda.synchronize()
    kc, ks, vc, vs = cache_np(*cache[:4], H, D)
    out, lse = out.float().cpu().numpy(), lse.cpu().numpy()
    for b in range(B):
        row = table[b].tolist()
        k = P.gather(kc, ks, row, lens[b], page, block)
        v = P.gather(vc, vs, row, lens[b], page, block)
        coarse = np.nan_to_num(P.coarse(vc, vs, row, lens[b], page, block))
        ref = P.decode(q[b].double().numpy(), k, v, n, 1 / math.sqrt(D), 0, Hq // H, coarse)
        check_decode_nan(out[b], lse[b].T, ref, 1 / math.sqrt(D))


def test_decode_empty_batch_and_no_queries():
    cache = [t.to(DEV) for t in build_cache([5], 16, 16, 1, 64, seed=1)]
    q = torch.zeros(0, 1, 2, 64, dtype=torch.bfloat16, device=DEV)
    bt = torch.zeros(0, 1, dtype=torch.int32, device=DEV)
    out, lse = G.gqa_attn_kv8_decode(q, *cache[:4], bt, i32([]))
    assert out.shape == q.shape and lse.shape == (0, 2, 1)
    q = torch.zeros(1, 0, 2, 64, dtype=torch.bfloat16, device=DEV)
    out, lse = G.gqa_attn_kv8_decode(q, *cache[:4], cache[4], i32([5]))
    assert out.shape == q.shape and lse.shape == (1, 2, 0)


def test_decode_reports_bad_lengths_pages_and_query_ranges():
    lens = [40, 40]
    k8, v8, ks, vs, table = build_cache(lens, 16, 16, 1, 64, seed=2)
    d = [t.to(DEV) for t in (k8, v8, ks, vs)]
    q = torch.randn(2, 1, 4, 64, device=DEV).bfloat16()
    bad = table.clone()
    bad[1, 1] = k8.shape[0]
    G.gqa_attn_kv8_decode(q, *d, bad.to(DEV), i32(lens))
    assert gqa_attn_get_device_error() == 3
    G.gqa_attn_kv8_decode(q, *d, table.to(DEV), i32([40, 49]))
    assert gqa_attn_get_device_error() == 3
    G.gqa_attn_kv8_decode(q[:, 0].contiguous(), *d, table.to(DEV), i32(lens),
                          cu_seqlens_q=i32([0, 1, 3]), max_seqlen_q=2)
    assert gqa_attn_get_device_error() == 2


def test_a_pool_past_four_gigabytes():
    """Rows, codes and scales whose offsets pass 32 bits: only the last pages are used."""
    pages, page, block, H, D = 4200, 256, 64, 32, 128       # 4.4 GB each of K and V
    k8 = torch.empty(pages, page, H, D, dtype=torch.uint8, device=DEV)
    v8 = torch.empty_like(k8)
    ks = torch.empty(pages, page // block, H, device=DEV)
    vs = torch.empty_like(ks)
    assert k8.numel() > 2 ** 32
    L = 300
    table = i32([[pages - 1, pages - 2]])
    slots = [(pages - 1) * page + i for i in range(page)] + \
        [(pages - 2) * page + i for i in range(L - page)]
    k, v = draw_kv(L, H, D, seed=3, spread=1.0)
    G.gqa_attn_kv8_append(k.to(DEV), v.to(DEV), i32(slots), k8, v8, ks, vs)
    g = torch.Generator().manual_seed(4)
    q = (1.5 * torch.randn(1, 1, 2 * H, D, generator=g)).bfloat16()
    out, lse = G.gqa_attn_kv8_decode(q.to(DEV), k8, v8, ks, vs, table, i32([L]))
    kg, vg = G.gqa_attn_kv8_gather(k8, v8, ks, vs, table, i32([0, L]), total=L)
    torch.cuda.synchronize()
    local = list(range(page, 2 * page)) + list(range(L - page))  # the last page first
    zc, zs = np.zeros((2 * page, H, D), np.uint8), np.full((2 * page // block, H), math.nan)
    (kc, ksc), (vc, vsc) = (P.append(x.double().numpy(), local, zc, zs, block) for x in (k, v))
    kk, vv = P.gather(kc, ksc, [1, 0], L, page, block), P.gather(vc, vsc, [1, 0], L, page, block)
    assert torch.equal(kg.cpu(), torch.from_numpy(kk).bfloat16())
    assert torch.equal(vg.cpu(), torch.from_numpy(vv).bfloat16())
    ref = P.decode(q[0].double().numpy(), kk, vv, 1, D ** -0.5, 0, 2,
                   P.coarse(vc, vsc, [1, 0], L, page, block))
    P.check_decode(out[0].float().cpu().numpy(), lse[0].T.cpu().numpy(), ref, D ** -0.5)


def test_append_many_single_tokens_and_long_runs_side_by_side():
    """Windows of 32 tokens that hold single tokens, whole blocks, and both."""
    H, D, page, block = 3, 64, 256, 256
    rng = np.random.default_rng(1)
    slots, pages = [], 0
    for n in [1] * 40 + [300, 1, 1, 256, 3, 700] + [2] * 20:
        off = int(rng.integers(0, page)) if n < 10 else 0
        slots += [pages * page + off % (page - n) + i if n < 10 else pages * page + i
                  for i in range(n)]
        pages += -(-n // page)
    k, v = draw_kv(len(slots), H, D, seed=12)
    run_append(k, v, slots, page, block, H, D, pages, seed=13)


def test_append_then_attend_without_waiting_on_either_side():
    """Back to back launches that may begin early still see all of what came before."""
    H, D, page = 8, 128, 64
    lens = [page * 4] * 16
    cache = build_cache(lens, page, 16, H, D, seed=50, garbage_rest=False)
    d = [t.to(DEV) for t in cache]
    q = torch.randn(16, 1, 32, D, device=DEV).bfloat16()
    k, v = (x.to(DEV) for x in draw_kv(16 * page, H, D, seed=51, spread=0.5))
    slots = torch.cat([d[4][:, 3:4] * page + torch.arange(page, device=DEV)], 1)
    slots = slots.reshape(-1).to(torch.int32)
    seq, ref = i32(lens), None
    for _ in range(30):
        d[0].view(-1, page, H, D)[d[4][:, 3].long()] = 0
        G.gqa_attn_kv8_append(k, v, slots, *d[:4])
        out, lse = G.gqa_attn_kv8_decode(q, *d, seq)
        ref = (out.clone(), lse.clone()) if ref is None else ref
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


# ----------------------------------------------------------------- a run of them together
class Server:
    """A small serving loop on the operators, with a plain 64-bit twin of its cache."""

    def __init__(self, B, page, block, H, D, pages, seed):
        self.B, self.page, self.block, self.H, self.D = B, page, block, H, D
        self.g = torch.Generator().manual_seed(seed)
        perm = torch.randperm(pages, generator=self.g).to(torch.int32)
        self.free = perm.to(DEV)
        self.start = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.table = torch.full((B, pages), -1, dtype=torch.int32, device=DEV)
        self.cached = torch.zeros(B, dtype=torch.int32, device=DEV)
        z = torch.randint(0, 256, (pages, page, H, D), generator=self.g).to(torch.uint8)
        self.k8, self.v8 = z.to(DEV), z.flip(0).contiguous().to(DEV)  # garbage, NaN too
        self.ks = torch.full((pages, page // block, H), math.nan, device=DEV)
        self.vs = self.ks.clone()
        self.twin = [t.cpu().numpy().reshape(-1, H, D) for t in (self.k8, self.v8)]
        self.twin_s = [t.cpu().double().numpy().reshape(-1, H) for t in (self.ks, self.vs)]

    def step(self, q, k, v, new, n_max, max_tokens):
        t = G.gqa_attn_kv_tables(self.cached, new, self.free, self.table, page_size=self.page,
                                 max_tokens=max_tokens, free_start=self.start)
        G.gqa_attn_kv8_append(k, v, t.slot_map, self.k8, self.v8, self.ks, self.vs)
        out, lse = G.gqa_attn_kv8_decode(q, self.k8, self.v8, self.ks, self.vs, self.table,
                                         t.seqlens_k, cu_seqlens_q=t.cu_seqlens_q,
                                         max_seqlen_q=n_max)
        self.cached.copy_(t.seqlens_k)
        self.start.copy_(t.free_end)
        return t, out, lse

    def check(self, t, q, k, v, new, out, lse):
        torch.cuda.synchronize()
        slots = t.slot_map.tolist()
        for i, x in enumerate((k, v)):
            self.twin[i], self.twin_s[i] = P.append(x.cpu().double().numpy(), slots,
                                                    self.twin[i], self.twin_s[i], self.block)
        table, lens, at, scale = self.table.tolist(), t.seqlens_k.tolist(), 0, self.D ** -0.5
        for b, n in enumerate(new):
            kk, vv = (P.gather(self.twin[i], self.twin_s[i], table[b], lens[b], self.page,
                               self.block) for i in range(2))
            coarse = P.coarse(self.twin[1], self.twin_s[1], table[b], lens[b], self.page,
                              self.block)
            ref = P.decode(q[at:at + n].cpu().double().numpy(), kk, vv, n, scale, 0,
                           q.shape[1] // self.H, coarse)
            P.check_decode(out[at:at + n].float().cpu().numpy(),
                           lse[:, at:at + n].T.cpu().numpy(), ref, scale)
            at += n


def draw_step(s, T, Hq):
    q = (1.5 * torch.randn(T, Hq, s.D, generator=s.g)).bfloat16()
    k = (torch.randn(T, s.H, s.D, generator=s.g) *
         torch.exp(torch.randn(T, s.H, 1, generator=s.g))).bfloat16()
    v = (torch.randn(T, s.H, s.D, generator=s.g) *
         torch.exp(torch.randn(T, s.H, 1, generator=s.g))).bfloat16()
    return [x.to(DEV) for x in (q, k, v)]


def test_serving_steps_together():
    s = Server(B=4, page=32, block=16, H=2, D=128, pages=40, seed=1)
    for new in ([40, 1, 17, 3], [1, 1, 1, 1], [4, 0, 1, 2], [1, 1, 1, 1], [33, 16, 1, 0]):
        T = sum(new) + 2
        q, k, v = draw_step(s, T, 8)
        t, out, lse = s.step(q, k, v, i32(new), max(new), T)
        s.check(t, q, k, v, new, out, lse)


def test_serving_steps_in_a_graph_on_a_side_stream():
    """Decode steps captured once and replayed, with the page cursor and the lengths
    advancing on the device; a second graph of the same kind alternates with it."""
    side = torch.cuda.Stream()
    servers, graphs, held = [], [], []
    for i in range(2):
        s = Server(B=3, page=16, block=16, H=2, D=64, pages=24, seed=10 + i)
        new = i32([1, 1, 1])
        prompt = draw_step(s, 9 + 20 + 1, 4)
        t, out, lse = s.step(*prompt, i32([9, 20, 1]), 20, 30)
        s.check(t, *prompt, [9, 20, 1], out, lse)
        bufs = draw_step(s, 3, 4)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        keep = [x.clone() for x in (s.cached, s.start)]
        with torch.cuda.graph(graph, stream=side):
            res = s.step(*bufs, new, 1, 3)
        for x, y in zip((s.cached, s.start), keep):
            x.copy_(y)
        servers.append((s, bufs))
        held.append(new)  # the graph reads it at every replay
        graphs.append((graph, res))
    for _ in range(20):
        for (s, bufs), (graph, _) in zip(servers, graphs):
            for x, y in zip(bufs, draw_step(s, 3, 4)):
                x.copy_(y)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for graph, _ in graphs:
                graph.replay()
        torch.cuda.synchronize()
        for (s, bufs), (_, (t, out, lse)) in zip(servers, graphs):
            s.check(t, *bufs, [1, 1, 1], out, lse)


def test_chunk_prefill_over_the_gathered_cache():
    """Cached tokens gathered to bf16 give gqa_attn's prefill the keys the cache holds."""
    s = Server(B=1, page=64, block=32, H=2, D=128, pages=8, seed=4)
    q, k, v = draw_step(s, 200, 8)
    s.step(q, k, v, i32([200]), 200, 200)
    q, k, v = draw_step(s, 100, 8)
    t, out, lse = s.step(q, k, v, i32([100]), 100, 100)
    kg, vg = G.gqa_attn_kv8_gather(s.k8, s.v8, s.ks, s.vs, s.table, t.cu_seqlens_k, total=300)
    o2, l2 = G.gqa_attn(q[None], kg[None], vg[None], causal=True)
    torch.cuda.synchronize()
    assert (l2[0] - lse).abs().max().item() <= 2e-3
    # two bf16 roundings and two roundings of the weights
    bar = 2.0 ** -7 * out.float().abs() + 2.0 ** -7 * vg.float().abs().max()
    assert bool(((o2[0].float() - out.float()).abs() <= bar).all())


def test_decode_calls_on_two_streams_at_once():
    caches = [[t.to(DEV) for t in build_cache([5000, 777], 64, 16, 2, 128, seed=40 + i)]
              for i in range(2)]
    qs = [torch.randn(2, 1, 8, 128, device=DEV).bfloat16() for _ in range(2)]
    lens = i32([5000, 777])
    ref = [G.gqa_attn_kv8_decode(q, *c, lens) for q, c in zip(qs, caches)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        got = []
        for st, q, c in zip(streams, qs, caches):
            with torch.cuda.stream(st):
                got.append(G.gqa_attn_kv8_decode(q, *c, lens))
        torch.cuda.synchronize()
        for (o, l), (o_ref, l_ref) in zip(got, ref):
            assert torch.equal(o, o_ref) and torch.equal(l, l_ref)
