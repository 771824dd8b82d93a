"""Decode over the 8-bit paged cache where the weights of a softmax or the scales of V lie far
apart: blocks much coarser or finer than their neighbours, attended to by some heads and not by
others.  Compared with the formula in 64 bits, within a share of sum p |v|."""
import math

import pytest
import torch

import exact_attention_gqa_b200 as G
from exact_attention_gqa_b200 import build, gqa_attn_get_device_error

pytestmark = pytest.mark.gpu
DEV = "cuda"
PAGE, BLOCK = 64, 16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    yield
    torch.cuda.synchronize()
    assert gqa_attn_get_device_error() == 0


def codes_of(x):
    """e4m3 codes (uint8) of x, rounded to nearest."""
    return x.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def values_of(codes):
    return codes.view(torch.float8_e4m3fn).double()


class Sequence:
    """One sequence's keys and values in a pool of shuffled pages.  The logits of query head g
    of a KV head are (to e4m3's rounding) what the caller asks for: its query is 1 in dimension
    g, where the keys hold them; the other dimensions carry noise.  Keys have a scale of their
    own, 1/4; values are codes times 2^v_exp."""

    def __init__(self, logits, v_codes, v_exp, seed):
        Hkv, self.G, self.L = logits.shape      # natural logits [Hkv, G, L]
        D = v_codes.shape[-1]                   # [L, Hkv, D] values of codes; v_exp [L / 16, Hkv]
        g = torch.Generator(device=DEV).manual_seed(seed)
        pages = -(-self.L // PAGE)
        n = pages * PAGE
        k = torch.zeros(n, Hkv, D, device=DEV)
        k[:self.L] = torch.randn(self.L, Hkv, D, generator=g, device=DEV)
        k[:self.L, :, :self.G] = logits.permute(2, 0, 1) * 4
        v = torch.zeros(n, Hkv, D, device=DEV)
        v[:self.L] = v_codes
        s = torch.ones(n // BLOCK, Hkv, device=DEV)
        s[:v_exp.shape[0]] = torch.exp2(v_exp.float())
        self.kc, self.vc = codes_of(k), codes_of(v)
        self.vs = s.double().repeat_interleave(BLOCK, 0)[:self.L]
        perm = torch.randperm(pages, generator=g, device=DEV)
        self.table = perm.to(torch.int32)       # logical page p lies in page perm[p]
        back = torch.argsort(perm)
        self.k8, self.v8 = (c.view(pages, PAGE, Hkv, D)[back].contiguous()
                            for c in (self.kc, self.vc))
        self.ks = torch.full((pages, PAGE // BLOCK, Hkv), 0.25, device=DEV)
        self.v_scale = s.view(pages, -1, Hkv)[back].contiguous()
        self.q = 0.01 * torch.randn(Hkv * self.G, D, generator=g, device=DEV)
        for h in range(Hkv * self.G):
            self.q[h, :self.G] = 0
            self.q[h, h % self.G] = 1
        self.q = self.q.bfloat16()

    def formula(self, hi, lo=0):
        """(out, lse, sum p |v|, largest p * scale times sum |code|, error of a logit) of a
        query that sees keys [lo, hi), each [Hq, D] or [Hq, 1], in 64 bits."""
        out = []
        for h in range(self.q.shape[0]):
            kv = h // self.G
            q, k = self.q[h].double(), values_of(self.kc[lo:hi, kv]) * 0.25
            code, vs = values_of(self.vc[lo:hi, kv]), self.vs[lo:hi, kv]
            z = k @ q
            m = z.max()
            p = torch.exp(z - m)
            total = p.sum()
            w = p / total * vs
            # q's terms and the fp32 sum of the products (test_kv8_gpu.py's bound)
            dz = q.abs().max() * k.abs().sum(1).max() * 2.0 ** -19
            out.append((w @ code, (m + torch.log(total))[None], w @ code.abs(),
                        w.max() * code.abs().sum(0), dz[None]))
        return [torch.stack(x) for x in zip(*out)]


# What the kernel's arithmetic allows.  A weight is rounded to f16 (half a step, 2^-11 of its
# power of two) and to nine bits (2^-9).  Where f16 has no normal numbers the steps are 2^-24
# and 2^-22, half of them 1.25 * 2^-23, and a row's largest weight, its V scale included, is
# 2^11 or more.
WEIGHT = 1.25 * 2.0 ** -9
FLOOR = 1.25 * 2.0 ** -34


def check(seq, out, lse, i, ref):
    """Rows out [B, Hq, D], lse [B, Hq] of the same query of B copies of seq."""
    o, l, a, floor, dz = ref
    assert bool(torch.isfinite(out.float()).all()) and bool(torch.isfinite(lse).all())
    # fp32 sums: 2^-16 within a product's 32 keys and the rescalings, and one rounding (down,
    # 2^-23) for each product added; a logit's error moves a weight and the normaliser.  The
    # result's bf16 rounding is half a step, 2^-8.
    sums = 2.0 ** -16 + seq.L / 32 * 2.0 ** -23
    bar = (WEIGHT + sums + 3 * dz) * a + FLOOR * floor + 2.0 ** -8 * 1.01 * o.abs()
    err = (out.double() - o).abs()
    # the reference and the logarithm that are added may each be 90 log2 units larger
    lbar = dz + 2.0 ** -19 * l.abs().clamp_min(1) + 2.0 ** -22 * 90 + seq.L / 128 * 2.0 ** -24
    lerr = (lse.double()[..., None] - l).abs()
    print("query %d: worst share of the bound: out %.3f, lse %.3f; off by %.2e of sum p |v|" %
          (i, (err / bar).max(), (lerr / lbar).max(), (err / a).max()))
    assert bool((err <= bar).all()), (err / a).max().item()
    assert bool((lerr <= lbar).all()), (lerr - lbar).max().item()


def attend(seq, B, n=1, window=0):
    """B copies of the sequence (the same pages) with n queries each, all against the formula.
    Few copies are cut into ranges of a few tiles, many are whole items of one CTA."""
    q = seq.q[None, None].expand(B, n, -1, -1).contiguous()
    table = seq.table[None].expand(B, -1).contiguous()
    lens = torch.full((B,), seq.L, dtype=torch.int32, device=DEV)
    out, lse = G.gqa_attn_kv8_decode(q, seq.k8, seq.v8, seq.ks, seq.v_scale, table, lens,
                                     window=window, scale=1.0)
    torch.cuda.synchronize()
    for i in range(n):
        hi = seq.L - n + i + 1
        check(seq, out[:, i], lse[:, :, i], i, seq.formula(hi, max(hi - window, 0) if window else 0))


def normal(shape, seed, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return std * torch.randn(shape, generator=g, device=DEV)


def values(L, Hkv, D, seed):
    """Codes' values in [1, 2): of one sign, so that lost weight shows in every dimension."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    return 1 + torch.randint(0, 8, (L, Hkv, D), generator=g, device=DEV) / 8


def coarse_block(L, Hkv, G_, D, e, at, seed, tail=0.0):
    """Block `at` of 16 keys is 2^e coarser than the rest.  Query head 0 of a KV head attends to
    it and to little else (not where it is alone), the others to all the rest: flat, or one
    early key and a tail `tail` nats below it."""
    z = normal((Hkv, G_, L), seed, 0.3) - tail
    z[:, :, 5] = 0
    own = slice(at * BLOCK, at * BLOCK + BLOCK)
    z[:, :, own] = -(e * math.log(2) + 30)
    if G_ > 1:
        z[:, 0] = normal((Hkv, L), seed + 1) - 30
        z[:, 0, own] = 5
    v_exp = torch.zeros(-(-L // BLOCK), Hkv, device=DEV)
    v_exp[at] = e
    return Sequence(z, values(L, Hkv, D, seed + 2), v_exp, seed + 3)


@pytest.mark.parametrize("Hkv,G_,D", [(2, 2, 128), (1, 1, 128), (1, 5, 128), (1, 12, 128),
                                      (2, 2, 64), (3, 1, 64), (2, 20, 64)])
@pytest.mark.parametrize("e", [3, 12, 20, 60, 90])
@pytest.mark.parametrize("B", [1, 300])
def test_coarse_block_that_one_head_attends_to(Hkv, G_, D, e, B):
    L = 1500
    for at in (0, 40, L // BLOCK - 1):
        for tail in (0.0, 6.2):
            attend(coarse_block(L, Hkv, G_, D, e, at, seed=at + e, tail=tail), B)


@pytest.mark.parametrize("Hkv,G_,D,n,window", [(2, 2, 128, 3, 0), (2, 4, 128, 8, 0),
                                               (2, 2, 64, 4, 1000), (1, 16, 128, 2, 777)])
@pytest.mark.parametrize("e", [12, 60])
def test_coarse_block_and_drafted_tokens(Hkv, G_, D, n, window, e):
    for B in (1, 150):
        attend(coarse_block(1500, Hkv, G_, D, e, 50, seed=e + n), B, n=n, window=window)


@pytest.mark.parametrize("Hkv,G_,n", [(2, 1, 1), (2, 3, 1), (3, 1, 3), (2, 8, 1), (2, 9, 2)])
@pytest.mark.parametrize("e", [20, 60])
def test_coarse_blocks_of_neighbouring_heads_one_after_the_other(Hkv, G_, n, e):
    """Heads of 64 dimensions that share a tile's rows of 128 bytes: when the second one meets
    its coarse block, the first one's references have fallen already."""
    L = 2000
    z = normal((Hkv, G_, L), e, 0.3)
    v_exp = torch.zeros(-(-L // BLOCK), Hkv, device=DEV)
    for h in range(Hkv):
        at = 20 + 40 * h
        v_exp[at, h] = e
        z[h, :, at * BLOCK:at * BLOCK + BLOCK] = -(e * math.log(2) + 30)
    for B in (1, 300):
        attend(Sequence(z, values(L, Hkv, 64, e), v_exp, e + 1), B, n=n)


def steps(L, D, up, down, order, seed):
    """Tiles of 128 keys whose scales grow by 2^up from each to the next while their logits fall
    by `down` bits (or the other way round): every head has its weight where p * scale is."""
    tile = torch.arange(L, device=DEV) // 128
    if order == "falling":
        tile = tile.max() - tile
    z = normal((2, 2, L), seed, 0.3) - (tile * down * math.log(2))[None, None]
    v_exp = (tile[::BLOCK] * up)[:, None].expand(-1, 2)
    return Sequence(z, values(L, 2, D, seed + 1), v_exp, seed + 2)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("up,down", [(16, 0), (16, 15), (28, 20), (24, 17.3), (30, 32)])
@pytest.mark.parametrize("order", ["growing", "falling"])
@pytest.mark.parametrize("B", [1, 300])
def test_scales_that_grow_from_tile_to_tile(D, up, down, order, B):
    # within 2^90 from the first tile to the last
    L = 128 * min(6, 1 + 90 // up) - 7
    attend(steps(L, D, up, down, order, seed=up), B)


# ------------------------------------------------------------------- peaked rows, long tails
def sink(L, Hkv, G_, D, drop, spread, seed, sink_value=0.0):
    """The first key outweighs each other one by `drop` nats and has a value near 0, so that the
    output is what the tail adds up to: `spread` is its logits' deviation."""
    z = normal((Hkv, G_, L), seed, spread).clamp(-3 * spread, 3 * spread) - drop
    z[:, :, 0] = 0
    v = values(L, Hkv, D, seed + 1)
    v[0] = sink_value
    return Sequence(z, v, torch.zeros(-(-L // BLOCK), Hkv, device=DEV), seed + 2)


@pytest.mark.parametrize("Hkv,G_,D", [(1, 2, 128), (1, 6, 128), (1, 16, 128), (1, 24, 128),
                                      (2, 2, 64), (2, 5, 64), (2, 9, 64)])
@pytest.mark.parametrize("drop", [8, 12, 14, 17])
@pytest.mark.parametrize("B", [1, 300])
def test_attention_sink_and_a_long_tail(Hkv, G_, D, drop, B):
    for L in (1000, 33000):
        attend(sink(L, Hkv, G_, D, drop, 1.5, seed=L + drop), B)


@pytest.mark.parametrize("drop", [14.2, 20])
@pytest.mark.parametrize("B", [1, 300])
def test_flat_tails_of_many_keys(drop, B):
    """All values 1, or 0 at the sink; at 14.2 nats 2^20 keys outweigh it."""
    for L, value in ((131072, 0.0), (1 << 20, 1.0), (1 << 20, 0.0)):
        s = sink(L, 1, 2, 64, drop, 0.0, seed=L, sink_value=value)
        attend(s, B)


@pytest.mark.parametrize("window", [0, 2048])
def test_attention_sink_before_drafted_tokens(window):
    """And one that leaves the windows of the last queries."""
    for B in (1, 100):
        attend(sink(2050, 2, 4, 128, 13, 1.0, seed=B), B, n=4, window=window)


@pytest.mark.parametrize("Hkv,G_,D", [(2, 2, 128), (1, 8, 128), (1, 20, 128), (2, 2, 64),
                                      (4, 7, 64)])
@pytest.mark.parametrize("spread", [1.0, 4.0])
@pytest.mark.parametrize("B", [1, 200])
def test_scales_with_no_order(Hkv, G_, D, spread, B):
    """Every block's scale between 2^-20 and 2^20, logits near to each other or far apart."""
    for seed in range(3):
        L = 5000 + seed
        g = torch.Generator(device=DEV).manual_seed(seed)
        z = normal((Hkv, G_, L), seed, spread).clamp(-25, 25)
        v_exp = torch.randint(-20, 21, (-(-L // BLOCK), Hkv), generator=g, device=DEV)
        v = values_of(torch.randint(0, 0x7f, (L, Hkv, D), generator=g, device=DEV)
                      .to(torch.uint8)).float()
        sign = torch.randint(0, 2, v.shape, generator=g, device=DEV) * 2 - 1
        attend(Sequence(z, v * sign, v_exp, seed + 9), B)


def test_blocks_of_zeros_beside_the_largest_scale():
    """What appending leaves: blocks of zeros have the scale 2^-126, a block with a value near
    bf16's largest one of 2^119.  One head attends to it, the other 2^-200 times less."""
    for at in (0, 10, 30):
        for B in (1, 200):
            L = 700
            z = normal((1, 2, L), at, 0.3)
            own = slice(at * BLOCK, at * BLOCK + BLOCK)
            z[0, 0] -= 30
            z[0, 0, own] = 0
            z[0, 1] += 40
            z[0, 1, own] = -100
            v_exp = torch.full((-(-L // BLOCK), 1), 10.0, device=DEV)
            v = values(L, 1, 128, at)
            v_exp[::3] = -126
            v[(torch.arange(L, device=DEV) // BLOCK) % 3 == 0] = 0
            v_exp[at] = 119
            v[own] = 1.5
            attend(Sequence(z, v, v_exp, at), B)
