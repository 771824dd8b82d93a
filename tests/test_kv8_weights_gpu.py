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


# What the kernel's arithmetic allows.  A weight is two e4m3 terms, half a step of the second
# being 2^-8 of it.
WEIGHT = 2.0 ** -8
FLOOR = 0.0


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
