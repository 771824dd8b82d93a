// Attention of the newest positions of each sequence over the 8-bit paged cache with block
// scales (kv8_cache.cuh): one position (decode) or a few (drafted tokens).
//
// Bound: HBM.  Every visible key and value is read once, at one byte an element, for about
// four operations a byte; the kernel's task is to keep the copies streaming.
//
// Both products run on the 8-bit codes as they lie in the cache, with no conversion: the
// 5th-generation MMA takes e4m3 operands from shared memory, and its M side (128 wide)
// holds what is long,
//   S^T [128 keys, rows]  = K tile [128 keys, 128 bytes]   x Q^T,
//   O^T [128 dims, rows]  = V tile^T [128 dims, 128 keys]  x P^T,
// so that one thread owns one key in the softmax and one dimension in the output.  The other
// sides are split into 8-bit terms, which are further columns of the same MMA (its N side has
// room).  q, in bf16, is two e4m3 terms, x = hi + lo / 16: e4m3 keeps four significant bits,
// so hi holds the upper four of bf16's eight and the remainder, at most half a unit of hi's
// last place, fits the other: q is exact down to 2^-21 of its row's largest element.  p has a
// range to keep as well, because a long tail of small weights counts: it is rounded to f16,
// whose upper byte is an e5m2 value of three significant bits, and taken apart into three
// such, x = hi + mid / 8 + lo / 64.  So p is off by 1.25 * 2^-9 of itself (half a step of
// nine bits, and f16's own), and by 1.25 * 2^-34 of its row's largest where it is smaller than
// 2^-25 of that.
//
// Scales: a key's K scale multiplies its logit.  Its V scale is folded into its weight,
// relative to vrun, the largest V scale met so far or one within 2^3 below it, so that O^T can
// stay in tensor memory and be summed there by the MMA.  With z the logit in log2 units and
// d = log2(vs / vrun), a row's reference m is kept at or above max_j (z_j + max(d_j, -90)) - 3:
// weights 2^11 * 2^(z - m) vs / vrun stay at or below 2^14, where none of their terms leaves
// e5m2's range, and the normaliser's terms 2^(z - m) at or below 2^96.  The 3 let references
// and vrun stay as they are in most tiles: a tile is computed with the last ones, every thread
// checks its own keys, and only where one is above the maxima are taken over all keys (a warp
// reduction a row, and an exchange), what is summed so far is rescaled and the tile computed
// again.  Where vrun grows by 2^e all d fall by e, so m falls with them, down to what the
// tile's own keys ask for and no further than the normaliser has room: the row of a head that
// does not attend to the coarse block keeps its weights' size, although another row of its KV
// head made vrun grow.  vrun follows when references are taken anew, and in any case where a
// scale is 2^3 above it.
//
// Heads of 64 dimensions go in pairs: a 128-byte row holds two KV heads.  Of the four MMAs
// over a row's bytes (K = 32), two are one head's and two the other's, each pair with its own
// head's query columns: no head meets the other's codes, which a padding with zeros would not
// keep out (NaN times 0).  Each half of O^T is read by its own head's rows (the MMA's idle
// half costs nothing here).
//
// Work: the (sequence, row unit) items of one head group are laid end to end, in tiles of
// 128 keys, and cut into equal ranges, whatever the lengths.  A range is taken by a team
// of CTAs, one for each head group (`width` of them): they walk the same keys side by
// side, so that the 128-byte pieces of one token's row are read at about the same time,
// which is what DRAM wants (one query, batch 16 at 32768 keys: 203 us before, 184 with it).
// An item that ends up in several ranges leaves one fp32 partial in each, joined by
// kv8_combine, a programmatic dependent launch.
//
// Roles: one warp copies and looks pages up, one issues the MMAs, one or two warpgroups do
// the softmax.
//
// Measured (device time in a CUDA graph; 32 query heads on 8, D 128): one query, batch 16 at
// 32768 keys 168 to 170 us (6.3 to 6.4 TB/s of the cache's data), batch 64 ragged up to 8192
// 98 us, 8 sequences of up to 8192 with four queries each 38 us, one of 1000 keys 12 us.
#pragma once
#include "kv8_cache.cuh"

namespace gqa {

struct Kv8DecodeParams {
    const __nv_bfloat16* q;   // [rows, Hq, D]
    __nv_bfloat16* out;       // like q
    float* lse;               // dense [B, Hq, Sq], packed [Hq, total_q]
    const float* k_scale;     // [num_pages * page_size / sb, Hkv]
    const float* v_scale;
    const int* block_table;   // [B, max_pages]
    const int* seqlens_k;     // [B]
    const int* cu_seqlens_q;  // [B + 1] or null: Sq queries each
    float* part_o;            // [CTAs, 2, R, 128] fp32 partials of a CTA's cut items
    float2* part_ml;          // [CTAs, 2, R] reference (log2 units) and sum
    int4* cut;                // [CTAs][2] the item that starts in a CTA's range and ends in
                              // another's, and its sequence
    int B, Sq, total_q, Hq, Hkv, G;
    int groups, units;        // head groups (KV heads, or pairs of them); row units of each
    int width, teams;         // CTAs of a team (divides groups), teams of the grid
    int num_pages, page_shift, sb_shift, max_pages, window;
    float scale_log2;
};

// ROWS query rows (query head x position, of both heads of a pair) per CTA and pass
template <int ROWS>
struct Kv8Cfg {
    static constexpr int WGS = ROWS >= 16 ? 2 : 1;      // consumer warpgroups, rows split
    static constexpr int RW = ROWS / WGS;               // rows of each
    // Three CTAs with two stages each, for 4 rows (more do not fit), measured against two with
    // three: batch 16 at 32768 keys 182 / 169 us, ragged batch of 64 95.3 / 97.7, one sequence
    // of 32768 25.8 / 25.3.
    static constexpr int CTAS_PER_SM = 2;
    // Stages of K, and of V and scales: what fits shared memory.  For 16 rows, 8 x 4 and 16 x 4
    // drafted: two of K and three of V 37.1 and 116.6 us, three and two 38.0 and 123.0, three
    // of both with one buffer of P 38.9 and 121.6.
    static constexpr int STK = ROWS < 16 ? 3 : 2;
    static constexpr int STV = ROWS <= 16 ? 3 : 2;
    static constexpr int TILE = 128 * 128;              // bytes of K or V per stage
    static constexpr int N = ROWS <= 8 ? 16 : 2 * ROWS;  // S^T's columns: a row's hi and lo
    static constexpr int NQ = ROWS <= 8 ? 32 : 2 * ROWS;  // q's: of a pair, N / 2 or 16 a head
    static constexpr int NP = (3 * ROWS + 15) / 16 * 16;  // O^T's and P's: hi, mid and lo
    static_assert(2 * NP * 128 >= ROWS * 512, "an item's results fit P's buffers");
    static constexpr int OFF_K = 0;
    static constexpr int OFF_V = STK * TILE;
    static constexpr int OFF_Q = OFF_V + STV * TILE;
    static constexpr int OFF_P = OFF_Q + NQ * 128;      // two buffers; an item's results
    static constexpr int OFF_SC = OFF_P + 2 * NP * 128;  // [STV][K, V][2 halves][8 groups]
    static constexpr int OFF_RED = OFF_SC + STV * 128;  // [ROWS][4 warps]
    static constexpr int OFF_ROW = OFF_RED + 16 * ROWS;  // [2][2][ROWS] logit factor, reference
    static constexpr int OFF_LIM = OFF_ROW + 32 * ROWS;  // [2][ROWS] keys a row sees: from, to
    static constexpr int OFF_TOP = OFF_LIM + 16 * ROWS;  // [2][ROWS] next reference, ordered int
    static constexpr int OFF_VRUN = OFF_TOP + 8 * ROWS;  // [2][2 halves] vrun, its log2, its
                                                         // inverse, what counts as far above
    static constexpr int OFF_OUT = OFF_VRUN + 64;        // [2][ROWS] position or -1, head
    static constexpr int OFF_NAN = OFF_OUT + 16 * ROWS;  // [2][ROWS] dimensions: 128 bits
    static constexpr int OFF_SEG = OFF_NAN + 32 * ROWS;  // [8] Kv8Segment
    static constexpr int OFF_BAR = OFF_SEG + 8 * 64;
    static constexpr int N_BAR = 2 * STK + 3 * STV + 8;
    static constexpr int OFF_MISC = OFF_BAR + 8 * N_BAR;
    static constexpr int SMEM_BYTES = OFF_MISC + 64 + 1024;
    static constexpr int TMEM_COLS = NQ == 32 ? 128 : 256;  // two of S^T, one of O^T
    static constexpr int CONSUMERS = 128 * WGS;
    static constexpr int THREADS = CONSUMERS + 64;      // and the producer's and the MMA warp
    static_assert((SMEM_BYTES + 1024) * CTAS_PER_SM <= 228 * 1024, "shared memory of an SM");
    static_assert(2 * NQ + NP <= TMEM_COLS && TMEM_COLS * CTAS_PER_SM <= 512, "tensor memory");
};

// Instruction descriptor, kind::f8f6f4: the B operand's format (bits [10, 13)) e5m2, not e4m3
constexpr uint32_t kBIsE5m2 = 1u << 10;

// Reference of a row that no key has reached: any logit is above it, and it stays finite
constexpr float kNoKey = -1e30f;
// Reference of a row that pads a pass: no logit is above it, and no weight is seen in fp32
constexpr float kNoRow = 1e30f;
// How far below vrun a V scale may lie (log2) and its keys' logits still set the reference:
// the normaliser's terms reach 2^(6 - kFar) (a fall of 3 is not checked), and 2^30 keys of them
// fp32's range
constexpr float kFar = -90.f;
// A weight whose logit is its row's reference and whose V scale is vrun
constexpr float kTopWeight = 2048.f;

struct Kv8Seq {
    int q0, n, len;  // first query row, queries, keys
};
__device__ __forceinline__ Kv8Seq kv8_seq(const Kv8DecodeParams& p, int b) {
    Kv8Seq s;
    s.q0 = b * p.Sq;
    s.n = p.Sq;
    if (p.cu_seqlens_q) {
        s.q0 = p.cu_seqlens_q[b];
        s.n = p.cu_seqlens_q[b + 1] - s.q0;
        if (s.n < 0 || s.n > p.Sq || s.q0 < 0 || s.q0 > p.total_q - s.n) {
            raise_device_error(kDevBadTile);
            s.n = 0;
        }
    }
    const int cap = p.max_pages << p.page_shift;
    s.len = p.seqlens_k[b];
    if (s.len < 0 || s.len > cap) {
        raise_device_error(kDevBadKvIndex);
        s.len = min(max(s.len, 0), cap);
    }
    return s;
}

// Keys [lo, hi) that some row of unit u sees (SUB positions x heads of one KV head each)
struct Kv8Keys {
    int lo, hi;
    __device__ __forceinline__ int first() const { return lo >> 7; }
    __device__ __forceinline__ int tiles() const {
        return hi > lo ? ((hi + 127) >> 7) - (lo >> 7) : 0;
    }
};
template <int SUB>
__device__ __forceinline__ Kv8Keys kv8_keys(const Kv8DecodeParams& p, const Kv8Seq& s, int u) {
    const int i0 = u * SUB / p.G;
    const int i1 = min((u * SUB + SUB - 1) / p.G, s.n - 1);
    Kv8Keys k = {0, 0};
    if (i0 < s.n) {
        k.hi = max(s.len - s.n + i1 + 1, 0);
        if (p.window > 0) k.lo = max(s.len - s.n + i0 + 1 - p.window, 0);
    }
    return k;
}

// What a CTA's range is measured in: an item with n > 0 tiles counts n + kItemStart, its
// first kItemStart units standing for its start.  Beginning another item (its q, the first
// tile's two passes, the last one's results) takes a CTA 4 to 6 us, a tile about 1.3; with
// equal numbers of tiles the CTAs with more items were that much behind.  Measured at 0 / 2 /
// 4: window batch of 32 (D 64) 46.2 / 40.8 / 40.1 us, 4 drafted tokens for 8 41.8 / 39.2 /
// 37.8, ragged batch of 64 100.7 / 97.6 / 97.7, one sequence of 1000 keys 11.6 / 12.3 / 12.3.
constexpr int kItemStart = 4;
__device__ __forceinline__ int kv8_cost(int tiles) { return tiles > 0 ? tiles + kItemStart : 0; }
// Units are numbered with 31 bits (the host refuses more).  `units` of them go to `teams`
// teams, at most as many: team t starts at floor(units * t / teams).
__device__ __forceinline__ int kv8_range_start(int units, int team, int teams) {
    const int each = units / teams, rest = units - each * teams;
    return each * team + rest * team / teams;
}

// A warp's walk over its CTA's range of tiles: segments of consecutive items.  The lanes
// hold the lengths of 32 sequences, so a step to the next one seldom reads memory.
template <int SUB>
struct Kv8Walk {
    int b, hs, u;        // the item: sequence, set of `width` head groups, row unit
    int off;             // its units already passed
    int left;            // units of this CTA still to come
    int base;            // lane l holds sequence base + l
    Kv8Seq held;
    Kv8Seq seq;
    Kv8Keys keys;
    int n;               // its tiles
    __device__ __forceinline__ void hold(const Kv8DecodeParams& p, int base_) {
        base = base_;
        const int mine = base + int(threadIdx.x & 31);
        held = {0, 0, 0};
        if (mine < p.B) held = kv8_seq(p, mine);
    }
    __device__ __forceinline__ void load(const Kv8DecodeParams& p) {
        if (b - base >= 32) hold(p, b);
        const int l = b - base;
        seq.q0 = __shfl_sync(0xffffffffu, held.q0, l);
        seq.n = __shfl_sync(0xffffffffu, held.n, l);
        seq.len = __shfl_sync(0xffffffffu, held.len, l);
        keys = kv8_keys<SUB>(p, seq, u);
        n = keys.tiles();
    }
    __device__ __forceinline__ int held_units(const Kv8DecodeParams& p) const {
        int t = 0;
        for (int v = 0; v < p.units; ++v) t += kv8_cost(kv8_keys<SUB>(p, held, v).tiles());
        return t * (p.groups / p.width);
    }
    // Adds up the units of one head group (the result) and goes to the first of the range
    // of team `team` of `teams`; start: that unit's number.
    __device__ __forceinline__ int find(const Kv8DecodeParams& p, int team, int& teams,
                                        int& start) {
        const int sets = p.groups / p.width, lane = threadIdx.x & 31;
        hold(p, 0);
        int t = held_units(p), all = t;
        for (int x = 32; x < p.B; x += 32) {
            hold(p, x);
            all += held_units(p);
        }
        all = __reduce_add_sync(0xffffffffu, all);
        teams = max(min(all, p.teams), 1);
        left = start = 0;
        if (team >= teams || all == 0) return all;
        start = kv8_range_start(all, team, teams);
        left = kv8_range_start(all, team + 1, teams) - start;
        if (p.B > 32) {
            hold(p, 0);
            t = held_units(p);
        }
        off = start;
        hs = u = 0;
        while (true) {  // 32 sequences at a time
            int inc = t;
#pragma unroll
            for (int x = 1; x < 32; x <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, inc, x);
                if (lane >= x) inc += o;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, off < inc);
            if (past) {
                const int l = __ffs(past) - 1;
                b = base + l;
                off -= __shfl_sync(0xffffffffu, inc - t, l);
                t = __shfl_sync(0xffffffffu, t, l);
                break;
            }
            off -= __shfl_sync(0xffffffffu, inc, 31);
            hold(p, base + 32);
            t = held_units(p);
        }
        if (sets > 1) {
            t /= sets;
            hs = off / t;
            off -= hs * t;
        }
        load(p);
        while (off >= kv8_cost(n)) {
            off -= kv8_cost(n);
            ++u;
            load(p);
        }
        return all;
    }
    // units, and tiles [first, first + tiles) of the item, in this CTA's range
    __device__ __forceinline__ int segment() const { return min(kv8_cost(n) - off, left); }
    __device__ __forceinline__ int first() const { return max(off - kItemStart, 0); }
    __device__ __forceinline__ int tiles() const {
        return max(off + segment() - kItemStart, 0) - first();
    }
    __device__ __forceinline__ void next(const Kv8DecodeParams& p) {
        left -= segment();
        off = 0;
        if (left <= 0) return;
        do {
            if (++u == p.units) {
                u = 0;
                if (++hs == p.groups / p.width) {
                    hs = 0;
                    ++b;
                }
            }
            load(p);
        } while (n == 0);
    }
};

// What the consumers need to know of a CTA's consecutive tiles of one item
struct Kv8Segment {
    int tiles, first;  // tiles here (0: no more segments), the first one's number
    int b, hg, u;      // the item
    int slot;          // this CTA's partial of it; -1: the item is whole
    Kv8Seq seq;
    Kv8Keys keys;
};
static_assert(sizeof(Kv8Segment) <= 64, "");

// float bits as an int that orders like the float, and back
__device__ __forceinline__ int ordered(float x) {
    const int i = __float_as_int(x);
    return i < 0 ? i ^ 0x7fffffff : i;
}
__device__ __forceinline__ float unordered(int i) {
    return __int_as_float(i < 0 ? i ^ 0x7fffffff : i);
}

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y)
        : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(taddr)
        : "memory");
}
// Rows [r0, r0 + C) of an accumulator whose column r is row r's hi term and column ROWS + r
// its lo term.
template <int ROWS, int C>
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, int r0, float (&hi)[C],
                                             float (&lo)[C]) {
    static_assert((ROWS == 4 && C == 4) || C == 8, "");
    uint32_t a[8], b[8];
    tmem_ld8(taddr + r0, a);
    if constexpr (C == 8) tmem_ld8(taddr + ROWS + r0, b);
    tmem_ld_wait();
    reg_fence(a);
    if constexpr (C == 8) reg_fence(b);
#pragma unroll
    for (int i = 0; i < C; ++i) {
        hi[i] = __uint_as_float(a[i]);
        lo[i] = __uint_as_float(C == 8 ? b[i] : a[4 + i]);
    }
}
// Logits (hi and lo terms) of rows r0 .. of S^T.  Of a pair's columns, NQ / 2 are each head's:
// hi of its rows, then lo.
template <int ROWS, bool PAIR, int C>
__device__ __forceinline__ void tmem_ld_logits(uint32_t taddr, int r0, float (&hi)[C],
                                               float (&lo)[C]) {
    if constexpr (!PAIR) {
        tmem_ld_rows<ROWS, C>(taddr, r0, hi, lo);
    } else {
        constexpr int SUB = ROWS / 2, HALF = Kv8Cfg<ROWS>::NQ / 2;
        uint32_t a[8], b[8];
        if constexpr (C > SUB) {  // these are rows of both heads
            static_assert(C == 2 * SUB && C <= 8, "");
            tmem_ld8(taddr, a);
            tmem_ld8(taddr + HALF, b);
        } else {  // of one
            static_assert(C == 8 && SUB % 8 == 0, "");
            const uint32_t at = taddr + r0 / SUB * HALF + r0 % SUB;
            tmem_ld8(at, a);
            tmem_ld8(at + SUB, b);
        }
        tmem_ld_wait();
        reg_fence(a);
        reg_fence(b);
#pragma unroll
        for (int i = 0; i < C; ++i) {
            if constexpr (C > SUB) {
                hi[i] = __uint_as_float(i < SUB ? a[i] : b[i - SUB]);
                lo[i] = __uint_as_float(i < SUB ? a[SUB + i] : b[i]);
            } else {
                hi[i] = __uint_as_float(a[i]);
                lo[i] = __uint_as_float(b[i]);
            }
        }
    }
}
// Rows [r0, r0 + C) of O^T, whose column t * ROWS + r is row r's term t (hi, mid, lo): the sums
// of weights relative to the rows' references, and a rescaling.
template <int ROWS, int C>
struct OutTerms {
    static_assert((ROWS == 4 && C == 4) || C == 8, "");
    static constexpr int LOADS = C == 8 ? 3 : 2;  // of 8 columns: a term, or two of four rows
    static __device__ __forceinline__ uint32_t column(int r0, int i) {
        return C == 8 ? i * ROWS + r0 : i * 8;
    }
    static __device__ __forceinline__ void sum(uint32_t taddr, int r0, float (&x)[C]) {
        uint32_t a[LOADS][8];
#pragma unroll
        for (int i = 0; i < LOADS; ++i) tmem_ld8(taddr + column(r0, i), a[i]);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < LOADS; ++i) reg_fence(a[i]);
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const float hi = __uint_as_float(a[0][j]);
            const float mid = __uint_as_float(C == 8 ? a[1][j] : a[0][4 + j]);
            const float lo = __uint_as_float(a[LOADS - 1][j]);
            constexpr float k = 1.f / kTopWeight;
            x[j] = fmaf(lo, k / 64, fmaf(mid, k / 8, hi * k));
        }
    }
    static __device__ __forceinline__ void scale(uint32_t taddr, int r0, const float (&by)[C]) {
        uint32_t a[LOADS][8];
#pragma unroll
        for (int i = 0; i < LOADS; ++i) tmem_ld8(taddr + column(r0, i), a[i]);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            reg_fence(a[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                a[i][j] = __float_as_uint(__uint_as_float(a[i][j]) * by[j % C]);
            tmem_st8(taddr + column(r0, i), a[i]);
        }
        tmem_st_wait();
    }
};

__device__ __forceinline__ void prefetch_l2(const void* at) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
}
// Whether the phase of `bar` with parity `parity` has completed; never waits
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// Four values as two e4m3 terms each (byte i: value i), x = hi + lo / shift
__device__ __forceinline__ void split_e4m3x4(float x0, float x1, float x2, float x3, float shift,
                                             uint32_t& hi, uint32_t& lo) {
    hi = pack_e4m3x4(x0, x1, x2, x3);
    uint32_t h01, h23;
    e4m3x4_to_f16x4(hi, h01, h23);
    add_f16x2_to_f32(h01 ^ 0x80008000u, x0, x1);
    add_f16x2_to_f32(h23 ^ 0x80008000u, x2, x3);
    lo = pack_e4m3x4(x0 * shift, x1 * shift, x2 * shift, x3 * shift);
}
// Four weights, at most 2^14, as three e5m2 terms each (byte i: weight i), x = hi + mid / 8 +
// lo / 64.  The upper byte of an f16 is the e5m2 value next to it towards 0; what is left
// is exact in f16, and eight times that is in range again.  The last term is rounded to
// nearest: half a unit of a byte is added below it (all terms are >= 0; a NaN stays in hi).
__device__ __forceinline__ void split_e5m2x4(float x0, float x1, float x2, float x3,
                                             uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    uint32_t a, b;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(a) : "f"(x1), "f"(x0));
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(b) : "f"(x3), "f"(x2));
    hi = __byte_perm(a, b, 0x7531);
    auto rest = [](uint32_t x) {  // eight times what x's upper bytes leave
        uint32_t r;
        asm("{\n\t.reg .b32 t;\n\tsub.f16x2 t, %1, %2;\n\tmul.f16x2 %0, t, %3;\n\t}"
            : "=r"(r)
            : "r"(x), "r"(x & 0xff00ff00u), "r"(0x48004800u));
        return r;
    };
    a = rest(a), b = rest(b);
    mid = __byte_perm(a, b, 0x7531);
    a = rest(a), b = rest(b);
    lo = __byte_perm(a + 0x00800080u, b + 0x00800080u, 0x7531);
}
// Descriptor of an operand of 16-byte chunks along M or N with no swizzle, the chunks of
// consecutive k next to each other: kgroup bytes from eight k to the next eight, chunk
// bytes from one chunk to the next (leading and stride offset of this layout).
__device__ __forceinline__ uint64_t mn_chunk_desc(uint32_t smem_addr, uint32_t kgroup,
                                                  uint32_t chunk) {
    return uint64_t((smem_addr >> 4) & 0x3FFFu) | uint64_t(kgroup >> 4) << 16 |
           uint64_t(chunk >> 4) << 32 | uint64_t(1) << 46;
}
__device__ __forceinline__ void st_shared_v2(uint32_t addr, uint32_t a, uint32_t b) {
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}
template <int THREADS>
__device__ __forceinline__ void consumers_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}
template <int THREADS>
__device__ __forceinline__ bool consumers_any(bool x) {
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, %2, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(int(x)), "n"(THREADS)
        : "memory");
    return r != 0;
}

// Bit 7 of each byte that is a NaN code (0x7f or 0xff)
__device__ __forceinline__ uint32_t nan_codes(uint32_t x) {
    return ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}
// Zeroes the NaN codes of V's row for `key` (row n of a tile, 128-byte swizzle) and notes
// their dimensions, 128 bits a query row, for the rows that see the key.
template <int ROWS>
__device__ __noinline__ void take_out_nan(uint32_t* v, int n, int key, const int2* limits,
                                          uint32_t* noted) {
    for (int j = 0; j < 32; ++j) {
        const uint32_t nan = nan_codes(v[j]);
        if (nan == 0u) continue;
        v[j] &= ~((nan >> 7) * 0xffu);
        const int d = (((j >> 2) ^ (n & 7)) << 4) + (j & 3) * 4;
        const uint32_t bits = (nan >> 7 & 1u) | (nan >> 14 & 2u) | (nan >> 21 & 4u) |
                              (nan >> 28 & 8u);
        for (int r = 0; r < ROWS; ++r)
            if (key >= limits[r].x && key < limits[r].y)
                atomicOr(noted + r * 4 + (d >> 5), bits << (d & 31));
    }
}

// Where row `r` of unit u belongs: position i of its sequence and query head h
template <int ROWS, bool PAIR>
__device__ __forceinline__ bool kv8_row(const Kv8DecodeParams& p, const Kv8Seq& s, int hg, int u,
                                        int r, int& i, int& h) {
    constexpr int SUB = PAIR ? ROWS / 2 : ROWS;
    const int half = PAIR ? r / SUB : 0;
    const int sub = u * SUB + (r - half * SUB);
    const int kvh = PAIR ? 2 * hg + half : hg;
    i = sub / p.G;
    h = kvh * p.G + (sub - i * p.G);
    return i < s.n && kvh < p.Hkv;
}

// Dimension `dim` (0..127, of both heads of a pair) of a finished row r, position i of its
// sequence and query head h: from its sums over the keys of weights (relative to 2^ref)
// times values, and of weights
template <int ROWS, bool PAIR>
__device__ __forceinline__ void kv8_store(const Kv8DecodeParams& p, const Kv8Seq& seq, int b,
                                          int i, int h, int r, int dim, float acc, float sum,
                                          float ref) {
    constexpr int D = PAIR ? 64 : 128;
    if (!PAIR || dim / 64 == r / (ROWS / 2))
        p.out[(size_t(seq.q0 + i) * p.Hq + h) * D + (dim & (D - 1))] =
            __float2bfloat16_rn(sum == 0.f ? 0.f : acc / sum);
    if (dim == 0)
        p.lse[p.cu_seqlens_q ? size_t(h) * p.total_q + seq.q0 + i
                             : (size_t(b) * p.Hq + h) * p.Sq + i] =
            sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.69314718055994531f;
}

template <int ROWS, bool PAIR>
__global__ void __launch_bounds__(Kv8Cfg<ROWS>::THREADS, Kv8Cfg<ROWS>::CTAS_PER_SM)
    kv8_decode(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
               const Kv8DecodeParams p) {
    using C = Kv8Cfg<ROWS>;
    constexpr int SUB = PAIR ? ROWS / 2 : ROWS;
    constexpr int RW = C::RW, CT = C::CONSUMERS, PRODUCER = C::CONSUMERS / 32;
    constexpr int CH = ROWS < 8 ? ROWS : 8;  // rows per accumulator load
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full_k = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* s_done = full_k + C::STK;  // S^T computed: its K stage is free
    uint64_t* full_v = s_done + C::STK;
    uint64_t* full_s = full_v + C::STV;  // scales
    uint64_t* o_done = full_s + C::STV;  // O^T summed: its V stage, scales and P are free
    uint64_t* p_ready = o_done + C::STV;  // [2] P written, S^T read
    uint64_t* seg_ready = p_ready + 2;   // [2] a segment's description written
    uint64_t* seg_free = seg_ready + 2;  // [2] the segment is finished
    uint64_t* q_ready = seg_free + 2;    // [2] the segment's q written
    int* misc = reinterpret_cast<int*>(smem + C::OFF_MISC);
    volatile int* abort_flag = misc;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 1);
    Kv8Segment* segments = reinterpret_cast<Kv8Segment*>(smem + C::OFF_SEG);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < C::N_BAR; ++i) mbar_init(full_k + i, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == PRODUCER + 1) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();  // at once: the SM's other CTAs cannot allocate before
        if (lane == 0) {
            tma_prefetch_desc(&tm_k);
            tma_prefetch_desc(&tm_v);
        }
    }
    griddep_wait();  // whatever wrote the cache, the tables and q has completed

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == PRODUCER) {
        // ------------------------------------------------------------ producer
        // A tile is one copy per page it touches (128 rows at most), one lane each, and the
        // scales of its eight groups of 16 keys (a scale block is 16 keys or more) of each
        // head.  The warp looks the pages of a batch of tiles up at once, a lane for each
        // tile and box and for each tile, head and group, one batch ahead and across
        // segments.
        // A tile's scales are waited for before the next one's copies, on purpose: they lie in a
        // 32-byte sector that the CTAs of a team share, so that all of them wait for the same
        // one and stay in step.  With asynchronous copies of the scales nothing held a team
        // together, its CTAs drifted up to 17 us apart (below 1 here; batch 16, 32768 keys),
        // the pieces of a token's row were no longer read at the same time, and that batch
        // took 188 us against 164 at that time.
        const int team = blockIdx.x / p.width, member = blockIdx.x - team * p.width;
        Kv8Walk<SUB> walk;
        int teams, range;
        const int all = walk.find(p, team, teams, range);
        const int total = walk.left;
        constexpr int BATCH = PAIR ? 2 : 4;
        const int box = min(1 << p.page_shift, 128), boxes = 128 / box;
        const int mine = lane * BATCH / 32;  // this lane's tile of a batch
        const int half = PAIR ? (lane >> 3) & 1 : 0, grp = lane & 7;
        struct Batch {
            int t, t1;   // its tiles (none: no more batches)
            int seg;     // their segment, if they are its first, else -1
            int lo, hi;  // the segment's keys
            int b, hg;   // and its sequence and head group
        };
        Batch seg_now = {0, 0, -1, 0, 0, 0, 0};  // what is left of the segment being cut up
        int segs = 0;
        auto next_batch = [&](Batch& x) {
            if (seg_now.t >= seg_now.t1) {
                // (an item may be in the range with nothing but its start)
                while (walk.left > 0 && walk.tiles() == 0) walk.next(p);
                if (walk.left <= 0) {
                    x.t = x.t1 = 0;
                    x.seg = -1;
                    return;
                }
                Kv8Segment g;
                g.tiles = walk.tiles();
                g.first = walk.keys.first() + walk.first();
                g.b = walk.b, g.hg = walk.hs * p.width + member, g.u = walk.u;
                g.seq = walk.seq, g.keys = walk.keys;
                const bool starts = walk.first() == 0, whole = starts && g.tiles == walk.n;
                g.slot = whole ? -1 : segs == 0 ? 0 : 1;
                if (starts && !whole && lane == 0) {
                    // for the combine: the item, the teams it is in (the one with its last
                    // tile is where it ends), and this CTA's partial
                    const int end = range + (total - walk.left) - walk.off + kv8_cost(walk.n);
                    const int parts = int(((long long)end * teams - 1) / all) - team + 1;
                    p.cut[2 * blockIdx.x] = make_int4(g.b, g.hg, g.u, 2 * parts + g.slot);
                    p.cut[2 * blockIdx.x + 1] = make_int4(g.seq.q0, g.seq.n, g.seq.len, 0);
                }
                // (eight slots: at most two segments ahead of the batch that is copied, and
                // that one's segment waits for the last but one before it)
                if (lane == 0) segments[segs & 7] = g;
                for (int r = lane; r < ROWS && segs > 0; r += 32) {  // q is wanted soon
                    int i, h;
                    if (kv8_row<ROWS, PAIR>(p, g.seq, g.hg, g.u, r, i, h)) {
                        const __nv_bfloat16* q =
                            p.q + (size_t(g.seq.q0 + i) * p.Hq + h) * (PAIR ? 64 : 128);
                        prefetch_l2(q);
                        if (!PAIR) prefetch_l2(q + 64);
                    }
                }
                seg_now = {g.first, g.first + g.tiles, segs++, g.keys.lo, g.keys.hi, g.b, g.hg};
                walk.next(p);
            }
            x = seg_now;
            x.t1 = min(x.t + BATCH, x.t1);
            seg_now.t = x.t1;
            seg_now.seg = -1;
        };
        // Rows without a visible key are read from a page that has one: their own table entry
        // may name no page.
        auto copies = [&](const Batch& x) { return x.t + mine < x.t1 && half == 0 && grp < boxes; };
        auto seen = [&](const Batch& x) {
            const int a = (x.t + mine) * 128 + grp * 16;
            return x.t + mine < x.t1 && a < x.hi && a + 16 > x.lo &&
                   (PAIR ? 2 * x.hg + half : x.hg) < p.Hkv;
        };
        int box_page = 0, grp_page = 0;  // of the batch looked up last, this lane's
        auto look_up = [&](const Batch& x) {
            const int* row = p.block_table + size_t(x.b) * p.max_pages;
            const int t = x.t + mine, a = t * 128 + grp * box;
            const int key = a < x.hi && a + box > x.lo ? a : max(x.lo, t * 128);
            // (a lane without a box or a group reads the row's first entry, and uses none)
            box_page = row[copies(x) ? key >> p.page_shift : 0];
            grp_page = row[seen(x) ? (t * 128 + grp * 16) >> p.page_shift : 0];
        };
        auto slot = [&](int page, int at) {
            if (page < 0 || page >= p.num_pages) {
                raise_device_error(kDevBadKvIndex);
                page = 0;
            }
            return (page << p.page_shift) + (at & ((1 << p.page_shift) - 1));
        };
        int c = 0, copied[2] = {0, 0};  // tiles; copies of K and of V issued
        bool ok = true;
        Batch now;
        if (lane == 0) p.cut[2 * blockIdx.x].x = -1;  // unless an item is cut
        __syncwarp();
        next_batch(now);
        if (lane == 0 && now.seg == 0) mbar_arrive(seg_ready);
        if (now.t < now.t1) look_up(now);
        while (now.t < now.t1) {
            const bool copies_now = copies(now), seen_now = seen(now);
            int z = 0;               // first row of this lane's box
            size_t scale_at = 0;     // where this lane's group's scales are
            if (copies_now) z = slot(box_page, (now.t + mine) * 128 + grp * box);
            if (seen_now)
                scale_at = size_t(slot(grp_page, (now.t + mine) * 128 + grp * 16) >> p.sb_shift) *
                               p.Hkv +
                           (PAIR ? 2 * now.hg + half : now.hg);
            Batch next;
            next_batch(next);
            if (next.t < next.t1) look_up(next);
            if (now.seg > 0) {
                const int buf = now.seg & 1;
                ok = mbar_wait_warp(seg_free + buf, ((now.seg >> 1) & 1) ^ 1, abort_flag);
                if (!ok) break;
                if (lane == 0) mbar_arrive(seg_ready + buf);
                __syncwarp();
            }
            for (int t = now.t; t < now.t1; ++t, ++c) {
                const bool turn = mine == t - now.t;  // this lane's tile
                const int sk = c % C::STK, s = c % C::STV;
                ok = mbar_wait_warp(s_done + sk, ((c / C::STK) & 1) ^ 1, abort_flag);
                if (!ok) break;
                // (here and not before that wait: about 1 %; behind K's or V's copy the ragged
                // batch of 64 takes 101.5 or 119.2 us instead of 97.7, 16 at 32768 keys 166.9 or
                // 164.4 instead of 168.6)
                float ks = 0.f, vs = 0.f;
                if (turn && seen_now) {
                    ks = p.k_scale[scale_at];
                    vs = p.v_scale[scale_at];
                }
                if (lane == 0) mbar_arrive_expect_tx(full_k + sk, C::TILE);
                __syncwarp();
                if (turn && copies_now)
                    tma_load_2d(smem + C::OFF_K + sk * C::TILE + grp * box * 128, &tm_k,
                                full_k + sk, now.hg * 128, z);
                ++copied[0];
                ok = mbar_wait_warp(o_done + s, ((c / C::STV) & 1) ^ 1, abort_flag);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(full_v + s, C::TILE);
                __syncwarp();
                if (turn && copies_now)
                    tma_load_2d(smem + C::OFF_V + s * C::TILE + grp * box * 128, &tm_v,
                                full_v + s, now.hg * 128, z);
                ++copied[1];
                // V's stage being free, so is the stage of scales: every consumer warp has
                // read them before that tile's P V was issued.  Groups without a visible key
                // get scales of 0.
                if (turn) {
                    float* sc =
                        reinterpret_cast<float*>(smem + C::OFF_SC) + s * 32 + half * 8 + grp;
                    sc[0] = ks, sc[16] = vs;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(full_s + s);
            }
            if (!ok) break;
            now = next;
        }
        // no more segments
        if (ok && mbar_wait_warp(seg_free + (segs & 1), ((segs >> 1) & 1) ^ 1, abort_flag) &&
            lane == 0) {
            segments[segs & 7].tiles = 0;
            mbar_arrive(seg_ready + (segs & 1));
        }
        // every issued copy lands before the CTA may release the memory
        if (lane == 0) {
#pragma unroll
            for (int kv = 0; kv < 2; ++kv)
                for (int s = 0; s < (kv ? C::STV : C::STK); ++s) {
                    const int st = kv ? C::STV : C::STK;
                    const int n = copied[kv] / st + (s < copied[kv] % st ? 1 : 0);
                    const uint64_t t0 = globaltimer_ns();
                    while (n > 0 && !mbar_try_wait((kv ? full_v : full_k) + s, (n - 1) & 1))
                        if (globaltimer_ns() - t0 > kWaitLimitNs) {
                            raise_device_error(kDevWaitTimeout);
                            break;
                        }
                }
        }
    } else if (warp == PRODUCER + 1) {
        // ------------------------------------------------------------ MMA issuer
        // S^T of the next tile goes out as soon as its keys are here and the tile before
        // the last has left the buffer; P V as soon as P and the values are.  (Issuing four
        // MMAs takes a few hundred cycles, so no consumer does it.)
        if (lane == 0) {
            const uint32_t idesc_s = idesc_e4m3_f32(128, PAIR ? C::NQ / 2 : C::N, 0, 0);
            const uint32_t idesc_o = idesc_e4m3_f32(128, C::NP, 1, 1) | kBIsE5m2;
            const uint64_t dk = sw128_desc(smem_u32(smem + C::OFF_K), 16, 1024);
            const uint64_t dv = sw128_desc(smem_u32(smem + C::OFF_V), C::TILE, 1024);
            const uint64_t dq = sw128_desc(smem_u32(smem + C::OFF_Q), 16, 1024);
            // P: [NP / 16 chunks][128 keys][16 columns]
            const uint64_t dp = mn_chunk_desc(smem_u32(smem + C::OFF_P), 128, 2048);
            int x = 0, y = 0;  // next tile of S^T, of P V
            bool ok = true;
            for (int seg = 0; ok; ++seg) {
                ok = mbar_wait(q_ready + (seg & 1), (seg >> 1) & 1, abort_flag);
                const int tiles = ok ? segments[seg & 7].tiles : 0;
                if (tiles == 0) break;
                const int first = y, end = y + tiles;
                uint64_t since = globaltimer_ns();  // of the last issue, as the clock checks see it
                int polls = 0, issued = x + y;
                while (ok && y < end) {
                    if (x < end && x < y + 2 && mbar_test(full_k + x % C::STK, (x / C::STK) & 1)) {
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const int col = PAIR ? (kk >> 1) * (C::NQ / 2) : 0;
                            umma_ss_f8(tmem + (x & 1) * C::NQ + col,
                                       dk + (((x % C::STK) * C::TILE + kk * 32) >> 4),
                                       dq + ((col * 128 + kk * 32) >> 4), idesc_s,
                                       PAIR ? kk & 1 : kk > 0);
                        }
                        umma_commit(s_done + x % C::STK);
                        ++x;
                    }
                    if (y < x && mbar_test(p_ready + (y & 1), (y >> 1) & 1) &&
                        mbar_test(full_v + y % C::STV, (y / C::STV) & 1)) {
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_ss_f8(tmem + 2 * C::NQ,
                                       dv + (((y % C::STV) * C::TILE + kk * 32 * 128) >> 4),
                                       dp + (((y & 1) * (C::NP * 128) + kk * 512) >> 4),
                                       idesc_o,
                                       y > first || kk > 0);
                        umma_commit(o_done + y % C::STV);
                        ++y;
                    }
                    if ((++polls & 63) == 0) {
                        const uint64_t now = globaltimer_ns();
                        if (issued != x + y) {
                            issued = x + y;
                            since = now;
                        }
                        if (now - since > kWaitLimitNs) {
                            raise_device_error(kDevWaitTimeout);
                            *abort_flag = 1;
                        }
                        ok = *abort_flag == 0;
                    }
                }
            }
        }
    } else {
        // ------------------------------------------------------------ consumers
        const int wg = warp >> 2;            // this warpgroup's rows: [R0, R0 + RW)
        const int R0 = wg * RW;
        const int t128 = tid & 127;          // this thread's key of a tile, and its dimension
        // P is [NP / 16 chunks][128 keys][16 columns]: a thread stores its key's columns
        const uint32_t sp = smem_u32(smem + C::OFF_P) + t128 * 16;
        const uint32_t t_s = tmem + (uint32_t((warp & 3) * 32) << 16);  // this warp's lanes
        const uint32_t t_o = t_s + 2 * C::NQ;
        float* red = reinterpret_cast<float*>(smem + C::OFF_RED);
        float* l_max = reinterpret_cast<float*>(misc + 4);  // [wg or half][4] largest normaliser
        float2* const all_rows = reinterpret_cast<float2*>(smem + C::OFF_ROW);
        int2* const all_limits = reinterpret_cast<int2*>(smem + C::OFF_LIM);
        int* const all_next = reinterpret_cast<int*>(smem + C::OFF_TOP);
        int2* const all_out = reinterpret_cast<int2*>(smem + C::OFF_OUT);
        uint32_t* const all_nan = reinterpret_cast<uint32_t*>(smem + C::OFF_NAN);
        float4* const all_vrun = reinterpret_cast<float4*>(smem + C::OFF_VRUN);
        float* so = reinterpret_cast<float*>(smem + C::OFF_P);  // [ROWS][128], P unused
        const int my_half = PAIR ? t128 >> 6 : 0;  // of this thread's dimension
        // the KV heads (of a pair) of this warpgroup's rows: half0 and, with NH = 2, half0 + 1
        constexpr int NH = PAIR && C::WGS == 1 ? 2 : 1;
        const int half0 = PAIR && C::WGS == 2 ? wg : 0;
        auto half_of = [](int r) { return NH == 2 ? r / SUB : 0; };  // of row R0 + r
        int c = 0;
        // After a wait that gave up (device error word set) a warp waits no more, so that all
        // come to the same barriers; what it computes is thrown away.
        bool dead = false;
        bool dry = true;
        auto wait = [&](uint64_t* bar, int phase) {
            if (!dead && !dry) dead = !mbar_wait_warp(bar, phase & 1, abort_flag);
        };
        auto wait_o = [&](int x) { wait(o_done + x % C::STV, x / C::STV); };  // P V of tile x
        int gen = 0;  // which of the two copies of the rows' references and of vrun is in use
        // Writes segment seg's q rows as two e4m3 terms; false: there is none.
        auto stage_q = [&](int seg) {
            const int buf = seg & 1;
            wait(seg_ready + buf, seg >> 1);
            if (consumers_any<CT>(dead)) return false;
            const Kv8Segment& g = segments[seg & 7];
            const bool any = g.tiles > 0;
            if (any) {
                constexpr int D = PAIR ? 64 : 128, MINE = ROWS * 32 / CT;  // rows of a warp
                const uint32_t sq = smem_u32(smem + C::OFF_Q);  // its last S^T has been read
                const int d0 = PAIR ? (lane * 4) & 63 : lane * 4;
                uint2 w[MINE];
#pragma unroll
                for (int j = 0; j < MINE; ++j) {
                    const int r = warp * MINE + j;
                    int i, h;
                    const bool valid = kv8_row<ROWS, PAIR>(p, g.seq, g.hg, g.u, r, i, h);
                    if (lane < 4) all_nan[(buf * ROWS + r) * 4 + lane] = 0u;
                    w[j] = make_uint2(0u, 0u);
                    if (valid && (!PAIR || (lane >> 4) == r / SUB))
                        w[j] = *reinterpret_cast<const uint2*>(
                            p.q + (size_t(g.seq.q0 + i) * p.Hq + h) * D + d0);
                    if (lane == 0) {
                        const int end = g.seq.len - g.seq.n + i + 1;
                        all_limits[buf * ROWS + r] =
                            make_int2(p.window > 0 ? end - p.window : 0, min(end, g.keys.hi));
                        all_next[buf * ROWS + r] = ordered(-INFINITY);
                        all_out[buf * ROWS + r] = make_int2(valid ? i : -1, h);
                    }
                }
#pragma unroll
                for (int j = 0; j < MINE; ++j) {
                    const int r = warp * MINE + j;
                    const uint32_t big =
                        max(max((w[j].x << 16) & 0x7fffffffu, w[j].x & 0x7fff0000u),
                            max((w[j].y << 16) & 0x7fffffffu, w[j].y & 0x7fff0000u));
                    const uint32_t amax = __reduce_max_sync(0xffffffffu, big);
                    // power-of-two factor that brings the row's largest |q| to [128, 256)
                    const int e = max(int(amax >> 23), 8);
                    const float up = __uint_as_float(uint32_t(261 - e) << 23);
                    uint32_t hi, lo;
                    split_e4m3x4(bf16_lo(w[j].x) * up, bf16_hi(w[j].x) * up,
                                 bf16_lo(w[j].y) * up, bf16_hi(w[j].y) * up, 16.f, hi, lo);
                    auto put = [&](int n, uint32_t codes) {  // operand row n, this lane's dims
                        const uint32_t at = (((lane >> 2) ^ (n & 7)) << 4) + (lane & 3) * 4;
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(sq + n * 128 + at),
                                     "r"(codes)
                                     : "memory");
                    };
                    if constexpr (PAIR) {  // (a lane's dimensions are in its head's half)
                        const int col = r / SUB * (C::NQ / 2) + r % SUB;
                        put(col, hi);
                        put(col + SUB, lo);
                    } else {
                        put(r, hi);
                        put(ROWS + r, lo);
                    }
                    // a row with an infinity or a NaN has no factor: its logits are NaN
                    if (lane == 0)
                        all_rows[(buf * 2 + gen) * ROWS + r] = make_float2(
                            amax >= 0x7f800000u
                                ? NAN
                                : __uint_as_float(uint32_t(e - 7) << 23) * p.scale_log2,
                            all_out[buf * ROWS + r].x >= 0 ? kNoKey : kNoRow);
                }
                fence_proxy_async();
            }
            consumers_sync<CT>();
            if (tid == 0) mbar_arrive(q_ready + buf);
            return any;
        };
        // Segment -1 is a dry run of one tile on whatever tensor and shared memory hold, with
        // no waits and nothing handed on: it brings the instructions of a tile into the SM's
        // cache while the first keys are on their way.  Behind other kernels (and a flush of
        // L2), on an event clock of 2 us steps: one sequence of 1000 keys 23.6 -> 21.5 us, of
        // 32768 39.9 -> 37.9, larger batches a step.  In back to back calls, which find the
        // instructions there: windowed batch of 32 42.1 -> 40.1, the other cases 1 to 4 %.
        bool more = true;
        for (int seg = -1; more; ++seg) {
            const Kv8Segment& g = segments[seg & 7];
            const int segment = dry ? 1 : g.tiles;
            const int2* const limits = all_limits + (seg & 1) * ROWS;
            int* const next_ref = all_next + (seg & 1) * ROWS;
            const Kv8Keys keys = g.keys;
            float l[RW];
#pragma unroll
            for (int r = 0; r < RW; ++r) l[r] = 0.f;
            // keys that every row sees, in tiles between which no mask is needed
            const int t0 = dry ? 0 : g.first;
            const int last = g.seq.len - g.seq.n;  // position of query 0
            const int i_lo = g.u * SUB / p.G;
            const int i_hi = min((g.u * SUB + SUB - 1) / p.G, g.seq.n - 1);
            const int all_hi = last + i_lo + 1;
            const int all_lo = p.window > 0 ? max(last + i_hi + 1 - p.window, 0) : 0;
            for (int t = t0; t < t0 + segment; ++t, ++c) {
                const int s = c % C::STV;
                const float2* rows = all_rows + ((seg & 1) * 2 + gen) * ROWS;
                const float4* vrun = all_vrun + gen * 2;
                const int key = t * 128 + t128;
                wait(full_s + s, c / C::STV);
                float4 sc[NH];   // this key's K scale, log2 of its V scale, V scale
                float vref[NH];  // the tile's largest V scale
#pragma unroll
                for (int j = 0; j < NH; ++j) {
                    const float* at = reinterpret_cast<const float*>(smem + C::OFF_SC) + s * 32 +
                                      (half0 + j) * 8;
                    const float4 a = *reinterpret_cast<const float4*>(at + 16);
                    const float4 b = *reinterpret_cast<const float4*>(at + 20);
                    vref[j] = fmaxf(fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)),
                                    fmaxf(fmaxf(b.x, b.y), fmaxf(b.z, b.w)));
                    const float v = at[16 + (t128 >> 4)];
                    sc[j] = make_float4(at[t128 >> 4], __log2f(v), v, 0.f);
                }
                // P's buffer is free once the tile before the last has used it
                if (c >= 2) wait_o(c - 2);
                wait(s_done + c % C::STK, c / C::STK);
                tc_fence_after();
                const bool edge = t * 128 < all_lo || t * 128 + 128 > all_hi;
                const uint32_t t_sc = t_s + (c & 1) * C::NQ;
                const uint32_t sp_c = sp + (c & 1) * (C::NP * 128);
                // logits of rows R0 + r0 .. in log2 units, -inf where not seen
                auto logits = [&](int r0, float (&f)[CH]) {
                    float lo[CH];
                    tmem_ld_logits<ROWS, PAIR, CH>(t_sc, R0 + r0, f, lo);
#pragma unroll
                    for (int j = 0; j < CH; ++j)
                        f[j] = fmaf(lo[j], 0.0625f, f[j]) *
                               (sc[half_of(r0 + j)].x * rows[R0 + r0 + j].x);
                    if (edge) {
#pragma unroll
                        for (int j = 0; j < CH; ++j) {
                            const int2 lim = limits[R0 + r0 + j];
                            if (key < lim.x || key >= lim.y) f[j] = -INFINITY;
                        }
                    }
                };
                // the weights relative to the rows' references: their terms u, and P
                float u[RW];
                // Whether this tile has a V scale far above vrun, so that its references are taken
                // from all of its keys
                bool far = t == t0;
#pragma unroll
                for (int j = 0; j < NH; ++j) far |= vref[j] > vrun[half0 + j].w;
                for (int pass = 0;; ++pass) {
                    bool high = pass == 0;
                    if (pass > 0 || !far) {
                        uint32_t hi[RW / 4], mid[RW / 4], lo[RW / 4];
                        float above[NH], d[NH], g[NH];
#pragma unroll
                        for (int j = 0; j < NH; ++j) {
                            const float4 v = vrun[half0 + j];
                            above[j] = -INFINITY;
                            d[j] = fmaxf(sc[j].y - v.y, kFar);
                            g[j] = sc[j].z * v.z * kTopWeight;
                        }
#pragma unroll
                        for (int r0 = 0; r0 < RW; r0 += CH) {
                            float f[CH];
                            logits(r0, f);
#pragma unroll
                            for (int j = 0; j < CH; j += 4) {
                                float w[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const int r = r0 + j + e, half = half_of(r);
                                    const float x = f[j + e] - rows[R0 + r].y;
                                    above[half] = fmaxf(above[half], x);
                                    u[r] = ex2_approx(x);
                                    w[e] = u[r] * g[half];
                                }
                                const int k = (r0 + j) / 4;
                                split_e5m2x4(w[0], w[1], w[2], w[3], hi[k], mid[k], lo[k]);
                            }
                        }
                        // columns: hi of every row, then mid, then lo
                        if constexpr (RW == 4) {
                            st_shared_v4(sp_c, hi[0], mid[0], lo[0], 0u);
                        } else if constexpr (ROWS == 8) {
                            st_shared_v4(sp_c, hi[0], hi[1], mid[0], mid[1]);
                            st_shared_v2(sp_c + 2048, lo[0], lo[1]);
                        } else if constexpr (RW == 8) {
                            st_shared_v2(sp_c + R0, hi[0], hi[1]);
                            st_shared_v2(sp_c + 2048 + R0, mid[0], mid[1]);
                            st_shared_v2(sp_c + 4096 + R0, lo[0], lo[1]);
                        } else {
                            st_shared_v4(sp_c + wg * 2048, hi[0], hi[1], hi[2], hi[3]);
                            st_shared_v4(sp_c + (2 + wg) * 2048, mid[0], mid[1], mid[2], mid[3]);
                            st_shared_v4(sp_c + (4 + wg) * 2048, lo[0], lo[1], lo[2], lo[3]);
                        }
                        // (the second pass has its tile's own references)
                        high = pass == 0 &&
                               (above[0] + d[0] > 3.f || above[NH - 1] + d[NH - 1] > 3.f);
                    }
                    if (__any_sync(0xffffffffu, high)) {
                        // what this warp's keys ask of the references (next_ref is at -inf)
                        float d[NH];  // relative to what vrun becomes
#pragma unroll
                        for (int j = 0; j < NH; ++j)
                            d[j] = fmaxf(
                                sc[j].y - __log2f(t == t0 ? vref[j]
                                                          : fmaxf(vref[j], vrun[half0 + j].x)),
                                kFar);
                        float top = -INFINITY;  // lane r: the warp's largest z + d of row r
#pragma unroll
                        for (int r0 = 0; r0 < RW; r0 += CH) {
                            float f[CH];
                            logits(r0, f);
#pragma unroll
                            for (int j = 0; j < CH; ++j) {
                                const float mx = warp_max(f[j] + d[half_of(r0 + j)]);
                                if (lane == r0 + j) top = mx;
                            }
                        }
                        if (lane < RW) atomicMax(next_ref + R0 + lane, ordered(top));
                        if (far && t > t0) {
#pragma unroll
                            for (int j = 0; j < NH; ++j) {
                                float x = 0.f;
#pragma unroll
                                for (int r = 0; r < RW; ++r)
                                    if (half_of(r) == j) x = fmaxf(x, l[r]);
                                x = warp_max(x);
                                if (lane == 0) l_max[j * 4 + warp] = x;
                            }
                        }
                    }
                    // V rows that no query sees may hold any code: a weight of 0 times NaN
                    // would still reach O.  In a row that only some see, a NaN is taken out
                    // and noted for those.
                    if (pass == 0 && wg == 0 && !dry && edge) {
                        wait(full_v + s, c / C::STV);
                        uint4* const v = reinterpret_cast<uint4*>(smem + C::OFF_V +
                                                                  s * C::TILE + t128 * 128);
                        if (key < keys.lo || key >= keys.hi) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) v[j] = make_uint4(0u, 0u, 0u, 0u);
                        } else if (key < all_lo || key >= all_hi) {
                            uint32_t any = 0u;
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const uint4 x = v[j];
                                any |= nan_codes(x.x) | nan_codes(x.y) | nan_codes(x.z) |
                                       nan_codes(x.w);
                            }
                            if (any)
                                take_out_nan<ROWS>(reinterpret_cast<uint32_t*>(v), t128, key,
                                                   limits, all_nan + (seg & 1) * ROWS * 4);
                        }
                    }
                    fence_proxy_async();
                    tc_fence_before();
                    if (!consumers_any<CT>(high)) break;
                    if (t > t0) wait_o(c - 1);
                    tc_fence_after();
                    gen ^= 1;
                    float2* const new_rows = all_rows + ((seg & 1) * 2 + gen) * ROWS;
                    float4* const new_vrun = all_vrun + gen * 2;
                    float v[NH], ratio[NH], fall[NH];
#pragma unroll
                    for (int j = 0; j < NH; ++j) {
                        const float v0 = t > t0 ? vrun[half0 + j].x : 0.f;
                        v[j] = fmaxf(vref[j], v0);
                        ratio[j] = v[j] > 0.f ? v0 / v[j] : 0.f;
                        fall[j] = t > t0 && vref[j] > v0 ? __log2f(v[j]) - vrun[half0 + j].y : 0.f;
                        if (far && t > t0) {  // no further than the normaliser has room
                            const float* x = l_max + (wg + j) * 4;
                            const float most = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
                            fall[j] = fminf(fminf(fall[j], 1000.f),
                                            fmaxf(-kFar - __log2f(most), 0.f));
                        }
                    }
                    auto next_of = [&](int r, float fall) {  // of row R0 + r
                        return fmaxf(fmaxf(rows[R0 + r].y - fall, kNoKey),
                                     unordered(next_ref[R0 + r]));
                    };
#pragma unroll
                    for (int r0 = 0; r0 < RW; r0 += CH) {
                        float alpha[CH];
#pragma unroll
                        for (int j = 0; j < CH; ++j) {
                            const int r = r0 + j;
                            alpha[j] = ex2_approx(rows[R0 + r].y - next_of(r, fall[half_of(r)]));
                            l[r] *= alpha[j];
                            alpha[j] *= ratio[half_of(r)];
                        }
                        if (t > t0) OutTerms<ROWS, CH>::scale(t_o, R0 + r0, alpha);
                    }
                    if (t128 < RW)
                        new_rows[R0 + t128] =
                            make_float2(rows[R0 + t128].x,
                                        next_of(t128, half_of(t128) ? fall[NH - 1] : fall[0]));
                    if (t128 < NH && (PAIR || wg == 0)) {
                        const float x = t128 ? v[NH - 1] : v[0];
                        new_vrun[half0 + t128] =
                            make_float4(x, __log2f(x), x > 0.f ? 1.f / x : 0.f,
                                        far ? 8.f * x : vrun[half0 + t128].w);
                    }
                    rows = new_rows;
                    vrun = new_vrun;
                    tc_fence_before();
                    consumers_sync<CT>();
                    // (read by all; the next maxima are taken behind another barrier)
                    if (t128 < RW) next_ref[R0 + t128] = ordered(-INFINITY);
                }
                if (tid == 0 && !dry) mbar_arrive(p_ready + (c & 1));
#pragma unroll
                for (int r = 0; r < RW; ++r) l[r] += u[r];
            }
            // --- end of the segment: the next one's q, so that its first S^T can start, then
            // this one's sums over the keys and its rows' results
            if (dry) {
                dry = false;
                c = 0;
                more = stage_q(0);
                continue;
            }
            more = stage_q(seg + 1);
            if (!more) griddep_launch_dependents();
            wait_o(c - 1);
            tc_fence_after();
            const bool lost = consumers_any<CT>(dead);
            const float2* const rows = all_rows + ((seg & 1) * 2 + gen) * ROWS;
            const float unit = all_vrun[gen * 2 + my_half].x;
#pragma unroll
            for (int r0 = 0; r0 < RW; r0 += CH) {
                float o[CH];
                OutTerms<ROWS, CH>::sum(t_o, R0 + r0, o);
#pragma unroll
                for (int j = 0; j < CH; ++j) {  // (so is read back by this thread)
                    so[(R0 + r0 + j) * 128 + t128] = o[j] * unit;
                    float x = l[r0 + j];
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1)
                        x += __shfl_xor_sync(0xffffffffu, x, off);
                    if (lane == 0) red[(R0 + r0 + j) * 4 + (warp & 3)] = x;
                }
            }
            tc_fence_before();
            consumers_sync<CT>();
            const size_t part = size_t(blockIdx.x) * 2 + g.slot;
#pragma unroll 2
            for (int r = R0; r < R0 + RW; ++r) {
                const float4 x = reinterpret_cast<float4*>(red)[r];
                float sum = (x.x + x.y) + (x.z + x.w);
                float acc = so[r * 128 + t128];
                if (all_nan[((seg & 1) * ROWS + r) * 4 + (t128 >> 5)] >> (t128 & 31) & 1u)
                    acc = NAN;
                // a wait gave up (device error word set): an empty result, so that no stale
                // memory is picked up
                if (lost) sum = 0.f, acc = 0.f;
                if (g.slot >= 0) {
                    p.part_o[(part * ROWS + r) * 128 + t128] = acc;
                    if (t128 == 0) p.part_ml[part * ROWS + r] = make_float2(rows[r].y, sum);
                } else {
                    const int2 at = all_out[(seg & 1) * ROWS + r];
                    if (at.x >= 0)
                        kv8_store<ROWS, PAIR>(p, g.seq, g.b, at.x, at.y, r, t128, acc, sum,
                                              rows[r].y);
                }
            }
            consumers_sync<CT>();  // red, the segment's rows and P are free again
            if (tid == 0) mbar_arrive(seg_free + (seg & 1));
        }
    }
    if (warp >= PRODUCER) griddep_launch_dependents();
    tc_fence_before();
    __syncthreads();
    if (warp == PRODUCER + 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// Joins the partials of the items that several teams shared, and writes the rows of items
// that no key reaches.  With reference M = max_s m_s (log2 units): sum = sum_s 2^(m_s - M)
// sum_s, O = sum_s 2^(m_s - M) O_s / sum, L = ln 2 (M + log2 sum).
// blockIdx.x: the one item that this CTA of kv8_decode may have begun and not ended, and
// every gridDim.x-th item's check for keys; blockIdx.y: four of its rows.  Eight warps, two
// to a row; a warp takes eight partials at a time, all loads in flight together (what
// bounds this kernel is latency), with an online rescaling of its own.
constexpr int kCombineWarps = 8;
constexpr int kCombineRows = 4;  // of a CTA
template <int ROWS, bool PAIR>
__global__ void __launch_bounds__(32 * kCombineWarps) kv8_combine(const Kv8DecodeParams p) {
    constexpr int SUB = PAIR ? ROWS / 2 : ROWS;
    constexpr int CR = kCombineRows, WPR = kCombineWarps / CR;
    __shared__ __align__(16) float so[kCombineWarps][128];
    __shared__ float2 sml[kCombineWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r0 = blockIdx.y * CR;
    griddep_wait();
    const int4 cut = p.cut[2 * blockIdx.x], of = p.cut[2 * blockIdx.x + 1];
    if (cut.x >= 0) {
        const int b = cut.x, hg = cut.y, u = cut.z, parts = cut.w >> 1;
        const Kv8Seq seq = {of.x, of.y, of.z};
        const int r = r0 + warp / WPR;
        float m = kNoKey, sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
        for (int x0 = warp % WPR; x0 < parts; x0 += 8 * WPR) {
            float2 ml[8];
            float4 o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int x = x0 + j * WPR;
                ml[j] = make_float2(kNoKey, 0.f);
                o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (x < parts) {
                    const size_t at = (size_t(blockIdx.x + x * p.width) * 2 +
                                       (x == 0 ? cut.w & 1 : 0)) * ROWS + r;
                    ml[j] = p.part_ml[at];
                    o[j] = reinterpret_cast<const float4*>(p.part_o + at * 128)[lane];
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float m1 = fmaxf(m, ml[j].x);
                const float a = ex2_approx(m - m1), f = ex2_approx(ml[j].x - m1);
                m = m1;
                sum = sum * a + f * ml[j].y;
                acc[0] = acc[0] * a + f * o[j].x;
                acc[1] = acc[1] * a + f * o[j].y;
                acc[2] = acc[2] * a + f * o[j].z;
                acc[3] = acc[3] * a + f * o[j].w;
            }
        }
        reinterpret_cast<float4*>(so[warp])[lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        if (lane == 0) sml[warp] = make_float2(m, sum);
        __syncthreads();
        for (int x = tid; x < CR * 128; x += 32 * kCombineWarps) {
            const int row = x >> 7, dim = x & 127;
            int i, h;
            if (!kv8_row<ROWS, PAIR>(p, seq, hg, u, r0 + row, i, h)) continue;
            float M = kNoKey, total = 0.f, out = 0.f;
#pragma unroll
            for (int w = 0; w < WPR; ++w) M = fmaxf(M, sml[row * WPR + w].x);
#pragma unroll
            for (int w = 0; w < WPR; ++w) {
                const float f = ex2_approx(sml[row * WPR + w].x - M);
                total += f * sml[row * WPR + w].y;
                out += f * so[row * WPR + w][dim];
            }
            kv8_store<ROWS, PAIR>(p, seq, b, i, h, r0 + row, dim, out, total, M);
        }
    }
    const int items = p.B * p.groups * p.units;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int bh = item / p.units, u = item - bh * p.units;
        const int b = bh / p.groups, hg = bh - b * p.groups;
        const Kv8Seq seq = kv8_seq(p, b);
        if (kv8_keys<SUB>(p, seq, u).tiles() > 0) continue;
        for (int x = tid; x < CR * 128; x += 32 * kCombineWarps) {
            const int row = r0 + (x >> 7);
            int i, h;
            if (kv8_row<ROWS, PAIR>(p, seq, hg, u, row, i, h))
                kv8_store<ROWS, PAIR>(p, seq, b, i, h, row, x & 127, 0.f, 0.f, kNoKey);
        }
    }
}

}  // namespace gqa
