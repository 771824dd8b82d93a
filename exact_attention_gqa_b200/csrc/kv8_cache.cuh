// The 8-bit paged KV cache with a scale for each block of tokens and head: its tables,
// its writer and its reader back to bf16 (the attention over it is kv8_decode.cuh).
//
// A stored value is code * scale, the code in e4m3 and the scale a power of two.  A power
// of two loses nothing against a free scale, because e4m3 is a floating-point format: its
// relative step does not depend on where in its range a value lies.  What it gains: x / s
// is exact, so a code is x rounded once, and when a block's scale grows by 2^n its codes
// are divided by 2^n exactly, apart from the bits that fall below the subnormal step.  So
// tokens can be written one at a time into a block without their error adding up.
#pragma once
#include "decode.cuh"

namespace gqa {

constexpr int kDevNoPages = 4;  // the free pages ran out, or a row of the block table did

struct KvTablesParams {
    const int* cached_lens;  // [B]
    const int* new_lens;     // [B]
    const int* free_pages;   // [n_free]
    const int* free_start;   // [1] or null (0)
    int* block_table;        // [B, max_pages]
    int* slot_map;           // [max_tokens]
    int* seqlens_k;          // [B]
    int* cu_seqlens_q;       // [B + 1]
    int* cu_seqlens_k;       // [B + 1]
    int* free_end;           // [1]
    int B, n_free, max_pages, page_shift, max_tokens;
};

__device__ __forceinline__ int sat_i32(long long x) {
    return x > INT32_MAX ? INT32_MAX : int(x);
}

// Index of the last entry of the non-decreasing cu[0..n] that is <= x, below n (0 <= x <
// cu[n]): the sequence that owns packed row x.
template <typename Ptr>
__device__ __forceinline__ int owner_of(Ptr cu, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= x)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Block table rows, slot map and prefix sums from the request lengths.  Every CTA repeats
// the scan over the B requests (two loads and a block scan, so no CTA waits for another
// and one launch does it all) and then takes its share of the slots and of the pages.
constexpr int kTablesThreads = 512;
__global__ void __launch_bounds__(kTablesThreads) kv_tables(const KvTablesParams p) {
    extern __shared__ int sm_tables[];
    int* cu_q = sm_tables;          // [B + 1] new tokens before request b
    int* pg = sm_tables + p.B + 1;  // [B + 1] new pages before request b
    __shared__ long long warp_sum[3][kTablesThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ps = 1 << p.page_shift;
    griddep_launch_dependents();
    griddep_wait();
    const long long cap = (long long)p.max_pages << p.page_shift;
    const int per = (p.B + kTablesThreads - 1) / kTablesThreads;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    auto lengths = [&](int b, int& had, int& add) {
        had = p.cached_lens[b];
        add = p.new_lens[b];
        if (had < 0 || add < 0 || (long long)had + add > cap) {
            raise_device_error(kDevNoPages);
            had = int(min((long long)max(had, 0), cap));
            add = int(min((long long)max(add, 0), cap - had));
        }
    };
    long long sum[3] = {0, 0, 0};  // new tokens, new pages, tokens
    for (int b = b0; b < b1; ++b) {
        int had, add;
        lengths(b, had, add);
        sum[0] += add;
        sum[1] += ((long long)had + add + ps - 1) / ps - ((long long)had + ps - 1) / ps;
        sum[2] += (long long)had + add;
    }
    long long inc[3] = {sum[0], sum[1], sum[2]};
#pragma unroll
    for (int off = 1; off < 32; off <<= 1)
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const long long o = __shfl_up_sync(0xffffffffu, inc[i], off);
            if (lane >= off) inc[i] += o;
        }
    if (lane == 31)
        for (int i = 0; i < 3; ++i) warp_sum[i][warp] = inc[i];
    __syncthreads();
    long long at[3];
    for (int i = 0; i < 3; ++i) {
        at[i] = inc[i] - sum[i];
        for (int w = 0; w < warp; ++w) at[i] += warp_sum[i][w];
    }
    const bool first = blockIdx.x == 0;
    for (int b = b0; b < b1; ++b) {
        int had, add;
        lengths(b, had, add);
        cu_q[b] = sat_i32(at[0]);
        pg[b] = sat_i32(at[1]);
        if (first) {
            p.cu_seqlens_q[b] = sat_i32(at[0]);
            p.cu_seqlens_k[b] = sat_i32(at[2]);
            p.seqlens_k[b] = had + add;
        }
        at[0] += add;
        at[1] += ((long long)had + add + ps - 1) / ps - ((long long)had + ps - 1) / ps;
        at[2] += (long long)had + add;
    }
    const int start = p.free_start ? max(*p.free_start, 0) : 0;
    if (p.B == 0 ? tid == 0 : b0 < p.B && b1 == p.B) {  // the thread with the last request
        cu_q[p.B] = sat_i32(at[0]);
        pg[p.B] = sat_i32(at[1]);
        if (first) {
            p.cu_seqlens_q[p.B] = sat_i32(at[0]);
            p.cu_seqlens_k[p.B] = sat_i32(at[2]);
            *p.free_end = sat_i32(start + at[1]);
            if (start + at[1] > p.n_free || at[0] > p.max_tokens)
                raise_device_error(kDevNoPages);
        }
    }
    __syncthreads();
    const int tokens = cu_q[p.B], pages = pg[p.B];
    auto free_page = [&](long long f) { return f < p.n_free ? p.free_pages[f] : -1; };
    // (unsigned: one stride past the largest count is more than an int holds)
    const unsigned stride = gridDim.x * kTablesThreads;
    for (unsigned f = blockIdx.x * kTablesThreads + tid; f < unsigned(pages); f += stride) {
        const int b = owner_of(pg, p.B, f);
        int had, add;
        lengths(b, had, add);
        p.block_table[size_t(b) * p.max_pages + (had + ps - 1) / ps + (int(f) - pg[b])] =
            free_page((long long)start + f);
    }
    for (unsigned t = blockIdx.x * kTablesThreads + tid; t < unsigned(p.max_tokens);
         t += stride) {
        int slot = -1;
        if (t < unsigned(tokens)) {
            const int b = owner_of(cu_q, p.B, t);
            int had, add;
            lengths(b, had, add);
            const int pos = had + (int(t) - cu_q[b]);
            const int lp = pos >> p.page_shift, lp0 = (had + ps - 1) / ps;
            // a page of the cached tokens is in the table already; a new one is not read
            // back from there, because another CTA may be about to write it
            const long long f = (long long)start + pg[b] + (lp - lp0);
            const bool cached = lp < lp0;
            const int page =
                cached ? p.block_table[size_t(b) * p.max_pages + lp] : free_page(f);
            const long long at = ((long long)page << p.page_shift) + (pos & (ps - 1));
            if (page >= 0 && at <= INT32_MAX)
                slot = int(at);
            else if (cached || f < p.n_free)  // not merely short of pages: no pool has this one
                raise_device_error(kDevBadKvIndex);
        }
        p.slot_map[t] = slot;
    }
}

// ------------------------------------------------------------------------------ append
struct Kv8AppendParams {
    struct Side {
        const __nv_bfloat16* x;  // new keys or values, rows of Hkv * D
        long long stride;        // elements from one token to the next
        uint8_t* codes;          // [num_pages * page_size, Hkv, D]
        float* scale;            // [num_pages * page_size / sb, Hkv]
    };
    Side k, v;
    const int* slot_map;  // [T]
    int T, Hkv, sb_shift;
    int slots;  // num_pages * page_size
    int wide;   // warps that share a long run (a power of two, 8 at most)
};

// The smallest power of two s, at least 2^-126, with a <= 448 s (448 = 1.75 * 2^8); a is
// finite and >= 0.
__device__ __forceinline__ float pow2_scale(float a) {
    const uint32_t u = __float_as_uint(a);
    const int e = int(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float(uint32_t(max(e, -126) + 127) << 23);
}

constexpr float kBf16Max = 3.3895313892515355e38f;

// The larger of each half of a and |x| of eight bf16, as two bf16 (the maximum passes over
// NaN).
__device__ __forceinline__ uint32_t amax8(const uint4& x, uint32_t a) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("max.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(w[i] & 0x7fff7fffu));
    return a;
}

// eight bf16 times inv -> eight e4m3 codes (rounded to nearest even, saturating)
__device__ __forceinline__ uint2 encode8(const uint4& x, float inv) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    const uint64_t inv2 = f2_pack(inv, inv);
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f2_unpack(fmul2(f2_pack(bf16_lo(w[i]), bf16_hi(w[i])), inv2), f[2 * i], f[2 * i + 1]);
    return make_uint2(pack_e4m3x4(f[0], f[1], f[2], f[3]), pack_e4m3x4(f[4], f[5], f[6], f[7]));
}

// four codes -> four fp32 (exact)
__device__ __forceinline__ void decode4(uint32_t c, float (&f)[4]) {
    uint32_t lo, hi;
    e4m3x4_to_f16x4(c, lo, hi);
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(f[0]), "=f"(f[1])
        : "r"(lo));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(f[2]), "=f"(f[3])
        : "r"(hi));
}

// A run is the tokens of one scale block; its first token is its leader.  blockIdx.x takes
// the leaders among 32 tokens, and its gridDim.y CTAs share the tasks (leader, K or V, head;
// heads next to each other, as they are in memory).  A warp reads its rows of a task once,
// into registers (four 16-byte loads a lane); a run of no more rows than that is one warp's
// task, and if the 32 tokens hold a longer run, `wide` warps share each task (rows beyond
// what they hold are read twice).
// Bound: for prompts HBM by its bytes (2 in, 1 out an element), in fact the instructions and
// the trips to memory before a run's loads (slots, then rows); latency for a decode step.
// Measured (8 heads, D 128): 4 prompts of up to 8192 tokens, blocks of 64, 51.7 us, 3.9 TB/s;
// a step of 64 tokens 2.9 us.  Two CTAs an SM instead of four: 72.4 and 2.9 us; two with
// eight held loads: 51.2 and 3.3, but 90.7 instead of 66.3 in blocks of 256 and 23.7 instead
// of 17.0 for 2048 single tokens.
constexpr int kAppendHeld = 4;  // 16-byte loads of a lane
static_assert((kAppendHeld & (kAppendHeld - 1)) == 0, "`wide` must divide a CTA's warps");
template <int D>
__global__ void __launch_bounds__(256, 4) kv8_append(const Kv8AppendParams p) {
    constexpr int LPR = D / 8;       // lanes of one row, eight elements each
    constexpr int RPW = 32 / LPR;    // rows a warp handles at a time
    constexpr int HELD = kAppendHeld;
    __shared__ float sm_amax[2][8];
    __shared__ int sm_restart[2][8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t0 = blockIdx.x * 32;
    griddep_wait();
    const int sb = 1 << p.sb_shift;
    auto block_of = [&](int t) {  // token t's scale block, -1: none
        if (t < 0 || t >= p.T) return -1;
        const int s = p.slot_map[t];
        return s >= 0 && s < p.slots ? s >> p.sb_shift : -1;
    };
    const int mine = block_of(t0 + lane), after = block_of(t0 + 32 + lane);
    int before = block_of(t0 - 1);
    if (blockIdx.y == 0 && warp == 0 && mine < 0 && t0 + lane < p.T &&
        p.slot_map[t0 + lane] != -1)
        raise_device_error(kDevBadKvIndex);
    const int left = __shfl_up_sync(0xffffffffu, mine, 1);
    if (lane > 0) before = left;
    const uint32_t starts = __ballot_sync(0xffffffffu, mine != before);
    const uint32_t leaders = __ballot_sync(0xffffffffu, mine >= 0 && mine != before);
    if (leaders == 0) return;
    // the runs' lengths: up to the next start, the last one's maybe beyond these 32
    const uint32_t later = lane < 31 ? starts >> (lane + 1) << (lane + 1) : 0u;
    int my_n = (leaders >> lane & 1) ? (later ? __ffs(later) - 1 : 32) - lane : 0;
    const int last = 31 - __clz(leaders);
    if (__shfl_sync(0xffffffffu, later, last) == 0) {
        const int blk = __shfl_sync(0xffffffffu, mine, last);
        int n = 0, next = after;
        while (true) {
            const uint32_t in = __ballot_sync(0xffffffffu, next == blk);
            if (in != 0xffffffffu) {
                n += __ffs(~in) - 1;
                break;
            }
            n += 32;
            next = block_of(t0 + 32 + n + lane);
        }
        if (lane == last) my_n += n;
    }
    const int longest = __reduce_max_sync(0xffffffffu, my_n);
    const int team = longest > HELD * RPW ? p.wide : 1;  // warps of a task
    const int teams = 8 / team, my_team = warp / team, wi = warp - my_team * team;
    const int tasks = __popc(leaders) * 2 * p.Hkv;
    const int r = wi * RPW + lane / LPR, c = lane % LPR, step = team * RPW;
    const size_t row = size_t(p.Hkv) * D;
    int parity = 0;
    struct Task {
        const __nv_bfloat16* x;  // this lane's elements of the run's first row
        long long stride;
        float* scale;
        uint8_t* codes;          // and of the block's first
        int t, n;                // the run
        float s0;                // the block's scale before
        uint4 held[HELD];
        int at[HELD];            // the rows' positions in the block
    };
    auto load = [&](const Task& k, int i) {
        return *reinterpret_cast<const uint4*>(k.x + (long long)i * k.stride);
    };
    auto fetch = [&](Task& k, int task) {
        const int which = task / p.Hkv, h = task - which * p.Hkv;
        const Kv8AppendParams::Side& io = which & 1 ? p.v : p.k;
        const int l = __fns(leaders, 0, (which >> 1) + 1);  // the leader's lane
        const int blk = __shfl_sync(0xffffffffu, mine, l);
        k.n = __shfl_sync(0xffffffffu, my_n, l);
        k.t = t0 + l;
        k.stride = io.stride;
        k.x = io.x + (long long)k.t * io.stride + h * D + c * 8;
        k.scale = io.scale + (size_t(blk) * p.Hkv + h);
        k.codes = io.codes + (size_t(blk) << p.sb_shift) * row + h * D + c * 8;
        k.s0 = *k.scale;
#pragma unroll
        for (int j = 0; j < HELD; ++j) {
            const int i = r + j * step;
            k.held[j] = make_uint4(0u, 0u, 0u, 0u);
            k.at[j] = 1;
            if (i < k.n) {
                k.held[j] = load(k, i);
                k.at[j] = p.slot_map[k.t + i];
            }
        }
    };
    auto finish = [&](const Task& k) {
        uint32_t a2 = 0u;
        bool restart = false;
#pragma unroll
        for (int j = 0; j < HELD; ++j) {
            a2 = amax8(k.held[j], a2);
            restart |= (k.at[j] & (sb - 1)) == 0;
        }
        for (int i = r + HELD * step; i < k.n; i += step) {
            a2 = amax8(load(k, i), a2);
            restart |= (p.slot_map[k.t + i] & (sb - 1)) == 0;
        }
        // (bits of numbers >= 0 order as the numbers do)
        float a = __uint_as_float(__reduce_max_sync(0xffffffffu, max(a2 << 16, a2 & 0xffff0000u)));
        restart = __any_sync(0xffffffffu, restart);
        if (team > 1) {
            if (lane == 0) {
                sm_amax[parity][warp] = a;
                sm_restart[parity][warp] = restart;
            }
            // (every warp has read the old scale before the first writes the new one)
            asm volatile("bar.sync %0, %1;" ::"r"(my_team + 1), "r"(team * 32) : "memory");
            for (int w = my_team * team; w < (my_team + 1) * team; ++w) {
                a = fmaxf(a, sm_amax[parity][w]);
                restart |= sm_restart[parity][w] != 0;
            }
            parity ^= 1;
        }
        float s = pow2_scale(fminf(a, kBf16Max));  // infinity: the largest finite value
        // a scale that no append wrote (not finite, not positive) holds nothing to keep
        if (!restart && k.s0 > 0.f && k.s0 < INFINITY) {
            const uint32_t u = __float_as_uint(k.s0);
            const float up = (u & 0x7fffffu) ? __uint_as_float(((u >> 23) + 1) << 23) : k.s0;
            s = fmaxf(s, fminf(fmaxf(up, 1.1754943508222875e-38f), 1.7014118346046923e38f));
            if (s != k.s0) {
                const float f = k.s0 / s;
                for (int i = r; i < sb; i += step) {
                    bool now = false;  // written by this call
                    for (int j = 0; j < k.n; ++j)
                        now |= (p.slot_map[k.t + j] & (sb - 1)) == i;
                    if (now) continue;
                    uint2* d = reinterpret_cast<uint2*>(k.codes + i * row);
                    const uint2 o = *d;
                    float y[4], z[4];
                    decode4(o.x, y);
                    decode4(o.y, z);
                    *d = make_uint2(pack_e4m3x4(y[0] * f, y[1] * f, y[2] * f, y[3] * f),
                                    pack_e4m3x4(z[0] * f, z[1] * f, z[2] * f, z[3] * f));
                }
            }
        }
        if (lane == 0 && wi == 0) *k.scale = s;
        const float inv = 1.f / s;
#pragma unroll
        for (int j = 0; j < HELD; ++j)
            if (r + j * step < k.n)
                *reinterpret_cast<uint2*>(k.codes + (k.at[j] & (sb - 1)) * row) =
                    encode8(k.held[j], inv);
        for (int i = r + HELD * step; i < k.n; i += step) {
            const int off = p.slot_map[k.t + i] & (sb - 1);
            *reinterpret_cast<uint2*>(k.codes + off * row) = encode8(load(k, i), inv);
        }
    };
    for (int task = blockIdx.y * teams + my_team; task < tasks; task += gridDim.y * teams) {
        Task k;
        fetch(k, task);
        finish(k);
    }
}

// ------------------------------------------------------------------------------ gather
struct Kv8GatherParams {
    struct Side {
        const uint8_t* codes;
        const float* scale;
        __nv_bfloat16* out;  // [total, Hkv, D]
    };
    Side k, v;
    const int* block_table;   // [B, max_pages]
    const int* cu_seqlens_k;  // [B + 1]
    int B, total, Hkv, D, num_pages, page_shift, sb_shift, max_pages;
};

// kGatherRows packed rows of K or V (blockIdx.y) per CTA: their source rows are looked up
// once, then every thread converts 8 elements at a time (so that a warp's stores are whole
// 512-byte pieces), eight loads in flight.
// Bound: HBM by its bytes (1 in, 2 out an element).  Measured: 4 sequences of up to 8192
// tokens, 8 heads, D 128, 19.5 us a pass over several states, 6.0 TB/s.  A single launch of
// that size leaves most of what it writes in L2 and takes 21 us, with DRAM a third busy and
// half of the issue slots used: there it is the trips to memory and the instructions.
constexpr int kGatherRows = 32;
__global__ void __launch_bounds__(256) kv8_gather(const Kv8GatherParams p) {
    static_assert(kGatherRows % 32 == 0, "whole warps look the rows up");
    __shared__ int src[kGatherRows];  // row of the pool, -1: none
    const int row0 = blockIdx.x * kGatherRows;
    griddep_wait();
    if (threadIdx.x < kGatherRows) {
        const int t = row0 + threadIdx.x;
        int s = -1;
        int b = 0, first = 0, end;
        if (p.B <= 32) {  // the lanes hold the prefix sums: one load, five steps of registers
            const int lane = threadIdx.x & 31;
            const int cu = p.cu_seqlens_k[min(lane, p.B - 1)];
            end = p.cu_seqlens_k[p.B];
#pragma unroll
            for (int step = 16; step > 0; step >>= 1) {
                const int at = __shfl_sync(0xffffffffu, cu, min(b + step, 31));
                if (b + step < p.B && at <= t) b += step;
            }
            first = __shfl_sync(0xffffffffu, cu, b);
        } else {
            end = p.cu_seqlens_k[p.B];
            b = owner_of(p.cu_seqlens_k, p.B, t);
            first = p.cu_seqlens_k[b];
        }
        if (t < p.total && t < end) {
            const int pos = t - first;
            const int lp = pos >> p.page_shift;
            int page = (pos >= 0 && lp < p.max_pages)
                           ? p.block_table[size_t(b) * p.max_pages + lp]
                           : -1;
            if (page < 0 || page >= p.num_pages) {
                raise_device_error(kDevBadKvIndex);
                page = 0;
            }
            s = (page << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
        }
        src[threadIdx.x] = s;
    }
    __syncthreads();
    const Kv8GatherParams::Side& io = blockIdx.y == 0 ? p.k : p.v;
    const uint32_t chunks = uint32_t(p.Hkv) * p.D / 8;  // of one row
    const uint32_t end = kGatherRows * chunks;
    const int per_head = p.D == 128 ? 4 : 3;  // log2 of a head's chunks
    const uint32_t rows_on = 256 / chunks, chunks_on = 256 - rows_on * chunks;
    uint32_t i = threadIdx.x / chunks, c = threadIdx.x - i * chunks;  // this chunk's row, place
    for (uint32_t e0 = threadIdx.x; e0 < end; e0 += 8 * 256) {
        uint2 o[8];
        float f[8];
        uint4* out[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int s = e0 + j * 256 < end ? src[i] : -1;
            out[j] = nullptr;
            if (s >= 0) {
                o[j] = reinterpret_cast<const uint2*>(io.codes + size_t(s) * chunks * 8)[c];
                f[j] = io.scale[size_t(s >> p.sb_shift) * p.Hkv + (c >> per_head)];
                out[j] = reinterpret_cast<uint4*>(io.out + size_t(row0 + i) * chunks * 8) + c;
            }
            i += rows_on;
            c += chunks_on;
            if (c >= chunks) c -= chunks, ++i;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (!out[j]) continue;
            float x[4], y[4];
            decode4(o[j].x, x);
            decode4(o[j].y, y);
            __stcs(out[j], make_uint4(pack_bf16x2(x[0] * f[j], x[1] * f[j]),
                                      pack_bf16x2(x[2] * f[j], x[3] * f[j]),
                                      pack_bf16x2(y[0] * f[j], y[1] * f[j]),
                                      pack_bf16x2(y[2] * f[j], y[3] * f[j])));
        }
    }
}

}  // namespace gqa
