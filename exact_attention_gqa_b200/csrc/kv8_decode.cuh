// Attention of the newest positions of each sequence over the 8-bit paged cache with block
// scales (kv8_cache.cuh).
#pragma once
#include "kv8_cache.cuh"

namespace gqa {

struct Kv8DecodeParams {
    const __nv_bfloat16* q;   // [rows, Hq, D]
    __nv_bfloat16* out;       // like q
    float* lse;               // dense [B, Hq, Sq], packed [Hq, total_q]
    const uint8_t* k8;
    const uint8_t* v8;
    const float* k_scale;     // [num_pages * page_size / sb, Hkv]
    const float* v_scale;
    const int* block_table;   // [B, max_pages]
    const int* seqlens_k;     // [B]
    const int* cu_seqlens_q;  // [B + 1] or null: Sq queries each
    int B, Sq, total_q, Hq, Hkv, G;
    int num_pages, page_shift, sb_shift, max_pages, window;
    float scale_log2;
};

// One CTA per (query head, query, sequence); each of its four warps takes every fourth
// key, with an online softmax of its own, and the four are joined at the end.
template <int D>
__global__ void __launch_bounds__(128) kv8_decode_simple(const Kv8DecodeParams p) {
    constexpr int PER = D / 32;
    const int h = blockIdx.x, i = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int q0 = b * p.Sq, n = p.Sq;
    if (p.cu_seqlens_q) {
        q0 = __ldg(p.cu_seqlens_q + b);
        n = __ldg(p.cu_seqlens_q + b + 1) - q0;
        if (n < 0 || n > p.Sq || q0 < 0 || q0 > p.total_q - n) {
            raise_device_error(kDevBadTile);
            return;
        }
    }
    if (i >= n) return;
    const int cap = p.max_pages << p.page_shift;
    int len = __ldg(p.seqlens_k + b);
    if (len < 0 || len > cap) {
        raise_device_error(kDevBadKvIndex);
        len = min(max(len, 0), cap);
    }
    const int end = max(len - n + i + 1, 0);
    const int start = p.window > 0 ? max(end - p.window, 0) : 0;
    const int kvh = h / p.G;
    const size_t row = size_t(q0 + i) * p.Hq + h;
    float q[PER], o[PER];
    for (int e = 0; e < PER; ++e) {
        q[e] = __bfloat162float(p.q[row * D + lane * PER + e]);
        o[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int j = start + warp; j < end; j += 4) {
        int page = __ldg(p.block_table + size_t(b) * p.max_pages + (j >> p.page_shift));
        if (page < 0 || page >= p.num_pages) {
            raise_device_error(kDevBadKvIndex);
            page = 0;
        }
        const int s = (page << p.page_shift) + (j & ((1 << p.page_shift) - 1));
        const size_t at = (size_t(s) * p.Hkv + kvh) * D + lane * PER;
        const size_t sc = size_t(s >> p.sb_shift) * p.Hkv + kvh;
        float acc = 0.f, x[4];
        uint32_t w = 0;
        for (int e = 0; e < PER; ++e) w |= uint32_t(p.k8[at + e]) << (8 * e);
        decode4(w, x);
        for (int e = 0; e < PER; ++e) acc += q[e] * x[e];
        for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
        const float z = acc * p.k_scale[sc] * p.scale_log2;
        const float m1 = fmaxf(m, z);
        const float alpha = exp2f(m - m1), u = exp2f(z - m1);
        w = 0;
        for (int e = 0; e < PER; ++e) w |= uint32_t(p.v8[at + e]) << (8 * e);
        decode4(w, x);
        const float f = u * p.v_scale[sc];
        for (int e = 0; e < PER; ++e) o[e] = o[e] * alpha + f * x[e];
        l = l * alpha + u;
        m = m1;
    }
    __shared__ float so[4][D], sm[4], sl[4];
    for (int e = 0; e < PER; ++e) so[warp][lane * PER + e] = o[e];
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
    __syncthreads();
    const float M = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    float L = 0.f, acc = 0.f;
    for (int w = 0; w < 4; ++w) {
        const float f = M == -INFINITY ? 0.f : exp2f(sm[w] - M);
        L += f * sl[w];
        if (threadIdx.x < D) acc += f * so[w][threadIdx.x];
    }
    if (threadIdx.x < D)
        p.out[row * D + threadIdx.x] = __float2bfloat16_rn(L > 0.f ? acc / L : 0.f);
    if (threadIdx.x == 0) {
        const size_t at = p.cu_seqlens_q ? size_t(h) * p.total_q + q0 + i
                                         : (size_t(b) * p.Hq + h) * p.Sq + i;
        p.lse[at] = L > 0.f ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
    }
}

}  // namespace gqa
