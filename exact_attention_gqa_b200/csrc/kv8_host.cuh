// Host side of the 8-bit paged cache's entry points declared in include/gqa_attn.h
// (gqa_attn_kv_tables, gqa_attn_kv8_append, gqa_attn_kv8_gather, gqa_attn_kv8_decode).
// Uses the argument checks and the device table of gqa_attn.cu.
#pragma once
#include "kv8_decode.cuh"

namespace {

bool pow2_at_least(int x, int least) { return x >= least && (x & (x - 1)) == 0; }

// The pool's shape: pages, tokens per page and per scale block, heads and head dimension.
int check_pool(int num_pages, int page_size, int scale_block, int Hkv, int D) {
    if (Hkv <= 0 || num_pages < 1 || !pow2_at_least(page_size, 16) ||
        !pow2_at_least(scale_block, 16) || scale_block > page_size)
        return GQA_ERR_SHAPE;
    if (D != 64 && D != 128) return GQA_ERR_HEADDIM;
    if ((long long)num_pages * page_size > INT32_MAX || (long long)Hkv * D > (1 << 24))
        return GQA_ERR_SHAPE;
    return GQA_OK;
}

constexpr int kTablesMaxRequests = 16384;  // two ints of shared memory each

}  // namespace

extern "C" {

int gqa_attn_kv_tables(const int* cached_lens, const int* new_lens, const int* free_pages,
                       const int* free_start, int* block_table, int* slot_map, int* seqlens_k,
                       int* cu_seqlens_q, int* cu_seqlens_k, int* free_end, int B, int n_free,
                       int max_pages, int page_size, int max_tokens, cudaStream_t stream) {
    if (B < 0 || B > kTablesMaxRequests || n_free < 0 || max_pages < 0 || max_tokens < 0 ||
        !pow2_at_least(page_size, 16) || (long long)max_pages * page_size > INT32_MAX ||
        (B > 0 && max_pages < 1))
        return GQA_ERR_SHAPE;
    if (!cu_seqlens_q || !cu_seqlens_k || !free_end || (max_tokens > 0 && !slot_map) ||
        (n_free > 0 && !free_pages) ||
        (B > 0 && (!cached_lens || !new_lens || !block_table || !seqlens_k)))
        return GQA_ERR_NULL;
    for (const int* x : {cached_lens, new_lens, free_pages, free_start,
                         static_cast<const int*>(block_table), static_cast<const int*>(slot_map),
                         static_cast<const int*>(seqlens_k),
                         static_cast<const int*>(cu_seqlens_q),
                         static_cast<const int*>(cu_seqlens_k),
                         static_cast<const int*>(free_end)})
        if (!aligned(x, 4)) return GQA_ERR_ALIGN;
    if (free_start == free_end) return GQA_ERR_SHAPE;  // read by every CTA, written by one
    DeviceInfo* dev = nullptr;
    int rc = device_info(&dev);
    if (rc != GQA_OK) return rc;
    gqa::KvTablesParams p;
    p.cached_lens = cached_lens;
    p.new_lens = new_lens;
    p.free_pages = free_pages;
    p.free_start = free_start;
    p.block_table = block_table;
    p.slot_map = slot_map;
    p.seqlens_k = seqlens_k;
    p.cu_seqlens_q = cu_seqlens_q;
    p.cu_seqlens_k = cu_seqlens_k;
    p.free_end = free_end;
    p.B = B;
    p.n_free = n_free;
    p.max_pages = max_pages;
    p.page_shift = log2_exact(page_size);
    p.max_tokens = max_tokens;
    const int smem = 2 * (B + 1) * int(sizeof(int));
    rc = ensure_smem_limit(gqa::kv_tables, 1 << 19,
                           2 * (kTablesMaxRequests + 1) * int(sizeof(int)));
    if (rc != GQA_OK) return rc;
    const int want = (max_tokens + gqa::kTablesThreads - 1) / gqa::kTablesThreads;
    const int grid = std::max(1, std::min(want, dev->sms));
    gqa::kv_tables<<<grid, gqa::kTablesThreads, smem, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

int gqa_attn_kv8_append(const void* k, const void* v, const int* slot_map, void* k8, void* v8,
                        float* k_scale, float* v_scale, int T, int Hkv, int D,
                        long long k_stride, long long v_stride, int num_pages, int page_size,
                        int scale_block, cudaStream_t stream) {
    const int rc = check_pool(num_pages, page_size, scale_block, Hkv, D);
    if (rc != GQA_OK) return rc;
    if (T < 0 || k_stride < 0 || v_stride < 0) return GQA_ERR_SHAPE;
    if (T == 0) return GQA_OK;
    if (!k || !v || !slot_map || !k8 || !v8 || !k_scale || !v_scale) return GQA_ERR_NULL;
    if (T > 1 && (k_stride < (long long)Hkv * D || v_stride < (long long)Hkv * D))
        return GQA_ERR_SHAPE;  // rows that overlap
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k8, 16) || !aligned(v8, 16) ||
        !aligned(slot_map, 4) || !aligned(k_scale, 4) || !aligned(v_scale, 4) ||
        k_stride % 8 != 0 || v_stride % 8 != 0)
        return GQA_ERR_ALIGN;
    const long long grid = ((long long)T * Hkv + 7) / 8;
    if (grid > INT32_MAX) return GQA_ERR_SHAPE;
    DeviceInfo* dev = nullptr;
    const int drc = device_info(&dev);
    if (drc != GQA_OK) return drc;
    gqa::Kv8AppendParams p;
    p.k = {static_cast<const __nv_bfloat16*>(k), k_stride, static_cast<uint8_t*>(k8), k_scale};
    p.v = {static_cast<const __nv_bfloat16*>(v), v_stride, static_cast<uint8_t*>(v8), v_scale};
    p.slot_map = slot_map;
    p.T = T;
    p.Hkv = Hkv;
    p.sb_shift = log2_exact(scale_block);
    p.slots = num_pages * page_size;
    const dim3 g(static_cast<unsigned>(grid), 2);
    if (D == 128)
        gqa::kv8_append<128><<<g, 256, 0, stream>>>(p);
    else
        gqa::kv8_append<64><<<g, 256, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

int gqa_attn_kv8_gather(const void* k8, const void* v8, const float* k_scale,
                        const float* v_scale, const int* block_table, const int* cu_seqlens_k,
                        void* k, void* v, int B, int total, int Hkv, int D, int num_pages,
                        int page_size, int max_pages, int scale_block, cudaStream_t stream) {
    const int rc = check_pool(num_pages, page_size, scale_block, Hkv, D);
    if (rc != GQA_OK) return rc;
    if (B < 0 || total < 0 || max_pages < 1 || (long long)max_pages * page_size > INT32_MAX)
        return GQA_ERR_SHAPE;
    if (B == 0 || total == 0) return GQA_OK;
    if (!k8 || !v8 || !k_scale || !v_scale || !block_table || !cu_seqlens_k || !k || !v)
        return GQA_ERR_NULL;
    if (!aligned(k8, 16) || !aligned(v8, 16) || !aligned(k, 16) || !aligned(v, 16) ||
        !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(block_table, 4) ||
        !aligned(cu_seqlens_k, 4))
        return GQA_ERR_ALIGN;
    DeviceInfo* dev = nullptr;
    const int drc = device_info(&dev);
    if (drc != GQA_OK) return drc;
    gqa::Kv8GatherParams p;
    p.k = {static_cast<const uint8_t*>(k8), k_scale, static_cast<__nv_bfloat16*>(k)};
    p.v = {static_cast<const uint8_t*>(v8), v_scale, static_cast<__nv_bfloat16*>(v)};
    p.block_table = block_table;
    p.cu_seqlens_k = cu_seqlens_k;
    p.B = B;
    p.total = total;
    p.Hkv = Hkv;
    p.D = D;
    p.num_pages = num_pages;
    p.page_shift = log2_exact(page_size);
    p.sb_shift = log2_exact(scale_block);
    p.max_pages = max_pages;
    const dim3 g((total + gqa::kGatherRows - 1) / gqa::kGatherRows, 2);
    gqa::kv8_gather<<<g, 256, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

size_t gqa_attn_kv8_decode_workspace_bytes(int B, int Sq, int Hq, int Hkv, int D) {
    (void)B, (void)Sq, (void)Hq, (void)Hkv, (void)D;
    return 0;
}

int gqa_attn_kv8_decode(const void* q, const void* k8, const void* v8, const float* k_scale,
                        const float* v_scale, const int* block_table, const int* seqlens_k,
                        const int* cu_seqlens_q, void* out, float* lse, void* workspace,
                        size_t workspace_bytes, int B, int Sq, int total_q, int Hq, int Hkv,
                        int D, int num_pages, int page_size, int max_pages, int scale_block,
                        float scale, int window, cudaStream_t stream) {
    int rc = check_pool(num_pages, page_size, scale_block, Hkv, D);
    if (rc != GQA_OK) return rc;
    if (B < 0 || Sq < 0 || total_q < 0 || window < 0 || max_pages < 1 ||
        (long long)max_pages * page_size > INT32_MAX)
        return GQA_ERR_SHAPE;
    rc = check_shape(B, Hq, Hkv, Sq, 0, D, scale, 1, -1, cu_seqlens_q != nullptr, false);
    if (rc != GQA_OK) return rc;
    if (B == 0 || Sq == 0 || (cu_seqlens_q && total_q == 0)) return GQA_OK;
    if (!q || !k8 || !v8 || !k_scale || !v_scale || !block_table || !seqlens_k || !out || !lse)
        return GQA_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k8, 16) || !aligned(v8, 16) || !aligned(out, 16) ||
        !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(block_table, 4) ||
        !aligned(seqlens_k, 4) || !aligned(cu_seqlens_q, 4) || !aligned(lse, 4) ||
        !aligned(workspace, 16))
        return GQA_ERR_ALIGN;
    if (B > 65535 || Sq > 65535) return GQA_ERR_SHAPE;
    if (workspace_bytes < gqa_attn_kv8_decode_workspace_bytes(B, Sq, Hq, Hkv, D))
        return GQA_ERR_WORKSPACE;
    DeviceInfo* dev = nullptr;
    rc = device_info(&dev);
    if (rc != GQA_OK) return rc;
    gqa::Kv8DecodeParams p;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.out = static_cast<__nv_bfloat16*>(out);
    p.lse = lse;
    p.k8 = static_cast<const uint8_t*>(k8);
    p.v8 = static_cast<const uint8_t*>(v8);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.block_table = block_table;
    p.seqlens_k = seqlens_k;
    p.cu_seqlens_q = cu_seqlens_q;
    p.B = B;
    p.Sq = Sq;
    p.total_q = total_q;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.num_pages = num_pages;
    p.page_shift = log2_exact(page_size);
    p.sb_shift = log2_exact(scale_block);
    p.max_pages = max_pages;
    p.window = window;
    p.scale_log2 = scale * kLog2e;
    const dim3 g(Hq, Sq, B);
    if (D == 128)
        gqa::kv8_decode_simple<128><<<g, 128, 0, stream>>>(p);
    else
        gqa::kv8_decode_simple<64><<<g, 128, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

}  // extern "C"
