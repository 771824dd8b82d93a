// Host side of the 8-bit paged cache's entry points declared in include/gqa_attn.h
// (gqa_attn_kv_tables, gqa_attn_kv8_append, gqa_attn_kv8_gather, gqa_attn_kv8_decode).
// Uses the argument checks and the device table of gqa_attn.cu.
#pragma once
#include <type_traits>

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

// The cache as rows of Hkv * D bytes, copied in boxes of 128 bytes (one head of 128
// dimensions or two of 64) by box_rows, 128-byte swizzle.
bool make_map_kv8(CUtensorMap* m, const void* base, long long rows, int width, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {cuuint64_t(width), cuuint64_t(rows)};
    cuuint64_t strides[1] = {cuuint64_t(width)};
    cuuint32_t box[2] = {128u, cuuint32_t(box_rows)};
    cuuint32_t estr[2] = {1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A launch that may begin while the kernel before it in the stream ends: every kernel of
// this file waits for that one (griddep_wait) before it touches global memory, and reads it
// by ordinary loads: read-only ones (__ldg) are for data that nothing writes while the kernel
// is there, and this one may be there while the one before it writes.
template <typename... Params, typename... Args>
int launch_pdl(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t stream,
               const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

// How a kv8 decode's query rows are cut: `rows` per pass (both heads' of a pair at D = 64),
// as few as hold all G * Sq rows of a KV head, 32 at most; then several units.
constexpr int kKv8MaxCtas = 480;
struct Kv8Plan {
    int rows, groups, units;
    long long items;
    size_t off_ml, off_o, bytes;  // workspace: cut items, partial sums, partial outputs
};
Kv8Plan kv8_plan(int B, int Sq, int Hq, int Hkv, int D) {
    Kv8Plan pl;
    const long long sub = (long long)(Hq / Hkv) * Sq;  // rows of one KV head
    const int heads = D == 64 ? 2 : 1;
    pl.rows = 4;
    while (pl.rows < 32 && pl.rows < sub * heads) pl.rows *= 2;
    pl.groups = (Hkv + heads - 1) / heads;
    pl.units = int((sub * heads + pl.rows - 1) / pl.rows);
    pl.items = (long long)B * pl.groups * pl.units;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    pl.off_ml = up(size_t(kKv8MaxCtas) * 32);
    pl.off_o = pl.off_ml + up(size_t(kKv8MaxCtas) * 2 * pl.rows * 8);
    pl.bytes = pl.off_o + size_t(kKv8MaxCtas) * 2 * pl.rows * 128 * 4;
    return pl;
}

constexpr int kAppendShare = 4;
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
    // inputs that every CTA reads and outputs that one writes
    for (const int* in : {cached_lens, new_lens, free_pages, free_start})
        for (const int* out : {slot_map, seqlens_k, cu_seqlens_q, cu_seqlens_k, free_end})
            if (in && in == out) return GQA_ERR_SHAPE;
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
    const long long want = ((long long)max_tokens + gqa::kTablesThreads - 1) / gqa::kTablesThreads;
    const int grid = int(std::max(1ll, std::min<long long>(want, dev->sms)));
    return launch_pdl(gqa::kv_tables, dim3(grid), gqa::kTablesThreads, smem, stream, p);
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
    const int held = gqa::kAppendHeld * 256 / D;  // rows
    p.wide = std::max(1, std::min(8, scale_block / held));
    // CTAs for each 32 tokens: as many as run at a time (four an SM), up to a warp for each
    // (token, K or V, head); for prompts kAppendShare, each with a few tasks then.  2048
    // single tokens: 16.9 us (20.3 with a warp for each task), 4 prompts of up to 8192
    // tokens: 51.9 us (54.9 with 8 CTAs for each 32, 125 with a warp for each task).
    const int windows = (T + 31) / 32;
    const int all = (32 * 2 * Hkv + 7) / 8;
    const int share =
        std::max(std::min(kAppendShare, all), std::min(all, 4 * dev->sms / windows));
    const dim3 g(windows, share);
    return launch_pdl(D == 128 ? gqa::kv8_append<128> : gqa::kv8_append<64>, g, 256, 0, stream, p);
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
    return launch_pdl(gqa::kv8_gather, g, 256, 0, stream, p);
}

size_t gqa_attn_kv8_decode_workspace_bytes(int B, int Sq, int Hq, int Hkv, int D) {
    if (B <= 0 || Sq <= 0 || Hkv <= 0 || Hq <= 0 || Hq % Hkv != 0 || (D != 64 && D != 128))
        return 0;
    return kv8_plan(B, Sq, Hq, Hkv, D).bytes;
}

int gqa_attn_kv8_decode(const void* q, const void* k8, const void* v8, const float* k_scale,
                        const float* v_scale, const int* block_table, const int* seqlens_k,
                        const int* cu_seqlens_q, void* out, float* lse, void* workspace,
                        size_t workspace_bytes, int B, int Sq, int total_q, int Hq, int Hkv,
                        int D, int num_pages, int page_size, int max_pages, int scale_block,
                        float scale, int window, cudaStream_t stream) {
    int rc = check_pool(num_pages, page_size, scale_block, Hkv, D);
    if (rc != GQA_OK) return rc;
    const long long cap = (long long)max_pages * page_size;  // keys a sequence can have
    if (B < 0 || Sq < 0 || Sq > 65535 || total_q < 0 || window < 0 || max_pages < 1 ||
        cap > (1 << 30))
        return GQA_ERR_SHAPE;
    if (window >= cap) window = 0;  // every key
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
    const Kv8Plan pl = kv8_plan(B, Sq, Hq, Hkv, D);
    // tiles of 128 keys, and items' starts, are numbered with 31 bits
    if ((double)pl.items * ((cap + 127) / 128 + gqa::kItemStart) > INT32_MAX)
        return GQA_ERR_SHAPE;
    if (!workspace || workspace_bytes < pl.bytes) return GQA_ERR_WORKSPACE;
    DeviceInfo* dev = nullptr;
    rc = device_info(&dev);
    if (rc != GQA_OK) return rc;
    gqa::Kv8DecodeParams p;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.out = static_cast<__nv_bfloat16*>(out);
    p.lse = lse;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.block_table = block_table;
    p.seqlens_k = seqlens_k;
    p.cu_seqlens_q = cu_seqlens_q;
    char* ws = static_cast<char*>(workspace);
    p.cut = reinterpret_cast<int4*>(ws);
    p.part_ml = reinterpret_cast<float2*>(ws + pl.off_ml);
    p.part_o = reinterpret_cast<float*>(ws + pl.off_o);
    p.B = B;
    p.Sq = Sq;
    p.total_q = total_q;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.groups = pl.groups;
    p.units = pl.units;
    p.num_pages = num_pages;
    p.page_shift = log2_exact(page_size);
    p.sb_shift = log2_exact(scale_block);
    p.max_pages = max_pages;
    p.window = window;
    p.scale_log2 = scale * kLog2e;
    const int box = std::min(page_size, 128);
    CUtensorMap tk, tv;
    if (!make_map_kv8(&tk, k8, (long long)num_pages * page_size, Hkv * D, box) ||
        !make_map_kv8(&tv, v8, (long long)num_pages * page_size, Hkv * D, box))
        return GQA_ERR_CUDA;
    const int sms = dev->sms;
    auto launch = [&](auto rows, auto pair, int bit) -> int {
        using C = gqa::Kv8Cfg<rows()>;
        const int r = ensure_smem_limit(gqa::kv8_decode<rows(), pair()>, 1 << bit, C::SMEM_BYTES);
        if (r != GQA_OK) return r;
        // a team's CTAs: as many head groups as divide them all, 16 at most; a team per
        // tile of one head group at most
        p.width = std::min(pl.groups, 16);
        while (pl.groups % p.width) --p.width;
        const long long tiles = pl.items / p.width * ((cap + 127) / 128);
        p.teams = int(std::min<long long>(
            tiles, std::min(C::CTAS_PER_SM * sms, kKv8MaxCtas) / p.width));
        const int grid = p.teams * p.width;
        const int r2 = launch_pdl(gqa::kv8_decode<rows(), pair()>, dim3(grid), C::THREADS,
                                  C::SMEM_BYTES, stream, tk, tv, p);
        if (r2 != GQA_OK) return r2;
        return launch_pdl(gqa::kv8_combine<rows(), pair()>,
                          dim3(grid, rows() / gqa::kCombineRows), 32 * gqa::kCombineWarps,
                          0, stream, p);
    };
    auto pick = [&](auto pair, int bit) {
        using std::integral_constant;
        switch (pl.rows) {
            case 4: return launch(integral_constant<int, 4>(), pair, bit);
            case 8: return launch(integral_constant<int, 8>(), pair, bit + 1);
            case 16: return launch(integral_constant<int, 16>(), pair, bit + 2);
            default: return launch(integral_constant<int, 32>(), pair, bit + 3);
        }
    };
    return D == 64 ? pick(std::true_type(), 20) : pick(std::false_type(), 24);
}

}  // extern "C"
