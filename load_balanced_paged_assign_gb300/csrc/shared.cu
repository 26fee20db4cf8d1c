// Host side of decode attention over shared prefixes: argument checks, tensor maps and
// launches.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "shared.h"

using namespace hpc;

namespace {

constexpr int kMaxDevices = 64;

// What the plan takes the work to cost (see SharedPlan), in us of one CTA: head_us an
// eighth of a page against two row tiles, with what a CTA's work has around it; tail_us a
// tile and stream_us its share of HBM's time; the starts what a unit costs beside its
// pages, in the same units.  One number serves all batches of a type, and most batches have
// a better one.  Steps in us, each number with one to either side of it.
//   BF16: 64 requests of 64 heads behind 8K tokens, tails 0.1 to 2K (53.7 as it is); 40 behind
//   12.5K (52.2); 37 in five groups of 15 heads, three tokens (28.5, two row blocks)
//     head_us 0.100, 0.140       53.5, 56.7;  55.0, 50.0;  29.2, 28.9
//     tail_us 0.50, 0.75         57.5, 53.8;  49.4, 54.0;  (0.66, 0.96)  28.6, 29.6
//     head_start 16, 48          53.8, 53.9;  51.9, 50.9;  28.8, 28.4
//     tail_start 0, 4            57.3, 55.3;  50.1, 54.7;  37.3, 29.1
//   E4M3: 128 of 16 heads behind 32K, tails 16 to 4K (47.5); 64 of 64 behind 8K (42.6); 48 in
//   three groups behind 4K, two tokens (42.2, two row blocks)
//     head_us 0.090, 0.128       48.7, 50.0;  40.9, 41.5;  40.5, 41.6
//     tail_us 0.30, 0.43         50.0, 48.6;  41.6, 40.8;  (0.33, 0.48)  41.6, 40.5
//     head_start 16, 48          50.4, 47.5;  43.4, 41.5;  41.4, 41.9
//     tail_start 0, 4            53.8, 48.3;  43.9, 40.5;  51.4, 40.8
//   block scales: 128 behind 32K (51.3); 64 behind 8K (44.4); 48 in six groups, two tokens
//   (40.6, two row blocks)
//     head_us 0.100, 0.130       51.4, 52.5;  44.0, 42.4;  40.9, 41.9
//     tail_us 0.30, 0.43         51.4, 53.2;  42.3, 43.9;  (0.33, 0.48)  41.6, 40.5
//     head_start 16, 48          54.6, 51.4;  46.3, 42.3;  41.5, 41.4
//     tail_start 0, 4            59.4, 51.2;  44.8, 43.4;  49.5, 41.6
//   stream_us times 1/2 and 2 (it counts where tails are nearly all of the work): 64 of 64
//   heads behind 1K, tails of 2K to 6K, BF16 158.6 and 155.5 (155.7), E4M3 89.1 and 88.9
//   (89.1); 32 pairs behind a page, BF16 60.3 and 61.0 (60.2); times 4 70.8
struct Cost {
    float head_us, tail_us, stream_us;
    int head_start, tail_start;
};
constexpr int kHeadStart = 32;

// (nb blocks of 8 query rows per KV head and request)
Cost cost_of(hpc_kv_dtype dt, int heads, int nb) {
    if (dt == HPC_KV_BF16) return {0.118f, nb == 1 ? 0.62f : 0.80f, 4.96e-3f, kHeadStart, 2};
    const float tile = (nb == 1 ? 0.36f : 0.40f) * heads, stream = 2.48e-3f * heads;
    if (dt == HPC_KV_FP8_E4M3) return {0.108f, tile, stream, kHeadStart, nb == 1 ? 2 : 3};
    return {0.115f, tile, stream, kHeadStart, nb == 1 ? 2 : 3};
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

hpc_status cuda_status(cudaError_t e) { return e == cudaSuccess ? HPC_OK : HPC_ERR_CUDA; }

// KV heads of a tail descriptor (see attn_tc.cuh).
int tail_heads(hpc_kv_dtype dt, int32_t Hkv) { return dt != HPC_KV_BF16 && Hkv % 2 == 0 ? 2 : 1; }

hpc_status check_shape(int32_t B, int32_t Hq, int32_t Hkv, int32_t q_len, int32_t max_pages,
                       int32_t groups, int32_t num_ctas, hpc_kv_dtype dt) {
    if (B < 0 || Hq <= 0 || Hkv <= 0 || q_len < 1 || max_pages <= 0 || groups < 0 || num_ctas < 2)
        return HPC_ERR_ARG;
    if (dt != HPC_KV_BF16 && dt != HPC_KV_FP8_E4M3 && dt != HPC_KV_E4M3_BLOCK) return HPC_ERR_ARG;
    if (Hq % Hkv != 0 || Hq / Hkv > HPC_MAX_GROUP) return HPC_ERR_UNSUPPORTED;
    if (q_len > HPC_MAX_QUERY_ROWS || q_len * (Hq / Hkv) > HPC_MAX_QUERY_ROWS)
        return HPC_ERR_UNSUPPORTED;
    if (B > HPC_MAX_SHARED_BATCH || groups > HPC_MAX_SHARED_GROUPS || num_ctas > 1 << 16)
        return HPC_ERR_UNSUPPORTED;
    // Costs, tile counts, query rows and token indices stay in int32.  A page costs 4 a row
    // tile and 1 more for an odd number of them, of which n requests (two at least) have n / 8
    // + 1 at most: 3 n, below 3 2^28 in all; the units' starts are below 2^30.  The plan's
    // quotients, KV heads among them, are exact below 2^20.
    if ((int64_t)B * max_pages * Hkv >= (int64_t)1 << 28 ||
        (int64_t)B * q_len * Hq >= (int64_t)1 << 30 ||
        (int64_t)max_pages * HPC_PAGE_SIZE >= (int64_t)1 << 30 || Hkv >= 1 << 20 ||
        head_units(B, Hq / Hkv, Hkv, q_len, groups) * kHeadStart >= (int64_t)1 << 30)
        return HPC_ERR_UNSUPPORTED;
    return HPC_OK;
}

// Tensor map over Q, whose box is a row tile: all query heads of a KV head of
// head_tokens(G) query tokens (BF16: of one 64-dim half).
hpc_status make_q_map(CUtensorMap *m, const void *q, int64_t tokens, int32_t Hq, int32_t G,
                      bool fp8) {
    auto encode = tensor_map_encoder();
    if (!encode) return HPC_ERR_CUDA;
    std::memset(m, 0, sizeof(*m));
    cuuint32_t elem[4] = {1, 1, 1, 1};
    CUresult r;
    if (fp8) {
        cuuint64_t dims[3] = {128, (cuuint64_t)Hq, (cuuint64_t)tokens};
        cuuint64_t strides[2] = {128, (cuuint64_t)Hq * 128};
        cuuint32_t box[3] = {128, (cuuint32_t)G, (cuuint32_t)head_tokens(G)};
        r = encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(q), dims, strides, box,
                   elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    } else {
        cuuint64_t dims[4] = {64, 2, (cuuint64_t)Hq, (cuuint64_t)tokens};
        cuuint64_t strides[3] = {128, 256, (cuuint64_t)Hq * 256};
        cuuint32_t box[4] = {64, 1, (cuuint32_t)G, (cuuint32_t)head_tokens(G)};
        r = encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(q), dims, strides,
                   box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    }
    return r == CUDA_SUCCESS ? HPC_OK : HPC_ERR_CUDA;
}

hpc_status check_map(const hpc_shared_map *m) {
    if (!m) return HPC_ERR_ARG;
    const hpc_task_map &t = m->tail;
    if (!t.desc || !t.bin_ptr || !t.chunk_count || !t.chunk_off || !t.meta || !m->head ||
        !m->head_o || !m->head_lse)
        return HPC_ERR_ARG;
    if (!aligned16(t.desc) || !aligned16(m->head) || (reinterpret_cast<uintptr_t>(m->head_o) & 31))
        return HPC_ERR_ARG;
    return HPC_OK;
}

hpc_status plan_shared(const int32_t *d_seqlens, int32_t B, int32_t Hq, int32_t Hkv,
                       int32_t max_pages, const int32_t *d_group_starts,
                       const int32_t *d_prefix_pages, int32_t num_groups, int32_t num_ctas,
                       int32_t min_tiles, hpc_kv_dtype dt, int32_t q_len, hpc_shared_map *map,
                       hpc_stream_t stream) {
    hpc_status st = check_shape(B, Hq, Hkv, q_len, max_pages, num_groups, num_ctas, dt);
    if (st != HPC_OK) return st;
    if (min_tiles < 0 || min_tiles >= 1 << 27) return HPC_ERR_ARG;
    if ((B > 0 && !d_seqlens) || (num_groups > 0 && (!d_group_starts || !d_prefix_pages)))
        return HPC_ERR_ARG;
    st = check_map(map);
    if (st != HPC_OK) return st;
    int64_t need[3];
    st = hpc_decode_shared_capacity(B, Hq, Hkv, q_len, num_groups, num_ctas, need);
    if (st != HPC_OK) return st;
    if (map->tail.cap_desc < need[0] || map->tail.cap_bins < num_ctas + 1 ||
        (int64_t)map->tail.cap_units < (int64_t)B * Hkv || map->cap_head < need[1] ||
        map->cap_slots < need[2])
        return HPC_ERR_WORKSPACE;
    const int G = Hq / Hkv, heads = tail_heads(dt, Hkv);
    SharedPlan p;
    p.seqlens = d_seqlens;
    p.starts = d_group_starts;
    p.prefix = d_prefix_pages;
    p.B = B;
    p.groups = num_groups;
    p.Hkv = Hkv;
    p.heads = heads;
    p.G = G;
    p.max_pages = max_pages;
    p.q_len = q_len;
    p.num_ctas = num_ctas;
    p.floor = min_tiles;
    const Cost c = cost_of(dt, heads, q_len * G > 8 ? 2 : 1);
    p.head_us = c.head_us;
    p.tail_us = c.tail_us;
    p.stream_us = c.stream_us;
    p.head_start = c.head_start;
    p.tail_start = c.tail_start;
    p.desc = reinterpret_cast<int4 *>(map->tail.desc);
    p.bin_ptr = map->tail.bin_ptr;
    p.chunk_count = map->tail.chunk_count;
    p.chunk_off = map->tail.chunk_off;
    p.meta = map->tail.meta;
    p.head = head_plan(map->head, B, head_units(B, G, Hkv, q_len, num_groups), num_ctas);
    st = cuda_status(launch_shared_plan(p, static_cast<cudaStream_t>(stream)));
    if (st != HPC_OK) return st;
    hpc_task_map &t = map->tail;
    t.B = B;
    t.Hkv = Hkv;
    t.num_ctas = num_ctas;
    t.persistent = 4 | 1 | (heads - 1) << 1;  // (no other call takes it)
    t.min_tiles = min_tiles;
    t.max_pages = max_pages;
    t.q_len = q_len;
    t.window = t.sinks = 0;
    map->Hq = Hq;
    map->num_groups = num_groups;
    map->kv_dtype = (int32_t)dt;
    return HPC_OK;
}

}  // namespace

extern "C" {

hpc_status hpc_decode_shared_capacity(int32_t B, int32_t Hq, int32_t Hkv, int32_t q_len,
                                      int32_t num_groups, int32_t num_ctas, int64_t sizes[3]) {
    const hpc_status st = check_shape(B, Hq, Hkv, q_len, 1, num_groups, num_ctas, HPC_KV_BF16);
    if (st != HPC_OK) return st;
    if (!sizes) return HPC_ERR_ARG;
    const int64_t units = head_units(B, Hq / Hkv, Hkv, q_len, num_groups);
    // (descriptors of head pairs fill two of the split buffer's)
    sizes[0] = 2 * (int64_t)num_ctas + (int64_t)B * Hkv;
    sizes[1] = head_ints(B, units, num_ctas);
    sizes[2] = units > 0 ? 2 * (units + num_ctas) : 1;
    return HPC_OK;
}

hpc_status hpc_decode_plan_shared(const int32_t *d_seqlens, int32_t B, int32_t Hq, int32_t Hkv,
                                  int32_t max_pages_per_req, const int32_t *d_group_starts,
                                  const int32_t *d_prefix_pages, int32_t num_groups,
                                  int32_t num_ctas, int32_t min_tiles_per_cta,
                                  hpc_kv_dtype kv_dtype, int32_t q_len, hpc_shared_map *map,
                                  hpc_stream_t stream) {
    return plan_shared(d_seqlens, B, Hq, Hkv, max_pages_per_req, d_group_starts, d_prefix_pages,
                       num_groups, num_ctas, min_tiles_per_cta, kv_dtype, q_len, map, stream);
}

hpc_status hpc_decode_attn_shared(const void *d_q, const float *d_q_scale, const void *d_k_cache,
                                  const void *d_v_cache, int32_t num_pages, float k_scale,
                                  float v_scale, const float *d_kv_scale, hpc_kv_dtype kv_dtype,
                                  const int32_t *d_block_table, int32_t max_pages_per_req,
                                  const int32_t *d_seqlens, int32_t B, int32_t Hq, int32_t Hkv,
                                  int32_t head_dim, int32_t q_len, float sm_scale,
                                  const hpc_shared_map *map, float *d_part_o, float *d_part_lse,
                                  void *d_out, hpc_stream_t stream) {
    hpc_status st = check_map(map);
    if (st != HPC_OK) return st;
    const hpc_task_map &m = map->tail;
    if (head_dim != HPC_HEAD_DIM) return HPC_ERR_UNSUPPORTED;
    st = check_shape(B, Hq, Hkv, q_len, max_pages_per_req, map->num_groups, m.num_ctas, kv_dtype);
    if (st != HPC_OK) return st;
    const bool block = kv_dtype == HPC_KV_E4M3_BLOCK, fp8 = kv_dtype != HPC_KV_BF16;
    if (block != (d_kv_scale != nullptr) || !aligned16(d_kv_scale)) return HPC_ERR_ARG;
    if (num_pages <= 0 || !d_k_cache || !d_v_cache || !d_part_o || !d_part_lse) return HPC_ERR_ARG;
    if (B > 0 && (!d_q || !d_block_table || !d_seqlens || !d_out)) return HPC_ERR_ARG;
    if (fp8 && B > 0 && !d_q_scale) return HPC_ERR_ARG;
    if (!aligned16(d_q) || !aligned16(d_k_cache) || !aligned16(d_v_cache) ||
        !aligned16(d_part_o) || !aligned16(d_out))
        return HPC_ERR_ARG;
    if (block || !fp8) k_scale = v_scale = 1.f;
    const float score_scale = sm_scale * 1.4426950408889634f * k_scale;
    if (!std::isfinite(score_scale) || !std::isfinite(v_scale)) return HPC_ERR_ARG;
    // the plan of this batch's shape
    const int heads = tail_heads(kv_dtype, Hkv);
    if (m.persistent != (4 | 1 | (heads - 1) << 1) || m.B != B || m.Hkv != Hkv ||
        m.q_len != q_len || m.max_pages != max_pages_per_req || map->Hq != Hq ||
        map->kv_dtype != (int32_t)kv_dtype)
        return HPC_ERR_ARG;
    if (B == 0) return HPC_OK;
    const int G = Hq / Hkv;

    SharedMaps maps;
    st = make_q_map(&maps.q, d_q, (int64_t)B * q_len, Hq, G, fp8);
    if (st == HPC_OK) st = cache_tensor_map(&maps.k, d_k_cache, num_pages, Hkv, fp8);
    if (st == HPC_OK) st = cache_tensor_map(&maps.v, d_v_cache, num_pages, Hkv, fp8);
    if (st == HPC_OK && fp8) st = heads_tensor_map(&maps.tk, d_k_cache, num_pages, Hkv, heads);
    if (st == HPC_OK && fp8) st = heads_tensor_map(&maps.tv, d_v_cache, num_pages, Hkv, heads);
    if (st != HPC_OK) return st;
    if (!fp8) maps.tk = maps.k, maps.tv = maps.v;

    AttnParams t = {};
    t.bin_ptr = m.bin_ptr;
    t.desc = reinterpret_cast<const int4 *>(m.desc);
    t.chunk_count = m.chunk_count;
    t.chunk_off = m.chunk_off;
    t.seqlens = d_seqlens;
    t.block_table = d_block_table;
    t.q = d_q;
    t.q_scale = d_q_scale;
    t.part_o = d_part_o;
    t.part_lse = d_part_lse;
    t.meta = m.meta;
    t.bin_counter = m.meta + 4;
    t.num_bins = m.num_ctas;
    t.min_tiles = m.min_tiles;
    t.B = B;
    t.Hq = Hq;
    t.Hkv = Hkv / heads;
    t.G = heads * G;
    t.max_pages = max_pages_per_req;
    t.num_pages = num_pages;
    t.q_len = q_len;
    t.R = q_len * t.G;
    t.score_scale = score_scale;
    t.v_scale = v_scale;
    t.window = kNoWindow;
    t.kv_scale = d_kv_scale;

    HeadArgs h = {};
    h.plan = head_plan(map->head, B, head_units(B, G, Hkv, q_len, map->num_groups), m.num_ctas);
    h.block_table = d_block_table;
    h.q_scale = d_q_scale;
    h.kv_scale = d_kv_scale;
    h.part_o = map->head_o;
    h.part_lse = map->head_lse;
    h.meta = m.meta;
    h.B = B;
    h.Hq = Hq;
    h.Hkv = Hkv;
    h.G = G;
    h.q_len = q_len;
    h.max_pages = max_pages_per_req;
    h.num_pages = num_pages;
    h.score_scale = score_scale;
    h.v_scale = v_scale;

    const int nb = q_len * G > 8 ? 2 : 1;
    const AttnConfig cfg = kv_dtype == HPC_KV_BF16 ? shared_config_bf16(nb)
                           : block                 ? shared_config_block(nb, heads)
                                                   : shared_config_e4m3(nb, heads);
    // per device and variant: the shared-memory attribute is set
    static std::atomic<unsigned> ready[kMaxDevices];
    const unsigned bit = 1u << ((int)kv_dtype * 4 + (heads - 1) * 2 + nb - 1);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return HPC_ERR_CUDA;
    if (!(ready[dev].load() & bit)) {
        if (cudaFuncSetAttribute(cfg.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 cfg.smem_bytes) != cudaSuccess)
            return HPC_ERR_CUDA;
        ready[dev].fetch_or(bit);
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = kv_dtype == HPC_KV_BF16
                              ? launch_shared_bf16(nb, maps, t, h, m.num_ctas, s)
                          : block ? launch_shared_block(nb, heads, maps, t, h, m.num_ctas, s)
                                  : launch_shared_e4m3(nb, heads, maps, t, h, m.num_ctas, s);
    if (e != cudaSuccess) return HPC_ERR_CUDA;
    return cuda_status(launch_shared_join(t, h, d_out, s));
}

hpc_status hpc_decode_step_shared(const void *d_q, const float *d_q_scale, const void *d_k_cache,
                                  const void *d_v_cache, int32_t num_pages, float k_scale,
                                  float v_scale, const float *d_kv_scale, hpc_kv_dtype kv_dtype,
                                  const int32_t *d_block_table, int32_t max_pages_per_req,
                                  const int32_t *d_seqlens, const int32_t *d_group_starts,
                                  const int32_t *d_prefix_pages, int32_t num_groups, int32_t B,
                                  int32_t Hq, int32_t Hkv, int32_t head_dim, int32_t q_len,
                                  float sm_scale, int32_t num_ctas, int32_t min_tiles_per_cta,
                                  hpc_shared_map *map, float *d_part_o, float *d_part_lse,
                                  void *d_out, hpc_stream_t stream) {
    const hpc_status st = plan_shared(d_seqlens, B, Hq, Hkv, max_pages_per_req, d_group_starts,
                                      d_prefix_pages, num_groups, num_ctas, min_tiles_per_cta,
                                      kv_dtype, q_len, map, stream);
    if (st != HPC_OK) return st;
    return hpc_decode_attn_shared(d_q, d_q_scale, d_k_cache, d_v_cache, num_pages, k_scale,
                                  v_scale, d_kv_scale, kv_dtype, d_block_table, max_pages_per_req,
                                  d_seqlens, B, Hq, Hkv, head_dim, q_len, sm_scale, map, d_part_o,
                                  d_part_lse, d_out, stream);
}

}  // extern "C"
