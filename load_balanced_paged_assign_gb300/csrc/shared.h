// Decode attention over shared prefixes: what its plan, its kernels and its host
// side share.
//
// Requests of a group begin with the same pages.  Their queries' attention over
// those pages (the head) is computed for all of them at once: the group's query rows
// of a KV head, 128 to a tile, against every shared page, which is read once for up
// to 256 rows.  What a request has behind them (the tail) is decode attention as
// ever, with descriptors that begin behind the shared pages.  Both leave normalised
// partials and their log-sum-exps, and the join weighs a row's partials from both.
#pragma once

#include "internal.h"

namespace hpc {

constexpr int kHeadRows = 128;  // query rows of a tile

// The head's plan, in map->head (int32):
//   hdr   [8]  {CTAs with head work, head descriptors, their budget, cost, units, 0 ..}
//   req   [B] int4 {shared tiles, the group's first unit, its first query token, its row tiles}
//   bin   [num_ctas + 1] first descriptor of each CTA's
//   unit  [units] int2 {first descriptor, descriptors}
//   desc  [descriptors][2] int4 {KV head, first query token, end of the group's query tokens,
//         the request whose table row is read}, {first tile, end, 1: two row tiles, 0}
// A unit is a KV head of a group and a pair of its row tiles (or the last one alone).
// Descriptor d leaves the partials of its first row tile in slot 2 d, the second's in
// slot 2 d + 1; a row tile that is alone leaves two, of every other page.
struct HeadPlan {
    int32_t *hdr;
    int4 *req;
    int32_t *bin;
    int2 *unit;
    int4 *desc;
};

// Query tokens of a row tile: as many as have all of a KV head's query heads in it.
__host__ __device__ constexpr int head_tokens(int G) { return kHeadRows / G; }

inline int64_t head_units(int64_t B, int G, int Hkv, int q_len, int64_t groups) {
    // a group has at least two requests and ceil(tiles / 2) pairs: at most tokens / (2
    // tokens of a tile) + 1
    const int64_t with = groups < B / 2 ? groups : B / 2;
    return with > 0 ? Hkv * (B * q_len / (2 * head_tokens(G)) + with) : 0;
}

inline int64_t head_ints(int64_t B, int64_t units, int64_t num_ctas) {
    const int64_t bins = (num_ctas + 1 + 3) / 4 * 4, pairs = (2 * units + 3) / 4 * 4;
    return 8 + 4 * B + bins + pairs + 8 * (units + num_ctas);
}

inline HeadPlan head_plan(int32_t *at, int64_t B, int64_t units, int64_t num_ctas) {
    HeadPlan h;
    h.hdr = at;
    at += 8;
    h.req = reinterpret_cast<int4 *>(at);
    at += 4 * B;
    h.bin = at;
    at += (num_ctas + 1 + 3) / 4 * 4;
    h.unit = reinterpret_cast<int2 *>(at);
    at += (2 * units + 3) / 4 * 4;
    h.desc = reinterpret_cast<int4 *>(at);
    return h;
}

struct SharedPlan {
    const int32_t *seqlens, *starts, *prefix;
    int B, groups, Hkv, heads, G, max_pages, q_len, num_ctas, floor;
    float head_us;    // of one unit of the head's cost (an eighth of a page of two row tiles)
    float tail_us;    // of a tail descriptor's tile in a CTA
    float stream_us;  // of a tail tile where HBM is what all CTAs wait for
    int head_start, tail_start;  // what a unit costs beside its pages
    int4 *desc;
    int32_t *bin_ptr, *chunk_count, *chunk_off, *meta;
    HeadPlan head;
};

struct HeadArgs {
    HeadPlan plan;
    const int32_t *block_table;
    const float *q_scale, *kv_scale;
    float *part_o, *part_lse;
    int32_t *meta;
    int B, Hq, Hkv, G, q_len, max_pages, num_pages;
    float score_scale;  // sm_scale * log2(e), times k_scale for E4M3
    float v_scale;
};

struct SharedMaps {  // over Q, the pages of one head, and the pages as the tail's kernel reads them
    CUtensorMap q, k, v, tk, tv;
};

cudaError_t launch_shared_plan(const SharedPlan &p, cudaStream_t s);
cudaError_t launch_shared_join(const AttnParams &t, const HeadArgs &h, void *out, cudaStream_t s);

// The attention kernel for a cache type, nb blocks of 8 rows and `heads` KV heads in a
// tail descriptor.
cudaError_t launch_shared_bf16(int nb, const SharedMaps &m, const AttnParams &t, const HeadArgs &h,
                               int grid, cudaStream_t s);
cudaError_t launch_shared_e4m3(int nb, int heads, const SharedMaps &m, const AttnParams &t,
                               const HeadArgs &h, int grid, cudaStream_t s);
cudaError_t launch_shared_block(int nb, int heads, const SharedMaps &m, const AttnParams &t,
                                const HeadArgs &h, int grid, cudaStream_t s);
AttnConfig shared_config_bf16(int nb);
AttnConfig shared_config_e4m3(int nb, int heads);
AttnConfig shared_config_block(int nb, int heads);

}  // namespace hpc
