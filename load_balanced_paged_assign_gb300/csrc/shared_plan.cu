// The plan of decode attention over shared prefixes, and the join of its partials.
//
// One CTA.  A request shares its group's pages where all of its queries see all of
// them; a group shares at all where two requests do.  Its row tiles (128 query rows of
// a KV head, pairs of them) times the shared pages are the head's work, the requests'
// tiles behind them the tail's; each has CTAs of its own, as many as its part of the
// time is.  Both are then cut as the plain plan cuts its tiles: units in a fixed order,
// bins of one budget, in closed form.  All integers: the map depends on the lengths
// alone.
#include <cuda_bf16.h>

#include "block_scan.cuh"
#include "ptx.cuh"
#include "shared.h"

namespace hpc {
namespace {

constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ int clamp_live(const SharedPlan &p, int L) {
    return min(max(L, 0), p.max_pages * kTile);
}

// Cost of a page: 2 against a pair of row tiles, 1 against a single one.  A unit's
// cost is even, so that bins of even budgets begin at tiles.
__device__ __forceinline__ int pair_cost(int np) { return 2 * np; }
__device__ __forceinline__ int single_cost(int np) { return (np + 1) & ~1; }

__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const SharedPlan p) {
    // [B] tail tiles of the requests up to each; of each group: shared pages, first
    // sharing request, row tiles, units and cost of the groups before it
    extern __shared__ int s_mem[];
    int *s_end = s_mem;
    int *g_np = s_end + p.B, *g_lead = g_np + p.groups, *g_nb = g_lead + p.groups;
    int *g_unit = g_nb + p.groups, *g_cost = g_unit + p.groups + 1;
    __shared__ int s_scan[32];
    __shared__ unsigned s_flags;
    __shared__ int s_bad, s_np;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    if (tid == 0) s_flags = 0, s_bad = 0;
    __syncthreads();
    unsigned flags = 0;

    // lengths into shared memory, flagged where out of range; the groups' bounds
    for (int r = tid; r < p.B; r += blockDim.x) {
        const int L = p.seqlens[r];
        if (L < 0 || L > p.max_pages * kTile) flags |= HPC_FLAG_BAD_SEQLEN;
        s_end[r] = clamp_live(p, L);
        p.head.req[r] = make_int4(0, 0, 0, 0);
    }
    for (int g = tid; g < p.groups; g += blockDim.x) {
        const int a = p.starts[g], b = p.starts[g + 1];
        if (a < 0 || b < a || b > p.B) s_bad = 1;
        const int np = p.prefix[g];
        if (np < 0 || np > p.max_pages) flags |= HPC_FLAG_BAD_SEQLEN;
    }
    __syncthreads();
    const bool bad = s_bad != 0;
    if (bad) flags |= HPC_FLAG_BAD_SEQLEN;

    // who shares: a warp per group
    const int tpb = head_tokens(p.G);
    for (int g = warp; g < p.groups; g += warps) {
        const int a = bad ? 0 : p.starts[g], b = bad ? 0 : p.starts[g + 1];
        int np = p.prefix[g];
        if (np < 0 || np > p.max_pages) np = 0;
        int count = 0, lead = p.B, last = -1;
        for (int r = a + lane; r < b; r += 32)
            if (np > 0 && s_end[r] - p.q_len + 1 >= np * kTile) {
                ++count;
                lead = min(lead, r);
                last = r;
            }
        count = __reduce_add_sync(kFull, count);
        lead = __reduce_min_sync(kFull, lead);
        last = __reduce_max_sync(kFull, last);
        if (lane == 0) {
            g_np[g] = count >= 2 ? np : 0;
            g_lead[g] = lead;
            g_nb[g] = count >= 2 ? ((last - lead + 1) * p.q_len + tpb - 1) / tpb : 0;
        }
    }
    __syncthreads();

    // units and costs of the groups
    int units = 0, cost = 0;
    for (int base = 0; base < p.groups; base += blockDim.x) {
        const int g = base + tid;
        int u = 0, c = 0;
        if (g < p.groups && g_np[g] > 0) {
            const int np = g_np[g], nb = g_nb[g];
            u = p.Hkv * ((nb + 1) / 2);
            c = p.Hkv * ((nb / 2) * pair_cost(np) + (nb & 1) * single_cost(np));
        }
        int tu, tc;
        const int iu = block_inclusive_scan(u, s_scan, tu);
        const int ic = block_inclusive_scan(c, s_scan, tc);
        if (g < p.groups) {
            g_unit[g] = units + iu - u;
            g_cost[g] = cost + ic - c;
        }
        units += tu;
        cost += tc;
    }
    if (tid == 0) g_unit[p.groups] = units, g_cost[p.groups] = cost;
    __syncthreads();

    // the requests' part in it
    for (int g = warp; g < p.groups; g += warps) {
        const int np = g_np[g];
        if (np == 0) continue;
        const int lead = g_lead[g], nb = g_nb[g], u0 = g_unit[g];
        for (int r = p.starts[g] + lane; r < p.starts[g + 1]; r += 32) {
            if (s_end[r] - p.q_len + 1 < np * kTile) continue;
            p.head.req[r] = make_int4(np, u0, lead * p.q_len, nb);
            s_end[r] -= np * kTile;  // the tail's tokens
        }
    }
    __syncthreads();

    // tail tiles per request and their running sum
    int N = 0;
    for (int base = 0; base < p.B; base += blockDim.x) {
        const int r = base + tid;
        const int n = r < p.B ? (s_end[r] + kTile - 1) / kTile : 0;
        int total;
        const int incl = block_inclusive_scan(n, s_scan, total);
        if (r < p.B) s_end[r] = N + incl;
        N += total;
    }
    const int tail_units = p.Hkv / p.heads;  // per request
    const int T = tail_units * N;

    // CTAs: where the tail's HBM time is what everything takes, no more for it than
    // that needs; else in proportion to the times
    if (tid == 0) {
        const long long C = p.num_ctas;
        const long long head = (long long)cost * p.head_ns, tail = (long long)T * p.tail_ns;
        const long long even = (head + tail + C - 1) / C;
        const long long stream = (long long)T * p.tail_ps / 1000;
        const long long time = max(max(even, stream), 1LL);
        long long n = (head + time - 1) / time;
        n = max(min(n, T > 0 ? C - 1 : C), cost > 0 ? 1LL : 0LL);
        s_np = (int)n;
    }
    __syncthreads();
    const int want = s_np;
    const int budget = want > 0 ? (max((cost + want - 1) / want, 2 * max(p.floor, 1)) + 1) & ~1 : 2;
    const int np_ctas = (cost + budget - 1) / budget;

    // the head's descriptors
    int num_head = 0;
    for (int base = 0; base < units; base += blockDim.x) {
        const int u = base + tid;
        int cnt = 0, S = 0, g = 0, h = 0, pair = 0, n = 0, w = 1;
        if (u < units) {
            int lo = 0, hi = p.groups;  // the last group with g_unit <= u that has units
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (g_unit[mid] <= u) lo = mid;
                else hi = mid;
            }
            g = lo;
            const int nb = g_nb[g], pairs = (nb + 1) / 2, i = u - g_unit[g];
            n = g_np[g];
            h = i / pairs;
            pair = i - h * pairs;
            w = 2 * pair + 1 < nb ? 2 : 1;
            const int per_head = (nb / 2) * pair_cost(n) + (nb & 1) * single_cost(n);
            S = g_cost[g] + h * per_head + pair * pair_cost(n);
            cnt = (S + w * (n - 1)) / budget - S / budget + 1;
        }
        int total;
        const int incl = block_inclusive_scan(cnt, s_scan, total);
        if (u < units) {
            const int off = num_head + incl - cnt, bin0 = S / budget;
            p.head.unit[u] = make_int2(off, cnt);
            const int lead = g_lead[g] * p.q_len, first = lead + 2 * pair * tpb;
            // (row tiles of the group are counted from its first sharing request to its last)
            const int end = min(lead + g_nb[g] * tpb, p.starts[g + 1] * p.q_len);
            for (int i = 0; i < cnt; ++i) {
                const int lo = i == 0 ? 0 : ((bin0 + i) * budget - S + w - 1) / w;
                const int hi = i == cnt - 1 ? n : ((bin0 + i + 1) * budget - S + w - 1) / w;
                p.head.desc[2 * (off + i)] = make_int4(h, first, end, g_lead[g]);
                p.head.desc[2 * (off + i) + 1] = make_int4(lo, hi, w - 1, 0);
                if (i > 0 || S == bin0 * budget) p.head.bin[bin0 + i] = off + i;
            }
        }
        num_head += total;
    }
    for (int b = np_ctas + tid; b <= p.num_ctas; b += blockDim.x) p.head.bin[b] = num_head;

    // the tail's, behind the head's CTAs
    const int tail_ctas = max(p.num_ctas - np_ctas, 1);
    const int tail_budget = max((T + tail_ctas - 1) / tail_ctas, max(p.floor, 1));
    int num_desc = 0;
    for (int base = 0; base < tail_units * p.B; base += blockDim.x) {
        const int u = base + tid;
        int cnt = 0, h = 0, r = 0, n = 0, S = 0;
        if (u < tail_units * p.B) {
            h = u / p.B;
            r = u - h * p.B;
            n = s_end[r] - (r ? s_end[r - 1] : 0);
            S = h * N + s_end[r] - n;
            cnt = n ? (S + n - 1) / tail_budget - S / tail_budget + 1 : 0;
        }
        int total;
        const int incl = block_inclusive_scan(cnt, s_scan, total);
        if (u < tail_units * p.B) {
            const int off = num_desc + incl - cnt, skip = p.head.req[r].x;
            p.chunk_count[u] = cnt;
            p.chunk_off[u] = off;
            for (int i = 0; i < cnt; ++i) {
                const int bin = S / tail_budget + i;
                const int bin_lo = bin * tail_budget;
                const int lo = max(S, bin_lo), hi = (int)min((long long)(S + n), (long long)bin_lo + tail_budget);
                p.desc[off + i] = make_int4(h, r, skip + lo - S, skip + hi - S);
                if (lo == bin_lo) p.bin_ptr[np_ctas + bin] = off + i;
            }
        }
        num_desc += total;
    }
    const int used = np_ctas + (T + tail_budget - 1) / tail_budget;
    for (int b = used + tid; b <= p.num_ctas; b += blockDim.x) p.bin_ptr[b] = num_desc;
    for (int b = tid; b < np_ctas; b += blockDim.x) p.bin_ptr[b] = 0;
    flags = __reduce_or_sync(kFull, flags);
    if (flags && lane == 0) atomicOr(&s_flags, flags);
    __syncthreads();
    if (tid == 0) {
        p.head.hdr[0] = np_ctas;
        p.head.hdr[1] = num_head;
        p.head.hdr[2] = budget;
        p.head.hdr[3] = cost;
        p.head.hdr[4] = units;
        p.head.hdr[5] = p.head.hdr[6] = p.head.hdr[7] = 0;
        p.meta[0] = T;
        p.meta[1] = tail_budget;
        p.meta[2] = num_desc;
        p.meta[3] = (int)s_flags;
        p.meta[4] = p.meta[5] = p.meta[6] = p.meta[7] = 0;
    }
}

// ------------------------------------------------------------------ join
constexpr int kJoinWarps = 4;
constexpr float kJoinLog2e = 1.4426950408889634f;

struct JoinArgs {
    const float *tail_o, *tail_lse, *head_o, *head_lse;
    const int32_t *chunk_count, *chunk_off;
    HeadPlan plan;
    int B, Hq, G, q_len;  // G query heads of a KV head
    int tail_heads;       // KV heads of a tail descriptor
};

// One warp per query row, lane i dims 4 i .. 4 i + 3: out = sum_c w_c o_c / sum_c w_c with
// w_c = exp(lse_c - max), over the row's partials of the tail and of the head.
__global__ void __launch_bounds__(32 * kJoinWarps)
    shared_join_kernel(const JoinArgs a, __nv_bfloat16 *__restrict__ out) {
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x * kJoinWarps + (threadIdx.x >> 5);  // (r * q_len + i) * Hq + hq
    if (row >= a.B * a.q_len * a.Hq) return;
    const int ri = row / a.Hq, hq = row - ri * a.Hq;
    const int r = ri / a.q_len, i = ri - r * a.q_len;
    const int Gt = a.tail_heads * a.G, ht = hq / Gt;
    const int R = a.q_len * Gt, g = i * Gt + (hq - ht * Gt);
    const int n_tail = a.chunk_count[ht * a.B + r], off = a.chunk_off[ht * a.B + r];
    const int4 req = a.plan.req[r];
    int n_head = 0, slot0 = 0, step = 1, rho = 0;
    if (req.x > 0) {
        const int h = hq / a.G, tpb = head_tokens(a.G);
        const int tok = ri - req.z, tile = tok / tpb;
        const int2 un = a.plan.unit[req.y + h * ((req.w + 1) / 2) + tile / 2];
        n_head = un.y;
        slot0 = 2 * un.x + (tile & 1);
        step = 2;
        rho = (tok - tile * tpb) * a.G + (hq - h * a.G);
    }
    const int n = n_tail + n_head;
    auto at = [&](int c, const float *tail, const float *head, int width) {
        return c < n_tail ? tail + ((size_t)(off + c) * R + g) * width
                          : head + ((size_t)(slot0 + step * (c - n_tail)) * kHeadRows + rho) * width;
    };
    float m = -INFINITY;
    for (int c = lane; c < n; c += 32) m = fmaxf(m, *at(c, a.tail_lse, a.head_lse, 1));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float wsum = 0.f;
    for (int base = 0; base < n; base += 32) {
        const int cnt = min(32, n - base);
        const float wl =
            lane < cnt ? ex2((*at(base + lane, a.tail_lse, a.head_lse, 1) - m) * kJoinLog2e) : 0.f;
        float ws = wl;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ws += __shfl_xor_sync(kFull, ws, o);
        wsum += ws;
        for (int k = 0; k < cnt; k += 4) {
            float4 x[4];
            float w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[j] = __shfl_sync(kFull, wl, (k + j) & 31);
                x[j] = k + j < cnt
                           ? reinterpret_cast<const float4 *>(
                                 at(base + k + j, a.tail_o, a.head_o, kHeadDim))[lane]
                           : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc.x += w[j] * x[j].x;
                acc.y += w[j] * x[j].y;
                acc.z += w[j] * x[j].z;
                acc.w += w[j] * x[j].w;
            }
        }
    }
    const float inv = n > 0 && m != -INFINITY ? 1.f / wsum : 0.f;
    if (inv == 0.f) acc = make_float4(0.f, 0.f, 0.f, 0.f);
    uint2 packed;
    packed.x = pack_bf16x2(acc.x * inv, acc.y * inv);
    packed.y = pack_bf16x2(acc.z * inv, acc.w * inv);
    reinterpret_cast<uint2 *>(out + (size_t)row * kHeadDim)[lane] = packed;
}

template <class... P, class... A>
cudaError_t launch_dependent(void (*kernel)(P...), int grid, int threads, size_t smem,
                             cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_shared_plan(const SharedPlan &p, cudaStream_t s) {
    const size_t smem = ((size_t)p.B + 5 * (size_t)p.groups + 2) * sizeof(int);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(
            shared_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    const long long work = max(max((long long)p.B * (p.Hkv / p.heads), (long long)p.num_ctas + 1),
                               32LL * p.groups);
    const int threads = (int)min(max((work + 31) / 32 * 32, 64LL), (long long)kPlanThreads);
    return launch_dependent(shared_plan_kernel, 1, threads, smem, s, p);
}

cudaError_t launch_shared_join(const AttnParams &t, const HeadArgs &h, void *out, cudaStream_t s) {
    const int64_t rows = (int64_t)h.B * h.q_len * h.Hq;
    if (rows == 0) return cudaSuccess;
    JoinArgs a;
    a.tail_o = t.part_o;
    a.tail_lse = t.part_lse;
    a.head_o = h.part_o;
    a.head_lse = h.part_lse;
    a.chunk_count = t.chunk_count;
    a.chunk_off = t.chunk_off;
    a.plan = h.plan;
    a.B = h.B;
    a.Hq = h.Hq;
    a.G = h.G;
    a.q_len = h.q_len;
    a.tail_heads = t.G / h.G;
    return launch_dependent(shared_join_kernel, (int)((rows + kJoinWarps - 1) / kJoinWarps),
                            32 * kJoinWarps, 0, s, a, static_cast<__nv_bfloat16 *>(out));
}

}  // namespace hpc
