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

// The head's cost of a page: against a pair of row tiles, and against one that is alone.
// Measured 0.80 and 0.50 us.
constexpr int kPairCost = 8, kAloneCost = 5;

// Costs are positions on a line that bins of one budget cut: a unit of n pages of cost w
// begins with `start` positions for what it costs beside them (Q, its partials), and a
// page belongs to the bin in which it begins.  A bin is longer than `start` + w, so that
// some page begins in each.

// a / b for quotients below 2^20, with `inv` = 1 / b: off by one at most before the
// correction.  (One reciprocal for all quotients of a divisor: a division is 100 cycles of
// latency, and this kernel is a chain of them.)
__device__ __forceinline__ int quotient(int a, int b, float inv) {
    const int q = (int)((float)a * inv), r = a - q * b;
    return q + (r >= b) - (r < 0);
}

// Descriptors of a unit that spans several bins: a thread writes the first kOwn of its
// own unit, its warp the others (a long prefix of few requests is one unit of as many
// descriptors as there are CTAs).  The cooperative way costs 300 cycles a unit, a
// thread's own 60 a descriptor.
constexpr int kOwn = 16;

template <class Write>
__device__ __forceinline__ void write_chunks(int cnt, Write write) {
    const int lane = threadIdx.x & 31;
    for (int i = 0; i < min(cnt, kOwn); ++i) write(lane, i, false);
    for (unsigned many = __ballot_sync(kFull, cnt > kOwn); many; many &= many - 1) {
        const int of = __ffs(many) - 1, n = __shfl_sync(kFull, cnt, of);
        for (int i0 = kOwn; i0 < n; i0 += 32) write(of, i0 + lane, true);
    }
}

__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const SharedPlan p) {
    // of each request: its length, then the tail tiles of the requests up to it; its
    // group where it shares, else -1; the tails up to it.  Of each group: first request, shared pages, first
    // sharing request, row tiles, units and cost of the groups before it
    extern __shared__ int s_mem[];
    int *s_end = s_mem, *s_of = s_end + p.B, *s_tail = s_of + p.B;
    int *g_start = s_tail + p.B, *g_np = g_start + p.groups + 1, *g_lead = g_np + p.groups;
    int *g_nb = g_lead + p.groups, *g_unit = g_nb + p.groups, *g_cost = g_unit + p.groups;
    __shared__ int s_scan[4 * 32];
    __shared__ unsigned s_flags;
    __shared__ int s_bad, s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    if (tid == 0) s_flags = 0, s_bad = 0, s_last = -1;
    // the arguments' lines of the constant bank, cold, while the kernel before still runs
    asm volatile("" ::"l"(p.seqlens), "r"(p.floor), "f"(p.head_us), "r"(p.tail_start), "l"(p.desc),
                 "l"(p.meta), "l"(p.head.hdr), "l"(p.head.desc));
    grid_dependency_wait();
    grid_launch_dependents();
    unsigned flags = 0;
    for (int i = tid; i < p.B || i <= p.groups; i += blockDim.x) {
        // (the three loads in flight together)
        const int L = i < p.B ? p.seqlens[i] : 0;
        const int start = p.groups > 0 && i <= p.groups ? p.starts[i] : 0;
        const int np = i < p.groups ? p.prefix[i] : 0;
        const bool bad_len = L < 0 || L > p.max_pages * kTile, bad_np = np < 0 || np > p.max_pages;
        if (bad_len || bad_np) flags |= HPC_FLAG_BAD_SEQLEN;
        if (i < p.B) {
            s_end[i] = clamp_live(p, L);
            s_of[i] = -1;
        }
        if (i <= p.groups) g_start[i] = start;
        if (i < p.groups) g_np[i] = bad_np ? 0 : np;
    }
    __syncthreads();
    for (int g = tid; g < p.groups; g += blockDim.x)
        if (g_start[g] < 0 || g_start[g + 1] < g_start[g] || g_start[g + 1] > p.B) s_bad = 1;
    if (p.groups > 0) __syncthreads();
    const bool bad = s_bad != 0;  // (not read before the barrier where it may be written)
    if (bad) flags |= HPC_FLAG_BAD_SEQLEN;

    // who shares: a warp per group
    const int tpb = head_tokens(p.G);
    for (int g = warp; g < p.groups; g += warps) {
        const int a = bad ? 0 : g_start[g], b = bad ? 0 : g_start[g + 1], np = g_np[g];
        const int need = np * kTile + p.q_len - 1;
        int count = 0, lead = p.B, last = -1;
        for (int r = a + lane; r < b && np > 0; r += 32)
            if (s_end[r] >= need) {
                ++count;
                lead = min(lead, r);
                last = r;
            }
        count = __reduce_add_sync(kFull, count);
        lead = __reduce_min_sync(kFull, lead);
        last = __reduce_max_sync(kFull, last);
        if (count >= 2)
            for (int r = a + lane; r < b; r += 32)
                if (s_end[r] >= need) {
                    s_of[r] = g;
                    s_end[r] -= np * kTile;  // the tail's tokens
                }
        __syncwarp();
        if (lane == 0) {
            g_lead[g] = lead;
            g_nb[g] = count >= 2 ? ((last - lead + 1) * p.q_len + tpb - 1) / tpb : 0;
            if (count < 2) g_np[g] = 0;
        }
    }
    __syncthreads();

    // units, pages' costs of the groups, tail tiles and tails of the requests, and their
    // running sums
    int units = 0, pages = 0, tiles = 0, tails = 0;
    for (int base = 0; base < max(p.B, p.groups); base += blockDim.x) {
        const int i = base + tid;
        int v[4] = {0, 0, 0, 0}, total[4];
        if (i < p.groups && g_np[i] > 0) {
            const int np = g_np[i], nb = g_nb[i];
            v[0] = p.Hkv * ((nb + 1) / 2);
            v[1] = p.Hkv * np * ((nb / 2) * kPairCost + (nb & 1) * kAloneCost);
        }
        if (i < p.B) v[2] = (s_end[i] + kTile - 1) / kTile;
        v[3] = v[2] > 0;
        const int u = v[0], c = v[1];
        block_inclusive_scans(v, s_scan, total);
        if (i < p.groups) {
            g_unit[i] = units + v[0] - u;
            g_cost[i] = pages + v[1] - c;
            if (u > 0) atomicMax(&s_last, i);  // the last group with units
        }
        if (i < p.B) {
            s_end[i] = tiles + v[2];
            s_tail[i] = tails + v[3];
        }
        units += total[0];
        pages += total[1];
        tiles += total[2];
        tails += total[3];
    }
    __syncthreads();  // the sums are complete
    const int tail_units = p.Hkv / p.heads;  // per request

    // What a unit costs beside its pages counts where a CTA has several microseconds of
    // work; with less, the floor alone says how finely units are cut.
    const float head_us = (float)pages * p.head_us, tail_us = (float)(tail_units * tiles) * p.tail_us;
    const bool busy = head_us + tail_us > 2.f * p.num_ctas;
    const int start = busy ? p.head_start : 0, tail_start = busy ? p.tail_start : 0;
    const int cost = pages + units * start;
    const int N = tiles + tails * tail_start, T = tail_units * N;
    // CTAs: where the tail's HBM time is what everything takes, no more for it than
    // that needs; else in proportion to the times
    const float head = (float)cost * p.head_us, tail = (float)T * p.tail_us;
    const float time = fmaxf((head + tail) / p.num_ctas, (float)(tail_units * tiles) * p.stream_us);
    const int most = T > 0 ? p.num_ctas - 1 : p.num_ctas;
    const int want = cost > 0 ? max((int)fminf(ceilf(head / time), (float)most), 1) : 0;
    const int budget = max(want > 0 ? (cost + want - 1) / want : 0,
                           start + kPairCost * max(p.floor, 1));
    // up to the bin in which the last page begins
    const int np_ctas =
        units > 0 ? (cost - (g_nb[s_last] & 1 ? kAloneCost : kPairCost)) / budget + 1 : 0;
    const int tail_ctas = max(p.num_ctas - np_ctas, 1);
    const int tail_budget = max((T + tail_ctas - 1) / tail_ctas, tail_start + max(p.floor, 1));
    const float budget_inv = 1.f / (float)budget, tail_inv = 1.f / (float)tail_budget;
    const float B_inv = 1.f / (float)max(p.B, 1);

    for (int r = tid; r < p.B; r += blockDim.x) {
        const int g = s_of[r];
        p.head.req[r] = g < 0 ? make_int4(0, 0, 0, 0)
                              : make_int4(g_np[g], g_unit[g], g_lead[g] * p.q_len, g_nb[g]);
    }
    auto group_of = [&](int u) {  // the last group with g_unit <= u: it has units
        int lo = 0, hi = p.groups;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (g_unit[mid] <= u) lo = mid;
            else hi = mid;
        }
        return lo;
    };
    // the descriptors of the head and, behind its CTAs, of the tail
    int num_head = 0, num_desc = 0;
    for (int base = 0; base < max(units, tail_units * p.B); base += blockDim.x) {
        const int u = base + tid;
        int hc = 0, hS = 0, hbin = 0, hh = 0, first = 0, end = 0, lead = 0, n = 0, w = 1,
            prev = 0;
        if (u < units) {
            const int lo = group_of(u);
            const int nb = g_nb[lo], pairs = (nb + 1) / 2, i = u - g_unit[lo];
            n = g_np[lo];
            hh = quotient(i, pairs, 1.f / (float)pairs);
            const int pair = i - hh * pairs;
            w = 2 * pair + 1 < nb ? kPairCost : kAloneCost;
            hS = g_cost[lo] + u * start +
                 hh * n * ((nb / 2) * kPairCost + (nb & 1) * kAloneCost) + pair * n * kPairCost +
                 start;  // of its first page
            // what a page of the unit before costs
            if (pair == 0 && hh == 0 && u > 0) {
                prev = g_nb[group_of(u - 1)] & 1;
            } else {
                prev = pair == 0 ? nb & 1 : 0;
            }
            prev = prev ? kAloneCost : kPairCost;
            hbin = quotient(hS, budget, budget_inv);
            hc = quotient(hS + w * (n - 1), budget, budget_inv) - hbin + 1;
            lead = g_lead[lo];
            first = lead * p.q_len + 2 * pair * tpb;
            end = min(lead * p.q_len + nb * tpb, g_start[lo + 1] * p.q_len);
        }
        int tc = 0, th = 0, r = 0, tn = 0, tS = 0, tbin = 0, skip = 0;
        if (u < tail_units * p.B) {
            th = quotient(u, p.B, B_inv);
            r = u - th * p.B;
            tn = s_end[r] - (r ? s_end[r - 1] : 0);
            // of its first tile
            tS = th * N + s_end[r] - tn + s_tail[r] * tail_start;
            tbin = quotient(tS, tail_budget, tail_inv);
            tc = tn ? quotient(tS + tn - 1, tail_budget, tail_inv) - tbin + 1 : 0;
            if (s_of[r] >= 0) skip = g_np[s_of[r]];
        }
        int v[2] = {hc, tc}, total[2];
        block_inclusive_scans(v, s_scan, total);
        const int hoff = num_head + v[0] - hc, toff = num_desc + v[1] - tc;
        num_head += total[0];
        num_desc += total[1];
        if (u < units) p.head.unit[u] = make_int2(hoff, hc);
        if (u < tail_units * p.B) {
            p.chunk_count[u] = tc;
            p.chunk_off[u] = toff;
        }
        write_chunks(hc, [&](int of, int i, bool all) {
            auto get = [&](int x) { return all ? __shfl_sync(kFull, x, of) : x; };
            const int S = get(hS), cnt = get(hc), n_ = get(n), w_ = get(w), off = get(hoff);
            const int prev_ = get(prev);
            const int4 a = make_int4(get(hh), get(first), get(end), get(lead));
            const int bin = get(hbin) + i;
            if (i >= cnt) return;
            const bool two = w_ == kPairCost;
            auto page_at = [&](int x) {
                return two ? (x + kPairCost - 1) / kPairCost : (x + kAloneCost - 1) / kAloneCost;
            };
            const int lo = i == 0 ? 0 : page_at(bin * budget - S);
            const int hi = i == cnt - 1 ? n_ : page_at((bin + 1) * budget - S);
            p.head.desc[2 * (off + i)] = a;
            p.head.desc[2 * (off + i) + 1] = make_int4(lo, hi, two, 0);
            // the first that begins in its bin: the unit before has its last page earlier
            if (i > 0 || S - start - prev_ < bin * budget) p.head.bin[bin] = off + i;
        });
        write_chunks(tc, [&](int of, int i, bool all) {
            auto get = [&](int x) { return all ? __shfl_sync(kFull, x, of) : x; };
            const int S = get(tS), cnt = get(tc), n_ = get(tn), off = get(toff);
            const int h_ = get(th), r_ = get(r), sk = get(skip);
            const int bin = get(tbin) + i, bin_lo = bin * tail_budget;
            if (i >= cnt) return;
            const int lo = max(S, bin_lo), hi = min(S + n_ - bin_lo, tail_budget) + bin_lo;
            p.desc[off + i] = make_int4(h_, r_, sk + lo - S, sk + hi - S);
            if (S - tail_start <= bin_lo) p.bin_ptr[np_ctas + bin] = off + i;
        });
    }
    for (int b = np_ctas + tid; b <= p.num_ctas; b += blockDim.x) p.head.bin[b] = num_head;
    const int used = np_ctas + (T + tail_budget - 1) / tail_budget;
    for (int b = used + tid; b <= p.num_ctas; b += blockDim.x) p.bin_ptr[b] = num_desc;
    for (int b = tid; b < np_ctas; b += blockDim.x) p.bin_ptr[b] = 0;
    flags = __reduce_or_sync(kFull, flags);
    if (flags && lane == 0) atomicOr(&s_flags, flags);
    __syncthreads();
    if (tid == 0) {
        int4 *hdr = reinterpret_cast<int4 *>(p.head.hdr);
        hdr[0] = make_int4(np_ctas, num_head, budget, cost);
        hdr[1] = make_int4(units, 0, 0, 0);
        p.meta[0] = tail_units * tiles;
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
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x * kJoinWarps + (threadIdx.x >> 5);  // (r * q_len + i) * Hq + hq
    const bool any = row < a.B * a.q_len * a.Hq;
    // The plan is read ahead of the attention's end: its kernel had finished before the
    // attention's let this one start.
    int n_tail = 0, off = 0, n_head = 0, slot0 = 0, step = 1, rho = 0, R = 1, g = 0;
    if (any) {
        const int ri = row / a.Hq, hq = row - ri * a.Hq;
        const int r = ri / a.q_len, i = ri - r * a.q_len;
        const int Gt = a.tail_heads * a.G, ht = hq / Gt;
        R = a.q_len * Gt;
        g = i * Gt + (hq - ht * Gt);
        n_tail = a.chunk_count[ht * a.B + r];
        off = a.chunk_off[ht * a.B + r];
        const int4 req = a.plan.req[r];
        if (req.x > 0) {
            const int h = hq / a.G, tpb = head_tokens(a.G);
            const int tok = ri - req.z, tile = tok / tpb;
            const int2 un = a.plan.unit[req.y + h * ((req.w + 1) / 2) + tile / 2];
            const bool alone = tile + 1 == req.w && (tile & 1) == 0;
            n_head = alone ? 2 * un.y : un.y;
            slot0 = 2 * un.x + (tile & 1);
            step = alone ? 1 : 2;
            rho = (tok - tile * tpb) * a.G + (hq - h * a.G);
        }
    }
    grid_dependency_wait();
    if (!any) return;
    const int n = n_tail + n_head;
    auto at = [&](int c, const float *tail, const float *head, int width) {
        return c < n_tail ? tail + ((size_t)(off + c) * R + g) * width
                          : head + ((size_t)(slot0 + step * (c - n_tail)) * kHeadRows + rho) * width;
    };
    // the first rows on their way with the log-sum-exps (nothing is read twice but the
    // latter of rows with more than 32 partials)
    constexpr int kAhead = 8;
    float4 x[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
        x[j] = j < n ? reinterpret_cast<const float4 *>(at(j, a.tail_o, a.head_o, kHeadDim))[lane]
                     : make_float4(0.f, 0.f, 0.f, 0.f);
    const float own = lane < n ? *at(lane, a.tail_lse, a.head_lse, 1) : -INFINITY;
    float m = own;
    for (int c = 32 + lane; c < n; c += 32) m = fmaxf(m, *at(c, a.tail_lse, a.head_lse, 1));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float wsum = 0.f;
    for (int base = 0; base < n; base += 32) {
        const int cnt = min(32, n - base);
        float wl = 0.f;
        if (lane < cnt)
            wl = ex2(((base ? *at(base + lane, a.tail_lse, a.head_lse, 1) : own) - m) * kJoinLog2e);
        float ws = wl;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ws += __shfl_xor_sync(kFull, ws, o);
        wsum += ws;
        for (int k = 0; k < cnt; k += kAhead) {
            if (base | k) {
#pragma unroll
                for (int j = 0; j < kAhead; ++j)
                    if (k + j < cnt)
                        x[j] = reinterpret_cast<const float4 *>(
                            at(base + k + j, a.tail_o, a.head_o, kHeadDim))[lane];
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const float w = __shfl_sync(kFull, wl, (k + j) & 31);
                if (k + j >= cnt || !(w > 0.f)) continue;  // (no values where no weight is)
                acc.x += w * x[j].x;
                acc.y += w * x[j].y;
                acc.z += w * x[j].z;
                acc.w += w * x[j].w;
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
    const size_t smem = (3 * (size_t)p.B + 6 * (size_t)p.groups + 1) * sizeof(int);
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
