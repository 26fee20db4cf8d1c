// The plan of decode attention over shared prefixes, and the join of its partials.
//
// One CTA.  A request shares its group's pages where all of its queries see all of
// them; a group shares at all where two requests do.  Its row tiles (128 query rows of
// a KV head, pairs of them) times the shared pages are the head's work, the requests'
// tiles behind them the tail's; each has CTAs of its own, as many as its part of the
// time is.  Both are then cut as the plain plan cuts its tiles: units in a fixed order,
// bins of one budget, in closed form, all in integers.  How the CTAs are shared out and
// which budgets that gives is reckoned in fp32 from measured costs (shared.cu), which
// depend on the cache type, the rows of a request and KV head and the heads of a
// descriptor.  So the map is a function of the lengths, the groups, the shape, the number
// of CTAs and the floor.
#include <cuda_bf16.h>

#include "block_scan.cuh"
#include "ptx.cuh"
#include "shared.h"

namespace hpc {
namespace {

constexpr unsigned kFull = 0xffffffffu;

// The head's cost of a page: against a pair of row tiles, and against one that is alone.
// What a page more of a long prefix takes a CTA, with no tails (64 and 16 requests of 64 heads
// on 8, 16K to 128K tokens): 0.72 us and 0.80 (BF16, whose lone tiles wait for HBM), 0.89 and
// 0.62 (E4M3), 0.86 and 0.64 (block scales); beside tails a lone tile's pages cost less.
// Steps with 5, 6 and 7: 12 requests of 64 heads on 8 behind 8K tokens, E4M3, 27.4, 29.6 and
// 29.6 us, block scales 28.0, 30.3 and 32.6; 48 in six groups, block scales, 40.6, 41.8 and
// 42.1; 37 in five groups, BF16, 28.4, 28.4 and 29.6, and 40 behind 12.5K tokens (a pair and a
// lone tile) 52.2, 49.8 and 48.2: one number for all types, of which 6 would suit BF16 better.
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

// The kernel is one chain of dependent steps over code that runs once, 5 us of 10,000
// cycles at first.  So the head's units and the tail's are warps of their own, requests
// find their groups for themselves, and loops are not unrolled.
constexpr int kHeadThreads = 64;

// A unit of either kind, by the thread that owns it: its first page's position, pages, their
// cost, bins, descriptors.
struct Unit {
    int S = 0, n = 0, w = 1, bin = 0, count = 0;
};

__device__ __forceinline__ Unit unit_of(int S, int n, int w, int budget, float inv) {
    Unit u;
    u.S = S;
    u.n = n;
    u.w = w;
    if (n == 0) return u;
    u.bin = quotient(S, budget, inv);
    u.count = quotient(S + w * (n - 1), budget, inv) - u.bin + 1;
    return u;
}

// Descriptors of a unit that spans several bins: put(owner's lane or -1 for one's own, i,
// first page, end) for each.  A thread writes the first kOwn of its own unit, its warp the
// others (a long prefix of few requests is one unit of as many descriptors as there are
// CTAs).
constexpr int kOwn = 16;

__device__ __forceinline__ int page_from(int x, int w) {  // the first that begins at x or later
    return w == kPairCost    ? (x + kPairCost - 1) / kPairCost
           : w == kAloneCost ? (x + kAloneCost - 1) / kAloneCost
                             : x;
}

template <class Put>
__device__ __forceinline__ void write_chunks(const Unit &u, int budget, Put put) {
    const int lane = threadIdx.x & 31;
    int lo = 0;
#pragma unroll 1
    for (int i = 0; i < min(u.count, kOwn); ++i) {
        const int hi = i == u.count - 1 ? u.n : page_from((u.bin + i + 1) * budget - u.S, u.w);
        put(-1, i, lo, hi);
        lo = hi;
    }
#pragma unroll 1
    for (unsigned many = __ballot_sync(kFull, u.count > kOwn); many; many &= many - 1) {
        const int of = __ffs(many) - 1, count = __shfl_sync(kFull, u.count, of);
        const int S = __shfl_sync(kFull, u.S, of), n = __shfl_sync(kFull, u.n, of);
        const int w = __shfl_sync(kFull, u.w, of), bin = __shfl_sync(kFull, u.bin, of);
#pragma unroll 1
        for (int i0 = kOwn; i0 < count; i0 += 32) {
            const int i = i0 + lane;
            put(of, i < count ? i : -1, page_from((bin + i) * budget - S, w),
                i == count - 1 ? n : page_from((bin + i + 1) * budget - S, w));
        }
    }
}

// The last group whose entry in `first` is not behind i.
__device__ __forceinline__ int last_from(const int *first, int groups, int i) {
    int lo = 0, hi = groups;
#pragma unroll 1
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const SharedPlan p) {
    // of each request: its length, then the tail tiles of the requests up to it; its
    // group where it shares, else -1; the tails up to it.  Of each group: first request,
    // shared pages, sharing requests, the first and last of them, units and cost of the
    // groups before it
    extern __shared__ int s_mem[];
    int *s_end = s_mem, *s_of = s_end + p.B, *s_tail = s_of + p.B;
    int *g_start = s_tail + p.B, *g_np = g_start + p.groups + 1, *g_count = g_np + p.groups;
    int *g_lead = g_count + p.groups, *g_last = g_lead + p.groups;
    int *g_unit = g_last + p.groups, *g_cost = g_unit + p.groups;
    __shared__ int s_scan[4 * 32];
    __shared__ unsigned s_flags;
    __shared__ int s_bad, s_first, s_last;
    const int tid = threadIdx.x, lane = tid & 31, threads = blockDim.x;
    if (tid == 0) s_flags = 0, s_bad = 0, s_first = p.groups, s_last = -1;
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();
    unsigned flags = 0;
#pragma unroll 1
    for (int i = tid; i < p.B || i <= p.groups; i += threads) {
        // (the loads in flight together)
        const int L = i < p.B ? p.seqlens[i] : 0;
        const int start = p.groups > 0 && i <= p.groups ? p.starts[i] : 0;
        const int next = i < p.groups ? p.starts[i + 1] : start;
        const int np = i < p.groups ? p.prefix[i] : 0;
        const bool bad_len = L < 0 || L > p.max_pages * kTile, bad_np = np < 0 || np > p.max_pages;
        if (start < 0 || next < start || next > p.B) s_bad = 1;
        if (bad_len || bad_np) flags |= HPC_FLAG_BAD_SEQLEN;
        if (i < p.B) s_end[i] = min(max(L, 0), p.max_pages * kTile);
        if (i <= p.groups) g_start[i] = start;
        if (i < p.groups) {
            g_np[i] = bad_np ? 0 : np;
            g_count[i] = 0;
            g_lead[i] = p.B;
            g_last[i] = -1;
        }
    }
    __syncthreads();
    const bool bad = s_bad != 0;
    if (bad) flags |= HPC_FLAG_BAD_SEQLEN;

    // who shares: a request all of whose queries see all of its group's pages, with another
    // one that does
    const int tpb = head_tokens(p.G);
#pragma unroll 1
    for (int r0 = tid - lane; r0 < p.B; r0 += threads) {
        const int r = r0 + lane;
        int g = -1;
        if (r < p.B && !bad && p.groups > 0 && r >= g_start[0] && r < g_start[p.groups]) {
            const int lo = last_from(g_start, p.groups, r);
            if (g_np[lo] > 0 && s_end[r] >= g_np[lo] * kTile + p.q_len - 1) g = lo;
        }
        if (r < p.B) s_of[r] = g;
        // (one set of atomics for a warp whose requests share one group, as most do)
        const int top = __reduce_max_sync(kFull, g);
        const unsigned same = __ballot_sync(kFull, g == top), any = __ballot_sync(kFull, g >= 0);
        if (any == 0) continue;
        if ((any & ~same) == 0) {
            if (lane == __ffs(any) - 1) {
                atomicAdd(g_count + g, __popc(any));
                atomicMin(g_lead + g, r);
                atomicMax(g_last + g, r0 + 31 - __clz(any));
            }
        } else if (g >= 0) {
            atomicAdd(g_count + g, 1);
            atomicMin(g_lead + g, r);
            atomicMax(g_last + g, r);
        }
    }
    __syncthreads();

    // units and pages' costs of the groups, tail tiles and tails of the requests, and
    // their running sums
    auto row_tiles = [&](int g) {
        return ((g_last[g] - g_lead[g] + 1) * p.q_len + tpb - 1) / tpb;
    };
    int units = 0, pages = 0, tiles = 0, tails = 0;
#pragma unroll 1
    for (int base = 0; base < max(p.B, p.groups); base += threads) {
        const int i = base + tid;
        int v[4] = {0, 0, 0, 0}, total[4];
        if (i < p.groups && g_count[i] >= 2) {
            const int nb = row_tiles(i);
            v[0] = p.Hkv * ((nb + 1) / 2);
            v[1] = p.Hkv * g_np[i] * ((nb / 2) * kPairCost + (nb & 1) * kAloneCost);
            atomicMin(&s_first, i);  // the first and the last group with units
            atomicMax(&s_last, i);
        }
        if (i < p.B) {
            int L = s_end[i];
            const int g = s_of[i];
            if (g >= 0 && g_count[g] >= 2) L -= g_np[g] * kTile;
            else s_of[i] = -1;
            v[2] = (L + kTile - 1) / kTile;
            v[3] = v[2] > 0;
        }
        const int u = v[0], c = v[1];
        block_inclusive_scans(v, s_scan, total);
        if (i < p.groups) {
            g_unit[i] = units + v[0] - u;
            g_cost[i] = pages + v[1] - c;
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
    const int tail_units = p.Hkv / p.heads;  // per request

    // What a unit costs beside its pages counts where a CTA has several microseconds of
    // work; with less, the floor alone says how finely units are cut.  (Steps with thresholds of
    // 0, 1, 2 and 8 us: 4 requests behind 960 tokens, BF16, 14.1, 13.2, 13.2 and 13.3 us; 8
    // behind 2K, 64 heads, E4M3, 17.8, 17.8, 21.5 and 21.5; 16 behind 4K, 16 heads, 21.4, 26.5,
    // 26.5 and 26.5; 12 behind 8K, 64 heads, 27.4, 27.4, 27.4 and 30.4: a lower one would suit
    // the batches between better.)
    const float head_us = (float)pages * p.head_us, tail_us = (float)(tail_units * tiles) * p.tail_us;
    const bool busy = head_us + tail_us > 2.f * p.num_ctas;
    int start = busy ? p.head_start : 0;
    const int tail_start = busy ? p.tail_start : 0;
    int cost = pages + units * start;
    const int N = tiles + tails * tail_start, T = tail_units * N;
    // CTAs: where the tail's HBM time is what everything takes, no more for it than
    // that needs; else in proportion to the times
    const float head = (float)cost * p.head_us, tail = (float)T * p.tail_us;
    const float stream = (float)(tail_units * tiles) * p.stream_us;
    const float time = fmaxf((head + tail) / p.num_ctas, stream);
    const int most = T > 0 ? p.num_ctas - 1 : p.num_ctas;
    const int want = cost > 0 ? max((int)fminf(ceilf(head / time), (float)most), 1) : 0;
    int budget = max(want > 0 ? (cost + want - 1) / want : 0,
                     start + kPairCost * max(p.floor, 1));
    __syncthreads();  // the sums are complete
    const int last_nb = units > 0 ? row_tiles(s_last) : 0;
    int last_w = last_nb & 1 ? kAloneCost : kPairCost;
    if (busy && s_first == s_last && (last_nb == 1 || !(last_nb & 1))) {
        // Units alike (one group's, all of pairs or all alone): the same number of CTAs for
        // each, and bins that end with the units, so that no CTA has parts of two: a second
        // descriptor costs as much as `start`, and the slowest CTA is waited for.
        const int pages_cost = last_w * g_np[s_last];
        float best = time + p.head_start * p.head_us;
        for (int k = max(want / units, 1), i = 0; i < 2; ++i, ++k) {
            const int ctas = units * k, b = (pages_cost + k - 1) / k;
            if (ctas > most || b < k + kPairCost * max(p.floor, 1)) break;
            const float t = fmaxf((b + p.head_start) * p.head_us,
                                  fmaxf(T > 0 ? tail / (p.num_ctas - ctas) : 0.f, stream));
            if (t < best) {
                best = t;
                budget = b;
                start = k * b - pages_cost;  // (below k: what fills the unit's last bin)
            }
        }
        cost = pages + units * start;
    }
    // up to the bin in which the last page begins
    const int np_ctas = units > 0 ? (cost - last_w) / budget + 1 : 0;
    const int tail_ctas = max(p.num_ctas - np_ctas, 1);
    const int tail_budget = max((T + tail_ctas - 1) / tail_ctas, tail_start + max(p.floor, 1));

    // the descriptors of the head, by the last warps, and of the tail, by the others
    const bool for_head = p.groups > 0 && tid >= threads - kHeadThreads;
    const int own_threads = for_head ? kHeadThreads : threads - (p.groups > 0 ? kHeadThreads : 0);
    const int own = for_head ? tid - (threads - kHeadThreads) : tid;
    const int line = for_head ? budget : tail_budget;
    const float line_inv = 1.f / (float)line, B_inv = 1.f / (float)max(p.B, 1);
    int num_head = 0, num_desc = 0;
#pragma unroll 1
    for (int k = 0;; ++k) {
        const int u = k * own_threads + own;
        Unit un;
        int h = 0, x = 0, y = 0, z = 0, prev = 0;  // head: group's numbers; tail: request, pages before
        if (for_head && u < units) {
            // (the last group with g_unit <= u has units)
            const int g = last_from(g_unit, p.groups, u), nb = row_tiles(g), pairs = (nb + 1) / 2, i = u - g_unit[g];
            h = quotient(i, pairs, 1.f / (float)pairs);
            const int pair = i - h * pairs, n = g_np[g];
            // of its first page
            const int S = g_cost[g] + u * start + start + pair * n * kPairCost +
                          h * n * ((nb / 2) * kPairCost + (nb & 1) * kAloneCost);
            un = unit_of(S, n, 2 * pair + 1 < nb ? kPairCost : kAloneCost, line, line_inv);
            // what a page of the unit before costs
            prev = pair > 0            ? 0
                   : h > 0 || u == 0 ? nb & 1
                                     : row_tiles(last_from(g_unit, p.groups, u - 1)) & 1;
            prev = prev ? kAloneCost : kPairCost;
            z = g_lead[g];
            x = z * p.q_len + 2 * pair * tpb;
            y = min(z * p.q_len + nb * tpb, g_start[g + 1] * p.q_len);
        } else if (!for_head && u < tail_units * p.B) {
            h = quotient(u, p.B, B_inv);
            x = u - h * p.B;
            const int n = s_end[x] - (x ? s_end[x - 1] : 0);
            if (s_of[x] >= 0) y = g_np[s_of[x]];
            // of its first tile
            un = unit_of(h * N + s_end[x] - n + s_tail[x] * tail_start, n, 1, line, line_inv);
        }
        int v[2] = {for_head ? un.count : 0, for_head ? 0 : un.count}, total[2];
        block_inclusive_scans(v, s_scan, total);
        const int off = (for_head ? num_head + v[0] : num_desc + v[1]) - un.count;
        num_head += total[0];
        num_desc += total[1];
        if (for_head && u < units) p.head.unit[u] = make_int2(off, un.count);
        if (!for_head && u < tail_units * p.B) {
            p.chunk_count[u] = un.count;
            p.chunk_off[u] = off;
        }
        if (for_head) {
            write_chunks(un, line, [&](int of, int i, int lo, int hi) {
                int a = h, b = x, c = y, d = z, at = off, bin = un.bin, w = un.w;
                if (of >= 0) {
                    a = __shfl_sync(kFull, h, of), b = __shfl_sync(kFull, x, of);
                    c = __shfl_sync(kFull, y, of), d = __shfl_sync(kFull, z, of);
                    at = __shfl_sync(kFull, off, of), bin = __shfl_sync(kFull, un.bin, of);
                    w = __shfl_sync(kFull, un.w, of);
                    if (i < 0) return;
                }
                p.head.desc[2 * (at + i)] = make_int4(a, b, c, d);
                p.head.desc[2 * (at + i) + 1] = make_int4(lo, hi, w == kPairCost, 0);
                // the first that begins in its bin: the unit before has its last page earlier
                if (i > 0 || un.S - start - prev < bin * line) p.head.bin[bin + i] = at + i;
            });
        } else {
            write_chunks(un, line, [&](int of, int i, int lo, int hi) {
                int a = h, b = x, c = y, at = off, bin = un.bin;
                if (of >= 0) {
                    a = __shfl_sync(kFull, h, of), b = __shfl_sync(kFull, x, of);
                    c = __shfl_sync(kFull, y, of), at = __shfl_sync(kFull, off, of);
                    bin = __shfl_sync(kFull, un.bin, of);
                    if (i < 0) return;
                }
                p.desc[at + i] = make_int4(a, b, c + lo, c + hi);
                if (i > 0 || un.S - tail_start <= bin * line) p.bin_ptr[np_ctas + bin + i] = at + i;
            });
        }
        // (the same number of rounds for all threads)
        if ((k + 1) * kHeadThreads >= units &&
            (k + 1) * (threads - (p.groups > 0 ? kHeadThreads : 0)) >= tail_units * p.B)
            break;
    }
#pragma unroll 1
    for (int r = tid; r < p.B; r += threads) {
        const int g = s_of[r];
        p.head.req[r] = g < 0 ? make_int4(0, 0, 0, 0)
                              : make_int4(g_np[g], g_unit[g], g_lead[g] * p.q_len, row_tiles(g));
    }
    const int used = np_ctas + (T + tail_budget - 1) / tail_budget;
#pragma unroll 1
    for (int b = tid; b <= p.num_ctas; b += threads) {
        if (b >= np_ctas) p.head.bin[b] = num_head;
        if (b >= used) p.bin_ptr[b] = num_desc;
        if (b < np_ctas) p.bin_ptr[b] = 0;
    }
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
// CTAs of an SM: as many rows in flight as there are registers for (with eight the kernel
// spilled and took 3.5 us longer).
constexpr int kJoinWarps = 4, kJoinCtas = 7;
constexpr int kJoinAhead = 6;  // partials of a row on their way together
constexpr float kJoinLog2e = 1.4426950408889634f;

struct JoinArgs {
    const float *tail_o, *tail_lse, *head_o, *head_lse;
    const int32_t *chunk_count, *chunk_off;
    HeadPlan plan;
    int B, Hq, G, q_len;  // G query heads of a KV head
    int tail_heads;       // KV heads of a tail descriptor
};

// One warp per query row, lane i dims 4 i .. 4 i + 3: out = sum_c w_c o_c / sum_c w_c with
// w_c = exp(lse_c - max), over the row's partials of the tail and of the head.  A partial
// that is NaN, or whose lse is, makes the row NaN.
__global__ void __launch_bounds__(32 * kJoinWarps, kJoinCtas)
    shared_join_kernel(const JoinArgs a, __nv_bfloat16 *__restrict__ out) {
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x * kJoinWarps + (threadIdx.x >> 5);  // (r * q_len + i) * Hq + hq
    const bool any = row < a.B * a.q_len * a.Hq;
    // The plan is read ahead of the attention's end: its kernel had finished before the
    // attention's let this one start.
    int n_tail = 0, n = 0;
    size_t tail = 0, head = 0;  // the row's first partial, in rows
    uint32_t tail_step = 0, head_step = 0;
    if (any) {
        const int ri = row / a.Hq, hq = row - ri * a.Hq;
        const int r = ri / a.q_len, i = ri - r * a.q_len;
        const int Gt = a.tail_heads * a.G, ht = hq / Gt;
        n_tail = n = a.chunk_count[ht * a.B + r];
        tail_step = a.q_len * Gt;
        tail = (size_t)a.chunk_off[ht * a.B + r] * tail_step + i * Gt + (hq - ht * Gt);
        const int4 req = a.plan.req[r];
        if (req.x > 0) {
            const int h = hq / a.G, tpb = head_tokens(a.G);
            const int tok = ri - req.z, tile = tok / tpb;
            const int2 un = a.plan.unit[req.y + h * ((req.w + 1) / 2) + tile / 2];
            const bool alone = tile + 1 == req.w && (tile & 1) == 0;
            n += alone ? 2 * un.y : un.y;
            head_step = (alone ? 1 : 2) * kHeadRows;
            head = (size_t)(2 * un.x + (tile & 1)) * kHeadRows + (tok - tile * tpb) * a.G +
                   (hq - h * a.G);
        }
    }
    grid_dependency_wait();
    if (!any) return;
    auto lse = [&](int c) {
        return c < n_tail ? a.tail_lse[tail + (size_t)c * tail_step]
                          : a.head_lse[head + (size_t)(c - n_tail) * head_step];
    };
    float4 x[kJoinAhead];
    auto load = [&](int k) {  // partials k .. (none past the last)
#pragma unroll
        for (int j = 0; j < kJoinAhead; ++j) {
            const int c = k + j;
            if (c >= n) break;
            const float *p = c < n_tail
                                 ? a.tail_o + (tail + (size_t)c * tail_step) * kHeadDim
                                 : a.head_o + (head + (size_t)(c - n_tail) * head_step) * kHeadDim;
            x[j] = reinterpret_cast<const float4 *>(p)[lane];
        }
    };
    load(0);  // (on their way with the log-sum-exps)
    const float own = lane < n ? lse(lane) : -INFINITY;
    float m = own;
    for (int c = 32 + lane; c < n; c += 32) m = fmaxf(m, lse(c));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    // ws: the weights of kRound partials, one per lane; -1: no values are there (a head's
    // partial that saw no page, whose lse says so).  A weight that is zero because the lse lies
    // far below the others' counts: NaN times zero is NaN.
    float wsum = 0.f, ws = -1.f;
    constexpr int kRound = 32 / kJoinAhead * kJoinAhead;
    int in = kRound;  // the round's partials before k
#pragma unroll 1
    for (int k = 0; k < n; k += kJoinAhead, in += kJoinAhead) {
        if (in == kRound) {
            in = 0;
            const float l = k == 0 ? own : k + lane < n ? lse(k + lane) : -INFINITY;
            ws = l != -INFINITY ? ex2((l - m) * kJoinLog2e) : k + lane < n_tail ? 0.f : -1.f;
        }
#pragma unroll
        for (int j = 0; j < kJoinAhead; ++j) {
            const float w = __shfl_sync(kFull, ws, in + j);
            if (k + j >= n || w < 0.f) continue;
            wsum += w;
            acc.x += w * x[j].x;
            acc.y += w * x[j].y;
            acc.z += w * x[j].z;
            acc.w += w * x[j].w;
        }
        load(k + kJoinAhead);
    }
    const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
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
    auto smem_bytes = [](size_t B, size_t groups) { return (3 * B + 7 * groups + 1) * sizeof(int); };
    const size_t smem = smem_bytes(p.B, p.groups);
    if (smem > 48 * 1024) {
        // always the largest size: the attribute is the process's, and one that followed the
        // calls could be lowered by another thread between here and the launch
        const cudaError_t e = cudaFuncSetAttribute(
            shared_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
            (int)smem_bytes(HPC_MAX_SHARED_BATCH, HPC_MAX_SHARED_GROUPS));
        if (e != cudaSuccess) return e;
    }
    const long long work = max((long long)p.B * (p.Hkv / p.heads), (long long)p.groups + 1);
    const int own = p.groups > 0 ? kHeadThreads : 0;
    const int threads =
        own + (int)min(max((work + 31) / 32 * 32, 64LL), (long long)(kPlanThreads - own));
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
