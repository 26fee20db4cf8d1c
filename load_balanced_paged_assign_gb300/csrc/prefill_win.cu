// Windowed extend / prefill attention with sinks over the paged BF16 cache, on
// the fifth-generation tensor cores: query position p sees token j <= p when
// j > p - window or j < sinks.
//
// Two 128-row Q tiles share every KV page: S = Q_x K^T into TMEM, one softmax
// thread per row (online, in fp32: a reference that moves when a score passes it
// by 2^8, P written over the scores as BF16, half a step of 2^-8), O_x += P V with
// P read from TMEM.  Within an item the tensor pipe bounds it: at N = 64 the scores'
// MMAs are limited by their operands' reads from shared memory (A 32 KB + B 16 KB at
// 128 bytes a cycle, 384 cycles; O's take 256), 1250 cycles a page for both Q tiles,
// timed alone in alternation, where a page takes 1430 (softmax 1075, its wait for the
// scores 355).  Of the launch that is 78%: an item of 8192 queries with a window of
// 1024 takes 31.9k cycles, 24.7k of them for its 17.3 pages, 0.7k until its first
// scores, 3.0k from its last to its output (0.9k of it the last product) and 3.5k for
// its bookkeeping and its share of the launch's start.  So the pipe multiplies in 57%
// of the launch's cycles (1024 of 1430 would be 72%).
//   * The unit is a page, not two.  A Q tile has two 64-column score buffers in
//     TMEM, and its scores run two pages ahead of its products, so that the
//     softmax of a page meets the next one's scores ready (with one buffer of 128,
//     and one issuing warp for both Q tiles, it waited for 2100 to 2600 of a tile's
//     5300 cycles).  Only pages that some row sees are computed, and 64 scores leave
//     registers for the masks.
//   * Each Q tile has its own MMA warp: an issuing warp stands still while its
//     MMAs wait for the pipe, and one for both tiles left the pipe idle for half
//     of a page.  What these warps compute per page is held to a few uniform
//     instructions, and one barrier stands for a page of K and V.
//   * Where the GQA group is even a pair is the same rows of two heads: both Q
//     tiles see the same pages (18 instead of 20 with a window of 1024) and end
//     together.  Else it is two Q tiles of one head.
//   * The CTAs are persistent, one per SM: the next item's Q and pages come in
//     while this one's last scores are taken, and its first scores are computed
//     while the output goes out, by TMA through shared memory.  (Reading O out by
//     warps of their own gains nothing, 231 us against 231 with the softmax at 128
//     registers and 246 with more; stores of 32 bytes a lane instead of TMA: 238.)
//   * Tokens that no query of the pair sees (past L_r, or before the window and no
//     sink) may hold anything: a warp of its own zeroes their V rows once the page
//     has landed (0 * NaN would reach O) and passes every page on.
// 8192 queries of 64 heads with a window of 1024 and 64 sinks (273 GFLOP): 237 us,
// 1150 TFLOP/s (250 us in long runs, under the power limit); 2 x 1000 behind 3111
// tokens with a window of 2000 (132 GFLOP): 127 us; 512 with 128: 12.7 us.
//
// All barrier phases are counted across items.  Every wait is bounded; on a
// timeout the CTA raises the error flag, waits (bounded) for its copies and
// MMAs in flight, frees TMEM and leaves.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>

#include "internal.h"
#include "prefill_common.cuh"
#include "tcgen05.cuh"

namespace hpc {
namespace {

constexpr int kStages = 4;                    // depth of the ring, in pages of K and V
constexpr int kPageHalf = kTile * 128;        // 64 tokens x 64 dims
constexpr int kPageBytes = 2 * kPageHalf;     // a page of K or V of one head
constexpr int kCleanWarp = kMmaWarp + kQT;    // (an MMA warp for each Q tile)
constexpr int kWinThreads = (kCleanWarp + 1) * 32;
// TMEM: the scores of Q tile x's even and odd pages at 128 x and 128 x + 64
// (P over their first 32 columns), O_x at kOCol + 128 x
constexpr int kOffQ = 0;
constexpr int kOffK = kOffQ + kQT * kTileBytes;
constexpr int kOffV = kOffK + kStages * kPageBytes;
constexpr int kOffO = kOffV + kStages * kPageBytes;  // [x]: half of an output tile, BF16
constexpr int kOffBar = kOffO + kQT * kHalf;
// barriers: q_full, q_free, full[S], ready[S], empty[S], s_full[x][2],
// p_full[x][2], o_done[x][2], o_free[x], mma_done, end
constexpr int kNumBars = 2 + 3 * kStages + 7 * kQT + 2;
constexpr int kOffMisc = kOffBar + kNumBars * 8;  // tmem slot, abort word
constexpr int kSmemBytes = kOffMisc + 16 + 1024;  // + alignment slack
static_assert(kSmemBytes <= 227 * 1024, "shared memory over the per-CTA limit");

struct WinArgs {
    const int32_t *seqlens;
    const int32_t *block_table;
    int32_t *flags;
    int B, Hq, G, q_len, max_pages, num_pages, n_qp;
    int heads;         // query heads of a pair: 2 (of one Q tile each), or 1 (of two)
    int pairs, items;  // items: `pairs` pairs of Q tiles, then single Q tiles
    int window, sinks;
    float score_scale;  // sm_scale * log2(e)
};

// What a Q tile sees of an item's KV pages: the first n1, and those from n1 +
// gap on, cnt in all.
struct Seen {
    int n1, gap, cnt;
    __device__ __forceinline__ bool sees(int c) const {
        return c < n1 || (c >= n1 + gap && c < gap + cnt);
    }
};

// One item: a request and a pair of Q tiles (or one of them, the first of the
// two then), with the KV pages it reads.  A pair is the same rows of two query
// heads of a KV head, which see the same pages, where the group is even, and
// else two tiles of one head.
struct Item {
    bool single;
    int r, hq, i0, L;
    int dh, di;            // the second tile's head and first row, less the first's
    int n;                 // its KV pages
    int sink_pages, skip;  // pages that hold sinks; pages left out behind them
    int lo;                // first token of the window of its first query
    Seen a, b;             // what the first and the second Q tile see of its pages

    // the item's page c among the request's
    __device__ __forceinline__ int page(int c) const { return c < sink_pages ? c : c + skip; }
    // (selected, not indexed: an item stays in registers)
    __device__ __forceinline__ Seen seen(int x) const { return x ? b : a; }
    // no query of the pair sees token t: past the end, or before the window
    // and no sink
    __device__ __forceinline__ bool dead(int t, int sinks) const {
        return t >= L || (t < lo && t >= sinks);
    }
    // page g holds such a token
    __device__ __forceinline__ bool dirty(int g, int sinks) const {
        const int t = g * kTile;
        return t + kTile > L || max(t, sinks) < min(t + kTile, lo);
    }
};

// The pair of item idx.  Where the pairs leave a last round that fills at most
// half of the CTAs, its pairs are halved (see the launch).
__device__ __forceinline__ int pair_of(const WinArgs &a, int idx) {
    return idx < a.pairs ? idx : a.pairs + ((idx - a.pairs) >> 1);
}

// Item idx: the last query tiles first, the heads that share a KV head side by
// side (they read the same K and V at the same time).
__device__ __forceinline__ Item item_of(const WinArgs &a, int item, int L) {
    Item it;
    const int idx = pair_of(a, item);
    it.single = item >= a.pairs;
    const int per_req = a.Hq / a.heads, per_qp = a.B * per_req;
    const int qp = a.n_qp - 1 - idx / per_qp, rem = idx % per_qp;
    const int second = it.single ? (item - a.pairs) & 1 : 0;
    it.dh = a.heads - 1;
    it.di = a.heads == 2 ? 0 : kQB;
    it.r = rem / per_req;
    it.hq = rem % per_req * a.heads + second * it.dh;
    it.i0 = qp * (kQB + it.di) + second * it.di;
    it.L = L;
    it.lo = max(L - a.q_len + it.i0 + 1 - a.window, 0);
    it.sink_pages = a.sinks / kTile + (a.sinks % kTile ? 1 : 0);
    it.skip = max(it.lo / kTile - it.sink_pages, 0);
    it.n = 0;
    auto seen = [&](int x) {
        Seen v = {0, 0, 0};
        const int first = it.i0 + x * it.di;
        // the last token its last query sees, the first of its first query's window
        const int lim = min(L - a.q_len + min(first + kQB - 1, a.q_len - 1), L - 1);
        const int lo = max(L - a.q_len + first + 1 - a.window, 0);
        if (first < a.q_len && lim >= 0 && (x == 0 || !it.single)) {
            const int last = lim / kTile;
            v.n1 = min(it.sink_pages, last + 1);
            v.gap = max(lo / kTile - it.skip, it.sink_pages) - v.n1;
            v.cnt = max(last + 1 - it.skip - v.gap, v.n1);
            // (a window's first page is not behind the last token its query sees, so
            // with pages left out there are some behind them)
            it.n = max(it.n, last + 1 - it.skip);
        }
        return v;
    };
    it.a = seen(0);
    it.b = seen(1);
    return it;
}

// A value that is the same in every lane, as one that the compiler knows to be:
// the MMAs take their operands from uniform registers, and moving each there
// costs more than the MMA.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __reduce_or_sync(0xffffffffu, v); }

// acc += a BF16 value, without widening it first (the widened pairs in paired adds:
// 241 us for 8192 queries instead of 237).
__device__ __forceinline__ void add_bf16(float &acc, uint16_t x) {
    asm("add.f32.bf16 %0, %1, %0;" : "+f"(acc) : "h"(x));
}

// The low bits up to and with bit k.
__device__ __forceinline__ uint64_t bits_to(int k) {
    return k < 0 ? 0ull : k >= 63 ? ~0ull : (2ull << k) - 1;
}

__device__ __forceinline__ int clamped_len(const WinArgs &a, int item) {
    const int per_req = a.Hq / a.heads;
    const int L = __ldg(a.seqlens + pair_of(a, item) % (a.B * per_req) / per_req);
    return min(max(L, 0), a.max_pages * kTile);
}

__global__ void __launch_bounds__(kWinThreads, 1)
    prefill_win_kernel(const __grid_constant__ CUtensorMap tq,
                       const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv,
                       const __grid_constant__ CUtensorMap to, const WinArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kOffBar);
    uint64_t *q_full = bars, *q_free = bars + 1;
    uint64_t *full = bars + 2;             // [stage]: K and V of a page have landed
    uint64_t *ready = full + kStages;      // [stage]: and the dead rows of V are zeroed
    uint64_t *empty = ready + kStages;     // [stage]: its products are done
    uint64_t *s_full = empty + kStages;    // [x][b]: the scores of an even or odd page
    uint64_t *p_full = s_full + 2 * kQT;    // [x][b]: its P written (four warps)
    uint64_t *o_done = p_full + 2 * kQT;    // [x][b]: O_x += P V of that page complete
    uint64_t *o_free = o_done + 2 * kQT;    // [x]: O_x read out (four warps)
    uint64_t *mma_done = o_free + kQT, *end = mma_done + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + kOffMisc);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + kOffMisc + 4);

    const int warp = (int)uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        // arrivals: one (an expect-tx arrival or a tcgen05.commit), but from a Q
        // tile's four warps on p_full and o_free, all eight at the end, and for
        // both Q tiles on q_free, empty and mma_done
        for (int b = 0; b < kNumBars; ++b) {
            uint64_t *bar = &bars[b];
            int n = 1;
            if (bar == q_free || bar == mma_done || (bar >= empty && bar < s_full)) n = kQT;
            if ((bar >= p_full && bar < o_done) || (bar >= o_free && bar < mma_done)) n = 4;
            if (bar == end) n = kSoftmaxWarps;
            mbar_init(bar, n);
        }
        *abort = 0;
        fence_barrier_init();
        prefetch_tensormap(&tq);
        prefetch_tensormap(&tk);
        prefetch_tensormap(&tv);
        prefetch_tensormap(&to);
    }
    if (warp == kMmaWarp) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(*tmem_slot);
    grid_dependency_wait();  // Q, the caches and the lengths may come from the previous kernel

    const int step = gridDim.x;
    bool ok = true;
    int next_L = clamped_len(a, blockIdx.x);  // (the grid is at most the items)

    if (warp == kProducerWarp) {
        const uint64_t pol = policy_evict_normal();
        uint32_t kt = 0;       // pages issued
        uint32_t q_items = 0;  // items whose Q has been issued
        for (int idx = blockIdx.x; ok && idx < a.items; idx += step) {
            const Item it = item_of(a, idx, (int)uniform(next_L));
            if (lane == 0 && a.flags && it.hq == 0 && it.i0 == 0) {
                const int raw = __ldg(a.seqlens + it.r);
                if (raw < 0 || raw > a.max_pages * kTile)
                    atomicOr(a.flags, (int)HPC_FLAG_BAD_SEQLEN);
            }
            if (idx + step < a.items) next_L = clamped_len(a, idx + step);
            if (it.n == 0) continue;
            if (q_items > 0 && !mbar_wait_warp(q_free, (q_items - 1) & 1u, abort)) {
                ok = false;
                break;
            }
            if (lane == 0) {
                uint32_t bytes = 0;
#pragma unroll
                for (int x = 0; x < kQT; ++x) bytes += it.seen(x).cnt > 0 ? kTileBytes : 0;
                mbar_arrive_expect_tx(q_full, bytes);
#pragma unroll
                for (int x = 0; x < kQT; ++x)
                    if (it.seen(x).cnt > 0)
                        for (int h = 0; h < 2; ++h)
                            tma_load_4d(smem + kOffQ + x * kTileBytes + h * kHalf, &tq, q_full, 0,
                                        h, it.hq + x * it.dh,
                                        it.r * a.q_len + it.i0 + x * it.di, pol);
            }
            ++q_items;
            const int32_t *bt = a.block_table + (size_t)it.r * a.max_pages;
            const int hkv = it.hq / a.G;
            int pg = -1;
            for (int j = 0; j < it.n; ++j, ++kt) {
                if ((j & 31) == 0)  // the entries of 32 pages, one per lane
                    pg = j + lane < it.n ? __ldg(bt + it.page(j + lane)) : 0;
                const int page = __shfl_sync(0xffffffffu, pg, j & 31);
                const bool good = page >= 0 && page < a.num_pages;
                if (!good && lane == 0 && a.flags) atomicOr(a.flags, (int)HPC_FLAG_BAD_PAGE);
                const int s = (int)(kt % kStages);
                ok = mbar_wait_warp(&empty[s], ((kt / kStages) & 1u) ^ 1u, abort);
                if (!ok) break;
                if (lane == 0 && !good) {
                    mbar_arrive(&full[s]);
                } else if (lane == 0) {
                    mbar_arrive_expect_tx(&full[s], 2 * kPageBytes);
                    uint8_t *k = smem + kOffK + s * kPageBytes, *v = smem + kOffV + s * kPageBytes;
                    for (int h = 0; h < 2; ++h)
                        tma_load_5d(k + h * kPageHalf, &tk, &full[s], 0, h, hkv, 0, page, pol);
                    for (int h = 0; h < 2; ++h)
                        tma_load_5d(v + h * kPageHalf, &tv, &full[s], 0, h, hkv, 0, page, pol);
                }
            }
        }
        // no copy may land after the CTA has left: the last one issued into
        // each buffer (bounded)
        __syncwarp();
        if (!ok || *abort) {
            volatile int no_abort = 0;
            if (q_items > 0) mbar_wait(q_full, (q_items - 1) & 1u, &no_abort);
            for (uint32_t t = kt > kStages ? kt - kStages : 0; t < kt; ++t)
                mbar_wait(&full[t % kStages], (t / kStages) & 1u, &no_abort);
            __syncwarp();
        }
    } else if (warp < kCleanWarp && warp >= kMmaWarp) {
        const int x = warp - kMmaWarp;  // the Q tile
        const uint32_t idesc_s = idesc_bf16_f32(kQB, kTile);
        const uint32_t idesc_o = idesc_bf16_f32_bmn(kQB, kHeadDim);
        const uint64_t dq0 = smem_desc_k128(smem_u32(smem + kOffQ));
        const uint64_t dk0 = smem_desc_k128(smem_u32(smem + kOffK));
        const uint64_t dv0 = smem_desc_mn128(smem_u32(smem + kOffV), kPageHalf);
        const uint64_t dq = dq0 + (uint64_t)((x * kTileBytes) >> 4);
        // S = Q_x K^T of a page into score buffer b (K page in stage s)
        auto issue_s = [&](uint32_t b, uint32_t s) {
            const uint64_t dk = dk0 + (uint64_t)((s * kPageBytes) >> 4);
#pragma unroll
            for (int k = 0; k < kHeadDim / 16; ++k) {
                const uint32_t in = (k & 3) * 32;  // bytes within a half's rows
                umma_bf16(tmem + 128 * x + 64 * b, dq + (((k >> 2) * kHalf + in) >> 4),
                          dk + (((k >> 2) * kPageHalf + in) >> 4), idesc_s, k > 0);
            }
            umma_commit(&s_full[2 * x + b]);
        };
        // O_x += P V of a page (V page in stage s), P from TMEM
        auto issue_pv = [&](uint32_t b, uint32_t s, bool acc) {
            const uint64_t dv = dv0 + (uint64_t)((s * kPageBytes) >> 4);
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
                umma_bf16_ts(tmem + kOCol + 128 * x, tmem + 128 * x + 64 * b + 8 * k,
                             dv + (uint64_t)((k * 16 * 128) >> 4), idesc_o, acc || k > 0);
            umma_commit(&o_done[2 * x + b]);
            umma_commit(&empty[s]);  // (this page's scores are done too)
        };
        uint32_t kt = 0, q_items = 0;
        uint32_t sp = 0, pp = 0;  // score pages issued, P pages taken
        uint32_t outs = 0;        // items whose O_x has been claimed
        for (int idx = blockIdx.x; ok && idx < a.items; idx += step) {
            const Item it = item_of(a, idx, (int)uniform(next_L));
            if (idx + step < a.items) next_L = clamped_len(a, idx + step);
            if (it.n == 0) continue;
            const Seen sn = it.seen(x);
            const int n1 = sn.n1, gap = sn.gap, cnt = sn.cnt;
            ok = mbar_wait_warp(q_full, q_items & 1u, abort);
            ++q_items;
            // The scores run two pages ahead of the products: both buffers are then
            // in use, one at the softmax and one being filled.  (Pages that the Q
            // tile does not see are passed by: at most two together, and all of an
            // item have landed when the next one's Q has, so a stage's phases are
            // met in order.)
            uint32_t ks = kt + (n1 == 0 ? gap : 0), vs = ks;  // pages of the next scores, products
            for (int c = -2; c < cnt; ++c) {
                const bool next = c + 2 < cnt;
                // behind a gap the next page waits for the stage that this product frees
                const bool late = next && ks - vs >= kStages;
                if (next && !late)
                    ok = mbar_wait_warp(&ready[ks % kStages], (ks / kStages) & 1u, abort);
                if (ok && c >= 0) {
                    ok = mbar_wait_warp(&p_full[2 * x + (pp & 1u)], (pp >> 1) & 1u, abort);
                    if (ok && c == 0 && outs++ > 0)  // O_x of the item before is out
                        ok = mbar_wait_warp(&o_free[x], (outs - 2) & 1u, abort);
                }
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    if (c >= 0) issue_pv(pp & 1u, vs % kStages, c > 0);
                    if (next && !late) issue_s(sp & 1u, ks % kStages);
                }
                __syncwarp();
                if (late) {
                    ok = mbar_wait_warp(&ready[ks % kStages], (ks / kStages) & 1u, abort);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) issue_s(sp & 1u, ks % kStages);
                    __syncwarp();
                }
                if (c + 3 == cnt || (c == -2 && cnt < 2)) {  // the item's last scores
                    if (elect_one()) umma_commit(q_free);
                    __syncwarp();
                }
                if (c >= 0) {
                    ++pp;
                    vs += c + 1 == n1 ? gap + 1 : 1;
                }
                if (next) {
                    ++sp;
                    ks += c + 3 == n1 ? gap + 1 : 1;
                }
            }
            kt += it.n;
        }
        // arrives once every MMA issued has completed (TMEM is freed after it)
        if (elect_one()) umma_commit(mma_done);
        __syncwarp();
    } else if (warp == kCleanWarp) {
        // zeroes the V rows that no query of the pair sees, and lets go of a page
        // for a Q tile that does not see it
        uint32_t kt = 0;
        for (int idx = blockIdx.x; ok && idx < a.items; idx += step) {
            const Item it = item_of(a, idx, (int)uniform(next_L));
            if (idx + step < a.items) next_L = clamped_len(a, idx + step);
            for (int j = 0; j < it.n; ++j, ++kt) {
                const uint32_t s = kt % kStages;
                ok = mbar_wait_warp(&full[s], (kt / kStages) & 1u, abort);
                if (!ok) break;
                const int g = it.page(j);
                if (it.dirty(g, a.sinks)) {
                    const uint32_t vs = smem_u32(smem + kOffV + s * kPageBytes);
                    for (int e = lane; e < kTile * 8; e += 32)
                        if (it.dead(g * kTile + (e >> 3), a.sinks))
                            for (int h = 0; h < 2; ++h)
                                sts128(vs + h * kPageHalf + e * 16, 0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (lane == 0) {
                    mbar_arrive(&ready[s]);
#pragma unroll
                    for (int x = 0; x < kQT; ++x)
                        if (!it.seen(x).sees(j)) mbar_arrive(&empty[s]);
                }
            }
        }
    } else {
        // softmax of Q tile x: thread = one query row, warp w reads TMEM
        // lanes 32 (w mod 4) ..
        const int x = warp >> 2, q4 = warp & 3;
        const int rho = 32 * q4 + lane;
        const uint32_t row = tmem + ((uint32_t)(32 * q4) << 16);
        const uint32_t scol = row + 128 * x, ocol = row + kOCol + 128 * x;
        const float sc = a.score_scale;
        uint32_t ns = 0;  // score pages taken
        for (int idx = blockIdx.x; ok && idx < a.items; idx += step) {
            const Item it = item_of(a, idx, (int)uniform(next_L));
            if (idx + step < a.items) next_L = clamped_len(a, idx + step);
            if (x > 0 && it.single) continue;
            const int first = it.i0 + x * it.di;
            // the tokens the row sees, and those that all of the warp's rows see
            const int p0 = it.L - a.q_len + first + 32 * q4;
            const int lim = min(p0 + lane, it.L - 1), lo = p0 + lane + 1 - a.window;
            const int lim_all = min(p0, it.L - 1), lo_all = p0 + 32 - a.window;
            const Seen sn = it.seen(x);
            float m_ref = -INFINITY, l = 0.f;
            bool started = false;
            for (int c = 0; c < sn.cnt; ++c) {
                const int t = it.page(c < sn.n1 ? c : c + sn.gap) * kTile;
                const uint32_t b = ns & 1u;
                if (!mbar_wait_warp(&s_full[2 * x + b], (ns >> 1) & 1u, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t ra[32], rb[32];
                tmem_ld32_nowait(scol + 64 * b, ra);
                tmem_ld32_nowait(scol + 64 * b + 32, rb);
                tmem_wait_ld32x2(ra, rb);
                float s[kTile];
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    s[c] = __uint_as_float(ra[c]);
                    s[32 + c] = __uint_as_float(rb[c]);
                }
                // some row of the warp does not see all of it: the diagonal or the
                // end, or tokens before a window that are no sinks
                if (t + kTile - 1 > lim_all || (t < lo_all && t + kTile > a.sinks)) {
                    const uint64_t sees = bits_to(lim - t) &
                                          (~bits_to(lo - 1 - t) | bits_to(a.sinks - 1 - t));
                    const uint32_t w0 = (uint32_t)sees, w1 = (uint32_t)(sees >> 32);
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        if (!(w0 >> c & 1u)) s[c] = -INFINITY;
                        if (!(w1 >> c & 1u)) s[32 + c] = -INFINITY;
                    }
                }
                float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < kTile / 2; ++c)
                    mx4[c & 3] = fmax3(mx4[c & 3], s[2 * c], s[2 * c + 1]);
                const float mx = fmax3(fmaxf(mx4[0], mx4[1]), mx4[2], mx4[3]);
                const float m_tile = mx * sc;
                const bool need = m_tile > m_ref + kRescaleLog2;
                const float new_ref = need ? m_tile : m_ref;
                const float factor = need ? ex2(m_ref - new_ref) : 1.f;
                const float base = new_ref == -INFINITY ? 0.f : new_ref;
                // P as packed BF16 pairs, over the first half of the scores
                uint32_t pk[32];
                const float2 sc2 = make_float2(sc, sc), nb2 = make_float2(-base, -base);
#pragma unroll
                for (int c = 0; c < 32; ++c) {  // two columns per instruction
                    const float2 e = __ffma2_rn(make_float2(s[2 * c], s[2 * c + 1]), sc2, nb2);
                    pk[c] = pack_bf16x2(ex2(e.x), ex2(e.y));
                }
                tmem_st32_nowait(scol + 64 * b, pk);
                // The sum takes the weights as they were rounded: the heaviest one's
                // rounding then cancels against its own in the product, which a row with
                // one heavy token needs, however many it sees (a token that holds nearly
                // all of the weight comes out to its BF16 rounding; with the unrounded
                // sum, 2% faster, twice as far off).
                float ps[8] = {};
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    add_bf16(ps[2 * (c & 3)], (uint16_t)pk[c]);
                    add_bf16(ps[2 * (c & 3) + 1], (uint16_t)(pk[c] >> 16));
                }
                l = l * factor + (((ps[0] + ps[1]) + (ps[2] + ps[3])) +
                                  ((ps[4] + ps[5]) + (ps[6] + ps[7])));
                if (started && __any_sync(0xffffffffu, need)) {
                    // O_x is settled once its last product is done (the product two
                    // before that, the same barrier's last, was issued before these
                    // scores' own: the phase cannot be mistaken)
                    if (!mbar_wait_warp(&o_done[2 * x + (b ^ 1u)], ((ns - 1) >> 1) & 1u, abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        float o[64];
                        tmem_ld32x2(ocol + 64 * hf, ocol + 64 * hf + 32, o);
#pragma unroll
                        for (int c = 0; c < 64; ++c) o[c] *= factor;
                        tmem_st32x2(ocol + 64 * hf, ocol + 64 * hf + 32, o);
                    }
                }
                started = true;
                tmem_wait_st32(pk);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[2 * x + b]);
                m_ref = new_ref;
                ++ns;
            }
            // epilogue: O / l as BF16 (zeros for rows that see nothing)
            bool have = ok && started;
            if (have) {
                if (!mbar_wait_warp(&o_done[2 * x + ((ns - 1) & 1u)], ((ns - 1) >> 1) & 1u, abort))
                    ok = have = false;
                else
                    tc_fence_after();
            }
            // through shared memory (64 dims at a time, the swizzle of the tensor
            // map) and out by TMA, which leaves the rows past q_len alone
            const float inv = l > 0.f ? 1.f / l : 0.f;
            const bool store = ok && !*abort && first < a.q_len;
            uint8_t *stage = smem + kOffO + x * kHalf + rho * 128;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                float o[64];
                if (have) {
                    tmem_ld32x2(ocol + 64 * hf, ocol + 64 * hf + 32, o);
                    if (hf == 1) {  // the next item's products may begin
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&o_free[x]);
                    }
#pragma unroll
                    for (int c = 0; c < 64; ++c) o[c] *= inv;
                } else {
#pragma unroll
                    for (int c = 0; c < 64; ++c) o[c] = 0.f;
                }
                // this warp's last store has left its 32 rows (each warp stores
                // its own, so no other is waited for)
                if (lane == 0) bulk_wait_read();
                __syncwarp();
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    *reinterpret_cast<uint4 *>(stage + ((u ^ (rho & 7)) << 4)) =
                        make_uint4(pack_bf16x2(o[8 * u], o[8 * u + 1]),
                                   pack_bf16x2(o[8 * u + 2], o[8 * u + 3]),
                                   pack_bf16x2(o[8 * u + 4], o[8 * u + 5]),
                                   pack_bf16x2(o[8 * u + 6], o[8 * u + 7]));
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && store && first + 32 * q4 < a.q_len) {
                    tma_store_5d(&to, smem + kOffO + x * kHalf + 32 * q4 * 128, 0, hf,
                                 it.hq + x * it.dh, first + 32 * q4, it.r);
                    bulk_commit_group();
                }
            }
        }
        if (lane == 0) bulk_wait_all();  // (complete before the CTA leaves)
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(end);
    }

    if (!ok) {
        if (a.flags && lane == 0) atomicOr(a.flags, (int)HPC_FLAG_TIMEOUT);
        *abort = 1;
    }
    if (warp == kMmaWarp) {
        // no MMA may still write TMEM, and no softmax warp read it, when it is
        // freed (bounded, like every wait)
        volatile int no_abort = 0;
        mbar_wait(mma_done, 0, &no_abort);
        mbar_wait(end, 0, &no_abort);
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Tensor map over the output [B, q_len, Hq, 128] BF16 as {64 dims, 2 halves,
// Hq, q_len, B}, box {64, 1, 1, 32, 1}: one 64-dim half of a warp's 32 query
// rows of one head; rows past q_len are outside the tensor.
hpc_status make_out_map(CUtensorMap *m, void *out, int32_t B, int32_t q_len, int32_t Hq) {
    auto encode = tensor_map_encoder();
    if (!encode) return HPC_ERR_CUDA;
    std::memset(m, 0, sizeof(*m));
    const cuuint64_t row = (cuuint64_t)Hq * 256;
    cuuint64_t dims[5] = {64, 2, (cuuint64_t)Hq, (cuuint64_t)q_len, (cuuint64_t)B};
    cuuint64_t strides[4] = {128, 256, row, row * (cuuint64_t)q_len};
    cuuint32_t box[5] = {64, 1, 1, 32, 1};
    cuuint32_t elem[5] = {1, 1, 1, 1, 1};
    const CUresult res = encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, out, dims, strides, box,
                                elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_NONE,
                                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return res == CUDA_SUCCESS ? HPC_OK : HPC_ERR_CUDA;
}

std::atomic<int> g_win_sms[64];  // per device: SMs, once the kernel's attribute is set

}  // namespace
}  // namespace hpc

using namespace hpc;

extern "C" hpc_status hpc_prefill_attn_win(const void *d_q, const void *d_k_cache,
                                           const void *d_v_cache, int32_t num_pages,
                                           const int32_t *d_block_table,
                                           int32_t max_pages_per_req, const int32_t *d_seqlens,
                                           int32_t B, int32_t Hq, int32_t Hkv, int32_t head_dim,
                                           int32_t q_len, int32_t window, int32_t sinks,
                                           float sm_scale, void *d_out, int32_t *d_flags,
                                           hpc_stream_t stream) {
    if (window < 0 || sinks < 0 || (window == 0 && sinks != 0)) return HPC_ERR_ARG;
    if (window >= kNoWindow || sinks >= kNoWindow) return HPC_ERR_UNSUPPORTED;
    if (window == 0)
        return hpc_prefill_attn(d_q, d_k_cache, d_v_cache, num_pages, d_block_table,
                                max_pages_per_req, d_seqlens, B, Hq, Hkv, head_dim, q_len,
                                sm_scale, d_out, d_flags, stream);
    if (B < 0 || Hq <= 0 || Hkv <= 0 || max_pages_per_req <= 0 || q_len < 1 || num_pages <= 0)
        return HPC_ERR_ARG;
    if (head_dim != HPC_HEAD_DIM || Hq % Hkv != 0) return HPC_ERR_UNSUPPORTED;
    // scores are masked before they are scaled: the scale may not turn -inf
    // round, nor be flushed to zero, nor make a zero score NaN
    const float score_scale = sm_scale * 1.4426950408889634f;  // times log2(e)
    if (!std::isfinite(score_scale) || !(sm_scale >= FLT_MIN)) return HPC_ERR_ARG;
    if (B == 0) return HPC_OK;
    if (!d_q || !d_k_cache || !d_v_cache || !d_block_table || !d_seqlens || !d_out)
        return HPC_ERR_ARG;
    if (!aligned16(d_q) || !aligned16(d_k_cache) || !aligned16(d_v_cache) || !aligned16(d_out))
        return HPC_ERR_ARG;
    const int G = Hq / Hkv, heads = G % 2 == 0 ? 2 : 1;
    const int rows = heads == 2 ? kQB : kQT * kQB;  // query rows that a pair spans
    const int64_t n_qp = ((int64_t)q_len + rows - 1) / rows;
    const int64_t pairs = n_qp * B * (Hq / heads);
    // (items + a grid's stride, query rows and token indices stay in int32)
    if (pairs >= ((int64_t)1 << 29) || (int64_t)B * q_len >= ((int64_t)1 << 31) ||
        q_len >= kNoWindow || (int64_t)max_pages_per_req * HPC_PAGE_SIZE >= ((int64_t)1 << 30))
        return HPC_ERR_UNSUPPORTED;

    CUtensorMap tq, tk, tv, to;
    hpc_status st = make_q_map(&tq, d_q, (int64_t)B * q_len, Hq);
    if (st == HPC_OK) st = make_out_map(&to, d_out, B, q_len, Hq);
    if (st == HPC_OK) st = cache_tensor_map(&tk, d_k_cache, num_pages, Hkv, false);
    if (st == HPC_OK) st = cache_tensor_map(&tv, d_v_cache, num_pages, Hkv, false);
    if (st != HPC_OK) return st;

    WinArgs a;
    a.seqlens = d_seqlens;
    a.block_table = d_block_table;
    a.flags = d_flags;
    a.B = B;
    a.Hq = Hq;
    a.G = G;
    a.heads = heads;
    a.q_len = q_len;
    a.max_pages = max_pages_per_req;
    a.num_pages = num_pages;
    a.n_qp = (int)n_qp;
    a.window = window;
    a.sinks = sinks;
    a.score_scale = score_scale;

    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return HPC_ERR_CUDA;
    int sms = g_win_sms[dev].load();
    if (sms == 0) {
        if (cudaFuncSetAttribute(prefill_win_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSmemBytes) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            sms < 1)
            return HPC_ERR_CUDA;
        g_win_sms[dev].store(sms);
    }
    // Pairs go round the CTAs.  A last round of few pairs is halved into single
    // Q tiles, which take about 0.65 of a pair's time (they share no K/V tile and
    // overlap nothing): worth it where the halves still fit one round.
    const int64_t rest = pairs % sms;
    a.pairs = (int)(pairs > sms && 2 * rest <= sms ? pairs - rest : pairs);
    a.items = (int)(a.pairs + 2 * (pairs - a.pairs));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min<int64_t>(a.items, sms));
    cfg.blockDim = dim3(kWinThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prefill_win_kernel, tq, tk, tv, to, a) == cudaSuccess
               ? HPC_OK
               : HPC_ERR_CUDA;
}
