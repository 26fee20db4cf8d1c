// Windowed extend / prefill attention with sinks over the paged BF16 cache, on
// the fifth-generation tensor cores: query position p sees token j <= p when
// j > p - window or j < sinks.
//
// The tile work is the causal kernel's (prefill.cu): two 128-row Q tiles share
// every 128-token K/V tile, S_x = Q_x K^T into TMEM, one softmax thread per row
// writing P over the scores, O_x += P_x V with P read from TMEM.  What differs
// follows from a window's items being short (a window of 1024 tokens is 10
// tiles where a causal 8K prompt averages 33):
//   * the CTAs are persistent, one per SM, and an item's start and end overlap
//     its neighbours': the producer brings the next item's Q as soon as the last
//     scores are computed and keeps the K/V ring filled across items, the next
//     item's first scores are issued while this one's output is read out, and
//     TMEM and barriers are set up once.  (One CTA per item, as the causal
//     kernel has them, took 390 us instead of 375 on 8192 queries of 64 heads
//     with a window of 1024, and 202 instead of 186 on 2 x 1000 with 2000.)
//   * an item's KV pages are its sink pages and those from its first query's
//     window on, numbered through and taken two to a tile (so a tile may join
//     the last sink page and the first window page); no other page is looked up
//     or loaded, and the second Q tile skips a tile that only the first one sees;
//   * a tile's masked scores are overwritten in TMEM before the softmax reads
//     them, and the output goes out by TMA through shared memory: both kept the
//     softmax warps from their next tile, a masked tile for as long again as its
//     softmax, the output rows for 4700 cycles an item;
//   * a tile with a dead row (past L_r, or before the window and no sink) has
//     those rows of V zeroed by the producer once they have landed, and is
//     handed over on its own barrier (0 * NaN would reach O).
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

constexpr int kOffQ = 0;
constexpr int kOffK = kOffQ + kQT * kTileBytes;
constexpr int kOffV = kOffK + kKStages * kTileBytes;
constexpr int kOffO = kOffV + kVStages * kTileBytes;  // [x]: half of an output tile, BF16
constexpr int kOffBar = kOffO + kQT * kHalf;
// barriers: q_full, q_free, k_full[2], k_empty[2], v_full[2], v_empty[2],
// v_clean[2], s_full[2], p_full[2], o_done[2], o_free[2], mma_done, end
constexpr int kNumBars = 2 + 2 * kKStages + 3 * kVStages + 4 * kQT + 2;
constexpr int kOffMisc = kOffBar + kNumBars * 8;  // tmem slot, abort word
constexpr int kSmemBytes = kOffMisc + 16 + 1024;  // + alignment slack
static_assert(kSmemBytes <= 227 * 1024, "shared memory over the per-CTA limit");

struct WinArgs {
    const int32_t *seqlens;
    const int32_t *block_table;
    __nv_bfloat16 *out;
    int32_t *flags;
    int B, Hq, G, q_len, max_pages, num_pages, n_qp;
    int pairs, items;  // items: `pairs` pairs of Q tiles, then single Q tiles
    int window, sinks;
    float score_scale;  // sm_scale * log2(e)
};

// One item: a request, a query head and a pair of Q tiles (or one of them, the
// first of the two then), with the KV pages it reads.
struct Item {
    bool single;
    int r, hq, i0, L;
    int tiles[kQT];      // causal extent of each Q tile, in the item's tiles
    int n;               // KV tiles of the item: two of its pages each
    int lo;              // first token of the window of the pair's first query
    int sink_pages, skip;  // pages that hold sinks; pages left out behind them
    int alone;           // tile that only the first Q tile sees, or -1

    // the item's page c among the request's, and tile j's token of column c
    __device__ __forceinline__ int page(int c) const { return c < sink_pages ? c : c + skip; }
    __device__ __forceinline__ int token(int j, int c) const {
        return page(2 * j + (c >> 6)) * kTile + (c & 63);
    }
    __device__ __forceinline__ bool active(int x, int j) const {
        return j < tiles[x] && (x == 0 || j != alone);
    }
    // no query of the pair sees token t: past the end, or before the window
    // and no sink
    __device__ __forceinline__ bool dead(int t, int sinks) const {
        return t >= L || (t < lo && t >= sinks);
    }
    // page g holds such a token, or one that is not
    __device__ __forceinline__ bool dirty_page(int g, int sinks) const {
        const int t = g * kTile;
        return t + kTile > L || max(t, sinks) < min(t + kTile, lo);
    }
    __device__ __forceinline__ bool needs_page(int g, int sinks) const {
        const int t = g * kTile;
        return t < L && (t + kTile > lo || t < sinks);
    }
    __device__ __forceinline__ bool dirty(int j, int sinks) const {
        return dirty_page(page(2 * j), sinks) || dirty_page(page(2 * j + 1), sinks);
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
    const int per_qp = a.B * a.Hq;
    const int qp = a.n_qp - 1 - idx / per_qp, rem = idx % per_qp;
    it.r = rem / a.Hq;
    it.hq = rem % a.Hq;
    it.i0 = qp * kQT * kQB + (it.single ? ((item - a.pairs) & 1) * kQB : 0);
    it.L = L;
    it.lo = max(L - a.q_len + it.i0 + 1 - a.window, 0);
    it.sink_pages = a.sinks / kTile + (a.sinks % kTile ? 1 : 0);
    it.skip = max(it.lo / kTile - it.sink_pages, 0);
    it.n = 0;
#pragma unroll
    for (int x = 0; x < kQT; ++x) {
        const int first = it.i0 + x * kQB;
        // last token that the tile's rows see
        const int lim_last = min(L - a.q_len + min(first + kQB - 1, a.q_len - 1), L - 1);
        it.tiles[x] = 0;
        // (the extent ends behind the first row's window: it has pages behind
        // the gap, or the gap is empty)
        if (first < a.q_len && lim_last >= 0 && (x == 0 || !it.single))
            it.tiles[x] = (lim_last / kTile + 1 - it.skip + 1) / 2;
        it.n = max(it.n, it.tiles[x]);
    }
    // the second Q tile's windows begin two pages later
    it.alone = it.lo > 0 && it.lo / kTile >= it.sink_pages && it.sink_pages % 2 == 0
                   ? it.sink_pages / 2
                   : -1;
    return it;
}

// Sets the scores of a tile (128 TMEM columns from `col`, the pages of tokens
// tok0 .. and tok1 ..) that the row does not see to -inf: query i of a request
// of L tokens sees tokens <= lim that are >= lo or < sinks.  Done in TMEM, 32
// columns at a time, before the softmax reads them: the warp's rows i0 .. i0 +
// 31 are consecutive, so whole groups are seen or hidden by all of them and only
// the groups that a border crosses are read and compared.  Out of line: it is
// rare, and the softmax needs its registers.
__device__ __noinline__ void mask_tile(uint32_t col, int tok0, int tok1, int i0, int L, int q_len,
                                       int window, int sinks) {
    const int p0 = L - q_len + i0, i = i0 + (int)(threadIdx.x & 31);
    const int lim0 = min(p0, L - 1), lim31 = min(p0 + 31, L - 1);
    const int lo0 = p0 + 1 - window, lo31 = lo0 + 31;
    const int lim = min(L - q_len + i, L - 1), lo = L - q_len + i + 1 - window;
#pragma unroll 1
    for (int w = 0; w < 4; ++w) {
        const int t = (w < 2 ? tok0 : tok1) + 32 * (w & 1);
        if (t + 31 <= lim0 && (t >= lo31 || t + 31 < sinks)) continue;  // all see all of it
        uint32_t r[32];
        if (t > lim31 || (t + 31 < lo0 && t >= sinks)) {  // none sees any
#pragma unroll
            for (int c = 0; c < 32; ++c) r[c] = 0xff800000u;
        } else {
            tmem_ld32_nowait(col + 32 * w, r);
            tmem_wait_ld32(r);
            if (t >= sinks) {  // one interval [lo, lim]
                const unsigned span = (unsigned)(lim - lo);
                const int from = lo - t;
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    if ((unsigned)(c - from) > span) r[c] = 0xff800000u;
            } else {
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    if (c > lim - t || (c < lo - t && c >= sinks - t)) r[c] = 0xff800000u;
            }
        }
        tmem_st32_nowait(col + 32 * w, r);
        tmem_wait_st32(r);
    }
}

__device__ __forceinline__ int clamped_len(const WinArgs &a, int item) {
    const int L = __ldg(a.seqlens + pair_of(a, item) % (a.B * a.Hq) / a.Hq);
    return min(max(L, 0), a.max_pages * kTile);
}

__global__ void __launch_bounds__(kThreads, 1)
    prefill_win_kernel(const __grid_constant__ CUtensorMap tq,
                       const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv,
                       const __grid_constant__ CUtensorMap to, const WinArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kOffBar);
    uint64_t *q_full = bars, *q_free = bars + 1;
    uint64_t *k_full = bars + 2, *k_empty = k_full + kKStages;
    uint64_t *v_full = k_empty + kKStages, *v_empty = v_full + kVStages;
    uint64_t *v_clean = v_empty + kVStages;  // [stage]: a V tile with its dead rows zeroed
    uint64_t *s_full = v_clean + kVStages;   // [x]: S_x complete (and every MMA before it)
    uint64_t *p_full = s_full + kQT;         // [x]: P_x written (four warps)
    uint64_t *o_done = p_full + kQT;         // [x]: O_x += P_x V complete
    uint64_t *o_free = o_done + kQT;         // [x]: O_x read out (four warps)
    uint64_t *mma_done = o_free + kQT, *end = mma_done + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + kOffMisc);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + kOffMisc + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        // one arrival (an expect-tx arrival or a tcgen05.commit) per phase,
        // except where a Q tile's four warps arrive, and all eight at the end
        for (int b = 0; b < kNumBars; ++b) {
            const bool per_warp = (&bars[b] >= p_full && &bars[b] < o_done) ||
                                  (&bars[b] >= o_free && &bars[b] < mma_done);
            mbar_init(&bars[b], per_warp ? 4 : &bars[b] == end ? kSoftmaxWarps : 1);
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
    const uint32_t tmem = *tmem_slot;
    grid_dependency_wait();  // Q, the caches and the lengths may come from the previous kernel

    const int step = gridDim.x;
    bool ok = true;
    int next_L = clamped_len(a, blockIdx.x);  // (the grid is at most the items)

    if (warp == kProducerWarp) {
        const uint64_t pol = policy_evict_normal();
        uint32_t kt = 0;           // tiles issued
        uint32_t q_items = 0;      // items whose Q has been issued
        bool pending = false;      // tile kt - 1 has dead rows to zero
        Item was;                  // ... of this item
        int was_j = 0;
        auto clean = [&]() {
            const int s = (int)((kt - 1) % kVStages);
            if (!warp_wait(&v_full[s], ((kt - 1) / kVStages) & 1u, abort)) return false;
            uint8_t *vs = smem + kOffV + s * kTileBytes;
            for (int e = lane; e < kKB * 8; e += 32)
                if (was.dead(was.token(was_j, e >> 3), a.sinks))
                    for (int h = 0; h < 2; ++h)
                        sts128(smem_u32(vs + h * kHalf + e * 16), 0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&v_clean[s]);
            return true;
        };
        for (int idx = blockIdx.x; ok && idx < a.items; idx += step) {
            const Item it = item_of(a, idx, next_L);
            if (lane == 0 && a.flags && it.hq == 0 && it.i0 == 0) {
                const int raw = __ldg(a.seqlens + it.r);
                if (raw < 0 || raw > a.max_pages * kTile)
                    atomicOr(a.flags, (int)HPC_FLAG_BAD_SEQLEN);
            }
            if (idx + step < a.items) next_L = clamped_len(a, idx + step);
            if (it.n == 0) continue;
            if (q_items > 0 && !warp_wait(q_free, (q_items - 1) & 1u, abort)) {
                ok = false;
                break;
            }
            if (lane == 0) {
                uint32_t bytes = 0;
#pragma unroll
                for (int x = 0; x < kQT; ++x) bytes += it.tiles[x] > 0 ? kTileBytes : 0;
                mbar_arrive_expect_tx(q_full, bytes);
#pragma unroll
                for (int x = 0; x < kQT; ++x)
                    if (it.tiles[x] > 0)
                        for (int h = 0; h < 2; ++h)
                            tma_load_4d(smem + kOffQ + x * kTileBytes + h * kHalf, &tq, q_full, 0,
                                        h, it.hq, it.r * a.q_len + it.i0 + x * kQB, pol);
            }
            ++q_items;
            const int32_t *bt = a.block_table + (size_t)it.r * a.max_pages;
            const int hkv = it.hq / a.G;
            int pg = -1;
            for (int j = 0; j < it.n; ++j) {
                if ((j & 15) == 0) {  // the pages of 16 tiles, one per lane; -2: not needed
                    const int g = it.page(2 * j + lane);
                    pg = it.needs_page(g, a.sinks) ? max(__ldg(bt + g), -1) : -2;
                }
                const int p0 = __shfl_sync(0xffffffffu, pg, (2 * j) & 31);
                const int p1 = __shfl_sync(0xffffffffu, pg, (2 * j + 1) & 31);
                const bool l0 = p0 >= 0 && p0 < a.num_pages, l1 = p1 >= 0 && p1 < a.num_pages;
                if (((p0 != -2 && !l0) || (p1 != -2 && !l1)) && lane == 0 && a.flags)
                    atomicOr(a.flags, (int)HPC_FLAG_BAD_PAGE);
                const uint32_t bytes = (uint32_t)((l0 ? 1 : 0) + (l1 ? 1 : 0)) * 2 * kTile * 128;
#pragma unroll
                for (int kv = 0; kv < 2 && ok; ++kv) {
                    // V of the tile before has landed by now, or nearly: its dead
                    // rows go before this tile's V has room
                    if (kv == 1 && pending) {
                        pending = false;
                        ok = clean();
                        if (!ok) break;
                    }
                    const int st = kv == 0 ? kKStages : kVStages, s = (int)(kt % st);
                    uint64_t *full = kv == 0 ? &k_full[s] : &v_full[s];
                    ok = warp_wait(kv == 0 ? &k_empty[s] : &v_empty[s], ((kt / st) & 1u) ^ 1u,
                                   abort);
                    if (ok && lane == 0) {
                        if (bytes == 0) {
                            mbar_arrive(full);
                        } else {
                            mbar_arrive_expect_tx(full, bytes);
                            const CUtensorMap *map = kv == 0 ? &tk : &tv;
                            uint8_t *dst = smem + (kv == 0 ? kOffK : kOffV) + s * kTileBytes;
                            for (int h = 0; h < 2; ++h) {
                                if (l0)
                                    tma_load_5d(dst + h * kHalf, map, full, 0, h, hkv, 0, p0, pol);
                                if (l1)
                                    tma_load_5d(dst + h * kHalf + kTile * 128, map, full, 0, h,
                                                hkv, 0, p1, pol);
                            }
                        }
                    }
                }
                if (!ok) break;
                ++kt;
                pending = it.dirty(j, a.sinks);
                was = it;
                was_j = j;
            }
        }
        if (ok && pending && !clean()) ok = false;
        // no copy may land after the CTA has left: the last one issued into
        // each buffer (bounded)
        __syncwarp();
        if (!ok || *abort) {
            volatile int no_abort = 0;
            if (q_items > 0) mbar_wait(q_full, (q_items - 1) & 1u, &no_abort);
            for (uint32_t t = kt > 2 ? kt - 2 : 0; t < kt; ++t) {
                mbar_wait(&k_full[t % kKStages], (t / kKStages) & 1u, &no_abort);
                mbar_wait(&v_full[t % kVStages], (t / kVStages) & 1u, &no_abort);
            }
            __syncwarp();
        }
    } else if (warp == kMmaWarp) {
        const uint32_t idesc_s = idesc_bf16_f32(kQB, kKB);
        const uint32_t idesc_o = idesc_bf16_f32_bmn(kQB, kHeadDim);
        const uint64_t dq0 = smem_desc_k128(smem_u32(smem + kOffQ));
        const uint64_t dk0 = smem_desc_k128(smem_u32(smem + kOffK));
        const uint64_t dv0 = smem_desc_mn128(smem_u32(smem + kOffV), kHalf);
        // S_x = Q_x K^T into x's score columns (K tile in stage s)
        auto issue_s = [&](int x, uint32_t s) {
            const uint64_t dq = dq0 + (uint64_t)((x * kTileBytes) >> 4);
            const uint64_t dk = dk0 + (uint64_t)((s * kTileBytes) >> 4);
#pragma unroll
            for (int k = 0; k < kHeadDim / 16; ++k) {
                const uint32_t off = ((k >> 2) * kHalf + (k & 3) * 32) >> 4;
                umma_bf16(tmem + 128 * x, dq + off, dk + off, idesc_s, k > 0);
            }
            umma_commit(&s_full[x]);
        };
        // O_x += P_x V (V tile in stage s), P_x from TMEM
        auto issue_pv = [&](int x, uint32_t s, bool acc) {
            const uint64_t dv = dv0 + (uint64_t)((s * kTileBytes) >> 4);
#pragma unroll
            for (int k = 0; k < kKB / 16; ++k)
                umma_bf16_ts(tmem + kOCol + 128 * x, tmem + 128 * x + 8 * k,
                             dv + (uint64_t)((k * 16 * 128) >> 4), idesc_o, acc || k > 0);
            umma_commit(&o_done[x]);
        };
        uint32_t kt = 0, q_items = 0;
        uint32_t cleaned[kVStages] = {};  // zeroed tiles taken from each stage
        uint32_t np[kQT] = {};            // P tiles taken
        uint32_t outs[kQT] = {};          // items whose O_x has been claimed
        for (int idx = blockIdx.x; ok && idx < a.items; idx += step) {
            const Item it = item_of(a, idx, next_L);
            if (idx + step < a.items) next_L = clamped_len(a, idx + step);
            if (it.n == 0) continue;
            bool started[kQT] = {};
            ok = warp_wait(q_full, q_items & 1u, abort) &&
                 warp_wait(&k_full[kt % kKStages], (kt / kKStages) & 1u, abort);
            ++q_items;
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                for (int x = 0; x < kQT; ++x)
                    if (it.active(x, 0)) issue_s(x, kt % kKStages);
                umma_commit(&k_empty[kt % kKStages]);
                if (it.n == 1) umma_commit(q_free);
            }
            __syncwarp();
            for (int j = 0; ok && j < it.n; ++j, ++kt) {
                const uint32_t s = kt % kVStages, s1 = (kt + 1) % kKStages;
                const bool next = j + 1 < it.n;
                if (it.dirty(j, a.sinks)) {
                    ok = warp_wait(&v_clean[s], cleaned[s] & 1u, abort);
                    ++cleaned[s];
                } else {
                    ok = warp_wait(&v_full[s], (kt / kVStages) & 1u, abort);
                }
                if (ok && next)
                    ok = warp_wait(&k_full[s1], ((kt + 1) / kKStages) & 1u, abort);
#pragma unroll
                for (int x = 0; x < kQT; ++x) {
                    if (!ok) break;
                    const bool now = it.active(x, j), then = next && it.active(x, j + 1);
                    if (now) {
                        ok = warp_wait(&p_full[x], np[x] & 1u, abort);
                        ++np[x];
                        if (ok && !started[x]) {  // the item before has been read out of O_x
                            if (outs[x] > 0) ok = warp_wait(&o_free[x], (outs[x] - 1) & 1u, abort);
                            ++outs[x];
                        }
                        if (!ok) break;
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        if (now) issue_pv(x, s, started[x]);
                        if (then) issue_s(x, s1);
                    }
                    __syncwarp();
                    started[x] |= now;
                }
                if (!ok) break;
                if (elect_one()) {
                    umma_commit(&v_empty[s]);  // after both Q tiles' products with V_j
                    if (next) umma_commit(&k_empty[s1]);  // after both Q tiles' scores with K_j+1
                    if (j + 2 == it.n) umma_commit(q_free);  // the item's last scores
                }
                __syncwarp();
            }
        }
        // arrives once every MMA issued has completed (TMEM is freed after it)
        if (elect_one()) umma_commit(mma_done);
        __syncwarp();
    } else {
        // softmax of Q tile x: thread = one query row, warp w reads TMEM
        // lanes 32 (w mod 4) ..
        const int x = warp >> 2, q4 = warp & 3;
        const int rho = 32 * q4 + lane;
        const uint32_t row = tmem + ((uint32_t)(32 * q4) << 16);
        const uint32_t scol = row + 128 * x, ocol = row + kOCol + 128 * x;
        const float sc = a.score_scale;
        uint32_t ns = 0;  // score tiles taken
        for (int idx = blockIdx.x; ok && idx < a.items; idx += step) {
            const Item it = item_of(a, idx, next_L);
            if (idx + step < a.items) next_L = clamped_len(a, idx + step);
            if (x > 0 && it.single) continue;
            const int tiles = it.tiles[x], L = it.L, first = it.i0 + x * kQB;
            // the last token its first row sees, the first of its last row's window
            const int lim_first = min(L - a.q_len + first, L - 1);
            const int lo_last = L - a.q_len + min(first + kQB, a.q_len) - a.window;
            float m_ref = -INFINITY, l = 0.f;
            bool started = false;
            for (int j = 0; j < tiles; ++j) {
                if (!it.active(x, j)) continue;
                if (!warp_wait(&s_full[x], ns & 1u, abort)) {
                    ok = false;
                    break;
                }
                ++ns;
                tc_fence_after();
                const int tok0 = it.token(j, 0), tok1 = it.token(j, kTile);
                // some row does not see all of it: the diagonal or the end, or
                // tokens before a window that are no sinks
                if (tok1 + kTile - 1 > lim_first || (tok0 < lo_last && tok0 + kTile > a.sinks) ||
                    (tok1 < lo_last && tok1 + kTile > a.sinks))
                    mask_tile(scol, tok0, tok1, first + 32 * q4, L, a.q_len, a.window, a.sinks);
                // the row's 128 scores in two halves: the second half loads while
                // the first is reduced
                uint32_t ra[32], rb[32], rc[32], rd[32];
                tmem_ld32_nowait(scol, ra);
                tmem_ld32_nowait(scol + 32, rb);
                tmem_wait_ld32x2(ra, rb);
                tmem_ld32_nowait(scol + 64, rc);
                tmem_ld32_nowait(scol + 96, rd);
                float s[128];
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    s[c] = __uint_as_float(ra[c]);
                    s[32 + c] = __uint_as_float(rb[c]);
                }
                float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 32; ++c) mx4[c & 3] = fmax3(mx4[c & 3], s[2 * c], s[2 * c + 1]);
                tmem_wait_ld32x2(rc, rd);
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    s[64 + c] = __uint_as_float(rc[c]);
                    s[96 + c] = __uint_as_float(rd[c]);
                }
#pragma unroll
                for (int c = 32; c < 64; ++c)
                    mx4[c & 3] = fmax3(mx4[c & 3], s[2 * c], s[2 * c + 1]);
                const float mx = fmax3(fmaxf(mx4[0], mx4[1]), mx4[2], mx4[3]);
                const float m_tile = mx * sc;
                const bool need = m_tile > m_ref + kRescaleLog2;
                const float new_ref = need ? m_tile : m_ref;
                const float factor = need ? ex2(m_ref - new_ref) : 1.f;
                const float base = new_ref == -INFINITY ? 0.f : new_ref;
                // P as packed BF16 pairs, written over the first 64 score columns
                // in two stores: the first is in flight while the second half is
                // computed
                uint32_t pa[32], pb[32];
                float2 ps[4] = {};
                const float2 sc2 = make_float2(sc, sc), nb2 = make_float2(-base, -base);
#pragma unroll
                for (int c = 0; c < 32; ++c) {  // two columns per instruction
                    const float2 e = __ffma2_rn(make_float2(s[2 * c], s[2 * c + 1]), sc2, nb2);
                    const float p0 = ex2(e.x), p1 = ex2(e.y);
                    ps[c & 3] = __fadd2_rn(ps[c & 3], make_float2(p0, p1));
                    pa[c] = pack_bf16x2(p0, p1);
                }
                tmem_st32_nowait(scol, pa);
#pragma unroll
                for (int c = 32; c < 64; ++c) {
                    const float2 e = __ffma2_rn(make_float2(s[2 * c], s[2 * c + 1]), sc2, nb2);
                    const float p0 = ex2(e.x), p1 = ex2(e.y);
                    ps[c & 3] = __fadd2_rn(ps[c & 3], make_float2(p0, p1));
                    pb[c - 32] = pack_bf16x2(p0, p1);
                }
                const float2 pq = __fadd2_rn(__fadd2_rn(ps[0], ps[1]), __fadd2_rn(ps[2], ps[3]));
                l = l * factor + (pq.x + pq.y);
                // O_x is settled: its product with the previous tile completed
                // before these scores did
                if (started && __any_sync(0xffffffffu, need)) {
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
                tmem_st32_nowait(scol + 32, pb);
                tmem_wait_st32x2(pa, pb);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[x]);
                m_ref = new_ref;
            }
            // epilogue: O / l as BF16 (zeros for rows that see nothing)
            bool have = ok && started;
            if (have) {
                if (!warp_wait(&o_done[x], (ns - 1) & 1u, abort))
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
                    tma_store_5d(&to, smem + kOffO + x * kHalf + 32 * q4 * 128, 0, hf, it.hq,
                                 first + 32 * q4, it.r);
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
    // round, nor be flushed to zero
    if (!std::isfinite(sm_scale) || !(sm_scale >= FLT_MIN)) return HPC_ERR_ARG;
    if (B == 0) return HPC_OK;
    if (!d_q || !d_k_cache || !d_v_cache || !d_block_table || !d_seqlens || !d_out)
        return HPC_ERR_ARG;
    if (!aligned16(d_q) || !aligned16(d_k_cache) || !aligned16(d_v_cache) || !aligned16(d_out))
        return HPC_ERR_ARG;
    const int64_t n_qp = ((int64_t)q_len + kQT * kQB - 1) / (kQT * kQB);
    const int64_t pairs = n_qp * B * Hq;
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
    a.out = static_cast<__nv_bfloat16 *>(d_out);
    a.flags = d_flags;
    a.B = B;
    a.Hq = Hq;
    a.G = Hq / Hkv;
    a.q_len = q_len;
    a.max_pages = max_pages_per_req;
    a.num_pages = num_pages;
    a.n_qp = (int)n_qp;
    a.window = window;
    a.sinks = sinks;
    a.score_scale = sm_scale * 1.4426950408889634f;

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
    cfg.blockDim = dim3(kThreads);
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
