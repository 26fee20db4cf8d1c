// Decode attention over shared prefixes on the fifth-generation tensor cores: one
// grid, whose first CTAs compute the heads (queries of a whole group against the pages
// that its requests share), the others the tails (each request's own pages, as decode
// ever does: attn_kernel.cuh over BF16 pages, attn_tc.cuh over 8-bit ones).
//
// The head reads a page once for up to 256 query rows and is bound by the tensor pipe
// and the softmax; the tail by HBM.  So the plan gives each CTAs of its own, and both
// run at the same time.
//
// A head's CTA has two halves, each with its softmax warps, its issuing warp and its
// accumulator: S = Q_x K^T of a page into TMEM, one softmax thread per row (online in
// fp32, with a reference that moves when a score passes it by 2^8; P in 16 bits over the
// scores), O_x += P V with P read from TMEM; two score buffers for each half, and its
// scores two of its pages ahead of the products.  Every row sees every token of every
// page here, so there are no masks.  The halves take a row tile of 128 queries each, and
// every page; where a row tile is alone (the last of an odd number) they take every
// other page of it, and leave a partial each.
//
// 8-bit pages: scores on E4M3 MMAs from the codes as they land; V is widened by warps
// of its own into a second ring, to f16, in which all E4M3 values are exact.  Weights are
// f16 (rounded to 2^-11), times 2^6 so that the smallest keep their bits: at most 2^14.
// Block scales of V multiply the weights, and the reference follows score + log2(scale),
// as the decode kernel's does (attn_tc.cuh), so that this bound holds whatever the scales
// and a sum of products stays below 2^23 a token.  (Weights in BF16, whose range holds the
// scales, with a reference that follows the scores alone: sums over 2400 tokens of scale
// 2^100 pass 2^128, and the error of a step is 0.0018 to 0.0021 of its norm, not 0.0017.)
//
// Every wait is bounded; on a timeout the CTA raises the flag, waits (bounded) for its
// copies and MMAs in flight, frees TMEM and leaves.
#pragma once

#include <cuda_bf16.h>

#include "attn_tc.cuh"
#include "shared.h"
#include "tcgen05.cuh"

namespace hpc {

constexpr int kHeadSoftmax = 8;  // warps: four for each row tile
constexpr int kHeadProducer = kHeadSoftmax, kHeadMma = kHeadProducer + 1, kHeadWiden = kHeadMma + 2;
constexpr uint32_t kHeadTmem = 512;  // S_x / P_x from 128 x on; O_x at 256 + 128 x
constexpr int kHeadOCol = 256;
constexpr int kScaleRing = 16;  // pages whose block scales are held
constexpr float kHeadLazy = 8.f;

template <hpc_kv_dtype KV>
struct HeadTraits {
    static constexpr bool k8 = KV != HPC_KV_BF16, kBlk = KV == HPC_KV_E4M3_BLOCK;
    static constexpr int kWarps = k8 ? 16 : 12;
    static constexpr int kWideners = k8 ? kWarps - kHeadWiden : 0;
    static constexpr int kRow = k8 ? 128 : 256;            // bytes of a row
    static constexpr int kQBytes = kHeadRows * kRow;       // of a row tile
    static constexpr int kPageBytes = kTile * kRow;        // of K or V
    static constexpr int kWideBytes = kTile * 256;
    // Pages in the first ring (K; 8-bit: and V's codes) and in the second (V as the
    // products take it).  Even numbers: a page's place says which half takes it where
    // they alternate.
    static constexpr int S = k8 ? 6 : 4;
    static constexpr int W = k8 ? 4 : 6;
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + 2 * kQBytes;
    static constexpr int kOffCodes = kOffK + S * kPageBytes;
    static constexpr int kOffV = kOffCodes + (k8 ? S * kPageBytes : 0);
    static constexpr int kOffScale = kOffV + W * kWideBytes;
    static constexpr int kOffBar = kOffScale + (kBlk ? kScaleRing * kPageScales * 4 : 0);
    // q_full, q_free, full[S], empty[S], v_full[W], v_free[W], s_full[2][2],
    // p_full[2][2], o_done[2][2], o_free[2], mma_done, end
    static constexpr int kNumBars = 2 + 2 * S + 2 * W + 12 + 2 + 2;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;  // TMEM address, abort word
    static constexpr int kSmemBytes = kOffMisc + 16 + 1024;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
    // a half's scores are at most two of its pages ahead of its softmax, so where the
    // halves alternate a page's scales have been read when S + 5 later ones are on their way
    static_assert(kScaleRing >= S + 6 && S % 2 == 0 && W % 2 == 0, "rings");
};

struct HeadItem {
    int h, tok, end, req;  // KV head, first query token, end of the group's, table row
    int lo, hi;            // pages
    bool two;              // two row tiles
    int slot;
};

__device__ __forceinline__ HeadItem head_item(const HeadPlan &p, int d) {
    const int4 x = __ldg(p.desc + 2 * d), y = __ldg(p.desc + 2 * d + 1);
    return {x.x, x.y, x.z, x.w, y.x, y.y, y.z != 0, 2 * d};
}

// The pages of an item that half x takes, in the CTA's count of pages (`kt` before the
// item): all, or every other one, by the place they have in the rings.
struct HeadPages {
    uint32_t at, step;
    int n;
};

__device__ __forceinline__ HeadPages head_pages(const HeadItem &it, uint32_t kt, int x) {
    const int n = it.hi - it.lo;
    if (it.two) return {kt, 1, n};
    const int skip = (int)(kt ^ (uint32_t)x) & 1;
    return {kt + skip, 2, (n - skip + 1) >> 1};
}

__device__ __forceinline__ float head_max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// acc += a BF16 value, without widening it first.
__device__ __forceinline__ void head_add_bf16(float &acc, uint16_t x) {
    asm("add.f32.bf16 %0, %1, %0;" : "+f"(acc) : "h"(x));
}

__device__ __forceinline__ void store_f32x8(float *p, const float *v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p),
                 "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])),
                 "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
                 "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
                 "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
                 : "memory");
}

// 3-D tiled TMA load.
__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, uint64_t *bar,
                                            int c0, int c1, int c2, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

// The head work of this CTA: descriptors first .. last - 1.
template <hpc_kv_dtype KV>
__device__ __forceinline__ void head_cta(const SharedMaps &m, const HeadArgs &a, int first,
                                         int last) {
    using Tr = HeadTraits<KV>;
    constexpr int S = Tr::S, W = Tr::W;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Tr::kOffBar);
    uint64_t *q_full = bars, *q_free = bars + 1;
    uint64_t *full = bars + 2;         // [stage]: K of a page has landed (8-bit: and V's codes)
    uint64_t *empty = full + S;        // [stage]: its scores are done (and V is widened)
    uint64_t *v_full = empty + S;      // [slot]: V is there
    uint64_t *v_free = v_full + W;     // [slot]: its products are done
    uint64_t *s_full = v_free + W;     // [x][b]: the scores of an even or odd page of x
    uint64_t *p_full = s_full + 4;        // [x][b]: its P written (four warps)
    uint64_t *o_done = p_full + 4;        // [x][b]: O_x += P V of that page complete
    uint64_t *o_free = o_done + 4;        // [x]: O_x read out (four warps)
    uint64_t *mma_done = o_free + 2, *end = mma_done + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Tr::kOffMisc);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + Tr::kOffMisc + 4);
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int b = 0; b < Tr::kNumBars; ++b) {
            uint64_t *bar = &bars[b];
            int n = 1;
            // Both halves' last scores, and all of V widened.  So when the next item's Q
            // lands, all pages of this one have, and V of each is or has been in place: a
            // half that left a page to the other meets no phase of its barriers early.
            if (bar == q_free) n = 2 + Tr::kWideners;
            if (bar >= empty && bar < empty + S) n = 2 + Tr::kWideners;
            if (bar >= v_full && bar < v_full + W) n = Tr::k8 ? Tr::kWideners : 1;
            if (bar >= v_free && bar < v_free + W) n = 2;
            // (block scales: beside the scores' commit, the word of a thread that has seen
            // the page land)
            if (Tr::kBlk && bar >= s_full && bar < p_full) n = 2;
            if ((bar >= p_full && bar < o_done) || (bar >= o_free && bar < mma_done)) n = 4;
            if (bar == mma_done) n = 2;
            if (bar == end) n = kHeadSoftmax;
            mbar_init(bar, n);
        }
        *abort = 0;
        fence_barrier_init();
        prefetch_tensormap(&m.q);
        prefetch_tensormap(&m.k);
        prefetch_tensormap(&m.v);
    }
    if (warp == kHeadMma) {
        tmem_alloc(tmem_slot, kHeadTmem);
        tmem_relinquish();
    }
    grid_launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
    const int tpb = head_tokens(a.G);
    bool ok = true;

    if (warp == kHeadProducer) {
        uint64_t keep;  // the pages are read by the other row tiles' CTAs too
        asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(keep));
        const uint32_t q_tile = (uint32_t)(tpb * a.G * Tr::kRow);
        uint32_t kt = 0, items = 0, v_pages = 0;
        for (int d = first; ok && d < last; ++d) {
            const HeadItem it = head_item(a.plan, d);
            if (items > 0 && !mbar_wait_warp(q_free, (items - 1) & 1u, abort)) {
                ok = false;
                break;
            }
            if (lane == 0) {
                mbar_arrive_expect_tx(q_full, it.two ? 2 * q_tile : q_tile);
                for (int x = 0; x < (it.two ? 2 : 1); ++x) {
                    uint8_t *q = smem + Tr::kOffQ + x * Tr::kQBytes;
                    const int tok = it.tok + x * tpb;
                    if (Tr::k8) {
                        tma_load_3d(q, &m.q, q_full, 0, it.h * a.G, tok, keep);
                    } else {
                        for (int hf = 0; hf < 2; ++hf)
                            tma_load_4d(q + hf * (kHeadRows * 128), &m.q, q_full, 0, hf,
                                        it.h * a.G, tok, keep);
                    }
                }
            }
            ++items;
            const int32_t *bt = a.block_table + (size_t)it.req * a.max_pages;
            int pg = 0;
            for (int j = it.lo; j < it.hi; ++j, ++kt) {
                const int e = (j - it.lo) & 31;
                if (e == 0) {  // the entries of 32 pages, one per lane
                    pg = j + lane < it.hi ? __ldg(bt + j + lane) : 0;
                    if (pg < 0 || pg >= a.num_pages) {
                        atomicOr(a.meta + 3, (int)HPC_FLAG_BAD_PAGE);
                        pg = 0;
                    }
                }
                const int page = __shfl_sync(kFullMask, pg, e);
                const int s = (int)(kt % S), v = (int)(kt % W);
                // V before K: who sees K land knows that V's place was free
                if (!Tr::k8) {
                    ok = mbar_wait_warp(&v_free[v], ((kt / W) & 1u) ^ 1u, abort);
                    if (!ok) break;
                    if (lane == 0) {
                        if (!it.two) mbar_arrive(&v_free[v]);  // for the half that leaves it
                        mbar_arrive_expect_tx(&v_full[v], Tr::kPageBytes);
                        for (int hf = 0; hf < 2; ++hf)
                            tma_load_5d(smem + Tr::kOffV + v * Tr::kPageBytes + hf * (kTile * 128),
                                        &m.v, &v_full[v], 0, hf, it.h, 0, page, keep);
                    }
                    ++v_pages;
                }
                ok = mbar_wait_warp(&empty[s], ((kt / S) & 1u) ^ 1u, abort);
                if (!ok) break;
                if (lane == 0) {
                    if (!it.two) mbar_arrive(&empty[s]);
                    uint8_t *k = smem + Tr::kOffK + s * Tr::kPageBytes;
                    if (Tr::k8) {
                        mbar_arrive_expect_tx(
                            &full[s], 2 * Tr::kPageBytes + (Tr::kBlk ? kPageScales * 4 : 0));
                        tma_load_4d(k, &m.k, &full[s], 0, it.h, 0, page, keep);
                        tma_load_4d(smem + Tr::kOffCodes + s * Tr::kPageBytes, &m.v, &full[s], 0,
                                    it.h, 0, page, keep);
                        if (Tr::kBlk)
                            bulk_load(smem + Tr::kOffScale + (kt % kScaleRing) * kPageScales * 4,
                                      a.kv_scale + ((size_t)page * a.Hkv + it.h) * kPageScales,
                                      kPageScales * 4, &full[s]);
                    } else {
                        mbar_arrive_expect_tx(&full[s], Tr::kPageBytes);
                        for (int hf = 0; hf < 2; ++hf)
                            tma_load_5d(k + hf * (kTile * 128), &m.k, &full[s], 0, hf, it.h, 0,
                                        page, keep);
                    }
                }
            }
        }
        // no copy may land after the CTA has left: the last one issued into each
        // buffer (bounded)
        __syncwarp();
        if (!ok || *abort) {
            volatile int no_abort = 0;
            if (items > 0) mbar_wait(q_full, (items - 1) & 1u, &no_abort);
            for (uint32_t t = kt > S ? kt - S : 0; t < kt; ++t)
                mbar_wait(&full[t % S], (t / S) & 1u, &no_abort);
            for (uint32_t t = v_pages > W ? v_pages - W : 0; t < v_pages; ++t)
                mbar_wait(&v_full[t % W], (t / W) & 1u, &no_abort);
            __syncwarp();
        }
    } else if (warp == kHeadMma || warp == kHeadMma + 1) {
        const int x = warp - kHeadMma;  // the half
        constexpr uint32_t id_s = Tr::k8 ? idesc_e4m3_f32(kHeadRows, kTile, false, false)
                                         : idesc_bf16_f32(kHeadRows, kTile);
        // (8-bit pages: f16 weights and values, the type bits of both zero)
        constexpr uint32_t id_o = idesc_bf16_f32_bmn(kHeadRows, kHeadDim) &
                                  (Tr::k8 ? ~((1u << 7) | (1u << 10)) : ~0u);
        const uint64_t dq0 = smem_desc_k128(smem_u32(smem + Tr::kOffQ));
        const uint64_t dk0 = smem_desc_k128(smem_u32(smem + Tr::kOffK));
        const uint64_t dv0 = smem_desc_mn128(smem_u32(smem + Tr::kOffV), kTile * 128);
        auto issue_s = [&](uint32_t b, uint64_t dq, uint32_t page) {
            const uint32_t s = page % S;
            const uint64_t dk = dk0 + (uint64_t)((s * Tr::kPageBytes) >> 4);
            if (Tr::k8) {
#pragma unroll
                for (int k = 0; k < kHeadDim / 32; ++k)
                    umma_e4m3(tmem + 128 * x + 64 * b, dq + 2 * k, dk + 2 * k, id_s, k > 0);
            } else {
#pragma unroll
                for (int k = 0; k < kHeadDim / 16; ++k) {
                    const uint32_t in = (k & 3) * 32;  // bytes within a half's rows
                    umma_bf16(tmem + 128 * x + 64 * b,
                              dq + (((k >> 2) * (kHeadRows * 128) + in) >> 4),
                              dk + (((k >> 2) * (kTile * 128) + in) >> 4), id_s, k > 0);
                }
            }
            if (Tr::kBlk) mbar_arrive(&s_full[2 * x + b]);
            umma_commit(&s_full[2 * x + b]);
            umma_commit(&empty[s]);
        };
        auto issue_pv = [&](uint32_t b, uint32_t page, bool acc) {
            const uint32_t s = page % W;
            const uint64_t dv = dv0 + (uint64_t)((s * Tr::kWideBytes) >> 4);
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
                umma_bf16_ts(tmem + kHeadOCol + 128 * x, tmem + 128 * x + 64 * b + 8 * k,
                             dv + (uint64_t)((k * 16 * 128) >> 4), id_o, acc || k > 0);
            umma_commit(&o_done[2 * x + b]);
            umma_commit(&v_free[s]);
        };
        uint32_t kt = 0, items = 0;
        uint32_t sp = 0, pp = 0;  // score pages issued, P pages taken
        uint32_t outs = 0;        // items whose O_x has been claimed
        for (int d = first; ok && d < last; ++d) {
            const HeadItem it = head_item(a.plan, d);
            ok = mbar_wait_warp(q_full, items & 1u, abort);
            ++items;
            if (!ok) break;
            const HeadPages pg = head_pages(it, kt, x);
            const uint64_t dq = dq0 + (uint64_t)((it.two ? x * Tr::kQBytes : 0) >> 4);
            if (pg.n == 0) {
                if (elect_one()) mbar_arrive(q_free);
                __syncwarp();
            }
            for (int c = -2; c < pg.n; ++c) {
                const bool next = c + 2 < pg.n;
                const uint32_t ks = pg.at + (uint32_t)(c + 2) * pg.step;
                const uint32_t vs = pg.at + (uint32_t)c * pg.step;
                if (next) ok = mbar_wait_warp(&full[ks % S], (ks / S) & 1u, abort);
                if (ok && c >= 0) {
                    ok = mbar_wait_warp(&p_full[2 * x + (pp & 1u)], (pp >> 1) & 1u, abort) &&
                         mbar_wait_warp(&v_full[vs % W], (vs / W) & 1u, abort);
                    if (ok && c == 0 && outs++ > 0)  // O_x of the item before is out
                        ok = mbar_wait_warp(&o_free[x], (outs - 2) & 1u, abort);
                }
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    if (c >= 0) issue_pv(pp & 1u, vs, c > 0);
                    if (next) issue_s(sp & 1u, dq, ks);
                    // the item's last scores
                    if (c + 3 == pg.n) umma_commit(q_free);
                }
                __syncwarp();
                if (c >= 0) ++pp;
                if (next) ++sp;
            }
            kt += it.hi - it.lo;
        }
        // arrives once every MMA issued has completed (TMEM is freed after it)
        if (elect_one()) umma_commit(mma_done);
        __syncwarp();
    } else if (Tr::k8 && warp >= kHeadWiden) {
        // V of a page, as it landed (rows of 128 codes, 16-byte groups swizzled), into
        // the two halves of 64 dims that the products take
        constexpr int NW = Tr::kWideners > 0 ? Tr::kWideners : 1;
        const int w = warp - kHeadWiden;
        uint32_t kt = 0;
        for (int d = first; ok && d < last; ++d) {
            const HeadItem it = head_item(a.plan, d);
            for (int j = it.lo; j < it.hi; ++j, ++kt) {
                const uint32_t s = kt % S, t = kt % W;
                ok = mbar_wait_warp(&full[s], (kt / S) & 1u, abort) &&
                     mbar_wait_warp(&v_free[t], ((kt / W) & 1u) ^ 1u, abort);
                if (!ok) break;
                const uint32_t src = smem_u32(smem + Tr::kOffCodes + s * Tr::kPageBytes);
                const uint32_t dst = smem_u32(smem + Tr::kOffV + t * Tr::kWideBytes);
                for (int e = 32 * w + lane; e < kTile * 8; e += 32 * NW) {
                    const int row = e >> 3, c = e & 7;  // token, 16 dims
                    const uint4 v = lds128(src + row * 128 + ((c ^ (row & 7)) << 4));
                    uint32_t o[8];
                    e4m3x4_to_f16x2x2(v.x, o[0], o[1]);
                    e4m3x4_to_f16x2x2(v.y, o[2], o[3]);
                    e4m3x4_to_f16x2x2(v.z, o[4], o[5]);
                    e4m3x4_to_f16x2x2(v.w, o[6], o[7]);
                    const uint32_t to = dst + (c >> 2) * (kTile * 128) + row * 128;
                    const int g = 2 * (c & 3);
                    sts128(to + ((g ^ (row & 7)) << 4), o[0], o[1], o[2], o[3]);
                    sts128(to + (((g + 1) ^ (row & 7)) << 4), o[4], o[5], o[6], o[7]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&v_full[t]);
                    mbar_arrive(&empty[s]);
                    if (!it.two && w == 0) mbar_arrive(&v_free[t]);  // for the half that leaves it
                }
            }
            if (ok && lane == 0) mbar_arrive(q_free);
        }
    } else if (warp < kHeadSoftmax) {
        // softmax of half x: thread = one query row, warp w reads TMEM lanes 32 (w mod 4) ..
        const int x = warp >> 2, q4 = warp & 3;
        const int rho = 32 * q4 + lane;
        const uint32_t row = tmem + ((uint32_t)(32 * q4) << 16);
        const uint32_t scol = row + 128 * x, ocol = row + kHeadOCol + 128 * x;
        const int tok_in = rho / a.G, g = rho - tok_in * a.G;
        // 8-bit pages: weights times 2^6 (see above)
        constexpr float kUp = Tr::k8 ? 6.f : 0.f;
        // Block scales: a term of the weights' sum is up to 2^88 times its weight (of a V
        // scale that counts as 2^-88 in the reference), so the sum is kept times 2^-8: below
        // 2^124 for the 2^30 tokens that a request may have.
        constexpr float kUnit = Tr::kBlk ? kSumUnit : 1.f;
        uint32_t ns = 0;  // score pages taken
        uint32_t kt = 0;
        for (int d = first; ok && d < last; ++d) {
            const HeadItem it = head_item(a.plan, d);
            const HeadPages pg = head_pages(it, kt, x);
            const int tok = it.tok + (it.two ? x * tpb : 0) + tok_in;
            const bool valid = tok_in < tpb && tok < it.end;
            float sc = a.score_scale;
            if (Tr::k8 && valid) sc *= __ldg(a.q_scale + (size_t)tok * a.Hq + it.h * a.G + g);
            if (!valid) sc = 0.f;  // (their scores may be anything)
            // a negative factor turns the maximum round: then the scores are scaled first
            const bool turned = __any_sync(kFullMask, sc < 0.f);
            float m_ref = -INFINITY, l = 0.f;
            for (int c = 0; c < pg.n; ++c) {
                const uint32_t b = ns & 1u;
                if (!mbar_wait_warp(&s_full[2 * x + b], (ns >> 1) & 1u, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t ra[32], rb[32];
                tmem_ld32_nowait(scol + 64 * b, ra);
                tmem_ld32_nowait(scol + 64 * b + 32, rb);
                const float *scales = reinterpret_cast<const float *>(
                    smem + Tr::kOffScale +
                    ((pg.at + (uint32_t)c * pg.step) % kScaleRing) * kPageScales * 4);
                tmem_wait_ld32x2(ra, rb);
                float s[kTile];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    s[i] = __uint_as_float(ra[i]);
                    s[32 + i] = __uint_as_float(rb[i]);
                }
                float f = sc;
                float lv[kPageScales / 2], vf[kPageScales / 2];  // V's scales, and their logarithms
                if (Tr::kBlk) {
#pragma unroll
                    for (int i = 0; i < kPageScales / 2; ++i) {
                        const float v = scales[kPageScales / 2 + i];
                        lv[i] = lg2(fmaxf(v, kMinVRef));
                        vf[i] = v < kMinVScale ? 0.f : v;
                    }
                }
                if (Tr::kBlk || turned) {
#pragma unroll
                    for (int i = 0; i < kTile; ++i)
                        s[i] *= Tr::kBlk ? scales[i / kScaleBlock] * sc : sc;
                    f = 1.f;
                }
                float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < kTile / 2; ++i) {
                    const int to = Tr::kBlk ? 2 * i / kScaleBlock : i & 3;
                    mx4[to] = head_max3(mx4[to], s[2 * i], s[2 * i + 1]);
                }
                if (Tr::kBlk) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) mx4[i] += lv[i];
                }
                const float m_tile = head_max3(fmaxf(mx4[0], mx4[1]), mx4[2], mx4[3]) * f;
                const bool need = m_tile > m_ref + kHeadLazy;
                const float new_ref = need ? m_tile : m_ref;
                // (in two steps: with block scales the reference may move by more than the
                // 126 that one holds, and the sum has terms that much larger than O's)
                const float step = need ? ex2((m_ref - new_ref) * (Tr::kBlk ? 0.5f : 1.f)) : 1.f;
                const float factor = Tr::kBlk ? step * step : step;
                const float base = (new_ref == -INFINITY ? 0.f : new_ref) - kUp;
                uint32_t pk[32];  // P as packed pairs, over the first half of the scores
                const float2 f2 = make_float2(f, f), nb2 = make_float2(-base, -base);
                float ps[8] = {};
                float2 *ps2 = reinterpret_cast<float2 *>(ps);
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float2 e = __ffma2_rn(make_float2(s[2 * i], s[2 * i + 1]), f2, nb2);
                    const float w0 = ex2(e.x), w1 = ex2(e.y);
                    if (Tr::kBlk) {
                        const float v = vf[2 * i / kScaleBlock];
                        pk[i] = pack_f16x2(w0 * v, w1 * v);
                        ps2[i & 3] = __ffma2_rn(make_float2(w0, w1), make_float2(kUnit, kUnit),
                                                ps2[i & 3]);
                    } else if (Tr::k8) {
                        pk[i] = pack_f16x2(w0, w1);
                        ps2[i & 3] = __fadd2_rn(ps2[i & 3], make_float2(w0, w1));
                    } else {
                        pk[i] = pack_bf16x2(w0, w1);
                    }
                }
                tmem_st32_nowait(scol + 64 * b, pk);
                // BF16: the sum takes the weights as they were rounded: the heaviest one's
                // rounding then cancels against its own in the product.  (f16 weights are
                // rounded to 2^-11.)
                if (KV == HPC_KV_BF16) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        head_add_bf16(ps[2 * (i & 3)], (uint16_t)pk[i]);
                        head_add_bf16(ps[2 * (i & 3) + 1], (uint16_t)(pk[i] >> 16));
                    }
                }
                if (Tr::kBlk) l *= step;
                l = l * step + (((ps[0] + ps[1]) + (ps[2] + ps[3])) +
                                  ((ps[4] + ps[5]) + (ps[6] + ps[7])));
                if (c > 0 && __any_sync(kFullMask, need)) {
                    // O_x is settled once its last product is done (the product two
                    // before that was issued before these scores' own: the phase cannot
                    // be mistaken)
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
                        for (int i = 0; i < 64; ++i) o[i] *= factor;
                        tmem_st32x2(ocol + 64 * hf, ocol + 64 * hf + 32, o);
                    }
                }
                tmem_wait_st32(pk);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[2 * x + b]);
                m_ref = new_ref;
                ++ns;
            }
            if (!ok) break;
            kt += it.hi - it.lo;
            const size_t at = (size_t)(it.slot + x) * kHeadRows + rho;
            // (l is NaN where a score is: so is the sum's logarithm, and the row)
            constexpr float kLow = kUp + (Tr::kBlk ? kSumLog2 : 0.f);
            if (valid) a.part_lse[at] = l == 0.f ? -INFINITY : (m_ref - kLow + lg2(l)) * kLn2;
            if (pg.n == 0) continue;  // (a partial of no weight: its values are not read)
            if (!mbar_wait_warp(&o_done[2 * x + ((ns - 1) & 1u)], ((ns - 1) >> 1) & 1u, abort)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const float inv = l == 0.f ? 0.f : (KV == HPC_KV_FP8_E4M3 ? a.v_scale : kUnit) / l;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                float o[64];
                tmem_ld32x2(ocol + 64 * hf, ocol + 64 * hf + 32, o);
                if (hf == 1) {  // the next item's products may begin
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&o_free[x]);
                }
#pragma unroll
                for (int i = 0; i < 64; ++i) o[i] *= inv;
                if (valid) {
#pragma unroll
                    for (int i = 0; i < 64; i += 8)
                        store_f32x8(a.part_o + at * kHeadDim + 64 * hf + i, o + i);
                }
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(end);
    }

    if (!ok) {
        if (lane == 0) atomicOr(a.meta + 3, (int)HPC_FLAG_TIMEOUT);
        *abort = 1;
    }
    if (warp == kHeadMma) {
        // no MMA may still write TMEM, and no softmax warp read it, when it is freed
        // (bounded, like every wait)
        volatile int no_abort = 0;
        mbar_wait(mma_done, 0, &no_abort);
        mbar_wait(end, 0, &no_abort);
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kHeadTmem);
    }
}

// The grid's kernel: Tail is what the CTAs without head work run.
template <hpc_kv_dtype KV, class Tail>
__global__ void __launch_bounds__(32 * HeadTraits<KV>::kWarps, 1)
    shared_kernel(const __grid_constant__ SharedMaps m, const __grid_constant__ AttnParams t,
                  const __grid_constant__ HeadArgs a) {
    grid_dependency_wait();  // the plan says which
    const int first = __ldg(a.plan.bin + blockIdx.x), last = __ldg(a.plan.bin + blockIdx.x + 1);
    if (first < last) head_cta<KV>(m, a, first, last);
    else Tail::run(m.tk, m.tv, t);
}

template <hpc_kv_dtype KV, class Tail>
struct SharedVariant {
    static constexpr int kThreads = 32 * HeadTraits<KV>::kWarps;
    static constexpr int kSmemBytes = HeadTraits<KV>::kSmemBytes > Tail::kSmemBytes
                                          ? HeadTraits<KV>::kSmemBytes
                                          : Tail::kSmemBytes;
    static_assert(kThreads >= Tail::kThreads, "threads");
    static AttnConfig config() {
        return {reinterpret_cast<const void *>(&shared_kernel<KV, Tail>), kSmemBytes, kThreads};
    }
    static cudaError_t launch(const SharedMaps &m, const AttnParams &t, const HeadArgs &h, int grid,
                              cudaStream_t s) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmemBytes;
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, shared_kernel<KV, Tail>, m, t, h);
    }
};

// The tail over 8-bit pages.
template <int RB, int HEADS, bool BLK>
struct TcTail {
    static constexpr int kThreads = kTcThreads, kSmemBytes = TcTraits<RB, HEADS, BLK>::kSmemBytes;
    static __device__ __forceinline__ void run(const CUtensorMap &tk, const CUtensorMap &tv,
                                               const AttnParams &t) {
        attn_tc_cta<RB, HEADS, BLK>(tk, tv, t);
    }
};

}  // namespace hpc
