// Decode attention over an 8-bit (E4M3) paged cache on the fifth-generation
// tensor cores, with a window and sinks (or none), and with one scale per
// cache or (BLK) one for each 16 tokens and head.  It drains the bins of the
// task map as the kernel in attn_kernel.cuh does, and shares its first-bin
// derivation, split buffer, chunk counting and merges.
//
// Why tcgen05 here: with up to 16 query rows per KV head the warp-level MMAs
// keep a warp busy for ~500 instructions per 16 tokens (widening V to f16,
// the fragments' moves, the softmax in accumulator layout); two such warps per
// scheduler reach 60% of the HBM rate.  Here tokens are the TMEM lanes:
//   S^T[token, row] = K[token, :] . Q^T       A = K as it lands (K-major, 128-
//       byte swizzle), B = Q;                  M = 128 tokens, N = 16 rows
//   O[dim, row] += V^T[dim, token] . P[token, row]   A = V as it lands (MN-
//       major), B = P, written by the softmax threads, one token each
// so one thread owns a token's scores of all rows, V is never converted, and a
// warp spends ~200 instructions per 32 tokens.
//
// Head pairs (HEADS = 2, an even number of KV heads): the rows of a page that
// belong to one 8-bit head are 128 bytes at a stride of Hkv * 128, and HBM
// serves such pieces at 4.3 .. 5.9 TB/s; two neighbouring heads make 256-byte
// pieces, which it serves at 6.7 (streams without arithmetic, 1 GB).  So a
// descriptor is a pair of heads, a stage one page of both (lanes 0-63 the first
// head's tokens, 64-127 the second's), and the map counts pairs.  An odd number
// of heads keeps one head per descriptor and two pages per stage.
//
// P in 8 bits would lose the weights' precision, so it goes in as three E5M2
// columns per row, w = h0 + h1 / 8 + h2 / 64: h0 the E5M2 of w, h1 that of 8
// times what h0 left, h2 of 8 times what h1 left (each difference exact in
// f16).  Each rounds by at most 2^-3 of what it is given: 2^-9 of the weight in
// all (BF16 weights, as the BF16 kernels have, 2^-8), down to steps of 2^-22
// with the largest weight between 2^3 and 2^14.5: E5M2's range, not E4M3's
// precision, is what a long tail of small weights needs.  The three products
// are separate accumulator columns, joined in fp32 at the end.  The softmax's
// sum takes the fp32 weight.
//
// Warps: 0 producer (TMA; K, V, Q and scales of a stage), 1 issues the first
// products, 2 the second (one warp for both took 1660 cycles a stage, more than
// HBM does), 4-7 and 8-11 two softmax warpgroups that take the stages in turn,
// 12-15 join and write.  Each softmax group keeps its own running reference m,
// sum and accumulator, so neither waits for the other; at its last stage of a
// descriptor it publishes the sum and the reference and goes on, and the join
// group brings the two accumulators together (a softmax group that did so
// itself stopped for 2 to 3 us at every descriptor).  The reference moves only
// when a weight would pass 2^14.5 (one barrier vote per stage); the group then
// rescales its accumulator in TMEM.
// Measured (queries, plan and merges included; the part of the measured copy
// rate that the cache's bytes alone make):
//   64 requests of 1K to 128K, 8 heads on 1, block scales, 560 MB: 89 us, 93%
//   64 of 512 to 16K, 64 heads on 8, two tokens, block scales, 731 MB: 122 us, 88%
//   128 of 1K to 32K, 16 on 2, window 1024, 69 MB: 23 us, 44%
//   48 of 500 to 16K, 48 on 8, two tokens, window 2048, 155 MB: 41 us, 56%
// The long streams run at the rate of HBM; what the short ones add is fixed: 5 us
// from the launch to the first stage's landing (lengths, block table, tiles, one
// after the other) and 6 to 8 us from the last landing to the end (softmax and
// product 2, join 2, the merges of units split between CTAs 1.5 to 2.5).
// With 16 rows per KV head (draft tokens, or a group above 8) the 128 registers that
// 512 threads leave are not enough for the softmax warps: 60 bytes are spilled with
// head pairs and 112 with single heads.  With 8 rows nothing is.
// Every wait is bounded.  Named barriers are reached by all four warps of a
// group: a wait that failed is voted on there, and the group leaves together.
#pragma once

#include <cuda_fp16.h>

#include "attn_kernel.cuh"
#include "tcgen05.cuh"

namespace hpc {

struct TcInfo {  // of a stage, written by the producer
    int kv_head, req, tile0, ntiles;
    int flags, seqlen, desc_idx, count;
    int chunk_off, skip, left, ord;  // left: stages of the descriptor after this one
    float qscale[2 * kMaxRows];  // of head y's row r at 16 y + r
    int group;  // softmax group (0, 1) of the descriptor's first stage
    int pad[3];
};
static_assert(sizeof(TcInfo) == 192, "TcInfo layout");

struct TcJoin {  // of a descriptor, for the join group
    DescInfo di;
    int only, end;  // only: the group (0, 1) that handled it alone, or -1; end: no more
    int group;      // the group that handled its first stage
};
static_assert(sizeof(TcJoin) == 32, "TcJoin layout");

constexpr int kTcTokens = 2 * kTile;    // of a stage: the MMA's 128 lanes
constexpr int kTcThreads = 32 * 16;
constexpr int kTcGroup = 128;           // threads of a softmax or join warpgroup
constexpr float kTcTop = 3.f;           // log2 of the largest weight when the reference moves
constexpr float kTcMax = 14.5f;         // log2 of the largest weight ever (E5M2 holds 1.75 2^15)
// A V scale below 2^-100 counts as zero.  In the reference none counts as less
// than 2^-88: the softmax's sum, of terms of up to 2^(14.5 + 88), must hold all
// tokens of a request (below 2^30; it is kept times 2^-8, and so stays below 2^125),
// and a weight at the reference's top (2^3) then still stands 2^10 above the three
// parts' last step at a scale of 2^-100.
constexpr float kMinVScale = 7.888609052210118e-31f;  // 2^-100
constexpr float kMinVRef = 3.2311742677852644e-27f;   // 2^-88
constexpr float kSumLog2 = -8.f, kSumUnit = 1.f / 256;  // of the sum: what its terms are times
constexpr int kTcOrds = 4;              // descriptors whose join data may be alive at once
constexpr int kTcPubs = 8 + 2;          // arrivals that publish one: the groups' warps, two products

// RB: query rows per KV head, padded to 8 or 16.  HEADS: KV heads of a
// descriptor (AttnParams' Hkv, G and R count descriptors' heads, their query
// heads and their rows).
template <int RB, int HEADS, bool BLK>
struct TcTraits {
    static constexpr int kPages = 2 / HEADS;                 // per stage
    static constexpr int STAGES = RB == 16 ? 5 : 6;
    static constexpr int kTileBytes = kTile * kHeadDim;      // one page of K or V, one head
    static constexpr int kStageKV = 2 * kTileBytes;          // 16 KB
    static constexpr int kQBytes = HEADS * RB * kHeadDim;
    static constexpr int kQRows = HEADS * RB < 16 ? 16 : HEADS * RB;  // N of the first product
    static constexpr int kPCols = RB == 16 ? 48 : 32;        // N of the second product
    static constexpr int kPBytes = kTcTokens * kPCols;
    static constexpr int kScaleBytes = BLK ? 2 * kPageScales * 4 : 0;
    static constexpr int kOffK = 0;
    static constexpr int kOffV = kOffK + STAGES * kStageKV;
    static constexpr int kOffQs = kOffV + STAGES * kStageKV;     // Q swizzled: [2][kQRows]
    static constexpr int kOffP = kOffQs + 2 * kQRows * kHeadDim;  // [2]
    static constexpr int kOffQ = kOffP + 2 * kPBytes;            // Q as it lands, per stage
    static constexpr int kOffInfo = kOffQ + STAGES * kQBytes;
    static constexpr int kOffScale = kOffInfo + STAGES * (int)sizeof(TcInfo);
    static constexpr int kOffRed = kOffScale + STAGES * kScaleBytes;  // [2][4 warps][16] floats
    static constexpr int kOffSum = kOffRed + 2 * 4 * 16 * 4;     // [ords][2][4][16] row sums
    static constexpr int kOffRef = kOffSum + kTcOrds * 2 * 4 * 16 * 4;  // [ords][2][32]
    static constexpr int kOffFac = kOffRef + kTcOrds * 2 * 32 * 4;  // [2 groups][32], join [3][32]
    static constexpr int kOffJoin = kOffFac + 5 * 32 * 4;           // [ords]
    static constexpr int kOffLast = kOffJoin + kTcOrds * (int)sizeof(TcJoin);
    // full[S], empty[S], s_full[2], p_full[2], o_done[2], o_free[2], pub[ords],
    // end, mma_done
    static constexpr int kOffBar = kOffLast + (kMaxLast + 1) * (int)sizeof(SlotInfo);
    static constexpr int kNumBars = 2 * STAGES + 8 + kTcOrds + 2;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;  // abort, TMEM address
    static constexpr int kSmemBytes = kOffMisc + 16 + 1024;
    static constexpr uint32_t kTmemCols = HEADS == 2 ? 512 : 256;
    // TMEM columns: S of group x; O of descriptor parity d, group x, head y
    static constexpr uint32_t s_col(int x) { return kQRows * x; }
    static constexpr uint32_t o_col(int d, int x, int y) {
        return 2 * kQRows + kPCols * ((2 * d + x) * HEADS + y);
    }
    static_assert(2 * kQRows + 4 * HEADS * kPCols <= kTmemCols, "TMEM columns");
    static_assert(kOffP % 1024 == 0 && kOffQ % 128 == 0, "operand alignment");
    static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};

struct TcBars {
    uint64_t *full, *empty, *s_full, *p_full, *o_done, *o_free, *pub, *end, *mma_done;
};

template <typename Tr>
__device__ __forceinline__ TcBars tc_bars(uint8_t *smem) {
    TcBars b;
    b.full = reinterpret_cast<uint64_t *>(smem + Tr::kOffBar);
    b.empty = b.full + Tr::STAGES;
    b.s_full = b.empty + Tr::STAGES;
    b.p_full = b.s_full + 2;
    b.o_done = b.p_full + 2;
    b.o_free = b.o_done + 2;
    b.pub = b.o_free + 2;
    b.end = b.pub + kTcOrds;
    b.mma_done = b.end + 1;
    return b;
}

// ------------------------------------------------------------------ wrappers
// Instruction descriptor of kind::f8f6f4: E4M3 A, E4M3 or E5M2 B, FP32
// accumulator.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N, bool a_mn, bool b_mn,
                                                      bool b_e5m2 = false) {
    return (1u << 4) | (b_e5m2 ? 1u << 10 : 0u) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// MN-major operand without swizzle: core matrices of 8 K indices x 16 bytes of
// MN (128 bytes, K index by K index), `k_bytes` from one group of 8 K to the
// next (leading offset), `mn_bytes` from one 16-byte group of MN to the next
// (stride offset).
__device__ __forceinline__ uint64_t smem_desc_mn_plain(uint32_t saddr, uint32_t k_bytes,
                                                       uint32_t mn_bytes) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(k_bytes >> 4) << 16) |
           ((uint64_t)(mn_bytes >> 4) << 32) | (1ull << 46);
}

__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}

// 8 or 16 columns of this thread's TMEM lane, waited for.
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t t, float (&v)[N]) {
    static_assert(N == 8 || N == 16, "columns");
    uint32_t r[N];
    if constexpr (N == 8)
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
            "tcgen05.wait::ld.sync.aligned;"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
              "=r"(r[7])
            : "r"(t)
            : "memory");
    else
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, "
            "%10, %11, %12, %13, %14, %15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
              "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
              "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(t)
            : "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]);
}

// The same in two steps: issued, then waited for (the registers are tied
// through the wait, so nothing uses them before it).
template <int N>
__device__ __forceinline__ void tmem_ld_cols_nowait(uint32_t t, uint32_t (&r)[N]) {
    static_assert(N == 8 || N == 16, "columns");
    if constexpr (N == 8)
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
              "=r"(r[7])
            : "r"(t)
            : "memory");
    else
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, "
            "%10, %11, %12, %13, %14, %15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
              "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
              "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(t)
            : "memory");
}

template <int N>
__device__ __forceinline__ void tmem_wait_cols(uint32_t (&r)[N], float (&v)[N]) {
    if constexpr (N == 8)
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                       "+r"(r[6]), "+r"(r[7])
                     :
                     : "memory");
    else
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                       "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                       "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                     :
                     : "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]);
}

template <int N>
__device__ __forceinline__ void tmem_st_cols(uint32_t t, const float (&v)[N]) {
    uint32_t r[N];
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = __float_as_uint(v[i]);
    if constexpr (N == 8)
        asm volatile(
            "tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};\n\t"
            "tcgen05.wait::st.sync.aligned;" ::"r"(r[0]),
            "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(t)
            : "memory");
    else
        asm volatile(
            "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, "
            "%9, %10, %11, %12, %13, %14, %15};\n\ttcgen05.wait::st.sync.aligned;" ::"r"(r[0]),
            "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
            "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
            "r"(r[15]), "r"(t)
            : "memory");
}

__device__ __forceinline__ void mbar_arrive_n(uint64_t *bar, uint32_t n) {
    asm volatile(
        "{\n\t.reg .b64 st;\n\t"
        "mbarrier.arrive.release.cta.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
        "r"(n)
        : "memory");
}

// True in every thread of the group if it is in one (all four warps reach it).
__device__ __forceinline__ bool group_any(int id, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(pred ? 1u : 0u), "r"(id)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                       uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

// Two f16 values -> two E5M2 codes (the low half's in the low byte), and back.
__device__ __forceinline__ uint32_t e5m2x2_of_f16x2(uint32_t x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t f16x2_of_e5m2x2(uint32_t x) {
    uint32_t r;
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(r) : "h"((uint16_t)x));
    return r;
}
// 8 (a - b) for two f16 values: exact for what an E5M2 rounding b of a left.
__device__ __forceinline__ uint32_t rest8(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("{\n\t.reg .b32 t;\n\tsub.rn.f16x2 t, %1, %2;\n\tmul.rn.f16x2 %0, t, %3;\n\t}"
        : "=r"(d)
        : "r"(a), "r"(b), "r"(0x48004800u));  // {8, 8}
    return d;
}

// Sums (or maxima) of v[0 .. N-1] over the warp's lanes: on return lane l holds
// that of row l / (32 / N).
template <int N, bool MAX>
__device__ __forceinline__ float warp_reduce_rows(float (&v)[N], int lane) {
    int o = 16;
#pragma unroll
    for (int n = N; n > 1; n >>= 1, o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float keep = up ? v[n / 2 + i] : v[i], give = up ? v[i] : v[n / 2 + i];
            const float got = __shfl_xor_sync(kFullMask, give, o);
            v[i] = MAX ? fmaxf(keep, got) : keep + got;
        }
    }
    float s = v[0];
    for (; o > 0; o >>= 1) {
        const float got = __shfl_xor_sync(kFullMask, s, o);
        s = MAX ? fmaxf(s, got) : s + got;
    }
    return s;
}

// A value that is the same in every lane, as one that the compiler knows to be.
__device__ __forceinline__ int uniform(int v) {
    return (int)__reduce_or_sync(kFullMask, (unsigned)v);
}

// ------------------------------------------------------------------ producer
// One descriptor through the ring; see stream_desc in attn_kernel.cuh for the
// derived-descriptor cases (desc_idx < 0) and the deferred map look-up.
template <int RB, int HEADS, bool BLK>
__device__ __forceinline__ bool tc_stream(const CUtensorMap *tmap_k, const CUtensorMap *tmap_v,
                                          const AttnParams &p, uint8_t *smem, int h, int r, int tb,
                                          int te, int desc_idx, int bin, FlyWalk *walk,
                                          int bin_pos, ProducerState &ps, int &ord,
                                          uint64_t policy, volatile int *abort) {
    using Tr = TcTraits<RB, HEADS, BLK>;
    constexpr int STAGES = Tr::STAGES;
    const int lane = threadIdx.x & 31;
    TcInfo *info = reinterpret_cast<TcInfo *>(smem + Tr::kOffInfo);
    const TcBars bar = tc_bars<Tr>(smem);
    if (tb >= te) return true;
    h = uniform(h), r = uniform(r), tb = uniform(tb), te = uniform(te);
    const int L = clamp_len(p, p.seqlens[r]);
    const int skip = window_skip(L, p.q_len, p.window, p.sink_tiles);
    const int u = h * p.B + r, group = (int)(ps.it & 1u);
    // lane: row i G + g' of the descriptor, g' = y Gh + g of its head y
    float qs = 1.f;
    int qs_at = -1;
    if (lane < p.R) {
        const int i = lane / p.G, gg = lane - i * p.G, Gh = p.G / HEADS, y = gg / Gh;
        qs = p.q_scale[((size_t)r * p.q_len + i) * p.Hq + h * p.G + gg];
        qs_at = kMaxRows * y + i * Gh + gg - y * Gh;
    }
    const uint32_t q_group = (uint32_t)(p.G * kHeadDim);
    const uint32_t q_bytes = q_group * (uint32_t)p.q_len;
    const size_t q_token_stride = (size_t)p.Hq * kHeadDim;
    const uint8_t *q_src = static_cast<const uint8_t *>(p.q) +
                           ((size_t)r * p.q_len * p.Hq + (size_t)h * p.G) * kHeadDim;
    const int32_t *bt_row = p.block_table + (size_t)r * p.max_pages;
    auto entry = [&](int t) {
        return min(t < p.sink_tiles ? t : t + skip, p.max_pages - 1);
    };
    int page0 = 0;
    if (lane < min(32, te - tb)) page0 = bt_row[entry(tb + lane)];

    for (int t0 = tb; t0 < te; t0 += 32) {  // 32 block-table entries at a time
        const int nt = min(32, te - t0);
        int page = 0;
        if (lane < nt) {
            page = t0 == tb ? page0 : bt_row[entry(t0 + lane)];
            if (page < 0 || page >= p.num_pages) {
                ps.late_flags |= HPC_FLAG_BAD_PAGE;
                page = 0;
            }
        }
        for (int k = 0; k < nt; k += Tr::kPages) {
            const int ns = min(Tr::kPages, nt - k), t = t0 + k;
            const int pg0 = uniform(__shfl_sync(kFullMask, page, k));
            const int pg1 = uniform(__shfl_sync(kFullMask, page, min(k + 1, 31)));
            const bool first = t == tb, last = t + ns == te;
            const bool defer = last && desc_idx < 0 && !walk && !ps.waited;
            int idx = desc_idx, count = 0, chunk_off = 0;
            if (last && walk) {
                walk_chunk(p, *walk, idx, count, chunk_off);
            } else if (last && !defer) {
                wait_for_map(ps);
                if (idx < 0) idx = p.bin_ptr[bin] + bin_pos;
                if (p.chunk_count) {
                    count = p.chunk_count[u];
                    chunk_off = p.chunk_off[u];
                }
            }
            const int stage = ps.it % STAGES;
            if (!warp_wait(&bar.empty[stage], ((ps.it / STAGES) & 1u) ^ 1u, abort)) return false;
            uint64_t *full = &bar.full[stage];
            TcInfo &si = info[stage];
            if (elect_one()) {
                mbar_expect_tx(full, (uint32_t)(ns * HEADS) *
                                             (2u * Tr::kTileBytes + (BLK ? kPageScales * 4u : 0u)) +
                                         (first ? q_bytes : 0u));
                uint8_t *sk = smem + Tr::kOffK + stage * Tr::kStageKV;
                uint8_t *sv = smem + Tr::kOffV + stage * Tr::kStageKV;
#pragma unroll
                for (int s = 0; s < Tr::kPages; ++s) {
                    if (s >= ns) break;
                    const int pg = s ? pg1 : pg0;
                    tma_load_4d(sk + s * Tr::kTileBytes, tmap_k, full, 0, 0, HEADS * h, pg, policy);
                    tma_load_4d(sv + s * Tr::kTileBytes, tmap_v, full, 0, 0, HEADS * h, pg, policy);
                    if (BLK)
                        bulk_load(smem + Tr::kOffScale + stage * Tr::kScaleBytes +
                                      s * kPageScales * 4,
                                  p.kv_scale + ((size_t)pg * p.Hkv + h) * HEADS * kPageScales,
                                  HEADS * kPageScales * 4, full);
                }
                if (first)
                    for (int i = 0; i < p.q_len; ++i)
                        bulk_load(smem + Tr::kOffQ + stage * Tr::kQBytes + i * q_group,
                                  q_src + i * q_token_stride, q_group, full);
                si.kv_head = h;
                si.req = r;
                si.tile0 = t;
                si.ntiles = ns;
                si.flags = (first ? kFirst : 0) | (last ? kLast : 0);
                si.seqlen = L;
                si.skip = skip;
                si.left = (te - t - ns + Tr::kPages - 1) / Tr::kPages;
                si.ord = ord;
                si.group = group;
            }
            if (defer) {  // the stage's copies are on their way
                wait_for_map(ps);
                idx = p.bin_ptr[bin] + bin_pos;
                if (p.chunk_count) {
                    count = p.chunk_count[u];
                    chunk_off = p.chunk_off[u];
                }
            }
            if (qs_at >= 0) si.qscale[qs_at] = qs;
            __syncwarp();
            if (lane == 0) {
                si.desc_idx = idx;
                si.count = count;
                si.chunk_off = chunk_off;
                mbar_arrive(full);  // releases the stage's fields with its bytes
            }
            ++ps.it;
        }
    }
    ++ord;
    return true;
}

template <int RB, int HEADS, bool BLK>
__device__ __forceinline__ void tc_producer(const CUtensorMap *tmap_k, const CUtensorMap *tmap_v,
                                            const AttnParams &p, uint8_t *smem,
                                            volatile int *abort) {
    using Tr = TcTraits<RB, HEADS, BLK>;
    constexpr int STAGES = Tr::STAGES;
    const int lane = threadIdx.x & 31;
    TcInfo *info = reinterpret_cast<TcInfo *>(smem + Tr::kOffInfo);
    const TcBars bar = tc_bars<Tr>(smem);
    const uint64_t policy = policy_evict_first();
    ProducerState ps{0u, false, 0u};
    bool ok = true;
    int ord = 0, skip = 0;
    const bool dynamic = p.num_bins > (int)gridDim.x;
    bool walked = false;
    // the first bin's descriptors from the lengths, as in attn_producer
    if (p.fly && p.B <= kWalkMaxBatch) {
        FlyWalk w;
        walk_init<true>(p, blockIdx.x, w);
        int streamed = 0;
        while (ok && w.te > w.tb) {
            const bool derive = streamed + (w.te - w.tb) < kWalkTiles;
            ok = tc_stream<RB, HEADS, BLK>(tmap_k, tmap_v, p, smem, w.h, w.r, w.tb, w.te, -1,
                                            blockIdx.x, derive ? &w : nullptr, w.k, ps, ord,
                                            policy, abort);
            ++skip;
            streamed += w.te - w.tb;
            if (!derive) break;
            walk_next(p, w);
        }
        walked = ok && w.te == w.tb && !ps.waited && !dynamic;
    } else if (p.fly) {
        int h, r, tb, te;
        if (first_descriptor<true>(p, blockIdx.x, h, r, tb, te) && te > tb) {
            ok = tc_stream<RB, HEADS, BLK>(tmap_k, tmap_v, p, smem, h, r, tb, te, -1, blockIdx.x,
                                            nullptr, 0, ps, ord, policy, abort);
            skip = 1;
        }
    }
    if (!walked) wait_for_map(ps);
    int bin = blockIdx.x;
    while (ok && !walked) {
        int grab = 0;
        if (dynamic && lane == 0) grab = atomicAdd(p.bin_counter, 1);
        const int d_begin = p.bin_ptr[bin] + (bin == (int)blockIdx.x ? skip : 0);
        const int d_end = p.bin_ptr[bin + 1];
        for (int d = d_begin; d < d_end && ok; ++d) {
            const int4 ds = p.desc[d];
            ok = tc_stream<RB, HEADS, BLK>(tmap_k, tmap_v, p, smem, ds.x, ds.y, ds.z, ds.w, d,
                                            bin, nullptr, 0, ps, ord, policy, abort);
        }
        if (!dynamic) break;
        grab = __shfl_sync(kFullMask, grab, 0);
        if (grab == p.num_bins - 1 && lane == 0) *p.bin_counter = 0;
        bin = (int)gridDim.x + grab;
        if (bin >= p.num_bins) break;
    }
    for (int e = 0; e < 2 && ok; ++e) {  // a terminator for each softmax group
        const int stage = ps.it % STAGES;
        if (!warp_wait(&bar.empty[stage], ((ps.it / STAGES) & 1u) ^ 1u, abort)) {
            ok = false;
            break;
        }
        if (lane == 0) {
            info[stage].flags = kEnd | (e == 0 ? kFirst : 0);
            info[stage].ord = ord;
            mbar_arrive(&bar.full[stage]);
        }
        ++ps.it;
    }
    if (!ok) ps.late_flags |= HPC_FLAG_TIMEOUT;
    const unsigned flags = __reduce_or_sync(kFullMask, ps.late_flags);
    if (flags) {
        wait_for_map(ps);  // meta[3] is written by the assign kernel
        if (lane == 0) atomicOr(p.meta + 3, (int)flags);
    }
    // no copy this warp issued may land after the CTA has left (bounded)
    volatile int no_abort = 0;
    const uint32_t from = ps.it > (uint32_t)STAGES ? ps.it - STAGES : 0u;
    for (uint32_t j = from; j < ps.it; ++j)
        mbar_wait(&bar.full[j % STAGES], (j / STAGES) & 1u, &no_abort);
    __syncwarp();
}

// ------------------------------------------------------------------ MMA issue

// First products: S of each stage, once it has landed and its group has taken
// the scores of the stage before the last.
template <int RB, int HEADS, bool BLK>
__device__ __forceinline__ bool tc_scores(const AttnParams &p, uint8_t *smem, uint32_t tmem,
                                          volatile int *abort) {
    using Tr = TcTraits<RB, HEADS, BLK>;
    constexpr int STAGES = Tr::STAGES;
    const int lane = threadIdx.x & 31;
    const TcInfo *info = reinterpret_cast<const TcInfo *>(smem + Tr::kOffInfo);
    const TcBars bar = tc_bars<Tr>(smem);
    constexpr uint32_t kId = idesc_e4m3_f32(128, Tr::kQRows, false, false);
    const uint64_t dk0 = smem_desc_k128(smem_u32(smem + Tr::kOffK));
    const uint64_t dq0 = smem_desc_k128(smem_u32(smem + Tr::kOffQs));
    int ends = 0;
    for (uint32_t it = 0; ends < 2; ++it) {
        const int s = it % STAGES, x = it & 1;
        if (!warp_wait(&bar.full[s], (it / STAGES) & 1u, abort)) return false;
        const int flags = uniform(info[s].flags), ord = uniform(info[s].ord);
        if (!(flags & kEnd) && (flags & kFirst)) {  // Q into the swizzled operand, padded with zeros
            // (the buffer's last descriptor, ord - 2, has had all its scores taken)
            const uint8_t *q = smem + Tr::kOffQ + s * Tr::kQBytes;
            uint8_t *dst = smem + Tr::kOffQs + (ord & 1) * Tr::kQRows * kHeadDim;
            if (it >= 2 && !warp_wait(&bar.p_full[x], ((it >> 1) - 1) & 1u, abort)) return false;
            const int Gh = p.G / HEADS, Rh = p.R / HEADS;
            for (int c = lane; c < Tr::kQRows * 8; c += 32) {
                const int row = c >> 3, col = c & 7;
                // operand row y RB + r, r = i Gh + g; as it lands: i G + y Gh + g
                const int y = row / RB, r = row - y * RB, i = r / Gh;
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (y < HEADS && r < Rh)
                    v = *reinterpret_cast<const uint4 *>(
                        q + (i * p.G + y * Gh + (r - i * Gh)) * 128 + col * 16);
                *reinterpret_cast<uint4 *>(dst + row * 128 + ((col ^ (row & 7)) << 4)) = v;
            }
            fence_proxy_async_smem();
            __syncwarp();
        } else if (it >= 2 && !warp_wait(&bar.p_full[x], ((it >> 1) - 1) & 1u, abort)) {
            return false;
        }
        if (elect_one()) {
            if (flags & kEnd) {
                mbar_arrive(&bar.s_full[x]);
            } else {
                tc_fence_after();
                const uint64_t dk = dk0 + (uint64_t)((s * Tr::kStageKV) >> 4);
                const uint64_t dq = dq0 + (uint64_t)(((ord & 1) * Tr::kQRows * kHeadDim) >> 4);
#pragma unroll
                for (int k = 0; k < kHeadDim / 32; ++k)
                    umma_e4m3(tmem + Tr::s_col(x), dk + 2 * k, dq + 2 * k, kId, k > 0);
                umma_commit(&bar.s_full[x]);
            }
        }
        if (flags & kEnd) ++ends;
        __syncwarp();
    }
    return true;
}

// Second products: O += V^T P of each stage, once its group has written P.
template <int RB, int HEADS, bool BLK>
__device__ __forceinline__ bool tc_products(const AttnParams &p, uint8_t *smem, uint32_t tmem,
                                            volatile int *abort) {
    using Tr = TcTraits<RB, HEADS, BLK>;
    constexpr int STAGES = Tr::STAGES;
    const TcInfo *info = reinterpret_cast<const TcInfo *>(smem + Tr::kOffInfo);
    const TcBars bar = tc_bars<Tr>(smem);
    constexpr uint32_t kId = idesc_e4m3_f32(128, Tr::kPCols, true, true, true);
    const uint64_t dv0 = smem_desc_mn128(smem_u32(smem + Tr::kOffV), 16);
    // token groups of 8 are 128 bytes apart, 16-byte column groups 2 KB
    const uint64_t dp0 = smem_desc_mn_plain(smem_u32(smem + Tr::kOffP), 128, 16 * kTcTokens);
    int ord_of[2] = {-1, -1};  // descriptor a group's accumulator belongs to
    int opened = -1;           // last descriptor whose accumulators were claimed
    for (uint32_t it = 0;; ++it) {
        const int s = it % STAGES, x = it & 1;
        if (!warp_wait(&bar.full[s], (it / STAGES) & 1u, abort)) return false;
        const int flags = uniform(info[s].flags), ord = uniform(info[s].ord);
        const int left = uniform(info[s].left);
        if (flags & kEnd) return true;
        // its group's last stage of the descriptor: the join waits for it (a
        // descriptor of one stage stands for both groups)
        const int pubs = left > 1 ? 0 : left == 0 && (flags & kFirst) ? 2 : 1;
        if (!warp_wait(&bar.p_full[x], (it >> 1) & 1u, abort)) return false;
        if (ord > opened) {  // descriptor ord - 2 has been read out of these columns
            if (ord >= 2 && !warp_wait(&bar.o_free[ord & 1], ((ord >> 1) - 1) & 1, abort))
                return false;
            opened = ord;
        }
        if (elect_one()) {
            tc_fence_after();
            const uint64_t dv = dv0 + (uint64_t)((s * Tr::kStageKV) >> 4);
            const uint64_t dp = dp0 + (uint64_t)((x * Tr::kPBytes) >> 4);
            const uint32_t o0 = tmem + Tr::o_col(ord & 1, x, 0);
            constexpr int kSteps = kTcTokens / 32 / HEADS;  // of 32 tokens, per head
#pragma unroll
            for (int k = 0; k < kTcTokens / 32; ++k) {
                const uint32_t o = o0 + Tr::kPCols * (k / kSteps);
                const bool acc = ord_of[x] == ord || k % kSteps > 0;
                umma_e4m3(o, dv + (uint64_t)((k * 32 * 128) >> 4),
                          dp + (uint64_t)((k * 32 * 16) >> 4), kId, acc);
            }
            umma_commit(&bar.empty[s]);
            umma_commit(&bar.o_done[x]);
            if (pubs > 0) umma_commit(&bar.pub[ord % kTcOrds]);
            if (pubs > 1) umma_commit(&bar.pub[ord % kTcOrds]);
        }
        ord_of[x] = ord;
        __syncwarp();
    }
}

// ------------------------------------------------------------------ softmax
template <int RB, int HEADS, bool BLK>
__device__ __forceinline__ bool tc_softmax(const AttnParams &p, uint8_t *smem, uint32_t tmem,
                                           int x, volatile int *abort) {
    using Tr = TcTraits<RB, HEADS, BLK>;
    constexpr int STAGES = Tr::STAGES;
    const int lane = threadIdx.x & 31, q4 = (threadIdx.x >> 5) & 3;
    const int tid = 32 * q4 + lane;  // token of the stage, then dim of the output
    const int bid = 1 + x;           // named barrier of the group
    const int hd = HEADS == 2 ? q4 >> 1 : 0;       // the head this thread's token belongs to
    const int pos = HEADS == 2 ? 0 : tid >> 6;     // its page of the stage
    const int Gh = p.G / HEADS, Rh = p.R / HEADS;  // query heads and rows of one KV head
    const TcInfo *info = reinterpret_cast<const TcInfo *>(smem + Tr::kOffInfo);
    const TcBars bar = tc_bars<Tr>(smem);
    float *red = reinterpret_cast<float *>(smem + Tr::kOffRed) + x * 64;
    float *sums = reinterpret_cast<float *>(smem + Tr::kOffSum);
    float *refs = reinterpret_cast<float *>(smem + Tr::kOffRef);
    float *fac = reinterpret_cast<float *>(smem + Tr::kOffFac) + x * 32;
    TcJoin *joins = reinterpret_cast<TcJoin *>(smem + Tr::kOffJoin);
    const uint32_t lane_base = tmem + ((uint32_t)(32 * q4) << 16);
    const uint32_t p_row = smem_u32(smem + Tr::kOffP) + x * Tr::kPBytes + tid * 16;

    float m[RB], l[RB], sc[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) m[r] = l[r] = sc[r] = 0.f;
    int cur = -1;  // descriptor the state belongs to
    for (uint32_t n = 0;; ++n) {  // this group's n-th stage
        const uint32_t it = 2 * n + x;
        const int s = it % STAGES;
        // the scores are ready, the stage's fields and scales with them
        bool ok = warp_wait(&bar.s_full[x], n & 1u, abort);
        float d[RB];
        uint32_t dr[RB];
        tc_fence_after();
        tmem_ld_cols_nowait<RB>(lane_base + Tr::s_col(x) + hd * RB, dr);
        ok = ok && warp_wait(&bar.full[s], (it / STAGES) & 1u, abort);
        const int flags = info[s].flags;
        const bool end = flags & kEnd;
        if (!ok || end) {  // leave together (the others meet both votes below)
            tmem_wait_cols<RB>(dr, d);
            // (the slot written below was last used by a descriptor that has been
            // joined once this group's last product is done)
            if (ok && n > 0) ok = warp_wait(&bar.o_done[x], (n - 1) & 1u, abort);
            group_any(bid, true);
            if (group_any(bid, !ok)) return false;
            if (flags & kFirst) {  // the first terminator: tell the join group
                const int slot = info[s].ord % kTcOrds;
                if (tid == 0) joins[slot].end = 1;
                __syncwarp();
                if (lane == 0) mbar_arrive_n(&bar.pub[slot], q4 == 0 ? 4 : 2);
            }
            return true;
        }
        const int ord = info[s].ord, L = info[s].seqlen, ntiles = info[s].ntiles;
        int tile = info[s].tile0 + pos;
        if (tile >= p.sink_tiles) tile += info[s].skip;
        const int tok = tile * kTile + (tid & 63);
        bool fresh = false;  // first stage of this descriptor for this group
        if (ord != cur) {
            cur = ord;
            fresh = true;
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                sc[r] = r < Rh ? p.score_scale * info[s].qscale[kMaxRows * hd + r] : 0.f;
                m[r] = r < Rh ? -3e38f : 3e38f;  // (a padding row never moves)
                l[r] = 0.f;
            }
        }
        const int lo0 = L - p.q_len + 1 - p.window;
        const bool live = pos < ntiles && tok < L && (tok >= lo0 || tok < p.sinks);
        float kf = 1.f, vf = 1.f, lv = 0.f;
        if (BLK) {
            const float *bs = reinterpret_cast<const float *>(
                                  smem + Tr::kOffScale + s * Tr::kScaleBytes) +
                              (tid >> 6) * kPageScales + ((tid & 63) / kScaleBlock);
            kf = live ? bs[0] : 0.f;
            vf = live ? bs[kPageScales / 2] : 0.f;
            lv = lg2(fmaxf(vf, kMinVRef));
            vf = vf < kMinVScale ? 0.f : vf;
        }
        // every row sees the warp's 32 tokens: no masks
        const int w0 = tok - lane;
        const bool full = pos < ntiles && w0 + 31 < L - p.q_len + 1 &&
                          (w0 + p.window >= L || w0 + 31 < p.sinks);
        tmem_wait_cols<RB>(dr, d);
        float top = kNegInf;
        if (!full) {  // a masked score is -inf whatever the operands held
            int qi = 0, g = 0;
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                const int limit = L - p.q_len + 1 + qi;
                if (!(live && tok < limit && (tok + p.window >= limit || tok < p.sinks)))
                    d[r] = kNegInf;
                else
                    d[r] *= kf * sc[r];
                if (++g == Gh) g = 0, qi = min(qi + 1, p.q_len - 1);
            }
        } else {
#pragma unroll
            for (int r = 0; r < RB; ++r) d[r] *= kf * sc[r];
        }
#pragma unroll
        for (int r = 0; r < RB; ++r) top = fmaxf(top, d[r] - m[r]);
        if (group_any(bid, top + lv > kTcMax)) {
            // (a rescale follows the group's previous product)
            if (!fresh && n > 0) ok = warp_wait(&bar.o_done[x], (n - 1) & 1u, abort);
            if (group_any(bid, !ok)) return false;  // a warp's wait failed, here or above
            if (!fresh) tc_fence_after();
            // move the reference: the rows' largest weights of this stage
            __syncwarp();
            {
                float v[RB];
#pragma unroll
                for (int r = 0; r < RB; ++r) v[r] = d[r] + lv;
                const float t = warp_reduce_rows<RB, true>(v, lane);
                constexpr int kPer = 32 / RB;  // lanes that hold the same row
                if (lane % kPer == 0) red[q4 * 16 + lane / kPer] = t;
            }
            named_bar_sync(bid, kTcGroup);
            float al[RB];
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                const float v = HEADS == 2
                                    ? fmaxf(red[32 * hd + r], red[32 * hd + 16 + r])
                                    : fmaxf(fmaxf(red[r], red[16 + r]), fmaxf(red[32 + r], red[48 + r]));
                const float mn = fmaxf(m[r], v - kTcTop);
                const float move = m[r] - mn;
                al[r] = ex2(move);
                m[r] = mn;
                // Block scales: the reference may move by 200, and the sum's terms are that
                // much larger than O's, but one factor holds 2^-126 at the least.  So in two
                // steps, or by the sum's logarithm (off by 2^-22 of itself, 2e-5 of the sum at
                // the most): 123.1 and 125.8 us with 8 rows (64
                // requests of 64 heads, 8K to 10K tokens; 123.1 without either), 49.1 and 48.6
                // with 16 (48 requests of 48 heads, two tokens each; 48.0).
                if (!BLK) {
                    l[r] *= al[r];
                } else if (RB == 8) {
                    const float half = ex2(0.5f * move);
                    l[r] = l[r] * half * half;
                } else {
                    l[r] = ex2(lg2(l[r]) + move);
                }
            }
            // O (lanes: dims) from the old reference's units to the new one's; both
            // heads' factors are needed in every thread
            if (tid % 64 == 0)
#pragma unroll
                for (int r = 0; r < RB; ++r)
                    if (HEADS == 2 || tid == 0) fac[16 * hd + r] = al[r];
            named_bar_sync(bid, kTcGroup);  // (red may be written again)
            if (!fresh) {
#pragma unroll
                for (int y = 0; y < HEADS; ++y) {
                    const uint32_t oc = lane_base + Tr::o_col(ord & 1, x, y);
#pragma unroll
                    for (int c = 0; c < 3; ++c) {
                        float o[RB];
                        tmem_ld_cols<RB>(oc + RB * c, o);
#pragma unroll
                        for (int r = 0; r < RB; ++r)
                            o[r] *= HEADS == 2 ? fac[16 * y + r] : al[r];
                        tmem_st_cols<RB>(oc + RB * c, o);
                    }
                }
            }
        }
        // weights, their sum, and their three 8-bit parts
        uint32_t h0[RB / 2], h1[RB / 2], h2[RB / 2];
#pragma unroll
        for (int i = 0; i < RB / 2; ++i) {
            const float a = ex2(d[2 * i] - m[2 * i]), b = ex2(d[2 * i + 1] - m[2 * i + 1]);
            l[2 * i] = fmaf(a, kSumUnit, l[2 * i]);
            l[2 * i + 1] = fmaf(b, kSumUnit, l[2 * i + 1]);
            const uint32_t w = BLK ? pack_f16x2(a * vf, b * vf) : pack_f16x2(a, b);
            h0[i] = e5m2x2_of_f16x2(w);
            const uint32_t r1 = rest8(w, f16x2_of_e5m2x2(h0[i]));
            h1[i] = e5m2x2_of_f16x2(r1);
            h2[i] = e5m2x2_of_f16x2(rest8(r1, f16x2_of_e5m2x2(h1[i])));
        }
        // the previous weights have been multiplied (a wait that fails sets the
        // abort word, which the group's next wait meets)
        if (n > 0) warp_wait(&bar.o_done[x], (n - 1) & 1u, abort);
        if constexpr (RB == 16) {
            sts128(p_row, h0[0] | h0[1] << 16, h0[2] | h0[3] << 16, h0[4] | h0[5] << 16,
                   h0[6] | h0[7] << 16);
            sts128(p_row + 2048, h1[0] | h1[1] << 16, h1[2] | h1[3] << 16, h1[4] | h1[5] << 16,
                   h1[6] | h1[7] << 16);
            sts128(p_row + 4096, h2[0] | h2[1] << 16, h2[2] | h2[3] << 16, h2[4] | h2[5] << 16,
                   h2[6] | h2[7] << 16);
        } else {
            sts128(p_row, h0[0] | h0[1] << 16, h0[2] | h0[3] << 16, h1[0] | h1[1] << 16,
                   h1[2] | h1[3] << 16);
            sts128(p_row + 2048, h2[0] | h2[1] << 16, h2[2] | h2[3] << 16, 0u, 0u);
        }
        if (!live) {  // this token's V row may hold anything: zero it
            const uint32_t v = smem_u32(smem + Tr::kOffV) + s * Tr::kStageKV + tid * 128;
#pragma unroll
            for (int c = 0; c < 8; ++c) sts128(v + 16 * c, 0u, 0u, 0u, 0u);
        }
        const int left = info[s].left, group = info[s].group;
        const DescInfo di = {info[s].req, info[s].kv_head, info[s].desc_idx, info[s].count,
                             info[s].chunk_off};
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[x]);  // the warp's weights, its reads of the stage
        if (left >= 2) continue;

        // ---- this group's last stage of the descriptor: publish sum and reference
        const int slot = ord % kTcOrds;
        const bool alone = (flags & kFirst) && left == 0;  // the descriptor's only stage
        {
            const float t = warp_reduce_rows<RB, false>(l, lane);
            constexpr int kPer = 32 / RB;  // lanes that hold the same row
            if (lane % kPer == 0) sums[((slot * 2 + x) * 4 + q4) * 16 + lane / kPer] = t;
            if (HEADS == 2 ? tid % 64 == 0 : tid == 0)
#pragma unroll
                for (int r = 0; r < RB; ++r) refs[(slot * 2 + x) * 32 + 16 * hd + r] = m[r];
            if (tid == 0 && left == 0) joins[slot] = TcJoin{di, alone ? x : -1, 0, group};
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_n(&bar.pub[slot], alone ? 2 : 1);
    }
}

// ------------------------------------------------------------------ join
// Of each descriptor in turn: the two groups' accumulators, in the units of
// their references, under one normalisation, as BF16 output or partial.
template <int RB, int HEADS, bool BLK>
__device__ __forceinline__ bool tc_join(const AttnParams &p, uint8_t *smem, uint32_t tmem,
                                        volatile int *abort) {
    using Tr = TcTraits<RB, HEADS, BLK>;
    const int lane = threadIdx.x & 31, q4 = (threadIdx.x >> 5) & 3;
    const int tid = 32 * q4 + lane;  // dim of the output
    const int bid = 3;
    const TcBars bar = tc_bars<Tr>(smem);
    const float *sums = reinterpret_cast<const float *>(smem + Tr::kOffSum);
    const float *refs = reinterpret_cast<const float *>(smem + Tr::kOffRef);
    float *fac = reinterpret_cast<float *>(smem + Tr::kOffFac) + 64;
    const TcJoin *joins = reinterpret_cast<const TcJoin *>(smem + Tr::kOffJoin);
    SlotInfo *last = reinterpret_cast<SlotInfo *>(smem + Tr::kOffLast);  // [0].flags: count
    const uint32_t lane_base = tmem + ((uint32_t)(32 * q4) << 16);
    const int Gh = p.G / HEADS, Rh = p.R / HEADS;
    const bool fused = p.out != nullptr;
    grid_dependency_wait();  // before this grid's first global writes
    for (int ord = 0;; ++ord) {
        const int slot = ord % kTcOrds;
        const bool ok = warp_wait(&bar.pub[slot], (ord / kTcOrds) & 1, abort);
        if (group_any(bid, !ok)) return false;
        const TcJoin j = joins[slot];
        if (j.end) return true;
        const DescInfo di = j.di;
        if (tid < 16 * HEADS && tid % 16 < RB) {  // head tid / 16, row tid % 16
            const int y = tid / 16, r = tid % 16;
            float ls[2], z[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {  // the two softmax groups
                const float *sk = sums + (slot * 2 + k) * 64 + 32 * y + r;
                z[k] = j.only == (k ^ 1) ? 0.f
                       : HEADS == 2      ? sk[0] + sk[16]
                                         : (sk[0] + sk[16]) + (sk[32] + sk[48]);
                ls[k] = z[k] > 0.f ? refs[(slot * 2 + k) * 32 + tid] + (lg2(z[k]) - kSumLog2)
                                   : kNegInf;
            }
            const float M = fmaxf(ls[0], ls[1]);
            const float e0 = z[0] > 0.f ? ex2(ls[0] - M) : 0.f;
            const float e1 = z[1] > 0.f ? ex2(ls[1] - M) : 0.f;
            const float Z = e0 + e1;
            // out = sum_k O_k / z_k * e_k / Z (z in units of 1 / kSumUnit)
            fac[tid] = z[0] > 0.f ? p.v_scale * e0 / (z[0] * Z) * kSumUnit : 0.f;
            fac[32 + tid] = z[1] > 0.f ? p.v_scale * e1 / (z[1] * Z) * kSumUnit : 0.f;
            fac[64 + tid] = Z > 0.f ? (M + lg2(Z)) * kLn2 : kNegInf;  // natural-log LSE
        }
        named_bar_sync(bid, kTcGroup);
        // the group of the descriptor's first stage first: where a stage stands in
        // the CTA's stream (a race, with more bins than CTAs) decides which one that
        // is, and may not decide how the sum below rounds
        const int group = uniform(j.group);
        float out[HEADS][RB];
        tc_fence_after();
#pragma unroll
        for (int y = 0; y < HEADS; ++y) {
#pragma unroll
            for (int r = 0; r < RB; ++r) out[y][r] = 0.f;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int k = n ^ group;
                if (j.only == (k ^ 1)) continue;
                const uint32_t oc = lane_base + Tr::o_col(ord & 1, k, y);
                uint32_t ra[RB], rb[RB], rc[RB];
                tmem_ld_cols_nowait<RB>(oc, ra);
                tmem_ld_cols_nowait<RB>(oc + RB, rb);
                tmem_ld_cols_nowait<RB>(oc + 2 * RB, rc);
                float a[RB], b[RB], c[RB];
                tmem_wait_cols<RB>(ra, a);
                tmem_wait_cols<RB>(rb, b);
                tmem_wait_cols<RB>(rc, c);
#pragma unroll
                for (int r = 0; r < RB; ++r)  // (a row that saw nothing: factor 0, finite O)
                    out[y][r] = fmaf(fmaf(fmaf(c[r], 0.125f, b[r]), 0.125f, a[r]),
                                     fac[32 * k + 16 * y + r], out[y][r]);
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.o_free[ord & 1]);
        if (fused && di.count == 1) {
            __nv_bfloat16 *base = static_cast<__nv_bfloat16 *>(p.out) +
                                  ((size_t)di.req * p.q_len * p.Hq + di.kv_head * p.G) * kHeadDim +
                                  tid;
#pragma unroll
            for (int y = 0; y < HEADS; ++y) {
                __nv_bfloat16 *dst = base + y * Gh * kHeadDim;
                int g = 0;
#pragma unroll
                for (int r = 0; r < RB; ++r) {
                    if (r < Rh) *dst = __float2bfloat16_rn(out[y][r]);
                    dst += kHeadDim;
                    if (++g == Gh) g = 0, dst += (size_t)(p.Hq - Gh) * kHeadDim;
                }
            }
        } else {
            float *base = p.part_o + (size_t)di.desc_idx * p.R * kHeadDim + tid;
#pragma unroll
            for (int y = 0; y < HEADS; ++y) {
                float *dst = base + y * Gh * kHeadDim;
                int g = 0;
#pragma unroll
                for (int r = 0; r < RB; ++r) {
                    if (r < Rh) *dst = out[y][r];
                    dst += kHeadDim;
                    if (++g == Gh) g = 0, dst += (p.G - Gh) * kHeadDim;
                }
            }
            if (tid < p.R) {
                const int i = tid / p.G, gg = tid - i * p.G, y = gg / Gh;
                p.part_lse[(size_t)di.desc_idx * p.R + tid] = fac[64 + 16 * y + i * Gh + gg - y * Gh];
            }
            if (fused) {  // count this chunk of a split unit
                named_bar_sync(bid, kTcGroup);  // the group's stores precede the release below
                if (q4 == 0) {
                    int completes = 0;
                    if (lane == 0) {
                        int *ctr = p.unit_done + di.kv_head * p.B + di.req;
                        if (atom_add_acq_rel_gpu(ctr, 1) == di.count - 1) {
                            *ctr = 0;  // every chunk counted: ready for the next launch
                            const int at = last[0].flags++;
                            if (at < kMaxLast) last[1 + at].di = di;
                            completes = at < kMaxLast ? 1 : 2;
                        }
                    }
                    completes = __shfl_sync(kFullMask, completes, 0);
                    if (completes == 2)  // list full: merge here, alone
                        for (int rho = 0; rho < p.R; ++rho) merge_unit_head<8>(p, di, rho);
                }
            }
        }
        named_bar_sync(bid, kTcGroup);  // fac may be written again
    }
}

// ------------------------------------------------------------------ kernel
template <int RB, int HEADS, bool BLK>
__device__ __forceinline__ void attn_tc_cta(const CUtensorMap &tmap_k, const CUtensorMap &tmap_v,
                                            const AttnParams &p) {
    using Tr = TcTraits<RB, HEADS, BLK>;
    constexpr int STAGES = Tr::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const TcBars bar = tc_bars<Tr>(smem);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + Tr::kOffMisc);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Tr::kOffMisc + 4);
    SlotInfo *last = reinterpret_cast<SlotInfo *>(smem + Tr::kOffLast);
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&bar.full[s], 1);   // producer arrive + bytes
            mbar_init(&bar.empty[s], 1);  // the second product's commit
        }
        for (int y = 0; y < 2; ++y) {
            mbar_init(&bar.s_full[y], 1);         // the first product's commit
            mbar_init(&bar.p_full[y], 4);         // the group's warps
            mbar_init(&bar.o_done[y], 1);
            mbar_init(&bar.o_free[y], 4);
        }
        for (int y = 0; y < kTcOrds; ++y) mbar_init(&bar.pub[y], kTcPubs);
        mbar_init(bar.end, 12);  // softmax and join warps
        mbar_init(bar.mma_done, 2);
        *abort = 0;
        last[0].flags = 0;
        fence_barrier_init();
        prefetch_tensormap(&tmap_k);
        prefetch_tensormap(&tmap_v);
    }
    if (warp == 0) {  // needs the barriers only, which it has set up itself
        __syncwarp();
        asm volatile("barrier.cta.arrive 4, %0;" ::"n"(kTcThreads) : "memory");
        grid_launch_dependents();
        tc_producer<RB, HEADS, BLK>(&tmap_k, &tmap_v, p, smem, abort);
        return;
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, Tr::kTmemCols);
        tmem_relinquish();
    }
    {  // caller inputs into L2 while the assign kernel may still be running
        const size_t bt_bytes = (size_t)p.B * p.max_pages * 4;
        const size_t q_bytes = (size_t)p.B * p.q_len * p.Hq * kHeadDim;
        const char *bt = reinterpret_cast<const char *>(p.block_table);
        const char *q = static_cast<const char *>(p.q);
        const size_t first = ((size_t)blockIdx.x * blockDim.x + threadIdx.x) * 128;
        const size_t step = (size_t)gridDim.x * blockDim.x * 128;
        for (size_t off = first; off < bt_bytes; off += step) prefetch_l2(bt + off);
        for (size_t off = first; off < q_bytes; off += step) prefetch_l2(q + off);
    }
    grid_launch_dependents();
    tc_fence_before();
    asm volatile("barrier.cta.sync 4, %0;" ::"n"(kTcThreads) : "memory");
    tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
    if (warp == 3) {  // fused mode: requests without live tokens get zero rows
        if (!p.out) return;
        grid_dependency_wait();
        const int row_vec = p.q_len * p.Hq * kHeadDim * 2 / 16;
        for (int r = blockIdx.x; r < p.B; r += gridDim.x) {
            if (p.seqlens[r] > 0) continue;
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) +
                                                   (size_t)r * p.q_len * p.Hq * kHeadDim);
            for (int i = lane; i < row_vec; i += 32) dst[i] = make_uint4(0, 0, 0, 0);
        }
        return;
    }
    const bool ok = warp == 1    ? tc_scores<RB, HEADS, BLK>(p, smem, tmem, abort)
                    : warp == 2  ? tc_products<RB, HEADS, BLK>(p, smem, tmem, abort)
                    : warp >= 12 ? tc_join<RB, HEADS, BLK>(p, smem, tmem, abort)
                                 : tc_softmax<RB, HEADS, BLK>(p, smem, tmem, (warp - 4) >> 2, abort);
    if (!ok) {
        grid_dependency_wait();  // meta[3] is written by the assign kernel
        if (lane == 0) atomicOr(p.meta + 3, (int)HPC_FLAG_TIMEOUT);
        *abort = 1;
    }
    if (warp == 1 || warp == 2) {
        // TMEM is freed once every MMA issued has completed and the other
        // groups have read their last columns (bounded, like every wait)
        if (elect_one()) umma_commit(bar.mma_done);
        __syncwarp();
        if (warp == 2) return;
        volatile int no_abort = 0;
        mbar_wait(bar.mma_done, 0, &no_abort);
        mbar_wait(bar.end, 0, &no_abort);
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, Tr::kTmemCols);
        return;
    }
    // End of the stream: all groups' warps merge the split units this CTA owes, two
    // rows of a unit per warp at a time, their loads in flight together (four took
    // 1 us longer in short launches: more of them sit in one warp, and their code is
    // fetched for a single run).
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar.end);
    if (!warp_wait(bar.end, 0, abort) || !p.out || *abort) return;
    grid_dependency_wait();
    const int nlast = min(last[0].flags, kMaxLast);
    const int w = warp - 4, items = nlast * p.R;
    for (int item = 2 * w; item < items; item += 2 * 12) {
        DescInfo dd[2];
        int rr[2];
        bool few = true;
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // (past the end: the last row again)
            const int e = min(item + k, items - 1);
            dd[k] = last[1 + e / p.R].di;
            rr[k] = e % p.R;
            few &= dd[k].count <= 32;
        }
        if (few) {
            merge_unit_rows<4, 2>(p, dd, rr);
        } else {
            for (int k = 0; k < 2 && item + k < items; ++k) merge_unit_head<8>(p, dd[k], rr[k]);
        }
    }
}

template <int RB, int HEADS, bool BLK>
__global__ void __launch_bounds__(kTcThreads, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap tmap_k,
                   const __grid_constant__ CUtensorMap tmap_v, const AttnParams p) {
    attn_tc_cta<RB, HEADS, BLK>(tmap_k, tmap_v, p);
}

template <int RB, int HEADS, bool BLK>
struct TcVariant {
    using Tr = TcTraits<RB, HEADS, BLK>;
    static AttnConfig config() {
        return {reinterpret_cast<const void *>(&attn_tc_kernel<RB, HEADS, BLK>), Tr::kSmemBytes,
                kTcThreads};
    }
    static cudaError_t launch(const CUtensorMap &tk, const CUtensorMap &tv, const AttnParams &p,
                              int grid, cudaStream_t s) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3(kTcThreads);
        cfg.dynamicSmemBytes = Tr::kSmemBytes;
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, attn_tc_kernel<RB, HEADS, BLK>, tk, tv, p);
    }
};

}  // namespace hpc
