// The block-scaled 8-bit KV cache: the prologue that writes it (QK-Norm, RoPE,
// quantisation of K and V by blocks of 16 tokens and head, the query) and the
// read-back to BF16 pages.
//
// Quantisation.  The scale of a block is the smallest power of two s with
// max |y| <= 448 s, so y / s is exact and the only rounding is E4M3's (half a
// step, 2^-4 of the value).  E4M3 being a floating-point type, a power of two
// costs no precision against max / 448 but at the bottom of the range (codes
// below 2^-6 are subnormal), and a block that grows over several calls is
// re-scaled exactly.
//
// Both stream a token's data through once (its fused QKV row in, queries and
// codes out; codes in, BF16 rows out); the comments at the kernels say how the
// work is cut and what they reach.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "internal.h"
#include "ptx.cuh"
#include "rope_rows.cuh"

namespace hpc {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kMaxE4m3 = 448.f;

// The smallest power of two s >= 2^-126 with a <= 448 s, for a >= 0 finite:
// a = f 2^e with 1 <= f < 2, and 448 = 1.75 * 2^8.
__device__ __forceinline__ float pow2_scale(float a) {
    const uint32_t b = __float_as_uint(a);
    const int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);  // biased
    return __uint_as_float((uint32_t)max(e, 1) << 23);
}

__device__ __forceinline__ float block_scale_or_zero(float s) {
    return s > 0.f && s <= 3.402823466e38f ? s : 0.f;
}

// ------------------------------------------------------------------ write
constexpr int kBwWarps = 8;
constexpr int kBwThreads = 32 * kBwWarps;
constexpr int kBwMaxChunk = 8;  // tokens a CTA owns at most
constexpr int kBwTokens = kBwMaxChunk + kScaleBlock - 1;  // and those its last run may add
static_assert(kBwMaxChunk + kScaleBlock + 1 <= 32, "a warp scans a CTA's tokens and one more run");

struct BlockWriteArgs {
    const uint16_t *qkv;
    int64_t stride;  // elements between token rows
    const uint16_t *q_w;
    const uint16_t *k_w;
    const int32_t *positions;
    const int32_t *token_req;
    const int32_t *block_table;
    const double *freq;  // [64] or nullptr: built per CTA from base
    uint8_t *k_cache;
    uint8_t *v_cache;
    float *kv_scale;
    void *q_out;
    float *q_scale_out;
    int32_t *flags;
    double base;
    float eps;
    int N, Hq, Hkv, B, max_pages, num_pages, chunk;
};

struct RunInfo {
    int first, len;  // the run's first token (index in the CTA's table) and its tokens
};

struct BlockWriteShared {
    float ang[kBwTokens * 128];  // per token and group of 4 frequencies: 4 cosines, 4 sines
    float fhi[64], flo[64];  // the frequencies over pi, in two floats
    long long slot[32];  // page * 64 + offset, or -1
    int pos[32];
    RunInfo run[kBwMaxChunk];
    int runs, tokens;  // runs that start here; tokens whose angles are needed
};

// x^(-1/2) and 448 / m to about a rounding: a step of Newton's method from the
// approximations (2 ulp), for a value that a whole row of codes follows.  (Zero
// and infinity, of rows with infinities, stay as they are.)  The quotient is taken
// of maxima between kQueryLow and kQueryHigh.
__device__ __forceinline__ float root_inverse(float x) {
    const float y = rsqrtf(x);
    const float r = fmaf(0.5f * y, fmaf(-x * y, y, 1.f), y);
    return y > 0.f && y <= 3.402823466e38f ? r : y;
}
constexpr float kQueryLow = 7.888609052210118e-31f;  // 2^-100
constexpr float kQueryHigh = 1.2676506002282294e30f;  // 2^100
__device__ __forceinline__ float quotient448(float m) {
    const float y = __fdividef(kMaxE4m3, m);
    const float r = fmaf(fmaf(-y, m, kMaxE4m3), y * (1.f / kMaxE4m3), y);
    return y > 0.f && y <= 3.402823466e38f ? r : y;
}

// cos and sin of pi pos (hi + lo), to about their own rounding (a code near a
// tie between two E4M3 values follows the angle's error).  The product's integer
// part goes exactly, its rounding error and the low part are added with what
// that addition loses, d, which the functions' first derivatives bring in.
__device__ __forceinline__ float2 half_turns(int pos, float hi, float lo) {
    const float p = (float)pos;  // exact: 0 <= pos < 2^24 for valid tokens
    const float prod = p * hi;
    const float e = fmaf(p, lo, fmaf(p, hi, -prod));
    const float r = prod - 2.f * rintf(0.5f * prod);  // exact, in [-1, 1]
    const float t = r + e, b = t - r;
    const float d = 3.14159265f * ((r - (t - b)) + (e - b));
    float s, c;
    sincospif(t, &s, &c);
    return make_float2(fmaf(-d, s, c), fmaf(d, c, s));
}

__device__ __forceinline__ void load_angles(const float *tab, int s, float (&c)[4], float (&sn)[4],
                                            float (&nsn)[4]) {
    const float4 *a4 = reinterpret_cast<const float4 *>(tab + 8 * s);
    const float4 c4 = a4[0], s4 = a4[1];
    c[0] = c4.x, c[1] = c4.y, c[2] = c4.z, c[3] = c4.w;
    sn[0] = s4.x, sn[1] = s4.y, sn[2] = s4.z, sn[3] = s4.w;
#pragma unroll
    for (int k = 0; k < 4; ++k) nsn[k] = -sn[k];
}

// y = the norm and the rotation (NF: in this order) of a row, in place.
template <int LAYOUT, bool NF>
__device__ __forceinline__ void norm_rope(float (&x)[8], const float (&w)[8], const float (&c)[4],
                                          const float (&sn)[4], const float (&nsn)[4], float eps) {
    float ss = sumsq8(x);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(kAll, ss, o);
    const float inv = root_inverse(fmaf(ss, 1.0f / kHeadDim, eps));
    if constexpr (NF) {
        mul8(x, w);
        rotate<LAYOUT>(x, c, sn, nsn);
    } else {
        rotate<LAYOUT>(x, c, sn, nsn);
        mul8(x, w);
    }
    scale8(x, inv);
}

// Largest finite magnitude of the 8 values.
__device__ __forceinline__ float absmax8_finite(const float (&x)[8]) {
    float a = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float v = fabsf(x[k]);
        if (v <= 3.402823466e38f) a = fmaxf(a, v);
    }
    return a;
}

// x / s for the 8 values: exact for a power of two, else the IEEE quotient
// (both keep an infinity, which the conversion then saturates).
__device__ __forceinline__ void quotient8(float (&x)[8], float s) {
    const uint32_t b = __float_as_uint(s);
    const int e = (int)(b >> 23);
    if ((b & 0x7fffffu) == 0 && e >= 1 && e <= 252) {
        scale8(x, __uint_as_float((uint32_t)(254 - e) << 23));
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = __fdiv_rn(x[k], s);
    }
}

// One run's rows of one KV head, K or V: half-warp `half` holds rows 2 i +
// half of the run, all of them in registers as the BF16 words they came in, so
// each row is read once; K's norm and rotation are computed for the block's
// maximum and again for the codes (a tenth of a prompt's rows; the fp32 values
// would take twice the registers and cost a resident CTA).
template <int LAYOUT, bool NF, bool KEY>
__device__ __forceinline__ void write_run(const BlockWriteArgs &a, const BlockWriteShared &sh,
                                          int t0, const RunInfo run, int head, int lane) {
    constexpr int kRowPairs = kScaleBlock / 2;
    constexpr int kHeld = KEY ? LAYOUT : HPC_ROPE_INTERLEAVED;  // V rows: 8 dims in a row
    const int half = lane >> 4, s = lane & 15;
    const char *src = reinterpret_cast<const char *>(
        a.qkv + (size_t)(t0 + run.first) * a.stride +
        (size_t)(a.Hq + (KEY ? 0 : a.Hkv) + head) * kHeadDim);
    uint4 v[kRowPairs];
#pragma unroll
    for (int i = 0; i < kRowPairs; ++i) {
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (2 * i < run.len && 2 * i + half < run.len)
            v[i] = load_words<kHeld>(src + (size_t)(2 * i + half) * a.stride * 2, s);
    }
    // where the block is, which of its slots the run writes
    const long long slot0 = sh.slot[run.first];
    const long long page = slot0 / kTile;
    const int blk = (int)(slot0 % kTile) / kScaleBlock;
    float *scale = a.kv_scale + (page * a.Hkv + head) * kPageScales +
                   (KEY ? 0 : kPageScales / 2) + blk;
    const float was = *scale;
    const int my_off = lane < run.len ? (int)(sh.slot[run.first + lane] % kScaleBlock) : 0;
    const unsigned written = __reduce_or_sync(kAll, lane < run.len ? 1u << my_off : 0u);
    const bool fresh = written & 1u;
    const bool twice = __popc(written) < run.len;  // a position comes twice: the later one stays

    float w[8];
    if constexpr (KEY) unpack8(load_words<LAYOUT>(reinterpret_cast<const char *>(a.k_w), s), w);
    auto row = [&](int i, float (&x)[8]) {
        unpack8(v[i], x);
        if constexpr (KEY) {
            float c[4], sn[4], nsn[4];
            load_angles(sh.ang + min(run.first + 2 * i + half, kBwTokens - 1) * 128, s, c, sn, nsn);
            norm_rope<LAYOUT, NF>(x, w, c, sn, nsn, a.eps);
        }
    };
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < kRowPairs; ++i) {
        if (2 * i >= run.len) continue;
        float x[8];
        row(i, x);
        if (2 * i + half < run.len) amax = fmaxf(amax, absmax8_finite(x));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, o));
    const float fit = pow2_scale(amax);
    const float old = fresh ? 0.f : block_scale_or_zero(was);
    const float sc = fmaxf(old, fit);
    if (lane == 0 && sc != was) *scale = sc;

    uint8_t *base = (KEY ? a.k_cache : a.v_cache) +
                    ((size_t)(page * kTile + blk * kScaleBlock) * a.Hkv + head) * kHeadDim;
    const size_t step = (size_t)a.Hkv * kHeadDim;  // bytes between slots
    if (!fresh && sc != was) {  // the other slots' codes at the grown scale
        const float ratio = old / sc;
        for (int i = 0; i < kRowPairs; ++i) {
            const int slot = 2 * i + half;
            if (written >> slot & 1u) continue;
            uint2 *p = reinterpret_cast<uint2 *>(base + slot * step + 8 * s);
            const uint2 q = *p;
            uint32_t h[4];
            e4m3x4_to_f16x2x2(q.x, h[0], h[1]);
            e4m3x4_to_f16x2x2(q.y, h[2], h[3]);
            float y[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 f = f16x2_to_f32x2(h[k]);
                y[2 * k] = f.x * ratio;
                y[2 * k + 1] = f.y * ratio;
            }
            *p = make_uint2(e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7]));
        }
    }
#pragma unroll
    for (int i = 0; i < kRowPairs; ++i) {
        if (2 * i >= run.len) continue;
        const int j = 2 * i + half;
        bool store = j < run.len;
        const int off = (int)(sh.slot[run.first + min(j, run.len - 1)] % kScaleBlock);
        if (twice)
            for (int k = j + 1; k < run.len; ++k)
                store &= (int)(sh.slot[run.first + k] % kScaleBlock) != off;
        float x[8];
        row(i, x);
        quotient8(x, sc);
        if (store) store_e4m3<kHeld>(reinterpret_cast<char *>(base + off * step), s, x);
    }
}

// Query rows 8 b .. 8 b + 7 of a token (half-warp `half` holds 8 b + 2 i + half):
// their words, and from them the outputs.
template <int LAYOUT>
__device__ __forceinline__ void load_queries(const BlockWriteArgs &a, int t, int b, int lane,
                                             uint4 (&v)[4]) {
    const int half = lane >> 4, s = lane & 15;
    const char *src = reinterpret_cast<const char *>(a.qkv + (size_t)t * a.stride);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = load_words<LAYOUT>(src + (size_t)min(8 * b + 2 * i + half, a.Hq - 1) * kRowBytes, s);
}

template <int LAYOUT, bool NF, bool Q8>
__device__ __forceinline__ void write_queries(const BlockWriteArgs &a, const float *tab, int t,
                                              int b, int lane, const uint4 (&v)[4]) {
    const int half = lane >> 4, s = lane & 15;
    float c[4], sn[4], nsn[4], w[8];
    load_angles(tab, s, c, sn, nsn);
    unpack8(load_words<LAYOUT>(reinterpret_cast<const char *>(a.q_w), s), w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (8 * b + 2 * i >= a.Hq) continue;
        const int row = 8 * b + 2 * i + half;
        float x[8];
        unpack8(v[i], x);
        norm_rope<LAYOUT, NF>(x, w, c, sn, nsn, a.eps);
        const size_t out = (size_t)t * a.Hq + row;
        if constexpr (Q8) {
            float m = absmax8(x);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
            // codes = y * 448 / max|y|, the scale max|y| / 448 (1 for a zero row)
            const bool live = m > 0.f;
            float mid = m;
            if (live && !(m >= kQueryLow && m <= kQueryHigh)) {  // 448 / m may leave fp32's range
                const float lift = m < kQueryLow ? kQueryHigh : kQueryLow;  // exact, for the maximum too
                scale8(x, lift);
                mid = m * lift;
            }
            scale8(x, live ? quotient448(mid) : 0.f);
            if (row < a.Hq) {
                store_e4m3<LAYOUT>(static_cast<char *>(a.q_out) + out * kHeadDim, s, x);
                if (s == 0) a.q_scale_out[out] = live ? m * (1.0f / kMaxE4m3) : 1.f;
            }
        } else if (row < a.Hq) {
            store_bf16<LAYOUT>(static_cast<char *>(a.q_out) + out * kRowBytes, s, x);
        }
    }
}

// A CTA owns `chunk` consecutive tokens: their query rows, and the runs that
// start among them (a run may reach up to 15 tokens further; the CTA owning
// those writes only their queries).  One warp finds the runs: token t starts
// one if its (request, position / 16) is not its predecessor's.  Work items
// (a run's rows of one head, K or V; 8 query rows of a token) go round the
// eight warps.  Each row is read once, straight into registers (16 bytes a
// lane, 4 to 8 rows in flight per half-warp), the next query item's while this
// one's are worked on.  8192 tokens of 64 + 2 x 8 heads, BF16 queries (319 MB):
// 66 us, 71% of the measured copy rate (71 us without the look-ahead); chunks of
// 6 to 15 tokens are within 1%, four resident CTAs (64 registers) spill and two
// take 81 us, and prefetching the rows to L2 at the start costs 9 us more.  What
// bounds it is the latency of each item's chain of shuffles and conversions at 24
// warps per SM, the warps the registers allow.
constexpr int kBwCtas = 3;  // resident CTAs per SM the register budget must allow
template <int LAYOUT, bool NF, bool Q8>
__global__ void __launch_bounds__(kBwThreads, kBwCtas)
    rope_norm_block_kernel(const BlockWriteArgs a) {
    __shared__ __align__(16) BlockWriteShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dependency_wait();  // everything read may come from the kernel before
    const int t0 = blockIdx.x * a.chunk, own = min(a.chunk, a.N - t0);
    if (tid >= 64 && tid < 128) {
        const int i = tid - 64;
        const double f = a.freq ? a.freq[i] : pow(a.base, -(double)i / 64.0);
        const double g = f * 0.318309886183790671538;  // 1 / pi
        const float hi = (float)g;
        sh.fhi[i] = hi;
        sh.flo[i] = (float)(g - (double)hi);
    }
    if (warp == 0) {  // lane l: token t0 - 1 + l
        const int t = t0 - 1 + lane;
        const bool mine = lane >= 1 && lane <= own;
        long long key = -1, slot = -1;
        int pos = 0;
        if (t >= 0 && t < a.N) {
            pos = a.positions[t];
            const int req = a.token_req ? a.token_req[t] : t;
            unsigned bad = HPC_FLAG_BAD_SEQLEN;
            if (req >= 0 && req < a.B && pos >= 0 && pos < a.max_pages * kTile) {
                const int page = a.block_table[(size_t)req * a.max_pages + pos / kTile];
                bad = HPC_FLAG_BAD_PAGE;
                if (page >= 0 && page < a.num_pages) {
                    bad = 0;
                    slot = (long long)page * kTile + pos % kTile;
                    key = ((long long)req << 32) | (pos / kScaleBlock);
                }
            }
            if (bad && mine && a.flags) atomicOr(a.flags, (int)bad);
        }
        const long long before = __shfl_up_sync(kAll, key, 1);
        const bool same = lane >= 1 && key >= 0 && key == before;
        const unsigned follows = __ballot_sync(kAll, same);
        const bool starts = mine && key >= 0 && !same;
        const unsigned leaders = __ballot_sync(kAll, starts);
        int end = own;
        if (starts) {
            int len = __ffs(~(follows >> (lane + 1)));  // 1 + the tokens that follow in the run
            if (len > kScaleBlock) {  // more tokens than the block has slots
                if (a.flags) atomicOr(a.flags, (int)HPC_FLAG_BAD_SEQLEN);
                len = kScaleBlock;
            }
            sh.run[__popc(leaders & ((1u << lane) - 1u))] = RunInfo{lane - 1, len};
            end = max(end, lane - 1 + len);
        }
        end = __reduce_max_sync(kAll, end);
        if (lane >= 1) {
            sh.pos[lane - 1] = pos;
            sh.slot[lane - 1] = slot;
        }
        if (lane == 0) {
            sh.runs = __popc(leaders);
            sh.tokens = end;
        }
    }
    __syncthreads();
    for (int i = tid; i < sh.tokens * 64; i += kBwThreads) {
        const int f = i & 63, k = i >> 6;
        store_angle(sh.ang + k * 128, f, half_turns(sh.pos[k], sh.fhi[f], sh.flo[f]));
    }
    __syncthreads();
    const int per_run = 2 * a.Hkv, kv_items = sh.runs * per_run;
    const int per_token = (a.Hq + 7) / 8, items = kv_items + own * per_token;
    int it = warp;
    for (; it < kv_items; it += kBwWarps) {
        const int r = it / per_run, h = it - r * per_run;
        if (h < a.Hkv) write_run<LAYOUT, NF, true>(a, sh, t0, sh.run[r], h, lane);
        else write_run<LAYOUT, NF, false>(a, sh, t0, sh.run[r], h - a.Hkv, lane);
    }
    // (an item's rows are loaded while the last one's are worked on)
    uint4 v[4], next[4];
    int k = (it - kv_items) / per_token, b = it - kv_items - k * per_token;
    if (it < items) load_queries<LAYOUT>(a, t0 + k, b, lane, v);
    while (it < items) {
        it += kBwWarps;
        const int k1 = (it - kv_items) / per_token, b1 = it - kv_items - k1 * per_token;
        if (it < items) load_queries<LAYOUT>(a, t0 + k1, b1, lane, next);
        write_queries<LAYOUT, NF, Q8>(a, sh.ang + k * 128, t0 + k, b, lane, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = next[i];
        k = k1;
        b = b1;
    }
}

using WriteFn = void (*)(const BlockWriteArgs);

template <int LAYOUT>
WriteFn write_kernel(bool nf, bool q8) {
    if (nf) return q8 ? rope_norm_block_kernel<LAYOUT, true, true>
                      : rope_norm_block_kernel<LAYOUT, true, false>;
    return q8 ? rope_norm_block_kernel<LAYOUT, false, true>
              : rope_norm_block_kernel<LAYOUT, false, false>;
}

// ------------------------------------------------------------------ read back
constexpr int kRdThreads = 256;

struct BlockReadArgs {
    const uint8_t *k_cache;
    const uint8_t *v_cache;
    const float *kv_scale;
    const int32_t *block_table;
    const int32_t *starts;
    const int32_t *seqlens;
    const int32_t *out_table;
    uint8_t *k_out;
    uint8_t *v_out;
    int32_t *flags;
    int B, Hkv, max_pages, out_max_pages, num_pages, out_num_pages;
};

// The tokens of request r to read: [start, end), clamped to both tables.
__device__ __forceinline__ int2 read_range(const BlockReadArgs &a, int r, unsigned &bad) {
    const int cap = min(a.max_pages, a.out_max_pages) * kTile;
    int L = a.seqlens[r], st = a.starts ? a.starts[r] : 0;
    if (L < 0 || L > cap || st < 0) bad |= HPC_FLAG_BAD_SEQLEN;
    L = min(max(L, 0), cap);
    st = min(max(st, 0), L);
    return make_int2(st, L);
}

// 16 codes at scale f as 16 BF16 values, stored by one 32-byte instruction.
__device__ __forceinline__ void widen16(uint4 q, float f, uint4 *dst) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint32_t o[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t h0, h1;
        e4m3x4_to_f16x2x2(w[k], h0, h1);
        const float2 a = f16x2_to_f32x2(h0), b = f16x2_to_f32x2(h1);
        o[2 * k] = pack_bf16x2(a.x * f, a.y * f);
        o[2 * k + 1] = pack_bf16x2(b.x * f, b.y * f);
    }
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(o[0]),
                 "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                 : "memory");
}

// The requests' blocks of 16 tokens, numbered through, go round the persistent
// CTAs (each finds a block's request in a prefix sum over the requests, built
// once per CTA), so a batch of very different lengths, or one request alone,
// loads the SMs evenly.  A block's tokens are contiguous for all heads: a
// thread takes 16 codes (16 bytes in, 32 out) of K and the same of V at a
// time, two of each in flight.  8192 tokens of 8 heads (17 MB in, 34 MB out): 9 to
// 10 us, a launch and the loads' latency (long scoreboard 10 a warp instruction; DRAM
// at 19% of its peak, as the output still sits in L2 when it ends).
__global__ void __launch_bounds__(kRdThreads) kv_read_block_kernel(const BlockReadArgs a) {
    extern __shared__ int s_end[];  // [B] blocks of the requests up to and with r
    __shared__ int s_scan[kRdThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dependency_wait();
    unsigned bad = 0;
    int total = 0;
    for (int base = 0; base < a.B; base += kRdThreads) {
        const int r = base + tid;
        int n = 0;
        if (r < a.B) {
            const int2 x = read_range(a, r, bad);
            n = x.y > x.x ? (x.y - 1) / kScaleBlock - x.x / kScaleBlock + 1 : 0;
        }
        int v = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kAll, v, o);
            if (lane >= o) v += y;
        }
        if (lane == 31) s_scan[warp] = v;
        __syncthreads();
        int add = total, all = 0;
#pragma unroll
        for (int k = 0; k < kRdThreads / 32; ++k) {
            if (k < warp) add += s_scan[k];
            all += s_scan[k];
        }
        if (r < a.B) s_end[r] = add + v;
        total += all;
        __syncthreads();
    }
    if (bad && blockIdx.x == 0 && a.flags) atomicOr(a.flags, (int)bad);
    const int per_token = a.Hkv * (kHeadDim / 16);  // 16-code vectors
    for (int p = blockIdx.x; p < total; p += gridDim.x) {
        int lo = 0, hi = a.B - 1;  // the first request whose blocks end past p
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (s_end[mid] > p) hi = mid;
            else lo = mid + 1;
        }
        unsigned ignored = 0;
        const int2 x = read_range(a, lo, ignored);
        const int block = x.x / kScaleBlock + p - (lo ? s_end[lo - 1] : 0);
        const int tile = block / (kTile / kScaleBlock), sub = block % (kTile / kScaleBlock);
        const int src = a.block_table[(size_t)lo * a.max_pages + tile];
        const int dst = a.out_table[(size_t)lo * a.out_max_pages + tile];
        if (src < 0 || src >= a.num_pages || dst < 0 || dst >= a.out_num_pages) {
            if (tid == 0 && a.flags) atomicOr(a.flags, (int)HPC_FLAG_BAD_PAGE);
            continue;
        }
        const int first = block * kScaleBlock;  // the block's first token
        const int from = max(x.x - first, 0) * per_token;
        const int to = min(x.y - first, kScaleBlock) * per_token;
        const size_t in0 = ((size_t)src * kTile + sub * kScaleBlock) * per_token;
        const size_t out0 = ((size_t)dst * kTile + sub * kScaleBlock) * per_token;
        const float *sc = a.kv_scale + (size_t)src * a.Hkv * kPageScales + sub;
        const uint4 *kc = reinterpret_cast<const uint4 *>(a.k_cache) + in0;
        const uint4 *vc = reinterpret_cast<const uint4 *>(a.v_cache) + in0;
        uint4 *ko = reinterpret_cast<uint4 *>(a.k_out) + 2 * out0;
        uint4 *vo = reinterpret_cast<uint4 *>(a.v_out) + 2 * out0;
        for (int i = from + tid; i < to; i += 2 * kRdThreads) {
            const int j = i + kRdThreads;
            const bool two = j < to;
            const float *si = sc + (i / (kHeadDim / 16)) % a.Hkv * kPageScales;
            const float *sj = sc + (j / (kHeadDim / 16)) % a.Hkv * kPageScales;
            const uint4 k0 = kc[i], v0 = vc[i];
            const uint4 k1 = two ? kc[j] : k0, v1 = two ? vc[j] : v0;
            const float fk0 = si[0], fv0 = si[kPageScales / 2];
            const float fk1 = sj[0], fv1 = sj[kPageScales / 2];
            widen16(k0, fk0, ko + 2 * i);
            widen16(v0, fv0, vo + 2 * i);
            if (two) {
                widen16(k1, fk1, ko + 2 * j);
                widen16(v1, fv1, vo + 2 * j);
            }
        }
    }
}

bool aligned32(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

std::atomic<int> g_sms[64];  // per device, once asked for

// SMs of the current device, or -1.
int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return -1;
    sms = g_sms[dev].load();
    if (sms == 0) {
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return -1;
        g_sms[dev].store(sms);
    }
    return sms;
}

// A launch as a programmatic dependent of the previous kernel in the stream.
template <typename Fn, typename Args>
cudaError_t launch_dependent(Fn fn, int grid, int threads, int smem, cudaStream_t s,
                             const Args &args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, args);
}

}  // namespace
}  // namespace hpc

extern "C" hpc_status hpc_rope_norm_block(
    const void *d_qkv, int64_t qkv_row_stride, const void *d_q_norm_w, const void *d_k_norm_w,
    const int32_t *d_positions, const int32_t *d_token_req, int32_t num_tokens, int32_t Hq,
    int32_t Hkv, int32_t head_dim, const int32_t *d_block_table, int32_t max_pages_per_req,
    int32_t B, void *d_k_cache, void *d_v_cache, float *d_kv_scale, int32_t num_pages,
    void *d_q_out, float *d_q_scale_out, int32_t *d_flags, const hpc_rope_norm_params *params,
    hpc_stream_t stream) {
    using namespace hpc;
    if (!params || num_tokens < 0 || Hq <= 0 || Hkv <= 0 || B < 0 || max_pages_per_req <= 0 ||
        num_pages <= 0)
        return HPC_ERR_ARG;
    if (head_dim != HPC_HEAD_DIM || Hq % Hkv != 0 || Hq > (1 << 16)) return HPC_ERR_UNSUPPORTED;
    if (!std::isfinite(params->eps) || params->eps < 0.f || !std::isfinite(params->rope_base) ||
        params->rope_base <= 0.f)
        return HPC_ERR_ARG;
    if (params->rope_layout != HPC_ROPE_HALVES && params->rope_layout != HPC_ROPE_INTERLEAVED)
        return HPC_ERR_ARG;
    if (params->norm_first != 0 && params->norm_first != 1) return HPC_ERR_ARG;
    if (params->freq && !aligned16(params->freq)) return HPC_ERR_ARG;
    if ((int64_t)B * max_pages_per_req >= (int64_t)1 << 31) return HPC_ERR_UNSUPPORTED;
    // cache positions must stay exact in fp32 (the RoPE angle is formed there)
    if ((int64_t)max_pages_per_req * kTile > kMaxPosition) return HPC_ERR_UNSUPPORTED;
    if (num_tokens == 0) return HPC_OK;
    if (!d_qkv || !d_q_norm_w || !d_k_norm_w || !d_positions || !d_block_table || !d_k_cache ||
        !d_v_cache || !d_kv_scale || !d_q_out)
        return HPC_ERR_ARG;
    const int64_t heads = (int64_t)Hq + 2 * (int64_t)Hkv;
    if (qkv_row_stride < heads * HPC_HEAD_DIM || qkv_row_stride % 8 != 0) return HPC_ERR_ARG;
    if (!aligned16(d_qkv) || !aligned16(d_q_norm_w) || !aligned16(d_k_norm_w) ||
        !aligned16(d_k_cache) || !aligned16(d_v_cache) || !aligned16(d_kv_scale) ||
        !aligned16(d_q_out))
        return HPC_ERR_ARG;
    if (!d_token_req && num_tokens > B) return HPC_ERR_ARG;  // token t is request t

    BlockWriteArgs a;
    a.qkv = static_cast<const uint16_t *>(d_qkv);
    a.stride = qkv_row_stride;
    a.q_w = static_cast<const uint16_t *>(d_q_norm_w);
    a.k_w = static_cast<const uint16_t *>(d_k_norm_w);
    a.positions = d_positions;
    a.token_req = d_token_req;
    a.block_table = d_block_table;
    a.freq = params->freq;
    a.k_cache = static_cast<uint8_t *>(d_k_cache);
    a.v_cache = static_cast<uint8_t *>(d_v_cache);
    a.kv_scale = d_kv_scale;
    a.q_out = d_q_out;
    a.q_scale_out = d_q_scale_out;
    a.flags = d_flags;
    a.base = (double)params->rope_base;
    a.eps = params->eps;
    a.N = num_tokens;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.B = B;
    a.max_pages = max_pages_per_req;
    a.num_pages = num_pages;
    const int sms = sm_count();
    if (sms < 1) return HPC_ERR_CUDA;
    // few tokens: one a CTA, for the shortest chain; many: as many as still
    // give every SM four CTAs
    a.chunk = kBwMaxChunk;
    while (a.chunk > 1 && num_tokens < (int64_t)a.chunk * 4 * sms) a.chunk /= 2;
    const bool q8 = d_q_scale_out != nullptr;
    const WriteFn fn = params->rope_layout == HPC_ROPE_HALVES
                           ? write_kernel<HPC_ROPE_HALVES>(params->norm_first != 0, q8)
                           : write_kernel<HPC_ROPE_INTERLEAVED>(params->norm_first != 0, q8);
    const int grid = (num_tokens - 1) / a.chunk + 1;
    return launch_dependent(fn, grid, kBwThreads, 0, static_cast<cudaStream_t>(stream), a) ==
                   cudaSuccess
               ? HPC_OK
               : HPC_ERR_CUDA;
}

extern "C" hpc_status hpc_kv_read_block(const void *d_k_cache, const void *d_v_cache,
                                        const float *d_kv_scale, int32_t num_pages,
                                        const int32_t *d_block_table, int32_t max_pages_per_req,
                                        const int32_t *d_starts, const int32_t *d_seqlens,
                                        int32_t B, int32_t Hkv, int32_t head_dim, void *d_k_out,
                                        void *d_v_out, int32_t out_num_pages,
                                        const int32_t *d_out_block_table,
                                        int32_t out_max_pages_per_req, int32_t *d_flags,
                                        hpc_stream_t stream) {
    using namespace hpc;
    if (B < 0 || Hkv <= 0 || max_pages_per_req <= 0 || out_max_pages_per_req <= 0 ||
        num_pages <= 0 || out_num_pages <= 0)
        return HPC_ERR_ARG;
    if (head_dim != HPC_HEAD_DIM || B > HPC_MAX_BATCH || Hkv > (1 << 16))
        return HPC_ERR_UNSUPPORTED;
    const int64_t pages = std::min(max_pages_per_req, out_max_pages_per_req);
    if (pages * HPC_PAGE_SIZE >= (int64_t)1 << 30 || pages * B >= (int64_t)1 << 28)
        return HPC_ERR_UNSUPPORTED;
    if (B == 0) return HPC_OK;
    if (!d_k_cache || !d_v_cache || !d_kv_scale || !d_block_table || !d_seqlens || !d_k_out ||
        !d_v_out || !d_out_block_table)
        return HPC_ERR_ARG;
    if (!aligned16(d_k_cache) || !aligned16(d_v_cache) || !aligned16(d_kv_scale) ||
        !aligned32(d_k_out) || !aligned32(d_v_out))
        return HPC_ERR_ARG;
    BlockReadArgs a;
    a.k_cache = static_cast<const uint8_t *>(d_k_cache);
    a.v_cache = static_cast<const uint8_t *>(d_v_cache);
    a.kv_scale = d_kv_scale;
    a.block_table = d_block_table;
    a.starts = d_starts;
    a.seqlens = d_seqlens;
    a.out_table = d_out_block_table;
    a.k_out = static_cast<uint8_t *>(d_k_out);
    a.v_out = static_cast<uint8_t *>(d_v_out);
    a.flags = d_flags;
    a.B = B;
    a.Hkv = Hkv;
    a.max_pages = max_pages_per_req;
    a.out_max_pages = out_max_pages_per_req;
    a.num_pages = num_pages;
    a.out_num_pages = out_num_pages;
    const int smem = B * (int)sizeof(int);
    if (smem > 40 * 1024 &&
        cudaFuncSetAttribute(kv_read_block_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             HPC_MAX_BATCH * (int)sizeof(int)) != cudaSuccess)
        return HPC_ERR_CUDA;
    const int sms = sm_count();
    if (sms < 1) return HPC_ERR_CUDA;
    const int grid = (int)std::min<int64_t>(pages * (HPC_PAGE_SIZE / kScaleBlock) * B,
                                            (int64_t)sms * (smem > 24 * 1024 ? 2 : 8));
    return launch_dependent(kv_read_block_kernel, grid, kRdThreads, smem,
                            static_cast<cudaStream_t>(stream), a) == cudaSuccess
               ? HPC_OK
               : HPC_ERR_CUDA;
}
