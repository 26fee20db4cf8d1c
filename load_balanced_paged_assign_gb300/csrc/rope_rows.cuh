// Head-row arithmetic shared by the prologues (rope_norm.cu, block_cache.cu):
// how a half-warp holds a row, the rotation, the RMS and the E4M3 conversion.
#pragma once

#include "internal.h"
#include "ptx.cuh"

namespace hpc {
namespace {

constexpr int kRowBytes = kHeadDim * 2;  // one BF16 head row
constexpr int kMaxPosition = 1 << 24;    // positions are exact in fp32 below this

// ------------------------------------------------------------ lane layout
// A head row is handled by one half-warp (16 lanes, 8 dims each), so a warp
// instruction covers two rows and a row reduction takes four shuffles.
// Sub-lane s = lane & 15 holds, and pairs under the rotation:
//   halves:      dims 4s..4s+3 and 64+4s..67+4s; pairs (x[k], x[4+k])
//   interleaved: dims 8s..8s+7;                  pairs (x[2k], x[2k+1])
// In both layouts pair k of sub-lane s has frequency 4s + k.

__device__ __forceinline__ void unpack2(uint32_t w, float &lo, float &hi) {
    lo = bf16lo_to_f32(w);
    hi = bf16hi_to_f32(w);
}

template <int LAYOUT>
__device__ __forceinline__ uint4 load_words(const char *row, int s) {
    if (LAYOUT == HPC_ROPE_HALVES) {
        const uint2 lo = *reinterpret_cast<const uint2 *>(row + 8 * s);
        const uint2 hi = *reinterpret_cast<const uint2 *>(row + 128 + 8 * s);
        return make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
    return *reinterpret_cast<const uint4 *>(row + 16 * s);
}

template <int LAYOUT>
__device__ __forceinline__ void store_words(char *row, int s, uint4 v) {
    if (LAYOUT == HPC_ROPE_HALVES) {
        *reinterpret_cast<uint2 *>(row + 8 * s) = make_uint2(v.x, v.y);
        *reinterpret_cast<uint2 *>(row + 128 + 8 * s) = make_uint2(v.z, v.w);
    } else {
        *reinterpret_cast<uint4 *>(row + 16 * s) = v;
    }
}

__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
    unpack2(v.x, x[0], x[1]);
    unpack2(v.y, x[2], x[3]);
    unpack2(v.z, x[4], x[5]);
    unpack2(v.w, x[6], x[7]);
}

// E4M3 (round to nearest even, saturating) of four values, y[0] in the low byte.
__device__ __forceinline__ uint32_t e4m3x4(float y0, float y1, float y2, float y3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y1), "f"(y0));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y3), "f"(y2));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

template <int LAYOUT>
__device__ __forceinline__ void store_e4m3(char *row, int s, const float (&y)[8]) {
    const uint32_t a = e4m3x4(y[0], y[1], y[2], y[3]), b = e4m3x4(y[4], y[5], y[6], y[7]);
    if (LAYOUT == HPC_ROPE_HALVES) {
        *reinterpret_cast<uint32_t *>(row + 4 * s) = a;
        *reinterpret_cast<uint32_t *>(row + 64 + 4 * s) = b;
    } else {
        *reinterpret_cast<uint2 *>(row + 8 * s) = make_uint2(a, b);
    }
}

template <int LAYOUT>
__device__ __forceinline__ void store_bf16(char *row, int s, const float (&y)[8]) {
    store_words<LAYOUT>(row, s,
                        make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                   pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7])));
}

// The rotation of this sub-lane's four pairs: c, sn = cos, sin of its four
// frequencies, nsn = -sin.  In the halves layout pairs k and k + 1 sit in
// consecutive registers, so two pairs take one paired FP32 instruction
// (each lane of which rounds like the scalar one).
template <int LAYOUT>
__device__ __forceinline__ void rotate(float (&x)[8], const float (&c)[4], const float (&sn)[4],
                                       const float (&nsn)[4]) {
    if constexpr (LAYOUT == HPC_ROPE_HALVES) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float2 p = make_float2(x[2 * h], x[2 * h + 1]);
            const float2 q = make_float2(x[4 + 2 * h], x[5 + 2 * h]);
            const float2 cc = make_float2(c[2 * h], c[2 * h + 1]);
            const float2 p2 = __ffma2_rn(p, cc, __fmul2_rn(q, make_float2(nsn[2 * h], nsn[2 * h + 1])));
            const float2 q2 = __ffma2_rn(q, cc, __fmul2_rn(p, make_float2(sn[2 * h], sn[2 * h + 1])));
            x[2 * h] = p2.x, x[2 * h + 1] = p2.y;
            x[4 + 2 * h] = q2.x, x[5 + 2 * h] = q2.y;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float p = x[2 * k], q = x[2 * k + 1];
            x[2 * k] = fmaf(p, c[k], q * nsn[k]);
            x[2 * k + 1] = fmaf(q, c[k], p * sn[k]);
        }
    }
}

// x[k] *= m[k] for the 8 values, two per instruction.
__device__ __forceinline__ void mul8(float (&x)[8], const float (&m)[8]) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const float2 v = __fmul2_rn(make_float2(x[2 * h], x[2 * h + 1]),
                                    make_float2(m[2 * h], m[2 * h + 1]));
        x[2 * h] = v.x, x[2 * h + 1] = v.y;
    }
}

// x[k] *= m for the 8 values, two per instruction.
__device__ __forceinline__ void scale8(float (&x)[8], float m) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const float2 v = __fmul2_rn(make_float2(x[2 * h], x[2 * h + 1]), make_float2(m, m));
        x[2 * h] = v.x, x[2 * h + 1] = v.y;
    }
}

// Sum of squares of the 8 values (two partial sums, paired).
__device__ __forceinline__ float sumsq8(const float (&x)[8]) {
    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const float2 v = make_float2(x[2 * h], x[2 * h + 1]);
        acc = __ffma2_rn(v, v, acc);
    }
    return acc.x + acc.y;
}

// max(a, b, c) in one instruction.
__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ float absmax8(const float (&x)[8]) {
    return fmax3(fmax3(fabsf(x[0]), fabsf(x[1]), fabsf(x[2])),
                 fmax3(fabsf(x[3]), fabsf(x[4]), fabsf(x[5])), fmaxf(fabsf(x[6]), fabsf(x[7])));
}

// (cos, sin) of frequency i into a buffer of the angle table.
__device__ __forceinline__ void store_angle(float *tab, int i, float2 cs) {
    tab[(i >> 2) * 8 + (i & 3)] = cs.x;
    tab[(i >> 2) * 8 + 4 + (i & 3)] = cs.y;
}

}  // namespace
}  // namespace hpc
