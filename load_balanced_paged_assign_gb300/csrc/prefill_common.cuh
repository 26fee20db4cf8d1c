// What the causal (prefill.cu) and the windowed (prefill_win.cu) prompt
// attention share: the Q tiles' shape, small wrappers, the tensor map over the
// queries.
#pragma once

#include <cuda_bf16.h>

#include <cstring>

#include "internal.h"
#include "tcgen05.cuh"

namespace hpc {
namespace {

constexpr int kQB = 128;                 // query rows per Q tile (UMMA M)
constexpr int kQT = 2;                   // Q tiles per CTA
constexpr int kHalf = 128 * 128;         // 128 rows x 64 BF16: one 128-byte column block
constexpr int kTileBytes = 2 * kHalf;    // a 128 x 128 BF16 tile (Q, K or V)
constexpr int kSoftmaxWarps = 4 * kQT;
constexpr int kProducerWarp = kSoftmaxWarps, kMmaWarp = kSoftmaxWarps + 1;
constexpr uint32_t kTmemCols = 512;      // S_x / P_x from 128 x on; O_x at 256 + 128 x
constexpr int kOCol = 256;
constexpr float kRescaleLog2 = 8.f;      // P <= 2^8 between reference moves

__device__ __forceinline__ uint64_t policy_evict_normal() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// max(a, b, c) in one instruction.
__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                       uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Tensor map over Q [B * q_len, Hq, 128] BF16 as {64 dims, 2 halves, Hq,
// tokens}, box {64, 1, 1, 128}: one 64-dim half of 128 consecutive query
// tokens of one head, rows of 128 bytes (the swizzle span).
hpc_status make_q_map(CUtensorMap *m, const void *q, int64_t tokens, int32_t Hq) {
    auto encode = tensor_map_encoder();
    if (!encode) return HPC_ERR_CUDA;
    std::memset(m, 0, sizeof(*m));
    cuuint64_t dims[4] = {64, 2, (cuuint64_t)Hq, (cuuint64_t)tokens};
    cuuint64_t strides[3] = {128, 256, (cuuint64_t)Hq * 256};
    cuuint32_t box[4] = {64, 1, 1, kQB};
    cuuint32_t elem[4] = {1, 1, 1, 1};
    CUresult res = encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(q), dims,
                          strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return res == CUDA_SUCCESS ? HPC_OK : HPC_ERR_CUDA;
}

}  // namespace
}  // namespace hpc
