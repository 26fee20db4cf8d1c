// Prefix sums over a block, used by the planners.
#pragma once

namespace hpc {

// Inclusive block-wide prefix sum over blockDim.x (a multiple of 32) values;
// also returns the block total.  Uses `scratch` (32 ints) and synchronises.
__device__ __forceinline__ int block_inclusive_scan(int v, int *scratch, int &total) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    if (lane == 31) scratch[wid] = v;
    __syncthreads();
    if (wid == 0) {
        int w = lane < nwarps ? scratch[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        scratch[lane] = w;
    }
    __syncthreads();
    if (wid > 0) v += scratch[wid - 1];
    total = scratch[nwarps - 1];
    __syncthreads();
    return v;
}

// The same of N values at once (in place; the totals in `total`); `scratch` holds 32 N.
template <int N>
__device__ __forceinline__ void block_inclusive_scans(int (&v)[N], int *scratch, int (&total)[N]) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int y = __shfl_up_sync(0xffffffffu, v[k], o);
            if (lane >= o) v[k] += y;
        }
    if (lane == 31)
#pragma unroll
        for (int k = 0; k < N; ++k) scratch[32 * k + wid] = v[k];
    __syncthreads();
    // every warp sums the warps' totals for itself
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int w = lane < nwarps ? scratch[32 * k + lane] : 0;
        v[k] += __reduce_add_sync(0xffffffffu, lane < wid ? w : 0);
        total[k] = __reduce_add_sync(0xffffffffu, w);
    }
    __syncthreads();
}

}  // namespace hpc
