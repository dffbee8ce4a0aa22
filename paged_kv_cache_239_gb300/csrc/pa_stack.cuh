// pa_stack.cuh -- what the kernels that work on the device free stack share.
#pragma once

#include <cuda_runtime.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

// The stack's height, held to what the array can hold (flagged if it was not).
__device__ __forceinline__ int stack_height(const int* stack, long long num_blocks,
                                            unsigned* status) {
    const int h = ld_dep(stack);
    if (h >= 0 && h <= num_blocks) return h;
    if (threadIdx.x == 0) atomicOr(status, kStatusBadLength);
    return h < 0 ? 0 : (int)num_blocks;
}

// Exclusive prefix sum of `v` over the CTA; `total` receives the sum.
__device__ __forceinline__ int cta_exclusive_scan(int v, int* s_warp, int& total) {
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(kFullMask, incl, o);
        if (lane >= o) incl += t;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int w = lane < (blockDim.x >> 5) ? s_warp[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(kFullMask, w, o);
            if (lane >= o) w += t;
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    const int before = warp > 0 ? s_warp[warp - 1] : 0;
    total = s_warp[(blockDim.x >> 5) - 1];
    __syncthreads();
    return before + incl - v;
}

}  // namespace pa
