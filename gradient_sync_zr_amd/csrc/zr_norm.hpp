// What the forward and the backward pass of the layer norm share: the lanes'
// share of a row, and sums over a row.
//
// A row is held in registers by TPR lanes, NV vectors of 8 columns each, so
// that every input byte is read once. A block has B = max(TPR, 256) threads
// and B / TPR rows at a time.
#pragma once

#include "zr_ckpt.hpp"
#include "zr_internal.hpp"

namespace zr {

__device__ __forceinline__ int existing(int64_t cols, int64_t c) {
    const int64_t left = cols - c;
    return left >= 8 ? 8 : (left > 0 ? (int)left : 0);
}

// Threads of a block whose rows have TPR lanes.
constexpr int norm_block(int tpr) { return tpr > kThreads ? tpr : kThreads; }

// Which of the block's rows a thread has: the same for a whole wave where a row
// takes one or more, and then kept in scalar registers, as are the addresses
// that follow from it.
template <int TPR, int B = norm_block(TPR)>
__device__ __forceinline__ int row_group() {
    if constexpr (B == TPR) return 0;
    const int g = threadIdx.x / TPR;
    return TPR >= 64 ? __builtin_amdgcn_readfirstlane(g) : g;
}

// Sums of N values each over the TPR lanes of a row. red: N floats per wave of
// the block, free again once every wave has passed a later barrier.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*red)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum<(TPR < 64 ? TPR : 64)>(v[i]);
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64;
        const int wave = threadIdx.x / 64, first = wave / W * W;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) red[wave][i] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += red[first + w][i];
    }
}

}  // namespace zr
