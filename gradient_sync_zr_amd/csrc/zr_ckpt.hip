// Packing and unpacking of 8-bit activation checkpoints.
//
// Both are streams: bf16 is 2 bytes in and 33/32 out (or the reverse) per
// element, and the arithmetic of a block (its largest magnitude over 4 lanes,
// one multiply and conversion per element) hides behind it. A lane takes
// vectors of 8 columns, 256 lanes apart, kCkptVecs of them with all loads in
// front, over the rows laid end to end (each padded to whole blocks, so the 4
// lanes of a block never part). Bound by memory: 65536x4096 bf16 to e4m3 packs in
// 147 to 152 us (5.4 to 5.5 TB/s) and unpacks in 134 (6.1); with 8 vectors a lane 168 and 146,
// without the accesses past the caches 172 and 143.
#include <hip/hip_runtime.h>

#include "zr_ckpt.hpp"
#include "zr_internal.hpp"

namespace zr {
namespace {

constexpr int kCkptVecs = 4;  // vectors per lane and tile
constexpr int kCkptTile = kThreads * kCkptVecs;

// Row (from the tile's first) and column of vector i of a tile that starts at
// vector `rem` of its first row, V vectors per row.
__device__ __forceinline__ void place(uint32_t rem, uint32_t i, uint32_t V, uint32_t* drow, int* c) {
    const uint32_t at = rem + i;
    const uint32_t r = at / V;
    *drow = r;
    *c = (int)(at - r * V) * 8;
}

template <int DT>
__global__ __launch_bounds__(kThreads) void pack_kernel(const void* x, int64_t ld, int64_t rows, int64_t cols,
                                                        char* ckpt, int e4m3, int64_t tiles) {
    const int64_t pitch = ckpt_pitch(cols);
    const uint32_t V = (uint32_t)(pitch / 8);
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t first = t * kCkptTile, row0 = first / V;
        const uint32_t rem = (uint32_t)(first - row0 * V);
        Raw8<DT> raw[kCkptVecs];
        int n[kCkptVecs], c[kCkptVecs];
        int64_t row[kCkptVecs];
#pragma unroll
        for (int k = 0; k < kCkptVecs; ++k) {
            uint32_t dr;
            place(rem, threadIdx.x + k * kThreads, V, &dr, &c[k]);
            row[k] = row0 + dr;
            const int64_t left = cols - c[k];
            n[k] = row[k] < rows ? (left >= 8 ? 8 : (left > 0 ? (int)left : 0)) : -1;
            if (n[k] >= 0) raw[k] = fetch8<DT, true>(row_at<DT>(x, ld, rows, cols, row[k]), c[k], n[k]);
        }
#pragma unroll
        for (int k = 0; k < kCkptVecs; ++k) {
            if (n[k] < 0) continue;  // rows end with whole blocks, so a block's lanes leave together
            float f[8];
            settle8(raw[k], c[k], n[k]);
            widen8(raw[k], f);
            uint32_t amax;
            if constexpr (DT == kBf16)
                amax = block_amax(raw[k].v);
            else
                amax = block_amax(f);
            ckpt_store8(ckpt + row[k] * pitch, (uint8_t*)ckpt + rows * pitch + row[k] * (pitch / kCkptBlock), c[k], f,
                        amax, e4m3 != 0);
        }
    }
}

template <int FMT>
__global__ __launch_bounds__(kThreads) void unpack_kernel(const char* ckpt, int64_t rows, int64_t cols, char* x,
                                                          int64_t ld, int dt, int64_t tiles) {
    const int64_t pitch = ckpt_pitch(cols);
    const uint32_t V = (uint32_t)(pitch / 8);
    const int64_t es = dt == kBf16 ? 2 : 4;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t first = t * kCkptTile, row0 = first / V;
        const uint32_t rem = (uint32_t)(first - row0 * V);
        Raw8<FMT> raw[kCkptVecs];
        int n[kCkptVecs], c[kCkptVecs];
        int64_t row[kCkptVecs];
#pragma unroll
        for (int k = 0; k < kCkptVecs; ++k) {
            uint32_t dr;
            place(rem, threadIdx.x + k * kThreads, V, &dr, &c[k]);
            row[k] = row0 + dr;
            const int64_t left = cols - c[k];
            n[k] = row[k] < rows ? (left >= 8 ? 8 : (left > 0 ? (int)left : 0)) : 0;
            if (n[k] > 0) raw[k] = fetch8<FMT, true>(row_at<FMT>(ckpt, 0, rows, cols, row[k]), c[k], n[k]);
        }
#pragma unroll
        for (int k = 0; k < kCkptVecs; ++k) {
            if (n[k] == 0) continue;
            float f[8];
            widen8(raw[k], f);
            store8<true>(x + row[k] * ld * es, dt, c[k], n[k], f);
        }
    }
}

int64_t tiles_of(int64_t rows, int64_t cols) {
    return (rows * (ckpt_pitch(cols) / 8) + kCkptTile - 1) / kCkptTile;
}

}  // namespace

hipError_t launch_ckpt_pack(const void* x, zr_dtype dt, int64_t rows, int64_t cols, int64_t ld, zr_dtype fmt,
                            void* ckpt, hipStream_t stream) {
    const int64_t tiles = tiles_of(rows, cols);
    const dim3 grid(grid_for(tiles, kThreads)), block(kThreads);
    const int e4m3 = fmt == ZR_CKPT_E4M3;
    if (dt == ZR_BF16)
        pack_kernel<kBf16><<<grid, block, 0, stream>>>(x, ld, rows, cols, (char*)ckpt, e4m3, tiles);
    else
        pack_kernel<kFp32><<<grid, block, 0, stream>>>(x, ld, rows, cols, (char*)ckpt, e4m3, tiles);
    return hipGetLastError();
}

hipError_t launch_ckpt_unpack(const void* ckpt, zr_dtype fmt, int64_t rows, int64_t cols, void* x, zr_dtype dt,
                              int64_t ld, hipStream_t stream) {
    const int64_t tiles = tiles_of(rows, cols);
    const dim3 grid(grid_for(tiles, kThreads)), block(kThreads);
    if (fmt == ZR_CKPT_E4M3)
        unpack_kernel<kE4m3><<<grid, block, 0, stream>>>((const char*)ckpt, rows, cols, (char*)x, ld, dt, tiles);
    else
        unpack_kernel<kInt8><<<grid, block, 0, stream>>>((const char*)ckpt, rows, cols, (char*)x, ld, dt, tiles);
    return hipGetLastError();
}

}  // namespace zr
