// Packing of 4-bit blocks (e2m1), their unpacking, and packing of a matrix's
// transpose in every format (the backward pass multiplies by a weight's transpose,
// whose blocks run along the other axis).
//
// Streams: 65536x4096 of bf16 to e2m1 takes 131 to 136 us (5.0 to 5.2 TB/s), back
// 112 to 118; 16384x4096 35.
#include <hip/hip_runtime.h>

#include "zr_e2m1.hpp"
#include "zr_internal.hpp"

namespace zr {
namespace {

constexpr int kVecs = 4;  // vectors of 8 columns per lane and tile
constexpr int kTile = kThreads * kVecs;

// Row (from the tile's first) and column of vector i of a tile that starts at
// vector `rem` of its first row, V vectors per row.
__device__ __forceinline__ void place(uint32_t rem, uint32_t i, uint32_t V, uint32_t* drow, int* c) {
    const uint32_t at = rem + i;
    const uint32_t r = at / V;
    *drow = r;
    *c = (int)(at - r * V) * 8;
}

// As the 8-bit pack: lanes take vectors of 8 columns over the rows laid end to
// end, each padded to whole blocks, so that the 4 lanes of a block never part.
template <int DT>
__global__ __launch_bounds__(kThreads) void pack_small_kernel(const void* x, int64_t ld, int64_t rows, int64_t cols,
                                                              char* ckpt, int64_t tiles) {
    const int64_t pitch = ckpt_pitch(cols);
    const uint32_t V = (uint32_t)(pitch / 8);
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t first = t * kTile, row0 = first / V;
        const uint32_t rem = (uint32_t)(first - row0 * V);
        Raw8<DT> raw[kVecs];
        int n[kVecs], c[kVecs];
        int64_t row[kVecs];
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            uint32_t dr;
            place(rem, threadIdx.x + k * kThreads, V, &dr, &c[k]);
            row[k] = row0 + dr;
            const int64_t left = cols - c[k];
            n[k] = row[k] < rows ? (left >= 8 ? 8 : (left > 0 ? (int)left : 0)) : -1;
            if (n[k] >= 0) raw[k] = fetch8<DT, true>(row_at<DT>(x, ld, rows, cols, row[k]), c[k], n[k]);
        }
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            if (n[k] < 0) continue;
            float f[8];
            settle8(raw[k], c[k], n[k]);
            widen8(raw[k], f);
            uint32_t amax;
            if constexpr (DT == kBf16)
                amax = block_amax(raw[k].v);
            else
                amax = block_amax(f);
            const uint32_t s = e2m1_byte(amax);
            st<true>((uint32_t*)(ckpt + row[k] * (pitch / 2) + c[k] / 2), e2m1_encode8(f, s));
            if ((c[k] & (kCkptBlock - 1)) == 0)
                ((uint8_t*)ckpt)[rows * (pitch / 2) + row[k] * (pitch / kCkptBlock) + c[k] / kCkptBlock] = (uint8_t)s;
        }
    }
}

__global__ __launch_bounds__(kThreads) void unpack_small_kernel(const char* ckpt, int64_t rows, int64_t cols, char* x,
                                                                int64_t ld, int dt, int64_t tiles) {
    const int64_t pitch = ckpt_pitch(cols);
    const uint32_t V = (uint32_t)(pitch / 8);
    const int64_t es = dt == kBf16 ? 2 : 4;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t first = t * kTile, row0 = first / V;
        const uint32_t rem = (uint32_t)(first - row0 * V);
        uint32_t q[kVecs], s[kVecs];
        int n[kVecs], c[kVecs];
        int64_t row[kVecs];
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            uint32_t dr;
            place(rem, threadIdx.x + k * kThreads, V, &dr, &c[k]);
            row[k] = row0 + dr;
            const int64_t left = cols - c[k];
            n[k] = row[k] < rows ? (left >= 8 ? 8 : (left > 0 ? (int)left : 0)) : 0;
            q[k] = s[k] = 0;
            if (n[k] > 0) {
                q[k] = __builtin_nontemporal_load((const uint32_t*)(ckpt + row[k] * (pitch / 2) + c[k] / 2));
                s[k] = ((const uint8_t*)ckpt)[rows * (pitch / 2) + row[k] * (pitch / kCkptBlock) + c[k] / kCkptBlock];
            }
        }
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            if (n[k] == 0) continue;
            float f[8];
            e2m1_decode8(q[k], ckpt_scale(s[k]), f);
            store8<true>(x + row[k] * ld * es, dt, c[k], n[k], f);
        }
    }
}

// The transpose: a wave takes 64 columns of x and, in turn, `turns` blocks of 32
// rows, a column to a lane. A lane holds a whole block, so its largest magnitude
// needs no other lane; loads are 64 neighbouring elements of a row, and a lane
// writes its blocks side by side. 11008x4096 of bf16 takes 44 us to e4m3 and 36.5 to
// e2m1, 4096x4096 16 and 13: the codes of 64 rows of the result leave in pieces of
// 32 bytes (16 of e2m1) a block, which caches collect.
template <int DT, int FMT>
__global__ __launch_bounds__(kThreads) void pack_t_kernel(const void* x, int64_t ld, int64_t rows, int64_t cols, char* ckpt,
                                                          int turns, int64_t tiles_c, int64_t tiles) {
    const int64_t blocks = ckpt_pitch(rows) / kCkptBlock;  // of an output row
    const int64_t codes = code_bytes<FMT>(rows);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t tr = t / tiles_c, c = ((t - tr * tiles_c) * (kThreads / 64) + wave) * 64 + lane;
        if (c >= cols) continue;
#pragma unroll 1
        for (int b = 0; b < turns; ++b) {
            const int64_t block = tr * turns + b, row = block * kCkptBlock;
            if (block >= blocks) break;
            // rows behind the last are read from it, and are zeros
            float f[kCkptBlock];
            const int have = rows - row < kCkptBlock ? (int)(rows - row) : kCkptBlock;
#pragma unroll
            for (int k = 0; k < kCkptBlock; ++k) {
                const int64_t at = (row + (k < have ? k : have - 1)) * ld + c;
                if constexpr (DT == kBf16)
                    f[k] = load_elem((const uint16_t*)x + at);
                else
                    f[k] = load_elem((const float*)x + at);
            }
            if (have < kCkptBlock) {
#pragma unroll
                for (int k = 0; k < kCkptBlock; ++k) f[k] = k < have ? f[k] : 0.0f;
            }
            uint32_t amax = 0;
#pragma unroll
            for (int k = 0; k < kCkptBlock; ++k) {
                const uint32_t m = __float_as_uint(f[k]) & 0x7FFFFFFFu;
                amax = m > amax ? m : amax;
            }
            const uint32_t s = format_byte<FMT>(amax);
            u32x4* out = (u32x4*)(ckpt + c * codes + block * (FMT == kE2m1 ? 16 : 32));
            if constexpr (FMT == kE2m1) {
                *out = u32x4{e2m1_encode8(f, s), e2m1_encode8(f + 8, s), e2m1_encode8(f + 16, s), e2m1_encode8(f + 24, s)};
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const u32x2 lo = ckpt_encode8(f + 16 * h, s, FMT == kE4m3), hi = ckpt_encode8(f + 16 * h + 8, s, FMT == kE4m3);
                    out[h] = u32x4{lo.x, lo.y, hi.x, hi.y};
                }
            }
            ((uint8_t*)ckpt)[cols * codes + c * blocks + block] = (uint8_t)s;
        }
    }
}

template <int DT>
void pack_t_run(const void* x, int64_t ld, int64_t rows, int64_t cols, char* ckpt, zr_dtype fmt, hipStream_t stream) {
    const int64_t tiles_c = (cols + kThreads - 1) / kThreads, blocks = (rows + kCkptBlock - 1) / kCkptBlock;
    // four blocks to a lane (a line of codes) where that leaves enough for the chip
    const int turns = tiles_c * blocks >= 4096 ? 4 : 1;
    const int64_t tiles = tiles_c * ((blocks + turns - 1) / turns);
    const dim3 grid(grid_for(tiles, kThreads)), block(kThreads);
    if (fmt == ZR_CKPT_E2M1)
        pack_t_kernel<DT, kE2m1><<<grid, block, 0, stream>>>(x, ld, rows, cols, ckpt, turns, tiles_c, tiles);
    else if (fmt == ZR_CKPT_E4M3)
        pack_t_kernel<DT, kE4m3><<<grid, block, 0, stream>>>(x, ld, rows, cols, ckpt, turns, tiles_c, tiles);
    else
        pack_t_kernel<DT, kInt8><<<grid, block, 0, stream>>>(x, ld, rows, cols, ckpt, turns, tiles_c, tiles);
}

int64_t tiles_of(int64_t rows, int64_t cols) { return (rows * (ckpt_pitch(cols) / 8) + kTile - 1) / kTile; }

}  // namespace

hipError_t launch_pack_small(const void* x, zr_dtype dt, int64_t rows, int64_t cols, int64_t ld, void* ckpt,
                             hipStream_t stream) {
    const int64_t tiles = tiles_of(rows, cols);
    const dim3 grid(grid_for(tiles, kThreads)), block(kThreads);
    if (dt == ZR_BF16)
        pack_small_kernel<kBf16><<<grid, block, 0, stream>>>(x, ld, rows, cols, (char*)ckpt, tiles);
    else
        pack_small_kernel<kFp32><<<grid, block, 0, stream>>>(x, ld, rows, cols, (char*)ckpt, tiles);
    return hipGetLastError();
}

hipError_t launch_unpack_small(const void* ckpt, int64_t rows, int64_t cols, void* x, zr_dtype dt, int64_t ld,
                               hipStream_t stream) {
    const int64_t tiles = tiles_of(rows, cols);
    unpack_small_kernel<<<grid_for(tiles, kThreads), kThreads, 0, stream>>>((const char*)ckpt, rows, cols, (char*)x, ld, dt,
                                                                            tiles);
    return hipGetLastError();
}

hipError_t launch_pack_t(const void* x, zr_dtype dt, int64_t rows, int64_t cols, int64_t ld, void* ckpt, zr_dtype fmt,
                         hipStream_t stream) {
    if (dt == ZR_BF16)
        pack_t_run<kBf16>(x, ld, rows, cols, (char*)ckpt, fmt, stream);
    else
        pack_t_run<kFp32>(x, ld, rows, cols, (char*)ckpt, fmt, stream);
    return hipGetLastError();
}

}  // namespace zr
