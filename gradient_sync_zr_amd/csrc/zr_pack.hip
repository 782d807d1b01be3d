// Packing of 4-bit blocks (e2m1), their unpacking, and packing of a matrix's
// transpose in every format (the backward pass multiplies by a weight's transpose,
// whose blocks run along the other axis).
//
// Streams: 65536x4096 of bf16 to e2m1 takes 106 us (6.4 TB/s), back 116 (5.9);
// 16384x4096 28 and 32.
#include <hip/hip_runtime.h>

#include <type_traits>

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

// Codes and exponent of vector i of the rows laid end to end.
__device__ __forceinline__ void put_small(uint32_t* codes, uint8_t* scales, int64_t i, uint32_t q, uint32_t s) {
    st<true>(codes + i, q);
    if ((i & 3) == 0) scales[i / 4] = (uint8_t)s;
}

// Rows of whole blocks without gaps are one row, and a vector's place is its number.
// (With rows, columns and their division the instructions take longer than memory:
// 65536x4096 of bf16 136 us.)
template <int DT>
__global__ __launch_bounds__(kThreads) void pack_flat_kernel(const void* x, int64_t vectors, char* ckpt) {
    uint8_t* const scales = (uint8_t*)ckpt + vectors * 4;
    const int64_t tiles = (vectors + kTile - 1) / kTile;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t first = t * kTile;
        auto tile = [&](auto whole) {
            Raw8<DT> raw[kVecs];
#pragma unroll
            for (int k = 0; k < kVecs; ++k) {
                const int64_t i = first + threadIdx.x + k * kThreads;
                if (whole || i < vectors) raw[k] = fetch8<DT, true>({(const char*)x + i * (DT == kBf16 ? 16 : 32), nullptr}, 0, 8);
            }
#pragma unroll
            for (int k = 0; k < kVecs; ++k) {
                const int64_t i = first + threadIdx.x + k * kThreads;
                if (!whole && i >= vectors) continue;  // a block's lanes leave together
                settle8(raw[k], 0, 8);
                if constexpr (DT == kBf16) {
                    const uint32_t s = e2m1_byte(block_amax(raw[k].v));
                    put_small((uint32_t*)ckpt, scales, i, e2m1_encode8(raw[k].v, s), s);
                } else {
                    float f[8];
                    widen8(raw[k], f);
                    const uint32_t s = e2m1_byte(block_amax(f));
                    put_small((uint32_t*)ckpt, scales, i, e2m1_encode8(f, s), s);
                }
            }
        };
        if (vectors - first >= kTile)  // the same for the block
            tile(std::true_type{});
        else
            tile(std::false_type{});
    }
}

__global__ __launch_bounds__(kThreads) void unpack_flat_kernel(const char* ckpt, int64_t vectors, char* x, int dt) {
    const uint8_t* const scales = (const uint8_t*)ckpt + vectors * 4;
    const int64_t tiles = (vectors + kTile - 1) / kTile, es = dt == kBf16 ? 16 : 32;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t first = t * kTile;
        auto tile = [&](auto whole) {
            uint32_t q[kVecs], s[kVecs];
#pragma unroll
            for (int k = 0; k < kVecs; ++k) {
                const int64_t i = first + threadIdx.x + k * kThreads;
                if (!whole && i >= vectors) continue;
                q[k] = __builtin_nontemporal_load((const uint32_t*)ckpt + i);
                s[k] = scales[i / 4];
            }
#pragma unroll
            for (int k = 0; k < kVecs; ++k) {
                const int64_t i = first + threadIdx.x + k * kThreads;
                if (!whole && i >= vectors) continue;
                float f[8];
                e2m1_decode8(q[k], ckpt_scale(s[k]), f);
                store8<true>(x + i * es, dt, 0, 8, f);
            }
        };
        if (vectors - first >= kTile)
            tile(std::true_type{});
        else
            tile(std::false_type{});
    }
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
            put_small((uint32_t*)ckpt, (uint8_t*)ckpt + rows * (pitch / 2), first + threadIdx.x + k * kThreads,
                      e2m1_encode8(f, s), s);
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

// The transpose: a block takes 256 columns of x and TURNS blocks of 32 rows, a column
// to a lane. A lane holds a whole block, so its largest magnitude needs no other lane;
// loads are 64 neighbouring elements of a row, and a lane writes its blocks' codes at
// once, 64 bytes of a row of the result. (A block at a time the pieces met in the caches
// only while they held all rows' lines: 16384x16384 of bf16 378 us to e4m3, 224 so; with
// 128 bytes the registers leave two waves a SIMD, 249.) 11008x4096 of bf16
// takes 37 us to e4m3 and 34 to e2m1, 4096x4096 15 and 12.
template <int DT, int FMT, int TURNS>
__global__ __launch_bounds__(kThreads) void pack_t_kernel(const void* x, int64_t ld, int64_t rows, int64_t cols, char* ckpt,
                                                          int64_t tiles_c, int64_t tiles) {
    constexpr int WORDS = FMT == kE2m1 ? 1 : 2;           // of 16 bytes, of a block's codes
    const int64_t blocks = ckpt_pitch(rows) / kCkptBlock;  // of an output row
    const int64_t codes = code_bytes<FMT>(rows);
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t tr = t / tiles_c, c = (t - tr * tiles_c) * kThreads + threadIdx.x, first = tr * TURNS;
        if (c >= cols) continue;
        u32x4 q[TURNS][WORDS];
        uint32_t s[TURNS];
#pragma unroll
        for (int b = 0; b < TURNS; ++b) {
            const int64_t row = (first + b) * kCkptBlock;
            if (first + b >= blocks) break;
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
            s[b] = format_byte<FMT>(amax);
            if constexpr (FMT == kE2m1) {
                q[b][0] = u32x4{e2m1_encode8(f, s[b]), e2m1_encode8(f + 8, s[b]), e2m1_encode8(f + 16, s[b]),
                                e2m1_encode8(f + 24, s[b])};
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const u32x2 lo = ckpt_encode8(f + 16 * h, s[b], FMT == kE4m3), hi = ckpt_encode8(f + 16 * h + 8, s[b], FMT == kE4m3);
                    q[b][h] = u32x4{lo.x, lo.y, hi.x, hi.y};
                }
            }
        }
        u32x4* const out = (u32x4*)(ckpt + c * codes) + first * WORDS;
        uint8_t* const scales = (uint8_t*)ckpt + cols * codes + c * blocks + first;
#pragma unroll
        for (int b = 0; b < TURNS; ++b) {
            if (first + b >= blocks) break;
#pragma unroll
            for (int h = 0; h < WORDS; ++h) out[b * WORDS + h] = q[b][h];
            scales[b] = (uint8_t)s[b];
        }
    }
}

template <int DT, int FMT>
void pack_t_run(const void* x, int64_t ld, int64_t rows, int64_t cols, char* ckpt, hipStream_t stream) {
    const int64_t tiles_c = (cols + kThreads - 1) / kThreads, blocks = (rows + kCkptBlock - 1) / kCkptBlock;
    // 64 bytes of codes to a lane where that leaves enough for the chip
    constexpr int TURNS = FMT == kE2m1 ? 4 : 2;
    const bool many = tiles_c * blocks >= 4096;
    const int64_t tiles = tiles_c * (many ? (blocks + TURNS - 1) / TURNS : blocks);
    const dim3 grid(grid_for(tiles, kThreads)), block(kThreads);
    if (many)
        pack_t_kernel<DT, FMT, TURNS><<<grid, block, 0, stream>>>(x, ld, rows, cols, ckpt, tiles_c, tiles);
    else
        pack_t_kernel<DT, FMT, 1><<<grid, block, 0, stream>>>(x, ld, rows, cols, ckpt, tiles_c, tiles);
}

template <int DT>
void pack_t_pick(const void* x, int64_t ld, int64_t rows, int64_t cols, char* ckpt, zr_dtype fmt, hipStream_t stream) {
    if (fmt == ZR_CKPT_E2M1)
        pack_t_run<DT, kE2m1>(x, ld, rows, cols, ckpt, stream);
    else if (fmt == ZR_CKPT_E4M3)
        pack_t_run<DT, kE4m3>(x, ld, rows, cols, ckpt, stream);
    else
        pack_t_run<DT, kInt8>(x, ld, rows, cols, ckpt, stream);
}

int64_t tiles_of(int64_t rows, int64_t cols) { return (rows * (ckpt_pitch(cols) / 8) + kTile - 1) / kTile; }

bool flat(int64_t rows, int64_t cols, int64_t ld) { return cols % kCkptBlock == 0 && (ld == cols || rows == 1); }

}  // namespace

hipError_t launch_pack_small(const void* x, zr_dtype dt, int64_t rows, int64_t cols, int64_t ld, void* ckpt,
                             hipStream_t stream) {
    const int64_t tiles = tiles_of(rows, cols);
    const dim3 grid(grid_for(tiles, kThreads)), block(kThreads);
    if (flat(rows, cols, ld)) {
        if (dt == ZR_BF16)
            pack_flat_kernel<kBf16><<<grid, block, 0, stream>>>(x, rows * (cols / 8), (char*)ckpt);
        else
            pack_flat_kernel<kFp32><<<grid, block, 0, stream>>>(x, rows * (cols / 8), (char*)ckpt);
        return hipGetLastError();
    }
    if (dt == ZR_BF16)
        pack_small_kernel<kBf16><<<grid, block, 0, stream>>>(x, ld, rows, cols, (char*)ckpt, tiles);
    else
        pack_small_kernel<kFp32><<<grid, block, 0, stream>>>(x, ld, rows, cols, (char*)ckpt, tiles);
    return hipGetLastError();
}

hipError_t launch_unpack_small(const void* ckpt, int64_t rows, int64_t cols, void* x, zr_dtype dt, int64_t ld,
                               hipStream_t stream) {
    const int64_t tiles = tiles_of(rows, cols);
    if (flat(rows, cols, ld)) {
        unpack_flat_kernel<<<grid_for(tiles, kThreads), kThreads, 0, stream>>>((const char*)ckpt, rows * (cols / 8), (char*)x, dt);
        return hipGetLastError();
    }
    unpack_small_kernel<<<grid_for(tiles, kThreads), kThreads, 0, stream>>>((const char*)ckpt, rows, cols, (char*)x, ld, dt,
                                                                            tiles);
    return hipGetLastError();
}

hipError_t launch_pack_t(const void* x, zr_dtype dt, int64_t rows, int64_t cols, int64_t ld, void* ckpt, zr_dtype fmt,
                         hipStream_t stream) {
    if (dt == ZR_BF16)
        pack_t_pick<kBf16>(x, ld, rows, cols, (char*)ckpt, fmt, stream);
    else
        pack_t_pick<kFp32>(x, ld, rows, cols, (char*)ckpt, fmt, stream);
    return hipGetLastError();
}

}  // namespace zr
