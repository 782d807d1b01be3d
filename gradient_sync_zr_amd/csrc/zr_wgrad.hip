// Weight and bias gradient of a linear layer whose input was kept as an 8-bit
// checkpoint:
//     dW[o, i] = sum over rows t of dY[t, o] * X[t, i],   db[o] = sum dY[t, o]
//
// A matrix product whose two operands both have the summed index outermost. A
// block computes a BM x BN tile of dW from slabs of BK rows: dY's slab goes to
// LDS as it is, the checkpoint's is decoded to bf16 on the way (every held
// value is exact in bf16), and both are read back transposed, 4 rows of one
// column per lane and instruction (ds_read_b64_tr_b16), as the operands of
// v_mfma_f32_32x32x16_bf16. Sums are fp32. fp32 dY is cut into three bf16
// terms that add up to it exactly (8 mantissa bits each), so its product with
// the checkpoint keeps fp32 accuracy on the bf16 matrix units.
//
// LDS rows are a multiple of 256 bytes, so the four rows that one transposed
// read touches would lie in the same banks; each row's 64-byte windows are
// exchanged by the row's number modulo 4, which spreads the read over all 64.
//
// Two slabs in LDS alternate: the next slab's loads are issued before the
// current one is multiplied and land in registers meanwhile.
//
// When dW has fewer tiles than the chip has places for blocks, the rows are
// split too; the parts go to the workspace in fp32 and a second kernel joins
// them in order, so results do not change from run to run.
//
// The small form (tiles of 128 x 128, four waves of 64 x 64) reads 64 KB from
// LDS and writes 32 for a slab of 64 rows, 768 cycles at 128 bytes each, and
// multiplies for 515; two blocks a CU hide each other's barriers:
// 16384x11008x4096 in 2,168 us, 681 TFLOP/s. With fp32 dY it does three times the
// products: 16384x4096x4096 in 1,600 to 1,640 us, 1,005 to 1,030 TFLOP/s of the
// matrix units. Loads two slabs ahead (which leave room for one block a CU) and
// operands read two steps ahead, as in the large form, both measured slower here
// (21232x176x1312: 69 and 43 us, not 41).
#include <hip/hip_runtime.h>

#include "zr_ckpt.hpp"
#include "zr_internal.hpp"

namespace zr {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

struct WgradArgs {
    const void* dy;
    const char* codes;
    const uint8_t* scales;
    float* part;  // splits > 1: [splits][out * in + out]
    void *dw, *db;
    int64_t rows, out, in, ld_dy, ld_dw, pitch, span;
    int grad_dt, accumulate, tiles_m, tiles_n, splits;
    int64_t slabs, full, rest, parts, share;  // the large form's (WgradShare)
};

// 16 codes of one block as 16 bf16 values (8 words).
template <int FMT>
__device__ __forceinline__ void decode16(const u32x4& q, uint32_t s, uint32_t w[8]) {
    const float scale = ckpt_scale(s);
    const uint32_t c[4] = {q.x, q.y, q.z, q.w};
    if constexpr (FMT == kE4m3) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            w[2 * k] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[k], scale, false));
            w[2 * k + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[k], scale, true));
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t h = c[k >> 1] >> (16 * (k & 1));
            const float a = (float)(int)(int8_t)h * scale, b = (float)(int)(int8_t)(h >> 8) * scale;
            // exact in bf16: the upper halves are the values
            w[k] = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
        }
    }
}

// Three bf16 terms (upper halves of a word each) that add up to v: each takes
// the next 8 mantissa bits. (Bits of v below 2^-133, which bf16 does not reach,
// are dropped: |v| < 2^-110 only.) An infinity has one term.
__device__ __forceinline__ void split3(float v, uint32_t t[3]) {
    const uint32_t u = __float_as_uint(v);
    t[0] = u & 0xFFFF0000u;
    const bool inf = (u & 0x7FFFFFFFu) == 0x7F800000u;
    const float r = inf ? 0.0f : v - __uint_as_float(t[0]);
    t[1] = __float_as_uint(r) & 0xFFFF0000u;
    const float r2 = r - __uint_as_float(t[1]);
    t[2] = __float_as_uint(r2) & 0xFFFF0000u;
}

// The same value in every lane, kept in scalar registers (a division's result
// comes in vector ones).
__device__ __forceinline__ int uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane((int)v); }

// Blocks are dealt to the 8 XCDs in turn: neighbours among `total` items for
// the blocks of one XCD, so that their slabs meet in that XCD's L2.
__device__ __forceinline__ uint32_t by_xcd(uint32_t item, uint32_t total) {
    const uint32_t x = item % 8, i = item / 8, q = total / 8, r = total % 8;
    return (x < r ? x * (q + 1) : r * (q + 1) + (x - r) * q) + i;
}

// Row and column of tile t, in groups of 8 rows of tiles.
__device__ __forceinline__ void tile_place(const WgradArgs& a, uint32_t t, int* tm, int* tn) {
    constexpr uint32_t GM = 8;
    const uint32_t per = GM * (uint32_t)a.tiles_n;
    const uint32_t group = t / per, in_group = t - group * per, first = group * GM;
    const uint32_t gm = (uint32_t)a.tiles_m - first < GM ? (uint32_t)a.tiles_m - first : GM;
    const uint32_t n = in_group / gm;
    *tm = uniform(first + in_group - n * gm);
    *tn = uniform(n);
}

// A wave's accumulators to dW or the workspace; `at` is this lane's first
// element, of which `rows` rows and `cols` columns from it exist (ALL: all of
// the tile's). D's layout: lane & 31 is the column, element e the row
// (e / 4) * 8 + (lane / 32) * 4 + e % 4. Old values are read 16 at a time, so
// that they do not wait for each other.
template <typename E, bool ALL, int MT, int NT>
__device__ __forceinline__ void put_tile(const f32x16 (&acc)[MT][NT], E* at, int64_t ld, int64_t rows, int64_t cols,
                                         bool add) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float old[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) old[e] = 0.0f;
            if (add) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int r = m * 32 + (e >> 2) * 8 + (e & 3);
                    if (ALL || (r < rows && n * 32 < cols)) old[e] = load_elem(at + r * ld + n * 32);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int r = m * 32 + (e >> 2) * 8 + (e & 3);
                if (ALL || (r < rows && n * 32 < cols)) store_elem(at + r * ld + n * 32, acc[m][n][e] + old[e]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
}

// The same for a wave's part of a tile that begins at element (o, i) of dW.
template <int MT, int NT>
__device__ __forceinline__ void put_dw(const f32x16 (&acc)[MT][NT], const WgradArgs& a, int64_t o, int64_t i, int lane) {
    const bool all = o + MT * 32 <= a.out && i + NT * 32 <= a.in;
    o += (lane >> 5) * 4;
    i += lane & 31;
    const int64_t at = o * a.ld_dw + i, rows = a.out - o, cols = a.in - i;
    if (a.grad_dt == kBf16) {
        uint16_t* p = (uint16_t*)a.dw + at;
        if (all)
            put_tile<uint16_t, true>(acc, p, a.ld_dw, rows, cols, a.accumulate);
        else
            put_tile<uint16_t, false>(acc, p, a.ld_dw, rows, cols, a.accumulate);
    } else {
        float* p = (float*)a.dw + at;
        if (all)
            put_tile<float, true>(acc, p, a.ld_dw, rows, cols, a.accumulate);
        else
            put_tile<float, false>(acc, p, a.ld_dw, rows, cols, a.accumulate);
    }
}

template <int DD, int FMT, int BM, int BN, int WM, int WN, int BK>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64, 2) void wgrad_kernel(WgradArgs a) {
    constexpr int T = (BM / WM) * (BN / WN) * 64;  // threads
    constexpr int P = DD == kFp32 ? 3 : 1;         // bf16 terms of dY
    constexpr int PA = BM * 2, PB = BN * 2;        // LDS row bytes
    constexpr int CA = BM / 8, CB = BN / 16;       // chunks per row: 8 of dY, 16 codes
    constexpr int NA = BK * CA / T, NB = BK * CB / T;
    constexpr int MT = WM / 32, NT = WN / 32;
    static_assert(BK * CA % T == 0 && BK * CB % T == 0 && T % CA == 0, "whole chunks per thread");
    constexpr int SA = BK * PA, SB = BK * PB, STAGE = P * SA + SB;
    __shared__ __attribute__((aligned(1024))) char lds[2 * STAGE];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave / (BN / WN), wn = wave % (BN / WN);
    const int64_t total = (int64_t)a.tiles_m * a.tiles_n * a.splits;

    // This lane's place in a transposed read: 16 lanes hold 4 rows of 16
    // columns and get one column each.
    const int r4 = (lane >> 2) & 3, rbase = (lane >> 5) * 8 + r4;
    int offA[MT], offB[NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
        offA[m] = rbase * PA + (((wm * WM + m * 32) * 2) ^ (r4 << 6)) + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
#pragma unroll
    for (int n = 0; n < NT; ++n)
        offB[n] = P * SA + rbase * PB + (((wn * WN + n * 32) * 2) ^ (r4 << 6)) + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;

    for (int64_t item = blockIdx.x; item < total; item += gridDim.x) {
        int tm, tn;
        const uint32_t at = by_xcd((uint32_t)item, (uint32_t)total), tiles = (uint32_t)(a.tiles_m * a.tiles_n);
        const int part = uniform(at / tiles);
        tile_place(a, at % tiles, &tm, &tn);
        const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
        const int64_t kb = part * a.span, ke = kb + a.span < a.rows ? kb + a.span : a.rows;
        const bool bias = a.db && tn == 0;

        f32x16 acc[MT][NT];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[m][n][e] = 0.0f;
        float sums[8] = {0, 0, 0, 0, 0, 0, 0, 0};

        const int64_t behind_chunk = a.out - (m0 + (tid % CA) * 8);
        const int chunk = behind_chunk >= 8 ? 8 : (behind_chunk > 0 ? (int)behind_chunk : 0);  // columns of its chunks
        Raw8<DD> ra[NA];
        u32x4 rb[NB];
        uint32_t rs[NB];
        auto fetch = [&](int64_t k) {
#pragma unroll
            for (int j = 0; j < NA; ++j) {
                const int id = tid + j * T;
                const int64_t row = k + id / CA, col = m0 + (id % CA) * 8;
                const int n = row < ke ? chunk : 0;
                ra[j] = fetch8<DD, false>({(const char*)a.dy + row * a.ld_dy * (DD == kBf16 ? 2 : 4), nullptr}, (int)col, n);
            }
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const int id = tid + j * T;
                const int64_t row = k + id / CB, col = n0 + (id % CB) * 16;
                rb[j] = u32x4{0, 0, 0, 0};
                rs[j] = 127;
                if (row < ke && col < a.pitch) {
                    rb[j] = *(const u32x4*)(a.codes + row * a.pitch + col);
                    rs[j] = a.scales[row * (a.pitch / kCkptBlock) + col / kCkptBlock];
                }
            }
        };
        auto stage = [&](char* buf) {
#pragma unroll
            for (int j = 0; j < NA; ++j) {
                const int id = tid + j * T, t = id / CA, c = id % CA;
                char* at = buf + t * PA + ((c * 16) ^ ((t & 3) << 6));
                settle8(ra[j], (int)(m0 + c * 8), chunk);
                if constexpr (DD == kBf16) {
                    *(u32x4*)at = ra[j].v;
                } else {
                    float f[8];
                    uint32_t w[3][4];
                    widen8(ra[j], f);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t lo[3], hi[3];
                        split3(f[2 * e], lo);
                        split3(f[2 * e + 1], hi);
#pragma unroll
                        for (int p = 0; p < 3; ++p) w[p][e] = (lo[p] >> 16) | hi[p];
                    }
#pragma unroll
                    for (int p = 0; p < 3; ++p) *(u32x4*)(at + p * SA) = u32x4{w[p][0], w[p][1], w[p][2], w[p][3]};
                }
                if (bias) {
                    float f[8];
                    widen8(ra[j], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) sums[e] += f[e];
                }
            }
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const int id = tid + j * T, t = id / CB, c = id % CB;
                uint32_t w[8];
                decode16<FMT>(rb[j], rs[j], w);
                char* at = buf + P * SA + t * PB;
                *(u32x4*)(at + ((c * 32) ^ ((t & 3) << 6))) = u32x4{w[0], w[1], w[2], w[3]};
                *(u32x4*)(at + ((c * 32 + 16) ^ ((t & 3) << 6))) = u32x4{w[4], w[5], w[6], w[7]};
            }
        };
        auto operand = [&](const char* at, int pitch) {
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)at);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(at + 4 * pitch));
            return __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        };
        auto multiply = [&](const char* buf) {
#pragma unroll
            for (int k = 0; k < BK; k += 16) {
                bf16x8 fb[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) fb[n] = operand(buf + offB[n] + k * PB, PB);
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    bf16x8 fa[MT];
#pragma unroll
                    for (int m = 0; m < MT; ++m) fa[m] = operand(buf + offA[m] + p * SA + k * PA, PA);
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[m], fb[n], acc[m][n], 0, 0, 0);
                }
            }
        };

        if (kb < ke) {
            fetch(kb);
            stage(lds);
            __syncthreads();
            int cur = 0;
            for (int64_t k = kb; k < ke; k += BK) {
                const bool more = k + BK < ke;
                if (more) fetch(k + BK);
                multiply(lds + cur * STAGE);
                if (more) stage(lds + (cur ^ 1) * STAGE);
                __syncthreads();
                cur ^= 1;
            }
        }

        float* const mine = a.splits > 1 ? a.part + (int64_t)part * (a.out * a.in + a.out) : nullptr;
        const int64_t o0 = m0 + wm * WM, i0 = n0 + wn * WN;
        if (mine) {
            const int64_t o = o0 + (lane >> 5) * 4, i = i0 + (lane & 31);
            put_tile<float, false>(acc, mine + o * a.in + i, a.in, a.out - o, a.in - i, false);
        } else {
            put_dw(acc, a, o0, i0, lane);
        }
        if (bias) {  // the threads that hold the same 8 columns
            float* s = (float*)lds;
#pragma unroll
            for (int e = 0; e < 8; ++e) s[(tid / CA) * BM + (tid % CA) * 8 + e] = sums[e];
            __syncthreads();
            for (int c = tid; c < BM; c += T) {
                float v = 0.0f;
#pragma unroll
                for (int r = 0; r < T / CA; ++r) v += s[r * BM + c];
                const int64_t o = m0 + c;
                if (o >= a.out) continue;
                if (mine)
                    mine[a.out * a.in + o] = v;
                else
                    put_grad(a.db, o, v, a.grad_dt, a.accumulate);
            }
            __syncthreads();
        }
    }
}

// The large form, for bf16 dY: tiles of 256 x 256, eight waves of 128 x 64. A
// slab of 64 rows costs a CU 2,061 cycles of matrix units and reads 192 KB from
// LDS (1,536 cycles at 128 bytes a cycle) where four tiles of 128 x 128 would
// read 256 KB. Each wave's 128 fp32 accumulators leave 128 registers for
// operands and the next slab. 16384x11008x4096 takes 1,330 to 1,480 us from run
// to run (1,000 to 1,110 TFLOP/s at 2.0 GHz; 688 tiles are 2.7 rounds of 256),
// where the library's bf16 product of such operands takes 1,570 to 1,640;
// 2048x4096x4096 71 to 82 us, the library's 65 to 70. The matrix units are busy
// 54% of the time and LDS 41%: the rest is the steps' latency. Operands three
// steps ahead do not fit the registers.
constexpr int kBigThreads = 512, kBigBK = 64;

// v plus the two bf16 values of a word.
__device__ __forceinline__ float sum2(uint32_t w, float v) {
    const bf16x2 one = {(__bf16)1.0f, (__bf16)1.0f};
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), one, v, false);
}

template <int FMT>
__global__ __launch_bounds__(kBigThreads) void wgrad_big_kernel(WgradArgs a) {
    constexpr int BM = kWgradBig, BN = kWgradBig, WM = 128, WN = 64, BK = kBigBK, T = kBigThreads;
    constexpr int PA = BM * 2, PB = BN * 2;
    constexpr int MT = WM / 32, NT = WN / 32;
    constexpr int SA = BK * PA, SB = BK * PB, STAGE = SA + SB;
    constexpr int RA = T / (BM / 8), RB = T / (BN / 16);  // rows that one round of loads covers
    constexpr int NA = BK / RA, NB = BK / RB;
    __shared__ __attribute__((aligned(1024))) char lds[2 * STAGE];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / (BN / WN), wn = wave % (BN / WN);
    const int r4 = (lane >> 2) & 3, rbase = (lane >> 5) * 8 + r4;
    const int low = rbase * PA + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;  // PA == PB
    // operand m of dY lies at offA ^ (m << 6), n of X at offB ^ (n << 6): the
    // windows' exchange has bits 6 and 7 to itself (wn's bit 7 is in offB's)
    const int offA = (low | (r4 << 6)) + wm * WM * 2;
    const int offB = SA + ((low | (r4 << 6)) ^ ((wn & 1) << 7)) + (wn >> 1) * 256;
    static_assert(WM * 2 % 256 == 0 && WN == 64, "operand offsets");
    // where this thread's chunks go; rows of a round are a multiple of 4 apart
    const int ta = tid / (BM / 8), ca = tid % (BM / 8), tb = tid / (BN / 16), cb = tid % (BN / 16);
    const int putA = ta * PA + ((ca * 16) ^ ((ta & 3) << 6));
    const int putB = SA + tb * PB + ((cb * 32) ^ ((tb & 3) << 6));
    const int64_t sp = a.pitch / kCkptBlock;

    const uint32_t full = (uint32_t)a.full, rest = (uint32_t)a.rest, total = full + rest * (uint32_t)a.parts;
    for (uint32_t item = blockIdx.x; item < total; item += gridDim.x) {
        // the parts of one share of the rows lie together, tile by tile
        uint32_t tile;
        int64_t k0 = 0, k1 = a.slabs;
        float* mine = nullptr;  // a part of a tile goes to its slot of the workspace
        if (item < full) {
            tile = by_xcd(item, full);
        } else {
            const uint32_t p = by_xcd(item - full, rest * (uint32_t)a.parts), part = uniform(p / rest);
            tile = full + p - part * rest;
            k0 = part * a.share;
            k1 = k0 + a.share < k1 ? k0 + a.share : k1;
            if (a.parts > 1) mine = a.part + p * kWgradSlot;
        }
        int tm, tn;
        tile_place(a, tile, &tm, &tn);
        const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
        const int64_t kb = k0 * BK, ke = k1 * BK < a.rows ? k1 * BK : a.rows;
        const bool bias = a.db && tn == 0 && wn == 0;
        // columns behind the last are read from the last chunk and not stored
        const int64_t col_a = m0 + ca * 8 <= a.out - 8 ? m0 + ca * 8 : a.out - 8;
        const int64_t col_b = n0 + cb * 16 < a.pitch ? n0 + cb * 16 : a.pitch - 16;
        // in the last tile of an `out` that is not whole chunks, the last chunk
        // that exists in part is read from `out - 8` and moved into place
        const bool ragged = m0 + BM > a.out && a.out % 8 != 0;
        const int late = (int)(m0 + ca * 8 - col_a) * 16;  // bits, 0 in other chunks
        const int64_t from = m0 <= a.out - 8 ? m0 : a.out - 8;  // no chunk starts before it
        const uint32_t va = (uint32_t)(col_a - from) * 2, vb = (uint32_t)(col_b - n0);
        // byte offsets of rows within a slab, in 32 bits (a slab is below 2^31 bytes)
        const uint32_t la = (uint32_t)a.ld_dy * 2, lb = (uint32_t)a.pitch;
        const uint32_t ta_la = (uint32_t)ta * la, tb_lb = (uint32_t)tb * lb;
        const char* pa = (const char*)a.dy + (kb * a.ld_dy + from) * 2;
        const char* pb = a.codes + kb * a.pitch + n0;
        const uint8_t* ps = a.scales + kb * sp + n0 / kCkptBlock;

        f32x16 acc[MT][NT];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[m][n][e] = 0.0f;
        float sums[MT] = {0, 0, 0, 0};  // bias: this lane's columns of dY over half of the rows
        u32x4 ra[NA], rb[NB];
        uint32_t rs[NB];
        // Rows behind the last are read from it, and staged as zeros.
        int64_t left = ke - kb;  // rows from the next slab on
        int have = 0;            // rows of the slab in the registers
        auto fetch = [&] {
            have = left < BK ? (int)left : BK;
            const uint32_t last_a = (uint32_t)(have - 1) * la, last_b = (uint32_t)(have - 1) * lb;
            // opaque, so that the six rows' offsets are computed here and do not
            // occupy registers through the loop
            uint32_t row_a = ta_la, row_b = tb_lb;
            asm volatile("" : "+v"(row_a), "+v"(row_b));
#pragma unroll
            for (int j = 0; j < NA; ++j) {
                const uint32_t row = row_a + (uint32_t)(j * RA) * la;
                ra[j] = *(const u32x4_a2*)(pa + ((row < last_a ? row : last_a) + va));
            }
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const uint32_t row = row_b + (uint32_t)(j * RB) * lb, at = (row < last_b ? row : last_b) + vb;
                rb[j] = *(const u32x4*)(pb + at);
                rs[j] = *(ps + at / kCkptBlock);  // a row of exponents is a 32nd of one of codes
            }
            pa += (int64_t)BK * a.ld_dy * 2;
            pb += (int64_t)BK * a.pitch;
            ps += (int64_t)BK * sp;
            left -= BK;
        };
        // The last slab's zeros and the ragged chunk's move are behind branches
        // (kept as such by the empty asm): as selects they would cost every slab
        // 30 of its 150 vector instructions.
        auto put_a = [&](char* buf, int j) {
            if (ragged || have < BK) {
                asm volatile("");
                if (ragged) ra[j] = behind(ra[j], late);
                if (ta + j * RA >= have) ra[j] = u32x4{0, 0, 0, 0};
            }
            *(u32x4*)(buf + putA + j * RA * PA) = ra[j];
        };
        auto put_b = [&](char* buf, int j) {
            uint32_t w[8];
            if (have < BK) {
                asm volatile("");
                if (tb + j * RB >= have) {
                    rb[j] = u32x4{0, 0, 0, 0};
                    rs[j] = 127;
                }
            }
            decode16<FMT>(rb[j], rs[j], w);
            *(u32x4*)(buf + putB + j * RB * PB) = u32x4{w[0], w[1], w[2], w[3]};
            *(u32x4*)(buf + putB + 16 + j * RB * PB) = u32x4{w[4], w[5], w[6], w[7]};
        };
        auto operand = [&](const char* at) {
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)at);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(at + 4 * PA));
            return __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        };
        if (kb < ke) {
            const int slabs = (int)((ke - kb + BK - 1) / BK);
            fetch();
#pragma unroll
            for (int j = 0; j < NA; ++j) put_a(lds, j);
#pragma unroll
            for (int j = 0; j < NB; ++j) put_b(lds, j);
            if (slabs > 1) fetch();
            __syncthreads();
            // A slab is 16 steps: 16 rows at a time, 32 of the wave's 128 columns
            // of dY in each. The operands of a step are read two steps before it
            // (X's up to four), so that matrix instructions do not wait for LDS;
            // the next slab goes from registers to the other buffer in steps 1 to
            // 6, the loads of the one after it are issued in step 8, and the
            // barrier that publishes the other buffer stands before step 14, whose
            // reads are the first from it. Behind the last slab the other buffer
            // holds nothing of use: it is written and read, and not multiplied.
            bf16x8 fa[4], fb[2][NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) fb[0][n] = operand(lds + (offB ^ (n << 6)));
            fa[0] = operand(lds + offA);
            fa[1] = operand(lds + (offA ^ (1 << 6)));
            int cur = 0;
#pragma unroll 1
            for (int k = 0; k < slabs; ++k) {
                const char* buf = lds + cur * STAGE;
                char* other = lds + (cur ^ 1) * STAGE;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if (i == 14) __syncthreads();
                    const int ahead = (i + 2) & 15;
                    fa[ahead & 3] = operand((i < 14 ? buf : other) + (offA ^ ((ahead & 3) << 6)) + (ahead >> 2) * 16 * PA);
                    if ((i & 3) == 2) {
                        const int ks = ((i >> 2) + 1) & 3;
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            fb[ks & 1][n] = operand((i < 14 ? buf : other) + (offB ^ (n << 6)) + ks * 16 * PB);
                    }
                    if (i >= 1 && i < 1 + NA) put_a(other, i - 1);
                    if (i >= 1 + NA && i < 1 + NA + NB) put_b(other, i - 1 - NA);
                    if (i == 8 && k + 2 < slabs) fetch();
                    if (bias) {
                        const u32x4 w = __builtin_bit_cast(u32x4, fa[i & 3]);
                        sums[i & 3] = sum2(w.x, sum2(w.y, sum2(w.z, sum2(w.w, sums[i & 3]))));
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        acc[i & 3][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i & 3], fb[(i >> 2) & 1][n],
                                                                               acc[i & 3][n], 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                }
                cur ^= 1;
            }
            __syncthreads();
        }

        if (mine)
            put_tile<float, true>(acc, mine + (wm * WM + (lane >> 5) * 4) * BN + wn * WN + (lane & 31), BN, BM, BN, false);
        else
            put_dw(acc, a, m0 + wm * WM, n0 + wn * WN, lane);
        if (bias) {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const float v = sums[m] + __shfl_xor(sums[m], 32, 64);
                const int c = wm * WM + m * 32 + (lane & 31);
                if (lane >= 32) continue;
                if (mine)
                    mine[BM * BN + c] = v;
                else if (m0 + c < a.out)
                    put_grad(a.db, m0 + c, v, a.grad_dt, a.accumulate);
            }
        }
    }
}

// Sums the parts of the large form's rest tiles, in order: an item is four
// rows of a tile, or (the last of its 65) the tile's part of the bias.
__global__ __launch_bounds__(kThreads) void wgrad_big_join_kernel(WgradArgs a) {
    constexpr int BM = kWgradBig, BN = kWgradBig;
    for (int64_t item = blockIdx.x; item < a.rest * 65; item += gridDim.x) {
        const int64_t t = item / 65;
        const int q = (int)(item % 65);
        int tm, tn;
        tile_place(a, (uint32_t)(a.full + t), &tm, &tn);
        const float* src = a.part + t * kWgradSlot + q * 4 * BN + threadIdx.x * (q < 64 ? 4 : 1);
        const int64_t next = a.rest * kWgradSlot;
        if (q == 64) {
            if (!a.db || tn != 0) continue;
            float v = 0.0f;
            for (int64_t p = 0; p < a.parts; ++p) v += src[p * next];
            const int64_t o = (int64_t)tm * BM + threadIdx.x;
            if (o < a.out) put_grad(a.db, o, v, a.grad_dt, a.accumulate);
            continue;
        }
        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int64_t p = 0; p < a.parts; p += 4) {  // four parts' loads in flight
            f32x4 w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[e] = p + e < a.parts ? (f32x4)*(const f32x4_a4*)(src + (p + e) * next) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int e = 0; e < 4; ++e) v += w[e];
        }
        const int64_t o = (int64_t)tm * BM + q * 4 + threadIdx.x / 64, i = (int64_t)tn * BN + (threadIdx.x & 63) * 4;
        if (o >= a.out) continue;
        if (i + 4 <= a.in && a.grad_dt == kFp32) {
            f32x4_a4* p = (f32x4_a4*)((float*)a.dw + o * a.ld_dw + i);
            *p = a.accumulate ? (f32x4)*p + v : v;
            continue;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i + e < a.in) put_grad(a.dw, o * a.ld_dw + i + e, v[e], a.grad_dt, a.accumulate);
    }
}

// Sums the parts, in order. A thread takes V neighbouring elements and has the
// loads of 8 / V parts in flight: one element where there are few outputs (of
// many parts), four where there are many. Items are runs of 256 V columns of a
// row of dW, and after them runs of db.
template <int V>
__global__ __launch_bounds__(kThreads) void wgrad_join_kernel(WgradArgs a) {
    constexpr int N = 8 / V;
    const int64_t run = kThreads * V, segs = (a.in + run - 1) / run, bsegs = a.db ? (a.out + run - 1) / run : 0;
    const int64_t stride = a.out * a.in + a.out;
    for (int64_t item = blockIdx.x; item < a.out * segs + bsegs; item += gridDim.x) {
        const bool bias = item >= a.out * segs;
        const int64_t o = bias ? a.out : item / segs;
        const int64_t c = (bias ? item - a.out * segs : item % segs) * run + threadIdx.x * V;
        const int64_t left = (bias ? a.out : a.in) - c;
        if (left <= 0) continue;
        const float* src = a.part + o * a.in + c;
        float v[V];
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = 0.0f;
        for (int s = 0; s < a.splits; s += N) {
            float t[N][V];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const float* q = src + (s + k) * stride;
                if (V == 4 && left >= 4 && s + k < a.splits) {
                    const f32x4 w = *(const f32x4_a4*)q;
                    t[k][0] = w.x; t[k][1 % V] = w.y; t[k][2 % V] = w.z; t[k][3 % V] = w.w;
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e) t[k][e] = e < left && s + k < a.splits ? q[e] : 0.0f;
                }
            }
#pragma unroll
            for (int k = 0; k < N; ++k)
#pragma unroll
                for (int e = 0; e < V; ++e) v[e] += t[k][e];
        }
        const int64_t at = bias ? c : o * a.ld_dw + c;
        void* const out = bias ? a.db : a.dw;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if (e < left) put_grad(out, at + e, v[e], a.grad_dt, a.accumulate);
        }
    }
}

template <int FMT>
hipError_t run_large(const WgradArgs& a, hipStream_t stream) {
    wgrad_big_kernel<FMT><<<grid_for(a.full + a.rest * a.parts, kBigThreads), kBigThreads, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.parts == 1) return e;
    wgrad_big_join_kernel<<<grid_for(a.rest * 65, kThreads), kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

template <int DD, int FMT>
hipError_t run_small(const WgradArgs& a, hipStream_t stream) {
    const int64_t total = (int64_t)a.tiles_m * a.tiles_n * a.splits;
    wgrad_kernel<DD, FMT, kWgradTile, kWgradTile, 64, 64, DD == kBf16 ? 64 : 32><<<grid_for(total, 256), 256, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    const int v = a.out * a.in >= (int64_t)1 << 20 ? 4 : 1;
    const int64_t n = kThreads * v;
    const int64_t items = a.out * ((a.in + n - 1) / n) + (a.db ? (a.out + n - 1) / n : 0);
    if (v == 4)
        wgrad_join_kernel<4><<<grid_for(items, kThreads), kThreads, 0, stream>>>(a);
    else
        wgrad_join_kernel<1><<<grid_for(items, kThreads), kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ckpt_wgrad(const Wgrad& w, hipStream_t stream) {
    const WgradCut cut = wgrad_cut(w.rows, w.out, w.in);
    const WgradShare share = wgrad_share(w.rows, w.out, w.in);
    const bool large = wgrad_can_be_large(w) && share.us < cut.us, e4m3 = w.format == ZR_CKPT_E4M3;
    const int tile = large ? kWgradBig : kWgradTile;
    WgradArgs a{};
    a.dy = w.dy;
    a.pitch = ckpt_pitch(w.in);
    a.codes = (const char*)w.ckpt;
    a.scales = (const uint8_t*)w.ckpt + w.rows * a.pitch;
    a.part = (float*)w.workspace;
    a.dw = w.dw;
    a.db = w.dbias;
    a.rows = w.rows; a.out = w.out; a.in = w.in; a.ld_dy = w.ld_dy; a.ld_dw = w.ld_dw;
    a.span = cut.span;
    a.grad_dt = w.grad_dt; a.accumulate = w.accumulate;
    a.tiles_m = (int)((w.out + tile - 1) / tile);
    a.tiles_n = (int)((w.in + tile - 1) / tile);
    a.splits = cut.splits;
    a.slabs = share.slabs; a.full = share.full; a.rest = share.rest; a.parts = share.parts; a.share = share.share;
    if (large) return e4m3 ? run_large<kE4m3>(a, stream) : run_large<kInt8>(a, stream);
    if (w.dy_dt == ZR_BF16) return e4m3 ? run_small<kBf16, kE4m3>(a, stream) : run_small<kBf16, kInt8>(a, stream);
    return e4m3 ? run_small<kFp32, kE4m3>(a, stream) : run_small<kFp32, kInt8>(a, stream);
}

}  // namespace zr
