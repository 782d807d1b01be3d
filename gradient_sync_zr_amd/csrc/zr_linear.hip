// Product of two packed matrices, as a linear layer's forward pass has it:
//     z[t, o] = sum_i x[t, i] * w[o, i] + bias[o]
// with x and w in blocks of 32 columns (e4m3 or e2m1 codes and one power of two
// each), which are the operands of the scaled matrix instructions: a lane brings
// the codes and the exponent bytes of its row, and no value is decoded.
//
// What the instructions do with the products decides between two ways:
//  - e2m1 by e2m1: products and sums are exact up to the fp32 accumulator;
//  - with e4m3 on either side the products that one lane brings are added with 13
//    bits below the largest of them (measured: 2^16 + 2^2 keeps both, 2^16 + 2^1 does
//    not), which is below what a bf16 result keeps and not below fp32's. So bf16
//    results take the scaled instructions, and for fp32 results both operands are
//    decoded to bf16 on their way from LDS (every held value is exact there) and
//    go through the bf16 instructions, which sum in fp32. Against 64 bits a bf16 result
//    is then off by as much as one that is summed in fp32 (1.66e-3 of the result's norm
//    both, 1x4096x4096 and 8192x4096x4096; one or two elements in a hundred are the other
//    neighbour of a border). Decoding would take 1.8 times as long, and for few rows up to
//    a sixth longer of weights in 8 bits and a third in 4 (one token by 4096x11008 12.6
//    us for 11.3, and 10.0 for 7.7).
//
// Reached, in TFLOP/s (with what the same instructions reach alone, held by the card's
// power): e2m1 2,980 to 3,180 at 16384x11008x4096 and 3,870 to 3,960 at 8192^3 (6,500),
// e4m3 2,260 to 2,500 (3,400 to 3,700), decoded 1,250 to 1,340 (bf16: 1,390 to 1,620);
// the library's bf16 product reaches 1,235 and 1,375. The matrix units are busy 45 to 50%
// (e2m1) and 56 to 64% (e4m3) of the time, at a clock of 1.7 to 1.8 GHz of 2.4, where the
// instructions alone keep them busy throughout at a lower one; LDS is busy 37 to 43%,
// and waves wait 30 to 34% of their cycles. Of a stage's 1.27 us 0.95 remain without the
// loads to LDS, and a tile costs 5 us in front of its loop and behind it. Four waves of
// 128x128 instead of eight of 128x64 took 463 us for 424 (16384x11008x4096 of e2m1, the
// product behind its packing), operands read 3 or 4 steps ahead and two stages of 128-byte
// rows the same.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "zr_e2m1.hpp"
#include "zr_internal.hpp"
#include "zr_norm.hpp"

namespace zr {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct LinArgs {
    const char *w, *x;          // codes
    const uint8_t *ws, *xs;     // exponents
    const void* bias;
    void* z;
    float* part;                // parts > 1: [parts][rows][out]
    int64_t rows, out, wrow, xrow, sp, ld_z;  // bytes of a row of codes, of exponents
    int64_t turns, share;       // turns of 512 columns, of a part
    int bias_dt, z_dt, accumulate, tiles_o, tiles_t, parts;
};

__device__ __forceinline__ int uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane((int)v); }

// Blocks are dealt to the 8 XCDs in turn: neighbours among `total` items for
// the blocks of one XCD, so that their operands meet in that XCD's L2.
__device__ __forceinline__ uint32_t by_xcd(uint32_t item, uint32_t total) {
    const uint32_t x = item % 8, i = item / 8, q = total / 8, r = total % 8;
    return (x < r ? x * (q + 1) : r * (q + 1) + (x - r) * q) + i;
}

// 16 codes (e4m3: 16 bytes; e2m1: 8) as two bf16 operands.
template <int FMT>
__device__ __forceinline__ void decode16(const u32x4& q, float scale, bf16x8 f[2]) {
    uint32_t w[8];
    if constexpr (FMT == kE2m1) {
        const uint32_t c[2] = {q.x, q.y};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            w[4 * k] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[k], scale, 0));
            w[4 * k + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[k], scale, 1));
            w[4 * k + 2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[k], scale, 2));
            w[4 * k + 3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[k], scale, 3));
        }
    } else {
        const uint32_t c[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            w[2 * k] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[k], scale, false));
            w[2 * k + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[k], scale, true));
        }
    }
    f[0] = __builtin_bit_cast(bf16x8, u32x4{w[0], w[1], w[2], w[3]});
    f[1] = __builtin_bit_cast(bf16x8, u32x4{w[4], w[5], w[6], w[7]});
}

// The scale of an exponent byte for the decoding (0 where the block does not
// exist: its codes count for nothing beside the other operand's, 0 as well).
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// Eight neighbouring results of a row, with bias and old values, rounded once; or,
// into a part of the workspace, as they are.
__device__ __forceinline__ void put8(const LinArgs& a, float* part, int64_t t, int64_t o, const float v[8]) {
    const int64_t left = a.out - o;
    const int n = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
    if (n == 0) return;
    float f[8];
    if (part) {
        store8<false>((char*)(part + t * a.out + o), kFp32, 0, n, v);
        return;
    }
    load_param8(a.bias ? (const char*)a.bias + o * (a.bias_dt == kBf16 ? 2 : 4) : nullptr, a.bias_dt, 0, n, 0.0f, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] += v[e];
    char* const z = (char*)a.z + (t * a.ld_z + o) * (a.z_dt == kBf16 ? 2 : 4);
    if (a.accumulate) {
        float old[8];
        load_param8(z, a.z_dt, 0, n, 0.0f, old);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] += old[e];
    }
    store8<true>(z, a.z_dt, 0, n, f);  // past the caches: 16384x11008x4096 of e2m1, behind its packing, 475 us without, 431 with
}

// ------------------------------------------------------------- tiled form
// LDS holds a stage's rows, of 64 or 32 bytes, in 16-byte chunks: lines of 128 bytes
// (two rows or four), two lines across its 64 banks. A chunk's place in its line is
// exchanged by the number of the pair of lines, so that the 16 chunks of 16
// neighbouring rows, which a read takes at once, lie in different banks. (Exchanged by
// the line's number, half of the reads' cycles were conflicts. What is left is the
// exponents': a word of each row at a stride of 16 bytes, 288 of LDS's 768 cycles for a
// 256 x 256 tile's 128 columns of e2m1, beside 1,024 of the matrix units.) The loads write LDS
// directly, a wave's 64 chunks in a row, so the exchange is made in the addresses
// that the lanes load from. 32 rows further down it is the same.
template <int RB>
__device__ __forceinline__ int chunk_swap(int line) {
    return (line >> 1) & (RB == 64 ? 7 : 3);
}

template <int RB>
__device__ __forceinline__ int chunk_at(int row, int c) {
    constexpr int ROWS = 128 / RB;
    const int line = row / ROWS, at = row % ROWS * (RB / 16) + c;
    return line * 128 + ((at ^ chunk_swap<RB>(line)) << 4);
}

// Row and chunk that belong to the LDS slot.
template <int RB>
__device__ __forceinline__ void chunk_of(int slot, int* row, int* c) {
    const int line = slot >> 3, p = (slot & 7) ^ chunk_swap<RB>(line);
    *row = line * (128 / RB) + p / (RB / 16);
    *c = p % (RB / 16);
}

typedef __attribute__((address_space(3))) char* lptr;

// 16 bytes of every lane from base + offset to LDS, at `to` (the same for the wave)
// plus `down` plus 16 times the lane. Written in assembly because the compiler, which cannot
// tell the stages apart, waits for its own such loads before every read of LDS;
// the kernel waits once, in front of the barrier that publishes a stage. There
// is no register that the load still writes to. A scalar write of M0 has to be one wait
// state ahead of a load to LDS, which takes its place from M0; nobody else puts it in
// (the compiler inserts nothing inside an asm, and uses M0 for nothing else here), and
// the build reads the unit's machine code for it.
__device__ __forceinline__ void load_lds16(const char* base, uint32_t offset, uint32_t to, int down) {
    asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(offset), "s"(base), "i"(down)
                 : "m0", "scc", "memory");
}

// 16 exponent bytes of a row from byte `at` (< sp) on, the row `row` bytes behind
// `base`; those behind the row's `sp` are 0. Nothing is read from `size` bytes on, the
// buffer's end: the last rows' bytes are then read early, from the codes' side, and
// moved into place.
__device__ __forceinline__ u32x4 exponents16(const uint8_t* base, int row, int at, int sp, int size) {
    typedef u32x4 u32x4_a1 __attribute__((aligned(1)));
    int over = row + at + 16 - size;
    over = over > 0 ? over : 0;
    const u32x4 v = behind((u32x4)*(const u32x4_a1*)(base + (row + at - over)), over * 8);
    const int left = sp - at < 16 ? sp - at : 16;
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int n = left - 4 * k;  // bytes of this word that the row has
        w[k] = n >= 4 ? w[k] : (n <= 0 ? 0u : w[k] & ((1u << (8 * n)) - 1));
    }
    return u32x4{w[0], w[1], w[2], w[3]};
}

// Waits until at most N of the wave's loads are in flight (they end in order).
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"i"(N) : "memory");
}

// Orders what a wave's lanes wrote to LDS before what its other lanes read behind this,
// for the compiler: a wave's LDS accesses are carried out in their order, so it costs no
// instruction.
__device__ __forceinline__ void wave_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// A tile's product. Eight (four) waves have WO outputs of WT tokens each; the
// weight's rows are the matrix instructions' A, so that a lane ends with one token
// and neighbouring outputs.
//
// A stage is BK codes of every row, and LDS holds STAGES of them, so that loads have the
// time of two stages and more to arrive. A stage goes through in units of 64 codes
// (32 where operands are decoded), and a unit by 32 of the wave's outputs: steps of NT
// matrix instructions each, whose operands are read AHEAD steps earlier. The barrier
// that publishes a stage stands before the first of these reads; by then all of the stage
// before has been read, and its place takes the loads of the stage STAGES - 1 behind
// the published one. A turn of the loop is the stages of 512 codes, whose exponents
// are loaded at once, a turn ahead. Stages behind the last have exponents of 0, and
// the loads ahead of the last are of it once more.
//
// (Two waves a SIMD are asked for so that the accumulators stay in VGPRs: with room for
// more registers they were kept as AGPRs, and moved back and forth in every step. 2048^3
// of e2m1 took 19.7 us for 11.3.)
template <int FW, int FX, bool EXACT, int BO, int BT, int WO, int WT>
__global__ __launch_bounds__((BO / WO) * (BT / WT) * 64, 2) void linear_kernel(LinArgs a) {
    constexpr int T = (BO / WO) * (BT / WT) * 64;
    constexpr bool PAIR4 = FW == kE2m1 && FX == kE2m1;
    constexpr int BK = PAIR4 ? 128 : 64, STAGES = 4;
    constexpr int RW = FW == kE2m1 ? BK / 2 : BK, RX = FX == kE2m1 ? BK / 2 : BK;
    constexpr int SW = BO * RW, SX = BT * RX;
    constexpr int NW = SW / 16 / T, NX = SX / 16 / T, LOADS = NW + NX;
    constexpr int SPT = kLinearGroup / BK;  // stages of a turn
    constexpr int SCALES = (BO + BT) * 16;
    constexpr int MT = WO / 32, NT = WT / 32;
    constexpr int UNIT = EXACT ? 32 : 64, ST = BK / UNIT * MT, STEPS = SPT * ST, AHEAD = 2;
    static_assert(SW / 16 % T == 0 && SX / 16 % T == 0 && BO + BT == T, "whole chunks per thread");
    static_assert(ST >= AHEAD && STEPS % 4 == 0 && SPT % STAGES == 0 && STAGES == 4, "the rings' turns");
    constexpr int RESULTS = T / 64 * WO * 32 * 4, EXPS = STAGES * (SW + SX), LDS = EXPS + 2 * SCALES;
    // the weight's stages, x's, exponents twice; the stages within an instruction's offset
    __shared__ __attribute__((aligned(1024))) char lds[RESULTS > LDS ? RESULTS : LDS];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wo = wave / (BT / WT), wt = wave % (BT / WT);
    const int r = lane & 31, g = lane >> 5;
    // where a lane's first chunk lies; the others are at exchanges of bits 4 and 5
    constexpr bool HALF_W = EXACT && FW == kE2m1, HALF_X = EXACT && FX == kE2m1;
    const int place_w = wo * WO * RW + chunk_at<RW>(r, HALF_W ? 0 : g) + (HALF_W ? 8 * g : 0);
    const int place_x = STAGES * SW + wt * WT * RX + chunk_at<RX>(r, HALF_X ? 0 : g) + (HALF_X ? 8 * g : 0);
    const int scale_w = EXPS + (wo * WO + r) * 16, scale_x = EXPS + (BO + wt * WT + r) * 16;
    const uint32_t to = (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)(uintptr_t)(lptr)lds + (uint32_t)wave * 1024));
    const uint32_t total = (uint32_t)a.tiles_o * (uint32_t)a.tiles_t * (uint32_t)a.parts;

#pragma unroll 1
    for (uint32_t item = blockIdx.x; item < total; item += gridDim.x) {
        const uint32_t at = by_xcd(item, total), tiles = (uint32_t)(a.tiles_o * a.tiles_t);
        const int part = uniform(at / tiles);
        // tiles in groups of 8 rows of tiles
        const uint32_t t = at % tiles, per = 8 * (uint32_t)a.tiles_o, group = t / per, in_group = t - group * per;
        const uint32_t gm = (uint32_t)a.tiles_t - group * 8 < 8 ? (uint32_t)a.tiles_t - group * 8 : 8;
        const int tile_o = uniform(in_group / gm), tt = uniform(group * 8 + in_group % gm);
        const int64_t o0 = (int64_t)tile_o * BO, t0 = (int64_t)tt * BT;
        // the part's turns (they fit 32 bits: columns do)
        const int g0 = (int)(part * a.share), g1 = (int)((part + 1) * a.share < a.turns ? (part + 1) * a.share : a.turns);

        // this thread's chunks, from the tile's first row on: rows behind the last are
        // read from it, and not stored
        const char* const tw = a.w + o0 * a.wrow;
        const char* const tx = a.x + t0 * a.xrow;
        uint32_t pw[NW], px[NX];
        int cw = 0, cx = 0;
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            int row;
            chunk_of<RW>(j * T + tid, &row, &cw);
            const int64_t most = a.out - 1 - o0;
            pw[j] = (uint32_t)(row < most ? row : (int)most) * (uint32_t)a.wrow;
        }
#pragma unroll
        for (int j = 0; j < NX; ++j) {
            int row;
            chunk_of<RX>(j * T + tid, &row, &cx);
            const int64_t most = a.rows - 1 - t0;
            px[j] = (uint32_t)(row < most ? row : (int)most) * (uint32_t)a.xrow;
        }
        auto fetch = [&](auto BUF, int s) {
            constexpr int buf = decltype(BUF)::value;
            // columns behind the last are read from it: their exponents are 0
            const uint32_t bw = (uint32_t)(s * RW) + cw * 16, bx = (uint32_t)(s * RX) + cx * 16;
            const uint32_t lw = (uint32_t)a.wrow - 16, lx = (uint32_t)a.xrow - 16;
            const uint32_t ow = bw < lw ? bw : lw, ox = bx < lx ? bx : lx;
#pragma unroll
            for (int j = 0; j < NW; ++j) load_lds16(tw, pw[j] + ow, to, buf * SW + j * T * 16);
#pragma unroll
            for (int j = 0; j < NX; ++j) load_lds16(tx, px[j] + ox, to, STAGES * SW + buf * SX + j * T * 16);
        };
        // the row whose exponents this thread brings, 16 at a time: the weight's or x's, the
        // same for a wave
        const bool of_w = wave * 64 < BO;
        const uint8_t* const eb = of_w ? a.ws + o0 * a.sp : a.xs + t0 * a.sp;
        const int64_t erows = of_w ? a.out - o0 : a.rows - t0, ebytes = erows * a.sp;
        const int esize = ebytes < (1 << 30) ? (int)ebytes : 1 << 30, esp = (int)a.sp;  // a tile's are below 2^27
        const int erow = tid - (of_w ? 0 : BO), eat = (erow < erows ? erow : (int)erows - 1) * esp;
        // exponents of a turn to half h: directly, where rows are whole words of them and the
        // row has all 16, else by registers, where all loads are waited for
        auto fetch_exponents = [&](int turn, int half) {
            if (esp % 4 == 0 && turn * 16 + 16 <= esp) {
                load_lds16((const char*)eb, (uint32_t)(eat + turn * 16), to + (uint32_t)half, EXPS);
            } else {
                *(u32x4*)(lds + EXPS + half + tid * 16) = exponents16(eb, eat, turn * 16, esp, esize);
            }
        };

        f32x16 acc[MT][NT];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 16; ++k) acc[m][n][k] = 0.0f;

        typedef std::conditional_t<EXACT, u32x4, i32x8> Raw;
        Raw fw[4], fx[2][NT];
        bf16x8 dx[NT][2];  // decoded
        uint32_t ew[2][MT], ex[2][NT];
        auto operand = [&](int at, int u, int down, auto fmt) -> Raw {
            constexpr bool four = decltype(fmt)::value == kE2m1;
            if constexpr (EXACT) {
                if constexpr (four) {
                    const u32x2 h = *(const u32x2*)(lds + (at ^ (u * 16)) + down);
                    return u32x4{h.x, h.y, 0, 0};
                } else {
                    return *(const u32x4*)(lds + (at ^ (u * 32)) + down);
                }
            } else if constexpr (four) {  // chunk g of a unit's two
                const u32x4 q = *(const u32x4*)(lds + (at ^ (u * 32)) + down);
                return i32x8{(int)q.x, (int)q.y, (int)q.z, (int)q.w, 0, 0, 0, 0};
            } else {  // chunks g and 2 + g of a unit's four
                const u32x4 p = *(const u32x4*)(lds + at + down);
                const u32x4 q = *(const u32x4*)(lds + (at ^ 32) + down);
                return i32x8{(int)p.x, (int)p.y, (int)p.z, (int)p.w, (int)q.x, (int)q.y, (int)q.z, (int)q.w};
            }
        };
        // operands of step j of a turn
        auto read_w = [&](auto J) {
            constexpr int j = decltype(J)::value % STEPS, buf = j / ST % STAGES, i = j % ST;
            fw[j & 3] = operand(place_w, i / MT, buf * SW + (i % MT) * 32 * RW, std::integral_constant<int, FW>{});
        };
        auto read_x = [&](auto J) {
            constexpr int j = decltype(J)::value % STEPS, buf = j / ST % STAGES, u = j % ST / MT;
#pragma unroll
            for (int n = 0; n < NT; ++n)
                fx[j / MT & 1][n] = operand(place_x, u, buf * SX + n * 32 * RX, std::integral_constant<int, FX>{});
        };
        // exponents of 128 codes: a word of each row, moved so that a lane's blocks (g and
        // 2 + g) are in the bytes that the instructions select
        auto read_exponents = [&](auto Q, int half) {
            constexpr int q = decltype(Q)::value;
#pragma unroll
            for (int m = 0; m < MT; ++m) ew[q & 1][m] = *(const uint32_t*)(lds + scale_w + half + m * 512 + 4 * q);
#pragma unroll
            for (int n = 0; n < NT; ++n) ex[q & 1][n] = *(const uint32_t*)(lds + scale_x + half + n * 512 + 4 * q);
        };
        auto align_exponents = [&](auto Q) {
            constexpr int q = decltype(Q)::value;
            if constexpr (!EXACT) {
#pragma unroll
                for (int m = 0; m < MT; ++m) ew[q & 1][m] >>= 8 * g;
#pragma unroll
                for (int n = 0; n < NT; ++n) ex[q & 1][n] >>= 8 * g;
            }
        };
        auto multiply = [&](auto J) {
            constexpr int j = decltype(J)::value, m = j % MT, unit = j / MT;  // of the turn
            constexpr int q = unit * UNIT / 128 & 1, in = unit * UNIT % 128 / UNIT;
            if constexpr (EXACT) {
                if constexpr (m == 0) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) decode16<FX>(fx[unit & 1][n], scale_of((ex[q][n] >> (8 * in)) & 255), dx[n]);
                }
                bf16x8 dw[2];
                decode16<FW>(fw[j & 3], scale_of((ew[q][m] >> (8 * in)) & 255), dw);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(dw[h], dx[n][h], acc[m][n], 0, 0, 0);
            } else {
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    acc[m][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        fw[j & 3], fx[unit & 1][n], acc[m][n], FW == kE2m1 ? 4 : 0, FX == kE2m1 ? 4 : 0, in * 2, (int)ew[q][m],
                        in * 2, (int)ex[q][n]);
            }
            // keeps the step's matrix instructions here: nothing else orders them among
            // the loads and barriers of a turn
#pragma unroll
            for (int n = 0; n < NT; ++n) asm volatile("" : "+v"(acc[m][n]));
            __builtin_amdgcn_sched_barrier(0);
        };

        __syncthreads();  // the last item's LDS is free
        fetch_exponents(g0, 0);
        fetch(std::integral_constant<int, 0>{}, g0 * SPT);
        fetch(std::integral_constant<int, 1>{}, g0 * SPT + 1);
        fetch(std::integral_constant<int, 2>{}, g0 * SPT + 2);
        wait_loads<2 * LOADS>();
        __syncthreads();
        fetch(std::integral_constant<int, 3>{}, g0 * SPT + 3);
        read_exponents(std::integral_constant<int, 0>{}, 0);
        read_x(std::integral_constant<int, 0>{});
        read_w(std::integral_constant<int, 0>{});
        read_w(std::integral_constant<int, 1>{});
        int half = 0;  // where this turn's exponents lie
#pragma unroll 1
        for (int turn = g0; turn < g1; ++turn) {
            // behind the last turn the last exponents once more, which no product takes
            fetch_exponents(turn + 1 < g1 ? turn + 1 : turn, half ^ SCALES);
            auto steps = [&](auto self, auto J) {
                constexpr int j = decltype(J)::value, next = j + AHEAD;
                if constexpr (j < STEPS) {
                    if constexpr (next % ST == 0) {  // the first reads of a stage
                        constexpr int s = next / ST, code = s % SPT * BK;
                        wait_loads<2 * LOADS>();
                        __syncthreads();
                        fetch(std::integral_constant<int, (s + STAGES - 1) % STAGES>{}, turn * SPT + s + STAGES - 1);
                        read_x(std::integral_constant<int, next>{});
                        read_w(std::integral_constant<int, next>{});
                        if constexpr (code % 128 == 0)
                            read_exponents(std::integral_constant<int, code / 128>{}, s == SPT ? half ^ SCALES : half);
                    } else {
                        if constexpr (next % MT == 0) read_x(std::integral_constant<int, next>{});
                        read_w(std::integral_constant<int, next>{});
                    }
                    if constexpr (j * UNIT / MT % 128 == 0 && j % MT == 0)
                        align_exponents(std::integral_constant<int, j / MT * UNIT / 128>{});
                    multiply(J);
                    self(self, std::integral_constant<int, j + 1>{});
                }
            };
            steps(steps, std::integral_constant<int, 0>{});
            half ^= SCALES;
        }
        wait_loads<0>();  // the loads ahead, before their places are used

        // D: a lane has token lane & 31 and, four at a time, outputs (k / 4) * 8 + g * 4
        // on. The wave's results go through LDS, 32 tokens at a time (16-byte chunks
        // exchanged by the token), to be written as rows of neighbouring outputs.
        __syncthreads();
        float* const mine = a.parts > 1 ? a.part + (int64_t)part * a.rows * a.out : nullptr;
        char* const own = lds + wave * (WO * 32 * 4);
        constexpr int CH = WO / 4, LANES = WO / 8;  // chunks of a token, lanes of 8 outputs
        int ol = lane;  // opaque: addresses made from it are not kept in registers through the product
        asm volatile("" : "+v"(ol));
        const int rr = ol & 31, rg = ol >> 5;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int c = m * 8 + k * 2 + rg;
                    *(f32x4*)(own + rr * (WO * 4) + ((c ^ (rr & (CH - 1))) << 4)) =
                        f32x4{acc[m][n][4 * k], acc[m][n][4 * k + 1], acc[m][n][4 * k + 2], acc[m][n][4 * k + 3]};
                }
            wave_lds_order();
            __builtin_amdgcn_sched_barrier(0);
            const int64_t o = o0 + wo * WO + (ol % LANES) * 8;
#pragma unroll 1
            for (int k = 0; k < 32; k += 64 / LANES) {
                const int q = k + ol / LANES, c = (ol % LANES) * 2;
                const f32x4 lo = *(const f32x4*)(own + q * (WO * 4) + ((c ^ (q & (CH - 1))) << 4));
                const f32x4 hi = *(const f32x4*)(own + q * (WO * 4) + (((c + 1) ^ (q & (CH - 1))) << 4));
                const int64_t tok = t0 + wt * WT + n * 32 + q;
                if (tok >= a.rows || o >= a.out) continue;
                const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                put8(a, mine, tok, o, v);
            }
            wave_lds_order();
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

// Sums the parts, in order, eight neighbouring outputs a thread.
__global__ __launch_bounds__(kThreads) void linear_join_kernel(LinArgs a) {
    const int64_t eights = (a.out + 7) / 8, next = a.rows * a.out;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < a.rows * eights; i += (int64_t)gridDim.x * kThreads) {
        const int64_t t = i / eights, o = (i - t * eights) * 8;
        const int n = existing(a.out, o);
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int p = 0; p < a.parts; ++p) {
            float f[8];
            load_param8(a.part + p * next + t * a.out + o, kFp32, 0, n, 0.0f, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += f[e];
        }
        put8(a, nullptr, t, o, v);
    }
}

// -------------------------------------------------------------- few rows
// Up to 64 tokens: the weight's bytes count, and each goes from memory to the
// matrix instruction's registers once. A block of 8 waves takes 16 outputs; its
// waves take every 8th turn of 512 columns, in 4 steps whose loads are in flight
// at once, with a turn's exponents in one load, and are added in LDS. (Rows of codes too
// long for the tiled form's 32-bit offsets come here too, 64 tokens at a time.) One token
// by 4096x4096 of e4m3 takes 6.2 us (of e2m1 5.0 to 5.7), of which a launch alone is 3.6, by
// 32768x8192 46 to 51 us (5.4 to 6.0 TB/s; of e2m1 34 to 38).
struct Piece {  // a row's 128 codes, one lane's quarter
    u32x4 p, q;
};

template <int FMT, bool EXACT>
__device__ __forceinline__ Piece piece(const char* row, int64_t bytes, int64_t s, int g) {
    Piece v;
    auto within = [&](int64_t at, int n) { return at < bytes - n ? at : bytes - n; };
    if constexpr (FMT == kE2m1 && !EXACT) {
        v.p = *(const u32x4*)(row + within(s * 64 + g * 16, 16));
        v.q = u32x4{0, 0, 0, 0};
    } else if constexpr (FMT == kE2m1) {
        const u32x2 x = *(const u32x2*)(row + within(s * 64 + g * 8, 8)), y = *(const u32x2*)(row + within(s * 64 + 32 + g * 8, 8));
        v.p = u32x4{x.x, x.y, 0, 0};
        v.q = u32x4{y.x, y.y, 0, 0};
    } else {
        v.p = *(const u32x4*)(row + within(s * 128 + g * 16, 16));
        v.q = *(const u32x4*)(row + within(s * 128 + 64 + g * 16, 16));
    }
    return v;
}

// A lane's exponents of a row's turn, a byte for each of its 4 steps: of block g, or,
// where operands are decoded, of the blocks of its two pieces.
template <bool EXACT>
struct Exps {
    uint32_t p, q;
};
template <bool EXACT>
__device__ __forceinline__ Exps<EXACT> turn_exps(const uint8_t* exps, int64_t row, int64_t rows, int64_t sp, int64_t turn, int g) {
    const int64_t left = (rows - row) * sp;  // to the buffer's end
    const u32x4 v = exponents16(exps + row * sp, 0, (int)turn * 16, (int)sp, left < (1 << 30) ? (int)left : 1 << 30);
    auto column = [&](int b) {
        const uint32_t sel = 0x0c0c0400u + 0x0101u * (uint32_t)b;
        return __builtin_amdgcn_perm(v.y, v.x, sel) | __builtin_amdgcn_perm(v.w, v.z, sel) << 16;
    };
    return EXACT ? Exps<EXACT>{column(g / 2), column(2 + g / 2)} : Exps<EXACT>{column(g), 0};
}

template <int FW, int FX, bool EXACT, int NG>
__global__ __launch_bounds__(512) void linear_few_kernel(LinArgs a) {
    constexpr int U = NG == 1 ? 4 : 2;
    __shared__ f32x4 red[8][NG][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    for (int64_t item = blockIdx.x; item < (int64_t)a.tiles_o * a.tiles_t; item += gridDim.x) {
        const int64_t tt = item / a.tiles_o, t0 = tt * (NG * 16), o0 = (item - tt * a.tiles_o) * 16;
        const int64_t o = o0 + r < a.out ? o0 + r : a.out - 1;
        const char* const w = a.w + o * a.wrow;
        f32x4 acc[NG];
#pragma unroll
        for (int n = 0; n < NG; ++n) acc[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int64_t turn = wave; turn < a.turns; turn += 8) {
            const Exps<EXACT> ew = turn_exps<EXACT>(a.ws, o, a.out, a.sp, turn, g);
            int64_t t[NG];
            Exps<EXACT> ex[NG];
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                t[n] = t0 + n * 16 + r < a.rows ? t0 + n * 16 + r : a.rows - 1;
                ex[n] = turn_exps<EXACT>(a.xs, t[n], a.rows, a.sp, turn, g);
            }
            auto half = [&](auto U0) {
                constexpr int u0 = decltype(U0)::value;
                Piece fw[U], fx[U][NG];
#pragma unroll
                for (int u = 0; u < U; ++u) fw[u] = piece<FW, EXACT>(w, a.wrow, turn * 4 + u0 + u, g);
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int n = 0; n < NG; ++n) fx[u][n] = piece<FX, EXACT>(a.x + t[n] * a.xrow, a.xrow, turn * 4 + u0 + u, g);
                auto step = [&](auto UU) {
                    constexpr int u = decltype(UU)::value, k = u0 + u;  // of the turn
#pragma unroll
                    for (int n = 0; n < NG; ++n) {
                        const Piece &p = fw[u], &q = fx[u][n];
                        if constexpr (EXACT) {
                            bf16x8 x[2], y[2];
                            decode16<FW>(p.p, scale_of((ew.p >> (8 * k)) & 255), x);
                            decode16<FX>(q.p, scale_of((ex[n].p >> (8 * k)) & 255), y);
                            acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[0], y[0], acc[n], 0, 0, 0);
                            acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[1], y[1], acc[n], 0, 0, 0);
                            decode16<FW>(p.q, scale_of((ew.q >> (8 * k)) & 255), x);
                            decode16<FX>(q.q, scale_of((ex[n].q >> (8 * k)) & 255), y);
                            acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[0], y[0], acc[n], 0, 0, 0);
                            acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[1], y[1], acc[n], 0, 0, 0);
                        } else {
                            const i32x8 x = {(int)p.p.x, (int)p.p.y, (int)p.p.z, (int)p.p.w, (int)p.q.x, (int)p.q.y, (int)p.q.z, (int)p.q.w};
                            const i32x8 y = {(int)q.p.x, (int)q.p.y, (int)q.p.z, (int)q.p.w, (int)q.q.x, (int)q.q.y, (int)q.q.z, (int)q.q.w};
                            acc[n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc[n], FW == kE2m1 ? 4 : 0,
                                                                                      FX == kE2m1 ? 4 : 0, k, (int)ew.p, k, (int)ex[n].p);
                        }
                    }
                };
                step(std::integral_constant<int, 0>{});
                step(std::integral_constant<int, 1>{});
                if constexpr (U == 4) {
                    step(std::integral_constant<int, 2>{});
                    step(std::integral_constant<int, 3>{});
                }
            };
            half(std::integral_constant<int, 0>{});
            if constexpr (U == 2) half(std::integral_constant<int, 2>{});
        }
#pragma unroll
        for (int n = 0; n < NG; ++n) red[wave][n][lane] = acc[n];
        __syncthreads();
        // red[.][n][g * 16 + token]: outputs g * 4 on; two of them are eight neighbours
        for (int i = threadIdx.x; i < NG * 32; i += 512) {
            const int n = i / 32, l = (i & 15) + (i & 16) * 2;
            float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] += red[k][n][l][e];
                    v[4 + e] += red[k][n][l + 16][e];
                }
            const int64_t t = t0 + n * 16 + (l & 15);
            if (t < a.rows) put8(a, nullptr, t, o0 + (l >> 4) * 4, v);
        }
        __syncthreads();
    }
}

template <int FW, int FX, bool EXACT>
hipError_t run(LinArgs& a, const LinearCut& cut, hipStream_t stream) {
    if (cut.form == 0) {
        a.tiles_o = (int)((a.out + 15) / 16);
        a.tiles_t = (int)((a.rows + 63) / 64);
        const int grid = grid_for((int64_t)a.tiles_o * a.tiles_t, 512);
        if (a.rows <= 16)
            linear_few_kernel<FW, FX, EXACT, 1><<<grid, 512, 0, stream>>>(a);
        else if (a.rows <= 32)
            linear_few_kernel<FW, FX, EXACT, 2><<<grid, 512, 0, stream>>>(a);
        else
            linear_few_kernel<FW, FX, EXACT, 4><<<grid, 512, 0, stream>>>(a);
        return hipGetLastError();
    }
    const int tile = cut.form == 1 ? 128 : 256;
    a.tiles_o = (int)((a.out + tile - 1) / tile);
    a.tiles_t = (int)((a.rows + tile - 1) / tile);
    const int64_t total = (int64_t)a.tiles_o * a.tiles_t * a.parts, places = device_cu_count() * (cut.form == 1 ? 2 : 1);
    const int64_t blocks = total < places ? total : places;  // blocks walk over the tiles
    if (cut.form == 1)
        linear_kernel<FW, FX, EXACT, 128, 128, 64, 64><<<grid_for(blocks, 256), 256, 0, stream>>>(a);
    else
        linear_kernel<FW, FX, EXACT, 256, 256, 128, 64><<<grid_for(blocks, 512), 512, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.parts == 1) return e;
    const int64_t items = (a.rows * ((a.out + 7) / 8) + kThreads - 1) / kThreads;
    linear_join_kernel<<<grid_for(items, kThreads), kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear(const Linear& f, hipStream_t stream) {
    const bool w4 = f.w_format == ZR_CKPT_E2M1, x4 = f.x_format == ZR_CKPT_E2M1;
    const LinearKind kind = w4 && x4 ? (f.z_dt == ZR_FP32 ? kLinearFourWide : kLinearFour)
                                     : (f.z_dt == ZR_FP32 ? kLinearDecoded : kLinearScaled);
    const LinearCut cut = linear_cut(f.rows, f.out, f.in, kind);
    const int64_t pitch = ckpt_pitch(f.in);
    LinArgs a{};
    a.w = (const char*)f.w; a.x = (const char*)f.x;
    a.wrow = w4 ? pitch / 2 : pitch; a.xrow = x4 ? pitch / 2 : pitch;
    a.ws = (const uint8_t*)f.w + f.out * a.wrow;
    a.xs = (const uint8_t*)f.x + f.rows * a.xrow;
    a.sp = pitch / kCkptBlock;
    a.bias = f.bias; a.z = f.z; a.part = (float*)f.workspace;
    a.rows = f.rows; a.out = f.out; a.ld_z = f.ld_z;
    a.bias_dt = f.bias_dt; a.z_dt = f.z_dt; a.accumulate = f.accumulate;
    a.turns = cut.turns; a.share = cut.share; a.parts = cut.parts;
    if (w4 && x4) return run<kE2m1, kE2m1, false>(a, cut, stream);
    if (kind == kLinearDecoded) {
        if (w4) return run<kE2m1, kE4m3, true>(a, cut, stream);
        return x4 ? run<kE4m3, kE2m1, true>(a, cut, stream) : run<kE4m3, kE4m3, true>(a, cut, stream);
    }
    if (w4) return run<kE2m1, kE4m3, false>(a, cut, stream);
    return x4 ? run<kE4m3, kE2m1, false>(a, cut, stream) : run<kE4m3, kE4m3, false>(a, cut, stream);
}

}  // namespace zr
