// Device codec of the 8-bit activation checkpoints, and the row-vector loads
// and stores that the norm and checkpoint kernels share.
//
// A checkpoint of a rows x cols tensor is cut into blocks of 32 columns. A
// block is one exponent byte s = 127 + e and 32 codes; a code stands for its
// e4m3 or int8 value times 2^e. e is the smallest integer >= -124 with
// max|x| <= M * 2^e, M = 448 (e4m3) or 127 (int8), so no code overflows, the
// scaling by 2^-e is exact in fp32, and a code is one rounding to nearest
// even of the true value. A power-of-two scale also makes every held value
// exact in bf16 (at most 7 significant bits; at e >= -124 the smallest step,
// 2^-9 * 2^e, is not below bf16's 2^-133), so a matrix product can take the
// decoded values as bf16 operands without a further rounding.
//
// A block that holds a NaN or an infinity has s = 255 and zero codes, and
// decodes to NaN throughout (0 * infinity). A block whose rounding would pass
// the largest fp32 (e = 120 for e4m3, 122 for int8) keeps its codes at the
// largest finite value below 2^128 instead.
#pragma once

#include "zr.h"
#include "zr_device.hpp"

namespace zr {

constexpr int kCkptBlock = 32;     // columns per block
constexpr int kCkptMinByte = 3;    // 127 - 124
constexpr uint32_t kCkptNan = 255; // exponent byte of a block that is not finite

// Bytes per row of codes; a row of exponents has pitch / 32.
__host__ __device__ __forceinline__ int64_t ckpt_pitch(int64_t cols) {
    return (cols + kCkptBlock - 1) / kCkptBlock * kCkptBlock;
}

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
// The same vectors at element alignment: rows of any stride and base are read
// and written with wide accesses (gfx950 allows them at any alignment).
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));

// 16 bytes of bf16 or fp32 elements at the elements' alignment; NT: past the
// caches. (A template over these types would drop their alignment.)
template <bool NT>
__device__ __forceinline__ u32x4 ld16(const uint16_t* p) {
    const u32x4_a2* q = (const u32x4_a2*)p;
    return NT ? (u32x4)__builtin_nontemporal_load(q) : (u32x4)*q;
}
template <bool NT>
__device__ __forceinline__ f32x4 ld32(const float* p) {
    const f32x4_a4* q = (const f32x4_a4*)p;
    return NT ? (f32x4)__builtin_nontemporal_load(q) : (f32x4)*q;
}
template <bool NT>
__device__ __forceinline__ void st16(uint16_t* p, u32x4 v) {
    if constexpr (NT)
        __builtin_nontemporal_store(v, (u32x4_a2*)p);
    else
        *(u32x4_a2*)p = v;
}
template <bool NT>
__device__ __forceinline__ void st32(float* p, f32x4 v) {
    if constexpr (NT)
        __builtin_nontemporal_store(v, (f32x4_a4*)p);
    else
        *(f32x4_a4*)p = v;
}

// Formats and sources as the kernels' template arguments (zr_dtype values).
constexpr int kBf16 = ZR_BF16, kFp32 = ZR_FP32, kE4m3 = ZR_CKPT_E4M3, kInt8 = ZR_CKPT_INT8;

// Exponent byte of a block whose largest magnitude has the fp32 bits `amax`.
// Adding all mantissa bits above M's carries into the exponent exactly when
// the magnitude's mantissa is larger than M's (1.75 or 127/64).
__device__ __forceinline__ uint32_t ckpt_byte(uint32_t amax, bool e4m3) {
    if (amax >= 0x7F800000u) return kCkptNan;
    const int k = e4m3 ? (int)((amax + 0x1FFFFFu) >> 23) - 8 : (int)((amax + 0x01FFFFu) >> 23) - 6;
    return (uint32_t)(k < kCkptMinByte ? kCkptMinByte : k);
}

// 2^-e and 2^e of an exponent byte (kCkptNan: 0 and infinity).
__device__ __forceinline__ float ckpt_inverse(uint32_t s) {
    return s == kCkptNan ? 0.0f : __uint_as_float((254u - s) << 23);
}
__device__ __forceinline__ float ckpt_scale(uint32_t s) {
    return __uint_as_float(s == 0 ? 0x00400000u : s << 23);
}

// Four bytes, the lowest of each word.
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(d, c, 0x0c0c0400u);
    return lo | (hi << 16);
}

// Codes of 8 values of a block with exponent byte s.
__device__ __forceinline__ u32x2 ckpt_encode8(const float f[8], uint32_t s, bool e4m3) {
    const float inv = ckpt_inverse(s);
    float v[8];
    u32x2 q;
    if (e4m3) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = f[e] * inv;
        if (s == 247u) {  // 248 and more would round to 2^128
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __builtin_amdgcn_fmed3f(v[e], -240.0f, 240.0f);
        }
        int a = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
        a = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], a, true);
        int b = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
        b = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], b, true);
        q = u32x2{(uint32_t)a, (uint32_t)b};
    } else {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = f[e] * inv;
        if (s == 249u) {  // 63.5 and more would round to 2^128
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __builtin_amdgcn_fmed3f(v[e], -63.0f, 63.0f);
        }
        // adding 1.5 * 2^23 rounds to an integer (to nearest even) whose two's
        // complement is then the low byte
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w[e] = __float_as_uint(__fadd_rn(v[e], 12582912.0f));
        q = u32x2{low_bytes(w[0], w[1], w[2], w[3]), low_bytes(w[4], w[5], w[6], w[7])};
    }
    if (s == kCkptNan) q = u32x2{0, 0};
    return q;
}

// 8 codes as the values they have at scale 1.
template <int FMT>
__device__ __forceinline__ void ckpt_codes8(const u32x2& q, float f[8]) {
    if constexpr (FMT == kE4m3) {
        const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(q.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(q.x, true);
        const f32x2 c = __builtin_amdgcn_cvt_pk_f32_fp8(q.y, false), d = __builtin_amdgcn_cvt_pk_f32_fp8(q.y, true);
        f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
        f[4] = c.x; f[5] = c.y; f[6] = d.x; f[7] = d.y;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = (float)(int)(int8_t)((e < 4 ? q.x : q.y) >> (8 * (e & 3)));
    }
}

// Values of 8 codes of a block with scale 2^e.
template <int FMT>
__device__ __forceinline__ void ckpt_decode8(const u32x2& q, float scale, float f[8]) {
    ckpt_codes8<FMT>(q, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= scale;
}

// Two values rounded to bf16 (nearest even; a NaN stays one), the first in the
// low half: one v_cvt_pk_bf16_f32.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    const bf16x2 r = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, r);
}

// ------------------------------------------------------------ row vectors
// A lane's vector is 8 consecutive columns; 4 lanes hold a block.
template <int DT>
struct Raw8 {};
template <>
struct Raw8<kBf16> {
    u32x4 v;
};
template <>
struct Raw8<kFp32> {
    f32x4 a, b;
};
template <>
struct Raw8<kE4m3> {
    u32x2 q;
    uint32_t s;
};
template <>
struct Raw8<kInt8> {
    u32x2 q;
    uint32_t s;
};

// A row source: `row` is the row's first element (or code), `scales` its
// first exponent byte (checkpoints only).
struct RowPtr {
    const char* row;
    const uint8_t* scales;
};

// base: first element of a strided tensor, or a checkpoint buffer.
template <int DT>
__device__ __forceinline__ RowPtr row_at(const void* base, int64_t ld, int64_t rows, int64_t cols, int64_t row) {
    const char* p = (const char*)base;
    if constexpr (DT == kBf16) return {p + row * ld * 2, nullptr};
    if constexpr (DT == kFp32) return {p + row * ld * 4, nullptr};
    const int64_t pitch = ckpt_pitch(cols);
    return {p + row * pitch, (const uint8_t*)p + rows * pitch + row * (pitch / kCkptBlock)};
}

// The 128 bits behind the first `bits` of v, zeros after them (all from 128 on).
__device__ __forceinline__ u32x4 behind(const u32x4& v, int bits) {
    uint64_t lo = ((uint64_t)v.y << 32) | v.x, hi = ((uint64_t)v.w << 32) | v.z;
    if (bits >= 64) {
        lo = hi;
        hi = 0;
    }
    const int by = bits & 63;
    if (by) lo = (lo >> by) | (hi << (64 - by));
    hi >>= by;
    return bits >= 128 ? u32x4{0, 0, 0, 0} : u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// Loads the vector at column c (a multiple of 8) of which n = clamp(cols - c,
// 0, 8) elements exist. A row's last, short vector is read 8 - n columns early,
// as a whole one, and settle8 moves it into place: single elements, put together
// behind a branch, would be waited for at the load (rows of 4095 columns took
// 1.6 times as long forward and twice backward as of 4096). Only rows of less
// than 8 columns are read by the element.
//
// NT: a stream, read once, past the caches (as the stores of streams are): pack
// and unpack of 65536x4096 bf16 took 273 us with both, 300 without. Codes are read
// through them (16384x4096 forward from e4m3: 47 us, past them 50).
template <int DT, bool NT>
__device__ __forceinline__ Raw8<DT> fetch8(const RowPtr& p, int c, int n) {
    Raw8<DT> r;
    if constexpr (DT == kBf16) {
        r.v = u32x4{0, 0, 0, 0};
        if (n > 0 && c + n >= 8) {
            r.v = ld16<NT>((const uint16_t*)p.row + c - (8 - n));
        } else if (n > 0) {
            const uint16_t* s = (const uint16_t*)p.row;
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < n) w[e >> 1] |= (uint32_t)s[e] << (16 * (e & 1));
            r.v = u32x4{w[0], w[1], w[2], w[3]};
        }
    } else if constexpr (DT == kFp32) {
        r.a = r.b = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (n > 0 && c + n >= 8) {
            const float* s = (const float*)p.row + c - (8 - n);
            r.a = ld32<NT>(s);
            r.b = ld32<NT>(s + 4);
        } else if (n > 0) {
            const float* s = (const float*)p.row;
            float w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < n) w[e] = s[e];
            r.a = f32x4{w[0], w[1], w[2], w[3]};
            r.b = f32x4{w[4], w[5], w[6], w[7]};
        }
    } else {
        if (n > 0) {
            r.q = *(const u32x2*)(p.row + c);
            r.s = p.scales[c / kCkptBlock];
        } else {
            r.q = u32x2{0, 0};
            r.s = 127;
        }
    }
    return r;
}

// Moves what fetch8 read to its place: the n elements first, zeros behind them
// (a checkpoint's padding is zero by itself, NaN in a block that is not finite).
template <int DT>
__device__ __forceinline__ void settle8(Raw8<DT>& r, int c, int n) {
    if (n == 8 || c + n < 8) return;
    if constexpr (DT == kBf16) {
        r.v = behind(r.v, (8 - n) * 16);
    } else if constexpr (DT == kFp32) {
        const int k = 8 - n;
        float t[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
        for (int by = 4; by >= 1; by /= 2)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (k & by) t[e] = e + by < 8 ? t[e + by] : 0.0f;
        r.a = f32x4{t[0], t[1], t[2], t[3]};  // n == 0: zeros were fetched
        r.b = f32x4{t[4], t[5], t[6], t[7]};
    }
}

// Both, for values that are used at once.
template <int DT>
__device__ __forceinline__ Raw8<DT> load8(const RowPtr& p, int c, int n) {
    Raw8<DT> r = fetch8<DT, false>(p, c, n);
    settle8(r, c, n);
    return r;
}

__device__ __forceinline__ void widen8(const Raw8<kBf16>& r, float f[8]) {
    const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[2 * e] = __uint_as_float(w[e] << 16);
        f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void widen8(const Raw8<kFp32>& r, float f[8]) {
    f[0] = r.a.x; f[1] = r.a.y; f[2] = r.a.z; f[3] = r.a.w;
    f[4] = r.b.x; f[5] = r.b.y; f[6] = r.b.z; f[7] = r.b.w;
}
__device__ __forceinline__ void widen8(const Raw8<kE4m3>& r, float f[8]) {
    ckpt_decode8<kE4m3>(r.q, ckpt_scale(r.s), f);
}
__device__ __forceinline__ void widen8(const Raw8<kInt8>& r, float f[8]) {
    ckpt_decode8<kInt8>(r.q, ckpt_scale(r.s), f);
}

// Elements of the vector that exist; zero behind them.
__device__ __forceinline__ void keep_first(float f[8], int n) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = e < n ? f[e] : 0.0f;
}

// The first n values rounded to dt (ZR_BF16 or ZR_FP32) at column c of a row.
template <bool NT>
__device__ __forceinline__ void store8(char* row, int dt, int c, int n, const float f[8]) {
    if (dt == kBf16) {
        uint16_t* p = (uint16_t*)row + c;
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = bf16_pair(f[2 * e], f[2 * e + 1]);
        if (n == 8) {
            st16<NT>(p, u32x4{w[0], w[1], w[2], w[3]});
        } else {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < n) p[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        }
    } else {
        float* p = (float*)row + c;
        if (n == 8) {
            st32<NT>(p, f32x4{f[0], f[1], f[2], f[3]});
            st32<NT>(p + 4, f32x4{f[4], f[5], f[6], f[7]});
        } else {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < n) p[e] = f[e];
        }
    }
}

// Eight parameters (a weight's or a bias's) from column c on; `none` where
// the pointer is null or the column does not exist.
__device__ __forceinline__ void load_param8(const void* p, int dt, int c, int n, float none, float f[8]) {
    if (!p) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = none;
    } else if (dt == kBf16) {
        widen8(load8<kBf16>({(const char*)p, nullptr}, c, n), f);
    } else {
        widen8(load8<kFp32>({(const char*)p, nullptr}, c, n), f);
    }
}

// A sum to an element of a gradient.
__device__ __forceinline__ void put_grad(void* p, int64_t at, float v, int grad_dt, bool add) {
    if (grad_dt == kBf16) {
        uint16_t* q = (uint16_t*)p + at;
        store_elem(q, add ? load_elem(q) + v : v);
    } else {
        float* q = (float*)p + at;
        store_elem(q, add ? load_elem(q) + v : v);
    }
}

// ------------------------------------------------------------- reductions
// Sums over the lanes of a row within a wave: DPP steps inside 16 lanes, then
// two exchanges across the wave.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
    const int o = __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true);
    return v + __int_as_float(o);
}
template <int LANES>
__device__ __forceinline__ float wave_sum(float v) {
    v = dpp_add<0xB1>(v);   // lane ^ 1
    v = dpp_add<0x4E>(v);   // lane ^ 2
    v = dpp_add<0x141>(v);  // mirrored within 8
    v = dpp_add<0x140>(v);  // mirrored within 16
    if constexpr (LANES >= 64) {
        // swaps of 16 and 32 lanes leave a lane's own and its partner's value
        auto both = [](auto r) { return __uint_as_float(r[0]) + __uint_as_float(r[1]); };
        v = both(__builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false));
        v = both(__builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false));
    }
    return v;
}

// The largest of m over the 4 lanes of a block.
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
    uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, true);
    m = o > m ? o : m;
    o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, true);
    return o > m ? o : m;
}

// Largest magnitude (fp32 bits) of a block, of fp32 values or of bf16 pairs
// (two at a time); a NaN is larger than all else.
__device__ __forceinline__ uint32_t block_amax(const float f[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t b = __float_as_uint(f[e]) & 0x7FFFFFFFu;
        m = b > m ? b : m;
    }
    return block_max(m);
}
__device__ __forceinline__ uint32_t block_amax(const u32x4& w) {
    auto pair = [](uint32_t a) { return __builtin_bit_cast(u16x2, a & 0x7FFF7FFFu); };
    const u16x2 m = __builtin_elementwise_max(__builtin_elementwise_max(pair(w.x), pair(w.y)),
                                              __builtin_elementwise_max(pair(w.z), pair(w.w)));
    return block_max(m.x > m.y ? m.x : m.y) << 16;
}

// Encodes a lane's vector, of largest magnitude amax in its block, at column c
// (< pitch; the block's 4 lanes are all here) of a checkpoint row; values
// behind the row's end must be zero.
__device__ __forceinline__ void ckpt_store8(char* codes, uint8_t* scales, int c, const float f[8], uint32_t amax,
                                            bool e4m3) {
    const uint32_t s = ckpt_byte(amax, e4m3);
    st<true>((u32x2*)(codes + c), ckpt_encode8(f, s, e4m3));
    if ((c & (kCkptBlock - 1)) == 0) scales[c / kCkptBlock] = (uint8_t)s;
}

}  // namespace zr
