// The 4-bit blocks' codec (e2m1: values 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
// negatives), beside the 8-bit ones of zr_ckpt.hpp: the same blocks of 32 columns
// and exponent bytes, with M = 6, and two codes to a byte, the even column in the
// low half. Held values are exact in bf16, as those are.
#pragma once

#include "zr_ckpt.hpp"

namespace zr {

constexpr int kE2m1 = ZR_CKPT_E2M1;

// Bytes of a row of codes.
template <int FMT>
__host__ __device__ __forceinline__ int64_t code_bytes(int64_t cols) {
    return FMT == kE2m1 ? ckpt_pitch(cols) / 2 : ckpt_pitch(cols);
}

// Exponent byte of a block whose largest magnitude has the fp32 bits `amax` (as
// ckpt_byte: the mantissa is held against M's, 1.5).
__device__ __forceinline__ uint32_t e2m1_byte(uint32_t amax) {
    if (amax >= 0x7F800000u) return kCkptNan;
    const int k = (int)((amax + 0x3FFFFFu) >> 23) - 2;
    return (uint32_t)(k < kCkptMinByte ? kCkptMinByte : k);
}

// Codes of 8 values of a block with exponent byte s, the first in the lowest bits.
// The conversion rounds to nearest even and keeps a zero's sign.
__device__ __forceinline__ uint32_t e2m1_encode8(const float f[8], uint32_t s) {
    const float inv = ckpt_inverse(s);
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = f[e] * inv;
    if (s == 253u) {  // 3.5 and more would round to 2^128
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __builtin_amdgcn_fmed3f(v[e], -3.0f, 3.0f);
    }
    uint32_t q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], 1.0f, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], 1.0f, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], 1.0f, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], 1.0f, 3);
    return s == kCkptNan ? 0u : q;
}

// The same of 8 bf16 values as they lie in memory: the conversion divides by the scale,
// and nothing is widened.
__device__ __forceinline__ uint32_t e2m1_encode8(const u32x4& w, uint32_t s) {
    if (s == 253u) {
        float f[8];
        widen8(Raw8<kBf16>{w}, f);
        return e2m1_encode8(f, s);
    }
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    auto pair = [](uint32_t a) { return __builtin_bit_cast(bf16x2, a); };
    const float scale = __uint_as_float(s << 23);
    uint32_t q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, pair(w.x), scale, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, pair(w.y), scale, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, pair(w.z), scale, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, pair(w.w), scale, 3);
    return s == kCkptNan ? 0u : q;
}

// Values of 8 codes of a block with scale 2^e.
__device__ __forceinline__ void e2m1_decode8(uint32_t q, float scale, float f[8]) {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 3);
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
    f[4] = c.x; f[5] = c.y; f[6] = d.x; f[7] = d.y;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= scale;
}

// Exponent byte of a block, by a format known at compile time.
template <int FMT>
__device__ __forceinline__ uint32_t format_byte(uint32_t amax) {
    return FMT == kE2m1 ? e2m1_byte(amax) : ckpt_byte(amax, FMT == kE4m3);
}

}  // namespace zr
