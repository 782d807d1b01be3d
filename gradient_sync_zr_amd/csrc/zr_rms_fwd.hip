// RMS norm, forward, with the residual's addition in front. Per row of n columns:
//     h    = x + r, rounded to the residual stream's type (h = x without r)
//     rstd = 1 / sqrt(sum h^2 / n + eps),  y = h * rstd * w
// in fp32 (waves' sums joined in fp64), of h as its later readers have it. One pass over the row's
// registers: blocks walk over the rows with the weight in registers and the next
// row's loads in flight while a row is summed and written. Rows over 16384
// columns are read twice (and h is then summed up twice).
//
// Memory bounds it: 16384x4096 bf16 with residual, h and y takes 91 to 92 us (5.9 TB/s).
// With y packed (8192x4096 from fp32 x, h written) 47 us. A row is summed once by
// its wave or block, so the shuffles and the one barrier of a row are what the next
// row's loads cover.
#include <hip/hip_runtime.h>

#include "zr_norm.hpp"

namespace zr {
namespace {

struct RmsFwdArgs {
    const void *x, *w;
    const char* res;
    char *h, *y, *ckpt_h, *ckpt_y;
    float* rstd;
    int64_t rows, cols, ld_x, ld_res, ld_h, ld_y;
    int param_dt, h_dt, y_dt, e4m3;
    float eps;
};

// Sum over the TPR lanes of a row, those of its waves in fp64. With the formula's own
// roundings behind it that makes rstd the same as that of sums in another order in
// three rows of four or more (with a reciprocal square root in one of two), and its
// last bit moves one value in 10^5 over the border between two in bf16. red: a float per
// wave, free again once every wave has passed a later barrier.
template <int TPR>
__device__ __forceinline__ double row_sum64(float v, float* red) {
    v = wave_sum<(TPR < 64 ? TPR : 64)>(v);
    if constexpr (TPR <= 64) return v;
    constexpr int W = TPR / 64;
    const int wave = threadIdx.x / 64, first = wave / W * W;
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < W; ++w) s += (double)red[first + w];
    return s;
}
__device__ __forceinline__ float rstd_of(double sum, double inv_n, float eps) {
    return 1.0f / sqrtf((float)(sum * inv_n) + eps);
}

// A vector of bf16 or fp32 by a type known at run time, bf16 in the first half.
__device__ __forceinline__ Raw8<kFp32> fetch_as(const char* row, int dt, int c, int n) {
    Raw8<kFp32> r;
    if (dt == kBf16) {
        r.a = __builtin_bit_cast(f32x4, fetch8<kBf16, true>({row, nullptr}, c, n).v);
        r.b = r.a;
    } else {
        r = fetch8<kFp32, true>({row, nullptr}, c, n);
    }
    return r;
}
__device__ __forceinline__ void widen_as(Raw8<kFp32>& r, int dt, int c, int n, float f[8]) {
    if (dt == kBf16) {
        Raw8<kBf16> b{__builtin_bit_cast(u32x4, r.a)};
        settle8(b, c, n);
        widen8(b, f);
    } else {
        settle8(r, c, n);
        widen8(r, f);
    }
}

// Rounds a vector to bf16, as stored.
__device__ __forceinline__ void as_bf16(float f[8]) {
    const u32x4 v = {bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7])};
    widen8(Raw8<kBf16>{v}, f);
}

__device__ __forceinline__ void put_block(const RmsFwdArgs& a, char* ckpt, int64_t row, int64_t pitch, int c,
                                          const float f[8]) {
    ckpt_store8(ckpt + row * pitch, (uint8_t*)ckpt + a.rows * pitch + row * (pitch / kCkptBlock), c, f, block_amax(f),
                a.e4m3 != 0);
}

// x's vector becomes h's, which is written.
__device__ __forceinline__ void add_residual(const RmsFwdArgs& a, int64_t row, int c, int n, Raw8<kFp32>& r, float f[8]) {
    float o[8];
    widen_as(r, a.h_dt, c, n, o);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] += o[e];
    if (a.h_dt == kBf16) as_bf16(f);
    if (a.h && n > 0) store8<true>(a.h + row * a.ld_h * (a.h_dt == kBf16 ? 2 : 4), a.h_dt, c, n, f);
}

// y of h's vector, then its checkpoint, of y as its readers have it.
__device__ __forceinline__ void put_rms(const RmsFwdArgs& a, int64_t row, int64_t pitch, int c, int n, float f[8],
                                        const float w[8], float rstd) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = f[e] * rstd * w[e];
    if (a.y && n > 0) store8<true>(a.y + row * a.ld_y * (a.y_dt == kBf16 ? 2 : 4), a.y_dt, c, n, f);
    if (a.ckpt_y) {
        if (n < 8) keep_first(f, n);
        if (a.y_dt == kBf16) as_bf16(f);
        put_block(a, a.ckpt_y, row, pitch, c, f);
    }
}

template <int XD, int TPR, int NV>
__global__ __launch_bounds__(norm_block(TPR)) void rms_fwd_kernel(RmsFwdArgs a) {
    constexpr int B = norm_block(TPR), G = B / TPR;
    static_assert(TPR <= 64 || G == 1, "barriers need one row per block");
    __shared__ float red[2][B / 64];
    const int lane = threadIdx.x % TPR, group = row_group<TPR>();
    const int64_t pitch = ckpt_pitch(a.cols);
    const double inv_n = 1.0 / (double)a.cols;
    float w[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (v * TPR + lane) * 8;
        load_param8(a.w, a.param_dt, c, existing(a.cols, c), 1.0f, w[v]);
    }
    Raw8<XD> raw[NV];
    Raw8<kFp32> res[NV];
    auto fetch = [&](int64_t row) {
        const RowPtr p = row_at<XD>(a.x, a.ld_x, a.rows, a.cols, row);
        const char* q = a.res + row * a.ld_res * (a.h_dt == kBf16 ? 2 : 4);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8, n = existing(a.cols, c);
            raw[v] = fetch8<XD, true>(p, c, n);
            if (a.res) res[v] = fetch_as(q, a.h_dt, c, n);
        }
    };
    int parity = 0;
    const int64_t first = (int64_t)blockIdx.x * G + group, step = (int64_t)gridDim.x * G;
    if (first < a.rows) fetch(first);
    for (int64_t row = first; row < a.rows; row += step) {
        float f[NV][8];
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8, n = existing(a.cols, c);
            settle8(raw[v], c, n);
            widen8(raw[v], f[v]);
            if (XD > kFp32 && n < 8) keep_first(f[v], n);
            if (a.res) add_residual(a, row, c, n, res[v], f[v]);
#pragma unroll
            for (int e = 0; e < 8; ++e) s = __builtin_fmaf(f[v][e], f[v][e], s);
        }
        if (row + step < a.rows) fetch(row + step);
        // two sets of slots in turn: a set is written again only after the other
        // set's barrier, which every reader of the first has passed
        const float rstd = rstd_of(row_sum64<TPR>(s, red[parity]), inv_n, a.eps);
        parity ^= 1;
        if (lane == 0 && a.rstd) a.rstd[row] = rstd;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8;
            if (c >= pitch) continue;
            if (a.ckpt_h) put_block(a, a.ckpt_h, row, pitch, c, f[v]);
            put_rms(a, row, pitch, c, existing(a.cols, c), f[v], w[v], rstd);
        }
    }
}

// Rows of any width, one per block of 1024, read once per pass. h may take x's or
// the residual's place: the second pass then reads h.
template <int XD>
__global__ __launch_bounds__(1024) void rms_fwd_wide_kernel(RmsFwdArgs a) {
    __shared__ float red[2][16];
    int parity = 0;
    const int64_t pitch = ckpt_pitch(a.cols);
    const int es = a.h_dt == kBf16 ? 2 : 4;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const RowPtr p = row_at<XD>(a.x, a.ld_x, a.rows, a.cols, row);
        const char* const q = a.res + row * a.ld_res * es;
        char* const h = a.h + row * a.ld_h * es;
        auto vector = [&](int64_t c, int n, float f[8]) {  // x, or x + r
            widen8(load8<XD>(p, (int)c, n), f);
            if (n < 8) keep_first(f, n);
            if (a.res) {
                float o[8];
                load_param8(q, a.h_dt, (int)c, n, 0.0f, o);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] += o[e];
                if (a.h_dt == kBf16) as_bf16(f);
            }
        };
        float s = 0.0f;
        for (int64_t c = threadIdx.x * 8; c < pitch; c += 8192) {
            const int n = existing(a.cols, c);
            float f[8];
            vector(c, n, f);
            if (a.res && a.h && n > 0) store8<false>(h, a.h_dt, (int)c, n, f);
            if (a.ckpt_h) put_block(a, a.ckpt_h, row, pitch, (int)c, f);
            float t = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) t = __builtin_fmaf(f[e], f[e], t);
            s += t;
        }
        const float rstd = rstd_of(row_sum64<1024>(s, red[parity]), 1.0 / (double)a.cols, a.eps);
        parity ^= 1;
        if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
        for (int64_t c = threadIdx.x * 8; c < pitch; c += 8192) {
            const int n = existing(a.cols, c);
            float f[8], w[8];
            if (a.res && a.h)  // this thread wrote it
                load_param8(h, a.h_dt, (int)c, n, 0.0f, f);
            else
                vector(c, n, f);
            load_param8(a.w, a.param_dt, (int)c, n, 1.0f, w);
            put_rms(a, row, pitch, (int)c, n, f, w, rstd);
        }
    }
}

template <int XD, int TPR, int NV>
hipError_t fwd_run(const RmsFwdArgs& a, hipStream_t stream) {
    constexpr int B = norm_block(TPR), G = B / TPR;
    const int64_t groups = (a.rows + G - 1) / G, most = 1024 * kThreads / B;
    rms_fwd_kernel<XD, TPR, NV><<<grid_for(groups < most ? groups : most, B), B, 0, stream>>>(a);
    return hipGetLastError();
}

template <int XD>
hipError_t fwd_pick(const RmsFwdArgs& a, hipStream_t stream) {
    const int64_t n = a.cols;
    if (n <= 128) return fwd_run<XD, 16, 1>(a, stream);
    if (n <= 512) return fwd_run<XD, 64, 1>(a, stream);
    if (n <= 1024) return fwd_run<XD, 64, 2>(a, stream);
    if (n <= 2048) return fwd_run<XD, 256, 1>(a, stream);
    if (n <= 4096) return fwd_run<XD, 256, 2>(a, stream);
    if (n <= 8192) return fwd_run<XD, 512, 2>(a, stream);
    if (n <= 12288) return fwd_run<XD, 512, 3>(a, stream);
    if (n <= 16384) return fwd_run<XD, 512, 4>(a, stream);
    rms_fwd_wide_kernel<XD><<<grid_for(a.rows, 1024), 1024, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm_fwd(const RmsFwd& f, hipStream_t stream) {
    RmsFwdArgs a{};
    a.x = f.x; a.w = f.weight; a.res = (const char*)f.residual;
    a.h = (char*)f.h; a.y = (char*)f.y; a.ckpt_h = (char*)f.ckpt_h; a.ckpt_y = (char*)f.ckpt_y;
    a.rstd = f.rstd;
    a.rows = f.rows; a.cols = f.cols; a.ld_x = f.ld_x; a.ld_res = f.ld_res; a.ld_h = f.ld_h; a.ld_y = f.ld_y;
    a.param_dt = f.param_dt; a.h_dt = f.h_dt; a.y_dt = f.y_dt; a.e4m3 = f.ckpt_format == ZR_CKPT_E4M3;
    a.eps = f.eps;
    switch (f.x_dt) {
        case ZR_BF16: return fwd_pick<kBf16>(a, stream);
        case ZR_FP32: return fwd_pick<kFp32>(a, stream);
        case ZR_CKPT_E4M3: return fwd_pick<kE4m3>(a, stream);
        default: return fwd_pick<kInt8>(a, stream);
    }
}

}  // namespace zr
