// Layer norm, forward, over rows of activations or of their 8-bit checkpoints.
// Per row of n columns:
//     mean = sum x / n,  rstd = 1 / sqrt(sum (x - mean)^2 / n + eps)
//     y    = (x - mean) * rstd * w + b
// Mean and variance come from the row's registers in two passes (no
// cancellation), all in fp32. Blocks walk over the rows with the weight and
// bias in registers and the next row's loads in flight while a row is reduced
// and written. Of rows over 16384 columns the fp32 copy does not fit beside the
// weights: they are read from memory in each of three passes (4096x20000 bf16 100
// us, 3.3 TB/s).
//
// Bound by memory, and by the arithmetic of checkpoints: 16384x4096 bf16 takes 48
// to 50 us (5.4 TB/s; 86 before the next row's loads were in flight and the weights
// kept), 64 with x's checkpoint, 36 to 42 from an e4m3 checkpoint (4.8 to 5.7 TB/s;
// 45 while every vector was masked by the element and lanes 16 and 32 apart were
// added through LDS), 46 from one checkpoint to another (3.0 TB/s: decoding and
// encoding); from fp32 72 us, 87 with x's checkpoint. 24576x11008 179 us (6.0 TB/s,
// 201 so), 154 (216) from e4m3, and 343 with the checkpoint of y too: there three
// vectors a lane take 156 to 158 registers, one block of 512 a CU, whose waves are
// too few to hide the encoding. A wave's own mean and squares, joined with one
// barrier a row, instead of two passes with two: 43 us where they took 40, as the
// vector instructions count, not the barriers. Two vectors of 8 columns a lane
// measured best: with one (512 lanes a row) 16384x4096 took 59 us for 52; and 1024
// blocks of 256 (512 of 512), which up to 8192 columns are what the chip holds at
// once (2048: 56). Beyond, from bf16 and fp32, it holds half of them, and they go in
// two rounds.
#include <hip/hip_runtime.h>

#include "zr_norm.hpp"

namespace zr {
namespace {

struct FwdArgs {
    const void *x, *w, *b;
    char *y, *ckpt_x, *ckpt_y;
    float *mean, *rstd;
    int64_t rows, cols, ld_x, ld_y;
    int param_dt, y_dt, e4m3;
    float eps;
};

__device__ __forceinline__ void put_ckpt(const FwdArgs& a, char* ckpt, int64_t row, int64_t pitch, int c,
                                         const float f[8], uint32_t amax) {
    ckpt_store8(ckpt + row * pitch, (uint8_t*)ckpt + a.rows * pitch + row * (pitch / kCkptBlock), c, f, amax,
                a.e4m3 != 0);
}

// One vector of the output at column c < pitch, of the centred row: y rounded
// to its type, then its checkpoint, of y as its readers have it.
__device__ __forceinline__ void put_y(const FwdArgs& a, int64_t row, int64_t pitch, int c, int n, float f[8],
                                      const float w[8], const float b[8], float rstd) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = __builtin_fmaf(f[e] * rstd, w[e], b[e]);
    if (a.y && n > 0) store8<true>(a.y + row * a.ld_y * (a.y_dt == kBf16 ? 2 : 4), a.y_dt, c, n, f);
    if (a.ckpt_y) {
        if (a.cols & 7) keep_first(f, n);
        if (n == 0) keep_first(f, 0);
        uint32_t amax;
        if (a.y_dt == kBf16) {
            const u32x4 h = {bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7])};
            widen8(Raw8<kBf16>{h}, f);
            amax = block_amax(h);
        } else {
            amax = block_amax(f);
        }
        put_ckpt(a, a.ckpt_y, row, pitch, c, f, amax);
    }
}

template <int XD, int TPR, int NV>
__global__ __launch_bounds__(norm_block(TPR)) void fwd_kernel(FwdArgs a) {
    constexpr int B = norm_block(TPR), G = B / TPR;
    __shared__ float red[2][B / 64][1];
    const int lane = threadIdx.x % TPR, group = row_group<TPR>();
    const int64_t pitch = ckpt_pitch(a.cols);
    const float inv_n = 1.0f / (float)a.cols;
    // the same for all threads: masks of single elements are stepped over, not
    // issued, where every vector is whole or absent
    const bool ragged = (a.cols & 7) != 0;
    float w[NV][8], b[NV][8];  // read again for each row instead, 24576x11008 took 354 us for 217
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (v * TPR + lane) * 8, n = existing(a.cols, c);
        load_param8(a.w, a.param_dt, c, n, 1.0f, w[v]);
        load_param8(a.b, a.param_dt, c, n, 0.0f, b[v]);
    }
    Raw8<XD> raw[NV];
    auto fetch = [&](int64_t row) {
        const RowPtr p = row_at<XD>(a.x, a.ld_x, a.rows, a.cols, row);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8;
            raw[v] = fetch8<XD, true>(p, c, existing(a.cols, c));
        }
    };
    const int64_t first = (int64_t)blockIdx.x * G + group, step = (int64_t)gridDim.x * G;
    if (first < a.rows) fetch(first);
    // rows of more than a wave: one per block and turn, so the block's threads
    // leave the loop together
    for (int64_t row = first; row < a.rows; row += step) {
        float f[NV][8];
        float s[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8, n = existing(a.cols, c);
            if (ragged) settle8(raw[v], c, n);
            widen8(raw[v], f[v]);
            if (XD > kFp32 && ragged) keep_first(f[v], n);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[0] += f[v][e];
        }
        if (row + step < a.rows) fetch(row + step);
        row_sums<TPR>(s, red[0]);
        const float mean = s[0] * inv_n;
        s[0] = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8, n = existing(a.cols, c);
            if (XD <= kFp32 && a.ckpt_x && c < pitch) put_ckpt(a, a.ckpt_x, row, pitch, c, f[v], block_amax(f[v]));
            const float m = n > 0 ? mean : 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) f[v][e] -= m;
            if (ragged) keep_first(f[v], n);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[0] = __builtin_fmaf(f[v][e], f[v][e], s[0]);
        }
        row_sums<TPR>(s, red[1]);
        const float rstd = rsqrtf(s[0] * inv_n + a.eps);  // one unit in the last place, as root and division
        if (lane == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8;
            if (c < pitch) put_y(a, row, pitch, c, existing(a.cols, c), f[v], w[v], b[v], rstd);
        }
    }
}

// Rows of any width, one per block of 1024, read once per pass.
template <int XD>
__global__ __launch_bounds__(1024) void fwd_wide_kernel(FwdArgs a) {
    __shared__ float red[2][16][1];
    const int64_t pitch = ckpt_pitch(a.cols);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const RowPtr p = row_at<XD>(a.x, a.ld_x, a.rows, a.cols, row);
        float s[1] = {0.0f};
        for (int64_t c = threadIdx.x * 8; c < pitch; c += 8192) {
            const int n = existing(a.cols, c);
            float f[8];
            widen8(load8<XD>(p, (int)c, n), f);
            if (n < 8) keep_first(f, n);
            if (XD <= kFp32 && a.ckpt_x) put_ckpt(a, a.ckpt_x, row, pitch, (int)c, f, block_amax(f));
            float t = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) t += f[e];
            s[0] += t;
        }
        row_sums<1024>(s, red[0]);
        const float mean = s[0] / (float)a.cols;
        s[0] = 0.0f;
        for (int64_t c = threadIdx.x * 8; c < pitch; c += 8192) {
            const int n = existing(a.cols, c);
            float f[8];
            widen8(load8<XD>(p, (int)c, n), f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] -= mean;
            if (n < 8) keep_first(f, n);
            float t = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) t = __builtin_fmaf(f[e], f[e], t);
            s[0] += t;
        }
        row_sums<1024>(s, red[1]);
        const float rstd = rsqrtf(s[0] / (float)a.cols + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        for (int64_t c = threadIdx.x * 8; c < pitch; c += 8192) {
            const int n = existing(a.cols, c);
            float f[8], w[8], b[8];
            widen8(load8<XD>(p, (int)c, n), f);
            load_param8(a.w, a.param_dt, (int)c, n, 1.0f, w);
            load_param8(a.b, a.param_dt, (int)c, n, 0.0f, b);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] -= mean;
            put_y(a, row, pitch, (int)c, n, f, w, b, rstd);
        }
    }
}

template <int XD, int TPR, int NV>
hipError_t fwd_run(const FwdArgs& a, hipStream_t stream) {
    constexpr int B = norm_block(TPR), G = B / TPR;
    const int64_t groups = (a.rows + G - 1) / G;
    const int64_t most = 1024 * kThreads / B;
    fwd_kernel<XD, TPR, NV><<<grid_for(groups < most ? groups : most, B), B, 0, stream>>>(a);
    return hipGetLastError();
}

template <int XD>
hipError_t fwd_pick(const FwdArgs& a, hipStream_t stream) {
    const int64_t n = a.cols;
    if (n <= 128) return fwd_run<XD, 16, 1>(a, stream);
    if (n <= 512) return fwd_run<XD, 64, 1>(a, stream);
    if (n <= 1024) return fwd_run<XD, 64, 2>(a, stream);
    if (n <= 2048) return fwd_run<XD, 256, 1>(a, stream);
    if (n <= 4096) return fwd_run<XD, 256, 2>(a, stream);
    if (n <= 8192) return fwd_run<XD, 512, 2>(a, stream);
    if (n <= 12288) return fwd_run<XD, 512, 3>(a, stream);
    if (n <= 16384) return fwd_run<XD, 512, 4>(a, stream);
    fwd_wide_kernel<XD><<<grid_for(a.rows, 1024), 1024, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_layernorm_fwd(const NormFwd& f, hipStream_t stream) {
    FwdArgs a{};
    a.x = f.x; a.w = f.weight; a.b = f.bias;
    a.y = (char*)f.y; a.ckpt_x = (char*)f.ckpt_x; a.ckpt_y = (char*)f.ckpt_y;
    a.mean = f.mean; a.rstd = f.rstd;
    a.rows = f.rows; a.cols = f.cols; a.ld_x = f.ld_x; a.ld_y = f.ld_y;
    a.param_dt = f.param_dt; a.y_dt = f.y_dt; a.e4m3 = f.ckpt_format == ZR_CKPT_E4M3;
    a.eps = f.eps;
    switch (f.x_dt) {
        case ZR_BF16: return fwd_pick<kBf16>(a, stream);
        case ZR_FP32: return fwd_pick<kFp32>(a, stream);
        case ZR_CKPT_E4M3: return fwd_pick<kE4m3>(a, stream);
        default: return fwd_pick<kInt8>(a, stream);
    }
}

}  // namespace zr
