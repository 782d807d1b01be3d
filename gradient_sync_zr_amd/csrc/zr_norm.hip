// Layer norm, forward and backward, over rows of activations or of their
// 8-bit checkpoints.
//
// Forward, per row of n columns:
//     mean = sum x / n,  rstd = 1 / sqrt(sum (x - mean)^2 / n + eps)
//     y    = (x - mean) * rstd * w + b
// Backward, with xh = (x - mean) * rstd and g = dy * w:
//     dx = rstd * (g - sum(g) / n - xh * sum(g * xh) / n)
//     dw = sum over rows of dy * xh,  db = sum over rows of dy
//
// A row is held in registers by TPR lanes, NV vectors of 8 columns each, so
// every input byte is read once: the forward pass takes mean and variance
// from the registers (two passes, no cancellation), the backward pass its two
// row sums. Rows too wide for that (over 16384 columns) are read again from
// memory in each pass. All statistics and sums
// are fp32.
//
// The weight's and the bias's gradient are column sums over all rows. A block
// keeps its columns' sums in registers over the strip of rows that it walks
// and leaves one fp32 partial row per strip in the workspace; a second, small
// kernel joins the strips in a fixed order, so the result does not change
// from run to run (no atomics).
#include <hip/hip_runtime.h>

#include "zr_ckpt.hpp"
#include "zr_internal.hpp"

namespace zr {
namespace {

__device__ __forceinline__ int existing(int64_t cols, int64_t c) {
    const int64_t left = cols - c;
    return left >= 8 ? 8 : (left > 0 ? (int)left : 0);
}

// Sum over the TPR lanes of a row. red: one float per wave of the block, free
// again once every wave has passed a later barrier.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
    v = wave_sum<(TPR < 64 ? TPR : 64)>(v);
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64;
        const int wave = threadIdx.x / 64, first = wave / W * W;
        if ((threadIdx.x & 63) == 0) red[wave] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < W; ++i) v += red[first + i];
    }
    return v;
}

// ---------------------------------------------------------------- forward
struct FwdArgs {
    const void *x, *w, *b;
    char *y, *ckpt_x, *ckpt_y;
    float *mean, *rstd;
    int64_t rows, cols, ld_x, ld_y;
    int param_dt, y_dt, e4m3;
    float eps;
};

// One vector of the output: y (rounded to its type), then its checkpoint.
__device__ __forceinline__ void fwd_store(const FwdArgs& a, int64_t row, int64_t pitch, int c, int n, float f[8],
                                          float mean, float rstd) {
    float w[8], b[8];
    load_param8(a.w, a.param_dt, c, n, 1.0f, w);
    load_param8(a.b, a.param_dt, c, n, 0.0f, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = __builtin_fmaf((f[e] - mean) * rstd, w[e], b[e]);
    if (a.y && n > 0) store8(a.y + row * a.ld_y * (a.y_dt == kBf16 ? 2 : 4), a.y_dt, c, n, f);
    if (a.ckpt_y && c < pitch) {
        // what is held is y as its readers have it
        if (a.y_dt == kBf16) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = bf16_widen(bf16_round(f[e]));
        }
        if (n < 8) keep_first(f, n);
        ckpt_store8(a.ckpt_y + row * pitch, (uint8_t*)a.ckpt_y + a.rows * pitch + row * (pitch / kCkptBlock), c, f,
                    a.e4m3 != 0);
    }
}

template <int XD, int TPR, int NV>
__global__ __launch_bounds__(TPR > kThreads ? TPR : kThreads) void fwd_kernel(FwdArgs a, int64_t groups) {
    constexpr int B = TPR > kThreads ? TPR : kThreads, G = B / TPR;
    __shared__ float red[2][B / 64];
    const int lane = threadIdx.x % TPR;
    const int64_t pitch = ckpt_pitch(a.cols);
    for (int64_t g = blockIdx.x; g < groups; g += gridDim.x) {
        const int64_t row = g * G + threadIdx.x / TPR;
        if (TPR <= 64 && row >= a.rows) continue;  // wider rows: one row per block, always there
        const RowPtr p = row_at<XD>(a.x, a.ld_x, a.rows, a.cols, row);
        Raw8<XD> raw[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8;
            raw[v] = load8<XD>(p, c, existing(a.cols, c));
        }
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8, n = existing(a.cols, c);
            float f[8];
            widen8(raw[v], f);
            if (n < 8) keep_first(f, n);
            if (XD <= kFp32 && a.ckpt_x && c < pitch)
                ckpt_store8(a.ckpt_x + row * pitch,
                            (uint8_t*)a.ckpt_x + a.rows * pitch + row * (pitch / kCkptBlock), c, f, a.e4m3 != 0);
#pragma unroll
            for (int e = 0; e < 8; ++e) s += f[e];
        }
        const float mean = row_sum<TPR>(s, red[0]) / (float)a.cols;
        s = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int n = existing(a.cols, (v * TPR + lane) * 8);
            float f[8];
            widen8(raw[v], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] -= mean;
            if (n < 8) keep_first(f, n);
#pragma unroll
            for (int e = 0; e < 8; ++e) s = __builtin_fmaf(f[e], f[e], s);
        }
        const float rstd = 1.0f / sqrtf(row_sum<TPR>(s, red[1]) / (float)a.cols + a.eps);
        if (lane == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8;
            if (c >= pitch) continue;  // whole blocks, so whole quads of lanes
            float f[8];
            widen8(raw[v], f);
            fwd_store(a, row, pitch, c, existing(a.cols, c), f, mean, rstd);
        }
    }
}

// Rows of any width, one per block of 1024, read once per pass.
template <int XD>
__global__ __launch_bounds__(1024) void fwd_wide_kernel(FwdArgs a) {
    __shared__ float red[2][16];
    const int64_t pitch = ckpt_pitch(a.cols);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const RowPtr p = row_at<XD>(a.x, a.ld_x, a.rows, a.cols, row);
        float s = 0.0f;
        for (int64_t c = threadIdx.x * 8; c < pitch; c += 8192) {
            const int n = existing(a.cols, c);
            float f[8];
            widen8(load8<XD>(p, (int)c, n), f);
            if (n < 8) keep_first(f, n);
            if (XD <= kFp32 && a.ckpt_x)
                ckpt_store8(a.ckpt_x + row * pitch,
                            (uint8_t*)a.ckpt_x + a.rows * pitch + row * (pitch / kCkptBlock), (int)c, f, a.e4m3 != 0);
            float t = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) t += f[e];
            s += t;
        }
        const float mean = row_sum<1024>(s, red[0]) / (float)a.cols;
        s = 0.0f;
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
            s += t;
        }
        const float rstd = 1.0f / sqrtf(row_sum<1024>(s, red[1]) / (float)a.cols + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        for (int64_t c = threadIdx.x * 8; c < pitch; c += 8192) {
            const int n = existing(a.cols, c);
            float f[8];
            widen8(load8<XD>(p, (int)c, n), f);
            fwd_store(a, row, pitch, (int)c, n, f, mean, rstd);
        }
    }
}

template <int XD, int TPR, int NV>
hipError_t fwd_run(const FwdArgs& a, hipStream_t stream) {
    constexpr int B = TPR > kThreads ? TPR : kThreads, G = B / TPR;
    const int64_t groups = (a.rows + G - 1) / G;
    fwd_kernel<XD, TPR, NV><<<grid_for(groups), B, 0, stream>>>(a, groups);
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
    if (n <= 8192) return fwd_run<XD, 256, 4>(a, stream);
    if (n <= 16384) return fwd_run<XD, 512, 4>(a, stream);
    fwd_wide_kernel<XD><<<grid_for(a.rows), 1024, 0, stream>>>(a);
    return hipGetLastError();
}

// --------------------------------------------------------------- backward
struct BwdArgs {
    const void *dy, *x, *w;
    const float *mean, *rstd;
    char* dx;
    float* part;  // [strips][2][cols], or null: no parameter gradients
    int64_t rows, cols, ld_dy, ld_x, ld_dx;
    int param_dt, dx_dt, add_dx;
};

template <int XD, int DD, int TPR, int NV>
__global__ __launch_bounds__(TPR > kThreads ? TPR : kThreads) void bwd_kernel(BwdArgs a) {
    constexpr int B = TPR > kThreads ? TPR : kThreads, G = B / TPR;
    constexpr int C = TPR * NV * 8;  // columns a group of lanes covers
    __shared__ float red[4][B / 64];
    __shared__ float join[G > 1 ? G : 1][G > 1 ? C : 1];
    const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
    const float inv_n = 1.0f / (float)a.cols;
    float dw[NV][8], db[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[v][e] = db[v][e] = 0.0f;

    Raw8<XD> rx[NV];
    Raw8<DD> rd[NV];
    float mean = 0.0f, rstd = 0.0f;
    auto fetch = [&](int64_t row) {
        const bool here = row < a.rows;
        const int64_t at = here ? row : 0;
        const RowPtr px = row_at<XD>(a.x, a.ld_x, a.rows, a.cols, at), pd = row_at<DD>(a.dy, a.ld_dy, a.rows, a.cols, at);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8, n = here ? existing(a.cols, c) : 0;
            rx[v] = load8<XD>(px, c, n);
            rd[v] = load8<DD>(pd, c, n);
        }
        mean = here ? a.mean[at] : 0.0f;
        rstd = here ? a.rstd[at] : 0.0f;
    };
    int parity = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * G; row0 < a.rows; row0 += (int64_t)gridDim.x * G) {
        const int64_t row = row0 + group;
        fetch(row);
        const bool here = row < a.rows;
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8, n = here ? existing(a.cols, c) : 0;
            float x[8], d[8], w[8];
            widen8(rx[v], x);
            widen8(rd[v], d);
            load_param8(a.w, a.param_dt, c, n, 1.0f, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = (x[e] - mean) * rstd;
            if (n < 8) keep_first(x, n);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dw[v][e] = __builtin_fmaf(d[e], x[e], dw[v][e]);
                db[v][e] += d[e];
                const float g = d[e] * w[e];
                s1 = __builtin_fmaf(g, x[e], s1);
                s2 += g;
            }
        }
        if (a.dx) {
            // two sets of slots in turn: a set is written again only after the
            // other set's barrier, which every reader of the first has passed
            const float c1 = row_sum<TPR>(s1, red[parity]) * inv_n;
            const float c2 = row_sum<TPR>(s2, red[parity + 2]) * inv_n;
            parity ^= 1;
            if (here) {
                char* out = a.dx + row * a.ld_dx * (a.dx_dt == kBf16 ? 2 : 4);
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const int c = (v * TPR + lane) * 8, n = existing(a.cols, c);
                    if (n == 0) continue;
                    float x[8], d[8], w[8];
                    widen8(rx[v], x);
                    widen8(rd[v], d);
                    load_param8(a.w, a.param_dt, c, n, 1.0f, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float xh = (x[e] - mean) * rstd;
                        d[e] = (d[e] * w[e] - c2 - xh * c1) * rstd;
                    }
                    if (a.add_dx) {
                        float old[8];
                        load_param8(out, a.dx_dt, c, n, 0.0f, old);
#pragma unroll
                        for (int e = 0; e < 8; ++e) d[e] += old[e];
                    }
                    store8(out, a.dx_dt, c, n, d);
                }
            }
        }
    }
    if (!a.part) return;
    float* out = a.part + (int64_t)blockIdx.x * 2 * a.cols;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if constexpr (G > 1) {
            __syncthreads();
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e) join[group][(v * TPR + lane) * 8 + e] = which ? db[v][e] : dw[v][e];
            __syncthreads();
            for (int c = threadIdx.x; c < a.cols; c += B) {
                float t = 0.0f;
#pragma unroll
                for (int g = 0; g < G; ++g) t += join[g][c];
                out[which * a.cols + c] = t;
            }
        } else {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (v * TPR + lane) * 8, n = existing(a.cols, c);
                if (n > 0) store8((char*)(out + which * a.cols), kFp32, c, n, which ? db[v] : dw[v]);
            }
        }
    }
}

// Rows of any width: one block per row for dx, then column sums by tiles of
// 2048 columns over strips of rows.
template <int XD, int DD>
__global__ __launch_bounds__(1024) void bwd_wide_dx_kernel(BwdArgs a) {
    __shared__ float red[4][16];
    const float inv_n = 1.0f / (float)a.cols;
    int parity = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const RowPtr px = row_at<XD>(a.x, a.ld_x, a.rows, a.cols, row), pd = row_at<DD>(a.dy, a.ld_dy, a.rows, a.cols, row);
        const float mean = a.mean[row], rstd = a.rstd[row];
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t c = threadIdx.x * 8; c < a.cols; c += 8192) {
            const int n = existing(a.cols, c);
            float x[8], d[8], w[8];
            widen8(load8<XD>(px, (int)c, n), x);
            widen8(load8<DD>(pd, (int)c, n), d);
            load_param8(a.w, a.param_dt, (int)c, n, 1.0f, w);
            float t1 = 0.0f, t2 = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = (x[e] - mean) * rstd;
            if (n < 8) keep_first(x, n);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float g = d[e] * w[e];
                t1 = __builtin_fmaf(g, x[e], t1);
                t2 += g;
            }
            s1 += t1;
            s2 += t2;
        }
        const float c1 = row_sum<1024>(s1, red[parity]) * inv_n;
        const float c2 = row_sum<1024>(s2, red[parity + 2]) * inv_n;
        parity ^= 1;
        char* out = a.dx + row * a.ld_dx * (a.dx_dt == kBf16 ? 2 : 4);
        for (int64_t c = threadIdx.x * 8; c < a.cols; c += 8192) {
            const int n = existing(a.cols, c);
            float x[8], d[8], w[8];
            widen8(load8<XD>(px, (int)c, n), x);
            widen8(load8<DD>(pd, (int)c, n), d);
            load_param8(a.w, a.param_dt, (int)c, n, 1.0f, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = (d[e] * w[e] - c2 - (x[e] - mean) * rstd * c1) * rstd;
            if (a.add_dx) {
                float old[8];
                load_param8(out, a.dx_dt, (int)c, n, 0.0f, old);
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] += old[e];
            }
            store8(out, a.dx_dt, (int)c, n, d);
        }
    }
}

template <int XD, int DD>
__global__ __launch_bounds__(kThreads) void bwd_wide_sums_kernel(BwdArgs a, int strips) {
    const int64_t tiles = (a.cols + kThreads * 8 - 1) / (kThreads * 8);
    for (int64_t t = blockIdx.x; t < tiles * strips; t += gridDim.x) {
        const int s = (int)(t / tiles);
        const int64_t c = ((t - s * tiles) * kThreads + threadIdx.x) * 8;
        const int n = existing(a.cols, c);
        if (n == 0) continue;
        float dw[8], db[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[e] = db[e] = 0.0f;
        for (int64_t row = s; row < a.rows; row += strips) {
            float x[8], d[8];
            widen8(load8<XD>(row_at<XD>(a.x, a.ld_x, a.rows, a.cols, row), (int)c, n), x);
            widen8(load8<DD>(row_at<DD>(a.dy, a.ld_dy, a.rows, a.cols, row), (int)c, n), d);
            const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dw[e] = __builtin_fmaf(d[e], (x[e] - mean) * rstd, dw[e]);
                db[e] += d[e];
            }
        }
        float* out = a.part + (int64_t)s * 2 * a.cols;
        store8((char*)out, kFp32, (int)c, n, dw);
        store8((char*)(out + a.cols), kFp32, (int)c, n, db);
    }
}

// Joins the strips' partial sums, [strips][2][cols], in a fixed order: each of
// 16 groups of lanes takes every 16th strip of 64 columns.
__global__ __launch_bounds__(1024) void bwd_join_kernel(const float* part, int strips, int64_t cols, void* dw, void* db,
                                                        int grad_dt, int accumulate) {
    __shared__ float sum[16][64];
    const int lane = threadIdx.x & 63, group = threadIdx.x >> 6;
    const int64_t tiles = (2 * cols + 63) / 64;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t at = t * 64 + lane;
        float s = 0.0f;
        if (at < 2 * cols)
            for (int k = group; k < strips; k += 16) s += part[(int64_t)k * 2 * cols + at];
        __syncthreads();
        sum[group][lane] = s;
        __syncthreads();
        if (group == 0 && at < 2 * cols) {
            s = 0.0f;
#pragma unroll
            for (int g = 0; g < 16; ++g) s += sum[g][lane];
            void* out = at < cols ? dw : db;
            const int64_t o = at < cols ? at : at - cols;
            if (out && grad_dt == kBf16) {
                uint16_t* q = (uint16_t*)out + o;
                store_elem(q, accumulate ? load_elem(q) + s : s);
            } else if (out) {
                float* q = (float*)out + o;
                store_elem(q, accumulate ? load_elem(q) + s : s);
            }
        }
    }
}

template <int XD, int DD, int TPR, int NV>
hipError_t bwd_run(const BwdArgs& a, int strips, hipStream_t stream) {
    constexpr int B = TPR > kThreads ? TPR : kThreads;
    bwd_kernel<XD, DD, TPR, NV><<<strips, B, 0, stream>>>(a);
    return hipGetLastError();
}

template <int XD, int DD>
hipError_t bwd_pick(const BwdArgs& a, int strips, hipStream_t stream) {
    const int64_t n = a.cols;
    if (n <= 128) return bwd_run<XD, DD, 16, 1>(a, strips, stream);
    if (n <= 512) return bwd_run<XD, DD, 64, 1>(a, strips, stream);
    if (n <= 1024) return bwd_run<XD, DD, 64, 2>(a, strips, stream);
    if (n <= 2048) return bwd_run<XD, DD, 256, 1>(a, strips, stream);
    if (n <= 4096) return bwd_run<XD, DD, 256, 2>(a, strips, stream);
    if (n <= 8192) return bwd_run<XD, DD, 256, 4>(a, strips, stream);
    if (n <= 16384) return bwd_run<XD, DD, 512, 4>(a, strips, stream);
    if (a.part) {  // before dx, which may take dy's or x's place
        const int64_t tiles = (n + kThreads * 8 - 1) / (kThreads * 8);
        bwd_wide_sums_kernel<XD, DD><<<grid_for(tiles * strips), kThreads, 0, stream>>>(a, strips);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.dx) bwd_wide_dx_kernel<XD, DD><<<grid_for(a.rows), 1024, 0, stream>>>(a);
    return hipGetLastError();
}

template <int XD>
hipError_t bwd_pick_dy(const BwdArgs& a, zr_dtype dy_dt, int strips, hipStream_t stream) {
    return dy_dt == ZR_BF16 ? bwd_pick<XD, kBf16>(a, strips, stream) : bwd_pick<XD, kFp32>(a, strips, stream);
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

hipError_t launch_layernorm_bwd(const NormBwd& f, hipStream_t stream) {
    BwdArgs a{};
    a.dy = f.dy; a.x = f.x; a.w = f.weight; a.mean = f.mean; a.rstd = f.rstd;
    a.dx = (char*)f.dx;
    a.rows = f.rows; a.cols = f.cols; a.ld_dy = f.ld_dy; a.ld_x = f.ld_x; a.ld_dx = f.ld_dx;
    a.param_dt = f.param_dt; a.dx_dt = f.dx_dt; a.add_dx = f.add_dx;
    const bool grads = f.dweight || f.dbias;
    a.part = grads ? (float*)f.workspace : nullptr;
    const int strips = layernorm_strips(f.rows, f.cols);
    hipError_t e = hipSuccess;
    if (strips > 0) {
        switch (f.x_dt) {
            case ZR_BF16: e = bwd_pick_dy<kBf16>(a, f.dy_dt, strips, stream); break;
            case ZR_FP32: e = bwd_pick_dy<kFp32>(a, f.dy_dt, strips, stream); break;
            case ZR_CKPT_E4M3: e = bwd_pick_dy<kE4m3>(a, f.dy_dt, strips, stream); break;
            default: e = bwd_pick_dy<kInt8>(a, f.dy_dt, strips, stream); break;
        }
        if (e != hipSuccess) return e;
    }
    if (!grads) return e;
    const int64_t tiles = (2 * f.cols + 63) / 64;
    bwd_join_kernel<<<grid_for(tiles), 1024, 0, stream>>>((const float*)f.workspace, strips, f.cols, f.dweight, f.dbias,
                                                          f.grad_dt, f.accumulate);
    return hipGetLastError();
}

}  // namespace zr
