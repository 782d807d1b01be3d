// RMS norm, backward, over rows of h (the norm's input after the residual's
// addition) or of its 8-bit checkpoint. With xh = h * rstd and g = dy * w, per row
// of n columns:
//     dh = rstd * (g - xh * sum(g * xh) / n)        (h's, x's and the residual's)
//     dw = sum over rows of dy * xh
// all in fp32. The weight's gradient is a column sum over all rows: a block keeps
// its columns' sums in registers over the strip of rows that it walks and leaves
// one fp32 partial row in the workspace; a second kernel joins the strips in a
// fixed order, so the result does not change from run to run (no atomics). Rows
// over 12288 columns are read in each of two passes, and once more for dw.
//
// Memory bounds it: 16384x4096 from an e4m3 checkpoint takes 75 to 77 us, join
// included, for 75 at 6.28 TB/s. Small ones are bound by their two launches and the
// rows' chain of sums: 4097x1023 fp32 13.8 us and 4.1 for the join.
#include <hip/hip_runtime.h>

#include "zr_norm.hpp"

namespace zr {
namespace {

struct RmsBwdArgs {
    const void *dy, *h, *w;
    const float* rstd;
    char* dx;
    float* part;  // [strips][cols], or null: no gradient or the one below
    void* dw;     // written by the only block, or null
    int grad_dt, accumulate;
    int64_t rows, cols, ld_dy, ld_h, ld_dx;
    int param_dt, dx_dt, add_dx;
};

// xh = h * rstd of a vector: a checkpoint's power of two goes into the factor.
template <int XD>
__device__ __forceinline__ void scaled8(const Raw8<XD>& r, float rstd, float f[8]) {
    if constexpr (XD <= kFp32) {
        widen8(r, f);
    } else {
        ckpt_codes8<XD>(r.q, f);
        rstd *= ckpt_scale(r.s);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= rstd;
}

template <int XD, int DD, int TPR, int NV, int B>
__global__ __launch_bounds__(B) void rms_bwd_kernel(RmsBwdArgs a) {
    constexpr int G = B / TPR;
    // a block's groups leave the loop at different turns, so only a block of one
    // group may have barriers in it
    static_assert(TPR <= 64 || B == TPR, "barriers need one row per block");
    constexpr int C = TPR * NV * 8;  // columns that a row's lanes cover
    __shared__ float red[2][B / 64][1];
    __shared__ float join[G > 1 ? G : 1][G > 1 ? C : 1];
    const int lane = threadIdx.x % TPR, group = row_group<TPR, B>();
    const float inv_n = 1.0f / (float)a.cols;
    float w[NV][8], dw[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (v * TPR + lane) * 8;
        load_param8(a.w, a.param_dt, c, existing(a.cols, c), 1.0f, w[v]);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[v][e] = 0.0f;
    }
    Raw8<XD> rx[NV];
    Raw8<DD> rd[NV];
    float rstd_next = 0.0f;
    const int dx_es = a.dx_dt == kBf16 ? 2 : 4;
    auto fetch = [&](int64_t row) {
        const RowPtr px = row_at<XD>(a.h, a.ld_h, a.rows, a.cols, row), pd = row_at<DD>(a.dy, a.ld_dy, a.rows, a.cols, row);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8, n = existing(a.cols, c);
            rx[v] = fetch8<XD, true>(px, c, n);
            rd[v] = fetch8<DD, true>(pd, c, n);
        }
        rstd_next = a.rstd[row];
    };
    int parity = 0;
    const int64_t first = (int64_t)blockIdx.x * G + group, step = (int64_t)gridDim.x * G;
    if (first < a.rows) fetch(first);
    for (int64_t row = first; row < a.rows; row += step) {
        const float rstd = rstd_next;
        char* out = a.dx + row * a.ld_dx * dx_es;
        // dx before (bf16 in the first half): in flight during the sums
        Raw8<kFp32> old[NV];
        if (a.add_dx) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (v * TPR + lane) * 8, n = existing(a.cols, c);
                if (a.dx_dt == kBf16)
                    old[v].a = __builtin_bit_cast(f32x4, fetch8<kBf16, true>({out, nullptr}, c, n).v);
                else
                    old[v] = fetch8<kFp32, true>({out, nullptr}, c, n);
            }
        }
        float xh[NV][8], g[NV][8];
        float s[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8, n = existing(a.cols, c);
            settle8(rx[v], c, n);
            settle8(rd[v], c, n);
            scaled8<XD>(rx[v], rstd, xh[v]);
            widen8(rd[v], g[v]);
            if (n < 8) keep_first(xh[v], n);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dw[v][e] = __builtin_fmaf(g[v][e], xh[v][e], dw[v][e]);
                g[v][e] *= w[v][e];
                s[0] = __builtin_fmaf(g[v][e], xh[v][e], s[0]);
            }
        }
        if (row + step < a.rows) fetch(row + step);
        if (!a.dx) continue;
        // two sets of slots in turn: a set is written again only after the
        // other set's barrier, which every reader of the first has passed
        row_sums<TPR>(s, red[parity]);
        parity ^= 1;
        const float k1 = -(s[0] * inv_n) * rstd;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8, n = existing(a.cols, c);
            if (n == 0) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) g[v][e] = __builtin_fmaf(g[v][e], rstd, xh[v][e] * k1);
            if (a.add_dx) {
                float o[8];
                if (a.dx_dt == kBf16) {
                    Raw8<kBf16> b{__builtin_bit_cast(u32x4, old[v].a)};
                    settle8(b, c, n);
                    widen8(b, o);
                } else {
                    settle8(old[v], c, n);
                    widen8(old[v], o);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) g[v][e] += o[e];
            }
            store8<true>(out, a.dx_dt, c, n, g[v]);
        }
    }
    // the block's sums: to the workspace, or as the gradient
    if (!a.part && !a.dw) return;
    float* const out = a.part ? a.part + (int64_t)blockIdx.x * a.cols : nullptr;
    if constexpr (G > 1) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e) join[group][(v * TPR + lane) * 8 + e] = dw[v][e];
        __syncthreads();
        for (int c = threadIdx.x; c < a.cols; c += B) {
            float t = 0.0f;
#pragma unroll
            for (int r = 0; r < G; ++r) t += join[r][c];
            if (out)
                out[c] = t;
            else
                put_grad(a.dw, c, t, a.grad_dt, a.accumulate);
        }
    } else {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8, n = existing(a.cols, c);
            if (n == 0) continue;
            if (out) {
                store8<false>((char*)out, kFp32, c, n, dw[v]);
            } else {
                float old[8];
                load_param8(a.accumulate ? a.dw : nullptr, a.grad_dt, c, n, 0.0f, old);
#pragma unroll
                for (int e = 0; e < 8; ++e) old[e] += dw[v][e];
                store8<false>((char*)a.dw, a.grad_dt, c, n, old);
            }
        }
    }
}

// Rows of any width: one block per row for dx, then column sums by tiles of
// 2048 columns over strips of rows.
template <int XD, int DD>
__global__ __launch_bounds__(1024) void rms_bwd_wide_dx_kernel(RmsBwdArgs a) {
    __shared__ float red[2][16][1];
    const float inv_n = 1.0f / (float)a.cols;
    int parity = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const RowPtr px = row_at<XD>(a.h, a.ld_h, a.rows, a.cols, row), pd = row_at<DD>(a.dy, a.ld_dy, a.rows, a.cols, row);
        const float rstd = a.rstd[row];
        float s[1] = {0.0f};
        for (int64_t c = threadIdx.x * 8; c < a.cols; c += 8192) {
            const int n = existing(a.cols, c);
            float x[8], d[8], w[8];
            scaled8<XD>(load8<XD>(px, (int)c, n), rstd, x);
            widen8(load8<DD>(pd, (int)c, n), d);
            load_param8(a.w, a.param_dt, (int)c, n, 1.0f, w);
            if (n < 8) keep_first(x, n);
            float t = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) t = __builtin_fmaf(d[e] * w[e], x[e], t);
            s[0] += t;
        }
        row_sums<1024>(s, red[parity]);
        parity ^= 1;
        const float k1 = -(s[0] * inv_n) * rstd;
        char* out = a.dx + row * a.ld_dx * (a.dx_dt == kBf16 ? 2 : 4);
        for (int64_t c = threadIdx.x * 8; c < a.cols; c += 8192) {
            const int n = existing(a.cols, c);
            float x[8], d[8], w[8];
            scaled8<XD>(load8<XD>(px, (int)c, n), rstd, x);
            widen8(load8<DD>(pd, (int)c, n), d);
            load_param8(a.w, a.param_dt, (int)c, n, 1.0f, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = __builtin_fmaf(d[e] * w[e], rstd, x[e] * k1);
            if (a.add_dx) {
                float old[8];
                load_param8(out, a.dx_dt, (int)c, n, 0.0f, old);
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] += old[e];
            }
            store8<true>(out, a.dx_dt, (int)c, n, d);
        }
    }
}

template <int XD, int DD>
__global__ __launch_bounds__(kThreads) void rms_bwd_wide_sums_kernel(RmsBwdArgs a, int strips) {
    const int64_t tiles = (a.cols + kThreads * 8 - 1) / (kThreads * 8);
    for (int64_t t = blockIdx.x; t < tiles * strips; t += gridDim.x) {
        const int s = (int)(t / tiles);
        const int64_t c = ((t - s * tiles) * kThreads + threadIdx.x) * 8;
        const int n = existing(a.cols, c);
        if (n == 0) continue;
        float dw[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[e] = 0.0f;
        for (int64_t row = s; row < a.rows; row += strips) {
            float x[8], d[8];
            scaled8<XD>(load8<XD>(row_at<XD>(a.h, a.ld_h, a.rows, a.cols, row), (int)c, n), a.rstd[row], x);
            widen8(load8<DD>(row_at<DD>(a.dy, a.ld_dy, a.rows, a.cols, row), (int)c, n), d);
#pragma unroll
            for (int e = 0; e < 8; ++e) dw[e] = __builtin_fmaf(d[e], x[e], dw[e]);
        }
        store8<false>((char*)(a.part + (int64_t)s * a.cols), kFp32, (int)c, n, dw);
    }
}

// Joins the strips' partial sums, [strips][cols], in a fixed order: each of 16
// groups of lanes takes every 16th strip of 64 columns.
__global__ __launch_bounds__(1024) void rms_bwd_join_kernel(const float* part, int strips, int64_t cols, void* dw,
                                                            int grad_dt, int accumulate) {
    __shared__ float sum[16][64];
    const int lane = threadIdx.x & 63, group = threadIdx.x >> 6;
    const int64_t tiles = (cols + 63) / 64;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t at = t * 64 + lane;
        float s = 0.0f;
        for (int k = group; k < strips; k += 128) {  // eight loads in flight
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = at < cols && k + 16 * e < strips ? part[(int64_t)(k + 16 * e) * cols + at] : 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s += v[e];
        }
        __syncthreads();
        sum[group][lane] = s;
        __syncthreads();
        if (group == 0 && at < cols) {
            s = 0.0f;
#pragma unroll
            for (int g = 0; g < 16; ++g) s += sum[g][lane];
            put_grad(dw, at, s, grad_dt, accumulate);
        }
    }
}

template <int XD, int DD, int TPR, int NV, int B = norm_block(TPR)>
hipError_t bwd_run(const RmsBwdArgs& a, int strips, hipStream_t stream) {
    rms_bwd_kernel<XD, DD, TPR, NV, B><<<strips, B, 0, stream>>>(a);
    return hipGetLastError();
}

template <int XD, int DD>
hipError_t bwd_pick(const RmsBwdArgs& a, int strips, hipStream_t stream) {
    const int64_t n = a.cols;
    // one block for all rows: as many of them at once as it can hold
    if (strips == 1 && n <= 128) return bwd_run<XD, DD, 16, 1, 1024>(a, strips, stream);
    if (strips == 1 && n <= 512) return bwd_run<XD, DD, 64, 1, 1024>(a, strips, stream);
    if (strips == 1 && n <= 1024) return bwd_run<XD, DD, 64, 2, 512>(a, strips, stream);
    if (n <= 128) return bwd_run<XD, DD, 16, 1>(a, strips, stream);
    if (n <= 512) return bwd_run<XD, DD, 64, 1>(a, strips, stream);
    if (n <= 1024) return bwd_run<XD, DD, 64, 2>(a, strips, stream);
    if (n <= 2048) return bwd_run<XD, DD, 256, 1>(a, strips, stream);
    if (n <= 4096) return bwd_run<XD, DD, 512, 1>(a, strips, stream);
    if (n <= 8192) return bwd_run<XD, DD, 512, 2>(a, strips, stream);
    if (n <= 12288) return bwd_run<XD, DD, 512, 3>(a, strips, stream);
    if (a.part) {  // before dx, which may take dy's or h's place
        const int64_t tiles = (n + kThreads * 8 - 1) / (kThreads * 8);
        rms_bwd_wide_sums_kernel<XD, DD><<<grid_for(tiles * strips, kThreads), kThreads, 0, stream>>>(a, strips);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.dx) rms_bwd_wide_dx_kernel<XD, DD><<<grid_for(a.rows, 1024), 1024, 0, stream>>>(a);
    return hipGetLastError();
}

template <int XD>
hipError_t bwd_pick_dy(const RmsBwdArgs& a, zr_dtype dy_dt, int strips, hipStream_t stream) {
    return dy_dt == ZR_BF16 ? bwd_pick<XD, kBf16>(a, strips, stream) : bwd_pick<XD, kFp32>(a, strips, stream);
}

}  // namespace

hipError_t launch_rmsnorm_bwd(const RmsBwd& f, hipStream_t stream) {
    RmsBwdArgs a{};
    a.dy = f.dy; a.h = f.h; a.w = f.weight; a.rstd = f.rstd;
    a.dx = (char*)f.dx;
    a.rows = f.rows; a.cols = f.cols; a.ld_dy = f.ld_dy; a.ld_h = f.ld_h; a.ld_dx = f.ld_dx;
    a.param_dt = f.param_dt; a.dx_dt = f.dx_dt; a.add_dx = f.add_dx;
    const int strips = layernorm_strips(f.rows, f.cols);
    const bool joined = rmsnorm_workspace(f.rows, f.cols) > 0 || strips == 0;
    a.part = f.dweight && joined ? (float*)f.workspace : nullptr;
    if (!joined) {
        a.dw = f.dweight;
        a.grad_dt = f.grad_dt; a.accumulate = f.accumulate;
    }
    hipError_t e = hipSuccess;
    if (strips > 0) {
        switch (f.h_dt) {
            case ZR_BF16: e = bwd_pick_dy<kBf16>(a, f.dy_dt, strips, stream); break;
            case ZR_FP32: e = bwd_pick_dy<kFp32>(a, f.dy_dt, strips, stream); break;
            case ZR_CKPT_E4M3: e = bwd_pick_dy<kE4m3>(a, f.dy_dt, strips, stream); break;
            default: e = bwd_pick_dy<kInt8>(a, f.dy_dt, strips, stream); break;
        }
        if (e != hipSuccess) return e;
    }
    if (!f.dweight || !joined) return e;
    rms_bwd_join_kernel<<<grid_for((f.cols + 63) / 64, 1024), 1024, 0, stream>>>((const float*)f.workspace, strips, f.cols,
                                                                                 f.dweight, f.grad_dt, f.accumulate);
    return hipGetLastError();
}

}  // namespace zr
