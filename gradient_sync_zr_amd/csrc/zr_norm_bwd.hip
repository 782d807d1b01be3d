// Layer norm, backward, over rows of activations or of their 8-bit
// checkpoints. With xh = (x - mean) * rstd and g = dy * w, per row of n columns:
//     dx = rstd * (g - sum(g) / n - xh * sum(g * xh) / n)
//     dw = sum over rows of dy * xh,  db = sum over rows of dy
// all in fp32. Rows over 12288 columns, whose fp32 copies do not fit the registers
// beside the column sums, are read from memory in each pass: x and dy twice for dx,
// and once more for the parameters' gradients (4096x16384 bf16 150 us, 2.7 TB/s).
//
// The weight's and the bias's gradient are column sums over all rows. A block
// keeps its columns' sums in registers over the strip of rows that it walks
// and leaves one fp32 partial row per strip in the workspace; a second, small
// kernel joins the strips in a fixed order, so the result does not change
// from run to run (no atomics).
//
// At 8 bytes an element the arithmetic is near the memory's time, so it is
// kept small: x's decoding is one multiply-add on the code (code * 2^e - mean,
// rounded once), xh and g stay in registers between the row's sums and dx, and
// dx is two multiply-adds. The next row's loads are in flight meanwhile.
//
// Bound by memory: 16384x4096 bf16 78 us (5.2 TB/s), 96 with dx added to (5.6),
// 24576x11008 from int8 240 (5.65 TB/s; 532 before the arithmetic was cut and the
// loads put ahead). 512 strips, two blocks of 256 or one of 512 per CU, measured
// best at 1024 columns (65536x1024: 78 us, with 1024 strips 90) and are taken up to
// 4096, though the forms up to 512 and from 1025 to 2048 columns, of 100 to 119
// registers, would leave room for twice as many (262144x128: 44 us, 4.6 TB/s); 256
// beyond, where a block of 512 has the CU's registers.
#include <hip/hip_runtime.h>

#include "zr_norm.hpp"

namespace zr {
namespace {

struct BwdArgs {
    const void *dy, *x, *w;
    const float *mean, *rstd;
    char* dx;
    float* part;  // [strips][2][cols], or null: no parameter gradients or those below
    void *dw, *db;  // written by the only block, or null
    int grad_dt, accumulate;
    int64_t rows, cols, ld_dy, ld_x, ld_dx;
    int param_dt, dx_dt, add_dx;
};

// (x - mean) of a vector: for a checkpoint one multiply-add per code.
template <int XD>
__device__ __forceinline__ void centered8(const Raw8<XD>& r, float mean, float f[8]) {
    if constexpr (XD <= kFp32) {
        widen8(r, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] -= mean;
    } else {
        const float scale = ckpt_scale(r.s);
        ckpt_codes8<XD>(r.q, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __builtin_fmaf(f[e], scale, -mean);
    }
}

template <int XD, int DD, int TPR, int NV, int B>
__global__ __launch_bounds__(B) void bwd_kernel(BwdArgs a) {
    constexpr int G = B / TPR;
    // a block's groups leave the loop at different turns, so only a block of one
    // group may have barriers in it
    static_assert(TPR <= 64 || B == TPR, "barriers need one row per block");
    constexpr int C = TPR * NV * 8;  // columns that a row's lanes cover
    // three vectors with one source in fp32 leave no registers for old dx
    constexpr bool LATE = NV == 3 && (XD == kFp32 || DD == kFp32);
    __shared__ float red[2][B / 64][2];
    __shared__ float join[G > 1 ? G : 1][G > 1 ? C : 1];
    const int lane = threadIdx.x % TPR, group = row_group<TPR, B>();
    const float inv_n = 1.0f / (float)a.cols;
    float w[NV][8], dw[NV][8], db[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (v * TPR + lane) * 8;
        load_param8(a.w, a.param_dt, c, existing(a.cols, c), 1.0f, w[v]);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[v][e] = db[v][e] = 0.0f;
    }
    Raw8<XD> rx[NV];
    Raw8<DD> rd[NV];
    float mean_next = 0.0f, rstd_next = 0.0f;
    const int dx_es = a.dx_dt == kBf16 ? 2 : 4;
    auto fetch = [&](int64_t row) {
        const RowPtr px = row_at<XD>(a.x, a.ld_x, a.rows, a.cols, row), pd = row_at<DD>(a.dy, a.ld_dy, a.rows, a.cols, row);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8, n = existing(a.cols, c);
            rx[v] = fetch8<XD, true>(px, c, n);
            rd[v] = fetch8<DD, true>(pd, c, n);
        }
        mean_next = a.mean[row];
        rstd_next = a.rstd[row];
    };
    int parity = 0;
    const int64_t first = (int64_t)blockIdx.x * G + group, step = (int64_t)gridDim.x * G;
    if (first < a.rows) fetch(first);
    for (int64_t row = first; row < a.rows; row += step) {
        const float mean = mean_next, rstd = rstd_next;
        char* out = a.dx + row * a.ld_dx * dx_es;
        // dx before (bf16 in the first half): in flight during the sums, and waited
        // for before the next row's loads
        Raw8<kFp32> old[LATE ? 1 : NV];
        auto fetch_old = [&](int v) {
            const int c = (v * TPR + lane) * 8, n = existing(a.cols, c);
            if (a.dx_dt == kBf16)
                old[LATE ? 0 : v].a = __builtin_bit_cast(f32x4, fetch8<kBf16, true>({out, nullptr}, c, n).v);
            else
                old[LATE ? 0 : v] = fetch8<kFp32, true>({out, nullptr}, c, n);
        };
        if (!LATE && a.add_dx) {
#pragma unroll
            for (int v = 0; v < NV; ++v) fetch_old(v);
        }
        float xh[NV][8], g[NV][8];
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8, n = existing(a.cols, c);
            settle8(rx[v], c, n);
            settle8(rd[v], c, n);
            centered8<XD>(rx[v], mean, xh[v]);
            widen8(rd[v], g[v]);
            if (n < 8) keep_first(xh[v], n);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xh[v][e] *= rstd;
                dw[v][e] = __builtin_fmaf(g[v][e], xh[v][e], dw[v][e]);
                db[v][e] += g[v][e];
                g[v][e] *= w[v][e];
                s[0] = __builtin_fmaf(g[v][e], xh[v][e], s[0]);
                s[1] += g[v][e];
            }
        }
        if (row + step < a.rows) fetch(row + step);
        if (!a.dx) continue;
        // two sets of slots in turn: a set is written again only after the
        // other set's barrier, which every reader of the first has passed
        row_sums<TPR>(s, red[parity]);
        parity ^= 1;
        const float k1 = -(s[0] * inv_n) * rstd, k2 = -(s[1] * inv_n) * rstd;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * 8, n = existing(a.cols, c);
            if (n == 0) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) g[v][e] = __builtin_fmaf(g[v][e], rstd, __builtin_fmaf(xh[v][e], k1, k2));
            if (a.add_dx) {
                float o[8];
                if (LATE) fetch_old(v);
                if (a.dx_dt == kBf16) {
                    Raw8<kBf16> h{__builtin_bit_cast(u32x4, old[LATE ? 0 : v].a)};
                    settle8(h, c, n);
                    widen8(h, o);
                } else {
                    settle8(old[LATE ? 0 : v], c, n);
                    widen8(old[LATE ? 0 : v], o);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) g[v][e] += o[e];
            }
            store8<true>(out, a.dx_dt, c, n, g[v]);
        }
    }
    // the block's sums: to the workspace, or as the gradients
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        void* const grad = which ? a.db : a.dw;
        if (!a.part && !grad) continue;
        float* const out = a.part ? a.part + ((int64_t)blockIdx.x * 2 + which) * a.cols : nullptr;
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
                for (int r = 0; r < G; ++r) t += join[r][c];
                if (out)
                    out[c] = t;
                else
                    put_grad(grad, c, t, a.grad_dt, a.accumulate);
            }
        } else {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (v * TPR + lane) * 8, n = existing(a.cols, c);
                if (n == 0) continue;
                if (out) {
                    store8<false>((char*)out, kFp32, c, n, which ? db[v] : dw[v]);
                } else {
                    float old[8];
                    load_param8(a.accumulate ? grad : nullptr, a.grad_dt, c, n, 0.0f, old);
#pragma unroll
                    for (int e = 0; e < 8; ++e) old[e] += which ? db[v][e] : dw[v][e];
                    store8<false>((char*)grad, a.grad_dt, c, n, old);
                }
            }
        }
    }
}

// Rows of any width: one block per row for dx, then column sums by tiles of
// 2048 columns over strips of rows.
template <int XD, int DD>
__global__ __launch_bounds__(1024) void bwd_wide_dx_kernel(BwdArgs a) {
    __shared__ float red[2][16][2];
    const float inv_n = 1.0f / (float)a.cols;
    int parity = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const RowPtr px = row_at<XD>(a.x, a.ld_x, a.rows, a.cols, row), pd = row_at<DD>(a.dy, a.ld_dy, a.rows, a.cols, row);
        const float mean = a.mean[row], rstd = a.rstd[row];
        float s[2] = {0.0f, 0.0f};
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
            s[0] += t1;
            s[1] += t2;
        }
        row_sums<1024>(s, red[parity]);
        parity ^= 1;
        const float c1 = s[0] * inv_n, c2 = s[1] * inv_n;
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
            store8<true>(out, a.dx_dt, (int)c, n, d);
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
        store8<false>((char*)out, kFp32, (int)c, n, dw);
        store8<false>((char*)(out + a.cols), kFp32, (int)c, n, db);
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
        for (int k = group; k < strips; k += 128) {  // eight loads in flight
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = at < 2 * cols && k + 16 * e < strips ? part[(int64_t)(k + 16 * e) * 2 * cols + at] : 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s += v[e];
        }
        __syncthreads();
        sum[group][lane] = s;
        __syncthreads();
        if (group == 0 && at < 2 * cols) {
            s = 0.0f;
#pragma unroll
            for (int g = 0; g < 16; ++g) s += sum[g][lane];
            void* out = at < cols ? dw : db;
            if (out) put_grad(out, at < cols ? at : at - cols, s, grad_dt, accumulate);
        }
    }
}

template <int XD, int DD, int TPR, int NV, int B = norm_block(TPR)>
hipError_t bwd_run(const BwdArgs& a, int strips, hipStream_t stream) {
    bwd_kernel<XD, DD, TPR, NV, B><<<strips, B, 0, stream>>>(a);
    return hipGetLastError();
}

template <int XD, int DD>
hipError_t bwd_pick(const BwdArgs& a, int strips, hipStream_t stream) {
    const int64_t n = a.cols;
    // one block for all rows: as many of them at once as it can hold (16x768 from
    // 8.6 us with 4 at once to 6.8 with 8)
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
    if (a.part) {  // before dx, which may take dy's or x's place
        const int64_t tiles = (n + kThreads * 8 - 1) / (kThreads * 8);
        bwd_wide_sums_kernel<XD, DD><<<grid_for(tiles * strips, kThreads), kThreads, 0, stream>>>(a, strips);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.dx) bwd_wide_dx_kernel<XD, DD><<<grid_for(a.rows, 1024), 1024, 0, stream>>>(a);
    return hipGetLastError();
}

template <int XD>
hipError_t bwd_pick_dy(const BwdArgs& a, zr_dtype dy_dt, int strips, hipStream_t stream) {
    return dy_dt == ZR_BF16 ? bwd_pick<XD, kBf16>(a, strips, stream) : bwd_pick<XD, kFp32>(a, strips, stream);
}

}  // namespace

hipError_t launch_layernorm_bwd(const NormBwd& f, hipStream_t stream) {
    BwdArgs a{};
    a.dy = f.dy; a.x = f.x; a.w = f.weight; a.mean = f.mean; a.rstd = f.rstd;
    a.dx = (char*)f.dx;
    a.rows = f.rows; a.cols = f.cols; a.ld_dy = f.ld_dy; a.ld_x = f.ld_x; a.ld_dx = f.ld_dx;
    a.param_dt = f.param_dt; a.dx_dt = f.dx_dt; a.add_dx = f.add_dx;
    const bool grads = f.dweight || f.dbias;
    const int strips = layernorm_strips(f.rows, f.cols);
    const bool joined = layernorm_workspace(f.rows, f.cols) > 0 || strips == 0;
    a.part = grads && joined ? (float*)f.workspace : nullptr;
    if (!joined) {
        a.dw = f.dweight; a.db = f.dbias;
        a.grad_dt = f.grad_dt; a.accumulate = f.accumulate;
    }
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
    if (!grads || !joined) return e;
    const int64_t tiles = (2 * f.cols + 63) / 64;
    bwd_join_kernel<<<grid_for(tiles, 1024), 1024, 0, stream>>>((const float*)f.workspace, strips, f.cols, f.dweight, f.dbias,
                                                          f.grad_dt, f.accumulate);
    return hipGetLastError();
}

}  // namespace zr
