// The global norm of many tensors, the coefficient that clips it, and tensors
// multiplied by that coefficient.
//     norm = scale * sqrt(sum g^2),  coef = scale * min(1, max_norm / norm)
//
// Squares are taken and summed in fp64: those of all finite fp32 values lie in
// its normal range (2^-298 to 2^256), so nothing overflows or vanishes whatever
// the gradients' size. Blocks walk over tiles and leave one partial sum each; a
// single block adds them in order, so the result does not change from run to run.
//
// The norm is one read: tiles of 8192 elements, whose loads are all in front, past
// the caches where the tensors exceed them (2^30 bf16 elements 320 us for 396 with
// 4096 and cached). 2^30 elements take 615 to 670 us of fp32 (6.4 to 7.0 TB/s) and
// 320 of bf16 (6.7); 2^27 take 81 and 44. The fp64 arithmetic, 2 operations per
// element, is hidden. Up to 16384 elements go through one block in one launch, where
// two launches cost 3.6 us more. Scaling reads and writes once: 2^30 elements of fp32
// in place 5.6 TB/s, to bf16 6.28. Tiles inside a tensor have a path without the quads'
// borders, whose branches held the loads apart (2^26 of bf16 in place 43 us for 48), and
// a tensor's last tile loads its whole vectors at once too (the norm of 290 ragged bf16
// tensors, 31M elements, 20 us for 27).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "zr_ckpt.hpp"
#include "zr_multi.hpp"

namespace zr {
namespace {

typedef Multi<1, kNormPer> NormTable;
typedef Multi<2, kScalePer> ScaleTable;

__device__ __forceinline__ double swap_add(double v, int lanes) { return v + __shfl_xor(v, lanes, 64); }

// Sum of v over a block of T threads, in lane 0 of wave 0.
template <int T>
__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
    for (int k = 1; k < 64; k *= 2) v = swap_add(v, k);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x / 64] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < T / 64; ++w) s += red[w];
    return s;
}

struct NormOut {
    float *norm, *coef;
    double scale, max_norm;
};

__device__ __forceinline__ void put_norm(const NormOut& o, double sum) {
    const double norm = o.scale * sqrt(sum);
    // a norm that is not finite leaves no coefficient
    const bool finite = sum < __builtin_inf();
    const double coef = finite ? (norm > o.max_norm ? o.scale * (o.max_norm / norm) : o.scale) : __builtin_nan("");
    if (o.norm) *o.norm = (float)norm;
    if (o.coef) *o.coef = (float)coef;
}

// Vectors of a lane in a tile, of 16 bytes: 8 of 4 fp32 elements, or 4 of 8 bf16.
template <typename T>
constexpr int kNormVecs = kNormTile / kThreads / (16 / (int)sizeof(T));

// The squares of this thread's share of the launch's tiles, all of a tile's loads in
// front. NT: past the caches.
template <typename T, bool NT>
__device__ __forceinline__ double squares(const NormTable& m, int first, int step) {
    constexpr int E = 16 / (int)sizeof(T), V = kNormVecs<T>;
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    int slot = 0;
    const int tiles = m.tile0[m.count];
    for (int t = first; t < tiles; t += step) {
        slot = multi_slot(m, slot, t);
        const int64_t begin = (int64_t)(t - m.tile0[slot]) * kNormTile, left = m.n[slot] - begin;
        const int c = (int)(threadIdx.x % kThreads) * E;
        const T* p = (const T*)m.p[0][slot] + begin + c;
        auto add = [&](const float f[E]) {
#pragma unroll
            for (int e = 0; e < E; ++e) s[e & 3] = __builtin_fma((double)f[e], (double)f[e], s[e & 3]);
        };
        auto vectors = [&](auto whole) {
            u32x4 raw[V];
#pragma unroll
            for (int k = 0; k < V; ++k) {
                raw[k] = u32x4{0, 0, 0, 0};
                if (!whole && left - c - k * kThreads * E < E) continue;
                if constexpr (sizeof(T) == 2)
                    raw[k] = ld16<NT>((const uint16_t*)p + k * kThreads * E);
                else
                    raw[k] = __builtin_bit_cast(u32x4, ld32<NT>((const float*)p + k * kThreads * E));
            }
#pragma unroll
            for (int k = 0; k < V; ++k) {
                float f[E];
                if constexpr (sizeof(T) == 2) {
                    widen8(Raw8<kBf16>{raw[k]}, f);
                } else {
                    const f32x4 v = __builtin_bit_cast(f32x4, raw[k]);
                    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
                }
                add(f);
            }
        };
        if (left >= kNormTile) {  // the same for the block
            vectors(std::true_type{});
        } else {
            vectors(std::false_type{});
            // the tensor's last elements, less than a vector: one to a thread
            const int64_t last = left / E * E + threadIdx.x % kThreads;
            if (last < left) {
                const float f = load_elem(p - c + last);
                s[0] = __builtin_fma((double)f, (double)f, s[0]);
            }
        }
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

template <typename T, bool NT>
__global__ __launch_bounds__(kThreads) void norm_kernel(NormTable m, double* part) {
    __shared__ double red[kThreads / 64];
    const double s = block_sum<kThreads>(squares<T, NT>(m, blockIdx.x, gridDim.x), red);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// Everything in one block, where there is little.
template <typename T>
__global__ __launch_bounds__(1024) void norm_one_kernel(NormTable m, NormOut o) {
    __shared__ double red[16];
    const double s = block_sum<1024>(squares<T, false>(m, threadIdx.x / kThreads, 1024 / kThreads), red);
    if (threadIdx.x == 0) put_norm(o, s);
}

__global__ __launch_bounds__(1024) void norm_join_kernel(const double* part, int count, NormOut o) {
    __shared__ double red[16];
    double s = 0.0;
    for (int i = threadIdx.x; i < count; i += 1024) s += part[i];
    s = block_sum<1024>(s, red);
    if (threadIdx.x == 0) put_norm(o, s);
}

// In place a coefficient of 1 leaves nothing to do.
template <typename T, typename U>
__global__ __launch_bounds__(kThreads) void scale_kernel(ScaleTable m, const float* coef, int in_place) {
    const float k1 = *coef;
    if (in_place && k1 == 1.0f) return;
    int slot = 0;
    const int tiles = m.tile0[m.count];
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
        slot = multi_slot(m, slot, t);
        const T* const p = (const T*)m.p[0][slot];
        U* const q = (U*)m.p[1][slot];
        const int64_t begin = (int64_t)(t - m.tile0[slot]) * kMultiTile - line_skew(q, sizeof(U)), n = m.n[slot];
        auto quads = [&](auto whole) {
            auto span = [&](int64_t at) { return whole ? Span{0, 4} : quad_span(at, n); };
            float f[kMultiQuads][4];
#pragma unroll
            for (int k = 0; k < kMultiQuads; ++k) {
                const int64_t at = begin + (threadIdx.x + k * kThreads) * 4;
                load_quad4<T, true>(p + at, span(at), f[k]);
            }
#pragma unroll
            for (int k = 0; k < kMultiQuads; ++k) {
                const int64_t at = begin + (threadIdx.x + k * kThreads) * 4;
#pragma unroll
                for (int e = 0; e < 4; ++e) f[k][e] *= k1;
                store_quad4<U, true>(q + at, span(at), f[k]);
            }
        };
        // the same for the block; without the quads' borders all loads go out in front
        if (begin >= 0 && n - begin >= kMultiTile)
            quads(std::true_type{});
        else
            quads(std::false_type{});
    }
}

}  // namespace

hipError_t launch_grad_norm(const GradNorm& f, hipStream_t stream) {
    const void* const* const lists[1] = {f.grads};
    const NormOut o{f.norm, f.coef, (double)f.scale, (double)f.max_norm};
    double* const part = (double*)f.workspace;
    // what the caches hold stays there for the call that scales it or takes the step
    int64_t total = 0;
    for (int i = 0; i < f.n; ++i) total += f.numels[i];
    const bool far = total * (f.dt == ZR_BF16 ? 2 : 4) > kCachedBytes;
    NormTable m;
    int next = multi_fill<kNormTile, -1>(&m, 0, f.n, lists, f.numels), parts = 0;
    if (next == f.n && m.tile0[m.count] <= 4 && total <= kNormOneElems) {
        if (f.dt == ZR_BF16)
            norm_one_kernel<uint16_t><<<1, 1024, 0, stream>>>(m, o);
        else
            norm_one_kernel<float><<<1, 1024, 0, stream>>>(m, o);
        return hipGetLastError();
    }
    while (m.count > 0) {
        const int64_t tiles = m.tile0[m.count];
        const int grid = grid_for(tiles < kNormBlocks ? tiles : kNormBlocks, kThreads);
        if (f.dt == ZR_BF16 && far)
            norm_kernel<uint16_t, true><<<grid, kThreads, 0, stream>>>(m, part + parts);
        else if (f.dt == ZR_BF16)
            norm_kernel<uint16_t, false><<<grid, kThreads, 0, stream>>>(m, part + parts);
        else if (far)
            norm_kernel<float, true><<<grid, kThreads, 0, stream>>>(m, part + parts);
        else
            norm_kernel<float, false><<<grid, kThreads, 0, stream>>>(m, part + parts);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        parts += grid;
        next = multi_fill<kNormTile, -1>(&m, next, f.n, lists, f.numels);
    }
    norm_join_kernel<<<1, 1024, 0, stream>>>(part, parts, o);
    return hipGetLastError();
}

hipError_t launch_grad_scale(const GradScale& f, hipStream_t stream) {
    const bool in_place = !f.outs;
    const void* const* const lists[2] = {f.grads, in_place ? f.grads : (const void* const*)f.outs};
    ScaleTable m;
    const int es = f.out_dt == ZR_BF16 ? 2 : 4;
    for (int next = multi_fill<kMultiTile, 1>(&m, 0, f.n, lists, f.numels, es); m.count > 0;
         next = multi_fill<kMultiTile, 1>(&m, next, f.n, lists, f.numels, es)) {
        const int grid = grid_for(m.tile0[m.count], kThreads);
        if (f.dt == ZR_BF16 && f.out_dt == ZR_BF16)
            scale_kernel<uint16_t, uint16_t><<<grid, kThreads, 0, stream>>>(m, f.coef, in_place);
        else if (f.dt == ZR_BF16)
            scale_kernel<uint16_t, float><<<grid, kThreads, 0, stream>>>(m, f.coef, in_place);
        else if (f.out_dt == ZR_BF16)
            scale_kernel<float, uint16_t><<<grid, kThreads, 0, stream>>>(m, f.coef, in_place);
        else
            scale_kernel<float, float><<<grid, kThreads, 0, stream>>>(m, f.coef, in_place);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace zr
