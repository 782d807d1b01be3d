// AdamW over many tensors, with the gradients multiplied by a coefficient that
// lies on the device (the clipping's), so that clipping costs no pass:
//     g' = coef * g
//     m  = beta1 * m + (1 - beta1) * g'
//     v  = beta2 * v + (1 - beta2) * g'^2
//     p  = (1 - lr * decay) * p - lr / (1 - beta1^t) * m / (sqrt(v / (1 - beta2^t)) + eps)
// in fp32, and p rounded to bf16 as the shard that the all-gather takes. A
// coefficient that is not finite leaves everything as it was. Steps so left out may be
// counted on the device: t is then the step less those, and the corrections come from
// there, as the host does not know of them (hidden: 337 us for 335 of 2^26 from bf16).
//
// A stream of 30 bytes per element (fp32 gradients, shards written), read and
// written past the caches: 2^26 elements take 359 us (5.6 TB/s), 335 (5.6) from bf16
// gradients, which is what the card moves with as much written as read (a scaling from
// fp32 to fp32: 5.6); with cached accesses 389. Tiles inside a tensor have a path
// without the quads' borders, whose branches held the loads apart (bf16 365 without it).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "zr_multi.hpp"

namespace zr {
namespace {

typedef Multi<5, kAdamPer> AdamTable;

struct AdamArgs {
    const float* coef;
    int64_t* left_out;  // steps left out so far, or null
    int64_t step;
    double lr, b1, b2;
    float beta1, rest1, beta2, rest2, keep, rate, inv2, eps;
    int count;  // this launch counts the step that it leaves out
};

// b^t by squaring, t >= 1: off by less than t roundings of fp64.
__device__ double power(double b, int64_t t) {
    double r = 1.0;
#pragma unroll 1
    for (; t > 0; t >>= 1) {
        if (t & 1) r *= b;
        b *= b;
    }
    return r;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamTable t5, AdamArgs a, int shards) {
    const float coef = a.coef ? *a.coef : 1.0f;
    if (!(__builtin_fabsf(coef) < __builtin_inff())) {
        // nobody reads it in a step that is left out
        if (a.count && blockIdx.x == 0 && threadIdx.x == 0) *a.left_out += 1;
        return;
    }
    const int64_t less = a.left_out ? *a.left_out : 0;
    if (less > 0) {  // the same for all; otherwise the host's corrections hold
        const int64_t t = a.step - less > 1 ? a.step - less : 1;
        a.rate = (float)(a.lr / (1.0 - power(a.b1, t)));
        a.inv2 = (float)(1.0 / (1.0 - power(a.b2, t)));
    }
    int slot = 0;
    const int tiles = t5.tile0[t5.count];
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
        slot = multi_slot(t5, slot, t);
        float* const pp = (float*)t5.p[1][slot];
        const int64_t begin = (int64_t)(t - t5.tile0[slot]) * kMultiTile - line_skew(pp, 4), n = t5.n[slot];
        const T* const pg = (const T*)t5.p[0][slot];
        float* const pm = (float*)t5.p[2][slot];
        float* const pv = (float*)t5.p[3][slot];
        uint16_t* const ps = (uint16_t*)t5.p[4][slot];
        auto quads = [&](auto whole) {
#pragma unroll
            for (int k = 0; k < kMultiQuads; ++k) {
                const int64_t at = begin + (threadIdx.x + k * kThreads) * 4;
                if (!whole && at >= n) break;
                const Span l = whole ? Span{0, 4} : quad_span(at, n);
                float g[4], p[4], m[4], v[4];
                load_quad4<float, true>(pp + at, l, p);
                load_quad4<float, true>(pm + at, l, m);
                load_quad4<float, true>(pv + at, l, v);
                load_quad4<T, true>(pg + at, l, g);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = g[e] * coef;
                    m[e] = __builtin_fmaf(a.beta1, m[e], a.rest1 * x);
                    v[e] = __builtin_fmaf(a.beta2, v[e], a.rest2 * x * x);
                    const float root = __fsqrt_rn(v[e] * a.inv2) + a.eps;
                    p[e] = __builtin_fmaf(a.keep, p[e], -a.rate * __fdiv_rn(m[e], root));
                }
                store_quad4<float, true>(pp + at, l, p);
                store_quad4<float, true>(pm + at, l, m);
                store_quad4<float, true>(pv + at, l, v);
                if (shards) store_quad4<uint16_t, true>(ps + at, l, p);
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

hipError_t launch_adamw(const AdamW& f, hipStream_t stream) {
    const void* const* const lists[5] = {f.grads, (const void* const*)f.params, (const void* const*)f.exp_avg,
                                         (const void* const*)f.exp_avg_sq, (const void* const*)f.shards};
    AdamArgs a{};
    a.coef = f.coef;
    a.left_out = f.left_out;
    a.step = f.step;
    a.lr = f.lr; a.b1 = f.beta1; a.b2 = f.beta2;
    a.count = f.left_out != nullptr;
    a.beta1 = (float)f.beta1; a.rest1 = (float)(1.0 - f.beta1);
    a.beta2 = (float)f.beta2; a.rest2 = (float)(1.0 - f.beta2);
    a.keep = (float)(1.0 - f.lr * f.weight_decay);
    a.rate = (float)(f.lr / (1.0 - __builtin_pow(f.beta1, (double)f.step)));
    a.inv2 = (float)(1.0 / (1.0 - __builtin_pow(f.beta2, (double)f.step)));
    a.eps = (float)f.eps;
    AdamTable m;
    for (int next = multi_fill<kMultiTile, 1>(&m, 0, f.n, lists, f.numels); m.count > 0; next = multi_fill<kMultiTile, 1>(&m, next, f.n, lists, f.numels)) {
        const int grid = grid_for(m.tile0[m.count], kThreads);
        if (f.grad_dt == ZR_BF16)
            adamw_kernel<uint16_t><<<grid, kThreads, 0, stream>>>(m, a, f.shards != nullptr);
        else
            adamw_kernel<float><<<grid, kThreads, 0, stream>>>(m, a, f.shards != nullptr);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        a.count = 0;
    }
    return hipSuccess;
}

}  // namespace zr
