// Lists of tensors for the kernels that walk over many at once: addresses and
// sizes in the kernel's arguments, the tensors cut into tiles that never cross
// from one to the next, so that a block's tile has one address for each list.
//
// A tile is read and written by quads of 4 elements, 64 lanes' quads side by
// side, at element alignment: tensors start anywhere.
#pragma once

#include "zr_device.hpp"
#include "zr_internal.hpp"

namespace zr {

constexpr int kMultiQuads = 4;                            // quads of a thread and tile
constexpr int kMultiTile = kThreads * 4 * kMultiQuads;    // elements

// NP lists of up to PER tensors; tile t of the launch lies in the tensor m with
// tile0[m] <= t < tile0[m + 1].
template <int NP, int PER>
struct Multi {
    const void* p[NP][PER];
    int64_t n[PER];
    int32_t tile0[PER + 1];
    int32_t count;
};

// Fills `m` with the tensors from `first` on (lists[k] may be null) in tiles of TILE
// elements; tensors of no elements are stepped over. Returns the first that is left.
template <int TILE, int NP, int PER>
inline int multi_fill(Multi<NP, PER>* m, int first, int n, const void* const* const (&lists)[NP], const int64_t* numels) {
    m->count = 0;
    m->tile0[0] = 0;
    int i = first;
    for (; i < n && m->count < PER; ++i) {
        if (numels[i] == 0) continue;
        const int at = m->count++;
        for (int k = 0; k < NP; ++k) m->p[k][at] = lists[k] ? lists[k][i] : nullptr;
        m->n[at] = numels[i];
        m->tile0[at + 1] = m->tile0[at] + (int32_t)((numels[i] + TILE - 1) / TILE);
    }
    while (i < n && numels[i] == 0) ++i;
    return i;
}

// The tensor of tile t, from a lower bound on; the same in every lane.
template <int NP, int PER>
__device__ __forceinline__ int multi_slot(const Multi<NP, PER>& m, int from, int t) {
    return m.count == 1 ? 0 : __builtin_amdgcn_readfirstlane(find_slot(m.tile0, m.count, from, t));
}

// Quads at element alignment.
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef f32x4 quad_f32 __attribute__((aligned(4)));

template <bool NT>
__device__ __forceinline__ Quad<uint16_t> quad_at(const uint16_t* p) {
    const u32x2_a2* q = (const u32x2_a2*)p;
    return {NT ? (u32x2)__builtin_nontemporal_load(q) : (u32x2)*q};
}
template <bool NT>
__device__ __forceinline__ Quad<float> quad_at(const float* p) {
    const quad_f32* q = (const quad_f32*)p;
    return {NT ? (f32x4)__builtin_nontemporal_load(q) : (f32x4)*q};
}
template <bool NT>
__device__ __forceinline__ void quad_to(uint16_t* p, const Quad<uint16_t>& v) {
    if constexpr (NT)
        __builtin_nontemporal_store(v.v, (u32x2_a2*)p);
    else
        *(u32x2_a2*)p = v.v;
}
template <bool NT>
__device__ __forceinline__ void quad_to(float* p, const Quad<float>& v) {
    if constexpr (NT)
        __builtin_nontemporal_store(v.v, (quad_f32*)p);
    else
        *(quad_f32*)p = v.v;
}

// The quad at p of which `left` elements exist (4: all): zeros behind them.
template <typename T, bool NT>
__device__ __forceinline__ void load_quad4(const T* p, int left, float f[4]) {
    if (left >= 4) {
        widen4(quad_at<NT>(p), f);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = e < left ? load_elem(p + e) : 0.0f;
    }
}
template <typename T, bool NT>
__device__ __forceinline__ void store_quad4(T* p, int left, const float f[4]) {
    if (left >= 4) {
        quad_to<NT>(p, pack4<T>(f));
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < left) store_elem(p + e, f[e]);
    }
}

}  // namespace zr
