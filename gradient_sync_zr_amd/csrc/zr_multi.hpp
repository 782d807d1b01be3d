// Lists of tensors for the kernels that walk over many at once: addresses and
// sizes in the kernel's arguments, the tensors cut into tiles that never cross
// from one to the next, so that a block's tile has one address for each list.
//
// A tile is read and written by quads of 4 elements, 64 lanes' quads side by
// side, at element alignment: tensors start anywhere. The tiles of a call that writes
// start on the 128-byte lines of what it writes (the first tile begins `skew` elements
// before its tensor): AdamW of 2^25 parameters off the lines took 198 us for 173.
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

// Elements of es bytes that lie between the line's start and p.
__host__ __device__ __forceinline__ int line_skew(const void* p, int es) {
    return (int)((uintptr_t)p / (unsigned)es & (128u / (unsigned)es - 1));
}

// Fills `m` with the tensors from `first` on (lists[k] may be null) in tiles of TILE
// elements, on the lines of list BY, of elements of es bytes (BY < 0: from the
// tensors' starts); tensors of no elements are stepped over. Returns the first that is
// left.
template <int TILE, int BY, int NP, int PER>
inline int multi_fill(Multi<NP, PER>* m, int first, int n, const void* const* const (&lists)[NP], const int64_t* numels,
                      int es = 4) {
    m->count = 0;
    m->tile0[0] = 0;
    int i = first;
    for (; i < n && m->count < PER; ++i) {
        if (numels[i] == 0) continue;
        const int at = m->count++;
        for (int k = 0; k < NP; ++k) m->p[k][at] = lists[k] ? lists[k][i] : nullptr;
        m->n[at] = numels[i];
        const int64_t with_skew = numels[i] + (BY < 0 ? 0 : line_skew(m->p[BY < 0 ? 0 : BY][at], es));
        m->tile0[at + 1] = m->tile0[at] + (int32_t)((with_skew + TILE - 1) / TILE);
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

// The part of a quad that a tensor of n elements has: elements lo to hi - 1, where
// the quad starts at element `at` (which may be before the tensor).
struct Span {
    int lo, hi;
    __device__ __forceinline__ bool whole() const { return lo <= 0 && hi >= 4; }
};
__device__ __forceinline__ Span quad_span(int64_t at, int64_t n) {
    return {at < 0 ? (int)-at : 0, n - at < 4 ? (int)(n - at) : 4};
}

// The quad at p: zeros where it does not exist.
template <typename T, bool NT>
__device__ __forceinline__ void load_quad4(const T* p, Span s, float f[4]) {
    if (s.whole()) {
        widen4(quad_at<NT>(p), f);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = e >= s.lo && e < s.hi ? load_elem(p + e) : 0.0f;
    }
}
template <typename T, bool NT>
__device__ __forceinline__ void store_quad4(T* p, Span s, const float f[4]) {
    if (s.whole()) {
        quad_to<NT>(p, pack4<T>(f));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e >= s.lo && e < s.hi) store_elem(p + e, f[e]);
    }
}

}  // namespace zr
