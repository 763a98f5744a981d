// rows.hpp -- typed row access of the operators around the recurrences
// (layer norm, embedding, linear attention): fp32 and bf16 elements in device
// memory, fp32 in registers, moved in vectors of V elements.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"

namespace prn {

typedef __bf16 bf16;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Elements of T that one 16-byte access moves.
template <typename T> constexpr int kVec = 16 / (int)sizeof(T);

template <typename T, int V>
struct alignas(sizeof(T) * V) VecT {
    T v[V];
};

template <typename T, int V>
__device__ __forceinline__ void load_vec(const T *p, float (&f)[V]) {
    const VecT<T, V> x = *reinterpret_cast<const VecT<T, V> *>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = (float)x.v[i];
}
// Elements that a launch reads exactly once (streamed past the caches, like
// ld_once); 16-byte vectors, ordinary loads of single elements.
template <typename T, int V>
__device__ __forceinline__ VecT<T, V> load_once(const T *p) {
    if constexpr (sizeof(T) * V == 16) {
        union {
            u32x4 w;
            VecT<T, V> v;
        } x;
        x.w = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
        return x.v;
    } else {
        return *reinterpret_cast<const VecT<T, V> *>(p);
    }
}
// Rounds to T (bf16: to nearest, ties to even).
template <typename T, int V>
__device__ __forceinline__ void store_vec(T *p, const float (&f)[V]) {
    VecT<T, V> x;
#pragma unroll
    for (int i = 0; i < V; ++i) x.v[i] = (T)f[i];
    *reinterpret_cast<VecT<T, V> *>(p) = x;
}
// Groups of kVec elements that begin at any element, moved in words of 4
// bytes, four at a time: a group of bf16 that begins inside a word is put
// together from the five words that hold it (its own elements lie in each, so
// each is memory of the same allocation).  Where a row is shorter than a
// group, its n elements move singly; the last group of a longer row is taken
// back to end with the row (group_at), so that two lanes share some columns
// and no group needs a branch of its own.
typedef u32x4 u32x4_any __attribute__((aligned(4)));
typedef uint32_t u32x3_any __attribute__((ext_vector_type(3), aligned(4)));
template <typename T>
__device__ __forceinline__ void load_any(const T *p, int n, float (&f)[kVec<T>]) {
    constexpr int V = kVec<T>;
    if (n < V) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = i < n ? (float)p[i] : 0.0f;
        return;
    }
    union {
        uint32_t w[4];
        T v[V];
    } x;
    const uint32_t odd = (uint32_t)(uintptr_t)p & 2u;
    const uint32_t *q = reinterpret_cast<const uint32_t *>((uintptr_t)p - odd);
    const u32x4 a = *reinterpret_cast<const u32x4_any *>(q);
    uint32_t last = 0;
    if (sizeof(T) == 2) last = q[3 + (odd >> 1)];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x.w[i] = sizeof(T) == 2 ? __builtin_amdgcn_alignbit(i < 3 ? a[i + 1] : last, a[i], odd << 3) : a[i];
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = (float)x.v[i];
}
template <typename T>
__device__ __forceinline__ void store_any(T *p, int n, const float (&f)[kVec<T>]) {
    constexpr int V = kVec<T>;
    if (n < V) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < n) p[i] = (T)f[i];
        return;
    }
    union {
        uint32_t w[4];
        T v[V];
    } x;
#pragma unroll
    for (int i = 0; i < V; ++i) x.v[i] = (T)f[i];
    if (sizeof(T) == 2 && ((uintptr_t)p & 2u)) {
        u32x3_any m;
#pragma unroll
        for (int i = 0; i < 3; ++i) m[i] = __builtin_amdgcn_alignbit(x.w[i + 1], x.w[i], 16);
        p[0] = x.v[0];
        *reinterpret_cast<u32x3_any *>(p + 1) = m;
        p[V - 1] = x.v[V - 1];
    } else {
        *reinterpret_cast<u32x4_any *>(p) = u32x4{x.w[0], x.w[1], x.w[2], x.w[3]};
    }
}
// Where the group that holds column c of a row of D begins.
template <typename T, bool VEC>
__device__ __forceinline__ int group_at(int c, int D) {
    return VEC || D < kVec<T> ? c : min(c, D - kVec<T>);
}
// A group of a row: VEC, if every row's groups are whole and 16-byte aligned.
// D: the row's elements (below kVec: the only group's).
template <typename T, bool VEC>
__device__ __forceinline__ void load_group(const T *p, int D, float (&f)[kVec<T>]) {
    if constexpr (VEC) load_vec<T, kVec<T>>(p, f);
    else load_any<T>(p, D, f);
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_group(T *p, int D, const float (&f)[kVec<T>]) {
    if constexpr (VEC) store_vec<T, kVec<T>>(p, f);
    else store_any<T>(p, D, f);
}

// Sum over the 64 lanes of a wave, in every lane: neighbours within rows of
// 16, then across rows, on the vector unit (no LDS traffic).
template <int CTRL, int ROWS>
__device__ __forceinline__ float add_dpp(float v) {
    return v + __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ float lanes_sum(float v) {
    v = add_dpp<0x111, 0xf>(v);  // row_shr:1
    v = add_dpp<0x112, 0xf>(v);  // row_shr:2
    v = add_dpp<0x114, 0xf>(v);  // row_shr:4
    v = add_dpp<0x118, 0xf>(v);  // row_shr:8: lane 15 of a row has the row's sum
    v = add_dpp<0x142, 0xa>(v);  // row_bcast:15 into rows 1 and 3
    v = add_dpp<0x143, 0xc>(v);  // row_bcast:31 into rows 2 and 3
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// Sum over each row of 16 lanes, in every lane of it (rotations by 8, 4, 2, 1).
__device__ __forceinline__ float lanes16_sum(float v) {
    v = add_dpp<0x128, 0xf>(v);
    v = add_dpp<0x124, 0xf>(v);
    v = add_dpp<0x122, 0xf>(v);
    return add_dpp<0x121, 0xf>(v);
}

}  // namespace prn
