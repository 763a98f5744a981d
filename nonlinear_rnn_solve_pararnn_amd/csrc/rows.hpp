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

}  // namespace prn
