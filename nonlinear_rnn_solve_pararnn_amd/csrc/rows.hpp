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
// Rounds to T (bf16: to nearest, ties to even).
template <typename T, int V>
__device__ __forceinline__ void store_vec(T *p, const float (&f)[V]) {
    VecT<T, V> x;
#pragma unroll
    for (int i = 0; i < V; ++i) x.v[i] = (T)f[i];
    *reinterpret_cast<VecT<T, V> *>(p) = x;
}

}  // namespace prn
