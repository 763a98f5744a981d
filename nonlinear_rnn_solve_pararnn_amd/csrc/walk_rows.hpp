// walk_rows.hpp -- where the walk kernel (walk.hpp) finds the rows of its
// operands: a chunk's bytes, the groups of 8 elements that a thread loads, and
// which of a group's elements are the chunk's own.  Host- and device-callable,
// so that a host program can check every offset.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace prn {
namespace walk {

constexpr int kThreads = 256;

constexpr uint32_t kNowhere = 0x80000000u;  // above every buffer's size, also after a chunk's bytes are taken off

// Rows of one operand as a walk's segment sees them, from column c0 on, in
// chunks of C positions.
struct Rows {
    const char *p;       // the first chunk, if it is whole: its lowest address
    int64_t step;        // bytes from a chunk to the next one
    uint32_t row_bytes;  // below 2^24 (checked on the host)
    uint32_t tail;       // bytes of a row from p on
    int rev;

    // Address and bytes of chunk i of cnt positions (none: nothing to read or write).
    __host__ __device__ __forceinline__ const char *at(int i, int cnt, int C) const {
        return p + i * step + (rev ? (C - cnt) * (int64_t)row_bytes : 0);
    }
    __host__ __device__ __forceinline__ uint32_t bytes(int cnt) const {
        return cnt == 0 ? 0u : (uint32_t)(cnt - 1) * row_bytes + tail;
    }
    // The same in whole words of memory, for rows of 2-byte elements that begin
    // anywhere: the buffer begins `skew` bytes before the chunk's first element
    // and ends with the word that holds the last one.  Its first and its last
    // word may each hold one element of others (see Groups::past).
    __host__ __device__ __forceinline__ static uint32_t word_skew(const char *first) { return (uint32_t)(uintptr_t)first & 3u; }
    __host__ __device__ __forceinline__ uint32_t word_bytes(uint32_t skew, int cnt) const {
        return cnt == 0 ? 0u : (skew + bytes(cnt) + 3u) & ~3u;
    }
    // Offset of a chunk's row r in it, if the chunk is whole; shift() less in a shorter one.
    __host__ __device__ __forceinline__ uint32_t row_at(int r, int C) const { return (uint32_t)(rev ? C - 1 - r : r) * row_bytes; }
    __host__ __device__ __forceinline__ uint32_t shift(int cnt, int C) const { return rev ? (uint32_t)(C - cnt) * row_bytes : 0u; }
};
// first: position 0's address; row: bytes from a position to the next; tail: bytes of a row.
__host__ __device__ __forceinline__ Rows rows_from(const char *first, int64_t row, uint32_t tail, int64_t L, int64_t begin, int C,
                                                   int rev) {
    return {first + (rev ? L - begin - C : begin) * row, rev ? -row * C : row * C, (uint32_t)row, tail, rev};
}

// A thread's groups of 8 elements of a tile of W columns.
template <int W, int C>
struct Groups {
    static constexpr int kGroups = W / 8, kN = (C * kGroups + kThreads - 1) / kThreads;
    // Where the groups of a row divide the threads, a thread's groups are the
    // same columns kThreads / kGroups rows apart and one offset tells them all.
    static constexpr bool kEven = kThreads % kGroups == 0;
    static constexpr int kStep = kThreads / kGroups;
    uint32_t at[kEven ? 1 : kN];  // offsets in a whole chunk
    int left;                     // columns the operand has
    int thread;

    __host__ __device__ __forceinline__ void init(const Rows &v, int elem_bytes, int thread_) {
        thread = thread_;
        left = (int)(v.tail / (uint32_t)elem_bytes);
#pragma unroll
        for (int n = 0; n < (kEven ? 1 : kN); ++n)
            at[n] = row(n) < C && column(n) < left ? v.row_at(row(n), C) + (uint32_t)(column(n) * elem_bytes) : kNowhere;
    }
    __host__ __device__ __forceinline__ static int row_of(int thread, int n) { return (int)((uint32_t)(thread + n * kThreads) / kGroups); }
    __host__ __device__ __forceinline__ int row(int n) const { return row_of(thread, n); }
    __host__ __device__ __forceinline__ int column(int n) const { return (int)((uint32_t)(thread + n * kThreads) % kGroups) * 8; }
    __host__ __device__ __forceinline__ uint32_t offset(const Rows &v, int n, uint32_t shift) const {
        return kEven ? at[0] + ((uint32_t)(v.rev ? -n : n) * kStep * v.row_bytes - shift) : at[kEven ? 0 : n] - shift;
    }
    // Whether a thread's group n is a row past the last of cnt positions.  Such a
    // row may have found an element of others in the buffer's end words, or (rows
    // that overlap) elements of its own rows inside it, and a NaN there would
    // reach the chunk's results through products with zero.
    __host__ __device__ __forceinline__ static bool past(int thread, int n, int cnt) { return row_of(thread, n) >= cnt; }
    // How many of group n's elements are its row's; what follows them in memory belongs to others.
    __host__ __device__ __forceinline__ int own(int n) const { return left - column(n); }
    // Word k of a group of which `valid` elements of elem_bytes are its own.
    __host__ __device__ __forceinline__ static uint32_t own_word(uint32_t x, int k, int elem_bytes, int valid) {
        const int per = 4 / elem_bytes;
        if (per == 2 && valid == k * per + 1) x &= 0xffffu;
        return valid <= k * per ? 0u : x;
    }
};

}  // namespace walk
}  // namespace prn
