// delta_walk.hpp -- the walks of the gated delta rule over its chunks: states
// and outputs, or states alone, from the first chunk on, and the gradient of
// the state from the last chunk back (formulas: delta.hpp, delta_back.hip).
//
// One workgroup walks one (batch row, head) for 64 columns of V; wave w owns
// columns 16 w .. 16 w + 15 and keeps its [D1, 16] columns of S in fp32
// registers, in the layout of walk.hpp, where they are a matrix operand as they
// stand.  The rows of K and of T are read in the order of row_of, so that K S,
// the right side and U come out as the operands of the next product as well:
// between the chunk's operands in LDS and its results nothing crosses the
// waves.  A chunk has one barrier where two chunks fit in LDS (kStages), else two.
//
// A wave is alone on its SIMD in most launches (a (batch row, head) pair has
// only dv / 16 of them), so the chunk's chain of dependent steps is what bounds
// it.  LDS reads are issued a step ahead of the matrix instructions that use
// them, results side by side take turns in the matrix unit, and results are
// stored after the next chunk's operands have arrived (loads and stores are
// waited for in their order).  B=8, L=2048, H=16, 128x128, bf16: 153 us, some
// 5400 cycles a chunk, 2200 of them vector and 1540 matrix instructions.  With S, U
// and P at 16 bits in outputs (which then rounded some values the other way than
// fp32 does) 146; measured like that on a slower card, against 157: before the second
// stage in LDS 163, with T and P in registers 172, with reads left to the compiler
// and one result after the other 199, with the stores before the wait as well 210;
// planes split off by two-element dot products (seven instructions for two numbers,
// not eleven) 169.
#pragma once

#include <type_traits>

#include "delta.hpp"

namespace prn {
namespace delta {

using walk::Ahead;
using walk::kNB;
using walk::kNowhere;
using walk::kTileRow;
using walk::read_row;
using walk::read_tr;
using walk::Rows;
using walk::same_in_lanes;
using walk::split3;
using walk::state_row;
using walk::tile_at;
using walk::u32x2;

enum class Role {
    Out,    // S and o
    State,  // S alone
    Grad    // D, with do in V's place
};

// A [rows, cols] matrix of states in memory.
struct StateAt {
    float *p;
    int64_t row;  // elements from a row to the next
    int rows, cols;
};

// What one workgroup walks.
struct Job {
    HeadView q, k, v;   // v: null for zeros
    int64_t L;
    int b, h, hk, dk, dv;
    int c0;             // first column of V
    int from, to, all;  // chunks: the walk's, and how many there are
    float scale;
    const char *rec;    // of the (batch row, head) pair
    StateAt init;       // null for zeros (or the identity's columns)
    int identity;
    StateAt fin;        // null if not wanted
    // Out
    void *out;          // [B, L, H, dv]
    int H, out4;
    // State and Grad in the backward pass: U or dR, and the states at the ends of every span
    float *rows, *states;
    int64_t row, span_chunks;
};

template <typename T, int D1>
struct alignas(16) WalkLds {
    bf16 K[kPlanes<T> * C * kTileRow<D1>], Q[kPlanes<T> * C * kTileRow<D1>], V[kPlanes<T> * C * kTileRow<kNB>];
    bf16x8 mats[12][64];  // planes of T's two tiles, then of P's
    Gates gates;
};

// Workgroups a CU that a walk's registers are shared out for, and chunks in LDS:
// two where they fit, so that a chunk's operands arrive while the one before is
// at work and it has one barrier.  B=8, L=2048, H=16, 128x128, bf16: the forward
// walk and the two of the backward pass 172 and 360 us with one workgroup, 163
// and 301 with two; the forward walk 163 with one chunk, 157 with two.
template <typename T, int D1> constexpr int kWgs = walk_wgs(sizeof(T) == 2, D1);
template <typename T, int D1> constexpr int kStages = 2 * kWgs<T, D1> * sizeof(WalkLds<T, D1>) <= 160 * 1024 ? 2 : 1;

// Eight numbers of a lane (a column of its wave's, positions 8 q ..) with the
// first ones that are not finite, and all after them, taken out.  Returns the
// first such position of the lane's column, C for none.
__device__ __forceinline__ int take_odd(float (&v)[8], int q) {
    float probe = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) probe = fmaf(v[i], 0.0f, probe);
    if (!__any(probe != 0.0f)) return C;
    int first = C;
#pragma unroll
    for (int i = 7; i >= 0; --i)
        if (abs_bits(v[i]) >= kInfBits) first = 8 * q + i;
    first = min(first, __shfl_xor(first, 16));
    first = min(first, __shfl_xor(first, 32));
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (8 * q + i >= first) v[i] = 0.0f;
    return first;
}

// BACK: records as the backward pass has them; nothing is made of values that are not finite.
template <typename T, int D1, bool VEC, Role ROLE, bool BACK>
__device__ __forceinline__ void walk_chunks(const Job &j, WalkLds<T, D1> (&lds)[kStages<T, D1>]) {
    constexpr bool kOut = ROLE == Role::Out, kGrad = ROLE == Role::Grad, kUseQ = kOut || kGrad;
    constexpr int kP = kPlanes<T>;  // planes of operands (all that is computed has three)
    constexpr int NA = D1 / 16, NT = D1 / 32;
    constexpr int kPX = C * kTileRow<D1>, kPZ = C * kTileRow<kNB>;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, m = lane & 15, q = lane >> 4;
    const int tr_i = m >> 2, tr_c = m & 3;  // this lane's row and column group in a transposing read
    const int col = j.c0 + wave * 16 + m;
    const int last = (int)(j.L - (int64_t)(j.all - 1) * C);

    f32x4 S[NA];
#pragma unroll
    for (int t = 0; t < NA; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = state_row(t, q, r);
            float s = j.identity && row == col ? 1.0f : 0.0f;
            if (j.init.p != nullptr && col < j.init.cols && row < j.init.rows) s = j.init.p[row * j.init.row + col];
            S[t][r] = BACK ? __builtin_canonicalizef(s) : s;  // no signalling NaN (a launch tag) goes into the workspace
        }

    const Rows rq = walk::rows_of<T>(view_of(j.q), j.b, j.hk, j.L, 0, C, 0, 0, j.dk), rk = walk::rows_of<T>(view_of(j.k), j.b, j.hk, j.L, 0, C, 0, 0, j.dk),
               rv = walk::rows_of<T>(view_of(j.v), j.b, j.h, j.L, 0, C, 0, j.c0, j.dv);
    const Rows ro = kOut ? walk::rows_of<T>({j.out, j.L * j.H * j.dv, (int64_t)j.H * j.dv, j.dv}, j.b, j.h, j.L, 0, C, 0, j.c0, j.dv) : rv;
    const int oc = wave * 16 + 4 * q;
    const uint32_t out_at = j.c0 + oc < j.dv ? ro.row_at(m, C) + oc * (uint32_t)sizeof(T) : kNowhere;
    const bool has_v = j.v.p != nullptr;

    Ahead<T, D1, C, VEC> aq, ak;
    Ahead<T, kNB, C, VEC> av;
    if (kUseQ) aq.init(rq);
    ak.init(rk);
    av.init(rv);
    float gate_ahead = 0.0f;
    constexpr int kMats = kUseQ ? 12 : 6, kMyMats = (kMats + 3) / 4;
    bf16x8 mat_ahead[kMyMats];  // this wave's share of T and P
    const int n_chunks = j.to - j.from;
    auto chunk_at = [&](int i) { return kGrad ? j.to - 1 - i : j.from + i; };
    auto positions = [&](int c) { return c < j.all - 1 ? C : last; };
    auto record = [&](int i) { return j.rec + (int64_t)chunk_at(min(i, n_chunks - 1)) * kRecord<BACK>; };
    auto load = [&](int i) {
        const int c = chunk_at(i), cnt = i < n_chunks ? positions(c) : 0;
        ak.load(rk, c, cnt);
        if (kUseQ) aq.load(rq, c, cnt);
        av.load(rv, c, has_v ? cnt : 0);
        const char *r = record(i);
        if (threadIdx.x < sizeof(Gates) / 4) gate_ahead = reinterpret_cast<const float *>(r)[threadIdx.x];
#pragma unroll
        for (int n = 0; n < kMyMats; ++n) {
            const int tile = wave * kMyMats + n;
            const int at = tile < 6 ? (kGrad ? kAtTt : kAtT) + tile * kTile : (kGrad ? kAtPt : kAtP) + (tile - 6) * kTile;
            if (kMats % 4 == 0 || tile < kMats) mat_ahead[n] = *reinterpret_cast<const bf16x8 *>(r + at + lane * 16);
        }
    };
    // a chunk's results on their way out
    using Bits = std::conditional_t<sizeof(T) == 2, u32x2, u32x4>;
    using Bit = std::conditional_t<sizeof(T) == 2, uint16_t, uint32_t>;
    struct alignas(sizeof(Bits)) Four {
        Bit v[4];
    } done[2];
    float done_rows[8];
    auto write = [&](int i) {
        const int c = chunk_at(i);
        if constexpr (kOut) {
            const __amdgpu_buffer_rsrc_t buf = walk::chunk_of(ro, c, positions(c), C);
#pragma unroll
            for (int it = 0; it < 2; ++it) {
                const uint32_t at = out_at + (uint32_t)it * 16 * ro.row_bytes;
                if (j.out4) {
                    if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(Bits, done[it]), buf, at, 0, 0);
                    else __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(Bits, done[it]), buf, at, 0, 0);
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const uint32_t ar = j.c0 + oc + r < j.dv ? at + r * (uint32_t)sizeof(T) : kNowhere;
                        if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b16(done[it].v[r], buf, ar, 0, 0);
                        else __builtin_amdgcn_raw_buffer_store_b32(done[it].v[r], buf, ar, 0, 0);
                    }
                }
            }
        } else if (BACK && j.rows != nullptr) {
#pragma unroll
            for (int n = 0; n < 8; ++n) j.rows[((int64_t)c * C + 8 * q + n) * j.row + col] = done_rows[n];
        }
    };

    // chunk i's operands into LDS, from registers
    auto put = [&](int i, WalkLds<T, D1> &l) {
        const int cnt = positions(chunk_at(i));
        ak.store(rk, l.K);
        if (kUseQ) aq.store(rq, l.Q);
        av.store(rv, l.V);
        if (threadIdx.x < sizeof(Gates) / 4) reinterpret_cast<float *>(&l.gates)[threadIdx.x] = gate_ahead;
#pragma unroll
        for (int n = 0; n < kMyMats; ++n)
            if (kMats % 4 == 0 || wave * kMyMats + n < kMats) l.mats[wave * kMyMats + n][lane] = mat_ahead[n];
        if constexpr (!VEC) {
            if (cnt < C) {
                walk::clear_past<kP, D1, C>(l.K, threadIdx.x, cnt);
                if (kUseQ) walk::clear_past<kP, D1, C>(l.Q, threadIdx.x, cnt);
                walk::clear_past<kP, kNB, C>(l.V, threadIdx.x, cnt);
            }
        }
    };
    // what leaves a chunk late, and a span's state before it
    auto leave = [&](int i) {
        const int c = chunk_at(i);
        if (i > 0) write(i - 1);
        if (BACK && j.states != nullptr) {
            const int span = (int)j.span_chunks, s = c / span;
            if (kGrad ? c == j.all - 1 || c - s * span == span - 1 : c == s * span) {
                float *to = j.states + (int64_t)s * D1 * j.row + col;
#pragma unroll
                for (int t = 0; t < NA; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) to[state_row(t, q, r) * j.row] = S[t][r];
            }
        }
    };
    auto compute = [&](WalkLds<T, D1> &l) {
        // K S in rows of positions, Q S in rows of columns; operands are read, and
        // S split, a step ahead of the matrix instructions that use them
        struct Step {
            bf16x8 k[2][kP], q[2][kP], s[3];
        } step[2];
        auto ahead = [&](int t, Step &to) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int p = 0; p < kP; ++p) {
                    to.k[u][p] = read_row(&l.K[p * kPX + tile_at<D1>(row_of(u, m), 4 * t + q)]);
                    if (kOut) to.q[u][p] = read_row(&l.Q[p * kPX + tile_at<D1>(16 * u + m, 4 * t + q)]);
                }
            const float v[8] = {S[2 * t][0],     S[2 * t][1],     S[2 * t][2],     S[2 * t][3],
                                S[2 * t + 1][0], S[2 * t + 1][1], S[2 * t + 1][2], S[2 * t + 1][3]};
            split3(v, to.s);
        };
        f32x4 ks[2] = {}, o[2] = {};
        bf16x8 z[kP];
        float ge[8];  // f (or r) of the lane's positions
        ahead(0, step[0]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (t + 1 < NT) {
                ahead(t + 1, step[(t + 1) & 1]);
            } else {
                const int grp = 2 * wave + (tr_c >> 1), in = 4 * (tr_c & 1);
#pragma unroll
                for (int p = 0; p < kP; ++p)
                    z[p] = walk::join(read_tr(&l.V[p * kPZ + tile_at<kNB>(8 * q + tr_i, grp) + in]),
                                      read_tr(&l.V[p * kPZ + tile_at<kNB>(8 * q + tr_i + 4, grp) + in]));
#pragma unroll
                for (int n = 0; n < 8; ++n) ge[n] = (kGrad ? l.gates.r : l.gates.f)[8 * q + n];
            }
            const Step &now = step[t & 1];
            mfma_each(now.k, now.s, ks);
            if constexpr (kOut) mfma_each_right(now.s, now.q, o);
            __builtin_amdgcn_sched_barrier(0);
        }
        float gb[8];
#pragma unroll
        for (int n = 0; n < 8; ++n) gb[n] = l.gates.b[8 * q + n];
        bf16x8 Tm[2][3];
#pragma unroll
        for (int n = 0; n < 6; ++n) Tm[n / 3][n % 3] = l.mats[n][lane];
        // the tiles of K^T (and Q^T) for the state's update, a step ahead of their use
        struct Across {
            bf16x8 k[2][kP], q[2][kP];
        } across[2];
        auto columns = [&](int t, Across &to) {
            auto tile = [&](const bf16 *X, int n, int p) {
                const int grp = 4 * t + tr_c, in = 4 * n;
                return walk::join(read_tr(&X[p * kPX + tile_at<D1>(8 * q + tr_i, grp) + in]),
                                  read_tr(&X[p * kPX + tile_at<D1>(8 * q + tr_i + 4, grp) + in]));
            };
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int p = 0; p < kP; ++p) {
                    to.k[n][p] = tile(l.K, n, p);
                    if (kGrad) to.q[n][p] = tile(l.Q, n, p);
                }
        };
        columns(0, across[0]);
        // the right side, in the result's place: b (v - f K S), or P^T do' + r K D
        float x[8];
        bf16x8 xp[3], wp[3];
        int odd = C;
        if constexpr (kGrad) {
            f32x4 y[2];
#pragma unroll
            for (int n = 0; n < 8; ++n) y[n >> 2][n & 3] = ge[n] * ks[n >> 2][n & 3];
            bf16x8 zz[kP];
#pragma unroll
            for (int p = 0; p < kP; ++p) zz[p] = z[p];
            bf16x8 Pm[2][3];
#pragma unroll
            for (int n = 0; n < 6; ++n) Pm[n / 3][n % 3] = l.mats[6 + n][lane];
            mfma_each(Pm, zz, y);
#pragma unroll
            for (int n = 0; n < 8; ++n) x[n] = y[n >> 2][n & 3];
        } else {
#pragma unroll
            for (int n = 0; n < 8; ++n) x[n] = gb[n] * fmaf(-ge[n], ks[n >> 2][n & 3], walk::plane_sum(z, n));
            if constexpr (!BACK) odd = take_odd(x, q);
        }
        f32x4 ua[2] = {};
        if constexpr (BACK) {  // what is a position's own where beta is 0 (any number, in padding) stays with it
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                const bool alone = writes_none(gb[n]);
                ua[n >> 2][n & 3] = alone ? x[n] : 0.0f;
                x[n] = alone ? 0.0f : x[n];
            }
        }
        split3(x, xp);
        mfma_each(Tm, xp, ua);
        const float carry = __uint_as_float(same_in_lanes(__float_as_uint(l.gates.carry)));
        const bool fast = same_in_lanes(__float_as_uint(l.gates.fast)) != 0;
        if constexpr (kGrad) {  // f do' while T^T is at work
#pragma unroll
            for (int n = 0; n < 8; ++n) ge[n] = l.gates.f[8 * q + n];
#pragma unroll
            for (int n = 0; n < 8; ++n) x[n] = j.scale * ge[n] * walk::plane_sum(z, n);
            split3(x, wp);
        } else {
#pragma unroll
            for (int n = 0; n < 8; ++n) ge[n] = l.gates.r[8 * q + n];
        }
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            x[n] = ua[n >> 2][n & 3];
            if (BACK) done_rows[n] = x[n];
        }
        if constexpr (kOut) {
            split3(x, xp);
#pragma unroll
            for (int it = 0; it < 2; ++it) o[it] *= l.gates.f[16 * it + m] * j.scale;
            bf16x8 Pm[2][3];
#pragma unroll
            for (int n = 0; n < 6; ++n) Pm[n / 3][n % 3] = l.mats[6 + n][lane];
            mfma_each_right(xp, Pm, o);
        }
        // the state after the chunk: K^T (r U), or Q^T (f do') - K^T (f b dR)
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            x[n] *= kGrad ? -ge[n] * gb[n] : ge[n];
            if (BACK && writes_none(gb[n])) x[n] = 0.0f;
        }
        split3(x, xp);
        if (fast) {
            asm volatile("");  // a branch: the compiler would work out both and select
#pragma unroll
            for (int t = 0; t < NA; ++t) S[t] *= carry;
        } else {
            const f32x4 c4 = {carry, carry, carry, carry};
#pragma unroll
            for (int t = 0; t < NA; ++t) S[t] = __builtin_elementwise_fma(S[t], c4, S[t]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (t + 1 < NT) columns(t + 1, across[(t + 1) & 1]);
            f32x4 two[2] = {S[2 * t], S[2 * t + 1]};
            if constexpr (kGrad) mfma_each(across[t & 1].q, wp, two);
            mfma_each(across[t & 1].k, xp, two);
            S[2 * t] = two[0];
            S[2 * t + 1] = two[1];
            __builtin_amdgcn_sched_barrier(0);
        }
        if (!BACK && __any(odd < C)) {
            const float nan = __builtin_nanf("");
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int first = __shfl(odd, 4 * q + r);  // of column 4 q + r
#pragma unroll
                for (int it = 0; it < 2; ++it)
                    if (16 * it + m >= first) o[it][r] = nan;
            }
            if (odd < C) {
#pragma unroll
                for (int t = 0; t < NA; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) S[t][r] = nan;
            }
        }
        if constexpr (kOut) {
#pragma unroll
            for (int it = 0; it < 2; ++it)
#pragma unroll
                for (int r = 0; r < 4; ++r) done[it].v[r] = __builtin_bit_cast(Bit, (T)o[it][r]);
        }
    };
    load(0);
    if constexpr (kStages<T, D1> == 2) {
        put(0, lds[0]);
        load(1);
        lds_barrier();
        auto step = [&](int i, WalkLds<T, D1> &now, WalkLds<T, D1> &next) {
            if (i + 1 < n_chunks) put(i + 1, next);
            leave(i);
            load(i + 2);
            compute(now);
            lds_barrier();
        };
        for (int i = 0; i < n_chunks; i += 2) {
            step(i, lds[0], lds[kStages<T, D1> - 1]);
            if (i + 1 < n_chunks) step(i + 1, lds[kStages<T, D1> - 1], lds[0]);
        }
    } else {
        for (int i = 0; i < n_chunks; ++i) {
            lds_barrier();  // the last chunk's reads are done
            put(i, lds[0]);
            leave(i);
            load(i + 1);
            lds_barrier();
            compute(lds[0]);
        }
    }
    write(n_chunks - 1);
    if (j.fin.p != nullptr && col < j.fin.cols) {
#pragma unroll
        for (int t = 0; t < NA; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = state_row(t, q, r);
                if (row < j.fin.rows) j.fin.p[row * j.fin.row + col] = S[t][r];
            }
    }
}

// ---------------------------------------------------------------- segments
// Few (batch row, head) pairs leave CUs idle, so long sequences are cut into
// segments that are walked side by side.  A segment takes a state S to
// M S + N: one pass over all segments finds N (from zero) and M (the identity's
// columns, nothing written), a join goes through them in order, and the walks
// themselves start from the states it leaves.  D goes back the same way, with
// M's transpose.
struct SegArgs {
    int n;       // segments
    int chunks;  // of one
    float *S, *D, *M;  // [pairs][n][D1][wide], of M [..][wide_k]: own parts, then the states before (S) or after (D) the segment
    int wide, wide_k;
};
template <int D1>
__device__ __forceinline__ StateAt seg_at(float *p, const SegArgs &s, int bh, int seg, int wide) {
    return {p + ((int64_t)bh * s.n + seg) * D1 * wide, wide, D1, wide};
}

struct JoinArgs {
    SegArgs s;
    const float *init, *fin;  // the sequence's own S before the first and D after the last position, or null
    int dk, dv, cols;         // cols: blocks of 16 columns
};
// A workgroup joins 16 columns of one (batch row, head); wave w has 32 rows.
// The products are fp32's in three planes.  Bound by latency: one step a segment,
// 1.3 us for heads of up to 64; those above 128 do not have the registers for M (988
// bytes a lane in memory) and take some 20, 40 where S and D are joined.
template <int D1, bool GRAD>
__device__ __forceinline__ void join_columns(const JoinArgs &a, int bh, int blk, bf16x8 (&lds)[3][D1 / 32][64]) {
    constexpr int NT = D1 / 32;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, m = lane & 15, q = lane >> 4;
    const int col = blk * 16 + m;
    const float *from = GRAD ? a.fin : a.init;
    f32x4 cur[2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = state_row(2 * wave + u, q, r);
            const float s = from != nullptr && col < a.dv && row < a.dk ? from[((int64_t)bh * a.dk + row) * a.dv + col] : 0.0f;
            cur[u][r] = __builtin_canonicalizef(s);  // no signalling NaN (a launch tag) goes into the workspace
        }
    float mat[2][NT][8];
    f32x4 own[2];
    auto seg_of = [&](int i) { return GRAD ? a.s.n - 1 - i : i; };
    auto load = [&](int i) {
        const int seg = seg_of(i);
        const StateAt at = seg_at<D1>(GRAD ? a.s.D : a.s.S, a.s, bh, seg, a.s.wide), mt = seg_at<D1>(a.s.M, a.s, bh, seg, a.s.wide_k);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int r = 0; r < 4; ++r) own[u][r] = at.p[state_row(2 * wave + u, q, r) * at.row + col];
            const int row = 32 * wave + row_of(u, m);
#pragma unroll
            for (int t = 0; t < NT; ++t)
                if (GRAD) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) mat[u][t][e] = mt.p[(32 * t + 8 * q + e) * mt.row + row];
                } else {
                    *reinterpret_cast<f32x4 *>(&mat[u][t][0]) = *reinterpret_cast<const f32x4 *>(&mt.p[row * mt.row + 32 * t + 8 * q]);
                    *reinterpret_cast<f32x4 *>(&mat[u][t][4]) = *reinterpret_cast<const f32x4 *>(&mt.p[row * mt.row + 32 * t + 8 * q + 4]);
                }
        }
    };
    if (a.s.n > 1) load(0);
    for (int i = 0; i < a.s.n; ++i) {
        const StateAt at = seg_at<D1>(GRAD ? a.s.D : a.s.S, a.s, bh, seg_of(i), a.s.wide);
        // (this segment's own part has been read)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) at.p[state_row(2 * wave + u, q, r) * at.row + col] = cur[u][r];
        if (i + 1 == a.s.n) return;
        const float v[8] = {cur[0][0], cur[0][1], cur[0][2], cur[0][3], cur[1][0], cur[1][1], cur[1][2], cur[1][3]};
        bf16x8 p[3];
        split3(v, p);
        lds_barrier();  // the last step's reads are done
#pragma unroll
        for (int k = 0; k < 3; ++k) lds[k][wave][lane] = p[k];
        lds_barrier();
        f32x4 sum[2] = {own[0], own[1]};
        bf16x8 mp[NT][2][3];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int u = 0; u < 2; ++u) split3(mat[u][t], mp[t][u]);
        if (i + 2 < a.s.n) load(i + 1);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            bf16x8 s[3];
#pragma unroll
            for (int k = 0; k < 3; ++k) s[k] = lds[k][t][lane];
            mfma_each(mp[t], s, sum);
        }
        cur[0] = sum[0];
        cur[1] = sum[1];
    }
}

template <int D1>
__global__ __launch_bounds__(D1 * 2) void join_kernel(JoinArgs a) {
    __shared__ bf16x8 lds[3][D1 / 32][64];
    const uint32_t blk = blockIdx.x % (uint32_t)a.cols, bh = blockIdx.x / (uint32_t)a.cols;
    if (blockIdx.y == 0) join_columns<D1, false>(a, (int)bh, (int)blk, lds);
    else join_columns<D1, true>(a, (int)bh, (int)blk, lds);
}

}  // namespace delta
}  // namespace prn
