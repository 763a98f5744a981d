// delta.hpp -- the gated delta rule in chunks of 32 positions: what the chunks'
// own products are (prep_kernel) and where they are kept.
//
//   S_t = e^(g_t) (I - b_t k_t^T k_t) S_{t-1} + b_t k_t^T v_t,  o_t = scale q_t S_t.
// With u_t = b_t (v_t - e^(g_t) k_t S_{t-1}) this is S_t = e^(g_t) S_{t-1} + k_t^T u_t.
// In a chunk that starts from S, with G_i the sum of its g up to position i,
// f_i = e^(G_i), r_i = e^(G_last - G_i) and E_ij = e^(G_i - G_j):
//   A_ij = b_i E_ij k_i.k_j (j < i),  T = (I + A)^-1,  P_ij = scale E_ij q_i.k_j (j <= i),
//   U = T (b (V - f (K S))),  o = scale f (Q S) + P U,  S <- f_last S + (r K)^T U.
// T and P need no state: one wave a chunk finds them, all chunks side by side
// (prep_kernel), and the walk over the chunks multiplies with them.
//
// G is summed in double: its differences stay exact where a strong decay
// stands before slow ones.  T comes from forward substitution in the 16x16
// blocks on the diagonal, which is stable where keys repeat (the powers of A
// that a product form of the inverse takes grow like binomials there).
#pragma once

#include "mixer.hpp"
#include "walk.hpp"

namespace prn {
namespace delta {

using walk::bf16x8;
using walk::kPlanes;

constexpr int C = 32;  // positions a chunk
// Backward pass: what stands in a beta's place that is no larger, as the gradient
// of beta divides u by it.  Such a position reaches no other one (writes_none).
constexpr float kTinyBeta = 1e-20f;
__device__ __forceinline__ bool writes_none(float beta) { return fabsf(beta) <= kTinyBeta; }

// What is kept of a chunk: gates, then matrices as operands of the 32-wide
// matrix instructions, plane by plane, 16 bytes a lane.  T (and in the backward
// pass its transpose and that of P) have their rows in the order in which a
// result's registers are the next operand (see row_of); P has them as they come.
struct Gates {
    float b[C], f[C], r[C];
    float carry, fast;  // walk.hpp's Carry of the whole chunk
    float pad[30];
};
constexpr int kTile = 1024;  // bytes of one plane of 16 rows
// T and P, or T, its transpose and that of P, of three planes of two tiles each
template <bool BACK> constexpr int64_t kRecord = sizeof(Gates) + (BACK ? 18 : 12) * kTile;
constexpr int kAtT = sizeof(Gates), kAtP = kAtT + 6 * kTile;       // forward
constexpr int kAtTt = kAtT + 6 * kTile, kAtPt = kAtTt + 6 * kTile;  // backward

// Position that lane m of operand tile u stands for: the registers of the
// result, tile by tile, are then eight consecutive positions of one lane.
__device__ __forceinline__ int row_of(int u, int m) { return 8 * (m >> 2) + 4 * u + (m & 3); }

// (batch row, head) pairs in groups of 8, then the `per` workgroups that read the
// same rows: consecutive workgroups go to the 8 XCDs in turn, so all workgroups
// of one pair meet in one L2.
struct Where {
    int bh, b, h, sub;
    bool any;
};
__device__ __forceinline__ Where where(int per_, int pairs, int heads) {
    auto scalar = [](uint32_t x) { return (int)__builtin_amdgcn_readfirstlane(x); };
    const uint32_t per = (uint32_t)per_;
    const uint32_t grp = blockIdx.x / (8 * per), rest = blockIdx.x - grp * 8 * per;
    const uint32_t bh = grp * 8 + (rest & 7);
    Where w;
    w.bh = scalar(bh);
    w.b = scalar(bh / (uint32_t)heads);
    w.h = w.bh - w.b * heads;
    w.sub = scalar(rest >> 3);
    w.any = w.bh < pairs;
    return w;
}

__host__ __device__ __forceinline__ WalkView view_of(const HeadView &v) { return {v.p, v.st[0], v.st[1], v.st[2]}; }

// Whether rows move as 16-byte vectors.  Rows that overlap are left to the
// loads of any alignment, whose rows past the last position are cleared.  Where
// all positions have one row, the rows past the last one are that row again: T,
// P, b and f are zero there.
inline bool view_vec(const HeadView &v, int d, int es) {
    const int64_t n = 16 / es;
    return d % n == 0 && aligned16(v.p) && v.st[0] % n == 0 && v.st[1] % n == 0 && v.st[2] % n == 0 && (v.st[1] >= d || v.st[1] == 0);
}

// Width of the state's rows that a walk is built for.
inline int walk_width(int dk) { return dk <= 32 ? 32 : dk <= 64 ? 64 : dk <= 128 ? 128 : 256; }
// Workgroups a CU that a walk's registers are shared out for.
constexpr int walk_wgs(bool bf16, int width) { return width > 128 || (!bf16 && width > 64) ? 1 : 2; }
inline int64_t chunks_of(int64_t L) { return (L + C - 1) / C; }
// delta.hip
int segments(int64_t pairs, int walks, int blocks, int64_t chunks, bool bf16, int width);
// delta_back.hip
size_t back_ws(const DeltaArgs &p);
hipError_t backward(const DeltaArgs &p, char *scratch, hipStream_t s);

// Sums of products of planes, smallest first, of N results side by side: each
// matrix instruction waits for the one before it on its result.
template <int N, int NA, int NB>
__device__ __forceinline__ void mfma_each(const bf16x8 (&a)[N][NA], const bf16x8 (&b)[NB], f32x4 (&c)[N]) {
#pragma unroll
    for (int s = 2; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB)
#pragma unroll
                for (int n = 0; n < N; ++n) c[n] = walk::mfma(a[n][i], b[s - i], c[n]);
}
template <int N, int NA, int NB>
__device__ __forceinline__ void mfma_each_right(const bf16x8 (&a)[NA], const bf16x8 (&b)[N][NB], f32x4 (&c)[N]) {
#pragma unroll
    for (int s = 2; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB)
#pragma unroll
                for (int n = 0; n < N; ++n) c[n] = walk::mfma(a[i], b[n][s - i], c[n]);
}

struct PrepArgs {
    HeadView q, k, log_decay, beta;
    int64_t L, items;  // items: chunks of all (batch row, head) pairs
    int H, group, dk, chunks;
    float scale;
    char *rec;
};

// Eight elements of a row from column c on, zeros past its end, as planes.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T *row, int c, int d, bool in, bf16x8 (&p)[kPlanes<T>]) {
    struct alignas(16) {
        T v[8];
    } x;
    if constexpr (VEC) {
        constexpr int kV = kVec<T>;
#pragma unroll
        for (int h = 0; h < 8 / kV; ++h) {
            const u32x4 z = {0u, 0u, 0u, 0u};
            u32x4 w = z;
            if (in && c + h * kV < d) w = *reinterpret_cast<const u32x4 *>(row + c + h * kV);
            *reinterpret_cast<u32x4 *>(&x.v[h * kV]) = w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x.v[i] = in && c + i < d ? row[c + i] : (T)0.0f;
    }
    walk::planes_of(x.v, p);
}

// Eight numbers as planes without an infinity in them (one would look like a launch tag in the workspace).
__device__ __forceinline__ void store_planes(char *at, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (abs_bits(v[i]) >= kInfBits) v[i] = __builtin_nanf("");
    bf16x8 p[3];
    walk::split3(v, p);
#pragma unroll
    for (int n = 0; n < 3; ++n) *reinterpret_cast<bf16x8 *>(at + n * kTile) = p[n];
}

__device__ __forceinline__ f32x4 mfma32(float a, float b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

// A wave a chunk.  Bound by memory where there are many: rows of q and k are read
// once, records written once.  B=8, L=2048, H=16, 128x128, bf16: 59 us for 134 MB
// read and 104 written, in the backward pass 66 for 134 and 154.
template <typename T, int D1, bool VEC, bool BACK>
__global__ __launch_bounds__(256) void prep_kernel(PrepArgs a) {
    constexpr int kP = kPlanes<T>, NT = D1 / 32, W = 36;
    __shared__ __align__(16) float Am[4][C * W], Tm[4][C * W];
    __shared__ double Gs[4][C];
    __shared__ float bs[4][C];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, m = lane & 15, q = lane >> 4;
    const int64_t want = (int64_t)blockIdx.x * 4 + wave, item = min(want, a.items - 1);
    const int bh = (int)((uint32_t)item / (uint32_t)a.chunks), chunk = (int)((uint32_t)item - (uint32_t)bh * (uint32_t)a.chunks);
    const int b = (int)((uint32_t)bh / (uint32_t)a.H), h = bh - b * a.H, hk = h / a.group;
    const int64_t begin = (int64_t)chunk * C;
    const int cnt = (int)min((int64_t)C, a.L - begin);
    float *A = Am[wave], *Tw = Tm[wave];
    double *G = Gs[wave];

    // gates: G in units of log 2, so that an exponential is one instruction
    const int p = lane & 31;
    const bool in = p < cnt;
    auto gate = [&](const HeadView &v) { return static_cast<const float *>(v.p)[b * v.st[0] + (begin + p) * v.st[1] + h * v.st[2]]; };
    float g = in ? gate(a.log_decay) : 0.0f;
    float beta = in ? gate(a.beta) : 0.0f;
    if (BACK && writes_none(beta)) beta = kTinyBeta;
    if (g < -1e5f) g = -1e5f;  // e^g is 0 from -104 on
    const bool bad_gate = abs_bits(g) >= kInfBits || abs_bits(beta) >= kInfBits;
    double sum = bad_gate ? 0.0 : (double)g * 1.4426950408889634;
#pragma unroll
    for (int d = 1; d < C; d *= 2) {
        const double up = __shfl_up(sum, d, C);
        if (p >= d) sum += up;
    }
    if (lane < C) {
        G[p] = sum;
        bs[wave][p] = beta;
    }
    __syncthreads();

    // k.k and q.k: tiles (0, 0), (1, 0), (1, 1)
    f32x4 kk[3] = {}, qk[3] = {};
    {
        const T *kp = static_cast<const T *>(a.k.p) + b * a.k.st[0] + begin * a.k.st[1] + hk * a.k.st[2];
        const T *qp = static_cast<const T *>(a.q.p) + b * a.q.st[0] + begin * a.q.st[1] + hk * a.q.st[2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            bf16x8 kf[2][kP], qf[2][kP];
#pragma unroll
            for (int it = 0; it < 2; ++it) {
                const int row = 16 * it + m;
                load8<T, VEC>(kp + row * a.k.st[1], 32 * t + 8 * q, a.dk, row < cnt, kf[it]);
                load8<T, VEC>(qp + row * a.q.st[1], 32 * t + 8 * q, a.dk, row < cnt, qf[it]);
            }
            kk[0] = walk::mfma_planes(kf[0], kf[0], kk[0]);
            kk[1] = walk::mfma_planes(kf[1], kf[0], kk[1]);
            kk[2] = walk::mfma_planes(kf[1], kf[1], kk[2]);
            qk[0] = walk::mfma_planes(qf[0], kf[0], qk[0]);
            qk[1] = walk::mfma_planes(qf[1], kf[0], qk[1]);
            qk[2] = walk::mfma_planes(qf[1], kf[1], qk[2]);
        }
    }

    // The first position whose key or gate is not finite: T is found as if the chunk ended before it.
    // (lane 16 q + m holds the diagonal's element m where m / 4 is q, so a mask's first bit is its first position)
    auto odd = [&](const f32x4 &t) { return __ballot(m >> 2 == q && abs_bits(t[m & 3]) >= kInfBits); };
    const uint64_t odd_gate = __ballot(bad_gate) & 0xffffffffu, odd0 = odd(kk[0]), odd1 = odd(kk[2]);
    int bad = C;
    if (odd_gate) bad = (int)__builtin_ctzll(odd_gate);
    if (odd1) bad = min(bad, 16 + ((int)__builtin_ctzll(odd1) & 15));
    if (odd0) bad = min(bad, (int)__builtin_ctzll(odd0) & 15);

    auto weight = [&](int i, int j) { return fast_exp2((float)(G[i] - G[j])); };
    float e[3][4];
#pragma unroll
    for (int n = 0; n < 3; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = (n > 0 ? 16 : 0) + 4 * q + r, j = (n > 1 ? 16 : 0) + m;
            e[n][r] = j <= i ? weight(i, j) : 0.0f;
            A[i * W + j] = j < i && i < bad ? bs[wave][i] * e[n][r] * kk[n][r] : 0.0f;
        }
    __syncthreads();

    // T's blocks on the diagonal, a lane a column
    {
        const int blk = (lane >> 4) & 1;
        float t[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const f32x4 *row = reinterpret_cast<const f32x4 *>(&A[(16 * blk + i) * W + 16 * blk]);
            float s = i == m ? 1.0f : 0.0f;
#pragma unroll
            for (int l4 = 0; l4 < (i + 3) / 4; ++l4) {
                const f32x4 x = row[l4];
#pragma unroll
                for (int l = 0; l < 4; ++l)
                    if (4 * l4 + l < i) s = fmaf(-x[l], t[4 * l4 + l], s);
            }
            t[i] = s;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (lane < 32) Tw[(16 * blk + i) * W + 16 * blk + m] = t[i];
            else if (lane < 48) Tw[i * W + 16 + m] = 0.0f;
        }
    }
    __syncthreads();
    // the block below: -T22 (A21 T11)
    f32x4 x = {};
#pragma unroll
    for (int s = 0; s < 4; ++s) x = mfma32(A[(16 + m) * W + 4 * s + q], Tw[(4 * s + q) * W + m], x);
#pragma unroll
    for (int r = 0; r < 4; ++r) A[(4 * q + r) * W + 16 + m] = x[r];
    __syncthreads();
    f32x4 y = {};
#pragma unroll
    for (int s = 0; s < 4; ++s) y = mfma32(Tw[(16 + m) * W + 16 + 4 * s + q], A[(4 * s + q) * W + 16 + m], y);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r) Tw[(16 + 4 * q + r) * W + m] = -y[r];
    // P, over A
#pragma unroll
    for (int n = 0; n < 3; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = (n > 0 ? 16 : 0) + 4 * q + r, j = (n > 1 ? 16 : 0) + m;
            A[i * W + j] = j <= i ? a.scale * e[n][r] * qk[n][r] : 0.0f;
            if (n == 0) A[i * W + 16 + m] = 0.0f;
        }
    __syncthreads();

    if (want >= a.items) return;
    char *rec = a.rec + item * kRecord<BACK>;
    if (lane < C) {
        Gates *to = reinterpret_cast<Gates *>(rec);
        to->b[p] = p < bad ? beta : __builtin_nanf("");  // tells the walk
        to->f[p] = in ? fast_exp2((float)sum) : 0.0f;
        to->r[p] = fast_exp2((float)(G[C - 1] - sum));
        if (p == C - 1) {
            const float whole = fast_exp2((float)sum), rest = expm1f((float)(sum * 0.6931471805599453));
            const bool fast = rest < -0.5f;
            to->carry = fast ? whole : rest;
            to->fast = fast ? 1.0f : 0.0f;
        }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int row = row_of(u, m);
        float v[8];
        auto across = [&](const float *src, int i) {
            *reinterpret_cast<f32x4 *>(&v[0]) = *reinterpret_cast<const f32x4 *>(&src[i * W + 8 * q]);
            *reinterpret_cast<f32x4 *>(&v[4]) = *reinterpret_cast<const f32x4 *>(&src[i * W + 8 * q + 4]);
        };
        auto down = [&](const float *src, int j) {
#pragma unroll
            for (int n = 0; n < 8; ++n) v[n] = src[(8 * q + n) * W + j];
        };
        across(Tw, row);
        store_planes(rec + kAtT + u * 3 * kTile + lane * 16, v);
        if constexpr (!BACK) {
            across(A, 16 * u + m);
            store_planes(rec + kAtP + u * 3 * kTile + lane * 16, v);
        } else {
            down(Tw, row);
            store_planes(rec + kAtTt + u * 3 * kTile + lane * 16, v);
            down(A, row);
            store_planes(rec + kAtPt + u * 3 * kTile + lane * 16, v);
        }
    }
}

}  // namespace delta
}  // namespace prn
