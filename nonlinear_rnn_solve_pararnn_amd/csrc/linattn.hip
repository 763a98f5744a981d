// linattn.hip -- linear attention with a decay per head: the walk over whole
// sequences on fp32 matrix instructions, and the single-token step.
#include "linattn.hpp"

namespace prn {

namespace {

constexpr int kThreads = 256;
constexpr int kC = 32;   // positions a chunk
constexpr int kNB = 64;  // columns of Z a workgroup: 16 a wave

__device__ __forceinline__ f32x4 mfma4(float a, float b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// Rows [p0, p0 + kC) of one operand (columns [c0, c0 + W)) into shared
// memory, zeros past the sequence's end and past column d.
template <typename T, int W>
__device__ __forceinline__ void stage(float *lds, int stride, const WalkView &v, int64_t base, int64_t L, int rev,
                                      int64_t p0, int c0, int d, bool vec) {
    const T *src = static_cast<const T *>(v.p) + base;
    if (vec) {
        constexpr int V = kVec<T>;
        for (int i = threadIdx.x; i < kC * (W / V); i += kThreads) {
            const int r = i / (W / V), c = (i - r * (W / V)) * V;
            const int64_t p = p0 + r;
            float f[V];
#pragma unroll
            for (int k = 0; k < V; ++k) f[k] = 0.0f;
            if (p < L && c0 + c < d) load_vec<T, V>(src + (rev ? L - 1 - p : p) * v.st + c0 + c, f);
#pragma unroll
            for (int k = 0; k < V; ++k) lds[r * stride + c + k] = f[k];
        }
    } else {
        for (int i = threadIdx.x; i < kC * W; i += kThreads) {
            const int r = i / W, c = i - r * W;
            const int64_t p = p0 + r;
            lds[r * stride + c] = p < L && c0 + c < d ? (float)src[(rev ? L - 1 - p : p) * v.st + c0 + c] : 0.0f;
        }
    }
}

// One workgroup walks the sequence of one (batch row, head) for 64 columns
// of Z, 16 a wave.  A wave keeps its [D1, 16] columns of T in accumulator
// registers for the whole walk; their layout (row 4 (lane / 16) + r of each
// 16-row tile, column lane % 16) is also that of a B operand whose k index
// runs over the same rows, so T is multiplied without leaving the registers.
template <typename T, int D1>
__global__ __launch_bounds__(kThreads) void walk_kernel(WalkArgs a) {
    constexpr int SX = D1 + 4, SZ = kNB + 4, SP = kC + 4, NA = D1 / 16;
    __shared__ float X[kC * SX], Y[kC * SX], Z[kC * SZ], P[kC * SP];
    __shared__ int odd_z;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, m = lane & 15, q = lane >> 4;
    // (batch row, head) pairs in groups of 8, the column blocks and walks of
    // a group in turn: all that read the same rows run on the same XCD
    const int64_t per = (int64_t)a.walks * a.nblk;
    const int64_t grp = (int64_t)blockIdx.x / (8 * per), rest = (int64_t)blockIdx.x - grp * 8 * per;
    const int64_t bh = grp * 8 + (rest & 7);
    const int sub = (int)(rest >> 3);
    if (bh >= a.B * a.H) return;
    const Walk &w = a.w[sub / a.nblk];
    const int c0 = (sub % a.nblk) * kNB;
    if (c0 >= w.d2) return;
    const int64_t b = bh / a.H, h = bh - b * a.H;
    const float g = walk_gate(a.log_decay, h), g2 = g * kLog2e;
    const int col = c0 + wave * 16 + m;
    const bool in = col < w.d2;

    f32x4 S[NA];
#pragma unroll
    for (int t = 0; t < NA; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 16 * t + 4 * q + r;
            S[t][r] = w.init != nullptr && in && row < w.d1
                          ? w.init[bh * w.d1 * w.d2 + (int64_t)row * w.im + (int64_t)col * w.in] : 0.0f;
        }

    const int64_t bx = b * w.X.sb + h * w.X.sh, by = b * w.Y.sb + h * w.Y.sh, bz = b * w.Z.sb + h * w.Z.sh;
    const float em1_full = walk_em1(g, kC);
    for (int64_t p0 = 0; p0 < a.L; p0 += kC) {
        const int cnt = (int)min((int64_t)kC, a.L - p0);
        __syncthreads();
        if (threadIdx.x == 0) odd_z = 0;
        stage<T, D1>(X, SX, w.X, bx, a.L, w.rev, p0, 0, w.d1, a.vec);
        stage<T, D1>(Y, SX, w.Y, by, a.L, w.rev, p0, 0, w.d1, a.vec);
        stage<T, kNB>(Z, SZ, w.Z, bz, a.L, w.rev, p0, c0, w.d2, a.vec);
        __syncthreads();
        // P = wi e^(g(i-j)) (X Y^T) below and on the diagonal, as its
        // transpose, so that a lane's four results are consecutive j
        if (wave < 3) {
            const int it = wave == 0 ? 0 : 1, jt = wave == 2 ? 1 : 0;
            f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int t = 0; t < NA; ++t) {
                const f32x4 y = *reinterpret_cast<const f32x4 *>(&Y[(jt * 16 + m) * SX + 16 * t + 4 * q]);
                const f32x4 x = *reinterpret_cast<const f32x4 *>(&X[(it * 16 + m) * SX + 16 * t + 4 * q]);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc = mfma4(y[r], x[r], acc);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int n = (it - jt) * 16 + m - (4 * q + r);
                acc[r] = n >= 0 ? acc[r] * (w.wi * fast_exp2(g2 * (float)n)) : 0.0f;
            }
            *reinterpret_cast<f32x4 *>(&P[(it * 16 + m) * SP + jt * 16 + 4 * q]) = acc;
        } else {
            // a value of Z that is not finite must not reach the positions
            // before it through a zero of P: it is left out of the product
            // and added to the positions from its own on
            bool bad = false;
            for (int i = lane; i < kC * kNB; i += 64) bad = bad || abs_bits(Z[(i / kNB) * SZ + i % kNB]) >= kInfBits;
            if (bad) odd_z = 1;
        }
        // the part of the state before the chunk
        f32x4 o[2];
#pragma unroll
        for (int it = 0; it < 2; ++it) {
            f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int t = 0; t < NA; ++t) {
                const f32x4 x = *reinterpret_cast<const f32x4 *>(&X[(it * 16 + m) * SX + 16 * t + 4 * q]);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc = mfma4(x[r], S[t][r], acc);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[r] *= w.wo * fast_exp2(g2 * (float)(it * 16 + 4 * q + r + 1 - w.e));
            o[it] = acc;
        }
        __syncthreads();
        const bool odd = odd_z != 0;
#pragma unroll
        for (int it = 0; it < 2; ++it)
#pragma unroll
            for (int jt = 0; jt <= it; ++jt) {
                const f32x4 p = *reinterpret_cast<const f32x4 *>(&P[(it * 16 + m) * SP + jt * 16 + 4 * q]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float z = Z[(jt * 16 + 4 * q + r) * SZ + wave * 16 + m];
                    if (odd && abs_bits(z) >= kInfBits) z = 0.0f;
                    o[it] = mfma4(p[r], z, o[it]);
                }
            }
        if (odd) {
            for (int j = 0; j < cnt; ++j) {
                const float z = Z[j * SZ + wave * 16 + m];
                if (abs_bits(z) < kInfBits) continue;
#pragma unroll
                for (int it = 0; it < 2; ++it)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int i = it * 16 + 4 * q + r;
                        if (j <= i) o[it][r] = fmaf(P[i * SP + j], z, o[it][r]);
                    }
            }
        }
#pragma unroll
        for (int it = 0; it < 2; ++it)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t p = p0 + it * 16 + 4 * q + r;
                if (p < a.L && in) {
                    const int64_t t = w.rev ? a.L - 1 - p : p;
                    static_cast<T *>(w.out)[((b * a.L + t) * a.H + h) * w.d2 + col] = (T)o[it][r];
                }
            }
        // T over the chunk
        const float em1 = cnt == kC ? em1_full : walk_em1(g, cnt);
#pragma unroll
        for (int t = 0; t < NA; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[t][r] = fmaf(S[t][r], em1, S[t][r]);
#pragma unroll
        for (int jt = 0; jt < 2; ++jt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int j = jt * 16 + 4 * q + r, n = cnt - 1 - j;
                const float wz = n >= 0 ? w.wt * fast_exp2(g2 * (float)(n + w.e)) : 0.0f;
                const float z = Z[j * SZ + wave * 16 + m] * wz;
#pragma unroll
                for (int t = 0; t < NA; ++t) S[t] = mfma4(Y[j * SX + 16 * t + m], z, S[t]);
            }
    }
    if (w.fin != nullptr && in) {
#pragma unroll
        for (int t = 0; t < NA; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * t + 4 * q + r;
                if (row < w.d1) w.fin[bh * w.d1 * w.d2 + (int64_t)row * w.im + (int64_t)col * w.in] = S[t][r];
            }
    }
}

template <typename T>
hipError_t run_walks(const WalkArgs &a, hipStream_t s) {
    int d1 = 0;
    for (int i = 0; i < a.walks; ++i) d1 = std::max(d1, a.w[i].d1);
    const int64_t bh = a.B * a.H;
    const unsigned grid = (unsigned)((bh + 7) / 8 * 8 * a.walks * a.nblk);
    if (d1 <= 64) walk_kernel<T, 64><<<grid, kThreads, 0, s>>>(a);
    else if (d1 <= 128) walk_kernel<T, 128><<<grid, kThreads, 0, s>>>(a);
    else walk_kernel<T, 256><<<grid, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

bool view_vec(const WalkView &v, int d, int es) {
    const int64_t n = 16 / es;
    return d % n == 0 && aligned16(v.p) && v.sb % n == 0 && v.st % n == 0 && v.sh % n == 0;
}

// Whether every operand of every walk moves as 16-byte vectors.
bool walks_vec(const WalkArgs &a, int es) {
    for (int i = 0; i < a.walks; ++i)
        if (!view_vec(a.w[i].X, a.w[i].d1, es) || !view_vec(a.w[i].Y, a.w[i].d1, es) || !view_vec(a.w[i].Z, a.w[i].d2, es))
            return false;
    return true;
}

// ---------------------------------------------------------------- single token
//   S' = e^g S + k^T v,  o = scale q S'
// Reads and writes the state once and is bound by that.  One workgroup a
// (batch row, head): threads are columns (V of them each) by rows, the rows'
// partial products with q meet in shared memory.
struct StepArgs {
    int64_t BH, H;
    int dk, dv, cols, lanes;  // lanes (a power of two) threads over the columns
    const void *q, *k, *v;
    int64_t qb, qh, kb, kh, vb, vh;
    const float *log_decay, *state;
    float scale;
    void *o;
    float *out_state;
};

constexpr int kMaxHead = 256;

template <typename T, int V>
__global__ __launch_bounds__(kThreads) void step_kernel(StepArgs a) {
    __shared__ float qk[2][kMaxHead];
    __shared__ float part[kThreads * V];
    const int64_t bh = blockIdx.x, b = bh / a.H, h = bh - b * a.H;
    for (int i = threadIdx.x; i < a.dk; i += kThreads) {
        qk[0][i] = (float)static_cast<const T *>(a.q)[b * a.qb + h * a.qh + i] * a.scale;
        qk[1][i] = (float)static_cast<const T *>(a.k)[b * a.kb + h * a.kh + i];
    }
    __syncthreads();
    const float lam = expf(a.log_decay[h]);
    const int tx = threadIdx.x & (a.lanes - 1), ty = threadIdx.x / a.lanes, rows = kThreads / a.lanes;
    const int c = tx * V;
    const bool in = c < a.dv;
    float v[V], acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        v[i] = in ? (float)static_cast<const T *>(a.v)[b * a.vb + h * a.vh + c + i] : 0.0f;
        acc[i] = 0.0f;
    }
    const float *src = a.state + bh * a.dk * a.dv + c;
    float *dst = a.out_state + bh * a.dk * a.dv + c;
    if (in) {
        constexpr int U = 8;  // rows in flight a thread
        for (int r0 = ty; r0 < a.dk; r0 += rows * U) {
            float s[U][V];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = r0 + u * rows;
                if (r < a.dk) load_vec<float, V>(src + (int64_t)r * a.dv, s[u]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = r0 + u * rows;
                if (r < a.dk) {
                    const float qr = qk[0][r], kr = qk[1][r];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        s[u][i] = fmaf(kr, v[i], lam * s[u][i]);
                        acc[i] = fmaf(qr, s[u][i], acc[i]);
                    }
                    store_vec<float, V>(dst + (int64_t)r * a.dv, s[u]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) part[(ty * a.lanes + tx) * V + i] = acc[i];
    __syncthreads();
    for (int n = threadIdx.x; n < a.dv; n += kThreads) {
        float sum = 0.0f;
        for (int y = 0; y < rows; ++y) sum += part[y * a.lanes * V + n];
        static_cast<T *>(a.o)[bh * a.dv + n] = (T)sum;
    }
}

}  // namespace

size_t linattn_ws(const LinattnArgs &, bool) { return kScratchOffset; }

hipError_t linattn_forward(const LinattnArgs &p, const Ws &, hipStream_t s) {
    WalkArgs a{};
    a.walks = 1;
    a.B = p.B;
    a.L = p.L;
    a.H = p.H;
    a.log_decay = p.log_decay;
    const WalkView q{p.q, p.st[0][0], p.st[0][1], p.st[0][2]}, k{p.k, p.st[1][0], p.st[1][1], p.st[1][2]},
        v{p.v, p.st[2][0], p.st[2][1], p.st[2][2]};
    a.w[0] = {q, k, v, p.o, p.state, p.out_state, p.dv, 1, p.dk, p.dv, 0, 0, p.scale, p.scale, 1.0f};
    a.nblk = (p.dv + kNB - 1) / kNB;
    a.vec = walks_vec(a, p.bf16 ? 2 : 4);
    return p.bf16 ? run_walks<bf16>(a, s) : run_walks<float>(a, s);
}

hipError_t linattn_backward(const LinattnArgs &p, const Ws &, hipStream_t s) {
    WalkArgs a{};
    a.walks = 3;
    a.B = p.B;
    a.L = p.L;
    a.H = p.H;
    a.log_decay = p.log_decay;
    const WalkView q{p.q, p.st[0][0], p.st[0][1], p.st[0][2]}, k{p.k, p.st[1][0], p.st[1][1], p.st[1][2]},
        v{p.v, p.st[2][0], p.st[2][1], p.st[2][2]}, g{p.grad_o, p.st[3][0], p.st[3][1], p.st[3][2]};
    a.w[0] = {g, v, k, p.grad_q, p.state, nullptr, 1, p.dv, p.dv, p.dk, 0, 0, p.scale, p.scale, 1.0f};
    a.w[1] = {v, g, q, p.grad_k, p.grad_out_state, nullptr, 1, p.dv, p.dv, p.dk, 1, 1, p.scale, 1.0f, p.scale};
    a.w[2] = {k, q, g, p.grad_v, p.grad_out_state, p.grad_state, p.dv, 1, p.dk, p.dv, 1, 1, p.scale, 1.0f, p.scale};
    a.nblk = (std::max(p.dk, p.dv) + kNB - 1) / kNB;
    a.vec = walks_vec(a, p.bf16 ? 2 : 4);
    return p.bf16 ? run_walks<bf16>(a, s) : run_walks<float>(a, s);
}

hipError_t linattn_step(const LinattnArgs &p, hipStream_t s) {
    const bool al = p.dv % 4 == 0 && aligned16(p.state) && aligned16(p.out_state);
    const int cols = al ? p.dv / 4 : p.dv;
    int lanes = 1;
    while (lanes < cols) lanes *= 2;
    const StepArgs a{p.B * p.H, p.H, p.dk, p.dv, cols, lanes, p.q, p.k, p.v,
                     p.st[0][0], p.st[0][2], p.st[1][0], p.st[1][2], p.st[2][0], p.st[2][2],
                     p.log_decay, p.state, p.scale, p.o, p.out_state};
    const unsigned grid = (unsigned)a.BH;
    if (p.bf16) {
        if (al) step_kernel<bf16, 4><<<grid, kThreads, 0, s>>>(a);
        else step_kernel<bf16, 1><<<grid, kThreads, 0, s>>>(a);
    } else {
        if (al) step_kernel<float, 4><<<grid, kThreads, 0, s>>>(a);
        else step_kernel<float, 1><<<grid, kThreads, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace prn
