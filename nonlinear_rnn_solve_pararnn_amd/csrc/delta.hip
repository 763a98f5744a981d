// delta.hip -- the gated delta rule: walks over whole sequences and the
// single-token step (formulas and chunks: delta.hpp).
#include "delta.hpp"

namespace prn {

namespace delta {

using walk::Ahead;
using walk::kNB;
using walk::kNowhere;
using walk::kThreads;
using walk::kTileRow;
using walk::read_row;
using walk::read_tr;
using walk::Rows;
using walk::s16x4;
using walk::split3;
using walk::state_row;
using walk::tile_at;
using walk::u32x2;

struct WalkArgs {
    WalkView q, k, v;
    void *out;          // dense [B, L, H, dv]
    const float *init;  // states before the first position or null for zeros
    float *fin;         // after the last one, or null
    int64_t B, L, H;
    int group, dk, dv, chunks, nblk;
    int out4;           // rows of out may be stored four elements at a time
    float scale;
    const char *rec;
};

// Part of the work of a chunk that every walk shares: eight numbers of a lane
// (a column of its wave's, positions 8 q ..) with the first ones that are not
// finite, and all after them, taken out.  Returns the first such position of
// the lane's column, C for none.
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

template <typename T, int D1>
constexpr int kWgs = D1 > 128 ? 1 : 2;

// One workgroup walks one (batch row, head) for 64 columns of V; wave w owns
// columns 16 w .. 16 w + 15 and keeps its [D1, 16] columns of S in fp32
// registers, in the layout of walk.hpp, where they are a matrix operand as they
// stand.  The rows of K and of T are read in the order of row_of, so that K S,
// the right side and U come out as the operands of the next product as well:
// between the chunk's operands in LDS and its outputs nothing crosses the
// waves, and a chunk has two barriers.
template <typename T, int D1, bool VEC>
__global__ __launch_bounds__(kThreads, (kWgs<T, D1>)) void walk_kernel(WalkArgs a) {
    constexpr int kP = kPlanes<T>, kO = kP == 3 ? 3 : 2;  // planes of operands; of S and U where an output is formed
    constexpr int NA = D1 / 16, NT = D1 / 32;
    constexpr int kPX = C * kTileRow<D1>, kPZ = C * kTileRow<kNB>;
    __shared__ __align__(16) bf16 K[kP * kPX], Q[kP * kPX], V[kP * kPZ];
    __shared__ __align__(16) Gates gates;
    const Where wh = where(a.nblk, (int)(a.B * a.H), (int)a.H);
    if (!wh.any) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, m = lane & 15, q = lane >> 4;
    const int tr_i = m >> 2, tr_c = m & 3;  // this lane's row and column group in a transposing read
    const int c0 = wh.sub * kNB, col = c0 + wave * 16 + m;
    const int last = (int)(a.L - (int64_t)(a.chunks - 1) * C);

    f32x4 S[NA];
#pragma unroll
    for (int t = 0; t < NA; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = state_row(t, q, r);
            S[t][r] = a.init != nullptr && col < a.dv && row < a.dk ? a.init[((int64_t)wh.bh * a.dk + row) * a.dv + col] : 0.0f;
        }

    const int hk = wh.h / a.group;
    const Rows rq = walk::rows_of<T>(a.q, wh.b, hk, a.L, 0, C, 0, 0, a.dk), rk = walk::rows_of<T>(a.k, wh.b, hk, a.L, 0, C, 0, 0, a.dk),
               rv = walk::rows_of<T>(a.v, wh.b, wh.h, a.L, 0, C, 0, c0, a.dv),
               ro = walk::rows_of<T>({a.out, a.L * a.H * a.dv, a.H * a.dv, a.dv}, wh.b, wh.h, a.L, 0, C, 0, c0, a.dv);
    const char *rec = a.rec + (int64_t)wh.bh * a.chunks * kRecord<T, false>;
    const int oc = wave * 16 + 4 * q;
    const uint32_t out_at = c0 + oc < a.dv ? ro.row_at(m, C) + oc * (uint32_t)sizeof(T) : kNowhere;
    const uint32_t out_step = 16 * ro.row_bytes;

    Ahead<T, D1, C, VEC> aq, ak;
    Ahead<T, kNB, C, VEC> av;
    aq.init(rq);
    ak.init(rk);
    av.init(rv);
    float gate_ahead = 0.0f;
    bf16x8 Ta[2][3], Pa[2][kPP<T>];
    auto positions = [&](int i) { return i < a.chunks - 1 ? C : i == a.chunks - 1 ? last : 0; };
    auto load = [&](int i) {
        const int cnt = positions(i);
        ak.load(rk, i, cnt);
        aq.load(rq, i, cnt);
        av.load(rv, i, cnt);
        const char *r = rec + (int64_t)min(i, a.chunks - 1) * kRecord<T, false>;
        if (threadIdx.x < sizeof(Gates) / 4) gate_ahead = reinterpret_cast<const float *>(r)[threadIdx.x];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int p = 0; p < 3; ++p) Ta[u][p] = *reinterpret_cast<const bf16x8 *>(r + kAtT + (u * 3 + p) * kTile + lane * 16);
#pragma unroll
            for (int p = 0; p < kPP<T>; ++p) Pa[u][p] = *reinterpret_cast<const bf16x8 *>(r + kAtP + (u * kPP<T> + p) * kTile + lane * 16);
        }
    };
    load(0);

    for (int i = 0; i < a.chunks; ++i) {
        const int cnt = positions(i);
        bf16x8 Tm[2][3], Pm[2][kPP<T>];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int p = 0; p < 3; ++p) Tm[u][p] = Ta[u][p];
#pragma unroll
            for (int p = 0; p < kPP<T>; ++p) Pm[u][p] = Pa[u][p];
        }
        lds_barrier();  // the last chunk's reads are done
        ak.store(rk, K);
        aq.store(rq, Q);
        av.store(rv, V);
        if (threadIdx.x < sizeof(Gates) / 4) reinterpret_cast<float *>(&gates)[threadIdx.x] = gate_ahead;
        load(i + 1);
        if constexpr (!VEC) {
            if (cnt < C) {
                walk::clear_past<kP, D1, C>(K, threadIdx.x, cnt);
                walk::clear_past<kP, D1, C>(Q, threadIdx.x, cnt);
                walk::clear_past<kP, kNB, C>(V, threadIdx.x, cnt);
            }
        }
        lds_barrier();

        // K S in rows of positions, Q S in rows of columns
        f32x4 ks[2] = {}, o[2] = {};
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float v[8] = {S[2 * t][0],     S[2 * t][1],     S[2 * t][2],     S[2 * t][3],
                                S[2 * t + 1][0], S[2 * t + 1][1], S[2 * t + 1][2], S[2 * t + 1][3]};
            bf16x8 sp[3], so[kO];
            split3(v, sp);
#pragma unroll
            for (int p = 0; p < kO; ++p) so[p] = sp[p];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                bf16x8 kr[kP], qr[kP];
#pragma unroll
                for (int p = 0; p < kP; ++p) {
                    kr[p] = read_row(&K[p * kPX + tile_at<D1>(row_of(u, m), 4 * t + q)]);
                    qr[p] = read_row(&Q[p * kPX + tile_at<D1>(16 * u + m, 4 * t + q)]);
                }
                ks[u] = walk::mfma_planes(kr, sp, ks[u]);
                o[u] = walk::mfma_planes(so, qr, o[u]);
            }
        }
        // the right side b (v - f K S), in U's place
        float x[8];
        {
            bf16x8 z[kP];
            const int grp = 2 * wave + (tr_c >> 1), in = 4 * (tr_c & 1);
#pragma unroll
            for (int p = 0; p < kP; ++p)
                z[p] = walk::join(read_tr(&V[p * kPZ + tile_at<kNB>(8 * q + tr_i, grp) + in]),
                                  read_tr(&V[p * kPZ + tile_at<kNB>(8 * q + tr_i + 4, grp) + in]));
#pragma unroll
            for (int n = 0; n < 8; ++n)
                x[n] = gates.b[8 * q + n] * fmaf(-gates.f[8 * q + n], ks[n >> 2][n & 3], walk::plane_sum(z, n));
        }
        const int odd = take_odd(x, q);
        bf16x8 xp[3];
        split3(x, xp);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const f32x4 ua = walk::mfma_planes(Tm[u], xp, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
            for (int r = 0; r < 4; ++r) x[4 * u + r] = ua[r];
        }
        // outputs
        split3(x, xp);
        {
            bf16x8 up[kO];
#pragma unroll
            for (int p = 0; p < kO; ++p) up[p] = xp[p];
#pragma unroll
            for (int it = 0; it < 2; ++it) {
                o[it] *= gates.f[16 * it + m] * a.scale;
                o[it] = walk::mfma_planes(up, Pm[it], o[it]);
            }
        }
        // the state after the chunk
        const Carry carry{gates.carry, gates.fast != 0.0f};
#pragma unroll
        for (int n = 0; n < 8; ++n) x[n] *= gates.r[8 * q + n];
        split3(x, xp);
#pragma unroll
        for (int t = 0; t < NA; ++t) {
#pragma unroll
            for (int r = 0; r < 4; ++r) S[t][r] = carry(S[t][r]);
            bf16x8 y[kP];
            const int grp = 4 * (t >> 1) + tr_c, in = 4 * (t & 1);
#pragma unroll
            for (int p = 0; p < kP; ++p)
                y[p] = walk::join(read_tr(&K[p * kPX + tile_at<D1>(8 * q + tr_i, grp) + in]),
                                  read_tr(&K[p * kPX + tile_at<D1>(8 * q + tr_i + 4, grp) + in]));
            S[t] = walk::mfma_planes(y, xp, S[t]);
        }
        if (__any(odd < C)) {
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
        const __amdgpu_buffer_rsrc_t buf = walk::chunk_of(ro, i, cnt, C);
#pragma unroll
        for (int it = 0; it < 2; ++it) {
            VecT<T, 4> v;
#pragma unroll
            for (int r = 0; r < 4; ++r) v.v[r] = (T)o[it][r];
            const uint32_t at = out_at + (uint32_t)it * out_step;
            if (a.out4) {
                if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b64(*reinterpret_cast<u32x2 *>(&v), buf, at, 0, 0);
                else __builtin_amdgcn_raw_buffer_store_b128(*reinterpret_cast<u32x4 *>(&v), buf, at, 0, 0);
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const uint32_t ar = c0 + oc + r < a.dv ? at + r * (uint32_t)sizeof(T) : kNowhere;
                    if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b16(*reinterpret_cast<uint16_t *>(&v.v[r]), buf, ar, 0, 0);
                    else __builtin_amdgcn_raw_buffer_store_b32(*reinterpret_cast<uint32_t *>(&v.v[r]), buf, ar, 0, 0);
                }
            }
        }
    }
    if (a.fin != nullptr && col < a.dv) {
#pragma unroll
        for (int t = 0; t < NA; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = state_row(t, q, r);
                if (row < a.dk) a.fin[((int64_t)wh.bh * a.dk + row) * a.dv + col] = S[t][r];
            }
    }
}

// ---------------------------------------------------------------- single token
//   u = b (v - e^g k S),  S' = e^g S + k^T u,  o = scale (e^g q S + (q.k) u)
// Reads and writes the state once and is bound by that: k S and q S are formed
// in the one pass that brings S into registers, S' leaves from there.  A
// workgroup takes 64 columns of one (batch row, head); its threads are columns
// (V of them each) by rows.
constexpr int kStepCols = 64, kMaxHead = 256;

struct StepArgs {
    int64_t H;
    int group, dk, dv, nblk;
    HeadView q, k, v, log_decay, beta;
    const float *state;
    float scale;
    void *o;
    float *out_state;
};

// R rows a thread
template <typename T, int V, int R>
__global__ __launch_bounds__(kThreads) void step_kernel(StepArgs a) {
    constexpr int kTx = kStepCols / V, kTy = kThreads / kTx;
    __shared__ float qk[2][kMaxHead];
    __shared__ float part[2][kTy][kStepCols], dots[kThreads / 64];
    const uint32_t bh = blockIdx.x / (uint32_t)a.nblk, blk = blockIdx.x - bh * (uint32_t)a.nblk;
    const int64_t b = bh / (uint32_t)a.H, h = bh - b * a.H, hk = h / a.group;
    const int tx = threadIdx.x & (kTx - 1), ty = threadIdx.x / kTx;
    const int c = (int)blk * kStepCols + tx * V;
    const bool in = c < a.dv;
    const float *src = a.state + (int64_t)bh * a.dk * a.dv + c;
    float s[R][V];
#pragma unroll
    for (int u = 0; u < R; ++u) {
        const int r = ty + u * kTy;
#pragma unroll
        for (int i = 0; i < V; ++i) s[u][i] = 0.0f;
        if (in && r < a.dk) load_vec<float, V>(src + (int64_t)r * a.dv, s[u]);
    }
    const T *q = static_cast<const T *>(a.q.p) + b * a.q.st[0] + hk * a.q.st[2], *k = static_cast<const T *>(a.k.p) + b * a.k.st[0] + hk * a.k.st[2];
    float dot = 0.0f;
    if ((int)threadIdx.x < a.dk) {
        const float qr = (float)q[threadIdx.x], kr = (float)k[threadIdx.x];
        qk[0][threadIdx.x] = qr;
        qk[1][threadIdx.x] = kr;
        dot = qr * kr;
    }
    dot = lanes_sum(dot);
    if ((threadIdx.x & 63) == 0) dots[threadIdx.x >> 6] = dot;
    const float decay = expf(static_cast<const float *>(a.log_decay.p)[b * a.log_decay.st[0] + h * a.log_decay.st[2]]);
    const float beta = static_cast<const float *>(a.beta.p)[b * a.beta.st[0] + h * a.beta.st[2]];
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = in ? (float)static_cast<const T *>(a.v.p)[b * a.v.st[0] + h * a.v.st[2] + c + i] : 0.0f;
    __syncthreads();
    float acc[2][V] = {};
#pragma unroll
    for (int u = 0; u < R; ++u) {
        const int r = ty + u * kTy;
        if (r < a.dk) {
            const float qr = qk[0][r], kr = qk[1][r];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                s[u][i] *= decay;
                acc[0][i] = fmaf(qr, s[u][i], acc[0][i]);
                acc[1][i] = fmaf(kr, s[u][i], acc[1][i]);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < V; ++i) part[n][ty][tx * V + i] = acc[n][i];
    __syncthreads();
    const float qdk = (dots[0] + dots[1]) + (dots[2] + dots[3]);
    float ks[V] = {}, u_of[V];
#pragma unroll
    for (int y = 0; y < kTy; ++y)
#pragma unroll
        for (int i = 0; i < V; ++i) ks[i] += part[1][y][tx * V + i];
#pragma unroll
    for (int i = 0; i < V; ++i) u_of[i] = beta * (v[i] - ks[i]);
    if (!in) return;
    float *dst = a.out_state + (int64_t)bh * a.dk * a.dv + c;
#pragma unroll
    for (int u = 0; u < R; ++u) {
        const int r = ty + u * kTy;
        if (r < a.dk) {
            const float kr = qk[1][r];
#pragma unroll
            for (int i = 0; i < V; ++i) s[u][i] = fmaf(kr, u_of[i], s[u][i]);
            store_vec<float, V>(dst + (int64_t)r * a.dv, s[u]);
        }
    }
    if (ty == 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float sum = 0.0f;
#pragma unroll
            for (int y = 0; y < kTy; ++y) sum += part[0][y][tx * V + i];
            static_cast<T *>(a.o)[(int64_t)bh * a.dv + c + i] = (T)(a.scale * fmaf(qdk, u_of[i], sum));
        }
    }
}

namespace {

int walk_width(int d1) { return d1 <= 32 ? 32 : d1 <= 64 ? 64 : d1 <= 128 ? 128 : 256; }

int blocks_of(int cols) { return (cols + kNB - 1) / kNB; }

int64_t chunks_of(int64_t L) { return (L + C - 1) / C; }

template <typename T, int D1, bool VEC>
hipError_t forward_launch(const DeltaArgs &p, char *scratch, hipStream_t s) {
    const int64_t chunks = chunks_of(p.L), items = p.B * p.H * chunks;
    const PrepArgs prep{p.q, p.k, p.log_decay, p.beta, p.L, items, (int)p.H, (int)(p.H / p.Hk), p.dk, (int)chunks, p.scale, scratch};
    prep_kernel<T, D1, VEC, false><<<(unsigned)((items + 3) / 4), 256, 0, s>>>(prep);
    WalkArgs a{};
    a.q = view_of(p.q);
    a.k = view_of(p.k);
    a.v = view_of(p.v);
    a.out = p.o;
    a.init = p.state;
    a.fin = p.out_state;
    a.B = p.B;
    a.L = p.L;
    a.H = p.H;
    a.group = (int)(p.H / p.Hk);
    a.dk = p.dk;
    a.dv = p.dv;
    a.chunks = (int)chunks;
    a.nblk = blocks_of(p.dv);
    a.out4 = p.dv % 4 == 0 && aligned_to(p.o, 4 * sizeof(T));
    a.scale = p.scale;
    a.rec = scratch;
    walk_kernel<T, D1, VEC><<<(unsigned)((p.B * p.H + 7) / 8 * 8 * a.nblk), kThreads, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T, bool VEC>
hipError_t forward_width(const DeltaArgs &p, char *scratch, hipStream_t s) {
    switch (walk_width(p.dk)) {
        case 32: return forward_launch<T, 32, VEC>(p, scratch, s);
        case 64: return forward_launch<T, 64, VEC>(p, scratch, s);
        case 128: return forward_launch<T, 128, VEC>(p, scratch, s);
        default: return forward_launch<T, 256, VEC>(p, scratch, s);
    }
}

template <typename T>
hipError_t forward_type(const DeltaArgs &p, char *scratch, hipStream_t s) {
    const int es = sizeof(T);
    const bool vec = view_vec(p.q, p.dk, es) && view_vec(p.k, p.dk, es) && view_vec(p.v, p.dv, es);
    return vec ? forward_width<T, true>(p, scratch, s) : forward_width<T, false>(p, scratch, s);
}

template <typename T>
void step_launch(const DeltaArgs &p, const StepArgs &a, hipStream_t s) {
    const unsigned grid = (unsigned)(p.B * p.H * a.nblk);
    if (p.dv % 4 == 0 && aligned16(p.state) && aligned16(p.out_state)) {
        if (p.dk <= 128) step_kernel<T, 4, 8><<<grid, kThreads, 0, s>>>(a);
        else step_kernel<T, 4, 16><<<grid, kThreads, 0, s>>>(a);
    } else {
        if (p.dk <= 128) step_kernel<T, 1, 32><<<grid, kThreads, 0, s>>>(a);
        else step_kernel<T, 1, 64><<<grid, kThreads, 0, s>>>(a);
    }
}

}  // namespace
}  // namespace delta

size_t delta_ws(const DeltaArgs &p, bool backward) {
    if (backward) return kScratchOffset + delta::back_ws(p);
    const size_t items = (size_t)(p.B * p.H * delta::chunks_of(p.L));
    const int64_t rec = p.bf16 ? delta::kRecord<bf16, false> : delta::kRecord<float, false>;
    return kScratchOffset + items * rec;
}

hipError_t delta_forward(const DeltaArgs &p, const Ws &ws, hipStream_t s) {
    char *scratch = ws.p + kScratchOffset;
    return p.bf16 ? delta::forward_type<bf16>(p, scratch, s) : delta::forward_type<float>(p, scratch, s);
}

hipError_t delta_backward(const DeltaArgs &p, const Ws &ws, hipStream_t s) { return delta::backward(p, ws.p + kScratchOffset, s); }

hipError_t delta_step(const DeltaArgs &p, hipStream_t s) {
    const delta::StepArgs a{p.H, (int)(p.H / p.Hk), p.dk, p.dv, delta::blocks_of(p.dv), p.q, p.k, p.v, p.log_decay, p.beta,
                            p.state, p.scale, p.o, p.out_state};
    if (p.bf16) delta::step_launch<bf16>(p, a, s);
    else delta::step_launch<float>(p, a, s);
    return hipGetLastError();
}

}  // namespace prn
