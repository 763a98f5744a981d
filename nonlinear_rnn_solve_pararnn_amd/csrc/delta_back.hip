// delta_back.hip -- gradients of the gated delta rule (formulas of a chunk:
// delta.hpp).
//
// With do' = scale do, D the gradient of the state and u_t, dR_t = dLoss/d(u_t / b_t):
//   dR = T^T (P^T do + r (K D)),  D <- f_last D + (f Q)^T do' - (f b K)^T dR,
// which needs no S, as the walk that finds U and S needs no D: both run side by
// side in one launch (back_walk_kernel), whole workgroups either way, and leave
// U, dR and their states at the ends of every span of positions.  u_t and dR_t
// belong to their position, not to the chunk they were found in, so the rest is
// worked out in spans of any length (grad_kernel), all spans side by side.
// With S before the span, D after it, dr = b dR and j < i in both sums,
//   dv = dr,  db = dR.u / b,
//   dq = scale f (do S^T) + MP K,  MP_ij = E_ij do'_i.u_j (j <= i),
//   dk = r (U D^T) - f (dr S^T) + MP^T Q + (MA + MA^T) K,  MA_ij = -E_ij dr_i.u_j,
//   dg_t = f_last <D, S> + sum of those products that e^(g_t) is part of: of rows
//          from t on with S, of rows before t with D, of pairs i >= t > j.
// The last line adds terms that the gate does take part in; the shorter
// identity dg_t - dg_(t+1) = do_t.o_t - dv_t.v_t adds up others that cancel.
//
// Precision: walks as in the forward pass; S, D, U, dr, MP and MA in three planes
// whatever the tensors are, so that bf16 gradients are fp32's, rounded once.  (MP
// and MA at 16 bits took 2% off grad_kernel: B=8, L=2048, H=16, 128x128, 350 and
// 358 us on one card.)
#include "delta_walk.hpp"

namespace prn {
namespace delta {

using walk::mfma_planes;

struct BackArgs {
    HeadView q, k, v, grad_o, log_decay, beta;
    const float *init, *fin;  // S before the first position, D after the last one; null for zeros
    float *grad_init;         // or null
    int64_t L;
    int pairs, H, group, dk, dv, chunks, nblk, nblk_k, spans, span_chunks, width;  // width: rows of a state in memory
    float scale;
    const char *rec;
    float *U, *dR;  // [pairs][spans span][64 nblk]
    float *S, *D;   // [pairs][spans][width][64 nblk]
    float *part_q, *part_k;  // [B, L, H, dk] where heads share q and k, or null
    void *grad_q, *grad_k, *grad_v;
    float *grad_g, *grad_b;
    int out8, out4;  // rows of grad_v, and of grad_q and grad_k, may be stored eight or four elements at a time
    SegArgs seg;
};

// Positions a span of grad_kernel: as many as its operands in LDS and registers
// allow, as the walks write S and D once a span.  B=8, L=2048, H=16, 128x128,
// bf16: walks and grad_kernel 436 and 406 us with 32, 305 and 395 with 64.
constexpr int span_of(bool bf16, int D) { return bf16 && D <= 128 ? 64 : 32; }

template <typename T>
__device__ __forceinline__ Job job_of(const BackArgs &a, const Where &wh) {
    Job j{};
    j.q = a.q;
    j.k = a.k;
    j.L = a.L;
    j.b = wh.b;
    j.h = wh.h;
    j.hk = (int)__builtin_amdgcn_readfirstlane(wh.h / a.group);  // the division runs on the vector unit
    j.dk = a.dk;
    j.dv = a.dv;
    j.all = a.chunks;
    j.scale = a.scale;
    j.rec = a.rec + (int64_t)wh.bh * a.chunks * kRecord<true>;
    return j;
}

// The two walks: workgroups that take S from the first chunk on, and those
// that take D from the last one back.
template <typename T, int D1, bool VEC>
__global__ __launch_bounds__(walk::kThreads, (kWgs<T, D1>)) void back_walk_kernel(BackArgs a) {
    __shared__ WalkLds<T, D1> lds[kStages<T, D1>];
    const Where wh = where(a.nblk * 2 * a.seg.n, a.pairs, a.H);
    if (!wh.any) return;
    const int part = (int)__builtin_amdgcn_readfirstlane(wh.sub / a.nblk), blk = wh.sub - part * a.nblk, seg = part >> 1;
    Job j = job_of<T>(a, wh);
    j.c0 = blk * kNB;
    j.from = seg * a.seg.chunks;
    j.to = min(j.from + a.seg.chunks, a.chunks);
    j.row = a.nblk * kNB;
    j.span_chunks = a.span_chunks;
    const int64_t state = (int64_t)wh.bh * a.dk * a.dv, rows = (int64_t)wh.bh * a.spans * a.span_chunks * C * j.row,
                  states = (int64_t)wh.bh * a.spans * D1 * j.row;
    if (part & 1) {
        j.v = a.grad_o;
        if (a.seg.n > 1) j.init = seg_at<D1>(a.seg.D, a.seg, wh.bh, seg, a.seg.wide);
        else if (a.fin != nullptr) j.init = {const_cast<float *>(a.fin) + state, a.dv, a.dk, a.dv};
        if (a.grad_init != nullptr && seg == 0) j.fin = {a.grad_init + state, a.dv, a.dk, a.dv};
        j.rows = a.dR + rows;
        j.states = a.D + states;
        walk_chunks<T, D1, VEC, Role::Grad, true>(j, lds);
    } else {
        j.v = a.v;
        if (a.seg.n > 1) j.init = seg_at<D1>(a.seg.S, a.seg, wh.bh, seg, a.seg.wide);
        else if (a.init != nullptr) j.init = {const_cast<float *>(a.init) + state, a.dv, a.dk, a.dv};
        j.rows = a.U + rows;
        j.states = a.S + states;
        walk_chunks<T, D1, VEC, Role::State, true>(j, lds);
    }
}

// The segments' own parts: of S, of D, and M.
template <typename T, int D1, bool VEC>
__global__ __launch_bounds__(walk::kThreads, (kWgs<T, D1>)) void back_segment_kernel(BackArgs a) {
    __shared__ WalkLds<T, D1> lds[kStages<T, D1>];
    const int per = 2 * a.nblk + a.nblk_k;
    const Where wh = where(per * a.seg.n, a.pairs, a.H);
    if (!wh.any) return;
    const int seg = (int)__builtin_amdgcn_readfirstlane(wh.sub / per), blk = wh.sub - seg * per;
    Job j = job_of<T>(a, wh);
    j.from = seg * a.seg.chunks;
    j.to = min(j.from + a.seg.chunks, a.chunks);
    if (blk >= a.nblk && blk < 2 * a.nblk) {
        if (seg == 0) return;
        j.v = a.grad_o;
        j.c0 = (blk - a.nblk) * kNB;
        j.fin = seg_at<D1>(a.seg.D, a.seg, wh.bh, seg, a.seg.wide);
        walk_chunks<T, D1, VEC, Role::Grad, true>(j, lds);
    } else {
        j.identity = blk >= 2 * a.nblk;
        if (!j.identity && seg == a.seg.n - 1) return;
        j.c0 = (j.identity ? blk - 2 * a.nblk : blk) * kNB;
        if (j.identity) j.dv = 1 << 20;  // every column there is
        else j.v = a.v;
        j.fin = j.identity ? seg_at<D1>(a.seg.M, a.seg, wh.bh, seg, a.seg.wide_k) : seg_at<D1>(a.seg.S, a.seg, wh.bh, seg, a.seg.wide);
        walk_chunks<T, D1, VEC, Role::State, true>(j, lds);
    }
}

// ---------------------------------------------------------------- the rest, span by span
// (The walks before it write S, D, U and dR, 0.79 GB, and read 0.57 at the size
// below, in 295 us: 4.6 TB/s, memory's rate.)
// A wave owns 16 rows of S and D (16 elements of k and q) and the gradients of
// those elements at all positions of the span; S and D go from memory straight
// into operands, each element once.  LDS holds the rows of do, U and dr, then,
// in their place, those of q and k and the matrices MP and MA + MA^T.
constexpr int grad_tiles(bool bf16, int D) { return D >= 128 && span_of(bf16, D) == 32 ? 2 : 1; }
template <typename T, int D>
struct GradLds {
    static constexpr int kN = span_of(sizeof(T) == 2, D), kP = kPlanes<T>, kM = 3, kW = grad_tiles(sizeof(T) == 2, D), kWaves = D / 16 / kW;
    static constexpr int kRowsX = kN * kTileRow<D>, kRowsV = kN * kTileRow<kNB>, kRowsM = kN * kTileRow<kN>;
    struct First {
        bf16 go[kP * kRowsV], u[3 * kRowsV], dr[3 * kRowsV];
    };
    struct Second {
        bf16 k[kP * kRowsX], q[kP * kRowsX], mp[kM * kRowsM], ma[kM * kRowsM];
    };
    union alignas(16) {
        First first;
        Second second;
    };
    double G[kN];
    float f[kN], r[kN];
    float y[kWaves][kN], x[kWaves][kN], z[kWaves];  // the waves' shares of a row's products with S and with D, and of <D, S>
    float row[2][kN / 16][kN], col[2][kN / 16][kN]; // sums of pairs of either kind: of a row in a tile of columns, of a column in one of rows
};

// A wave has kW tiles of 16 elements of q and k.  With two, rows read from LDS
// serve both, and a workgroup leaves room for another one on its CU, whose loads
// go on while this one multiplies (fp32 heads of 65 to 128 spill 28 to 52 bytes a
// lane so).  With one (heads of up to 64, and bf16 up to 128) a workgroup goes
// through several spans and has the next one's first operands on their way while
// it works on the pairs.
// B=8, L=2048, H=16, 128x128, bf16: 1.0 GB read and 0.2 written in 351 us, 3.5
// TB/s, which is not memory's rate: a workgroup's phases follow each other on its
// CU (LDS and matrix instructions of the products with S and D take half of them).
// The whole backward pass 740 us with a workgroup a span, 700 so; grad_kernel with
// two tiles and two workgroups a CU 438-510 us where it took 395.  B=3, L=1000,
// H=10, 48x80, fp32: grad_kernel 62 us with one tile, 54 with two.
template <typename T, int D> constexpr bool kAhead = grad_tiles(sizeof(T) == 2, D) == 1;
template <typename T, int D> constexpr int kGradThreads = D * 4 / grad_tiles(sizeof(T) == 2, D);
template <typename T, int D, bool VEC>
__global__ __launch_bounds__((kGradThreads<T, D>), 2) void grad_kernel(BackArgs a) {
    using Lds = GradLds<T, D>;
    constexpr int N = Lds::kN, kP = Lds::kP, kM = Lds::kM, kWaves = Lds::kWaves, kW = Lds::kW, kThreadsG = kGradThreads<T, D>;
    constexpr int kX = Lds::kRowsX, kV = Lds::kRowsV, kMx = Lds::kRowsM, NI = N / 16, NS = N / 32, kTiles = NI * (NI + 1) / 2;
    __shared__ Lds l;
    struct Item {
        uint32_t bh, span, b, h, hk;
        int64_t begin;
        int cnt;
    };
    auto item_of = [&](uint32_t i) {  // (the divisions run on the vector unit; addresses want scalar registers)
        Item w;
        w.bh = same_in_lanes(i / (uint32_t)a.spans);
        w.span = i - w.bh * (uint32_t)a.spans;
        w.b = same_in_lanes(w.bh / (uint32_t)a.H);
        w.h = w.bh - w.b * (uint32_t)a.H;
        w.hk = same_in_lanes(w.h / (uint32_t)a.group);
        w.begin = (int64_t)w.span * N;
        w.cnt = (int)min((int64_t)N, a.L - w.begin);
        return w;
    };
    auto after = [&](Item w) {
        w.begin += N;
        if (++w.span == (uint32_t)a.spans) {
            w.span = 0;
            w.begin = 0;
            ++w.bh;
            if (++w.h == (uint32_t)a.H) {
                w.h = 0;
                ++w.b;
            }
            w.hk = same_in_lanes(w.h / (uint32_t)a.group);
        }
        w.cnt = (int)min((int64_t)N, a.L - w.begin);
        return w;
    };
    const int wide = a.nblk * kNB;  // columns in memory
    constexpr int kKeysAt = kThreadsG / (D / 8), kMyKeys = N / kKeysAt;
    int wave, lane, m, q, tr_i, tr_c, key_grp, key_row, grp, r0, tid;
    bool has_s;
    uint32_t lane_at;
    // Where this thread stands, worked out again for each span: kept over the loop, the
    // addresses made of it would take the registers that operands are ahead in.
    auto stand = [&]() {
        tid = threadIdx.x;
        if (kAhead<T, D>) asm volatile("" : "+v"(tid));
        wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        lane = tid & 63;
        m = lane & 15;
        q = lane >> 4;
        tr_i = m >> 2;
        tr_c = m & 3;
        key_grp = tid % (D / 8);
        key_row = tid / (D / 8);
        grp = tid & 7;
        r0 = tid >> 3;
        has_s = wave * kW * 16 < a.width;  // narrower keys have no rows there: the first ones stand in, for elements that nothing reads
        lane_at = (uint32_t)(m * wide + 8 * q);
    };

    // Rows of do, U and dr go through LDS 64 columns at a time, dv and db on the
    // way; products with S and D: lane m is position 16 it + m, registers are
    // elements 16 (kW wave + w) + 4 q ..; raw do_i.u_j and dr_i.u_j: tiles on and below the
    // diagonal go round the waves, a result's rows are i.
    bf16x8 key[kMyKeys][kP], query[kMyKeys][kP];
    auto load_keys = [&](const Item &of) {
        const T *kp = static_cast<const T *>(a.k.p) + of.b * a.k.st[0] + of.begin * a.k.st[1] + of.hk * a.k.st[2];
        const T *qp = static_cast<const T *>(a.q.p) + of.b * a.q.st[0] + of.begin * a.q.st[1] + of.hk * a.q.st[2];
#pragma unroll
        for (int n = 0; n < kMyKeys; ++n) {
            const int row = key_row + n * kKeysAt;
            load8<T, VEC>(kp + row * a.k.st[1], key_grp * 8, a.dk, row < of.cnt, key[n]);
            load8<T, VEC>(qp + row * a.q.st[1], key_grp * 8, a.dk, row < of.cnt, query[n]);
        }
    };
    constexpr int kRowsAt = kThreadsG / 8, kMyRows = (N + kRowsAt - 1) / kRowsAt;
    constexpr int kUnits = 2 * kTiles, kMine = (kUnits + kWaves - 1) / kWaves;
    auto unit_of = [&](int n) { return min(wave + n * kWaves, kUnits - 1); };
    auto tile_of = [&](int unit, int &it, int &jt) {
        const int tile = unit >= kTiles ? unit - kTiles : unit;
        it = tile < 1 ? 0 : tile < 3 ? 1 : tile < 6 ? 2 : 3;
        jt = tile - it * (it + 1) / 2;
    };
    bf16x8 go[kMyRows][kP];
    float u[kMyRows][8], d[kMyRows][8], beta[kMyRows];
    auto load_rows = [&](const Item &of, int blk) {
        const T *gop = static_cast<const T *>(a.grad_o.p) + of.b * a.grad_o.st[0] + of.begin * a.grad_o.st[1] + of.h * a.grad_o.st[2];
        const float *bp = static_cast<const float *>(a.beta.p) + of.b * a.beta.st[0] + of.begin * a.beta.st[1] + of.h * a.beta.st[2];
        const int64_t base = ((int64_t)of.bh * a.spans + of.span) * N * wide;
        const float *u_rows = a.U + base, *r_rows = a.dR + base;
#pragma unroll
        for (int n = 0; n < kMyRows; ++n) {
            const int row = r0 + n * kRowsAt, c = blk * kNB + grp * 8;
            const bool in = row < of.cnt && c < wide;
            load8<T, VEC>(gop + row * a.grad_o.st[1], c, a.dv, in, go[n]);
#pragma unroll
            for (int i = 0; i < 8; ++i) u[n][i] = d[n][i] = 0.0f;
            if (blk == 0) beta[n] = row < of.cnt ? bp[row * a.beta.st[1]] : 0.0f;
            if (in) {
                const uint32_t at = (uint32_t)(row * wide + c);
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    *reinterpret_cast<f32x4 *>(&u[n][i]) = *reinterpret_cast<const f32x4 *>(u_rows + at + i);
                    *reinterpret_cast<f32x4 *>(&d[n][i]) = *reinterpret_cast<const f32x4 *>(r_rows + at + i);
                }
            }
        }
    };
    float sv[kW][8], dv[kW][8];
    auto load_state = [&](const Item &of, int t) {
        const int64_t state = (((int64_t)of.bh * a.spans + of.span) * a.width + (has_s ? wave * kW * 16 : 0)) * wide;
        const float *s_rows = a.S + state, *d_rows = a.D + state;
#pragma unroll
        for (int w = 0; w < kW; ++w)
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                const uint32_t at = lane_at + (uint32_t)(16 * w * wide + min(32 * t, wide - 32) + i);
                *reinterpret_cast<f32x4 *>(&sv[w][i]) = *reinterpret_cast<const f32x4 *>(s_rows + at);
                *reinterpret_cast<f32x4 *>(&dv[w][i]) = *reinterpret_cast<const f32x4 *>(d_rows + at);
            }
    };
    float gate = 0.0f;  // of this thread's position
    auto load_gate = [&](const Item &of) {
        const int p = tid;
        if (p < N) gate = p < of.cnt ? static_cast<const float *>(a.log_decay.p)[of.b * a.log_decay.st[0] + (of.begin + p) * a.log_decay.st[1] + of.h * a.log_decay.st[2]] : 0.0f;
    };

    // (a workgroup's spans follow each other)
    uint32_t left = 1, first = blockIdx.x;
    if (kAhead<T, D>) {
        const uint32_t items = (uint32_t)a.pairs * (uint32_t)a.spans;
        const uint32_t each = items / gridDim.x, over = items - each * gridDim.x;
        left = each + (blockIdx.x < over ? 1 : 0);
        first = blockIdx.x * each + min(blockIdx.x, over);
    }
    stand();
    Item w = item_of(first);
    load_rows(w, 0);
    load_state(w, 0);
    load_gate(w);
    for (;;) {
        if (kAhead<T, D>) stand();
        const uint32_t b = w.b, h = w.h;
        const int64_t begin = w.begin;
        const int cnt = w.cnt;
        f32x4 aq[kW][NI] = {}, as[kW][NI] = {}, ad[kW][NI] = {}, pair[kMine] = {};
        {
            float dot[kMyRows] = {}, z = 0.0f, b_of[kMyRows];
#pragma unroll
            for (int n = 0; n < kMyRows; ++n) b_of[n] = beta[n];
            // (blocks that dv does not reach are zeros: a loop of any other number moves all sums between registers)
#pragma unroll
            for (int blk = 0; blk < D / kNB; ++blk) {
#pragma unroll
                for (int n = 0; n < kMyRows; ++n) {
                    const int row = r0 + n * kRowsAt, at = tile_at<kNB>(row, grp), c = blk * kNB + grp * 8;
                    if (N < kRowsAt && row >= N) continue;  // (whole waves)
                    const bool none = writes_none(b_of[n]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        dot[n] = fmaf(u[n][i], d[n][i], dot[n]);
                        d[n][i] = none ? 0.0f : b_of[n] * d[n][i];
                        u[n][i] = none ? 0.0f : u[n][i];
                    }
                    if (row < cnt) {
                        T *gv = static_cast<T *>(a.grad_v) + (((int64_t)b * a.L + begin) * a.H + h) * a.dv + (int64_t)row * a.H * a.dv + c;
                        if (a.out8) {
                            constexpr int kVec8 = kVec<T>;
                            if (c < a.dv) {
#pragma unroll
                                for (int o = 0; o < 8; o += kVec8) {
                                    float w[kVec8];
#pragma unroll
                                    for (int i = 0; i < kVec8; ++i) w[i] = d[n][o + i];
                                    store_vec<T, kVec8>(gv + o, w);
                                }
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                if (c + i < a.dv) gv[i] = (T)d[n][i];
                        }
                    }
                    bf16x8 p3[3];
                    split3(u[n], p3);
#pragma unroll
                    for (int p = 0; p < 3; ++p) *reinterpret_cast<bf16x8 *>(&l.first.u[p * kV + at]) = p3[p];
                    split3(d[n], p3);
#pragma unroll
                    for (int p = 0; p < 3; ++p) *reinterpret_cast<bf16x8 *>(&l.first.dr[p * kV + at]) = p3[p];
#pragma unroll
                    for (int p = 0; p < kP; ++p) *reinterpret_cast<bf16x8 *>(&l.first.go[p * kV + at]) = go[n][p];
                }
                // the next rows, ahead of the products
                auto load_next = [&]() {
                    if (blk + 1 < D / kNB) load_rows(w, blk + 1);
                    else load_keys(w);
                };
                load_next();
                __syncthreads();
                if (blk == 0 && tid < N) {  // the gates' factors, which the second half reads
                    const int p = tid;
                    double sum = (double)(gate < -1e5f ? -1e5f : gate) * 1.4426950408889634;
#pragma unroll
                    for (int n = 1; n < N; n *= 2) {
                        const double up = __shfl_up(sum, n, N);
                        if (p >= n) sum += up;
                    }
                    const double whole = __shfl(sum, N - 1, N);
                    l.G[p] = sum;
                    l.f[p] = fast_exp2((float)sum);
                    l.r[p] = fast_exp2((float)(whole - sum));
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    bf16x8 sp[kW][3], x[kP], y[3];
#pragma unroll
                    for (int w = 0; w < kW; ++w) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) z = fmaf(sv[w][i], blk * 2 + t < a.nblk * 2 ? dv[w][i] : 0.0f, z);
                        split3(sv[w], sp[w]);
                    }
#pragma unroll
                    for (int it = 0; it < NI; ++it) {
                        const int at = tile_at<kNB>(16 * it + m, 4 * t + q);
#pragma unroll
                        for (int p = 0; p < kP; ++p) x[p] = read_row(&l.first.go[p * kV + at]);
#pragma unroll
                        for (int p = 0; p < 3; ++p) y[p] = read_row(&l.first.dr[p * kV + at]);
#pragma unroll
                        for (int w = 0; w < kW; ++w) {
                            aq[w][it] = mfma_planes(sp[w], x, aq[w][it]);
                            as[w][it] = mfma_planes(sp[w], y, as[w][it]);
                        }
                        __builtin_amdgcn_sched_barrier(0);  // or reads are brought forward into registers that are not there
                    }
#pragma unroll
                    for (int w = 0; w < kW; ++w) split3(dv[w], sp[w]);
                    if (blk * 2 + t + 1 < D / 32) load_state(w, blk * 2 + t + 1);
#pragma unroll
                    for (int it = 0; it < NI; ++it) {
                        const int at = tile_at<kNB>(16 * it + m, 4 * t + q);
#pragma unroll
                        for (int p = 0; p < 3; ++p) y[p] = read_row(&l.first.u[p * kV + at]);
#pragma unroll
                        for (int w = 0; w < kW; ++w) ad[w][it] = mfma_planes(sp[w], y, ad[w][it]);
                        __builtin_amdgcn_sched_barrier(0);
                    }
#pragma unroll
                    for (int n = 0; n < kMine; ++n) {
                        const int unit = unit_of(n);
                        int it, jt;
                        tile_of(unit, it, jt);
                        const int ai = tile_at<kNB>(16 * it + m, 4 * t + q), aj = tile_at<kNB>(16 * jt + m, 4 * t + q);
                        bf16x8 y[3];
#pragma unroll
                        for (int p = 0; p < 3; ++p) y[p] = read_row(&l.first.u[p * kV + aj]);
                        // (what a unit is is known beforehand but for those in the middle)
                        const bool erase = n * kWaves >= kTiles || ((n + 1) * kWaves > kTiles && unit >= kTiles);
                        if (erase) {
                            bf16x8 x[3];
#pragma unroll
                            for (int p = 0; p < 3; ++p) x[p] = read_row(&l.first.dr[p * kV + ai]);
                            pair[n] = mfma_planes(x, y, pair[n]);
                        } else {
                            bf16x8 x[kP];
#pragma unroll
                            for (int p = 0; p < kP; ++p) x[p] = read_row(&l.first.go[p * kV + ai]);
                            pair[n] = mfma_planes(x, y, pair[n]);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
                __syncthreads();
            }
            z = lanes_sum(z);
            if (lane == 0) l.z[wave] = has_s ? z : 0.0f;
#pragma unroll
            for (int n = 0; n < kMyRows; ++n) {
                const int row = r0 + n * kRowsAt;
#pragma unroll
                for (int s = 1; s < 8; s *= 2) dot[n] += __shfl_xor(dot[n], s, 8);
                if (grp == 0 && row < cnt && a.grad_b != nullptr) {
                    a.grad_b[((int64_t)b * a.L + begin + row) * a.H + h] = dot[n] / (writes_none(b_of[n]) ? kTinyBeta : b_of[n]);
                }
            }
        }

        // rows of q and k in their place
        {
#pragma unroll
            for (int n = 0; n < kMyKeys; ++n) {
                const int at = tile_at<D>(key_row + n * kKeysAt, key_grp);
#pragma unroll
                for (int p = 0; p < kP; ++p) {
                    *reinterpret_cast<bf16x8 *>(&l.second.k[p * kX + at]) = key[n][p];
                    *reinterpret_cast<bf16x8 *>(&l.second.q[p * kX + at]) = query[n][p];
                }
            }
            // the tiles above those on the diagonal that are read with them
            for (int i = tid; i < 2 * kM * NS * 16 * 2; i += kThreadsG) {
                const int half = i & 1, r = i >> 1 & 15, s = (i >> 5) % NS, k = (i >> 5) / NS;
                const bf16x8 zero = {};
                *reinterpret_cast<bf16x8 *>(&(k < kM ? l.second.mp : l.second.ma)[(k < kM ? k : k - kM) * kMx + tile_at<N>(32 * s + 16 + r, 4 * s + half)]) = zero;
            }
        }
        // the next span's first operands, on their way while this one's pairs are at work
        if (kAhead<T, D>) stand();
        const bool more = kAhead<T, D> && --left > 0;
        if (more) {
            w = after(w);
            load_rows(w, 0);
            load_state(w, 0);
            load_gate(w);
        }
        __syncthreads();
        f32x4 dots[kMine] = {};
        auto add_dots = [&](int n, int t) {
            const int unit = unit_of(n);
            int it, jt;
            tile_of(unit, it, jt);
            const bf16 *left = unit >= kTiles ? l.second.k : l.second.q;
            bf16x8 x[kP], y[kP];
#pragma unroll
            for (int p = 0; p < kP; ++p) {
                x[p] = read_row(&left[p * kX + tile_at<D>(16 * it + m, 4 * t + q)]);
                y[p] = read_row(&l.second.k[p * kX + tile_at<D>(16 * jt + m, 4 * t + q)]);
            }
            dots[n] = mfma_planes(x, y, dots[n]);
        };
        if (kAhead<T, D>) {  // side by side where there are registers for it
#pragma unroll
            for (int t = 0; t < D / 32; ++t)
#pragma unroll
                for (int n = 0; n < kMine; ++n) add_dots(n, t);
        }
#pragma unroll
        for (int n = 0; n < kMine; ++n) {
            if (wave + n * kWaves >= kUnits) continue;
            if (!kAhead<T, D>) {
#pragma unroll
                for (int t = 0; t < D / 32; ++t) add_dots(n, t);
            }
            const int unit = unit_of(n);
            int it, jt;
            tile_of(unit, it, jt);
            const bool erase = unit >= kTiles;
            float cols = 0.0f, mine[8] = {};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * it + 4 * q + r, j = 16 * jt + m;
                const float e = j <= i ? fast_exp2((float)(l.G[i] - l.G[j])) : 0.0f;
                const float w = erase ? (j < i ? -e * pair[n][r] : 0.0f) : a.scale * e * pair[n][r];
                const float both = j < i ? w * dots[n][r] : 0.0f;
                cols += both;
                const float rows = lanes16_sum(both);
                if (m == 0) l.row[erase][jt][i] = rows;
                mine[r] = w;
            }
            // MP and MA are kept by columns: a lane's four results are neighbours there
            bf16x8 p[kM];
            walk::to_planes(mine, p);
            bf16 *to = &(erase ? l.second.ma : l.second.mp)[tile_at<N>(16 * jt + m, 2 * it + (q >> 1)) + 4 * (q & 1)];
#pragma unroll
            for (int k = 0; k < kM; ++k) *reinterpret_cast<u32x2 *>(to + k * kMx) = *reinterpret_cast<const u32x2 *>(&p[k]);
            cols += __shfl_xor(cols, 16);
            cols += __shfl_xor(cols, 32);
            if (q == 0) l.col[erase][it][16 * jt + m] = cols;
        }
        __syncthreads();

        // the products with S and D weighted; a row's products with them are the gates' share
#pragma unroll
        for (int it = 0; it < NI; ++it) {
            const int pos = 16 * it + m;
            const float f = l.f[pos], r = l.r[pos];
            float x = 0.0f, y = 0.0f;
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                const int at = tile_at<D>(pos, 2 * (wave * kW + w) + (q >> 1)) + 4 * (q & 1);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    float qv = 0.0f, kv = 0.0f;
#pragma unroll
                    for (int p = 0; p < kP; ++p) {
                        qv += (float)l.second.q[p * kX + at + n];
                        kv += (float)l.second.k[p * kX + at + n];
                    }
                    aq[w][it][n] *= f * a.scale;
                    as[w][it][n] *= f;
                    ad[w][it][n] *= r;
                    y = fmaf(qv, aq[w][it][n], fmaf(-kv, as[w][it][n], y));
                    x = fmaf(kv, ad[w][it][n], x);
                    ad[w][it][n] -= as[w][it][n];
                }
            }
            x += __shfl_xor(x, 16);
            y += __shfl_xor(y, 16);
            x += __shfl_xor(x, 32);
            y += __shfl_xor(y, 32);
            if (q == 0) {
                l.x[wave][pos] = x;
                l.y[wave][pos] = y;
            }
        }
        // the pairs: dq += MP K, dk += MP^T Q + (MA + MA^T) K
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const int row = 32 * s + 8 * q + tr_i, in = 4 * (tr_c & 1);
            bf16x8 kt[kW][kP], qt[kW][kP];
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                const int grp = 2 * (wave * kW + w) + (tr_c >> 1);
#pragma unroll
                for (int p = 0; p < kP; ++p) {
                    kt[w][p] = walk::join(read_tr(&l.second.k[p * kX + tile_at<D>(row, grp) + in]), read_tr(&l.second.k[p * kX + tile_at<D>(row + 4, grp) + in]));
                    qt[w][p] = walk::join(read_tr(&l.second.q[p * kX + tile_at<D>(row, grp) + in]), read_tr(&l.second.q[p * kX + tile_at<D>(row + 4, grp) + in]));
                }
            }
#pragma unroll
            for (int it = 0; it < NI; ++it) {
                bf16x8 x[kM];
                auto down = [&](const bf16 *M) {  // lane m: row 16 it + m of M, elements j
                    const int g2 = 2 * it + (tr_c >> 1);
#pragma unroll
                    for (int p = 0; p < kM; ++p)
                        x[p] = walk::join(read_tr(&M[p * kMx + tile_at<N>(row, g2) + in]), read_tr(&M[p * kMx + tile_at<N>(row + 4, g2) + in]));
                };
                auto along = [&](const bf16 *M) {  // lane m: column 16 it + m, elements i
#pragma unroll
                    for (int p = 0; p < kM; ++p) x[p] = read_row(&M[p * kMx + tile_at<N>(16 * it + m, 4 * s + q)]);
                };
                if (s <= it / 2) {
                    down(l.second.mp);
#pragma unroll
                    for (int w = 0; w < kW; ++w) aq[w][it] = mfma_planes(kt[w], x, aq[w][it]);
                    down(l.second.ma);
#pragma unroll
                    for (int w = 0; w < kW; ++w) ad[w][it] = mfma_planes(kt[w], x, ad[w][it]);
                }
                if (s >= it / 2) {
                    along(l.second.mp);
#pragma unroll
                    for (int w = 0; w < kW; ++w) ad[w][it] = mfma_planes(qt[w], x, ad[w][it]);
                    along(l.second.ma);
#pragma unroll
                    for (int w = 0; w < kW; ++w) ad[w][it] = mfma_planes(kt[w], x, ad[w][it]);
                }
            }
        }
#pragma unroll
        for (int it = 0; it < NI; ++it) {
            const int pos = 16 * it + m;
            if (pos >= cnt) continue;
            const int64_t row = b * a.L + begin + pos;
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                const int c = 16 * (wave * kW + w) + 4 * q;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float v[4];
#pragma unroll
                    for (int n = 0; n < 4; ++n) v[n] = k ? ad[w][it][n] : aq[w][it][n];
                    if (a.part_q != nullptr) {
                        float *to = (k ? a.part_k : a.part_q) + (row * a.H + h) * a.dk + c;
#pragma unroll
                        for (int n = 0; n < 4; ++n)
                            if (c + n < a.dk) to[n] = v[n];
                    } else {
                        T *to = static_cast<T *>(k ? a.grad_k : a.grad_q) + (row * a.H + h) * a.dk + c;
                        if (a.out4) {
                            if (c < a.dk) store_vec<T, 4>(to, v);
                        } else {
#pragma unroll
                            for (int n = 0; n < 4; ++n)
                                if (c + n < a.dk) to[n] = (T)v[n];
                        }
                    }
                }
            }
        }
        const float f_last = l.f[N - 1];
        __syncthreads();
        if (wave == kWaves - 1 && a.grad_g != nullptr) {  // (the others go on to the next span)
            const int p = lane & (N - 1), t = p >> 4;
            double x = 0.0, y = 0.0, z = 0.0;
            for (int w = 0; w < kWaves; ++w) {
                x += l.x[w][p];
                y += l.y[w][p];
                z += l.z[w];
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int n = 0; n < NI; ++n) {
                    if (n <= t) y += l.row[k][n][p];
                    if (n >= t) y -= l.col[k][n][p];
                }
            const double own = x;
#pragma unroll
            for (int d = 1; d < N; d *= 2) {
                const double before = __shfl_up(x, d, N), after = __shfl_down(y, d, N);
                if (p >= d) x += before;
                if (p + d < N) y += after;
            }
            if (lane < cnt) a.grad_g[(b * a.L + begin + p) * a.H + h] = (float)((double)f_last * z + y + (x - own));
        }
        if (!more) return;
    }
}

template <typename T, int D, bool VEC>
void grad_launch(const BackArgs &a, hipStream_t s) {
    constexpr int kThreadsG = kGradThreads<T, D>;
    static const int per_cu = blocks_per_cu(reinterpret_cast<const void *>(grad_kernel<T, D, VEC>), kThreadsG);
    const int64_t items = (int64_t)a.pairs * a.spans, slots = (int64_t)per_cu * device_cu_count();
    grad_kernel<T, D, VEC><<<(unsigned)(kAhead<T, D> ? std::min(items, slots) : items), kThreadsG, 0, s>>>(a);
}

// Gradients of shared heads: out [rows, Hk, dk] = sums of part [rows, Hk, group, dk] over the group, in its order.
template <typename T>
__global__ __launch_bounds__(256) void share_kernel(const float *part_q, const float *part_k, void *out_q, void *out_k, int64_t n, int group, int dk) {
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (at >= n) return;
    const int64_t head = at / dk;
    const float *src = (blockIdx.y ? part_k : part_q) + head * group * dk + (at - head * dk);
    float sum = 0.0f;
    for (int g = 0; g < group; ++g) sum += src[(int64_t)g * dk];
    static_cast<T *>(blockIdx.y ? out_k : out_q)[at] = (T)sum;
}

namespace {

// Width that the span kernel is built for: the wider of the two heads'.
int span_width(const DeltaArgs &p) {
    const int d = std::max(p.dk, p.dv);
    return d <= 64 ? 64 : d <= 128 ? 128 : 256;
}

// Where the parts of the workspace begin.
struct BackPlan {
    int64_t chunks, spans;
    int span, segs, seg_chunks;
    size_t u, dr, s, d, pq, pk, seg_s, seg_d, seg_m, total;
    bool parts;
};
BackPlan back_plan(const DeltaArgs &p) {
    BackPlan w{};
    const int64_t pairs = p.B * p.H, D1 = walk_width(p.dk), wide = (p.dv + kNB - 1) / kNB * kNB, wide_k = (D1 + kNB - 1) / kNB * kNB;
    w.span = span_of(p.bf16, span_width(p));
    w.chunks = chunks_of(p.L);
    w.spans = (p.L + w.span - 1) / w.span;
    w.segs = segments(pairs, 2, (int)(wide / kNB), w.chunks, p.bf16, (int)D1);
    w.seg_chunks = (int)((w.chunks + w.segs - 1) / w.segs);
    w.segs = (int)((w.chunks + w.seg_chunks - 1) / w.seg_chunks);
    w.parts = p.H > p.Hk;
    size_t at = 0;
    auto take = [&](int64_t floats) {
        const size_t here = at;
        at += ((size_t)floats * 4 + 255) / 256 * 256;
        return here;
    };
    take(pairs * w.chunks * kRecord<true> / 4);
    w.u = take(pairs * w.spans * w.span * wide);
    w.dr = take(pairs * w.spans * w.span * wide);
    w.s = take(pairs * w.spans * D1 * wide);
    w.d = take(pairs * w.spans * D1 * wide);
    w.pq = take(w.parts ? pairs * p.L * p.dk : 0);
    w.pk = take(w.parts ? pairs * p.L * p.dk : 0);
    const int64_t slots = w.segs > 1 ? pairs * w.segs * D1 : 0;
    w.seg_s = take(slots * wide);
    w.seg_d = take(slots * wide);
    w.seg_m = take(slots * wide_k);
    w.total = at;
    return w;
}

template <typename T, int D1, bool VEC>
hipError_t back_walks(const DeltaArgs &p, const BackPlan &w, BackArgs &a, char *scratch, hipStream_t s) {
    const int64_t pairs = p.B * p.H, items = pairs * w.chunks, eights = (pairs + 7) / 8 * 8;
    const PrepArgs prep{p.q, p.k, p.log_decay, p.beta, p.L, items, (int)p.H, a.group, p.dk, (int)w.chunks, p.scale, scratch};
    prep_kernel<T, D1, VEC, true><<<(unsigned)((items + 3) / 4), 256, 0, s>>>(prep);
    if (w.segs > 1) {
        back_segment_kernel<T, D1, VEC><<<(unsigned)(eights * (2 * a.nblk + a.nblk_k) * w.segs), walk::kThreads, 0, s>>>(a);
        const JoinArgs join{a.seg, p.state, p.grad_out_state, p.dk, p.dv, a.nblk * (kNB / 16)};
        join_kernel<D1><<<dim3((unsigned)(pairs * join.cols), 2), D1 * 2, 0, s>>>(join);
    }
    back_walk_kernel<T, D1, VEC><<<(unsigned)(eights * a.nblk * 2 * w.segs), walk::kThreads, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T, bool VEC>
hipError_t back_launch(const DeltaArgs &p, char *scratch, hipStream_t s) {
    const BackPlan w = back_plan(p);
    const int64_t pairs = p.B * p.H;
    auto at = [&](size_t n) { return reinterpret_cast<float *>(scratch + n); };
    BackArgs a{};
    a.q = p.q;
    a.k = p.k;
    a.v = p.v;
    a.grad_o = p.grad_o;
    a.log_decay = p.log_decay;
    a.beta = p.beta;
    a.init = p.state;
    a.fin = p.grad_out_state;
    a.grad_init = p.grad_state;
    a.L = p.L;
    a.pairs = (int)pairs;
    a.H = (int)p.H;
    a.group = (int)(p.H / p.Hk);
    a.dk = p.dk;
    a.dv = p.dv;
    a.chunks = (int)w.chunks;
    a.nblk = (p.dv + kNB - 1) / kNB;
    a.nblk_k = (walk_width(p.dk) + kNB - 1) / kNB;  // a matrix M is square
    a.spans = (int)w.spans;
    a.span_chunks = w.span / C;
    a.width = walk_width(p.dk);
    a.scale = p.scale;
    a.rec = scratch;
    a.U = at(w.u);
    a.dR = at(w.dr);
    a.S = at(w.s);
    a.D = at(w.d);
    a.part_q = w.parts ? at(w.pq) : nullptr;
    a.part_k = w.parts ? at(w.pk) : nullptr;
    a.grad_q = p.grad_q;
    a.grad_k = p.grad_k;
    a.grad_v = p.grad_v;
    a.grad_g = p.grad_log_decay;
    a.grad_b = p.grad_beta;
    a.out8 = p.dv % 8 == 0 && aligned16(p.grad_v);
    a.out4 = p.dk % 4 == 0 && aligned_to(p.grad_q, 4 * sizeof(T)) && aligned_to(p.grad_k, 4 * sizeof(T));
    a.seg = {w.segs, w.seg_chunks, at(w.seg_s), at(w.seg_d), at(w.seg_m), a.nblk * kNB, a.nblk_k * kNB};
    hipError_t e;
    switch (a.width) {
        case 32: e = back_walks<T, 32, VEC>(p, w, a, scratch, s); break;
        case 64: e = back_walks<T, 64, VEC>(p, w, a, scratch, s); break;
        case 128: e = back_walks<T, 128, VEC>(p, w, a, scratch, s); break;
        default: e = back_walks<T, 256, VEC>(p, w, a, scratch, s); break;
    }
    if (e != hipSuccess) return e;
    switch (span_width(p)) {
        case 64: grad_launch<T, 64, VEC>(a, s); break;
        case 128: grad_launch<T, 128, VEC>(a, s); break;
        default: grad_launch<T, 256, VEC>(a, s); break;
    }
    if (w.parts) {
        const int64_t n = p.B * p.L * p.Hk * p.dk;
        share_kernel<T><<<dim3((unsigned)((n + 255) / 256), 2), 256, 0, s>>>(a.part_q, a.part_k, a.grad_q, a.grad_k, n, a.group, p.dk);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t back_type(const DeltaArgs &p, char *scratch, hipStream_t s) {
    const int es = sizeof(T);
    const bool vec = view_vec(p.q, p.dk, es) && view_vec(p.k, p.dk, es) && view_vec(p.v, p.dv, es) && view_vec(p.grad_o, p.dv, es);
    return vec ? back_launch<T, true>(p, scratch, s) : back_launch<T, false>(p, scratch, s);
}

}  // namespace

size_t back_ws(const DeltaArgs &p) { return back_plan(p).total; }
hipError_t backward(const DeltaArgs &p, char *scratch, hipStream_t s) {
    return p.bf16 ? back_type<bf16>(p, scratch, s) : back_type<float>(p, scratch, s);
}

}  // namespace delta
}  // namespace prn
