// delta.hip -- the gated delta rule over whole sequences and its single-token
// step (formulas and chunks: delta.hpp; the walks: delta_walk.hpp).
#include "delta_walk.hpp"

namespace prn {

namespace delta {

struct ForwardArgs {
    HeadView q, k, v;
    void *out;
    const float *init;
    float *fin;
    int64_t L;
    int pairs, H, group, dk, dv, chunks, nblk, nblk_k, out4;
    float scale;
    const char *rec;
    SegArgs seg;
};

__device__ __forceinline__ Job job_of(const ForwardArgs &a, const Where &wh, int64_t record) {
    Job j{};
    j.q = a.q;
    j.k = a.k;
    j.v = a.v;
    j.L = a.L;
    j.b = wh.b;
    j.h = wh.h;
    j.hk = (int)__builtin_amdgcn_readfirstlane(wh.h / a.group);  // the division runs on the vector unit
    j.dk = a.dk;
    j.dv = a.dv;
    j.all = a.chunks;
    j.scale = a.scale;
    j.rec = a.rec + (int64_t)wh.bh * a.chunks * record;
    j.H = a.H;
    return j;
}

template <typename T, int D1, bool VEC>
__global__ __launch_bounds__(walk::kThreads, (kWgs<T, D1>)) void walk_kernel(ForwardArgs a) {
    __shared__ WalkLds<T, D1> lds[kStages<T, D1>];
    const Where wh = where(a.nblk * a.seg.n, a.pairs, a.H);
    if (!wh.any) return;
    const int seg = (int)__builtin_amdgcn_readfirstlane(wh.sub / a.nblk), blk = wh.sub - seg * a.nblk;
    Job j = job_of(a, wh, kRecord<false>);
    j.c0 = blk * kNB;
    j.from = seg * a.seg.chunks;
    j.to = min(j.from + a.seg.chunks, a.chunks);
    const int64_t state = (int64_t)wh.bh * a.dk * a.dv;
    if (a.seg.n > 1) j.init = seg_at<D1>(a.seg.S, a.seg, wh.bh, seg, a.seg.wide);
    else if (a.init != nullptr) j.init = {const_cast<float *>(a.init) + state, a.dv, a.dk, a.dv};
    if (a.fin != nullptr && j.to == a.chunks) j.fin = {a.fin + state, a.dv, a.dk, a.dv};
    j.out = a.out;
    j.out4 = a.out4;
    walk_chunks<T, D1, VEC, Role::Out, false>(j, lds);
}

// The segments' own parts: blocks of V's columns from zero, then of the identity's.
template <typename T, int D1, bool VEC>
__global__ __launch_bounds__(walk::kThreads, (kWgs<T, D1>)) void segment_kernel(ForwardArgs a) {
    __shared__ WalkLds<T, D1> lds[kStages<T, D1>];
    const int per = a.nblk + a.nblk_k;
    const Where wh = where(per * (a.seg.n - 1), a.pairs, a.H);
    if (!wh.any) return;
    const int seg = (int)__builtin_amdgcn_readfirstlane(wh.sub / per), blk = wh.sub - seg * per;
    Job j = job_of(a, wh, kRecord<false>);
    j.from = seg * a.seg.chunks;
    j.to = j.from + a.seg.chunks;
    j.identity = blk >= a.nblk;
    j.c0 = (j.identity ? blk - a.nblk : blk) * kNB;
    if (j.identity) {
        j.v.p = nullptr;
        j.dv = 1 << 20;  // every column there is
    }
    j.fin = j.identity ? seg_at<D1>(a.seg.M, a.seg, wh.bh, seg, a.seg.wide_k) : seg_at<D1>(a.seg.S, a.seg, wh.bh, seg, a.seg.wide);
    walk_chunks<T, D1, VEC, Role::State, false>(j, lds);
}

// ---------------------------------------------------------------- single token
//   u = b (v - e^g k S),  S' = e^g S + k^T u,  o = scale (e^g q S + (q.k) u)
// Reads and writes the state once and is bound by that: k S and q S are formed
// in the one pass that brings S into registers, S' leaves from there.  A
// workgroup takes 64 columns of one (batch row, head); its threads are columns
// (V of them each) by rows.  B=128, H=16, 128x128, bf16: 55 us (the kernel 48), 4.9
// TB/s; B=1: 11 us, most of it the host's.  Rows that are not 16-byte vectors move
// an element a thread, 2.8 TB/s: 128x127 95 us.  (A form of 32 rows a thread for
// dk up to 128 there, as R is 8 and 16 for vectors, spilled 1796 bytes a lane and
// took 3650.)
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
__global__ __launch_bounds__(walk::kThreads) void step_kernel(StepArgs a) {
    constexpr int kTx = kStepCols / V, kTy = walk::kThreads / kTx;
    __shared__ float qk[2][kMaxHead];
    __shared__ float part[2][kTy][kStepCols], dots[walk::kThreads / 64];
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

int blocks_of(int cols) { return (cols + kNB - 1) / kNB; }
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

struct ForwardPlan {
    int64_t chunks;
    int segs, seg_chunks;
    size_t seg_s, seg_m, total;  // where the segments' states are
};
ForwardPlan forward_plan(const DeltaArgs &p) {
    ForwardPlan w{};
    const int D1 = walk_width(p.dk);
    const int64_t pairs = p.B * p.H;
    w.chunks = chunks_of(p.L);
    w.segs = segments(pairs, 1, blocks_of(p.dv), w.chunks, p.bf16, D1);
    w.seg_chunks = (int)((w.chunks + w.segs - 1) / w.segs);
    w.segs = (int)((w.chunks + w.seg_chunks - 1) / w.seg_chunks);
    const size_t slots = w.segs > 1 ? (size_t)(pairs * w.segs) * D1 * 4 : 0;
    w.seg_s = round256((size_t)(pairs * w.chunks) * kRecord<false>);
    w.seg_m = w.seg_s + round256(slots * blocks_of(p.dv) * kNB);
    w.total = w.seg_m + slots * blocks_of(D1) * kNB;
    return w;
}

template <typename T, int D1, bool VEC>
hipError_t forward_launch(const DeltaArgs &p, char *scratch, hipStream_t s) {
    const ForwardPlan w = forward_plan(p);
    const int64_t pairs = p.B * p.H, items = pairs * w.chunks;
    const int group = (int)(p.H / p.Hk);
    const PrepArgs prep{p.q, p.k, p.log_decay, p.beta, p.L, items, (int)p.H, group, p.dk, (int)w.chunks, p.scale, scratch};
    prep_kernel<T, D1, VEC, false><<<(unsigned)((items + 3) / 4), 256, 0, s>>>(prep);
    ForwardArgs a{};
    a.q = p.q;
    a.k = p.k;
    a.v = p.v;
    a.out = p.o;
    a.init = p.state;
    a.fin = p.out_state;
    a.L = p.L;
    a.pairs = (int)pairs;
    a.H = (int)p.H;
    a.group = group;
    a.dk = p.dk;
    a.dv = p.dv;
    a.chunks = (int)w.chunks;
    a.nblk = blocks_of(p.dv);
    a.nblk_k = blocks_of(D1);  // a matrix M is square
    a.out4 = p.dv % 4 == 0 && aligned_to(p.o, 4 * sizeof(T));
    a.scale = p.scale;
    a.rec = scratch;
    a.seg = {w.segs, w.seg_chunks, reinterpret_cast<float *>(scratch + w.seg_s), nullptr, reinterpret_cast<float *>(scratch + w.seg_m),
             a.nblk * kNB, a.nblk_k * kNB};
    const int64_t eights = (pairs + 7) / 8 * 8;
    if (w.segs > 1) {
        segment_kernel<T, D1, VEC><<<(unsigned)(eights * (a.nblk + a.nblk_k) * (w.segs - 1)), walk::kThreads, 0, s>>>(a);
        const JoinArgs join{a.seg, p.state, nullptr, p.dk, p.dv, a.nblk * (kNB / 16)};
        join_kernel<D1><<<dim3((unsigned)(pairs * join.cols), 1), D1 * 2, 0, s>>>(join);
    }
    walk_kernel<T, D1, VEC><<<(unsigned)(eights * a.nblk * w.segs), walk::kThreads, 0, s>>>(a);
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
        if (p.dk <= 128) step_kernel<T, 4, 8><<<grid, walk::kThreads, 0, s>>>(a);
        else step_kernel<T, 4, 16><<<grid, walk::kThreads, 0, s>>>(a);
    } else {
        step_kernel<T, 1, 64><<<grid, walk::kThreads, 0, s>>>(a);
    }
}

}  // namespace

// Segments of a sequence of `chunks` that each (batch row, head) pair's `walks`
// (one forward, S and D backward) go through for `blocks` of 64 columns, 1 for
// none: as many as the CUs hold with two workgroups each, of 8 chunks at the
// least, and more than 8 if they keep 16 chunks, where the estimate below says
// that they take less time than the whole walk.  It counts in chunks of a walk:
// both passes' workgroups in rounds of what fits on the card (two workgroups on a
// CU take 1.4 times as long as one), a segment's own part at 0.8 of a walk, 3
// chunks until a workgroup is under way, and the join of a segment, twice for S
// and D.  Heads above 128 join slowly, and take no segments where fewer than four
// workgroups' room is there for each of the whole walk's.
// Against whole walks, 540 sizes (seven types and widths, both passes, 8 to 104
// workgroups, L=1024 to 8192): 0.3% slower on average than the better of the two and
// 11% at most; segments wherever they fit 6% and twice (B=1, L=1024, H=20, 256x256,
// bf16 140 whole, 286 with 4), none 44%.  Where they pay, us, with their number in brackets: H=16,
// 128x128, bf16: B=1, L=4096: 286 whole, 129 (8), 147 (16); B=2, L=4096: 298 whole, 207
// (4), 204 (8); B=1, L=1024: 85 whole, 90 (2), 67 (4).  fp32, B=1, H=8, L=32768: 64x64:
// 2682 whole, 320 (32), 328 (64); 64x128: 420 (16), 350 (32).  Backward, H=8, L=2048,
// 128x128: bf16 204 whole, 120 (8), fp32 322 whole, 172 (8).
int segments(int64_t pairs, int walks, int blocks, int64_t chunks, bool bf16, int width) {
    const int64_t cus = device_cu_count(), groups = pairs * walks * blocks;
    const int64_t most = 2 * cus / groups, n = std::min({most, chunks / 8, std::max<int64_t>(8, chunks / 16)});
    const int wgs = walk_wgs(bf16, width), key_blocks = blocks_of(width);
    if (most < 5 || n < 4 || (width > 128 && most < 8)) return 1;
    auto rounds = [&](int64_t workgroups) {
        const int64_t full = workgroups / (wgs * cus), rest = workgroups - full * wgs * cus;
        const double whole = wgs == 2 ? 1.4 : 1.0;
        return (double)full * whole + (rest == 0 ? 0.0 : rest <= cus ? 1.0 : whole);
    };
    const double join = walks * (width <= 64 ? 0.5 : width <= 128 ? 1.0 : bf16 ? 5.0 : 2.9);
    // (a backward pass takes M of the last segment as well)
    const double own = 0.8 * rounds(groups * (n - 1) + pairs * key_blocks * (walks == 2 ? n : n - 1));
    const double cut = (own + rounds(groups * n)) * ((double)chunks / (double)n + 3.0) + join * (double)n;
    return cut < rounds(groups) * ((double)chunks + 3.0) ? (int)n : 1;
}

}  // namespace delta

size_t delta_ws(const DeltaArgs &p, bool backward) {
    return kScratchOffset + (backward ? delta::back_ws(p) : delta::forward_plan(p).total);
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
