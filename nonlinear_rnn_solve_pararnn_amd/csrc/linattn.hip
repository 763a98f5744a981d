// linattn.hip -- linear attention with a decay per head: the walks over whole
// sequences (walk.hpp) and the single-token step.
#include "walk.hpp"

namespace prn {

namespace {

constexpr int kThreads = 256;

// Width of the state's rows a walk is built for.
int walk_width(int d1) { return d1 <= 32 ? 32 : d1 <= 64 ? 64 : d1 <= 96 ? 96 : d1 <= 128 ? 128 : 256; }

struct WalkPlan {
    int d1, nblk, walks, segs, chunk;
    int64_t seg_len;
    size_t bytes;  // segment states
};

// A walk is sequential, so few (batch row, head, column block) walks leave
// CUs idle.  Below one walk a CU the sequence is cut into segments whose own
// states are found first and joined, as many as keep two workgroups on every
// CU in one round (B=1, L=32771, H=8, 64x128 fp32: 32 segments 186 us, 48 199,
// 64 194); from one walk a CU on the second reading of Y and Z costs more than
// it gains (B=8, L=2048, H=16, 128x128 bf16: 95 us whole, 122 in two).
WalkPlan walk_plan(const LinattnArgs &p, bool backward) {
    auto blocks = [](int cols) { return (cols + walk::kNB - 1) / walk::kNB; };
    WalkPlan w;
    w.walks = backward ? 3 : 1;
    w.d1 = walk_width(backward ? std::max(p.dk, p.dv) : p.dk);
    w.nblk = backward ? blocks(std::max(p.dk, p.dv)) : blocks(p.dv);
    const int64_t cus = device_cu_count(), pairs = p.B * p.H;
    const int64_t groups = pairs * (backward ? 2 * blocks(p.dk) + blocks(p.dv) : blocks(p.dv));
    // fp32: 32 positions, as three planes of 64 would leave room for one
    // workgroup a CU; bf16: see kWgs
    w.chunk = p.bf16 && groups <= 2 * cus && p.L > walk::kShort ? 64 : 32;
    const int C = w.chunk;
    const int64_t chunks = (p.L + C - 1) / C;
    int64_t segs = groups >= cus ? 1 : std::min<int64_t>(2 * cus / groups, chunks / 4);
    if (segs < 2) segs = 1;
    w.seg_len = (chunks + segs - 1) / segs * C;
    w.segs = (int)((p.L + w.seg_len - 1) / w.seg_len);
    w.bytes = w.segs > 1 ? (size_t)pairs * w.walks * w.nblk * w.segs * 4 * (w.d1 / 16) * 64 * 16 : 0;
    return w;
}

// Rows that overlap are left to the loads of any alignment, whose rows past the
// last position are cleared: here they would find elements of the last rows.
bool view_vec(const WalkView &v, int d, int es) {
    const int64_t n = 16 / es;
    return d % n == 0 && aligned16(v.p) && v.sb % n == 0 && v.st % n == 0 && v.sh % n == 0 && (v.st >= d || v.st == 0);
}

// Whether every operand of every walk moves as 16-byte vectors.
bool walks_vec(const WalkArgs &a, int es) {
    for (int i = 0; i < a.walks; ++i)
        if (!view_vec(a.w[i].X, a.w[i].d1, es) || !view_vec(a.w[i].Y, a.w[i].d1, es) || !view_vec(a.w[i].Z, a.w[i].d2, es))
            return false;
    return true;
}

template <typename T, int D1, int C, bool VEC>
void walk_launch(const WalkArgs &a, hipStream_t s) {
    const int64_t pairs = (a.B * a.H + 7) / 8 * 8 * a.walks * a.nblk;
    if (a.segs > 1) {
        walk::walk_kernel<T, D1, C, VEC, walk::Part::State><<<(unsigned)(pairs * (a.segs - 1)), walk::kThreads, 0, s>>>(a);
        const int64_t tiles = (int64_t)a.walks * a.B * a.H * a.nblk * 4 * (D1 / 16);
        walk::join_kernel<D1><<<(unsigned)tiles, walk::kThreads, 0, s>>>(a);
    }
    walk::walk_kernel<T, D1, C, VEC, walk::Part::Whole><<<(unsigned)(pairs * a.segs), walk::kThreads, 0, s>>>(a);
}

template <typename T, int C, bool VEC>
void walk_width_launch(const WalkArgs &a, int d1, hipStream_t s) {
    switch (d1) {
        case 32: walk_launch<T, 32, C, VEC>(a, s); break;
        case 64: walk_launch<T, 64, C, VEC>(a, s); break;
        case 96: walk_launch<T, 96, C, VEC>(a, s); break;
        case 128: walk_launch<T, 128, C, VEC>(a, s); break;
        default: walk_launch<T, 256, C, VEC>(a, s); break;
    }
}

template <typename T, int C>
void walk_vec_launch(const WalkArgs &a, int d1, hipStream_t s) {
    if (walks_vec(a, sizeof(T))) walk_width_launch<T, C, true>(a, d1, s);
    else walk_width_launch<T, C, false>(a, d1, s);
}

template <typename T>
hipError_t run_walks(WalkArgs &a, const WalkPlan &w, const Ws &ws, hipStream_t s) {
    a.walks = w.walks;
    a.nblk = w.nblk;
    a.segs = w.segs;
    a.seg_len = w.seg_len;
    a.seg_state = reinterpret_cast<float *>(ws.p + kScratchOffset);
    for (int i = 0; i < a.walks; ++i)
        a.w[i].out4 = a.w[i].d2 % 4 == 0 && aligned_to(a.w[i].out, 4 * sizeof(T));
    if constexpr (sizeof(T) == 2) {
        if (w.chunk == 64) {
            walk_vec_launch<T, 64>(a, w.d1, s);
            return hipGetLastError();
        }
    }
    walk_vec_launch<T, 32>(a, w.d1, s);
    return hipGetLastError();
}

// ---------------------------------------------------------------- single token
//   S' = e^g S + k^T v,  o = scale q S'
// Reads and writes the state once and is bound by that.  One workgroup a
// (batch row, head): threads are columns (V of them each) by rows, eight rows'
// loads in flight a thread, the rows' partial products with q meet in shared
// memory.  B=128, H=16, 128x128: 53.8 us, 270 MB at 5.0 TB/s (a copy's rate);
// B=1: 5.4 us, where 16 workgroups wait for one round trip to memory.
struct StepArgs {
    int64_t BH, H;
    int dk, dv, lanes;  // lanes (a power of two) threads over the columns
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

size_t linattn_ws(const LinattnArgs &p, bool backward) { return kScratchOffset + walk_plan(p, backward).bytes; }

hipError_t linattn_forward(const LinattnArgs &p, const Ws &ws, hipStream_t s) {
    WalkArgs a{};
    a.walks = 1;
    a.B = p.B;
    a.L = p.L;
    a.H = p.H;
    a.log_decay = p.log_decay;
    const WalkView q{p.q, p.st[0][0], p.st[0][1], p.st[0][2]}, k{p.k, p.st[1][0], p.st[1][1], p.st[1][2]},
        v{p.v, p.st[2][0], p.st[2][1], p.st[2][2]};
    a.w[0] = {q, k, v, p.o, p.state, p.out_state, p.dv, 1, p.dk, p.dv, 0, 0, p.scale, p.scale, 1.0f, 0};
    const WalkPlan w = walk_plan(p, false);
    return p.bf16 ? run_walks<bf16>(a, w, ws, s) : run_walks<float>(a, w, ws, s);
}

hipError_t linattn_backward(const LinattnArgs &p, const Ws &ws, hipStream_t s) {
    WalkArgs a{};
    a.walks = 3;
    a.B = p.B;
    a.L = p.L;
    a.H = p.H;
    a.log_decay = p.log_decay;
    const WalkView q{p.q, p.st[0][0], p.st[0][1], p.st[0][2]}, k{p.k, p.st[1][0], p.st[1][1], p.st[1][2]},
        v{p.v, p.st[2][0], p.st[2][1], p.st[2][2]}, g{p.grad_o, p.st[3][0], p.st[3][1], p.st[3][2]};
    a.w[0] = {g, v, k, p.grad_q, p.state, nullptr, 1, p.dv, p.dv, p.dk, 0, 0, p.scale, p.scale, 1.0f, 0};
    a.w[1] = {v, g, q, p.grad_k, p.grad_out_state, nullptr, 1, p.dv, p.dv, p.dk, 1, 1, p.scale, 1.0f, p.scale, 0};
    a.w[2] = {k, q, g, p.grad_v, p.grad_out_state, p.grad_state, p.dv, 1, p.dk, p.dv, 1, 1, p.scale, 1.0f, p.scale, 0};
    const WalkPlan w = walk_plan(p, true);
    return p.bf16 ? run_walks<bf16>(a, w, ws, s) : run_walks<float>(a, w, ws, s);
}

hipError_t linattn_step(const LinattnArgs &p, hipStream_t s) {
    const bool al = p.dv % 4 == 0 && aligned16(p.state) && aligned16(p.out_state);
    const int cols = al ? p.dv / 4 : p.dv;
    int lanes = 1;
    while (lanes < cols) lanes *= 2;
    const StepArgs a{p.B * p.H, p.H, p.dk, p.dv, lanes, p.q, p.k, p.v,
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
