// headnorm.hip -- norms of queries and keys for each head, with the position
// rotation in the same pass, and their gradients.
//
//   r = 1 / sqrt(m(x^2) + eps),  m the mean (RMS) or the sum (unit length),
//   n = x r w,  y = n with its first R elements turned in pairs (c, c'):
//   y_c = n_c cos - n_c' sin,  y_c' = n_c' cos + n_c sin.
// Backward, with the rotation undone on the gradient first (g = Rot^T dy):
//   dw = sum over rows of g x r,  dx = r (g w - x r m(g w x r)).
//
// Bound by memory: a row is read once (its partner elements again, from the
// first-level cache) and written once.  A head's row is 16 lanes wide, so a
// wave has four rows on their way and row sums stay on the vector unit; a group
// of 16 lanes takes several heads of one position in turn, which share the
// cosines and sines it has loaded.  B=8, L=2048, 16 + 16 heads of 128, bf16, full
// rotation: 55 us forward (274 MB, 5.0 TB/s, a large copy's rate), 94 backward (408
// MB, 4.3 TB/s, 5 us of it the weights' sums).
#include "mixer.hpp"
#include "rows.hpp"

namespace prn {

namespace {

constexpr int kThreads = 256, kLanes = 16, kGroups = kThreads / kLanes;

struct Params {
    HeadnormArgs a;
    int64_t tokens;
    int heads;     // heads a group takes in turn
    int parts[2];  // groups a token's heads need: queries, keys
    float *part;   // [gridDim.x][2][d] partial dw, or null
};

// The elements c = (lane + 16 j) V + i of a row.
template <int V>
__device__ __forceinline__ int column(int lane, int j) { return (lane + kLanes * j) * V; }

// How a launch rotates: not at all, (i, i + R/2), (2i, 2i + 1), or whichever the
// arguments say (single elements).  Kernels of their own need a third of the
// registers less: 72 -> 56 us forward and 123 -> 94 backward at the size above.
enum Turned { kNone, kHalves, kPairs, kAny };
template <int M>
__device__ __forceinline__ bool pairs(const HeadnormArgs &a) { return M == kAny ? a.interleaved != 0 : M == kPairs; }
template <int M>
__device__ __forceinline__ bool turned(const HeadnormArgs &a, int c) { return M != kNone && c < a.R; }

// Where the rotation's partner of the V elements from c on begins.
template <int M>
__device__ __forceinline__ int partner(const HeadnormArgs &a, int c) {
    if (pairs<M>(a)) return c ^ 1;
    return c < a.R / 2 ? c + a.R / 2 : c - a.R / 2;
}

template <typename T, int V>
__device__ __forceinline__ VecT<T, V> load_row(const T *p) { return *reinterpret_cast<const VecT<T, V> *>(p); }

// Sixteen bytes of floats at a time where a group's elements are consecutive.
template <int V>
__device__ __forceinline__ void load_floats(const float *p, float (&f)[V]) {
    if constexpr (V % 4 == 0) {
        typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const f32x4_any x = *reinterpret_cast<const f32x4_any *>(p + i);
#pragma unroll
            for (int k = 0; k < 4; ++k) f[i + k] = x[k];
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = p[i];
    }
}

// A group's share of the rotation: the cosine and the signed sine of each of
// its elements (y_c = n_c cos + n_partner sin; back: the angle's opposite), one
// and zero where there is none.
template <int V, int NV, int M>
struct Turn {
    float cos[NV][V], sin[NV][V];

    __device__ __forceinline__ void load(const HeadnormArgs &a, int64_t token, int64_t t, int lane, bool back) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                cos[j][i] = 1.0f;
                sin[j][i] = 0.0f;
            }
        if (M == kNone || a.R == 0) return;
        int64_t pos;
        if (a.positions == nullptr) pos = t;
        else pos = a.wide ? static_cast<const int64_t *>(a.positions)[token] : (int64_t) static_cast<const int32_t *>(a.positions)[token];
        const bool in = pos >= 0 && pos < a.P;
        const float *row = a.table + (in ? pos : 0) * a.R;
        const float nan = __builtin_nanf("");
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = column<V>(lane, j);
            if (c >= a.R) continue;
            if (V > 1 && !pairs<M>(a)) {  // all of them on one side
                const int k = c >= a.R / 2 ? c - a.R / 2 : c;
                load_floats<V>(row + k, cos[j]);
                load_floats<V>(row + a.R / 2 + k, sin[j]);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (c + i < a.R) {
                        const int k = pairs<M>(a) ? (c + i) >> 1 : c >= a.R / 2 ? c - a.R / 2 : c;
                        cos[j][i] = row[k];
                        sin[j][i] = row[a.R / 2 + k];
                    }
            }
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (c + i < a.R) {
                    const bool second = pairs<M>(a) ? (c + i) & 1 : c >= a.R / 2;
                    if (second == back) sin[j][i] = -sin[j][i];
                    if (!in) cos[j][i] = sin[j][i] = nan;
                }
        }
    }
};

// Partners of a row's elements in it (interleaved vectors hold their own; past
// the rotated ones any finite value does: the elements themselves).
template <typename T, int V, int M>
__device__ __forceinline__ void load_partner(const HeadnormArgs &a, const T *row, int c, const VecT<T, V> &own, VecT<T, V> &to) {
    if (M == kNone) return;
    if (V > 1 && pairs<M>(a)) {
#pragma unroll
        for (int i = 0; i < V; ++i) to.v[i] = own.v[i ^ 1];
    } else {
        to = load_row<T, V>(row + (c < a.R ? partner<M>(a, c) : c));
    }
}

struct Item {
    int64_t token;
    int which, head, heads;  // queries or keys, the first head, how many
};
__device__ __forceinline__ Item item_of(const Params &p, int64_t n) {
    const uint32_t per = (uint32_t)(p.parts[0] + p.parts[1]);
    const uint32_t token = (uint32_t)n / per, part = (uint32_t)n - token * per;
    Item it;
    it.token = token;
    it.which = part >= (uint32_t)p.parts[0];
    const int H = (int)(it.which ? p.a.Hk : p.a.Hq);
    it.head = (int)(part - (it.which ? p.parts[0] : 0)) * p.heads;
    it.heads = min(p.heads, H - it.head);
    return it;
}
template <typename T>
__device__ __forceinline__ const T *row_of(const HeadView &v, int64_t b, int64_t t, int head) {
    return static_cast<const T *>(v.p) + b * v.st[0] + t * v.st[1] + head * v.st[2];
}

// Rows of a group that are on their way at once.
template <int V, int NV> constexpr int kAhead = V > 1 && NV == 1 ? 2 : 1;

template <typename T, int V, int NV, int M>
__global__ __launch_bounds__(kThreads) void headnorm_fwd_kernel(Params p) {
    constexpr int U = kAhead<V, NV>;
    const HeadnormArgs &a = p.a;
    const int lane = threadIdx.x & (kLanes - 1);
    const int64_t items = p.tokens * (p.parts[0] + p.parts[1]);
    const int64_t n = (int64_t)blockIdx.x * kGroups + threadIdx.x / kLanes;
    if (n >= items) return;
    const Item it = item_of(p, n);
    const int64_t b = (uint32_t)it.token / (uint32_t)a.L, t = it.token - b * a.L;
    const int64_t H = it.which ? a.Hk : a.Hq;
    const float *wp = it.which ? a.w[1] : a.w[0];
    const HeadView x = it.which ? a.x[1] : a.x[0];
    const T *first = row_of<T>(x, b, t, it.head);
    float *r_out = it.which ? a.r[1] : a.r[0];
    T *y = static_cast<T *>(it.which ? a.y[1] : a.y[0]) + (it.token * H + it.head) * a.d;
    VecT<T, V> own[U][NV], other[U][NV];
    auto load = [&](int h0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const T *row = first + min(h0 + u, it.heads - 1) * x.st[2];
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = column<V>(lane, j);
                if (c < a.d) {
                    own[u][j] = load_row<T, V>(row + c);
                    load_partner<T, V, M>(a, row, c, own[u][j], other[u][j]);
                }
            }
        }
    };
    // y = r (x (w cos) + x_partner (w_partner sin))
    Turn<V, NV, M> turn;
    turn.load(a, it.token, t, lane, false);
    if (wp != nullptr) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = column<V>(lane, j);
            if (c >= a.d) continue;
            float w[V], wo[V];
            load_floats<V>(wp + c, w);
            if (V > 1 && pairs<M>(a)) {
#pragma unroll
                for (int i = 0; i < V; ++i) wo[i] = w[i ^ 1];
            } else {
                load_floats<V>(wp + (turned<M>(a, c) ? partner<M>(a, c) : c), wo);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                turn.cos[j][i] *= w[i];
                turn.sin[j][i] *= wo[i];
            }
        }
    }
    for (int h0 = 0; h0 < it.heads; h0 += U) {
        load(h0);
        float f[U][NV][V], o[U][NV][V], sum[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            sum[u] = 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const bool in = column<V>(lane, j) < a.d;
                    f[u][j][i] = in ? (float)own[u][j].v[i] : 0.0f;
                    o[u][j][i] = in && M != kNone ? (float)other[u][j].v[i] : 0.0f;
                    sum[u] = fmaf(f[u][j][i], f[u][j][i], sum[u]);
                }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float s = lanes16_sum(sum[u]);
            const float r = 1.0f / sqrtf((a.l2 ? s : s / (float)a.d) + a.eps);
            if (h0 + u >= it.heads) continue;
            if (lane == 0 && r_out != nullptr) r_out[it.token * H + it.head + h0 + u] = r;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = column<V>(lane, j);
                if (c < a.d) {
                    float v[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        // an infinity beside a zero sine is no number of this element's
                        const float n = f[u][j][i] * turn.cos[j][i];
                        v[i] = r * (turned<M>(a, c + i) ? fmaf(o[u][j][i], turn.sin[j][i], n) : n);
                    }
                    store_vec<T, V>(y + (int64_t)(h0 + u) * a.d + c, v);
                }
            }
        }
    }
}

// A launch's groups are a multiple of a token's parts, so that a group has the
// same heads of every token it comes to: one weight and one sum of gradients.
// (At the 128 registers of four waves a SIMD the rotated forms of eight elements a
// lane spill 12 to 44 bytes, single elements of d above 64 116.)
template <typename T, int V, int NV, int M>
__global__ __launch_bounds__(kThreads, NV * V <= 8 ? 4 : 2) void headnorm_bwd_kernel(Params p) {
    constexpr int U = 1;
    const HeadnormArgs &a = p.a;
    const int lane = threadIdx.x & (kLanes - 1), grp = threadIdx.x / kLanes;
    const int64_t items = p.tokens * (p.parts[0] + p.parts[1]), first_item = (int64_t)blockIdx.x * kGroups + grp;
    const Item mine = item_of(p, first_item);
    const int which = mine.which;
    const int64_t H = which ? a.Hk : a.Hq;
    const float *wp = which ? a.w[1] : a.w[0];
    const HeadView x = which ? a.x[1] : a.x[0], g = which ? a.g[1] : a.g[0];
    float w[NV][V], acc[NV][V] = {};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < V; ++i) w[j][i] = 1.0f;
        if (wp != nullptr && column<V>(lane, j) < a.d) load_floats<V>(wp + column<V>(lane, j), w[j]);
    }
    for (int64_t n = first_item; n < items; n += (int64_t)gridDim.x * kGroups) {
        const Item it = item_of(p, n);
        const int64_t b = (uint32_t)it.token / (uint32_t)a.L, t = it.token - b * a.L;
        const T *first = row_of<T>(x, b, t, mine.head), *gfirst = row_of<T>(g, b, t, mine.head);
        const float *r_in = (which ? a.r[1] : a.r[0]) + it.token * H + mine.head;
        T *out = static_cast<T *>(which ? a.y[1] : a.y[0]) + (it.token * H + mine.head) * a.d;
        Turn<V, NV, M> turn;
        turn.load(a, it.token, t, lane, true);
#pragma unroll 1
        for (int h0 = 0; h0 < mine.heads; h0 += U) {
            VecT<T, V> own[U][NV], dy[U][NV], other[U][NV];
            float r[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = min(h0 + u, mine.heads - 1);
                const T *row = first + h * x.st[2], *grow = gfirst + h * g.st[2];
                r[u] = r_in[h];
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int c = column<V>(lane, j);
                    if (c < a.d) {
                        own[u][j] = load_row<T, V>(row + c);
                        dy[u][j] = load_row<T, V>(grow + c);
                        load_partner<T, V, M>(a, grow, c, dy[u][j], other[u][j]);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (h0 + u >= mine.heads) continue;
                float xh[NV][V], v[NV][V], sum = 0.0f;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int c = column<V>(lane, j);
                    if (c < a.d)
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            xh[j][i] = (float)own[u][j].v[i] * r[u];
                            float gn = (float)dy[u][j].v[i] * turn.cos[j][i];
                            if (turned<M>(a, c + i)) gn = fmaf((float)other[u][j].v[i], turn.sin[j][i], gn);
                            acc[j][i] = fmaf(gn, xh[j][i], acc[j][i]);
                            v[j][i] = gn * w[j][i];
                            sum = fmaf(v[j][i], xh[j][i], sum);
                        }
                }
                sum = lanes16_sum(sum);
                if (!a.l2) sum /= (float)a.d;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int c = column<V>(lane, j);
                    if (c < a.d) {
#pragma unroll
                        for (int i = 0; i < V; ++i) v[j][i] = r[u] * (v[j][i] - xh[j][i] * sum);
                        store_vec<T, V>(out + (int64_t)(h0 + u) * a.d + c, v[j]);
                    }
                }
            }
        }
    }
    if (p.part == nullptr) return;
    // the sums of the groups of either tensor, in their order
    __shared__ float buf[kGroups][kLanes * V];
    __shared__ int whose[kGroups];
    if (lane == 0) whose[grp] = which;
    float *part = p.part + (int64_t)blockIdx.x * 2 * a.d;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) buf[grp][lane * V + i] = acc[j][i];
        __syncthreads();
        for (int k = threadIdx.x; k < 2 * kLanes * V; k += kThreads) {
            const int of = k >= kLanes * V, at = k - of * kLanes * V, c = kLanes * V * j + at;
            float sum = 0.0f;
#pragma unroll
            for (int m = 0; m < kGroups; ++m)
                if (whose[m] == of) sum += buf[m][at];
            if (c < a.d) part[of * a.d + c] = sum;
        }
    }
}

// dw = sum of the G partials, always in the same order: 64 columns a workgroup, 16 threads a column.
__global__ __launch_bounds__(1024) void headnorm_reduce_kernel(const float *part, int G, int d, float *gq, float *gk) {
    __shared__ float buf[16][64];
    const int lane = threadIdx.x & 63, grp = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane;
    float *out = blockIdx.y == 0 ? gq : gk;
    if (out == nullptr) return;
    float v = 0.0f;
    if (c < d) {
#pragma unroll 8
        for (int g = grp; g < G; g += 16) v += part[((int64_t)g * 2 + blockIdx.y) * d + c];
    }
    buf[grp][lane] = v;
    __syncthreads();
    if (grp == 0 && c < d) {
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) v += buf[i][lane];
        out[c] = v;
    }
}

bool view_vec(const HeadView &v, int n) {
    return aligned16(v.p) && v.st[0] % n == 0 && v.st[1] % n == 0 && v.st[2] % n == 0;
}

// Whether every row moves as 16-byte vectors whose rotation partners are one too.
bool rows_vec(const HeadnormArgs &a, int es, bool back) {
    const int n = 16 / es;
    if (a.d % n != 0 || (!a.interleaved && a.R / 2 % n != 0)) return false;
    for (int i = 0; i < (a.Hk ? 2 : 1); ++i)
        if (!view_vec(a.x[i], n) || !aligned16(a.y[i]) || (back && !view_vec(a.g[i], n))) return false;
    return true;
}

// Heads a group takes in turn: as many as leave four waves a SIMD, 8 at the most.
// At the size above 56 and 94 us, with one head each 126 and 159.
Params params(const HeadnormArgs &a) {
    Params p{};
    p.a = a;
    p.tokens = a.B * a.L;
    const int64_t rows = p.tokens * (a.Hq + a.Hk), want = (int64_t)device_cu_count() * kGroups * 4;
    p.heads = (int)std::max<int64_t>(1, std::min<int64_t>(8, rows / want));
    p.parts[0] = (int)((a.Hq + p.heads - 1) / p.heads);
    p.parts[1] = (int)((a.Hk + p.heads - 1) / p.heads);
    return p;
}

int64_t groups(const Params &p) { return (p.tokens * (p.parts[0] + p.parts[1]) + kGroups - 1) / kGroups; }

// Workgroups of the backward pass, which keep the weights' gradients in
// registers over all their rows: a multiple of a token's parts where there are
// more items than groups.
int bwd_grid(const Params &p) {
    const int64_t parts = p.parts[0] + p.parts[1], cap = std::max<int64_t>((int64_t)device_cu_count() * 4, parts);
    const int64_t n = groups(p);
    return (int)(n <= cap ? n : cap / parts * parts);
}

template <typename T, int V, int NV, int M>
hipError_t launch(const Params &p, bool back, hipStream_t s) {
    if (back) headnorm_bwd_kernel<T, V, NV, M><<<bwd_grid(p), kThreads, 0, s>>>(p);
    else headnorm_fwd_kernel<T, V, NV, M><<<(unsigned)groups(p), kThreads, 0, s>>>(p);
    return hipGetLastError();
}

template <typename T, int NV>
hipError_t launch_vec(const Params &p, bool back, hipStream_t s) {
    constexpr int V = kVec<T>;
    if (p.a.R == 0) return launch<T, V, NV, kNone>(p, back, s);
    return p.a.interleaved ? launch<T, V, NV, kPairs>(p, back, s) : launch<T, V, NV, kHalves>(p, back, s);
}

template <typename T>
hipError_t run(const Params &p, bool back, hipStream_t s) {
    const int d = p.a.d;
    if (rows_vec(p.a, sizeof(T), back)) {
        constexpr int V = kVec<T>;
        if (d <= kLanes * V) return launch_vec<T, 1>(p, back, s);
        if (d <= kLanes * V * 2) return launch_vec<T, 2>(p, back, s);
        if constexpr (V == 4) return launch_vec<T, 4>(p, back, s);
    }
    if (d <= kLanes * 4) return launch<T, 1, 4, kAny>(p, back, s);
    if (d <= kLanes * 8) return launch<T, 1, 8, kAny>(p, back, s);
    return launch<T, 1, 16, kAny>(p, back, s);
}

}  // namespace

size_t headnorm_ws(const HeadnormArgs &a) {
    return kScratchOffset + (size_t)bwd_grid(params(a)) * 2 * a.d * sizeof(float);
}

hipError_t headnorm_forward(const HeadnormArgs &a, hipStream_t s) {
    const Params p = params(a);
    return a.bf16 ? run<bf16>(p, false, s) : run<float>(p, false, s);
}

hipError_t headnorm_backward(const HeadnormArgs &a, const Ws &ws, hipStream_t s) {
    Params p = params(a);
    const bool want = a.gw[0] != nullptr || a.gw[1] != nullptr;
    if (want) p.part = reinterpret_cast<float *>(ws.p + kScratchOffset);
    const hipError_t e = a.bf16 ? run<bf16>(p, true, s) : run<float>(p, true, s);
    if (e != hipSuccess || !want) return e;
    headnorm_reduce_kernel<<<dim3((a.d + 63) / 64, 2), 1024, 0, s>>>(p.part, bwd_grid(p), a.d, a.gw[0], a.gw[1]);
    return hipGetLastError();
}

}  // namespace prn
