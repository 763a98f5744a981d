// layernorm.hip -- layer norm over the last dimension of [rows, D], with the
// residual sum before it, and its backward pass.
//
//   s = x + r (rounded to the tensors' type),  mu = sum s / D,
//   v = sum (s - mu)^2 / D,  rstd = 1 / sqrt(v + eps),
//   xh = (s - mu) rstd,  y = xh w + b.
//   g = dy w,  dx = rstd (g - mean(g) - xh mean(g xh)) + ds,
//   dw = sum over rows of dy xh,  db = sum over rows of dy.
//
// Both passes are bound by memory: a few operations per element against 2 to
// 4 tensors moved.  A row therefore stays in registers from its one load to
// its store (E elements a thread, in vectors of V), so the centred second
// pass of the variance costs no traffic.  R threads share a row: 16 lanes for
// rows up to 128 elements, a wave up to 1024 (no barrier), the workgroup
// above.  All statistics and sums are fp32.
//
// Measured: forward with residual, 32768x1024 fp32, 98 us (537 MB, 5.5 TB/s);
// backward with a gradient of the sum, dw and db, 8192x4096 bf16, 49 + 5 us
// (268 MB, 5.5 TB/s in the first); a copy of 1 GiB runs at 5.1 TB/s.  Rows that
// are not whole 16-byte vectors move an element at a time: 20000x1283 fp32
// forward and backward 107 and 130 us (3.8, 3.2 TB/s), bf16 90 and 130 us (2.3,
// 1.6); groups put together from whole words were no better here (one set of
// tensors, in part from the caches: fp32 99 and 80 us where elements took 83 and
// 90, bf16 64 and 89 where they took 60 and 80), as that work sits between a
// row's loads and the next's.  Rows above 8192 elements are read several times
// by one workgroup each: 4096x16384 fp32 forward 339, backward 451 us (3.2, 2.4
// TB/s of its least traffic).
#include "rows.hpp"
#include "sequence.hpp"

namespace prn {

namespace {

constexpr int kThreads = 256;

// Sums over the R threads that share a row: 16 lanes, a wave, or the
// workgroup, where buf holds a pair a wave and alternates between calls
// (`half`) so that one barrier a call is enough.
template <int R>
__device__ __forceinline__ float2 row_sums(float a, float b, float2 (&buf)[2][4], int half) {
    if (R == 16) return make_float2(lanes16_sum(a), lanes16_sum(b));
    a = lanes_sum(a);
    b = lanes_sum(b);
    if (R == 64) return make_float2(a, b);
    if ((threadIdx.x & 63) == 0) buf[half][threadIdx.x >> 6] = make_float2(a, b);
    __syncthreads();
    const float2 p = buf[half][0], q = buf[half][1], r = buf[half][2], t = buf[half][3];
    return make_float2((p.x + q.x) + (r.x + t.x), (p.y + q.y) + (r.y + t.y));
}
template <int R>
__device__ __forceinline__ float row_sum(float v, float2 (&buf)[2][4], int half) {
    return row_sums<R>(v, 0.0f, buf, half).x;
}

struct LnFwdArgs {
    int64_t rows;
    int D;
    const void *x, *res;
    const float *w, *b;
    float eps;
    void *s, *y;
    float *mean, *rstd;
};

// A workgroup keeps its columns' weight and bias in registers over its rows
// and loads a row ahead (32768x1024 fp32 with residual: 98 us, 109 with one
// row a wave and the weights read again for each; 20000x1283, one set of tensors
// in part from the caches: 86 us, 171).
template <typename T, int V, int R, int E>
__global__ __launch_bounds__(kThreads) void ln_fwd_kernel(LnFwdArgs a) {
    constexpr int NV = E / V, kRows = kThreads / R;
    __shared__ float2 buf[2][4];
    const int li = threadIdx.x & (R - 1);
    const int64_t step = (int64_t)gridDim.x * kRows;
    const float n = (float)a.D;
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.res);
    float w[NV][V], b[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (li + j * R) * V + i;
            w[j][i] = c < a.D && a.w != nullptr ? a.w[c] : 1.0f;
            b[j][i] = c < a.D && a.b != nullptr ? a.b[c] : 0.0f;
        }
    struct Row {
        VecT<T, V> x[NV], res[NV];
    };
    Row next;
    auto load = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (li + j * R) * V;
            if (c < a.D) {
                next.x[j] = load_once<T, V>(x + row * a.D + c);
                if (res != nullptr) next.res[j] = load_once<T, V>(res + row * a.D + c);
            }
        }
    };
    int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / R;
    if (row < a.rows) load(row);
    for (; row < a.rows; row += step) {
        const int64_t base = row * a.D;
        const Row cur = next;
        if (row + step < a.rows) load(row + step);
        float f[NV][V];
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (li + j * R) * V;
#pragma unroll
            for (int i = 0; i < V; ++i) f[j][i] = 0.0f;
            if (c < a.D) {
#pragma unroll
                for (int i = 0; i < V; ++i) f[j][i] = (float)cur.x[j].v[i];
                if (res != nullptr) {
#pragma unroll
                    for (int i = 0; i < V; ++i) f[j][i] = (float)(T)(f[j][i] + (float)cur.res[j].v[i]);
                    store_vec<T, V>(static_cast<T *>(a.s) + base + c, f[j]);
                }
            }
#pragma unroll
            for (int i = 0; i < V; ++i) sum += f[j][i];
        }
        const float mu = row_sum<R>(sum, buf, 0) / n;
        float sq = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (li + j * R) * V;
            if (c < a.D) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    f[j][i] -= mu;
                    sq = fmaf(f[j][i], f[j][i], sq);
                }
            }
        }
        const float rstd = 1.0f / sqrtf(row_sum<R>(sq, buf, 1) / n + a.eps);
        if (li == 0) {
            if (a.mean != nullptr) a.mean[row] = mu;
            if (a.rstd != nullptr) a.rstd[row] = rstd;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (li + j * R) * V;
            if (c < a.D) {
#pragma unroll
                for (int i = 0; i < V; ++i) f[j][i] = fmaf(f[j][i] * rstd, w[j][i], b[j][i]);
                store_vec<T, V>(static_cast<T *>(a.y) + base + c, f[j]);
            }
        }
    }
}

// Rows too long for the registers (above 8192): one workgroup a row, read
// three times.
template <typename T>
__global__ __launch_bounds__(kThreads) void ln_fwd_long_kernel(LnFwdArgs a) {
    __shared__ float2 buf[2][4];
    const float n = (float)a.D;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t base = row * a.D;
        const T *x = static_cast<const T *>(a.x) + base;
        const T *r = a.res != nullptr ? static_cast<const T *>(a.res) + base : nullptr;
        T *s = static_cast<T *>(a.s) + base, *y = static_cast<T *>(a.y) + base;
        float sum = 0.0f;
        for (int c = threadIdx.x; c < a.D; c += kThreads) {
            float v = (float)x[c];
            if (r != nullptr) {
                v = (float)(T)(v + (float)r[c]);
                s[c] = (T)v;
            }
            sum += v;
        }
        const T *src = r != nullptr ? s : x;  // each thread reads back what it wrote itself
        const float mu = row_sum<256>(sum, buf, 0) / n;
        float sq = 0.0f;
        for (int c = threadIdx.x; c < a.D; c += kThreads) {
            const float d = (float)src[c] - mu;
            sq = fmaf(d, d, sq);
        }
        const float rstd = 1.0f / sqrtf(row_sum<256>(sq, buf, 1) / n + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean != nullptr) a.mean[row] = mu;
            if (a.rstd != nullptr) a.rstd[row] = rstd;
        }
        for (int c = threadIdx.x; c < a.D; c += kThreads) {
            const float w = a.w != nullptr ? a.w[c] : 1.0f, b = a.b != nullptr ? a.b[c] : 0.0f;
            y[c] = (T)fmaf(((float)src[c] - mu) * rstd, w, b);
        }
    }
}

struct LnBwdArgs {
    int64_t rows;
    int D;
    const void *s;
    const float *w, *mean, *rstd;
    const void *dy, *ds;
    void *dx;
    float *part;  // [gridDim.x][2][D] partial dw, db, or null
};

// The workgroups keep their columns' dw and db in registers over all their
// rows, so there are only as many partial sums as workgroups; the few waves
// that leaves on a CU keep memory busy by loading a row ahead.
template <typename T, int V, int R, int E>
__global__ __launch_bounds__(kThreads) void ln_bwd_kernel(LnBwdArgs a) {
    constexpr int NV = E / V, kRows = kThreads / R;
    __shared__ float2 buf[2][4];
    __shared__ float comb[kRows > 1 ? (kRows - 1) * R * V : 1];
    const int li = threadIdx.x & (R - 1);
    const int64_t step = (int64_t)gridDim.x * kRows;
    const float n = (float)a.D;
    const T *s = static_cast<const T *>(a.s), *dy = static_cast<const T *>(a.dy), *ds = static_cast<const T *>(a.ds);
    float w[NV][V], gw[NV][V], gb[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (li + j * R) * V + i;
            w[j][i] = c < a.D ? (a.w != nullptr ? a.w[c] : 1.0f) : 0.0f;
            gw[j][i] = gb[j][i] = 0.0f;
        }
    struct Row {
        VecT<T, V> s[NV], dy[NV], ds[NV];
        float mu, rstd;
    };
    Row next;
    auto load = [&](int64_t row) {
        next.mu = a.mean[row];
        next.rstd = a.rstd[row];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (li + j * R) * V;
            if (c < a.D) {
                const int64_t at = row * a.D + c;
                next.s[j] = load_once<T, V>(s + at);
                next.dy[j] = load_once<T, V>(dy + at);
                if (ds != nullptr) next.ds[j] = load_once<T, V>(ds + at);
            }
        }
    };
    int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / R;
    if (row < a.rows) load(row);
    for (int half = 0; row < a.rows; row += step, half ^= 1) {
        const Row cur = next;
        if (row + step < a.rows) load(row + step);
        float xh[NV][V], g[NV][V];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (li + j * R) * V;
            if (c < a.D) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float d = (float)cur.dy[j].v[i];
                    xh[j][i] = ((float)cur.s[j].v[i] - cur.mu) * cur.rstd;
                    gw[j][i] = fmaf(d, xh[j][i], gw[j][i]);
                    gb[j][i] += d;
                    g[j][i] = d * w[j][i];
                    s1 += g[j][i];
                    s2 = fmaf(g[j][i], xh[j][i], s2);
                }
            }
        }
        const float2 sums = row_sums<R>(s1, s2, buf, half);
        const float c1 = sums.x / n, c2 = sums.y / n;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (li + j * R) * V;
            if (c < a.D) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    g[j][i] = cur.rstd * (g[j][i] - fmaf(xh[j][i], c2, c1));
                    if (ds != nullptr) g[j][i] += (float)cur.ds[j].v[i];
                }
                store_vec<T, V>(static_cast<T *>(a.dx) + row * a.D + c, g[j]);
            }
        }
    }
    if (a.part == nullptr) return;
    float *part = a.part + (int64_t)blockIdx.x * 2 * a.D;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (li + j * R) * V;
            float v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = q == 0 ? gw[j][i] : gb[j][i];
            if (kRows > 1) {  // the sums of the rows side by side, in their order
                const int grp = threadIdx.x / R;
                __syncthreads();
                if (grp > 0)
#pragma unroll
                    for (int i = 0; i < V; ++i) comb[((grp - 1) * V + i) * R + li] = v[i];
                __syncthreads();
                if (grp == 0)
#pragma unroll
                    for (int g = 0; g < kRows - 1; ++g)
#pragma unroll
                        for (int i = 0; i < V; ++i) v[i] += comb[(g * V + i) * R + li];
            }
            if (c < a.D && threadIdx.x < R) {
#pragma unroll
                for (int i = 0; i < V; ++i) part[(int64_t)q * a.D + c + i] = v[i];
            }
        }
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void ln_bwd_long_kernel(LnBwdArgs a) {
    __shared__ float2 buf[2][4];
    const float n = (float)a.D;
    int half = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t base = row * a.D;
        const T *s = static_cast<const T *>(a.s) + base, *dy = static_cast<const T *>(a.dy) + base;
        const T *ds = a.ds != nullptr ? static_cast<const T *>(a.ds) + base : nullptr;
        T *dx = static_cast<T *>(a.dx) + base;
        const float mu = a.mean[row], rstd = a.rstd[row];
        float s1 = 0.0f, s2 = 0.0f;
        for (int c = threadIdx.x; c < a.D; c += kThreads) {
            const float g = (float)dy[c] * (a.w != nullptr ? a.w[c] : 1.0f);
            s1 += g;
            s2 = fmaf(g, ((float)s[c] - mu) * rstd, s2);
        }
        const float2 c = row_sums<256>(s1, s2, buf, half);
        const float c1 = c.x / n, c2 = c.y / n;
        half ^= 1;
        for (int c = threadIdx.x; c < a.D; c += kThreads) {
            const float g = (float)dy[c] * (a.w != nullptr ? a.w[c] : 1.0f);
            const float xh = ((float)s[c] - mu) * rstd;
            float v = rstd * (g - fmaf(xh, c2, c1));
            if (ds != nullptr) v += (float)ds[c];
            dx[c] = (T)v;
        }
    }
}

// Rows of a few elements: a lane a row, in double.  Their gradient is what is
// left of g after its mean and its part along xh are taken out, and of two
// elements only eps keeps anything: in fp32 that would be rounding error.
constexpr int kShortRow = 4;
template <typename T>
__global__ __launch_bounds__(kThreads) void ln_bwd_short_kernel(LnBwdArgs a) {
    float gw[kShortRow] = {}, gb[kShortRow] = {};
    for (int64_t row = (int64_t)blockIdx.x * kThreads + threadIdx.x; row < a.rows; row += (int64_t)gridDim.x * kThreads) {
        const int64_t base = row * a.D;
        const double mu = a.mean[row], rstd = a.rstd[row];
        double xh[kShortRow], g[kShortRow], s1 = 0.0, s2 = 0.0;
#pragma unroll
        for (int i = 0; i < kShortRow; ++i)
            if (i < a.D) {
                const float dy = (float)static_cast<const T *>(a.dy)[base + i];
                xh[i] = ((double)(float)static_cast<const T *>(a.s)[base + i] - mu) * rstd;
                gw[i] = fmaf(dy, (float)xh[i], gw[i]);
                gb[i] += dy;
                g[i] = (double)dy * (a.w != nullptr ? (double)a.w[i] : 1.0);
                s1 += g[i];
                s2 += g[i] * xh[i];
            }
        const double c1 = s1 / a.D, c2 = s2 / a.D;
#pragma unroll
        for (int i = 0; i < kShortRow; ++i)
            if (i < a.D) {
                double v = rstd * (g[i] - c1 - xh[i] * c2);
                if (a.ds != nullptr) v += (double)(float)static_cast<const T *>(a.ds)[base + i];
                static_cast<T *>(a.dx)[base + i] = (T)(float)v;
            }
    }
    if (a.part == nullptr) return;
    __shared__ float buf[4];
    float *part = a.part + (int64_t)blockIdx.x * 2 * a.D;
#pragma unroll
    for (int i = 0; i < 2 * kShortRow; ++i) {
        const int c = i >> 1;
        const float v = lanes_sum(i & 1 ? gb[c] : gw[c]);
        if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
        __syncthreads();
        if (threadIdx.x == 0 && c < a.D) part[(i & 1) * a.D + c] = (buf[0] + buf[1]) + (buf[2] + buf[3]);
        __syncthreads();
    }
}

// Partial dw, db of long rows: workgroup (x, y) adds the rows y, y + gridDim.y, ... of its 256 columns.
template <typename T>
__global__ __launch_bounds__(kThreads) void ln_bwd_cols_kernel(LnBwdArgs a) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= a.D) return;
    float gw = 0.0f, gb = 0.0f;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const float g = (float)static_cast<const T *>(a.dy)[row * a.D + c];
        const float xh = ((float)static_cast<const T *>(a.s)[row * a.D + c] - a.mean[row]) * a.rstd[row];
        gw = fmaf(g, xh, gw);
        gb += g;
    }
    float *part = a.part + (int64_t)blockIdx.y * 2 * a.D;
    part[c] = gw;
    part[a.D + c] = gb;
}

// dw, db = sum of the G partials, always in the same order: 64 columns a
// workgroup, 16 threads a column.
__global__ __launch_bounds__(1024) void ln_reduce_kernel(const float *part, int G, int D, float *gw, float *gb) {
    __shared__ float buf[16][64];
    const int lane = threadIdx.x & 63, grp = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane;
    float *out = blockIdx.y == 0 ? gw : gb;
    if (out == nullptr) return;
    float v = 0.0f;
    if (c < D) {
#pragma unroll 8
        for (int g = grp; g < G; g += 16) v += part[((int64_t)g * 2 + blockIdx.y) * D + c];
    }
    buf[grp][lane] = v;
    __syncthreads();
    if (grp == 0 && c < D) {
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) v += buf[i][lane];
        out[c] = v;
    }
}

// Rows up to kNarrow elements: 16 lanes each, four rows a wave (100000x64 fp32:
// forward with residual 21 us, backward 24; 37 and 51 with a wave a row, of
// which 16 lanes work; bf16 17 and 20, 42 and 51 so; 32768x128 fp32 14 and 16,
// 17 and 23 so; one set of tensors).
constexpr int64_t kNarrow = 128;
// Rows that a workgroup takes at once.
int64_t rows_at_once(int64_t D) { return D <= kNarrow ? 16 : D <= 1024 ? 4 : 1; }

template <typename T, int V>
void ln_fwd_launch(const LnFwdArgs &a, hipStream_t s) {
    const int64_t cap = (int64_t)device_cu_count() * 4;
    const int g = (int)std::min<int64_t>((a.rows + rows_at_once(a.D) - 1) / rows_at_once(a.D), cap);
    if (a.D <= kNarrow) ln_fwd_kernel<T, V, 16, 8><<<g, kThreads, 0, s>>>(a);
    else if (a.D <= 512) ln_fwd_kernel<T, V, 64, 8><<<g, kThreads, 0, s>>>(a);
    else if (a.D <= 1024) ln_fwd_kernel<T, V, 64, 16><<<g, kThreads, 0, s>>>(a);
    else if (a.D <= 4096) ln_fwd_kernel<T, V, 256, 16><<<g, kThreads, 0, s>>>(a);
    else ln_fwd_kernel<T, V, 256, 32><<<g, kThreads, 0, s>>>(a);
}

template <typename T, int V>
void ln_bwd_launch(const LnBwdArgs &a, int G, hipStream_t s) {
    if (a.D <= kNarrow) ln_bwd_kernel<T, V, 16, 8><<<G, kThreads, 0, s>>>(a);
    else if (a.D <= 512) ln_bwd_kernel<T, V, 64, 8><<<G, kThreads, 0, s>>>(a);
    else if (a.D <= 1024) ln_bwd_kernel<T, V, 64, 16><<<G, kThreads, 0, s>>>(a);
    else if (a.D <= 4096) ln_bwd_kernel<T, V, 256, 16><<<G, kThreads, 0, s>>>(a);
    else ln_bwd_kernel<T, V, 256, 32><<<G, kThreads, 0, s>>>(a);
}

constexpr int64_t kLongRow = 8192;  // above it a row does not fit the registers

template <typename T>
hipError_t ln_fwd(const LnFwdArgs &a, hipStream_t s) {
    const bool vec = a.D % kVec<T> == 0 && aligned16(a.x) && aligned16(a.y) &&
                     (a.res == nullptr || (aligned16(a.res) && aligned16(a.s)));
    if (a.D > kLongRow)
        ln_fwd_long_kernel<T><<<(int)std::min<int64_t>(a.rows, (int64_t)device_cu_count() * 8), kThreads, 0, s>>>(a);
    else if (vec) ln_fwd_launch<T, kVec<T>>(a, s);
    else ln_fwd_launch<T, 1>(a, s);
    return hipGetLastError();
}

template <typename T>
hipError_t ln_bwd(const LnBwdArgs &a, int G, float *gw, float *gb, hipStream_t s) {
    const bool vec = a.D % kVec<T> == 0 && aligned16(a.s) && aligned16(a.dy) && aligned16(a.dx) &&
                     (a.ds == nullptr || aligned16(a.ds));
    if (a.D > kLongRow) {
        if (a.part != nullptr)  // first: it reads what grad_x may overwrite
            ln_bwd_cols_kernel<T><<<dim3((a.D + kThreads - 1) / kThreads, G), kThreads, 0, s>>>(a);
        ln_bwd_long_kernel<T><<<(int)std::min<int64_t>(a.rows, (int64_t)device_cu_count() * 8), kThreads, 0, s>>>(a);
    } else if (a.D <= kShortRow) ln_bwd_short_kernel<T><<<G, kThreads, 0, s>>>(a);
    else if (vec) ln_bwd_launch<T, kVec<T>>(a, G, s);
    else ln_bwd_launch<T, 1>(a, G, s);
    if (a.part != nullptr)
        ln_reduce_kernel<<<dim3((a.D + 63) / 64, 2), 1024, 0, s>>>(a.part, G, a.D, gw, gb);
    return hipGetLastError();
}

}  // namespace

// Partials of the weight's gradient: one workgroup's rows each.
int layernorm_parts(int64_t rows, int64_t D) {
    const int64_t per = D <= kShortRow ? kThreads : rows_at_once(D);
    const int64_t cap = D > kLongRow ? 64 : (int64_t)device_cu_count() * 2;
    return (int)std::min<int64_t>((rows + per - 1) / per, cap);
}

hipError_t layernorm_forward(const LayernormFwdArgs &q, hipStream_t s) {
    const LnFwdArgs a{q.rows, (int)q.D, q.x, q.residual, q.weight, q.bias, q.eps, q.sum, q.y, q.mean, q.rstd};
    return q.bf16 ? ln_fwd<bf16>(a, s) : ln_fwd<float>(a, s);
}

hipError_t layernorm_backward(const LayernormBwdArgs &q, const Ws &ws, hipStream_t s) {
    const bool want = q.grad_w != nullptr || q.grad_b != nullptr;
    const LnBwdArgs a{q.rows, (int)q.D, q.s, q.weight, q.mean, q.rstd, q.grad_y, q.grad_sum, q.grad_x,
                      want ? reinterpret_cast<float *>(ws.p + kScratchOffset) : nullptr};
    const int G = layernorm_parts(q.rows, q.D);
    return q.bf16 ? ln_bwd<bf16>(a, G, q.grad_w, q.grad_b, s) : ln_bwd<float>(a, G, q.grad_w, q.grad_b, s);
}

}  // namespace prn
