// embedding.hip -- embedding lookup with scaling, and its gradient by sorted
// tokens.
//
//   out[n] = scale table[ids[n]]
//   dtable[r] = scale * sum over n with ids[n] = r, in ascending n, of grad[n]
//
// The lookup is a gather of whole rows, bound by memory: 32768 rows of
// 50000x1024 bf16 in 18.5 us, 134 MB at 7.3 TB/s, as frequent rows come from
// the caches.  The gradient sorts
// the (id, position) pairs by a stable radix sort, cuts the sorted list into
// chunks of equal length and adds each run of equal ids within a chunk: a
// natural text's most frequent token has thousands of rows, so the work is
// split by sorted positions, not by table rows.  Runs that cross chunks leave
// fp32 partial sums that a second kernel adds in order.  There are no
// floating-point atomics: the result depends on the inputs alone.
// Measured: 8192 tokens into 32768x1024 fp32, 48 us (four launches of the sort
// with the clearing beside them 33, sums 12, join 5; 168 MB move at the least,
// 33 us at a copy's 5.1 TB/s); 65536 tokens into 50000x2048 bf16, 138 us
// (51, 78, 9; 473 MB, 93 us).  Streaming the gradient's loads past the caches
// takes 74 us instead of 78 for the sums of the second and 13.4 instead of
// 11.8 for those of the first, whose gradient the caches still hold, and was
// left out.
#include "rows.hpp"
#include "sequence.hpp"

namespace prn {

namespace {

constexpr int kThreads = 256;

// An id as a sort key: ids outside the table become V, which sorts last.
__device__ __forceinline__ uint32_t id_key(const void *ids, int wide, int64_t n, int64_t V) {
    const int64_t id = wide ? static_cast<const int64_t *>(ids)[n] : (int64_t)static_cast<const int32_t *>(ids)[n];
    return id >= 0 && id < V ? (uint32_t)id : (uint32_t)V;
}

// ---------------------------------------------------------------- lookup
struct EmbFwdArgs {
    int64_t N, V;
    int D, wide, lanes;  // lanes (a power of two) share a row
    const void *ids, *table;
    float scale;
    void *out;
};

constexpr int kLookRows = 4;  // rows whose loads a thread keeps in flight

// Rows that begin at any element: 65536 rows of 50000x2047 bf16, uniform ids, in
// 140 us (210 an element at a time; 109 for 2048 columns).
template <typename T, bool VEC>
__global__ __launch_bounds__(kThreads) void emb_lookup_kernel(EmbFwdArgs a) {
    constexpr int V = kVec<T>;
    const int li = threadIdx.x & (a.lanes - 1);
    const int per = kThreads / a.lanes;  // rows a workgroup takes at once
    const int64_t n0 = (int64_t)blockIdx.x * per * kLookRows + threadIdx.x / a.lanes;
    uint32_t key[kLookRows];
#pragma unroll
    for (int r = 0; r < kLookRows; ++r) {
        const int64_t n = n0 + (int64_t)r * per;
        key[r] = n < a.N ? id_key(a.ids, a.wide, n, a.V) : (uint32_t)a.V;
    }
    const float bad = __uint_as_float(0x7fc00000u);
    for (int c0 = li * V; c0 < a.D; c0 += a.lanes * V) {
        const int c = group_at<T, VEC>(c0, a.D);
        float f[kLookRows][V];
#pragma unroll
        for (int r = 0; r < kLookRows; ++r) {
            if (key[r] < (uint32_t)a.V) load_group<T, VEC>(static_cast<const T *>(a.table) + (int64_t)key[r] * a.D + c, a.D, f[r]);
            else
#pragma unroll
                for (int i = 0; i < V; ++i) f[r][i] = bad;
        }
#pragma unroll
        for (int r = 0; r < kLookRows; ++r) {
            const int64_t n = n0 + (int64_t)r * per;
            if (n >= a.N) continue;
#pragma unroll
            for (int i = 0; i < V; ++i) f[r][i] *= a.scale;
            store_group<T, VEC>(static_cast<T *>(a.out) + n * a.D + c, a.D, f[r]);
        }
    }
}

// ---------------------------------------------------------------- zero rows
// Every row of the gradient is cleared while the ids are sorted (a share in
// each launch of the sort, by workgroups of their own): the sort has work for
// few CUs, and rows that no id names need no search.  Named rows are written
// twice for that, at most N of V + N.  The stores are streamed: kept in the
// caches as ordinary ones are, their way to memory costs the sums that follow
// (65536 x 2048 bf16: 93 us instead of 78).
struct ZeroArgs {
    char *out;
    int64_t bytes;
    int first;  // workgroups of the launch before those that clear
};
constexpr int kZeroBlocks = 1024;

__device__ __forceinline__ void zero_share(const ZeroArgs &z, int share, int shares) {
    // 16-byte pieces [lo, hi) of this share; the first also takes what is left at either end
    const int64_t head = min(z.bytes, (int64_t)((16 - ((uintptr_t)z.out & 15)) & 15)), whole = (z.bytes - head) / 16;
    u32x4 *v = reinterpret_cast<u32x4 *>(z.out + head);
    const u32x4 zero = {0u, 0u, 0u, 0u};
    const int64_t lo = whole * share / shares, hi = whole * (share + 1) / shares;
    const int64_t me = (int64_t)((int)blockIdx.x - z.first) * blockDim.x + threadIdx.x;
    const int64_t all = (int64_t)((int)gridDim.x - z.first) * blockDim.x;
    int64_t i = lo + me;
    for (; i + 3 * all < hi; i += 4 * all) {
#pragma unroll
        for (int u = 0; u < 4; ++u) __builtin_nontemporal_store(zero, v + i + u * all);
    }
    for (; i < hi; i += all) __builtin_nontemporal_store(zero, v + i);
    if (share == 0) {
        if (me < head) z.out[me] = 0;
        if (me < z.bytes - head - whole * 16) z.out[head + whole * 16 + me] = 0;
    }
}

// ---------------------------------------------------------------- sort
constexpr int kBins = 256;          // 8 bits of the key a pass
constexpr int kSmallN = 4096;       // sorted by one workgroup in LDS
constexpr int kSmallThreads = 1024;
constexpr int kMaxTiles = 128;      // workgroups of a pass over a longer list

// Lanes of the wave whose digit equals this lane's (valid lanes only).
__device__ __forceinline__ uint64_t same_digit(uint32_t d, bool valid) {
    uint64_t m = __ballot(valid);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        const uint64_t one = __ballot((d >> b) & 1u);
        m &= ((d >> b) & 1u) ? one : ~one;
    }
    return m;
}

// Exclusive sum of one value per thread over the first 256 threads of a
// workgroup (all of its threads call this).
__device__ __forceinline__ uint32_t scan256(uint32_t v, uint32_t *tmp) {
    const int t = threadIdx.x, lane = t & 63;
    uint32_t inc = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = __shfl_up(inc, d, 64);
        if (lane >= d) inc += o;
    }
    if (t < kBins && lane == 63) tmp[t >> 6] = inc;
    __syncthreads();
    uint32_t before = 0;
    for (int w = 0; w < (t >> 6) && w < 4; ++w) before += tmp[w];
    __syncthreads();
    return before + inc - v;
}

struct SortArgs {
    int64_t N, V;
    int wide, passes;
    const void *ids;
    uint32_t *key[2], *pos[2];
    uint32_t *hist;  // [tiles][256]
    int64_t tile;    // elements a workgroup (a multiple of 256)
};

// A wave's places for up to U groups of 64 elements in their order: the
// counters' additions of one wave are done in the order they are issued, so
// none waits for the one before it.
template <int U>
__device__ __forceinline__ void take_places(uint32_t *counter, const uint32_t (&d)[U], int count, uint32_t (&to)[U]) {
    const int lane = threadIdx.x & 63;
    uint64_t same[U];
    uint32_t base[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const bool valid = u * 64 + lane < count;
        same[u] = same_digit(d[u], valid);
        base[u] = 0;
        if (valid && lane == __ffsll((unsigned long long)same[u]) - 1) base[u] = atomicAdd(&counter[d[u]], (uint32_t)__popcll(same[u]));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int first = same[u] != 0 ? __ffsll((unsigned long long)same[u]) - 1 : lane;
        to[u] = __shfl(base[u], first, 64) + (uint32_t)__popcll(same[u] & ((1ull << lane) - 1ull));
    }
}

// The whole list in one workgroup: wave w keeps the elements [w per, (w + 1) per) in order.
__global__ __launch_bounds__(kSmallThreads) void emb_sort_small_kernel(SortArgs a, ZeroArgs zero) {
    if ((int)blockIdx.x >= zero.first) {
        zero_share(zero, 0, 1);
        return;
    }
    constexpr int U = kSmallN / kSmallThreads, NW = kSmallThreads / 64;
    __shared__ uint32_t key[kSmallN];
    __shared__ uint16_t pos[kSmallN];
    __shared__ uint32_t cnt[NW][kBins];
    __shared__ uint32_t tmp[4];
    const int t = threadIdx.x, w = t >> 6, lane = t & 63;
    const int N = (int)a.N;
    const int per = (N + kSmallThreads - 1) / kSmallThreads * 64, lo = w * per, count = max(0, min(N - lo, per));
    uint32_t k[U], d[U], to[U];
    uint16_t q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int n = u * 64 + lane;
        k[u] = n < count ? id_key(a.ids, a.wide, lo + n, a.V) : 0u;
        q[u] = (uint16_t)(lo + n);
    }
    for (int p = 0; p < a.passes; ++p) {
#pragma unroll
        for (int i = 0; i < NW * kBins / kSmallThreads; ++i) (&cnt[0][0])[t + i * kSmallThreads] = 0;
        if (p > 0)
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (u * 64 + lane < count) {
                    k[u] = key[lo + u * 64 + lane];
                    q[u] = pos[lo + u * 64 + lane];
                }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            d[u] = (k[u] >> (8 * p)) & 255u;
            if (u * 64 + lane < count) atomicAdd(&cnt[w][d[u]], 1u);
        }
        __syncthreads();
        uint32_t c[NW], total = 0;
        if (t < kBins)
#pragma unroll
            for (int v = 0; v < NW; ++v) c[v] = cnt[v][t];
#pragma unroll
        for (int v = 0; v < NW; ++v) total += t < kBins ? c[v] : 0u;
        uint32_t run = scan256(total, tmp);
        if (t < kBins)
#pragma unroll
            for (int v = 0; v < NW; ++v) {
                cnt[v][t] = run;
                run += c[v];
            }
        __syncthreads();
        take_places<U>(cnt[w], d, count, to);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u * 64 + lane < count) {
                key[to[u]] = k[u];
                pos[to[u]] = q[u];
            }
        __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int n = t + u * kSmallThreads;
        if (n < N) {
            a.key[0][n] = key[n];
            a.pos[0][n] = pos[n];
        }
    }
}

__device__ __forceinline__ uint32_t key_at(const SortArgs &a, int p, int64_t n) {
    return p == 0 ? id_key(a.ids, a.wide, n, a.V) : a.key[(p - 1) & 1][n];
}

// Digit counts of each workgroup's elements in pass p.
__global__ __launch_bounds__(kThreads) void emb_hist_kernel(SortArgs a, int p, ZeroArgs zero) {
    if ((int)blockIdx.x >= zero.first) {
        zero_share(zero, 2 * p, 2 * a.passes);
        return;
    }
    __shared__ uint32_t cnt[kBins];
    cnt[threadIdx.x] = 0;
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * a.tile, hi = min(a.N, lo + a.tile);
    for (int64_t n = lo + threadIdx.x; n < hi; n += kThreads) atomicAdd(&cnt[(key_at(a, p, n) >> (8 * p)) & 255u], 1u);
    __syncthreads();
    a.hist[(int64_t)blockIdx.x * kBins + threadIdx.x] = cnt[threadIdx.x];
}

// Moves each workgroup's elements to their places in pass p, keeping the
// order of equal digits: wave w takes the w-th quarter of the tile in order.
__global__ __launch_bounds__(kThreads) void emb_scatter_kernel(SortArgs a, int p, ZeroArgs zero) {
    if ((int)blockIdx.x >= zero.first) {
        zero_share(zero, 2 * p + 1, 2 * a.passes);
        return;
    }
    __shared__ uint32_t cnt[4][kBins];
    __shared__ uint32_t tmp[4];
    const int t = threadIdx.x, w = t >> 6, lane = t & 63;
    const int64_t end = min(a.N, ((int64_t)blockIdx.x + 1) * a.tile);
    const int64_t lo = (int64_t)blockIdx.x * a.tile + w * (a.tile / 4), hi = min(end, lo + a.tile / 4);
#pragma unroll
    for (int v = 0; v < 4; ++v) cnt[v][t] = 0;
    __syncthreads();
    for (int64_t n = lo + lane; n < hi; n += 64) atomicAdd(&cnt[w][(key_at(a, p, n) >> (8 * p)) & 255u], 1u);
    uint32_t before = 0, total = 0;
#pragma unroll 16
    for (int g = 0; g < zero.first; ++g) {
        const uint32_t c = a.hist[(int64_t)g * kBins + t];
        total += c;
        before += g < (int)blockIdx.x ? c : 0u;
    }
    uint32_t run = scan256(total, tmp) + before;  // its barriers also order the counts above
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        const uint32_t c = cnt[v][t];
        cnt[v][t] = run;
        run += c;
    }
    __syncthreads();
    constexpr int U = 4;
    for (int64_t n0 = lo; n0 < hi; n0 += U * 64) {
        const int count = (int)min(hi - n0, (int64_t)U * 64);
        uint32_t k[U], q[U], d[U], to[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t n = n0 + u * 64 + lane;
            const bool valid = u * 64 + lane < count;
            k[u] = valid ? key_at(a, p, n) : 0u;
            q[u] = p == 0 ? (uint32_t)n : (valid ? a.pos[(p - 1) & 1][n] : 0u);
            d[u] = (k[u] >> (8 * p)) & 255u;
        }
        take_places<U>(cnt[w], d, count, to);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u * 64 + lane < count) {
                a.key[p & 1][to[u]] = k[u];
                a.pos[p & 1][to[u]] = q[u];
            }
    }
}

// ---------------------------------------------------------------- sums
struct EmbSumArgs {
    int64_t N, V, pad;  // pad: the row whose gradient stays zero, or -1
    int D;
    const uint32_t *key, *pos;
    const void *grad;
    float scale;
    void *out;
    float *part;     // [chunks][2][D]: sums of a run that came from the chunk before, of one that goes on
    int run;         // sorted positions a chunk (at most 64)
    int64_t chunks, cols;  // column blocks of 64 * V
};

constexpr int kBatch = 8;         // rows whose loads are in flight
constexpr uint32_t kNoKey = ~0u;  // above every key

// A wave takes a chunk for 64 groups of columns (65536 tokens, 50000x2047 bf16:
// the whole gradient 156 us; 139 for 2048 columns; an element at a time, uniform
// ids, 271 where this takes 168).
template <typename T, bool VEC>
__global__ __launch_bounds__(kThreads) void emb_sum_kernel(EmbSumArgs a) {
    constexpr int V = kVec<T>;
    const int lane = threadIdx.x & 63;
    const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (item >= a.chunks * a.cols) return;
    const int64_t chunk = item / a.cols;
    const int c0 = (int)(item - chunk * a.cols) * 64 * V + lane * V, c = group_at<T, VEC>(c0, a.D);
    const int64_t n0 = chunk * a.run;
    const int cnt = (int)min((int64_t)a.run, a.N - n0);
    const uint32_t mykey = a.key[n0 + min(lane, cnt - 1)], mypos = a.pos[n0 + min(lane, cnt - 1)];
    const uint32_t prev = n0 > 0 ? a.key[n0 - 1] : kNoKey;
    const uint32_t next = n0 + cnt < a.N ? a.key[n0 + cnt] : kNoKey;
    const bool in = c0 < a.D;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    bool from_start = true;  // the current run began at the chunk's first position
    uint32_t cur = __builtin_amdgcn_readlane(mykey, 0);
    auto flush = [&](bool to_end) {
        if (cur < (uint32_t)a.V && (int64_t)cur != a.pad && in) {
            const bool head = from_start && prev == cur, tail = to_end && next == cur;
            if (head || tail) {
                float *p = a.part + ((chunk * 2 + (head ? 0 : 1)) * a.D + c);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (VEC || i < a.D) p[i] = acc[i];
            } else {
                float f[V];
#pragma unroll
                for (int i = 0; i < V; ++i) f[i] = acc[i] * a.scale;
                store_group<T, VEC>(static_cast<T *>(a.out) + (int64_t)cur * a.D + c, a.D, f);
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    };
    for (int b = 0; b < cnt; b += kBatch) {
        float f[kBatch][V];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int64_t row = (int64_t)__builtin_amdgcn_readlane(mypos, min(b + u, cnt - 1));
            if (in) load_group<T, VEC>(static_cast<const T *>(a.grad) + row * a.D + c, a.D, f[u]);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (b + u < cnt) {
                const uint32_t k = __builtin_amdgcn_readlane(mykey, b + u);
                if (k != cur) {
                    flush(false);
                    cur = k;
                    from_start = false;
                }
                if (in)
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[i] += f[u][i];
            }
        }
    }
    flush(true);
}

// Runs that cross chunks: the wave of the chunk where such a run begins adds
// its partial sums in order, V columns a lane.
template <typename T, int V>
__global__ __launch_bounds__(kThreads) void emb_join_kernel(EmbSumArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (item >= a.chunks * a.cols) return;
    const int64_t chunk = item / a.cols;
    const int c = (int)(item - chunk * a.cols) * 64 * V + lane * V;
    const int64_t n0 = chunk * a.run, n1 = n0 + a.run;  // n1: the next chunk's first position
    if (n1 >= a.N) return;
    const uint32_t k = a.key[n1], end = a.key[n1 - 1], begin = a.key[n0], before = n0 > 0 ? a.key[n0 - 1] : kNoKey;
    if (end != k || k >= (uint32_t)a.V || (int64_t)k == a.pad) return;
    if (begin == k && before == k) return;  // the run begins earlier
    int64_t past = chunk + 1;  // the first chunk that does not begin with the run's id
    while (true) {
        const int64_t q = past + lane;
        const uint64_t ends = __ballot(q >= a.chunks || a.key[min(q, a.chunks - 1) * a.run] != k);
        if (ends != 0) {
            past += __ffsll((unsigned long long)ends) - 1;
            break;
        }
        past += 64;
    }
    if (c >= a.D) return;
    float acc[V];
    load_vec<float, V>(a.part + (chunk * 2 + 1) * a.D + c, acc);
    constexpr int U = 8;
    for (int64_t q0 = chunk + 1; q0 < past; q0 += U) {
        float f[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (q0 + u < past) load_vec<float, V>(a.part + (q0 + u) * 2 * a.D + c, f[u]);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (q0 + u < past)
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] += f[u][i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] *= a.scale;
    store_vec<T, V>(static_cast<T *>(a.out) + (int64_t)k * a.D + c, acc);
}

// Layout of the gradient's scratch.
struct EmbWs {
    int tiles, run;
    int64_t tile, chunks;
    size_t key[2], pos[2], hist, part, total;
};
EmbWs emb_ws(int64_t N, int64_t D) {
    EmbWs w;
    size_t off = kScratchOffset;
    auto take = [&](size_t n) {
        const size_t at = off;
        off += (n + 255) / 256 * 256;
        return at;
    };
    const bool small = N <= kSmallN;
    w.tile = std::max<int64_t>(512, ((N + kMaxTiles - 1) / kMaxTiles + 255) / 256 * 256);
    w.tiles = (int)((N + w.tile - 1) / w.tile);
    // chunks of up to 64 entries (one a lane), shorter where that makes fewer
    // than four waves a SIMD.  65536 x 2048 bf16 (four with 64 entries): 91 us +
    // 10 us for the joins, with 32 entries 94 + 17; 65536 x 128 bf16 (one with
    // 64): the whole gradient 48 us, with 16 entries 36; 8192 x 1024 fp32 (one
    // with 16): sums and joins 12 + 5, with 8 entries 12 + 8; 4000 x 256 bf16
    // (a quarter with 16): the whole gradient 22 us, with 8 entries 19 (the whole
    // gradients with uniform ids).
    const int64_t per_simd = N * ((D + 511) / 512) / (4 * device_cu_count());
    w.run = per_simd >= 256 ? 64 : per_simd >= 128 ? 32 : per_simd >= 16 ? 16 : 8;
    w.chunks = (N + w.run - 1) / w.run;
    for (int i = 0; i < 2; ++i) {
        w.key[i] = i == 0 || !small ? take((size_t)N * 4) : w.key[0];
        w.pos[i] = i == 0 || !small ? take((size_t)N * 4) : w.pos[0];
    }
    w.hist = take((size_t)w.tiles * kBins * 4);
    w.part = take((size_t)w.chunks * 2 * (size_t)D * 4);
    w.total = off;
    return w;
}

template <typename T, bool VEC>
hipError_t emb_sums(EmbSumArgs &a, hipStream_t s) {
    constexpr int V = kVec<T>;
    a.cols = (a.D + 64 * V - 1) / (64 * V);
    emb_sum_kernel<T, VEC><<<(unsigned)((a.chunks * a.cols + 3) / 4), kThreads, 0, s>>>(a);
    if (a.chunks == 1) return hipGetLastError();  // no run crosses chunks
    constexpr int J = VEC ? 4 : 1;
    a.cols = (a.D + 64 * J - 1) / (64 * J);
    emb_join_kernel<T, J><<<(unsigned)((a.chunks * a.cols + 3) / 4), kThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

size_t embedding_ws(int64_t N, int64_t D) { return emb_ws(N, D).total; }

hipError_t embedding_forward(const EmbeddingArgs &q, hipStream_t s) {
    const int es = q.bf16 ? 2 : 4, vec = 16 / es;
    const bool al = q.D % vec == 0 && aligned16(q.table) && aligned16(q.out);
    const int64_t vecs = (q.D + vec - 1) / vec;
    int lanes = 1;
    while (lanes < 64 && lanes < vecs) lanes *= 2;
    const EmbFwdArgs a{q.N, q.V, (int)q.D, q.wide_ids, lanes, q.ids, q.table, q.scale, q.out};
    const int64_t per = (int64_t)kThreads / lanes * kLookRows;
    const unsigned grid = (unsigned)((q.N + per - 1) / per);
    if (q.bf16) {
        if (al) emb_lookup_kernel<bf16, true><<<grid, kThreads, 0, s>>>(a);
        else emb_lookup_kernel<bf16, false><<<grid, kThreads, 0, s>>>(a);
    } else {
        if (al) emb_lookup_kernel<float, true><<<grid, kThreads, 0, s>>>(a);
        else emb_lookup_kernel<float, false><<<grid, kThreads, 0, s>>>(a);
    }
    return hipGetLastError();
}

hipError_t embedding_backward(const EmbeddingArgs &q, const Ws &ws, hipStream_t s) {
    const EmbWs w = emb_ws(q.N, q.D);
    SortArgs o{};
    o.N = q.N;
    o.V = q.V;
    o.wide = q.wide_ids;
    o.ids = q.ids;
    o.tile = w.tile;
    o.hist = reinterpret_cast<uint32_t *>(ws.p + w.hist);
    for (int i = 0; i < 2; ++i) {
        o.key[i] = reinterpret_cast<uint32_t *>(ws.p + w.key[i]);
        o.pos[i] = reinterpret_cast<uint32_t *>(ws.p + w.pos[i]);
    }
    o.passes = 1;
    while (o.passes < 4 && (q.V >> (8 * o.passes)) != 0) ++o.passes;  // V itself is a key
    ZeroArgs zero{static_cast<char *>(q.out), q.V * q.D * (q.bf16 ? 2 : 4), w.tiles};
    const int blocks = (int)std::min<int64_t>((zero.bytes + 16383) / 16384, kZeroBlocks);
    int at = 0;
    if (q.N <= kSmallN) {
        zero.first = 1;  // a workgroup here fills a CU
        emb_sort_small_kernel<<<1 + std::min(blocks, device_cu_count() - 1), kSmallThreads, 0, s>>>(o, zero);
    } else {
        for (int p = 0; p < o.passes; ++p) {
            emb_hist_kernel<<<w.tiles + blocks, kThreads, 0, s>>>(o, p, zero);
            emb_scatter_kernel<<<w.tiles + blocks, kThreads, 0, s>>>(o, p, zero);
        }
        at = (o.passes - 1) & 1;
    }
    EmbSumArgs a{q.N, q.V, q.padding, (int)q.D, o.key[at], o.pos[at], q.table, q.scale, q.out,
                 reinterpret_cast<float *>(ws.p + w.part), w.run, w.chunks, 0};
    const int vec = q.bf16 ? 8 : 4;
    const bool al = q.D % vec == 0 && aligned16(q.table) && aligned16(q.out);
    if (q.bf16) return al ? emb_sums<bf16, true>(a, s) : emb_sums<bf16, false>(a, s);
    return al ? emb_sums<float, true>(a, s) : emb_sums<float, false>(a, s);
}

}  // namespace prn
