// walk.hpp -- the walk kernel of linear attention (the primitive of
// linattn.hpp) on bf16 matrix instructions, for bf16 and fp32 operands.
//
// Chunks of C positions.  Within a chunk, with the decays applied in fp32:
//   P = (X Y^T) * wi e^(g(i-j)) on and below the diagonal,
//   out = P Z + wo e^(g(i+1-e)) X T,
//   T <- e^(gC) T + sum_j Y_j^T (wt e^(g(C-1-j+e)) Z_j).
// One workgroup walks one segment of one (batch row, head) for 64 columns of
// Z; wave w owns columns 16 w .. 16 w + 15 and keeps its [D1, 16] columns of T
// in fp32 registers.  T is a matrix operand straight from there: in the
// layout of a 16x16 result a lane holds column lane % 16 and four rows, and
// the order of rows over tiles is chosen (row 32 t + 8 (lane / 16) + 4 u + r in
// register r of tile 2 t + u) so that two tiles are the eight consecutive k of
// one operand of the next product.  Only P crosses the waves, through LDS.
//
// Precision.  An fp32 number is three bf16 numbers of 8 bits each, exactly;
// a product of two such sums takes the six products whose size is at least
// 2^-16 of the first, which leaves an error of 2^-23 or so.  fp32 operands are
// held as three planes throughout.  bf16 operands are one plane, exact as they
// come, and T is fp32 in both: the decayed Z that it adds up is split into
// three planes, so the state of a bf16 model is as good as that of an fp32 one.
// For the bf16 outputs alone, P and the copy of T that the rows are multiplied
// with are rounded to bf16 once.  Sums of many such products are then off by
// about as much as their own rounding (B=8, L=2048, H=16, 128x128: outputs and
// gradients 2.3e-3 from 64 bits, of which the last rounding alone is 1.7e-3);
// two planes each leave that rounding alone and cost 45% (forward there, 95 to
// 138 us; backward at B=1, 58 to 64).  Where few terms are summed two planes are
// taken: of T in heads of up to 32, of P in chunks of 32 positions, which all
// short sequences have.
//
// (A first form of the kernel on fp32 matrix instructions, with bf16 tensors
// widened, took 647 us where this one takes 92: B=8, L=2048, H=16, 128x128.)
//
// What bounds it (B=8, L=2048, H=16, 128x128, bf16): 268 MB forward, 52 us at
// the rate of a copy, 470 MB backward, 92 us; matrix instructions 18 us of the
// forward pass.  It takes 92 us forward and 197 us backward.  Neither
// memory (the loads and stores alone 75 and 162 us) nor the arithmetic (all
// but the loads 83 and 175) fills the time; a workgroup's three barriers a chunk
// leave both idle in turn.  Tried and not kept, beside 102 us forward and 256
// backward at the time: three chunks in LDS and one barrier (the accumulators
// then move between register files, 103 and 329), two waves sharing 16 columns
// with half the positions each (115, 337), workgroups of 32 columns (116, 365),
// outputs through LDS in whole rows (98, 263).
#pragma once

#include "linattn.hpp"
#include "walk_rows.hpp"

namespace prn {
namespace walk {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kNB = 64;  // columns of Z a workgroup

template <typename T> constexpr int kPlanes = sizeof(T) == 2 ? 1 : 3;

// Element offset of 8-element group `grp` of row `row` in an LDS tile of W
// columns.  Rows of 64, 128 and 256 columns are swizzled so that both the row
// reads (16 rows, one group) and the transposing reads (4 rows, 4 groups) of
// 16 lanes fall on different banks; other widths are padded by one group.
template <int W>
__device__ __forceinline__ int tile_at(int row, int grp) {
    if (W == 128 || W == 256) return row * W + ((grp ^ (((row & 3) << 2) | (-(row >> 2) & 3))) << 3);
    if (W == 64) return row * W + ((grp ^ ((((row >> 1) & 1) << 2) | (-(row >> 2) & 3))) << 3);
    return row * (W + 8) + (grp << 3);
}
template <int W> constexpr int kTileRow = (W == 64 || W == 128 || W == 256) ? W : W + 8;

__device__ __forceinline__ bf16x8 read_row(const bf16 *p) { return *reinterpret_cast<const bf16x8 *>(p); }

// Transposing read: the 16 lanes of a group give the addresses of four rows
// of 16 columns (lane 4 i + c: row i, columns 4 c ..); lane m receives column m of the four rows.
__device__ __forceinline__ s16x4 read_tr(const bf16 *p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(p));
}
__device__ __forceinline__ bf16x8 join(s16x4 a, s16x4 b) {
    union {
        s16x4 s[2];
        bf16x8 v;
    } u;
    u.s[0] = a;
    u.s[1] = b;
    return u.v;
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Sum of the products of two numbers given as NA and NB planes, smallest first.
template <int NA, int NB>
__device__ __forceinline__ f32x4 mfma_planes(const bf16x8 (&a)[NA], const bf16x8 (&b)[NB], f32x4 c) {
#pragma unroll
    for (int s = 2; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB) c = mfma(a[i], b[s - i], c);
    return c;
}

// The upper halves of two words as one (two truncated bf16).
__device__ __forceinline__ uint32_t upper_halves(uint32_t lo, uint32_t hi) { return __builtin_amdgcn_perm(hi, lo, 0x07060302u); }

// Eight fp32 numbers as three planes of bf16, exactly (8 bits each).
__device__ __forceinline__ void split3(const float (&f)[8], bf16x8 (&p)[3]) {
    union {
        uint32_t w[4];
        bf16x8 v;
    } u[3];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a = f[2 * i], b = f[2 * i + 1];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const uint32_t wa = __float_as_uint(a), wb = __float_as_uint(b);
            u[k].w[i] = upper_halves(wa, wb);
            if (k < 2) {
                a -= __uint_as_float(wa & 0xffff0000u);
                b -= __uint_as_float(wb & 0xffff0000u);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) p[k] = u[k].v;
}
__device__ __forceinline__ void round1(const float (&f)[8], bf16x8 (&p)[1]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[0][i] = (bf16)f[i];
}
__device__ __forceinline__ void split2(const float (&f)[8], bf16x8 (&p)[2]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        p[0][i] = (bf16)f[i];
        p[1][i] = (bf16)(f[i] - (float)p[0][i]);
    }
}
template <int N>
__device__ __forceinline__ void to_planes(const float (&f)[8], bf16x8 (&p)[N]) {
    if constexpr (N == 3) split3(f, p);
    else if constexpr (N == 2) split2(f, p);
    else round1(f, p);
}
template <int N>
__device__ __forceinline__ float plane_sum(const bf16x8 (&p)[N], int i) {
    float v = (float)p[0][i];
#pragma unroll
    for (int k = 1; k < N; ++k) v += (float)p[k][i];
    return v;
}

// Buffer accesses: an offset at or past `bytes` reads zeros and writes nothing.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, (int)bytes, 0x00020000);
}
// Chunk i of cnt positions; the same in whole words, `skew` bytes before it.
// (Their sizes are the same in every lane, which the compiler may lose sight of:
// each access would then be a loop over the lanes' resources.)
__device__ __forceinline__ uint32_t same_in_lanes(uint32_t x) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)x); }
__device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk_of(const Rows &v, int i, int cnt, int C) {
    return buffer_of(v.at(i, cnt, C), same_in_lanes(v.bytes(cnt)));
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk_words_of(const Rows &v, int i, int cnt, int C, uint32_t &skew) {
    const char *first = v.at(i, cnt, C);
    skew = Rows::word_skew(first);
    return buffer_of(first - skew, same_in_lanes(v.word_bytes(skew, cnt)));
}
template <typename T>
__device__ __forceinline__ Rows rows_of(const WalkView &v, int64_t b, int64_t h, int64_t L, int64_t begin, int C, int rev,
                                        int c0, int d) {
    const char *first = static_cast<const char *>(v.p) + (b * v.sb + h * v.sh + c0) * (int64_t)sizeof(T);
    return rows_from(first, v.st * (int64_t)sizeof(T), (uint32_t)((d - c0) * (int)sizeof(T)), L, begin, C, rev);
}

// Group n of a thread, as the planes of its 8 elements, into an LDS tile.
template <int W, int C, int kP>
__device__ __forceinline__ void put_group(bf16 *lds, int thread, int n, const bf16x8 (&p)[kP]) {
    constexpr int kGroups = Groups<W, C>::kGroups;
    const int i = thread + n * kThreads, r = i / kGroups, grp = i - r * kGroups;
    if (C * kGroups % kThreads != 0 && r >= C) return;
#pragma unroll
    for (int k = 0; k < kP; ++k) *reinterpret_cast<bf16x8 *>(lds + k * C * kTileRow<W> + tile_at<W>(r, grp)) = p[k];
}
// Zeros over a thread's rows past the last position.
template <int kP, int W, int C>
__device__ __forceinline__ void clear_past(bf16 *lds, int thread, int cnt) {
    uint32_t none = 0;
    asm volatile("" : "+v"(none));  // or the zeros take registers in every chunk
    bf16x8 zero[kP];
#pragma unroll
    for (int k = 0; k < kP; ++k) {
        const u32x4 z = {none, none, none, none};
        zero[k] = *reinterpret_cast<const bf16x8 *>(&z);
    }
#pragma unroll 1
    for (int n = 0; n < Groups<W, C>::kN; ++n)
        if (Groups<W, C>::past(thread, n, cnt)) put_group<W, C>(lds, thread, n, zero);
}
__device__ __forceinline__ void planes_of(const bf16 (&v)[8], bf16x8 (&p)[1]) { p[0] = *reinterpret_cast<const bf16x8 *>(&v[0]); }
__device__ __forceinline__ void planes_of(const float (&v)[8], bf16x8 (&p)[3]) { split3(v, p); }

// A thread's share of one tile, loaded ahead of its use.  VEC: rows are
// 16-byte aligned and whole numbers of 16-byte pieces.
template <typename T, int W, int C, bool VEC>
struct Ahead {
    Groups<W, C> g;
    struct alignas(16) {
        T v[8];
    } r[Groups<W, C>::kN];

    __device__ __forceinline__ void init(const Rows &v) { g.init(v, sizeof(T), threadIdx.x); }
    // The cnt positions of chunk i; zeros past the ends.
    __device__ __forceinline__ void load(const Rows &v, int chunk, int cnt) {
        constexpr int kV = 16 / (int)sizeof(T);
        const __amdgpu_buffer_rsrc_t buf = chunk_of(v, chunk, cnt, C);
        const uint32_t shift = v.shift(cnt, C);
#pragma unroll
        for (int n = 0; n < g.kN; ++n) {
            const uint32_t o = g.offset(v, n, shift);
#pragma unroll
            for (int h = 0; h < 8 / kV; ++h) {
                // the second half of a group may lie past the row's end
                const uint32_t oh = h == 0 ? o : (g.column(n) + h * kV < g.left ? o + 16 * h : kNowhere);
                *reinterpret_cast<u32x4 *>(&r[n].v[h * kV]) = __builtin_amdgcn_raw_buffer_load_b128(buf, oh, 0, 0);
            }
        }
    }
    __device__ __forceinline__ void store(const Rows &, bf16 *lds) const {
#pragma unroll
        for (int n = 0; n < g.kN; ++n) {
            bf16x8 p[kPlanes<T>];
            planes_of(r[n].v, p);
            put_group<W, C>(lds, threadIdx.x, n, p);
        }
    }
};

// Rows that begin at any element: groups of fp32 are loaded from 4-byte
// aligned addresses, groups of bf16 as the five words of memory that hold
// them, and put straight when they go into LDS (forward at B=4, L=4000, H=8,
// 77x101 bf16: 88 us, 138 with a load an element; 60 with 80x104).
template <typename T, int W, int C>
struct Ahead<T, W, C, false> {
    Groups<W, C> g;
    static constexpr bool kHalves = sizeof(T) == 2;
    static constexpr int kWords = 2 * (int)sizeof(T);  // of a group
    uint32_t r[Groups<W, C>::kN][kWords + 1];
    uint32_t shift;                                    // of the loaded chunk's offsets, less the skew

    __device__ __forceinline__ void init(const Rows &v) { g.init(v, sizeof(T), threadIdx.x); }
    __device__ __forceinline__ void load(const Rows &v, int chunk, int cnt) {
        uint32_t skew = 0;
        const __amdgpu_buffer_rsrc_t buf = kHalves ? chunk_words_of(v, chunk, cnt, C, skew) : chunk_of(v, chunk, cnt, C);
        shift = v.shift(cnt, C) - skew;
#pragma unroll
        for (int n = 0; n < g.kN; ++n) {
            const uint32_t o = g.offset(v, n, shift) & ~3u;
#pragma unroll
            for (int h = 0; h < kWords / 4; ++h) {
                const u32x4 x = __builtin_amdgcn_raw_buffer_load_b128(buf, o + 16 * h, 0, 0);
#pragma unroll
                for (int k = 0; k < 4; ++k) r[n][4 * h + k] = x[k];
            }
            r[n][kWords] = kHalves ? __builtin_amdgcn_raw_buffer_load_b32(buf, o + 16, 0, 0) : 0u;
        }
    }
    __device__ __forceinline__ void store(const Rows &v, bf16 *lds) const {
#pragma unroll
        for (int n = 0; n < g.kN; ++n) {
            const uint32_t bits = kHalves ? (g.offset(v, n, shift) & 2u) << 3 : 0u;
            const int valid = g.own(n);
            union {
                uint32_t w[kWords];
                T v[8];
            } u;
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
                const uint32_t x = kHalves ? __builtin_amdgcn_alignbit(r[n][k + 1], r[n][k], bits) : r[n][k];
                u.w[k] = g.own_word(x, k, sizeof(T), valid);
            }
            bf16x8 p[kPlanes<T>];
            planes_of(u.v, p);
            put_group<W, C>(lds, threadIdx.x, n, p);
        }
    }
};

// Which part of the work a workgroup does (every count fits 31 bits: the
// grid does).  The divisions run on the vector unit; their results are put
// back into scalar registers, where addresses and branches want them.
struct Where {
    int bh, b, h;
    int walk, blk, seg;
    bool any;
};
// (batch row, head) pairs in groups of 8, then everything that reads the
// same rows: consecutive workgroups go to the 8 XCDs in turn, so all blocks of
// one pair meet in one L2.
__device__ __forceinline__ Where where(const WalkArgs &a, int segs) {
    auto scalar = [](uint32_t x) { return (int)__builtin_amdgcn_readfirstlane(x); };
    const uint32_t per = (uint32_t)(a.walks * a.nblk * segs), heads = (uint32_t)a.H;
    const uint32_t grp = blockIdx.x / (8 * per), rest = blockIdx.x - grp * 8 * per;
    const uint32_t bh = grp * 8 + (rest & 7), sub = rest >> 3, pair = sub / (uint32_t)segs, walk = pair / (uint32_t)a.nblk;
    Where w;
    w.bh = scalar(bh);
    w.b = scalar(bh / heads);
    w.h = w.bh - w.b * (int)heads;
    w.seg = scalar(sub - pair * (uint32_t)segs);
    w.walk = scalar(walk);
    w.blk = scalar(pair - walk * (uint32_t)a.nblk);
    w.any = w.bh < (int)(a.B * a.H) && w.blk * kNB < a.w[w.walk].d2;
    return w;
}

// Where segment states are kept between the launches: the registers of wave
// `wave` of a block, tile by tile.
template <int D1>
__device__ __forceinline__ f32x4 *seg_state(const WalkArgs &a, const Where &w, int seg, int wave) {
    const int64_t slot = ((w.walk * a.B * a.H + w.bh) * a.nblk + w.blk) * a.segs + seg;
    return reinterpret_cast<f32x4 *>(a.seg_state) + (slot * 4 + wave) * (D1 / 16) * 64;
}
// Row of T that register r of tile t holds in lanes of group q.
__device__ __forceinline__ int state_row(int t, int q, int r) { return 32 * (t >> 1) + 8 * q + 4 * (t & 1) + r; }

// Workgroups a CU that the registers are shared out for.  Where a launch has
// more than two a CU, bf16 takes chunks of 32 positions, whose smaller tiles
// leave room for three (backward at B=8, L=2048, H=16, 128x128: 202 us, 241
// with chunks of 64); with one or two a CU the longer chunk, with half as many
// barriers, is mostly ahead (backward at B=4, L=2048, H=16, 64x64: 77 us, 82 with
// 32; at B=1, L=4096, H=16, 96x96: 81, 88; the training forward pass the same, 95
// and 96), but for sequences of up to kShort positions, where it makes no
// difference to the time.
constexpr int64_t kShort = 256;
// fp32 keeps two: with three, walks have fewer registers than their loads ahead
// need (B=1, L=32771, H=8, 64x128: the call 186 us, 193 with three; backward at
// B=3, L=1000, H=10, 48x80: 70, 79; at B=8, L=1024, H=8, 64x64: 81, 86).
template <typename T, int D1, int C>
constexpr int kWgs = D1 > 128 ? 1 : sizeof(T) == 2 && C == 32 ? 3 : 2;

enum class Part {
    Whole,  // outputs and T
    State   // only the segment's own part of T (from zero), for the join
};

template <typename T, int D1, int C, bool VEC, Part PART>
__global__ __launch_bounds__(kThreads, (kWgs<T, D1, C>)) void walk_kernel(WalkArgs a) {
    constexpr bool kOut = PART == Part::Whole;
    constexpr int kP = kPlanes<T>;                 // planes of X, Y, Z
    constexpr int kR = kP == 3 ? 3 : C == 64 ? 1 : 2;  // planes of P
    constexpr int kS = kP == 3 ? 3 : D1 == 32 ? 2 : 1;  // planes of the operand copy of T
    constexpr int NA = D1 / 16, NT = D1 / 32, NS = C / 32, NI = C / 16;
    constexpr int kPX = C * kTileRow<D1>, kPZ = C * kTileRow<kNB>, kPP = C * kTileRow<C>;  // elements of a plane
    __shared__ __align__(16) bf16 X[kOut ? kP * kPX : 8], Y[kP * kPX], Z[kP * kPZ], P[kOut ? kR * kPP : 8];
    __shared__ __align__(16) float dec_z[C];
    const Where wh = where(a, kOut ? a.segs : a.segs - 1);
    if (!wh.any) return;
    const Walk &w = a.w[wh.walk];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, m = lane & 15, q = lane >> 4;
    const int tr_i = m >> 2, tr_c = m & 3;         // this lane's row and column group in a transposing read
    const int c0 = wh.blk * kNB, col = c0 + wave * 16 + m;
    const float g = walk_gate(a.log_decay, wh.h), g2 = g * kLog2e;
    const int64_t begin = (int64_t)wh.seg * a.seg_len, end = min(a.L, begin + a.seg_len);
    const int chunks = (int)((end - begin + C - 1) / C), last = (int)(end - begin - (int64_t)(chunks - 1) * C);

    f32x4 S[NA];
    if (kOut && a.segs > 1) {
        const f32x4 *src = seg_state<D1>(a, wh, wh.seg, wave) + lane;
#pragma unroll
        for (int t = 0; t < NA; ++t) S[t] = src[t * 64];
    } else {
#pragma unroll
        for (int t = 0; t < NA; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = state_row(t, q, r);
                S[t][r] = kOut && w.init != nullptr && col < w.d2 && row < w.d1
                              ? w.init[(int64_t)wh.bh * w.d1 * w.d2 + (int64_t)row * w.im + (int64_t)col * w.in] : 0.0f;
            }
    }

    // decays: of P's elements in tiles on the diagonal and one below it, of a
    // row's share of T, and (in LDS) of the positions' shares of T
    float dec_d[4], dec_o[4], dec_row[NI];
    const float dec16 = fast_exp2(16.0f * g2);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int n = m - 4 * q - r;
        dec_d[r] = n >= 0 ? w.wi * fast_exp2(g2 * (float)n) : 0.0f;
        dec_o[r] = w.wi * fast_exp2(g2 * (float)(n + 16));
    }
#pragma unroll
    for (int it = 0; it < NI; ++it) dec_row[it] = w.wo * fast_exp2(g2 * (float)(16 * it + m + 1 - w.e));
    if (threadIdx.x < C) dec_z[threadIdx.x] = w.wt * fast_exp2(g2 * (float)(C - 1 - (int)threadIdx.x + w.e));
    const Carry carry_full = walk_carry(g, C), carry_last = last == C ? carry_full : walk_carry(g, last);

    if constexpr (kOut) {
        // the tiles of P right of the diagonal that share a 32-wide read with it stay zero
        for (int i = threadIdx.x; i < kR * kPP / 8; i += kThreads) {
            const bf16x8 z = {};
            *reinterpret_cast<bf16x8 *>(&P[i * 8]) = z;
        }
    }

    auto rows = [&](const WalkView &v, int from, int d) { return rows_of<T>(v, wh.b, wh.h, a.L, begin, C, w.rev, from, d); };
    const Rows rx = rows(w.X, 0, w.d1), ry = rows(w.Y, 0, w.d1), rz = rows(w.Z, c0, w.d2),
               ro = rows({w.out, a.L * a.H * w.d2, a.H * w.d2, w.d2}, c0, w.d2);
    // the pass that only carries T is bound by the loads' latency and has the
    // registers to keep two chunks on their way
    constexpr int kDepth = kOut ? 1 : 2;
    Ahead<T, D1, C, VEC> ax, ay[kDepth];
    Ahead<T, kNB, C, VEC> az[kDepth];
    if (kOut) ax.init(rx);
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
        ay[d].init(ry);
        az[d].init(rz);
    }
    const int oc = wave * 16 + 4 * q;
    // this lane's row of the first 16-row tile of out, four columns from its own
    const uint32_t out_at = c0 + oc < w.d2 ? ro.row_at(m, C) + oc * (uint32_t)sizeof(T) : kNowhere;
    const uint32_t out_step = (uint32_t)(w.rev ? -16 : 16) * ro.row_bytes;

    auto positions = [&](int i) { return i < chunks - 1 ? C : i == chunks - 1 ? last : 0; };
    auto load = [&](int i, int d) {  // chunk i (past the last one: zeros) into registers
        const int cnt = positions(i);
        if (kOut) ax.load(rx, i, cnt);
        ay[d].load(ry, i, cnt);
        az[d].load(rz, i, cnt);
    };
    auto put = [&](int d) {
        if (kOut) ax.store(rx, X);
        ay[d].store(ry, Y);
        az[d].store(rz, Z);
    };
#pragma unroll
    for (int d = 0; d < kDepth; ++d) load(d, d);

    // The products of a chunk run as one sequence of batches, each a few
    // operand reads and the matrix instructions that use them, with the reads
    // of batch k + 1 issued before the products of batch k (the compiler,
    // short of registers, would put every read right before its use and wait):
    //   P: the tiles below and on the diagonal go round
    //     the waves (the last one is formed more than once if they don't come
    //     out even), each as its transpose, so that a lane's four results are
    //     consecutive j;
    //   the rows' share of T, transposed (lane m is position 16 it + m,
    //     registers are four columns);
    //   T over the chunk.
    constexpr int kTiles = NI * (NI + 1) / 2, kMine = (kTiles + 3) / 4;
    constexpr bool kLong = kP == 1 && C == 64;                             // longer batches, where the registers allow
    constexpr int kU1 = kLong ? 2 : 1, kU3 = kLong ? 4 : 2;                // units a batch
    constexpr int kB1 = kOut ? (kMine * NT + kU1 - 1) / kU1 : 0, kB2 = kOut ? NT : 0,
                  kB3s = (NA + kU3 - 1) / kU3, kB3 = NS * kB3s;
    constexpr int kFrags = kLong ? 4 : 2 * kP;
    static_assert(NI * kP <= kFrags && 2 * kU1 * kP <= kFrags && kU3 * kP <= kFrags, "a batch fits its buffer");
    struct Frags {
        bf16x8 v[kFrags];
    };
    int my_it[kMine], my_jt[kMine];
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
        const int tile = min(wave + 4 * k, kTiles - 1);
        my_it[k] = tile < 1 ? 0 : tile < 3 ? 1 : tile < 6 ? 2 : 3;
        my_jt[k] = tile - my_it[k] * (my_it[k] + 1) / 2;
    }
    auto carry_state = [&](bool whole) {
        const Carry carry = whole ? carry_full : carry_last;
        if (carry.fast) {
            asm volatile("");  // a branch: the compiler would work out both and select
#pragma unroll
            for (int t = 0; t < NA; ++t) S[t] *= carry.f;
        } else {
            const f32x4 f = {carry.f, carry.f, carry.f, carry.f};
#pragma unroll
            for (int t = 0; t < NA; ++t) S[t] = __builtin_elementwise_fma(S[t], f, S[t]);
        }
    };
    auto products = [&](int cnt, bool whole, bf16x8 (&z)[NS][kP], f32x4 (&o)[NI]) {
        // rows 16 it + m are laid out like rows m
        int y_off[kMine], x_off[kMine];
#pragma unroll
        for (int k = 0; k < kMine; ++k) {
            y_off[k] = __builtin_amdgcn_readfirstlane(my_jt[k] * 16 * kTileRow<D1>);
            x_off[k] = __builtin_amdgcn_readfirstlane(my_it[k] * 16 * kTileRow<D1>);
        }
        Frags buf[2];
        f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
        bf16x8 zw[3];
        auto read = [&](int k, Frags &f) {
            if (k < kB1) {
#pragma unroll
                for (int u = 0; u < kU1; ++u) {
                    const int unit = k * kU1 + u, mine = unit / NT, t = unit % NT;
                    if (unit < kMine * NT)
#pragma unroll
                        for (int p = 0; p < kP; ++p) {
                            f.v[(2 * u) * kP + p] = read_row(&Y[p * kPX + tile_at<D1>(m, 4 * t + q) + y_off[mine]]);
                            f.v[(2 * u + 1) * kP + p] = read_row(&X[p * kPX + tile_at<D1>(m, 4 * t + q) + x_off[mine]]);
                        }
                }
            } else if (k < kB1 + kB2) {
                const int t = k - kB1;
#pragma unroll
                for (int it = 0; it < NI; ++it)
#pragma unroll
                    for (int p = 0; p < kP; ++p)
                        f.v[it * kP + p] = read_row(&X[p * kPX + tile_at<D1>(it * 16 + m, 4 * t + q)]);
            } else {
                const int s = (k - kB1 - kB2) / kB3s, t0 = (k - kB1 - kB2) % kB3s * kU3;
#pragma unroll
                for (int u = 0; u < kU3; ++u)
                    if (t0 + u < NA)
#pragma unroll
                        for (int p = 0; p < kP; ++p) {
                            const int t = t0 + u, row = 32 * s + 8 * q + tr_i, grp = 4 * (t >> 1) + tr_c, in = 4 * (t & 1);
                            f.v[u * kP + p] = join(read_tr(&Y[p * kPX + tile_at<D1>(row, grp) + in]),
                                                   read_tr(&Y[p * kPX + tile_at<D1>(row + 4, grp) + in]));
                        }
            }
        };
        auto use = [&](int k, const Frags &f) {
            if (k < kB1) {
#pragma unroll
                for (int u = 0; u < kU1; ++u) {
                    const int unit = k * kU1 + u, mine = unit / NT, t = unit % NT;
                    if (unit >= kMine * NT) continue;
                    bf16x8 y[kP], x[kP];
#pragma unroll
                    for (int p = 0; p < kP; ++p) {
                        y[p] = f.v[(2 * u) * kP + p];
                        x[p] = f.v[(2 * u + 1) * kP + p];
                    }
                    acc = mfma_planes(y, x, acc);
                    if (t != NT - 1) continue;
                    const int it = my_it[mine], jt = my_jt[mine];
                    const float far = it - jt == 3 ? dec16 * dec16 : it - jt == 2 ? dec16 : 1.0f;
                    float v[8] = {};
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        v[r] = acc[r] * (it == jt ? dec_d[r] : dec_o[r] * far);
                        if (it == jt && m < 4 * q + r) v[r] = 0.0f;  // whatever Y holds there
                        acc[r] = 0.0f;
                    }
                    bf16x8 pv[kR];
                    to_planes(v, pv);
                    bf16 *to = &P[tile_at<C>(it * 16 + m, 2 * jt + (q >> 1)) + 4 * (q & 1)];
#pragma unroll
                    for (int p = 0; p < kR; ++p) *reinterpret_cast<u32x2 *>(to + p * kPP) = *reinterpret_cast<const u32x2 *>(&pv[p]);
                }
            } else if (k < kB1 + kB2) {
                const int t = k - kB1;
                const float v[8] = {S[2 * t][0],     S[2 * t][1],     S[2 * t][2],     S[2 * t][3],
                                    S[2 * t + 1][0], S[2 * t + 1][1], S[2 * t + 1][2], S[2 * t + 1][3]};
                bf16x8 sp[kS];
                to_planes(v, sp);
#pragma unroll
                for (int it = 0; it < NI; ++it) {
                    bf16x8 x[kP];
#pragma unroll
                    for (int p = 0; p < kP; ++p) x[p] = f.v[it * kP + p];
                    o[it] = mfma_planes(sp, x, t == 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : o[it]);
                }
                if (t == NT - 1)
#pragma unroll
                    for (int it = 0; it < NI; ++it)
#pragma unroll
                        for (int r = 0; r < 4; ++r) o[it][r] *= dec_row[it];
            } else {
                const int s = (k - kB1 - kB2) / kB3s, t0 = (k - kB1 - kB2) % kB3s * kU3;
                if (t0 == 0) {
                    float v[8];
                    if (whole) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] = plane_sum(z[s], i) * dec_z[32 * s + 8 * q + i];
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int n = cnt - 1 - (32 * s + 8 * q + i);
                            v[i] = n >= 0 ? plane_sum(z[s], i) * (w.wt * fast_exp2(g2 * (float)(n + w.e))) : 0.0f;
                        }
                    }
                    split3(v, zw);
                }
#pragma unroll
                for (int u = 0; u < kU3; ++u)
                    if (t0 + u < NA) {
                        bf16x8 y[kP];
#pragma unroll
                        for (int p = 0; p < kP; ++p) y[p] = f.v[u * kP + p];
                        S[t0 + u] = mfma_planes(y, zw, S[t0 + u]);
                    }
            }
        };
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int p = 0; p < kP; ++p) {
                const int row = 32 * s + 8 * q + tr_i, grp = 2 * wave + (tr_c >> 1), in = 4 * (tr_c & 1);
                z[s][p] = join(read_tr(&Z[p * kPZ + tile_at<kNB>(row, grp) + in]),
                               read_tr(&Z[p * kPZ + tile_at<kNB>(row + 4, grp) + in]));
            }
        read(0, buf[0]);
        auto ahead = [&](int k) {
            if (k + 1 < kB1 + kB2 + kB3) read(k + 1, buf[(k + 1) & 1]);
            __builtin_amdgcn_sched_barrier(0);
        };
#pragma unroll
        for (int k = 0; k < kB1 + kB2; ++k) {
            ahead(k);
            use(k, buf[k & 1]);
        }
#pragma unroll
        for (int k = kB1 + kB2; k < kB1 + kB2 + kB3; ++k) {
            ahead(k);
            if (k == kB1 + kB2) carry_state(whole);
            use(k, buf[k & 1]);
        }
    };
    // out += P Z.  Values of Z that are not finite must not reach earlier
    // positions through a zero of P: then (their columns of T have become so)
    // they are left out of the product and added to the positions from their own on.
    auto within = [&](int cnt, bf16x8 (&z)[NS][kP], f32x4 (&o)[NI]) {
        bf16x8 pr[NI][NS][kR];
#pragma unroll
        for (int it = 0; it < NI; ++it)
#pragma unroll
            for (int s = 0; s <= it / 2; ++s)
#pragma unroll
                for (int p = 0; p < kR; ++p) pr[it][s][p] = read_row(&P[p * kPP + tile_at<C>(it * 16 + m, 4 * s + q)]);
        const bool odd = __any(abs_bits(S[0][0]) >= kInfBits);
        if (odd) {
#pragma unroll
            for (int s = 0; s < NS; ++s)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const bool bad = abs_bits((float)z[s][0][i]) >= kInfBits;
#pragma unroll
                    for (int p = 0; p < kP; ++p)
                        if (bad) z[s][p][i] = (bf16)0.0f;
                }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int it = 0; it < NI; ++it)
#pragma unroll
            for (int s = 0; s <= it / 2; ++s) o[it] = mfma_planes(z[s], pr[it][s], o[it]);
        if (odd) {
#pragma unroll 1
            for (int j = 0; j < cnt; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int c = oc + r;
                    const float zv = (float)Z[tile_at<kNB>(j, c >> 3) + (c & 7)];  // the first plane is as little finite
                    if (abs_bits(zv) < kInfBits) continue;
#pragma unroll
                    for (int it = 0; it < NI; ++it)
                        if (j <= 16 * it + m)
                            o[it][r] = fmaf((float)P[tile_at<C>(16 * it + m, j >> 3) + (j & 7)], zv, o[it][r]);
                }
        }
    };
    auto write = [&](int i, int cnt, const f32x4 (&o)[NI]) {
        const __amdgpu_buffer_rsrc_t buf = chunk_of(ro, i, cnt, C);
        const uint32_t shift = ro.shift(cnt, C);
#pragma unroll
        for (int it = 0; it < NI; ++it) {
            VecT<T, 4> v;
#pragma unroll
            for (int r = 0; r < 4; ++r) v.v[r] = (T)o[it][r];
            const uint32_t at = out_at + ((uint32_t)it * out_step - shift);
            if (w.out4) {
                if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b64(*reinterpret_cast<u32x2 *>(&v), buf, at, 0, 0);
                else __builtin_amdgcn_raw_buffer_store_b128(*reinterpret_cast<u32x4 *>(&v), buf, at, 0, 0);
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const uint32_t ar = c0 + oc + r < w.d2 ? at + r * (uint32_t)sizeof(T) : kNowhere;
                    if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b16(*reinterpret_cast<uint16_t *>(&v.v[r]), buf, ar, 0, 0);
                    else __builtin_amdgcn_raw_buffer_store_b32(*reinterpret_cast<uint32_t *>(&v.v[r]), buf, ar, 0, 0);
                }
            }
        }
    };

    auto step = [&](int i, int d) {
        const int cnt = positions(i);
        lds_barrier();  // the last chunk's reads are done
        put(d);
        load(i + kDepth, d);
        if constexpr (!VEC) {  // with VEC they have found nothing in the buffer (see view_vec)
            if (cnt < C) {
                // the thread's index is found again: kept for the one chunk that
                // may be short it would take a register in all of them
                uint32_t all = ~0u;
                asm volatile("" : "+s"(all));
                const int thread = wave * 64 + (int)__builtin_amdgcn_mbcnt_hi(all, __builtin_amdgcn_mbcnt_lo(all, 0));
                if (kOut) clear_past<kP, D1, C>(X, thread, cnt);
                clear_past<kP, D1, C>(Y, thread, cnt);
                clear_past<kP, kNB, C>(Z, thread, cnt);
            }
        }
        lds_barrier();
        f32x4 o[NI];
        bf16x8 z[NS][kP];
        products(cnt, cnt == C, z, o);
        if constexpr (kOut) {
            lds_barrier();  // P is whole
            within(cnt, z, o);
            write(i, cnt, o);
        }
    };
    for (int i = 0; i < chunks; i += kDepth)
#pragma unroll
        for (int d = 0; d < kDepth; ++d)
            if (i + d < chunks) step(i + d, d);

    if constexpr (!kOut) {
        f32x4 *dst = seg_state<D1>(a, wh, wh.seg, wave) + lane;
#pragma unroll
        for (int t = 0; t < NA; ++t) dst[t * 64] = S[t];
    } else if (w.fin != nullptr && end == a.L && col < w.d2) {
#pragma unroll
        for (int t = 0; t < NA; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = state_row(t, q, r);
                if (row < w.d1) w.fin[(int64_t)wh.bh * w.d1 * w.d2 + (int64_t)row * w.im + (int64_t)col * w.in] = S[t][r];
            }
    }
}

// From every segment's own part of T to T before every segment, in place: a
// workgroup a 16x16 tile, a thread an element.  Bound by latency (few
// elements, one step a segment), so 16 segments' loads are in flight.
template <int D1>
__global__ __launch_bounds__(kThreads) void join_kernel(WalkArgs a) {
    constexpr int NA = D1 / 16;
    const uint32_t item = blockIdx.x, blk_of = item / (4 * NA), pairs = (uint32_t)(a.B * a.H);
    const int t = (int)(item % NA), wave = (int)(item / NA % 4);
    Where wh;
    wh.blk = (int)(blk_of % (uint32_t)a.nblk);
    wh.bh = (int)(blk_of / (uint32_t)a.nblk % pairs);
    wh.walk = (int)(blk_of / (uint32_t)a.nblk / pairs);
    const Walk &w = a.w[wh.walk];
    if (wh.blk * kNB >= w.d2) return;
    const int lane = threadIdx.x >> 2, r = threadIdx.x & 3;  // whose register this element is
    const int row = state_row(t, lane >> 4, r), col = wh.blk * kNB + wave * 16 + (lane & 15);
    const Carry carry = walk_carry(walk_gate(a.log_decay, wh.bh % (int)a.H), a.seg_len);
    float s = w.init != nullptr && col < w.d2 && row < w.d1
                  ? w.init[(int64_t)wh.bh * w.d1 * w.d2 + (int64_t)row * w.im + (int64_t)col * w.in] : 0.0f;
    s = __builtin_canonicalizef(s);  // no signalling NaN (a launch tag) goes into the workspace
    float *at = reinterpret_cast<float *>(seg_state<D1>(a, wh, 0, wave) + t * 64) + threadIdx.x;
    const int64_t step = 4 * NA * 64 * 4;
    constexpr int U = 16;
    for (int s0 = 0; s0 < a.segs; s0 += U) {
        float own[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s0 + u < a.segs - 1) own[u] = at[(s0 + u) * step];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s0 + u < a.segs) at[(s0 + u) * step] = s;
            if (s0 + u < a.segs - 1) s = carry(s) + own[u];
        }
    }
}

}  // namespace walk
}  // namespace prn
