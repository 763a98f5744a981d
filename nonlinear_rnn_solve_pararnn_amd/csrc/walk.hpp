// walk.hpp -- the walk kernel of linear attention (the primitive of
// linattn.hpp) on bf16 matrix instructions, for bf16 and fp32 operands.
//
// Chunks of C positions.  Within a chunk, with the decays applied in fp32:
//   P = (X Y^T) * wi e^(g(i-j)) on and below the diagonal,
//   out = P Z + wo e^(g(i+1-e)) X T,
//   T <- T + T (e^(gC) - 1) + sum_j Y_j^T (wt e^(g(C-1-j+e)) Z_j).
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
// held as three planes throughout.  bf16 operands are one plane: exact as they
// come, and the products X Y^T and Y^T (decayed Z) keep everything because the
// decayed Z is split into three; P and the operand copy of T are rounded to
// bf16 once, which puts an error the size of the result's own rounding on it.
#pragma once

#include "linattn.hpp"

namespace prn {
namespace walk {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kNB = 64;  // columns of Z a workgroup

template <typename T> constexpr int kPlanes = sizeof(T) == 2 ? 1 : 3;

// Element offset of 8-element group `grp` of row `row` in an LDS tile of W
// columns.  Rows of 64, 128 and 256 columns are swizzled so that both the row
// reads (16 rows, one group) and the transposing reads (4 rows, 4 groups) of
// 16 lanes fall on different banks; other widths are padded by one group.
template <int W>
__device__ __forceinline__ int tile_at(int row, int grp) {
    if (W == 128 || W == 256) return row * W + ((grp ^ (((row & 3) << 2) | ((row >> 2) & 3))) << 3);
    if (W == 64) return row * W + ((grp ^ ((((row >> 1) & 1) << 2) | ((row >> 2) & 3))) << 3);
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
template <int N>
__device__ __forceinline__ void to_planes(const float (&f)[8], bf16x8 (&p)[N]) {
    if constexpr (N == 3) split3(f, p);
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
constexpr uint32_t kNowhere = 0x80000000u;  // above every buffer's size, also after a chunk's bytes are taken off

// Rows of one operand as a walk sees them, from column c0 on.
struct Rows {
    const char *p;      // row 0 of the sequence
    int64_t row_bytes;  // below 2^24 (checked on the host)
    uint32_t tail;      // bytes of a row from p on
    int64_t L;
    int rev;

    // Bytes and address of the chunk of cnt positions from p0.
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk(int64_t p0, int cnt) const {
        return buffer_of(p + (rev ? L - p0 - cnt : p0) * row_bytes, (uint32_t)(cnt - 1) * (uint32_t)row_bytes + tail);
    }
    // Offset of a chunk's row r in it, if the chunk is whole; (C - cnt) * row_bytes less in a reversed shorter one.
    __device__ __forceinline__ uint32_t row_at(int r, int C) const { return (uint32_t)(rev ? C - 1 - r : r) * (uint32_t)row_bytes; }
    __device__ __forceinline__ uint32_t shift(int cnt, int C) const { return rev ? (uint32_t)(C - cnt) * (uint32_t)row_bytes : 0u; }
};
template <typename T>
__device__ __forceinline__ Rows rows_of(const WalkView &v, int64_t b, int64_t h, int64_t L, int rev, int c0, int d) {
    return {static_cast<const char *>(v.p) + (b * v.sb + h * v.sh + c0) * (int64_t)sizeof(T), v.st * (int64_t)sizeof(T),
            (uint32_t)(d - c0) * (uint32_t)sizeof(T), L, rev};
}

// A thread's share of one tile of W columns (groups of 8 elements), loaded
// ahead of its use.  VEC: rows are 16-byte aligned and whole numbers of
// 16-byte pieces; otherwise elements are loaded one by one.
template <typename T, int W, int C, bool VEC>
struct Ahead {
    static constexpr int kGroups = W / 8, kN = (C * kGroups + kThreads - 1) / kThreads, kV = 16 / (int)sizeof(T);
    struct alignas(16) {
        T v[8];
    } r[kN];
    uint32_t at[kN];   // offsets in a whole chunk
    int left;          // columns the operand has

    __device__ __forceinline__ void init(const Rows &v) {
        left = (int)(v.tail / sizeof(T));
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            const int i = threadIdx.x + n * kThreads, row = i / kGroups, c = (i - row * kGroups) * 8;
            at[n] = row < C && c < left ? v.row_at(row, C) + c * (uint32_t)sizeof(T) : kNowhere;
        }
    }
    // Positions p0 .. p0 + cnt of the walk; zeros past the ends.
    __device__ __forceinline__ void load(const Rows &v, int64_t p0, int cnt) {
        const __amdgpu_buffer_rsrc_t buf = v.chunk(p0, cnt);
        const uint32_t shift = v.shift(cnt, C);
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            const uint32_t o = at[n] - shift;
            if constexpr (VEC) {
#pragma unroll
                for (int h = 0; h < 8 / kV; ++h) {
                    // the second half of a group may lie past the row's end
                    const uint32_t oh = h == 0 ? o : ((int)((threadIdx.x + n * kThreads) % kGroups) * 8 + h * kV < left ? o + 16 * h : kNowhere);
                    *reinterpret_cast<u32x4 *>(&r[n].v[h * kV]) = __builtin_amdgcn_raw_buffer_load_b128(buf, oh, 0, 0);
                }
            } else {
                const int c = (int)((threadIdx.x + n * kThreads) % kGroups) * 8;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t ok = c + k < left ? o + k * (uint32_t)sizeof(T) : kNowhere;
                    if constexpr (sizeof(T) == 2) {
                        const uint16_t x = __builtin_amdgcn_raw_buffer_load_b16(buf, ok, 0, 0);
                        r[n].v[k] = *reinterpret_cast<const T *>(&x);
                    } else {
                        const uint32_t x = __builtin_amdgcn_raw_buffer_load_b32(buf, ok, 0, 0);
                        r[n].v[k] = *reinterpret_cast<const T *>(&x);
                    }
                }
            }
        }
    }

    __device__ __forceinline__ void store(bf16 *lds) const {
        constexpr int kP = kPlanes<T>, kPlane = C * kTileRow<W>;
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            const int i = threadIdx.x + n * kThreads, row = i / kGroups, grp = i - row * kGroups;
            if (C * kGroups % kThreads != 0 && row >= C) continue;
            bf16x8 p[kP];
            if constexpr (kP == 1) {
                p[0] = *reinterpret_cast<const bf16x8 *>(&r[n].v[0]);
            } else {
                float f[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] = (float)r[n].v[k];
                split3(f, p);
            }
#pragma unroll
            for (int k = 0; k < kP; ++k) *reinterpret_cast<bf16x8 *>(lds + k * kPlane + tile_at<W>(row, grp)) = p[k];
        }
    }
};

// Which part of the work a workgroup does.
struct Where {
    int64_t bh, b, h;
    int walk, blk, seg;
    bool any;
};
// (batch row, head) pairs in groups of 8, then everything that reads the
// same rows: consecutive workgroups go to the 8 XCDs in turn, so all blocks of
// one pair meet in one L2.
__device__ __forceinline__ Where where(const WalkArgs &a, int segs) {
    const int64_t per = (int64_t)a.walks * a.nblk * segs;
    const int64_t grp = (int64_t)blockIdx.x / (8 * per), rest = (int64_t)blockIdx.x - grp * 8 * per;
    Where w;
    w.bh = grp * 8 + (rest & 7);
    const int sub = (int)(rest >> 3), pair = sub / segs;
    w.seg = sub - pair * segs;
    w.walk = pair / a.nblk;
    w.blk = pair - w.walk * a.nblk;
    w.b = w.bh / a.H;
    w.h = w.bh - w.b * a.H;
    w.any = w.bh < a.B * a.H && w.blk * kNB < a.w[w.walk].d2;
    return w;
}

// Where segment states are kept between the launches: the registers of wave
// `wave` of a block, tile by tile.
template <int D1>
__device__ __forceinline__ f32x4 *seg_state(const WalkArgs &a, const Where &w, int seg, int wave) {
    const int64_t slot = (((int64_t)w.walk * a.B * a.H + w.bh) * a.nblk + w.blk) * a.segs + seg;
    return reinterpret_cast<f32x4 *>(a.seg_state) + (slot * 4 + wave) * (D1 / 16) * 64;
}
// Row of T that register r of tile t holds in lanes of group q.
__device__ __forceinline__ int state_row(int t, int q, int r) { return 32 * (t >> 1) + 8 * q + 4 * (t & 1) + r; }

// STATE: only the segment's own part of T (from zero), for the join.
template <typename T, int D1, int C, bool VEC, bool STATE>
__global__ __launch_bounds__(kThreads, D1 > 128 ? 1 : 2) void walk_kernel(WalkArgs a) {
    constexpr int kP = kPlanes<T>;                 // planes of X, Y, Z, P
    constexpr int kS = kP == 1 ? 1 : 3;            // planes of the operand copy of T
    constexpr int NA = D1 / 16, NT = D1 / 32, NS = C / 32, NI = C / 16;
    constexpr int kPX = C * kTileRow<D1>, kPZ = C * kTileRow<kNB>, kPP = C * kTileRow<C>;
    __shared__ __align__(16) bf16 X[STATE ? 8 : kP * kPX], Y[kP * kPX], Z[kP * kPZ], P[STATE ? 8 : kP * kPP];
    const Where wh = where(a, STATE ? a.segs - 1 : a.segs);
    if (!wh.any) return;
    const Walk &w = a.w[wh.walk];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, m = lane & 15, q = lane >> 4;
    const int tr_i = m >> 2, tr_c = m & 3;         // this lane's row and column group in a transposing read
    const int c0 = wh.blk * kNB, col = c0 + wave * 16 + m;
    const float g = walk_gate(a.log_decay, wh.h), g2 = g * kLog2e;
    const int64_t begin = (int64_t)wh.seg * a.seg_len, end = min(a.L, begin + a.seg_len);

    f32x4 S[NA];
    if (!STATE && a.segs > 1) {
        const f32x4 *src = seg_state<D1>(a, wh, wh.seg, wave) + lane;
#pragma unroll
        for (int t = 0; t < NA; ++t) S[t] = src[t * 64];
    } else {
#pragma unroll
        for (int t = 0; t < NA; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = state_row(t, q, r);
                S[t][r] = !STATE && w.init != nullptr && col < w.d2 && row < w.d1
                              ? w.init[wh.bh * w.d1 * w.d2 + (int64_t)row * w.im + (int64_t)col * w.in] : 0.0f;
            }
    }

    // decays: of P's elements in tiles on the diagonal and one below it, of a
    // row's share of T, of the positions' shares of T
    float dec_d[4], dec_o[4], dec_row[NI], dec_z[NS][8];
    const float dec16 = fast_exp2(16.0f * g2);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int n = m - 4 * q - r;
        dec_d[r] = n >= 0 ? w.wi * fast_exp2(g2 * (float)n) : 0.0f;
        dec_o[r] = w.wi * fast_exp2(g2 * (float)(n + 16));
    }
#pragma unroll
    for (int it = 0; it < NI; ++it) dec_row[it] = w.wo * fast_exp2(g2 * (float)(16 * it + m + 1 - w.e));
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) dec_z[s][i] = w.wt * fast_exp2(g2 * (float)(C - 1 - 32 * s - 8 * q - i + w.e));
    const float em1_full = walk_em1(g, C);

    if constexpr (!STATE) {
        // the tiles of P right of the diagonal that share a 32-wide read with it stay zero
        for (int i = threadIdx.x; i < kP * kPP / 8; i += kThreads) {
            const bf16x8 z = {};
            *reinterpret_cast<bf16x8 *>(&P[i * 8]) = z;
        }
    }

    const Rows rx = rows_of<T>(w.X, wh.b, wh.h, a.L, w.rev, 0, w.d1), ry = rows_of<T>(w.Y, wh.b, wh.h, a.L, w.rev, 0, w.d1),
               rz = rows_of<T>(w.Z, wh.b, wh.h, a.L, w.rev, c0, w.d2);
    const Rows ro = rows_of<T>({w.out, a.L * a.H * w.d2, a.H * w.d2, w.d2}, wh.b, wh.h, a.L, w.rev, c0, w.d2);
    Ahead<T, D1, C, VEC> ax, ay;
    Ahead<T, kNB, C, VEC> az;
    const int first = (int)min((int64_t)C, end - begin);
    if (!STATE) {
        ax.init(rx);
        ax.load(rx, begin, first);
    }
    ay.init(ry);
    ay.load(ry, begin, first);
    az.init(rz);
    az.load(rz, begin, first);
    uint32_t out_at[NI];  // this lane's row of each 16-row tile of out, four columns from its own
    const int oc = wave * 16 + 4 * q;
#pragma unroll
    for (int it = 0; it < NI; ++it)
        out_at[it] = c0 + oc < w.d2 ? ro.row_at(16 * it + m, C) + oc * (uint32_t)sizeof(T) : kNowhere;

    for (int64_t p0 = begin; p0 < end; p0 += C) {
        const int cnt = (int)min((int64_t)C, end - p0);
        lds_barrier();  // the last chunk's reads are done
        if (!STATE) ax.store(X);
        ay.store(Y);
        az.store(Z);
        if (p0 + C < end) {
            const int next = (int)min((int64_t)C, end - p0 - C);
            if (!STATE) ax.load(rx, p0 + C, next);
            ay.load(ry, p0 + C, next);
            az.load(rz, p0 + C, next);
        }
        lds_barrier();

        f32x4 o[NI];
        if constexpr (!STATE) {
            // P, a tile's transpose at a time (a lane's results are then four
            // consecutive j); the NI (NI + 1) / 2 tiles go round the waves
            constexpr int kTiles = NI * (NI + 1) / 2;
#pragma unroll
            for (int k = 0; k < (kTiles + 3) / 4; ++k) {
                const int tile = wave + 4 * k;
                if (tile < kTiles) {
                    const int it = tile < 1 ? 0 : tile < 3 ? 1 : tile < 6 ? 2 : 3, jt = tile - it * (it + 1) / 2;
                    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        bf16x8 y[kP], x[kP];
#pragma unroll
                        for (int p = 0; p < kP; ++p) {
                            y[p] = read_row(&Y[p * kPX + tile_at<D1>(jt * 16 + m, 4 * t + q)]);
                            x[p] = read_row(&X[p * kPX + tile_at<D1>(it * 16 + m, 4 * t + q)]);
                        }
                        acc = mfma_planes(y, x, acc);
                    }
                    const float far = it - jt == 3 ? dec16 * dec16 : it - jt == 2 ? dec16 : 1.0f;
                    float f[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        f[r] = it == jt ? acc[r] * dec_d[r] : acc[r] * (dec_o[r] * far);
                        if (it == jt && m < 4 * q + r) f[r] = 0.0f;  // whatever Y holds there
                    }
                    bf16 *to = &P[tile_at<C>(it * 16 + m, 2 * jt + (q >> 1)) + 4 * (q & 1)];
                    if constexpr (kP == 1) {
                        VecT<bf16, 4> v;
#pragma unroll
                        for (int r = 0; r < 4; ++r) v.v[r] = (bf16)f[r];
                        *reinterpret_cast<VecT<bf16, 4> *>(to) = v;
                    } else {
                        const float f8[8] = {f[0], f[1], f[2], f[3], 0.0f, 0.0f, 0.0f, 0.0f};
                        bf16x8 p[3];
                        split3(f8, p);
#pragma unroll
                        for (int k2 = 0; k2 < 3; ++k2)
                            *reinterpret_cast<u32x2 *>(to + k2 * kPP) = *reinterpret_cast<const u32x2 *>(&p[k2]);
                    }
                }
            }
            // the rows' share of T, transposed: lane m is position 16 it + m, registers four columns
#pragma unroll
            for (int it = 0; it < NI; ++it) o[it] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float f[8] = {S[2 * t][0],     S[2 * t][1],     S[2 * t][2],     S[2 * t][3],
                                    S[2 * t + 1][0], S[2 * t + 1][1], S[2 * t + 1][2], S[2 * t + 1][3]};
                bf16x8 sp[kS];
                to_planes(f, sp);
#pragma unroll
                for (int it = 0; it < NI; ++it) {
                    bf16x8 x[kP];
#pragma unroll
                    for (int p = 0; p < kP; ++p) x[p] = read_row(&X[p * kPX + tile_at<D1>(it * 16 + m, 4 * t + q)]);
                    o[it] = mfma_planes(sp, x, o[it]);
                }
            }
#pragma unroll
            for (int it = 0; it < NI; ++it)
#pragma unroll
                for (int r = 0; r < 4; ++r) o[it][r] *= dec_row[it];
        }

        // T over the chunk
        const float em1 = cnt == C ? em1_full : walk_em1(g, cnt);
#pragma unroll
        for (int t = 0; t < NA; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[t][r] = fmaf(S[t][r], em1, S[t][r]);
        bf16x8 z[NS][kP];
#pragma unroll
        for (int s = 0; s < NS; ++s) {
#pragma unroll
            for (int p = 0; p < kP; ++p) {
                const int row = 32 * s + 8 * q + tr_i, grp = 2 * wave + (tr_c >> 1), in = 4 * (tr_c & 1);
                z[s][p] = join(read_tr(&Z[p * kPZ + tile_at<kNB>(row, grp) + in]),
                               read_tr(&Z[p * kPZ + tile_at<kNB>(row + 4, grp) + in]));
            }
            float f[8];
            if (cnt == C) {
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = plane_sum(z[s], i) * dec_z[s][i];
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int n = cnt - 1 - (32 * s + 8 * q + i);
                    f[i] = n >= 0 ? plane_sum(z[s], i) * (w.wt * fast_exp2(g2 * (float)(n + w.e))) : 0.0f;
                }
            }
            bf16x8 zw[3];
            split3(f, zw);
#pragma unroll
            for (int t = 0; t < NA; ++t) {
                bf16x8 y[kP];
#pragma unroll
                for (int p = 0; p < kP; ++p) {
                    const int row = 32 * s + 8 * q + tr_i, grp = 4 * (t >> 1) + tr_c, in = 4 * (t & 1);
                    y[p] = join(read_tr(&Y[p * kPX + tile_at<D1>(row, grp) + in]),
                                read_tr(&Y[p * kPX + tile_at<D1>(row + 4, grp) + in]));
                }
                S[t] = mfma_planes(y, zw, S[t]);
            }
        }

        if constexpr (!STATE) {
            lds_barrier();  // P is whole
            // an infinity or NaN of Z has made T so, in its column's every row
            const bool odd = __any(abs_bits(S[0][0]) >= kInfBits);
            if (odd) {
                // values of Z that are not finite must not reach earlier
                // positions through a zero of P: they are left out here and
                // added to the positions from their own on below
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
#pragma unroll
            for (int it = 0; it < NI; ++it)
#pragma unroll
                for (int s = 0; s <= it / 2; ++s) {
                    bf16x8 pr[kP];
#pragma unroll
                    for (int p = 0; p < kP; ++p) pr[p] = read_row(&P[p * kPP + tile_at<C>(it * 16 + m, 4 * s + q)]);
                    o[it] = mfma_planes(z[s], pr, o[it]);
                }
            if (odd) {
                for (int j = 0; j < cnt; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int c = wave * 16 + 4 * q + r;
                        const float zv = (float)Z[tile_at<kNB>(j, c >> 3) + (c & 7)];  // the first plane is as little finite
                        if (abs_bits(zv) < kInfBits) continue;
#pragma unroll
                        for (int it = 0; it < NI; ++it)
                            if (j <= 16 * it + m)
                                o[it][r] = fmaf((float)P[tile_at<C>(16 * it + m, j >> 3) + (j & 7)], zv, o[it][r]);
                    }
            }
            const __amdgpu_buffer_rsrc_t buf = ro.chunk(p0, cnt);
            const uint32_t shift = ro.shift(cnt, C);
#pragma unroll
            for (int it = 0; it < NI; ++it) {
                VecT<T, 4> v;
#pragma unroll
                for (int r = 0; r < 4; ++r) v.v[r] = (T)o[it][r];
                const uint32_t at = out_at[it] - shift;
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
        }
    }

    if constexpr (STATE) {
        f32x4 *dst = seg_state<D1>(a, wh, wh.seg, wave) + lane;
#pragma unroll
        for (int t = 0; t < NA; ++t) dst[t * 64] = S[t];
    } else if (w.fin != nullptr && end == a.L && col < w.d2) {
#pragma unroll
        for (int t = 0; t < NA; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = state_row(t, q, r);
                if (row < w.d1) w.fin[wh.bh * w.d1 * w.d2 + (int64_t)row * w.im + (int64_t)col * w.in] = S[t][r];
            }
    }
}

// From every segment's own part of T to T before every segment, in place.
template <int D1>
__global__ __launch_bounds__(kThreads) void join_kernel(WalkArgs a) {
    constexpr int NA = D1 / 16;
    const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);  // one tile of one wave of one block
    const int64_t tiles = (int64_t)a.walks * a.B * a.H * a.nblk * 4 * NA;
    if (item >= tiles) return;
    const int t = (int)(item % NA), wave = (int)(item / NA % 4);
    const int64_t blk_of = item / (4 * NA);
    Where wh;
    wh.blk = (int)(blk_of % a.nblk);
    wh.bh = blk_of / a.nblk % (a.B * a.H);
    wh.walk = (int)(blk_of / a.nblk / (a.B * a.H));
    const Walk &w = a.w[wh.walk];
    if (wh.blk * kNB >= w.d2) return;
    const int lane = threadIdx.x & 63, m = lane & 15, q = lane >> 4, col = wh.blk * kNB + wave * 16 + m;
    const float em1 = walk_em1(walk_gate(a.log_decay, wh.bh % a.H), a.seg_len);
    f32x4 s;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int row = state_row(t, q, r);
        s[r] = w.init != nullptr && col < w.d2 && row < w.d1
                   ? w.init[wh.bh * w.d1 * w.d2 + (int64_t)row * w.im + (int64_t)col * w.in] : 0.0f;
    }
    f32x4 *at = seg_state<D1>(a, wh, 0, wave) + t * 64 + lane;
    const int64_t step = 4 * NA * 64;
    constexpr int U = 8;
    for (int s0 = 0; s0 < a.segs; s0 += U) {
        f32x4 own[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s0 + u < a.segs - 1) own[u] = at[(s0 + u) * step];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s0 + u < a.segs) at[(s0 + u) * step] = s;
            if (s0 + u < a.segs - 1)
#pragma unroll
                for (int r = 0; r < 4; ++r) s[r] = fmaf(s[r], em1, s[r]) + own[u][r];
        }
    }
}

}  // namespace walk
}  // namespace prn
