// linattn.hpp -- linear attention with a decay per head as one primitive, the
// walk, that the forward pass and all three gradients are instances of.
//
// With positions p = 0 .. L-1 in the walk's order (reversed in time for two
// of the gradients), gates g = log decay of the head and e in {0, 1}:
//   out_p = wi sum_{r<=p} e^(g(p-r)) (X_p.Y_r) Z_r + wo e^(g(p+1-e)) X_p T_0
//   T_end = e^(gL) T_0 + wt sum_r e^(g(L-1-r+e)) Y_r^T Z_r
// per batch row and head, X, Y of width d1, Z and out of width d2, T [d1, d2]:
//   o   X, Y, Z = q, k, v            e = 0, T = S
//   dq  X, Y, Z = do, v, k           e = 0, T = S^T
//   dk  X, Y, Z = v, do, q reversed  e = 1, T = D^T
//   dv  X, Y, Z = k, q, do reversed  e = 1, T = D
// S_t = e^g S_{t-1} + k_t^T v_t is the state, D_t = dLoss/dS_t; a reversed
// walk carries e^g D, so that the gradient of the final state enters with
// weight 1 and the walk ends on the gradient of the initial state.
#pragma once

#include "rows.hpp"
#include "sequence.hpp"

namespace prn {

// One operand: element (b, t, h, i) is p[b sb + t st + h sh + i].
struct WalkView {
    const void *p;
    int64_t sb, st, sh;
};

struct Walk {
    WalkView X, Y, Z;
    void *out;          // dense [B, L, H, d2]
    const float *init;  // T_0 or null for zeros; element (m, n) of a (b, h) at m im + n in
    float *fin;         // T_end or null, same layout as init
    int im, in;
    int d1, d2;
    int rev, e;
    float wi, wo, wt;
    int out4;           // rows of out may be stored four elements at a time
};

struct WalkArgs {
    Walk w[3];
    int walks;
    int64_t B, L, H;
    const float *log_decay;
    int nblk;   // column blocks of 64 a walk, at most
    int segs;          // pieces of the sequence that are walked side by side
    int64_t seg_len;   // positions a piece (a multiple of the chunk)
    float *seg_state;  // T of every piece, in the walk's register layout
};

// The head's decay, kept above -infinity so that 0 * g is 0 (a NaN stays one).
__device__ __forceinline__ float walk_gate(const float *log_decay, int64_t h) {
    const float g = log_decay[h];
    return g < -1e30f ? -1e30f : g;
}

// The state's factor over n positions, in double and rounded once.  Slow decays
// are carried as T + T (e^(g n) - 1), whose rounding does not repeat from chunk
// to chunk the way that of a factor near 1 does; where less than half is left,
// e^(g n) itself is the factor, as what is left of T + T (e^(g n) - 1) would be
// that factor's rounding error of 2^-25.
struct Carry {
    float f;
    bool fast;
    __device__ __forceinline__ float operator()(float t) const { return fast ? t * f : fmaf(t, f, t); }
};
__device__ __forceinline__ Carry walk_carry(float g, int64_t n) {
    const double e = exp((double)g * (double)n);  // e - 1 is off by 2^-53 of T, whatever its size
    const bool fast = e < 0.5;
    const float f = (float)(fast ? e : e - 1.0);
    // the same in every lane
    return {__uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(f))), (bool)__builtin_amdgcn_readfirstlane(fast)};
}

}  // namespace prn
