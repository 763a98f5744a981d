// mixer.hpp -- host entry points of the operators of a delta-rule mixer
// (delta.hip, headnorm.hip), called by the C ABI (api.hip) after argument
// validation, like those of sequence.hpp.
#pragma once

#include "sequence.hpp"

namespace prn {

// One operand: element (b, t, h, i) is p[b st[0] + t st[1] + h st[2] + i].
struct HeadView {
    const void *p;
    int64_t st[3];
};

struct DeltaArgs {
    int bf16;
    int64_t B, L, H, Hk;  // Hk divides H: head h of v shares head h / (H / Hk) of q and k
    int dk, dv;
    HeadView q, k, v, grad_o;
    HeadView log_decay, beta;  // fp32, one element a head
    const float *state;
    float scale;
    void *o;
    float *out_state;
    const float *grad_out_state;
    void *grad_q, *grad_k, *grad_v;
    float *grad_log_decay, *grad_beta, *grad_state;
};
hipError_t delta_forward(const DeltaArgs &a, const Ws &ws, hipStream_t s);
hipError_t delta_backward(const DeltaArgs &a, const Ws &ws, hipStream_t s);
hipError_t delta_step(const DeltaArgs &a, hipStream_t s);
// Workspace bytes of a call (only the shape's fields of `a` are read).
size_t delta_ws(const DeltaArgs &a, bool backward);

struct HeadnormArgs {
    int bf16;
    int64_t B, L, Hq, Hk;  // Hk = 0: no second tensor
    int d, R;
    int l2, interleaved;
    HeadView x[2], g[2];   // inputs and (backward) gradients of the outputs: queries, keys
    const float *w[2];
    const float *table;    // [P, R]: cosines, then sines, or null
    int64_t P;
    const void *positions; // [B, L] or null: position t of a row is its own index
    int wide;              // positions have 64 bits
    float eps;
    void *y[2];            // outputs, or gradients of the inputs
    float *r[2];           // 1 / norm of every row: an output of the forward pass
    float *gw[2];
};
hipError_t headnorm_forward(const HeadnormArgs &a, hipStream_t s);
hipError_t headnorm_backward(const HeadnormArgs &a, const Ws &ws, hipStream_t s);
size_t headnorm_ws(const HeadnormArgs &a);

}  // namespace prn
