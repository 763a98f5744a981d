// sequence.hpp -- host entry points of the operators around the recurrences
// (linattn.hip, layernorm.hip, embedding.hip), called by the C ABI (api.hip)
// after argument validation, like those of launch.hpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "launch.hpp"

namespace prn {

// The operators' scratch lies kScratchOffset bytes into the caller's workspace
// (past the ticket header) and holds only results of fp32 arithmetic and
// integers below 2^30, none of which look like a launch tag, so a workspace
// stays ready for every entry point.
constexpr size_t kScratchOffset = 256;

struct LinattnArgs {
    int bf16;
    int64_t B, L, H;
    int dk, dv;
    const void *q, *k, *v, *grad_o;
    int64_t st[4][3];  // strides of q, k, v, grad_o over batch rows, positions and heads
    const float *log_decay, *state;
    float scale;
    void *o;
    float *out_state;
    const float *grad_out_state;
    void *grad_q, *grad_k, *grad_v;
    float *grad_state;
};
hipError_t linattn_forward(const LinattnArgs &a, const Ws &ws, hipStream_t s);
hipError_t linattn_backward(const LinattnArgs &a, const Ws &ws, hipStream_t s);
hipError_t linattn_step(const LinattnArgs &a, hipStream_t s);
// Workspace bytes of a call (only the shape's fields of `a` are read).
size_t linattn_ws(const LinattnArgs &a, bool backward);

struct LayernormFwdArgs {
    int bf16;
    int64_t rows, D;
    const void *x, *residual;
    const float *weight, *bias;
    float eps;
    void *sum, *y;
    float *mean, *rstd;
};
hipError_t layernorm_forward(const LayernormFwdArgs &a, hipStream_t s);
struct LayernormBwdArgs {
    int bf16;
    int64_t rows, D;
    const void *s;
    const float *weight, *mean, *rstd;
    const void *grad_y, *grad_sum;
    void *grad_x;
    float *grad_w, *grad_b;
};
hipError_t layernorm_backward(const LayernormBwdArgs &a, const Ws &ws, hipStream_t s);
// Partial rows of the weight's and bias's gradients (2 D floats each).
int layernorm_parts(int64_t rows, int64_t D);

struct EmbeddingArgs {
    int bf16, wide_ids;
    int64_t N, V, D, padding;  // padding: -1 for none
    const void *ids, *table;   // table: the gradient of the rows in the backward pass
    float scale;
    void *out;
};
hipError_t embedding_forward(const EmbeddingArgs &a, hipStream_t s);
hipError_t embedding_backward(const EmbeddingArgs &a, const Ws &ws, hipStream_t s);
size_t embedding_ws(int64_t N, int64_t D);

}  // namespace prn
