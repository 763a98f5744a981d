// api.hip -- the C ABI declared in include/pararnn.h: host-side argument
// validation, workspace checks and dispatch to the kernel launchers.
#include <math.h>
#include <stdlib.h>
#include <string.h>

#include "pararnn.h"
#include "launch.hpp"
#include "sequence.hpp"

using namespace prn;

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 40;

bool dims_ok(int64_t B, int64_t L, int64_t H) {
    if (B <= 0 || L <= 0 || H <= 0) return false;
    if (B > kMaxDim || L > kMaxDim || H > kMaxDim) return false;
    // B*L*H elements must be addressable and the grid must fit in 2^31 blocks
    const double n = (double)B * (double)L * (double)H;
    return n < 9.0e15;
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

int status_of(hipError_t e) { return e == hipSuccess ? PARARNN_OK : PARARNN_ERR_HIP; }

bool grid_ok(int64_t ntiles) { return ntiles > 0 && ntiles < ((int64_t)1 << 31); }

// Whether the n-float arrays at p and q share any byte (a null one shares none).
bool overlaps(const float *p, const float *q, int64_t n) {
    if (p == nullptr || q == nullptr) return false;
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q, len = (uintptr_t)n * sizeof(float);
    return a < b + len && b < a + len;
}

// Zeros for trace entries [from, to) that no iteration will write.
int clear_trace_tail(float *trace, int32_t from, int32_t to, hipStream_t s) {
    FillRange fr[1] = {{trace + from, (uint64_t)(to - from), 0, 4}};
    return status_of(fill(fr, 1, s));
}

// Newton from zero reproduces the sequential result after L iterations (and
// iteration L + 1 confirms it with a zero update), so caps above L + 1 change
// nothing but the number of launches: they are taken as L + 1 (a trace still
// receives zeros up to the caller's cap).
int32_t eff_cap(int32_t max_iter, int64_t L) {
    return (int64_t)max_iter > L + 1 ? (int32_t)(L + 1) : max_iter;
}

// The chained kernel keeps records of every iteration, so its workspace
// grows with the cap; above kChainMaxCap the per-iteration path is used.
bool chain_ok(int32_t cap) { return cap <= kChainMaxCap; }


// Path of a Newton forward.  The GRU takes the fused on-chip kernel while
// the sequence fits one workgroup's registers; longer sequences (and the
// LSTM) take the chained kernel, which keeps each chunk on chip for all its
// iterations, unless the cap is above kChainMaxCap.  The chained kernel lets
// each workgroup own whole chains of chunks when there are at least as many
// chains as workgroup slots, and chains chunks across workgroups otherwise.
// PARARNN_GRU_PATH=fused|chain|local|step and PARARNN_LSTM_PATH=chain|local|step
// override the choice (for testing every path; "chain" and "local" force the
// two forms of the chained kernel, "local" only with channel lanes; a chain
// request above kChainMaxCap still takes the per-iteration path).
enum class Path { Fused, Chain, Step, Invalid };
Path env_path(const char *name) {
    const char *env = getenv(name);
    if (env == nullptr) return Path::Invalid;
    if (strcmp(env, "fused") == 0) return Path::Fused;
    if (strcmp(env, "chain") == 0 || strcmp(env, "local") == 0) return Path::Chain;
    if (strcmp(env, "step") == 0) return Path::Step;
    return Path::Invalid;
}
// Form of the chained kernel: 1 workgroups own whole chains, 0 chunks are
// chained across workgroups, -1 chosen from the shape.
int env_chain_local(const char *name) {
    const char *env = getenv(name);
    if (env == nullptr) return -1;
    if (strcmp(env, "local") == 0) return 1;
    if (strcmp(env, "chain") == 0) return 0;
    return -1;
}
Path gru_path(int64_t L, int32_t cap) {
    const bool fits = fused_c_for(L) != 0;
    const Path p = env_path("PARARNN_GRU_PATH");
    if (p == Path::Fused) return fits ? Path::Fused : Path::Invalid;
    if (p == Path::Step) return p;
    if (p == Path::Chain) return chain_ok(cap) ? p : Path::Step;
    return fits ? Path::Fused : (chain_ok(cap) ? Path::Chain : Path::Step);
}
Path lstm_path(int32_t cap) {
    const Path p = env_path("PARARNN_LSTM_PATH");
    return (p == Path::Step || !chain_ok(cap)) ? Path::Step : Path::Chain;
}

// Workspace of a Newton forward: that of the kernel the call takes (the
// fused kernel and the chained kernel's whole-chain form use none; the query
// returns the 256-byte minimum for them).
constexpr size_t kMinWs = 256;
size_t gru_fwd_ws(int64_t B, int64_t L, int64_t H, int32_t cap) {
    switch (gru_path(L, cap)) {
        case Path::Chain:
            if (gru_chain_owns_chains(B, L, H, env_chain_local("PARARNN_GRU_PATH"))) return kMinWs;
            return chain_ws(kCfgGruChain, 1, B, L, H, cap).total;
        case Path::Step: return newton_ws(kCfgGruStep, 1, B, L, H, cap).total;
        default: return kMinWs;
    }
}
// The 4x4 blocks take the lane-group kernel (blkrow.hip) unless
// PARARNN_BLK4_PATH=thread asks for the one-thread-per-block scan.
bool blk4_rows() {
    const char *env = getenv("PARARNN_BLK4_PATH");
    return !(env != nullptr && strcmp(env, "thread") == 0);
}
size_t blk4_ws(int64_t B, int64_t L, int64_t H) {
    return blk4_rows() ? blkrow_ws(4, B, L, H).total : scan_ws(kCfgLinBlk4, 4, B, L, H).total;
}

size_t lstm_fwd_ws(int64_t B, int64_t L, int64_t H, int32_t cap) {
    if (lstm_path(cap) == Path::Step) return newton_ws(kCfgLstmStep, 2, B, L, H, cap).total;
    if (lstm_chain_owns_chains(B, L, H, env_chain_local("PARARNN_LSTM_PATH"))) return kMinWs;
    return chain_ws(kCfgLstmChain, 2, B, L, H, cap).total;
}

// ---- operators around the recurrences: sizes and operand strides
constexpr int64_t kMaxHeadDim = 256;

bool type_ok(int32_t dtype) { return dtype == PARARNN_F32 || dtype == PARARNN_BF16; }

constexpr int64_t kMaxRowBytes = (int64_t)1 << 24;  // a chunk of 64 rows stays within 32-bit offsets

// A launch counts its threads in 32 bits: workgroups of 256.
bool blocks_ok(int64_t n) { return n < (int64_t)1 << 24; }

// What a call launches: the walk of the outputs, the gradients' three, or the token's step.
enum class LinattnPass { Forward, Backward, Step };

bool linattn_dims_ok(LinattnPass pass, int32_t dtype, int64_t B, int64_t L, int64_t H, int64_t dk, int64_t dv) {
    if (!type_ok(dtype) || dk < 1 || dk > kMaxHeadDim || dv < 1 || dv > kMaxHeadDim) return false;
    auto blocks = [](int64_t cols) { return (cols + 63) / 64; };
    // workgroups a (batch row, head); sequences are cut into segments only where there are few of them
    const int64_t per = pass == LinattnPass::Forward ? blocks(dv) : pass == LinattnPass::Backward ? 3 * blocks(std::max(dk, dv)) : 1;
    return dims_ok(B, L, H) && dims_ok(B, L, H * kMaxHeadDim) && blocks_ok((B * H + 7) * per) &&
           H * std::max(dk, dv) * 4 < kMaxRowBytes;
}

LinattnArgs linattn_shape(int32_t dtype, int64_t B, int64_t L, int64_t H, int64_t dk, int64_t dv) {
    LinattnArgs a{};
    a.bf16 = dtype == PARARNN_BF16;
    a.B = B;
    a.L = L;
    a.H = H;
    a.dk = (int)dk;
    a.dv = (int)dv;
    return a;
}

// Operands q, k, v (and grad_o) with their strides over (batch row, position,
// head), dense if none are given; false where a pointer is not aligned to its
// elements, or a stride is negative or (of a position) too large.
bool linattn_inputs(LinattnArgs &a, const void *const *in, int n, const int64_t *strides) {
    const void **to[4] = {&a.q, &a.k, &a.v, &a.grad_o};
    for (int i = 0; i < n; ++i) {
        *to[i] = in[i];
        if (!aligned(in[i], a.bf16 ? 2 : 4)) return false;
        const int64_t d = i < 2 ? a.dk : a.dv;
        for (int j = 0; j < 3; ++j) {
            a.st[i][j] = strides ? strides[i * 3 + j] : (j == 0 ? a.L * a.H * d : j == 1 ? a.H * d : d);
            if (a.st[i][j] < 0 || (j == 1 && a.st[i][j] * 4 >= kMaxRowBytes)) return false;
        }
    }
    return true;
}

// Whether the states' in- and output share memory without being the same.
bool states_cross(const LinattnArgs &a, const float *in, const float *out) {
    return in != out && overlaps(in, out, a.B * a.H * a.dk * a.dv);
}

bool layernorm_dims_ok(int32_t dtype, int64_t rows, int64_t D) {
    return type_ok(dtype) && dims_ok(rows, D, 1) && D < ((int64_t)1 << 24);
}

bool embedding_dims_ok(int32_t dtype, int64_t N, int64_t V, int64_t D) {
    const int64_t most = (int64_t)1 << 30;
    // the lookup takes at least 16 rows a workgroup, the sums four times 64
    // positions (fewer where that makes few workgroups) of at least 64 columns
    return type_ok(dtype) && dims_ok(N, D, 1) && dims_ok(V, D, 1) && N < most && V < most && D < ((int64_t)1 << 24) &&
           blocks_ok(N / 16 + 1) && blocks_ok((N / 64 + 1) * (D / 64 + 1) / 4 + 32768);
}

}  // namespace

extern "C" {

const char *pararnn_status_string(int status) {
    switch (status) {
        case PARARNN_OK: return "ok";
        case PARARNN_ERR_INVALID: return "invalid argument";
        case PARARNN_ERR_HIP: return "HIP error";
        case PARARNN_ERR_UNSUPPORTED: return "unsupported";
        case PARARNN_ERR_TOO_LARGE: return "needs more scratch than the library's static buffer holds";
        default: return "unknown status";
    }
}

size_t pararnn_workspace_bytes(int32_t op, int64_t B, int64_t L, int64_t H, int32_t max_iter) {
    if (!dims_ok(B, L, H)) return 0;
    switch (op) {
        case PARARNN_OP_LINSCAN_DIAG: return scan_ws(kCfgLinDiag, 1, B, L, H).total;
        case PARARNN_OP_LINSCAN_BLK2: return scan_ws(kCfgLinBlk2, 2, B, L, H).total;
        case PARARNN_OP_GRU_FORWARD:
            if (max_iter < 1) return 0;
            return gru_fwd_ws(B, L, H, eff_cap(max_iter, L));
        case PARARNN_OP_LSTM_FORWARD:
            if (max_iter < 1) return 0;
            return lstm_fwd_ws(B, L, H, eff_cap(max_iter, L));
        case PARARNN_OP_LINSCAN_BLK4: return blk4_ws(B, L, H);
        case PARARNN_OP_LINSCAN_BLK8: return blkrow_ws(8, B, L, H).total;
        case PARARNN_OP_HGRU4_FORWARD:
        case PARARNN_OP_HGRU8_FORWARD: {
            const int k = op == PARARNN_OP_HGRU8_FORWARD ? 8 : 4;
            if (max_iter < 1 || !dims_ok(B, L, H * k)) return 0;
            return hgru_ws(k, B, L, H, eff_cap(max_iter, L)).total;
        }
        case PARARNN_OP_HGRU4_BACKWARD:
        case PARARNN_OP_HGRU8_BACKWARD: {
            const int k = op == PARARNN_OP_HGRU8_BACKWARD ? 8 : 4;
            if (!dims_ok(B, L, H * k)) return 0;
            return hgru_adj_ws(k, B, L, H).total;
        }
        case PARARNN_OP_GRU_ADJOINT: return gru_adjoint_ws(B, L, H);
        case PARARNN_OP_LSTM_ADJOINT: return lstm_adjoint_ws(B, L, H);
        default: return 0;
    }
}

int rnn_linscan_diag(int64_t B, int64_t L, int64_t H, const float *a, const float *b,
                     const float *h0, float *h, void *ws, size_t ws_bytes, void *stream) {
    if (!dims_ok(B, L, H) || !a || !b || !h || !ws) return PARARNN_ERR_INVALID;
    if (!grid_ok(scan_shape(kCfgLinDiag, B, L, H).ntiles)) return PARARNN_ERR_INVALID;
    if (ws_bytes < scan_ws(kCfgLinDiag, 1, B, L, H).total || !aligned(ws, 256)) return PARARNN_ERR_INVALID;
    return status_of(linscan_diag(B, L, H, a, b, h0, h, Ws{static_cast<char *>(ws), ws_bytes},
                                  static_cast<hipStream_t>(stream)));
}

int rnn_linscan_blk2(int64_t B, int64_t L, int64_t H, const float *A, const float *b,
                     const float *h0, float *h, void *ws, size_t ws_bytes, void *stream) {
    if (!dims_ok(B, L, H) || !A || !b || !h || !ws) return PARARNN_ERR_INVALID;
    if (!aligned(A, 4) || !aligned(b, 4) || !aligned(h, 4) || (h0 && !aligned(h0, 4)))
        return PARARNN_ERR_INVALID;
    if (!grid_ok(scan_shape(kCfgLinBlk2, B, L, H).ntiles)) return PARARNN_ERR_INVALID;
    if (ws_bytes < scan_ws(kCfgLinBlk2, 2, B, L, H).total || !aligned(ws, 256)) return PARARNN_ERR_INVALID;
    return status_of(linscan_blk2(B, L, H, A, b, h0, h, Ws{static_cast<char *>(ws), ws_bytes},
                                  static_cast<hipStream_t>(stream)));
}

int rnn_linscan_blk(int32_t k, int64_t B, int64_t L, int64_t H, const float *A, const float *b,
                    const float *h0, float *h, void *ws, size_t ws_bytes, void *stream) {
    if (k == 2) return rnn_linscan_blk2(B, L, H, A, b, h0, h, ws, ws_bytes, stream);
    if (k < 1) return PARARNN_ERR_INVALID;
    if (k != 4 && k != 8) return PARARNN_ERR_UNSUPPORTED;
    if (!dims_ok(B, L, H) || !A || !b || !h || !ws) return PARARNN_ERR_INVALID;
    if (!aligned(A, 4) || !aligned(b, 4) || !aligned(h, 4) || (h0 && !aligned(h0, 4)))
        return PARARNN_ERR_INVALID;
    const Ws w{static_cast<char *>(ws), ws_bytes};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (k == 4 && !blk4_rows()) {
        if (!grid_ok(scan_shape(kCfgLinBlk4, B, L, H).ntiles)) return PARARNN_ERR_INVALID;
        if (ws_bytes < scan_ws(kCfgLinBlk4, 4, B, L, H).total || !aligned(ws, 256)) return PARARNN_ERR_INVALID;
        return status_of(linscan_blk(4, B, L, H, A, b, h0, h, w, s));
    }
    const BlkRowWs need = blkrow_ws(k, B, L, H);
    if (!grid_ok(need.ntiles)) return PARARNN_ERR_INVALID;
    if (ws_bytes < need.total || !aligned(ws, 256)) return PARARNN_ERR_INVALID;
    return status_of(linscan_blkrow(k, B, L, H, A, b, h0, h, w, s));
}

int pararnn_gru_forward(int64_t B, int64_t L, int64_t H, const float *pz, const float *pr,
                        const float *pc, const float *uz, const float *ur, const float *uc,
                        const float *h0, const float *h_init, float *h, float tol, int32_t max_iter,
                        int32_t *info, float *trace, void *ws, size_t ws_bytes, void *stream) {
    if (!dims_ok(B, L, H) || !pz || !pr || !pc || !uz || !ur || !uc || !h) return PARARNN_ERR_INVALID;
    if (!(tol >= 0.0f) || max_iter < 1) return PARARNN_ERR_INVALID;  // rejects NaN too
    if (overlaps(h_init, h, B * L * H)) return PARARNN_ERR_INVALID;
    const int32_t cap = eff_cap(max_iter, L);
    GruFwdArgs a{B,  L,   H,   pz,    pr,   pc,    uz,   ur,
                 uc, h0,  h_init, h,  tol,  cap,   info, trace,
                 env_chain_local("PARARNN_GRU_PATH")};
    hipStream_t s = static_cast<hipStream_t>(stream);
    const Path path = gru_path(L, cap);
    if (path == Path::Invalid) return PARARNN_ERR_UNSUPPORTED;
    if (path != Path::Fused && (!ws || ws_bytes < gru_fwd_ws(B, L, H, cap) || !aligned(ws, 256)))
        return PARARNN_ERR_INVALID;
    const int64_t ntiles = path == Path::Fused ? B * ((H + kFusedChannels - 1) / kFusedChannels)
                           : path == Path::Chain ? scan_shape(kCfgGruChain, B, L, H).ntiles
                                                 : scan_shape(kCfgGruStep, B, L, H).ntiles;
    if (!grid_ok(ntiles)) return PARARNN_ERR_INVALID;
    if (trace != nullptr && max_iter > cap) {
        const int st = clear_trace_tail(trace, cap, max_iter, s);
        if (st != PARARNN_OK) return st;
    }
    const Ws w{static_cast<char *>(ws), ws_bytes};
    if (path == Path::Fused) return status_of(gru_forward_fused(a, s));
    if (path == Path::Chain) return status_of(gru_forward_chain(a, w, s));
    return status_of(gru_forward_step(a, w, s));
}

int pararnn_lstm_forward(int64_t B, int64_t L, int64_t H, const float *pi, const float *pf,
                         const float *po, const float *pg, const float *ui, const float *uf,
                         const float *uo, const float *ug, const float *h0, const float *c0,
                         const float *h_init, const float *c_init, float *h, float *c, float tol,
                         int32_t max_iter, int32_t *info, float *trace, void *ws, size_t ws_bytes,
                         void *stream) {
    if (!dims_ok(B, L, H) || !pi || !pf || !po || !pg || !ui || !uf || !uo || !ug || !h || !c)
        return PARARNN_ERR_INVALID;
    if (!(tol >= 0.0f) || max_iter < 1) return PARARNN_ERR_INVALID;
    const int64_t n = B * L * H;
    if (overlaps(h_init, h, n) || overlaps(h_init, c, n) || overlaps(c_init, h, n) || overlaps(c_init, c, n))
        return PARARNN_ERR_INVALID;
    const int32_t cap = eff_cap(max_iter, L);
    if (!ws || ws_bytes < lstm_fwd_ws(B, L, H, cap) || !aligned(ws, 256)) return PARARNN_ERR_INVALID;
    LstmFwdArgs a{B,  L,  H,      pi,     pf, po, pg,  ui,  uf,   uo,    ug,
                  h0, c0, h_init, c_init, h,  c,  tol, cap, info, trace, env_chain_local("PARARNN_LSTM_PATH")};
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool chain = lstm_path(cap) == Path::Chain;
    if (!grid_ok(scan_shape(chain ? kCfgLstmChain : kCfgLstmStep, B, L, H).ntiles)) return PARARNN_ERR_INVALID;
    if (trace != nullptr && max_iter > cap) {
        const int st = clear_trace_tail(trace, cap, max_iter, s);
        if (st != PARARNN_OK) return st;
    }
    const Ws w{static_cast<char *>(ws), ws_bytes};
    if (chain) return status_of(lstm_forward_chain(a, w, s));
    return status_of(lstm_forward_step(a, w, s));
}

int pararnn_hgru_forward(int32_t k, int64_t B, int64_t L, int64_t NH, const float *pz, const float *pr,
                         const float *pc, const float *Uz, const float *Ur, const float *Uc, const float *h0,
                         const float *h_init, float *h, float tol, int32_t max_iter, int32_t *info, float *trace,
                         void *ws, size_t ws_bytes, void *stream) {
    if (k < 1) return PARARNN_ERR_INVALID;
    if (k != 4 && k != 8) return PARARNN_ERR_UNSUPPORTED;
    if (!dims_ok(B, L, NH) || !dims_ok(B, L, NH * k)) return PARARNN_ERR_INVALID;
    if (!pz || !pr || !pc || !Uz || !Ur || !Uc || !h) return PARARNN_ERR_INVALID;
    if (!(tol >= 0.0f) || max_iter < 1) return PARARNN_ERR_INVALID;
    if (overlaps(h_init, h, B * L * NH * k)) return PARARNN_ERR_INVALID;
    const int32_t cap = eff_cap(max_iter, L);
    const HgruWs need = hgru_ws(k, B, L, NH, cap);
    if (!grid_ok(need.sh.ntiles)) return PARARNN_ERR_INVALID;
    if (!ws || ws_bytes < need.total || !aligned(ws, 256)) return PARARNN_ERR_INVALID;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (trace != nullptr && max_iter > cap) {
        const int st = clear_trace_tail(trace, cap, max_iter, s);
        if (st != PARARNN_OK) return st;
    }
    const HgruFwdArgs a{k, B, L, NH, pz, pr, pc, Uz, Ur, Uc, h0, h_init, h, tol, cap, info, trace};
    return status_of(hgru_forward(a, Ws{static_cast<char *>(ws), ws_bytes}, s));
}

int pararnn_hgru_backward(int32_t k, int64_t B, int64_t L, int64_t NH, const float *pz, const float *pr,
                          const float *pc, const float *Uz, const float *Ur, const float *Uc, const float *h0,
                          const float *h, const float *grad_h, float *grad_pz, float *grad_pr, float *grad_pc,
                          float *grad_Uz, float *grad_Ur, float *grad_Uc, float *grad_h0, void *ws,
                          size_t ws_bytes, void *stream) {
    if (k < 1) return PARARNN_ERR_INVALID;
    if (k != 4 && k != 8) return PARARNN_ERR_UNSUPPORTED;
    if (!dims_ok(B, L, NH) || !dims_ok(B, L, NH * k)) return PARARNN_ERR_INVALID;
    if (!pz || !pr || !pc || !Uz || !Ur || !Uc || !h || !grad_h || !grad_pz || !grad_pr || !grad_pc)
        return PARARNN_ERR_INVALID;
    const int64_t n = B * L * NH * k;
    // h is read at other positions than the thread's own: no output may alias it
    if (overlaps(grad_pz, h, n) || overlaps(grad_pr, h, n) || overlaps(grad_pc, h, n)) return PARARNN_ERR_INVALID;
    if ((grad_Uz || grad_Ur || grad_Uc) && NH > 0x7fffffff) return PARARNN_ERR_INVALID;
    const HgruAdjWs need = hgru_adj_ws(k, B, L, NH);
    if (!grid_ok(need.sh.ntiles)) return PARARNN_ERR_INVALID;
    if (!ws || ws_bytes < need.total || !aligned(ws, 256)) return PARARNN_ERR_INVALID;
    HgruBwdArgs a{k, B, L, NH, pz, pr, pc, Uz, Ur, Uc, h0, h, grad_h, grad_pz, grad_pr, grad_pc,
                  {grad_Uz, grad_Ur, grad_Uc}, grad_h0};
    return status_of(hgru_backward(a, Ws{static_cast<char *>(ws), ws_bytes}, static_cast<hipStream_t>(stream)));
}

int pararnn_gru_sequential(int64_t B, int64_t L, int64_t H, const float *pz, const float *pr,
                           const float *pc, const float *uz, const float *ur, const float *uc,
                           const float *h0, float *h, void *stream) {
    if (!dims_ok(B, L, H) || !pz || !pr || !pc || !uz || !ur || !uc || !h) return PARARNN_ERR_INVALID;
    if (!grid_ok((B * H + 63) / 64)) return PARARNN_ERR_INVALID;
    GruFwdArgs a{B, L, H, pz, pr, pc, uz, ur, uc, h0, nullptr, h, 0.0f, 1, nullptr, nullptr, -1};
    return status_of(gru_rollout(a, static_cast<hipStream_t>(stream)));
}

int pararnn_lstm_sequential(int64_t B, int64_t L, int64_t H, const float *pi, const float *pf,
                            const float *po, const float *pg, const float *ui, const float *uf,
                            const float *uo, const float *ug, const float *h0, const float *c0,
                            float *h, float *c, void *stream) {
    if (!dims_ok(B, L, H) || !pi || !pf || !po || !pg || !ui || !uf || !uo || !ug || !h || !c)
        return PARARNN_ERR_INVALID;
    if (!grid_ok((B * H + 63) / 64)) return PARARNN_ERR_INVALID;
    LstmFwdArgs a{B, L, H, pi, pf, po, pg, ui, uf, uo, ug, h0, c0, nullptr, nullptr, h, c, 0.0f, 1, nullptr, nullptr, -1};
    return status_of(lstm_rollout(a, static_cast<hipStream_t>(stream)));
}

int pararnn_adjoint_backward(int32_t cell, int64_t B, int64_t L, int64_t H, const float *const *p,
                             const float *const *u, const float *h0, const float *c0,
                             const float *h, const float *c, const float *grad_h,
                             const float *grad_c, float *const *grad_p, float *const *grad_u,
                             float *grad_h0, float *grad_c0, void *ws, size_t ws_bytes,
                             void *stream) {
    if (cell != PARARNN_CELL_GRU && cell != PARARNN_CELL_LSTM) return PARARNN_ERR_INVALID;
    if (!dims_ok(B, L, H) || !p || !u || !h || !grad_h || !grad_p || !ws) return PARARNN_ERR_INVALID;
    const int ng = cell == PARARNN_CELL_GRU ? 3 : 4;
    AdjArgs a;
    memset(&a, 0, sizeof(a));
    a.B = B;
    a.L = L;
    a.H = H;
    for (int q = 0; q < ng; ++q) {
        if (!p[q] || !u[q] || !grad_p[q]) return PARARNN_ERR_INVALID;
        a.p[q] = p[q];
        a.u[q] = u[q];
        a.gp[q] = grad_p[q];
        a.gu[q] = grad_u ? grad_u[q] : nullptr;
    }
    a.h0 = h0;
    a.h = h;
    a.gh = grad_h;
    a.gh0 = grad_h0;
    bool want_u = false;
    for (int q = 0; q < ng; ++q) want_u = want_u || a.gu[q] != nullptr;
    if (want_u && H > 0x7fffffff) return PARARNN_ERR_INVALID;  // the dL/du reduction has one workgroup per channel
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (cell == PARARNN_CELL_GRU) {
        if (grad_c || grad_c0) return PARARNN_ERR_INVALID;
        if (!grid_ok(scan_shape(kCfgGruAdj, B, L, H).ntiles)) return PARARNN_ERR_INVALID;
        if (ws_bytes < gru_adjoint_ws(B, L, H) || !aligned(ws, 256)) return PARARNN_ERR_INVALID;
        return status_of(gru_adjoint(a, Ws{static_cast<char *>(ws), ws_bytes}, s));
    }
    if (!c) return PARARNN_ERR_INVALID;
    a.c0 = c0;
    a.c = c;
    a.gc = grad_c;
    a.gc0 = grad_c0;
    if (!grid_ok(scan_shape(kCfgLstmAdj, B, L, H).ntiles)) return PARARNN_ERR_INVALID;
    if (ws_bytes < lstm_adjoint_ws(B, L, H) || !aligned(ws, 256)) return PARARNN_ERR_INVALID;
    return status_of(lstm_adjoint(a, Ws{static_cast<char *>(ws), ws_bytes}, s));
}

// ---------------------------------------------------------------- operators around the recurrences
size_t pararnn_linattn_workspace_bytes(int32_t backward, int32_t dtype, int64_t B, int64_t L, int64_t H, int64_t dk,
                                       int64_t dv) {
    if (!linattn_dims_ok(backward ? LinattnPass::Backward : LinattnPass::Forward, dtype, B, L, H, dk, dv)) return 0;
    return linattn_ws(linattn_shape(dtype, B, L, H, dk, dv), backward != 0);
}

int pararnn_linattn_forward(int32_t dtype, int64_t B, int64_t L, int64_t H, int64_t dk, int64_t dv, const void *q,
                            const void *k, const void *v, const int64_t *strides, const float *log_decay,
                            const float *state, float scale, void *o, float *out_state, void *ws, size_t ws_bytes,
                            void *stream) {
    if (dk > kMaxHeadDim || dv > kMaxHeadDim) return PARARNN_ERR_UNSUPPORTED;
    if (!linattn_dims_ok(LinattnPass::Forward, dtype, B, L, H, dk, dv) || !q || !k || !v || !log_decay || !o)
        return PARARNN_ERR_INVALID;
    LinattnArgs a = linattn_shape(dtype, B, L, H, dk, dv);
    const void *in[3] = {q, k, v};
    if (!linattn_inputs(a, in, 3, strides)) return PARARNN_ERR_INVALID;
    if (!ws || ws_bytes < linattn_ws(a, false) || !aligned(ws, 256)) return PARARNN_ERR_INVALID;
    if (states_cross(a, state, out_state)) return PARARNN_ERR_INVALID;
    a.log_decay = log_decay;
    a.state = state;
    a.scale = scale;
    a.o = o;
    a.out_state = out_state;
    return status_of(linattn_forward(a, Ws{static_cast<char *>(ws), ws_bytes}, static_cast<hipStream_t>(stream)));
}

int pararnn_linattn_backward(int32_t dtype, int64_t B, int64_t L, int64_t H, int64_t dk, int64_t dv, const void *q,
                             const void *k, const void *v, const void *grad_o, const int64_t *strides,
                             const float *log_decay, const float *state, const float *grad_out_state, float scale,
                             void *grad_q, void *grad_k, void *grad_v, float *grad_state, void *ws, size_t ws_bytes,
                             void *stream) {
    if (dk > kMaxHeadDim || dv > kMaxHeadDim) return PARARNN_ERR_UNSUPPORTED;
    if (!linattn_dims_ok(LinattnPass::Backward, dtype, B, L, H, dk, dv) || !q || !k || !v || !grad_o || !log_decay ||
        !grad_q || !grad_k || !grad_v)
        return PARARNN_ERR_INVALID;
    LinattnArgs a = linattn_shape(dtype, B, L, H, dk, dv);
    const void *in[4] = {q, k, v, grad_o};
    if (!linattn_inputs(a, in, 4, strides)) return PARARNN_ERR_INVALID;
    if (!ws || ws_bytes < linattn_ws(a, true) || !aligned(ws, 256)) return PARARNN_ERR_INVALID;
    // both states are read by walks beside the one that ends on grad_state
    const int64_t n = B * H * dk * dv;
    if (overlaps(state, grad_state, n) || overlaps(grad_out_state, grad_state, n)) return PARARNN_ERR_INVALID;
    a.log_decay = log_decay;
    a.state = state;
    a.scale = scale;
    a.grad_out_state = grad_out_state;
    a.grad_q = grad_q;
    a.grad_k = grad_k;
    a.grad_v = grad_v;
    a.grad_state = grad_state;
    return status_of(linattn_backward(a, Ws{static_cast<char *>(ws), ws_bytes}, static_cast<hipStream_t>(stream)));
}

int pararnn_linattn_step(int32_t dtype, int64_t B, int64_t H, int64_t dk, int64_t dv, const void *q, const void *k,
                         const void *v, const int64_t *strides, const float *log_decay, const float *state, float scale,
                         void *o, float *out_state, void *stream) {
    if (dk > kMaxHeadDim || dv > kMaxHeadDim) return PARARNN_ERR_UNSUPPORTED;
    if (!linattn_dims_ok(LinattnPass::Step, dtype, B, 1, H, dk, dv) || !q || !k || !v || !log_decay || !state || !o || !out_state)
        return PARARNN_ERR_INVALID;
    LinattnArgs a = linattn_shape(dtype, B, 1, H, dk, dv);
    const void *in[3] = {q, k, v};
    if (!linattn_inputs(a, in, 3, strides) || states_cross(a, state, out_state)) return PARARNN_ERR_INVALID;
    a.log_decay = log_decay;
    a.state = state;
    a.scale = scale;
    a.o = o;
    a.out_state = out_state;
    return status_of(linattn_step(a, static_cast<hipStream_t>(stream)));
}

size_t pararnn_layernorm_workspace_bytes(int64_t rows, int64_t D) {
    if (!layernorm_dims_ok(PARARNN_F32, rows, D)) return 0;
    return kScratchOffset + (size_t)layernorm_parts(rows, D) * 2 * (size_t)D * sizeof(float);
}

int pararnn_layernorm_forward(int32_t dtype, int64_t rows, int64_t D, const void *x, const void *residual,
                              const float *weight, const float *bias, float eps, void *sum, void *y, float *mean,
                              float *rstd, void *stream) {
    if (!layernorm_dims_ok(dtype, rows, D) || !x || !y || (residual != nullptr) != (sum != nullptr))
        return PARARNN_ERR_INVALID;
    if (!(eps >= 0.0f)) return PARARNN_ERR_INVALID;
    const LayernormFwdArgs a{dtype == PARARNN_BF16, rows, D, x, residual, weight, bias, eps, sum, y, mean, rstd};
    return status_of(layernorm_forward(a, static_cast<hipStream_t>(stream)));
}

int pararnn_layernorm_backward(int32_t dtype, int64_t rows, int64_t D, const void *s, const float *weight,
                               const float *mean, const float *rstd, const void *grad_y, const void *grad_sum,
                               void *grad_x, float *grad_weight, float *grad_bias, void *ws, size_t ws_bytes,
                               void *stream) {
    if (!layernorm_dims_ok(dtype, rows, D) || !s || !mean || !rstd || !grad_y || !grad_x) return PARARNN_ERR_INVALID;
    if ((grad_weight || grad_bias) &&
        (!ws || ws_bytes < pararnn_layernorm_workspace_bytes(rows, D) || !aligned(ws, 256)))
        return PARARNN_ERR_INVALID;
    const LayernormBwdArgs a{dtype == PARARNN_BF16, rows, D, s, weight, mean, rstd, grad_y, grad_sum, grad_x,
                             grad_weight, grad_bias};
    return status_of(layernorm_backward(a, Ws{static_cast<char *>(ws), ws_bytes}, static_cast<hipStream_t>(stream)));
}

int pararnn_embedding_forward(int32_t dtype, int64_t N, int64_t V, int64_t D, const void *ids, int32_t id_bytes,
                              const void *table, float scale, void *out, void *stream) {
    if (!embedding_dims_ok(dtype, N, V, D) || (id_bytes != 4 && id_bytes != 8) || !ids || !table || !out)
        return PARARNN_ERR_INVALID;
    const EmbeddingArgs a{dtype == PARARNN_BF16, id_bytes == 8, N, V, D, -1, ids, table, scale, out};
    return status_of(embedding_forward(a, static_cast<hipStream_t>(stream)));
}

size_t pararnn_embedding_workspace_bytes(int64_t N, int64_t V, int64_t D) {
    return embedding_dims_ok(PARARNN_F32, N, V, D) ? embedding_ws(N, D) : 0;
}

int pararnn_embedding_backward(int32_t dtype, int64_t N, int64_t V, int64_t D, const void *ids, int32_t id_bytes,
                               const void *grad, float scale, int64_t padding_idx, void *grad_table, void *ws,
                               size_t ws_bytes, void *stream) {
    if (!embedding_dims_ok(dtype, N, V, D) || (id_bytes != 4 && id_bytes != 8) || !ids || !grad || !grad_table)
        return PARARNN_ERR_INVALID;
    if (padding_idx < -1 || padding_idx >= V) return PARARNN_ERR_INVALID;
    if (!ws || ws_bytes < embedding_ws(N, D) || !aligned(ws, 256)) return PARARNN_ERR_INVALID;
    const EmbeddingArgs a{dtype == PARARNN_BF16, id_bytes == 8, N, V, D, padding_idx, ids, grad, scale, grad_table};
    return status_of(embedding_backward(a, Ws{static_cast<char *>(ws), ws_bytes}, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
