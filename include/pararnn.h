/*
 * pararnn.h -- C ABI of libpararnn.so: parallel-in-time evaluation of
 * nonlinear RNNs by Newton's method with a parallel linear-recurrence scan,
 * for AMD Instinct MI355X (gfx950).
 *
 * The method (ParaRNN page, TL;DR and abstract; DEER summary page, first and
 * second paragraphs): the recurrence h_t = f(h_{t-1}, x_t) over a whole
 * sequence is one nonlinear system; Newton's method linearises every cell at
 * the current iterate and solves the resulting block bi-diagonal linear
 * system, which is a linear recurrence, with a parallel scan over the
 * sequence.  The GRU-style cell has a diagonal Jacobian and the LSTM-style
 * cell a 2x2 block-diagonal one (ParaRNN page, Fig. 2 caption).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Tensors are fp32, dense, row-major.  Sequence tensors are [B, L, H]
 *    with the channel index fastest ("channel-contiguous").  Per-channel
 *    weights u are [H], shared over batch and time.  Initial states are
 *    [B, H].  Output row t is the state after consuming input t; the initial
 *    state is not emitted.
 *  - Every pointer named as a tensor is a DEVICE pointer (hipMalloc'd or
 *    torch-allocated, at least 4-byte aligned).  The caller owns all memory,
 *    including the workspace; the library never allocates or frees and keeps
 *    no state of its own between calls beyond cached device properties (what
 *    persists lives in the caller's workspace).  Outputs must not alias
 *    inputs.
 *  - `ws`/`ws_bytes`: a device scratch buffer of at least
 *    pararnn_workspace_bytes(...) bytes (256-byte aligned); `ws_bytes` is
 *    its whole size.  It must be zero-filled before its first use
 *    (hipMemset, torch.zeros); every call leaves it ready for the next call
 *    of any entry point at any size that fits, so the caller never clears it
 *    again and must not write to it between calls.  Its first 16 bytes
 *    count the workgroups of a launch and number the launches; the
 *    look-back records of the scans carry the number of the launch that
 *    wrote them, which is why no call has to clear them.  Launch numbers
 *    repeat after 8,388,606 launches on one workspace: the launch that uses
 *    the last number clears all `ws_bytes` past the 16-byte header when its
 *    last workgroup finishes (about a millisecond per few hundred MB, once
 *    per period), so no record of an earlier period is ever read.
 *    Concurrent calls on different streams need different workspaces.  A
 *    workspace that was not zero-filled gives wrong results (the kernels
 *    still stay in bounds and finish).
 *  - `stream`: a hipStream_t passed as void* (NULL = the default stream).
 *    Every call only enqueues work on that stream and returns; it never
 *    synchronises.  Device-side outputs (including `info`) are valid once
 *    the stream has been synchronised.
 *  - Return value: PARARNN_OK, or a negative status.  Argument validation is
 *    done on the host before anything is enqueued (PARARNN_ERR_INVALID).  A
 *    failed launch returns PARARNN_ERR_HIP.  Non-convergence of Newton is NOT
 *    an error: the outputs hold the last iterate and info reports it.
 */
#ifndef PARARNN_H
#define PARARNN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
    PARARNN_OK = 0,
    PARARNN_ERR_INVALID = -1,     /* bad pointer, size, tolerance, cap or workspace */
    PARARNN_ERR_HIP = -2,         /* a HIP launch or runtime call failed */
    PARARNN_ERR_UNSUPPORTED = -3, /* combination not implemented */
    PARARNN_ERR_TOO_LARGE = -4    /* needs more than the library's static scratch buffer */
};

enum { PARARNN_CELL_GRU = 0, PARARNN_CELL_LSTM = 1 };

/* Operation codes for pararnn_workspace_bytes. */
enum {
    PARARNN_OP_LINSCAN_DIAG = 0,
    PARARNN_OP_LINSCAN_BLK2 = 1,
    PARARNN_OP_GRU_FORWARD = 2,
    PARARNN_OP_LSTM_FORWARD = 3,
    PARARNN_OP_GRU_ADJOINT = 4,
    PARARNN_OP_LSTM_ADJOINT = 5,
    PARARNN_OP_LINSCAN_BLK4 = 6,  /* rnn_linscan_blk with k = 4 */
    PARARNN_OP_LINSCAN_BLK8 = 7,  /* rnn_linscan_blk with k = 8 */
    PARARNN_OP_HGRU4_FORWARD = 8,  /* pararnn_hgru_forward with k = 4 (H = heads) */
    PARARNN_OP_HGRU8_FORWARD = 9,  /* pararnn_hgru_forward with k = 8 (H = heads) */
    PARARNN_OP_HGRU4_BACKWARD = 10, /* pararnn_hgru_backward with k = 4 (H = heads) */
    PARARNN_OP_HGRU8_BACKWARD = 11  /* pararnn_hgru_backward with k = 8 (H = heads) */
};

/*
 * Bytes of workspace that operation `op` needs at (B, L, H) with Newton
 * iteration cap `max_iter` (ignored by the scans and the adjoints).  For the
 * Newton forwards it is the need of the kernel the call will take, which
 * depends on the shape, the cap, the device (how many workgroups fit on it)
 * and the PARARNN_GRU_PATH / PARARNN_LSTM_PATH environment overrides as read
 * at the time of the query.  The GRU's fused kernel and the chained kernel's
 * form in which workgroups own whole chains need none: 256 bytes are
 * returned.  A call whose workspace is too small for its kernel returns
 * PARARNN_ERR_INVALID.  Returns 0 for invalid arguments.
 */
size_t pararnn_workspace_bytes(int32_t op, int64_t B, int64_t L, int64_t H,
                               int32_t max_iter);

/*
 * Diagonal linear recurrence, solved by a chunked parallel scan
 * (ParaRNN page, Fig. 2 left: the parallel reduction for diagonal systems;
 * DEER summary page: associative scan; minimal-RNN article: the recurrence a
 * parallel scan evaluates once gates do not depend on h):
 *     h[b,t,j] = a[b,t,j] * h[b,t-1,j] + b[b,t,j],   h[b,-1,j] = h0[b,j]
 * a, b, h: [B, L, H].  h0: [B, H], or NULL for zeros.
 */
int rnn_linscan_diag(int64_t B, int64_t L, int64_t H,
                     const float *a, const float *b, const float *h0,
                     float *h, void *ws, size_t ws_bytes, void *stream);

/*
 * 2x2 block linear recurrence (ParaRNN page, Fig. 2: the 2x2 block-diagonal
 * solver used by ParaLSTM):
 *     h[b,t,j,:] = A[b,t,j] @ h[b,t-1,j,:] + b[b,t,j,:]
 * A: [B, L, H, 2, 2] row-major blocks (a00, a01, a10, a11).
 * b, h: [B, L, H, 2].  h0: [B, H, 2] or NULL.  Any 4-byte alignment; with
 * A 16-byte aligned and b, h, h0 8-byte aligned, blocks and pairs move as
 * single vector accesses (faster).
 */
int rnn_linscan_blk2(int64_t B, int64_t L, int64_t H,
                     const float *A, const float *b, const float *h0,
                     float *h, void *ws, size_t ws_bytes, void *stream);

/*
 * k x k block linear recurrence: the 2x2 solver widened to small dense
 * blocks, such as the per-head Jacobians of a cell with dense recurrence
 * inside heads of k channels (ParaRNN page, Fig. 2 caption: block
 * bi-diagonal systems; DEER summary page, limitations paragraph: dense
 * Jacobians as the hidden size grows):
 *     h[b,t,j,:] = A[b,t,j] @ h[b,t-1,j,:] + b[b,t,j,:]
 * A: [B, L, H, k, k] row-major blocks (A[i][l] takes component l into i).
 * b, h: [B, L, H, k].  h0: [B, H, k] or NULL.
 * k = 2 is rnn_linscan_blk2 (its workspace query, PARARNN_OP_LINSCAN_BLK2).
 * k = 4 and k = 8 take the workspace of PARARNN_OP_LINSCAN_BLK4 and
 * PARARNN_OP_LINSCAN_BLK8 and any 4-byte alignment (with A 16-byte aligned,
 * block rows move as 16-byte accesses, faster).  The rows of each block are
 * spread over k lanes; PARARNN_BLK4_PATH=thread (read at the query and at
 * the call) makes k = 4 take the kernel with one thread per block instead.
 * Other k return PARARNN_ERR_UNSUPPORTED (k < 1: PARARNN_ERR_INVALID).
 */
int rnn_linscan_blk(int32_t k, int64_t B, int64_t L, int64_t H,
                    const float *A, const float *b, const float *h0,
                    float *h, void *ws, size_t ws_bytes, void *stream);

/*
 * GRU-style cell with diagonal recurrence (ParaGRU, ParaRNN page Fig. 2):
 *   z = sigmoid(pz + uz*h), r = sigmoid(pr + ur*h),
 *   c = tanh(pc + uc*(r*h)),  h' = (1 - z)*h + z*c
 * evaluated over the whole sequence by Newton's method (ParaRNN TL;DR;
 * DEER summary), from h = 0 or from a given initial iterate.
 * pz, pr, pc: [B, L, H] gate pre-projections (input projections and biases
 * already applied).  uz, ur, uc: [H].  h0: [B, H] or NULL.
 * h_init: [B, L, H] initial iterate (a warm start, such as the solution of a
 * nearby input), or NULL for zeros; read only, and it must not overlap h
 * (PARARNN_ERR_INVALID).  Newton from any iterate is exact after L
 * iterations, so the cap rule below holds for warm starts too; a start that
 * already solves the system returns after one iteration with a zero update.
 * h: [B, L, H] output.
 * tol >= 0: Newton stops once max|delta| <= tol (the only extra
 * hyper-parameter; DEER summary, second paragraph), measured after the
 * update and absolute.  Where the test is taken depends on the kernel:
 *  - L <= 512: over the whole sequence of each 16 channels of a batch row;
 *  - longer sequences with max_iter <= 64: each chunk of the sequence stops
 *    once it and every earlier chunk of its channels meet the bound, so the
 *    last chunk stops exactly when Newton over the whole sequence of those
 *    channels would (earlier chunks may freeze a few iterations sooner, with
 *    corrections of order tol^2 left);
 *  - max_iter > 64: over the whole tensor (one launch per iteration).
 * With tol = 0 nothing stops before the cap.  max_iter >= 1; caps above
 * L + 1 are taken as L + 1 (Newton from zero is exact after L iterations,
 * and iteration L + 1 confirms it).
 * info: device int32[2] {iterations, converged} or NULL.  iterations is the
 * largest number of updates any tile applied; converged is 1 only if every
 * tile met the tolerance.
 * trace: device float[max_iter] or NULL; receives max|delta| of each
 * iteration (0 for iterations not run).
 */
int pararnn_gru_forward(int64_t B, int64_t L, int64_t H,
                        const float *pz, const float *pr, const float *pc,
                        const float *uz, const float *ur, const float *uc,
                        const float *h0, const float *h_init, float *h, float tol,
                        int32_t max_iter, int32_t *info, float *trace,
                        void *ws, size_t ws_bytes, void *stream);

/*
 * LSTM-style cell with diagonal recurrence (ParaLSTM, ParaRNN page Fig. 2):
 * per channel the state is (c, h) and the Jacobian a 2x2 block.
 *   i = sigmoid(pi + ui*h'), f = sigmoid(pf + uf*h'), o = sigmoid(po + uo*h'),
 *   g = tanh(pg + ug*h'),  c = f*c' + i*g,  h = o*tanh(c)
 * Newton from (c, h) = 0, or from the initial iterates h_init, c_init
 * ([B, L, H] each, a NULL one taken as zeros; read only, neither may overlap
 * h or c); max|delta| is taken over both components.
 * pi, pf, po, pg: [B, L, H]; ui, uf, uo, ug: [H]; h0, c0: [B, H] or NULL;
 * h, c: [B, L, H] outputs.  tol, max_iter, info, trace as for the GRU,
 * except that this cell has no single-tile kernel: the chunk rule applies at
 * every L when max_iter <= 64.
 */
int pararnn_lstm_forward(int64_t B, int64_t L, int64_t H,
                         const float *pi, const float *pf, const float *po,
                         const float *pg, const float *ui, const float *uf,
                         const float *uo, const float *ug, const float *h0,
                         const float *c0, const float *h_init, const float *c_init,
                         float *h, float *c, float tol, int32_t max_iter,
                         int32_t *info, float *trace,
                         void *ws, size_t ws_bytes, void *stream);

/*
 * GRU with dense recurrence inside heads of k channels (k = 4 or 8): the
 * GRU-style cell above with each weight vector replaced by one k x k matrix
 * per head, acting on the state vector of the head where the diagonal cell
 * multiplies by u (a diagonal U is exactly the diagonal cell), so the
 * Jacobian is block-diagonal with dense k x k blocks (DEER summary page,
 * limitations paragraph: dense Jacobians, the GRU with 8-channel heads;
 * ParaRNN page, Fig. 2 caption: block bi-diagonal systems):
 *   z = sigmoid(pz + Uz h), r = sigmoid(pr + Ur h),
 *   c = tanh(pc + Uc (r*h)),  h' = (1 - z)*h + z*c
 * evaluated over the whole sequence by Newton's method, one launch per
 * iteration (launches after convergence exit at once; the host never waits),
 * each solving the block bi-diagonal system with the k x k scan.
 * pz, pr, pc: [B, L, NH, k] gate pre-projections; Uz, Ur, Uc: [NH, k, k]
 * row-major (U[n][i][l] takes component l into i); h0: [B, NH, k] or NULL;
 * h_init: [B, L, NH, k] initial iterate or NULL for zeros (must not overlap
 * h); h: [B, L, NH, k] output.  tol, max_iter, info, trace as for
 * pararnn_gru_forward, with max|delta| over the whole tensor (every cap
 * takes this path).  Workspace: PARARNN_OP_HGRU4_FORWARD /
 * PARARNN_OP_HGRU8_FORWARD with H = NH.  Other k return
 * PARARNN_ERR_UNSUPPORTED (k < 1: PARARNN_ERR_INVALID).
 */
int pararnn_hgru_forward(int32_t k, int64_t B, int64_t L, int64_t NH,
                         const float *pz, const float *pr, const float *pc,
                         const float *Uz, const float *Ur, const float *Uc,
                         const float *h0, const float *h_init, float *h, float tol,
                         int32_t max_iter, int32_t *info, float *trace,
                         void *ws, size_t ws_bytes, void *stream);

/*
 * Gradients through the converged solve of pararnn_hgru_forward (DEER
 * summary page: forward plus gradients; the adjoint is the transposed block
 * bi-diagonal system, ParaRNN page, Fig. 2 caption), by a reverse-time scan
 * of k x k blocks:
 *   nu_t = J_t^T (nu_{t+1} + g_t) with nu_L = 0,  lambda_t = g_t + nu_{t+1},
 *   dL/dpz = lambda dF/daz,  dL/dpc = lambda dF/dac,  dL/dpr = dL/dar,
 *   dL/dU = sum over batch rows and positions of the outer products of the
 *   pre-activation gradients with the vectors U multiplies (h for Uz and Ur,
 *   r*h for Uc),  dL/dh0 = nu_0,
 * for L = sum g*h, with the cell and J_t evaluated at the given states.
 * pz, pr, pc, Uz, Ur, Uc, h0 as for pararnn_hgru_forward; h: [B, L, NH, k]
 * the forward's solution; grad_h: [B, L, NH, k].  grad_pz, grad_pr,
 * grad_pc: [B, L, NH, k] outputs (overwritten; each may be its own p, none
 * may overlap h).  grad_Uz, grad_Ur, grad_Uc: [NH, k, k] outputs or NULL
 * (any of them requires NH < 2^31).  grad_h0: [B, NH, k] output or NULL.
 * Workspace: PARARNN_OP_HGRU4_BACKWARD / PARARNN_OP_HGRU8_BACKWARD with
 * H = NH (max_iter ignored).  Other k return PARARNN_ERR_UNSUPPORTED (k < 1:
 * PARARNN_ERR_INVALID).
 */
int pararnn_hgru_backward(int32_t k, int64_t B, int64_t L, int64_t NH,
                          const float *pz, const float *pr, const float *pc,
                          const float *Uz, const float *Ur, const float *Uc,
                          const float *h0, const float *h, const float *grad_h,
                          float *grad_pz, float *grad_pr, float *grad_pc,
                          float *grad_Uz, float *grad_Ur, float *grad_Uc, float *grad_h0,
                          void *ws, size_t ws_bytes, void *stream);

/*
 * Gradients through the converged solve (DEER summary: forward plus
 * gradients), by a reverse-time linear scan of the adjoint:
 *   lambda_t = g_t + J_{t+1}^T lambda_{t+1},  dL/dp_t = (df_t/dp_t)^T lambda_t,
 *   dL/du = sum_{b,t} lambda_t^T df_t/du,  dL/dh0 = J_0^T lambda_0,
 * for the loss L = sum g_h*h (+ sum g_c*c for the LSTM), with J and df/dp
 * evaluated at the forward states (h, c).
 * cell: PARARNN_CELL_GRU (3 gates z, r, c) or PARARNN_CELL_LSTM (4 gates
 * i, f, o, g).  p, u, grad_p, grad_u: HOST arrays of 3 or 4 DEVICE pointers.
 * h (and c for the LSTM): the forward outputs [B, L, H].  grad_h: [B, L, H];
 * grad_c: [B, L, H] or NULL (LSTM only; NULL means zero).  grad_p[k]:
 * [B, L, H] outputs (overwritten).  grad_u: NULL, or an array whose entries
 * are [H] outputs or NULL (any of them requires H < 2^31).  grad_h0,
 * grad_c0: [B, H] outputs or NULL.
 */
int pararnn_adjoint_backward(int32_t cell, int64_t B, int64_t L, int64_t H,
                             const float *const *p, const float *const *u,
                             const float *h0, const float *c0,
                             const float *h, const float *c,
                             const float *grad_h, const float *grad_c,
                             float *const *grad_p, float *const *grad_u,
                             float *grad_h0, float *grad_c0,
                             void *ws, size_t ws_bytes, void *stream);

/*
 * Sequential application of the GRU-style cell: one thread per channel
 * walks t = 0..L-1 in order, one cell evaluation per position, no Newton
 * iteration.  This is the evaluation the pages quote their speedups against
 * (ParaRNN page, abstract and Fig. 2 caption: speedup over sequential
 * application; DEER summary page, results: sequential GRU at L = 2^20), and
 * the exact answer Newton converges to.  It exposes only B*H-fold
 * parallelism.  Arguments, layouts and the cell as for pararnn_gru_forward
 * (no tolerance, cap, info, trace or workspace).
 */
int pararnn_gru_sequential(int64_t B, int64_t L, int64_t H,
                           const float *pz, const float *pr, const float *pc,
                           const float *uz, const float *ur, const float *uc,
                           const float *h0, float *h, void *stream);

/*
 * Sequential application of the LSTM-style cell (as above; arguments as for
 * pararnn_lstm_forward without tolerance, cap, info, trace or workspace).
 */
int pararnn_lstm_sequential(int64_t B, int64_t L, int64_t H,
                            const float *pi, const float *pf, const float *po,
                            const float *pg, const float *ui, const float *uf,
                            const float *uo, const float *ug, const float *h0,
                            const float *c0, float *h, float *c, void *stream);

/*
 * For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation): the GRU
 * Newton forward of pararnn_gru_forward from h = 0 (no initial iterate),
 * with its other arguments, results and errors, but no workspace argument.  Its workspace is a static device
 * array of the library, PARARNN_NOALLOC_SCRATCH_BYTES bytes on each device
 * it runs on, held until the process ends.  The first call on a device looks
 * up the array's address (with that device current) and zero-fills it with
 * one kernel on `stream`; no call allocates or frees anything.  A shape
 * whose workspace (pararnn_workspace_bytes(PARARNN_OP_GRU_FORWARD, ...))
 * exceeds the array returns PARARNN_ERR_TOO_LARGE before anything is
 * enqueued.  Every call on a device shares the one array: calls that overlap
 * in time on one device (other streams, other threads) race on it and must
 * not be issued; consecutive calls, in any order of shapes, are fine.
 * The device is the current one, which must be the device of `stream`.
 */
#define PARARNN_NOALLOC_SCRATCH_BYTES (64u << 20)
int pararnn_gru_forward_noalloc(int64_t B, int64_t L, int64_t H,
                                const float *pz, const float *pr, const float *pc,
                                const float *uz, const float *ur, const float *uc,
                                const float *h0, float *h, float tol, int32_t max_iter,
                                int32_t *info, float *trace, void *stream);

/*
 * Operators around the recurrences
 * --------------------------------
 * What a sequence model built on the recurrences needs next to them: linear
 * attention with a decay per head (a linear recurrence with a matrix state),
 * layer norm and the embedding lookup, each with its gradient.  Tensors are
 * fp32 or bf16 (`dtype`, all sequence tensors of a call alike); states,
 * decays, norm weights and statistics are always fp32, and so is every sum.
 * bf16 results are rounded to nearest even, once but in linear attention,
 * which says below what else it rounds.  Outputs are dense and must not alias
 * inputs unless stated.  Workspaces follow the rules above and may
 * be shared with every other entry point.  Results do not depend on timing:
 * the same inputs give the same bits.
 */
enum { PARARNN_F32 = 0, PARARNN_BF16 = 1 };

/*
 * Linear attention with decay: for each batch row and head, with g the head's
 * log decay (g <= 0; -infinity forgets everything at once),
 *     S_t = e^g S_{t-1} + k_t^T v_t,   o_t = scale q_t S_t,   S_{-1} = state.
 * q, k: [B, L, H, dk]; v, o: [B, L, H, dv]; state, out_state: [B, H, dk, dv]
 * fp32 (state NULL: zeros; out_state NULL: not wanted; out_state may be
 * state itself, but not overlap it otherwise).  log_decay: [H] fp32.
 * 1 <= dk, dv <= 256 (above: PARARNN_ERR_UNSUPPORTED).  B H is below 2^24, or
 * 2^24 over the column blocks of 64 in dv (three times those of the wider of
 * dk and dv in the backward pass).
 * strides: HOST array of {batch row, position, head} strides in elements for
 * q, k and v in turn (9 values), not negative, a position's below 2^22; the
 * last dimension is dense.  NULL: dense tensors (H max(dk, dv) < 2^22).
 * Operands whose rows are 16-byte aligned move faster.
 * A value that is not finite at position t of q, k or v affects no output
 * before t; from t on the affected outputs are not finite (an infinity may
 * come out as NaN).
 * Precision: states are carried in fp32, with the relative accuracy of fp32
 * whatever the decay.  fp32 products are formed of three parts of 8 bits, of
 * which the three smallest of nine products are left out (2^-23 of a product).
 * With bf16 tensors whole sequences round two things to bf16 on the way to an
 * output or a gradient: the copy of the state that a row is multiplied with
 * (heads above 32), and the weights of the positions within a chunk of 64;
 * outputs are then off by about 2.3e-3 in the 2-norm, of which their own
 * rounding is 1.7e-3.  States are not affected, nor is the single token's step.
 * How long a chunk is (32 positions keep the weights to 16 bits) and how many
 * pieces a sequence is walked in depend on L, on the head sizes and on B H, so
 * the same row may come out with other last bits in a batch of another size.
 */
size_t pararnn_linattn_workspace_bytes(int32_t backward, int32_t dtype, int64_t B, int64_t L, int64_t H, int64_t dk,
                                       int64_t dv);
int pararnn_linattn_forward(int32_t dtype, int64_t B, int64_t L, int64_t H, int64_t dk, int64_t dv,
                            const void *q, const void *k, const void *v, const int64_t *strides,
                            const float *log_decay, const float *state, float scale, void *o,
                            float *out_state, void *ws, size_t ws_bytes, void *stream);

/*
 * Its gradients for a loss with dLoss/do = grad_o ([B, L, H, dv]) and
 * dLoss/d(final state) = grad_out_state ([B, H, dk, dv] or NULL for zeros):
 *     D_t = e^g D_{t+1} + scale q_t^T do_t   (plus grad_out_state at L-1),
 *     dq_t = scale do_t S_t^T,  dk_t = v_t D_t^T,  dv_t = k_t D_t,
 *     dstate = e^g D_0.
 * The log decay is a constant of the model and gets no gradient.
 * strides: as above for q, k, v and grad_o (12 values).  grad_state: NULL if
 * not wanted; it must not overlap state or grad_out_state.
 */
int pararnn_linattn_backward(int32_t dtype, int64_t B, int64_t L, int64_t H, int64_t dk, int64_t dv,
                             const void *q, const void *k, const void *v, const void *grad_o,
                             const int64_t *strides, const float *log_decay, const float *state,
                             const float *grad_out_state, float scale, void *grad_q, void *grad_k,
                             void *grad_v, float *grad_state, void *ws, size_t ws_bytes, void *stream);

/*
 * One token of the recurrence above (its form for decoding): q, k [B, H, dk],
 * v, o [B, H, dv], state and out_state [B, H, dk, dv], both required;
 * out_state may be state itself.  strides: as above with the position's
 * stride ignored, or NULL.  No workspace.
 */
int pararnn_linattn_step(int32_t dtype, int64_t B, int64_t H, int64_t dk, int64_t dv, const void *q,
                         const void *k, const void *v, const int64_t *strides, const float *log_decay,
                         const float *state, float scale, void *o, float *out_state, void *stream);

/*
 * Layer norm over the last dimension of [rows, D], after an optional residual
 * sum: s = x + residual (rounded to dtype; s = x without one),
 *     y = (s - mean) rstd weight + bias,  rstd = 1 / sqrt(var + eps)
 * with the biased variance.  weight, bias: [D] fp32 or NULL (one, zero).
 * sum: [rows, D] output, given exactly when residual is.  mean, rstd: [rows]
 * fp32 outputs or NULL.  eps >= 0; D < 2^24.
 */
int pararnn_layernorm_forward(int32_t dtype, int64_t rows, int64_t D, const void *x, const void *residual,
                              const float *weight, const float *bias, float eps, void *sum, void *y,
                              float *mean, float *rstd, void *stream);

/*
 * Its gradients: s is the forward's sum (x without a residual), mean and rstd
 * its statistics; grad_sum: [rows, D], what reaches s past the norm, or NULL.
 *     xh = (s - mean) rstd, g = grad_y weight,
 *     grad_x = rstd (g - mean(g) - xh mean(g xh)) + grad_sum
 * (the gradient of x and of the residual alike), grad_weight = sum over rows
 * of grad_y xh, grad_bias = sum over rows of grad_y, [D] fp32 each or NULL.
 * grad_x may be grad_y or grad_sum itself.
 * ws: pararnn_layernorm_workspace_bytes (unused, may be NULL, when neither
 * weight nor bias gradient is wanted).
 */
size_t pararnn_layernorm_workspace_bytes(int64_t rows, int64_t D);
int pararnn_layernorm_backward(int32_t dtype, int64_t rows, int64_t D, const void *s, const float *weight,
                               const float *mean, const float *rstd, const void *grad_y,
                               const void *grad_sum, void *grad_x, float *grad_weight, float *grad_bias,
                               void *ws, size_t ws_bytes, void *stream);

/*
 * Embedding lookup: out[n] = scale table[ids[n]], table [V, D], out [N, D];
 * ids: int32 or int64 (id_bytes 4 or 8).  An id outside [0, V) reads nothing
 * and gives a row of NaN.  N < 2^28 - 16, V < 2^30, D < 2^24,
 * N D < 2^36.
 */
int pararnn_embedding_forward(int32_t dtype, int64_t N, int64_t V, int64_t D, const void *ids,
                              int32_t id_bytes, const void *table, float scale, void *out, void *stream);

/*
 * Its gradient: grad_table[r] = scale * sum of grad[n] over the n with
 * ids[n] = r in ascending n, for every row r of [V, D] (zeros where no id
 * names the row).  The ids are sorted, so the order of the sums is fixed.
 * padding_idx: a row that gets zeros, or -1.  Ids outside [0, V) are left out.
 */
size_t pararnn_embedding_workspace_bytes(int64_t N, int64_t V, int64_t D);
int pararnn_embedding_backward(int32_t dtype, int64_t N, int64_t V, int64_t D, const void *ids,
                               int32_t id_bytes, const void *grad, float scale, int64_t padding_idx,
                               void *grad_table, void *ws, size_t ws_bytes, void *stream);

/*
 * The gated delta rule: for each batch row and head, with g_t <= 0 the log
 * decay and b_t the write strength of the position,
 *     S_t = e^(g_t) (I - b_t k_t^T k_t) S_{t-1} + b_t k_t^T v_t,
 *     o_t = scale q_t S_t,   S_{-1} = state.
 * It is meant for keys of about unit length and b in [0, 1] (or [0, 2]): for
 * b |k|^2 above 2 the state grows along k.  A position with b = 0 and g = 0
 * leaves the state as it is, whatever finite v it has (padding).
 * q, k: [B, L, Hk, dk]; v, o: [B, L, H, dv], Hk a divisor of H: head h shares
 * q and k of head h / (H / Hk); log_decay, beta: [B, L, H] fp32; state,
 * out_state: [B, H, dk, dv] fp32 (state NULL: zeros; out_state NULL: not
 * wanted; out_state may be state itself).  No output may otherwise lie between
 * the first and the last element of another tensor of the call (refused; so
 * for the gradients and the single token).
 * 1 <= dk, dv <= 256 (above: PARARNN_ERR_UNSUPPORTED).  B H ceil(L / 32) is
 * below 2^26 - 4 (backward 2^22, and where heads share keys B L Hk dk below
 * 2^32) and B H below 2^23 over the blocks of 64 in the wider of dk and dv.
 * strides: HOST array of {batch row, position, head} strides in elements for
 * q, k, v, log_decay and beta in turn (15 values), not negative, those of
 * positions in q, k and v below 2^22; the last dimension of q, k and v is
 * dense.  NULL: dense tensors (H max(dk, dv) < 2^22).  Operands whose rows are
 * 16-byte aligned move faster.
 * A value that is not finite at position t of q changes o_t alone; in v it
 * makes its column of o NaN from t on and that column of the final state; in
 * k, log_decay or beta (a log decay of -infinity is one that forgets
 * everything, and finite) it makes every output of the head from t on NaN and
 * its final state.  No output before t is affected.  A key whose squares add
 * up past fp32 counts as not finite.
 * Precision: fp32 throughout (products formed of three parts of 8 bits, of which
 * the three smallest of nine products are left out: 2^-23 of a product), and
 * one rounding of each output to bf16.  What a chunk of 32 positions leaves of a
 * state that its keys write over (and of the state's gradient) is a difference, off
 * by 2^-22 or so of what was there.
 * Long sequences of few rows are walked in segments, whose number depends on
 * L, B H, the type and the heads' widths: the same row may get other last bits in
 * another batch.  The same call gives the same bits.  (A segment multiplies with the
 * matrix that it takes any state through: for keys and beta with which the state
 * grows, that may pass fp32 where the state itself does not.)
 */
size_t pararnn_delta_workspace_bytes(int32_t backward, int32_t dtype, int64_t B, int64_t L, int64_t H, int64_t Hk,
                                     int64_t dk, int64_t dv);
int pararnn_delta_forward(int32_t dtype, int64_t B, int64_t L, int64_t H, int64_t Hk, int64_t dk, int64_t dv,
                          const void *q, const void *k, const void *v, const float *log_decay, const float *beta,
                          const int64_t *strides, const float *state, float scale, void *o, float *out_state,
                          void *ws, size_t ws_bytes, void *stream);

/*
 * Its gradients for a loss with dLoss/do = grad_o ([B, L, H, dv]) and
 * dLoss/d(final state) = grad_out_state ([B, H, dk, dv] or NULL for zeros):
 * grad_q, grad_k [B, L, Hk, dk] (summed over the heads that share them),
 * grad_v [B, L, H, dv], grad_log_decay and grad_beta [B, L, H] fp32 (either may
 * be NULL) and grad_state [B, H, dk, dv] or NULL.  strides: as above and those of grad_o after them (18
 * values).  Where a value is not finite, the gradients are not defined.
 * Precision as above: fp32 throughout, and one rounding of each gradient.
 * The workspace grows with B H L (heads of 128x128, bf16: 3.7 KB a position and
 * head, 0.96 GB for B=8, L=2048, H=16; fp32 5.7; where heads share keys 8 dk bytes
 * more), the forward pass's is 0.4 KB a position and head.
 */
int pararnn_delta_backward(int32_t dtype, int64_t B, int64_t L, int64_t H, int64_t Hk, int64_t dk, int64_t dv,
                           const void *q, const void *k, const void *v, const float *log_decay, const float *beta,
                           const void *grad_o, const int64_t *strides, const float *state,
                           const float *grad_out_state, float scale, void *grad_q, void *grad_k, void *grad_v,
                           float *grad_log_decay, float *grad_beta, float *grad_state, void *ws, size_t ws_bytes,
                           void *stream);

/*
 * One token of the recurrence (its form for decoding): q, k [B, Hk, dk], v, o
 * [B, H, dv], log_decay, beta [B, H], state and out_state [B, H, dk, dv], both
 * required; out_state may be state itself.  strides: as above with the
 * positions' ignored, or NULL.  No workspace.  A value that is not finite goes
 * where the formula takes it: what is NaN after a sequence may be infinite here.
 */
int pararnn_delta_step(int32_t dtype, int64_t B, int64_t H, int64_t Hk, int64_t dk, int64_t dv, const void *q,
                       const void *k, const void *v, const float *log_decay, const float *beta, const int64_t *strides,
                       const float *state, float scale, void *o, float *out_state, void *stream);

/*
 * Norms of queries and keys for each head, with the position rotation in the
 * same pass.  For every row x of d elements of q [B, L, Hq, d] and k
 * [B, L, Hk, d] (k NULL and Hk = 0: q alone):
 *     r = 1 / sqrt(mean(x^2) + eps)  (PARARNN_NORM_RMS) or
 *     r = 1 / sqrt(sum(x^2) + eps)   (PARARNN_NORM_L2),   n = x r w,
 * and the first R elements of n are turned in pairs by the position's angles:
 *     y_c = n_c cos_i - n_c' sin_i,  y_c' = n_c' cos_i + n_c sin_i,
 * with c, c' = i, i + R / 2, or 2 i, 2 i + 1 (interleaved).  weight: [d] fp32 of
 * each tensor, or NULL for ones.  table: [P, R] fp32, a position's R / 2
 * cosines and then its R / 2 sines; R even, R <= d; R = 0 (table NULL): no
 * rotation.  positions: [B, L] int32 or int64 (position_bytes 4 or 8), or NULL
 * for 0 .. L-1; a position outside [0, P) turns the rotated elements to NaN
 * (and reads nothing).
 * yq, yk: dense outputs in dtype; rq [B, L, Hq], rk [B, L, Hk]: r, fp32, or NULL.
 * strides: HOST array of {batch row, position, head} strides of q and k (6
 * values, not negative, last dimension dense) or NULL for dense tensors.
 * No output (here and of the gradients) may lie between the first and the last
 * element of another tensor of the call (refused).
 * 2 <= d <= 256 (above: PARARNN_ERR_UNSUPPORTED), eps >= 0, B L (Hq + Hk) < 2^28.
 */
enum { PARARNN_NORM_RMS = 0, PARARNN_NORM_L2 = 1 };
int pararnn_headnorm_forward(int32_t dtype, int64_t B, int64_t L, int64_t Hq, int64_t Hk, int64_t d, const void *q,
                             const void *k, const int64_t *strides, const float *wq, const float *wk,
                             const float *table, int64_t P, int64_t R, const void *positions,
                             int32_t position_bytes, int32_t kind, int32_t interleaved, float eps, void *yq, void *yk,
                             float *rq, float *rk, void *stream);

/*
 * Its gradients: with the rotation undone on the gradients of the outputs (g),
 *     dw = sum over rows of g x r,  dx = r (g w - x r m(g w x r)),
 * m the mean or the sum.  strides: of q, k, grad_yq and grad_yk (12 values) or
 * NULL; rq, rk: the forward pass's; grad_q, grad_k: dense; grad_wq, grad_wk: [d]
 * fp32 or NULL (ws: unused, may be NULL, when both are).
 */
size_t pararnn_headnorm_workspace_bytes(int64_t B, int64_t L, int64_t Hq, int64_t Hk, int64_t d);
int pararnn_headnorm_backward(int32_t dtype, int64_t B, int64_t L, int64_t Hq, int64_t Hk, int64_t d, const void *q,
                              const void *k, const void *grad_yq, const void *grad_yk, const int64_t *strides,
                              const float *wq, const float *wk, const float *rq, const float *rk, const float *table,
                              int64_t P, int64_t R, const void *positions, int32_t position_bytes, int32_t kind,
                              int32_t interleaved, void *grad_q, void *grad_k, float *grad_wq, float *grad_wk,
                              void *ws, size_t ws_bytes, void *stream);

/* Short text for a status code (static storage). */
const char *pararnn_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* PARARNN_H */
