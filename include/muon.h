/* muon.h -- C ABI of libmuon: the Muon optimizer step with Newton-Schulz
 * orthogonalisation (standard, Gram and stabilised Gram forms) on NVIDIA B200.
 *
 * Sources of the operations (web pages, cited by title and section):
 *   [Moonlight] "Moonlight 16B Guide: Scalable MoE & Muon Optimizer":
 *       box "Scalable Muon Optimizer Step" (steps 1-4); section "The
 *       Newton-Schulz Iteration for Matrix Orthogonalization"; "Innovation 1:
 *       Decoupled Weight Decay in Muon"; "Innovation 2: Per-Parameter Update
 *       Scale Alignment"; listing "End-to-End PyTorch Implementation".
 *   [GramNS] "Gram Newton-Schulz" news write-up (Machine Heart, m.web578.cn):
 *       standard iteration and its three products; Gram rewrite; stabilised
 *       variant (float16 Gram iteration, restart after step 2).
 *
 * Conventions shared by every entry point
 *   - Every matrix is dense row-major in device memory (leading dimension =
 *     cols) and 16-byte aligned.  The caller owns all memory, including the
 *     workspace; the library allocates nothing and carries no data from one
 *     call to the next (it only caches per-device launch settings on first
 *     use: the SM count, shared-memory opt-ins, how many CTA pairs fit).
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *     default stream).  They take no lock on the launch path; the opt-in
 *     profiler and the allocation-free entry point's scratch lookup
 *     take a mutex.  The return value reports argument
 *     and launch errors only (MUON_OK, MUON_ERR_*).  Conditions found on the
 *     device are OR-ed into the optional per-matrix status words (device int
 *     array, one per matrix, zeroed by the call): MUON_STATUS_NONFINITE when
 *     an orthogonalised matrix holds Inf/NaN, MUON_STATUS_TIMEOUT when a
 *     device-side wait gave up (the kernel then returned without finishing).
 *   - A matrix of storage shape rows x cols is orthogonalised in its
 *     short-side-first orientation n x m (n = min, m = max): tall matrices
 *     are transposed on the way in and back on the way out [Moonlight
 *     listing, "ensure m <= n"; GramNS, X in R^{n x m}].
 *   - Calls that overlap on the GPU must not share a workspace.
 */
#ifndef MUON_H_
#define MUON_H_

#include <stddef.h>

#if defined(__GNUC__)
#define MUON_API __attribute__((visibility("default")))
#else
#define MUON_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MUON_BF16 = 0, MUON_FP16 = 1, MUON_FP32 = 2 } muon_dtype;

/* Which form of the Newton-Schulz iteration runs [GramNS]:
 *   STANDARD         X <- a X + (b A + c A^2) X, A = X X^T, per iteration
 *   GRAM             naive Gram form: R = X0 X0^T; Q_k = a I + b R + c R^2;
 *                    Q_acc <- Q_k Q_acc; R <- Q_k R Q_k; X = Q_acc X0
 *   GRAM_STABILIZED  Gram form restarted after iteration restart_after (and,
 *                    if restart_every > 0, every restart_every iterations
 *                    after it): X0 <- Q_acc X0, R <- X0 X0^T, Q_acc <- I */
typedef enum { MUON_NS_STANDARD = 0, MUON_NS_GRAM = 1, MUON_NS_GRAM_STABILIZED = 2 } muon_ns_mode;

enum {
  MUON_OK = 0,
  MUON_ERR_INVALID = -1,     /* null pointer, bad size/shape/count, misaligned pointer, bad enum */
  MUON_ERR_UNSUPPORTED = -2, /* dtype combination the kernels do not implement */
  MUON_ERR_WORKSPACE = -3,   /* ws_bytes below muon_*_workspace_size's minimum for one matrix */
  MUON_ERR_CUDA = -4         /* a CUDA launch or tensor-map encode failed */
};
#define MUON_STATUS_NONFINITE 1
#define MUON_STATUS_TIMEOUT 2

/* Newton-Schulz parameters.
 *   iters          K >= 1 iterations
 *   coeffs         host array of 3*iters floats, (a_k, b_k, c_k) per iteration;
 *                  the quintic (3.4445, -4.7750, 2.0315) or the cubic
 *                  (1.5, -0.5, 0) of [Moonlight, NS section]
 *   mode           muon_ns_mode
 *   restart_after  GRAM_STABILIZED only: iteration after which the Gram
 *                  matrix is rebuilt (1 <= restart_after < iters; 2 in [GramNS])
 *   restart_every  GRAM_STABILIZED only: 0 = rebuild once; e > 0 = also after
 *                  iterations restart_after + e, + 2e, ... before the last
 *                  (the periodic reading of [GramNS]'s "re-initialise")
 *   eps            X0 = U / (||U||_F + eps)  [Moonlight, NS section; listing eps]
 *   compute_dtype  MUON_BF16 or MUON_FP16: tcgen05 tensor cores, fp32
 *                  accumulate, 16-bit storage of X, A, B between the products
 *                  of the standard form; MUON_FP32: fp32 storage throughout
 *                  (any mode), products as 3xTF32 on the tensor cores (operands
 *                  split into TF32 hi + lo, fp32 sums per 32-deep k-block) when
 *                  min(rows, cols) >= 256, else fp32 FFMA (a matrix whose whole
 *                  chain fits in one block's shared memory runs it in one launch)
 *   gram_dtype     Gram modes on tensor cores: the 16-bit type of every matrix
 *                  the Gram chain stores (R, Q, Q_acc, X0 and the restart X),
 *                  MUON_FP16 (the stabilised variant's float16) or MUON_BF16 */
typedef struct {
  int iters;
  const float* coeffs;
  int mode;
  int restart_after;
  float eps;
  int compute_dtype;
  int gram_dtype;
  int restart_every;
} muon_ns_params;

/* One group of `count` parameters that share storage shape rows x cols.
 *   W  host array of `count` device pointers, rows x cols of w_dtype; updated
 *   G  host array of device pointers, rows x cols of g_dtype; read only
 *   M  host array of device pointers, rows x cols fp32 momentum; updated */
typedef struct {
  int rows, cols, count;
  int w_dtype, g_dtype;
  void* const* W;
  const void* const* G;
  float* const* M;
} muon_group;

/* Optimizer hyper-parameters of one step.
 *   lr, weight_decay  W <- (1 - lr wd) W - lr s(W) O   [Moonlight, Innovation 1, box step 4]
 *   momentum, nesterov  M <- mu M + (1 - mu) G [Moonlight, box step 1];
 *                     U = nesterov ? (1 - mu) G + mu M : M
 *   scale_coef        s(W) = scale_coef sqrt(max(rows, cols)) [Moonlight, Innovation 2]
 *   ns                the orthogonalisation */
typedef struct {
  float lr, momentum, weight_decay, scale_coef;
  int nesterov;
  muon_ns_params ns;
} muon_hparams;

/* Workspace bytes that let muon_step process every group in a single chunk
 * (the fastest setting).  A smaller workspace is accepted down to
 * muon_workspace_min; groups are then processed in chunks.  Returns 0 on
 * invalid arguments. */
MUON_API size_t muon_workspace_size(const muon_group* groups, int n_groups, const muon_hparams* hp);
MUON_API size_t muon_workspace_min(const muon_group* groups, int n_groups, const muon_hparams* hp);

/* One Muon step over n_groups groups  [Moonlight, box steps 1-4]:
 *   M <- mu M + (1 - mu) G;  U = nesterov ? (1 - mu) G + mu M : M
 *   O = NS(U / (||U||_F + eps))   (oriented n x m, see muon_ns_params)
 *   W <- (1 - lr wd) W - lr scale_coef sqrt(max(rows, cols)) O
 * Groups whose matrices orient to the same n x m (e.g. 2048 x 1408 and
 * 1408 x 2048) are orthogonalised together.
 *   ws, ws_bytes       device workspace (256-byte aligned)
 *   status_per_matrix  optional device int array, one word per matrix in
 *                      group order; zeroed, then OR-ed with MUON_STATUS_* */
MUON_API int muon_step(const muon_group* groups, int n_groups, const muon_hparams* hp, void* ws, size_t ws_bytes,
              int* status_per_matrix, void* stream);

/* One group of `count` row-major matrices, each tiled by down x across blocks
 * of rows x cols: a head's rows of an attention projection, its columns of the
 * output projection, gate and up of a fused weight, the experts of a stack.  As
 * muon_group, with the row pitch (in elements, at least across * cols) of the
 * matrices, and pointers that need no more than their elements' alignment
 * (rows that all start on 16 bytes are moved by 16-byte accesses, others element
 * by element).  Nothing outside the blocks is read or written; blocks of one
 * call must not overlap.  Blocks count in the order of the groups, their
 * matrices, block rows and block columns; a group has at most 2^20. */
typedef struct {
  int rows, cols, count;
  int down, across;
  int w_dtype, g_dtype;
  long long ld_w, ld_g, ld_m;
  void* const* W;
  const void* const* G;
  float* const* M;
} muon_block_group;

/* muon_step with every block as a matrix of its own: its own norm, its own
 * orthogonalisation, and the update scale sqrt(max(rows, cols)) of the block.
 * The results are muon_step's on dense copies of the blocks, bit for bit, except
 * for blocks with min(rows, cols) <= 128 and max <= 4096 in 16-bit standard chains
 * of at most 64 iterations: they run in one launch, which adds up X X^T in another
 * order, and differ by the chain's roundings.  That launch takes up to 512 blocks
 * whatever the workspace holds: the sizes count such blocks like others, and
 * muon_blocks_workspace_min is enough for its full speed. */
MUON_API size_t muon_blocks_workspace_size(const muon_block_group* groups, int n_groups, const muon_hparams* hp);
MUON_API size_t muon_blocks_workspace_min(const muon_block_group* groups, int n_groups, const muon_hparams* hp);
MUON_API int muon_step_blocks(const muon_block_group* groups, int n_groups, const muon_hparams* hp, void* ws,
                              size_t ws_bytes, int* status_per_block, void* stream);

/* In-place orthogonalisation of `count` matrices of storage shape rows x cols
 * and dtype `dtype` (X[i] is a device pointer; O replaces X in the same
 * orientation).  This is the listing's newton_schulz_orthogonalize without
 * the optimizer around it. */
MUON_API size_t muon_ns_workspace_size(int count, int rows, int cols, const muon_ns_params* ns);
MUON_API int muon_ns_batched(void* const* X, int count, int rows, int cols, int dtype, const muon_ns_params* ns, void* ws,
                    size_t ws_bytes, int* status_per_matrix, void* stream);

/* muon_ns_batched without a caller workspace, for callers that cannot
 * allocate device memory when they orthogonalise: a host whose caching
 * allocator already owns the GPU's memory (a raw cudaMalloc would fail or
 * fragment its pool), a loop that forbids allocation after start-up, or a
 * plugin that receives only input/output pointers.  The pages have no
 * counterpart of this entry point; it is a library convenience.
 *
 * The workspace is a fixed array of MUON_NOALLOC_SCRATCH_BYTES inside the
 * library, present on every GPU that loads the library until the process
 * exits.  The call allocates and frees nothing.  A shape whose one-matrix
 * workspace (muon_ns_workspace_size(1, rows, cols, ns)) exceeds the array is
 * rejected with MUON_ERR_WORKSPACE; larger counts of fitting matrices are
 * processed in chunks.  Results equal muon_ns_batched's.
 *
 * A call outside a stream capture looks up the array's device address on
 * the current device (cudaGetSymbolAddress) and remembers it; a call on a
 * capturing stream uses the address remembered by the last uncaptured call on
 * that device (none: MUON_ERR_CUDA), so make one uncaptured call before
 * capturing, and again after a cudaDeviceReset.  Every call uses the same
 * array, which keeps the previous call's contents (the call resets what must
 * start at zero): calls that can overlap on the GPU (other streams, other
 * host threads) race on it and must be serialised by the caller, e.g. on one
 * stream. */
#define MUON_NOALLOC_SCRATCH_BYTES (64u << 20)
MUON_API int muon_ns_batched_noalloc(void* const* X, int count, int rows, int cols, int dtype,
                                     const muon_ns_params* ns, int* status_per_matrix, void* stream);

/* ---------------------------------------------------------------- expert layers
 * What produces the gradients of a mixture-of-experts layer's weights: tokens
 * sorted by expert and back, and the experts' products with their gradients.
 *
 * A router sends each of `tokens` tokens to `topk` of `experts` experts.  An
 * assignment is a pair (t, j); its number is t * topk + j.
 *   offsets  device int array, experts + 1: expert e owns the sorted rows
 *            [offsets[e], offsets[e+1])
 *   slot     device int array, tokens x topk: the sorted row of an assignment,
 *            or a negative number for an assignment that no expert takes
 *   source   device int array, tokens x topk: the assignment behind every sorted
 *            row; behind the last row, those that no expert takes, in order
 * Matrices are row-major with a row pitch ld >= cols in elements and any
 * alignment of their elements; rows that start on 16 bytes are moved faster,
 * and the 16-bit products' operands need it for the tensor cores (see there).
 * Sorted rows that no expert owns are neither read into a result nor written.  All sums are held
 * in fp32 and rounded once, in an order that does not change from call to call.
 * Rows, columns and tokens * topk are at most 2^30, experts at most 1024 and
 * experts * outer (all weights' rows) at most 2^34.  What a call writes overlaps
 * nothing that it reads, unless its description says otherwise.
 *
 * muon_expert_sort: ids is tokens x topk of int32 or int64 (id_bytes 4 or 8),
 * row pitch ld_ids; an id outside [0, experts) goes to no expert.  The sort is
 * stable: an expert's rows keep the order of their assignments. */
MUON_API size_t muon_expert_sort_workspace_size(int tokens, int topk, int experts);
MUON_API int muon_expert_sort(const void* ids, int id_bytes, long long ld_ids, int tokens, int topk, int experts,
                              int* offsets, int* slot, int* source, void* ws, size_t ws_bytes, void* stream);

/* xs[slot[t, j]] = x[t].  x is tokens x cols, xs is rows x cols; slots of one
 * call are distinct, and those outside [0, rows) are skipped (here and below).
 * Its gradient is muon_expert_combine without weights. */
MUON_API int muon_expert_gather(const void* x, long long ld_x, const int* slot, int tokens, int topk, int cols, int dtype,
                                void* xs, long long ld_xs, long long rows, void* stream);

/* y[t] = sum_j weights[t, j] * ys[slot[t, j]], j ascending; zero for a token
 * that no expert takes.  weights is tokens x topk of w_dtype, dense; NULL: ones. */
MUON_API int muon_expert_combine(const void* ys, long long ld_ys, long long rows, const int* slot, const void* weights,
                                 int w_dtype, int tokens, int topk, int cols, int dtype, void* y, long long ld_y,
                                 void* stream);

/* The gradients of muon_expert_combine:
 *   dys[slot[t, j]]  = weights[t, j] * dy[t]
 *   dweights[t, j]   = <dy[t], ys[slot[t, j]]>, zero for an assignment that no expert takes
 * dweights (of w_dtype) may be NULL; ys is then not read.  dys may be ys. */
MUON_API int muon_expert_combine_backward(const void* dy, long long ld_dy, const void* ys, long long ld_ys, long long rows,
                                          const int* slot, const void* weights, int w_dtype, int tokens, int topk,
                                          int cols, int dtype, void* dys, long long ld_dys, void* dweights, void* stream);

/* The experts' products.  W[e] is outer x inner at w + e * stride_w, row pitch
 * ld_w; xs is rows x inner, ys and dys are rows x outer, one dtype for all.
 * Offsets are clamped to [0, rows] and read on the device: no count reaches the
 * host.  They may run backwards; a row that several experts then own gets one
 * expert's product, of no particular one.
 *   muon_expert_product       y[p]   = W[e] xs[p]            for e's rows p
 *   muon_expert_input_grad    dxs[p] = W[e]^T dys[p]         for e's rows p
 *   muon_expert_weight_grad   dW[e]  = sum_p dys[p] xs[p]^T  over e's rows p
 * dW[e] (outer x inner at dw + e * stride_dw) has the operands' type or fp32; an
 * expert without rows gets zeros.  accumulate (fp32 dW only) adds to dW instead.
 * 16-bit operands run on the tensor cores where base, pitch and expert stride are
 * multiples of 16 bytes (and the stride is not 0).  Others are first copied into
 * such rows in the workspace, where it holds muon_expert_workspace_size bytes;
 * without it, where that is 0 (small products), and in fp32 the CUDA cores run.
 * status: one optional device word, zeroed by the call, MUON_STATUS_TIMEOUT when
 * a device-side wait gave up and part of the result was not written.  Without a word
 * nothing reports that, as with the status words of muon_step. */
enum { MUON_EXPERT_PRODUCT = 0, MUON_EXPERT_INPUT_GRAD = 1, MUON_EXPERT_WEIGHT_GRAD = 2 };
/* Workspace bytes with which the product `kind` of these operands runs on the
 * tensor cores (a: xs or dys, b: w, or xs for the weight gradient); 0: none needed
 * or none used.  With it the product is summed by the tensor cores, whose fp32
 * additions truncate (the runs of an fp32 weight gradient aside, an error that grows
 * with the length of the sum: 1.9e-5 relative at 16384 terms), without it by fused
 * multiply-adds that round to nearest: the results differ by those roundings. */
MUON_API size_t muon_expert_workspace_size(int kind, const void* a, long long ld_a, const void* b, long long ld_b,
                                           long long stride_b, int experts, long long rows, int inner, int outer,
                                           int dtype);
MUON_API int muon_expert_product(const void* xs, long long ld_xs, const void* w, long long ld_w, long long stride_w,
                                 const int* offsets, int experts, long long rows, int inner, int outer, int dtype,
                                 void* y, long long ld_y, void* ws, size_t ws_bytes, int* status, void* stream);
MUON_API int muon_expert_input_grad(const void* dys, long long ld_dys, const void* w, long long ld_w, long long stride_w,
                                    const int* offsets, int experts, long long rows, int inner, int outer, int dtype,
                                    void* dxs, long long ld_dxs, void* ws, size_t ws_bytes, int* status, void* stream);
MUON_API int muon_expert_weight_grad(const void* dys, long long ld_dys, const void* xs, long long ld_xs,
                                     const int* offsets, int experts, long long rows, int inner, int outer, int dtype,
                                     void* dw, long long ld_dw, long long stride_dw, int dw_dtype, int accumulate,
                                     void* ws, size_t ws_bytes, int* status, void* stream);

/* Algorithmic FLOPs of one orthogonalisation of a rows x cols matrix, every
 * product counted as 2 * rows * cols * inner [GramNS cost list]. */
MUON_API double muon_ns_flops(int rows, int cols, const muon_ns_params* ns);

/* Opt-in launch profiler (tracing aid).  Between muon_profile_begin() and
 * muon_profile_end(), every kernel the library launches (the one to three of an
 * expert-layer call together) is bracketed by a pair
 * of CUDA events recorded on the launch stream; this is the only state the
 * library keeps between calls, and only while profiling is on.
 * muon_profile_end synchronises on those events and fills up to max_entries
 * rows, one per kernel kind that ran: its name, launch count, summed device
 * time, and for those launches
 *   flops       algorithmic FLOPs: every product 2 * M * N * K, the full
 *               product even where only a triangle is computed [GramNS cost list]
 *   exec_flops  FLOPs the kernels execute: tensor-core MMAs over whole tiles
 *               (zero padding included), only the tiles of a symmetric
 *               product's upper triangle, three TF32 MMAs per 3xTF32 product;
 *               equal to flops for the other kernels
 *   bytes       algorithmic bytes (each operand read once, result written once)
 * Returns the number of rows written, or a MUON_ERR_* code. */
typedef struct {
  const char* kernel;
  int launches;
  double ms;
  double flops;
  double exec_flops;
  double bytes;
} muon_profile_entry;
MUON_API int muon_profile_begin(void);
MUON_API int muon_profile_end(muon_profile_entry* out, int max_entries);

/* Static text for a MUON_* return code or status bit set. */
MUON_API const char* muon_status_string(int code);

#ifdef __cplusplus
}
#endif
#endif /* MUON_H_ */
