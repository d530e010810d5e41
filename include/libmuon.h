/*
 * libmuon — the Muon / Aurora-Muon matrix-optimizer step on AMD Instinct
 * MI355X (gfx950), as a C-ABI shared library.
 *
 * The operations follow two web pages:
 *   [Aurora page]  "modded-nanogpt Track 3 优化实录：Aurora 行均衡 polar +
 *                  Contra-Muon + u/w-floor 将 3.28 验证损失推进到 3175 步"
 *                  (www.xxmr.cn/news/295280);
 *   [Track-1 page] "Modded-NanoGPT 纪录解读：U-Net 式跳跃连接与学习率翻倍如何将
 *                  124M GPT 训练压到 7.23 分钟" (www.trdm.cn/news/788905).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Matrices are row-major, in device memory the caller owns. A descriptor
 *    names one matrix: element (i, j) lives at ptr + i * ld + j (elements).
 *    ld >= cols. ptr must be aligned to the element size. A matrix with
 *    rows == 0 or cols == 0 is skipped (its ptr may be NULL).
 *  - Batches: every call takes n descriptors of mixed shapes and types; each
 *    matrix is processed on its own (its own norms, preconditioner and power
 *    iteration) and the batch is fused into shared kernel launches.
 *  - Limits: rows, cols <= 65536, min(rows, cols) <= 16384,
 *    rows * cols < 2^31 and ld <= 2^40 per matrix.
 *  - Precision: a matrix whose input is MUON_BF16 runs Newton-Schulz on bf16
 *    matrix cores with fp32 accumulation; a MUON_F32 input runs it with fp32
 *    matrix-core arithmetic throughout. Norms, the preconditioner, the power
 *    iteration and every scalar are fp32.
 *  - Errors: no exception crosses the ABI. Calls return a muon_status; a
 *    negative value is an error. All arguments are validated on the host
 *    before anything is enqueued: on any error nothing is enqueued and no
 *    caller buffer is touched. muon_last_error() gives a message. (With
 *    MUON_FLAG_CHECK_FINITE a read-only device pass also checks the input
 *    values; a non-finite one is reported the same way, no buffer written.)
 *  - Asynchrony: compute calls enqueue on the handle's stream and return.
 *    Inputs must stay valid and unmodified until that stream reaches the
 *    work. Device faults surface as MUON_ERR_HIP on a later call or on the
 *    caller's synchronisation.
 *  - Determinism: reductions run in a fixed order with no floating-point
 *    atomics; two calls on the same inputs give bitwise-equal results.
 *  - Threads: a handle is not thread-safe; use one handle per thread.
 */
#ifndef LIBMUON_H
#define LIBMUON_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
typedef enum {
  MUON_F32 = 0,
  MUON_BF16 = 1
} muon_dtype;

/* Status codes. */
typedef enum {
  MUON_OK = 0,
  MUON_ERR_INVALID_ARG = -1,      /* NULL pointer, bad count, bad config value */
  MUON_ERR_UNSUPPORTED_DTYPE = -2,/* dtype not in muon_dtype, or momentum not F32 */
  MUON_ERR_SHAPE_MISMATCH = -3,   /* grad/momentum/weight/out shapes differ, ld < cols, limits */
  MUON_ERR_ALLOC = -4,            /* device workspace allocation failed */
  MUON_ERR_HIP = -5,              /* a HIP runtime call failed */
  MUON_ERR_NO_DEVICE = -6,        /* no usable gfx950 device */
  MUON_ERR_TOO_LARGE = -7,        /* muon_update_static: the batch does not fit the static scratch */
  MUON_ERR_NONFINITE = -8         /* MUON_FLAG_CHECK_FINITE: an input element is NaN or Inf */
} muon_status_code;
typedef int muon_status;

/* One row-major device matrix (see conventions above). */
typedef struct {
  void*   ptr;
  int64_t rows;
  int64_t cols;
  int64_t ld;
  int32_t dtype; /* muon_dtype */
} muon_matrix;

/*
 * Step hyper-parameters. muon_config_default() fills the values the Aurora
 * page locks (§"完整的超参配置表" and the signature defaults in §"源码实现" and
 * §"组合优化栈"): ns_steps 12, (ns_a, ns_b, ns_c) = (2, -1.5, 0.5),
 * ns_eps 1e-7, pp_iterations 2, pp_beta 0.5, pp_eps 1e-7, mu 0.95,
 * nesterov 1, power_steps 5, contra 0.4, target_uw 0.35, lr 0.0375, flags 0.
 *
 *   ns_steps, ns_a/b/c  Newton-Schulz iteration count and polynomial
 *                       X <- a X + (b A + c A^2) X, A = X X^T (1..64 steps).
 *   ns_eps              added to the Frobenius norm before normalising.
 *   pp_iterations       Aurora passes (0 = plain NS, no preconditioner; 1 =
 *                       row-normalise then polar; 0..8).
 *   pp_beta, pp_eps     damping exponent of the D update; clamp of row norms
 *                       (pp_eps) and squared row norms (pp_eps^2).
 *   mu, nesterov        momentum coefficient in [0, 1]; Nesterov blend flag.
 *   power_steps         power iterations for the operator-norm estimate (1..64).
 *   contra              Contra-Muon coefficient; the step subtracts contra/2
 *                       times the unit-operator-norm direction (0 = off).
 *   target_uw           u/w-floor target ratio (0 = off).
 *   lr                  learning rate of the parameter add.
 *   flags               bitwise OR of MUON_FLAG_* below (0 = the Aurora
 *                       page's step); unknown bits are rejected
 *                       (MUON_ERR_INVALID_ARG).
 */
typedef struct {
  int32_t  ns_steps;
  float    ns_a, ns_b, ns_c, ns_eps;
  int32_t  pp_iterations;
  float    pp_beta, pp_eps;
  float    mu;
  int32_t  nesterov;
  int32_t  power_steps;
  float    contra;
  float    target_uw;
  float    lr;
  uint32_t flags;
} muon_config;

/*
 * MUON_FLAG_SGD_MOMENTUM — the momentum form of the classic Muon recipe,
 * [Track-1 page] §"训练管线与系统实现" ("SGD momentum" with Nesterov), read as
 * the heavy-ball buffer with no dampening: M <- mu M + G, X = G + mu M
 * (X = M without Nesterov). Without the flag the step keeps the Aurora page's
 * moving average, M <- M + (1 - mu)(G - M), X = G + mu (M - G). The two give
 * the same direction at constant mu from a zero buffer (the buffers differ
 * by 1/(1 - mu)) and different ones under a momentum warm-up.
 * muon_config_classic sets it.
 *
 * MUON_FLAG_WIDE_ROWS — [Aurora page] §"复现与扩展建议" names a later result
 * that applies the row-balanced polar to a wide matrix (the MLP output
 * projection) and gives no formula. With this flag a wide matrix (rows <
 * cols) is equilibrated on its own rows, the short side: D = 1/max(row
 * norm, pp_eps), then the same damped update with target 1 (the squared
 * row norm of a polar factor with orthonormal rows). Tall and square
 * matrices are unaffected. Since such a polar factor's rows are already
 * orthonormal, later passes move D only where Newton-Schulz has not
 * converged; pp_iterations 1 is row-normalise-then-polar on the rows.
 *
 * MUON_FLAG_FP8_GRAM — lower-precision Newton-Schulz, a research option (not
 * from the pages, which run the optimizer's products in their training
 * precision; the 3.8B page uses FP8 only for the model's GEMMs, in its
 * post-mortem). For bf16 matrices that run Newton-Schulz in blocks
 * (rectangular, short side >= 512), the first Gram of each pass, A = X0 X0^T
 * with K = the long side, reads an fp8 (OCP e4m3) copy of X0 written by the
 * pass prologue with a per-matrix power-of-two scale q (q |X0| <= 448,
 * bounded by the largest equilibrated line or row norm), runs on the fp8
 * matrix cores and divides by q^2 in its epilogue. The sums over the long
 * side average the operands' rounding: measured error stays at the bf16
 * path's level (about 5e-3 relative Frobenius). Later Grams, the short-side
 * products and X' = Q X stay bf16 (fp8 there costs 1e-2 to 5e-2).
 *
 * MUON_FLAG_CHECK_FINITE — an input check for callers that want a NaN or
 * Inf to stop the step instead of spreading through it (the pages define
 * no such check; without the flag a non-finite input gives non-finite
 * results for its matrix only). Before anything is written, one read-only
 * pass over every matrix's grad (the polar input), momentum and weight
 * looks for NaN or Inf; the call then waits for that pass on its stream
 * (the one case where a compute call synchronises). If any element is not
 * finite the call returns MUON_ERR_NONFINITE, names the first such matrix
 * in muon_last_error(), and leaves every caller buffer as it was;
 * otherwise the step runs as without the flag, with bitwise-equal results.
 * Costs one read of the inputs and the synchronisation.
 */
#define MUON_FLAG_SGD_MOMENTUM 0x1u
#define MUON_FLAG_WIDE_ROWS    0x2u
#define MUON_FLAG_FP8_GRAM     0x4u
#define MUON_FLAG_CHECK_FINITE 0x8u
#define MUON_FLAG_ALL          0xFu

/* Per-kernel-class timing gathered when profiling is on (see muon_profile_*).
   Each *_ms is the wall time the class's event pairs cover: their summed
   durations less the time they overlap (launches on the handle's second
   stream run beside those on the call's stream). */
typedef struct {
  int64_t gemm_launches;      /* Newton-Schulz matrix-core launches */
  double  gemm_ms;            /* event time of those launches */
  double  gemm_counted_flop;  /* 4 s^2 L + 2 s^3 per iteration per matrix (s <= L) */
  double  gemm_executed_flop; /* flops the tiles actually issue (symmetric results' lower tiles
                                 skipped, and on their diagonal tiles the 32x32 blocks wholly
                                 below the diagonal) */
  double  gemm_algorithmic_flop; /* flops the products need: the upper half of each symmetric
                                    result, no padding (3 s^2 L + (4 r - 3) s^3 per block of r
                                    iterations) */
  int64_t stream_launches;    /* bandwidth-bound launches of the step itself: momentum and
                                 norms, the weight norm, power iteration, tail (and the latency
                                 kernels between) */
  double  stream_ms;
  double  stream_bytes;       /* algorithmic HBM bytes of those launches */
  int64_t aux_launches;       /* Aurora vector kernels feeding the products: the pass prologue
                                 (X0 = scale D o T in one or both orientations) and the D update */
  double  aux_ms;
  double  aux_bytes;          /* HBM bytes of those launches (source read, iterate pair written;
                                 D update: one read of U) */
} muon_profile;

typedef struct muon_handle muon_handle;

/* Fill *cfg with the page's locked values (listed above). cfg must not be NULL. */
void muon_config_default(muon_config* cfg);

/*
 * Fill *cfg with the classic Muon recipe of the Track-1 record page
 * (§"训练管线与系统实现"): SGD momentum 0.95 with Nesterov
 * (flags = MUON_FLAG_SGD_MOMENTUM), Newton-Schulz with
 * (ns_a, ns_b, ns_c) = (3.4445, -4.7750, 2.0315) for ns_steps 5, no Aurora
 * preconditioner (pp_iterations 0), no Contra term (contra 0), no u/w-floor
 * (target_uw 0), the sqrt(max(1, rows/cols)) scale, lr 0.04. The remaining
 * fields keep muon_config_default's values. cfg must not be NULL.
 * That recipe's fixed point is deliberately not 1, so its update is not an
 * exact orthogonalisation.
 */
void muon_config_classic(muon_config* cfg);

/*
 * Momentum warm-up of the same page: frac = min(step / warmup_steps, 1),
 * mu = (1 - frac) * mu_start + frac * mu_end (the page uses 0.85 -> 0.95
 * over 500 steps). A host-side scalar for muon_config.mu; step < 0 counts as
 * 0, warmup_steps <= 0 returns mu_end. Computed in double, returned as float.
 */
float muon_momentum_warmup(int64_t step, float mu_start, float mu_end, int64_t warmup_steps);

/* Static text for a status code. Never NULL. */
const char* muon_status_string(muon_status s);

/* Library version string ("major.minor.patch"). */
const char* muon_version(void);

/*
 * Create a handle bound to the current HIP device and to `stream`
 * (a hipStream_t; NULL = the default stream). The stream is borrowed, not
 * owned. The handle owns its device workspace and plan cache; both grow on
 * demand and are freed by muon_destroy. It also owns a second stream of
 * default priority, made by the first call that uses it: on sets whose
 * product launches are small, a call runs part of each Newton-Schulz pass
 * there (the one-iteration matrices beside the blocked ones, or half of a
 * set with only one kind), and `stream` waits for it before the pass ends,
 * so every call still completes in order on `stream`. Returns
 * MUON_ERR_NO_DEVICE when no gfx950 device is current.
 *
 * Tuning (environment). The layout and tile edge give bitwise the default's
 * results; a forced block length changes the rounding only:
 *   MUON_NS_VARIANT=1      read here: Newton-Schulz products on 256x256 tiles
 *                          with 4 waves of 128x128 instead of 8 of 64x128.
 *   MUON_NS_TILE=128|256   read when a plan is built (first call with a new
 *                          set of shapes): force the product tile edge;
 *                          otherwise launches with fewer than 768 256-tiles
 *                          use 128-tiles.
 *   MUON_NS_BLOCK=1..8     read when a plan is built: Newton-Schulz
 *                          iterations per block for every rectangular matrix
 *                          (default 4 where the coefficients allow, below 512
 *                          on the short side 1).
 *   MUON_NS_SIDE=0|1       read here: 0 keeps every launch on `stream`, 1
 *                          uses the second stream in every pass that has
 *                          both one-iteration and blocked matrices, however
 *                          large (bitwise the same results either way).
 *   MUON_FUSED_TAIL=0      read when a plan is built: bf16 matrices of
 *                          muon_update take the tail's norms in a reduction
 *                          pass over U, X and W (and the operator-norm
 *                          estimate in its own X v launch) instead of in the
 *                          final Newton-Schulz product's epilogue and a
 *                          read-only pass over W (the same sums in another
 *                          order).
 *   MUON_TALL_X0=0         read when a plan is built: bf16 matrices of
 *                          muon_update with both sides multiples of 256 get
 *                          both orientations of the pass's first iterate
 *                          from the prologue, instead of the first X' = Q X
 *                          (tall matrices) or the first Gram (wide or square
 *                          ones without the preconditioner) reading the
 *                          blended update and scaling its output (the
 *                          same products, rounded once less).
 * Tracing: MUON_ROCTX=1, read here, wraps each phase of a call (momentum,
 * power iteration, each Newton-Schulz pass, the Aurora D update, the tail)
 * in a ROCTx range for rocprofv3 --marker-trace; the ROCTx library is loaded
 * at run time and the ranges are skipped when it is absent.
 */
muon_status muon_create(muon_handle** handle, void* stream);

/* Free the handle and its workspace (waits for the stream first). NULL is a no-op. */
muon_status muon_destroy(muon_handle* handle);

/* Rebind the handle to another stream of the same device. */
muon_status muon_set_stream(muon_handle* handle, void* stream);

/* Message of the handle's last error ("" if none). Valid until the next call. */
const char* muon_last_error(const muon_handle* handle);

/*
 * Host-only validation of a muon_update batch with the same rules as
 * muon_update; enqueues nothing and needs no device. weight and update_out
 * may be NULL. msg (may be NULL) receives a message of up to msg_len bytes.
 */
muon_status muon_check_update_args(int n, const muon_matrix* grad,
                                   const muon_matrix* momentum,
                                   const muon_matrix* weight,
                                   const muon_matrix* update_out,
                                   const muon_config* cfg,
                                   char* msg, int msg_len);

/* Host-only validation of an ns_polar / aurora_orthogonalize batch. */
muon_status muon_check_polar_args(int n, const muon_matrix* in,
                                  const muon_matrix* out,
                                  const muon_config* cfg,
                                  char* msg, int msg_len);

/*
 * Host-only consistency check of the launch plan a compute call would build
 * for a batch (for tests and for debugging the planner; needs no device).
 * kind: 0 muon_update, 1 ns_polar, 2 aurora_orthogonalize; only rows, cols
 * and dtype of `shapes` are read; cfg may be NULL (defaults). It checks that
 * every workspace region lies inside the workspace and overlaps no other;
 * that every tile of every Newton-Schulz product list lies inside its
 * matrix's padded tile grid and sits in the list of that matrix's pass,
 * block length class and element type; that every tile a product needs is
 * listed exactly once (the upper triangle of the symmetric products, the
 * whole grid of X' = Q X); and that the streaming launch lists have
 * consistent block offsets (the momentum pass's n_rt x n_seg tiles per
 * matrix). Returns MUON_OK, or MUON_ERR_INVALID_ARG with the first violation
 * in msg (NUL-terminated, at most msg_len bytes); shapes past the library's
 * limits give MUON_ERR_SHAPE_MISMATCH.
 */
muon_status muon_debug_check_plan(int kind, int n, const muon_matrix* shapes,
                                  const muon_config* cfg, char* msg, int msg_len);

/*
 * Grow the workspace so that batches with these shapes and types run without
 * any further device allocation (so a timed or captured region allocates
 * nothing). Only rows, cols and dtype of `shapes` are read.
 */
muon_status muon_reserve(muon_handle* handle, int n, const muon_matrix* shapes);

/*
 * ns_polar — out_i = NS(in_i): the Newton-Schulz approximation of the polar
 * factor, [Aurora page] §"源码实现" (the shared NS primitive): divide by the
 * Frobenius norm + ns_eps, then ns_steps times X <- a X + (b A + c A^2) X with
 * A = X X^T formed on the short side.
 *   in[i]   input, any shape, F32 or BF16; read only.
 *   out[i]  output, same shape as in[i], F32 or BF16 (rounded to nearest
 *           even). An output may share memory with any input, in place or
 *           not: every input is read before the first output is written.
 *           Outputs must not share an element with one another
 *           (MUON_ERR_INVALID_ARG); column slices of one buffer do not.
 *   cfg     ns_* fields are used; NULL = defaults.
 */
muon_status ns_polar(muon_handle* handle, int n, const muon_matrix* in,
                     const muon_matrix* out, const muon_config* cfg);

/*
 * aurora_orthogonalize — leverage-equilibrated polar, [Aurora page]
 * §"Aurora 是什么", §"Aurora 的迭代伪代码" and §"源码实现": square inputs get
 * plain NS; otherwise, in the tall orientation (m > n), D = 1/max(row norm,
 * pp_eps) and pp_iterations passes of U = NS(D * G), multiplying D by
 * (n/m / max(row_sq, pp_eps^2))^pp_beta between passes. Wide inputs are
 * handled as their transpose without materialising it.
 *   in, out, cfg as for ns_polar (pp_* and ns_* fields used).
 */
muon_status aurora_orthogonalize(muon_handle* handle, int n,
                                 const muon_matrix* in, const muon_matrix* out,
                                 const muon_config* cfg);

/*
 * muon_update — one Aurora + Contra-Muon + u/w-floor optimizer step,
 * [Aurora page] §"组合优化栈" (muon_update, the Contra-Muon and u/w-floor
 * parts) and §"完整的超参配置表":
 *   M <- M + (1 - mu)(G - M); X = G + mu (M - G) (X = M without Nesterov);
 *   N = X / max(sigma, 1e-7), sigma from power_steps power iterations on
 *   X^T X started from ones/sqrt(cols) (restart from the first largest-norm
 *   column if that start is annihilated);
 *   U = aurora_orthogonalize(X); V = U - (contra/2) N, rescaled to ||U||_F
 *   (clamp 1e-10); V *= sqrt(max(1, rows/cols));
 *   if ||V||/||W|| < target_uw (both clamped at 1e-8): V *= target_uw ||W||/||V||;
 *   W <- W - lr V.
 *   grad[i]       G, F32 or BF16; read only (unlike the page's in-place
 *                 lerp, the blended update goes to workspace).
 *   momentum[i]   M, F32, same shape; updated in place.
 *   weight        NULL, or weight[i] = W (F32 or BF16, same shape) updated in
 *                 place (bf16 rounded to nearest even); weight[i].ptr NULL
 *                 means no weight (and no floor) for matrix i.
 *   update_out    NULL, or update_out[i] receives V after the floor and
 *                 before lr (F32 or BF16; ptr NULL = not wanted).
 *   cfg           NULL = defaults.
 * Every buffer the call writes (momentum, weight, update_out) must not share
 * an element with any other buffer of the call, of the same matrix or
 * another: MUON_ERR_INVALID_ARG names the first such pair. Grads may share
 * memory with one another (they are only read), and column slices of one
 * buffer (same ld, disjoint columns) share no element.
 */
muon_status muon_update(muon_handle* handle, int n, const muon_matrix* grad,
                        const muon_matrix* momentum, const muon_matrix* weight,
                        const muon_matrix* update_out, const muon_config* cfg);

/*
 * muon_update_static — muon_update for callers that cannot allocate device
 * memory during the call: code under HIP graph capture, tight serving or
 * training loops, harnesses that forbid allocation. Same arguments, rules,
 * validation, kernels and results as muon_update (bitwise), but the call
 * allocates nothing: its workspace and launch tables live in a file-scope
 * device array of 64 MiB per device (held until the process ends; its
 * address is taken once per device by muon_create, and a pinned 1 MiB table
 * stage is allocated there too), and no profiling events are recorded.
 *   Limit: the batch's workspace plus its launch tables must fit the 64 MiB
 *   (for example one 1024 x 3072 bf16 matrix, or a few 768 x 768 ones, with
 *   tables within 1 MiB); larger batches return MUON_ERR_TOO_LARGE with a
 *   message giving the bytes needed, before anything is enqueued.
 *   Sharing: every static call on a device uses that device's one array and
 *   leaves its contents there (nothing in it needs clearing: every call
 *   writes each part before reading it). Static calls that can overlap on
 *   one device (other handles, other streams) race: order them, e.g. on one
 *   stream.
 */
muon_status muon_update_static(muon_handle* handle, int n, const muon_matrix* grad,
                               const muon_matrix* momentum, const muon_matrix* weight,
                               const muon_matrix* update_out, const muon_config* cfg);

/*
 * ---------------------------------------------------------------------------
 * The rest of a training step: the head's loss with its gradient, the global
 * gradient norm with clipping, and AdamW for the parameters that Muon does
 * not take (embeddings, head, one-dimensional ones).
 *
 * The conventions above hold, with these differences. The tensors of the list
 * calls are any rows x cols with unit column stride, up to 2^42 elements (a
 * vector is one row, whose ld is not looked at); none of the Newton-Schulz
 * limits applies. Outputs share no element with any other buffer of the call
 * unless said below (MUON_ERR_INVALID_ARG). norm, coef, loss, grad_out and
 * grad_scale are device pointers to fp32 values. Lists travel in the kernel
 * arguments, so these calls upload nothing; they can be captured in a graph
 * once a first call of the same sizes has grown the handle's buffers. A buffer
 * that a later call outgrows is freed (that call waits for the stream), unless a
 * captured call used it: then it is kept until muon_destroy, so that the graph
 * stays valid. Like any call a graph must not run beside others of its handle.
 */

/*
 * muon_grad_norm - norm = sqrt(sum over all elements of all tensors of g^2),
 * the squares summed in 64 bits (no overflow for any fp32 gradient); with
 * coef not NULL also coef = min(1, max_norm / (norm + 1e-6)), NaN where the
 * norm is. An empty list has norm 0. max_norm > 0 is read only with coef.
 */
muon_status muon_grad_norm(muon_handle* handle, int n, const muon_matrix* grad, float max_norm,
                           float* norm, float* coef);

/*
 * muon_clip_grad_norm - muon_grad_norm, then out_i = coef grad_i (out NULL:
 * in place, and nothing is written when coef is 1). out_i may be grad_i
 * itself; its type may differ from grad_i's. coef must not be NULL.
 */
muon_status muon_clip_grad_norm(muon_handle* handle, int n, const muon_matrix* grad, const muon_matrix* out,
                                float max_norm, float* norm, float* coef);

/* out_i = coef in_i with coef on the device (out NULL: in place, nothing written when it is 1). */
muon_status muon_scale(muon_handle* handle, int n, const muon_matrix* in, const muon_matrix* out,
                       const float* coef);

/*
 * adamw_update - AdamW with decoupled weight decay, in place, for each tensor:
 *   g' = grad_scale g (grad_scale: device scalar, for example muon_grad_norm's
 *   coef; NULL = 1), m = beta1 m + (1 - beta1) g', v = beta2 v +
 *   (1 - beta2) g'^2, w = w (1 - lr weight_decay) - lr (m / (1 - beta1^step))
 *   / (sqrt(v / (1 - beta2^step)) + eps).
 *   grad, weight F32 or BF16 (each its own), exp_avg, exp_avg_sq F32; copy
 *   (array may be NULL, entries may be empty) receives the same fp32 result as
 *   the weight, rounded to the copy's own type, for a model that computes on
 *   16-bit copies of 32-bit weights; an F32 copy of a BF16 weight is therefore
 *   the value that the weight was rounded from, not the weight. All arithmetic
 *   is fp32; a BF16 weight is rounded to nearest even once a step. step counts
 *   from 1. Every tensor is read and written once.
 *   lr and step are constants of the launch: a graph that captured the call
 *   repeats them on every replay. step_at and lr_at (device pointers, each or
 *   both, NULL = the value here) are read when the kernel runs instead, so a
 *   graph can count its steps (a step below 1 gives weights that are not finite).
 * muon_adamw_config_default (start from it: fields may be added at the end): lr 0.01,
 * betas (0.8, 0.95), eps 1e-10, weight_decay 0 (the [Aurora page]'s AdamW beside
 * Muon), step 1, no device values.
 */
typedef struct {
  float lr, beta1, beta2, eps, weight_decay;
  int64_t step;
  const int64_t* step_at;
  const float* lr_at;
} muon_adamw_config;
void muon_adamw_config_default(muon_adamw_config* cfg);
muon_status adamw_update(muon_handle* handle, int n, const muon_matrix* grad, const muon_matrix* exp_avg,
                         const muon_matrix* exp_avg_sq, const muon_matrix* weight, const muon_matrix* copy,
                         const muon_adamw_config* cfg, const float* grad_scale);

/*
 * linear_cross_entropy(_grad) - softmax cross entropy of a language-model
 * head: z = hidden weight^T (N x V, fp32 accumulation; the loss alone
 * stores none of them), with softcap c > 0: z <- c tanh(z / c); loss_i = log sum_v
 * exp z_iv - z_i,target. The gradient is that of sum_i g_i loss_i, g_i = grad_out[i]
 * (reduction none), grad_out[0] (sum) or grad_out[0] / valid tokens (mean);
 * grad_out NULL = 1.
 *   hidden   N x D; weight V x D, same type, F32 or BF16 (D <= 65536,
 *            V <= 2^22, N <= 2^24; N may be 0)
 *   targets  N integers of target_bytes 4 or 8 each. Tokens whose target is
 *            ignore_index are left out: loss 0, gradient 0, and whatever
 *            their hidden rows hold (NaN too) is never read. Any other target
 *            outside [0, V) gives that token a NaN loss and no gradient.
 *   loss     N values (reduction none) or one; mean is over the valid tokens,
 *            0 if there is none
 *   dhidden, dweight  gradients, of the types of hidden and weight; one of
 *            them may be NULL (its product is left out)
 * BF16 inputs are multiplied on the bf16 matrix cores: a logit's gradient is
 * rounded to 10 bits of mantissa (its kept exponential) and then to bf16, but
 * the target's, most of a token's, counts with 16 bits; grad_out and 1 / valid
 * tokens multiply the fp32 sums. F32 inputs are fp32 throughout; statistics and
 * sums are fp32. The tokens are taken in pieces; with gradients a piece's V
 * exponentials a token (2 bytes each, F32 4) are kept beside its rows, as much as
 * the logits of these tokens would take.
 * Memory of the handle (each handle has its own; the Python binding has one a
 * thread): the pieces, up to 1 GiB, or 256 tokens' if these take more; partial
 * sums of each gradient, up to 256 MB; 12 bytes a token of the call; when a call takes more than one piece, an
 * fp32 V x D sum; a padded copy of a weight whose rows are not whole 16-byte
 * pieces that start on 16 bytes. A buffer that grows takes up to half as much
 * again, 256 MiB at most.
 */
typedef enum { MUON_REDUCE_NONE = 0, MUON_REDUCE_SUM = 1, MUON_REDUCE_MEAN = 2 } muon_reduction;
typedef struct {
  int32_t reduction;     /* muon_reduction */
  float   softcap;       /* 0 = off */
  int64_t ignore_index;
} muon_loss_config;
/* mean, no softcap, ignore_index -100 */
void muon_loss_config_default(muon_loss_config* cfg);
muon_status linear_cross_entropy(muon_handle* handle, const muon_matrix* hidden, const muon_matrix* weight,
                                 const void* targets, int target_bytes, const muon_loss_config* cfg, float* loss);
muon_status linear_cross_entropy_grad(muon_handle* handle, const muon_matrix* hidden, const muon_matrix* weight,
                                      const void* targets, int target_bytes, const muon_loss_config* cfg,
                                      const float* grad_out, float* loss, const muon_matrix* dhidden,
                                      const muon_matrix* dweight);

/*
 * linear_logprobs(_grad) - log probabilities of given tokens under a language-model
 * head, with the distribution's entropy and its likeliest tokens: z = hidden
 * weight^T as above (soft cap included), lse_i = log sum_v exp z_iv,
 *   logprobs_i = z_i,target - lse_i
 *   entropy_i  = - sum_v p_iv log p_iv, p_iv = exp(z_iv - lse_i)
 *   top_tokens_i, top_logprobs_i: the `top` largest logits in falling order,
 *   equal ones by rising token
 * No logits are stored. The gradient is that of sum_i grad_logprobs[i]
 * logprobs_i + grad_entropy[i] entropy_i; the alternatives have none.
 *   hidden, weight, targets   as for linear_cross_entropy. Tokens whose target
 *            is ignore_index have log probability, entropy and top_logprobs 0,
 *            top_tokens -1 and gradient 0, and their hidden rows are never read.
 *            Any other target outside [0, V) gives that token's log probability
 *            as NaN and no gradient; its entropy and alternatives do not depend on it.
 *   cfg      NULL = defaults; top in [0, MUON_TOP_MOST], at most V
 *   logprobs N values; entropy N values or NULL
 *   stats    N x 4 values or NULL, on 16 bytes: what linear_logprobs_grad
 *            needs of the call (each token's largest logit, log sum exp over it,
 *            entropy and log probability)
 *   top_logprobs, top_tokens  N x top each, row by row; not looked at with top 0
 *   grad_logprobs, grad_entropy  N values each; one may be NULL (zero)
 *   dhidden, dweight  as for linear_cross_entropy_grad
 * The alternatives are ranked by the raw logits (a soft cap keeps their order): the
 * top + 8 largest of the fp32 sums are summed again in 64 bits, so neighbours
 * nearer than an fp32 sum's error are in order too (a word is out only where its
 * fp32 sum is behind those of top + 8 others, in either precision). The target's
 * logit, too, is summed in 64 bits, and where there are alternatives the largest of
 * theirs counts so in the sums: where one is the largest by far its error would be all
 * of its log probability's, and the others' sum is kept apart from it. Where fewer
 * than `top` raw logits are above minus infinity the rest are token -1 with log
 * probability minus infinity; a NaN logit makes a token's values NaN and its
 * alternatives -1, and so does one of infinity that no cap bounds (the target's
 * leaves the alternatives' tokens).
 * The gradient takes the logits again, as its own product, and with the same
 * workspace as linear_cross_entropy_grad; a logit's gradient is rounded once, as
 * the products' operand, and the target's counts with 16 bits of a BF16's 8.
 */
#define MUON_TOP_MOST 32
typedef struct {
  int32_t top;           /* alternatives a token */
  float   softcap;       /* 0 = off */
  int64_t ignore_index;
} muon_logprob_config;
/* no alternatives, no softcap, ignore_index -100 */
void muon_logprob_config_default(muon_logprob_config* cfg);
muon_status linear_logprobs(muon_handle* handle, const muon_matrix* hidden, const muon_matrix* weight,
                            const void* targets, int target_bytes, const muon_logprob_config* cfg, float* logprobs,
                            float* entropy, float* stats, float* top_logprobs, int64_t* top_tokens);
muon_status linear_logprobs_grad(muon_handle* handle, const muon_matrix* hidden, const muon_matrix* weight,
                                 const void* targets, int target_bytes, const muon_logprob_config* cfg,
                                 const float* stats, const float* grad_logprobs, const float* grad_entropy,
                                 const muon_matrix* dhidden, const muon_matrix* dweight);

/*
 * residual_norm(_grad) - the end of one block and the start of the next, for
 * each row (token) of the residual stream x and of the block's result y:
 *   n      = y / sqrt(mean(y^2) + eps) * post_gain      (post_norm 0: n = y)
 *   out    = scale * x + gate * n
 *   hidden = out / sqrt(mean(out^2) + eps) * pre_gain   (pre_norm 0: none)
 * x alone (y NULL): out = scale * x, which need not be stored (out NULL) - the
 * norm before the first block. Arithmetic is fp32; out and hidden are each
 * rounded once, from the same fp32 sums. Squares are fp32, too: rows of values
 * past 2^56 can overflow them.
 *   x, out     N x D, D <= 16384, F32 or BF16, both of one type
 *   y, hidden  N x D, both of one type: x's, or BF16 beside an F32 x
 *   post_gain, pre_gain  D values (NULL: 1)
 *   gate       one value, D values, or N x D of y's type (NULL: 1)
 *   scale      one value or D values (NULL: 1)
 * Parameters are F32 or BF16, each its own; vectors are one row. eps > 0.
 * residual_norm_grad takes the gradients of out (dout) and hidden (dhidden; each
 * may be NULL: zero, not both), of the types of out and hidden, and gives those of
 * the inputs (grads; a NULL one is left out), each of its input's type and
 * shape. It makes out again from x and y; nothing else of the forward call is
 * needed. Outputs share no element with any other buffer of the call.
 * Workspace: fp32 sums of up to 3 D + 4 values for each of up to 1024 blocks.
 */
typedef struct {
  const muon_matrix *post_gain, *pre_gain, *gate, *scale;
  int32_t post_norm, pre_norm;
  float eps;
} muon_norm_params;
/* no parameters, both norms, eps 1e-6 */
void muon_norm_params_default(muon_norm_params* p);
typedef struct {
  const muon_matrix *x, *y, *post_gain, *gate, *scale, *pre_gain;
} muon_norm_grads;
muon_status residual_norm(muon_handle* handle, const muon_matrix* x, const muon_matrix* y,
                          const muon_norm_params* params, const muon_matrix* out, const muon_matrix* hidden);
muon_status residual_norm_grad(muon_handle* handle, const muon_matrix* x, const muon_matrix* y,
                               const muon_norm_params* params, const muon_matrix* dout, const muon_matrix* dhidden,
                               const muon_norm_grads* grads);

/*
 * Host-only validation with the rules of the calls above; enqueue nothing, need no device.
 * muon_check_norm_args has muon_grad_norm's rules with out NULL (the list is only read: a
 * tensor may be in it twice) and muon_clip_grad_norm's with out, coef apart, which that call
 * also needs; for a clip in place, which writes the list, give the list itself as out.
 */
muon_status muon_check_norm_args(int n, const muon_matrix* grad, const muon_matrix* out, float max_norm,
                                 const float* norm, const float* coef, char* msg, int msg_len);
muon_status muon_check_adamw_args(int n, const muon_matrix* grad, const muon_matrix* exp_avg,
                                  const muon_matrix* exp_avg_sq, const muon_matrix* weight, const muon_matrix* copy,
                                  const muon_adamw_config* cfg, const float* grad_scale, char* msg, int msg_len);
muon_status muon_check_loss_args(const muon_matrix* hidden, const muon_matrix* weight, const void* targets,
                                 int target_bytes, const muon_loss_config* cfg, const float* grad_out,
                                 const float* loss, const muon_matrix* dhidden, const muon_matrix* dweight,
                                 char* msg, int msg_len);
muon_status muon_check_logprob_args(const muon_matrix* hidden, const muon_matrix* weight, const void* targets,
                                    int target_bytes, const muon_logprob_config* cfg, const float* logprobs,
                                    const float* entropy, const float* stats, const float* top_logprobs,
                                    const int64_t* top_tokens, char* msg, int msg_len);
muon_status muon_check_logprob_grad_args(const muon_matrix* hidden, const muon_matrix* weight, const void* targets,
                                         int target_bytes, const muon_logprob_config* cfg, const float* stats,
                                         const float* grad_logprobs, const float* grad_entropy,
                                         const muon_matrix* dhidden, const muon_matrix* dweight, char* msg,
                                         int msg_len);
muon_status muon_check_residual_norm_args(const muon_matrix* x, const muon_matrix* y, const muon_norm_params* params,
                                          const muon_matrix* out, const muon_matrix* hidden, char* msg, int msg_len);
muon_status muon_check_residual_norm_grad_args(const muon_matrix* x, const muon_matrix* y,
                                               const muon_norm_params* params, const muon_matrix* dout,
                                               const muon_matrix* dhidden, const muon_norm_grads* grads, char* msg,
                                               int msg_len);

/*
 * Profiling of the library's own launches (for roofline reporting): when
 * enabled, each kernel launch is bracketed by HIP events on the handle's
 * stream and its time, its algorithmic flops or bytes are added to totals.
 * muon_profile_read synchronises those events and returns the totals since
 * the last reset.
 */
muon_status muon_profile_enable(muon_handle* handle, int enable);
muon_status muon_profile_reset(muon_handle* handle);
muon_status muon_profile_read(muon_handle* handle, muon_profile* out);

#ifdef __cplusplus
}
#endif

#endif /* LIBMUON_H */
