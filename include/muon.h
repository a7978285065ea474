/*
 * muon.h -- C ABI of the B200 (sm_100a) Muon / MONA optimizer step.
 *
 * The method (sources):
 *   [MONA]  "MONA - Muon-optimizer met Nesterov-versnelling" (gist.science,
 *           paper 2605.26842), section 2 "Methodologie: MONA", Kernalgoritme
 *           steps 1-4:
 *             D = G - G_prev;  A = beta_a A + (1 - beta_a) D;  Gt = G + alpha A;
 *             M = mu M + Gt;   O = Newton-Schulz(M);
 *             W = W - eta (gamma O + lambda W).
 *           "Ontwerprichtlijnen": the acceleration term is applied before the
 *           orthogonalisation, never after.
 *   [POLAR] quant_prune_distill post 677 (tgviewer.app): the Muon step
 *           substitutes the polar factor polar(X) = U V^T (X = U S V^T) of the
 *           momentum; it is found by Newton-Schulz.  Gram route:
 *           polar(X) = X (X^T X)^{-1/2} with the inverse square root also found
 *           by Newton-Schulz on the small Gram matrix, half of every symmetric
 *           product computed and mirrored, restarts, and a division by
 *           1.02-1.05 so that the eigenvalues stay inside [0, 1].
 *   [LiMuon] "LiMuon: Light and Fast Muon Optimizer for Large Models"
 *           (arxiv.sitesynth.xyz digest 2509.14562v1), section "Метод":
 *           Muon's momentum with the update taken from a randomized SVD
 *           (limuon_step_batched below).
 *
 * Iteration used by every entry point (readings of the pages, which name
 * Newton-Schulz but print no coefficients): on the wide view X (s x l,
 * s = min(rows, cols); a matrix with rows > cols is iterated transposed,
 * polar(X^T) = polar(X)^T) start from X0 = M / ((||M||_F + eps) f) and, for
 * k = 0 .. n_steps-1 with (a, b, c) = coeffs[k]:
 *     A = X X^T;   B = b A + c A A;   X = a X + B X
 * At every step k > 0 listed in `restarts` X is divided by f once more before
 * the step.  The Gram route evaluates the same polynomial through
 * R = X X^T:  h = a I + b R + c R^2,  Q <- h Q,  R <- h R h, and at a restart
 * k > 0: Xb <- Q Xb / f, R <- Xb Xb^T, Q <- I;  finally X = Q Xb.
 *
 * Conventions common to all entry points:
 *   - Every pointer named d_* or documented as "device" is CUDA device memory
 *     of the current device, owned by the caller.  Host arrays (schedule
 *     coefficients, restarts, parameter descriptors) are read during the call
 *     only and may be freed as soon as it returns.
 *   - The library allocates no memory.  Scratch space is the caller-provided
 *     `workspace` (device, >= the size returned by the matching *_size query,
 *     256-byte aligned).  Its contents need no initialisation and are
 *     clobbered.
 *   - Matrices are dense, row-major and contiguous (row stride = cols).
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL = legacy default
 *     stream) and the call returns without synchronising.  Argument errors
 *     are returned before anything is enqueued.  Faults seen on the device
 *     (non-finite norm, a wait that ran out) are OR-ed into *d_status
 *     (MUON_FLAG_* bits) when d_status is not NULL; the caller reads it after
 *     synchronising.  d_status is never cleared by the library.
 *   - Calls that share a workspace must be ordered on the GPU (same stream,
 *     or events); concurrent calls on one workspace race.
 */
#ifndef MUON_B200_H
#define MUON_B200_H

#include <stddef.h>

#if defined(__GNUC__)
#define MUON_API __attribute__((visibility("default")))
#else
#define MUON_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same handle type as cudaStream_t / CUstream. */
typedef struct CUstream_st* muon_stream_t;

typedef enum {
    MUON_OK = 0,
    MUON_ERR_INVALID_ARG = 1,   /* NULL pointer, bad size, bad enum, bad schedule */
    MUON_ERR_UNSUPPORTED = 2,   /* valid request the library cannot run (no sm_100 device, shape limits) */
    MUON_ERR_WORKSPACE = 3,     /* workspace NULL, misaligned or smaller than the size query */
    MUON_ERR_NONFINITE = 4,     /* host-side name for MUON_FLAG_NONFINITE */
    MUON_ERR_CUDA = 5,          /* a CUDA runtime/driver call failed (see cudaGetLastError) */
    MUON_ERR_TIMEOUT = 6        /* host-side name for MUON_FLAG_TIMEOUT */
} muon_status;

/* Bits OR-ed into *d_status by the device. */
#define MUON_FLAG_NONFINITE 1   /* a matrix had a non-finite Frobenius norm; its W was left unchanged */
#define MUON_FLAG_TIMEOUT   2   /* a kernel's internal wait ran out (about 4 s); its output is invalid */

typedef enum {
    MUON_BF16 = 0,
    MUON_FP16 = 1,
    MUON_FP32 = 2
} muon_dtype;

/* One Newton-Schulz step X <- a X + (b A + c A^2) X. */
typedef struct {
    float a, b, c;
} muon_ns_coeff;

typedef struct {
    int n_steps;                 /* >= 1, <= 64 */
    const muon_ns_coeff* coeffs; /* host array of n_steps entries */
    float eps;                   /* added to ||M||_F before dividing; >= 0 (1e-7 is the usual choice) */
    const int* restarts;         /* host array of step indices (0 allowed, ignored); may be NULL if n_restarts == 0 */
    int n_restarts;              /* >= 0, <= 64 */
    float scale_f;               /* >= 1: extra divisor at the start and at every restart (1.02-1.05 on the Gram route) */
    float gram_aspect;           /* optimizer steps only: a shape group whose long side is at least gram_aspect
                                    times its short side runs the Gram route (with restarts and scale_f);
                                    0 keeps every group on the direct iteration.  >= 0.  ns_polar and
                                    gram_polar ignore it. */
} muon_schedule;

/* Hyper-parameters of [MONA] section 2. */
typedef struct {
    float mu;       /* momentum */
    float eta;      /* learning rate */
    float lambda;   /* decoupled weight decay */
    float gamma;    /* scale of the orthogonalised update */
    float beta_a;   /* EMA factor of the acceleration buffer */
    float alpha;    /* weight of the acceleration term */
} muon_hparams;

/* One matrix parameter and its optimizer state (all device memory). */
typedef struct {
    int rows, cols;    /* >= 1 */
    void* W;           /* rows x cols, w_dtype, updated in place */
    const void* G;     /* rows x cols, w_dtype, this step's gradient (read only) */
    void* G_prev;      /* rows x cols, w_dtype, previous gradient; receives G */
    float* A;          /* rows x cols, fp32 acceleration buffer, updated in place */
    float* M;          /* rows x cols, fp32 momentum, updated in place */
    float gamma;       /* per-matrix gamma; NaN means "use hparams.gamma" */
    float* O_out;      /* optional rows x cols fp32: receives O (the orthogonalised momentum); NULL to skip */
} muon_param;

/*
 * Bytes of workspace muon_step_batched needs for these parameters under this
 * schedule.  params: host array of n descriptors (only rows/cols are read).
 * sched: the schedule the step will use (its gram_aspect decides which shape
 * groups need the Gram route's larger workspace); NULL sizes every group for
 * the direct iteration.
 * Returns MUON_ERR_INVALID_ARG for n < 1, NULL pointers, non-positive sizes or
 * an invalid schedule.
 */
MUON_API muon_status muon_workspace_size(const muon_param* params, int n, muon_dtype ns_dtype,
                                const muon_schedule* sched, size_t* bytes);

/*
 * One optimizer step ([MONA] section 2, steps 1-4) for n matrix parameters.
 *   1. One fused pass over every element: A, M, G_prev updated in place as in
 *      steps 1-4, the Frobenius norm of the new M accumulated per matrix, and
 *      M written in ns_dtype (wide view) to the workspace.
 *   2. The iteration above on every matrix (matrices with the same
 *      (short side, long side) are batched together): the direct iteration,
 *      or the Gram route for the shape groups sched->gram_aspect selects
 *      ([POLAR]: elongated matrices iterate on their small s x s Gram
 *      matrix; in exact arithmetic both routes give the same O).  A matrix
 *      whose short side is below 16 is iterated in fp32 on CUDA cores
 *      whatever ns_dtype says (its 16-bit intermediates would cost accuracy
 *      for no measurable time).
 *   3. W <- W - eta (gamma O + lambda W), fused into the last iteration step;
 *      O never reaches memory unless O_out is given.
 * w_dtype: element type of W, G and G_prev (MUON_BF16, MUON_FP16 or MUON_FP32).
 * ns_dtype: arithmetic of the iteration: MUON_BF16 / MUON_FP16 (tensor cores,
 *   fp32 accumulation, 16-bit operands) or MUON_FP32 (CUDA-core fp32).
 * hp: host struct.  sched: host struct (restarts divide by scale_f as above).
 * A matrix whose norm is not finite keeps its W and sets MUON_FLAG_NONFINITE.
 * W, G, G_prev, A, M of one parameter may not overlap another parameter's.
 */
MUON_API muon_status muon_step_batched(const muon_param* params, int n, muon_dtype w_dtype,
                              muon_dtype ns_dtype, const muon_hparams* hp,
                              const muon_schedule* sched, void* workspace, size_t ws_bytes,
                              int* d_status, muon_stream_t stream);

/*
 * MONA-Lite ([MONA] section "Efficientie en Implementatie"): the auxiliary
 * state kept in bfloat16 and the gradient difference formed in place, without
 * a stored previous gradient.  One buffer per parameter replaces G_prev and A:
 *     B = beta_a A - (1 - beta_a) G      (of the previous step; 0 at the start)
 * so that step 2 reads A_k = B + (1 - beta_a) G_k, and after step 4
 *     B <- beta_a A_k - (1 - beta_a) G_k   (rounded to bfloat16, RNE).
 * Unrounded this is exactly steps 1-4; the state shrinks from G_prev + A to
 * one bfloat16 matrix and the fused pass from 24 to 16 bytes per element
 * (bf16 W/G, fp32 M, 16-bit copy).
 */
typedef struct {
    int rows, cols;    /* >= 1 */
    void* W;           /* rows x cols, w_dtype, updated in place */
    const void* G;     /* rows x cols, w_dtype, this step's gradient (read only) */
    void* B;           /* rows x cols, bfloat16 auxiliary buffer, updated in place (zero initially) */
    float* M;          /* rows x cols, fp32 momentum, updated in place */
    float gamma;       /* per-matrix gamma; NaN means "use hparams.gamma" */
    float* O_out;      /* optional rows x cols fp32: receives O; NULL to skip */
} muon_lite_param;

/* Bytes of workspace muon_lite_step_batched needs (only rows/cols are read;
 * sched as for muon_workspace_size). */
MUON_API muon_status muon_lite_workspace_size(const muon_lite_param* params, int n, muon_dtype ns_dtype,
                                     const muon_schedule* sched, size_t* bytes);

/*
 * One MONA-Lite optimizer step for n matrix parameters: the fused pass above
 * (B and M updated in place, the norm of the new M, its 16-bit wide view),
 * then the same iteration and fused weight update as muon_step_batched, with
 * the same arguments, errors and ownership rules (B takes the place of G_prev
 * and A).
 */
MUON_API muon_status muon_lite_step_batched(const muon_lite_param* params, int n, muon_dtype w_dtype,
                                   muon_dtype ns_dtype, const muon_hparams* hp,
                                   const muon_schedule* sched, void* workspace, size_t ws_bytes,
                                   int* d_status, muon_stream_t stream);

/*
 * AdamW for vector-valued parameters ([MONA] section 2, "Ontwerprichtlijnen":
 * embeddings and biases keep standard AdamW, as in Muon; the page gives no
 * formulas, read as Adam with bias correction and decoupled weight decay):
 *     m <- beta1 m + (1 - beta1) g          v <- beta2 v + (1 - beta2) g^2
 *     W <- W - lr ( (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps) + weight_decay W )
 * evaluated in fp32 per element.  One streaming launch per 128 parameters.
 */
typedef struct {
    long long n;       /* elements (>= 1); any shape, contiguous */
    void* W;           /* n elements, w_dtype, updated in place */
    const void* G;     /* n elements, w_dtype (read only) */
    float* m;          /* n fp32 first moments, updated in place (zero initially) */
    float* v;          /* n fp32 second moments, updated in place (zero initially) */
} muon_vec_param;

typedef struct {
    float lr, beta1, beta2, eps, weight_decay;   /* 0 <= beta < 1, eps >= 0 */
} muon_adamw_hparams;

/*
 * One AdamW step (t = step >= 1, the bias-correction count) on n vector
 * parameters, asynchronous on `stream`.  Argument errors return before any
 * launch (MUON_ERR_INVALID_ARG: NULL pointers, n < 1, step < 1, non-finite or
 * out-of-range hyper-parameters).  An element whose gradient is not finite
 * keeps its W, m and v, and MUON_FLAG_NONFINITE is OR-ed into *d_status
 * (when given).  No workspace.
 */
MUON_API muon_status adamw_step_batched(const muon_vec_param* params, int n, muon_dtype w_dtype,
                               const muon_adamw_hparams* hp, int step, int* d_status,
                               muon_stream_t stream);

/*
 * One optimizer step for a whole model: the n matrix parameters exactly as
 * muon_step_batched, and the nvec vector-valued parameters (embeddings,
 * biases, norm weights: [MONA] section 2, "Ontwerprichtlijnen") with AdamW
 * exactly as adamw_step_batched -- their elements are further work items of
 * the step's fused pre-pass launch, so the model needs no separate AdamW pass.
 * vecs: host array of nvec descriptors (NULL when nvec == 0); every W and G
 * of them in w_dtype, m and v fp32.  adamw, step: as adamw_step_batched
 * (ignored when nvec == 0).  workspace: muon_workspace_size of the matrix
 * parameters under `sched` (the vectors need none).  Errors, ownership and
 * asynchrony as muon_step_batched and adamw_step_batched; a vector element
 * with a non-finite gradient keeps its state and sets MUON_FLAG_NONFINITE.
 */
MUON_API muon_status muon_model_step(const muon_param* params, int n, const muon_vec_param* vecs, int nvec,
                                     muon_dtype w_dtype, muon_dtype ns_dtype, const muon_hparams* hp,
                                     const muon_adamw_hparams* adamw, int step, const muon_schedule* sched,
                                     void* workspace, size_t ws_bytes, int* d_status, muon_stream_t stream);

/*
 * LiMuon ([LiMuon] section "Метод": Muon's momentum, with the update taken
 * from a randomized SVD of the momentum).  The page gives no formulas; read
 * as the basic randomized SVD of Halko, Martinsson and Tropp ("Finding
 * structure with randomness", 2011) in place of the Newton-Schulz iteration:
 *     M <- mu M + G
 *     Y = M Omega,  Q = orth(Y),  B = Q^T M = U~ S V^T,  U = Q U~
 *     O = U_r V_r^T over the r = rank largest singular values
 *     W <- W - eta (gamma O + lambda W)
 * Omega (cols x k, k = rank + oversample <= 64) is the caller's test matrix:
 * the method draws it (Gaussian, fresh or fixed) and passes it in.  Singular
 * values at or below 1e-5 of the largest count as zero and are left out, so a
 * rank-deficient M gives a partial isometry and M = 0 gives O = 0.  Y, Q and
 * the products run in fp32; the k x k Gram, Cholesky and eigen steps in fp64.
 */
typedef struct {
    int rows, cols;       /* >= 1 */
    void* W;              /* rows x cols, w_dtype, updated in place */
    const void* G;        /* rows x cols, w_dtype, this step's gradient (read only) */
    float* M;             /* rows x cols, fp32 momentum, updated in place (zero initially) */
    const float* Omega;   /* cols x k fp32 test matrix, row-major, read only; parameters with the
                             same cols may share one */
    float gamma;          /* per-matrix gamma; NaN means "use hparams.gamma" */
    float* O_out;         /* optional rows x cols fp32: receives O; NULL to skip */
} muon_rsvd_param;

typedef struct {
    float mu, eta, lambda, gamma;
    int rank;             /* r >= 1 */
    int oversample;       /* p >= 0; k = r + p <= 64 (else MUON_ERR_UNSUPPORTED) */
} muon_rsvd_hparams;

/* Bytes of workspace limuon_step_batched needs (only rows/cols are read). */
MUON_API muon_status limuon_workspace_size(const muon_rsvd_param* params, int n, const muon_rsvd_hparams* hp,
                                           size_t* bytes);

/*
 * One LiMuon step for n matrix parameters, asynchronous on `stream`: five
 * launches per 128 parameters (fused momentum pass and sketch; per-matrix
 * QR; projection; per-matrix eigen-decomposition; O fused with the weight
 * update, O never stored unless O_out is given).  workspace: device,
 * 256-byte aligned, at least limuon_workspace_size bytes; no state is kept
 * in it between calls.  Argument errors return before any launch.  A matrix
 * whose new momentum holds a non-finite value keeps its W, and
 * MUON_FLAG_NONFINITE is OR-ed into *d_status (when given).  Parameters may
 * not overlap one another (Omega excepted, which is only read).
 */
MUON_API muon_status limuon_step_batched(const muon_rsvd_param* params, int n, muon_dtype w_dtype,
                                         const muon_rsvd_hparams* hp, void* workspace, size_t ws_bytes,
                                         int* d_status, muon_stream_t stream);

/*
 * Activation checkpoints in 8 bits.  The matrix gradients the steps above read
 * are G = dY^T X of a linear layer's input X and output gradient dY, so X is
 * held from the forward to the backward pass.  A checkpoint holds it in one
 * byte per element: the columns of each row in blocks of 32, per block the
 * smallest e in [-120, 119] with max|x| <= 127 2^e, stored as the byte e + 127,
 * and per element the whole number q = x 2^-e rounded to nearest even (two's
 * complement, -127..127); the checkpoint stands for X^ = q 2^e.
 *   - |X^ - x| <= 2^(e-1), below 1/127 of the block's largest magnitude (half a
 *     step; e only exceeds the smallest exponent that fits at e = -120).
 *   - q 2^e has 7 significant bits, so it is exact in bfloat16 and float.
 *   - A block with a NaN, an infinity or a magnitude above 127 2^119 gets the
 *     byte 255 and codes 0, and stands for 32 NaNs.
 * Any row may hold nothing else than zeros.  rows == 0 is a valid empty
 * checkpoint (an expert without tokens); its pointers may be NULL.  Readers of a
 * checkpoint load q in whole aligned pieces of 16 bytes and e in whole aligned
 * words of 4, so bytes that share one with the checkpoint's are read (not used).
 */
typedef struct {
    int rows, cols;        /* 0 <= rows (tokens) <= 2^30, 1 <= cols <= 2^30 */
    signed char* q;        /* rows x cols codes, row r at q + r * ldq; 16-byte aligned */
    long long ldq;         /* >= cols, a multiple of 16 */
    unsigned char* e;      /* rows x ceil(cols / 32) exponent bytes, row r at e + r * lde */
    long long lde;         /* >= ceil(cols / 32) */
} muon_act8;

/* One matrix to encode (x is read, c written) or to decode (c read, x written). */
typedef struct {
    muon_act8 c;
    void* x;               /* c.rows x c.cols elements, row r at x + r * ldx elements */
    long long ldx;         /* >= cols */
} muon_act8_item;

/*
 * Encode n matrices of x_dtype.  Bytes of q and e outside rows x cols (rows x
 * ceil(cols / 32)) are left as they were.  A block that cannot be held raises
 * MUON_FLAG_NONFINITE in *d_status (when given).  One launch per 64 items;
 * asynchronous on `stream`; argument errors (MUON_ERR_INVALID_ARG) return
 * before any launch, but a batch of 64 whose elements exceed 2^41 (for rows that
 * are not 16-byte aligned 2^31 groups of eight rows) returns
 * MUON_ERR_UNSUPPORTED where it is reached.  No workspace.  What one item writes
 * may not overlap what another reads or writes.
 */
MUON_API muon_status act8_encode_batched(const muon_act8_item* items, int n, muon_dtype x_dtype, int* d_status,
                                         muon_stream_t stream);

/* Decode n checkpoints into x_dtype (exact in bfloat16 and float; rounded to
 * nearest even in fp16).  fp16 values from 65024 on are held as 65536, which fp16
 * takes as its largest value, 65504, so that a finite fp16 tensor stays finite and
 * within half a step; larger values, of checkpoints of other types, become infinite. */
MUON_API muon_status act8_decode_batched(const muon_act8_item* items, int n, muon_dtype x_dtype,
                                         muon_stream_t stream);

/*
 * Weight gradients of linear layers from checkpointed inputs.  Layer i maps
 * rows of `cols` values to rows of `out` values by a weight out x cols; its input
 * was X = X^ diag(gain) + 1 shift^T (gain NULL: 1, shift NULL: 0; a norm's weight
 * and bias, when the checkpoint holds the normalised rows that also serve the
 * norm's own backward pass), so its gradient is
 *     G = beta G + (dY^T X^) diag(gain) + dy_sum shift^T
 * with dy_sum = the column sums of dY (the layer's bias gradient).  beta = 0
 * overwrites G without reading it; rows == 0 leaves beta G (+ the shift term).
 * The product accumulates in fp32: 16-bit dY runs on tensor cores with X^ taken
 * in dY's type (exact in bfloat16; in fp16 rounded, see act8_decode_batched); fp32
 * dY is split into three bfloat16 parts that sum to it (but for bits below 2^-133).  The tensor cores'
 * running sum is truncated (up to 2^-23 of it every 16 tokens), so an fp32 G is summed
 * in segments of 6144 terms (tokens times parts) that are added rounded to nearest; a 16-bit G
 * in segments of 65,536.  Segments, and an fp32 G with beta = 1, are added to in memory, where values
 * below 2^-126 count as zeros.  The sums run in a
 * fixed order: equal inputs give equal bits.  A NaN block makes NaNs of its columns of
 * G (the step then flags the matrix and keeps its W).
 */
typedef struct {
    muon_act8 c;           /* X^: rows (tokens) x cols; e as above */
    const void* dY;        /* c.rows x out elements of dy_dtype, row r at dY + r * lddy elements */
    long long lddy;        /* >= out */
    int out;               /* 1 to 2^30 */
    void* G;               /* out x cols, w_dtype, contiguous */
    const void* gain;      /* cols elements of w_dtype, or NULL */
    const void* shift;     /* cols elements of w_dtype, or NULL; needs dy_sum */
    const float* dy_sum;   /* out fp32 values; NULL if and only if shift is NULL */
    float beta;            /* finite */
} muon_act8_grad_item;

/* Bytes of workspace act8_grad_batched needs for these items (pointers are
 * only inspected for their alignment). */
MUON_API muon_status act8_grad_workspace_size(const muon_act8_grad_item* items, int n, muon_dtype dy_dtype,
                                              muon_dtype w_dtype, size_t* bytes);

/*
 * The gradients of n layers (any mix of shapes; two items may share a
 * checkpoint or a dY; G's that overlap are refused), asynchronous on `stream`:
 * per 48 layers one launch, a second that joins ranges of tokens where layers have few
 * tiles or G's rows are not 16-byte aligned, and one ahead of them where dY has to be copied (fp32, or rows
 * that are not 16-byte aligned).  workspace: device, 256-byte aligned, at least
 * act8_grad_workspace_size bytes (NULL when that is 0); no state is kept in it
 * between calls, and calls that overlap on the GPU each need their own.
 * *d_status (when given) receives MUON_FLAG_TIMEOUT if a bounded wait inside the
 * kernel ran out.  Argument errors return before any launch.
 */
MUON_API muon_status act8_grad_batched(const muon_act8_grad_item* items, int n, muon_dtype dy_dtype,
                                       muon_dtype w_dtype, void* workspace, size_t ws_bytes, int* d_status,
                                       muon_stream_t stream);

/*
 * The seam between two blocks of a network: the norm behind a block, its gate
 * and residual scale, the residual sum, and the norm ahead of the next block, in
 * one pass over the rows; the backward pass works from 8-bit checkpoints of the
 * normalised rows and makes the vector gradients muon_model_step hands to
 * AdamW.  Row t, in fp32:
 *     n_f = (f - mean f) r_f   r_f = 1 / sqrt(mean (f - mean f)^2 + eps)   (MUON_NORM_LAYER)
 *     n_f = f r_f              r_f = 1 / sqrt(mean f^2 + eps)              (MUON_NORM_RMS)
 *     n_f = f                                                              (MUON_NORM_NONE)
 *     u   = n_f post_gain + post_bias
 *     x'  = skip x + scale gate u          rounded to x_dtype, stored in `out`
 *     y   = n pre_gain + pre_bias          n the normalised rows of the rounded x'
 * The gate of row t is row t / gate_rows of `gate` (1: a value for each token; the
 * tokens of a sequence: a row for each sequence; rows: one learned vector).
 * Means are fp32 sums with up to 42 roundings: a mean's error, at most 42 2^-24 times
 * the row's mean magnitude, reaches each of its normalised values times r.
 * Without f there is no residual sum: x' = x, and only y is made.  Without a
 * pre-norm (MUON_NORM_NONE) there is no y.  Inputs whose rows are not 16-byte aligned
 * are read as the aligned 4-byte words that hold them.
 */
typedef enum {
    MUON_NORM_NONE = 0,
    MUON_NORM_RMS = 1,
    MUON_NORM_LAYER = 2
} muon_norm;

/* Largest row the seams take (one row is held in the registers of one block). */
#define MUON_SEAM_MAX_COLS 16384

typedef struct {
    int rows, cols;             /* 0 <= rows <= 2^30; 1 <= cols <= MUON_SEAM_MAX_COLS */
    muon_norm post, pre;        /* norm of f; norm of x'.  post must be NONE without f */
    float eps;                  /* > 0 */
    float skip, scale;          /* finite; skip must be 1 without f */
    const void* x;  long long ldx;       /* rows x cols, x_dtype, as are f, gate, out and y; ld >= cols elements */
    const void* f;  long long ldf;       /* the block's output, or NULL */
    const void* gate; long long ldgate;  /* ceil(rows / gate_rows) x cols, or NULL; needs f */
    int gate_rows;                       /* >= 1 with a gate */
    const void *post_gain, *post_bias;   /* cols elements of w_dtype, or NULL; need f */
    const void *pre_gain, *pre_bias;     /* likewise; need a pre-norm */
    void* out; long long ldout;          /* x'; NULL if and only if f is NULL; may be x or f, with its ld */
    void* y;   long long ldy;            /* NULL if and only if pre is NONE; may not overlap the others */
    muon_act8 post_c;           /* receives n_f (rows x cols); q NULL: not kept.  Needs f */
    muon_act8 pre_c;            /* receives n; q NULL: not kept.  Needs a pre-norm */
    float* post_rstd;           /* receives r_f (rows); NULL to skip.  Needs a post-norm */
    float* pre_rstd;            /* receives r (rows); NULL to skip.  Needs a pre-norm */
} muon_seam;

/*
 * One seam, asynchronous on `stream`; one launch, no workspace.  Argument errors
 * return before the launch (MUON_ERR_UNSUPPORTED: cols beyond
 * MUON_SEAM_MAX_COLS).  A checkpoint block that cannot be held raises
 * MUON_FLAG_NONFINITE in *d_status (when given).
 */
MUON_API muon_status seam_forward(const muon_seam* seam, muon_dtype x_dtype, muon_dtype w_dtype, int* d_status,
                                  muon_stream_t stream);

/*
 * Gradients of a seam.  With g = dy pre_gain, n and n_f the checkpoints' values:
 *     d    = dout + r (g - [mean g] - n mean(g n))      ([..]: MUON_NORM_LAYER)
 *     dx   = skip d
 *     du   = scale gate d;   h = du post_gain
 *     df   = r_f (h - [mean h] - n_f mean(h n_f))       (MUON_NORM_NONE: df = h)
 *     dgate = the sum over the gate row's tokens of scale d (n_f post_gain + post_bias)
 *     d_pre_gain  = sum_t dy n       d_pre_bias  = sum_t dy
 *     d_post_gain = sum_t du n_f     d_post_bias = sum_t du
 * each of the last four as d_v = beta d_v + the sum (beta = 0: not read).  Sums over
 * tokens run in fp32 in a fixed order and are rounded once.
 */
typedef struct {
    int rows, cols;             /* as muon_seam */
    muon_norm post, pre;
    float skip, scale;
    const void* gate; long long ldgate; int gate_rows;
    const void *post_gain, *post_bias, *pre_gain;
    muon_act8 post_c;           /* needed for a post-norm, dgate or d_post_gain; q NULL otherwise allowed */
    muon_act8 pre_c;            /* needed for a pre-norm */
    const float *post_rstd, *pre_rstd;   /* needed for that norm */
    const void* dy;   long long lddy;    /* x_dtype, as all that follow; NULL if and only if pre is NONE */
    const void* dout; long long lddout;  /* gradient that reaches x' on the residual path; NULL: none */
    void* dx; long long lddx;            /* required; may be dout or dy, with its ld */
    void* df; long long lddf;            /* NULL: the seam had no f; may be dy or dout, with its ld, when dx is not */
    void* dgate; long long lddgate;      /* as gate; NULL to skip */
    void *d_post_gain, *d_post_bias, *d_pre_gain, *d_pre_bias;   /* cols elements of w_dtype; NULL to skip */
    float beta;                 /* finite */
} muon_seam_grad;

/* Bytes of workspace seam_backward needs (pointers are compared with NULL only). */
MUON_API muon_status seam_backward_workspace_size(const muon_seam_grad* seam, size_t* bytes);

/*
 * Asynchronous on `stream`: one launch, and a second one that joins the sums over
 * tokens where vector or shared gate gradients are asked for.  workspace: device,
 * 256-byte aligned, at least seam_backward_workspace_size bytes (NULL when that
 * is 0); no state is kept in it between calls, and calls that overlap on the GPU
 * each need their own.  Errors as seam_forward; d_status is not written (a
 * checkpoint's NaN blocks make NaN gradients, which the step flags).
 */
MUON_API muon_status seam_backward(const muon_seam_grad* seam, muon_dtype x_dtype, muon_dtype w_dtype,
                                   void* workspace, size_t ws_bytes, int* d_status, muon_stream_t stream);

/*
 * Bytes of workspace ns_polar / gram_polar need for a batch of rows x cols
 * matrices in `dtype`.
 */
MUON_API muon_status ns_polar_workspace_size(int batch, int rows, int cols, muon_dtype dtype,
                                    size_t* bytes);
MUON_API muon_status gram_polar_workspace_size(int batch, int rows, int cols, muon_dtype dtype,
                                      size_t* bytes);

/*
 * Orthogonalise a batch of matrices with the direct iteration ([POLAR]
 * Newton-Schulz).  X_in: device, batch matrices of rows x cols in `dtype`,
 * matrix i at X_in + i * batch_stride elements (batch_stride >= rows*cols).
 * X_out: device, same layout and dtype; may equal X_in.
 * dtype MUON_BF16 / MUON_FP16 run on tensor cores, MUON_FP32 on CUDA cores.
 * A MUON_BF16 batch is iterated in fp16 ([POLAR]: fp16 is the recommended
 * type; bfloat16's 8 significant bits lose the small singular directions at
 * condition numbers near 1e3): one extra read of the input sums its squares,
 * and the copy the iteration starts from is X / (||X||_F + eps), which fp16
 * holds without overflow.  Input and output stay bfloat16.
 */
MUON_API muon_status ns_polar(const void* X_in, void* X_out, int batch, int rows, int cols,
                     long long batch_stride, muon_dtype dtype, const muon_schedule* sched,
                     void* workspace, size_t ws_bytes, int* d_status, muon_stream_t stream);

/*
 * The same result through the Gram route ([POLAR] X (X^T X)^{-1/2}): all
 * iteration steps work on s x s symmetric matrices (upper tiles computed and
 * mirrored); the s x l operand is touched only at the start, at restarts and
 * at the end.  Arguments as ns_polar; sched->restarts and sched->scale_f
 * select the restart steps and the divisor f.
 */
MUON_API muon_status gram_polar(const void* X_in, void* X_out, int batch, int rows, int cols,
                       long long batch_stride, muon_dtype dtype, const muon_schedule* sched,
                       void* workspace, size_t ws_bytes, int* d_status, muon_stream_t stream);

/*
 * ns_polar without a workspace argument, for callers that cannot allocate
 * device memory when they need the orthogonalisation: code running during CUDA
 * graph capture, runtimes whose allocators forbid outside allocations, and
 * plugins that only receive pointers to existing buffers.  The pages describe
 * no such entry point; it exists for this library's users.
 *
 * It runs exactly the ns_polar iteration with a fixed scratch array compiled
 * into the library: ns_polar_noalloc_capacity() bytes (32 MiB) of device
 * memory that every GPU loading the library keeps until the process exits.
 * A request whose ns_polar_workspace_size exceeds that capacity returns
 * MUON_ERR_WORKSPACE without launching anything.  Nothing is allocated: no
 * cudaMalloc, cudaFree or allocating library routine is called.
 *   - The first call on each device looks up the scratch array's device
 *     address (cudaGetSymbolAddress, with that device current); make that
 *     first call before any stream capture.  The address is remembered with
 *     the id of the CUDA context it was taken in and looked up again when a
 *     call finds a different context current (after cudaDeviceReset, say);
 *     such a call, too, should come before any capture.
 *   - All calls on a device share the scratch, which keeps the previous
 *     call's contents (each call clears what must start at zero).  Calls that
 *     overlap on the GPU (unordered streams) race: order them.
 * Arguments and results are those of ns_polar.
 */
MUON_API muon_status ns_polar_noalloc(const void* X_in, void* X_out, int batch, int rows, int cols,
                                      long long batch_stride, muon_dtype dtype,
                                      const muon_schedule* sched, int* d_status, muon_stream_t stream);
/* Bytes of the fixed scratch behind ns_polar_noalloc. */
MUON_API size_t ns_polar_noalloc_capacity(void);

/*
 * Tracing aid (optional).  While enabled, every kernel the library launches
 * is bracketed by two CUDA events recorded on the launch stream, and the
 * launch's algorithmic work is noted: floating-point operations for the
 * Newton-Schulz products (a symmetric product counts the half it needs,
 * n*n*k; a full product 2*m*n*k) or bytes moved for the elementwise pass.
 * Events come from a fixed host-side pool created on first use (up to
 * MUON_TRACE_CAPACITY launches; later launches are not recorded).
 * muon_trace_read synchronises on the recorded events, copies up to `max`
 * records (oldest first) to `out` (host array), clears the log and returns
 * the number of records copied (or -1 on a CUDA error).
 */
#define MUON_TRACE_CAPACITY 8192
typedef enum {
    MUON_KERNEL_PREPASS = 0,   /* fused MONA pre-pass / input copy + norms (work = bytes) */
    MUON_KERNEL_SYM = 1,       /* tcgen05 symmetric product X X^T, A A, ... (work = flops) */
    MUON_KERNEL_UPD = 2,       /* tcgen05 update product X <- aX + BX, Q Xb (work = flops) */
    MUON_KERNEL_SIMT = 3,      /* fp32 CUDA-core product (work = flops) */
    MUON_KERNEL_OTHER = 4,     /* identity fill (work = bytes) */
    MUON_KERNEL_ADAMW = 5,     /* AdamW streaming pass over vector parameters (work = bytes) */
    MUON_KERNEL_RSVD = 6,      /* LiMuon streaming passes: momentum + sketch, projection, update (work = bytes) */
    MUON_KERNEL_RSVD_SMALL = 7, /* LiMuon per-matrix factorisations: QR, eigen-decomposition (work = bytes) */
    MUON_KERNEL_ACT8 = 8,      /* checkpoint encode / decode, gradient operand copies and joins (work = bytes) */
    MUON_KERNEL_ACT8_GRAD = 9, /* weight gradients from checkpoints (work = flops) */
    MUON_KERNEL_SEAM = 10      /* block seams and the joins of their sums (work = bytes) */
} muon_kernel_kind;

typedef struct {
    int kind;        /* muon_kernel_kind */
    double work;     /* algorithmic flops or bytes of this launch */
    float ms;        /* device time between the bracketing events */
} muon_trace_record;

MUON_API muon_status muon_trace_enable(int enable);
MUON_API int muon_trace_read(muon_trace_record* out, int max);

/*
 * Self-test of the failure path: one block runs the library's bounded wait
 * on a barrier that nothing completes, with a limit of wait_ms milliseconds
 * (1..4000); the wait gives up, ORs MUON_FLAG_TIMEOUT into *d_status (device,
 * required) and the kernel returns normally.  No pages' counterpart: it lets a
 * caller check that a stuck wait ends in a status word, not a hung GPU.
 */
MUON_API muon_status muon_wait_selftest(int wait_ms, int* d_status, muon_stream_t stream);

/* Static, NUL-terminated description of a status code. */
MUON_API const char* muon_status_string(muon_status status);

#ifdef __cplusplus
}
#endif

#endif /* MUON_B200_H */
