/*
 * shampoo.h -- C ABI of the MI355X (gfx950) Shampoo block-preconditioner library.
 *
 * One optimizer step of Shampoo's block preconditioner, for a stack of
 * B x B blocks, in five calls:
 *
 *   shampoo_accumulate       L <- alpha L + gamma G G^T,  R <- alpha R + gamma G^T G
 *   shampoo_scale_power      trace, damping eps and scale c (power iteration or Frobenius)
 *   shampoo_invroot_newton   X ~ c^{-1/p} ((F + eps I)/c)^{-1/p} by Newton-DB or coupled Newton
 *   shampoo_invroot_cheby    the same by a Chebyshev polynomial evaluated with Clenshaw
 *   shampoo_precondition     U = X_L G X_R
 *   shampoo_graft_update     theta <- theta - lr (||P||/||U||) U with P Adam's direction
 *
 * Beside it, for the tensors that are not blocked and for the layers whose
 * gradients the step consumes:
 *
 *   shampoo_grad_norm        norm of many tensors and the coefficient that clips it
 *   shampoo_adamw            an AdamW step over many tensors, moments in 32 or 8 bits
 *   shampoo_mx4_quantize     4-bit microscaled (MX4) copies of a matrix, along its rows and columns
 *   shampoo_mx4_product      C <- alpha A B^T + beta C on MX4 operands
 *   shampoo_mx4_linear       Y = mx4(X) W^T with an MX4 weight
 *   shampoo_mx8_quantize     8-bit microscaled (MX8) copies of activations
 *   shampoo_activation       f(a) or f(a) b, the inputs kept in MX8 for the gradient
 *   shampoo_join             a block's output normed, gated, added to the residual and normed for the next block
 *
 * Sources (cited by page title and section): "DASH: Faster Shampoo via Batched
 * Block Preconditioning and Efficient Inverse-Root Solvers", the howistudyai.com
 * explainer of the paper ([DASH] below; its sections "Building blocks",
 * "High-level flow" and "Step-by-step"), and the arXiv 2602.02016 abstract.
 *
 * Conventions shared by every call
 * --------------------------------
 *  - All matrix pointers are DEVICE pointers owned by the caller.  Matrices are
 *    fp32, row-major.  A factor stack is float[nfactors][B][B], contiguous; the
 *    stack of a step holds the n left factors first, then the n right factors
 *    (nfactors = 2 n; block i owns factors i and n + i).
 *  - B must be a multiple of 64 with 64 <= B <= 16384 (SHAMPOO_EUNSUPPORTED).
 *  - A call only validates its arguments, enqueues kernels on `stream` and
 *    returns; it never synchronises and never allocates device memory.  Scratch
 *    memory comes from the caller's workspace `ws` of `ws_bytes` bytes (size from
 *    shampoo_workspace_bytes); it must stay allocated until the stream has
 *    executed the call, and one workspace must not be shared by calls that may
 *    run concurrently.  (shampoo_graft_update_noalloc takes no workspace: it
 *    uses a static device array of the library instead.)
 *  - The stream and the memory are of the calling thread's current device (a
 *    stream of 0 is that device's default stream).
 *  - Argument errors are returned synchronously as negative codes and nothing is
 *    enqueued.  A count of 0 (no blocks / factors) is a valid no-op.
 *  - Numerical trouble is reported per factor in a caller int32 status array on
 *    the device (bits below); shampoo_scale_power writes it, the inverse-root
 *    calls OR further bits into it.  Results are deterministic: no floating-point
 *    atomics are used, so a call repeated on the same inputs gives the same bits.
 *  - No C++ exception crosses this interface.
 */
#ifndef SHAMPOO_MI355X_H
#define SHAMPOO_MI355X_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SHAMPOO_ABI_VERSION 4

/* Return codes. */
enum {
  SHAMPOO_OK = 0,
  SHAMPOO_EINVAL = -1,        /* a null pointer, a negative count, a parameter out of range */
  SHAMPOO_EUNSUPPORTED = -2,  /* a valid value this library does not implement (B, p, prec) */
  SHAMPOO_EWORKSPACE = -3,    /* workspace missing or smaller than shampoo_workspace_bytes */
  SHAMPOO_EHIP = -4,          /* the HIP runtime refused a launch */
  SHAMPOO_ESCRATCH = -5       /* larger than the static scratch of shampoo_graft_update_noalloc */
};

/* Per-factor status bits (int32 status[nfactors] on the device). */
enum {
  SHAMPOO_BLK_NONFINITE = 1,  /* trace, spectral estimate or an iterate is not finite; values propagate */
  SHAMPOO_BLK_ZERO = 2,       /* tr(F) == 0 (all-zero history): X = I is returned */
  SHAMPOO_BLK_NONPOS_RQ = 4,  /* spectral estimate <= 0: X = I is returned */
  SHAMPOO_BLK_RESID_GROWTH = 8 /* a Newton residual rose above twice the smallest earlier residual of its
                                  pass: rounding errors are growing (the iteration diverges in this
                                  precision); X is still returned.  [DASH] "Limitations" and
                                  "Scoreboard with context" name unstable low-precision and
                                  Frobenius-scaled Newton runs; the pages give no detector */
};

/* Operand precision of the matrix products. */
enum {
  SHAMPOO_F32 = 0,            /* fp32 in, fp32 MFMA, fp32 accumulate */
  SHAMPOO_BF16_IN = 1         /* operands rounded to bf16 (RNE), bf16 MFMA, fp32 accumulate */
};

/* Scaling modes of shampoo_scale_power. */
enum {
  SHAMPOO_SCALE_POWER = 0,
  SHAMPOO_SCALE_FROBENIUS = 1
};

/* Iterations of shampoo_invroot_newton. */
enum {
  SHAMPOO_NDB = 0,            /* Newton-DB, second pass on Y (the pages' chaining) */
  SHAMPOO_NDB_Z = 1,          /* Newton-DB, second pass on Z_1 / (3/2)^iters (a variant) */
  SHAMPOO_CN = 2,             /* coupled Newton */
  SHAMPOO_CN_F16 = 3          /* coupled Newton on fp16 operands, fp32 accumulate (B % 128 == 0) */
};

/* Modifier bit, OR-ed into `variant` (shampoo_invroot_newton) or `prec`
 * (shampoo_invroot_cheby).  By default every product whose result is a
 * polynomial in the factor -- Newton-DB's Y E and E Z, coupled Newton's X C
 * and powers of C, Clenshaw's A_s b -- is symmetric in exact arithmetic, so
 * only its upper-triangular tiles are computed and mirrored (the outputs are
 * exactly symmetric).  The coupling products Z Y and C^p M are computed in
 * full by default.  With this bit set every product is computed in full. */
#define SHAMPOO_FULL_PRODUCTS 0x100

/* Opt-in modifier bit for shampoo_invroot_newton: form the coupling products
 * (Newton-DB's P = Z Y, coupled Newton's C^p M) from upper tiles as well,
 * which saves about 40% of their MFMA work.  They are symmetric in exact
 * arithmetic, but with the full product the coupled iterations stay
 * self-correcting: measured in fp32 on factors with a condition number of
 * 1e8, the mirrored coupling product matches the full one while the
 * iteration converges and then lets rounding errors grow until the iterates
 * overflow (Newton-DB by k = 15 per pass, where the full product stays
 * accurate); coupled Newton on fp16 operands loses accuracy the same way
 * over many iterations.  Use only for well-conditioned factors or few
 * iterations.  Ignored together with SHAMPOO_FULL_PRODUCTS. */
#define SHAMPOO_SYM_COUPLING 0x200

/* Operation ids of shampoo_workspace_bytes. */
enum {
  SHAMPOO_OP_ACCUMULATE = 1,
  SHAMPOO_OP_SCALE = 2,
  SHAMPOO_OP_NEWTON = 3,
  SHAMPOO_OP_CHEBY = 4,
  SHAMPOO_OP_PRECONDITION = 5,
  SHAMPOO_OP_GRAFT = 6
};

/* A B x B block inside a larger row-major fp32 matrix (a layer gradient or
 * the update).  `ptr` is the device address of the block's element (0,0), `ld`
 * the row stride in elements.  A partial edge block has rows < B or cols < B;
 * its missing entries read as zero and are never written.  Valid descriptors
 * have 0 <= rows, cols <= B and ld >= cols; the table itself lives in device
 * memory.  A descriptor that fails these checks on the device is treated as
 * an all-zero block (an invalid output descriptor is not written).  Vector
 * loads are used when ptr is 16-byte aligned and ld % 4 == 0, scalar loads
 * otherwise.  SHAMPOO_BF16_IN products need B % 128 == 0. */
typedef struct shampoo_block {
  float* ptr;
  int64_t ld;
  int32_t rows;
  int32_t cols;
} shampoo_block;

/* Per-factor scale record written by shampoo_scale_power (device memory). */
typedef struct shampoo_scale {
  float c;       /* scale constant: A_s = (F + eps I) / c */
  float eps;     /* damping: eps = eps_rel * tr(F) / B */
  float lambda;  /* spectral estimate (power) or ||F + eps I||_F (Frobenius) */
  float trace;   /* tr(F) */
} shampoo_scale;

/*
 * shampoo_accumulate -- EMA of the Kronecker factors of every block.
 * [DASH] "Step-by-step", building the preconditioners (an EMA of G G^T and
 * G^T G per block) and stacking the blocks into one 3D tensor.
 *
 *   g_blocks  device array [nblocks] of gradient block descriptors (read only)
 *   factors   device float[2 nblocks][B][B], updated in place:
 *               factors[i]          <- alpha factors[i]          + gamma G_i G_i^T
 *               factors[nblocks+i]  <- alpha factors[nblocks+i]  + gamma G_i^T G_i
 *             (alpha = beta, gamma = 1 - beta for the EMA; start from zeros)
 *   prec      SHAMPOO_F32 or SHAMPOO_BF16_IN (G rounded to bf16 before the product)
 *   ws        workspace of shampoo_workspace_bytes(SHAMPOO_OP_ACCUMULATE, nblocks, B, 0, prec)
 *             (0 bytes for SHAMPOO_F32; ws may then be NULL)
 */
int shampoo_accumulate(const shampoo_block* g_blocks, int64_t nblocks, int B,
                       float* factors, float alpha, float gamma, int prec,
                       void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * shampoo_scale_power -- trace, damping and scale of every factor.
 * [DASH] "Building blocks" (multi-power-iteration; Frobenius versus spectral
 * scaling) and "Step-by-step", scaling each block.
 *
 *   factors    device float[nfactors][B][B] (not modified); A = F + eps I.
 *              F is taken to be symmetric, as a factor formed by
 *              shampoo_accumulate is: when B is a multiple of 256, rounds
 *              after the first form W = A^T V (reading F by columns).  For
 *              an F that is not symmetric that is the same iteration on A^T,
 *              which has A's eigenvalues.
 *   eps_rel    eps = eps_rel * tr(F) / B (>= 0)
 *   mode       SHAMPOO_SCALE_POWER: r start vectors v0, `steps` rounds of
 *                W = A V, columns normalised; then q_j = v_j^T A v_j,
 *                lambda = max_j q_j, c = safety * lambda
 *              SHAMPOO_SCALE_FROBENIUS: lambda = c = ||A||_F (v0 may be NULL)
 *   v0         device float[nfactors][B][r], 1 <= r <= 32, steps >= 1
 *   safety     > 0 (the pages divide by about twice the estimate: 2.0)
 *   scale_out  device shampoo_scale[nfactors]
 *   status     device int32[nfactors], overwritten: ZERO if tr(F) == 0,
 *              NONPOS_RQ if lambda <= 0, NONFINITE if trace or lambda is not finite
 */
int shampoo_scale_power(const float* factors, int64_t nfactors, int B, float eps_rel,
                        int mode, const float* v0, int r, int steps, float safety,
                        shampoo_scale* scale_out, int32_t* status,
                        void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * shampoo_invroot_newton -- inverse p-th roots by inverse-free Newton iterations.
 * [DASH] "Building blocks" (Newton-DB) and "Step-by-step", solvers (a) Newton-DB
 * and (b) coupled Newton.
 *
 *   A_s = (F + eps I) / c with (c, eps) from `scale`; x_out = c^{-1/p} g(A_s).
 *   variant SHAMPOO_NDB:   pass(Y0): Z = I; iters times { E = (3I - Z Y)/2;
 *                          Y <- Y E; Z <- E Z }.  p = 2: X = pass(A_s).Z;
 *                          p = 4: X = pass(pass(A_s).Y).Z.
 *           SHAMPOO_NDB_Z: p = 4: s = (3/2)^iters, X = sqrt(s) pass(pass(A_s).Z / s).Y
 *           SHAMPOO_CN:    X = I, M = A_s; iters times { C = ((p+1) I - M)/p;
 *                          X <- X C; M <- C^p M };  p in {1, 2, 4, 8}
 *           SHAMPOO_CN_F16: the same iteration with every product on fp16
 *                          operands (RNE) and fp32 accumulation; only fp16
 *                          copies of the iterates are kept, X is written in fp32
 *                          ([DASH] Scoreboard: coupled Newton in FP16)
 *   iters      iterations per pass, 1..100
 *   x_out      device float[nfactors][B][B]
 *   resid_out  NULL or device float[nfactors][passes * iters]: ||I - Z Y||_F before
 *              each Newton-DB iteration (passes = 1 for p = 2, else 2), or
 *              ||I - M||_F before each coupled-Newton iteration (passes = 1)
 *   status     device int32[nfactors]; factors flagged ZERO or NONPOS_RQ get
 *              X = I; NONFINITE is added when a residual is not finite, and
 *              RESID_GROWTH when a residual exceeds twice the smallest earlier
 *              residual of the same pass (in exact arithmetic the residuals of a
 *              pass never increase for a spectrum inside the iteration's
 *              convergence region, (0, 3) for Newton-DB and (0, p + 1) for
 *              coupled Newton).  The residuals are computed whether or not
 *              resid_out is given.
 *   ws         shampoo_workspace_bytes(SHAMPOO_OP_NEWTON, nfactors, B, variant, SHAMPOO_F32)
 */
int shampoo_invroot_newton(const float* factors, const shampoo_scale* scale,
                           int64_t nfactors, int B, int p, int variant, int iters,
                           float* x_out, float* resid_out, int32_t* status,
                           void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * shampoo_invroot_cheby -- inverse p-th roots by a Chebyshev polynomial.
 * [DASH] "Building blocks" (Chebyshev) and "Step-by-step", solver (d).
 *
 *   The polynomial interpolates f(x) = x^{-1/p} at the degree+1 first-kind
 *   Chebyshev nodes of [interval_eps, 1 + interval_eps] (fitted on the host in
 *   double precision).  With T = 2 A_s - I it is evaluated by Clenshaw's
 *   recurrence b_j = c_j I + 2 T b_{j+1} - b_{j+2}, X = c_0 I + T b_1 - b_2,
 *   i.e. degree - 1 matrix products; x_out = c^{-1/p} X.
 *   degree     1..256;  p >= 1;  interval_eps >= 0
 *   prec       SHAMPOO_F32, or SHAMPOO_BF16_IN (products on bf16 operands,
 *              the recurrence itself in fp32)
 *   status     as for shampoo_invroot_newton (ZERO / NONPOS_RQ give X = I)
 *   ws         shampoo_workspace_bytes(SHAMPOO_OP_CHEBY, nfactors, B, degree, prec)
 */
int shampoo_invroot_cheby(const float* factors, const shampoo_scale* scale,
                          int64_t nfactors, int B, int p, int degree, double interval_eps,
                          int prec, float* x_out, int32_t* status,
                          void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * shampoo_precondition -- U_i = X_L,i G_i X_R,i for every block.
 * [DASH] "High-level flow" and "Step-by-step" (the preconditioned direction).
 *
 *   x_roots   device float[2 nblocks][B][B]: X_L of block i at i, X_R at nblocks + i
 *   g_blocks  device array [nblocks] of gradient block descriptors (read only)
 *   u_blocks  device array [nblocks] of output descriptors; only the rows x cols
 *             part of each output block is written.  Output blocks must not overlap
 *             the gradient blocks or each other.
 *   prec      SHAMPOO_F32 or SHAMPOO_BF16_IN
 *   ws        shampoo_workspace_bytes(SHAMPOO_OP_PRECONDITION, nblocks, B, 0, prec)
 */
int shampoo_precondition(const float* x_roots, const shampoo_block* g_blocks,
                         int64_t nblocks, int B, const shampoo_block* u_blocks, int prec,
                         void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * shampoo_graft_update -- grafted parameter update of every block.
 * [DASH] "Step-by-step", grafting: the update keeps the Shampoo direction U
 * and takes its length from an Adam-like direction P.
 *
 *   Per block (elementwise over the block's rows x cols, taken from g_blocks):
 *     m <- beta1 m + (1 - beta1) g;  v <- beta2 v + (1 - beta2) g^2          (in place)
 *     P = (m / (1 - beta1^step)) / (sqrt(v / (1 - beta2^step)) + eps)
 *     s = ||P||_F / ||U||_F  (0 when ||U||_F = 0)
 *     theta <- theta - lr s U                                              (in place)
 *   g_blocks, u_blocks (U from shampoo_precondition), param_blocks, m_blocks,
 *   v_blocks   device arrays [nblocks] of descriptors of blocks of the same shape;
 *              the m and v blocks hold Adam's state (zeros before step 1)
 *   step       1-based step count for the bias corrections;  0 <= beta1, beta2 < 1;  eps >= 0
 *   scale_out  NULL or device float[nblocks]: s of every block
 *   ws         shampoo_workspace_bytes(SHAMPOO_OP_GRAFT, nblocks, B, 0, SHAMPOO_F32)
 */
int shampoo_graft_update(const shampoo_block* g_blocks, const shampoo_block* u_blocks,
                         const shampoo_block* param_blocks, const shampoo_block* m_blocks,
                         const shampoo_block* v_blocks, int64_t nblocks, int B, float lr, float beta1,
                         float beta2, float eps, int step, float* scale_out,
                         void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * shampoo_graft_update_noalloc -- shampoo_graft_update without a workspace.
 * For callers that cannot allocate device memory: code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation.  The
 * per-block partial norms live in a static device array of
 * SHAMPOO_NOALLOC_SCRATCH_BYTES that the library holds on every GPU it runs
 * on until the process ends; this call allocates nothing and frees nothing.
 * Arguments, results and errors are those of shampoo_graft_update, plus
 * SHAMPOO_ESCRATCH (nothing enqueued) when the partial norms need more than
 * the static array: nblocks * min(max(B / 64, 1), 64) * 8 bytes, rounded up to
 * 256, must not exceed SHAMPOO_NOALLOC_SCRATCH_BYTES (e.g. up to 8192 blocks
 * at B = 1024).  The array starts with no meaningful contents and every call
 * overwrites all of the part it reads before reading it.  All calls on one
 * GPU share that GPU's array: calls that may overlap in time on the same GPU
 * (different streams, or different host threads without ordering) race and
 * must not be issued.  The first call on a device looks up the array's
 * address there (SHAMPOO_EHIP if that fails).
 */
#define SHAMPOO_NOALLOC_SCRATCH_BYTES (1u << 20)
int shampoo_graft_update_noalloc(const shampoo_block* g_blocks, const shampoo_block* u_blocks,
                                 const shampoo_block* param_blocks, const shampoo_block* m_blocks,
                                 const shampoo_block* v_blocks, int64_t nblocks, int B, float lr, float beta1,
                                 float beta2, float eps, int step, float* scale_out, hipStream_t stream);

/* -------------------------------------------------------------------------
 * AdamW over many tensors
 * ---------------------------------------------------------------------- */

/* Element types of the tensors below. */
enum {
  SHAMPOO_T_F32 = 0,
  SHAMPOO_T_BF16 = 1
};

/* Storage of AdamW's moments. */
enum {
  SHAMPOO_STATE_F32 = 0,
  SHAMPOO_STATE_MX8 = 1       /* one byte each, a scale byte per 32 elements (shampoo_adamw) */
};

/* A tensor of n elements, dense in memory, taken in its flat order.  `ptr` is
 * its device address, aligned to its element size (nothing more is needed);
 * `offset` the place of its first element in the state buffers, a multiple
 * of SHAMPOO_GROUP.  The table lives in device memory. */
typedef struct shampoo_tensor {
  void* ptr;
  int64_t n;
  int64_t offset;
} shampoo_tensor;

/* A piece of a tensor: its elements [index * SHAMPOO_SEGMENT,
 * min(n, (index + 1) * SHAMPOO_SEGMENT)).  A segment list names every piece
 * of every tensor of a table once, in device memory. */
typedef struct shampoo_segment {
  int32_t tensor;
  int32_t index;
} shampoo_segment;

#define SHAMPOO_GROUP 32       /* elements that share a scale byte */
#define SHAMPOO_SEGMENT 2048

/*
 * shampoo_grad_norm -- Euclidean norm of many tensors taken as one vector.
 *
 *   tensors, segments  device tables (nsegments pieces; n and ptr are used)
 *   dtype      SHAMPOO_T_F32 or SHAMPOO_T_BF16, of all tensors
 *   max_norm   > 0 (may be infinite)
 *   out        device float[2]: norm, and min(1, max_norm / norm) -- 1 for a norm
 *              of 0, NaN for a norm that is not finite
 *   ws         shampoo_grad_norm_workspace_bytes(nsegments) bytes
 * Squares are summed in double in a fixed order: no fp32 gradient overflows
 * them, and a call repeated gives the same bits.  nsegments = 0 gives 0 and 1.
 */
int shampoo_grad_norm(const shampoo_tensor* tensors, const shampoo_segment* segments, int64_t nsegments,
                      int dtype, float max_norm, float* out, void* ws, size_t ws_bytes, hipStream_t stream);
size_t shampoo_grad_norm_workspace_bytes(int64_t nsegments);

/*
 * shampoo_adamw -- one AdamW step (decoupled weight decay) of many tensors.
 *
 *   Per element, in fp32:
 *     g <- c g                                   (c = *grad_scale, 1 if grad_scale is NULL)
 *     m <- beta1 m + (1 - beta1) g;  v <- beta2 v + (1 - beta2) g^2
 *     p <- p (1 - eta w) - eta / (1 - beta1^step) m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 *   with eta = lr hyper[t][0] and w = hyper[t][1] of the element's tensor t.
 *
 *   params, grads, copies   device tables of the same tensors in the same order
 *              (copies may be NULL: else p is also written there in bf16,
 *              rounded to nearest even; only with fp32 parameters).  The
 *              state offsets are those of `params`.  No two tensors of
 *              params and copies share memory (gradients may)
 *   hyper      device float[ntensors][2]: factor on lr, weight decay
 *   param_dtype, grad_dtype   SHAMPOO_T_F32 or SHAMPOO_T_BF16
 *   m, v       device state at the tensors' offsets, 16-byte aligned: float, or
 *              for SHAMPOO_STATE_MX8 codes of one byte with m_scale and v_scale,
 *              one byte per SHAMPOO_GROUP elements (both NULL for SHAMPOO_STATE_F32)
 *   nsegments  below 2^24 (SHAMPOO_EUNSUPPORTED: divide the list)
 *   step       1-based step count;  0 <= beta1, beta2 < 1;  eps >= 0
 *   seed       of the stochastic rounding below (unused for fp32 parameters
 *              with SHAMPOO_STATE_F32)
 *   grad_scale NULL or a device float: a clipping or unscaling factor.  If it
 *              is not finite the call changes nothing
 *
 * SHAMPOO_STATE_MX8: an m code is a sign and an OCP E4M3 value (bias 7), a v
 * code an unsigned E5M3 value (bias 15, every code finite); the value is the
 * code's times 2^(s - 127), s the group's scale byte, and NaN for s = 255.
 * With E the exponent field of the group's largest magnitude, s = max(E - 7, 1)
 * for m and max(E - 15, 1) for v (255 if E = 255: one entry that is not finite
 * makes its group NaN).  Codes round stochastically: where x lies the fraction
 * f of the way between two neighbours, the upper is taken if
 * f + (h + 1/2) / 65536 >= 1, so that small changes of a moment are kept on
 * average; h is the low (m) or high (v) half of the element's 32-bit hash, a
 * function of seed, step and its place in the state buffer.  A v code is at
 * least 1: a moment that rounds to 0 cannot leave eps alone under m.
 * bf16 parameters round stochastically by the same rule (16 other bits of the
 * hash), fp32 parameters to nearest even.
 *
 * The bias corrections and the hash's key are formed from step and seed when
 * the call is made.  Captured into a graph, the call repeats them on every
 * replay: one step's bias correction, and one step's random bits, so that the
 * rounding of 8-bit moments and bf16 parameters, unbiased over steps, is not so
 * over replays.  Capture a call for each step, or call outside the graph, where that
 * matters.
 */
int shampoo_adamw(const shampoo_tensor* params, const shampoo_tensor* grads, const shampoo_tensor* copies,
                  const float* hyper, int64_t ntensors, const shampoo_segment* segments, int64_t nsegments,
                  int param_dtype, int grad_dtype, int state, void* m, void* v, uint8_t* m_scale,
                  uint8_t* v_scale, double lr, double beta1, double beta2, double eps, int step, uint64_t seed,
                  const float* grad_scale, hipStream_t stream);

/* Values of n 8-bit moments (n a multiple of SHAMPOO_GROUP) as fp32 or bf16.
 * fp32 holds every value exactly, bf16 those from 2^-126 up; smaller ones are
 * rounded to nearest even (a v code of 1 beside the least scale is 2^-143,
 * which becomes 0).  Either of m and v may be NULL with its
 * scale and output. */
int shampoo_adamw_moments(const uint8_t* m, const uint8_t* m_scale, const uint8_t* v, const uint8_t* v_scale,
                          int64_t n, void* m_out, void* v_out, int dtype, hipStream_t stream);

/* -------------------------------------------------------------------------
 * MX4: 4-bit microscaled matrices
 * ---------------------------------------------------------------------- */

/* An MX4 matrix of R rows and C columns is a pair of byte arrays,
 *   codes  [R][Cp / 2]   two E2M1 values a byte, the lower column in the low half
 *   scales [R][Cp / 32]  one E8M0 byte s for 32 consecutive columns: 2^(s - 127)
 * with Cp = C rounded up to a multiple of 128; the columns from C to Cp hold
 * code 0.  Both arrays are 16-byte aligned.  (OCP microscaling MXFP4.)
 * Sides are at most 2^31, the columns of a product 2^24, and what would take
 * 2^24 workgroups or more (from 2^28 rows of B, 2^29 of x) is SHAMPOO_EUNSUPPORTED. */
#define SHAMPOO_MX4_PAD 128

/*
 * shampoo_mx4_quantize -- MX4 copies of x and / or of its transpose.
 *
 *   x          device matrix [rows][cols] of dtype, row stride ld >= cols
 *   codes, scales      MX4 matrix [rows][cols], or both NULL
 *   codes_t, scales_t  MX4 matrix [cols][rows] of x^T (32 consecutive rows of x
 *              share a scale), or both NULL
 * s = max(E - 2, 0) with E the exponent field of the group's largest
 * magnitude as fp32; values round to nearest even and saturate at 6 * 2^(s-127).
 * A group with an entry that is not finite gets codes 0 and s = 255 (NaN).
 */
int shampoo_mx4_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                         uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t, hipStream_t stream);

/* Values of an MX4 matrix, as fp32 or bf16 (which holds every value that
 * shampoo_mx4_quantize writes exactly), row stride ld >= cols. */
int shampoo_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* out,
                           int dtype, int64_t ld, hipStream_t stream);

/*
 * shampoo_mx4_product -- C <- alpha A B^T + beta C, fp32 accumulation.
 *
 *   A [M][K] and B [N][K]   MX4 matrices
 *   C          device matrix [M][N] of dtype, row stride ldc >= N, apart from A
 *              and B.  beta = 0: C is only written
 *   ws         shampoo_mx4_workspace_bytes(M, N, K) bytes (NULL if that is 0)
 */
int shampoo_mx4_product(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* b_codes,
                        const uint8_t* b_scales, int64_t M, int64_t N, int64_t K, float alpha, float beta, void* c,
                        int dtype, int64_t ldc, void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * shampoo_mx4_linear -- Y = mx4(X) W^T: X [M][K] is quantised along its rows
 * and multiplied by the MX4 weight W [N][K].
 *
 *   X          of dtype, row stride ldx;  Y [M][N] of dtype, row stride ldy,
 *              apart from X (SHAMPOO_EINVAL; other columns of one matrix are)
 *   ws         shampoo_mx4_linear_workspace_bytes(M, N, K) bytes
 */
int shampoo_mx4_linear(const void* x, int64_t ldx, const uint8_t* w_codes, const uint8_t* w_scales, int64_t M,
                       int64_t N, int64_t K, void* y, int64_t ldy, int dtype, void* ws, size_t ws_bytes,
                       hipStream_t stream);

/* Workspace sizes of the two calls above (0 for invalid sizes too). */
size_t shampoo_mx4_workspace_bytes(int64_t M, int64_t N, int64_t K);
size_t shampoo_mx4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K);

/* -------------------------------------------------------------------------
 * MX8: activations kept in 8 bits
 * ---------------------------------------------------------------------- */

/* An MX8 matrix of R rows and C columns is a pair of byte arrays,
 *   codes  [R][Cp]        sign + OCP E4M3 (bias 7), one value a byte
 *   scales [R][Cp / 32]   one byte s for 32 consecutive columns: 2^(s - 127)
 * with Cp = C rounded up to a multiple of 32; the columns from C to Cp are
 * those of zeros.  Both arrays are 16-byte aligned.  (The format of AdamW's 8-bit first moments,
 * by rows and rounded to nearest even.)  At most 2^31 rows and 2^29 columns; beyond these, and where 2^24 workgroups
 * would be needed, calls here and of the activations are SHAMPOO_EUNSUPPORTED. */

/*
 * shampoo_mx8_quantize -- MX8 copy of x, a device matrix [rows][cols] of dtype
 * with row stride ld >= cols.  s = max(E - 7, 1) with E the exponent field of
 * the group's largest magnitude as fp32; codes round to nearest even and none
 * saturates.  A group with an entry that is not finite gets s = 255, and codes
 * that are E4M3's NaN (0x7f).
 */
int shampoo_mx8_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                         uint8_t* scales, hipStream_t stream);

/* Values of an MX8 matrix (s = 255: NaN), as fp32 (exact) or bf16 (exact from 2^-126 up,
 * smaller ones rounded to nearest even), row stride ld >= cols. */
int shampoo_mx8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* out,
                           int dtype, int64_t ld, hipStream_t stream);

/* -------------------------------------------------------------------------
 * Activations
 * ---------------------------------------------------------------------- */

enum {
  SHAMPOO_ACT_SILU = 0,       /* x / (1 + exp(-x)) */
  SHAMPOO_ACT_GELU = 1,       /* x Phi(x), Phi the normal distribution */
  SHAMPOO_ACT_GELU_TANH = 2,  /* x (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))) / 2 */
  SHAMPOO_ACT_RELU = 3,       /* max(x, 0), slope 0 at 0 */
  SHAMPOO_ACT_RELU2 = 4       /* max(x, 0)^2 */
};

/*
 * shampoo_activation -- y = f(a), or y = f(a) b where b is given; fp32
 * arithmetic, rounded once.
 *
 *   a, b, y    device matrices [rows][cols] of dtype, row strides lda, ldb, ldy;
 *              b may be NULL; y apart from a and b.  a and b may be halves
 *              of one matrix
 *   a_codes .. b_scales   NULL, or MX8 matrices that receive a (and b, where
 *              there is one) for the backward pass
 */
int shampoo_activation(int act, const void* a, int64_t lda, const void* b, int64_t ldb, int64_t rows, int64_t cols,
                       int dtype, void* y, int64_t ldy, uint8_t* a_codes, uint8_t* a_scales, uint8_t* b_codes,
                       uint8_t* b_scales, hipStream_t stream);

/*
 * shampoo_activation_backward -- da = dy f'(a) [b], db = dy f(a).
 *
 *   gated      whether there is a b
 *   a, b       the inputs, or where a_codes is given, their MX8 copies (a and b
 *              are then not used)
 *   da, db     of dtype; either may be NULL.  They may be halves of one matrix
 */
int shampoo_activation_backward(int act, const void* dy, int64_t lddy, const void* a, int64_t lda, const void* b,
                                int64_t ldb, const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* b_codes,
                                const uint8_t* b_scales, int gated, int64_t rows, int64_t cols, int dtype, void* da,
                                int64_t ldda, void* db, int64_t lddb, hipStream_t stream);

/* -------------------------------------------------------------------------
 * Norms, and the join of a block with its residual
 * ---------------------------------------------------------------------- */

enum {
  SHAMPOO_NORM_NONE = 0,
  SHAMPOO_NORM_RMS = 1,
  SHAMPOO_NORM_LAYER = 2
};

enum {
  SHAMPOO_GATE_NONE = 0,
  SHAMPOO_GATE_ROWS = 1,   /* [rows / gate_rows][cols]: a row of the gate for every gate_rows rows */
  SHAMPOO_GATE_TOKEN = 2   /* [rows]: a number for each row */
};

/* N(x) = (x - mean) s w + b over each row: RMS: mean = 0, s = 1 / sqrt(mean of
 * x^2 + eps); layer: s = 1 / sqrt(variance + eps).  Vectors of `cols` elements,
 * NULL: w = 1, b = 0.  In fp32: a row whose squares overflow it (elements from
 * about 2^60) has s = 0. */
typedef struct shampoo_norm {
  int64_t kind;
  double eps;              /* > 0; as fp32 */
  const void* weight;
  int64_t weight_dtype;
  const void* bias;
  int64_t bias_dtype;
} shampoo_norm;

/*
 * A join: with the residual r and a block's output y,
 *   z = N1(y),  h = scale r + gate z,  u = N2(h)       (N1 = after, N2 = before)
 * Either norm may be absent (kind SHAMPOO_NORM_NONE: z = y, no u), and so may y:
 * then h = r, nothing is written for it, and the join is the norm of r.
 *
 * Every matrix is [rows][cols] in device memory with a row stride (ld_) of at
 * least cols, of stream_dtype (r, h and their gradients) or branch_dtype (y, u
 * and theirs): equal, or fp32 and bf16.  Outputs are apart from inputs and each
 * other.  1 <= cols <= SHAMPOO_NORM_COLS for what has rows.  All members are 8
 * bytes wide; unused ones are 0.
 */
#define SHAMPOO_NORM_COLS 16384
typedef struct shampoo_join {
  int64_t rows, cols, stream_dtype, branch_dtype;
  const void* residual;
  int64_t ld_residual;
  const void* branch;      /* NULL: a norm only */
  int64_t ld_branch;
  double scale;            /* as fp32 */
  shampoo_norm after, before;
  int64_t gate_kind;       /* SHAMPOO_GATE_*; the gate is dense */
  const void* gate;
  int64_t gate_dtype, gate_rows;
  /* Kept for the backward pass: MX8 copies of the inputs (all NULL: backward
   * is given the inputs themselves), and fp32 [rows][2] mean and s of each norm,
   * 8-byte aligned (NULL in a forward pass without a backward one). */
  uint8_t *residual_codes, *residual_scales, *branch_codes, *branch_scales;
  float *after_stats, *before_stats;
} shampoo_join;

/*
 * shampoo_join_forward -- h and u (each needed where the join has one).  The MX8
 * copies and statistics that have an address are written.
 */
int shampoo_join_forward(const shampoo_join* join, void* h, int64_t ld_h, void* u, int64_t ld_u, hipStream_t stream);

/* Gradients: of the outputs, where there is one (NULL: zero), and of what is
 * wanted (else NULL).  Those of parameters have the parameters' types, and
 * the gate's layout. */
typedef struct shampoo_join_grads {
  const void* d_h;
  int64_t ld_d_h;
  const void* d_u;
  int64_t ld_d_u;
  void* d_residual;
  int64_t ld_d_residual;
  void* d_branch;
  int64_t ld_d_branch;
  void *d_after_weight, *d_after_bias, *d_gate, *d_before_weight, *d_before_bias;
} shampoo_join_grads;

/*
 * shampoo_join_backward -- the inputs are taken as shampoo_join_forward kept them: with codes,
 * from these (residual and branch then only have to be not NULL where there is such an
 * input); the row statistics are read, never formed again.  Sums over rows
 * are of fixed order: the same call gives the same bits.  The residual's codes
 * are read only where there is d_u, the branch's only with a norm after
 * it, a gate or d_u.  Copies are as shampoo_mx8_quantize writes them (NaN codes beside s = 255).
 *   ws         shampoo_join_backward_workspace_bytes(join, grads) bytes: rows of fp32 sums for some hundred
 *              workgroups, and where gradients of a gate of rows or of the norm after the branch
 *              are wanted, one (with a bias of that norm up to two) for each run of gate_rows
 *              rows: with gate_rows = 1 as much as an fp32 matrix.
 *              shampoo_join_workspace_bytes(join): enough for any grads
 */
int shampoo_join_backward(const shampoo_join* join, const shampoo_join_grads* grads, void* ws, size_t ws_bytes,
                          hipStream_t stream);
/* 0 for a join that is refused, and for one without rows or columns. */
size_t shampoo_join_workspace_bytes(const shampoo_join* join);
size_t shampoo_join_backward_workspace_bytes(const shampoo_join* join, const shampoo_join_grads* grads);

/* Workspace size in bytes for an operation (op = SHAMPOO_OP_*).  `count` is
 * nfactors for SCALE/NEWTON/CHEBY and nblocks for ACCUMULATE/PRECONDITION;
 * `variant_or_degree` is the Newton variant or the Chebyshev degree (else 0);
 * `count` is nblocks for GRAFT too.
 * Returns 0 for invalid arguments as well as for operations that need none. */
size_t shampoo_workspace_bytes(int op, int64_t count, int B, int variant_or_degree, int prec);

/* Static English text for a return code (never NULL). */
const char* shampoo_strerror(int code);

/* SHAMPOO_ABI_VERSION of the built library. */
int shampoo_abi_version(void);

/* Kernel families for shampoo_timing_hook (bits, OR-able). */
enum {
  SHAMPOO_TIME_OFF = 0,
  SHAMPOO_TIME_NDB_PAIR = 1,   /* Newton-DB updates Y E and E Z, launched together (2 products) */
  SHAMPOO_TIME_NDB_P = 2,      /* Newton-DB product Z Y with the E = (3I - P)/2 epilogue */
  SHAMPOO_TIME_CLENSHAW = 4,   /* one Clenshaw product A_s b (fp32 or bf16) */
  SHAMPOO_TIME_CN_M = 8,       /* coupled Newton's product C^p M (fp32 or fp16) */
  SHAMPOO_TIME_ALL = 15
};

/*
 * shampoo_timing_hook -- measurement instrumentation (not part of the method).
 * While enabled, each launch of a kernel family in the bit set `families`
 * made by any later call records events[2 i] just before and events[2 i + 1]
 * just after the launch on that call's stream, and (when fam_out is not NULL)
 * writes the launch's family bit to fam_out[i], a HOST array, for
 * i < capacity; further launches are not recorded.  `events` are
 * caller-created HIP events (2 * capacity of them) that must outlive the
 * recorded launches.  families = SHAMPOO_TIME_OFF disables the hook.  The hook
 * is process-wide and not thread-safe; enabling it resets the count.
 * shampoo_timing_count returns how many launches have been recorded.
 */
int shampoo_timing_hook(int families, hipEvent_t* events, int32_t* fam_out, int capacity);
int shampoo_timing_count(void);

#ifdef __cplusplus
}
#endif

#endif /* SHAMPOO_MI355X_H */
