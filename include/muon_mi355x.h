/*
 * muon_mi355x.h: C ABI of the MI355X (gfx950) Muon / Dimuon optimizer step,
 * of AdamW for the parameters Muon does not take, and of the global gradient
 * norm that clips both.
 *
 * One Muon call updates a batch of independent 2-D weight matrices of mixed
 * shapes:
 *
 *   momentum      M_t = mu * M_{t-1} + G
 *                 ("Muon Optimizer 정리", section "업데이트 규칙", eq. (1))
 *   orthogonalise O_t = NS5(M_t).  Divide by the Frobenius norm, then apply
 *                 X <- aX + b(XX^T)X + c(XX^T)^2 X a set number of times,
 *                 with (a, b, c) = (3.4445, -4.7750, 2.0315).
 *                 (same page, eq. (2) and section "Newton-Schulz 직교화";
 *                 sitech.ge Muon blog, section "SVD-ի փոխարեն՝ Newton–Schulz")
 *   update        W_t = W_{t-1} - lr * O_t   (same page, eq. (3))
 *
 * Gram side: when m > n, the library iterates on X^T, so the Gram matrix is
 * min(m, n) square ("From PCG to Muon", section "Muon's Gram Matrix").
 *
 * dimuon_step adds the diagonal conditioning of "Dimuon: LoRA 에 맞춰 다시 짠
 * Muon" (optim-book, "Dimuon diagonal conditioning"):
 *   - row energies R_i and column energies C_j are sums of squares of the
 *     momentum as it was BEFORE this step's update (section
 *     "왜 「지난」 모멘텀인가");
 *   - each factor is d = (E / max(E) + eps)^(-1/4) (section "문제 4");
 *   - the factors scale the momentum before orthogonalisation and the result
 *     after it (section "양쪽에서 −1/4 제곱");
 *   - the step is then rescaled so that ||O||_F equals the Frobenius norm of
 *     the orthogonaliser's output (the norm is fixed afterwards);
 *   - if the previous momentum is all zero, the factors are 1 and the step
 *     equals muon_step bit for bit.
 *
 * R and C are float32 sums in a fixed pairwise order.  Each square is
 * fl(x*x) of the stored value x.  The sequence along the row (column) is
 * zero-padded to a power of two.  Adjacent pairs are then added level by
 * level, left + right, each addition rounded to float32.  The order depends
 * only on (m, n).
 *
 * Optional extensions, all off by default:
 *   - Nesterov input G + mu*M_t ("From PCG to Muon", "DL Optimizer w/ Line
 *     Search");
 *   - decoupled weight decay, and a per-matrix update scale ("Muon
 *     Optimizer 정리", section "참고: 대규모 학습으로의 확장");
 *   - a per-iteration (a, b, c) schedule, the mechanism of the Polar Express
 *     iteration the Dimuon page names.
 *
 * Conventions
 *   - Every matrix is row-major and contiguous.  Its element size follows
 *     the dtype in the config.  Device pointers must be 16-byte aligned.
 *   - The caller owns all memory, including the workspace.  The library
 *     allocates no device memory.  It does allocate pinned host staging
 *     buffers, from which the batch's descriptor table (a few KB per matrix
 *     batch) is copied into the workspace: muon_step and dimuon_step keep
 *     them per host thread, take one whose previous copy has completed or
 *     else allocate another (hipHostMalloc), up to 64 per thread, and free
 *     them when the thread exits (adamw_step and muon_grad_norm take theirs
 *     from the same pool); a plan holds one, freed by its destroy function.  The only host-side wait: a thread that already
 *     has 64 descriptor copies in flight waits for its oldest.
 *   - Every call is asynchronous on `stream` (a hipStream_t; NULL means the
 *     default stream).  Host-side validation runs before anything is
 *     enqueued.  An invalid call returns an error code and leaves every
 *     buffer untouched.
 *   - muon_step and dimuon_step upload the descriptor table (a few KB) into
 *     the workspace on every call.  Calls that share a workspace must be
 *     ordered, for example on one stream.
 *   - A plan (muon_plan_create) validates and uploads once; muon_plan_step
 *     then only launches kernels.  While a plan exists, its workspace and
 *     every buffer it names must stay allocated, and the caller must not
 *     write to the workspace.
 *   - Numerical edge cases are not errors.  ||M||_F = 0 gives O = 0.
 *     NaN and Inf propagate as IEEE arithmetic does.
 */
#ifndef MUON_MI355X_H
#define MUON_MI355X_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MUON_ABI_VERSION 1

typedef enum muon_dtype {
  MUON_F32 = 0,  /* IEEE binary32 */
  MUON_BF16 = 1  /* bfloat16: 8 significant bits, binary32 exponent range */
} muon_dtype_t;

typedef enum muon_status {
  MUON_OK = 0,
  MUON_ERR_INVALID_ARG = 1,  /* null pointer, bad size, count < 1, bad ns_steps, ... */
  MUON_ERR_DTYPE = 2,        /* unsupported dtype combination */
  MUON_ERR_WORKSPACE = 3,    /* workspace null, misaligned or too small */
  MUON_ERR_ALIAS = 4,        /* two buffers of the batch overlap where they must not */
  MUON_ERR_HIP = 5,          /* a HIP runtime call or kernel launch failed */
  MUON_ERR_UNSUPPORTED = 6,  /* shape outside the supported range, or a call that
                                cannot run under stream capture */
  MUON_ERR_MEMORY = 7        /* host memory exhausted */
} muon_status_t;

/* One matrix of the batch.  Sizes are in elements. */
typedef struct muon_matrix {
  void* w;              /* device, m*n of cfg.w_dtype; W_{t-1} in, W_t out */
  const void* g;        /* device, m*n of cfg.g_dtype; gradient, read only */
  void* mom;            /* device, m*n of cfg.mom_dtype; M_{t-1} in, M_t out */
  float* o_out;         /* device or NULL: m*n float32, receives O_t (before lr) */
  float* energy_out;    /* device or NULL: m+n float32, receives R then C
                           (dimuon_step only; ignored by muon_step) */
  int64_t m;            /* rows, 1 <= m <= 65536 */
  int64_t n;            /* columns, 1 <= n <= 65536 */
  float update_scale;   /* multiplies O in the update; 1 for plain Muon */
  float reserved0;
} muon_matrix_t;

#define MUON_CONFIG_FIELDS 0x4D43F702u   /* value of muon_config_t.fields */

typedef struct muon_config {
  float lr;                     /* learning rate eta */
  float momentum;               /* mu */
  int32_t ns_steps;             /* Newton-Schulz iterations, 0..32; 5 is NS5 */
  float a, b, c;                /* quintic coefficients */
  const float* coeff_schedule;  /* host or NULL: ns_steps triples (a_t, b_t, c_t)
                                   replacing (a, b, c) iteration by iteration */
  muon_dtype_t w_dtype;         /* F32 or BF16 */
  muon_dtype_t g_dtype;         /* F32 or BF16 */
  muon_dtype_t mom_dtype;       /* F32 or BF16 */
  muon_dtype_t ns_dtype;        /* BF16: bf16 MFMA products with fp32 accumulation;
                                   F32: fp32 products and accumulation */
  float dimuon_eps;             /* floor added to the relative energy (1e-4) */
  int32_t nesterov;             /* nonzero: orthogonalise G + mu*M_t instead of M_t */
  float weight_decay;           /* W_t = W_{t-1} - lr*(scale*O_t + weight_decay*W_{t-1}) */
  uint32_t fields;              /* MUON_CONFIG_FIELDS (muon_config_default writes it): the caller knows
                                   grad_scale.  With any other value grad_scale is not looked at:
                                   it lies where earlier versions had reserved words, which a caller
                                   that fills the struct by hand may never have set. */
  const float* grad_scale;      /* device or NULL: one float32 s, read by the step; the step then
                                   uses s*G (rounded to float32) wherever G stands.  The clip
                                   coefficient of muon_grad_norm (out + 1) goes here.  Must stay
                                   allocated while a plan uses it, and lie outside every buffer
                                   the step writes. */
  int32_t reserved[1];
} muon_config_t;

/* Fill `cfg` with the defaults: lr 0.02, mu 0.95, NS5 (3.4445, -4.7750,
 * 2.0315), bf16 everywhere, eps 1e-4, no Nesterov, no weight decay, no
 * gradient scale (and `fields`, so that grad_scale counts once it is set). */
void muon_config_default(muon_config_t* cfg);

/* Bytes of device workspace a call over this batch needs.  The value covers
 * both muon_step and dimuon_step.  It is written to *bytes.  Checks the
 * arguments as a step would, but does not check pointers to buffers.
 * Errors: INVALID_ARG, DTYPE, UNSUPPORTED. */
muon_status_t muon_workspace_bytes(const muon_matrix_t* mats, int64_t count,
                                   const muon_config_t* cfg, size_t* bytes);

/* One Muon step over `count` matrices (host array `mats`).  `workspace` is
 * device memory of at least muon_workspace_bytes() bytes, 256-byte aligned.
 * Enqueues on `stream` and returns without synchronising (a thread with 64
 * descriptor copies still in flight first waits for its oldest; see the
 * staging buffers above).
 * Errors: INVALID_ARG, DTYPE, WORKSPACE, ALIAS, UNSUPPORTED, HIP. */
muon_status_t muon_step(const muon_matrix_t* mats, int64_t count,
                        const muon_config_t* cfg, void* workspace,
                        size_t workspace_bytes, void* stream);

/* One Dimuon step.  Same arguments and errors as muon_step. */
muon_status_t dimuon_step(const muon_matrix_t* mats, int64_t count,
                          const muon_config_t* cfg, void* workspace,
                          size_t workspace_bytes, void* stream);

/* For callers that cannot allocate: code under HIP graph capture, tight
 * serving loops, harnesses that forbid allocation.  One Muon step
 * (dimuon = 0) or Dimuon step (dimuon != 0) with the semantics of
 * muon_step / dimuon_step, but with no workspace argument: the library's
 * own static device array of MUON_NOALLOC_MAX_BYTES (64 MiB, held by each
 * GPU the library runs on until the process ends) serves as the workspace,
 * and the descriptor table reaches it through kernel arguments.  The call
 * allocates nothing: no device memory, no pinned host memory.
 *   - The batch must fit: a batch whose muon_workspace_bytes() exceeds
 *     MUON_NOALLOC_MAX_BYTES is rejected with MUON_ERR_WORKSPACE before
 *     anything is enqueued.  (Thin batches fit easily: the 64 LoRA pairs
 *     of 8 x 4096 and 4096 x 8 need about 7 MB.)
 *   - `stream` must belong to the current device; the array of that device
 *     is used.  Every call on one GPU shares that GPU's array, which keeps
 *     the last call's contents (no call depends on them): calls that
 *     overlap on one GPU race and must be ordered, for example on one
 *     stream.
 *   - Results equal muon_step / dimuon_step bit for bit (the same kernels).
 * Errors: INVALID_ARG, DTYPE, WORKSPACE (batch too large), ALIAS,
 * UNSUPPORTED, HIP. */
#define MUON_NOALLOC_MAX_BYTES ((size_t)64 << 20)
muon_status_t muon_step_noalloc(const muon_matrix_t* mats, int64_t count,
                                const muon_config_t* cfg, int32_t dimuon,
                                void* stream);

/* Kernel kinds reported by the launch-event hook. */
typedef enum muon_launch_kind {
  MUON_LAUNCH_START = -1,     /* event recorded before the first launch */
  MUON_LAUNCH_THIN = 0,       /* thin path pass B: k x k iteration, next energies, apply, update */
  MUON_LAUNCH_MOMENTUM = 1,   /* (not emitted: the momentum runs in the prescale pass) */
  MUON_LAUNCH_CONDITION = 2,  /* energies -> Dimuon factors */
  MUON_LAUNCH_PRESCALE = 3,   /* (not emitted: see MOMENTUM_PRESCALE) */
  MUON_LAUNCH_NORM = 4,       /* Frobenius norm of the prescaled copy */
  MUON_LAUNCH_GRAM = 5,       /* A = X X^T */
  MUON_LAUNCH_POLY = 6,       /* B = b A + c A A */
  MUON_LAUNCH_COMBINE = 7,    /* X = a X + B X (Muon, bf16 weights with rows of whole 8-element
                                 runs: the last one also applies the weight update) */
  MUON_LAUNCH_POSTNORM = 8,   /* Dimuon norm fix */
  MUON_LAUNCH_UPDATE = 9,     /* O and the weight update (not emitted when the last combine
                                 updated every matrix) */
  MUON_LAUNCH_THIN_ENERGY = 10, /* thin path: energies of M_{t-1} (no cached energies) */
  MUON_LAUNCH_THIN_A = 11,    /* thin path pass A: momentum, Gram partials */
  MUON_LAUNCH_MOMENTUM_PRESCALE = 12, /* momentum, Dimuon energies of M_t, conditioned and
                                         normalised bf16/f32 copy (+ transpose), one pass */
  MUON_LAUNCH_ENERGY = 13,    /* energies of M_{t-1} (general path, no cached energies) */
  MUON_LAUNCH_ADAMW = 14,     /* AdamW step */
  MUON_LAUNCH_STATE_GET = 15, /* AdamW moments to values */
  MUON_LAUNCH_STATE_SET = 16, /* values to AdamW moments */
  MUON_LAUNCH_GRAD_NORM = 17  /* global gradient norm */
} muon_launch_kind_t;

/* Timing hook, per host thread; not part of the method.  When `events` is
 * non-NULL, each later step on this thread records events[0] on the step's
 * stream before its first launch and events[i] after its i-th launch.  The
 * kind of launch i is written to kinds[i] (kinds[0] = MUON_LAUNCH_START).
 * `events` are hipEvent_t the caller created on the stream's device.  At
 * most `n` events are recorded.  Pass NULL to switch the hook off.  The
 * return value is the number of events the last step recorded. */
int32_t muon_set_launch_events(void* const* events, int32_t* kinds, int32_t n);

/* Prepared batch for repeated steps (an optimizer's fixed parameter list).
 * Validation, planning and the descriptor upload happen once, in create.
 * Each muon_plan_step runs one Muon step (dimuon = 0) or one Dimuon step
 * (dimuon != 0) over the batch, with the same semantics as muon_step /
 * dimuon_step.  The config, including the coefficient schedule, is copied.
 * Errors of create: as muon_step; of step: INVALID_ARG (NULL plan), HIP. */
typedef struct muon_plan muon_plan_t;
muon_status_t muon_plan_create(const muon_matrix_t* mats, int64_t count,
                               const muon_config_t* cfg, int32_t dimuon,
                               void* workspace, size_t workspace_bytes,
                               void* stream, muon_plan_t** plan);
muon_status_t muon_plan_step(muon_plan_t* plan, void* stream);
/* A Dimuon plan keeps, in its workspace, the row/column energies of the
 * momentum its last step wrote (the next step's R and C), so the next step
 * need not read M_{t-1} an extra time to compute them.  Call
 * muon_plan_reset after writing to the momentum buffers outside the plan
 * (resume, reset); the next step then recomputes them.  Muon plans ignore it. */
muon_status_t muon_plan_reset(muon_plan_t* plan);
/* Learning rate used by later steps of the plan (must be finite). */
muon_status_t muon_plan_set_lr(muon_plan_t* plan, float lr);
/* Replay the plan's launch sequence as a HIP graph (enable != 0) or launch
 * its kernels one by one (enable = 0, the default).  With graphs on, the
 * first step in each state of the sequence captures it (on a private stream
 * the plan creates; a Dimuon plan alternates between two states) and every
 * step then launches the instantiated graph on `stream`.  Results are the
 * same bit for bit.  Steps that run eagerly even with graphs on: a Dimuon
 * plan's first step and the step after muon_plan_reset (they also compute
 * the energies of M_{t-1}), and steps timed through muon_set_launch_events.
 * muon_plan_set_lr with a new rate discards the captured graphs.
 * Errors: INVALID_ARG (NULL plan), HIP. */
muon_status_t muon_plan_set_graph(muon_plan_t* plan, int32_t enable);
/* Waits for the plan's upload to finish, then frees the plan (NULL is a no-op). */
void muon_plan_destroy(muon_plan_t* plan);

/* ------------------------------------------------------------------------
 * AdamW, for the parameters Muon does not take (embeddings, heads, norm
 * weights, biases): one call updates many tensors of any sizes.
 *
 *   y   = s * g                               (s: grad_scale, 1 if NULL)
 *   m_t = beta1 * m_{t-1} + (1 - beta1) * y
 *   v_t = beta2 * v_{t-1} + (1 - beta2) * y^2
 *   w_t = w_{t-1} - lr * ( lr_scale * m^ / (sqrt(v^) + eps) + weight_decay * w_{t-1} )
 *   with m^ = m_t / (1 - beta1^t),  v^ = v_t / (1 - beta2^t)
 *
 * (decoupled weight decay, as in muon_step; the sitech.ge Muon blog and "From
 * PCG to Muon" leave the parameters that are not hidden matrices to AdamW).
 * All arithmetic is in binary32 (a v_t below 2^-126 counts as zero under the
 * root); the weight is rounded to its dtype once, at the end, to nearest even.
 * With `master`, w_{t-1} is read from the float32 master copy, which takes w_t
 * unrounded, and w is only written.
 *
 * Moments in 32 bits (ADAMW_STATE_F32): m and v are float32, n elements each.
 *
 * Moments in 8 bits (ADAMW_STATE_BLOCK8): a tensor's elements are cut, in
 * memory order, into blocks of ADAMW_BLOCK (the last one may be shorter).
 * A block holds one float32 per moment and one byte per element and moment:
 *   m  = e4m3(code) * m_scale     m_scale = max|m| / 256 over the block.
 *        The code is OCP float8 e4m3 (torch.float8_e4m3fn); the block's
 *        largest |m| has the code of 256.  A block whose largest |m| is below
 *        2^-118 is stored as zeros, its scale too.
 *   v  = u(code) * v_scale        v_scale = max v over the block.
 *        u is an unsigned float with 5 exponent and 3 mantissa bits: u(0) = 0,
 *        u(255) = NaN, and u(c) is the binary32 with the bits
 *        (c + 768) << 20 otherwise, so u(248) = 1.  A v above zero never takes
 *        code 0: it is stored as at least u(1) = 1.125 * 2^-31, so that no
 *        element's denominator falls to eps.  (With a v_scale below 2^-94, or
 *        a beta2 below 1/2, beta2 times the smallest values may fall below
 *        2^-126, and then counts as zero under the root all the same.)
 * A non-finite m or v, and a negative v, has the code of NaN, and the block's
 * scale is that of its other elements.  m^ and v^ of a step come from the
 * new moments before they are rounded to codes.  Rounding to a code:
 *   ADAMW_ROUND_NEAREST     half a code step is added, then the value is cut.
 *        Once an element's v changes by less than half a code step (1/32 to
 *        1/16 of it) per step, its code stays where it is relative to the
 *        block's largest v.
 *   ADAMW_ROUND_STOCHASTIC  (r + 1/2) / 65536 of a code step is added, r in
 *        0..65535 from a counter hash: the expected value is the unrounded
 *        one (to 2^-17 of a code step).  r depends only on the seed, the step
 *        number t and the element's place in the batch, so a step repeats bit
 *        for bit.  With i the element's index in the batch (every tensor's
 *        first element at a multiple of ADAMW_BLOCK, in the batch's order),
 *        lo and hi meaning the lower and upper 32 bits, and all sums and
 *        products modulo 2^32:
 *          mix(x): x ^= x >> 16; x *= 0x6A09E667; x ^= x >> 15;
 *                  x *= 0xBB67AE85; x ^= x >> 16
 *          key  = mix(lo(seed) ^ mix(hi(seed) ^ mix(lo(t) ^ mix(hi(t) ^ 0x3C6EF372))))
 *          h    = mix(lo(i) + mix(key + hi(i)))
 *        m takes the lower 16 bits of h as r, v the upper 16.
 *
 * Numerical edge cases are not errors: NaN and Inf propagate, and eps = 0
 * with v = 0 divides by zero, as IEEE arithmetic does.
 *
 * Buffers: contiguous, 16-byte aligned (the scales 4-byte), none written by
 * the call overlapping another (gradients may share memory).  A tensor with
 * n = 0 is skipped and its pointers are not looked at.  Device memory,
 * workspaces, streams and errors are as in the Muon calls; plan calls make
 * the plan's device current while they run and restore the caller's.
 * ------------------------------------------------------------------------ */
#define ADAMW_BLOCK 256

typedef enum adamw_state {
  ADAMW_STATE_F32 = 0,
  ADAMW_STATE_BLOCK8 = 1
} adamw_state_t;

typedef enum adamw_rounding {
  ADAMW_ROUND_NEAREST = 0,
  ADAMW_ROUND_STOCHASTIC = 1
} adamw_rounding_t;

/* One tensor of the batch.  Sizes are in elements. */
typedef struct adamw_tensor {
  void* w;              /* device, n of cfg.w_dtype: w_{t-1} in (without master), w_t out */
  const void* g;        /* device, n of cfg.g_dtype: gradient, read only */
  void* m;              /* device, n float32 or n bytes: first moment, in and out */
  void* v;              /* device, n float32 or n bytes: second moment, in and out */
  float* m_scale;       /* device, ceil(n / ADAMW_BLOCK) float32 (BLOCK8 only) */
  float* v_scale;       /* device, ceil(n / ADAMW_BLOCK) float32 (BLOCK8 only) */
  float* master;        /* device or NULL: n float32 master weights (w_dtype BF16 only;
                           all tensors of a batch or none) */
  int64_t n;            /* elements, 0 <= n <= 2^40 */
  float lr_scale;       /* multiplies the Adam term of the update; 1 for plain AdamW */
  float weight_decay;
} adamw_tensor_t;

typedef struct adamw_config {
  double beta1, beta2;          /* in [0, 1) */
  float lr;
  float eps;                    /* >= 0 */
  uint64_t seed;                /* of the stochastic rounding */
  const float* grad_scale;      /* device or NULL: one float32 s (the clip coefficient of
                                   muon_grad_norm, out + 1); read by the step, lies outside
                                   every buffer the step writes */
  muon_dtype_t w_dtype;         /* F32 or BF16 */
  muon_dtype_t g_dtype;         /* F32 or BF16 */
  int32_t state;                /* adamw_state_t */
  int32_t rounding;             /* adamw_rounding_t (BLOCK8) */
  int32_t reserved[4];
} adamw_config_t;

/* Fill `cfg` with the defaults: betas 0.9 and 0.999, lr 1e-3, eps 1e-8, bf16
 * weights and gradients, 32-bit moments, stochastic rounding, seed 0. */
void adamw_config_default(adamw_config_t* cfg);

/* Bytes of device workspace a call or a plan over this batch needs.
 * Errors: INVALID_ARG, DTYPE, UNSUPPORTED (n above 2^40, more than 2^20
 * tensors, more than 2^23 - 1 units of 4096 elements), MEMORY. */
muon_status_t adamw_workspace_bytes(const adamw_tensor_t* tensors, int64_t count,
                                    const adamw_config_t* cfg, size_t* bytes);

/* One AdamW step over `count` tensors (host array); `step` is t, from 1 on
 * (at most 2^62).
 * Asynchronous on `stream`.  Uploads its descriptor table through a pinned
 * staging buffer, so it is refused while `stream` is being captured: capture
 * a plan's step instead.
 * Errors: INVALID_ARG, DTYPE, WORKSPACE, ALIAS, UNSUPPORTED, HIP, MEMORY. */
muon_status_t adamw_step(const adamw_tensor_t* tensors, int64_t count, const adamw_config_t* cfg,
                         int64_t step, void* workspace, size_t workspace_bytes, void* stream);

/* Prepared batch for repeated steps.  `steps_done` is the number of steps the
 * moments have already taken (0 for new ones).  The step number and the
 * learning rate live in the workspace and each step advances the number on
 * the device, so a captured adamw_plan_step replays as the next step, with
 * the rate set last.  Calls on one plan must be ordered, for example on one
 * stream.  set_lr, set_step, get_state and set_state are asynchronous on
 * `stream`, and can be captured too (a replay then sets the captured value).
 * Errors of create: as adamw_step; of the others: INVALID_ARG, ALIAS, DTYPE,
 * HIP. */
typedef struct adamw_plan adamw_plan_t;
muon_status_t adamw_plan_create(const adamw_tensor_t* tensors, int64_t count, const adamw_config_t* cfg,
                                int64_t steps_done, void* workspace, size_t workspace_bytes,
                                void* stream, adamw_plan_t** plan);
muon_status_t adamw_plan_step(adamw_plan_t* plan, void* stream);
/* Learning rate of later steps (finite). */
muon_status_t adamw_plan_set_lr(adamw_plan_t* plan, float lr, void* stream);
/* Number of steps done, for resuming (>= 0, below 2^62). */
muon_status_t adamw_plan_set_step(adamw_plan_t* plan, int64_t steps_done, void* stream);
/* The moments as values, for checkpoints and for moving between 32- and 8-bit
 * moments.  `m` and `v` are device buffers of adamw_state_elems() elements of
 * `dtype` (F32 or BF16), 16-byte aligned, overlapping no buffer of the plan;
 * tensor i's n values start at the sum over j < i of n_j rounded up to
 * ADAMW_BLOCK.  The gaps are left as they were.  set_state rounds to 8-bit
 * codes to nearest.  get_state in F32 followed by set_state keeps m's codes
 * where m_scale is a normal float32 number, and v's where v_scale is 2^-114
 * or more; with smaller scales the smallest values lose bits to float32's
 * own range, down to zero. */
muon_status_t adamw_plan_get_state(adamw_plan_t* plan, void* m, void* v, muon_dtype_t dtype, void* stream);
muon_status_t adamw_plan_set_state(adamw_plan_t* plan, const void* m, const void* v, muon_dtype_t dtype,
                                   void* stream);
muon_status_t adamw_state_elems(const adamw_tensor_t* tensors, int64_t count, int64_t* elems);
/* Waits for the plan's upload to finish, then frees the plan (NULL is a no-op). */
void adamw_plan_destroy(adamw_plan_t* plan);

/* ------------------------------------------------------------------------
 * Global gradient norm and clip coefficient over many tensors:
 *   out[0] = N = sqrt(sum over all elements of g^2)
 *   out[1] = 1 if N <= max_norm, else max_norm / N
 * out[1] is meant for grad_scale of muon_config_t and adamw_config_t: the
 * gradients are clipped where the steps read them, and no pass rewrites them.
 * tensor_norms (NULL or `count` float32) receives every tensor's own norm.
 * Squares and sums are binary64 in an order that depends only on the sizes
 * and dtypes, so no float32 gradient overflows the sum and results repeat bit
 * for bit.  NaN gives N = NaN and out[1] = NaN; Inf gives N = Inf and 0.
 * A tensor with n = 0 has norm 0.  max_norm > 0; +Inf measures only (out[1]
 * is 1, or NaN).  At most 2^20 tensors, and 2^24 - 1 pieces of 32 KB.
 * The gradients may share memory; out and tensor_norms overlap no other
 * buffer.  Workspace, stream and capture rules are those of adamw_step and
 * of its plan.
 * ------------------------------------------------------------------------ */
typedef struct muon_grad {
  const void* g;        /* device, n of dtype, 16-byte aligned */
  int64_t n;            /* elements, 0 <= n <= 2^40 */
  muon_dtype_t dtype;   /* F32 or BF16; a batch may mix them */
  int32_t reserved0;
} muon_grad_t;

muon_status_t muon_grad_norm_workspace_bytes(const muon_grad_t* grads, int64_t count, size_t* bytes);
muon_status_t muon_grad_norm(const muon_grad_t* grads, int64_t count, float max_norm, float* out,
                             float* tensor_norms, void* workspace, size_t workspace_bytes, void* stream);
typedef struct muon_grad_norm_plan muon_grad_norm_plan_t;
muon_status_t muon_grad_norm_plan_create(const muon_grad_t* grads, int64_t count, float max_norm, float* out,
                                         float* tensor_norms, void* workspace, size_t workspace_bytes,
                                         void* stream, muon_grad_norm_plan_t** plan);
muon_status_t muon_grad_norm_plan_run(muon_grad_norm_plan_t* plan, void* stream);
void muon_grad_norm_plan_destroy(muon_grad_norm_plan_t* plan);

/* Static description of a status code. */
const char* muon_status_string(muon_status_t status);

/* Detail message of the last failed call on this host thread ("" if none). */
const char* muon_last_error(void);

/* MUON_ABI_VERSION of the loaded library. */
int32_t muon_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MUON_MI355X_H */
