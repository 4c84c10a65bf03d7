/*
 * libmuon: the Muon optimizer step on one GB300 (sm_103a), C ABI.
 *
 * The step (HyperParallel FSDP Muon RFC, mindspore hyper-parallel issue
 * "HyperParallel FSDP Muon优化器性能优化 RFC"):
 *   1. momentum   M' = beta*M + G;  V = G + beta*M' (Nesterov) or V = M'
 *                 (section 1(1): the orthogonalised matrix is the gradient
 *                 momentum M_t);
 *   2. normalise  X0 = V / (||V||_F + eps) per matrix slice;
 *   3. Newton-Schulz, T steps on the slice, worked on transposed when M > N
 *                 (sections 1 and 2: needs the whole matrix, depends only on
 *                 the last two dims):
 *                   A = X X^T;  B = b*A + c*A*A;  X <- a*X + B*X;
 *   4. update     W' = W*(1 - lr*wd) - lr*s*O,  s = sqrt(max(1, M/N))
 *                 (section 6: AdamW-style decoupled weight decay).
 * Slices whose trailing dims agree are regrouped into one batch and each
 * [E, M, N] tensor contributes E independent slices (sections 2 and 3).
 *
 * Ownership: the caller allocates and owns every device buffer (parameters,
 * gradients, momentum, workspace).  A plan owns host memory only.  muon_step
 * is asynchronous on the given stream, allocates nothing and never
 * synchronises the host.
 *
 * Errors: every call returns a muon_status; nothing aborts or throws.
 * Arguments are validated before any launch.  Launch failures return
 * MUON_ERR_CUDA.  A device-side wait that runs out of its iteration budget
 * writes an error word into the workspace header; muon_workspace_error reads
 * it.  Every kernel of a step checks that word when it starts and returns
 * at once when it is set, and a kernel whose own wait gave up stores no
 * parameter and no momentum after that point: such a step leaves the
 * parameters of the slices not yet updated as they were (momenta may have
 * advanced).  The word stays set until the caller clears it.
 *
 * Environment (read by the library at each call):
 *   MUON_LOG=1        muon_plan prints the plan to stderr (one line per
 *                     group: dims, dtype, slices, tr, scale, kernel, chunk,
 *                     workspace).
 *   MUON_FAULT=alloc  muon_plan fails as if host memory ran out
 *                     (MUON_ERR_NOMEM), before allocating anything.
 *   MUON_FAULT=launch the step calls fail as if the first launch had
 *                     failed (MUON_ERR_CUDA), after validating their
 *                     arguments and before any device work.
 *   MUON_FAULT=timeout every bounded device wait of the step kernels gives
 *                     up at once (budget of zero polls): the step records
 *                     MUON_ERR_DEVICE_TIMEOUT in the error word; each kernel
 *                     still waits, with the normal budget, for the copies it
 *                     has in flight before it returns.
 * These fault switches exist to test the callers' error paths; unset, they
 * cost one getenv per call.
 */
#ifndef MUON_H_
#define MUON_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MUON_API __attribute__((visibility("default")))
#else
#define MUON_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MUON_OK = 0,
  MUON_ERR_INVALID_ARG = -1,       /* null pointer, bad count, bad option   */
  MUON_ERR_UNSUPPORTED_SHAPE = -2, /* ndim not in {2,3}, a zero dimension    */
  MUON_ERR_DTYPE = -3,             /* dtype not MUON_BF16 / MUON_F32         */
  MUON_ERR_ALIGNMENT = -4,         /* workspace not 256-byte aligned         */
  MUON_ERR_CUDA = -5,              /* a CUDA runtime call failed             */
  MUON_ERR_DEVICE_TIMEOUT = -6,    /* a bounded device wait gave up          */
  MUON_ERR_WORKSPACE = -7,         /* workspace smaller than the plan needs  */
  MUON_ERR_NOMEM = -8              /* host memory allocation failed          */
} muon_status;

/* element types of parameters and gradients (momentum is always fp32) */
enum { MUON_BF16 = 0, MUON_F32 = 1 };

/* arithmetic of the Newton-Schulz products */
enum {
  /* 16-bit tensor-core operands, fp32 accumulation.  Dense groups iterate
   * in fp16: the iterates are normalised (spectral norm <= 1.21), so fp16
   * cannot overflow and carries three more mantissa bits than bf16.  The
   * fused kernel of skinny groups keeps V in bf16 and runs the m x m
   * recursion in fp32; its two products take bf16 operands. */
  MUON_MODE_TC16 = 0,
  /* fp32 operands and accumulation throughout (accuracy mode) */
  MUON_MODE_FP32 = 1
};

/* which kernel family a group runs on (reported by muon_plan_group) */
enum { MUON_KERNEL_SKINNY = 0, MUON_KERNEL_DENSE = 1 };

/* One parameter: [M, N] (ndim 2) or [E, M, N] (ndim 3), row-major,
 * contiguous.  dims[k] for k >= ndim is ignored. */
typedef struct {
  int ndim;
  int64_t dims[3];
  int dtype; /* MUON_BF16 or MUON_F32 */
} muon_shape;

typedef struct {
  int mode;             /* MUON_MODE_TC16 (default) or MUON_MODE_FP32        */
  float eps;            /* normalisation eps, default 1e-7                   */
  size_t workspace_cap; /* bytes; 0 = no cap.  Dense groups are processed in
                           chunks of slices that fit the cap; chunking never
                           changes results (slices are independent).        */
  int skinny_max_m;     /* groups with min(M,N) <= this run on the fused
                           skinny kernel when they fit on chip (default 64,
                           0 or negative disables the skinny kernel)        */
  int scale_mode;       /* update scale s of a [M, N] slice (the RFC does
                           not fix it): MUON_SCALE_SQRT_RATIO (default) or
                           MUON_SCALE_RMS_MATCH                             */
} muon_options;

/* update scale s in W' = W (1 - lr wd) - lr s O, rounded once to float */
enum {
  MUON_SCALE_SQRT_RATIO = 0, /* s = sqrt(max(1, M/N))                          */
  MUON_SCALE_RMS_MATCH = 1   /* s = 0.2 sqrt(max(M, N)): an update whose RMS is
                                about 0.2, like a typical AdamW step          */
};

typedef struct muon_plan_s muon_plan_t;

typedef struct {
  int64_t M, N;   /* slice dims as stored                                 */
  int64_t m, n;   /* working dims: m = min(M,N), n = max(M,N)             */
  int dtype;
  int count;      /* slices in the group                                   */
  int tr;         /* 1 when M > N: the slice is worked on transposed       */
  float scale;    /* update scale s of the options' scale_mode (float)     */
  int kernel;     /* MUON_KERNEL_SKINNY or MUON_KERNEL_DENSE               */
  int cluster;    /* skinny: CTAs per slice (thread-block cluster size)    */
  int chunk;      /* dense: slices per chunk under the workspace cap       */
} muon_group_info;

/* Fill *opt with the defaults listed above. */
MUON_API void muon_options_default(muon_options* opt);

/*
 * Build a plan (host only; no device call).  RFC section 3: slices are
 * grouped by key (M, N, dtype) in order of first appearance while walking
 * parameters in call order and slices e = 0..E-1 within each; a slice's
 * index in its group is its order of encounter.  shapes: n entries, host.
 * opt may be null (defaults).  On success *out receives a plan to be freed
 * with muon_plan_destroy.
 */
MUON_API muon_status muon_plan(const muon_shape* shapes, int n, const muon_options* opt,
                      muon_plan_t** out);

/* Device workspace bytes muon_step needs for this plan (>= 256). */
MUON_API muon_status muon_plan_workspace_bytes(const muon_plan_t* plan, size_t* out);
MUON_API muon_status muon_plan_num_groups(const muon_plan_t* plan, int* out);
MUON_API muon_status muon_plan_num_slices(const muon_plan_t* plan, int* out);
MUON_API muon_status muon_plan_group(const muon_plan_t* plan, int g, muon_group_info* out);
/* group id and index within the group of slice `slice` of parameter `param` */
MUON_API muon_status muon_plan_slice(const muon_plan_t* plan, int param, int slice,
                            int* group, int* index);

/*
 * One Muon step for every parameter of the plan, enqueued on `stream`
 * (a cudaStream_t; null = legacy default stream).
 *   params[p]   device, dtype of shape p, updated in place (RNE rounding)
 *   grads[p]    device, same dtype and shape, read only
 *   momentum[p] device, fp32, same shape, updated in place
 *   coeffs      host, 3 floats (a, b, c); null = (3.4445, -4.7750, 2.0315)
 *   ns_steps    T >= 0
 *   workspace   device, 256-byte aligned, >= muon_plan_workspace_bytes.
 *               Any content is valid on entry.  Passing the same workspace
 *               to the next step of the same plan keeps, per dense slice, the
 *               power of two that scales its first iterate; when it still
 *               fits, the step skips one pass over that slice.  The results
 *               do not depend on it.
 * Parameter, gradient and momentum buffers must not overlap one another.
 */
MUON_API muon_status muon_step(const muon_plan_t* plan, void* const* params,
                      const void* const* grads, float* const* momentum,
                      float lr, float beta, float wd, int nesterov,
                      int ns_steps, const float* coeffs, void* workspace,
                      size_t ws_bytes, void* stream);

/*
 * muon_step that also writes the orthogonalised momentum O (fp32, the
 * parameter's own shape and layout) of every slice into ortho[p], a device
 * buffer per parameter.  Used to check O itself against a reference.
 */
MUON_API muon_status muon_step_ortho(const muon_plan_t* plan, void* const* params,
                            const void* const* grads, float* const* momentum,
                            float lr, float beta, float wd, int nesterov,
                            int ns_steps, const float* coeffs, void* workspace,
                            size_t ws_bytes, void* stream, float* const* ortho);

/*
 * muon_step on loss-scaled gradients (mixed-precision training with a loss
 * scaler; the Paddle Muon sharding PR's review of its AMP GradScaler path
 * shows the Muon step running behind such a scaler).
 *   grads hold S * G for a loss scale S; the step uses G = grads * inv_scale
 *   (the multiply is fused into the momentum update, no extra pass).
 *   found_inf: device int.  Before any state changes, every gradient value of
 *   every parameter is checked; *found_inf is set to 1 when one is inf or NaN,
 *   and then no parameter and no momentum is modified (the step is skipped),
 *   else *found_inf is set to 0 and the step runs.  The check reads every
 *   gradient once more (2 bytes per bf16 element).
 * inv_scale must be finite.  Other arguments are those of muon_step.
 */
MUON_API muon_status muon_step_amp(const muon_plan_t* plan, void* const* params,
                                   const void* const* grads, float* const* momentum,
                                   float lr, float beta, float wd, int nesterov,
                                   int ns_steps, const float* coeffs, float inv_scale,
                                   int* found_inf, void* workspace, size_t ws_bytes,
                                   void* stream);

/*
 * AdamW for the parameters Muon does not orthogonalise (1-D biases and norm
 * scales, or any tensor the caller keeps off the Muon path; the Paddle Muon
 * sharding PR keeps separate 2-D and 1-D gradient buffers because the two
 * kinds take different update rules).  Standard AdamW, bias-corrected, with
 * decoupled weight decay, step t >= 1:
 *   m' = b1*m + (1-b1)*g;  v' = b2*v + (1-b2)*g^2
 *   W' = W*(1 - lr*wd) - lr * (m'/(1-b1^t)) / (sqrt(v'/(1-b2^t)) + eps)
 *   n tensors, each contiguous with numel[i] elements (any shape): params[i]
 *   and grads[i] of `dtype`, exp_avg[i] and exp_avg_sq[i] fp32 (updated in
 *   place).  All device pointers; one launch per 256 tensors.
 * Returns MUON_ERR_INVALID_ARG for null pointers, t < 1, betas outside [0,1),
 * negative eps or non-finite hyper-parameters.
 */
MUON_API muon_status muon_adamw_step(int n, void* const* params, const void* const* grads,
                                     float* const* exp_avg, float* const* exp_avg_sq,
                                     const int64_t* numel, int dtype, float lr, float beta1,
                                     float beta2, float eps, float wd, int step, void* stream);

/*
 * Read the device error word of a workspace after synchronising `stream`.
 * *code receives MUON_OK or the first device-side error recorded
 * (MUON_ERR_DEVICE_TIMEOUT); when clear != 0 the word is reset to zero.
 */
MUON_API muon_status muon_workspace_error(const void* workspace, void* stream, int clear,
                                 int* code);

/*
 * muon_step without a workspace argument, for callers that cannot allocate
 * device memory: a host runtime that hands nearly all of the GPU's memory to
 * its own pooled allocator at start-up, leaving none for a library's
 * cudaMalloc, or a latency-bound caller that cannot afford a cudaMalloc,
 * which may block and synchronise the device.  The RFC has no counterpart of
 * this call.
 *
 * The scratch is one static device array of MUON_STATIC_WORKSPACE_BYTES,
 * held by every GPU that loads the library until the process exits; no call
 * allocates or frees anything.  Plans whose muon_plan_workspace_bytes exceed
 * that size are rejected with MUON_ERR_WORKSPACE before any device work.
 * The first call on each device, with that device current, looks up the
 * array's device address and caches it; make that first call before any
 * stream capture.  The cache assumes the device is not reset
 * (cudaDeviceReset) while the library is loaded.  `stream` must belong to the
 * current device (else MUON_ERR_INVALID_ARG).  Every call shares the array
 * and finds the previous call's contents there: the device error word is
 * cleared at each call, everything else is written before it is read.  Calls
 * whose work overlaps on the GPU (streams with no ordering between them) race
 * on the array.  A device-side wait that gave up during the step is reported
 * by muon_static_error, not by the return code.  Other arguments are those of
 * muon_step.
 */
#define MUON_STATIC_WORKSPACE_BYTES (32u << 20)
MUON_API muon_status muon_step_static(const muon_plan_t* plan, void* const* params,
                                      const void* const* grads, float* const* momentum,
                                      float lr, float beta, float wd, int nesterov,
                                      int ns_steps, const float* coeffs, void* stream);

/*
 * The device error word that the last muon_step_static on the current device
 * left in the static array, read after synchronising `stream` (which must
 * belong to the current device): *code receives MUON_OK or
 * MUON_ERR_DEVICE_TIMEOUT; when clear != 0 the word is reset to zero.  Call
 * it before the next muon_step_static, which clears the word.  Allocates
 * nothing.  The RFC has no counterpart of this call.
 */
MUON_API muon_status muon_static_error(void* stream, int clear, int* code);

/* kernel classes of muon_step_timed */
enum {
  MUON_KC_SKINNY = 0,  /* fused on-chip kernel of the skinny groups              */
  MUON_KC_FRONT = 1,   /* dense path: momentum, V, partial sums of V^2           */
  MUON_KC_NORM = 2,    /* dense path: 1/(||V|| + eps) and the 16-bit X0          */
  MUON_KC_GEMM = 3,    /* dense path: the tcgen05 (or fp32) Newton-Schulz products */
  MUON_KC_UPDATE = 4,  /* dense path: separate update kernel (O requested)       */
  MUON_KC_CHECK = 5,   /* loss-scaled step: non-finite check of the gradients    */
  MUON_KC_COUNT = 6
};
typedef struct {
  float ms[MUON_KC_COUNT];   /* device time summed over the launches of a class  */
  int launches[MUON_KC_COUNT];
} muon_kernel_times;

/*
 * muon_step with a CUDA event recorded on `stream` before every kernel
 * launch and after the last one; synchronises `stream` and writes the device
 * time of each kernel class into *times (host).  An event between two
 * launches keeps a kernel from overlapping its predecessor's tail, so the
 * classes can sum to slightly more than a muon_step of the same plan takes.
 * For measurement: it creates and destroys its events (host-side driver
 * objects, no device memory).  Other arguments are those of muon_step.
 */
MUON_API muon_status muon_step_timed(const muon_plan_t* plan, void* const* params,
                                     const void* const* grads, float* const* momentum,
                                     float lr, float beta, float wd, int nesterov, int ns_steps,
                                     const float* coeffs, void* workspace, size_t ws_bytes,
                                     void* stream, muon_kernel_times* times);

/*
 * muon_step on parameters, gradients and momenta held in HOST memory (an
 * optimizer whose state lives in host memory; on a Grace-Blackwell node the
 * GPU reaches it over NVLink-C2C).  `staging` is cut into
 * nbuf = staging_bytes / unit_bytes buffers (2 to 16) and the plan's slices
 * into units of whole slices that fit one; each unit's parameters, gradients
 * and momenta are copied to the device, stepped by the kernels of muon_step,
 * and its parameters and momenta copied back, the copies of one unit
 * overlapping the kernels of its neighbours (two copy streams of the call's
 * own).  The kernels do not wait as long as a unit's copies in and out take
 * at most about nbuf - 1 times as long as its kernels.
 *   params, grads, momentum  host pointers (page-locked memory gives full
 *                            copy bandwidth, and muon_host_alloc's keeps it
 *                            when the state is cold; pageable memory works,
 *                            slower), shapes and dtypes as for muon_step
 *   workspace, ws_bytes      device, as for muon_step
 *   staging, staging_bytes   device, 256-byte aligned
 *   unit_bytes               staging bytes of one unit, at least
 *                            muon_plan_host_unit_bytes; larger units mean
 *                            fewer launches and a longer pipeline fill and
 *                            drain
 * Asynchronous: the work is ordered before any later work on `stream`;
 * synchronise `stream` before reading the host buffers.  Returns
 * MUON_ERR_WORKSPACE when one slice does not fit unit_bytes or the staging
 * holds fewer than two units.  Other arguments are those of muon_step.  The
 * RFC has no counterpart of this call.
 */
MUON_API muon_status muon_step_host(const muon_plan_t* plan, void* const* params,
                                    const void* const* grads, float* const* momentum, float lr,
                                    float beta, float wd, int nesterov, int ns_steps,
                                    const float* coeffs, void* workspace, size_t ws_bytes,
                                    void* staging, size_t staging_bytes, size_t unit_bytes,
                                    void* stream);
/* smallest unit_bytes of muon_step_host: the largest slice's parameter,
 * gradient and momentum, each 256-byte aligned (host only, no device call) */
MUON_API muon_status muon_plan_host_unit_bytes(const muon_plan_t* plan, size_t* out);

/*
 * Page-locked host memory for the state muon_step_host streams: `bytes`
 * rounded up to the kernel's transparent-huge-page size (the PMD size, read
 * from sysfs; 2 MiB if it cannot be read), mapped at an address aligned to
 * it, advised for huge pages, faulted in and registered with the CUDA driver
 * (portable).  Huge pages keep the device's reads of state it has not touched
 * for a while at full speed; with the base pages of the ordinary allocators,
 * such cold reads ran at a fraction of the link's bandwidth on some
 * allocations.  Where the kernel has no transparent huge pages the memory is
 * still page-locked, on base pages.  *out (host) receives the address (NULL
 * on failure); the memory reads as zeros.  Returns MUON_ERR_INVALID_ARG for
 * bytes == 0 or out == NULL, MUON_ERR_NOMEM when the mapping fails (or under
 * MUON_FAULT=alloc), MUON_ERR_CUDA when the registration fails (no device,
 * or the driver refuses); nothing is held then.  Ownership: the caller's,
 * until muon_host_free.
 */
MUON_API muon_status muon_host_alloc(size_t bytes, void** out);
/* Unregisters and unmaps memory from muon_host_alloc.  NULL is a no-op;
 * MUON_ERR_INVALID_ARG for an address muon_host_alloc did not return (or
 * already freed).  No device work may still use the memory. */
MUON_API muon_status muon_host_free(void* p);

/* Kernel launches muon_step makes for this plan and ns_steps, for a step
 * without O outputs (for accounting; no device call). */
MUON_API muon_status muon_plan_launches(const muon_plan_t* plan, int ns_steps, int* out);

/*
 * Assignment of the plan's slices to `world` replicas that all hold every
 * parameter (HyperParallel FSDP Muon RFC, section 4, HSDP grouped
 * computation: each replica group orthogonalises only the parameters that a
 * greedy algorithm assigns to it for an even compute load, then the updated
 * parameters are broadcast; section 2: the E slices of an [E, M, N] tensor
 * are independent, so the unit of assignment is a slice).  Host only, no
 * device call; the result depends only on the plan's shapes and the
 * arguments, so every replica computes the same assignment without
 * communicating.
 *
 * Load of a slice (seconds on the roofline of one GPU):
 *   max(T (4 m^2 n + 2 m^3) / flops_per_s,  m n (3 es + 8) / bytes_per_s)
 * with m = min(M, N), n = max(M, N), T = ns_steps, es = 2 (bf16) or 4 (fp32):
 * standard Newton-Schulz flop count, and the optimizer state touched once
 * (gradient read, parameter read and written, fp32 momentum read and
 * written).  Greedy longest first: slices in decreasing load (equal loads:
 * lower global slice id first), each to the replica with the least summed
 * load so far (equal sums: lower rank).
 *   owner      host, muon_plan_num_slices ints, written: owner[s] is the rank
 *              of global slice s (parameters in plan order, slices e = 0..E-1
 *              of each)
 *   rank_load  host, `world` doubles, written, or null: summed load per rank
 * Errors: MUON_ERR_INVALID_ARG for a null plan or owner, world < 1,
 * ns_steps < 0, or a rate that is not finite and positive.
 */
MUON_API muon_status muon_plan_partition(const muon_plan_t* plan, int world, int ns_steps,
                                         double flops_per_s, double bytes_per_s, int* owner,
                                         double* rank_load);

/*
 * Operators of a training step that stand between its matrix products and
 * feed the optimizer: layer norm (alone, or behind dropout and the residual
 * add), dropout, and the expert router with its balance loss, each with its
 * gradient.  All are asynchronous on `stream`, allocate nothing, keep nothing
 * between calls and validate their arguments before any launch.  Activations
 * and logits are MUON_BF16 or MUON_F32; rows are `ld` elements apart (any
 * ld >= 0 for inputs; every output is dense).  Sums, means and softmax
 * statistics are held in fp32.  Results do not depend on scheduling: no
 * floating-point atomics.  Outputs must not overlap inputs or one another
 * unless said otherwise.  MUON_FAULT=launch applies (MUON_ERR_CUDA after
 * validation); pointers that are not aligned to their element type give
 * MUON_ERR_ALIGNMENT.
 *
 * Random bits of dropout: Philox4x32-10 (J. Salmon, M. Moraes, R. Dror, D.
 * Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011) with key =
 * seed and counter = offset + i / 8 for element i in row-major order; the
 * eight 16-bit halves of a block's four words, low half first, serve elements
 * 8 (i / 8) .. + 7.  With t = floor(65536 p + 1/2), element i is kept when its
 * half is >= t and is then multiplied by 65536 / (65536 - t), the exact
 * inverse of the probability used; a dropped element is an exact 0 whatever
 * it held.  The flags depend on (seed, offset, i) alone, so the gradient
 * recomputes them and no mask is stored.  A call uses ceil(n / 8) counters: the
 * next call with the same seed takes an offset at least that much higher.  A
 * captured graph replays the seed and offset it was captured with.
 */

/*
 * Layer norm of each row, optionally behind dropout and a residual add:
 *   s = residual + dropout(x);  y = (s - mean) * rstd * weight + bias,
 *   mean = mean(s), rstd = 1 / sqrt(mean((s - mean)^2) + eps)
 * over `cols`.  Statistics and y use s in fp32; `sum` receives s rounded.
 *   rows >= 0, cols in [1, 2^30]
 *   wdtype       type of weight and bias
 *   residual     null: s = dropout(x)
 *   weight, bias [cols], each may be null (1, 0)
 *   p            dropout probability in [0, 1]; 0: no random bits are drawn
 *   sum          [rows, cols] of dtype, or null (not needed)
 *   y            [rows, cols] of dtype
 *   mean, rstd   [rows] fp32, each may be null
 */
MUON_API muon_status muon_layer_norm(int64_t rows, int64_t cols, int dtype, int wdtype,
                                     const void* x, int64_t ldx, const void* residual,
                                     int64_t ldr, const void* weight, const void* bias, float eps,
                                     float p, uint64_t seed, uint64_t offset, void* sum, void* y,
                                     float* mean, float* rstd, void* stream);

/*
 * Gradient of muon_layer_norm.  With g = dy * weight and h = (sum - mean) *
 * rstd:
 *   d = rstd * (g - mean(g) - h * mean(g * h)) + dsum
 *   dresidual = d;  dx = dropout(d), with the forward pass's p, seed, offset
 *   dweight = sum over rows of dy * h;  dbias = sum over rows of dy
 *   sum          the forward pass's sum (its x when it had neither residual
 *                nor dropout), mean and rstd its statistics
 *   dsum         gradient that reaches s past the norm, or null (0)
 *   dx, dresidual, dweight, dbias   each may be null (not needed)
 *   workspace    device, 256-byte aligned, >= muon_layer_norm_workspace_bytes
 *                (any content); unused, and may be null, when neither dweight
 *                nor dbias is asked for
 */
MUON_API muon_status muon_layer_norm_backward(
    int64_t rows, int64_t cols, int dtype, int wdtype, const void* dy, int64_t lddy,
    const void* sum, int64_t ldsum, const float* mean, const float* rstd, const void* weight,
    const void* dsum, int64_t ldds, float p, uint64_t seed, uint64_t offset, void* dx,
    void* dresidual, void* dweight, void* dbias, void* workspace, size_t ws_bytes, void* stream);
MUON_API muon_status muon_layer_norm_workspace_bytes(int64_t rows, int64_t cols, size_t* out);

/*
 * y = residual + dropout(x) over 0 <= n <= 2^40 dense elements (residual null: 0).
 * The gradient of x is the same call on dy without a residual.  y may be x or
 * residual itself.
 */
MUON_API muon_status muon_dropout(int64_t n, int dtype, const void* x, const void* residual,
                                  float p, uint64_t seed, uint64_t offset, void* y, void* stream);

/*
 * Expert router: choice of k experts per token, their combine weights, the
 * per-expert counts and the balance loss.
 *   A token is routed when its mask is nonzero (or there is no mask) and some
 *   logit is above -inf.  p = softmax of its logits; its picks are the k
 *   largest logits, ties to the lowest index; an expert at -inf is never
 *   picked.  A missing pick (fewer than k experts above -inf, or a token that
 *   is not routed) has index -1 and weight 0.  weight = softmax over the picks
 *   (normalize != 0) or p at the pick.
 *   n = routed tokens, P_e = sum of p_e / n, c_e = picks of e:
 *   loss = experts * sum over e of c_e / (k n) * P_e   (1 when balanced; 0
 *   when n = 0)
 * What the logits of a masked token hold has no effect.  A NaN ranks above
 * every number; a routed token with a NaN or +inf has NaN weights, and so have
 * mean_prob and the loss.
 *   tokens >= 0 with tokens * k < 2^31, experts in [1, 1024], k in [1,
 *   min(experts, 32)]
 *   token_mask  [tokens] bytes, or null
 *   weights     [tokens, k] fp32;  index [tokens, k]
 *   counts      [experts + 1]: c_e, then n
 *   mean_prob   [experts] fp32: P_e;  loss one fp32
 *   workspace   device, 256-byte aligned, >= muon_route_workspace_bytes (any
 *               content)
 */
MUON_API muon_status muon_route(int64_t tokens, int experts, int k, int dtype, const void* logits,
                                int64_t ld, const uint8_t* token_mask, int normalize,
                                float* weights, int32_t* index, int32_t* counts, float* mean_prob,
                                float* loss, void* workspace, size_t ws_bytes, void* stream);
MUON_API muon_status muon_route_workspace_bytes(int64_t tokens, int experts, size_t* out);

/*
 * Gradient of muon_route's weights and loss with respect to the logits (the
 * counts are constants of the loss).
 *   index, counts   the forward pass's
 *   dweights        [tokens, k] fp32, or null (0)
 *   dloss           one fp32 on the device, or null (0)
 *   dlogits         [tokens, experts] of dtype; a token that is not routed gets
 *                   zeros
 * Other arguments are those of muon_route.  An index outside [0, experts) is
 * a missing pick.
 */
MUON_API muon_status muon_route_backward(int64_t tokens, int experts, int k, int dtype,
                                         const void* logits, int64_t ld, const uint8_t* token_mask,
                                         int normalize, const int32_t* index,
                                         const int32_t* counts, const float* dweights,
                                         const float* dloss, void* dlogits, void* stream);

/*
 * Operators over sequences, with the conventions above: a gated linear
 * recurrence, the norms of query and key heads with the rotation of positions,
 * log probabilities of given tokens, and a clipped policy loss on them, each
 * with its gradient.  Flags (starts, token_mask) are bytes: nonzero is true.
 * A call of no elements touches nothing but what is said to be written.
 */

/*
 * Gated linear recurrence over `length` tokens of each of `batch` sequences,
 * one recurrence a channel, with a = sigmoid(gate):
 *   p = 0 at a token that starts over, else the state before it
 *   h = a p + (1 - a) x   (mix != 0)   or   h = a p + x   (mix == 0)
 * h is the state behind the token.  A masked token changes nothing: its h is
 * the state before it, whatever its gate and x hold and whether it starts over.
 * The state is held in fp32; h is that rounded.  Gate, x and states are finite;
 * what a sequence's state is after a value that is not, up to the next start,
 * is not defined (other sequences and channels are not affected).
 *   0 <= batch, length < 2^31, dim in [1, 2^20], batch * ceil(dim / 64) < 2^27
 *   gate, x      [batch * length, dim] of dtype, rows ldg and ldx apart (any stride
 *                below 2^32); read in whole aligned 16 bytes, each of which holds
 *                an element of a row, so up to 14 bytes beside a row are read, too
 *   state        [batch, dim] fp32: the state before the first token; null: 0
 *   starts       [batch, length] bytes, or null: no token starts over
 *   token_mask   [batch, length] bytes: 0 for masked tokens; null: none
 *   h            [batch, length, dim] of dtype
 *   last         [batch, dim] fp32: the state behind the last token (`state` for
 *                no tokens), or null; may be `state` itself
 */
MUON_API muon_status muon_gated_scan(int64_t batch, int64_t length, int64_t dim, int dtype,
                                     const void* gate, int64_t ldg, const void* x, int64_t ldx,
                                     const float* state, const uint8_t* starts,
                                     const uint8_t* token_mask, int mix, void* h, float* last,
                                     void* stream);

/*
 * Gradient of muon_gated_scan.  With l the gradient of the state behind a
 * token (dh plus what reaches it through the next token, dlast for the last
 * one) and p as in the forward pass, from the rounded h:
 *   dx = (1 - a) l or l,   dgate = a (1 - a) l (p - x) or a (1 - a) l p
 *   dstate = what reaches the state before the first token
 * 0 for the gate and x of masked tokens.
 *   dh           [batch * length, dim] of dtype, rows lddh apart
 *   x            unused, and may be null, where mix == 0
 *   h            the forward pass's, rows ldh apart
 *   dlast        [batch, dim] fp32, or null (0)
 *   dgate, dx    [batch, length, dim] of dtype, each may be null (not needed)
 *   dstate       [batch, dim] fp32, or null; may be dlast itself
 * Other arguments are those of muon_gated_scan.
 */
MUON_API muon_status muon_gated_scan_backward(
    int64_t batch, int64_t length, int64_t dim, int dtype, const void* dh, int64_t lddh,
    const void* gate, int64_t ldg, const void* x, int64_t ldx, const void* h, int64_t ldh,
    const float* state, const float* dlast, const uint8_t* starts, const uint8_t* token_mask,
    int mix, void* dgate, void* dx, float* dstate, void* stream);

/*
 * RMS norm of each query and key head, and the rotation of its first `rotary`
 * elements by the angles of the token's position:
 *   n = x / sqrt(mean(x^2) + eps) * weight   over the dim elements of a head,
 *   in fp32: the squares' sum is below 2^128, and mean(x^2) + eps is at least 2^-126
 *   (y_i, y_j) = (n_i c - n_j s, n_j c + n_i s)   for pair m of rotary / 2, with
 *   c, s = cos[position, m], sin[position, m]; i, j = m, m + rotary / 2, or
 *   2 m, 2 m + 1 (neighbours != 0).  Elements from `rotary` on keep n.
 * A token whose position is outside of the table is no token: its heads are 0,
 * whatever they hold.
 *   0 <= tokens < 2^31, 0 <= heads <= 65536, dim in [1, 1024], rotary even, in
 *   [0, dim]
 *   wdtype         type of the weights
 *   q, k           [tokens, heads, dim] of dtype: tokens ldq and ldk apart,
 *                  heads q_step and k_step
 *   q_weight, k_weight   [dim], each may be null (1)
 *   cos, sin       [table, rotary / 2] fp32; unused where rotary == 0
 *   positions      [tokens], or null: token t has position t % period
 *   q_out, k_out   [tokens, heads, dim] of dtype
 */
MUON_API muon_status muon_norm_rotate_heads(
    int64_t tokens, int q_heads, int k_heads, int dim, int rotary, int dtype, int wdtype,
    const void* q, int64_t ldq, int64_t q_step, const void* k, int64_t ldk, int64_t k_step,
    const void* q_weight, const void* k_weight, float eps, const float* cos, const float* sin,
    int64_t table, const int64_t* positions, int64_t period, int neighbours, void* q_out,
    void* k_out, void* stream);

/*
 * Gradient of muon_norm_rotate_heads.  With g = dy rotated back, h = x * rstd:
 *   dx = rstd * (g * weight - h * mean(g * weight * h))
 *   dweight = sum over tokens and heads of g * h
 *   dq, dk         gradients of q_out and k_out, laid out as q and k are, with
 *                  strides of their own
 *   q_grad, k_grad [tokens, heads, dim] of dtype, each may be null (not needed)
 *   q_dweight, k_dweight [dim] of wdtype, each may be null
 *   workspace      device, 256-byte aligned, >= the bytes of
 *                  muon_norm_rotate_heads_workspace_bytes (any content); unused, and
 *                  may be null, where no weight gradient is asked for
 * Other arguments are those of muon_norm_rotate_heads.
 */
MUON_API muon_status muon_norm_rotate_heads_backward(
    int64_t tokens, int q_heads, int k_heads, int dim, int rotary, int dtype, int wdtype,
    const void* dq, int64_t lddq, int64_t dq_step, const void* dk, int64_t lddk, int64_t dk_step,
    const void* q, int64_t ldq, int64_t q_step, const void* k, int64_t ldk, int64_t k_step,
    const void* q_weight, const void* k_weight, float eps, const float* cos, const float* sin,
    int64_t table, const int64_t* positions, int64_t period, int neighbours, void* q_grad,
    void* k_grad, void* q_dweight, void* k_dweight, void* workspace, size_t ws_bytes,
    void* stream);
MUON_API muon_status muon_norm_rotate_heads_workspace_bytes(int64_t tokens, int q_heads,
                                                            int k_heads, int dim, size_t* out);

/*
 * Log probability of a given token under softmax(scale * logits), and the
 * logarithm of the softmax's sum:
 *   lse = log(sum over v of exp(scale * logits_v))
 *   log_probs = scale * logits_index - lse
 * A token whose index is outside of [0, vocab) is ignored: both are 0 whatever
 * its logits hold.  A logit of -inf has no share (scale > 0).  A row with a NaN, a
 * +inf or nothing above -inf has NaN in log_probs.
 *   0 <= tokens < 2^31, vocab in [1, 2^30], tokens * vocab <= 2^40, scale in
 *   (0, 2^127]
 *   logits       [tokens, vocab] of dtype, rows ld apart
 *   index        [tokens]
 *   log_probs, lse [tokens] fp32
 */
MUON_API muon_status muon_token_log_probs(int64_t tokens, int64_t vocab, int dtype,
                                          const void* logits, int64_t ld, const int64_t* index,
                                          float scale, float* log_probs, float* lse, void* stream);

/*
 * Gradient of muon_token_log_probs's log_probs:
 *   dlogits_v = scale * dlog_probs * ((v == index) - exp(min(scale * logits_v - lse, 0)))
 * (the minimum is the difference itself but for lse's rounding; it is 0 where scale *
 * logits_v and lse overflow below, so rows of finite logits have finite gradients).
 * An exponential under 2^-126 counts as 0.
 * A token that is ignored, or whose dlog_probs is 0, gets zeros, whatever its
 * logits hold.
 *   dlog_probs   [tokens] fp32
 *   dlogits      [tokens, vocab] of dtype; may be logits itself, where its rows are
 *                dense (ld == vocab)
 * Other arguments are those of muon_token_log_probs, lse its result.
 */
MUON_API muon_status muon_token_log_probs_backward(int64_t tokens, int64_t vocab, int dtype,
                                                   const float* dlog_probs, const void* logits,
                                                   int64_t ld, const int64_t* index,
                                                   const float* lse, float scale, void* dlogits,
                                                   void* stream);

/*
 * Clipped policy loss with a KL term, over `length` tokens of each of `batch`
 * sequences, with d = log_probs - old, A the advantage, r = exp(d) and
 * e = ref - log_probs:
 *   each = -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A) + kl_weight * k
 *   k = exp(e) - e - 1   (0 without ref)
 *   loss = sum of w each,  kl = sum of w k,
 *   clipped = sum of w over the tokens whose minimum is the clipped side, which
 *   is where d > log(1 + clip_high) and A >= 0, or d < log(1 - clip_low) and A < 0,
 *   decided on the exact difference
 *   w = 1 / tokens (all that count), or with by_sequence != 0
 *   w = 1 / (sequences that have a token * tokens of the sequence)
 * Masked tokens have no effect, whatever they hold, nor has ref where kl_weight is 0,
 * but on kl.  No token at all: all 0.
 *   0 <= batch, length < 2^31, batch * length < 2^40, 0 <= clip_low < 1,
 *   0 <= clip_high, both and kl_weight finite
 *   log_probs, old, ref  fp32 rows of `length`, ldl, ldo and ldr apart; ref may be
 *                null
 *   advantages   fp32 rows of `length`, lda apart, or one a sequence (lda < 0):
 *                [batch]
 *   token_mask   [batch, length] bytes, or null
 *   loss, kl, clipped    one fp32 each; the last two may be null
 *   weights      [batch] fp32: w of the sequence's tokens (0 where it has none)
 *   workspace    device, 256-byte aligned, >= muon_policy_loss_workspace_bytes
 *                (any content)
 */
MUON_API muon_status muon_policy_loss(int64_t batch, int64_t length, const float* log_probs,
                                      int64_t ldl, const float* old, int64_t ldo,
                                      const float* advantages, int64_t lda, const float* ref,
                                      int64_t ldr, const uint8_t* token_mask, double clip_low,
                                      double clip_high, float kl_weight, int by_sequence,
                                      float* loss, float* kl, float* clipped, float* weights,
                                      void* workspace, size_t ws_bytes, void* stream);
MUON_API muon_status muon_policy_loss_workspace_bytes(int64_t batch, int64_t length, size_t* out);

/*
 * Gradient of muon_policy_loss's loss with respect to log_probs (old, ref and
 * the advantages are constants):
 *   dlog_probs = dloss * w * ((clipped ? 0 : -r A) + kl_weight * (1 - exp(e)))
 * 0 at masked tokens.
 *   weights      the forward pass's
 *   dloss        one fp32 on the device, or null (1)
 *   dlog_probs   [batch, length] fp32; may be log_probs, old or ref itself, where its
 *                rows are dense
 * Other arguments are those of muon_policy_loss.
 */
MUON_API muon_status muon_policy_loss_backward(
    int64_t batch, int64_t length, const float* log_probs, int64_t ldl, const float* old,
    int64_t ldo, const float* advantages, int64_t lda, const float* ref, int64_t ldr,
    const uint8_t* token_mask, double clip_low, double clip_high, float kl_weight,
    const float* weights, const float* dloss, float* dlog_probs, void* stream);

MUON_API void muon_plan_destroy(muon_plan_t* plan);
MUON_API const char* muon_status_string(muon_status s);

#ifdef __cplusplus
}
#endif

#endif /* MUON_H_ */
