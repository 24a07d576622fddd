/*
 * mpopt.h -- C ABI of the GB300 mixed-precision optimizer step (libmpopt.so).
 *
 * One optimizer step over fp32 master weights ("main_param"), fp32 reduced
 * gradients ("main_grad") and fp32 optimizer state, ending with the bf16 copy
 * of every master weight written back to the model:
 *
 *   - AdamW for every tensor routed to it (opt_adamw_step), as defined in
 *     "02 · Optimizer：算法与 infra" §2 (Adam, bias correction, eps outside the
 *     square root) and §3 (decoupled weight decay, AdamW Algorithm 2);
 *   - Muon for 2-D hidden matrices (opt_muon_step), as defined in the same
 *     page §1 (momentum and Nesterov as lerp), §5.2 (Newton-Schulz quintic),
 *     §5.4 (decoupled decay, Eq. 3; update scaled by 0.2*sqrt(max(A, B)),
 *     Eq. 4), and in "优化器：AdamW、Muon 与分布式优化器", Muon section;
 *   - both at once with the routing rule of §5.5 / §14.2 (opt_mixed_step):
 *     a tensor is a Muon tensor when it is 2-D and not an embedding or an
 *     output (LM head) parameter; every other tensor goes to AdamW;
 *   - the bf16 writeback of §9.2 ("参数写回": master -> model copy), done in
 *     the same kernels, round-to-nearest-even.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Every data pointer is a DEVICE pointer owned by the caller (for example
 *    torch.Tensor.data_ptr()).  The library allocates nothing and keeps no
 *    state between calls: optimizer state lives in the caller's buffers and
 *    scratch space in the caller's workspace.
 *  - Updates are in place.  Tensors are dense, row-major, element-contiguous.
 *    fp32 pointers must be 4-byte aligned and bf16 pointers 2-byte aligned;
 *    any other alignment is handled (unaligned heads and tails take a scalar
 *    path).  Tensors in one call must not overlap.
 *  - Work is enqueued on `stream` (a cudaStream_t; NULL is the legacy default
 *    stream) and runs asynchronously.  Argument errors are detected on the host
 *    before anything is enqueued and return a status; nothing runs then.
 *    A failed launch returns OPT_ERR_CUDA (the CUDA error text is available
 *    from opt_last_cuda_error()).
 *  - Device-side waits in the tensor-core kernels are bounded in time.  A wait
 *    that runs out records a code in the workspace header; opt_device_status()
 *    reads it.  Each step clears the header first.
 *  - Thread safety: calls that share a workspace must be serialised on one
 *    stream.
 */
#ifndef MPOPT_H
#define MPOPT_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MPOPT_API __attribute__((visibility("default")))
#else
#define MPOPT_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  OPT_OK = 0,
  OPT_ERR_INVALID_ARG = 1,   /* null pointer, bad size/shape/hyper-parameter  */
  OPT_ERR_UNSUPPORTED = 2,   /* a case this library does not implement        */
  OPT_ERR_MISALIGNED = 3,    /* fp32 pointer not 4-byte / bf16 not 2-byte aligned */
  OPT_ERR_WORKSPACE = 4,     /* workspace null, too small or not 256-B aligned */
  OPT_ERR_CUDA = 5,          /* a CUDA runtime/driver call or launch failed    */
  OPT_ERR_DEVICE_TIMEOUT = 6 /* a bounded device-side wait ran out (device status) */
} opt_status;

/* Routing of one tensor (opt_tensor.kind). */
enum {
  OPT_KIND_AUTO = 0,   /* opt_mixed_step decides: Muon iff ndim == 2 and not
                          flagged OPT_FLAG_EMBEDDING_OR_OUTPUT                  */
  OPT_KIND_ADAMW = 1,
  OPT_KIND_MUON = 2
};

/* opt_tensor.flags */
enum { OPT_FLAG_EMBEDDING_OR_OUTPUT = 1 };

/* OR into opt_workspace_size's `routing` to size a workspace for
   opt_mixed_step_clipped (adds one float per 16K gradient elements). */
enum { OPT_WORKSPACE_CLIP = 0x10 };
/* OR into opt_workspace_size's `routing` to size the Newton-Schulz buffers of
   every shape for grouped iterations (opt_muon_hp.flags OPT_MUON_NS_GROUPED);
   without it only the shapes grouped by default get their two extra buffers. */
enum { OPT_WORKSPACE_GROUPED = 0x20 };

/*
 * AdamW hyper-parameters for one step ("02 · Optimizer：算法与 infra" §2, §3).
 *   lr            eta, the step size
 *   beta1, beta2  EMA factors of the first and second raw moments, in [0, 1)
 *   eps           added OUTSIDE the square root: mhat / (sqrt(vhat) + eps)
 *   weight_decay  lambda, decoupled: theta <- theta * (1 - lr*lambda) - lr*update
 *   step          t >= 1, the number of this step (bias corrections 1 - beta^t)
 * The per-step scalars 1-beta1, 1-beta2, 1-beta1^t, 1-beta2^t and 1-lr*lambda are
 * formed in double precision from these values and rounded once to float; each
 * element is then evaluated in fp32 in the order written above, every operation
 * rounded to nearest (no fused multiply-add).
 */
typedef struct {
  float lr;
  float beta1;
  float beta2;
  float eps;
  float weight_decay;
  int32_t reserved;
  int64_t step;
} opt_adamw_hp;

/*
 * Muon hyper-parameters ("02 · Optimizer：算法与 infra" §1, §5.2, §5.4, §14.1,
 * §14.6).
 *   lr            eta
 *   momentum      mu in [0, 1): m <- lerp(m, g, 1 - mu)
 *   weight_decay  lambda, decoupled, applied to W_{t-1}
 *   eps           Newton-Schulz normalisation X = G / (||G||_F + eps); 1e-7
 *   nesterov      nonzero: Newton-Schulz input lerp(g, m, mu); zero: m
 *   ns_steps      number of quintic iterations, 0..16 (5 on the pages)
 *   ns_a, ns_b, ns_c  quintic coefficients, (3.4445, -4.7750, 2.0315), used
 *                 for every iteration unless ns_schedule is given
 *   scale_coeff   free factor k of the update scale (0.2 on the pages)
 *   scale_mode    OPT_SCALE_SPECTRAL: k * sqrt(max(m, n)) (the default, §5.4
 *                 Eq. 4); OPT_SCALE_SHAPE: k * sqrt(max(1, m / n));
 *                 OPT_SCALE_UNIT_RMS: k * sqrt(m / n) (§14.6), where
 *                 m = rows (fan_out) and n = cols (fan_in) of the parameter
 *   flags         OPT_MUON_NO_ORTHOGONALIZE: plain momentum SGD,
 *                 W <- W (1 - lr lambda) - lr * k * gtilde (§1), no Newton-Schulz;
 *                 evaluation order of the iterations (at most one of):
 *                 OPT_MUON_NS_PER_ITERATION: every iteration as printed
 *                 (A = X X^T, C = a I + b A + c A A, X <- C X);
 *                 OPT_MUON_NS_GROUPED: up to three consecutive iterations
 *                 share one X X^T and one C X.  Every C_k is a polynomial in
 *                 the group's first Gram matrix, so A_{k+1} = C_k (A_k C_k)
 *                 and X_{k+g} = (C_{k+g-1} ... C_k) X_k hold exactly; only
 *                 the rounding differs.  Used for every shape whose workspace
 *                 group has room for two more fp16 [A][A] buffers per matrix.
 *                 Neither flag (the default): grouped for the shapes where it
 *                 saves tensor-core work (padded max side >= 2 x padded min
 *                 side, min side >= 1024, e.g. 4096 x 14336), per iteration
 *                 otherwise
 *   ns_schedule   optional HOST array of ns_steps triples (a, b, c), one per
 *                 iteration in order (a coefficient schedule); NULL: ns_a..c
 */
typedef struct {
  float lr;
  float momentum;
  float weight_decay;
  float eps;
  int32_t nesterov;
  int32_t ns_steps;
  float ns_a;
  float ns_b;
  float ns_c;
  float scale_coeff;
  int32_t scale_mode;
  int32_t flags;
  const float* ns_schedule;
} opt_muon_hp;

enum { OPT_SCALE_SPECTRAL = 0, OPT_SCALE_SHAPE = 1, OPT_SCALE_UNIT_RMS = 2 };
enum { OPT_MUON_NO_ORTHOGONALIZE = 1, OPT_MUON_NS_PER_ITERATION = 2, OPT_MUON_NS_GROUPED = 4 };

/*
 * One parameter tensor.
 *   main_param   fp32 [rows*cols]   master weights, updated in place
 *   main_grad    fp32 [rows*cols]   this step's gradient, read only
 *   exp_avg      fp32 [rows*cols]   AdamW first moment m / Muon momentum buffer
 *   exp_avg_sq   fp32 [rows*cols]   AdamW second moment v; ignored for Muon
 *   model_param  bf16 [rows*cols]   written with the rounded master; NULL means
 *                                   the model parameter is itself fp32 (it IS
 *                                   main_param) and nothing is written back
 *   rows, cols   the shape; a 1-D tensor of n elements is rows = 1, cols = n,
 *                ndim = 1.  Muon requires ndim == 2, rows >= 1, cols >= 1.
 *                rows*cols == 0 is allowed and does nothing.
 *   ndim         the parameter's dimensionality (used by OPT_KIND_AUTO)
 *   kind, flags  routing, see above
 *   scale_rows, scale_cols  Muon only: the shape whose (fan_out, fan_in) set
 *                the update scale; 0, 0 means this tensor's own shape.  A block
 *                of a split parameter (QKV split, "02 · Optimizer：算法与 infra"
 *                §5.5 / §14.4: Q, K and V rows orthogonalised separately) is
 *                passed as its own row-block view with the whole parameter's
 *                shape here.
 */
typedef struct {
  float* main_param;
  const float* main_grad;
  float* exp_avg;
  float* exp_avg_sq;
  uint16_t* model_param;
  int64_t rows;
  int64_t cols;
  int32_t ndim;
  int32_t kind;
  int32_t flags;
  int32_t reserved;
  int64_t scale_rows;
  int64_t scale_cols;
} opt_tensor;

/*
 * Bytes of device workspace that opt_mixed_step (and the other steps) need for
 * this tensor list: a 256-byte status header and the Newton-Schulz buffers of
 * the largest group of same-shape Muon matrices (the fp16 iterate twice, as a
 * ping-pong pair, the fp16 Gram matrix, the fp16 polynomial a I + b A + c A A,
 * norm partials; for the shapes that take grouped iterations by default, two
 * more fp16 [A][A] buffers).  Shapes are padded to multiples of 256.
 * AdamW needs no workspace: 0 for a list without Muon tensors.
 * `routing` selects how kinds are interpreted: OPT_KIND_AUTO as in
 * opt_mixed_step, OPT_KIND_ADAMW treats every tensor as AdamW, OPT_KIND_MUON
 * every tensor as Muon.  Returns 0 if the list is invalid.
 * A smaller workspace is accepted by the Muon path as long as one matrix of
 * each shape fits without the grouped-iteration buffers; matrices are then
 * processed in smaller groups, and without grouped iterations when not even
 * one matrix fits with their buffers.
 */
MPOPT_API size_t opt_workspace_size(const opt_tensor* tensors, int32_t n, int32_t routing);

/*
 * AdamW step over a list of n tensors (n >= 0): a multi-tensor kernel over
 * 16K-element chunks whose tensor table travels in the kernel's parameter
 * space, one launch per 400 tensors.  kind/flags are ignored.  exp_avg_sq
 * must be non-null.  No workspace is needed (workspace may be NULL).
 */
MPOPT_API opt_status opt_adamw_step(const opt_adamw_hp* hp, const opt_tensor* tensors, int32_t n,
                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * Muon step for one 2-D matrix t (t->ndim must be 2): momentum, Nesterov,
 * Newton-Schulz on the wide orientation (transposed when rows > cols),
 * W <- W (1 - lr*lambda) - lr * scale_coeff * sqrt(max(rows, cols)) * O, and
 * bf16 writeback.  exp_avg is the momentum buffer; exp_avg_sq is ignored.
 */
MPOPT_API opt_status opt_muon_step(const opt_muon_hp* hp, const opt_tensor* t,
                         void* workspace, size_t workspace_bytes, void* stream);

/*
 * The whole mixed step: routes each tensor (kind/flags), runs one AdamW
 * launch over all AdamW tensors, and Muon over all Muon matrices, batching
 * matrices of the same (min, max) shape into shared tensor-core launches.
 * hp_muon may be NULL when no tensor routes to Muon, hp_adamw when none
 * routes to AdamW.
 */
MPOPT_API opt_status opt_mixed_step(const opt_muon_hp* hp_muon, const opt_adamw_hp* hp_adamw,
                          const opt_tensor* tensors, int32_t n,
                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * opt_mixed_step with global gradient-norm clipping fused in front
 * ("02 · Optimizer：算法与 infra" §11.1; §11.4: one norm over the gradients of
 * both optimizer groups):
 *   total_norm = sqrt(sum over every tensor of ||main_grad||^2)
 *   clip_coeff = max_norm / (total_norm + 1e-6)
 *   every gradient is multiplied by clip_coeff when clip_coeff < 1.
 * The factor is computed on the device (fp32 sums of squares per 16K-element
 * chunk, added in double in a fixed order) and applied by the AdamW and Muon
 * kernels as they load each gradient; main_grad itself is not rewritten.
 * max_norm <= 0 disables clipping (no norm pass, outputs untouched).
 * total_norm_out and clip_scale_out are optional 4-byte-aligned DEVICE fp32
 * pointers receiving the norm and the factor applied.  Workspace:
 * opt_workspace_size(tensors, n, OPT_KIND_AUTO | OPT_WORKSPACE_CLIP).
 */
MPOPT_API opt_status opt_mixed_step_clipped(const opt_muon_hp* hp_muon, const opt_adamw_hp* hp_adamw, float max_norm,
                                            float* total_norm_out, float* clip_scale_out, const opt_tensor* tensors,
                                            int32_t n, void* workspace, size_t workspace_bytes, void* stream);

/*
 * main_param <- fp32(model_param) for every tensor that has a bf16 model copy
 * ("02 · Optimizer：算法与 infra" §9.2 reload_model_params: refresh the masters
 * after the model copy was changed from outside; "支持FP32优化器" §9.3-§9.4:
 * the plain-checkpoint and model-only restore branches).  Exact (bf16 widens
 * to fp32 without rounding).  fp32-native tensors (model_param NULL) are left
 * alone.  Only main_param, model_param and the shape are read; no workspace.
 * Note the fp32 tail the masters had is not recoverable this way: a resume
 * that must continue bit for bit restores main_param itself.
 */
MPOPT_API opt_status opt_reload_model_params(const opt_tensor* tensors, int32_t n, void* stream);

/*
 * Data-parallel sharding of one optimizer step over `world_size` ranks
 * ("02 · Optimizer：算法与 infra" §12.1-§12.2 and §14.3; "优化器：AdamW、Muon 与
 * 分布式优化器", distributed Muon, scheme ③).  Host-only: no device work, no
 * CUDA call; every rank computes the same plan from the same tensor list.
 *
 *   - AdamW tensors (the routing of opt_mixed_step, with `routing` as in
 *     opt_workspace_size) are laid end to end, in list order, in one index
 *     space of N elements, each starting at a multiple of `align_elems` (>= 1;
 *     the gaps belong to no tensor), which is cut into world_size contiguous
 *     ranges, ZeRO-1 style: rank r owns [rank_bounds[r], rank_bounds[r+1]).
 *     The cuts ignore tensor boundaries (a tensor may span ranks); every inner
 *     cut is a multiple of `align_elems`, so it falls at a multiple of
 *     `align_elems` of the tensor's own elements, and the ranges are as equal
 *     as that allows: rank_bounds[r] = min(N, round_up(r * N / world_size,
 *     align_elems)).
 *     Rank r steps only the elements it owns, with fp32 master, m and v of
 *     that size, and then every rank receives the bf16 values of the rest.
 *   - Muon tensors stay whole (Newton-Schulz needs the whole matrix): each has
 *     one owner rank, assigned by LPT bin-packing on its Newton-Schulz work
 *     2 (2 A^2 B + A^3) per iteration (largest first; each goes to the rank
 *     with the least work so far, the lowest rank on ties; equal sizes keep
 *     list order), so the plan is deterministic.
 *
 * Output, caller-owned host memory:
 *   entries[n]            per tensor: owner = the owning rank (Muon) or -1
 *                         (AdamW; and for empty tensors); flat_begin = the
 *                         tensor's first index in the AdamW index space
 *                         (AdamW) or -1 (Muon)
 *   rank_bounds[world_size + 1]   the AdamW ranges (rank_bounds[0] = 0,
 *                         rank_bounds[world_size] = N)
 *   rank_muon_work[world_size]    optional (NULL: not written): the
 *                         Newton-Schulz flops per iteration each rank owns
 * Only shapes, kinds and flags are read: the tensors' pointers may be null
 * (on a sharded rank the master and state of what it does not own need not
 * exist).  Errors: OPT_ERR_INVALID_ARG for world_size < 1, align_elems < 1,
 * null outputs, or a shape or kind opt_mixed_step would reject.
 */
typedef struct {
  int32_t owner;
  int32_t reserved;
  int64_t flat_begin;
} opt_shard_entry;

MPOPT_API opt_status opt_shard_plan(const opt_tensor* tensors, int32_t n, int32_t routing, int32_t world_size,
                                    int64_t align_elems, opt_shard_entry* entries, int64_t* rank_bounds,
                                    double* rank_muon_work);

/*
 * How opt_muon_step / opt_mixed_step evaluate the Newton-Schulz iterations of
 * one rows x cols matrix under `hp` (host only: nothing is launched, no GPU is
 * needed).  Writes the size of each group of consecutive iterations that
 * share one X X^T and one C X, in order (all 1: every iteration as written),
 * into group_sizes[0 .. *n_groups) and their count into *n_groups; the sizes
 * add up to hp->ns_steps.  The plan assumes a workspace from
 * opt_workspace_size (with OPT_WORKSPACE_GROUPED when hp->flags has
 * OPT_MUON_NS_GROUPED): a workspace without room for the grouped buffers
 * evaluates every iteration as written.
 * Grouping follows hp->flags (see opt_muon_hp), in groups of at most three,
 * and splits a group into single iterations when the product of its
 * polynomials could leave fp16's range: each iteration's largest |a + b l +
 * c l^2| over the squared singular values it can reach (from [0, 1] after the
 * normalisation, through the per-singular-value form of the iteration,
 * "02 · Optimizer：算法与 infra" §5.2) is multiplied over the group, and
 * groups above 4096 are split (the printed coefficients give about 42).
 * Errors: OPT_ERR_INVALID_ARG for a null pointer, an invalid hp, rows or cols
 * below 1, or capacity below hp->ns_steps.
 */
MPOPT_API opt_status opt_ns_plan(int64_t rows, int64_t cols, const opt_muon_hp* hp, int32_t* group_sizes,
                                 int32_t capacity, int32_t* n_groups);

/*
 * Copies `bytes` from page-locked host memory `src` (cudaHostAlloc, or
 * registered with cudaHostRegister) to device memory `dst` of the current
 * device, enqueued on `stream`, with a kernel whose threads load the host
 * buffer over the CPU-GPU link and store to device memory (32 CTAs, no
 * shared memory: it runs beside the optimizer's kernels on another stream
 * and leaves most SMs to them).  No counterpart on the pages: it serves callers whose gradients
 * arrive in host memory.  On GB300 hosts the copy engines' host-to-device
 * rate (cudaMemcpyAsync) from page-locked memory varies with the pages and
 * over time, down to 13-40 GB/s on some buffers of some hosts, while loads by
 * the SMs keep about 210 GB/s.
 *   dst, src  4-byte aligned (16-byte aligned for the vector path), not
 *             overlapping; bytes a multiple of 4.
 * Errors: OPT_ERR_INVALID_ARG for null pointers, a src that is not
 * page-locked host memory, or a dst that is not device memory of the current
 * device; OPT_ERR_MISALIGNED for the alignment rules; OPT_ERR_CUDA if the
 * launch fails.  bytes == 0 does nothing.
 */
MPOPT_API opt_status opt_copy_from_host(void* dst, const void* src, size_t bytes, void* stream);

/*
 * Newton-Schulz orthogonalisation alone ("02 · Optimizer：算法与 infra" §5.2):
 * O = NS_steps(G) for one fp32 rows x cols matrix G, same fp16 tensor-core
 * path as opt_muon_step.  G and O are device fp32 [rows*cols]; O may alias G.
 * Workspace: opt_workspace_size of a one-matrix Muon list of that shape.
 */
MPOPT_API opt_status opt_newton_schulz(const float* G, float* O, int64_t rows, int64_t cols,
                             int32_t ns_steps, float a, float b, float c, float eps,
                             void* workspace, size_t workspace_bytes, void* stream);

/*
 * opt_newton_schulz without a workspace, for callers that cannot allocate
 * device memory: code hosted by a runtime that owns every device allocation
 * and gives extensions no allocator, or a path whose memory budget is fixed in
 * advance.  No counterpart on the pages: this is an interface convenience, the
 * arithmetic is opt_newton_schulz's with every iteration evaluated as written
 * (as with OPT_MUON_NS_PER_ITERATION): the built-in scratch holds the buffers
 * of one iteration, not those of grouped iterations.
 *   - Scratch is a 20 MiB array of device memory built into the library (a
 *     static __device__ array).  Every GPU that loads the library holds it until
 *     the process exits.  This entry point calls no cudaMalloc, cudaFree or
 *     other allocating routine.
 *   - Size limit: min(rows, cols) <= 1024 and max(rows, cols) <= 4096; larger
 *     matrices return OPT_ERR_UNSUPPORTED (text in opt_last_cuda_error()).
 *   - The first call on each device looks up the array's device address there
 *     (cudaGetSymbolAddress with that device current), and so does the first
 *     call after the device's CUDA context was destroyed and created again
 *     (cudaDeviceReset): the library remembers the context's id with the
 *     address.  Make such a first call before any stream capture.
 *   - Every call on a device shares the one array, and the array keeps the last
 *     call's contents (the status word is cleared at the start of each call).
 *     Calls whose work overlaps on the GPU -- on different streams, or from
 *     different threads -- race on it: serialise them on one stream.
 *   - A device-side timeout is recorded in the array's header: read it with
 *     opt_noalloc_device_status() after the call.
 */
MPOPT_API opt_status opt_newton_schulz_noalloc(const float* G, float* O, int64_t rows, int64_t cols,
                                               int32_t ns_steps, float a, float b, float c, float eps,
                                               void* stream);

/*
 * Status of the last opt_newton_schulz_noalloc call on the current device:
 * synchronises `stream` and returns OPT_ERR_DEVICE_TIMEOUT if a kernel of
 * that call recorded a device-side timeout in the built-in array's header,
 * else OPT_OK (OPT_ERR_CUDA if the copy or the synchronisation fails).  Like
 * the call itself, no counterpart on the pages.
 */
MPOPT_API opt_status opt_noalloc_device_status(void* stream);

/*
 * Synchronises `stream` and reports whether a kernel of the last step on this
 * workspace recorded a device-side timeout (OPT_ERR_DEVICE_TIMEOUT) or not
 * (OPT_OK).  Returns OPT_ERR_CUDA if the synchronisation itself fails, and for
 * a workspace of opt_linear_* OPT_ERR_WORKSPACE if a call found that its header
 * had not been zero (see there).
 */
MPOPT_API opt_status opt_device_status(const void* workspace, void* stream);

/*
 * Self-test of the bounded device-side waits (for tests of the failure path).
 * Runs opt_newton_schulz on G (rows x cols; 5 iterations with the quintic
 * coefficients of "02 · Optimizer：算法与 infra" §5.2, eps 1e-7) with one TMA
 * stage of the first X X^T launch withheld: the even CTA of the first CTA pair
 * never signals it, so the MMA issuer's wait for that stage runs out after
 * about 2 s.  The kernel then records the timeout in the workspace header,
 * every role of the CTA pair leaves its loop (each of their waits is bounded
 * too), and the remaining launches run to completion on whatever the buffers
 * hold.  Nothing faults, and the CUDA context and the workspace stay usable:
 * opt_device_status() returns OPT_ERR_DEVICE_TIMEOUT, and the next call on
 * the same workspace clears the header and runs normally.  O receives
 * unspecified values.  Arguments, workspace size (opt_workspace_size of one
 * OPT_KIND_MUON tensor of this shape) and host-side errors are those of
 * opt_newton_schulz.
 */
MPOPT_API opt_status opt_selftest_wait_timeout(const float* G, float* O, int64_t rows, int64_t cols,
                                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * Feed-forward operators
 * ----------------------
 * The operators around the parameters: the bf16 model copies the step writes
 * are their weights, and the fp32 main_grad buffers the step reads are their
 * outputs.  A residual block is
 *
 *   h = x + residual;  y = rmsnorm(h) * gamma          opt_rmsnorm_forward
 *   u = act(y w1^T + b1)                                opt_linear_forward
 *   out = u w2^T + b2 + h                               opt_linear_forward
 *
 * and the gradients run through opt_linear_backward and opt_rmsnorm_backward
 * into main_grad.  Conventions beyond the shared ones:
 *
 *  - Matrices are row-major with elements of a row contiguous; `*_ld` is the
 *    distance between rows in elements (>= the row's length).  With one row
 *    the distance is not used.  Rows may be slices of wider rows.
 *  - Sums, norms and products are accumulated in fp32; an output is rounded
 *    once, to its own type, round-to-nearest-even.
 *  - 8-bit values are e4m3 with one fp32 scale per row, value = q * scale:
 *      scale = max(max_j |y_j|, 1e-30) / 448,   q_j = rne_e4m3(y_j * (1 / scale))
 *    so the largest magnitude of a row maps to 448, and a row of zeros has
 *    q = 0.  (y_j / scale in the second place of the product gives the same codes
 *    but where it lies within two fp32 roundings of the middle between two of
 *    them, which bf16 values meet: there either neighbour is the nearest.)  A NaN stays a NaN; a row that holds an infinity has scale = inf
 *    and stands for NaN throughout.
 *  - Zero rows (rows or m = 0) are allowed: nothing is read, and gradients of
 *    parameters are left as they are (accumulate) or set to zero.
 *  - The workspace of opt_linear_* and opt_rmsnorm_backward is 256-byte aligned
 *    device memory.  The first 256 bytes of a linear workspace must be zero
 *    before its first use (cudaMemset); every call leaves them zero unless a
 *    bounded device-side wait ran out.  opt_device_status() reports that, and
 *    the workspace must be zeroed again before its next use.  A header that was
 *    not zero costs a large product some of its tiles, whose outputs are then not
 *    written; nothing is accessed out of range, and opt_device_status() reports
 *    it too.
 */
enum { OPT_DTYPE_FP32 = 0, OPT_DTYPE_BF16 = 1, OPT_DTYPE_E4M3 = 2 };

/* Activations: u; max(u, 0) (a NaN stays one); u (1 + tanh(sqrt(2/pi) (u +
   0.044715 u^3))) / 2; u / (1 + exp(-u)).  The last two are 0 where the factor
   of u is below 2^-126 (silu: from u = -87 down, values under 1.1e-36). */
enum { OPT_ACT_NONE = 0, OPT_ACT_RELU = 1, OPT_ACT_GELU = 2, OPT_ACT_SILU = 3 };

/*
 * RMS norm with the residual's addition, one row (token) at a time, cols <= 49152:
 *   h = x + residual          (residual NULL: h = x)
 *   rstd = 1 / sqrt(mean_j h_j^2 + eps)
 *   y_j = h_j * rstd * gamma_j
 * y is formed from the unrounded h.  Outputs that are NULL are not written.  The
 * squares are summed in fp32, so the rms of a row is right from 1e-18 (below it
 * eps decides, or with eps = 0 nothing does) to 1.8e19 / sqrt(cols); the gradient
 * holds in the same range.
 */
typedef struct {
  const void* x;          /* [rows][cols], dtype                               */
  const void* residual;   /* [rows][cols], dtype, or NULL                      */
  const void* gamma;      /* [cols], gamma_dtype (FP32 or BF16)                */
  void* h;                /* [rows][cols], dtype; may be x or residual itself
                             (same pointer and row distance)                   */
  uint16_t* y;            /* [rows][cols] bf16                                 */
  uint8_t* q;             /* [rows][cols] e4m3 of y; needs q_scale             */
  float* q_scale;         /* [rows]; needs q                                   */
  float* rstd;            /* [rows]                                            */
  int64_t rows, cols;
  int64_t x_ld, residual_ld, h_ld, y_ld, q_ld;
  int32_t dtype;          /* FP32 or BF16                                      */
  int32_t gamma_dtype;
  float eps;              /* >= 0                                              */
  int32_t reserved;
} opt_rmsnorm_args;

MPOPT_API opt_status opt_rmsnorm_forward(const opt_rmsnorm_args* args, void* stream);

/*
 * Gradient of opt_rmsnorm_forward at h, with n_j = h_j rstd and g_j = dy_j gamma_j:
 *   dx_j = rstd (g_j - n_j mean_i(g_i n_i)) + dh_j     (x and residual both get dx)
 *   dgamma_j (+)= sum over rows of dy_j n_j            (fp32, in a fixed order)
 * cols <= 24576.  With dgamma the call needs a workspace of
 * opt_rmsnorm_workspace_size(rows, cols) bytes (its contents do not matter).
 */
typedef struct {
  const uint16_t* dy;     /* [rows][cols] bf16                                 */
  const void* h;          /* [rows][cols], dtype                               */
  const void* gamma;      /* [cols], gamma_dtype                               */
  const float* rstd;      /* [rows]                                            */
  const void* dh;         /* [rows][cols], dtype: gradient reaching h past the
                             norm, or NULL                                     */
  void* dx;               /* [rows][cols], dtype; may be dh itself, or NULL    */
  float* dgamma;          /* [cols] main_grad of gamma, or NULL                */
  int64_t rows, cols;
  int64_t dy_ld, h_ld, dh_ld, dx_ld;
  int32_t dtype;
  int32_t gamma_dtype;
  int32_t accumulate;     /* nonzero: dgamma += ...; zero: dgamma = ...        */
  int32_t reserved;
} opt_rmsnorm_grad_args;

MPOPT_API opt_status opt_rmsnorm_backward(const opt_rmsnorm_grad_args* args, void* workspace,
                                          size_t workspace_bytes, void* stream);
MPOPT_API size_t opt_rmsnorm_workspace_size(int64_t rows, int64_t cols);

/*
 * Rows in e4m3 with a scale each (see above): x [rows][cols] of dtype FP32 or
 * BF16, cols <= 49152.  For a weight [n][k] this is the operand that
 * opt_linear_forward reads in 8 bits.
 */
MPOPT_API opt_status opt_quantize_rows(const void* x, int64_t x_ld, int32_t dtype, int64_t rows, int64_t cols,
                                       uint8_t* q, int64_t q_ld, float* scale, void* stream);

/*
 * Linear layer with a fused epilogue, on the tensor cores:
 *   z = x w^T + bias;  y = act(z) + residual
 * Operands are both BF16, or both E4M3 with x_scale [m] and w_scale [n]
 * (products in 8 bits, fp32 sums, scaled in the epilogue).
 */
typedef struct {
  const void* x;            /* [m][k] dtype                                    */
  const void* w;            /* [n][k] dtype                                    */
  const float* x_scale;     /* [m], E4M3 only                                  */
  const float* w_scale;     /* [n], E4M3 only                                  */
  const void* bias;         /* [n] bias_dtype (FP32 or BF16), or NULL          */
  const uint16_t* residual; /* [m][n] bf16, or NULL                            */
  uint16_t* y;              /* [m][n] bf16; may be residual itself             */
  uint16_t* z;              /* [m][n] bf16 pre-activation for the gradient, or NULL */
  int64_t m, n, k;          /* m >= 0, n, k >= 1                               */
  int64_t x_ld, w_ld, residual_ld, y_ld, z_ld;
  int32_t dtype;            /* BF16 or E4M3                                    */
  int32_t bias_dtype;
  int32_t act;              /* OPT_ACT_*                                       */
  int32_t reserved;
} opt_linear_args;

MPOPT_API opt_status opt_linear_forward(const opt_linear_args* args, void* workspace, size_t workspace_bytes,
                                        void* stream);

/*
 * Gradients of z = x w^T + bias for a given dz (bf16):
 *   dx = (dz w) * act_prev'(z_prev)   bf16; with z_prev, x = act_prev(z_prev) is
 *        taken to be the previous layer's output and dx is that layer's dz
 *   dw (+)= dz^T x                    fp32 main_grad of w
 *   dbias (+)= column sums of dz      fp32 main_grad of the bias
 * Outputs that are NULL are not computed, and what only they need may be NULL.
 * Every sum has a fixed order: a call gives the same bits each time.  With
 * accumulate each element of dw is added once, in fp32, to what main_grad
 * holds (subnormal values, what it holds and the result, count as zeros).
 */
typedef struct {
  const uint16_t* dz;       /* [m][n] bf16                                     */
  const uint16_t* x;        /* [m][k] bf16 (for dw)                            */
  const uint16_t* w;        /* [n][k] bf16 (for dx)                            */
  const uint16_t* z_prev;   /* [m][k] bf16, or NULL                            */
  uint16_t* dx;             /* [m][k] bf16, or NULL                            */
  float* dw;                /* [n][k] fp32, dense, or NULL                     */
  float* dbias;             /* [n] fp32, or NULL                               */
  int64_t m, n, k;
  int64_t dz_ld, x_ld, w_ld, z_prev_ld, dx_ld;
  int32_t act_prev;         /* OPT_ACT_*; other than NONE, dx needs z_prev     */
  int32_t accumulate;       /* nonzero: dw, dbias += ...; zero: = ...          */
} opt_linear_grad_args;

MPOPT_API opt_status opt_linear_backward(const opt_linear_grad_args* args, void* workspace,
                                         size_t workspace_bytes, void* stream);

/*
 * Workspace bytes for opt_linear_forward and opt_linear_backward of these
 * sizes.  The tensor cores' operands are read in 16-byte pieces: an operand
 * whose base or row distance is not a multiple of 16 bytes is first copied
 * into the workspace.  flags 0: room for the operands whose dense layout
 * needs that; OPT_LINEAR_ANY_LAYOUT: room for all of them.
 *
 * With OPT_LINEAR_ANY_LAYOUT the workspace also serves every call whose m, n
 * and k are none larger; without it those of them whose operands need no copy.
 * A call that needs more is refused with OPT_ERR_WORKSPACE.  A layer that is
 * followed by one with n and k the other way round takes the larger of both sizes.
 */
enum { OPT_LINEAR_ANY_LAYOUT = 1 };
MPOPT_API size_t opt_linear_workspace_size(int64_t m, int64_t n, int64_t k, int32_t flags);

/*
 * Optional launch instrumentation (off by default).  After
 *   opt_profile_launches(events, info, capacity, &count)
 * every kernel this library launches from the calling thread is bracketed by
 * cudaEventRecord(events[2*i]) and cudaEventRecord(events[2*i+1]) on the
 * launch's stream, and info[i] describes it, for i = count, count+1, ...
 * while count < capacity (count is incremented by the library, also past
 * capacity, so the caller learns how many launches there were).  `events`
 * holds 2*capacity cudaEvent_t created by the caller; `info` and `count` are
 * host memory owned by the caller and must stay valid until
 * opt_profile_launches(NULL, NULL, 0, NULL) switches it off.
 */
typedef struct {
  int32_t kernel;   /* OPT_KERNEL_* */
  int32_t count;    /* matrices (Newton-Schulz, Muon stages) or tensors (AdamW) */
  int64_t a;        /* Newton-Schulz: A = min(rows, cols); AdamW: elements */
  int64_t b;        /* Newton-Schulz: B = max(rows, cols) */
} opt_launch_info;

enum {
  OPT_KERNEL_NS_GRAM = 0,      /* A = X X^T, fp16 tensor cores                   */
  OPT_KERNEL_NS_POLY = 1,      /* C = a I + b A + c A A, fp16 tensor cores       */
  OPT_KERNEL_NS_BX = 2,        /* X' = C X, fp16 tensor cores (last one updates W) */
  OPT_KERNEL_ADAMW = 3,
  OPT_KERNEL_MUON_PREP = 4,    /* momentum, Nesterov, norm partials (and, with
                                  Newton-Schulz, the fp16 iterate)              */
  OPT_KERNEL_MUON_NORM = 5,
  OPT_KERNEL_MUON_APPLY = 6,   /* ns_steps == 0 only                             */
  OPT_KERNEL_MUON_OPERANDS = 7, /* fix-up: normalised fp16 X0 rewritten for the
                                  matrices whose iterate left fp16's range       */
  OPT_KERNEL_GRAD_NORM = 8,     /* clipping: sums of squares of the gradients      */
  OPT_KERNEL_CLIP_FINALIZE = 9, /* clipping: total norm and factor                 */
  OPT_KERNEL_MUON_SAMPLE = 10,  /* per-matrix power-of-two scale of the iterate    */
  OPT_KERNEL_NS_SYM = 11,       /* grouped iterations: product of two commuting
                                   symmetric [A][A] matrices, fp16 tensor cores  */
  OPT_KERNEL_RMSNORM = 12,      /* feed-forward operators: a = rows (m), b = cols (n);
                                   count is 1                                    */
  OPT_KERNEL_RMSNORM_GRAD = 13,
  OPT_KERNEL_RMSNORM_DGAMMA = 14, /* joins the partial sums of dgamma            */
  OPT_KERNEL_QUANTIZE = 15,
  OPT_KERNEL_LINEAR = 16,       /* y                                             */
  OPT_KERNEL_LINEAR_DX = 17,
  OPT_KERNEL_LINEAR_DW = 18,
  OPT_KERNEL_LINEAR_DBIAS = 19,
  OPT_KERNEL_LINEAR_REPACK = 20, /* operands (count of them) copied to 16-byte
                                   aligned rows; a, b of the largest             */
  OPT_KERNEL_LINEAR_GRAD = 21   /* dx, dw and dbias of a short batch at once      */
};

MPOPT_API opt_status opt_profile_launches(void* const* events, opt_launch_info* info, int32_t capacity,
                                          int32_t* count);

/* Static text for a status code. */
MPOPT_API const char* opt_strerror(opt_status status);

/* Text of the last CUDA error seen by this thread's calls ("" if none). */
MPOPT_API const char* opt_last_cuda_error(void);

/* ABI version: (major << 16) | minor (2.0: Muon variants, scale shapes, clipping;
   2.1: feed-forward operators). */
MPOPT_API int32_t opt_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MPOPT_H */
