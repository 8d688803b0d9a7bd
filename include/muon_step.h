/*
 * muon_step.h -- C ABI of the MI355X (gfx950) Muon optimizer step over flat buffers.
 *
 * What is computed (page "Add initial Muon+M-FSDPv2 implementation",
 * Megatron-LM PR #6425, pseudocode block "Opt step", steps 1, 2, 4 and 6; and
 * class FsdpMuon on the page
 * "core.distributed.fsdp.src.megatron_fsdp.experimental.muon", methods
 * _compute_momentum_inputs, _orthogonalize_updates, _apply_local_updates):
 * for every 2-D matrix described by a muon_matrix_desc_t, with
 * G = gradient, M = momentum, W = weights, all rows x cols row-major,
 *
 *   M  <- beta*M + G                              (state update, step 1)
 *   U  <- G + beta*M   (Nesterov)   or   U <- M   (orthogonalization input, step 2)
 *   O  <- s * NS(U),  s = sqrt(max(1, rows/cols)) (orthogonalization, step 4)
 *   W  <- W*(1 - lr*wd) - lr*O                    (decoupled decay + update, step 6)
 *
 * NS is the quintic Newton-Schulz orthogonalization: X = U (or U^T when
 * rows > cols), X <- X / (||X||_F + 1e-7), then ns_steps times
 * A = X X^T, B = b A + c A A, X <- a X + B X with (a, b, c) =
 * (3.4445, -4.7750, 2.0315); the result is transposed back for tall matrices.
 * The pages name the orthogonalization without fixing its algorithm; the
 * quintic iteration is the one Muon is built on.
 *
 * Numerics.  The elementwise phases run in float32, one rounding per
 * operation, no fused multiply-add, in this order:
 *   M1 = fl(fl(beta*M) + G);  U = fl(fl(beta*M1) + G)  (U = M1 without Nesterov)
 *   f  = fl(1 - fl(lr*wd));   W1 = fl(W*f);  Wn = fl(W1 - fl(lr*O))
 * and bfloat16 weights are rounded once, to nearest even, on store.
 * The Frobenius norm is a deterministic float32 reduction.  Newton-Schulz
 * runs either on bfloat16 MFMA with float32 accumulation and float32
 * epilogues, X/A/B stored as bfloat16 (MUON_GEMM_BF16_MFMA), or entirely in
 * float32 on the float32 MFMA (MUON_GEMM_F32).  Matrices whose shorter side
 * is below 160 run in float32 in both modes (with bfloat16 iterates a matrix
 * with few singular values deviates from the exact iteration by up to ~12%);
 * in float32 no accumulation chain is longer than 32768 products.  The
 * first iterate is stored
 * as U itself (rounded to the Newton-Schulz type) and the normalization is
 * applied in float32 inside the first iteration: A0 = inv^2 (U U^T),
 * X1 = inv (a U + B0 U), inv = 1 / (||U||_F + 1e-7) -- the same iterates as
 * X0 = U / (||U||_F + 1e-7), with one rounding fewer.  Rank-deficient inputs:
 * the exact O lies in U's column and row spaces, and that part is computed to
 * the mode's accuracy; in U's null space each iteration multiplies rounding
 * noise by a = 3.4445, so O also carries a component there, about a^5 times
 * the products' rounding error: below 3e-4 of ||O|| in float32, but of the
 * order of ||O|| itself with bfloat16 iterates (use MUON_GEMM_F32 for inputs
 * of very low rank).  The bfloat16 mode's deviation also grows with
 * ns_steps, since rounding accumulates while the quintic keeps the singular
 * values oscillating in its band: on Gaussian inputs about 2e-3 relative at 2
 * iterations, 1e-2 at 5, 2.4e-2 at 10 and 5e-2 at 64 (float32: below 3e-5 at
 * 64).  With ns_steps == 0,
 * O = fl(s * X0) with X0 rounded to the Newton-Schulz type.  O = fl(s * x)
 * in float32.  Results are deterministic and do not depend on the order of
 * descriptors; muon_step equals muon_apply(muon_orthogonalize(muon_momentum))
 * bit for bit.
 *
 * Buffers.  All buffer pointers are device pointers allocated by the caller,
 * who keeps ownership.  Descriptor arrays are host memory read during the
 * call.  The workspace is caller-owned device memory, 256-byte aligned; its
 * contents are undefined after a call.  Calls that share a workspace must be
 * ordered on one stream and made one after the other: a call is several
 * launches, and those of calls made by two threads at once may mix.  With muon_workspace_bytes() bytes every matrix is
 * orthogonalized in one wave; a smaller workspace of at least
 * muon_workspace_min_bytes() bytes runs the matrices in waves, each wave's
 * intermediates fitting the workspace (the pages' optimizer likewise works
 * through its buffers one at a time on the caller's stream, FsdpMuon class
 * docstring).  Results do not depend on the wave split, bit for bit.
 *
 * Execution.  All work is enqueued on `stream` (0 = the null stream) and the
 * call returns without waiting for it.  The first call with a new descriptor
 * set (per device, GEMM mode and -- when it runs in waves -- workspace size)
 * builds a launch plan and uploads its tables: one device allocation and a
 * stream synchronization, so make that call outside graph capture and while
 * no stream of the process is being captured in global mode.  Later calls
 * with the same set allocate nothing and do not synchronize the host.  Plans
 * stay in a 64-entry least-recently-used cache; a plan used while its stream
 * is being captured into a HIP graph is pinned (never evicted, kept until the
 * process ends), since the graph keeps pointers to its tables.  An evicted
 * plan's tables are freed after a device synchronization.
 *
 * Errors.  The pages' optimizer validates its parameter-to-group mapping up
 * front and raises rather than run on a bad mapping (FsdpMuon._validate_parameter_groups
 * on the page "core.distributed.fsdp.src.megatron_fsdp.experimental.muon";
 * the review answer on the page "feat(fsdp): expose HSDP and HFSDP through
 * the MFSDP v2 adapter": an inconsistent layout is an error, never a quiet
 * wrong mapping).  Here every entry point returns MUON_OK (0) or a
 * negative muon_status_t instead of raising: nothing is thrown across the
 * ABI.  Every check except MUON_ERR_HIP runs before anything is enqueued, so
 * a failed call leaves every buffer untouched.  muon_last_error() returns a
 * thread-local message describing the last failure of this thread.  Values
 * that are NaN or infinite inside the buffers are not checked: they propagate.
 */
#ifndef MUON_STEP_H
#define MUON_STEP_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* One 2-D parameter inside the flat buffers (page "core.distributed.fsdp.src.
 * megatron_fsdp.experimental.muon": FsdpMuon handles 2-D parameters only,
 * held in flat FSDP buffers; the owner scatters slices of each full update to
 * their shard destinations, "Opt step" step 5 of PR #6425).
 *
 *   offset        element offset of the row-major rows x cols matrix in the
 *                 flat grads / momentum (and update) buffers; multiple of 4.
 *   rows, cols    matrix shape, each >= 1 and <= 2^20, rows*cols <= 2^34;
 *                 a set's matrices hold at most 2^36 elements in total
 *                 (MUON_ERR_BAD_SHAPE otherwise).
 *   param_offset  element offset of slice 0 in the flat params buffer.
 *   shard_stride  distance in elements between consecutive slices in params
 *                 (>= rows*cols/n_shards; ignored when n_shards == 1).
 *   n_shards      the flattened matrix is cut into n_shards contiguous slices
 *                 of rows*cols/n_shards elements; slice k of the update goes
 *                 to params[param_offset + k*shard_stride ...].  For
 *                 n_shards > 1 the slice length must be a multiple of 8.
 *   group         optimizer group of the matrix for muon_step_grouped
 *                 (0 <= group < n_groups); must be 0 for every other entry
 *                 point (muon_workspace_bytes accepts any group >= 0).
 * Every slice start must be 16-byte aligned within params.  Matrices must not
 * overlap each other in grads/momentum, nor slices each other in params. */
typedef struct muon_matrix_desc {
    int64_t offset;
    int64_t rows;
    int64_t cols;
    int64_t param_offset;
    int64_t shard_stride;
    int32_t n_shards;
    int32_t group;
} muon_matrix_desc_t;

typedef enum muon_status {
    MUON_OK = 0,
    MUON_ERR_NULL_POINTER = -1,        /* a required pointer is NULL */
    MUON_ERR_BAD_SHAPE = -2,           /* rows/cols < 1, numel % n_shards, slice length */
    MUON_ERR_OUT_OF_BOUNDS = -3,       /* a matrix or slice leaves its buffer */
    MUON_ERR_MISALIGNED = -4,          /* a matrix, slice or workspace start misaligned */
    MUON_ERR_OVERLAP = -5,             /* two descriptors' ranges intersect */
    MUON_ERR_ALIAS = -6,               /* two distinct buffers' address ranges intersect */
    MUON_ERR_BAD_ARG = -7,             /* bad n, dtype, mode, ns_steps, group or non-finite scalar */
    MUON_ERR_WORKSPACE_TOO_SMALL = -8, /* workspace smaller than muon_workspace_bytes() */
    MUON_ERR_HIP = -9,                 /* a HIP runtime call failed (message has details) */
    MUON_ERR_INTERNAL = -10            /* an exception, such as no host memory; message has details */
} muon_status_t;

/* Element type of the params buffer.  grads, momentum and updates are float32. */
enum { MUON_DTYPE_F32 = 0, MUON_DTYPE_BF16 = 1 };

/* Arithmetic of the Newton-Schulz chain. */
enum { MUON_GEMM_BF16_MFMA = 0, MUON_GEMM_F32 = 1 };

/* Bytes of device workspace with which muon_step / muon_orthogonalize run
 * these descriptors in one wave, for this GEMM mode (the plan-building
 * analogue of FsdpMuon's owner assignment, which is worked out once when the
 * optimizer is set up).  Host-only: makes no HIP call.  Validates the descriptors' shapes
 * (not their bounds).  out_bytes: host pointer receiving the size. */
int muon_workspace_bytes(const muon_matrix_desc_t* descs, int64_t n, int gemm_mode,
                         size_t* out_bytes);

/* Smallest workspace with which the descriptors run at all: the largest
 * single matrix's intermediates.  Between this and muon_workspace_bytes() the
 * matrices run in waves whose intermediates fit the workspace given (the
 * FsdpMuon class docstring: the step works through the buffers in turn on the
 * caller's stream).  Host-only, same validation as muon_workspace_bytes. */
int muon_workspace_min_bytes(const muon_matrix_desc_t* descs, int64_t n, int gemm_mode,
                             size_t* out_bytes);

/* The whole step ("Opt step" steps 1, 2, 4, 6 of PR #6425; FsdpMuon.step).
 *   params        device, n_param_elems elements of param_dtype; updated in place.
 *   grads         device, float32, n_state_elems elements; read only.
 *   momentum      device, float32, n_state_elems elements; updated in place.
 *   descs, n      host array of n descriptors (n == 0 is a no-op).
 *   lr, weight_decay, beta  finite float32 scalars.
 *   nesterov      0 or 1.   ns_steps  0..64.   gemm_mode  MUON_GEMM_*.
 *   workspace     device, 256-byte aligned, >= muon_workspace_min_bytes()
 *                 (>= muon_workspace_bytes() for one wave).
 * The four buffers must not alias one another. */
int muon_step(void* params, int param_dtype, int64_t n_param_elems, const float* grads,
              float* momentum, int64_t n_state_elems, const muon_matrix_desc_t* descs,
              int64_t n, float lr, float weight_decay, float beta, int nesterov, int ns_steps,
              int gemm_mode, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Momentum update and orthogonalization input alone ("Opt step" steps 1-2;
 * FsdpMuon._compute_momentum_inputs).  Writes U (float32) to u_out at each
 * descriptor's offset; momentum updated in place.  grads, momentum, u_out are
 * device buffers of n_state_elems float32 that must not alias.  Weight decay
 * is applied by muon_apply (decoupled), not here. */
int muon_momentum(const float* grads, float* momentum, float* u_out, int64_t n_state_elems,
                  const muon_matrix_desc_t* descs, int64_t n, float beta, int nesterov,
                  hipStream_t stream);

/* Orthogonalization alone ("Opt step" step 4; FsdpMuon._orthogonalize_updates):
 * o_out = s * NS(u) for every descriptor, both device float32 buffers of
 * n_elems elements laid out like grads.  o_out may equal u (in place) but must
 * not partially overlap it.  Workspace as for muon_step. */
int muon_orthogonalize(const float* u, float* o_out, int64_t n_elems,
                       const muon_matrix_desc_t* descs, int64_t n, int ns_steps, int gemm_mode,
                       void* workspace, size_t workspace_bytes, hipStream_t stream);

/* One optimizer group of muon_step_grouped: the pages' optimizer keeps its
 * settings per parameter group and maps every parameter to its group (page
 * "core.distributed.fsdp.src.megatron_fsdp.experimental.muon", FsdpMuon._step_group,
 * argument tensor_to_optimizer_group_index).  An array of groups lives in DEVICE
 * memory and is read by the kernels when they run, so a captured graph
 * replays with whatever values the array holds at replay time (optimizer
 * CUDA-graph support is among the features the Megatron-Bridge #5933 commit
 * message lists, quoted on the page "feat(fsdp): expose HSDP and HFSDP
 * through the MFSDP v2 adapter", PR #6873).  Values are not checked: NaN and
 * infinities propagate; nesterov is true when non-zero. */
typedef struct muon_group {
    float lr;
    float weight_decay;
    float beta;
    int32_t nesterov;
} muon_group_t;

/* The whole step with per-matrix optimizer groups and an optional bfloat16
 * model copy.  Matrix i uses groups[descs[i].group]; its results equal, bit for
 * bit, those of muon_step called with that group's scalars.
 *   groups, n_groups  DEVICE array of n_groups (1..65536) muon_group_t, read
 *                     during the kernels; must not overlap the other buffers.
 *   model_copy        NULL, or -- with param_dtype MUON_DTYPE_F32 only -- a
 *                     device bfloat16 buffer of n_param_elems elements, 16-byte
 *                     aligned and laid out like params: every updated weight
 *                     is also stored there, rounded to nearest even (float32
 *                     master weights with a refreshed bfloat16 model copy: the
 *                     pages' optimizer updates the model weights from the
 *                     optimizer's own copy, FsdpMuon class docstring and
 *                     FsdpMuon.step; the precision-aware optimizer listed in the
 *                     Megatron-Bridge #5933 commit message on the PR #6873 page).
 * Every other argument as muon_step.  Once the plan for a descriptor set
 * exists (built by the first call with that set, which synchronizes the
 * stream: make it outside graph capture), a call makes no allocation, memset
 * or host synchronization and may be captured into a HIP graph. */
int muon_step_grouped(void* params, int param_dtype, int64_t n_param_elems, void* model_copy,
                      const float* grads, float* momentum, int64_t n_state_elems,
                      const muon_matrix_desc_t* descs, int64_t n, const muon_group_t* groups,
                      int32_t n_groups, int ns_steps, int gemm_mode, void* workspace,
                      size_t workspace_bytes, hipStream_t stream);

/* Decay and update alone ("Opt step" step 6; FsdpMuon._apply_local_updates):
 * params slice k <- fl(fl(W*f) - fl(lr*O)), f = fl(1 - fl(lr*weight_decay)),
 * with O read from `updates` (device float32, n_update_elems, laid out like
 * grads) and slices scattered as the descriptors say.  params and updates
 * must not alias. */
int muon_apply(void* params, int param_dtype, int64_t n_param_elems, const float* updates,
               int64_t n_update_elems, const muon_matrix_desc_t* descs, int64_t n, float lr,
               float weight_decay, hipStream_t stream);

/* muon_step for callers that cannot allocate device memory: code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc.  Same
 * arguments and results (bit for bit) as muon_step, without the workspace:
 * every intermediate lives in a fixed device array of 320 MiB that the library
 * holds on each GPU it runs on, from its load until the process ends (8 MiB of
 * launch tables, 312 MiB of workspace; matrices that do not fit at once run in
 * waves).  The call makes no hipMalloc, hipFree or other allocation.  A matrix
 * whose intermediates alone exceed 312 MiB (for example 4096 x 16384 with
 * bfloat16 products), or a set whose launch tables exceed 8 MiB, is rejected
 * with MUON_ERR_WORKSPACE_TOO_SMALL before anything is enqueued.  The first
 * call with a new descriptor set on a device copies its launch tables into the
 * array and synchronizes `stream`; later calls with the same set copy nothing
 * and do not synchronize.  Under graph capture only a call with the set whose
 * tables are resident (the device's last one) can run: any other is rejected
 * with MUON_ERR_BAD_ARG before anything is enqueued, leaving the resident
 * tables in place.  All calls on one GPU share its array, which keeps
 * the last call's contents: calls that overlap on one GPU (different streams,
 * or threads without ordering) race and must not be made. */
int muon_step_noalloc(void* params, int param_dtype, int64_t n_param_elems, const float* grads,
                      float* momentum, int64_t n_state_elems, const muon_matrix_desc_t* descs,
                      int64_t n, float lr, float weight_decay, float beta, int nesterov,
                      int ns_steps, int gemm_mode, hipStream_t stream);

/* ------------------------------------------- gradient norm, clipping, AdamW
 *
 * What a training step needs beside the Muon step: the norm of ALL gradients
 * (matrices and the rest), the clipping that follows from it, and an optimizer
 * for the parameters that Muon skips ("Non-2D parameters are skipped. Use a
 * separate optimizer", FsdpMuon class docstring; "clip_grad" in the
 * Megatron-Bridge #5933 commit message).  All but muon_step_clipped keep no
 * plan and allocate nothing: every call of theirs, the first one too, may be
 * captured into a HIP graph.  muon_step_clipped has the plans of
 * muon_step_grouped, so its first call with a descriptor set is made outside
 * graph capture.  Nothing returns to the host: the norm and the clipping
 * coefficient stay in a record in device memory, which the consuming kernels
 * read when they run.  Errors, streams and ownership as above. */

/* One tensor of a list: `numel` consecutive elements (0..2^34; a list holds at
 * most 2^36) of type MUON_DTYPE_F32 or MUON_DTYPE_BF16 in device memory,
 * aligned to its elements only.  data may be NULL where numel is 0.  Lists are
 * host memory read during the call. */
typedef struct muon_tensor {
    void* data;
    int64_t numel;
    int32_t dtype;
    int32_t reserved;
} muon_tensor_t;

/* The clipping record, in DEVICE memory, 16-byte aligned, owned by the caller:
 *   sumsq  sum of the squares of all elements, float64
 *   norm   sqrt(sumsq), rounded to float32
 *   coef   min(1, max_norm / (sqrt(sumsq) + 1e-6)), rounded to float32
 * The sum is float64 from the first element on (squares of float32 are exact
 * there), so it neither overflows nor underflows.  A NaN among the elements
 * makes sumsq, norm and coef NaN; an infinity without a NaN gives sumsq = norm
 * = inf and coef = 0 (NaN where max_norm is infinite too), so that clipping
 * turns the infinite elements into NaN.  The same call gives the same bits; the
 * last bits of sumsq depend on the order of summation, that is on the list's
 * lengths, order and addresses and on whether tensor_norms are asked for. */
typedef struct __attribute__((aligned(16))) muon_clip {
    double sumsq;
    float norm;
    float coef;
} muon_clip_t;

/* Bytes of device workspace (256-byte aligned) of muon_grad_norm for this
 * list.  It depends on the lengths alone.  Host-only. */
int muon_clip_workspace_bytes(const muon_tensor_t* tensors, int64_t n, size_t* out_bytes);

/* Global 2-norm of the listed tensors, and the clipping coefficient.
 *   max_norm      >= 0; infinity never clips.
 *   clip          receives the record (n == 0: sumsq = norm = 0).
 *   tensor_norms  NULL, or device float32 [n]: the norm of every tensor.
 *   workspace     device, >= muon_clip_workspace_bytes(); calls that share it
 *                 (or a record) must be ordered on one stream and made one
 *                 after the other, not by two threads at once.
 * Tensors may overlap each other (each counts in full); the record, the norms
 * and the workspace may not overlap anything. */
int muon_grad_norm(const muon_tensor_t* tensors, int64_t n, float max_norm, muon_clip_t* clip,
                   float* tensor_norms, void* workspace, size_t workspace_bytes,
                   hipStream_t stream);

/* norm and coef of a record from its sumsq: after the caller has summed sumsq
 * over the ranks that hold parts of the gradient. */
int muon_clip_finish(muon_clip_t* clip, float max_norm, hipStream_t stream);

/* dst[i] = coef * src[i], in float32, rounded once to dst's type (nearest
 * even), for every element of every tensor.  Lists have the same lengths;
 * types may differ.  A dst may be its src (same address and type: in place; a
 * list that is so throughout is neither read nor written while coef is 1);
 * apart from that no dst may overlap another dst or a src. */
int muon_clip_grads(const muon_tensor_t* src, const muon_tensor_t* dst, int64_t n,
                    const muon_clip_t* clip, hipStream_t stream);

/* muon_step_grouped on the clipped gradient fl(coef * G), without a pass of its
 * own: the kernel that reads G multiplies.  Results equal, bit for bit, those of
 * muon_clip_grads into another float32 buffer followed by muon_step_grouped
 * with it; grads itself is only read.  clip must not overlap the other buffers.
 * The first call with a descriptor set (unless muon_step_grouped or muon_step
 * ran with it, in the same mode and workspace size) builds its plan, allocates and
 * synchronizes: make it outside graph capture, where it is refused with
 * MUON_ERR_BAD_ARG before anything is enqueued. */
int muon_step_clipped(void* params, int param_dtype, int64_t n_param_elems, void* model_copy,
                      const float* grads, float* momentum, int64_t n_state_elems,
                      const muon_matrix_desc_t* descs, int64_t n, const muon_group_t* groups,
                      int32_t n_groups, const muon_clip_t* clip, int ns_steps, int gemm_mode,
                      void* workspace, size_t workspace_bytes, hipStream_t stream);

/* One range of parameters of muon_adamw.
 *   offset        first element in grads / exp_avg / exp_avg_sq; multiple of 4,
 *                 below 2^36
 *   numel         0..2^34 elements (2^36 in all ranges)
 *   param_offset  first element in params (and model_copy); 16-byte aligned,
 *                 below 2^36
 *   group         row of the group table */
typedef struct muon_range {
    int64_t offset;
    int64_t numel;
    int64_t param_offset;
    int32_t group;
    int32_t reserved;
} muon_range_t;

/* One optimizer group of muon_adamw, in DEVICE memory and read by the kernels
 * when they run, like muon_group_t.  step is the number t >= 1 of the step to be
 * made, for the bias corrections; the caller raises it between steps.  Values
 * are not checked. */
typedef struct muon_adamw_group {
    float lr;
    float weight_decay;
    float beta1;
    float beta2;
    float eps;
    int32_t reserved;
    int64_t step;
} muon_adamw_group_t;

/* One AdamW step on ranges of flat buffers:
 *   g = fl(coef * G)  (coef of `clip`; g = G where clip is NULL)
 *   m <- fl(fl(beta1*m) + fl((1-beta1)*g))
 *   v <- fl(fl(beta2*v) + fl(fl((1-beta2)*g)*g))
 *   W <- fl(fl(W*f) - fl(a * fl(m / fl(fl(sqrt(v)*r) + eps))))
 *   f = fl(1 - fl(lr*wd)),  a = fl(lr / (1 - beta1^t)),  r = fl(1 / sqrt(1 - beta2^t))
 * in float32, each operation rounded on its own; a and r are computed in
 * float64 and rounded once.  bfloat16 weights are rounded once, to nearest
 * even, on store.
 *   params      device, n_param_elems of param_dtype, updated in place
 *   model_copy  NULL, or (float32 params only) device bfloat16 laid out like
 *               params, receives every updated weight rounded to nearest even
 *   grads       device, n_state_elems of grad_dtype, read only
 *   exp_avg, exp_avg_sq  device float32, n_state_elems, updated in place
 *   groups, n_groups     DEVICE array of 1..65536 groups (8-byte aligned)
 *   clip        NULL or a record
 * Every buffer starts 16-byte aligned.  Buffers must not overlap one another,
 * nor ranges each other.  Elements outside the ranges stay as they are. */
int muon_adamw(void* params, int param_dtype, int64_t n_param_elems, void* model_copy,
               const void* grads, int grad_dtype, float* exp_avg, float* exp_avg_sq,
               int64_t n_state_elems, const muon_range_t* ranges, int64_t n,
               const muon_adamw_group_t* groups, int32_t n_groups, const muon_clip_t* clip,
               hipStream_t stream);

/* ------------------------------------ 8-bit matrices and their products
 *
 * What the linear layers between two steps need where they run in 8 bits: an
 * 8-bit copy of the updated weights (the counterpart of model_copy, which is
 * bfloat16; the precision-aware optimizer of the Megatron-Bridge #5933 commit
 * message), the products that read it, and the product that adds a weight's
 * gradient to the float32 buffer that the step reads.  These calls keep no plan
 * and allocate nothing: every call, the first one too, may be captured into a
 * HIP graph.  Errors, streams and ownership as above. */

/* 8-bit floats: 4 exponent and 3 mantissa bits (largest number 448, no
 * infinities), 5 and 2 (largest 57344). */
enum { MUON_FP8_E4M3 = 0, MUON_FP8_E5M2 = 1 };

/* A rows x cols matrix of 8-bit floats with a float32 scale for each block of
 * block_rows x 128 elements (blocks at the ends are short): element (i, j) stands
 * for codes[i * row_stride + j] * scales[i / block_rows * scale_row + j / 128 *
 * scale_col].
 *   rows, cols   0..2^24, rows * cols <= 2^34
 *   block_rows   1 or 128
 *   row_stride   bytes between rows, cols..2^26; any alignment (products run
 *                fastest where codes, row_stride and cols are multiples of 16)
 *   scale_row, scale_col  elements between the scales of adjacent blocks, 1..2^32,
 *                none overlapping another; products read fastest with scale_row = 1
 * (A stride counts where there is more than one row, or block, to step to.) */
typedef struct muon_fp8 {
    void* codes;
    float* scales;
    int64_t rows, cols;
    int64_t row_stride;
    int64_t scale_row, scale_col;
    int32_t format;
    int32_t block_rows;
} muon_fp8_t;

/* A matrix into 8 bits: out, out_t or both (either may be NULL) receive x
 * (rows x cols of dtype, row_stride elements between rows, cols..2^26) and its
 * transpose, each in its own blocks.  For each block
 *   m = max(largest magnitude, 2^-100),  s = fl(m / L)     L = 448 or 57344
 *   code = x L / m rounded to nearest, to even in the middle (once)
 * A block that holds a NaN gets the scale NaN, one that holds an infinity an
 * infinite one; its codes say nothing.  x, codes and scales must not overlap: neither each other nor,
 * where there are gaps between rows, each other's span from the first element to
 * the last.  Elements in the gaps stay as they are. */
int muon_fp8_cast(const void* x, int dtype, int64_t rows, int64_t cols, int64_t row_stride,
                  const muon_fp8_t* out, const muon_fp8_t* out_t, hipStream_t stream);

/* Bytes of device workspace (256-byte aligned) of muon_fp8_matmul for m x n
 * products over k; 0 for most.  Host-only. */
int muon_fp8_workspace_bytes(int64_t m, int64_t n, int64_t k, size_t* out_bytes);

/* out = a b^T, or out += a b^T: a is m x k, b is n x k, out m x n of out_dtype
 * with out_row_stride elements between rows (n..2^26), m n <= 2^36.  Sums over a block of 128 along k
 * are float32, as is the sum of these times their two scales, whatever the sizes
 * of the two (where their product alone is no normal float32, and codes are not
 * zero, a product takes 10 to 20 times as long); the result is
 * rounded once (with accumulate, after out is added; out is then float32).  With a
 * bfloat16 out the 8-bit matrix instruction multiplies: it cuts each product at 2^-13
 * of the largest product of the group of 8 that it is added with, which for
 * operands of one size stays 100 times below the rounding of out; with a float32
 * out every product is exact (and the rate half).  k = 0
 * gives zeros, or leaves out as it is.  The same call gives the same bits.  An
 * element of out depends on its row of a and its row of b alone: NaN and
 * infinite scales and codes propagate there.  out must not overlap a, b or the
 * workspace (spans as above); a and b may overlap each other.  Calls that share
 * a workspace must be ordered on one stream and made one after the other. */
int muon_fp8_matmul(const muon_fp8_t* a, const muon_fp8_t* b, void* out, int out_dtype,
                    int64_t out_row_stride, int accumulate, void* workspace,
                    size_t workspace_bytes, hipStream_t stream);

/* -------------------------------------------- orthogonalization of stacks
 *
 * muon_orthogonalize for matrices outside flat buffers: the heads of a
 * projection, the experts of a layer, a gradient that is a view of a larger
 * tensor.  `count` matrices of rows x cols, row-major, in_stride elements apart
 * with in_row elements between rows (out likewise), float32 or bfloat16:
 *   X = U / (||U||_F + 1e-7)   (U^T where rows > cols), then for every step t
 *   A = X X^T, B = b_t A + c_t A A, X <- a_t X + B X;    O = scale X
 * X, A and B are held as pairs of float16 whose sum keeps 22 bits, scaled by
 * powers of two, and every product takes three of the four products of their halves
 * (the fourth lies below the pairs' own rounding), summed in float32: float32
 * accuracy (about 1e-6 relative to ||O|| for five steps of the default
 * coefficients on Gaussian input) at the rate of the 16-bit matrix cores.  The
 * norm is a float64 sum in fixed order.  The same call gives the same bits; a NaN or
 * an infinity makes its own matrix NaN and no other.  No plan, no allocation:
 * every call may be captured. */
typedef struct muon_stack {
    const void* in;
    void* out;
    int64_t count, rows, cols; /* count 0..2^20, sides 1..2^20, rows * cols <= 2^31 */
    int64_t in_stride, in_row; /* elements; in_row cols..2^31, in_stride 0..2^40 */
    int64_t out_stride, out_row; /* likewise */
    int32_t in_dtype, out_dtype;
} muon_stack_t;

/* Bytes of device workspace (256-byte aligned) of muon_orthogonalize_stack: the
 * whole stack's intermediates.  With less, but at least its `count`-th part
 * (one matrix of this stack: how a matrix is divided among workgroups depends on
 * how many there are), the matrices run in groups that fit, with identical
 * results.  Host-only. */
int muon_stack_workspace_bytes(const muon_stack_t* stack, size_t* out_bytes);

/*   coefficients  host, 3 * n_steps float32: (a, b, c) of every step.  Finite, and such
 *                 that the bound s on the largest singular value, which starts at 1
 *                 and is worked out from them, and |a| + |b| s^2 + |c| s^4 stay below 2^24.
 *   n_steps       0..64;  scale  finite
 * in and out must not overlap (spans from first to last element); the matrices of
 * in may overlap each other, those of out may not. */
int muon_orthogonalize_stack(const muon_stack_t* stack, const float* coefficients, int n_steps,
                             float scale, void* workspace, size_t workspace_bytes,
                             hipStream_t stream);

/* Kernel timing, a profiling aid (not part of the step's semantics).
 * Between muon_profile_begin() and muon_profile_end(), every kernel the
 * library launches, from any thread, is bracketed by two HIP events recorded
 * on the launch's own stream.  muon_profile_end() stops recording, waits for
 * the recorded events, and aggregates elapsed time by kernel name into `out`
 * (at most max_entries rows, host memory; *n_entries receives the number of
 * distinct kernels, which may exceed max_entries).  Names are
 * "front", "sumsq", "norm", "cast", "apply" and "ns_<stage>_t<tile>_<type>"
 * for the Newton-Schulz products (stage a: X X^T, b: b A + c A A, x: a X + B X;
 * tile 64/128/256; type bf16/f32); "grad_norm", "norm_solo", "tensor_norms",
 * "norm_finish", "clip_finish", "clip" and "adamw" for the clipping and AdamW
 * above; "fp8_cast", "fp8_matmul" and "fp8_join" for 8-bit matrices; "stack_norm",
 * "stack_split", "stack_a", "stack_b", "stack_x", "stack_join", "stack_scaled",
 * "stack_whole", "stack_gram", "stack_poly" and "stack_strip" for stacks.  Events
 * come from a pool the library owns; when timing is off the only cost is one flag
 * test per launch. */
typedef struct muon_kernel_time {
    char name[48];
    double total_ms;   /* sum of the launches' event-to-event times */
    int64_t launches;
} muon_kernel_time_t;

int muon_profile_begin(void);
int muon_profile_end(muon_kernel_time_t* out, int max_entries, int* n_entries);

/* Static name of a status code ("MUON_OK", "MUON_ERR_BAD_SHAPE", ...): the
 * kind of a rejected call, which the pages' optimizer reports by raising from
 * its up-front validation (FsdpMuon._validate_parameter_groups, page
 * "core.distributed.fsdp.src.megatron_fsdp.experimental.muon"; errors rather
 * than wrong mappings, review answers on the page "feat(fsdp): expose HSDP and
 * HFSDP through the MFSDP v2 adapter").  Any int is accepted; unknown codes
 * give "MUON_ERR_UNKNOWN".  The string is static: never free it. */
const char* muon_status_string(int status);

/* Message of the calling thread's last failure ("" if none): the text the
 * pages' validation would raise with (same passages as muon_status_string),
 * naming the offending descriptor, buffer or argument.  Thread-local, owned
 * by the library, valid until the thread's next failing call into this
 * library; never free it.  Successful calls leave it unchanged. */
const char* muon_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MUON_STEP_H */
