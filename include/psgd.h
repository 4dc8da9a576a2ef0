/*
 * psgd.h -- C ABI of the GB300-native PowerSGD communication-hook step.
 *
 * A data-parallel job of W workers is either simulated inside one GPU by W
 * replica gradient buckets resident in the same HBM -- the "allreduce" of the
 * pages is then a mean over those W buckets, folded into the kernels that read
 * them (psgd_step) -- or spread over W processes with one replica each, the
 * pages' two exchanges left to the caller's collective on library-owned
 * buffers (psgd_dp_*).  Every step of the method runs in CUDA kernels of this
 * library; the host side only plans, allocates (at create time) and enqueues.
 *
 * Sources (web pages; the operations are restated here, not copied):
 *   [DDP]  "DDP Communication Hooks" (PyTorch 1.11 documentation):
 *          "PowerSGD State" (PowerSGDState and its items 1-4),
 *          "PowerSGD Hooks" (powerSGD_hook steps 1-3.7, the vanilla-allreduce
 *          note, the error-feedback memory warning),
 *          "Default Communication Hooks" (allreduce_hook: the mean).
 *   [DDP2] "DDP Communication Hooks" (spec-zone.ru translation of a later
 *          version): "PowerSGD State" item 5, batch_tensors_with_same_shape.
 *   [AMP]  "Automatic Mixed Precision package - torch.cuda.amp",
 *          GradScaler: unscale, inf/NaN check, skipped step.
 *
 * Conventions for every call:
 *   - Return value: PSGD_OK (0) or a positive informational code on success,
 *     a negative PSGD_E* code on failure; psgd_last_error() then holds a
 *     message (thread-local, valid until the next failing call on the thread).
 *   - "device pointer" = CUDA global memory on the state's device; "host
 *     pointer" = ordinary (pageable or pinned) CPU memory.  The caller owns
 *     every pointer it passes; the library never frees or retains them past
 *     the call (psgd_step: past the enqueued work).
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  psgd_step enqueues only and never synchronises.
 *   - Host threads: calls on one state (or one group) must not overlap in
 *     time; different states may be driven from different threads at once
 *     (the library's process-wide launch settings are atomic or locked).
 *   - Elements of a bucket are in bucket order: tensor 0 first, each tensor
 *     row-major in its own shape, with no padding between tensors.
 */
#ifndef PSGD_H
#define PSGD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct psgd_state psgd_state; /* opaque, library-owned */

/* Type of the replica gradient buckets.  F16 / BF16: 16-bit gradients, as
 * produced by GradScaler-scaled half-precision training or by the pages'
 * fp16/bf16 compress wrappers ("Default Communication Hooks":
 * fp16_compress_wrapper / bf16_compress_wrapper cast the bucket to 16 bits);
 * the library computes in fp32 and returns fp32 (the cast back). */
typedef enum { PSGD_F32 = 0, PSGD_F16 = 1, PSGD_BF16 = 2 } psgd_dtype;

/* 8-bit floating point formats: e4m3 (largest value 448, no infinities) and e5m2 (57344). */
typedef enum { PSGD_E4M3 = 0, PSGD_E5M2 = 1 } psgd_code;

#define PSGD_OK 0
#define PSGD_SKIPPED_NONFINITE 1 /* [AMP] inf/NaN seen: step skipped, state kept   */
#define PSGD_BAD_TOKEN 2         /* an embedding met an id outside its table       */
#define PSGD_EINVAL (-1)         /* bad argument                                   */
#define PSGD_ENOMEM (-2)         /* device or host allocation failed               */
#define PSGD_ECUDA (-3)          /* a CUDA call failed                             */
#define PSGD_ETIMEOUT (-4)       /* a bounded device-side wait gave up             */

#define PSGD_MAX_RANK 32  /* largest matrix_approximation_rank ([DDP] item 1 names up to 32) */
#define PSGD_MAX_WORLD 64 /* largest number of simulated replicas W              */

/*
 * psgd_plan -- host-only planner query (no GPU needed).
 *
 * [DDP] powerSGD_hook step 1: views the flat bucket as per-parameter tensors
 * and splits them into a compressed group and an uncompressed group (every
 * tensor of fewer than 2 dimensions is uncompressed).  A tensor of >= 2 dims
 * is viewed as (shape[0], prod(shape[1:])) and compressed iff
 *   (rows + cols) * matrix_approximation_rank * min_compression_rate < rows * cols
 * ([DDP] "PowerSGD State" item 3; strict, evaluated in double precision).
 *
 *   dims, ndims, n_tensors : shapes, concatenated: tensor t has ndims[t]
 *                            entries of dims starting after the previous ones.
 *   compressed[n_tensors]  : out, 1 if the tensor is compressed.
 *   ranks[n_tensors]       : out, min(rank, rows, cols) if compressed, else 0.
 *   rows[n_tensors], cols[n_tensors] : out, the 2-D view (0,0 for < 2 dims).
 *   Any of the out arrays may be NULL.
 * Errors: PSGD_EINVAL for a negative dimension, n_tensors < 0 or rank outside
 * [1, PSGD_MAX_RANK].
 */
int psgd_plan(const int64_t* dims, const int32_t* ndims, int32_t n_tensors,
              int32_t matrix_approximation_rank, double min_compression_rate,
              int32_t* compressed, int32_t* ranks, int64_t* rows, int64_t* cols);

/*
 * psgd_state_create -- [DDP] PowerSGDState(...) for one bucket layout.
 *
 * Hyper-parameters keep the pages' names and meaning ([DDP] items 1-4,
 * [DDP2] item 5).  world_size = W simulated replicas.  grad_dtype is the type
 * of the replica buckets passed to psgd_step (F16 / BF16: 16-bit buckets).
 * Allocates on `device` everything a step needs: the per-replica error
 * feedback store, P/Q memory and all scratch; psgd_step allocates nothing.
 * The error store is kept twice (the current and the next step) so that a
 * skipped step ([AMP]) leaves the state bit-identical.
 * random_seed seeds the counter-based generator (Philox4x32-10) that draws
 * the initial standard-normal Q when none was injected with psgd_set_q.
 * Errors: PSGD_EINVAL (rank outside [1,32], world_size outside [1,64],
 * negative dims, start_powerSGD_iter < 0, min_compression_rate < 0 or NaN,
 * epsilon < 0, device ordinal 64 or above), PSGD_ENOMEM, PSGD_ECUDA (no such
 * device).  *out is NULL on failure.  Every creator takes the same device
 * rule; states on several devices may live in one process.
 */
int psgd_state_create(const int64_t* dims, const int32_t* ndims, int32_t n_tensors,
                      int32_t world_size, int32_t matrix_approximation_rank,
                      int64_t start_powerSGD_iter, double min_compression_rate,
                      int32_t use_error_feedback, int32_t warm_start,
                      float orthogonalization_epsilon, uint64_t random_seed,
                      int32_t batch_tensors_with_same_shape, psgd_dtype grad_dtype,
                      int32_t device, psgd_state** out);

/*
 * psgd_state_create_batched -- the state of [DDP] batched_powerSGD_hook
 * ("PowerSGD Hooks", batched_powerSGD_hook steps 1-9): the whole flat bucket
 * of `numel` elements is viewed as ONE square matrix of side
 * ceil(sqrt(numel)), zero beyond the bucket, compressed by one PowerSGD step
 * per psgd_step call, and the result truncated to `numel` elements.  There
 * is no compression-rate gate.  Error feedback covers the padded square
 * (psgd_error_numel = side * side; tensor 0 of psgd_tensor_info is the
 * square).  Other arguments as psgd_state_create; psgd_step and the other
 * calls work unchanged on the returned state.  Rows are read with 16-byte
 * vector accesses when side is a multiple of 4, element by element
 * otherwise.
 * Errors: PSGD_EINVAL (numel < 1, rank outside [1, 32], ...), PSGD_ENOMEM,
 * PSGD_ECUDA.
 */
int psgd_state_create_batched(int64_t numel, int32_t world_size, int32_t matrix_approximation_rank,
                              int64_t start_powerSGD_iter, int32_t use_error_feedback,
                              int32_t warm_start, float orthogonalization_epsilon,
                              uint64_t random_seed, psgd_dtype grad_dtype, int32_t device,
                              psgd_state** out);

/* Frees every device and host allocation of the state.  NULL is a no-op. */
void psgd_state_destroy(psgd_state* s);

/*
 * psgd_step -- one call of [DDP] powerSGD_hook on the W replicas.
 *
 *   grads[W] : host array of W device pointers; grads[w] is replica w's flat
 *              bucket of N elements of grad_dtype.  Read only.
 *   out      : device pointer, N floats: the bucket every replica receives
 *              (the hook's in-place update).  May alias grads[0] when
 *              grad_dtype is F32; must not overlap any other grads[w].
 *   inv_loss_scale : [AMP] unscale factor 1/scale multiplied into every
 *              gradient element (1.0f when no scaler is used).
 *   stream   : cudaStream_t; all work is enqueued on it, nothing waits.
 *
 * Semantics: while the call count is below start_powerSGD_iter, out is the
 * replica mean of every element ([DDP] vanilla-allreduce note).  Afterwards
 * the uncompressed tensors get their replica mean ([DDP] step 2) and each
 * compressed tensor M gets P Q^T with P = orth(mean_w M_w Q) and
 * Q = mean_w M_w^T P, M_w = replica w's gradient plus its error-feedback
 * residual, which then becomes M_w - P Q^T ([DDP] steps 3.1-3.7).  If any
 * unscaled gradient element is inf or NaN the step is skipped: state is left
 * as it was, `out` is unspecified, psgd_step_status reports
 * PSGD_SKIPPED_NONFINITE.  The call counter advances either way.
 * Errors (synchronous): PSGD_EINVAL (NULL pointers, overlap), PSGD_ECUDA.
 */
int psgd_step(psgd_state* s, const void* const* grads, float* out, float inv_loss_scale,
              void* stream);

/*
 * psgd_step_host -- psgd_step on HOST buffers: copies the W host buckets to
 * the device (one cudaMemcpyAsync per replica), runs the step and copies
 * `out` back to host memory.  Two device staging sets are allocated on the
 * first call (so the first call may return PSGD_ENOMEM) and alternated call
 * by call: the uploads run on an internal stream and wait only for the
 * download that last used the same set, the step runs on `stream` after the
 * uploads, and the download runs on a second internal stream after the step.
 * `stream` then waits for the download, so host_out is valid once `stream`
 * is synchronised, and consecutive calls overlap the next upload with the
 * current step and download.  Pinned host memory makes the copies
 * asynchronous; the host buffers must stay untouched until `stream` is
 * synchronised.
 *   host_grads[W] : host pointers, N elements of grad_dtype each.
 *   host_out      : host pointer, N floats.
 */
int psgd_step_host(psgd_state* s, const void* const* host_grads, float* host_out,
                   float inv_loss_scale, void* stream);

/*
 * psgd_set_graph -- enable (1) or disable (0) CUDA-graph replay of the steady
 * compressed step.  Once a state is past start_powerSGD_iter, has made its
 * first compressed step and warm-starts Q, every step enqueues the same
 * launches, and what is left to decide (skip on inf/NaN, the double-buffer
 * half, warm or fresh Q after a skipped first step) is decided on the device.
 * With graphs enabled, psgd_step captures that sequence once (on a private
 * stream, executing nothing) for its grads/out pointers and inv_loss_scale,
 * and afterwards enqueues it on `stream` with one cudaGraphLaunch while they
 * stay the same; other pointers or another scale capture again.  Results are
 * bit-identical to the launch-by-launch path.  Not used while profiling is on.
 * For callers that step with the same buffers every iteration and want the
 * host's launch cost out of the way (many small buckets).  Default: off.
 */
int psgd_set_graph(psgd_state* s, int32_t enable);

/* Graph captures and replays so far (either pointer may be NULL). */
int psgd_graph_stats(const psgd_state* s, int64_t* captures, int64_t* replays);

/*
 * psgd_step_status -- synchronises `stream` and returns the outcome of the
 * last step enqueued: PSGD_OK, PSGD_SKIPPED_NONFINITE, PSGD_ETIMEOUT (a
 * bounded wait inside a tensor-core kernel or at a grid barrier of the
 * cooperative Gram-Schmidt stage gave up; the step was not committed and the
 * state is as before it -- the call rebuilds the tensor-core operand images
 * of the committed factors, on `stream`, before returning), or PSGD_ECUDA.
 */
int psgd_step_status(psgd_state* s, void* stream);

/*
 * psgd_get_stats -- [DDP] "PowerSGD State": compression statistics.
 *   numel_before : elements of the bucket (N).
 *   numel_after  : elements exchanged per compressed step:
 *                  sum over compressed tensors of (rows + cols) * rank, plus
 *                  the uncompressed elements.
 *   iter         : psgd_step calls so far.
 * Any pointer may be NULL.
 */
int psgd_get_stats(const psgd_state* s, int64_t* numel_before, int64_t* numel_after,
                   int64_t* iter);

/*
 * psgd_tensor_info -- the planner's view of tensor `tensor`:
 * compressed flag, rows, cols, effective rank, first element in the bucket,
 * and first element in the packed error layout of psgd_get_error (-1 for an
 * uncompressed tensor).  Any out pointer may be NULL.
 */
int psgd_tensor_info(const psgd_state* s, int32_t tensor, int32_t* compressed,
                     int64_t* rows, int64_t* cols, int32_t* rank,
                     int64_t* bucket_offset, int64_t* packed_offset);

/* Elements of one replica's packed error buffer (psgd_get_error/set_error). */
int64_t psgd_error_numel(const psgd_state* s);

/*
 * psgd_set_q -- install Q for compressed tensor `tensor` from host memory,
 * cols x rank floats, row-major (rank = the tensor's effective rank).
 *   is_draw = 1 : the values are a standard-normal draw ([DDP] step 3.1: Q
 *                 is initialised from a standard normal distribution and
 *                 orthogonalised); it replaces the library's own draw the
 *                 next time the tensor needs a fresh Q (its first compressed
 *                 step, or every step when warm_start is 0) and is
 *                 orthogonalised there.
 *   is_draw = 0 : the values become the warm-start Q used as is by the next
 *                 compressed step (checkpoint restore).
 * Synchronous (blocks until the copy is done).  PSGD_EINVAL if the tensor is
 * not compressed.
 */
int psgd_set_q(psgd_state* s, int32_t tensor, const float* host_in, int32_t is_draw);

/* psgd_get_q -- the warm-start Q after the last committed step (cols x rank,
 * host memory; zeros before the first compressed step).  Synchronous. */
int psgd_get_q(psgd_state* s, int32_t tensor, float* host_out);

/* psgd_get_p -- the orthogonalised P of the last committed compressed step
 * (rows x rank, host memory; zeros before it).  Synchronous. */
int psgd_get_p(psgd_state* s, int32_t tensor, float* host_out);

/*
 * psgd_get_error / psgd_set_error -- replica `replica`'s error-feedback
 * residual ([DDP] "PowerSGD Hooks" warning: the extra memory that error
 * feedback needs), packed: compressed tensors in bucket order, each
 * row-major, at psgd_tensor_info's packed_offset; psgd_error_numel floats.
 * dev_out / dev_in are device pointers; the work is enqueued on `stream`.
 * PSGD_EINVAL when error feedback is off.
 */
int psgd_get_error(psgd_state* s, int32_t replica, float* dev_out, void* stream);
int psgd_set_error(psgd_state* s, int32_t replica, const float* dev_in, void* stream);

/* Bytes of device memory the state holds (error store, P/Q, scratch). */
size_t psgd_workspace_bytes(const psgd_state* s);

/*
 * psgd_set_error_store_halves -- keep the error-feedback store once (1) or
 * twice (2, the default).  The pages put error feedback's memory at the size
 * of the model's gradients ([DDP] "PowerSGD Hooks", the warning on error
 * feedback): one half is that, W x (compressed elements) floats per state.
 * With one half, pass 1 writes each step's M_w over the residual it has just
 * read, so the results are the same bits; but a step that meets an inf/NaN
 * has by then overwritten the store with that step's M_w, so its skip leaves
 * the factors as they were and the error feedback changed (reset it with
 * psgd_set_error, or keep two halves when gradients can be non-finite, as
 * with a GradScaler).  Must precede the first psgd_step (reallocates the
 * store, zeroed).  Errors: PSGD_EINVAL (NULL state, halves not 1 or 2, a step
 * already taken, a data-parallel state), PSGD_ENOMEM, PSGD_ECUDA.  A state
 * without error feedback has no store: the call then only returns PSGD_OK.
 */
int psgd_set_error_store_halves(psgd_state* s, int32_t halves);

/*
 * Kernel timing for measurement.  psgd_profile(s, 1) makes later psgd_step
 * calls record a CUDA event pair around every kernel they launch (on the
 * step's stream); 0 stops it.  psgd_profile_read synchronises the device,
 * then returns for kernel kind `kind` (0 .. psgd_profile_kinds()-1) its name,
 * the number of launches and the summed device time since the last read, and
 * the algorithmic bytes one launch must move (the roofline numerator); it
 * then clears that kind's record.  With launches and total_ms both NULL it
 * returns the name and bytes only and leaves the record.
 */
int psgd_profile(psgd_state* s, int32_t enable);
/*
 * psgd_profile_select -- as psgd_profile, for the kinds whose bit is set in
 * kind_mask only (bit k: kind k; 0 stops): a timed region that needs one
 * kernel's duration then carries two events per step, not two per kernel.
 * Returns PSGD_EINVAL for a NULL state.
 */
int psgd_profile_select(psgd_state* s, uint32_t kind_mask);
int32_t psgd_profile_kinds(void);
int psgd_profile_read(psgd_state* s, int32_t kind, const char** name, int64_t* launches,
                      double* total_ms, double* bytes_per_launch);

/*
 * psgd_project_q_static -- Q = M^T P for one matrix, allocating nothing.
 *
 * The pages have no counterpart: this entry point exists for callers that
 * cannot call cudaMalloc -- a job that reserved nearly all device memory up
 * front, code whose device memory must come from a framework's own
 * allocator, or latency-sensitive code that cannot afford cudaMalloc's
 * implicit synchronisation.  It computes what pass 2 of psgd_step computes
 * for one replica (Q(j, k) = sum_i M(i, j) P(i, k)), summing per block of
 * 512 rows in row order and then over the blocks in block order, with those
 * partial sums kept in a file-scope __device__ array of 2 Mi floats (8 MiB)
 * that every GPU loading this library holds until the process exits.
 *
 *   dev_m  : device pointer, rows x cols floats, row-major.
 *   dev_p  : device pointer, rows x rank floats, row-major.
 *   dev_q  : device pointer, cols x rank floats, row-major (output).
 *   rank   : 1 .. 32.
 *   stream : cudaStream_t; the work is enqueued on it.
 * Runs on the calling thread's current CUDA device; the first call on a
 * device looks up the array's device address (make that first call before
 * any stream capture).  Sizes with ceil(rows / 512) * next_pow2(rank) * cols
 * above 2 Mi return PSGD_EINVAL.  Every call overwrites the whole part of the
 * array it uses, so nothing carries over between calls, but calls that
 * overlap on the GPU (other streams, other threads) race on the array.
 * Errors: PSGD_EINVAL (NULL pointer, sizes), PSGD_ECUDA.
 */
int psgd_project_q_static(const float* dev_m, const float* dev_p, float* dev_q, int64_t rows,
                          int64_t cols, int32_t rank, void* stream);

/*
 * Bucket groups -- overlap across buckets.
 *
 * [DDP] "What Does a Communication Hook Operate On?": DDP splits the
 * gradients into buckets so that communication overlaps computation and calls
 * the hook once per bucket as it becomes ready; the PowerSGD state keeps its
 * error-feedback residuals and warm-start Qs per bucket.  A group holds one
 * psgd_state per bucket, all with the same hyper-parameters, and steps each
 * bucket on one of n_streams internal CUDA streams, so that one bucket's
 * latency-bound launches (Gram-Schmidt stage, reductions) run beside another
 * bucket's streaming passes.  The buckets' compressed tensors are numbered
 * across the group in bucket order for the Q draws, so a group draws the
 * same Qs as one state over the concatenated buckets.
 */
typedef struct psgd_group psgd_group; /* opaque, library-owned */

#define PSGD_MAX_GROUP_STREAMS 16

/*
 * psgd_group_create -- n_buckets buckets; bucket b holds tensors_per_bucket[b]
 * tensors, and dims/ndims list every tensor of every bucket in bucket order,
 * as psgd_state_create takes them for one bucket.  The other arguments are
 * psgd_state_create's and apply to every bucket; n_streams in [1, 16].
 * More than 8 streams overlap fully only when the process starts CUDA with
 * as many hardware work queues (CUDA_DEVICE_MAX_CONNECTIONS >= n_streams;
 * CUDA's default is 8) or replays the steps as graphs (psgd_set_graph).
 * Allocates every bucket's state and the streams on `device`.
 * Errors: PSGD_EINVAL, PSGD_ENOMEM, PSGD_ECUDA (nothing is left allocated).
 */
int psgd_group_create(int32_t n_buckets, const int32_t* tensors_per_bucket, const int64_t* dims,
                      const int32_t* ndims, int32_t world_size, int32_t matrix_approximation_rank,
                      int64_t start_powerSGD_iter, double min_compression_rate,
                      int32_t use_error_feedback, int32_t warm_start,
                      float orthogonalization_epsilon, uint64_t random_seed,
                      int32_t batch_tensors_with_same_shape, psgd_dtype grad_dtype,
                      int32_t n_streams, int32_t device, psgd_group** out);

/* Synchronises the group's streams and frees everything.  NULL is a no-op. */
void psgd_group_destroy(psgd_group* g);

/*
 * psgd_group_step -- psgd_step of bucket `bucket` (grads/out/inv_loss_scale
 * as there, sized for that bucket), enqueued on internal stream
 * bucket mod n_streams after the work enqueued so far on `stream`.  Returns
 * once enqueued; grads and out must stay valid until psgd_group_wait's
 * stream has reached the step.  Each bucket is stepped once per training
 * iteration, in any order.
 * Errors: psgd_step's, and PSGD_EINVAL for a bucket index out of range.
 */
int psgd_group_step(psgd_group* g, int32_t bucket, const void* const* grads, float* out,
                    float inv_loss_scale, void* stream);

/* Makes `stream` wait for every bucket step enqueued so far.  Enqueues only. */
int psgd_group_wait(psgd_group* g, void* stream);

/*
 * psgd_group_status -- psgd_group_wait, then synchronises `stream`:
 * PSGD_SKIPPED_NONFINITE if the last step of any bucket was skipped ([AMP]
 * inf/NaN; each bucket skips on its own inputs), else PSGD_OK.
 */
int psgd_group_status(psgd_group* g, void* stream);

/* Bucket b's state, owned by the group (introspection, Q and error views,
 * checkpointing); do not destroy it. */
int psgd_group_bucket(psgd_group* g, int32_t bucket, psgd_state** out);

/* Number of buckets (0 for NULL). */
int32_t psgd_group_size(const psgd_group* g);

/*
 * Data-parallel split of the step -- one replica per process.
 *
 * [DDP] "PowerSGD Hooks", powerSGD_hook: each worker computes its own
 * P = M_w Q and Q = M_w^T P, and the hook allreduces the uncompressed batch
 * (step 2), the Ps (step 3.3) and the Qs (step 3.6) across the workers;
 * "Default Communication Hooks", allreduce_hook: the result is the mean.
 * When each process (typically one per GPU) holds ONE replica, the linearity
 * fold that psgd_step uses for its W simulated replicas no longer applies,
 * and the step is split at its two exchanges:
 *
 *   psgd_dp_begin    pass 1 on the local replica: M = g * s + e, the local
 *                    P = M Q, the local uncompressed values and a skip flag,
 *                    all packed into one exchange buffer;
 *   (caller)         SUM-allreduce that buffer across the W processes;
 *   psgd_dp_project  P = sum / W, orthogonalise P, local Q = M^T P into a
 *                    second exchange buffer;
 *   (caller)         SUM-allreduce that buffer;
 *   psgd_dp_finish   Q = sum / W, out = P Q^T, uncompressed out = sum / W,
 *                    residual kept (factored), commit.
 *
 * The exchange buffers are library-owned device memory at fixed addresses
 * (psgd_dp_begin / psgd_dp_project return them with their float counts), so
 * the caller's collective (NCCL on device memory, or a host exchange through
 * a copy) reads and writes them in place; a SUM reduction with any
 * association order is expected.  The library itself makes no collective
 * call and reads no peer memory.  Every process must call the three stages
 * in order, step after step, with the same bucket layout and
 * hyper-parameters (random_seed included: the initial Q is drawn the same
 * on every process).  A non-finite input on any process raises that
 * process's flag in the exchanged buffer, so after the sum every process
 * skips the same step ([AMP]) and keeps its state bit-identical.  Before
 * start_powerSGD_iter the exchange buffer of psgd_dp_begin is `out` itself,
 * holding this replica's unscaled gradient (psgd_dp_project then returns
 * count 0), and psgd_dp_finish divides it by W; a non-finite sum skips.
 */

/*
 * psgd_dp_create -- the state of ONE process of a W-process data-parallel job
 * (W = world_size in [1, 64]).  Arguments as psgd_state_create; the state
 * holds this process's error-feedback residual (one replica) and the shared
 * factors.  psgd_step on it returns PSGD_EINVAL (use the three stages);
 * psgd_step_status, psgd_get_stats, psgd_tensor_info, psgd_set_q, psgd_get_q,
 * psgd_get_p, psgd_get_error / psgd_set_error (replica 0 = this process's),
 * psgd_workspace_bytes, psgd_profile* and psgd_state_destroy work as for any
 * state.  Errors: as psgd_state_create.
 */
int psgd_dp_create(const int64_t* dims, const int32_t* ndims, int32_t n_tensors, int32_t world_size,
                   int32_t matrix_approximation_rank, int64_t start_powerSGD_iter,
                   double min_compression_rate, int32_t use_error_feedback, int32_t warm_start,
                   float orthogonalization_epsilon, uint64_t random_seed,
                   int32_t batch_tensors_with_same_shape, psgd_dtype grad_dtype, int32_t device,
                   psgd_state** out);

/*
 * psgd_dp_begin -- first stage of one hook call on this process's replica.
 *   grad  : device pointer, this replica's flat bucket (N elements of
 *           grad_dtype); read here and, without error feedback, again by
 *           psgd_dp_project's kernels: keep it valid and unchanged until
 *           that call's work has run on `stream`.
 *   out   : device pointer, N floats, the bucket the hook returns (written
 *           by psgd_dp_finish; before start_powerSGD_iter also the exchange
 *           buffer).  Must not overlap grad unless grad == out (F32).
 *   inv_loss_scale, stream : as psgd_step.
 *   exchange, count : out; the device buffer (`count` floats) to
 *           SUM-allreduce across the W processes before psgd_dp_project.
 * Enqueues only.  Errors: PSGD_EINVAL (NULL pointers, stage out of order,
 * not a data-parallel state), PSGD_ECUDA.
 */
int psgd_dp_begin(psgd_state* s, const void* grad, float* out, float inv_loss_scale, void* stream,
                  float** exchange, int64_t* count);

/*
 * psgd_dp_project -- second stage, after the caller's SUM-allreduce of the
 * first exchange buffer: P = sum / W, Gram-Schmidt, local Q = M^T P.
 * exchange, count : out; the device buffer to SUM-allreduce before
 * psgd_dp_finish (count 0: nothing to exchange, as before
 * start_powerSGD_iter).  Enqueues only.  Errors: PSGD_EINVAL (stage out of
 * order), PSGD_ECUDA.
 */
int psgd_dp_project(psgd_state* s, void* stream, float** exchange, int64_t* count);

/*
 * psgd_dp_finish -- last stage, after the caller's SUM-allreduce of the
 * second exchange buffer (if any): Q = sum / W (the next warm-start Q),
 * out = P Q^T for the compressed tensors and the replica mean for the rest,
 * then the commit (or the skip).  psgd_step_status reports the outcome, the
 * same on every process.  Enqueues only.  Errors: PSGD_EINVAL (stage out of
 * order), PSGD_ECUDA.
 */
int psgd_dp_finish(psgd_state* s, void* stream);

/*
 * Training operators -- what fills the buckets.
 *
 * The gradients that psgd_step compresses come from a training step.  These
 * operators compute the parts of one that hang on a vocabulary and on the
 * normalisations between the matrix products: the embedding's lookup and the
 * dense gradient of its table, layer norm forward and backward, and
 * distillation from a teacher's top logits.  Each writes parameter gradients
 * straight into a caller's bucket: at any element offset, in the bucket's
 * type, replacing what is there or adding to it.
 *
 * Common to all of them:
 *   - dtype arguments name the type of the elements (F32, F16, BF16); all
 *     arithmetic and every sum is fp32, rounded once into an output.
 *   - strides are in elements and non-negative; rows are contiguous inside.
 *     Outputs may have any element alignment; operands whose addresses and
 *     strides are multiples of 16 bytes are accessed 16 bytes at a time.
 *   - an output may overlap no other operand unless the call says so; an
 *     operand reaches from its first to its last element, what lies between
 *     its rows included.
 *   - calls enqueue on `stream` and never synchronise; results are the same
 *     bits on every run on the same GPU model.
 */

/*
 * Embedding -- a table of `vocab` rows of `dim` elements.
 *
 * The handle holds the workspace of the gradient (the sorted tokens and the
 * partial rows) for up to max_tokens tokens a call, a lookup's among them;
 * calls on one handle must not overlap on the GPU (order them on one stream, or
 * with events).
 */
typedef struct psgd_embedding psgd_embedding; /* opaque, library-owned */

/* Errors: PSGD_EINVAL (vocab outside [1, 2^31 - 2], dim outside [1, 2^20],
 * max_tokens outside [0, 2^31 - 256], device above 63), PSGD_ENOMEM,
 * PSGD_ECUDA.  *out is NULL on failure. */
int psgd_embedding_create(int64_t vocab, int64_t dim, int64_t max_tokens, int32_t device, psgd_embedding** out);
void psgd_embedding_destroy(psgd_embedding* e); /* NULL is a no-op */
size_t psgd_embedding_workspace_bytes(const psgd_embedding* e);

/*
 * psgd_embedding_forward -- out_i = scale * weight[id_i].
 *
 *   weight : vocab rows, weight_stride apart.
 *   ids    : id_bits (32 or 64) bit signed integers, an (outer, inner) array:
 *            token (o, n) at o * ids_outer_stride + n * ids_inner_stride.
 *            An id outside [0, vocab) gives a row of zeros and is reported by
 *            psgd_embedding_status.
 *   out    : the tokens' rows, in the same (outer, inner) layout with strides
 *            of its own, either of which may be the larger one; rows must not
 *            overlap.
 * Errors: PSGD_EINVAL, PSGD_ECUDA.
 */
int psgd_embedding_forward(psgd_embedding* e, const void* weight, psgd_dtype weight_dtype, int64_t weight_stride,
                           const void* ids, int32_t id_bits, int64_t outer, int64_t inner,
                           int64_t ids_outer_stride, int64_t ids_inner_stride, float scale, void* out,
                           psgd_dtype out_dtype, int64_t out_outer_stride, int64_t out_inner_stride, void* stream);

/*
 * psgd_embedding_backward -- the gradient of the whole table:
 *   dweight_v = [dweight_v +] scale * sum over the tokens i with id_i = v of grad_i,
 * zero (or unchanged, with accumulate) for a row that no token names.
 *
 *   ids, grad   : as psgd_embedding_forward's ids and out; grad rows may
 *                 overlap (a broadcast gradient has stride 0).
 *   padding_idx : tokens with this id add nothing; -1: none.  Neither does an
 *                 id outside [0, vocab), which psgd_embedding_status reports.
 *   accumulate  : 0: dweight is overwritten; 1: added to.
 * Each row's sum runs over its tokens in position order, in pieces whose sums
 * are then added in a fixed order; where they are cut depends on the ids and the
 * token count alone (and on the GPU's multiprocessor count).
 * Errors: PSGD_EINVAL (more than max_tokens tokens among them), PSGD_ECUDA.
 */
int psgd_embedding_backward(psgd_embedding* e, const void* ids, int32_t id_bits, int64_t outer, int64_t inner,
                            int64_t ids_outer_stride, int64_t ids_inner_stride, const void* grad,
                            psgd_dtype grad_dtype, int64_t grad_outer_stride, int64_t grad_inner_stride,
                            float scale, int64_t padding_idx, int32_t accumulate, void* dweight,
                            psgd_dtype dweight_dtype, int64_t dweight_stride, void* stream);

/* Synchronises `stream`; PSGD_BAD_TOKEN if a call enqueued on it since the last
 * status call (or creation) met an id outside the table, else PSGD_OK. */
int psgd_embedding_status(psgd_embedding* e, void* stream);

/*
 * Layer norm over rows of `dim` elements.  The handle holds the partial sums
 * of the parameters' gradients; backward calls on one handle must not overlap
 * on the GPU, forward calls may.
 */
typedef struct psgd_layernorm psgd_layernorm; /* opaque, library-owned */

/* Errors: PSGD_EINVAL (dim outside [1, 2^20], device above 63), PSGD_ENOMEM,
 * PSGD_ECUDA.  *out is NULL on failure. */
int psgd_layernorm_create(int64_t dim, int32_t device, psgd_layernorm** out);
void psgd_layernorm_destroy(psgd_layernorm* n); /* NULL is a no-op */
size_t psgd_layernorm_workspace_bytes(const psgd_layernorm* n);

/*
 * psgd_layernorm_forward -- y = (x - mean) rstd weight + bias per row, with
 * rstd = (mean((x - mean)^2) + eps)^-1/2.
 *
 *   x, y         : `rows` rows (at most 2^30) of `dtype`, x_stride / y_stride
 *                  apart.
 *   weight, bias : dim elements of param_dtype; NULL: 1 and 0.
 *   mean, rstd   : out, one float a row (what the backward pass takes); may be
 *                  NULL.
 * The variance is a sum of squares in fp32: deviations below about 1e-19 count
 * as none (then rstd is eps^-1/2, infinite without an eps), above 1e19 they
 * overflow it (rstd 0).  The backward pass takes any mean and rstd.
 * Errors: PSGD_EINVAL, PSGD_ECUDA.
 */
int psgd_layernorm_forward(psgd_layernorm* n, const void* x, psgd_dtype dtype, int64_t x_stride, int64_t rows,
                           const void* weight, const void* bias, psgd_dtype param_dtype, float eps, void* y,
                           int64_t y_stride, float* mean, float* rstd, void* stream);

/*
 * psgd_layernorm_backward -- with xh = (x - mean) rstd and a = grad weight:
 *   dx      = rstd (a - mean(a) - xh mean(a xh))
 *   dweight = [dweight +] sum over rows of grad xh
 *   dbias   = [dbias +]   sum over rows of grad
 *
 *   grad, x, dx    : `rows` rows of `dtype`; dx may be NULL.
 *   weight         : dim elements of param_dtype; NULL: 1.
 *   dweight, dbias : dim elements of dparam_dtype; either may be NULL.  With
 *                    no rows they become 0 (unchanged with accumulate).
 * Errors: PSGD_EINVAL, PSGD_ECUDA.
 */
int psgd_layernorm_backward(psgd_layernorm* n, const void* grad, int64_t grad_stride, const void* x,
                            psgd_dtype dtype, int64_t x_stride, int64_t rows, const float* mean, const float* rstd,
                            const void* weight, psgd_dtype param_dtype, void* dx, int64_t dx_stride, void* dweight,
                            void* dbias, psgd_dtype dparam_dtype, int32_t accumulate, void* stream);

#define PSGD_DISTILL_MAX_K 1024 /* teacher entries per row */

/*
 * psgd_distill -- distillation of a student from a teacher's top logits.
 * For every row, with T = temperature:
 *   p_k     = softmax over the row's valid entries of teacher_k / T,
 *   q       = softmax over the vocabulary of logits / T,
 *   loss    = w T^2 sum_k p_k (log p_k - log q[index_k]),
 *   dlogits = grad_scale w T (q_j - sum over the k with index_k = j of p_k).
 *
 *   logits  : `rows` rows (below 2^28) of `vocab` elements (at most 2^30) of
 *             `dtype`.
 *   teacher, index : `rows` rows of k teacher logits and of the vocabulary
 *             entries (index_bits 32 or 64) they belong to.  An entry whose
 *             index lies outside [0, vocab) is not valid: a row with fewer
 *             than k entries is filled up with -1.  Equal indices add up.
 *             The largest valid logit of a row comes off before the division by
 *             T: only -infinity has no mass.
 *   weights : w, one float a row (a loss mask, or 1 / tokens); NULL: 1.
 *   losses  : out, one float a row.
 *   dlogits : out, rows of `dtype`; NULL: the losses only.  May be logits
 *             itself (same stride).
 * A row with w = 0, or with no valid entry whose teacher logit is above
 * -infinity, has loss 0 and gradient 0 whatever its logits hold.  Otherwise
 * a logit of -infinity has q_j = 0 (the loss is infinite if the teacher wants
 * it), and NaN, +infinity or a row of nothing but -infinity gives NaN.
 *   device  : the CUDA device that holds the operands.
 * Errors: PSGD_EINVAL, PSGD_ECUDA.
 */
int psgd_distill(const void* logits, psgd_dtype dtype, int64_t logits_stride, int64_t rows, int64_t vocab,
                 const void* teacher, psgd_dtype teacher_dtype, int64_t teacher_stride, const void* index,
                 int32_t index_bits, int64_t index_stride, int32_t k, float temperature, const float* weights,
                 float grad_scale, float* losses, void* dlogits, int64_t dlogits_stride, int32_t device, void* stream);

/*
 * Activations in 8 bits.  Every row is cut into blocks of 128 elements (the last
 * one may be shorter); a block has one fp32 scale, a power of two:
 *   scale = the least 2^e, e >= -126, with |x| <= M 2^e for the block's finite
 *           values (M = 448 for e4m3, 57344 for e5m2); 1 for a block of zeros
 *   code  = x / scale rounded to the format, ties to even (one rounding of x).
 * NaN becomes NaN; an infinity stays one in e5m2 and becomes NaN in e4m3.
 * `codes` are rows of dim bytes, `scales` rows of ceil(dim / 128) floats, both
 * without gaps.
 */

/*
 * psgd_activation_save -- codes and scales of `rows` rows of `dim` elements.
 * device : the CUDA device that holds the operands.
 * Errors: PSGD_EINVAL (rows above 2^30, dim above 2^30 among them), PSGD_ECUDA.
 */
int psgd_activation_save(const void* x, psgd_dtype dtype, int64_t x_stride, int64_t rows, int64_t dim, void* codes,
                         psgd_code code, float* scales, int32_t device, void* stream);

/*
 * psgd_activation_restore -- out = code * scale, rounded to out's type (exact in
 * fp32, and in bf16 but for its subnormals).  The scales may be any floats.
 * Errors: PSGD_EINVAL, PSGD_ECUDA.
 */
int psgd_activation_restore(const void* codes, psgd_code code, const float* scales, int64_t rows, int64_t dim,
                            void* out, psgd_dtype dtype, int64_t out_stride, int32_t device, void* stream);

/*
 * Root-mean-square norm over rows of `dim` elements.  The handle holds the partial
 * sums of the weight's gradient; backward calls on one handle must not overlap
 * on the GPU, forward calls may.
 */
typedef struct psgd_rmsnorm psgd_rmsnorm; /* opaque, library-owned */

/* Errors: PSGD_EINVAL (dim outside [1, 2^20], device above 63), PSGD_ENOMEM,
 * PSGD_ECUDA.  *out is NULL on failure. */
int psgd_rmsnorm_create(int64_t dim, int32_t device, psgd_rmsnorm** out);
void psgd_rmsnorm_destroy(psgd_rmsnorm* n); /* NULL is a no-op */
size_t psgd_rmsnorm_workspace_bytes(const psgd_rmsnorm* n);

/*
 * psgd_rmsnorm_forward -- per row
 *   s = x + residual, rounded to dtype,   rstd = (mean(s^2) + eps)^-1/2,   y = s rstd weight.
 *
 *   x, residual, y, summed : `rows` rows (at most 2^30) of `dtype`, strides of their own.
 *   residual : NULL: s = x.
 *   weight   : dim elements of param_dtype; NULL: 1.
 *   y        : out; or NULL, with
 *   codes, scales : out, y in 8 bits (from its fp32 value, without a rounding to
 *              dtype before).
 *   summed   : out, s (what the backward pass takes); may be NULL, or x or
 *              residual itself (same stride).
 *   rstd     : out, one float a row.
 * The sum of squares is fp32: |s| above 1e19 overflows it (rstd 0).
 * Errors: PSGD_EINVAL, PSGD_ECUDA.
 */
int psgd_rmsnorm_forward(psgd_rmsnorm* n, const void* x, psgd_dtype dtype, int64_t x_stride, int64_t rows,
                         const void* residual, int64_t residual_stride, const void* weight, psgd_dtype param_dtype,
                         float eps, void* y, int64_t y_stride, void* codes, psgd_code code, float* scales, void* summed,
                         int64_t summed_stride, float* rstd, void* stream);

/*
 * psgd_rmsnorm_backward -- with xh = s rstd and a = grad weight:
 *   dx      = rstd (a - xh mean(a xh)) [+ grad_summed]
 *   dweight = [dweight +] sum over rows of grad xh
 * dx is the gradient of x and of residual.
 *
 *   grad, grad_summed, dx : `rows` rows of `dtype`.
 *   summed        : s, of `dtype`; or NULL, with
 *   codes, scales : s in 8 bits (psgd_activation_save).
 *   grad_summed   : the gradient that reaches s past the norm; may be NULL.
 *   dx            : out; may be NULL, or grad or grad_summed itself (same stride).
 *   dweight       : out, dim elements of dparam_dtype; may be NULL.  Without rows it
 *                   becomes 0 (unchanged with accumulate).
 * Errors: PSGD_EINVAL, PSGD_ECUDA.
 */
int psgd_rmsnorm_backward(psgd_rmsnorm* n, const void* grad, psgd_dtype dtype, int64_t grad_stride, int64_t rows,
                          const void* summed, int64_t summed_stride, const void* codes, psgd_code code,
                          const float* scales, const float* rstd, const void* weight, psgd_dtype param_dtype,
                          const void* grad_summed, int64_t grad_summed_stride, void* dx, int64_t dx_stride,
                          void* dweight, psgd_dtype dparam_dtype, int32_t accumulate, void* stream);

/*
 * The weight gradient of a linear layer y = x W^T from its input's 8-bit
 * checkpoint, on the tensor cores.  The handle holds the restored checkpoint
 * (2 bytes for max_rows x ins), a piece of a gradient that TMA cannot read where it lies (an address or row stride
 * that is no multiple of 16 bytes, rows that overlap): at most 32 MB, or 512 MB where outs is no multiple of 8 (or 256 columns),
 * and a product's partial sums (512 KB for every two SMs).  Calls on one handle must not overlap on the GPU.
 */
typedef struct psgd_wgrad psgd_wgrad; /* opaque, library-owned */

/* outs, ins : rows and columns of W.  max_rows : rows of one call at most.
 * Errors: PSGD_EINVAL (features outside [1, 2^20], max_rows outside [0, 2^24],
 * device above 63), PSGD_ENOMEM, PSGD_ECUDA.  *out is NULL on failure. */
int psgd_wgrad_create(int64_t outs, int64_t ins, int64_t max_rows, int32_t device, psgd_wgrad** out);
void psgd_wgrad_destroy(psgd_wgrad* w); /* NULL is a no-op */
size_t psgd_wgrad_workspace_bytes(const psgd_wgrad* w);

/*
 * psgd_wgrad_backward -- dweight = [dweight +] grad^T x, with x = codes * scales
 * (psgd_activation_save) rounded to grad's type (exact in bf16; in f16 while it is in
 * range).
 *
 *   grad          : `rows` rows of outs elements, F16 or BF16 (the products are of
 *                   16-bit operands; sums are fp32).
 *   codes, scales : `rows` rows of ins elements.
 *   dweight       : outs rows of ins elements, dweight_stride apart, at any
 *                   element offset.  Without rows it becomes 0 (unchanged with
 *                   accumulate).
 * Errors: PSGD_EINVAL, PSGD_ECUDA.
 */
int psgd_wgrad_backward(psgd_wgrad* w, const void* grad, psgd_dtype dtype, int64_t grad_stride, int64_t rows,
                        const void* codes, psgd_code code, const float* scales, void* dweight,
                        psgd_dtype dweight_dtype, int64_t dweight_stride, int32_t accumulate, void* stream);

/* Synchronises `stream`; PSGD_ETIMEOUT if a bounded wait of a call enqueued on it gave
 * up since the last status call (its results are not valid), else PSGD_OK. */
int psgd_wgrad_status(psgd_wgrad* w, void* stream);

/*
 * Softmax cross entropy of a linear output layer, without its logits.
 *
 * The handle holds
 *   the tokens that count, twice in their type and once in fp32 (8 bytes for max_tokens x dim),
 *   a piece of the logits' gradient of at most 256 MB (or 256 columns of the vocabulary where those take more),
 *   a piece of a weight that TMA cannot read where it lies (an address or row stride that is no multiple of 16
 *   bytes, rows that overlap): at most 32 MB, or 256 MB where dim is no multiple of 8 (or 256 rows),
 *   partial sums: 512 KB for every two SMs, and eight bytes for every 128 logits;
 * 80 MB for one token of 50257 x 1600, 402 MB for 8192.  Calls on one handle must not overlap on the GPU.
 */
typedef struct psgd_linear_ce psgd_linear_ce; /* opaque, library-owned */

/* Errors: PSGD_EINVAL (vocab outside [1, 2^24], dim outside [1, 2^20], max_tokens
 * outside [0, 2^20], device above 63), PSGD_ENOMEM, PSGD_ECUDA.  *out is NULL on failure. */
int psgd_linear_ce_create(int64_t vocab, int64_t dim, int64_t max_tokens, int32_t device, psgd_linear_ce** out);
void psgd_linear_ce_destroy(psgd_linear_ce* c); /* NULL is a no-op */
size_t psgd_linear_ce_workspace_bytes(const psgd_linear_ce* c);

/*
 * psgd_linear_ce_forward -- for every token t, with z_tv = hidden_t . weight_v:
 *   lse_t    = log sum_v exp(z_tv),
 *   losses_t = w_t (lse_t - z_t,target).
 *
 *   hidden  : `tokens` rows of dim elements, F16 or BF16 (the products are of
 *             16-bit operands; sums are fp32).
 *   weight  : vocab rows of dim elements of the same type.
 *   targets : target_bits (32 or 64) bit signed integers, without gaps.
 *   weights : w, one float a token; NULL: 1.
 *   losses, lse : out, one float a token (lse is what the backward pass takes).
 * A token with a target outside [0, vocab) or with w = 0 does not count: its
 * loss and lse are 0 whatever its row holds, and it costs no arithmetic.  NaN or
 * +infinity among a row's logits gives NaN.
 * Errors: PSGD_EINVAL, PSGD_ECUDA.
 */
int psgd_linear_ce_forward(psgd_linear_ce* c, const void* hidden, psgd_dtype dtype, int64_t hidden_stride, int64_t tokens,
                           const void* weight, int64_t weight_stride, const void* targets, int32_t target_bits,
                           const float* weights, float* losses, float* lse, void* stream);

/*
 * psgd_linear_ce_backward -- with G_tv = grad_scale w_t (exp(z_tv - lse_t) - [v = target_t]):
 *   dhidden_t = sum_v G_tv weight_v
 *   dweight_v = [dweight_v +] sum_t G_tv hidden_t
 * The logits are computed again.  exp(z - lse) - [v = target], times r_t, is rounded
 * once to the operands' type before both products, where w_t = s r_t 2^e with s the
 * significand of the largest weight and 1 <= |r_t| < 2; hidden_t takes the power of two,
 * relative to the largest.  At the target it is exp(z - lse) - 1 without a cancellation but that of lse's own
 * rounding (z is the forward pass's), so a likely target's 1 - p is there to 2^-24 |lse|.
 *
 *   hidden, weight, targets, weights : as in the forward pass; lse: its output.
 *   dhidden : out, rows of the operands' type; may be NULL.  0 for a token that
 *             does not count.
 *   dweight : out, vocab rows of dim elements, at any element offset; may be NULL.
 * Errors: PSGD_EINVAL, PSGD_ECUDA.
 */
int psgd_linear_ce_backward(psgd_linear_ce* c, const void* hidden, psgd_dtype dtype, int64_t hidden_stride,
                            int64_t tokens, const void* weight, int64_t weight_stride, const void* targets,
                            int32_t target_bits, const float* lse, const float* weights, float grad_scale, void* dhidden,
                            int64_t dhidden_stride, void* dweight, psgd_dtype dweight_dtype, int64_t dweight_stride,
                            int32_t accumulate, void* stream);

/* As psgd_wgrad_status. */
int psgd_linear_ce_status(psgd_linear_ce* c, void* stream);

/*
 * psgd_build_id -- "psgd-source-hash:" followed by the SHA-256 (32 hex
 * digits) of the sources, header, flags and compiler version this library
 * was built from, so that a caller can check that the loaded binary matches
 * its sources.  The string is static.
 */
const char* psgd_build_id(void);

/* Message of the last failing call on this thread ("" if none). */
const char* psgd_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* PSGD_H */
