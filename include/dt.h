/*
 * dt.h -- collectives among P logical ranks that share one GPU.
 *
 * The operation set is the ThreadGroup collective set of the DTorch developer
 * guide page "集合通信组件" (collective communication component): §2.1 lists
 * the ThreadGroup methods (AllReduce, AllGatherIntoTensor, AllGather with
 * uneven shards, ReduceScatterTensor, AllToAll, Barrier) and §2.3 describes
 * ThreadGroupSameDeviceBackend, the backend used when every rank of the group
 * lives on the same GPU.  On top of that set come the fused gradient-bucket
 * all-reduce with 1/P scaling of "异步融合 AllReduce 流水线优化" (MindSpore
 * hyper-parallel issue #120, AllReduceParamGroup) and the notify/wait barrier
 * of "Barrier：仅信号（Signals Only）" (PyPTO distributed tutorial).
 *
 * Group-wide calls.  One call carries every rank's buffer (rank ==
 * DT_ALL_RANKS, pointer arrays with P entries) and runs as one kernel that
 * reads all P rank buffers directly from HBM.
 *
 * Rank-local calls.  As in DTorch, where every rank is a host thread that
 * calls ThreadGroup with its own tensor, each of P threads may call with
 * rank = its rank (0..P-1), one-entry pointer arrays and its own stream.  The
 * ranks meet on the host the way the MemoryTensorStore of §3.4 does (mutex,
 * condition variable, CUDA events): each rank records a ready event on its
 * stream, the last rank to arrive makes its stream wait on the others' ready
 * events and launches the one group-wide kernel, and every other rank's
 * stream waits on that launch's done event, so results are valid in each
 * rank's own stream order.  All ranks of a round must make the same call
 * (same collective, sizes, dtype, op, flags; AllGather's rows are each
 * rank's own) or every rank gets DT_ERR_INVALID.  A rank whose partners do
 * not all arrive within the group's time limit gets DT_ERR_TIMEOUT and the
 * group is poisoned until dt_group_reset.  Ranks of one group must not mix
 * rank-local and group-wide calls within a round.  dt_bucket_allreduce, the
 * layer norm and the vocabulary loss are group-wide only.
 *
 * Conventions shared by every entry point:
 *   Streams   `stream` is a cudaStream_t passed as void* (NULL = the legacy
 *             default stream).  A call enqueues its work on `stream` and
 *             returns without waiting for the GPU, like a collective in
 *             synchronous mode on the PyTorch page "通信与互联（05）" §四.2:
 *             results are valid in stream order.  Inputs must be produced in
 *             stream order, or the caller makes `stream` wait on an event.
 *   Buffers   Device pointers.  The caller owns them and keeps them alive
 *             until `stream` has passed the call (§五.5 of the same page).
 *             The group owns only its signal window, error word and bucket
 *             plan scratch.  dt_group_create allocates them; the plan scratch
 *             grows only when a bucket plan outgrows it or when every plan
 *             slot is pinned by a CUDA graph (see "CUDA graphs" below).
 *   Alignment Any alignment is accepted.  When every pointer and size is a
 *             multiple of 16 bytes the kernels move 16-byte vectors; otherwise
 *             they fall back to element-wise access with identical results.
 *   Errors    Argument errors are reported before anything is enqueued.  A
 *             device-side wait that runs out of time records DT_ERR_TIMEOUT
 *             in the group's error word; that code is returned by the next
 *             call on the group (and by dt_group_check), and the group then
 *             refuses work until dt_group_reset.  No call throws.
 *   Numerics  fp32 and bf16 reduce in fp32 registers, combining ranks in
 *             ascending rank order (rank 0 first, as the same-device
 *             AllReduce adds ranks 1..P-1 onto rank 0's tensor in order); bf16
 *             is rounded once, to nearest even, at the store; AVG divides the
 *             fp32 sum by P with IEEE division; int32 sums wrap modulo 2^32;
 *             MAX/MIN select an input element (a NaN wins; on equal values
 *             the lower rank's element is kept).
 */
#ifndef DT_H
#define DT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct dt_group *dt_group_t;
typedef struct dt_work *dt_work_t;

typedef enum {
    DT_OK = 0,
    DT_ERR_INVALID = 1,      /* bad argument; nothing was enqueued */
    DT_ERR_UNSUPPORTED = 2,  /* legal request the library does not support (AVG on int32, ...) */
    DT_ERR_CUDA = 3,         /* a CUDA runtime call failed */
    DT_ERR_TIMEOUT = 4,      /* a device-side wait ran out of time (see dt_group_check) */
    DT_ERR_OOM = 5,          /* the group could not allocate its own state */
    DT_ERR_POISONED = 6,     /* an earlier timeout left the group unusable until reset */
    DT_ERR_TOO_LARGE = 7,    /* request exceeds the fixed scratch of dt_bucket_allreduce_static */
    DT_NOT_READY = 8         /* dt_work_query: the work has not finished yet (not an error) */
} dt_status;

typedef enum { DT_F32 = 0, DT_BF16 = 1, DT_I32 = 2 } dt_dtype;

/* ReduceOpType of the ThreadGroup interface: kSum, kAvg, kMax, kMin.
 * DT_SUM_STEPWISE is the literal `result += DestGet(rank)` of the same-device
 * AllReduce ("集合通信组件" §2.3): ranks added in ascending order with every
 * add rounded to the element type, so bf16 rounds after each rank instead of
 * once at the end; for fp32 and int32 it equals DT_SUM. */
typedef enum { DT_SUM = 0, DT_AVG = 1, DT_MAX = 2, DT_MIN = 3, DT_SUM_STEPWISE = 4 } dt_redop;

#define DT_MAX_RANKS 16
#define DT_ALL_RANKS (-1)
/* Flag: every out[] entry names the same buffer; the result is written once.
 * The same-device AllReduce hands all ranks one shared result tensor. */
#define DT_SHARED_OUTPUT 0x1u
/* Default bucket cap: DDP's bucket_cap_mb = 25, read as 25 MiB. */
#define DT_DEFAULT_BUCKET_CAP_BYTES ((size_t)25 << 20)

/* Environment switches, read once per process:
 *   DT_TIMEOUT_MS  limit of every device wait and host rendezvous, in ms
 *                  (default 2000; read by dt_group_create)
 *   DT_LOG=1       every kernel launch and bucket plan is printed to stderr
 *   DT_PDL=0       kernels are launched without programmatic dependent launch
 *   DT_DEBUG=1     every launch is followed by a synchronisation of its stream
 *                  (not while the stream is being captured), so a kernel that
 *                  fails is reported by the call that launched it */

/* ------------------------------------------------------------------ groups */

/* Create a group of world_size (1..DT_MAX_RANKS) logical ranks on CUDA device
 * cuda_device.  Allocates the P x P int32 signal window, the error word and
 * two 1 MiB bucket-plan slots on that device; later calls allocate nothing
 * except a bucket all-reduce whose plan needs a larger or an extra slot.
 * The device-side wait limit is read from the environment variable
 * DT_TIMEOUT_MS (default 2000).  Like the TensorStore constructor, which
 * starts all participants from one state, the window starts at zero.
 * Returns DT_ERR_INVALID for a bad size or NULL out, DT_ERR_CUDA / DT_ERR_OOM
 * on a failed CUDA call (nothing is leaked). */
dt_status dt_group_create(int world_size, int cuda_device, dt_group_t *out);

/* Wait for the group's outstanding work, then free everything it owns. */
dt_status dt_group_destroy(dt_group_t g);

/* TensorStore::Reset analogue: zero the signal window and the error word on
 * `stream`, wait for that stream, clear the poisoned state and restart the
 * barrier generation at 0.  Blocks the calling thread. */
dt_status dt_group_reset(dt_group_t g, void *stream);

/* Report the first device-side error recorded so far without synchronising:
 * DT_OK, or the recorded code (the group is poisoned from then on).
 * rank/peer/generation of the failed wait are returned when the pointers are
 * not NULL. */
dt_status dt_group_check(dt_group_t g);
dt_status dt_group_error_detail(dt_group_t g, int *rank, int *peer, int *generation);

/* Number of ranks; number of barrier launches issued on the host since
 * create/reset (a barrier captured in a CUDA graph counts once, however
 * often the graph replays; the device-side generations live in the window). */
int dt_group_size(dt_group_t g);
int64_t dt_group_generation(dt_group_t g);

/* Change the device-side wait limit of later calls (milliseconds, >= 1). */
dt_status dt_group_set_timeout_ms(dt_group_t g, uint32_t timeout_ms);

const char *dt_status_string(dt_status st);

/* Kernels this library has launched in this process (all groups). */
uint64_t dt_launch_count(void);

/* CUDA graphs: group-wide calls may be captured in a stream capture.  Every
 * collective passes its rank pointers in the kernel's parameter block, and the
 * barrier keeps each rank's generation on the device, so replays advance the
 * window as eager calls would.  Make one eager call of each collective before
 * capturing it (the first call sets kernel attributes and caches launch
 * shapes).  A bucket all-reduce can be captured only after an eager call with
 * the same gradients, counts, dtype, op and cap (building a plan may allocate;
 * otherwise the call returns DT_ERR_UNSUPPORTED).  The captured call pins that
 * plan in the group: later bucket calls with other arguments use other plan
 * slots, so the graph keeps replaying against its own plan.  The group must
 * outlive every graph that holds its calls.  Rank-local calls meet on the host
 * and are not meant for capture. */

/* ------------------------------------------------------------- collectives */

/* AllReduce (P -> R): "集合通信组件" §2.1 AllReduce(input, reduceOpType) and
 * the three-phase same-device AllReduce of §2.3.
 *   in[r]   rank r's `count` elements of `dtype` (P entries)
 *   out[q]  rank q's result, `count` elements (P entries); out[q] may equal
 *           in[q] (in place).  With DT_SHARED_OUTPUT all out[] are one buffer
 *           written once; it may not overlap any input.
 * out[q][i] = scale( in[0][i] op in[1][i] op ... op in[P-1][i] ), scale = 1/P
 * for DT_AVG.  DT_AVG on DT_I32 -> DT_ERR_UNSUPPORTED. */
dt_status dt_allreduce(dt_group_t g, int rank, const void *const *in, void *const *out,
                       size_t count, int dtype, int op, unsigned flags, void *stream);

/* ReduceScatter (P -> S(0)): "集合通信组件" §2.1 ReduceScatterTensor.
 *   in[r]   rank r's P * recv_count elements: shard s is elements
 *           [s * recv_count, (s + 1) * recv_count) (dim 0 split evenly)
 *   out[r]  recv_count elements: the reduction over all ranks of shard r.
 * Outputs may not overlap inputs. */
dt_status dt_reduce_scatter(dt_group_t g, int rank, const void *const *in, void *const *out,
                            size_t recv_count, int dtype, int op, void *stream);

/* AllGather (S(0) -> R): "集合通信组件" §2.1 AllGatherIntoTensor (equal
 * shards, rows == NULL: every rank has rows_equal rows) and AllGather with
 * uneven shards (rows[r] rows on rank r).  In a rank-local call rows must be
 * NULL and rows_equal is the calling rank's own row count.  Rows are row_bytes bytes; rank r's
 * rows land at row offset rows[0] + ... + rows[r-1] of every out[q], which
 * holds the sum of all rows.  With DT_SHARED_OUTPUT every out[] is one buffer
 * written once.  Byte copies: any element type. */
dt_status dt_all_gather(dt_group_t g, int rank, const void *const *in, void *const *out,
                        const size_t *rows, size_t rows_equal, size_t row_bytes,
                        unsigned flags, void *stream);

/* AllToAll (S -> S, split and concatenated along dim 0): "集合通信组件"
 * §2.1 AllToAll.  in[i] is P chunks of chunk_bytes; chunk j of rank i goes
 * to rank j, which stacks what it receives in ascending source rank:
 *   out[j][i * chunk_bytes + k] = in[i][j * chunk_bytes + k]. */
dt_status dt_all_to_all(dt_group_t g, int rank, const void *const *in, void *const *out,
                        size_t chunk_bytes, void *stream);

/* ReplicateToShard (R -> S): "集合通信组件" §2.1 ReplicateToShard(input,
 * shardIdx) and the R -> S entry of the §2.5 placement matrix.  Every rank
 * holds the whole tensor (rows rows of row_bytes bytes, rows a multiple of
 * P); rank r keeps row block shard_idx[r] (NULL: block r) of the P equal
 * blocks: out[r] = in[r][shard_idx[r] * rows/P, (shard_idx[r] + 1) * rows/P).
 * Byte copies.  Rank-local: shard_idx points at the calling rank's own index
 * (NULL: its rank).  The sub-split coordinate of the page (nested meshes) is
 * not modelled. */
dt_status dt_replicate_to_shard(dt_group_t g, int rank, const void *const *in, void *const *out,
                                const int *shard_idx, size_t rows, size_t row_bytes, void *stream);

/* AllGatherIntoVec (S -> R, kept apart): "集合通信组件" §2.1
 * AllGatherIntoVec: every rank receives every rank's shard as a tensor of
 * its own.  out has P * P entries; out[q * P + r] (rows[r] rows, or
 * rows_equal when rows is NULL, of row_bytes bytes) receives rank r's shard
 * on rank q.  Rank-local: out has the calling rank's P entries, rows must be
 * NULL and rows_equal is the rank's own row count. */
dt_status dt_all_gather_into_vec(dt_group_t g, int rank, const void *const *in, void *const *out,
                                 const size_t *rows, size_t rows_equal, size_t row_bytes,
                                 void *stream);

/* AllToAll(srcDim, destDim) (S(src_dim) -> S(dest_dim)): "集合通信组件"
 * §2.1 AllToAll(input, srcDim, destDim) on 2-D tensors of R x C elements of
 * elem_bytes bytes (row-major).  Rank i splits its tensor along dest_dim into
 * P equal parts (h x w: R/P x C or R x C/P); part j goes to rank j, which
 * concatenates the parts it receives along src_dim in ascending source rank:
 * out[j] is (P h) x w for src_dim 0 and h x (P w) for src_dim 1.
 * (0, 0) is dt_all_to_all with chunk_bytes = R/P * C * elem_bytes. */
dt_status dt_all_to_all_2d(dt_group_t g, int rank, const void *const *in, void *const *out,
                           size_t R, size_t C, size_t elem_bytes, int src_dim, int dest_dim,
                           void *stream);

/* Fused gradient-bucket all-reduce: "异步融合 AllReduce 流水线优化"
 * (AllReduceParamGroup.issue_async_allreduce / wait_and_apply_grads: SUM
 * all-reduce of the fused gradient buffer, each gradient view then divided by
 * the replicate world size for AVG) with the bucketing of "通信与互联（05）"
 * §六.5 (DDP gathers gradients into bucket_cap_mb = 25 MB buckets).
 *   grads[t * P + p]  rank p's gradient t, counts[t] elements, updated in place
 *   dtype             DT_BF16 or DT_F32;  op  DT_SUM or DT_AVG
 *   bucket_cap_bytes  0 -> DT_DEFAULT_BUCKET_CAP_BYTES
 * Tensors are grouped in order into buckets (dt_bucket_plan); each bucket is
 * one kernel that reads and writes the gradients in place through a chunk
 * table (no flatten copy), and one signal-window barrier (the notify / wait
 * of dt_barrier, one generation each) runs between consecutive buckets: in an
 * extra last block of the earlier bucket's kernel, which waits until that
 * bucket's other blocks have finished.  The next bucket's kernel stores
 * nothing before that whole kernel has completed (its first blocks load
 * their first gradients while it drains: tensors no kernel of the call has
 * written yet).  The plan table is staged through the group's scratch; at
 * most one bucket call per group may be in flight. */
dt_status dt_bucket_allreduce(dt_group_t g, void *const *grads, const size_t *counts,
                              size_t n_tensors, int dtype, int op, size_t bucket_cap_bytes,
                              void *stream);

/* The bucket plan used above, on the host only (no GPU needed): greedy in the
 * given order, a bucket closes when the next tensor would take it past
 * cap_bytes, a tensor larger than the cap gets a bucket of its own.
 * bucket_of[t] receives tensor t's bucket; *n_buckets the bucket count. */
dt_status dt_bucket_plan(const size_t *counts, size_t n_tensors, size_t elem_bytes,
                         size_t cap_bytes, size_t *bucket_of, size_t *n_buckets);

/* Signal-window barrier: "Barrier：仅信号（Signals Only）".  The group keeps
 * an int32 window win[P][P] in HBM (row r of rank q's window is win[q][r]).
 * The g-th barrier (1-based generation, bumped by every call) is one kernel
 * in which each rank is one warp: rank r adds 1 (AtomicAdd) to win[q][r] of
 * every peer q != r, then waits until win[r][s] >= g (Ge) for every s != r.
 * Afterwards win[r][s] == g for s != r and win[r][r] == 0.  Stream order
 * orders the data around the barrier kernel, so its adds and polls are
 * relaxed GPU-scope atomics and loads.  Each wait gives up after the group's
 * time limit and records DT_ERR_TIMEOUT. */
dt_status dt_barrier(dt_group_t g, int rank, void *stream);

/* Allocation-free fused bucket all-reduce.  The pages have no counterpart:
 * this entry point exists for callers that cannot let a library allocate
 * device memory -- applications that own all device memory through their own
 * pool (a library's cudaMalloc escapes their accounting and can fail once the
 * pool has taken the device) and code on a latency-critical path that must
 * not stall other streams (cudaMalloc and cudaFree can synchronise the whole
 * device).  Such callers cannot create a dt_group.
 *   world_size        P (1..DT_MAX_RANKS); no group is needed
 *   grads, counts, n_tensors, dtype, op, bucket_cap_bytes, stream
 *                     as dt_bucket_allreduce; the results are identical
 * The tensor and pointer tables live in one fixed 1 MiB device array inside
 * this library (every GPU that loads the library holds it until the process
 * exits) and are staged from a fixed host array: the call allocates nothing.
 * Tables that do not fit (n_tensors * (P * 8 + 24) bytes plus 4 bytes per
 * thread block of every bucket: one block per 2048 bf16 or 1024 fp32
 * elements of each tensor, at most 16 per resident block slot, so about 40
 * full 25 MiB buckets) or more than 4096 buckets return DT_ERR_TOO_LARGE before anything
 * is enqueued.  Every call shares the array and leaves its contents behind;
 * calls that overlap on the GPU (unordered streams) race on it, calls on one
 * stream do not.  A call whose tables differ from the last ones copied to
 * this device copies them with a pageable cudaMemcpyAsync, which CUDA may
 * finish only after the work already queued on `stream`, so such a call can
 * block the host until then; a call that repeats the previous call's
 * gradients, counts, dtype, cap and ranks on the same device finds its
 * tables there and neither copies nor waits.  A call on a stream that is
 * being captured returns DT_ERR_UNSUPPORTED and enqueues nothing (a captured
 * copy would read the host array at replay time, after later calls have
 * rewritten it).  No signal barrier runs between buckets (there is no group
 * window); stream order orders them.  The first call on each device looks up
 * the array's device address with that device current.  The current CUDA
 * device must be the gradients'. */
dt_status dt_bucket_allreduce_static(int world_size, void *const *grads, const size_t *counts,
                                     size_t n_tensors, int dtype, int op,
                                     size_t bucket_cap_bytes, void *stream);

/* ------------------------------------------------ layer norm, group-wide */

/* Layer norm over the last dimension of every rank's rows, as a
 * sequence-parallel model has it: the activations are S(0) (rank r holds its
 * own rows), the weights R (one copy serves every rank on this GPU), and the
 * weights' gradients P, reduced over the ranks by the backward call itself.
 * Like the bucket all-reduce, these calls are group-wide only.
 *   x[r], y[r]     rank r's rows (rows[r], or rows_equal when rows is NULL) of
 *                  cols elements of dtype (DT_F32 or DT_BF16), dense; y[r] may
 *                  equal x[r] (in place).  A rank may have no rows.
 *   weight, bias   cols elements of weight_dtype (DT_F32 or DT_BF16), shared
 *                  by all ranks; NULL: ones, zeros
 *   mean, rstd     per rank rows[r] floats, written: what the backward call
 *                  reads; either array, or any entry, may be NULL
 *   eps            finite, >= 0
 * With mu the mean of a row and v the mean of (x - mu)^2, both fp32 and v from
 * the differences: rstd = 1 / sqrt(v + eps), y = (x - mu) * rstd * weight +
 * bias, rounded once.  A NaN or an infinity in a row makes that row NaN.  The
 * order of a row's sums depends on its width, type and alignment and on whether
 * the call has more than two rows an SM: the same call gives the same bits.
 * Every pointer must be a multiple of its element size; rows that all start on
 * 16-byte boundaries move as vectors, others element by element.  cols is
 * 1..2^24.  A buffer may otherwise overlap no output. */
dt_status dt_layer_norm(dt_group_t g, const void *const *x, const void *weight, const void *bias,
                        void *const *y, float *const *mean, float *const *rstd, const size_t *rows,
                        size_t rows_equal, size_t cols, float eps, int dtype, int weight_dtype,
                        void *stream);

/* The backward pass.  With h = (x - mean) * rstd and q = dy * weight:
 *   dx[r]     = rstd * (q - mean(q) - h * mean(q * h)), of dtype; may equal
 *               dy[r] (in place)
 *   dweight   = the sum over every row of every rank of dy * h, of
 *               weight_dtype; dbias the same of dy; either may be NULL.  op
 *               DT_SUM, or DT_AVG: divided by the number of ranks, the mean
 *               of the ranks' gradients.  With no rows at all they are 0.
 *   mean, rstd  as the forward call wrote them
 *   workspace   at least dt_layer_norm_workspace(g, cols) bytes of device
 *               memory, 16-byte aligned, free for other use once `stream` has
 *               passed the call; NULL when neither gradient is wanted
 * The sums over rows are fp32 and their order depends on the GPU and the
 * shapes only: repeated calls give the same bits. */
dt_status dt_layer_norm_backward(dt_group_t g, const void *const *x, const void *const *dy,
                                 const void *weight, const float *const *mean,
                                 const float *const *rstd, void *const *dx, void *dweight,
                                 void *dbias, const size_t *rows, size_t rows_equal, size_t cols,
                                 int dtype, int weight_dtype, int op, void *workspace,
                                 size_t workspace_bytes, void *stream);

/* Workspace bytes of dt_layer_norm_backward for rows of cols elements, any
 * number of them; 0 for an invalid argument. */
size_t dt_layer_norm_workspace(dt_group_t g, size_t cols);

/* ------------------------------------------- vocabulary loss, group-wide */

/* Softmax cross entropy of `tokens` hidden rows under a vocabulary whose rows
 * are S(0) over the ranks (rank r holds weight[r]), computed from the hidden
 * rows and the weights in one call: the logits are never stored, and the
 * reductions over the ranks (the maximum and the sum of exponentials here,
 * dhidden below) are part of it.  Group-wide only, like the layer norm.
 *   hidden       [tokens, dim], one copy for all ranks
 *   weight[r]    rank r's vocabulary rows, [vocab[r], dim] (vocab_equal rows
 *                each when vocab is NULL); rank r's first row has the index
 *                vocab[0] + ... + vocab[r - 1].  A rank may have none, all
 *                ranks together need one.
 *   targets      [tokens] int32 vocabulary indices on the device, or
 *                ignore_index: that token's loss and dhidden are 0, it is not
 *                counted, and its hidden row enters dweight as a product with
 *                0 (so a NaN or an infinity there makes dweight NaN).  Any
 *                other value outside the vocabulary is treated the same way
 *                and recorded as DT_ERR_INVALID in the group's error word
 *                (dt_group_error_detail: rank -1, peer = the token,
 *                generation = the value).
 *   dtype        of hidden and weight: DT_BF16 (products in the tensor cores,
 *                fp32 sums); DT_F32 is DT_ERR_UNSUPPORTED
 *   op           DT_SUM, or DT_AVG: the mean over the counted tokens (0 where
 *                none is counted)
 *   losses, lse  [tokens] floats: each token's loss, and log(sum(exp(logits)))
 *                for the backward call;  loss: one float.  Each may be NULL.
 *   workspace    dt_vocab_loss_workspace bytes (backward = 0) of device memory,
 *                256-byte aligned, free once `stream` has passed the call
 * hidden, weight are 2-byte aligned; rows of whole 16-byte vectors that start
 * on 16-byte boundaries are read in place, others are laid out again in the
 * workspace first.  tokens, the vocabulary and dim are at most 2^30, 2^30 and
 * 2^20.  No output may overlap another buffer. */
dt_status dt_vocab_loss(dt_group_t g, const void *hidden, const void *const *weight,
                        const size_t *vocab, size_t vocab_equal, const int32_t *targets,
                        size_t tokens, size_t dim, int dtype, int op, int32_t ignore_index,
                        float *losses, float *lse, float *loss, void *workspace,
                        size_t workspace_bytes, void *stream);

/* The gradient of that loss.  With p = exp(logit - lse) and c = grad_loss
 * (one float on the device; NULL: 1), divided by the counted tokens for DT_AVG:
 *   dhidden      [tokens, dim] of dtype: c * sum over the whole vocabulary of
 *                (p - [target]) * weight, the ranks' parts already reduced
 *   dweight[r]   [vocab[r], dim] of dtype: c * sum over the tokens of
 *                (p - [target]) * hidden; entries of ranks without rows may be
 *                NULL
 *   lse          as dt_vocab_loss wrote it
 *   workspace    dt_vocab_loss_workspace bytes with backward = 1
 * The logits are computed again as the loss computes them, a piece of the
 * vocabulary at a time; p - [target] is held in bf16 for that piece (at most 512
 * MiB, or 256 vocabulary rows' worth), every sum in fp32, and results are
 * rounded once.  The tensor cores cut off what of a product lies below a quarter of
 * the sum's last place: sums of n terms of one sign are about n * 5e-9 of themselves too
 * small beside that, and any n * 2^-25 of their largest part sum or term at most.
 * Repeated calls give the same bits. */
dt_status dt_vocab_loss_backward(dt_group_t g, const void *hidden, const void *const *weight,
                                 const size_t *vocab, size_t vocab_equal, const int32_t *targets,
                                 const float *lse, const float *grad_loss, size_t tokens,
                                 size_t dim, int dtype, int op, int32_t ignore_index,
                                 void *dhidden, void *const *dweight, void *workspace,
                                 size_t workspace_bytes, void *stream);

/* Workspace bytes of either call; 0 for an invalid argument. */
size_t dt_vocab_loss_workspace(dt_group_t g, const size_t *vocab, size_t vocab_equal,
                               size_t tokens, size_t dim, int dtype, int backward);

/* ------------------------------- linear layers over the ranks, group-wide */

/* The two linear layers of a block whose tokens are S(0) over the ranks (rank r
 * holds rows[r] of them, `dim` columns each) and whose inner features are S(0)
 * over the ranks as well (rank r holds features[r]).  The first gathers: every
 * rank's tokens meet every rank's features.  The second reduces: the ranks'
 * features are summed over and each rank keeps its own tokens.  The gather and the
 * reduce-scatter are part of the products: neither the gathered tokens nor the
 * ranks' partial sums are stored, and the sum over the ranks is rounded once.
 *
 * Both.  rows NULL: rows_equal tokens on each rank; features NULL: features_equal.
 * n is the sum of rows (n of them number the tokens in rank order); a rank may have
 * no tokens or no features, all ranks together need a feature.  dtype is that of
 * every tensor: DT_BF16, products in the tensor cores and fp32 sums; DT_F32 is
 * DT_ERR_UNSUPPORTED.  Tensors are dense and 2-byte aligned.  Few tokens and small
 * products read them in place; of larger ones those whose rows start on 16-byte
 * boundaries are, others are laid out again in the workspace first, as are tokens where the
 * tiles of 128 rows that the ranks' pieces end inside would cost more than that.
 * workspace: the query's bytes of device memory, 256-byte aligned, free for other use
 * once `stream` has passed the call.  No output may overlap another buffer, but for
 * the residual below.  n is at most 2^26, dim and the sum of features 2^22.  The
 * tensor cores cut off what of a product lies below a quarter of the sum's last place:
 * a sum of n terms is off by n * 2^-25 of its largest part sum or term at most.  Terms of
 * one sign and like size come out n * 5e-9 of their sum too small, terms of both signs as
 * near as fp32's rounding.  Calls repeated on the same buffers give the same bits; the same
 * values in others, aligned otherwise or with ranks' rows that follow one another where these
 * do not, may be summed in another order. */
#define DT_ACT_NONE 0
#define DT_ACT_RELU 1
#define DT_ACT_GELU 2 /* v * Phi(v), Phi the normal distribution (no tanh form) */
#define DT_ACT_SILU 3 /* v / (1 + exp(-v)); 0 below v = -87.3, where it is -1.1e-36 and nearer to 0 */

/* y[r] = act(X weight[r]^T + bias[r]), X [n, dim] the tokens of all ranks:
 *   x[r]        rank r's tokens, [rows[r], dim]
 *   weight[r]   [features[r], dim]
 *   bias        NULL, or bias[r] [features[r]]
 *   pre         NULL, or pre[r] [n, features[r]]: receives what act is taken of (itself
 *               rounded to dtype; act is taken of the fp32 sum), for the backward call
 *   y[r]        [n, features[r]] */
dt_status dt_gather_linear(dt_group_t g, const void *const *x, const void *const *weight,
                           const void *const *bias, void *const *pre, void *const *y,
                           const size_t *rows, size_t rows_equal, size_t dim, const size_t *features,
                           size_t features_equal, int dtype, int act, void *workspace,
                           size_t workspace_bytes, void *stream);

/* Its gradient.  With G_r = dy[r] act'(pre[r]) (dy[r] itself for DT_ACT_NONE, where pre
 * may be NULL), rounded to dtype as the products' operand (small products, a few
 * tokens of narrow layers among them, take what the rounding leaves as an operand too):
 *   dx[r]       rank r's rows of sum_q G_q weight[q], reduced over the ranks
 *   dweight[r]  G_r^T X
 *   dbias       NULL, or dbias[r]: the sum of G_r over the tokens, before its rounding
 * With no tokens at all dweight and dbias are 0. */
dt_status dt_gather_linear_backward(dt_group_t g, const void *const *x, const void *const *weight,
                                    const void *const *pre, const void *const *dy, void *const *dx,
                                    void *const *dweight, void *const *dbias, const size_t *rows,
                                    size_t rows_equal, size_t dim, const size_t *features,
                                    size_t features_equal, int dtype, int act, void *workspace,
                                    size_t workspace_bytes, void *stream);

/* Workspace bytes of either call; 0 for an invalid argument. */
size_t dt_gather_linear_workspace(dt_group_t g, const size_t *rows, size_t rows_equal, size_t dim,
                                  const size_t *features, size_t features_equal, int dtype,
                                  int backward);

/* y[r] = rank r's rows of (sum_q x[q] weight[q]^T + bias) + residual[r]:
 *   x[q]        rank q's features of all tokens, [n, features[q]]
 *   weight[q]   [dim, features[q]]
 *   bias        NULL, or [dim], added once
 *   residual    NULL, or residual[r] [rows[r], dim]
 *   y[r]        [rows[r], dim]; may be residual[r] itself (in place) */
dt_status dt_linear_reduce(dt_group_t g, const void *const *x, const void *const *weight,
                           const void *bias, const void *const *residual, void *const *y,
                           const size_t *rows, size_t rows_equal, size_t dim, const size_t *features,
                           size_t features_equal, int dtype, void *workspace, size_t workspace_bytes,
                           void *stream);

/* Its gradient.  With Y [n, dim] the dy of all ranks:
 *   dx[q]       Y weight[q], [n, features[q]]
 *   dweight[q]  Y^T x[q]
 *   dbias       NULL, or the sum of Y over the tokens, [dim]
 * (the residual's gradient is dy).  With no tokens dweight and dbias are 0. */
dt_status dt_linear_reduce_backward(dt_group_t g, const void *const *x, const void *const *weight,
                                    const void *const *dy, void *const *dx, void *const *dweight,
                                    void *dbias, const size_t *rows, size_t rows_equal, size_t dim,
                                    const size_t *features, size_t features_equal, int dtype,
                                    void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes of either call; 0 for an invalid argument. */
size_t dt_linear_reduce_workspace(dt_group_t g, const size_t *rows, size_t rows_equal, size_t dim,
                                  const size_t *features, size_t features_equal, int dtype,
                                  int backward);

/* ---------------------------------------- residual norm, group-wide */

/* What stands between two blocks, for every rank's rows at once: the norm of the
 * block's output, its gate, the residual sum, and the norm before the next block.
 * With rstd(v) = 1 / sqrt(mean(v^2) + eps) over a row (no mean is taken off):
 *   h = branch * rstd(branch)       y = residual_scale * x + gate * post_weight * h
 *   z = y * rstd(y) * pre_weight
 * x[r], branch[r], y[r], z[r] are rank r's [rows[r], cols] of dtype (rows NULL:
 * rows_equal rows each); a rank may have none.  post_weight, gate and pre_weight, each
 * [cols] of weight_dtype or NULL (1), serve all ranks.  dtype and weight_dtype are
 * DT_F32 or DT_BF16.  All sums are fp32, the second norm is of y before its rounding,
 * and y and z are rounded once.  rstd_post and rstd_pre, float arrays of rows[r] for
 * each rank (or NULL: not wanted), receive both reciprocals for the backward call.  y[r]
 * may be x[r] and z[r] may be branch[r] (in place); otherwise no output may overlap another
 * buffer.
 * Pointers are multiples of their element size; rows that all start on 16-byte boundaries
 * move as vectors.  cols is 1..2^24, residual_scale any finite number.  The same call gives
 * the same bits.
 * A NaN or an infinity goes through the formulas as it stands and reaches its own row's
 * results only.  A NaN in branch makes all of y and z and both reciprocals NaN; one in x its
 * element of y, all of z, and rstd_pre.  Of an infinity the reciprocal is 0 and its own norm
 * NaN: one in branch makes rstd_post 0, its element of y NaN and the others
 * residual_scale * x, all of z and rstd_pre NaN; one in x makes its element of y infinite
 * and of z NaN, rstd_pre and the rest of z 0.  Squares are summed in fp32: where the sum
 * passes it (a root mean square of 1.8e19 / sqrt(cols)) the reciprocal is 0 as well.  With
 * an eps of 0 a row whose squares are all 0 there, below 1e-23, has an infinite one, and NaN
 * or infinities for its norm. */
dt_status dt_residual_norm(dt_group_t g, const void *const *x, const void *const *branch,
                           const void *post_weight, const void *gate, const void *pre_weight,
                           float residual_scale, void *const *y, void *const *z,
                           float *const *rstd_post, float *const *rstd_pre, const size_t *rows,
                           size_t rows_equal, size_t cols, float eps, int dtype, int weight_dtype,
                           void *stream);

/* The backward pass.  y is as the forward call wrote it, dy the gradient that reaches y
 * from further on (NULL: none), dz that of z.  With n = y * rstd_pre, q = dz * pre_weight,
 * h = branch * rstd_post, d = dy + rstd_pre * (q - n * mean(q * n)) and c = d * gate *
 * post_weight:
 *   dx[r]         = residual_scale * d; may be dy[r] (in place)
 *   dbranch[r]    = rstd_post * (c - h * mean(c * h)); may be dz[r]
 *   dpost_weight  = gate * the sum over every row of every rank of d * h
 *   dgate         = post_weight * that sum
 *   dpre_weight   = the sum over every row of every rank of dz * n
 * the last three of weight_dtype, each may be NULL; op DT_SUM, or DT_AVG: divided by the
 * number of ranks.  With no rows at all they are 0.  A NaN or an infinity reaches its own
 * row's results and the weights' gradients only.  Reciprocals are squared in fp32: one of
 * 1.8e19 or more, which no eps of 1e-38 or more leaves, makes NaN or infinities.
 *   workspace     at least dt_residual_norm_workspace(g, cols) bytes of device memory,
 *                 16-byte aligned, free for other use once `stream` has passed the call;
 *                 NULL when none of the three is wanted
 * Sums are fp32 in an order that depends on the GPU and the shapes only. */
dt_status dt_residual_norm_backward(dt_group_t g, const void *const *branch, const void *const *y,
                                    const void *const *dy, const void *const *dz,
                                    const void *post_weight, const void *gate, const void *pre_weight,
                                    float residual_scale, const float *const *rstd_post,
                                    const float *const *rstd_pre, void *const *dx,
                                    void *const *dbranch, void *dpost_weight, void *dgate,
                                    void *dpre_weight, const size_t *rows, size_t rows_equal,
                                    size_t cols, int dtype, int weight_dtype, int op, void *workspace,
                                    size_t workspace_bytes, void *stream);

/* Workspace bytes of dt_residual_norm_backward for rows of cols elements, any number of
 * them; 0 for an invalid argument. */
size_t dt_residual_norm_workspace(dt_group_t g, size_t cols);

/* ----------------------------------------------------------- async work */

/* Asynchronous collectives, after the async mode of "通信与互联（05）" §四.3
 * (async_op=True): the collective runs on the backend's own stream, which
 * first waits for the caller's stream (syncStream), and the caller gets a
 * Work whose end event it waits on later; §五.5's rule holds: buffers of an
 * unfinished work are neither read nor written on any stream.
 *   dt_async_begin  makes the group's communication stream wait for the work
 *                   already on `stream` and returns that communication stream
 *                   in *comm_stream: pass it to the dt_* calls of the scope
 *                   (any collective, any number); one scope per group at a
 *                   time, opened and closed by one thread
 *   dt_async_end    closes the scope and returns a work handle whose end
 *                   event covers everything enqueued in the scope
 *   dt_work_wait    makes `stream` wait for the work (no host blocking)
 *   dt_work_query   DT_OK when the work has finished, DT_NOT_READY if not
 *   dt_work_free    returns the handle to its group (after waiting or
 *                   querying; freeing does not cancel the work)
 * Groups on different communication streams (for example the shard and
 * replicate groups of an HSDP mesh) run their works concurrently. */
dt_status dt_async_begin(dt_group_t g, void *stream, void **comm_stream);
dt_status dt_async_end(dt_group_t g, dt_work_t *work);
dt_status dt_work_wait(dt_work_t work, void *stream);
dt_status dt_work_query(dt_work_t work);
dt_status dt_work_free(dt_work_t work);

/* ------------------------------------------------------------- test hooks */

/* Copy the P x P window to host_out (row-major, win[q][r] at q * P + r) after
 * the work already on `stream`; blocks the calling thread. */
dt_status dt_debug_read_window(dt_group_t g, int32_t *host_out, void *stream);

/* The ordering example of the barrier page (built-in reveal): one kernel,
 * one block per rank; rank r copies in[r] to stage[r], passes the barrier,
 * then copies stage[(r + 1) % P] to out[r].  Each buffer holds `bytes`. */
dt_status dt_debug_ring_after_barrier(dt_group_t g, const void *const *in,
                                      void *const *stage, void *const *out, size_t bytes,
                                      void *stream);

/* Failure injection for tests: run one barrier kernel whose waits expect the
 * generation current + extra (extra >= 1), which no rank will reach, with a
 * wait limit of timeout_ms.  The waits give up, DT_ERR_TIMEOUT is recorded
 * in the error word and the kernel returns; the GPU stays usable. */
dt_status dt_debug_barrier_expect(dt_group_t g, int extra, uint32_t timeout_ms, void *stream);

/* ------------------------------------------------------------- tracing */

/* Per-block timeline of the library's kernels, recorded only by a library
 * built with DT_TIMELINE=1 in the environment (elsewhere both calls return
 * DT_ERR_UNSUPPORTED).  The pages trace collectives with profiler timelines
 * ("通信与互联（05）" §六: the communication kernels of each stream on their
 * own row); this records, for every thread block of every kernel launched
 * after dt_timeline_start, when it started, when it passed its wait on the
 * previous kernel (the bucket barrier block: when its barrier completed) and
 * when it ended, in %globaltimer nanoseconds.
 *   dt_timeline_start  (re)allocates room for max_records on the current
 *                      device and empties it; the last one wins
 *   dt_timeline_read   waits for the device, copies up to max_records records
 *                      to host memory and sets *n_records; records past the
 *                      room are dropped and counted in *n_records */
#define DT_TL_REDUCE 1          /* AllReduce / ReduceScatter, vector kernel */
#define DT_TL_REDUCE_SHIFT 2    /* the same, inputs at their own offsets */
#define DT_TL_COPY_BULK 3       /* AllGather / AllToAll, TMA bulk copies */
#define DT_TL_COPY_VEC 4        /* small copies */
#define DT_TL_COPY_SHIFT 5      /* copies at other offsets */
#define DT_TL_COPY_2D 6         /* AllToAll along other dims */
#define DT_TL_BUCKET 7          /* bucket all-reduce, data block */
#define DT_TL_BUCKET_BARRIER 8  /* bucket all-reduce, the barrier block after a bucket */
#define DT_TL_BARRIER 9         /* signal-window barrier kernel */
#define DT_TL_MARK 10           /* dt_timeline_mark: block = the caller's tag */
#define DT_TL_NORM 11           /* layer norm, either pass, and the join of its weight gradients */
#define DT_TL_VOCAB 12          /* vocabulary loss, either pass */
#define DT_TL_LINEAR 13         /* linear layers over the ranks, either pass */
#define DT_TL_RESIDUAL 14       /* residual norm, either pass, and the join of its weight gradients */
typedef struct {
    uint64_t grid;       /* the launch's %gridid */
    uint32_t kind;       /* DT_TL_* */
    uint32_t block;      /* blockIdx.x + gridDim.x * blockIdx.y */
    uint32_t sm;         /* %smid */
    uint32_t pad;
    uint64_t t_start, t_waited, t_end;
} dt_timeline_record;
dt_status dt_timeline_start(size_t max_records);
dt_status dt_timeline_read(dt_timeline_record *out, size_t max_records, size_t *n_records);
/* A mark on the timeline at this point of `stream`: a one-thread kernel
 * records DT_TL_MARK with block = tag, so a caller can bracket its own work
 * (a GEMM, a copy) and compare it with the collectives' blocks. */
dt_status dt_timeline_mark(void *stream, uint32_t tag);

/* ------------------------------------------------------- build flavours */

/* Which instrumented flavour this library is (a bit set; 0 = the default
 * build).  Each flavour is chosen by a variable in the environment of the
 * build and compiled into its own objects.
 *   DT_BUILD_NVTX      every entry point opens an NVTX range (DT_NVTX=1)
 *   DT_BUILD_TIMELINE  the kernel timeline above is recorded (DT_TIMELINE=1)
 *   DT_BUILD_BOUNDS    bounds-checked kernels (DT_BOUNDS=1): every global
 *                      load and store of the data kernels is checked against
 *                      the extent of its buffer as the call's arguments give
 *                      it.  An access outside is skipped and DT_ERR_INVALID
 *                      is recorded in the group's error word, with
 *                      dt_group_error_detail giving rank = the kernel
 *                      (DT_BOUNDS_* below), peer = the buffer (reductions:
 *                      input r as r, output q as 16 + q; copies: source
 *                      segment s as s, destination q as 256 + q; bucket
 *                      kernel: the tensor's index in its bucket) and
 *                      generation = the low 31 bits of the byte offset from
 *                      the buffer's start.  dt_bucket_allreduce_static
 *                      has no error word: its out-of-bounds accesses are only
 *                      skipped.  The checks cost time: for testing only.
 *                      DT_BOUNDS_TRIM=<bytes> in the environment of a
 *                      program using this flavour records every destination
 *                      extent that many bytes short (a self-test of the
 *                      checker: the stores it skips lie inside the buffers). */
#define DT_BUILD_NVTX 1u
#define DT_BUILD_TIMELINE 2u
#define DT_BUILD_BOUNDS 4u
#define DT_BOUNDS_REDUCE 1       /* AllReduce / ReduceScatter */
#define DT_BOUNDS_REDUCE_SHIFT 2 /* the same, inputs at their own offsets */
#define DT_BOUNDS_COPY_BULK 3
#define DT_BOUNDS_COPY_VEC 4
#define DT_BOUNDS_COPY_EDGE 5
#define DT_BOUNDS_COPY_SHIFT 6
#define DT_BOUNDS_COPY_2D 7
#define DT_BOUNDS_BUCKET 8
/* Layer norm; buffers: x r, dy 16 + r, y or dx 32 + r, mean 48 + r, rstd 64 + r,
 * weight 80, bias 81, dweight 82, dbias 83, workspace 84. */
#define DT_BOUNDS_NORM 9
/* Vocabulary loss; buffers: p - [target] 0, dhidden 1, targets 2, lse 3, losses 4,
 * loss 5, grad_loss 6, workspace 7, hidden rows laid out again 8, dweight 16 + r,
 * rank r's rows laid out again 32 + r.  (TMA's own loads stay in their tensor maps.) */
#define DT_BOUNDS_VOCAB 10
/* Linear layers over the ranks; buffers by rank r: y r, pre 16 + r, dx 32 + r, dweight
 * 48 + r, dbias 64 + r, bias 80 + r, residual 96 + r, and those laid out again x 112 + r,
 * weight 128 + r, dy 144 + r; workspace 160.  (TMA's own loads stay in their maps.) */
#define DT_BOUNDS_LINEAR 11
/* Residual norm; buffers: branch r, x or y 16 + r, dz 32 + r, dy 48 + r, y or dx 64 + r, z
 * or dbranch 80 + r, rstd_post 96 + r, rstd_pre 112 + r, post_weight 128, gate 129,
 * pre_weight 130, their gradients 131 to 133, workspace 134. */
#define DT_BOUNDS_RESIDUAL 12
uint32_t dt_build_flags(void);

#ifdef __cplusplus
}
#endif

#endif /* DT_H */
