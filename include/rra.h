/*
 * rra.h -- all-reduce, reduce-scatter and all-gather over N "virtual ranks"
 * held as separate buffers in one GPU's memory, plus the LL and LL128 wire
 * formats.  Plain C ABI: device and host pointers, sizes and enums; no C++
 * or PyTorch types.  Library: librra.so (sm_103a).
 *
 * Sources (web pages, cited by title and section):
 *   [ILP] "NCCL collectives, ring all-reduce & launching TP/PP"
 *         (inference-learning-path): "Direct answer", "Deep dive", "Code".
 *   [AIH] "Collective communication: NCCL's algorithms and protocols, and
 *         custom all-reduce in inference frameworks" (ai-infra-handbooks):
 *         "Algorithms: the ways to run one all-reduce", "Protocols: how do
 *         you know the data has arrived", "Reading nccl-tests",
 *         "Common environment variables and debugging", "Exercises" 2 and 3.
 *
 * Conventions shared by every call
 * --------------------------------
 * - A virtual rank r owns one input buffer bufs[r] and one output buffer
 *   outs[r], all device pointers on the current CUDA device.  bufs/outs are
 *   HOST arrays of nranks device pointers; they are read during the call
 *   only (copied into the kernel's parameters), never retained.
 * - Buffers are dense, 1-D, element type `dtype`, little-endian.  Each
 *   pointer must be aligned to the element size; 16-byte aligned buffers
 *   (what cudaMalloc and PyTorch give) take the 128-bit vector path, other
 *   alignments a slower element-wise path with identical results.
 * - The caller owns every buffer.  The library owns only the workspace made
 *   by rra_init() for the device.
 * - Calls are asynchronous on `stream` (a cudaStream_t; NULL = the legacy
 *   default stream), never allocate, never synchronize, and may be captured
 *   into a CUDA graph.  Argument errors are returned synchronously before
 *   any launch.  Errors found on the device (a bounded wait that expired, a
 *   wire flag that never matched) are recorded in the device status word
 *   and read with rra_query_status(), like an asynchronous communicator
 *   error.
 * - Calls that use the workspace (ring, two-shot, LL/LL128 unpack) on one
 *   device must not overlap on the GPU: issue them on one stream or order
 *   them, as with the operations of one communicator.
 * - count == 0 returns RRA_SUCCESS without a launch.
 * - Summation (op RRA_SUM): int32 wraps modulo 2^32; float32 adds in IEEE
 *   round-to-nearest in the order the schedule fixes; bfloat16 is widened
 *   to float32, summed in float32 in that order and rounded to bfloat16
 *   (nearest, ties to even) once, when the final value is stored.
 *
 * Environment (read by the library; none is needed, each overrides a
 * measured default; [AIH] "Common environment variables and debugging"
 * describes NCCL's counterparts)
 * ------------------------------------------------------------------------
 *   RRA_ALGO             schedule for RRA_ALGO_AUTO: ring, one_shot,
 *                        two_shot or tree (instead of the tuning table)
 *   RRA_TUNING_FILE      tuning table read by rra_init (default: tune/
 *                        gb300.txt beside the library)
 *   RRA_TIMEOUT_NS       bound of every device wait (500 ms), unless
 *                        rra_set_timeout_ns() sets one
 *   RRA_MAX_CTAS         CTA budget of every kernel (0: all), unless
 *                        rra_set_max_ctas() sets one
 *   RRA_DEBUG            1: print each call (schedule, grid, status) and
 *                        every CUDA error to stderr
 *   RRA_RING_PROTO       ring links for every buffer: staged, simple or ll
 *                        (per-warp forms); default by size (below)
 *   RRA_RING_LL_STAGED_MAX_BYTES  on 16-byte aligned buffers with 2 ranks
 *                        or more, chunks up to this many bytes take LL
 *                        lines (measured faster there; default 256 KiB from
 *                        3 ranks and 128 KiB at 2, bfloat16 128 KiB),
 *                        larger ones the staged form
 *   RRA_RING_LL_MAX_BYTES  on other buffers, the largest chunk the per-warp
 *                        ring sends as LL lines (64 KiB; larger: Simple)
 *   RRA_RING_CLUSTER     1: the ring on thread-block clusters
 *   RRA_RING_TILE, RRA_RING_G, RRA_RING_K, RRA_RING_STAGES,
 *   RRA_RING_CHANNELS    staged ring: units per message (<= 2368, 1536 for
 *                        bfloat16), messages per step (1-6 by the chunk's
 *                        size per channel), FIFO slots (G+3),
 *                        shared-memory stages, CTAs per rank
 *   RRA_STAGED_SMEM_KB   shared memory for the staged ring's and tree's
 *                        stages (224)
 *   RRA_TREE_TILE, RRA_TREE_G, RRA_TREE_K, RRA_TREE_LAG, RRA_TREE_STAGES,
 *   RRA_TREE_CHANNELS    staged tree: units per message (<= 2048, 1280 for
 *                        bfloat16), tiles per iteration (by size, at most
 *                        24, 12 for bfloat16), FIFO slots (G + 1),
 *                        iterations the broadcast trails the reduction (6),
 *                        stages, CTAs per rank
 *   RRA_TREE_PROTO       ll | staged: the tree's form (default: LL lines
 *                        wherever they fit the workspace's LL region, up to
 *                        RRA_TREE_LL_MAX_BYTES per rank (no limit; bfloat16
 *                        at 2 ranks 1 MiB); the staged tree otherwise)
 *   RRA_TWOSHOT_CLUSTER  1: two-shot on thread-block clusters
 *   RRA_TWOSHOT_CHANNELS CTAs per rank of two-shot
 *   RRA_TWOSHOT_LAG      tiles the two-shot's gather trails its reduce by
 *                        (and between its progress flags): 16 at 8 ranks, 8
 *                        below
 *   RRA_ONESHOT_TMA      1: one-shot with bulk copies through shared memory
 *   RRA_ONESHOT_PER_RANK 1: one-shot reads the n inputs once per rank, as
 *                        n GPUs would (out of place only; in place keeps
 *                        the combined form)
 *   RRA_DIRECT_GRID      grid of one-shot and the direct reduce-scatter and
 *                        all-gather: resident (SMs x occupancy, grid-stride)
 *                        or cover (one trip a thread); default: cover from
 *                        256 MB of floor bytes (one-shot) or 64 MB (the
 *                        others), resident below.  An SM budget keeps the
 *                        resident grid.
 */
#ifndef RRA_H
#define RRA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/** Same object as cudaStream_t; NULL means the legacy default stream. */
typedef struct CUstream_st* rra_stream_t;

/** Largest number of virtual ranks (and of LL/LL128 sources) per call. */
#define RRA_MAX_RANKS 8

typedef enum {
  RRA_OK = 0,
  RRA_SUCCESS = RRA_OK,        /* the same value under a second name */
  RRA_ERR_INVALID_ARG = 1,     /* null pointer, bad count, bad enum, misaligned pointer, flag 0 */
  RRA_ERR_UNSUPPORTED = 2,     /* valid but not supported here (e.g. nranks > RRA_MAX_RANKS) */
  RRA_ERR_ALIAS = 3,           /* input and output ranges overlap other than in place */
  RRA_ERR_NOT_INITIALIZED = 4, /* rra_init() was not called for the current device */
  RRA_ERR_CUDA = 5,            /* a CUDA runtime call failed (launch, query) */
  RRA_ERR_TIMEOUT = 6,         /* a bounded device wait expired (see rra_query_status) */
  RRA_ERR_WORKSPACE = 7        /* the workspace of rra_init is too small for the call's FIFO
                                  slots and flags (call rra_init with more workspace_bytes) */
} rra_status_t;

typedef enum { RRA_INT32 = 0, RRA_FLOAT32 = 1, RRA_BFLOAT16 = 2 } rra_dtype_t;

typedef enum { RRA_SUM = 0 } rra_op_t;

/** Schedules ([AIH] "Algorithms").  For reduce-scatter and all-gather,
 *  RRA_ALGO_DIRECT names the direct halves of two-shot (RRA_ALGO_TWO_SHOT
 *  is accepted as a synonym) and RRA_ALGO_RING the ring halves. */
typedef enum {
  RRA_ALGO_AUTO = 0,
  RRA_ALGO_RING = 1,
  RRA_ALGO_ONE_SHOT = 2,
  RRA_ALGO_TWO_SHOT = 3,
  RRA_ALGO_DIRECT = 4,
  /** all-gather only: the GPU's copy engines move the shards
   *  (cudaMemcpyAsync device to device), no SM runs a kernel ([AIH]
   *  "Protocols": transfer methods that use no SMs, like the copy engine). */
  RRA_ALGO_COPY_ENGINE = 5,
  /** all-reduce only: a double binary tree ([AIH] "Algorithms": tree
   *  (double binary tree), reduce up, broadcast down, O(log n) steps,
   *  large messages pipelined in chunks).  Tree 0 is the binary tree in
   *  heap order over the ranks (position p has children 2p+1 and 2p+2,
   *  rank r at position r), tree 1 the same tree over the ranks reversed
   *  (rank r at position n-1-r).  The first part of the message by the
   *  chunk plan for two parts (C = ceil(count/2) rounded up to whole
   *  16-byte vectors) is reduced on tree 0, the rest on tree 1.  A node
   *  sums its own data, then the partial of its child 2p+1, then that of
   *  its child 2p+2; each root's total, rounded once, travels down
   *  unchanged.  Needs 16-byte aligned buffers (else
   *  RRA_ERR_UNSUPPORTED).  Links through the workspace: LL lines for
   *  small messages ("Protocols": LL for small messages), whole-CTA
   *  messages staged by bulk copies for large ones. */
  RRA_ALGO_TREE = 6
} rra_algo_t;

/* ------------------------------------------------------------------------ */
/* set-up                                                                   */
/* ------------------------------------------------------------------------ */

/** Create the per-device state: the workspace (device status word, step
 *  flags, FIFO slots; 64 MiB of them, at most half, hold LL lines only) of
 *  `workspace_bytes` bytes (0 = 256 MiB, at least 1 MiB) on CUDA device
 *  `device`, which becomes current.  Fixed buffers
 *  made once, ahead of the calls, keep every call allocation-free and
 *  graph-capturable, as [AIH] "Exercises" 3 explains for custom
 *  all-reduce.  Calling it again for an initialised device is a no-op that
 *  returns RRA_SUCCESS.  Errors: RRA_ERR_INVALID_ARG (bad device),
 *  RRA_ERR_CUDA (allocation failed). */
rra_status_t rra_init(int device, size_t workspace_bytes);

/** Free the state rra_init made on every device (the pages' communicator
 *  teardown that ends the "init step before calls" of [ILP] "Code").  The
 *  caller must have synchronized every stream that used it; later calls
 *  that need the workspace return RRA_ERR_NOT_INITIALIZED until rra_init
 *  is called again.  Returns RRA_ERR_CUDA if freeing a workspace failed
 *  (the state is dropped all the same). */
rra_status_t rra_finalize(void);

/* ------------------------------------------------------------------------ */
/* collectives                                                              */
/* ------------------------------------------------------------------------ */

/** All-reduce ([ILP] "Direct answer": sum a tensor every rank holds; every
 *  rank ends with the result).  outs[r][i] = SUM_k bufs[k][i] for
 *  i < count, every r.
 *  - bufs[r], outs[r]: count elements each.  In place (outs[r] == bufs[r]
 *    for every r) is allowed; any other overlap is RRA_ERR_ALIAS.
 *  - algo: RING -- n-1 reduce-scatter steps then n-1 all-gather steps over
 *    the N chunks of the chunk plan ([ILP] "Deep dive", [AIH] "Algorithms");
 *    chunk c is summed in the order x_{c+1}, ..., x_{c-1}, x_c.
 *    ONE_SHOT -- every rank's result read directly from all n inputs,
 *    summed in ascending rank order.  TWO_SHOT -- rank r reduces chunk r
 *    (ascending order), then every rank reads the reduced chunks back.
 *    AUTO -- rra_select_algo().
 *  - Chunk plan: chunk length C = ceil(count/n) rounded up to whole
 *    16-byte vectors, chunk c = [min(cC,count), min((c+1)C,count)).
 *  - nranks in [1, RRA_MAX_RANKS]; nranks == 1 copies (or does nothing in
 *    place).
 *  Errors: RRA_ERR_INVALID_ARG, RRA_ERR_UNSUPPORTED, RRA_ERR_ALIAS,
 *  RRA_ERR_NOT_INITIALIZED (RING/TWO_SHOT/AUTO without rra_init),
 *  RRA_ERR_CUDA. */
rra_status_t rra_allreduce(const void* const* bufs, void* const* outs, int nranks, size_t count,
                           rra_dtype_t dtype, rra_op_t op, rra_algo_t algo, rra_stream_t stream);

/** Two-shot all-reduce that allocates nothing.  The pages have no
 *  counterpart: this exists for callers that may not allocate device
 *  memory, and so cannot call rra_init (which calls cudaMalloc for its
 *  workspace).  Examples: a plugin inside a framework whose allocator owns
 *  all device memory, or code under a memory budget that forbids new
 *  allocations after start-up.  It needs no rra_init.
 *  - Same arguments, result and summation order as rra_allreduce with
 *    RRA_ALGO_TWO_SHOT (outs[r][i] = SUM_k bufs[k][i], chunk r reduced in
 *    ascending rank order, then gathered back).  The caller passes the
 *    inputs and outputs; in place is allowed as there.
 *  - Scratch: the kernel's status block, call epoch and step flags live in
 *    a static device array of 16,640 bytes inside librra.so, which every
 *    GPU that loads the library holds until the process exits.  It holds
 *    flags for at most 8 ranks x 16 channels; more than 8 ranks is
 *    RRA_ERR_UNSUPPORTED.  Messages of any size are split over at most 16
 *    channels per rank (fewer under rra_set_max_ctas).
 *  - No cudaMalloc, cudaFree or allocating library routine is called.
 *    The first call on a device looks up the array's device address
 *    (cudaGetSymbolAddress, with that device current); make that first
 *    call before any stream capture.
 *  - Every call on a device shares the one array, which keeps the last
 *    call's contents (the flags carry a per-call epoch and need no
 *    clearing; the status block keeps the first device error until
 *    rra_query_status_static reads and clears it).  Calls that overlap on
 *    the GPU -- on two streams without ordering, or together with another
 *    copy of this call -- race on it.
 *  - Device waits are bounded by rra_set_timeout_ns; a wait that expires
 *    ends the kernel early with the outputs partly written, and
 *    rra_query_status_static then returns RRA_ERR_TIMEOUT.  Honours
 *    rra_debug_skip_rank.  Recorded in rra_dump_recent.
 *  Errors: RRA_ERR_INVALID_ARG, RRA_ERR_UNSUPPORTED, RRA_ERR_ALIAS,
 *  RRA_ERR_CUDA.  count == 0 returns RRA_SUCCESS without a launch. */
rra_status_t rra_allreduce_two_shot_static(const void* const* bufs, void* const* outs, int nranks,
                                           size_t count, rra_dtype_t dtype, rra_op_t op,
                                           rra_stream_t stream);

/** Status of rra_allreduce_two_shot_static on the current device, which
 *  allocates nothing either (the pages have no counterpart; it reads the
 *  static scratch array of that entry point, not the workspace of
 *  rra_init).  Synchronizes `stream`, copies the status block to the host
 *  and clears it.  Returns RRA_SUCCESS, the first device error recorded
 *  since the last query (RRA_ERR_TIMEOUT), or RRA_ERR_CUDA.  info (may be
 *  NULL) receives {code, rank, peer, index} as rra_query_status gives it. */
rra_status_t rra_query_status_static(rra_stream_t stream, int32_t info[4]);

/** Reduce-scatter ([ILP] "Direct answer": sum across ranks, each keeps only
 *  its slice).  bufs[r] holds nranks*recvcount elements; outs[r]
 *  (recvcount elements) receives slice r of the sum:
 *  outs[r][i] = SUM_k bufs[k][r*recvcount + i].
 *  - algo RING: chunk c is summed x_{c+1}, ..., x_{c-1}, x_c (the ring's
 *    reduce-scatter half).  DIRECT/TWO_SHOT/AUTO: ascending rank order.
 *  - In place: outs[r] == bufs[r] + r*recvcount elements for every r.
 *  Errors as rra_allreduce; ONE_SHOT is RRA_ERR_INVALID_ARG. */
rra_status_t rra_reduce_scatter(const void* const* bufs, void* const* outs, int nranks,
                                size_t recvcount, rra_dtype_t dtype, rra_op_t op, rra_algo_t algo,
                                rra_stream_t stream);

/** All-gather ([ILP] "Direct answer": each rank holds a shard, every rank
 *  ends with the concatenation).  bufs[r] holds sendcount elements; outs[r]
 *  holds nranks*sendcount: outs[r][q*sendcount + i] = bufs[q][i].
 *  - algo RING: the ring's all-gather half (n-1 forwarding steps).
 *    DIRECT/TWO_SHOT/AUTO: every rank reads every shard directly.
 *    COPY_ENGINE: nranks^2 device-to-device copies on `stream` (no kernel).
 *  - In place: bufs[r] == outs[r] + r*sendcount elements for every r.
 *  The data are copied bit for bit, whatever dtype says.
 *  Errors as rra_allreduce; ONE_SHOT is RRA_ERR_INVALID_ARG. */
rra_status_t rra_all_gather(const void* const* bufs, void* const* outs, int nranks,
                            size_t sendcount, rra_dtype_t dtype, rra_algo_t algo,
                            rra_stream_t stream);

/** All-reduce fused with RMSNorm ([AIH] "Source code": FlashInfer's fused
 *  all-reduce + RMSNorm for tensor-parallel activations).  bufs[r] and
 *  outs[r] hold rows x hidden elements, row-major.  Every rank gets
 *  outs[r][i][j] = s[i][j] * rsqrt(mean_j(s[i][j]^2) + eps) * gamma[j],
 *  where s = SUM_k bufs[k] summed in float32 in ascending rank order (the
 *  one-shot sum).  The normalisation runs in float32; the result is
 *  rounded to dtype once.
 *  - gamma: device pointer, hidden elements of dtype (must not overlap an
 *    output).
 *  - dtype: RRA_FLOAT32 or RRA_BFLOAT16; hidden in [1, 51200]; in place
 *    (outs[r] == bufs[r]) allowed.
 *  Errors: RRA_ERR_INVALID_ARG (int32, null, misaligned, hidden 0),
 *  RRA_ERR_UNSUPPORTED (hidden > 51200, nranks > RRA_MAX_RANKS),
 *  RRA_ERR_ALIAS, RRA_ERR_CUDA.  rows == 0 returns RRA_SUCCESS. */
rra_status_t rra_allreduce_rmsnorm(const void* const* bufs, void* const* outs, int nranks,
                                   size_t rows, size_t hidden, const void* gamma, float eps,
                                   rra_dtype_t dtype, rra_stream_t stream);

/* ------------------------------------------------------------------------ */
/* the training step around a tensor-parallel all-reduce                    */
/* ------------------------------------------------------------------------ */
/*
 * Operators that sit next to the all-reduce in a tensor-parallel training
 * step ([ILP] "Deep dive": a column-parallel layer, then a row-parallel
 * layer, then the all-reduce; [AIH] "Source code": the fused all-reduce +
 * RMSNorm).  Weights are held as one shard per virtual rank, separate
 * buffers; activations that every rank holds alike are passed once (their
 * n copies are the same bytes).  Where a multi-GPU step would all-reduce a
 * partial result (the softmax statistics, the input gradients), the sum
 * over ranks is part of the operator, in float32.
 *
 * Matrices are dense and row-major; dtype is RRA_BFLOAT16 for the
 * operators with matrix products (products of bfloat16 operands summed in
 * float32; others are RRA_ERR_UNSUPPORTED) and RRA_FLOAT32 or RRA_BFLOAT16
 * for the norm.  Matrices that a product reads (x, gates, ups, weights)
 * must be 16-byte aligned (else RRA_ERR_UNSUPPORTED: they are read by bulk
 * tensor copies); rows that are not whole 16-byte units (hidden % 8 != 0)
 * are first copied to padded rows in the workspace.  Every other buffer
 * needs its element's alignment only.
 *
 * The products need rra_init: their bounded internal waits (2 s) report to
 * the device status word, info = {RRA_ERR_TIMEOUT, CTA, -1, which wait}.
 * `workspace` is a device buffer of the caller, 256-byte aligned, of at
 * least the bytes the *_workspace_bytes function gives; its contents need no
 * preparation and mean nothing between calls.
 * Calls with different workspaces may overlap on the GPU; calls that share
 * one must be ordered.  Results do not depend on timing (no atomics).
 * Outputs must not overlap inputs, the workspace or one another
 * (RRA_ERR_ALIAS), but for the in-place forms named below.  A buffer of no
 * elements may be NULL. */

/** Activation of the gated feed-forward block. */
typedef enum {
  RRA_ACT_SILU = 0,     /* g / (1 + exp(-g)) */
  RRA_ACT_GELU_TANH = 1 /* 0.5 g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) */
} rra_act_t;

/** rra_allreduce_rmsnorm that also saves what the backward pass needs
 *  ([AIH] "Source code": the fused all-reduce + RMSNorm; its training
 *  counterpart).  outs as there, bit for bit; and
 *  - codes: rows x hidden bytes, s in 8 bits: per block of 128 columns of a
 *    row (the last one may be short), b = bfloat16(s), e the smallest
 *    integer in [-127, 120] with max |b| <= 448 * 2^e over the block's
 *    finite values, code = e4m3(b * 2^-e), nearest even; a value that is
 *    not finite becomes the NaN code;
 *  - scales: rows x ceil(hidden / 128) bytes, e + 127;
 *  - rstd: rows float32, 1 / sqrt(mean_j(s^2) + eps).
 *  Errors as rra_allreduce_rmsnorm (null codes, scales or rstd too). */
rra_status_t rra_allreduce_rmsnorm_save8(const void* const* bufs, void* const* outs, int nranks, size_t rows,
                                         size_t hidden, const void* gamma, float eps, void* codes, void* scales,
                                         float* rstd, rra_dtype_t dtype, rra_stream_t stream);

/** The activations a checkpoint of rra_allreduce_rmsnorm_save8 stands for
 *  ([AIH] "Source code", as above; the recomputation of a backward pass):
 *  out[i][j] = code * 2^e * rstd[i] * gamma[j], rounded to dtype once.
 *  rstd or gamma (dtype) may be NULL: that factor is left out (both NULL:
 *  the saved sum itself).  Errors: RRA_ERR_INVALID_ARG, RRA_ERR_UNSUPPORTED
 *  (hidden > 51200), RRA_ERR_ALIAS, RRA_ERR_CUDA. */
rra_status_t rra_rmsnorm_restore8(const void* codes, const void* scales, const float* rstd, const void* gamma,
                                  void* out, size_t rows, size_t hidden, rra_dtype_t dtype, rra_stream_t stream);

/** Workspace bytes of rra_allreduce_rmsnorm_backward8 ([AIH] "Source code";
 *  column sums of dgamma). */
size_t rra_allreduce_rmsnorm_backward8_workspace_bytes(size_t rows, size_t hidden);

/** Backward pass of rra_allreduce_rmsnorm_save8 ([AIH] "Source code", as
 *  above).  The ranks' gradients of the normalised rows are summed (float32,
 *  ascending ranks: the all-reduce a column-parallel layer's backward
 *  needs) and taken through the norm, the saved sum read from its 8-bit
 *  checkpoint:
 *    dy = SUM_k grads[k],  h = code * 2^e * rstd,  w = dy * gamma,
 *    dxs[r] = rstd * (w - h * mean_j(w * h))    for every r,
 *    dgamma[j] = SUM_i dy[i][j] * h[i][j]       (float32)
 *  dxs is the gradient of the sum and so of every rank's addend.  In place
 *  (dxs[r] == grads[r]) is allowed.  rows == 0 writes zeros to dgamma.
 *  Errors as rra_allreduce_rmsnorm; RRA_ERR_WORKSPACE. */
rra_status_t rra_allreduce_rmsnorm_backward8(const void* const* grads, void* const* dxs, int nranks, size_t rows,
                                             size_t hidden, const void* codes, const void* scales,
                                             const float* rstd, const void* gamma, float* dgamma, void* workspace,
                                             size_t workspace_bytes, rra_dtype_t dtype, rra_stream_t stream);

/** Workspace bytes of rra_gated_ffn (backward == 0) or
 *  rra_gated_ffn_backward ([ILP] "Deep dive": the column-parallel layer). */
size_t rra_gated_ffn_workspace_bytes(int nranks, size_t tokens, size_t hidden, size_t width, int backward);

/** Column-parallel half of a gated feed-forward block ([ILP] "Deep dive":
 *  column-parallel, then row-parallel).  x: tokens x hidden; gates[r],
 *  ups[r]: width x hidden; acts[r]: tokens x width,
 *    acts[r] = act(x gates[r]^T) * (x ups[r]^T),
 *  both projections, the activation and the product in one kernel, float32
 *  until the one rounding of acts.  tokens == 0 or width == 0 launches
 *  nothing.  Errors: RRA_ERR_INVALID_ARG (null, hidden 0, bad act,
 *  misaligned), RRA_ERR_UNSUPPORTED (dtype, a matrix not 16-byte aligned,
 *  an extent of 2^31 or more, nranks > RRA_MAX_RANKS),
 *  RRA_ERR_NOT_INITIALIZED, RRA_ERR_ALIAS, RRA_ERR_WORKSPACE,
 *  RRA_ERR_CUDA. */
rra_status_t rra_gated_ffn(const void* x, const void* const* gates, const void* const* ups, void* const* acts,
                           int nranks, size_t tokens, size_t hidden, size_t width, rra_act_t act,
                           rra_dtype_t dtype, void* workspace, size_t workspace_bytes, rra_stream_t stream);

/** Backward pass of rra_gated_ffn ([ILP] "Deep dive"): dacts[r] tokens x
 *  width in; dx tokens x hidden (the SUM over ranks, what a multi-GPU step
 *  all-reduces), dgates[r] and dups[r] width x hidden out.  The projections
 *  are computed again from x, not read; dg = dacts * u * act'(g) and
 *  du = dacts * act(g) are rounded to bfloat16 as operands of the gradient
 *  products (up to 128 tokens in two halves, with the rounding's rest as the
 *  second), whose sums are float32.  tokens == 0 writes zeros to dgates
 *  and dups; width == 0 zeros to dx.  Errors as rra_gated_ffn. */
rra_status_t rra_gated_ffn_backward(const void* x, const void* const* gates, const void* const* ups,
                                    const void* const* dacts, void* dx, void* const* dgates, void* const* dups,
                                    int nranks, size_t tokens, size_t hidden, size_t width, rra_act_t act,
                                    rra_dtype_t dtype, void* workspace, size_t workspace_bytes,
                                    rra_stream_t stream);

/** Workspace bytes of rra_vocab_loss (backward == 0) or
 *  rra_vocab_loss_backward ([ILP] "Deep dive": a layer's weights split over
 *  the ranks).  vocab: host array of nranks shard heights.  For the backward
 *  pass this holds pieces of the vocabulary of up to 512 MiB; it also
 *  accepts less, down to rra_vocab_loss_workspace_bytes(..., 2), which holds
 *  a piece of 256 columns (smaller pieces are slower, not different but for
 *  the rounding of dx's float32 sums). */
size_t rra_vocab_loss_workspace_bytes(int nranks, size_t tokens, size_t hidden, const size_t* vocab, int backward);

/** Softmax cross entropy over a vocabulary held as shards of the ranks
 *  ([ILP] "Deep dive"), the logits never kept.  x: tokens x hidden;
 *  weights[r]: vocab[r] x hidden (ranks' rows follow one another in the
 *  vocabulary; a shard may be empty); targets: tokens int64 (device);
 *    l = x W^T,  lse[t] = log SUM_v exp l[t][v],
 *    loss[t] = lse[t] - l[t][targets[t]]   (float32)
 *  loss[t] is 0 where targets[t] == ignore_index and NaN where it is any
 *  other value outside the vocabulary.  tokens == 0 launches nothing.
 *  Errors: RRA_ERR_INVALID_ARG (an empty vocabulary too), and as
 *  rra_gated_ffn. */
rra_status_t rra_vocab_loss(const void* x, const void* const* weights, const size_t* vocab, const int64_t* targets,
                            int nranks, size_t tokens, size_t hidden, int64_t ignore_index, float* loss,
                            float* lse, rra_dtype_t dtype, void* workspace, size_t workspace_bytes,
                            rra_stream_t stream);

/** Gradient of rra_vocab_loss ([ILP] "Deep dive"): grad_loss[t] float32 and
 *  the lse that call gave in; dx (tokens x hidden, summed over all shards)
 *  and dweights[r] (vocab[r] x hidden) out.  Piece by piece of the
 *  vocabulary the logits are computed again,
 *    dl[t][v] = (exp(l[t][v] - lse[t]) - [v == targets[t]]) * grad_loss[t]
 *  is rounded to bfloat16 as operand of the two gradient products, but for
 *  the target's entry, whose rest is added to both results in float32 (up to
 *  32 tokens the products of dweights take the rest of every entry, as
 *  bfloat16); the products' sums are float32.  A row whose target is ignore_index or outside
 *  the vocabulary has a zero gradient, whatever grad_loss holds there (its x
 *  still enters dweights, times zero, and has to be finite).
 *  tokens == 0 writes zeros to dweights.  Errors as rra_vocab_loss. */
rra_status_t rra_vocab_loss_backward(const void* x, const void* const* weights, const size_t* vocab,
                                     const int64_t* targets, const float* lse, const float* grad_loss, void* dx,
                                     void* const* dweights, int nranks, size_t tokens, size_t hidden,
                                     int64_t ignore_index, rra_dtype_t dtype, void* workspace,
                                     size_t workspace_bytes, rra_stream_t stream);

/* ------------------------------------------------------------------------ */
/* the serving step around a tensor-parallel all-reduce                     */
/* ------------------------------------------------------------------------ */
/*
 * Operators of a tensor-parallel forward pass in 4 bits ([AIH] "Source
 * code": the fused all-reduce + RMSNorm of inference frameworks; [ILP] "Deep
 * dive": a column-parallel layer, then a row-parallel layer, then the
 * all-reduce), and the choice of the next token from vocabulary-parallel
 * logits.  Shards, overlap (RRA_ERR_ALIAS), streams and graphs as for the
 * training step's operators; no call needs a workspace.  The products need
 * rra_init: their bounded internal waits (2 s) report to the device status
 * word.  Results do not depend on timing.
 *
 * MX4, microscaled 4-bit floating point: 32 consecutive columns of a row (the
 * last block may be short) share a scale 2^e, e the smallest integer >= -127
 * with max |x| <= 6 * 2^e; code = e2m1(x * 2^-e) (0, 0.5, 1, 1.5, 2, 3, 4, 6
 * and a sign), nearest, ties to even; nothing is clipped.  A block that holds
 * a value that is not finite has scale byte 255 (NaN) and codes 0, and reads,
 * and multiplies, as NaN.  A rows x cols matrix is
 * - codes: rows of 16 * ceil(cols / 32) bytes, column 2i in the low half of
 *   byte i, column 2i + 1 in the high half, zeros behind the last column;
 * - scales: rra_mx4_scale_bytes(rows, cols) bytes, tiles of 128 rows x 4
 *   blocks: the byte e + 127 of (row, block) is number
 *   row % 32 * 16 + row % 128 / 32 * 4 + block % 4 of the 512 of tile
 *   (row / 128, block / 4), the tiles of a row band side by side.  The calls
 *   that write a matrix write 0 for blocks behind the last one of a row and
 *   leave the bytes of rows behind the last one as they were; a matrix made
 *   elsewhere must not have 255 there for blocks behind the last one.
 * Both start on 16 bytes (else RRA_ERR_UNSUPPORTED).  Column-wise splits of a
 * matrix (a row-parallel layer's shards) are quantised each on its own.
 */

/** An MX4 matrix: device pointers.  Calls take host pointers to these, read
 *  during the call only. */
typedef struct {
  void* codes;
  void* scales;
} rra_mx4_t;

/** Bytes of a rows x cols MX4 matrix's scales: 512 * ceil(rows / 128) *
 *  ceil(cols / 128). */
size_t rra_mx4_scale_bytes(size_t rows, size_t cols);

/** x (rows x cols of dtype, RRA_FLOAT32 or RRA_BFLOAT16) in MX4.  Errors:
 *  RRA_ERR_INVALID_ARG, RRA_ERR_UNSUPPORTED (a part of out not 16-byte
 *  aligned, an extent of 2^31 - 1024 or more), RRA_ERR_ALIAS, RRA_ERR_CUDA. */
rra_status_t rra_mx4_quantize(const void* x, const rra_mx4_t* out, size_t rows, size_t cols, rra_dtype_t dtype,
                              rra_stream_t stream);

/** The values of an MX4 matrix: code * 2^e, rounded to dtype once (exact but
 *  for values below its normal range).  Errors as rra_mx4_quantize. */
rra_status_t rra_mx4_restore(const rra_mx4_t* in, void* out, size_t rows, size_t cols, rra_dtype_t dtype,
                             rra_stream_t stream);

/** All-reduce fused with the residual stream, RMSNorm and quantisation
 *  ([AIH] "Source code"): s = SUM_k bufs[k] + residual in float32, ascending
 *  ranks, the residual last; residual_out = s rounded to dtype (the next
 *  layer's residual); out = MX4 of (s * rstd) * gamma, where rstd is the
 *  float32 nearest to 1 / sqrt(mean_j(s^2) + eps) (but for ties within 2^-40)
 *  and both products round to float32, so that the codes depend on no order
 *  of summation.
 *  - residual, residual_out: rows x hidden of dtype; either may be NULL (no
 *    addition; the sum is not stored), and they may be the same.
 *  - gamma: hidden elements of dtype; hidden in [1, 51200].
 *  The squares and their sum have float32's range, its steps of 2^-149 too:
 *  with an eps that small, rows of values below 2^-55 lose bits of rstd.
 *  Errors as rra_allreduce_rmsnorm; RRA_ERR_UNSUPPORTED also for a part of out
 *  not 16-byte aligned. */
rra_status_t rra_allreduce_rmsnorm_mx4(const void* const* bufs, int nranks, size_t rows, size_t hidden,
                                       const void* gamma, float eps, const void* residual, void* residual_out,
                                       const rra_mx4_t* out, rra_dtype_t dtype, rra_stream_t stream);

/** Column-parallel product of MX4 matrices ([ILP] "Deep dive"), such as the
 *  vocabulary head: outs[r] (tokens x widths[r] of dtype, RRA_FLOAT32 or
 *  RRA_BFLOAT16) = X W_r^T for x: tokens x hidden and weights[r]: widths[r] x
 *  hidden.  Products are exact, sums float32, rounded to dtype once.
 *  tokens == 0, or all widths 0, launches nothing.  Errors:
 *  RRA_ERR_INVALID_ARG (null, hidden 0, dtype, misaligned),
 *  RRA_ERR_UNSUPPORTED (an MX4 part not 16-byte aligned, an extent of 2^31 -
 *  1024 or more, more than 2^29 tiles of 256 tokens x 128 weight rows, nranks >
 *  RRA_MAX_RANKS), RRA_ERR_NOT_INITIALIZED, RRA_ERR_ALIAS,
 *  RRA_ERR_CUDA. */
rra_status_t rra_mx4_product(const rra_mx4_t* x, const rra_mx4_t* weights, void* const* outs, int nranks,
                             size_t tokens, size_t hidden, const size_t* widths, rra_dtype_t dtype,
                             rra_stream_t stream);

/** Row-parallel product of MX4 matrices with its all-reduce ([ILP] "Deep
 *  dive"): out (tokens x hidden of dtype) = SUM_r X_r W_r^T for xs[r]: tokens
 *  x width and weights[r]: hidden x width, the sum over ranks in the float32
 *  accumulator.  width == 0 writes zeros; widths of 2^28 - 256 and more are
 *  RRA_ERR_UNSUPPORTED.  Errors as rra_mx4_product. */
rra_status_t rra_mx4_product_sum(const rra_mx4_t* xs, const rra_mx4_t* weights, void* out, int nranks, size_t tokens,
                                 size_t width, size_t hidden, rra_dtype_t dtype, rra_stream_t stream);

/** Column-parallel half of a gated feed-forward block in MX4 ([ILP] "Deep
 *  dive"): acts[r] (tokens x width, MX4) = act(X G_r^T) * (X U_r^T), float32
 *  until the quantisation, for x: tokens x hidden, gates[r] and ups[r]: width x
 *  hidden.  Errors as rra_mx4_product (a bad act too). */
rra_status_t rra_mx4_gated_ffn(const rra_mx4_t* x, const rra_mx4_t* gates, const rra_mx4_t* ups,
                               const rra_mx4_t* acts, int nranks, size_t tokens, size_t hidden, size_t width,
                               rra_act_t act, rra_stream_t stream);

/** The next token of each row, drawn from vocabulary-parallel logits ([ILP]
 *  "Deep dive": a layer's weights split over the ranks).  logits[r]: rows x
 *  vocab[r] of dtype (RRA_FLOAT32 or RRA_BFLOAT16), the vocabulary being the
 *  shards one after another.  Per row, w_j = exp((l_j - max l) / temperature):
 *  - top_k > 0 keeps the top_k largest logits;
 *  - top_p < 1 keeps, of those in falling order, the shortest run whose weight
 *    reaches top_p times theirs (one at least);
 *  - min_p > 0 keeps what weighs min_p or more;
 *  equal logits go by the lowest index.  token = the first index i with
 *  SUM_{j <= i, kept} w_j > uniform * SUM_{kept} w_j, logprob = log(w_token /
 *  SUM_{kept} w_j).  temperature == 0 (as top_k == 1) takes the largest logit.
 *  - uniform: rows float32 in [0, 1) (clamped); temperature, top_k, top_p,
 *    min_p: one value per row (device), or NULL for all rows 1, 0, 1, 0;
 *    logprob: rows float32, or NULL.
 *  - -infinity masks a token; a row of nothing else gives token -1, logprob
 *    -infinity; a row with a NaN logit or a temperature that is NaN or
 *    negative gives token -1, logprob NaN.  Where +infinity occurs its
 *    tokens share the whole weight.
 *  - Weights are held to 29 bits (20 at temperatures above 1e35) and in units
 *    of 2^-44 of the largest, and summed exactly: a token that weighs less than
 *    a unit is never drawn.  Temperatures between 0 and 1.5e-38 count as that.
 *  Vocabulary up to 368640 in all (else RRA_ERR_UNSUPPORTED); under an SM
 *  budget a row still takes the CTAs whose shared memory holds it, up to 8.
 *  Errors:
 *  RRA_ERR_INVALID_ARG, RRA_ERR_UNSUPPORTED, RRA_ERR_ALIAS, RRA_ERR_CUDA. */
rra_status_t rra_vocab_sample(const void* const* logits, const size_t* vocab, int nranks, size_t rows,
                              const float* uniform, const float* temperature, const int32_t* top_k,
                              const float* top_p, const float* min_p, int64_t* token, float* logprob,
                              rra_dtype_t dtype, rra_stream_t stream);

/* ------------------------------------------------------------------------ */
/* LL and LL128 wire formats ([AIH] "Protocols")                            */
/* ------------------------------------------------------------------------ */

/** Bytes of LL wire for a payload: 8 * ceil(payload_bytes / 4).  LL: every
 *  8-byte line holds 4 bytes of data and a 4-byte flag (50% efficiency). */
size_t rra_ll_wire_bytes(size_t payload_bytes);

/** Bytes of LL128 wire: 128 * ceil(payload_bytes / 120).  LL128: every
 *  128-byte line holds 120 bytes of data and an 8-byte flag (93.75%). */
size_t rra_ll128_wire_bytes(size_t payload_bytes);

/** LL pack: line i of `wire` (device, 16-byte aligned,
 *  rra_ll_wire_bytes(payload_bytes) bytes) gets payload bytes [4i, 4i+4) in
 *  its bytes 0..3 (zero past the payload's end) and `flag` (little-endian)
 *  in bytes 4..7.  Lines are written with single 16-byte stores, so a
 *  line's data and flag become visible together.  flag must be nonzero (0
 *  marks an empty line); callers use a step counter 1, 2, ...  `payload`
 *  is a device pointer (any alignment).  Errors: RRA_ERR_INVALID_ARG. */
rra_status_t rra_ll_pack(const void* payload, size_t payload_bytes, void* wire, uint32_t flag,
                         rra_stream_t stream);

/** LL unpack-and-reduce: for every line, poll each of the nsrc wires until
 *  its flag equals expected_flag (a bounded wait, rra_set_timeout_ns), then
 *  write the element-wise SUM of the nsrc data words, sources in ascending
 *  order, to out (payload_bytes bytes, a whole number of dtype elements).
 *  nsrc == 1 is a plain unpack.  wires: host array of nsrc device pointers
 *  (16-byte aligned).  A line whose flag never matches ends the wait with
 *  RRA_ERR_TIMEOUT in the status word: info = {code, source, -1, line}.
 *  Needs rra_init().  Errors: RRA_ERR_INVALID_ARG, RRA_ERR_UNSUPPORTED,
 *  RRA_ERR_NOT_INITIALIZED. */
rra_status_t rra_ll_unpack(const void* const* wires, int nsrc, void* out, size_t payload_bytes,
                           rra_dtype_t dtype, rra_op_t op, uint32_t expected_flag,
                           rra_stream_t stream);

/** LL128 pack: line j (128 bytes) of `wire` gets payload bytes
 *  [120j, 120j+120) in bytes 0..119 (zero past the end) and `flag` as a
 *  little-endian uint64 in bytes 120..127.  A warp writes four lines with
 *  32 16-byte stores.  Other rules as rra_ll_pack. */
rra_status_t rra_ll128_pack(const void* payload, size_t payload_bytes, void* wire, uint64_t flag,
                            rra_stream_t stream);

/** LL128 unpack-and-reduce: a warp reads four lines of each source (one
 *  16-byte load per lane), checks the four flags across the warp, and on a
 *  match sums the 120 data bytes of every line over the sources (ascending
 *  order).  Other rules as rra_ll_unpack. */
rra_status_t rra_ll128_unpack(const void* const* wires, int nsrc, void* out, size_t payload_bytes,
                              rra_dtype_t dtype, rra_op_t op, uint64_t expected_flag,
                              rra_stream_t stream);

/* ------------------------------------------------------------------------ */
/* status, selection, configuration                                         */
/* ------------------------------------------------------------------------ */

/** The asynchronous error of the calls issued so far, as NCCL reports an
 *  asynchronous communicator error ([AIH] "Common environment variables
 *  and debugging": a collective that hangs or fails is found from the
 *  device side, not from the launch).  Synchronize `stream`, then read and
 *  clear the current device's status word.  Returns RRA_SUCCESS, the
 *  recorded device error (RRA_ERR_TIMEOUT) or RRA_ERR_CUDA if the stream
 *  itself failed.  info (may be NULL) receives {code, rank, peer, index}:
 *  the rank (or LL source) whose wait expired, the rank it waited for (-1
 *  if none) and the step (ring, two-shot) or line (LL, LL128) index. */
rra_status_t rra_query_status(rra_stream_t stream, int32_t info[4]);

/** The schedule AUTO uses for an all-reduce of bytes_per_rank bytes per
 *  rank: from the measured table (rra_load_tuning; the table shipped
 *  beside the library is loaded by rra_init) when it has an entry for
 *  nranks and dtype; else from the alpha-beta cost model of [AIH]
 *  "Algorithms" with alpha and beta fitted on this GPU (the table's "ab"
 *  lines): the schedule with the least alpha * syncs(n) + beta * n * S,
 *  syncs being 2(n-1) for the ring, 1 for one-shot, 2 for two-shot and
 *  2 ceil(log2 n) for the tree; with no table loaded, one-shot (on one GPU
 *  every schedule moves the same 2nS bytes and one-shot has the fewest
 *  syncs).  AUTO never runs the tree on buffers that are not 16-byte
 *  aligned.  Never returns RRA_ALGO_AUTO. */
rra_algo_t rra_select_algo(int nranks, size_t bytes_per_rank, rra_dtype_t dtype);

/** Load a tuning table ([AIH] "Algorithms": the alpha-beta crossovers are
 *  only illustrative and must be measured on one's own machine; this is
 *  where the measured ones go): text lines "nranks dtype log2_bytes algo"
 *  (dtype int32|float32|bfloat16, algo ring|one_shot|two_shot|tree), and
 *  prior lines "ab dtype algo alpha_us beta_us_per_MiB" (alpha per
 *  synchronization, beta per MiB of nranks x bytes_per_rank); '#' starts a
 *  comment.  The entry with the largest log2_bytes <= ceil(log2(bytes))
 *  for (nranks, dtype) wins.  NULL clears the table.  Errors:
 *  RRA_ERR_INVALID_ARG (unreadable or malformed file; the old table stays). */
rra_status_t rra_load_tuning(const char* path);

/** Upper bound, in nanoseconds of %globaltimer, on every device-side wait
 *  (ring, tree and two-shot step flags, LL/LL128 line flags).  [AIH]
 *  "Common environment variables and debugging" describes collectives that
 *  wait forever for a rank that never arrives; here every such wait ends
 *  after this bound with RRA_ERR_TIMEOUT in the status word.  Default 500
 *  ms or RRA_TIMEOUT_NS from the environment; 0 restores the default.
 *  Also bounds the waits of rra_allreduce_two_shot_static. */
void rra_set_timeout_ns(uint64_t ns);

/** SM budget ([AIH] "Protocols": each channel is a CUDA block, and
 *  communication kernels compete with compute for SMs): at most
 *  `max_ctas` CTAs per launch (0 = no limit, the default, or RRA_MAX_CTAS
 *  from the environment).  Streaming kernels shrink their grid and loop
 *  longer; ring and two-shot use at most max_ctas / nranks channels (at
 *  least one); the tensor-core products of the training operators run as
 *  pairs of CTAs (at least one). */
void rra_set_max_ctas(int max_ctas);

/** Fault injection for tests: virtual rank `rank` posts no step flag in the
 *  following ring, two-shot (also rra_allreduce_two_shot_static) and tree
 *  calls (-1 turns it off), so its peers' waits expire with RRA_ERR_TIMEOUT
 *  naming it as `peer`.  The GPU stays usable. */
void rra_debug_skip_rank(int rank);

/** Static text for a status code, for the error reports [AIH] "Common
 *  environment variables and debugging" asks to read first when a
 *  collective fails. */
const char* rra_status_string(rra_status_t status);

/** Flight recorder ([AIH] "Common environment variables and debugging":
 *  a record of each rank's recent collectives): writes the last calls
 *  (sequence number, call, algo, nranks, count, dtype, grid, result; grid is
 *  the largest of a call's launches), one per line, oldest first, into buf (NUL-terminated, truncated to len).
 *  Returns the number of calls written. */
int rra_dump_recent(char* buf, size_t len);

#ifdef __cplusplus
}
#endif

#endif /* RRA_H */
