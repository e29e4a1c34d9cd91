/*
 * muon.h: C ABI of the whole-tensor Muon optimizer step on one gfx950 GPU.
 *
 * The operation. A data-parallel rank updates the whole matrices it owns with
 * no communication. This is the "optimizer step (local)" phase of the Canzona
 * analysis page (paper-graph-ui), section 3.4, DP per-iteration execution. The
 * step also equals ΔW = Muon_step(G, States_local) followed by P <- P + ΔW,
 * from the micro-group lifecycle in the same section (steps 2 and 4). The
 * update has the form W_{t+1} = W_t - eta * MatrixOp(W_t, grad W_t) (same page,
 * section 2). Muon's MatrixOp orthogonalises the whole gradient with
 * Newton-Schulz iterations, and the momentum buffer is state that stays on the
 * owning rank (section 3.4, "Task abstraction").
 *
 * For every matrix (rows r, cols c) one step computes:
 *   M' = beta*M + G                          momentum, updated in place
 *   U  = G + beta*M'   (nesterov; else M')
 *   X0 = U (or U^T if r > c, so X is m x n with m <= n) / (||U||_F + eps)
 *   T times: A = X X^T;  B = b*A + c*A*A;  X = a*X + B X
 *   O  = X (or X^T if r > c)
 *   W' = W - lr * sqrt(max(1, r/c)) * O      weights, updated in place
 *
 * Beside the step: the tensor-parallel local update, the host-side planners,
 * and the layer operators that make the gradients it reads.
 *
 * Conventions for every function:
 * - It returns muon_status (0 = MUON_OK) and never throws or aborts across the
 *   ABI. On error, muon_last_error() gives this thread's message.
 * - Pointers named w, g, m and delta are device pointers. They address
 *   row-major, contiguous matrices of the plan's dtype (MUON_BF16_F32_MASTER:
 *   fp32 w, m and delta with a bf16 g).
 * - Every other pointer is a host pointer.
 */
#ifndef MUON_H_
#define MUON_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MUON_OK = 0,
  MUON_ERR_INVALID_ARG = -1, /* null/negative/non-finite argument, bad shape   */
  MUON_ERR_ALIAS = -2,       /* two device ranges of the batch overlap         */
  MUON_ERR_ALIGN = -3,       /* a device pointer is not 16-byte aligned        */
  MUON_ERR_UNSUPPORTED = -4, /* dtype or option not supported                  */
  MUON_ERR_HIP = -5,         /* a HIP runtime call failed (message has it)     */
  MUON_ERR_OOM = -6          /* workspace allocation failed                    */
} muon_status;

typedef enum {
  MUON_F32 = 0,  /* W, G, M fp32; all arithmetic fp32 (fp32 MFMA)          */
  MUON_BF16 = 1, /* W, G, M bf16; bf16 MFMA with fp32 accumulation,         */
                 /* intermediates stored bf16 (round to nearest even)      */
  MUON_BF16_F32_MASTER = 2
                 /* fp32 master weights and momentum with bf16 gradients,  */
                 /* the training setup of the pages (Canzona analysis page, */
                 /* section 3.4, the Atomicity Constraint): W, M and delta  */
                 /* fp32, G bf16; X, A and B bf16 as for MUON_BF16, and     */
                 /* W' = W - lr*s*O formed in fp32 and stored fp32         */
} muon_dtype;

/* One matrix of the batch: rows x cols, row-major, contiguous.
 * w     weights, updated in place. May be NULL when delta is set.
 * g     gradient, read only.
 * m     momentum buffer, updated in place.
 * delta optional (NULL = none). When set, it receives
 *       Delta W = -lr*sqrt(max(1,r/c))*O, the update that the host rank
 *       returns in the micro-group lifecycle (Canzona analysis page, section
 *       3.4, step 2).
 * All four ranges must be 16-byte aligned and must not overlap any other
 * range of the batch. */
typedef struct {
  void* w;
  const void* g;
  void* m;
  void* delta;
  int64_t rows;
  int64_t cols;
} muon_matrix;

/* Hyperparameters. muon_hparams_default() fills in:
 * lr = 0.02, beta = 0.95, eps = 1e-7, (a,b,c) = (3.4445, -4.7750, 2.0315),
 * ns_steps = 5, nesterov = 1, dtype = MUON_BF16. */
typedef struct {
  float lr;
  float beta;     /* momentum, 0 <= beta < 1                               */
  float eps;      /* added to the Frobenius norm, eps >= 0                 */
  float a, b, c;  /* Newton-Schulz polynomial a*x + b*x^3 + c*x^5          */
  int32_t ns_steps; /* >= 0; 0 applies the normalised direction itself    */
  int32_t nesterov; /* 0 or 1                                              */
  int32_t dtype;    /* muon_dtype                                          */
} muon_hparams;

typedef struct muon_plan_s* muon_plan_t;

/* Fills *hp with the defaults listed above. Returns INVALID_ARG if hp is NULL. */
muon_status muon_hparams_default(muon_hparams* hp);

/* Builds a static plan for a batch of n matrices. The plan is computed once
 * and reused every step; the pages' planners likewise run once at
 * initialisation (Canzona analysis page, section 3.3 "Output and offline
 * nature").
 * mats  host array of n descriptors. The plan keeps the device pointers, so
 *       the tensors must stay allocated and unmoved until muon_plan_destroy.
 * hp    host pointer to the hyperparameters (copied).
 * out   receives the plan handle (NULL on error).
 * Every argument is validated before any HIP call. Errors: INVALID_ARG (n < 1,
 * null pointers, rows or cols < 1 or > 2^24 (> 2^23 for MUON_F32),
 * non-finite lr/beta/eps/a/b/c, beta outside [0,1), eps < 0, ns_steps < 0),
 * ALIAS, ALIGN, UNSUPPORTED (dtype). Then the
 * plan allocates and zeroes its device workspace on the current device: HIP
 * or OOM on failure. The call synchronises the device once, at its end. */
muon_status muon_plan(const muon_matrix* mats, int32_t n, const muon_hparams* hp,
                      muon_plan_t* out);

/* Device workspace bytes held by the plan (written to *bytes). */
muon_status muon_plan_workspace_bytes(muon_plan_t plan, size_t* bytes);

/* Enqueues one step over the whole batch on `stream` (a hipStream_t; NULL is
 * the null stream). It is asynchronous: no host synchronisation and no
 * allocation. Launch errors return HIP; faults surface at the caller's next
 * synchronisation. A plan must not be stepped concurrently on two streams,
 * because its work-queue counters live in its workspace. Matrices are
 * independent, and the result does not depend on descriptor order. For a
 * fixed plan the result is bitwise deterministic.
 * A step only launches kernels and records and waits on events (no memset,
 * copy or host synchronisation; the work-queue counters are cleared by the
 * step's own kernels), so it may be captured in a HIP graph on `stream` and
 * the graph replayed; a replay equals an eager step bit for bit. Kernel
 * timing (muon_plan_set_timing) must be off during capture. */
muon_status muon_step(muon_plan_t plan, void* stream);

/* Frees the plan and its workspace. NULL is a no-op. Synchronises the device. */
muon_status muon_plan_destroy(muon_plan_t plan);

/* Bytes of the static device scratch that muon_step_noalloc works in. */
#define MUON_NOALLOC_SCRATCH_BYTES (64u << 20)

/* One step that allocates nothing, for callers that cannot allocate device
 * memory: code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc. It computes what muon_plan, one muon_step and
 * muon_plan_destroy compute, bit for bit, but keeps its workspace (the
 * Newton-Schulz buffers, norm partials, work-queue counters and tile tables)
 * in a static device array of MUON_NOALLOC_SCRATCH_BYTES (64 MiB), one per
 * GPU, which the library holds from its first use on that GPU until the
 * process ends. It calls no hipMalloc or hipFree and creates no stream or
 * event: everything is enqueued on `stream` (a hipStream_t; NULL is the null
 * stream) as one chain of launches: a fill kernel clears the workspace,
 * small kernels copy the tables in (their bytes travel as kernel arguments),
 * then the step's kernels run. Host-side bookkeeping (building the tables) uses
 * ordinary host memory.
 * mats, n, hp: as for muon_plan (the same validation and errors), device
 * pointers on the current device. The tensors must stay valid until the step
 * has run on the stream.
 * Errors: those of muon_plan's validation; INVALID_ARG if the batch's
 * workspace exceeds the scratch (the message gives both sizes); HIP.
 * Every call on a GPU works in that GPU's one array, which keeps the last
 * call's contents: calls that overlap on one GPU (on two streams without an
 * ordering between them, or from two threads) race and give wrong results.
 * Calls issued one after another on one stream are safe. */
muon_status muon_step_noalloc(const muon_matrix* mats, int32_t n, const muon_hparams* hp, void* stream);

/* This thread's last error message ("" if none). Valid until this thread's
 * next call into the library. */
const char* muon_last_error(void);

/* Kernel kinds, for the timing counters below. */
typedef enum {
  MUON_K_MOMENTUM = 0, /* fused momentum + Nesterov + sum-of-squares partials */
  MUON_K_NORM = 1,     /* fixed-order norm reduction to 1/(||U||+eps)        */
  MUON_K_GRAM = 2,     /* symmetric A = X X^T (upper tiles, mirrored)        */
  MUON_K_SQUARE = 3,   /* B = b*A + c*A*A (upper tiles, mirrored)            */
  MUON_K_UPDATE = 4,   /* X = a*X + B X; on the last step, the weight apply  */
  MUON_K_APPLY = 5,    /* weight apply when ns_steps == 0                    */
  MUON_K_GRAM_REDUCE = 6, /* sum of split-K Gram pieces, then A's epilogue   */
  MUON_K_COUNT = 7
} muon_kernel_kind;

/* enable != 0: every later muon_step records a HIP event pair on its stream
 * around each kernel launch. Timing is off by default. */
muon_status muon_plan_set_timing(muon_plan_t plan, int32_t enable);

/* Waits for the recorded events and adds their durations to per-kind totals.
 * Then writes, for kind k in [0, MUON_K_COUNT):
 *   total_ms[k] = summed launch durations;
 *   launches[k] = number of launches.
 * Either array may be NULL. Totals accumulate until muon_plan_reset_timing. */
muon_status muon_plan_kernel_times(muon_plan_t plan, double* total_ms, int64_t* launches);
muon_status muon_plan_reset_timing(muon_plan_t plan);

/* Plan facts, for logs and benchmarks (host pointers; any may be NULL):
 * n_tiles[k] = tiles per launch of kind k (K1 tiles for MOMENTUM);
 * grid[k]    = workgroups launched per launch of kind k. */
muon_status muon_plan_info(muon_plan_t plan, int64_t* n_tiles, int64_t* grid);

/* ---------------------------------------------------------------------------
 * Tensor-parallel local update.
 *
 * Under tensor parallelism a rank holds shards of each weight matrix: a
 * column-parallel layer splits the output dimension (a block of rows of the
 * rows x cols W), a row-parallel layer the input dimension (a block of
 * columns) (Canzona analysis page, section 2, "The Core Problem"). The host
 * rank of a tensor runs muon_step on the whole matrix with delta set (and w
 * NULL); the update is then cut into the TP partition's slices, and every rank
 * adds its slices to its parameter shards, P_local <- P_local + Delta W_local,
 * element by element and with no communication (section 3.4, "The TP Task
 * Abstraction", micro-group lifecycle, steps 3 and 4).
 *
 * One shard: p and d are device pointers of the plan's dtype.
 * p     the local parameter shard, rows x cols, row stride ldp elements,
 *       updated in place;
 * d     its update slice, rows x cols, row stride ldd elements, read only
 *       (a view into a delta matrix, or a buffer the shard arrived in).
 * A column block of a row-major matrix is such a view: its first element and
 * the matrix's row stride. */
typedef struct {
  void* p;
  const void* d;
  int64_t rows;
  int64_t cols;
  int64_t ldp;
  int64_t ldd;
} muon_shard;

typedef struct muon_apply_plan_s* muon_apply_plan_t;

/* Builds a static plan over n shards; the TP layout is fixed at
 * initialisation, as the pages' assignment of tensors is. shards is a host
 * array; the plan keeps the device pointers. Every argument is validated
 * before any HIP call. Errors: INVALID_ARG (n < 1, null pointers, rows or
 * cols < 1 or > 2^24, ldp or ldd < cols, more than 2^31 - 1 tiles of 16 rows
 * x 1 KB),
 * ALIGN (p or d not aligned to the element size), ALIAS (an element of a p
 * view is also in another p view or in a d view; d views may share elements),
 * UNSUPPORTED (dtype). Two views with the same row stride are checked element
 * by element (column blocks of one matrix are disjoint); views with different
 * strides whose address ranges overlap are rejected. Then the plan copies its
 * shard table to the current device: HIP or OOM on failure. The call
 * synchronises the device once, at its end. */
muon_status muon_apply_plan(const muon_shard* shards, int32_t n, int32_t dtype,
                            muon_apply_plan_t* out);

/* Enqueues P_local <- P_local + Delta W_local for every shard of the plan on
 * `stream` (a hipStream_t; NULL is the null stream): one kernel, no
 * allocation, no host synchronisation. Each sum is formed in fp32 and stored
 * once (bf16: round to nearest even), which for two values of the storage type
 * is their exactly rounded sum. Shards are independent and the result does not
 * depend on their order. The call may be captured in a HIP graph on `stream`. */
muon_status muon_apply(muon_apply_plan_t plan, void* stream);

/* Frees the plan. NULL is a no-op. Synchronises the device. */
muon_status muon_apply_plan_destroy(muon_apply_plan_t plan);

/* ---------------------------------------------------------------------------
 * MFMA throughput probe (measurement, not part of the step). Enqueues one
 * kernel of `blocks` workgroups of 4 waves on `stream`; every wave issues
 * iters * 8 bf16 MFMAs of 32 x 32 x 16 (32768 flops each) back to back on
 * random register data and stores one sum per lane into out (a device buffer
 * of blocks * 256 floats). Timed by the caller, it gives the bf16 MFMA rate
 * the chip sustains on random data under its power limit, against which the
 * step's rate can be read. It is a measurement aid, not an operation of the
 * pages' method. Errors:
 * INVALID_ARG (out NULL, blocks outside [1, 2^20], iters < 1), HIP. */
muon_status muon_mfma_probe(float* out, int32_t blocks, int32_t iters, void* stream);

/* ---------------------------------------------------------------------------
 * Data-parallel static partition: which whole parameters each DP rank owns
 * (host only, no GPU). A rank's share is the batch it passes to muon_plan.
 *
 * The parameter buffer is a list of n_buckets buckets; bucket i is an ordered
 * run of bucket_len[i] atomic parameters. sizes[] holds the element count of
 * every parameter, bucket after bucket; loads[] (NULL: the sizes) holds its
 * load W(p). On return, cuts[i*(ranks+1) + r] .. cuts[i*(ranks+1) + r+1] - 1
 * are the parameters of bucket i that rank r owns (cuts are parameter indices
 * within the bucket: 0 first, bucket_len[i] last, non-decreasing), and
 * rank_loads[r] (if not NULL) is rank r's total load. Errors: INVALID_ARG
 * (null sizes, bucket_len or cuts; n_buckets < 1; ranks outside [1, 2^20];
 * an empty bucket; a size outside [1, 2^40]; a negative or non-finite load;
 * alpha outside [0, 1]). */

/* The Start_Index rule without load balancing (Canzona analysis page,
 * section 3.4, "Paradigm 3: Static Partitioning"): with S = |B_i| / R, a
 * parameter whose first element lies in [r S, (r+1) S) of its bucket belongs
 * to rank r (evaluated exactly, in integers). */
muon_status muon_dp_partition_static(const int64_t* sizes, const double* loads, const int32_t* bucket_len,
                                     int32_t n_buckets, int32_t ranks, int32_t* cuts, double* rank_loads);

/* The alpha-Balanced Greedy LPT algorithm (same section, "Algorithm 1"):
 * buckets in descending load order (equal loads keep their order); per bucket,
 * deficits d_r = max(0, mu - L_r) against the mean load mu, the target share
 * v_r = (1 - alpha)/R + alpha d_r / sum(d) (1/R when every deficit is 0), and
 * the cut of rank r < R-1 at the parameter boundary whose cumulative load is
 * closest to the cumulative target (the earlier one on a tie, never before
 * rank r-1's cut); the last rank takes the rest. O(N log N + N R log P) for N
 * buckets of at most P parameters. */
muon_status muon_dp_partition(const int64_t* sizes, const double* loads, const int32_t* bucket_len,
                              int32_t n_buckets, int32_t ranks, double alpha, int32_t* cuts, double* rank_loads);

/* TP micro groups (host only; Canzona analysis page, section 3.4, "The TP
 * Hierarchical Partitioning and Scheduling", the LPT with greedy rollback and
 * its min-heap solver). n tensors with costs cost[i] (their ID is i) are
 * sorted by (cost, ID) descending and packed, in that order, into groups: a
 * tensor joins the current group if the min-heap LPT assignment of the group
 * (by cost descending, each tensor to the least-loaded of `ranks` host ranks,
 * the lower rank on a tie) keeps every rank's load within c_max; otherwise the
 * group closes and the tensor starts the next one (a tensor heavier than
 * c_max alone forms its own group). On return order[] holds the IDs in
 * schedule order (every group a consecutive run), group_of[i] and host_of[i]
 * the group and host rank of tensor i, and *n_groups the number of groups.
 * Every tentative group is solved again, as the pages do: O(n K log K) for
 * groups of up to K tensors (milliseconds for thousands of tensors in groups
 * of tens). Errors: INVALID_ARG (null pointers, n < 1, ranks outside [1, 2^20], c_max
 * not finite and > 0, a negative or non-finite cost). */
muon_status muon_tp_micro_groups(const double* cost, int32_t n, int32_t ranks, double c_max, int32_t* order,
                                 int32_t* group_of, int32_t* host_of, int32_t* n_groups);

/* ---------------------------------------------------------------------------
 * Layer operators: what a training step runs around the optimizer step, from a
 * block's norms to the weight gradients that muon_step reads. Activations that
 * the backward pass needs are kept in 8 bits.
 *
 * These calls keep nothing: every one takes its descriptors by value of the
 * call, only launches kernels on `stream` (no allocation, copy, memset or host
 * synchronisation), and may be captured in a HIP graph. Results are bitwise
 * deterministic. Arguments are validated before any HIP call. rows may be 0
 * (weight gradients are then 0, or beta*C); views without rows may be NULL.
 * Device pointers named below address row-major views, rows x cols with a row
 * stride in elements (ld*, at least cols, at most 2^24); any alignment to the
 * element size and any stride is right, and views with 16-byte aligned rows and
 * cols a multiple of 8 take the fast path. Written views must not overlap any
 * other view of the call (ALIAS; column blocks of one buffer may lie side by
 * side, but views of different row strides in bytes must not reach into each
 * other's address range); views that are only read may share elements.
 *
 * 8-bit checkpoints. A row of cols elements is cut into groups of 32 columns
 * (the last may be shorter). A group has one exponent byte E; an element is
 * one byte q and stands for q * 2^(E-127), q being an int8 in [-127, 127]
 * (MUON_Q8_INT8) or an e4m3 number of at most 448 (MUON_Q8_E4M3).
 * Saving chooses the smallest E >= 17 with max|x| <= 127 * 2^(E-127) (int8; 448
 * for e4m3) over the group, so nothing saturates, and rounds x / 2^(E-127) to
 * nearest, ties to even. A group holding an infinity or a NaN gets E = 255 and
 * q = 0 and stands for NaNs, so that a bad activation shows up in the gradients.
 * Every finite value that a saved checkpoint stands for is exactly a bf16 number.
 * At the end of fp32's range some are not finite: int8 elements of at least
 * 1.984375 * 2^127 in a group whose largest is above that, and e4m3 elements of
 * at least 1.9375 * 2^127, round to 2^128, an infinity, as the largest fp32
 * numbers do in bf16. E of 0 to 16 is not written and not meant to be read.
 * int8 is the more accurate of the two for activations whose groups
 * are near Gaussian (0.7% against 2.6% relative error), e4m3 where elements of
 * a group differ by more than two orders of magnitude.
 *
 * q     rows x ldq bytes, 16-byte aligned, ldq a multiple of 16 and >= cols;
 *       the bytes between cols and the next multiple of 16 are padding, which
 *       the library may read and write;
 * e     rows x lde bytes, lde >= ceil(cols / 32). */
typedef enum { MUON_Q8_INT8 = 0, MUON_Q8_E4M3 = 1 } muon_q8_kind;

typedef struct {
  void* q;
  void* e;
  int64_t rows;
  int64_t cols;
  int64_t ldq;
  int64_t lde;
  int32_t kind; /* muon_q8_kind */
  int32_t reserved;
} muon_q8;

/* Saves x (out->rows x out->cols, row stride ldx, MUON_F32 or MUON_BF16) into
 * the checkpoint out. Errors: INVALID_ARG (null pointers, rows outside
 * [0, 2^30], cols outside [1, 2^24], strides), ALIGN, ALIAS, UNSUPPORTED
 * (dtype, kind), HIP. */
muon_status muon_q8_save(const void* x, int64_t ldx, int32_t dtype, const muon_q8* out, void* stream);

/* Loads a checkpoint: x gets the values it stands for (fp32, or bf16, which
 * holds them exactly). Same errors. */
muon_status muon_q8_load(const muon_q8* in, void* x, int64_t ldx, int32_t dtype, void* stream);

/* The norm site between two blocks: the norm after a block, its gate and the
 * residual scales, the residual sum, and the norm before the next block, row
 * by row in one pass:
 *   v = branch / rms(branch)             (v = branch if w_post is NULL)
 *   y = res_scale*residual + branch_scale * gate * w_post * v
 *   u = y / rms(y),   h = w_pre * u      rms(x) = sqrt(mean(x^2) + eps)
 * All arithmetic is fp32; y and h are rounded to dtype once, at the end (h is
 * formed from the unrounded y).
 * branch, residual  rows x cols, read only
 * w_pre, w_post     cols elements; w_post may be NULL (no norm after the block)
 * gate              NULL (1), cols elements with ld_gate = 0 (one gate for all
 *                   rows), or rows x cols with row stride ld_gate >= cols
 * y, h              rows x cols, written
 * rstd_y, rstd_b    rows floats, 1/rms(y) and 1/rms(branch), written if not
 *                   NULL, with or without w_post; a backward pass needs rstd_y, and rstd_b with w_post
 * u, v              8-bit checkpoints, written if their q is not NULL; a
 *                   backward pass needs u, and v with w_post or gate
 * cols is at most 32768. Up to 8192 columns (backward pass: 6144) a row is read
 * once and stays in registers; wider rows are read again from cache or spill, and
 * run at a fraction of the memory's rate (a backward pass of 16384 bf16 columns
 * takes 6 times its bytes' time). */
typedef struct {
  int64_t rows;
  int64_t cols;
  const void* branch;
  int64_t ld_branch;
  const void* residual;
  int64_t ld_residual;
  const void* w_pre;
  const void* w_post;
  const void* gate;
  int64_t ld_gate;
  void* y;
  int64_t ld_y;
  void* h;
  int64_t ld_h;
  float* rstd_y;
  float* rstd_b;
  muon_q8 u;
  muon_q8 v;
  float res_scale;
  float branch_scale;
  float eps;
  int32_t dtype; /* MUON_F32 or MUON_BF16, of every tensor but rstd, u and v */
} muon_norm_site;

/* Errors: INVALID_ARG (null pointers, sizes, strides, non-finite scales,
 * eps < 0), ALIGN, ALIAS, UNSUPPORTED (dtype, kind, cols > 32768), HIP. */
muon_status muon_norm_forward(const muon_norm_site* site, void* stream);

/* Gradients of a norm site from its checkpoints. dy and dh are the gradients
 * of y (NULL: zero) and h. With s the whole gradient of y,
 *   s          = dy + rstd_y*(du - u*mean(du*u)),     du = w_pre*dh
 *   d_residual = res_scale*s
 *   d_branch   = rstd_b*(dv - v*mean(dv*v)),          dv = branch_scale*s*gate*w_post
 *                (dv itself if w_post is NULL)
 *   d_w_pre    = sum over rows of dh*u
 *   d_w_post   = sum over rows of branch_scale*s*gate*v
 *   d_gate     = branch_scale*s*w_post*v, summed over rows if ld_gate is 0
 * d_w_pre, d_w_post (cols elements) and d_gate (cols elements, or rows x cols
 * with row stride ld_d_gate) may be NULL: not wanted. Weight gradients are
 * summed in fp32 in a fixed order and rounded to dtype once.
 * workspace: device memory of at least muon_norm_backward_workspace bytes,
 * 16-byte aligned, scratch of this call until it has run. */
typedef struct {
  const void* dy;
  int64_t ld_dy;
  const void* dh;
  int64_t ld_dh;
  void* d_residual;
  int64_t ld_d_residual;
  void* d_branch;
  int64_t ld_d_branch;
  void* d_w_pre;
  void* d_w_post;
  void* d_gate;
  int64_t ld_d_gate;
  void* workspace;
  size_t workspace_bytes;
} muon_norm_grads;

/* Reads rows, cols, w_pre, w_post, gate, rstd_y, rstd_b, u, v, the scales and
 * dtype of site (branch, residual, y and h may be NULL). Errors: those of
 * muon_norm_forward, and INVALID_ARG for a missing or short workspace or a
 * gradient of a weight that the site does not have. */
muon_status muon_norm_backward(const muon_norm_site* site, const muon_norm_grads* grads, void* stream);

/* Workspace bytes of muon_norm_backward for rows x cols (host, no GPU). */
muon_status muon_norm_backward_workspace(int64_t rows, int64_t cols, size_t* bytes);

/* One weight gradient of a linear layer Y = X W^T, from the saved input:
 *   G = dY^T (X diag(scale)) + beta*C
 * dy     rows x n, dtype, row stride ld_dy: the gradient of the output
 * x      rows x k checkpoint of the input
 * scale  NULL, or k elements of dtype: a norm weight, when x is the normalised
 *        row u of a norm site and the layer's input was h = w_pre * u
 * g      n x k, contiguous, g_dtype, 16-byte aligned: what muon_matrix.g takes
 * c      n x k, contiguous, g_dtype, 16-byte aligned: read if beta != 0; may
 *        be g itself (accumulation over micro batches)
 * bf16 dY: bf16 MFMA with fp32 accumulation; the products are exact, since
 * checkpoint values are bf16 numbers. fp32 dY is cut into three bf16 numbers
 * that add up to it (24 bits; of numbers below 2^-110 the bits down to 2^-133,
 * the smallest bf16 number), for fp32 accuracy on the bf16 matrix cores. Where x
 * stands for an infinity, its column of G is infinite or NaN, with fp32 dY NaN
 * in general (some of the three numbers are 0).
 * g is rounded to g_dtype once. */
typedef struct {
  const void* dy;
  int64_t ld_dy;
  muon_q8 x;
  const void* scale;
  void* g;
  const void* c;
  int64_t n;
  float beta;
  int32_t reserved;
} muon_wgrad_item;

/* Weight gradients of n_items layers in one go (few layers alone fill the
 * GPU). dtype (of dy and scale) and g_dtype are MUON_F32 or MUON_BF16; every
 * x has the same kind. Errors: INVALID_ARG (null pointers, n or cols outside
 * [1, 2^24], rows outside [0, 2^30], strides, non-finite beta, a short
 * workspace, checkpoints of different kinds, more than 2^22 output tiles), ALIGN, ALIAS (c == g is fine),
 * UNSUPPORTED, HIP. workspace is scratch of this call until it has run:
 * muon_wgrad_workspace bytes (which may be 0), 16-byte aligned.
 * muon_wgrad_workspace makes the same checks of the items, without a GPU. */
muon_status muon_wgrad(const muon_wgrad_item* items, int32_t n_items, int32_t dtype, int32_t g_dtype,
                       void* workspace, size_t workspace_bytes, void* stream);
muon_status muon_wgrad_workspace(const muon_wgrad_item* items, int32_t n_items, int32_t dtype, int32_t g_dtype,
                                 size_t* bytes);

/* How muon_wgrad runs these items, without a GPU: item i in output tiles of
 * tile[i] x tile[i] (256, 128 or 64, of its launch of 16 items), its sum over
 * rows in pieces[i] pieces that a second launch adds. Same checks and errors as
 * muon_wgrad_workspace. */
muon_status muon_wgrad_info(const muon_wgrad_item* items, int32_t n_items, int32_t dtype, int32_t g_dtype,
                            int32_t* tile, int32_t* pieces);

/* The gated feed-forward block of a layer,
 *   a = x Wgate^T,  b = x Wup^T,  s = act(a) * b,  y = s Wdown^T,
 * in two launches: both projections, the activation and the product are one. (fp32
 * operands, and bf16 ones that are not 16-byte aligned, are rewritten by a launch
 * before; where there are few tiles, a launch after joins the pieces of their sums.)
 * dtype is that of x, y and the weights. Sums are fp32; s is rounded to dtype
 * once, as the operand of the last product (to 16 bits where one or two rows keep
 * no checkpoints), y once. bf16: bf16 MFMA. fp32: every operand is cut into three
 * bf16 numbers that add up to it (24 bits, of numbers below 2^-110 fewer), and the
 * six products down to 2^-24 of the largest are summed: fp32 accuracy at six times
 * the work. Infinities are what they are in an fp32 sum, but for products with
 * numbers below 2^-62, which may be NaN.
 * x       rows x width
 * w_gate, w_up  inner x width, w_down  out x inner, contiguous (muon_matrix.w)
 * y       rows x out, written (NULL: only the checkpoints are wanted)
 * a, b, s rows x inner checkpoints of the unrounded a, b and s, written if their q
 *         is not NULL, all of the same kind; a backward pass needs a and b, the
 *         weight gradient of w_down (muon_wgrad) s
 * width, inner and out are at most 2^22, and so are the row strides of y, d_x, d_a
 * and d_b.
 * workspace: device memory of at least muon_mlp_exact_workspace bytes
 * (muon_mlp_workspace for any tensors of these sizes), 16-byte aligned, scratch of a
 * call until it has run; a call on it in a captured graph writes it anew with every
 * replay.
 * act: MUON_ACT_SILU a/(1+e^-a), MUON_ACT_GELU a Phi(a) (Phi the normal
 * distribution), MUON_ACT_GELU_TANH its approximation by a tanh, a (1 +
 * tanh(sqrt(2/pi) (a + 0.044715 a^3))) / 2, MUON_ACT_RELU max(a, 0). */
typedef enum { MUON_ACT_SILU = 0, MUON_ACT_GELU = 1, MUON_ACT_GELU_TANH = 2, MUON_ACT_RELU = 3 } muon_act;

typedef struct {
  int64_t rows;
  int64_t width;
  int64_t inner;
  int64_t out;
  const void* x;
  int64_t ld_x;
  const void* w_gate;
  const void* w_up;
  const void* w_down;
  void* y;
  int64_t ld_y;
  muon_q8 a;
  muon_q8 b;
  muon_q8 s;
  void* workspace;
  size_t workspace_bytes;
  int32_t act;   /* muon_act */
  int32_t dtype; /* MUON_F32 or MUON_BF16 */
} muon_mlp;

/* Errors: INVALID_ARG (null pointers, sizes, strides, a short workspace, a call
 * that writes nothing), ALIGN, ALIAS, UNSUPPORTED (dtype, act, kind), HIP. */
muon_status muon_mlp_forward(const muon_mlp* mlp, void* stream);

/* Gradients of the block from its checkpoints, dy (rows x out) being that of y:
 *   ds = dy Wdown,  d_a = ds * b * act'(a),  d_b = ds * act(a),
 *   d_x = d_a Wgate + d_b Wup   (NULL: not wanted)
 * d_a and d_b, rows x inner, are what muon_wgrad takes for w_gate and w_up. ds
 * stays fp32; d_a and d_b are rounded once, and d_x is summed from the rounded
 * ones. Reads rows, width, inner, out, the weights, a, b, act, dtype and the
 * workspace of mlp (x, y and s may be NULL). Same errors. */
typedef struct {
  const void* dy;
  int64_t ld_dy;
  void* d_x;
  int64_t ld_d_x;
  void* d_a;
  int64_t ld_d_a;
  void* d_b;
  int64_t ld_d_b;
} muon_mlp_grads;

/* The workspace may be the forward pass's: nothing in it is carried over. */
muon_status muon_mlp_backward(const muon_mlp* mlp, const muon_mlp_grads* grads, void* stream);

/* Workspace bytes that both passes of this block get along with, whatever the
 * alignment and the strides of its tensors (host, no GPU; reads rows, width, inner,
 * out and dtype). */
muon_status muon_mlp_workspace(const muon_mlp* mlp, size_t* bytes);

/* What one pass asks for with the tensors given, forward (grads NULL) or backward:
 * operands that are read where they lie take none of it, so that of aligned bf16
 * tensors it is s, or nothing, and the pieces of sums. x, the weights, dy, d_a and
 * d_b that are NULL count as unaligned ones (host, no GPU; reads those pointers and
 * their strides, and which of y, d_x and the checkpoints are wanted). */
muon_status muon_mlp_exact_workspace(const muon_mlp* mlp, const muon_mlp_grads* grads, size_t* bytes);

/* How a pass cuts its two products up, forward (grads NULL: the projections, y) or
 * backward (ds, d_x): the edge of the output tiles (0: a kernel for at most 16 rows, or
 * no product), how many tiles are summed whole, and the pieces that the sums of the
 * others are cut into (1: there are none). Two numbers each (host, no GPU; reads what
 * muon_mlp_exact_workspace reads). */
muon_status muon_mlp_info(const muon_mlp* mlp, const muon_mlp_grads* grads, int32_t* tile, int32_t* whole, int32_t* pieces);

/* Weights in 8 bits. An n x k weight is cut into blocks of 128 x 128 (those at the
 * edges may be smaller). A block has one exponent byte E, an element is one e4m3
 * byte q and stands for q * 2^(E-127); E and q are chosen as for a checkpoint (E =
 * 255 and q = 0, NaNs, where a block holds an infinity or a NaN).
 * q     n x ldq bytes, e4m3
 * qt    k x ldqt bytes, the same transposed, for products with W itself; or NULL
 * e     ceil(n / 128) x lde bytes, lde >= ceil(k / 128)
 * q and qt 16-byte aligned, ldq and ldqt multiples of 16; the bytes between k (n)
 * and the next multiple of 16 are padding, which the library may read and write. */
typedef struct {
  void* q;
  void* qt;
  void* e;
  int64_t n;
  int64_t k;
  int64_t ldq;
  int64_t ldqt;
  int64_t lde;
} muon_w8;

/* Saves w (n x k, row stride ldw, MUON_F32 or MUON_BF16); a training loop does so
 * after every step. Errors as for muon_q8_save. */
muon_status muon_w8_save(const void* w, int64_t ldw, int32_t dtype, const muon_w8* out, void* stream);
/* Loads the values that it stands for. */
muon_status muon_w8_load(const muon_w8* in, void* w, int64_t ldw, int32_t dtype, void* stream);

/* One product of a linear layer in 8-bit floating point:
 *   y = x W^T + beta*c   (rows x n), or, transposed,  y = x W + beta*c   (rows x k)
 * x      rows x k (transposed: rows x n) e4m3 checkpoint: the layer's input, or the
 *        gradient of its output, as muon_q8_save makes it
 * w      the weight; transposed needs its qt
 * y, c   rows x n (k), dtype, row strides ld_y and ld_c (n, k and these are at most
 *        2^22); c is read if beta != 0 and may be y itself
 * Products of elements are exact, sums are fp32, y is rounded once. bf16: the 8-bit
 * MFMA with scales, which adds 16 products of consecutive k (from a multiple of 16)
 * on a common grid of 2^-13 of the largest and drops what is below; these sums are
 * then added in fp32. fp32: the operands as bf16, exactly, and bf16 MFMA, at about
 * half the rate. A group of x or a block
 * of w that stands for NaNs makes its row or its columns of y NaN. */
typedef struct {
  muon_q8 x;
  muon_w8 w;
  void* y;
  int64_t ld_y;
  const void* c;
  int64_t ld_c;
  float beta;
  int32_t transposed;
} muon_linear8_item;

/* Products of n_items layers in one go. Errors: INVALID_ARG (null pointers, sizes,
 * strides, shapes, non-finite beta, a short workspace, more than 2^22 output
 * tiles), ALIGN, ALIAS, UNSUPPORTED (dtype, an int8 checkpoint), HIP. workspace:
 * muon_linear8_workspace bytes (which may be 0), 16-byte aligned, scratch of this
 * call until it has run. muon_linear8_workspace makes the same checks of the items,
 * without a GPU. */
muon_status muon_linear8(const muon_linear8_item* items, int32_t n_items, int32_t dtype, void* workspace,
                         size_t workspace_bytes, void* stream);
muon_status muon_linear8_workspace(const muon_linear8_item* items, int32_t n_items, int32_t dtype, size_t* bytes);
/* How muon_linear8 cuts each item's product up, as muon_mlp_info says it (after the
 * same checks of the items, without a GPU). n_items numbers each. */
muon_status muon_linear8_info(const muon_linear8_item* items, int32_t n_items, int32_t dtype, int32_t* tile, int32_t* whole,
                              int32_t* pieces);

#ifdef __cplusplus
}
#endif

#endif /* MUON_H_ */
