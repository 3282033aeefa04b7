/*
 * dmuon.h - C ABI of the owner-side batched Muon update on one GB300 GPU.
 *
 * The library runs, for a whole batch of 2-D weight matrices in one pass, the
 * update that a DMuon owner performs on the matrices it owns ("DMuon:
 * Efficient Distributed Muon Training with Near-Adam Overhead", gist.science
 * technical summary, section 2.1 "Owner-Centric Executiestrategie": the owner
 * keeps the optimizer state and runs the Newton-Schulz iteration and the
 * update once per matrix; section 1 "Probleemstelling": Newton-Schulz on the
 * momentum-aggregated gradient, built on the product X X^T). Per matrix W
 * (rows x cols, row-major, rows = dim 0), gradient G and momentum M:
 *
 *   M  <- mu*M + G;   U = G + mu*M (Nesterov) or U = M
 *   X  <- U / (||U||_F + eps), transposed when rows > cols (short side first)
 *   repeat ns_steps:  A = X X^T;  B = b*A + c*A*A;  X <- a*X + B*X
 *   W  <- W - lr * sqrt(max(1, rows/cols)) * X     (X back in W's orientation)
 *
 * The two calls follow the problem statement of the pages: a plan built once
 * from the list of matrix shapes, the Newton-Schulz step count, coefficients
 * and dtypes ("dmuon_plan"), and a step taking params, grads and momenta
 * ("dmuon_step"). Matrices of equal shape are batched into one bucket and
 * every phase runs all buckets in one launch (summary section 2,
 * "Batching"); tiles are ordered by computational cost, largest first, the
 * greedy fallback of the cost-based balancing in summary section 2.3.
 *
 * Conventions for every entry point:
 *  - Every call returns a dmuon_status; nothing else crosses the ABI. On an
 *    error, dmuon_last_error() returns a message (thread-local, valid until
 *    the next call on the same thread).
 *  - Argument errors are detected on the host before anything is launched.
 *  - "stream" is a cudaStream_t passed as void* (NULL = legacy default stream).
 *  - Device pointers must address memory of the current CUDA device.
 *  - The library never allocates device memory: the caller owns the
 *    workspace and every parameter, gradient and momentum buffer.
 *  - Device-detected conditions (non-finite norm, a pipeline wait that ran
 *    out of time) are bits of a status word in the workspace, never traps;
 *    read them with dmuon_read_device_status().
 */
#ifndef DMUON_H
#define DMUON_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  DMUON_OK = 0,
  DMUON_ERR_INVALID_ARG = -1, /* bad shape, count, pointer, size or value      */
  DMUON_ERR_UNSUPPORTED = -2, /* dtype combination or flag not supported       */
  DMUON_ERR_WORKSPACE = -3,   /* workspace NULL, too small or misaligned       */
  DMUON_ERR_CUDA = -4,        /* a CUDA runtime/driver call failed             */
  DMUON_ERR_NOT_BOUND = -5,   /* dmuon_step before dmuon_plan_bind             */
  DMUON_ERR_DEVICE = -6       /* a device-side result is wrong: a status bit is
                                 set, or a DMUON_FLAG_DEBUG_CHECKS check failed */
} dmuon_status;

typedef enum { DMUON_F32 = 0, DMUON_BF16 = 1 } dmuon_dtype;

/* Stored shape of one matrix: rows = dim 0, row-major, contiguous. */
typedef struct {
  int64_t rows;
  int64_t cols;
} dmuon_shape;

/* Storage dtypes of the step's tensors and the arithmetic mode.
 *   param:    DMUON_F32 or DMUON_BF16 (weights, updated in place)
 *   grad:     DMUON_F32 or DMUON_BF16 (read only)
 *   momentum: DMUON_F32 only (updated in place)
 *   compute:  DMUON_F32  = fp32 operands and fp32 accumulation everywhere;
 *             DMUON_BF16 = bf16 Newton-Schulz operands (X, A, B stored bf16)
 *                          with fp32 accumulation on the tensor cores.      */
typedef struct {
  int32_t param;
  int32_t grad;
  int32_t momentum;
  int32_t compute;
} dmuon_dtypes;

/* Plan flags. */
#define DMUON_FLAG_CAPTURE_UPDATE 0x1u /* keep the fp32 update X of the last step
                                          (read it with dmuon_read_update)      */
#define DMUON_FLAG_GRAM_NS 0x2u        /* matrices with max(rows,cols) >= 2*min(rows,cols)
                                          iterate in the m x m Gram space: G = X X^T
                                          once, then per step P = aI + bG + cG^2,
                                          Q <- P Q, G <- P G P; finally X = Q X0
                                          ("DMuon: Efficient Distributed Muon
                                          Training with Near-Adam Overhead",
                                          gist.science summary section 2, "Gram
                                          Space Recurrence"). Fewer flops when the
                                          matrix is wide (>= 26% fewer at 2:1);
                                          others keep the standard form.          */
#define DMUON_FLAG_PAIR_TILES 0x8u    /* 256 x 256 tiles on pairs of SMs (two-SM
                                          UMMA, thread-block clusters of 2; bf16
                                          only) for every bucket whose short side
                                          is a multiple of 256 and whose products
                                          run 256 wide. Without the flag the same
                                          holds for short sides of at least 1024
                                          (the default); other buckets use one-SM
                                          tiles. Test hook: with the environment
                                          variable DMUON_TEST_FORCE_PAIRS=1, every
                                          bucket with a short side >= 256 gets
                                          pairs (as DMUON_FLAG_TUNE may choose).  */
#define DMUON_FLAG_EPILOGUE_AX 0x10u   /* standard form: add the a*X_k term of the
                                          quintic step in the epilogue of the
                                          product B X_k (reading the X_k tile),
                                          with B = bA + cA^2. Without the flag
                                          the step runs as X_{k+1} = P X_k with
                                          P = aI + bA + cA^2 formed by the
                                          symmetric-product epilogue (a on the
                                          diagonal), and the last product reads
                                          no X_k tile: the same polynomial, one
                                          bf16 rounding of a + B_ii instead of
                                          an fp32 a*X term.                      */
#define DMUON_FLAG_STATIC_TILES 0x20u  /* tensor-core launches deal the cost-ordered
                                          tile list round-robin (CTA b, or CTA pair b,
                                          takes tiles b, b + grid, ...) instead of
                                          letting each CTA (pair) claim the next tile
                                          from the launch's counter as it becomes free.
                                          Same results bit for bit; kept to compare the
                                          two schedules.                           */
#define DMUON_FLAG_DEBUG_CHECKS 0x40u /* debugging aid: after every launch of a step
                                          the host waits for it, copies back the
                                          operands of a few sampled output elements
                                          (momentum, U, s, product elements, one on
                                          the diagonal, one mirror, updated weights)
                                          and recomputes them in double precision;
                                          dmuon_step returns DMUON_ERR_DEVICE, with
                                          the launch, matrix and element in
                                          dmuon_last_error(), when one is off by more
                                          than its rounding allows. Makes every step
                                          synchronous and slow; not for capture.
                                          Test hook: with the environment variable
                                          DMUON_TEST_SKIP_LAUNCH=<i>, launch i of
                                          each step is left out, so its outputs are
                                          stale and the checks must report them.  */
#define DMUON_FLAG_ONE_SM_TILES 0x80u /* every bucket uses one-SM tiles (128 rows,
                                          128 or 256 columns): no CTA pairs. Not
                                          together with DMUON_FLAG_PAIR_TILES or
                                          DMUON_FLAG_TUNE.                        */
#define DMUON_FLAG_TUNE 0x4u           /* at bind, time three tile configurations per
                                          bucket on the bound workspace (one-SM
                                          128 x 128 and 128 x 256 tiles, two-SM
                                          256 x 256 pairs where the short side is
                                          >= 256; each with its ring depth), keep
                                          the cheapest, and order tiles by measured
                                          time (see dmuon_plan_costs). Timings are
                                          cached for the process by (short side,
                                          long side, weight dtype, SM count,
                                          compute capability): a later plan with
                                          the same shapes binds without timing.
                                          bf16 only.                              */

/* Device status bits (dmuon_read_device_status). */
#define DMUON_DEV_NONFINITE_NORM 0x1u  /* ||U||_F was NaN or Inf for some matrix  */
#define DMUON_DEV_WAIT_TIMEOUT 0x2u    /* a pipeline wait ran out of time; the
                                          kernel returned early, results invalid */

/* Launch kinds reported by the profiler. */
#define DMUON_KIND_MOMENTUM 0 /* momentum + per-unit sums of squares + cast/transposed copy */
#define DMUON_KIND_GRAM 1     /* A = X X^T, upper tiles, mirrored                  */
#define DMUON_KIND_POLY 2     /* B = b*A + c*A A^T, upper tiles, mirrored          */
#define DMUON_KIND_GEMM 3     /* X' = a*X + B X (last step: W update epilogue)     */
#define DMUON_KIND_UPDATE0 4  /* W update straight from U (ns_steps == 0)          */
#define DMUON_KIND_SYMM 5     /* Gram-space form: product of two commuting
                                 symmetric m x m matrices, upper tiles, mirrored   */
#define DMUON_KIND_NORM 6     /* s = 1/(||U||_F + eps) per matrix from the partials */

typedef struct dmuon_plan_s* dmuon_plan_t;

/*
 * dmuon_plan - validate a batch description and build the host-side plan.
 *
 *  shapes[n_mats]     stored shape of each matrix; 1 <= rows, cols <= 2^20 and
 *                     rows*cols < 2^31.
 *  ns_steps           number of Newton-Schulz steps, 0..16.
 *  coeffs             host array of 3*n_coeff_triples floats (a, b, c, ...);
 *                     n_coeff_triples is 1 (same triple every step) or
 *                     ns_steps (one triple per step). NULL with 0 triples
 *                     selects (3.4445, -4.7750, 2.0315).
 *  eps                added to the Frobenius norm (not its square); >= 0.
 *  dtypes, flags      see above. momentum must be DMUON_F32.
 *  out                receives the plan handle (host memory, owned by the
 *                     library until dmuon_plan_destroy).
 *
 * Needs no GPU: only host memory is touched. Matrices with equal (short, long)
 * shape share a bucket; per phase the tiles of all buckets are listed and
 * sorted by cost (largest first).
 */
dmuon_status dmuon_plan(const dmuon_shape* shapes, int32_t n_mats, int32_t ns_steps,
                        const float* coeffs, int32_t n_coeff_triples, float eps,
                        dmuon_dtypes dtypes, uint32_t flags, dmuon_plan_t* out);

/* Bytes of device workspace the plan needs (host only). */
dmuon_status dmuon_plan_workspace_bytes(dmuon_plan_t plan, size_t* bytes);

/*
 * dmuon_plan_bind - attach a caller-owned device workspace and upload the
 * plan's tables into it (asynchronously, on stream).
 *
 *  d_workspace  device pointer, 1024-byte aligned, at least
 *               dmuon_plan_workspace_bytes() bytes; owned by the caller and
 *               used exclusively by this plan until it is destroyed or bound
 *               again. Its contents need not be initialised.
 *  Builds the TMA tensor maps for the workspace buffers. The plan's host
 *  staging of the tables must outlive the copies: it does (it is owned by the
 *  plan). Returns DMUON_ERR_WORKSPACE if the buffer is NULL, misaligned, too
 *  small or not memory of the current device, DMUON_ERR_UNSUPPORTED for bf16 compute on a GPU other than
 *  sm_103. Any failing bind leaves the plan unbound, also a plan that was
 *  bound before (dmuon_step then returns DMUON_ERR_NOT_BOUND until a bind
 *  succeeds). For tests, the environment variable DMUON_TEST_FAIL set to
 *  bind_check, bind_tables, bind_maps or bind_staging makes the bind fail at
 *  that point (before any CUDA call, after the tables are uploaded, while the
 *  tensor maps are built, or before the host staging is allocated).
 */
dmuon_status dmuon_plan_bind(dmuon_plan_t plan, void* d_workspace, size_t bytes, void* stream);

/*
 * dmuon_step - one Muon step for every matrix of the plan, asynchronous on
 * stream.
 *
 *  params[n_mats]   host array of device pointers; W_i, rows x cols,
 *                   param dtype, updated in place.
 *  grads[n_mats]    host array of device pointers; G_i, grad dtype, read only.
 *  momenta[n_mats]  host array of device pointers; M_i, fp32, updated in place.
 *  lr, mu           learning rate and momentum coefficient (finite).
 *  nesterov         0 = heavy ball (U = M), 1 = Nesterov (U = G + mu*M).
 *
 * Each pointer must be 16-byte aligned and the matrices must not overlap.
 * The host pointer arrays are read during the call only. The plan keeps the
 * last 4 distinct pointer sets resident on the device: a call whose pointers
 * equal one of them copies nothing (alternating gradient buffers cost no
 * copy after their first steps); otherwise the least recently used set is
 * replaced by a cudaMemcpyAsync from host memory on `stream`. With bf16
 * weights on the tensor-core path a resident set also holds a TMA tensor map
 * of every W (encoded on the host when the set is first seen, copied with the
 * pointers): the last Newton-Schulz product stores its updated W boxes
 * through them. Under CUDA-graph
 * capture, make one uncaptured call with the same pointers first so that none
 * is needed; the captured graph stays valid while that pointer set remains
 * one of the 4 resident ones.
 * Launches the momentum kernel and the per-matrix norm kernel, then
 * 3*ns_steps kernels per chunk of standard-form buckets and 4*ns_steps - 1
 * per chunk of Gram-space buckets (a chunk: up to 7 buckets sharing form and
 * tile widths); 2 + 1 kernels when ns_steps == 0. dmuon_plan_describe lists
 * them.
 */
dmuon_status dmuon_step(dmuon_plan_t plan, void* const* params, const void* const* grads,
                        void* const* momenta, float lr, float mu, int32_t nesterov, void* stream);

/*
 * dmuon_set_weight_events - order the weight writes of later steps against
 * work on other streams. Only the launches that write W (the last
 * Newton-Schulz product of each launch chunk, or the update kernel when
 * ns_steps == 0) touch the weights; the momentum pass and every earlier
 * product read only the gradients, the momenta and the workspace.
 *
 *  wait_before_write  a cudaEvent_t (as void*) or NULL: every later
 *                     dmuon_step makes its stream wait on it
 *                     (cudaStreamWaitEvent, on the event's most recent
 *                     record at the time of that dmuon_step call) just
 *                     before its first launch that writes W.
 *  after_write        a cudaEvent_t or NULL: every later dmuon_step
 *                     records it on its stream right after its last launch
 *                     that writes W.
 *
 * With both, a copy of step k's weights (to the host, say) can run on
 * another stream while step k+1's momentum pass and its first ns_steps - 1
 * Newton-Schulz steps run: the copy waits on after_write and records
 * wait_before_write. The events stay the caller's; they must stay valid
 * while set (NULL, NULL clears them). Host only; no effect on the results.
 */
dmuon_status dmuon_set_weight_events(dmuon_plan_t plan, void* wait_before_write, void* after_write);

/*
 * dmuon_read_device_status - synchronise stream, return the device status
 * bits accumulated since the last read (DMUON_DEV_*) in *bits, and clear
 * them. Returns DMUON_OK even when bits are set. The word travels through a
 * one-thread kernel into mapped page-locked host memory owned by the plan,
 * not through a copy, so the read does not wait behind large transfers that
 * other streams have in flight.
 */
dmuon_status dmuon_read_device_status(dmuon_plan_t plan, void* stream, uint32_t* bits);

/*
 * dmuon_read_update - copy the fp32 update X of matrix `mat` from the last
 * step (before lr and the shape scale, in W's rows x cols orientation) to
 * d_dst (device, rows*cols floats), asynchronously on stream. Needs a plan
 * made with DMUON_FLAG_CAPTURE_UPDATE.
 */
dmuon_status dmuon_read_update(dmuon_plan_t plan, int32_t mat, float* d_dst, void* stream);

/*
 * dmuon_plan_describe - JSON text describing the plan (buckets, tiles per
 * phase, launches per step, algorithmic flops and bytes per launch) written
 * to buf (at most len bytes, NUL-terminated); *needed receives the full
 * length + 1. Host only.
 */
dmuon_status dmuon_plan_describe(dmuon_plan_t plan, char* buf, size_t len, size_t* needed);

/*
 * Profiling: dmuon_profile_begin(plan, max_launches) makes the following
 * steps record a CUDA event pair around each launch (on the step's stream),
 * for up to max_launches launches (it creates the events: host-side CUDA
 * objects, no device memory). dmuon_profile_end synchronises the events and
 * writes, for each recorded launch i < cap, its kind (DMUON_KIND_*), its
 * duration in ms and its algorithmic work (flops for GEMM kinds, bytes for
 * streaming kinds); *n receives the number recorded. Profiling then stops.
 */
dmuon_status dmuon_profile_begin(dmuon_plan_t plan, int32_t max_launches);
dmuon_status dmuon_profile_end(dmuon_plan_t plan, int32_t* kinds, float* ms, double* work,
                               int32_t cap, int32_t* n);

/*
 * dmuon_plan_costs - predicted GPU milliseconds of each matrix's
 * Newton-Schulz work (its tiles times the measured time per tile, spread over
 * all SMs), from the timings a DMUON_FLAG_TUNE bind made. n must equal the
 * plan's matrix count; per_matrix_ms is a host array. Returns
 * DMUON_ERR_UNSUPPORTED for a plan that was not tuned. The costs can be
 * passed to dmuon_assign_owners ("DMuon: Efficient Distributed Muon Training
 * with Near-Adam Overhead", gist.science summary section 2.3: owners are
 * balanced on measured, not theoretical, costs).
 */
dmuon_status dmuon_plan_costs(dmuon_plan_t plan, double* per_matrix_ms, int32_t n);

/*
 * Per-CTA timing of the tensor-core launches (profiling). After
 * dmuon_profile_cta_times(plan, 1), every tensor-core launch of the following
 * steps records, per CTA, the global timer (ns) when the CTA started and when
 * it finished, in the workspace (each step overwrites the previous one's);
 * dmuon_profile_cta_times(plan, 0) stops it. dmuon_read_cta_times copies the
 * records of launch `launch` (its index in dmuon_plan_describe's launch list)
 * of the last recorded step to out[2*i] (start) and out[2*i+1] (end) for CTA
 * i < min(cap, *n_ctas), host memory, synchronising stream; *n_ctas receives
 * the launch's CTA count (both CTAs of each pair for two-SM tiles; 0 for
 * launches that keep no records: streaming kernels and fp32 mode).
 */
dmuon_status dmuon_profile_cta_times(dmuon_plan_t plan, int32_t enable);
dmuon_status dmuon_read_cta_times(dmuon_plan_t plan, int32_t launch, uint64_t* out, int32_t cap, int32_t* n_ctas,
                                  void* stream);

/* Number of kernels the library has launched through this plan so far. */
dmuon_status dmuon_launch_count(dmuon_plan_t plan, int64_t* count);

/*
 * dmuon_selftest_wait_timeout - run one small kernel whose pipeline wait can
 * never complete (nothing arrives on its barrier), with a wait limit of
 * limit_ns nanoseconds (1e6..5e9). The kernel gives up, records
 * DMUON_DEV_WAIT_TIMEOUT and returns; *bits receives the status it wrote.
 * Exercises the bounded-wait path of the pipelined kernels without a fault.
 * Synchronises stream. d_scratch: 256 device bytes owned by the caller.
 */
dmuon_status dmuon_selftest_wait_timeout(void* d_scratch, int64_t limit_ns, void* stream,
                                         uint32_t* bits);

/*
 * dmuon_momentum_norm_noalloc - the momentum and normalisation pass of ONE
 * matrix for callers that cannot allocate device memory: a framework whose
 * allocator already holds the whole GPU, a plugin handed only the tensors it
 * must update, or a runtime that forbids allocation in its steady state.
 * The pages have no counterpart; it is the plan-free form of the first
 * launch of dmuon_step, with its reduction scratch (per-tile partial sums)
 * in a static device array of the library instead of a workspace.
 *
 *  grad       device, rows x cols, grad_dtype (DMUON_F32 or DMUON_BF16), read only.
 *  momentum   device, rows x cols fp32, updated in place: M <- mu*M + G.
 *  u_out      device, m x u_ld elements of u_dtype, m = min(rows, cols),
 *             u_ld = round_up(max(rows, cols), 8): U = G + mu*M (Nesterov) or
 *             U = M, stored transposed when rows > cols (short side first).
 *  s_out      device, one float: 1 / (||U||_F + eps).
 *
 * Limit: ceil(rows/64) * ceil(cols/128) <= 65536 (e.g. 8192 x 8192 fits);
 * larger matrices return DMUON_ERR_UNSUPPORTED. The static array (256 KiB +
 * 256 B) stays allocated on every GPU that loads the library until the
 * process exits. The first call on a device looks up the array's device
 * address (cudaGetSymbolAddress) with that device current, and so does the
 * first call after the device's context was replaced (cudaDeviceReset); make
 * that first call before any stream capture. A CUDA error that earlier work
 * left pending is reported (DMUON_ERR_CUDA, left pending) before anything is
 * launched. The call allocates nothing: it launches two
 * kernels on stream (the tile pass, which writes one partial sum per tile,
 * and a one-block kernel that adds them in a fixed order and writes s_out).
 * 16-byte aligned grad, momentum and u_out (with cols % 4 == 0) take the
 * vectorised path; other alignments are accepted and go element by element.
 * Every call shares the array and it keeps the last call's contents; calls
 * that overlap on the GPU race and give wrong results.
 */
dmuon_status dmuon_momentum_norm_noalloc(const void* grad, float* momentum, void* u_out, float* s_out,
                                         int64_t rows, int64_t cols, int32_t grad_dtype, int32_t u_dtype,
                                         float mu, int32_t nesterov, float eps, void* stream);

/*
 * dmuon_assign_owners - choose one owner rank for every matrix so that the
 * largest predicted per-rank load is small ("DMuon: Efficient Distributed
 * Muon Training with Near-Adam Overhead", gist.science summary section 2.1:
 * one owner per matrix runs its update; section 2.3: minimise the predicted
 * makespan over owner ranks, greedy when the search space is large).
 *
 *  shapes[n_mats]   stored shapes (host).
 *  ns_steps         0..16; with costs == NULL the cost of a matrix is its
 *                   Newton-Schulz flops (symmetric products counted once;
 *                   ns_steps 0 counts as 1).
 *  costs            optional host array of n_mats finite costs >= 0 (e.g.
 *                   measured times); NULL = the flop count above.
 *  n_ranks          >= 1.
 *  owner_out        host array of n_mats: the owner rank of each matrix.
 *  load_out         optional host array of n_ranks: the summed cost per rank.
 *
 * Longest-processing-time-first greedy, then moves and swaps out of the
 * most-loaded rank while they lower the makespan. Deterministic: every rank
 * that calls it with the same arguments gets the same assignment. Host only.
 */
dmuon_status dmuon_assign_owners(const dmuon_shape* shapes, int32_t n_mats, int32_t ns_steps,
                                 const double* costs, int32_t n_ranks, int32_t* owner_out,
                                 double* load_out);

/*
 * dmuon_adamw_flat - one AdamW step over a flat buffer of n elements, for the
 * parameters the Muon predicate leaves out ("DMuon" project docs, section
 * "DMuon 能做什么": everything else is optimised by AdamW with its own
 * learning rate, adamw_lr). Decoupled weight decay and bias correction:
 *   p <- p*(1 - lr*wd);  m <- b1*m + (1-b1)*g;  v <- b2*v + (1-b2)*g^2
 *   p <- p - lr/(1-b1^t) * m / (sqrt(v)/sqrt(1-b2^t) + eps)
 *
 *  param        device, n elements of param_dtype (DMUON_F32/DMUON_BF16), in place.
 *  grad         device, n elements of grad_dtype, read only.
 *  exp_avg, exp_avg_sq  device, n fp32 each (m and v), in place.
 *  step         t >= 1 (the step being taken); 0 <= beta1, beta2 < 1; eps >= 0.
 * All four pointers 16-byte aligned. One kernel on stream; no allocation.
 */
dmuon_status dmuon_adamw_flat(void* param, const void* grad, float* exp_avg, float* exp_avg_sq, int64_t n,
                              int32_t param_dtype, int32_t grad_dtype, float lr, float beta1, float beta2,
                              float eps, float weight_decay, int32_t step, void* stream);

/*
 * ---- The language-model head: losses with their gradients, without the logits
 *
 * The parameters the Muon predicate leaves out include the head ("DMuon"
 * project docs, section "DMuon 能做什么": everything else goes to AdamW), and
 * every gradient a step consumes starts at the head's loss. These calls take
 * the head's input and weight and return the loss of each token and the
 * gradients of both, working through the vocabulary in pieces: the
 * tokens x vocab matrix of logits never exists.
 *
 *   hidden   H, tokens x dim, bf16 (row pitch ld_hidden elements)
 *   weight   W, vocab x dim, bf16 (row pitch ld_weight elements)
 *   z[t][v] = sum_d H[t][d] * W[v][d], accumulated by the tensor cores in fp32
 *             and kept in fp32. They truncate: z loses between nothing and
 *             2e-9 * dim of the largest partial sum, about 1.0e-9 * dim * z
 *             where terms are spread evenly (measured at 256 to 65536 dims). z
 *             is scaled by 1 + 1.0e-9 * dim, which leaves at most a quarter of
 *             that in the even case (a few percent from 4096 dims on), and up
 *             to 1.2e-9 * dim * z either way where they lie at one end.
 *             The logits that decide a loss come from plain fp32 FMAs: the
 *             target's, a teacher's entries of at least 1/8.
 *
 * A dmuon_head_t is made once per (max_tokens, vocab, dim, max_top) and bound to
 * a caller-owned workspace, like a plan; one call uses the workspace at a time
 * (calls on several streams must be ordered by the caller), and nothing in it
 * is kept from one call for the next except the status word.
 *
 * H, W and their gradients start on 16 bytes, and their row pitches are
 * multiples of 8 elements and at least dim. Outputs must not overlap inputs.
 */
typedef struct dmuon_head_s* dmuon_head_t;

/*
 * dmuon_head_create - host only. 1 <= max_tokens <= 2^20, 1 <= vocab <= 2^22,
 * 1 <= dim <= 2^16; max_top (0..256) is the longest teacher list a
 * distillation call may pass (0: none). The backward pass works through the
 * vocabulary in pieces of about 2^28 / max_tokens entries (256 at least), two
 * launches each, however few tokens a call has: a head made for the lengths it
 * is called with is faster than one made for many more.
 */
dmuon_status dmuon_head_create(int64_t max_tokens, int64_t vocab, int64_t dim, int32_t max_top, dmuon_head_t* out);

/* Bytes of device workspace the head needs (host only). */
dmuon_status dmuon_head_workspace_bytes(dmuon_head_t head, size_t* bytes);

/*
 * ... and with room for what dmuon_head_logprobs writes where alternatives are asked
 * for: the logits, 4 bytes for each token and entry, up to 512 MB (or 1 KB *
 * max_tokens). In a smaller workspace they have the place of the backward pass's
 * dz, 2 bytes for each (4 for heads of up to 64 tokens), and the call takes the
 * vocabulary in as many pieces more, one after another: 2048 tokens x 32000 x 2048
 * with 20 alternatives 235 us in place of 210, for 128 MB less.
 */
dmuon_status dmuon_head_scores_workspace_bytes(dmuon_head_t head, size_t* bytes);

/*
 * dmuon_head_bind - attach a caller-owned device workspace (1024-byte aligned,
 * its contents need not be initialised) and clear the status word in it,
 * asynchronously on stream. Errors as dmuon_plan_bind. `bytes` is at least what
 * dmuon_head_workspace_bytes says; up to dmuon_head_scores_workspace_bytes all of it
 * is used.
 */
dmuon_status dmuon_head_bind(dmuon_head_t head, void* d_workspace, size_t bytes, void* stream);

/*
 * dmuon_head_xent - softmax cross entropy of each token against its target:
 *
 *   lse[t]  = log sum_v exp(z[t][v])
 *   loss[t] = lse[t] - z[t][targets[t]]
 *
 *  targets   device, tokens int64. A target outside 0..vocab-1 (-100, say)
 *            marks a token that does not count: its loss is 0, and its rows of
 *            dz and dH are exact zeros whatever its logits are. (Its row of H
 *            has to be finite all the same: dW sums 0 * H.)
 *  tokens    0..max_tokens; 0 is a no-op.
 *  loss, lse device, tokens floats each.
 *
 * The target's share of the sum is kept apart from the others', so that the
 * loss of a token predicted with near certainty keeps its leading digits.
 * Asynchronous on stream, no allocation, deterministic.
 */
dmuon_status dmuon_head_xent(dmuon_head_t head, const void* hidden, int64_t ld_hidden, const void* weight,
                             int64_t ld_weight, const int64_t* targets, int64_t tokens, float* loss, float* lse,
                             void* stream);

/*
 * dmuon_head_xent_backward - gradients of sum_t grad_loss[t] * loss[t]:
 *
 *   dz[t][v] = grad_loss[t] * (exp(z[t][v] - lse[t]) - [v == targets[t]])   (0 for a token that does not count)
 *   dH = dz W,  dW = dz^T H
 *
 *  lse        device, tokens floats, as dmuon_head_xent wrote them.
 *  grad_loss  device, tokens floats (1/n for a mean over n tokens); not used
 *             of tokens that do not count.
 *  dhidden    device, tokens x dim bf16, pitch ld_dhidden, or NULL: not wanted.
 *  dweight    device, vocab x dim bf16, pitch ld_dweight, or NULL: not wanted
 *             (a frozen head). Overwritten, also when tokens is 0.
 *
 * z is formed again, piece by piece, and dz is rounded to bf16 once (of up to
 * 64 tokens: to the sum of two bf16), as the operand of two tensor-core
 * products that accumulate in fp32 over the whole vocabulary (dH) and all
 * tokens (dW). (What truncation takes there, at most about 2e-9 for each term
 * summed, is not put back: below the result's rounding up to a million terms.)
 */
dmuon_status dmuon_head_xent_backward(dmuon_head_t head, const void* hidden, int64_t ld_hidden, const void* weight,
                                      int64_t ld_weight, const int64_t* targets, int64_t tokens, const float* lse,
                                      const float* grad_loss, void* dhidden, int64_t ld_dhidden, void* dweight,
                                      int64_t ld_dweight, void* stream);

/*
 * dmuon_head_xent_backward_loss - the same, given the losses too:
 *
 *  loss       device, tokens floats, as dmuon_head_xent wrote them beside lse.
 *
 * dz of a target is then grad_loss * expm1(-loss), which has all the digits of
 * the loss. From z and lse, both rounded to 1e-6 at 16 to 32, 1 - p of the
 * target is off by about that much: 1 % of dz where the loss is 1e-4, all of it
 * below 1e-6 (it never has the wrong sign). The other entries are the same.
 */
dmuon_status dmuon_head_xent_backward_loss(dmuon_head_t head, const void* hidden, int64_t ld_hidden,
                                           const void* weight, int64_t ld_weight, const int64_t* targets,
                                           int64_t tokens, const float* lse, const float* loss,
                                           const float* grad_loss, void* dhidden, int64_t ld_dhidden, void* dweight,
                                           int64_t ld_dweight, void* stream);

/*
 * dmuon_head_distill - distillation from a teacher's top logits: the divergence
 * of the student's distribution over the whole vocabulary from the teacher's
 * over its list, both at a temperature:
 *
 *   q[t] = softmax(top_logits[t] / temperature) over the list's entries
 *   p[t] = softmax(z[t] / temperature) over the vocabulary
 *   lse[t]  = log sum_v exp(z[t][v] / temperature)
 *   loss[t] = temperature^2 * sum_k q[t][k] * (log q[t][k] - log p[t][top_ids[t][k]])
 *
 *  top_ids     device, tokens x top int64, contiguous, any order. An entry
 *              whose id is outside 0..vocab-1 or whose logit is -infinity is
 *              not in the list; a row without entries has loss 0. The ids of a
 *              row should differ; entries that share one add up.
 *  top_logits  device, tokens x top fp32, contiguous.
 *  top         1..max_top.
 *  temperature > 0, finite.
 */
dmuon_status dmuon_head_distill(dmuon_head_t head, const void* hidden, int64_t ld_hidden, const void* weight,
                                int64_t ld_weight, const int64_t* top_ids, const float* top_logits, int32_t top,
                                float temperature, int64_t tokens, float* loss, float* lse, void* stream);

/*
 * dmuon_head_distill_backward - gradients of sum_t grad_loss[t] * loss[t]:
 *
 *   dz[t][v] = grad_loss[t] * temperature * (p[t][v] - q[t][v])   (0 for a row without entries)
 *
 * lse as dmuon_head_distill wrote it; the rest as dmuon_head_xent_backward. p of
 * a listed entry is off by about 1e-6 of itself, which is most of p - q once
 * the student agrees with the teacher that closely.
 */
dmuon_status dmuon_head_distill_backward(dmuon_head_t head, const void* hidden, int64_t ld_hidden, const void* weight,
                                         int64_t ld_weight, const int64_t* top_ids, const float* top_logits,
                                         int32_t top, float temperature, int64_t tokens, const float* lse,
                                         const float* grad_loss, void* dhidden, int64_t ld_dhidden, void* dweight,
                                         int64_t ld_dweight, void* stream);

/*
 * dmuon_head_logprobs - the log probability of each token's target, the entropy of
 * what the model expected, and its likeliest entries (what a server returns beside
 * a generated token, and what a policy's gradient starts from), at a temperature:
 *
 *   zt[t][v]   = z[t][v] / temperature
 *   lse[t]     = log sum_v exp(zt[t][v])
 *   logp[t]    = zt[t][targets[t]] - lse[t]
 *   entropy[t] = - sum_v p log p,  p[t][v] = exp(zt[t][v] - lse[t])
 *   top_ids[t], top_logp[t]: the entries with the `top` largest z, largest first (of
 *                equal ones the lowest id first), and their log probabilities, which
 *                never rise along them; the target's is logp[t]
 *
 *  targets   device, tokens int64, or NULL: none is given. A target outside
 *            0..vocab-1 has the log probability 0; the rest of its token's
 *            results are the same.
 *  top       0..32, and not above vocab. With 0 top_ids and top_logp are not used.
 *  tokens    0..max_tokens; 0 is a no-op.
 *  logp, entropy, lse  device, tokens floats each.
 *  top_ids   device, tokens x top int64;  top_logp  the same, fp32.
 *
 * The target's share of the sum is kept apart from the others', as in
 * dmuon_head_xent, and the largest entry's from the rest, so that the log
 * probability of a target predicted with near certainty and the entropy of a token
 * with any nearly sure entry keep their leading digits (other entries' log
 * probabilities are off by about 1e-6 of their logit). Neighbours among the top
 * entries that are too near to tell in fp32 are put in order by sums with twice its
 * digits: those nearer than what the tensor cores' sums may be off by, which goes by
 * the products' absolute values (|hidden| . |weight|, of the target or, without one,
 * of some entry; others' rows may have twice as much). `top` + 8 entries are looked
 * at: where more than eight others lie within that of the last one, which of them is
 * among the top is the tensor cores' choice. A row whose logits are not finite has
 * unspecified top entries (ids within the vocabulary or -1).
 * Where alternatives are asked for, the logits of a piece of the vocabulary lie in
 * the workspace at a time (see dmuon_head_scores_workspace_bytes; in the smallest
 * workspace of a head for more than 2^19 tokens there is room for 2^19 at a time, and
 * calls with more are DMUON_ERR_WORKSPACE).
 * Asynchronous on stream, no allocation, deterministic.
 */
dmuon_status dmuon_head_logprobs(dmuon_head_t head, const void* hidden, int64_t ld_hidden, const void* weight,
                                 int64_t ld_weight, const int64_t* targets, float temperature, int32_t top,
                                 int64_t tokens, float* logp, float* entropy, float* lse, int64_t* top_ids,
                                 float* top_logp, void* stream);

/*
 * dmuon_head_logprobs_backward - gradients of
 * sum_t grad_logp[t] * logp[t] + grad_entropy[t] * entropy[t]:
 *
 *   dz[t][v] = (grad_logp[t] * ([v == targets[t]] - p[t][v])
 *               - grad_entropy[t] * p[t][v] * (log p[t][v] + entropy[t])) / temperature
 *
 *  targets, temperature  as the forward call had them.
 *  logp, entropy, lse    device, tokens floats, as dmuon_head_logprobs wrote
 *             them (logp may be NULL where targets is).
 *  grad_logp, grad_entropy  device, tokens floats, or NULL: zeros. grad_logp is
 *             not used of tokens without a target.
 * log p of an entry that is nearly sure and not the target is off by about 1e-6 of
 * its logit, and what grad_entropy adds there with it.
 * The rest as dmuon_head_xent_backward.
 */
dmuon_status dmuon_head_logprobs_backward(dmuon_head_t head, const void* hidden, int64_t ld_hidden, const void* weight,
                                          int64_t ld_weight, const int64_t* targets, float temperature, int64_t tokens,
                                          const float* logp, const float* entropy, const float* lse,
                                          const float* grad_logp, const float* grad_entropy, void* dhidden,
                                          int64_t ld_dhidden, void* dweight, int64_t ld_dweight, void* stream);

/* As dmuon_read_device_status, for the head's status word (DMUON_DEV_WAIT_TIMEOUT). */
dmuon_status dmuon_head_read_device_status(dmuon_head_t head, void* stream, uint32_t* bits);

/* Free the host-side head (the workspace stays the caller's). NULL is a no-op. */
void dmuon_head_destroy(dmuon_head_t head);

/*
 * ---- Tokens to experts and back
 *
 * What a mixture-of-experts layer does around its experts' products, whose
 * matrices are the largest sets Muon owns ("DMuon" project docs, section
 * "DMuon 能做什么": one owner per expert projection). Assignment i = t*top + k
 * sends token t to expert expert_ids[i]; an id outside 0..experts-1 marks an
 * assignment that is dropped. Rows are ordered by expert and, within one, by
 * assignment.
 *
 *   offsets[e]  rows offsets[e] .. offsets[e+1]-1 belong to expert e
 *   dest[i]     the row of assignment i, -1 when dropped
 *   source[r]   the assignment of row r, -1 past the last row in use
 *
 * Asynchronous on stream, no allocation, deterministic (no atomics whose order
 * could show). Outputs must not overlap inputs. Pointers and stream are of the
 * current device; the calls hold no handle to compare it with.
 */

/* Bytes of scratch dmuon_route_sort needs for up to these sizes (host only):
 * 0 <= tokens, 1 <= top <= 64, tokens*top <= 2^30, 1 <= experts <= 4096. */
dmuon_status dmuon_route_workspace_bytes(int64_t tokens, int32_t top, int32_t experts, size_t* bytes);

/*
 * dmuon_route_sort - order the assignments by expert.
 *  expert_ids  device, tokens x top int64, contiguous.
 *  dest, source  device, tokens*top int32 each;  offsets  device, experts+1 int32.
 *  d_workspace   device scratch, 256-byte aligned, free again when the call's work is done.
 */
dmuon_status dmuon_route_sort(const int64_t* expert_ids, int64_t tokens, int32_t top, int32_t experts, int32_t* dest,
                              int32_t* source, int32_t* offsets, void* d_workspace, size_t bytes, void* stream);

/*
 * dmuon_route_dispatch - the experts' input: xs[r] = x[source[r] / top], zeros
 * for rows not in use.
 *  x   device, tokens x dim of dtype (DMUON_F32/DMUON_BF16), row pitch ld_x.
 *  xs  device, tokens*top x dim, contiguous.
 * Any dim >= 1; rows that start on 16 bytes and are whole 16-byte pieces move
 * 16 bytes at a time, others element by element.
 */
dmuon_status dmuon_route_dispatch(const void* x, int64_t ld_x, const int32_t* dest, const int32_t* source, int64_t tokens,
                                  int32_t top, int64_t dim, int32_t dtype, void* xs, void* stream);

/*
 * dmuon_route_combine - the layer's output: y[t] = sum_k weights[t][k] * ys[dest[t][k]],
 * fp32 sums in the order of k, rounded once. Dropped assignments add nothing.
 *  weights  device, tokens x top fp32, or NULL: all 1. With NULL it is also the
 *           gradient of dmuon_route_dispatch (ys = the gradient of xs).
 *  y        device, tokens x dim, row pitch ld_y.
 */
dmuon_status dmuon_route_combine(const void* ys, const float* weights, const int32_t* dest, int64_t tokens, int32_t top,
                                 int64_t dim, int32_t dtype, void* y, int64_t ld_y, void* stream);

/*
 * dmuon_route_combine_backward - gradients of dmuon_route_combine:
 *   dys[dest[t][k]] = weights[t][k] * dy[t]   (zeros for rows not in use)
 *   dweights[t][k]  = sum_d dy[t][d] * ys[dest[t][k]][d]   (0 when dropped)
 *  dy        device, tokens x dim, row pitch ld_dy.
 *  dys       device, tokens*top x dim, contiguous;  dweights  device, tokens x top fp32.
 */
dmuon_status dmuon_route_combine_backward(const void* dy, int64_t ld_dy, const void* ys, const float* weights,
                                          const int32_t* dest, const int32_t* source, int64_t tokens, int32_t top,
                                          int64_t dim, int32_t dtype, void* dys, float* dweights, void* stream);

/*
 * ---- A mixture's experts for a few tokens
 *
 * What generating with a mixture-of-experts layer needs between its router and
 * its output, in three launches and without the rows in expert order: for
 * assignment i = t*top + k, which sends token t to expert e = expert_ids[i],
 *
 *   h[i] = silu(G_e x_t) * (U_e x_t)      without a gate: silu(U_e x_t)
 *   y[t] = sum_k weights[i] * D_e h[i]    silu(v) = v / (1 + exp(-v))
 *
 * An id outside 0..experts-1 marks an assignment that adds nothing, whatever its
 * weight; a token without others gets zeros. A token may name an expert more
 * than once. Only the matrices of experts that are named are read, from memory
 * once. Sums are fp32; h is held as the sum of two bf16, so that y has the one
 * rounding of its type.
 *
 * For tokens * top <= 2048, and made for far fewer: what it costs is the reading
 * of the experts' matrices. An expert's rows are gone through again for every
 * further 24 of its assignments (8 of 64 experts of 2048 x 1408: 64 tokens 200 us,
 * 128 250, 256 390). With more tokens the experts' own products between
 * dmuon_route_dispatch and dmuon_route_combine use the tensor cores better.
 *
 * Asynchronous on stream, no allocation, deterministic. Pointers and stream are
 * of the current device; the calls hold no handle to compare it with.
 */

/* Bytes of scratch dmuon_experts_forward needs for up to these sizes (host only):
 * 0 <= tokens, 1 <= top <= 64, tokens*top <= 2048, 1 <= experts <= 4096, 1 <= dim, inner <= 2^20, and no matrices
 * of more than 2^30 rows together. */
dmuon_status dmuon_experts_workspace_bytes(int64_t tokens, int32_t top, int32_t experts, int64_t dim, int64_t inner,
                                           size_t* bytes);

/*
 * dmuon_experts_forward
 *  x           device, tokens x dim bf16, row pitch ld_x.
 *  expert_ids  device, tokens x top int64, contiguous;  weights  the same, fp32.
 *  up, gate    device, experts x inner x dim bf16, contiguous; gate may be NULL.
 *  down        device, experts x dim x inner bf16, contiguous.
 *  y           device, tokens x dim bf16, row pitch ld_y.
 *  d_workspace device scratch, 256-byte aligned, its contents need not be
 *              initialised; free again when the call's work is done.
 * Any dim and inner: rows that start on 16 bytes and are whole 16-byte pieces
 * stream through shared memory. Others are read element by element, three to four
 * times as slowly; up and gate are too where it is x whose rows are others. The
 * output must not overlap an input. Where a matrix or h is infinite, y may be NaN in
 * place of an infinity.
 */
dmuon_status dmuon_experts_forward(const void* x, int64_t ld_x, const int64_t* expert_ids, const float* weights,
                                   int64_t tokens, int32_t top, int32_t experts, int64_t dim, int64_t inner,
                                   const void* up, const void* gate, const void* down, void* y, int64_t ld_y,
                                   void* d_workspace, size_t bytes, void* stream);

/* The status word (DMUON_DEV_WAIT_TIMEOUT) of the last call with tokens that used a workspace; each clears it first, and
 * before any it says nothing. */
dmuon_status dmuon_experts_read_device_status(const void* d_workspace, void* stream, uint32_t* bits);

/*
 * ---- The global gradient norm, and clipping
 *
 * Over all tensors of a call, as a training step takes it before its optimizers
 * (matrices on other GPUs are no part of it):
 *
 *   norm   = sqrt(sum over all elements of x^2)
 *   out[i] = grads[i] * min(1, max_norm / norm)
 *
 * Squares are summed in fp32 per vector and unit and in 64 bits beyond; where
 * they leave the range of fp32 (gradients of 1e-30 or 1e30), in 64 bits
 * throughout. A norm that is infinite or NaN, or above fp32's range so that norm
 * is infinite, clips nothing: the gradients stay (out becomes a copy of them), and
 * norm says so. Elements are multiplied by the quotient in fp32, in which it is
 * held too (below 2^-126 it loses digits), and rounded once.
 *
 *  grads    host array of n device pointers; each tensor is contiguous and
 *           aligned to its elements, which is enough.
 *  counts   host array of n: elements of each tensor (0: none, the pointer is
 *           not looked at).
 *  dtypes   host array of n: DMUON_F32 or DMUON_BF16.
 *  n        0..2^20. (norm is 0 where there are no elements.)
 *  norm     device, one float: the norm before clipping.
 *  d_workspace  device scratch, 256-byte aligned, its contents need not be
 *           initialised; free again when the call's work is done.
 *
 * The arrays are read before the call returns. Asynchronous on stream, no
 * allocation, deterministic. Pointers and stream are of the current device.
 */

/* Bytes of scratch the two calls need, whatever the tensors (host only). */
dmuon_status dmuon_clip_workspace_bytes(size_t* bytes);

/* dmuon_grad_norm - the norm alone. A tensor that is named twice counts twice. */
dmuon_status dmuon_grad_norm(const void* const* grads, const int64_t* counts, const int32_t* dtypes, int32_t n,
                             float* norm, void* d_workspace, size_t bytes, void* stream);

/*
 * dmuon_grad_clip - the norm, and the clipped gradients.
 *  out       host array of n device pointers of the gradients' types: out[i] may
 *            be grads[i] (in place) and must not overlap any other tensor of
 *            the call. In place nothing is written where nothing is clipped.
 *  max_norm  >= 0; infinity clips nothing.
 */
dmuon_status dmuon_grad_clip(const void* const* grads, void* const* out, const int64_t* counts, const int32_t* dtypes,
                             int32_t n, float max_norm, float* norm, void* d_workspace, size_t bytes, void* stream);

/* Free the host-side plan (the workspace stays the caller's). NULL is a no-op. */
void dmuon_plan_destroy(dmuon_plan_t plan);

/* Message of the last error on this thread ("" if none). */
const char* dmuon_last_error(void);

/* Library version: major*10000 + minor*100 + patch. */
int32_t dmuon_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DMUON_H */
