/*
 * moe.h -- C ABI of the GB300 (sm_103a) MoE-layer forward megakernel.
 *
 * The operation (what every call below computes) is the forward pass of one
 * Mixture-of-Experts layer, as described in
 *   Weave abstract (arXiv 2609.21483): routing, then dispatch of tokens to
 *     experts, the expert computation, and the combine back to token order,
 *     run as one persistent megakernel whose CTAs are split by a cost model
 *     into data-movement and computation workers once routing is known;
 *   xxqk.cn/news/665650 section 1 (router, top-k expert selection, the
 *     expert matrix products, weighted merge of the expert outputs) and
 *     section 2.1-2.3 (an in-kernel atomic task queue; per-task dependency
 *     counters that release a task when they reach zero; no global barrier);
 *   m.xxqk.cn/news/657744 section 2.1 (scheduling units: an expert's up
 *     projection, then its down projection, large GEMMs split along K) and
 *     section 5.1 (scheduling state lives in device memory passed to the
 *     kernel).
 *
 * Per token t (T tokens, model dim d, E routed experts, top-k, expert FFN
 * dim f, S in {0,1} always-on shared experts):
 *   L[t,e]  = sum_i x[t,i] * Wr[e,i] + b[e]                (fp32 accumulate)
 *   p[t,:]  = softmax(L[t,:]) over all E experts
 *   idx[t,:]= the k experts with the largest p (ties: lower expert index)
 *   w[t,j]  = p[t,idx[t,j]] / sum_j' p[t,idx[t,j']]         (renormalised)
 *   h       = bf16( silu(Wg[e] x_t) * (Wu[e] x_t) ),  silu(z) = z / (1 + e^-z)
 *   y_e     = Wd[e] h
 *   out[t]  = bf16( sum_j w[t,j] * y_{idx[t,j]}  +  y_shared )
 * Tokens are permuted into per-expert rows in the canonical order: experts
 * ascending, tokens ascending inside an expert.
 *
 * Conventions for every entry point:
 *   - bf16 tensors are IEEE bfloat16, row-major, contiguous, 16-byte aligned
 *     device pointers owned by the caller;
 *       x        [T, d]         token activations
 *       router_w [E, d]         router weight (nn.Linear layout)
 *       w_gate   [E+S, f, d]    gate projections, shared expert stored last
 *       w_up     [E+S, f, d]    up projections
 *       w_down   [E+S, d, f]    down projections
 *       out      [T, d]         overwritten (not accumulated)
 *   - a stream argument is a cudaStream_t passed as void* (NULL = the legacy
 *     default stream);
 *   - every int-returning call returns MOE_OK (0) or one of MOE_E_*; the
 *     message of the last failure on the calling thread is moe_last_error();
 *   - a handle serves one stream at a time; calls on one handle are not
 *     thread-safe;
 *   - a handle's workspace is on the device that was current at its reserve call, and
 *     that device is current at the later calls that use it.
 * Limits: d % 128 == 0, d <= 32768, f % 128 == 0, 1 <= k <= E <= 256,
 * k <= 16, S <= 1, 0 <= T <= T_max given to moe_layer_reserve, T_max <= 32768.
 */
#ifndef MOE_H_
#define MOE_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct moe_layer moe_layer_t;

/* status codes */
#define MOE_OK 0
#define MOE_E_INVAL 1   /* bad argument, alignment, size, or T > T_max    */
#define MOE_E_CUDA 2    /* a CUDA call or kernel launch failed             */
#define MOE_E_TIMEOUT 3 /* a device-side wait ran out of its time budget   */
#define MOE_E_DEVICE 4  /* the kernel found an inconsistent scheduler state */
#define MOE_E_NOMEM 5   /* device or pinned host allocation failed         */
#define MOE_E_STATE 6   /* call order: forward before reserve, etc.        */

/* execution modes (option MOE_OPT_MODE) */
#define MOE_MODE_PERSISTENT 0  /* one persistent megakernel, task queue      */
#define MOE_MODE_MULTIKERNEL 1 /* ablation: one kernel per stage, no queue   */
#define MOE_MODE_STATIC 2      /* ablation: one cooperative launch, tasks
                                  assigned round-robin per stage, grid-wide
                                  barriers between stages, no queue          */

/* option keys for moe_layer_set_option */
#define MOE_OPT_MODE 1         /* MOE_MODE_*                                   */
#define MOE_OPT_TIMEOUT_NS 2   /* device wait budget in ns (default 2e9)      */
#define MOE_OPT_MOVER_CTAS 3   /* >0: fixed number of mover workers (a CTA or
                                  a CTA pair each); 0 = the cost model        */
#define MOE_OPT_GRID_CTAS 4    /* >0: CTAs of the persistent (and static)
                                  grid, rounded down to whole workers (at
                                  least one); 0 = one CTA per SM (every SM
                                  pair the device keeps resident, for pairs) */
#define MOE_OPT_SPLIT_K 5      /* down-projection K splits (1,2,4; 0 = auto)  */
#define MOE_OPT_TOKENS_PER_TILE 6 /* max tokens per GEMM tile: 0 = auto, else
                                     16..256 in steps of 16, used rounded up
                                     to a multiple of 32                       */
#define MOE_OPT_FAULT_DROP_TASK 7 /* test only: -1 off; else drop the dependency
                                     notification of the n-th finished GEMM task,
                                     which must end in MOE_E_TIMEOUT            */
#define MOE_OPT_ROUTE_TOKENS 8 /* tokens per router tile: 64 or 128; 0 (default)
                                  = 64 when T <= 1024 and E >= 64, else 128.
                                  A forward with more than 256 router tiles
                                  fails with MOE_E_INVAL                      */
#define MOE_OPT_CLAIM_AHEAD 9  /* claim the next task while running one when at
                                  least this many tasks wait; -1 auto, 0 off  */
#define MOE_OPT_TRACE 10       /* >0: record up to this many task records per
                                  forward (allocates; see moe_layer_get_trace) */
#define MOE_OPT_RELEASE 11     /* when gate/up tiles become ready: 0 = all at
                                  once after the last gather, f-tile major;
                                  1 = per expert after its gathers (default) */
#define MOE_OPT_PREFETCH 12    /* 1 (default): while a GEMM tile finishes, the
                                  TMA producer starts loading the next tile
                                  claimed ahead; 0: off                        */
#define MOE_OPT_BANDS 13       /* 1 (default): the down tiles of the last
                                  quarter of d run at low priority and the
                                  combine is split in two d bands, so the
                                  first band's combine overlaps them; 0: one
                                  band                                         */
#define MOE_OPT_ROUTE_SPLITS 14 /* K splits of a router tile (1..8; 0 = auto:
                                  enough to spread the tiles over the SMs,
                                  8 k blocks per split at least); capped so
                                  that tiles x splits <= the SM count          */
#define MOE_OPT_L2_PREFETCH 15 /* persistent mode: bytes of the first gate/up
                                  weight tiles (experts in index order) to
                                  prefetch into L2 once the plan is published,
                                  while the gathers run; the plan keeps
                                  experts in index order then.
                                  -1 (default) = 96 MiB when S = 0 and the
                                  mean expert load is at most half a GEMM
                                  tile, else off; 0 = off                      */

#define MOE_OPT_PAIR 16        /* CTAs per worker: 2 = GEMM tiles on CTA pairs
                                  (clusters of two SMs sharing one tensor-core
                                  tile, tcgen05 .cta_group::2, M = 256), 1 =
                                  one CTA per tile (M = 128); 0 (default) =
                                  pairs when the mean rows per expert
                                  (T k / E) are at least 128                 */

#define MOE_OPT_FRONT_SPLIT 17 /* persistent mode, once routing is known:
                                  1 = only the cost model's mover workers
                                  prefer the gathers; the GEMM workers run
                                  the GEMM tiles that are ready and take
                                  gathers only when none is; 0 = every worker
                                  prefers gathers while any is left; -1
                                  (default) = 1 without a shared expert, 0
                                  with one                                   */

#define MOE_OPT_FAULT_DROP_TYPE 18 /* test only: 0 off; 2, 3 or 4 = drop every
                                      dependency notification of gather,
                                      gate/up or down tasks, which must end
                                      in MOE_E_TIMEOUT                        */
#define MOE_OPT_FAULT_CORRUPT_COUNT 19 /* test only: 0 off; else the plan adds
                                      this to the first expert's token count;
                                      its check (counts summing to T k) must
                                      end the pass in MOE_E_DEVICE           */
#define MOE_OPT_FAULT_REPUSH 20 /* test only, with MOE_OPT_DEBUG_CLAIMS: -1
                                  off; else the n-th finished gate/up task is
                                  pushed into the queue again, which the
                                  claimed-twice check must end in
                                  MOE_E_DEVICE (without the check the extra
                                  claim can end the queue's count early: the
                                  output is then undefined)                   */
#define MOE_OPT_DEBUG_CLAIMS 21 /* persistent mode: 1 = every task claimed
                                  sets a bit; a task claimed twice (or an id
                                  outside the layer's tasks) sets
                                  MOE_E_DEVICE, never a trap; 0 (default) off */

#define MOE_OPT_FOLD_GATHER 22 /* 1: a routed gate/up tile gathers its token
                                  rows from x itself (warps idle during its
                                  main loop copy them into the stages through
                                  perm, 16 bytes at a time), and the gather
                                  tasks only write perm and pos; 0 (default):
                                  the gather tasks copy the rows into a
                                  permuted buffer that the tiles load by TMA.
                                  Same bits either way; 1 is slower on this
                                  GPU (the copies keep too few bytes in
                                  flight)                                    */

/* statistics keys for moe_layer_get_stat (values of the last forward;
 * moe_layer_status must have been called after it) */
#define MOE_STAT_MOVER_CTAS 1  /* mover workers the cost model chose          */
#define MOE_STAT_TASKS 2       /* tasks executed (all types)                   */
#define MOE_STAT_GRID 3        /* CTAs launched for the persistent kernel
                                  (MOE_STAT_PAIR per worker)                  */
#define MOE_STAT_GEMM_TASKS 4  /* expert GEMM tasks executed                   */
#define MOE_STAT_MOVER_TASKS 5 /* gather + combine tasks executed              */
#define MOE_STAT_STOLEN 6      /* tasks a CTA ran from the other role's queue  */
#define MOE_STAT_AHEAD 7       /* tasks claimed ahead while another one ran    */
#define MOE_STAT_TRACE_RECORDS 8 /* task records the last forward produced     */
#define MOE_STAT_TILE_TOKENS 9 /* max tokens per GEMM tile of the last forward */
#define MOE_STAT_SPLIT_K 10    /* down-projection K splits of the last forward */
#define MOE_STAT_BANDS 11      /* d bands of the last forward (1 or 2)         */
#define MOE_STAT_Y_BYTES 12    /* bytes the combine read per down-projection
                                  output value in the last forward: 2 (bf16
                                  outputs) or 4 * split_k (fp32 partials)     */
#define MOE_STAT_COMBINE_TOKENS 13 /* tokens per combine tile of the last
                                      forward                                  */
#define MOE_STAT_PAIR 14       /* CTAs per worker of the last forward (1 or 2) */

/* Create a layer description.  Pure host call (no CUDA call, no allocation on
 * the device).  Returns NULL on invalid dimensions (see moe_last_error),
 * among them d > 32768: a gather copies whole bf16 token rows through the
 * pipeline's shared memory, which holds a 64 KB row under every tiling. */
moe_layer_t* moe_layer_create(int d, int f, int E, int k, int shared_experts);

/* Allocate the device workspace for up to T_max tokens on the current device
 * (routing arrays, permuted activations, expert intermediates, scheduler
 * state) and cache the device properties.  The only allocating call besides
 * moe_layer_forward_host's first use; call it before any stream capture.
 * May be called again to grow or shrink; a graph captured before that holds the
 * freed workspace and must not be replayed. */
int moe_layer_reserve(moe_layer_t* h, int T_max, void* stream);

/* Set the per-expert router bias (fp32 [E] device pointer, added to the
 * logits before softmax and top-k); NULL removes it.  The pointer is read at
 * every forward and must stay valid. */
int moe_layer_set_router_bias(moe_layer_t* h, const float* bias);

/* One forward pass of the layer on T tokens (device pointers, see the layout
 * above).  Asynchronous on `stream`; allocates nothing and never synchronises,
 * so it can be captured in a CUDA graph.  Device-side failures (timeouts,
 * inconsistent state) are reported by the next moe_layer_status. T == 0 is a
 * no-op. */
int moe_layer_forward(moe_layer_t* h, int T, const void* x, const void* router_w,
                      const void* w_gate, const void* w_up, const void* w_down, void* out,
                      void* stream);

/* The same forward pass on a routing that the caller gives, in place of the
 * layer's own router: idx [T, k] int32 and w [T, k] fp32 (device pointers,
 * 4-byte aligned), such as moe_router_forward writes them -- sigmoid scores,
 * groups, a balance bias, weights that are not renormalised.
 *   out[t] = bf16( sum_j w[t,j] * y_{idx[t,j]}  +  y_shared )
 * Each token's k experts are in [0, E) and distinct; else the pass ends in
 * MOE_E_DEVICE (moe_layer_status) and its output is undefined.  So the slots
 * that moe_router_forward left without an expert (idx -1: rows of padding, or
 * with fewer than k experts not masked) have to name some other expert of the
 * row first; their w is 0, and adds nothing as long as that expert's y is
 * finite.  The router bias does not enter.  Everything else (modes, options,
 * routing readback, status) is that of moe_layer_forward; with the same routing
 * the output has the same bits. */
int moe_layer_forward_routed(moe_layer_t* h, int T, const void* x, const int32_t* idx,
                             const float* w, const void* w_gate, const void* w_up,
                             const void* w_down, void* out, void* stream);

/* The forward pass with the residual add and the RMSNorm that end the MoE
 * megakernel (xxqk.cn/news/665650 section 1 lists them after the weighted
 * merge) fused into the combine.  Per token t, with layer[t] the value
 * moe_layer_forward rounds to bf16:
 *   out[t]      = bf16( residual[t] + layer[t] )          (fp32 add)
 *   norm_out[t] = bf16( out[t] * rsqrt(mean_c out[t,c]^2 + eps) * gamma )
 * the mean over the d values of out[t] as stored (bf16).  residual [T, d] and
 * gamma [d] are bf16 device pointers, norm_out [T, d] is overwritten; all
 * 16-byte aligned; 0 <= eps <= 1.  Everything else (routing, scheduling,
 * status, asynchrony, no allocation) is that of moe_layer_forward, except
 * that the combine covers whole rows (MOE_OPT_BANDS does not apply): each
 * combine task adds the residual rows, bulk-copied with the expert rows, and
 * then normalises its tile's rows. */
int moe_layer_forward_residual_norm(moe_layer_t* h, int T, const void* x, const void* router_w,
                                    const void* w_gate, const void* w_up, const void* w_down,
                                    const void* residual, const void* gamma, float eps,
                                    void* out, void* norm_out, void* stream);

/* The same forward pass with x and out in host memory: copies x to the
 * device, runs moe_layer_forward, copies out back and synchronises the
 * stream.  Weights are device pointers as above.  Host buffers may be
 * pageable or pinned; the first call allocates a device staging area for
 * T_max tokens.  Returns the device status of the pass as well. */
int moe_layer_forward_host(moe_layer_t* h, int T, const void* x_host, const void* router_w,
                           const void* w_gate, const void* w_up, const void* w_down,
                           void* out_host, void* stream);

/* The same forward pass without any allocation, for callers that cannot call
 * cudaMalloc: processes whose device memory is owned by another allocator (a
 * framework's caching allocator that must account for every byte), and
 * runtimes that forbid allocation after start-up (fixed memory budgets,
 * real-time or certified deployments).  (The pages have no counterpart: this
 * is an interface convenience, not part of the method.)  Needs only
 * moe_layer_create (host memory); no moe_layer_reserve.  Its scratch is a
 * fixed 32 MiB array inside this library's device code, which every GPU that
 * loads the library holds until the process exits.  Layers whose workspace
 * for T tokens exceeds it are rejected with MOE_E_INVAL and a message naming
 * the size needed (the decode-sized layer, T=256 d=4096 E=8 k=2 f=14336,
 * fits).  The first call on a device looks up the scratch array's device
 * address and sets kernel attributes (no allocation); make that first call
 * before any stream capture.  Later calls look the address up again and
 * redo that set-up if it changed (after a device reset).  Every call on a
 * device shares the one array and the array keeps the last call's contents:
 * the scheduler state is cleared at each call, but calls that overlap on the
 * GPU (two streams, two threads, two handles) race on it.  Inputs, outputs,
 * layouts, options and the asynchronous behaviour are those of
 * moe_layer_forward.  When the fp32 K-split partials of the down projection
 * do not fit the scratch, it keeps them in bf16 with one K split, so its
 * results may differ from moe_layer_forward's in the last bits (both stay
 * within the oracle's tolerance).  After a call, moe_layer_status and
 * moe_layer_get_routing on the same handle report this call (read from the
 * shared array: call them before another no-allocation forward runs on the
 * device); moe_layer_get_trace does not cover these calls. */
int moe_layer_forward_noalloc(moe_layer_t* h, int T, const void* x, const void* router_w,
                              const void* w_gate, const void* w_up, const void* w_down, void* out,
                              void* stream);

/* Copy the routing of the last forward into caller device buffers (any may be
 * NULL): idx int32 [T,k], w fp32 [T,k] (renormalised weights, slot order),
 * counts int32 [E], offsets int32 [E+1], perm int32 [T*k] (source token of
 * each permuted row), pos int32 [T,k] (permuted row of each (token, slot)).
 * Asynchronous on `stream`. */
int moe_layer_get_routing(moe_layer_t* h, int32_t* idx, float* w, int32_t* counts,
                          int32_t* offsets, int32_t* perm, int32_t* pos, void* stream);

/* Synchronise `stream`, then return and clear the sticky device status of the
 * last forward (MOE_OK, MOE_E_TIMEOUT or MOE_E_DEVICE), or MOE_E_CUDA when a
 * CUDA error is pending. */
int moe_layer_status(moe_layer_t* h, void* stream);

/* Automatic granularity calibration (the per-workload tuning of task
 * granularity discussed in xxqk.cn/news/665650 section 4.4 and
 * m.xxqk.cn/news/657744 section 5.2): times the forward pass on these inputs
 * for a few candidate settings -- tokens per GEMM tile (auto, 64, 128, 160,
 * 256), down-projection K splits (auto, 1, 2, 4), one or two d bands -- by
 * coordinate descent from the current options, `reps` timed passes each
 * (1..100, after one untimed pass), and keeps the fastest as the handle's
 * options (MOE_OPT_TOKENS_PER_TILE, MOE_OPT_SPLIT_K, MOE_OPT_BANDS).
 * Arguments are those of moe_layer_forward (out is overwritten, 1 <= T);
 * best_us (may be NULL) receives the best mean time in microseconds.  It runs
 * 10-20 forwards and synchronises the stream after each candidate, so call it
 * at set-up, not under stream capture; it allocates nothing (two CUDA events).
 * Candidates that fail (a tile too large, a device timeout) are skipped; the
 * MOE_STAT_TILE_TOKENS / _SPLIT_K / _BANDS statistics of the next forward
 * report the chosen tiling.  The expert selection of every candidate is the
 * same; K splits change the fp32 summation order, so outputs may differ from
 * the uncalibrated pass in their last bits. */
int moe_layer_calibrate(moe_layer_t* h, int T, const void* x, const void* router_w,
                        const void* w_gate, const void* w_up, const void* w_down, void* out,
                        int reps, float* best_us, void* stream);

/* Set an option (MOE_OPT_*).  Takes effect at the next forward. */
int moe_layer_set_option(moe_layer_t* h, int key, long long value);

/* Read a statistic (MOE_STAT_*) of the last forward whose status was read. */
long long moe_layer_get_stat(moe_layer_t* h, int key);

/* Copy the task trace of the last forward (option MOE_OPT_TRACE) into a host
 * buffer of `cap` records; synchronises `stream`.  Each record is four
 * uint64: (CTA index << 32) | task id, then three %globaltimer readings in ns:
 * when the CTA began claiming the task, when it began running it, and when
 * it had published its results.  Task id bits 28-31 hold the type (1 router
 * tile, 2 gather, 3 gate/up GEMM, 4 down GEMM, 5 combine).  Returns the
 * number of records copied, or -1 on error. */
int moe_layer_get_trace(moe_layer_t* h, uint64_t* records, int cap, void* stream);

/* Bytes of device workspace moe_layer_reserve(T_max) allocates (host-only;
 * -1 for a NULL handle or T_max < 0).  Not monotone in T_max: while four
 * fp32 K-split partials of the down-projection outputs of T_max tokens fit
 * in 512 MB the workspace holds them, beyond that only bf16 outputs. */
long long moe_layer_workspace_bytes(const moe_layer_t* h, int T_max);

/* Free the workspace and the handle.  NULL is ignored. */
void moe_layer_destroy(moe_layer_t* h);

/* ------------------------------------------------------------------ routing
 *
 * Routing of tokens to experts as an operator of its own, for scores, biases
 * and groups that the layer's built-in router (softmax, top-k, renormalise)
 * does not have, with its gradient for training; moe_layer_forward_routed and
 * moe_w4_forward take its result.  Per token, with the logits
 * l over E experts:
 *   s   = softmax(l) or sigmoid(l)                       (the scores)
 *   c   = s + bias; without a bias the order of l itself (what selects)
 *   groups of E / groups consecutive experts are ranked by their largest c
 *         (MOE_GROUP_MAX) or the sum of their two largest (MOE_GROUP_TOP2;
 *         without a bias, of their two largest s); the experts of the best
 *         groups_kept groups stay in the choice
 *   idx = the k largest c, the larger first
 *   w_j = scale * s_j, or scale * s_j / (sum of the kept s) if renormalised
 * Ties go to the lower expert and the lower group.  The bias (the balance
 * bias that training moves against the load) selects only: it is not in w.
 * A logit of -inf masks its expert out: it is never chosen and has the score 0.
 * A bias of -inf keeps its expert from being chosen, whatever its logit.  A
 * slot left without an expert (a row masked out altogether, say) gets idx -1
 * and w 0.  A NaN logit of an expert that is not masked ranks above every
 * number, and shows as NaN in w.  Scores, sums and weights are fp32, and the
 * sigmoid scores that select (not those in w) are within 4e-7: two choices
 * whose c are nearer than that and a few fp32 roundings may be taken either
 * way.  Without a bias (and groups ranked by the maximum) the choice is exact.
 *
 * Row t of the logits is at logits + t * row_stride elements (row_stride >=
 * E), fp32 or bf16, aligned to its type; idx [T, k] int32 and w [T, k] fp32
 * are overwritten; counts (int32 [E], may be NULL) is overwritten with each
 * expert's number of tokens.  Outputs must not overlap inputs.  Both calls
 * are asynchronous, allocate nothing and can be captured in a graph; a handle
 * holds settings alone and may be used by several streams and threads at
 * once.  T = 0 writes counts only. */
typedef struct moe_router moe_router_t;

#define MOE_SCORE_SOFTMAX 0
#define MOE_SCORE_SIGMOID 1
#define MOE_GROUP_MAX 0
#define MOE_GROUP_TOP2 1
#define MOE_TYPE_F32 0
#define MOE_TYPE_BF16 1

/* Limits: 1 <= k <= E <= 256, k <= 16; groups divides E, at most 32;
 * k <= groups_kept * E / groups; scale finite.  NULL on anything else. */
moe_router_t* moe_router_create(int E, int k, int score, int groups, int groups_kept, int group_score,
                                int renormalise, float scale);

int moe_router_forward(const moe_router_t* h, int T, const void* logits, int logits_type,
                       long long row_stride, const float* bias, int32_t* idx, float* w,
                       int32_t* counts, void* stream);

/* The gradient of the weights with respect to the logits, for the choice idx
 * that the forward pass made (the choice itself and the bias have none):
 * grad_w [T, k] fp32 -> grad_logits, every one of its E columns overwritten,
 * of the logits' type, rows grad_row_stride elements apart.  Slots with idx
 * outside [0, E) or naming a masked expert (logit -inf) are passed over; an
 * expert that a row names twice gets the sum.  grad_logits must not overlap the logits. */
int moe_router_backward(const moe_router_t* h, int T, const void* logits, int logits_type,
                        long long row_stride, const int32_t* idx, const float* grad_w,
                        void* grad_logits, long long grad_row_stride, void* stream);

void moe_router_destroy(moe_router_t* h);

/* -------------------------------------------------------------- 4-bit weights
 *
 * A matrix [rows, cols] of 4-bit weights is
 *   codes   [rows, cols / 2] bytes: column 2 i in the low half, 2 i + 1 in the
 *           high half of byte i
 *   scales  [rows, cols / group] bf16, a group being 32, 64 or 128 consecutive
 *           columns of a row
 *   zeros   [rows, cols / group] bytes, of which the low four bits count, or
 *           NULL: 8 everywhere
 *   value = (code - zero) * scale
 */

/* bf16 weights w [rows, cols] -> codes, scales and, if zeros is not NULL,
 * zero points.  Per group, with division and rounding (half to even) in fp32:
 *   without zeros: scale = bf16(max |w| / 7), code = 8 + clamp(round(w / scale), -8, 7)
 *   with zeros:    lo = min(0, min w), hi = max(0, max w), scale = bf16((hi - lo) / 15),
 *                  zero = clamp(round(-lo / scale), 0, 15),
 *                  code = clamp(round(w / scale) + zero, 0, 15)
 * A scale of 0 divides as 1.  A group with an infinity or a NaN gets the scale
 * NaN and codes at the zero point.  w and codes are 16-byte aligned, cols a multiple of
 * group.  Asynchronous, allocates nothing; no two tensors overlap. */
int moe_w4_quantize(long long rows, int cols, int group, const void* w, void* codes, void* scales,
                    void* zeros, void* stream);

/* The values as bf16 (one rounding): the way back, to moe_layer_forward for
 * prompts, whose products the tensor cores bound and not the weights' bytes. */
int moe_w4_dequantize(long long rows, int cols, int group, const void* codes, const void* scales,
                      const void* zeros, void* w, void* stream);

/* Experts on 4-bit weights, for decode batches (T <= 1024): given the routing
 * (idx, w) of moe_router_forward or of moe_layer_get_routing,
 *   h       = bf16( silu(Wg[e] x_t) * (Wu[e] x_t) )
 *   out[t]  = bf16( sum_j w[t,j] Wd[e_j] h_j  +  shared expert's, weight 1 )
 * with the weights' 4-bit values and fp32 sums.  (From a mean of 9 rows an
 * expert and 33 slots on, the kernels for larger batches round each weight to 11
 * bits; with fewer no weight is rounded.  So a token's bits may differ from one
 * batch size to another.)  Magnitudes of x and h are taken to lie below
 * 2^64, those below 2^-57 count as zero; scales between 2^-86 and 2^31, or 0.
 * In larger batches a scale under 2^-24 of its weight row's largest, and a value
 * of x or h under 2^-29 of its token row's, lose bits.  Slots with idx outside
 * [0, E) add nothing (the rows behind a padded batch's last sequence: idx -1);
 * an expert named twice by a row counts twice.  Shapes: gate and up
 * [E + S, f, d], down [E + S, d, f] (groups along the last axis), the shared
 * expert last.  Limits: those of moe_layer_create, and f <= 32768.
 * The handle owns a workspace and serves one stream at a time. */
typedef struct moe_w4 moe_w4_t;

typedef struct moe_w4_weight {
  const void* codes;
  const void* scales;
  const void* zeros; /* NULL for all three matrices or for none */
} moe_w4_weight;

moe_w4_t* moe_w4_create(int d, int f, int E, int k, int shared_experts, int group);

/* Allocate the workspace for up to T_max (1..1024) tokens, and room for the
 * scales (they are kept twice over, for small and for larger batches: 4 bytes
 * a group, and one for its zero point), on the current device.  The only
 * allocating call; may be called again, on the same device, to grow or shrink
 * the workspace: a graph captured before that holds the freed one and must not
 * be replayed. */
int moe_w4_reserve(moe_w4_t* h, int T_max, void* stream);

/* Bytes that moe_w4_reserve(T_max) allocates in all; -1 for a NULL handle or a T_max
 * outside 0..1024. */
long long moe_w4_workspace_bytes(const moe_w4_t* h, int T_max);

/* The matrices of every later forward (device pointers, 16-byte aligned).  The
 * codes are read where they are and stay the caller's; the scales and zero
 * points are copied, in the order in which the kernels take them, on `stream`
 * (call it again when they change).  After moe_w4_reserve.  A captured pass
 * reads the copies as they are when it is replayed, but the codes where they
 * were when it was captured: new weights in the old tensors reach it by this
 * call, others need another capture. */
int moe_w4_set_weights(moe_w4_t* h, const moe_w4_weight* gate, const moe_w4_weight* up,
                       const moe_w4_weight* down, void* stream);

/* One pass for T tokens, 0 <= T <= T_max (T = 0 does nothing): x and out
 * [T, d] bf16, idx [T, k] int32, w [T, k] fp32.  Asynchronous, allocates
 * nothing, can be captured in a graph. */
int moe_w4_forward(moe_w4_t* h, int T, const void* x, const int32_t* idx, const float* w, void* out,
                   void* stream);

/* Synchronise `stream`, then return and clear the device status of the passes
 * since the last call: MOE_OK, MOE_E_TIMEOUT (a wait inside a kernel ran out,
 * the pass's output is undefined), or MOE_E_CUDA when a CUDA error is pending. */
int moe_w4_status(moe_w4_t* h, void* stream);

void moe_w4_destroy(moe_w4_t* h);

/* --------------------------------------------------------------- 8-bit rows
 *
 * Activations kept for the backward pass in half their bytes.  Rows [rows, cols]
 * of bf16 or fp32 values are held as
 *   codes   [rows, cols] int8
 *   scales  [rows, ceil(cols / group)] bf16, a group being 32, 64 or 128
 *           consecutive columns of a row, its last one maybe shorter
 *   value = code * scale,  scale = bf16(max |v| / 127) over the group,
 *   code = clamp(round(v / scale), -127, 127)
 * with division and rounding (half to even) in fp32.  A scale of 0 divides as 1.
 * A group with an infinity or a NaN gets the scale NaN and codes 0.
 * moe_norm_forward writes such rows, and moe_norm_backward reads them. */
typedef struct moe_rows8 {
  void* codes;
  void* scales;
} moe_rows8;

/* v [rows, cols] of `type` (MOE_TYPE_F32, MOE_TYPE_BF16), contiguous -> codes and
 * scales; and the way back, rounded once to `type`.  Any cols; tensors are aligned
 * to their types (16 bytes, 8 for the codes, and cols a multiple of the group are
 * faster).  At most 2^30 cols and 2^38 values; where rows are not whole groups or not
 * aligned so, at most 2^34 - 8 pieces, rows * ceil(cols / 256).  Asynchronous, allocate
 * nothing; no two tensors overlap. */
int moe_rows8_quantize(long long rows, int cols, int type, int group, const void* v, void* codes, void* scales,
                       void* stream);
int moe_rows8_dequantize(long long rows, int cols, int type, int group, const void* codes, const void* scales, void* v,
                         void* stream);

/* ------------------------------------------------------ norms about a block
 *
 * What stands between two blocks of a network whose blocks read a normalised
 * residual stream: the norm behind a block (post), its gate and factor, the
 * residual add, and the norm in front of the next block (pre).  Per token, with
 * the residual r, the block's output y and a gate g:
 *   p    = N_post(y), or y
 *   out  = r + scale * g * p                   rounded to r's type
 *   norm = bf16(N_pre(out))                    of the rounded sum, or not at all
 *   N(x) = (x - m) * rstd * gain + shift,  rstd = 1 / sqrt(mean((x - m)^2) + eps),
 *          m = 0 (MOE_NORM_RMS, no shift) or mean(x) (MOE_NORM_LAYER)
 * with fp32 sums.  A gain of NULL is 1, a shift of NULL 0; with unit_offset a gain
 * is 1 + what is stored.  The gate: MOE_GATE_NONE 1; MOE_GATE_CHANNEL [d] of
 * the gains' type; MOE_GATE_TOKEN [T] fp32; MOE_GATE_ELEMENT [T, d] bf16, rows
 * gate_stride elements apart.
 *
 * y and norm are bf16, the residual and out of residual_type.  Row t of a tensor
 * is at its pointer + t * its stride elements (d <= stride, below 4 GB); every tensor is
 * aligned to its type, and rows of a multiple of 8 columns that are aligned to 16
 * bytes (codes to 8) are faster.  Any d from 1 to 32768, up to
 * 2^30 rows.  A row with an infinity or
 * a NaN makes itself NaN, no other. */
#define MOE_NORM_NONE 0
#define MOE_NORM_RMS 1
#define MOE_NORM_LAYER 2
#define MOE_GATE_NONE 0
#define MOE_GATE_CHANNEL 1
#define MOE_GATE_TOKEN 2
#define MOE_GATE_ELEMENT 3

typedef struct moe_norm moe_norm_t;

typedef struct moe_norm_params {
  const void *pre_gain, *pre_shift, *post_gain, *post_shift; /* [d] each, or NULL */
  const void* gate;                                          /* NULL with MOE_GATE_NONE */
  long long gate_stride;                                     /* MOE_GATE_ELEMENT */
  int type; /* MOE_TYPE_* of gains, shifts and a channel gate */
} moe_norm_params;

/* group: of the 8-bit rows.  eps finite and >= 0, scale finite.  NULL on anything
 * else. */
moe_norm_t* moe_norm_create(int d, int pre, int post, int gate, float eps, float scale, int unit_offset, int group);

/* out is written where y is given (it may be the residual itself, in place);
 * without y, post norm and gate, norm is that of the residual (the first block's).
 * stats [T, 4] fp32, 16-byte aligned, may be NULL: post norm's mean and rstd, pre
 * norm's mean and rstd, as the backward pass takes them (0 and 1 where there is no
 * norm).  out8 and y8, each may be NULL: out and y as 8-bit rows, codes [T, d]
 * contiguous, scales 4-byte aligned.  No other tensors overlap.  Asynchronous,
 * allocates nothing, can be captured in a graph; needs no workspace, so a handle
 * may be used by several streams and threads at once.  T = 0 does nothing; what has a row
 * a token (a gate, 8-bit rows) may then be null. */
int moe_norm_forward(const moe_norm_t* h, int T, int residual_type, const void* residual, long long residual_stride,
                     const void* y, long long y_stride, const moe_norm_params* params, void* out, long long out_stride,
                     void* norm, long long norm_stride, float* stats, const moe_rows8* out8, const moe_rows8* y8,
                     void* stream);

/* What the forward pass left: out and y as they were or as 8-bit rows (out: only if
 * grad_norm is given; y: only for the gradients that need it: any but grad_residual,
 * and grad_y with neither post norm nor gate). */
typedef struct moe_norm_kept {
  const void* out;
  long long out_stride;
  const moe_rows8* out8;
  const void* y;
  long long y_stride;
  const moe_rows8* y8;
  const float* stats; /* may be NULL where no norm is passed through */
} moe_norm_kept;

/* Gradients that are wanted, overwritten; NULL: not wanted.  fp32 [d], but those of
 * a token gate fp32 [T] and of an element gate bf16 [T, d]. */
typedef struct moe_norm_grads {
  float *pre_gain, *pre_shift, *post_gain, *post_shift;
  void* gate;
  long long gate_stride;
} moe_norm_grads;

/* Allocate the workspace (moe_norm_workspace_bytes: 20 MB, less for narrow rows,
 * 80 MB for the widest)
 * for gradients [d], on the current device.  Once is enough; the only allocating
 * call. */
int moe_norm_reserve(moe_norm_t* h, void* stream);
long long moe_norm_workspace_bytes(const moe_norm_t* h);

/* With u = (x - m) * rstd from what was kept and stats as they were saved:
 *   through a norm, for the gradient q of its output and t = q * gain,
 *     rstd * (t - u * mean(t u) - [layer] mean(t))
 *   G = grad_out + (grad_norm through the pre norm);   grad_residual = G
 *   P = scale * g * G;   grad_y = P through the post norm
 *   grad gain = sum over rows of q u, grad shift = sum of q  (q: grad_norm, or P)
 *   grad gate = scale * G * p, summed over the rows (channel) or columns (token)
 * grad_out (of residual_type) or grad_norm (bf16) may be NULL: zero.
 * grad_residual (of residual_type; may be grad_out itself, in place) and grad_y (bf16)
 * may be NULL: not wanted.  No other tensors overlap.  Sums over rows are fp32, without
 * atomics, in an order that the form of the call decides: T, the handle's settings,
 * residual_type, which tensors are given and whether out and y are kept in 8 bits,
 * and whether all rows are aligned (to 16 bytes, codes to 8, d a multiple of 8).
 * Calls of one form have the same bits wherever their tensors are; the same rows in
 * another form (unaligned, as part of a larger batch) may differ in the last ones, and so
 * may those of moe_norm_forward.  Asynchronous, allocates nothing, can be
 * captured in a graph; one stream at a time where gradients [d] are wanted (they
 * use the workspace; graphs replayed at once need handles of their own).  T = 0
 * writes zeros to the gradients [d]. */
int moe_norm_backward(const moe_norm_t* h, int T, int residual_type, const void* grad_out, long long grad_out_stride,
                      const void* grad_norm, long long grad_norm_stride, const moe_norm_params* params,
                      const moe_norm_kept* kept, void* grad_residual, long long grad_residual_stride, void* grad_y,
                      long long grad_y_stride, const moe_norm_grads* grads, void* stream);

void moe_norm_destroy(moe_norm_t* h);

/* ------------------------------------------------- the layer for a few tokens
 *
 * moe_layer_forward's and moe_layer_forward_routed's operation for 1 to 16 tokens
 * (decode, speculative decode), in one cooperative kernel that streams the chosen
 * experts' weights: the same tensors, layouts and limits.  What differs:
 *   - h is not rounded to bf16 but kept to 16 bits, with its weight w in it;
 *   - a logit of -inf masks its expert out, and so does a bias of -inf whatever the
 *     logit, as moe_router_forward has it; a NaN logit of an expert that is not
 *     masked ranks above every number, and shows as NaN in w; a slot without an
 *     expert gets idx -1 and w 0, and adds nothing;
 *   - a given routing may have empty slots (idx outside [0, E): the rows behind a
 *     padded batch's last sequence) and may name an expert twice in a row, which
 *     then counts twice; a row of empty slots gets the shared expert's output, or
 *     zeros;
 *   - weights of experts that a token did not choose do not reach it, an infinity
 *     or a NaN among them neither; in a chosen expert's w_down an infinity makes a
 *     NaN, or an infinity of its sign (h is the sum of two numbers, each times it).
 * The handle owns a workspace and serves one stream at a time; graphs that may run
 * at once need handles of their own.  Where a wait inside the kernel ran out, the later
 * passes do nothing until moe_decode_status has been called. */
typedef struct moe_decode moe_decode_t;

/* Limits: those of moe_layer_create, and f <= 32768.  NULL on anything else. */
moe_decode_t* moe_decode_create(int d, int f, int E, int k, int shared_experts);

/* Allocate the workspace for up to T_max (1..16) tokens, on the current device.  The
 * only allocating call; may be called again, on the same device, to grow or shrink
 * it: a graph captured before that holds the freed one and must not be replayed. */
int moe_decode_reserve(moe_decode_t* h, int T_max, void* stream);

/* Bytes that moe_decode_reserve(T_max) allocates; -1 for a NULL handle or a T_max
 * outside 0..16. */
long long moe_decode_workspace_bytes(const moe_decode_t* h, int T_max);

/* One pass for T tokens, 0 <= T <= T_max (T = 0 does nothing), with the layer's
 * router.  bias (fp32 [E]) may be NULL; idx [T, k] int32 and w [T, k] fp32, each may
 * be NULL, get the choice, the larger logit first.  Asynchronous, allocates nothing,
 * can be captured in a graph.  Outputs must not overlap inputs. */
int moe_decode_forward(moe_decode_t* h, int T, const void* x, const void* router_w, const float* bias, const void* w_gate,
                       const void* w_up, const void* w_down, void* out, int32_t* idx, float* w, void* stream);

/* The same on a given routing. */
int moe_decode_forward_routed(moe_decode_t* h, int T, const void* x, const int32_t* idx, const float* w, const void* w_gate,
                              const void* w_up, const void* w_down, void* out, void* stream);

/* Set an option: MOE_OPT_TIMEOUT_NS (from 1000; the default is 2e9), the limit of a pass's
 * waits; MOE_OPT_FAULT_DROP_TASK, test only: -1 off; 0 or 1 = one block does not
 * arrive at the grid's wait for the logits, or at that for h, which must end in
 * MOE_E_TIMEOUT.  Takes effect at the next forward. */
int moe_decode_set_option(moe_decode_t* h, int key, long long value);

/* Synchronise `stream`, then return and clear the device status of the passes
 * since the last call: MOE_OK, MOE_E_TIMEOUT (a wait of the kernel ran out, that pass's
 * output is undefined, and the passes after it did nothing), or MOE_E_CUDA when a CUDA
 * error is pending. */
int moe_decode_status(moe_decode_t* h, void* stream);

void moe_decode_destroy(moe_decode_t* h);

/* Message of the last failed call on this thread ("" if none). */
const char* moe_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H_ */
