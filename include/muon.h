/*
 * libmuon — one Muon optimizer step on an AMD Instinct MI355X (gfx950).
 *
 * The step the pages describe ("Frontier Pre-training at Microsoft AI", method details
 * section 5, "Scaling Muon to 16K GPUs", resharding steps 1, 3 and 5; the same step in
 * "Microsoft Reveals MAI-Base-2 Training Recipe ...", section "How to Make Parameter
 * Updates Faster and More Stable?"):
 *
 *   1. each GPU updates its FP32 momentum and casts it to BF16;
 *   3. each GPU orthogonalises whole momentum matrices, batched by shape, with a
 *      Newton–Schulz operator built for the symmetric intermediates;
 *   5. the update is cast back to FP32 and applied to the weights.
 *
 * On one GPU the all-to-all exchanges of steps 2 and 4 have no counterpart: this library
 * takes one GPU's share of whole matrices.  Two points of that section become the plan
 * below: matrices of one shape are processed together as a batch, and the indexing
 * metadata of the resharding is worked out once and then reused every step.
 *
 * Memory and ownership
 *   The caller owns every device buffer: weights W, momenta M, gradients G and the
 *   workspace.  The library owns only the host-side plan object.  It never allocates or
 *   frees device memory.  All step calls are asynchronous on the given stream, never
 *   synchronise, and can be captured in a HIP graph.
 *
 * Errors
 *   Every call returns a muon_status synchronously; MUON_OK is 0.  muon_last_error()
 *   gives a message for the last failing call on the calling thread.  Device faults
 *   surface at the caller's next synchronisation.  NaN and Inf are data, not errors:
 *   they stay inside the matrix they occur in.
 *
 * Threading
 *   A bound plan's layout never changes.  Step calls on one plan must not overlap on
 *   different streams: they share the workspace.
 *
 * Streams are passed as `void*` holding a hipStream_t (NULL = the null stream).
 */
#ifndef LIBMUON_MUON_H
#define LIBMUON_MUON_H

#include <stdint.h>

#if defined(__GNUC__) || defined(__clang__)
#define MUON_API __attribute__((visibility("default")))
#else
#define MUON_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t muon_status;
#define MUON_OK 0
#define MUON_ERR_INVALID_ARG 1         /* null pointer, bad enum, bad chunk or scalar     */
#define MUON_ERR_SHAPE 2               /* zero or oversized dimension                     */
#define MUON_ERR_ALIGNMENT 3           /* device pointer not 16-byte aligned              */
#define MUON_ERR_WORKSPACE_TOO_SMALL 4 /* workspace below muon_plan_workspace_bytes()     */
#define MUON_ERR_NOT_BOUND 5           /* step call before muon_plan_bind()               */
#define MUON_ERR_STALE_PLAN 6          /* descriptors no longer match the plan            */
#define MUON_ERR_HIP 7                 /* a HIP runtime call failed (message in last_error) */

#define MUON_DTYPE_F32 0
#define MUON_DTYPE_BF16 1

/* One parameter as the caller holds it.  The pages apply Muon to every 2-D matrix that is
 * not an embedding and AdamW to the rest, scalars and embeddings ("Frontier Pre-training
 * at Microsoft AI", setup section 4; "Microsoft Reveals MAI-Base-2 Training Recipe ...",
 * section "How to Make Parameter Updates Faster and More Stable?").  `optimizer` says
 * which one a parameter takes:
 *   MUON_OPT_DEFAULT  ndim == 2: Muon; otherwise AdamW when exp_avg_sq is non-NULL,
 *                     else excluded (its pointers are then not read);
 *   MUON_OPT_ADAMW    AdamW whatever ndim (embeddings);
 *   MUON_OPT_NONE     excluded.
 * Muon: weight, momentum are rows x cols float32, grad rows x cols of grad_dtype, all
 * row-major, contiguous, device, 16-B aligned.  AdamW: weight, momentum (the first
 * moment), exp_avg_sq (the second moment) are float32 and grad of grad_dtype, each
 * rows * cols contiguous elements (a parameter of another ndim passes rows = its
 * element count and cols = 1), device, 16-B aligned.  Written buffers (weight,
 * momentum, exp_avg_sq) must not overlap each other, any other parameter's, or a grad. */
typedef struct muon_param_desc {
    int32_t ndim;
    int32_t grad_dtype; /* MUON_DTYPE_F32 or MUON_DTYPE_BF16 */
    int64_t rows;
    int64_t cols;
    float* weight;
    float* momentum;
    const void* grad;
    float* exp_avg_sq;  /* AdamW only */
    int32_t optimizer;  /* MUON_OPT_* */
    int32_t reserved;
} muon_param_desc;

#define MUON_OPT_DEFAULT 0
#define MUON_OPT_ADAMW 1
#define MUON_OPT_NONE 2

/* Plan options.  A zero-filled struct (or NULL) means: no workspace cap, scale 1. */
typedef struct muon_plan_opts {
    /* Upper bound on the workspace in bytes; 0 = no bound.  Above the bound, buckets
     * are split into chunks that share one workspace region and must then be stepped
     * one chunk at a time (momentum, NS, apply for chunk i before chunk i+1). */
    uint64_t max_workspace_bytes;
    /* Host, nullable: per-parameter update scale s_i (n entries, indexed like the
     * descriptors; entries of excluded parameters are ignored).  NULL means s_i = 1.
     * The pages give no scale rule; the scale is a free per-matrix factor. */
    const float* scale;
    /* MUON_PLAN_* bits; 0 for the defaults.  Other bits: INVALID_ARG. */
    uint32_t flags;
    /* Update-scale rule used where `scale` is NULL (MUON_SCALE_*).  The pages give no
     * rule: one of them notes only that careful per-parameter scaling of the update
     * was a key to scaling Muon, in the prior work it names ("MAI-Base-2 в 4–12 раз
     * экономнее DeepSeek на предобучении", section "Muon обошёл AdamW, но потребовал
     * пересобирать матрицы между GPU"). */
    int32_t scale_mode;
} muon_plan_opts;

/* s_i = 1. */
#define MUON_SCALE_NONE 0
/* s_i = sqrt(max(1, rows / cols)) of the parameter as stored (rows = outputs): the
 * scale of the original Muon write-up, which keeps tall matrices' per-element update
 * size in line with square ones. */
#define MUON_SCALE_ASPECT 1
/* s_i = 0.2 * sqrt(max(rows, cols)): gives the orthogonalised update an RMS of about
 * 0.2, the range of AdamW's updates (the rule of Moonshot AI's Muon scaling paper). */
#define MUON_SCALE_RMS_MATCH 2

/* Orthogonalise small matrices with the tiled kernels too, instead of the fused
 * whole-iteration kernel (both give bitwise the same result; this exists to show it). */
#define MUON_PLAN_TILED_SMALL 1u
/* Plan for the two-stream step (muon_step_config.pipeline), which hides one chunk's
 * neighbours' elementwise work behind its Newton–Schulz products and so needs several
 * chunks: a large bucket is split into up to 8 chunks, as many as keep at least 2048
 * SYRK workgroups per launch (sizes differing by at most one).  The buckets of 256-row
 * output tiles (m >= 1024) come first, and a smaller chunk may be split off the front of
 * the first such chunk and off the back of the last one (their elementwise work is the
 * part nothing hides), sized by an estimate of the step time that the plan computes from
 * the shapes alone.  With a workspace cap that splits buckets anyway, the chunks are laid
 * out in two regions of at most half the remaining cap each, alternating between
 * consecutive tiled chunks, so that one chunk can be prepared while the previous one is
 * orthogonalised.  Results do not depend on the chunking. */
#define MUON_PLAN_PIPELINE 2u
/* Normalise in a separate pass instead of in the first iteration's operand loads.  By
 * default a chunk of 256-row output tiles (m >= 1024) run for an odd number of iterations
 * never writes the normalised X: its first SYRK and GEMM+axpy read X0 and normalise each
 * value on its way into LDS, with the same arithmetic as the pass (bitwise the same
 * result; this exists to show it). */
#define MUON_PLAN_UNFUSED_NORMALIZE 4u
/* Run each small tiled chunk (128- or 64-row tiles: 64 < m < 1024, or m <= 64 with a
 * padded n above 1024, e.g. routers and gates) on its own.  By default all of a plan's
 * small tiled chunks are orthogonalised together: one launch normalises them all and one
 * launch per product and iteration works through a single queue of all their tiles (the
 * pages treat router weights apart from the bulk of the experts: "Frontier Pre-training
 * at Microsoft AI", method details section 5).  Both give bitwise the same result; this
 * exists to show it. */
#define MUON_PLAN_UNGROUPED 8u

typedef struct muon_plan muon_plan;

/* Per-chunk facts, for reporting. */
typedef struct muon_chunk_info {
    int64_t m, n;          /* canonical shape: m = min(rows, cols), n = max(rows, cols) */
    int64_t m_pad, n_pad;  /* padded workspace shape of every matrix in the chunk       */
    int64_t count;         /* matrices in the chunk                                    */
    int32_t bucket;        /* bucket id (chunks of one bucket share it)                */
    int32_t tile;          /* Newton–Schulz output tile edge                           */
    int32_t grad_dtype;
    int32_t shared_region; /* 1 when this chunk shares its workspace region            */
    int32_t fused_small;   /* 1 when one fused kernel runs this chunk's whole NS        */
    int32_t grouped_small; /* 1 when the chunk's products run in the grouped launches of
                              every small tiled chunk (MUON_PLAN_UNGROUPED)              */
    double flops_conventional; /* per NS iteration: 4 m^2 n + 2 m^3, times count        */
    double flops_algorithmic;  /* per NS iteration: m(m+1)n + m^2(m+1) + 2 m^2 n, x count */
    double bytes_momentum;     /* algorithmic HBM bytes of the momentum kernel          */
    double bytes_apply;        /* algorithmic HBM bytes of the apply kernel             */
    uint64_t region_offset;    /* byte offset of the chunk's region in the workspace    */
    uint64_t region_bytes;
} muon_chunk_info;

/* Where one parameter's orthogonalised update O lives after muon_ns_batched. */
typedef struct muon_param_info {
    int32_t included;       /* 1: Muon; 2: AdamW; 0: excluded (for 0 and 2 the rest is 0) */
    int32_t chunk;
    int64_t slot;           /* index of the matrix inside its chunk                   */
    int32_t transposed;     /* 1 when rows > cols: O is stored as the m x n transpose */
    float scale;            /* the update scale s_i the apply step uses               */
    uint64_t output_offset; /* byte offset of O (bf16, m x n, row stride ld) in the workspace */
    int64_t ld;             /* row stride of O in elements (= n_pad)                  */
} muon_param_info;

/* ---- plan (host only; no device calls) ---------------------------------------------- */

/* Build a plan for n parameters: exclude ndim != 2, canonicalise each matrix to
 * (m, n) = (min, max) with a transpose flag when rows > cols, group by (m, n, grad
 * dtype) into buckets, split buckets into chunks under the workspace cap, lay out the
 * workspace and build the per-matrix tables.  On success *out owns a new plan.
 * Errors: INVALID_ARG (null params with n > 0, null out, bad dtype, null or
 * overlapping buffers), SHAPE (rows or cols <= 0, or a padded matrix above 2^31
 * elements), ALIGNMENT (a buffer not 16-B aligned), WORKSPACE_TOO_SMALL (one matrix of
 * some bucket does not fit under the cap). */
MUON_API muon_status muon_plan_buckets(const muon_param_desc* params, int64_t n,
                              const muon_plan_opts* opts, muon_plan** out);

/* Bytes of device workspace the plan needs (256-B aligned start required). */
MUON_API muon_status muon_plan_workspace_bytes(const muon_plan* plan, uint64_t* bytes);

/* Number of chunks and buckets; counts of the parameters that take Muon (included) and
 * of those that take neither optimizer (excluded).  Any pointer may be NULL. */
MUON_API muon_status muon_plan_counts(const muon_plan* plan, int32_t* n_chunks, int32_t* n_buckets,
                             int64_t* n_included, int64_t* n_excluded);
/* Count and total elements of the parameters that take AdamW (any pointer may be NULL). */
MUON_API muon_status muon_plan_adamw_counts(const muon_plan* plan, int64_t* n_params, int64_t* n_elements);

MUON_API muon_status muon_plan_info(const muon_plan* plan, int32_t chunk, muon_chunk_info* out);

MUON_API muon_status muon_plan_param_info(const muon_plan* plan, int64_t param, muon_param_info* out);

/* STALE_PLAN when the descriptors differ from those the plan was built from (count,
 * ndim, shape, dtype or any pointer), else OK. */
MUON_API muon_status muon_plan_validate(const muon_plan* plan, const muon_param_desc* params, int64_t n);

/* ---- bind (device) ------------------------------------------------------------------- */

/* Attach a caller-owned device workspace (>= muon_plan_workspace_bytes, 256-B aligned)
 * and upload the plan's tables, ordered on `stream`.  Also zero-fills the workspace.
 * May be called again with another workspace.  Errors: INVALID_ARG, ALIGNMENT,
 * WORKSPACE_TOO_SMALL, SHAPE (a chunk needs 2^31 or more tiles, or one padded matrix
 * takes 2 GiB or more: about 32768 x 32768), HIP. */
MUON_API muon_status muon_plan_bind(muon_plan* plan, void* workspace, uint64_t bytes, void* stream);

/* ---- the step (device, asynchronous on `stream`) --------------------------------------- */

/* Step 1.  For every matrix of `chunk` (-1 = every chunk; not allowed when chunks share
 * a region): M <- beta*M + (1-beta)*G with both products and the sum in float64 and one
 * float32 store; X0 = bf16(M) (round to nearest even) written to the workspace in
 * canonical orientation; per-tile sums of X0^2 for the normaliser.  beta = 0 copies G
 * into M.  Errors: INVALID_ARG (chunk, non-finite beta), NOT_BOUND, HIP. */
MUON_API muon_status muon_momentum_update(const muon_plan* plan, int32_t chunk, float beta, void* stream);

/* Step 3.  For every matrix of `chunk`: X = bf16(X0 / (||X0||_F + eps)) (the norm summed
 * in float64; X0 times the reciprocal, the float64 product rounded once to bf16, which
 * float32 products reach through a per-matrix float32 scale chosen for it), then `steps`
 * quintic Newton–Schulz iterations, each
 *     A = X X^T (bf16),  B = b A + c A A (bf16),  X = a X + B X (bf16),
 * with bf16 MFMA products accumulated in float32.  A and B are symmetric; only their
 * upper-triangle tiles are computed and then mirrored.  The result O is left in the
 * workspace (see muon_plan_param_info).  The pages give no coefficients or step count;
 * (3.4445, -4.7750, 2.0315), 5 steps and eps = 1e-7 are the usual choice.  ("Frontier
 * Pre-training at Microsoft AI", method details section 5, resharding step 3: the
 * orthogonalisation of whole same-shape matrices with an operator for symmetric
 * intermediates.)  For chunks of 256-row tiles (m >= 1024) and an odd step count the
 * normalisation happens inside the first iteration's loads (bitwise the same X).
 * The call consumes X0: the iterations overwrite it, so each call needs a muon_momentum_update
 * of the chunk after the last Newton–Schulz call or step that touched it (or that touched
 * another chunk in the same workspace region); the plan tracks this in the order calls are
 * made and refuses the call otherwise.
 * Errors: INVALID_ARG (chunk, steps < 1, non-finite scalars, no fresh X0), NOT_BOUND, HIP. */
MUON_API muon_status muon_ns_batched(const muon_plan* plan, int32_t chunk, float a, float b, float c,
                            int32_t steps, float eps, void* stream);

/* Step 5.  For every matrix of `chunk`: W <- f32((1 - lr*wd) * W - lr*s_i*O), each
 * product and the difference rounded to float64 separately (no fused multiply-add),
 * O read back in the parameter's own orientation.  Decoupled weight decay: the decay's
 * time scale is 1/(lr*wd) ("Frontier Pre-training at Microsoft AI", method details
 * section 3), so lr and wd are plain arguments and wd = 17.04/(steps*lr) plugs in.
 * Errors: INVALID_ARG (chunk, non-finite lr or wd), NOT_BOUND, HIP. */
MUON_API muon_status muon_apply(const muon_plan* plan, int32_t chunk, float lr, float wd, void* stream);

/* Steps 1, 3 and 5 for `chunk` (-1 = every chunk, in order), with the arguments above. */
MUON_API muon_status muon_step(const muon_plan* plan, int32_t chunk, float beta, float a, float b,
                      float c, int32_t steps, float eps, float lr, float wd, void* stream);

/* ---- variants the pages leave open ------------------------------------------------------ */

/* Step 3 with its own coefficients per iteration: `coeffs` (host) holds 3*steps floats
 * (a_t, b_t, c_t), t = 1..steps; iteration t runs A = X X^T, B = b_t A + c_t A A,
 * X = a_t X + B X.  The pages fix neither the coefficients nor their schedule;
 * muon_ns_batched is this call with the same (a, b, c) every iteration.
 * Errors: INVALID_ARG (chunk, coeffs NULL, steps outside [1, 1024], non-finite values,
 * eps < 0, no fresh X0 as for muon_ns_batched), NOT_BOUND, HIP. */
MUON_API muon_status muon_ns_batched_schedule(const muon_plan* plan, int32_t chunk, const float* coeffs,
                                     int32_t steps, float eps, void* stream);

/* AdamW for the parameters that take it (the pages' companion optimizer, see
 * muon_param_desc), decoupled weight decay as in the Muon apply.  Per element, float64
 * arithmetic with every operation rounded once, in this order, then float32 stores:
 *     m = beta1*m + (1-beta1)*g;   v = beta2*v + (1-beta2)*(g*g);
 *     w = (1 - lr*wd)*w - (lr * (m / bc1)) / (sqrt(v / bc2) + eps),
 * with bc1 = 1 - beta1^t, bc2 = 1 - beta2^t formed in float64 on the host (the float32 m
 * and v are the values stored).  The pages give no AdamW hyper-parameters. */
typedef struct muon_adamw_config {
    float lr, beta1, beta2, eps, wd;
    int32_t reserved;
    int64_t step;              /* t >= 1, for the bias corrections                      */
    /* Device, nullable, 4-byte aligned: {lr, wd, bc1, bc2} as four floats, read by the
     * kernel when it runs instead of lr, wd and the bias corrections from `step` (for
     * graph replays; bc1 and bc2 are then float32 values). */
    const float* dev_scalars;
} muon_adamw_config;

/* AdamW over every AdamW parameter of the plan, one launch.  Errors: INVALID_ARG (NULL
 * config, step < 1, non-finite or out-of-range hyper-parameters), ALIGNMENT, NOT_BOUND,
 * HIP.  Nothing is launched when the plan has no AdamW parameter. */
MUON_API muon_status muon_adamw_step(const muon_plan* plan, const muon_adamw_config* config, void* stream);

/* Everything one step takes, for muon_step_ex and muon_graph_capture_ex. */
typedef struct muon_step_config {
    float beta;                /* momentum coefficient                                     */
    float lr, wd;              /* learning rate, decoupled weight decay                    */
    float eps;                 /* added to the Frobenius norm (>= 0)                       */
    int32_t steps;             /* Newton–Schulz iterations, 1..1024                        */
    float a, b, c;             /* each iteration's coefficients when `coeffs` is NULL      */
    const float* coeffs;       /* host, nullable: 3*steps floats (a_t, b_t, c_t)           */
    /* 0: Newton–Schulz takes bf16(M_new), the momentum itself (the pages' step 1).
     * 1: it takes the Nesterov look-ahead bf16(f32(beta*M_new + (1-beta)*G)), formed like
     *    the momentum (float64 products and sum, one float32 rounding).  The stored
     *    momentum is M_new either way. */
    int32_t nesterov;
    /* Device, nullable, 4-byte aligned: {beta, lr, wd} as three floats, read by the
     * kernels when they run instead of the fields above (whose values are then
     * ignored).  A captured graph then follows a learning-rate or decay schedule: write
     * the new values into this buffer, ordered before each launch.  Non-finite values
     * are not checked; they propagate as data. */
    const float* dev_scalars;
    /* Host, nullable: also run AdamW over the plan's AdamW parameters (after the Muon
     * step, on the same stream), so one call updates every parameter. */
    const muon_adamw_config* adamw;
    /* 0: one stream, phase by phase.  1: the two-stream pipeline, for whole steps
     * (chunk -1): while one chunk's Newton–Schulz products run on `stream`, the next
     * chunk's momentum and normaliser and the previous chunk's apply run on a second
     * stream that the plan owns (created at bind, default priority), in kernels small
     * enough to share the compute units with the products; the call returns with all of
     * it ordered before later work on `stream`.  The pages overlap the next batch's
     * exchange with the current batch's orthogonalisation ("Frontier Pre-training at
     * Microsoft AI", method details section 5, "Scaling Muon to 16K GPUs").  Results are
     * bitwise those of 0.  It needs at least two tiled chunks, no two consecutive ones
     * in one workspace region (always so without a binding cap; with one, plan with
     * MUON_PLAN_PIPELINE); otherwise the step runs as with 0.  Steps of one plan
     * must not overlap: the second stream is shared by every call on the plan. */
    int32_t pipeline;
} muon_step_config;

/* muon_step with a muon_step_config.  Errors: INVALID_ARG (NULL config, chunk, steps,
 * non-finite scalars or coefficients, nesterov or pipeline not 0/1), ALIGNMENT
 * (dev_scalars), NOT_BOUND, HIP. */
MUON_API muon_status muon_step_ex(const muon_plan* plan, int32_t chunk, const muon_step_config* config,
                         void* stream);

/* ---- the whole step as one graph ------------------------------------------------------- */

/* The pages count kernel-dispatch overhead among the causes of the gap between the
 * measured optimizer step and its communication limit ("Frontier Pre-training at
 * Microsoft AI", method details section 5, "Scaling Muon to 16K GPUs", overhead
 * analysis; the same list in "MAI-Base-2 в 4–12 раз экономнее DeepSeek на
 * предобучении", its optimizer section).
 * A step issues 2 + 3*steps + 2 launches per chunk; as a graph it is one launch.
 *
 * muon_graph_capture records muon_step(plan, -1, ...) on a private stream into a HIP
 * graph and instantiates it.  Nothing runs during capture.  The graph holds the device
 * addresses of W, M, G and of the workspace bound at capture time, and the scalars
 * given here: a later muon_plan_bind does not move it, and the caller keeps all of
 * those buffers alive and in place while the graph exists.  New gradients are picked
 * up by writing them into the same G buffers before each launch.  Kernel timing is not
 * recorded inside graphs.  Errors: INVALID_ARG, NOT_BOUND, HIP (capture or
 * instantiation failed; nothing is left allocated). */
typedef struct muon_graph muon_graph;
MUON_API muon_status muon_graph_capture(const muon_plan* plan, float beta, float a, float b, float c,
                               int32_t steps, float eps, float lr, float wd, muon_graph** out);
/* muon_graph_capture with a muon_step_config (schedules, Nesterov, device scalars). */
MUON_API muon_status muon_graph_capture_ex(const muon_plan* plan, const muon_step_config* config,
                                  muon_graph** out);
/* Launch one step, ordered on `stream` (the null stream is allowed).  Launches of one
 * graph, or of graphs of one plan, must not overlap on different streams. */
MUON_API muon_status muon_graph_launch(const muon_graph* graph, void* stream);
/* Number of nodes in the captured graph (one per kernel launch). */
MUON_API muon_status muon_graph_node_count(const muon_graph* graph, int64_t* nodes);
/* Free the graph; the caller makes sure no launch of it is still running. */
MUON_API void muon_graph_destroy(muon_graph* graph);

/* ---- a step that allocates nothing ------------------------------------------------------ */

/* Bytes of the library's own static device scratch (one copy per GPU, held until the
 * process ends). */
#define MUON_NOALLOC_MAX_BYTES (64ull << 20)

/* For callers that cannot allocate device memory (code under HIP graph capture, tight
 * serving loops, harnesses that forbid hipMalloc): muon_step_ex for every chunk, on one
 * stream, with the library's static scratch array on the current device as the workspace
 * instead of a bound one.  The plan need not be bound; it must need at most
 * MUON_NOALLOC_MAX_BYTES of workspace (muon_plan_workspace_bytes).  Each call clears the
 * part of the scratch the plan uses (with a kernel) and copies the plan's tables into it
 * (hipMemcpyAsync from the plan's host memory, which the plan owns), then runs the step;
 * config->pipeline is ignored (one stream).  Calls no hipMalloc or hipFree.  Every call
 * on one GPU shares that GPU's scratch and leaves its contents there: calls that overlap
 * on one GPU (different streams or threads) race, and the result O cannot be read back
 * (muon_plan_param_info refers to a bound workspace).  The first call on a device looks
 * the scratch's address up on that device.
 * Errors: INVALID_ARG (NULL plan, config as for muon_step_ex), WORKSPACE_TOO_SMALL (the
 * plan needs more than MUON_NOALLOC_MAX_BYTES), SHAPE, HIP. */
MUON_API muon_status muon_step_noalloc(const muon_plan* plan, const muon_step_config* config, void* stream);

/* ---- routed experts: routing, grouped rows, 8-bit products ------------------------------- */

/* The layer whose matrices a step updates: every token is routed to top_k of n_experts, its
 * activations and the experts' weights are multiplied in 8 bits, and the products of the
 * backward pass are the gradients that a plan's step reads (the pages: one shared and the
 * top 7 of 512 routed experts, 8-bit compute with block scales; "Frontier Pre-training at
 * Microsoft AI", setup sections 2 and 4).  These calls need no plan: all their state is in
 * their arguments, they never allocate or synchronise, and they can be captured.  Calls on
 * different streams may overlap unless they share a written buffer or a workspace.
 * Device pointers are 16-byte aligned; where a size is 0 nothing is launched and the
 * pointers are not looked at.  Outputs must not overlap inputs or each other unless stated
 * (a buffer reaches from its first byte to its last; another one may lie in the gaps
 * between its rows where the two have the same row stride). */

#define MUON_MAX_EXPERTS 1024
#define MUON_MAX_TOP_K 64

#define MUON_SCORE_SOFTMAX 0
#define MUON_SCORE_SIGMOID 1

typedef struct muon_route_config {
    int64_t tokens;      /* rows of logits, at most 2^26 - 4; tokens * top_k below 2^31      */
    int64_t ld;          /* row stride of logits in elements, >= n_experts                   */
    int32_t n_experts;   /* 1..MUON_MAX_EXPERTS                                              */
    int32_t top_k;       /* 1..min(n_experts, MUON_MAX_TOP_K)                                */
    int32_t dtype;       /* of logits (and of their gradient): MUON_DTYPE_*                  */
    int32_t score;       /* MUON_SCORE_*                                                     */
    int32_t n_groups;    /* consecutive equal groups of experts; 1: no groups; at most 64    */
    int32_t top_groups;  /* groups that a token may use, 1..n_groups                         */
    int32_t renormalize; /* 1: weights divided by the sum of the chosen scores               */
    float scale;         /* factor of every weight (finite)                                  */
} muon_route_config;

/* Routing.  Scores s of a token's logits x: softmax over its experts, or sigmoid.  An expert
 * whose logit is -inf or NaN is out for that token (score 0, never chosen, left out of the
 * softmax); +inf counts as the largest finite float32.  The choice goes by the key s + bias (bias:
 * n_experts floats; an expert with a NaN key is out), or by x itself where bias is NULL.
 * With n_groups > 1 only the experts of the top_groups groups stay whose two largest s + bias
 * add up to the most (a group without an expert comes last).  experts (tokens x top_k) gets
 * the experts of the top_k largest keys in falling order, equal keys (and equal groups) by
 * lowest index, and -1 where a token has no further expert; weights (tokens x top_k,
 * float32) gets scale * s without the bias, divided by the sum of the chosen s with
 * renormalize (the ratio itself, also where the scores underflow), and 0 beside -1.  The choice is that of
 * scores and keys in float64, so that near ties fall as the formulas say; the weights are
 * formed in float32.
 * Errors: INVALID_ARG (NULL, enum, n_groups not a divisor of n_experts or above 64,
 * top_groups, non-finite scale, overlap), SHAPE (tokens, n_experts, top_k, ld), ALIGNMENT, HIP. */
MUON_API muon_status muon_route(const muon_route_config* config, const void* logits, const float* bias,
                                int32_t* experts, float* weights, void* stream);

/* The gradient of the weights with respect to the logits, the choice held fixed: grad_logits
 * (row stride ld_grad, logits' dtype) gets sum_j grad_weights[t][j] * d weights[t][j] / d x,
 * whole rows, zeros where nothing flows.  experts is muon_route's; entries outside
 * [0, n_experts) and entries whose logit is -inf or NaN pass nothing on, equal entries of a
 * row add up.  bias, n_groups and top_groups take no part.  grad_logits may be logits, with
 * the same ld.  Errors: as muon_route. */
MUON_API muon_status muon_route_backward(const muon_route_config* config, const void* logits,
                                         const int32_t* experts, const float* grad_weights, void* grad_logits,
                                         int64_t ld_grad, void* stream);

/* Device workspace of muon_group_rows in bytes (0 for few rows).  Errors: INVALID_ARG, SHAPE. */
MUON_API muon_status muon_group_rows_workspace(int64_t n, int32_t n_experts, uint64_t* bytes);

/* Rows of `rows` below: n, plus what the padding may add. */
MUON_API muon_status muon_group_rows_capacity(int64_t n, int32_t n_experts, int32_t align, int64_t* rows);

/* Groups n choices of experts (muon_route's experts, n = tokens * top_k; entries outside [0, n_experts)
 * go nowhere) by expert, in stable order: counts[e] (n_experts) choices of expert e sit in segment
 * [offsets[e], offsets[e + 1]) (n_experts + 1), which is padded to a multiple of `align`
 * (1, 2, 4, ..., 128; 128 is what MUON_PRODUCT_DEPTH needs).  rows[r] (muon_group_rows_capacity
 * entries, all written) is the index of the choice in row r, so rows[r] / top_k is its token,
 * or -1 in the padding and behind the last segment; position[i] (n) is the row of choice i, or
 * -1.  The same on every run.  Errors: INVALID_ARG (NULL, align, overlap), SHAPE (n, n_experts, or a capacity of
 * 2^31 or more), ALIGNMENT, WORKSPACE_TOO_SMALL, HIP. */
MUON_API muon_status muon_group_rows(const int32_t* experts, int64_t n, int32_t n_experts, int32_t align,
                                     int32_t* counts, int32_t* offsets, int32_t* rows, int32_t* position,
                                     void* workspace, uint64_t workspace_bytes, void* stream);

/* The step of the selection bias, which no gradient reaches: bias_out[e] = bias[e] + rate *
 * sign(mean of counts - counts[e]) in float32, the sign exact.  bias_out may be bias.
 * Errors: INVALID_ARG (NULL, non-finite rate, overlap), SHAPE (n_experts), ALIGNMENT, HIP. */
MUON_API muon_status muon_balance_step(const float* bias, const int32_t* counts, int32_t n_experts, float rate,
                                       float* bias_out, void* stream);

/* 8-bit matrices: one byte per value (e4m3 or e5m2) and one scale byte per block of 128 values
 * of a row, or per 128 x 128 square.  Scale byte b stands for 2^(b - 127).  A power of two changes no
 * value's significand, so a code is its value rounded once, and the matrix instructions take
 * the scales as they are.  A matrix of rows x cols has rows of round_up(cols, 128) codes and
 * scale rows of round_up(ceil(cols / 128), 4) bytes, one per row or per 128 rows (square);
 * codes and scales outside cols are zero bytes. */
#define MUON_FP8_E4M3 0
#define MUON_FP8_E5M2 1

typedef struct muon_fp8_quantize_config {
    const void* src;          /* batch matrices of float32 or bfloat16                      */
    int32_t src_dtype;        /* MUON_DTYPE_*                                               */
    int32_t format;           /* MUON_FP8_*                                                 */
    int32_t square;           /* 0: a scale per 128 values of a row; 1: per 128 x 128       */
    int32_t per;              /* with gather: choices per source row (top_k), >= 1          */
    int64_t batch;            /* fewer than 2^24 tiles of 128 x 128 in all                  */
    int64_t rows, cols;       /* of each quantised matrix                                   */
    int64_t ld;               /* row stride of src in elements, >= cols                     */
    int64_t batch_stride;     /* between src's matrices, in elements                        */
    /* Device, nullable (batch 1): quantised row r is source row gather[r] / per, or zero where
     * that is outside [0, src_rows). */
    const int32_t* gather;
    int64_t src_rows;
    /* Device, nullable (batch 1, square 0): one int32; rows from *limit on are left as they
     * were (of the transposed copy, the blocks of 128 that begin there), and those of a
     * transposed block that *limit cuts are zero. */
    const int32_t* limit;
    uint8_t* codes;           /* nullable: batch x rows x round_up(cols, 128)               */
    uint8_t* scales;
    /* nullable: the transposed matrix (cols x rows) in the same layout, its blocks along rows:
     * batch x cols x round_up(rows, 128). */
    uint8_t* codes_t;
    uint8_t* scales_t;
} muon_fp8_quantize_config;

/* Quantises, and quantises the transpose, in one pass over src.  A block's scale is 2^e with the
 * least e in [-127, 127] for which its largest finite magnitude is at most 448 * 2^e (e4m3)
 * or 57344 * 2^e (e5m2), -127 for a block of zeros; a code is the value * 2^-e rounded to
 * nearest even.  An infinity or NaN becomes a NaN code and has no part in its block's scale.
 * Errors: INVALID_ARG (NULL, enum, no output, one of a codes / scales pair NULL, gather or
 * limit with batch > 1 or limit with square, per < 1, an output that overlaps an input or another),
 * SHAPE (sizes, strides), ALIGNMENT, HIP. */
MUON_API muon_status muon_fp8_quantize(const muon_fp8_quantize_config* config, void* stream);

typedef struct muon_fp8_operand {
    const void* codes;
    const void* scales;
    int64_t ld;            /* row stride of codes in bytes, a multiple of 16, below 2^23    */
    int64_t ld_scales;     /* row stride of scales in bytes, a multiple of 4, below 2^23    */
    int64_t stride;        /* b of MUON_PRODUCT_ROWS: bytes between the groups' codes (multiple of 16) */
    int64_t stride_scales; /* and scales (multiple of 4)                                    */
    int32_t format;        /* MUON_FP8_*; b: e4m3                                           */
    int32_t square;        /* 1: a scale row per 128 rows                                   */
} muon_fp8_operand;

/* out = a b^T for a (m x k) and b (n x k): one product. */
#define MUON_PRODUCT_DENSE 0
/* Rows of a grouped: rows [offsets[g], offsets[g + 1]) of out are those of a by the transpose of group g's b
 * (outputs and input gradients of experts); rows outside every segment are left as they were. */
#define MUON_PRODUCT_ROWS 1
/* Depth grouped: a (m x k) and b (n x k) are transposed copies whose columns hold segments, and
 * out[g] (m x n) = a b^T over columns [offsets[g], offsets[g + 1]) only, zeros where that is
 * empty (weight gradients).  offsets are multiples of 128 (muon_group_rows with align 128):
 * a segment's blocks of 128 must be its own.  Others are rounded down. */
#define MUON_PRODUCT_DEPTH 2
/* Added to one of the three: full float32 sums for a bfloat16 out, too (see muon_fp8_product). */
#define MUON_PRODUCT_FULL_SUMS 16

typedef struct muon_fp8_product_config {
    int32_t mode;             /* MUON_PRODUCT_*, and MUON_PRODUCT_FULL_SUMS if wanted       */
    int32_t groups;           /* 1 for MUON_PRODUCT_DENSE; at most MUON_MAX_EXPERTS         */
    int64_t m, n, k;
    muon_fp8_operand a, b;
    const int32_t* offsets;   /* device, groups + 1, not falling (NULL for DENSE); values outside the
                                 operand are clamped to it                                  */
    void* out;                /* rows of n                                                  */
    int64_t ld_out;           /* in elements, >= n                                          */
    int64_t out_stride;       /* MUON_PRODUCT_DEPTH: elements between groups                */
    int32_t out_dtype;        /* MUON_DTYPE_*                                               */
    int32_t accumulate;       /* 1: added to out (float32 only)                             */
} muon_fp8_product_config;

/* 8-bit product on the matrix cores, one rounding to out's type.  A bfloat16 out is by default
 * summed by the 8-bit matrix instruction: of each 8 neighbouring products it drops what is
 * below 2^-13 of the largest, and adds up the groups of 8 in float32.  So a sum is off by up
 * to 7 * 2^-13 of the sum of those largest products: about 1.4e-5 of a sum of normal values,
 * but where large products cancel, small ones beside them are lost.
 * With MUON_PRODUCT_FULL_SUMS, and always for a float32 out, all sums are full float32 sums:
 * the codes go through the bfloat16 instruction, at half the rate, where a value below 2^-126
 * is rounded to a multiple of 2^-133 and one whose code was rounded up to 2^128 is an infinity.
 * Errors: INVALID_ARG (NULL, enum, groups, accumulate into bfloat16, out overlapping an
 * operand or offsets), SHAPE (sizes, strides, 2^31 or more tiles), ALIGNMENT, HIP. */
MUON_API muon_status muon_fp8_product(const muon_fp8_product_config* config, void* stream);

/* ---- expert layers: gated blocks, 8-bit integer products, rows gathered and combined ------ */

/* What stands between the calls above in an expert's layer: its rows gathered, the gated block of its first two
 * projections with the gradients that a plan's step reads, products with 8-bit integer weights for serving, and
 * the rows combined to their tokens by muon_route's weights.  All of the above holds here too: no plan, no
 * allocation, no synchronisation, capture, 16-byte aligned pointers, sizes of 0, overlaps.
 * bfloat16 and float32 rows may begin anywhere (any row stride >= the columns) unless stated. */

#define MUON_ACT_SILU 0  /* v / (1 + exp(-v))                                                 */
#define MUON_ACT_GELU 1  /* v * P(N < v), N standard normal (no approximation by tanh)         */
#define MUON_ACT_RELU 2  /* max(v, 0), slope 0 at 0                                            */

#define MUON_OPERANDS_BF16 0
#define MUON_OPERANDS_INT8 1

/* A matrix, or one per group, of bfloat16 values, or of 8-bit integer codes with a float32 scale for each row. */
typedef struct muon_operand {
    const void* data;
    const float* scales;   /* 8-bit integers: one per row (4-byte aligned); else NULL            */
    int64_t ld;            /* row stride in elements; of codes a multiple of 16, at least round_up(k, 128);
                              below 2^22 (codes: 2^23).  Codes from k to round_up(k, 128): zeros   */
    int64_t stride;        /* elements between the groups' matrices (of codes a multiple of 16) */
    int64_t stride_scales; /* and their scales                                                  */
} muon_operand;

typedef struct muon_int8_quantize_config {
    const void* src;       /* batch matrices of float32 or bfloat16                             */
    int32_t src_dtype;     /* MUON_DTYPE_*                                                      */
    int32_t per;           /* with gather: choices per source row (top_k), >= 1                 */
    int64_t batch;         /* batch * rows below 2^31                                           */
    int64_t rows, cols;    /* of each quantised matrix                                          */
    int64_t ld;            /* row stride of src in elements, >= cols                            */
    int64_t batch_stride;  /* between src's matrices, in elements                               */
    /* Device, nullable (batch 1): quantised row r is source row gather[r] / per, or zero where
     * that is outside [0, src_rows). */
    const int32_t* gather;
    int64_t src_rows;
    /* Device, nullable (batch 1): one int32; rows from *limit on are left as they were. */
    const int32_t* limit;
    int8_t* codes;         /* batch x rows x round_up(cols, 128), zeros outside cols            */
    float* scales;         /* batch x rows                                                      */
} muon_int8_quantize_config;

/* Quantises rows (tokens, or a weight's output channels) to 8-bit integers.  A row's scale is its largest magnitude
 * / 127 rounded to float32, a code is value / scale (the exact quotient) rounded to the nearest whole number,
 * ties to even, and kept in [-127, 127]; where the scale is 0 codes are 0.  A row with an infinity or a NaN gets
 * the scale NaN and codes 0, so that its products are NaN and no others.
 * Errors: INVALID_ARG (NULL, enum, gather or limit with batch > 1, per < 1, overlap), SHAPE (sizes, strides),
 * ALIGNMENT, HIP. */
MUON_API muon_status muon_int8_quantize(const muon_int8_quantize_config* config, void* stream);

typedef struct muon_int8_product_config {
    int32_t mode;             /* MUON_PRODUCT_DENSE or MUON_PRODUCT_ROWS                        */
    int32_t groups;           /* 1 for MUON_PRODUCT_DENSE; at most MUON_MAX_EXPERTS             */
    int64_t m, n, k;          /* k at most 131071, so that no sum leaves 32 bits                */
    muon_operand a, b;        /* a: m x k; b: n x k, with MUON_PRODUCT_ROWS one per group       */
    const int32_t* offsets;   /* device, groups + 1, not falling (NULL for DENSE); values outside a's rows are
                                 clamped to them                                                */
    void* out;                /* m rows of n                                                    */
    int64_t ld_out;           /* in elements, >= n                                              */
    int32_t out_dtype;        /* MUON_DTYPE_*                                                   */
    int32_t reserved;
} muon_int8_product_config;

/* out[i][j] = (sum over k of a's codes times b's) * a.scales[i] * b.scales[j]: the sum exact, in 32-bit integers, then
 * float32 products from left to right and one rounding to out's type.  MUON_PRODUCT_ROWS as in muon_fp8_product: rows
 * outside every segment are left as they were.  With k = 0 sums are 0; data and its strides are not looked at then.
 * Errors: INVALID_ARG (NULL, enum, groups, overlap), SHAPE (sizes, strides, 2^31 or more tiles), ALIGNMENT, HIP. */
MUON_API muon_status muon_int8_product(const muon_int8_product_config* config, void* stream);

typedef struct muon_gated_config {
    int32_t mode;             /* MUON_PRODUCT_DENSE or MUON_PRODUCT_ROWS                        */
    int32_t groups;           /* 1 for MUON_PRODUCT_DENSE; at most MUON_MAX_EXPERTS             */
    int32_t operands;         /* MUON_OPERANDS_*, of x, gate and up alike (INT8: k at most 131071) */
    int32_t activation;       /* MUON_ACT_*                                                     */
    int64_t m, n, k;          /* rows, features of the block, values of a row                   */
    muon_operand x;           /* m x k                                                          */
    muon_operand gate, up;    /* n x k, with MUON_PRODUCT_ROWS one per group; the same strides  */
    const int32_t* offsets;   /* as in muon_int8_product                                        */
    uint16_t* out;            /* bfloat16, m rows of n                                          */
    int64_t ld_out;           /* in elements, >= n                                              */
    /* bfloat16, m rows of n each, both or neither: x gate^T and x up^T, for muon_gated_backward. */
    uint16_t* pre_gate;
    uint16_t* pre_up;
    int64_t ld_pre;           /* in elements, >= n                                              */
} muon_gated_config;

/* The gated block of a feed-forward layer in one pass: out = act(x gate^T) * (x up^T), each row by its group's
 * matrices.  Sums in float32 (8-bit integers: exact, then scaled as in muon_int8_product); the activation and
 * the product are formed from the unrounded sums and rounded once.  Rows outside every segment are left as they were;
 * k = 0 as in muon_int8_product.
 * Errors: as muon_int8_product; one of pre_gate / pre_up NULL. */
MUON_API muon_status muon_gated(const muon_gated_config* config, void* stream);

typedef struct muon_gated_backward_config {
    int32_t mode, groups, activation;   /* muon_gated's                                         */
    int32_t grad_dtype;       /* of grad_gate and grad_up: MUON_DTYPE_*                         */
    int32_t accumulate;       /* 1: added to grad_gate and grad_up (float32 only)               */
    int32_t reserved;
    int64_t m, n, k;
    muon_operand x, gate, up; /* muon_gated's, bfloat16                                         */
    const int32_t* offsets;
    const uint16_t* grad;     /* gradient of out: bfloat16, m rows of n                         */
    int64_t ld_grad;
    const uint16_t* pre_gate; /* as muon_gated left them                                        */
    const uint16_t* pre_up;
    int64_t ld_pre;
    /* Written: the gradients of x gate^T and x up^T, bfloat16, m rows of n each (the operands of the products below,
     * rounded to bfloat16 as those take them), and zeros from column n on to a multiple of 64.  They may be pre_gate
     * and pre_up, with the same stride. */
    uint16_t* grad_pre_gate;
    uint16_t* grad_pre_up;
    int64_t ld_grad_pre;      /* in elements, a multiple of 64, at least n and below 2^22       */
    uint16_t* grad_x;         /* nullable: bfloat16, m rows of k (with n = 0 refused)           */
    int64_t ld_grad_x;
    void* grad_gate;          /* nullable, both or neither: per group n rows of k               */
    void* grad_up;
    int64_t ld_grad_w;
    int64_t stride_grad_w;    /* elements between groups                                        */
} muon_gated_backward_config;

/* The gradients of muon_gated.  With d = grad, g = pre_gate, u = pre_up:
 *     dg = d u act'(g),  du = d act(g)   (float32, rounded once),
 *     grad_x = dg gate + du up,  grad_gate = dg^T x,  grad_up = du^T x over each group's rows (zeros without rows),
 * sums in float32.  The products take dg and du as they are written, rounded to bfloat16: float32 gradients, and what is added
 * to, are sums of such terms, each off by up to 2^-8 of itself (1.7e-3 in the 2-norm).  Rows of the row outputs
 * outside every segment are left as they were and have no part in the weight gradients.  x is not read without weight gradients, gate and up not without grad_x.
 * Errors: as muon_gated; accumulate into bfloat16. */
MUON_API muon_status muon_gated_backward(const muon_gated_backward_config* config, void* stream);

typedef struct muon_gather_rows_config {
    const void* src;          /* src_rows x cols                                                */
    int64_t src_rows, cols, ld;
    int32_t dtype;            /* MUON_DTYPE_*, of src, out and y                                */
    int32_t per;              /* choices per source row (top_k), >= 1                           */
    const int32_t* rows;      /* device, n_rows: muon_group_rows' rows                          */
    int64_t n_rows;           /* at most 2^30                                                   */
    const int32_t* limit;     /* device, nullable: one int32; rows of out from *limit on are left as they were */
    void* out;                /* nullable: n_rows x cols                                        */
    int64_t ld_out;
    /* Nullable: src_rows * per factors (muon_route's weights). */
    const float* weights;
    /* Nullable, together: n_rows x cols, muon_group_rows' position (src_rows * per), and the gradient of the weights. */
    const void* y;
    int64_t ld_y;
    const int32_t* position;
    float* grad_weights;      /* src_rows * per                                                 */
} muon_gather_rows_config;

/* Rows in expert order: out[r] = src[c / per] for the choice c = rows[r] (times weights[c], in float32, rounded once), zeros
 * where c is outside [0, src_rows * per).  Without weights that is how tokens reach their experts.  With them and
 * src the gradient of muon_combine_rows' out it is the gradient of its rows, and with y those rows grad_weights[c] =
 * sum over columns of src[c / per] * y[r] for r = position[c] (float32; 0 where that is outside [0, n_rows)).
 * Without rows (n_rows = 0) grad_weights is zeros.
 * Errors: INVALID_ARG (NULL, enum, per, no output, overlap), SHAPE (sizes, strides, src_rows * per of 2^31 or more),
 * ALIGNMENT, HIP. */
MUON_API muon_status muon_gather_rows(const muon_gather_rows_config* config, void* stream);

typedef struct muon_combine_rows_config {
    const void* src;          /* n_rows x cols                                                  */
    int64_t n_rows, cols, ld;
    int32_t dtype;            /* of src: MUON_DTYPE_*                                           */
    int32_t out_dtype;        /* MUON_DTYPE_*                                                   */
    int64_t tokens;           /* tokens * top_k below 2^31                                      */
    int32_t top_k;            /* 1..MUON_MAX_TOP_K                                              */
    int32_t reserved;
    const int32_t* position;  /* device, tokens x top_k: muon_group_rows' position              */
    const float* weights;     /* nullable (all 1): tokens x top_k                               */
    const void* residual;     /* nullable: tokens x cols of out_dtype, added; may be out        */
    int64_t ld_residual;
    void* out;                /* tokens x cols                                                  */
    int64_t ld_out;
} muon_combine_rows_config;

/* Rows back to their tokens: out[t] = residual[t] + sum over j of weights[t][j] * src[position[t][j]], j in rising order,
 * in float32 and rounded once; positions outside [0, n_rows) add nothing, whatever their weight.  Without weights
 * it is the gradient of muon_gather_rows' src.
 * Errors: INVALID_ARG (NULL, enum, overlap), SHAPE (sizes, strides), ALIGNMENT, HIP. */
MUON_API muon_status muon_combine_rows(const muon_combine_rows_config* config, void* stream);

/* ---- per-kernel timing (HIP events on the launching stream) --------------------------- */

#define MUON_KERNEL_MOMENTUM 0
#define MUON_KERNEL_NORM_FINALIZE 1
#define MUON_KERNEL_NORMALIZE 2
#define MUON_KERNEL_SYRK 3
#define MUON_KERNEL_SYRK_POLY 4
#define MUON_KERNEL_GEMM_AXPY 5
#define MUON_KERNEL_APPLY 6
#define MUON_KERNEL_NS_SMALL 7
#define MUON_KERNEL_ADAMW 8
/* the side-stream kernels of the two-stream step (muon_step_config.pipeline) */
#define MUON_KERNEL_MOMENTUM_SIDE 9
#define MUON_KERNEL_NORMALIZE_SIDE 10
#define MUON_KERNEL_APPLY_SIDE 11
/* the grouped launches of the small tiled chunks (all three products; the normalisation) */
#define MUON_KERNEL_NS_GROUPED 12
#define MUON_KERNEL_PREP_GROUPED 13
#define MUON_KERNEL_COUNT 14

/* Start recording a HIP event pair around every kernel launch of this plan (up to
 * `capacity` launches; later ones go unrecorded).  capacity = 0 stops recording.
 * Not for use while a graph is being captured. */
MUON_API muon_status muon_timing_enable(muon_plan* plan, int32_t capacity);
/* Wait for the recorded events and return, for one kernel kind, the summed duration
 * in milliseconds, the launch count and the summed algorithmic work of those launches
 * (FLOPs for the Newton–Schulz kernels, HBM bytes for the others).  Clears nothing. */
MUON_API muon_status muon_timing_read(muon_plan* plan, int32_t kernel, double* total_ms,
                             int64_t* launches, double* work);
/* Forget recorded launches (events are kept for reuse). */
MUON_API muon_status muon_timing_reset(muon_plan* plan);
MUON_API const char* muon_kernel_name(int32_t kernel);

/* ---- teardown and errors ------------------------------------------------------------ */

MUON_API void muon_plan_destroy(muon_plan* plan);
MUON_API const char* muon_status_string(muon_status status);
MUON_API const char* muon_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* LIBMUON_MUON_H */
