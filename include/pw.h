/*
 * pw.h -- C ABI of libpw.so: a GB300-native (sm_103a) fused mixed-precision MoE layer
 * that reads Any-Precision bit-planes and per-row centroid LUTs directly, with a
 * device-resident weight page table, asynchronous page offload/reload and a greedy
 * quality-aware planner.
 *
 * Source of every operation: "PagedWeight: Efficient MoE LLM Serving with Dynamic
 * Quality-Aware Weight Quantization" (arXiv 2607.16184).
 *
 * Conventions shared by every call
 *   - Every call returns pw_status; nothing throws across the ABI.  pw_last_error()
 *     gives a message for the last failing call on a context (or, with ctx == NULL,
 *     on the calling thread).
 *   - A CUDA error met asynchronously (a failed kernel or copy) is sticky: the next call
 *     on the same context returns PW_ERR_CUDA.
 *   - Host inputs are copied; the caller keeps ownership.  Device pointers handed to a
 *     call (x, y, ids, w) are borrowed and must stay valid until the stream reaches the
 *     work.  The context owns planes, LUTs, the page table, pinned host pages and scratch.
 *   - A context is used by one host thread at a time.
 *   - Linear block i = (layer, expert, u), u = 0 gate_up, 1 down, is addressed by the
 *     block id (layer * E + expert) * 2 + u.
 *   - A gate_up block has N = 2*I rows (gate rows 0..I-1, then up rows I..2I-1) and K = H
 *     columns; a down block has N = H rows and K = I columns.
 *   - Bitwidths: a block stores bmax <= 8 bit-planes, plane 0 the most significant bit,
 *     so a b-bit code is the top b planes.  Supported bitwidths are the set bits of
 *     bits_mask (each between 1 and bmax).  A LUT for bitwidth b holds 2^b fp16
 *     centroids per output row.
 *   - Page p of a block is bit-plane p together with LUT_{p+1} when p+1 is supported.
 *     At committed bitwidth q the GPU holds planes 0..q-1 and LUT_c for supported c <= q;
 *     M^b (Eq. 3 of the paper) counts exactly those bytes.
 */
#ifndef PW_H
#define PW_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    PW_OK = 0,
    PW_ERR_INVALID = 1, /* bad argument: nothing was changed */
    PW_ERR_CUDA = 2,    /* a CUDA call failed (message in pw_last_error) */
    PW_ERR_OOM = 3,     /* device or pinned-host memory exhausted: nothing was changed */
    PW_ERR_STATE = 4,   /* the page state forbids the request (e.g. a page in transfer) */
    PW_ERR_TIMEOUT = 5, /* a bounded device wait gave up */
    PW_ERR_BUSY = 6,    /* an earlier transfer of the same block has not landed yet */
    PW_ERR_RANGE = 7    /* an fp16 activation overflowed or an output is not finite */
} pw_status;

typedef struct pw_ctx pw_ctx;
typedef void *pw_stream; /* a cudaStream_t; NULL means the legacy default stream */

enum {
    PW_FLAG_POISON = 1 /* fill retired device pages with 0xFF before reuse (testing) */
};

enum {
    PW_ACCUMULATE = 1, /* pw_moe_forward: y <- bf16(y + layer(x)); y may alias x */
    PW_PRENORM = 2     /* the layer reads RMSNorm(x) = x / sqrt(mean_h x^2 + 1e-6) (unit gain), the
                          way the pre-norm models of the paper's Table 1 feed their MoE blocks */
};

typedef struct {
    int L, E, H, I, K; /* layers, routed experts, hidden, expert intermediate, top-K */
    int Is;            /* shared-expert intermediate; 0 = no shared expert */
    int bmax;          /* bit-planes per block, 1..8 */
    uint32_t bits_mask;/* bit b set <=> bitwidth b supported */
    int renorm;        /* 1: routing weights renormalised over the chosen K */
    int device;        /* CUDA device ordinal */
    int max_tokens;    /* largest T accepted by the forward calls */
    int flags;         /* PW_FLAG_* */
} pw_desc;

/* ---------------------------------------------------------------- lifetime */

/* Create a context on desc->device.  The context holds the state the paper describes for one
 * model: the per-block weight pages and the device weight page table of Sec. 3.1 ("Paged
 * Weight Representation": committed bitwidth q_i, desired bitwidth d_i, per-page residency),
 * the compute and side streams of Sec. 3.3 ("Asynchronous Page Movement"), and the forward
 * scratch of the fused layer of Sec. 3.3.  The paper specifies no API; the call and its
 * plain-C signature are this library's own.  Requires H % 16 == 0, I % 8 == 0, Is % 8 == 0,
 * K <= E <= 256, K <= 8.  Allocates the page table, scratch for max_tokens tokens and
 * the two streams (compute stream = a new non-blocking stream, side stream for page
 * copies).  Errors: PW_ERR_INVALID on bad shapes, PW_ERR_CUDA / PW_ERR_OOM otherwise. */
pw_status pw_create(const pw_desc *desc, pw_ctx **out);
/* Release everything the context owns (device pages, pinned host pages, scratch, streams it
 * created); waits for its streams first.  NULL is ignored. */
void pw_destroy(pw_ctx *ctx);
/* Message of the last failing call on ctx (or of the calling thread when ctx is NULL); owned
 * by the library, valid until the next call on the same context or thread. */
const char *pw_last_error(const pw_ctx *ctx);
/* Library version string (static storage). */
const char *pw_version(void);

/* Stream on which commits (pw_set_bits, pw_offload's lowering, pw_commit's raising) and
 * the context's own copies are enqueued; by default a non-blocking stream the context
 * created.  Forward calls should run on the same stream so that a commit lands between
 * launches (PagedWeight Sec. 3.3: commit only at safe boundaries).  Switching waits for
 * the previous stream.  The caller keeps ownership of a stream it sets. */
pw_status pw_set_stream(pw_ctx *ctx, pw_stream stream);
pw_status pw_get_stream(pw_ctx *ctx, pw_stream *stream);

/* ---------------------------------------------------------------- weights */

/* Pack one linear block (PagedWeight Sec. 3.1 paged weight representation; APL overlaid
 * bit-planes, Sec. 2.2).
 *   idx: uint8 [N][K] codes < 2^bmax, row-major.
 *   lut: fp16 bits, the LUTs of every supported b in ascending b, concatenated:
 *        [N][2^b] for the smallest b, then the next, ...; entries in any order.
 *   q_init: initial committed bitwidth (supported).
 * idx and lut may both be host memory or both be device memory (detected).  Pages
 * 0..q_init-1 become GPU-resident, the rest CPU-resident in pinned host memory.
 * Re-packing a block replaces it (its pages must not be in transfer: PW_ERR_BUSY).
 * The device copy uses a kernel-private tiling of each plane; pw_unpack_indices
 * reproduces the plain codes. */
pw_status pw_pack(pw_ctx *ctx, int layer, int expert, int u, const uint8_t *idx,
                  const uint16_t *lut, int q_init);

/* Router of a layer (Sec. 2.1): Wr fp32 [E][H]; bias fp32 [E] or NULL.
 * Host or device pointers (detected). */
pw_status pw_set_router(pw_ctx *ctx, int layer, const float *Wr, const float *bias);

/* Shared expert of a layer (Table 1 counts shared experts): wgu bf16 bits [2*Is][H]
 * (gate rows, then up rows), wd bf16 bits [H][Is].  Host or device pointers.  The device
 * copy is fp16 (exact for bf16 values in [2^-14, 65504]; smaller ones keep an absolute
 * error below 2^-25); PW_ERR_INVALID if a weight exceeds 65504 in magnitude. */
pw_status pw_set_shared(pw_ctx *ctx, int layer, const uint16_t *wgu, const uint16_t *wd);

/* Gate the shared expert of `layer`: its output for token t is scaled by
 * sigmoid(x_t . wsg), x_t the layer input as the experts read it (RMS-normalised under
 * PW_PRENORM), computed in fp32 by the router.  This is the shared-expert gate of the
 * Qwen1.5-MoE model in Table 1; the pages describe no gating, so layers are ungated until
 * this is called.  wsg: fp32 [H], host or device, copied; NULL removes the gate.  Waits for
 * the context's stream.  PW_ERR_INVALID if the context has no shared expert. */
pw_status pw_set_shared_gate(pw_ctx *ctx, int layer, const float *wsg);

/* ---------------------------------------------------------------- forward */

/* One fused MoE layer (Sec. 3.3 "fused mixed-precision MoE kernel"): router logits in
 * fp32, softmax over E, top-K (ties to the lower expert id, listed by descending
 * probability), token-to-expert bucketing, gate_up with SiLU(gate)*up, down projection
 * and the routing-weighted combine y_t = sum_k r_tk o_tk (k order), plus the shared
 * expert.  Each block is read at the committed bitwidth q_i held in the device page
 * table when the launch runs.
 *   x: device bf16 [T][H]; y: device bf16 [T][H] (with PW_ACCUMULATE, y += layer(x);
 *   y may equal x).  ids (int32 [T][K]) and w (fp32 [T][K]) are optional device
 *   outputs (NULL to skip).  1 <= T <= max_tokens.  Asynchronous on `stream`; no host
 *   synchronisation and no allocation, so it can be captured in a CUDA graph.
 * Activations are handled in fp16 inside the expert kernels: |x| (after the RMS norm under
 * PW_PRENORM) and |h| must stay below 65504.  A value that rounds past it (or a NaN), and a
 * y that is not finite, set a flag in the context that pw_check reports as PW_ERR_RANGE. */
pw_status pw_moe_forward(pw_ctx *ctx, int layer, const void *x, int T, void *y,
                         int32_t *ids, float *w, int flags, pw_stream stream);

/* Wait for the compute stream and report whether a bounded wait inside an expert kernel
 * expired since the last check (PW_ERR_TIMEOUT; the outputs of that launch are invalid),
 * else whether an fp16 activation (x as the experts read it, or h) overflowed or a y came out
 * infinite or NaN (PW_ERR_RANGE; the outputs since the last check are invalid).  Both
 * flags are cleared by the call.  Also reports sticky CUDA errors.  No counterpart in the paper: the fused kernel of
 * Sec. 3.3 synchronises its warps on device barriers, and this library bounds every such
 * wait and reports the ones that gave up here. */
pw_status pw_check(pw_ctx *ctx);

/* The whole stack in place: for l = 0..L-1, x <- bf16(x + layer_l(RMSNorm(x))), i.e.
 * pw_moe_forward with PW_ACCUMULATE | PW_PRENORM and y = x.  x: device bf16 [T][H].  Asynchronous; launched as a CUDA graph replay after the first call
 * for a given (x, T, stream). */
pw_status pw_stack_forward(pw_ctx *ctx, void *x, int T, pw_stream stream);

/* End-to-end variant with host buffers: copies x_host (bf16 [T][H]) to the device,
 * runs pw_stack_forward, copies the result to y_host and waits for it.  Pinned host
 * buffers give full copy bandwidth; pageable ones work too. */
pw_status pw_stack_forward_host(pw_ctx *ctx, const void *x_host, int T, void *y_host);

/* Online routing statistics (Sec. 3.2 "Routing statistics"): per expert of `layer`, the
 * number of (token, k) selections and the sum of their routing weights since the last
 * reset, accumulated by every forward call.  Outputs are host double [E].  Waits for
 * the compute stream. */
pw_status pw_routing_stats(pw_ctx *ctx, int layer, double *count, double *weight_sum,
                           int reset);

/* Routed-input features phi of Eq. 5 (Sec. 3.2 "Prompt residual"), per expert of `layer`,
 * over every forward call since the last reset: with n_t the L2 norm of token t's input as
 * the experts read it (RMS-normalised under PW_PRENORM) and r the routing weight of each
 * (token, k) selection of the expert, phi[e] = (sum r n / sum r, sqrt(sum r n^2 / sum r),
 * max n); zeros for an expert no token reached.  Both linear blocks of an expert share its
 * phi.  Output host double [E][3].  Waits for the compute stream. */
pw_status pw_routing_features(pw_ctx *ctx, int layer, double *phi, int reset);

/* Decode kernel choice (no counterpart in the paper: its fused kernel, Sec. 3.3, has one
 * path; this switch offers a CUDA-core bit-plane GEMV for items too small to fill a tensor-core
 * tile in the memory-bound decode regime).  At decode batch sizes (T < 512) a routed work item -- a 128-row
 * tile of one expert's block times the tokens routed to that expert -- with at most
 * `max_tokens` tokens is computed on the CUDA cores (packed fp16 products of the decoded
 * centroids and the activations, summed in fp32 per 32 columns); larger items go to the
 * tensor cores.  0 sends every item to the tensor cores.  Default 0 (on GB300 the
 * tensor-core items measured faster at every decode size); valid 0..8, else
 * PW_ERR_INVALID.  Takes effect at the next forward launch (captured stack graphs are
 * dropped). */
pw_status pw_set_gemv_tokens(pw_ctx *ctx, int max_tokens);

/* Tracing (no counterpart in the paper; measurement only): while on, every forward records
 * five CUDA timing events per layer, before,
 * between and after its four kernels (router, gate_up, down, combine), on the launch
 * stream; stack graphs captured while on contain the event records.  The events are
 * owned by the context.  pw_profile_read waits for the latest recording of `layer` and
 * writes the four kernel durations in milliseconds to ms[0..3]. */
pw_status pw_set_profiling(pw_ctx *ctx, int on);
pw_status pw_profile_read(pw_ctx *ctx, int layer, float *ms);

/* Routing without allocation.  The paper has no counterpart: this entry point exists for
 * callers that cannot call cudaMalloc (or anything that allocates) where they route, e.g.
 * code running under a memory budget or allocator it does not own.  It runs the same
 * router kernel as pw_moe_forward -- fp32 logits, softmax, top-K, bucketing -- for layer
 * `layer` on device x (bf16 [T][H], 16-byte aligned), writing ids (int32 [T][K]) and w
 * (fp32 [T][K]) to the caller's device buffers.  flags: PW_PRENORM or 0.
 * Its scratch is a static device array of 8 MiB inside libpw.so (held by every GPU that
 * loads the library until the process exits); T is limited by it, and a T whose scratch
 * does not fit returns PW_ERR_INVALID.  The first call on a device looks up the array's
 * device address, so make it before any stream capture.  Calls share the array: calls
 * that overlap on the GPU (e.g. on two streams) race.  Online routing statistics are not
 * updated.  The call returns before the router runs: if the router's bounded wait for its
 * input copies gives up, a pw_check on the context made after the call's stream has run it
 * reports PW_ERR_TIMEOUT (and the ids and w of that call are invalid).  No cudaMalloc, cudaFree or other allocation happens
 * in the call. */
pw_status pw_route_noalloc(pw_ctx *ctx, int layer, const void *x, int T, int32_t *ids, float *w,
                           int flags, pw_stream stream);

/* ---------------------------------------------------------------- page table */

enum { PW_PAGE_GPU = 0, PW_PAGE_CPU = 1, PW_PAGE_TO_CPU = 2, PW_PAGE_TO_GPU = 3 };

typedef struct {
    int layer, expert, u;
    int N, K;
    int q;          /* committed bitwidth (read by the kernels) */
    int d;          /* desired bitwidth (set by the planner and by offload/reload) */
    int pending_q;  /* reload target waiting for its pages, or 0 */
    int state[8];   /* PW_PAGE_* per page 0..bmax-1 */
    int64_t M[9];   /* M^b bytes for b = 0..8 (-1 when b is not supported) */
} pw_block_info;

/* Commit bitwidth q for a block now (stream-ordered write of the device table entry on
 * the ctx stream).  Sec. 3.1 ("Paged Weight Representation"): the page table row holds the
 * committed bitwidth q_i the kernels read, and q_i may only name pages the GPU holds;
 * Sec. 3.3: a bitwidth changes only at a safe boundary, here between launches on the ctx
 * stream.  Every page below q must be GPU-resident (else PW_ERR_STATE, as for an unpacked
 * block); PW_ERR_BUSY while a transfer of the block is in flight; PW_ERR_INVALID if q is not
 * a supported bitwidth or block is out of range. */
pw_status pw_set_bits(pw_ctx *ctx, int block, int q);

/* Offload (Sec. 3.1, Sec. 3.3): lower the committed bitwidth of `block` to q_new first
 * (enqueued on the ctx stream), then copy pages q_new..q-1 to pinned host memory on the
 * side stream after the compute stream has passed the lowering.  The device pages are
 * released by the pw_commit call that sees the copy landed.  PW_ERR_STATE if q_new is
 * not a supported bitwidth below q or a page of the range is not GPU-resident;
 * PW_ERR_BUSY if a transfer of the block is in flight. */
pw_status pw_offload(pw_ctx *ctx, int block, int q_new);

/* Reload: allocate device pages q..q_new-1 and copy them in from pinned host memory on
 * the side stream; q stays unchanged until pw_commit sees the copy landed and then
 * raises q (Sec. 3.1: raise only once GPU-resident).  PW_ERR_OOM if device memory is
 * exhausted (nothing changed); PW_ERR_STATE / PW_ERR_BUSY as for pw_offload. */
pw_status pw_reload(pw_ctx *ctx, int block, int q_new);

/* Apply every transfer that has landed: retire offloaded device pages and commit the
 * raises of landed reloads on the ctx stream (Sec. 3.1: q_i rises only once the pages are
 * GPU-resident; Sec. 3.3 and Fig. 4: a reload becomes visible to the kernels at a later safe
 * commit point, and retired pages become free device memory).  *n_applied (may be NULL) receives the
 * number of raises committed.  Never blocks.  A failed copy rolls its block back
 * (pages stay or become CPU-resident, q is not raised) and returns PW_ERR_CUDA. */
pw_status pw_commit(pw_ctx *ctx, int *n_applied);

/* Wait for every transfer in flight (then pw_commit applies them).  Sec. 3.3's page movement
 * is asynchronous; this is the blocking point a caller uses before teardown or a test. */
pw_status pw_sync_io(pw_ctx *ctx);

/* One row of the weight page table and its host-side state (Sec. 3.1: the committed bitwidth
 * q_i, the desired bitwidth d_i, where each page lives, and M_i^b of Eq. 3 for every b).
 * info: caller storage.  PW_ERR_INVALID if block is out of range.  Does not wait. */
pw_status pw_query(pw_ctx *ctx, int block, pw_block_info *info);

typedef struct {
    int64_t resident_bytes;   /* sum over blocks of M_i^{q_i} (routed planes + LUTs) */
    int64_t device_pool_bytes;/* bytes reserved from cudaMalloc for pages */
    int64_t device_pool_free; /* of which free for reuse */
    int64_t pinned_bytes;     /* pinned host bytes reserved for CPU-resident pages */
    int64_t scratch_bytes;    /* forward scratch */
    int64_t held_bytes;       /* device bytes of the weight pages the GPU holds: resident, in
                                 transfer, or lowered but not yet retired by pw_commit */
} pw_mem_info;
/* Memory accounting of the context (Sec. 3.1 and Eq. 3: the GPU holds M_i^{q_i} bytes of
 * block i; Sec. 3.3: retired pages return to the device budget).  Does not wait. */
pw_status pw_memory(pw_ctx *ctx, pw_mem_info *info);

/* Host-side fault injection for testing the page I/O paths (no GPU fault is ever made; no
 * counterpart in the paper):
 * kind 1 = the n-th next page copy is reported failed instead of issued;
 * kind 2 = the n-th next device page allocation fails;
 * kind 3 = while n != 0, no transfer is observed as landed (the copies still run), so a
 * test can act while pages are in transfer;
 * kind 4 = with n != 0, the next forward's gate_up kernel withholds one barrier arrival of
 *   its first routed chunk (nothing asynchronous is held back), so that the bounded device
 *   wait on it expires: the launch's outputs are invalid and pw_check reports
 *   PW_ERR_TIMEOUT, after which the context is usable as before;
 * kind 5 = bounded device waits of the expert kernels give up after about n microseconds
 *   (n = 0: the default, about 2 s).
 * n = 0 clears kinds 1-4. */
pw_status pw_set_fault(pw_ctx *ctx, int kind, int n);

/* ---------------------------------------------------------------- planner */

typedef struct {
    int T_blk;          /* free-block threshold (Eq. 7) */
    int F_blk;          /* current number of free KV blocks (Eq. 7) */
    double B_KV;        /* bytes of one KV block (Eq. 7) */
    int R;              /* reload margin in blocks (reload when F_blk >= T_blk + R) */
    const double *mass; /* [L][E] routing mass (Eq. 1), or NULL: use the context's
                           online routing statistics (pw_plan_step only) */
    const double *phi;  /* [n_blocks][3] routed-input features (Eq. 5), or NULL: the
                           context's device features, pw_routing_features (pw_plan_step only) */
    const double *rho_hat; /* [n_blocks][n_bits-1] prompt residuals, transition j = bits[j+1] ->
                           bits[j], or NULL: Eq. 5 from phi.  A batch-level table from
                           pw_merge_requests (Sec. 3.2, batched serving); phi is then unused */
} pw_obs;

typedef struct {
    int n_bits;             /* number of supported bitwidths */
    const double *s;        /* [n_blocks][n_bits] offline sensitivity s_i^b (Eq. 2), b ascending */
    const double *head_w;   /* [2][n_bits-1][3] residual heads w_u^{b->b'} (Eq. 5); transition j: bits[j+1] -> bits[j] */
    const double *head_a;   /* [2][n_bits-1] */
    const double *head_c;   /* [2][n_bits-1] confidence c_u^{b->b'} (Eq. 6) */
    double alpha, rho_min, rho_max, eps; /* Eq. 6, Eq. 8 */
    int n_buckets;
    const double *mu;       /* [n_buckets] damage multipliers, bucket 0 hottest (Eq. 8) */
    const int *floors;      /* [n_buckets] bitwidth floors */
    int n_stages;           /* bitwidth-floor stages: stage s allows s+1 levels below q_i */
} pw_offline;

typedef struct {
    int block, from_bits, to_bits;
    double delta;           /* bytes released (offload) or restored (reload) */
} pw_plan_entry;

typedef struct {
    pw_plan_entry *entries; /* caller storage */
    int capacity;           /* entries available; PW_ERR_INVALID if too small */
    int n;                  /* entries written */
    int kind;               /* 0 no plan, 1 offload plan, 2 reload plan */
    int stage;              /* stage of the chosen offload plan, -1 otherwise */
    double D;               /* Eq. 7 byte target */
    double total;           /* bytes of the chosen plan */
} pw_plan;

/* A planner problem over explicit arrays (no context, no GPU). */
typedef struct {
    int n_blocks, n_bits, L, E;
    const int *bits;        /* [n_bits] ascending supported bitwidths */
    const int *q;           /* [n_blocks] committed bitwidths */
    const int *q_init;      /* [n_blocks] bitwidths reloads may restore up to */
    const int *utype;       /* [n_blocks] 0 gate_up, 1 down */
    const int *layer;       /* [n_blocks] */
    const int *expert;      /* [n_blocks] */
    const double *M;        /* [n_blocks][n_bits] M^b bytes (Eq. 3) */
} pw_plan_problem;

/* PlanStep (Algorithm 1 of Sec. 3.2) on an explicit problem: D from Eq. 7; for every
 * stage: score the legal single-level steps with Eqs. 4-6, 8, greedily take the lowest
 * d_hat / Delta until D is met (ties: larger Delta, then lower block); keep each stage's
 * plan; when D > 0 return the lowest stage meeting D, else the largest reduction.  When
 * D == 0 and F_blk >= T_blk + R, returns a reload plan instead (most damaging reduction
 * restored first while the bytes fit in (F_blk - T_blk - R) * B_KV).  Host only. */
pw_status pw_plan_host(const pw_plan_problem *prob, const pw_obs *obs,
                       const pw_offline *off, pw_plan *out);

/* One request's planner signals, for the batch-level merge. */
typedef struct {
    const double *mass;      /* [L][E] the request's routing mass (Eq. 1) */
    const double *rho_hat;   /* [n_blocks][n_bits-1] its prompt residuals (Eq. 5) */
    const double *conf;      /* [2][n_bits-1] its confidence scores c_u^{b->b'} (Eq. 6) */
    double rho_min, rho_max; /* its clipping bounds (Eq. 6) */
    double kv_blocks;        /* KV blocks the request holds: its weight in the merge */
} pw_request_signals;

/* Batched serving (Sec. 3.2): before planning, the signals of the batch's requests are
 * merged into a single batch-level table.  Routing masses, prompt residuals, confidence scores and clipping
 * bounds are each averaged with weights kv_blocks / sum(kv_blocks), requests summed in
 * order.  Outputs (caller storage): mass [L][E], rho_hat [n_blocks][n_bits-1], conf
 * [2][n_bits-1], *rho_min, *rho_max; plan with them by passing rho_hat in pw_obs and conf
 * and the bounds in pw_offline.  PW_ERR_INVALID if n_req < 1, a pointer is NULL, a weight
 * is negative or the weights do not sum to a positive number.  Host only. */
pw_status pw_merge_requests(const pw_request_signals *req, int n_req, int L, int E, int n_blocks,
                            int n_bits, double *mass, double *rho_hat, double *conf, double *rho_min,
                            double *rho_max);

/* PlanStep on the context's page table (q_i, M_i^b) and, when obs->mass is NULL, its
 * online routing statistics (Eq. 1).  Blocks with a page transfer in flight, or a landed
 * reload not yet committed, take no step (they are left out of the problem), so every
 * entry of the plan can be applied at once.  Writes the desired bitwidth d_i of every
 * planned block.  Applying the plan is the caller's pw_offload / pw_reload. */
pw_status pw_plan_step(pw_ctx *ctx, const pw_obs *obs, const pw_offline *off, pw_plan *out);

/* ---------------------------------------------------------------- KV-block allocator */

/* The KV blocks of a paged KV cache and the weight pages share one device budget: the pages
 * an offload retires become headroom for KV blocks, and the planner follows the free KV
 * blocks, the allocator headroom and the pending KV growth (Sec. 3.3).  This allocator hands
 * out logical block ids and keeps the free-block count F_blk that Eq. 7 (Sec. 3.2) turns into
 * the planner's byte target, with S the budget, W the weight-page bytes and B the block size:
 *   capacity  C = floor(max(0, S - W) / B) blocks
 *   U = blocks held by requests, P = blocks announced as pending growth
 *   F_blk = C - U - P  (negative when the budget is overcommitted; pass it as pw_obs.F_blk)
 *   headroom = S - W - U * B bytes
 * W is either set by the caller or read, on every call that needs it, from an attached
 * context (its pw_mem_info.held_bytes, so pages count until pw_commit retires them).  A
 * request is any int64 key.  Host only; an allocator is used by one thread at a time. */
typedef struct pw_kv pw_kv;

typedef struct {
    int64_t budget_bytes;     /* S */
    int64_t block_bytes;      /* B */
    int64_t weight_bytes;     /* W */
    int64_t capacity_blocks;  /* C */
    int64_t used_blocks;      /* U */
    int64_t pending_blocks;   /* P */
    int64_t free_blocks;      /* F_blk = C - U - P */
    int64_t headroom_bytes;   /* S - W - U * B */
} pw_kv_stats;

/* budget_bytes >= 0, block_bytes > 0 and budget_bytes / block_bytes < 2^31 (ids are int32),
 * else PW_ERR_INVALID.  W starts at 0. */
pw_status pw_kv_create(int64_t budget_bytes, int64_t block_bytes, pw_kv **out);
void pw_kv_destroy(pw_kv *kv);
/* W = weight_bytes (>= 0) from now on; detaches a context. */
pw_status pw_kv_set_weight_bytes(pw_kv *kv, int64_t weight_bytes);
/* W = ctx's held weight-page bytes from now on (ctx must outlive the attachment; NULL
 * detaches and keeps the last value read).  PW_ERR_* of pw_memory when reading fails. */
pw_status pw_kv_attach(pw_kv *kv, pw_ctx *ctx);
/* Request r expects to need n_blocks (>= 0) more blocks soon; replaces its previous
 * announcement.  The announced blocks count as taken in F_blk.  PW_ERR_OOM if host memory runs out; nothing has changed
 * then. */
pw_status pw_kv_announce(pw_kv *kv, int64_t request, int64_t n_blocks);
/* Grow request r by n_blocks (>= 0): c = min(n, r's announcement) of them come out of the
 * announcement, the other n - c must fit in F_blk (and their ids in host memory), else PW_ERR_OOM and nothing changes.
 * The granted ids -- the lowest free ones, ascending -- go to ids_out[0..n-1] (NULL: not
 * written). */
pw_status pw_kv_grow(pw_kv *kv, int64_t request, int64_t n_blocks, int32_t *ids_out);
/* Return every block of request r and drop its announcement; the count to *n_released
 * (may be NULL).  An unknown request releases nothing.  (A block that other requests hold too, see pw_kv_fork, stays
 * theirs and does not count.)  PW_ERR_OOM if host memory for the free ids runs out; nothing has changed then. */
pw_status pw_kv_release(pw_kv *kv, int64_t request, int64_t *n_released);
/* Request `child`, which holds no block (else PW_ERR_STATE), gets the first n_blocks blocks of `parent` (which holds as
 * many, else PW_ERR_INVALID): both hold them from then on, a block counts once in U, and it is free when its last holder has
 * returned it.  Costs no block.  A shared block is written to by nobody; pw_kv_unshare comes before that.  PW_ERR_OOM as by
 * pw_kv_release. */
pw_status pw_kv_fork(pw_kv *kv, int64_t parent, int64_t child, int64_t n_blocks);
/* Before request r writes to its block number `index` (PW_ERR_INVALID if it holds fewer): a block that others hold too is
 * replaced by a fresh one, granted as by pw_kv_grow (one block, PW_ERR_OOM).  *src is the block before and *dst the one from
 * now on, whose contents pw_kv_copy brings over; both the same where the block was the request's alone. */
pw_status pw_kv_unshare(pw_kv *kv, int64_t request, int64_t index, int32_t *src, int32_t *dst);
/* Return the blocks of request r behind its first n_keep (>= 0); how many became free to *n_released (may be NULL).
 * Announcements stay.  PW_ERR_OOM as by pw_kv_release. */
pw_status pw_kv_trim(pw_kv *kv, int64_t request, int64_t n_keep, int64_t *n_released);
/* Bring all blocks in use below the id `limit` (at least U, else PW_ERR_INVALID): those at or above it, ascending, go to
 * src[0 .. *n - 1], and the lowest free ids, which take their places in every request, to dst.  pw_kv_copy moves the
 * contents and renames the blocks in device tables.  With capacity < *n nothing is changed but *n (PW_ERR_INVALID).
 * PW_ERR_OOM as by pw_kv_release. */
pw_status pw_kv_compact(pw_kv *kv, int64_t limit, int32_t *src, int32_t *dst, int64_t capacity, int64_t *n);
/* Blocks request r holds and has announced (0 and 0 for an unknown request); either
 * pointer may be NULL.  The held count is the request's weight in pw_merge_requests. */
pw_status pw_kv_request(const pw_kv *kv, int64_t request, int64_t *held, int64_t *announced);
/* Request r's block table in the order granted: *n = its block count, and the first
 * min(*n, capacity) ids go to ids_out. */
pw_status pw_kv_blocks(const pw_kv *kv, int64_t request, int32_t *ids_out, int64_t capacity, int64_t *n);
pw_status pw_kv_get_stats(pw_kv *kv, pw_kv_stats *out);

/* ---------------------------------------------------------------- paged attention */

/* The KV blocks that pw_kv_* hands out hold the keys and values that the attention of a layer
 * reads (the paper's Sec. 3.3 takes the cache and its attention from the serving engine; these
 * calls have no counterpart there).  One engine step serves R requests; request r has
 * ctx_len[r] tokens in the cache and brings new_len[r] new ones.  Rows of q, k, v and o are the
 * new tokens, request after request.  Per step: pw_kv_map, then pw_attn_plan once for each kind
 * of mask; per layer: pw_attn_append, then pw_attn_forward.  All of them are asynchronous on
 * `stream`, allocate nothing and read lengths on the device only, so a step can be captured in
 * a CUDA graph and replayed with new lengths.
 *
 * The position of the row t of request r is p = ctx_len[r] + t - q_start[r], and key position j
 * of its cache lies in block table[row][j / block_tokens] at token j % block_tokens.  The row
 * sees the keys lo <= j < hi with
 *   lo = max(0, doc_start[t] if given, p - window + 1 if window > 0),
 *   hi = min(kv_len[r], max(p + 1, bidir_len[r] if given)),
 * and, with x_j = scale * (q . k_j), then x_j = softcap * tanh(x_j / softcap) if softcap > 0, then
 * x_j -= slope[head] * |p - j| if slopes are given,
 *   o = sum_j softmax(x)_j v_j,  lse = log sum_j exp(x_j)  (natural logarithm).
 * A row that sees no key gets o = 0 and lse = -infinity.  Keys and values a row does not see do
 * not reach it, whatever bits they hold.  (Infinities and NaN among the values of a step's requests cost time: rows in
 * whose key tiles they lie are computed again, by one warp a row at 0.1 to 0.4 us a key.)  Products of q and k and the softmax sums are fp32; the
 * probabilities are rounded to the cache's type for the product with v, which is summed in fp32. */
enum { PW_BF16 = 0, PW_FP16 = 1 };

typedef struct pw_attn pw_attn;

typedef struct {
    int L;                /* layers (caches to bind) */
    int n_heads;          /* query heads, a multiple of n_kv_heads; at most 128 per key/value head */
    int n_kv_heads;
    int head_dim;         /* a multiple of 8, at most 128 */
    int dtype;            /* of q, k, v, o and the caches: PW_BF16 or PW_FP16 */
    int n_blocks;         /* blocks of each cache; valid block ids are 0 .. n_blocks - 1 */
    int block_tokens;     /* tokens of a block: 16, 32, 64 or 128 */
    int max_requests;     /* largest R, at most 4096 */
    int max_tokens;       /* largest n_tokens, at most 2^20 */
    int max_shared_tokens;/* largest n_tokens of a step with n_groups > 0 (0: no such steps) */
    int n_plans;          /* plans kept at a time, 1..16 */
    int device;           /* CUDA device ordinal */
    int max_tree_tokens;  /* largest n_tokens of a step planned by pw_attn_plan_tree (0: no such steps) */
} pw_attn_desc;

/* One engine step.  Every pointer is device memory that stays the caller's. */
typedef struct {
    int R;                  /* requests, 1 .. max_requests */
    int n_tokens;           /* rows of slot and pos: at least the sum of new_len.  Rows past that sum
                               are padding: slot and pos -1, no cache write, o = 0 */
    int max_new;            /* the largest new_len, or an upper bound of it (it chooses tile sizes, and
                               with them the order in which sums are rounded) */
    int table_rows, table_stride; /* rows of table, and entries of a row */
    const int32_t *ctx_len; /* [R] */
    const int32_t *new_len; /* [R], each may be 0 */
    const int32_t *rows;    /* [R] table row of each request, or NULL: request r has row r */
    int32_t *table;         /* [table_rows][table_stride] block ids; entries of cached tokens are read */
    int32_t *q_start;       /* [R + 1] first row of each request */
    int32_t *kv_len;        /* [R] */
    int64_t *slot;          /* [n_tokens] block id * block_tokens + token within the block */
    int32_t *pos;           /* [n_tokens] */
    /* Groups of consecutive requests that share their first tokens: group g is the requests
     * group_start[g] .. group_start[g + 1] - 1, whose first shared_len[g] tokens (a multiple of
     * block_tokens, at most each request's ctx_len) lie in the same blocks.  group_start[0] = 0 and
     * group_start[n_groups] = R; a request alone or a shared_len of 0 is fine.  Those keys are then
     * read once for the group.  n_groups = 0: none, and both pointers are ignored. */
    int n_groups;
    const int32_t *group_start; /* [n_groups + 1] */
    const int32_t *shared_len;  /* [n_groups] */
} pw_kv_step;

/* Create an attention handle: plans, split workspace (about 40 MB), max_tokens * n_heads / 8 bytes of marks and, with
 * max_shared_tokens, 4 * max_shared_tokens * n_heads * (head_dim + 1) bytes for the shared prefixes' results; 32 *
 * max_tree_tokens bytes a plan, 4 * n_blocks bytes and 1792 * L bytes for trees, moved blocks and rotations.  The calls
 * of one handle run on one stream at a time (its workspace is shared by them), and by one host
 * thread.  PW_ERR_INVALID on a shape outside the ranges above, PW_ERR_CUDA / PW_ERR_OOM otherwise. */
pw_status pw_attn_create(const pw_attn_desc *desc, pw_attn **out);
/* Waits for the device's work and releases the handle.  NULL is ignored. */
void pw_attn_destroy(pw_attn *a);
/* The caches of a layer: element (block, token, head, d) of k is k[block * block_stride + token *
 * token_stride + head * head_stride + d] (strides in elements; v likewise), so a block may keep its
 * heads or its tokens outermost.  Addresses are multiples of 16 bytes, strides positive multiples of 8.
 * The memory stays the caller's and outlives the binding; k and v may be bound again.  Layers may share a cache, and k and v
 * may be one (the same address and strides); caches that are not the same share no element. */
pw_status pw_attn_bind(pw_attn *a, int layer, void *k, void *v, int64_t block_stride, int64_t token_stride,
                       int64_t head_stride);
/* Block tables and slot maps of a step, on the device from the lengths: q_start, kv_len, slot, pos, and
 * the table entries of the blocks that the new tokens open.  new_ids [n_ids] are those blocks' ids,
 * request after request in the order granted (pw_kv_grow): request r opens
 * ceil((ctx_len + new_len) / block_tokens) - ceil(ctx_len / block_tokens) blocks.  Ids beyond these are
 * left alone.  A negative length, too few ids or rows, a table row that is too short or an id outside the
 * cache is reported by pw_attn_check (PW_ERR_STATE); entries and slots concerned are -1. */
pw_status pw_kv_map(pw_attn *a, const pw_kv_step *step, const int32_t *new_ids, int n_ids, pw_stream stream);
/* Lay out the attention work of a mapped step under one mask into plan 0 .. n_plans - 1: per row its keys
 * [lo, hi), and the division of all key blocks among the SMs.  window >= 0 (0: none).  doc_start [n_tokens]
 * (NULL: none): position in its request at which the row's document begins, for packed documents.
 * bidir_len [R] (NULL: none): keys below it are seen by every row of the request.  The plan holds for every
 * layer of the step with this mask, until the next pw_attn_plan into it; step's table must stay valid, and
 * its entries are read by each pw_attn_forward: a block may be moved in between.
 * A captured pw_attn_forward may be replayed after its plan was laid out again with the same max_new, n_tokens, table,
 * table_stride and presence of groups, and follows the new lengths and masks.  After one with others (as far as they
 * change the tiles), or while a captured pw_attn_plan has not been replayed, it writes nothing and pw_attn_check
 * reports PW_ERR_STATE.
 * PW_ERR_INVALID also where table_stride and n_tokens allow for 2^31 or more key tiles of 128 over all tiles of
 * rows (a tile is 256 / (n_heads / n_kv_heads) tokens of a request, or max_new where that is less). */
pw_status pw_attn_plan(pw_attn *a, int plan, const pw_kv_step *step, int window, const int32_t *doc_start,
                       const int32_t *bidir_len, pw_stream stream);
/* Write the step's new keys and values to the layer's cache: row t, head h of k is k[t * k_token +
 * h * k_head + d] (strides in elements, multiples of 8; addresses multiples of 16 bytes; v likewise).
 * Rows with slot -1 are skipped. */
pw_status pw_attn_append(pw_attn *a, int layer, const pw_kv_step *step, const void *k, int64_t k_token,
                         int64_t k_head, const void *v, int64_t v_token, int64_t v_head, pw_stream stream);
/* Rotation of queries and keys by position, and norms of both before it.  Of each head the first rot_dim elements make
 * rot_dim / 2 pairs; pair i of a token is turned by the angle f = p * inv_freq[i], p the token's position on axis axis[i]:
 *   a' = scale (a cos f - b sin f),  b' = scale (a sin f + b cos f),
 * with sine and cosine off by less than 2^-22 at every int32 position and for every finite inv_freq (the angle's part of a
 * turn is computed in whole numbers, to 2 10^-9 radians).  Before that a head of q (k) is x / sqrt(mean x^2 + eps) *
 * q_gain (k_gain), where gains are given.  All of it is fp32, rounded once. */
typedef struct {
    int rot_dim;            /* a multiple of 8, at most head_dim; 0: nothing is turned */
    int interleaved;        /* pair i is the elements 2 i and 2 i + 1; else i and i + rot_dim / 2 */
    int n_axes;             /* positions of a token, 1..4 (time, height, width) */
    const double *inv_freq; /* host [rot_dim / 2], finite: radians for each position */
    const int32_t *axis;    /* host [rot_dim / 2], or NULL: every pair follows axis 0 */
    float scale;            /* of sine and cosine: 1 but where a long-context scheme says otherwise; finite */
    const float *q_gain, *k_gain; /* [head_dim], host or device (detected), or NULL: no norm */
    float eps;              /* >= 0, of the norms */
} pw_rope_desc;
/* Set a layer's rotation (everything in desc is copied).  Waits for the device's work, so not while a stream is captured; a
 * pw_attn_rope_append captured before it is to be captured again. */
pw_status pw_attn_set_rope(pw_attn *a, int layer, const pw_rope_desc *desc);
/* Norms, rotation and cache write of the step's rows in one pass: q to q_out, k and v to the layer's cache (v as it is).
 * q, q_out, k and v as in pw_attn_append, q and q_out with n_heads heads; q_out may be q itself (same strides) and overlaps
 * nothing else.  pos: int32 [n_axes][n_tokens], or NULL: step->pos for every axis (for drafted trees: pw_tree's pos).  Rows with slot -1 are
 * skipped: their rows of q_out stay as they were.  PW_ERR_STATE before pw_attn_set_rope and pw_attn_bind of the layer. */
pw_status pw_attn_rope_append(pw_attn *a, int layer, const pw_kv_step *step, const void *q, int64_t q_token, int64_t q_head,
                              void *q_out, int64_t qo_token, int64_t qo_head, const void *k, int64_t k_token, int64_t k_head,
                              const void *v, int64_t v_token, int64_t v_head, const int32_t *pos, pw_stream stream);
/* Drafted tokens that form a tree: the tree of request r is its last tree_len[r] keys, nodes 0, 1, ... from the tree's
 * start s = kv_len[r] - tree_len[r], new ones or written by earlier steps.  Node i follows node parent[r][i] < i, or the token
 * before the tree (-1).  Device memory that stays the caller's. */
enum { PW_TREE_NODES = 256 };
typedef struct {
    const int32_t *tree_len; /* [R] at most PW_TREE_NODES, parent_stride and kv_len[r]; 0: no tree, the request's rows see what
                                they see under pw_attn_plan */
    const int32_t *parent;   /* [R][parent_stride] */
    int parent_stride;
    int32_t *pos;            /* out [n_tokens], or NULL: positions of the rows, s + the node's depth (roots: 0) for nodes,
                                else as in step->pos; -1 for padding */
} pw_tree;
/* pw_attn_plan for a step with trees.  The row of a node sees the keys before the tree and, of the tree, the node itself and
 * its ancestors.  Windows and distance biases go by positions: node i stands at s + its depth, as a row and as a key.  A
 * length or a parent out of range is reported by pw_attn_check (PW_ERR_STATE): a tree_len counts as 0 then, a parent as -1.
 * A captured pw_attn_forward is replayed under the rules of pw_attn_plan, and with a plan of the call that it was captured
 * with.  PW_ERR_INVALID also where n_tokens exceeds max_tree_tokens. */
pw_status pw_attn_plan_tree(pw_attn *a, int plan, const pw_kv_step *step, int window, const pw_tree *tree, pw_stream stream);
/* Once drafts are verified: of each request's tree (as above; parents are not read) the nodes keep[r][0] < keep[r][1] < ...
 * < keep[r][n_keep[r] - 1], a path from a root, move to the tree's start: key and value of position s + keep[r][i] go to s + i, in all
 * layers' caches.  ctx_out [R] (NULL: not written): s + n_keep[r], the request's ctx_len in the next step; what lies
 * behind is free to be written again.  keep [R][keep_stride] and n_keep [R] are device memory.  A length, or a node that does not
 * ascend or lies outside the tree, is reported by pw_attn_check (PW_ERR_STATE); that request keeps what came before it.  (So is
 * a block id outside the cache; the tokens that would move there or from there stay, and ctx_out counts them.)  Two
 * requests' trees share no block.  A cache that several layers share is moved once.  PW_ERR_STATE if a layer's cache is not
 * bound, or if two begin at one address with other strides. */
pw_status pw_kv_keep(pw_attn *a, const pw_kv_step *step, const int32_t *tree_len, const int32_t *keep, int keep_stride,
                     const int32_t *n_keep, int32_t *ctx_out, pw_stream stream);
/* Copy the blocks src[i] to dst[i], i < n, in all layers' caches (src and dst: device int32).  With a table (device
 * [table_rows][table_stride], else NULL) its entries src[i] then become dst[i].  The dst are distinct and none of them is a
 * src; with a table the src are distinct, too.  Where they are not, what lies in those blocks and entries afterwards is not
 * specified.  Pairs with an id outside the cache are skipped and reported by pw_attn_check (PW_ERR_STATE).  n = 0 does
 * nothing.  PW_ERR_STATE if a layer's cache is not bound. */
pw_status pw_kv_copy(pw_attn *a, const int32_t *src, const int32_t *dst, int n, int32_t *table, int table_rows, int table_stride,
                     pw_stream stream);
/* Attention of the step's rows over the layer's cache, which holds the new tokens already: the formula
 * above.  q and o as k above, over n_heads heads; query head h reads key/value head h / (n_heads /
 * n_kv_heads).  lse: fp32 [n_tokens][n_heads] or NULL.  scale finite; softcap >= 0 (0: none); slopes: fp32
 * [n_heads] or NULL.  o may not alias q or the caches.  A block id outside the cache reads as zeros.
 * PW_ERR_STATE if the plan or the layer's cache was never set. */
pw_status pw_attn_forward(pw_attn *a, int layer, int plan, const void *q, int64_t q_token, int64_t q_head,
                          void *o, int64_t o_token, int64_t o_head, float *lse, float scale, float softcap,
                          const float *slopes, pw_stream stream);
/* Fault injection for testing (no GPU fault is ever made), as pw_set_fault's kinds: 4 = with n != 0, the next
 * pw_attn_forward withholds one barrier arrival, so that the bounded waits on it expire (its outputs are invalid
 * and pw_attn_check reports PW_ERR_TIMEOUT, after which the handle is usable as before); 5 = bounded device waits
 * give up after about n microseconds (0: the default, about 2 s; behind shared prefixes 0.3 ms later for each key that
 * a row may see).  PW_ERR_INVALID for another kind or n < 0. */
pw_status pw_attn_set_fault(pw_attn *a, int kind, int n);
/* Wait for `stream` and report what the handle's calls found since the last check: PW_ERR_TIMEOUT if a
 * bounded device wait expired, PW_ERR_STATE for the findings of pw_kv_map, pw_attn_plan_tree, pw_kv_keep and pw_kv_copy and
 * for a forward whose plan was laid out anew for another shape (message in pw_last_error(NULL)).
 * Clears what it reports. */
pw_status pw_attn_check(pw_attn *a, pw_stream stream);

/* ---------------------------------------------------------------- inspection */

/* b-bit codes of a block as the GPU kernels read them (the same device extraction code
 * as the forward): host uint8 [N][K].  Sec. 2.2 (Any-Precision LLM's overlaid bit-planes):
 * the b-bit code of an element is its top b bit-planes, plane 0 the most significant.
 * Pages 0..b-1 must be GPU-resident, else PW_ERR_STATE; PW_ERR_INVALID for a bad block or
 * b outside 1..bmax.  Waits for the ctx stream. */
pw_status pw_unpack_indices(pw_ctx *ctx, int block, int b, uint8_t *host_out);

/* Dequantised weights W^(b)[n][k] = LUT_b[n][code] as the GPU kernels produce them:
 * host fp16 bits [N][K].  Sec. 2.2: each output row has its own table of 2^b centroids per
 * supported bitwidth b, indexed by the b-bit code.  Pages 0..b-1 and LUT_b must be
 * GPU-resident, else PW_ERR_STATE; PW_ERR_INVALID for a bad block or unsupported b.
 * Waits for the ctx stream. */
pw_status pw_dequant(pw_ctx *ctx, int block, int b, uint16_t *host_out);

/* Self-check of the 5th-generation tensor-core path (tcgen05) on one CTA: D[128][N] =
 * A[128][K] * B[N][K]^T with fp16 A, B (row-major, device) and fp32 D (row-major, device),
 * 16 <= N <= 256 and 16 <= K <= 128, both multiples of 16.  flags bit 0: A goes through
 * tensor memory (written with tcgen05.st, read by the MMA from there) as the expert kernels'
 * dequantised weights do; otherwise both operands come from shared memory.  Other flag
 * bits are invalid.  *err (device int) is set to 1 if the bounded wait for the MMAs
 * expired.  Asynchronous on `stream`.  No counterpart in the paper: a hardware check. */
pw_status pw_tc_selftest(const uint16_t *A, const uint16_t *B, int N, int K, int flags, float *D, int *err,
                         pw_stream stream);

/* Pure host helpers (no context, no GPU) for checking the packer (Sec. 2.2 bit-planes,
 * Sec. 3.1 one page per plane).
 * pw_pack_planes_host: the plain plane layout -- planes [bmax][N][W] uint32,
 *   W = ceil(K/128)*4 words per row, bit j of word w is column 32w+j, plane 0 = MSB.
 * pw_tile_planes_host / pw_untile_planes_host: the kernel-private device tiling of
 *   those planes for a block of type u (gate_up rows are interleaved per 16-row tile)
 *   and its inverse.  Sizes: bmax * N * W words each. */
pw_status pw_pack_planes_host(const uint8_t *idx, int N, int K, int bmax, uint32_t *planes);
pw_status pw_tile_planes_host(const uint32_t *planes, int N, int K, int nplanes, int u,
                              uint32_t *tiled);
pw_status pw_untile_planes_host(const uint32_t *tiled, int N, int K, int nplanes, int u,
                                uint32_t *planes);

#ifdef __cplusplus
}
#endif
#endif /* PW_H */
