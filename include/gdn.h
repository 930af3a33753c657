/*
 * gdn.h — C ABI of the GB300 (sm_103a) Gated Delta Network chunked-prefill
 * forward pass (and its backward, gdn_chunk_bwd), and of the layer operators
 * around it: layer norm, the short causal convolution, the selective state
 * space scan and the single-token delta step.
 *
 * The operation (FlashQLA talk "Qwen系列模型线性注意力高性能优化实践", the
 * recurrent-form and GDN paragraphs): for every sequence n and head h, with the
 * state S in R^{dv x dk},
 *
 *     S_t = S_{t-1} alpha_t (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,
 *     o_t = scale * S_t q_t,            alpha_t = exp(g_t),
 *
 * computed chunk by chunk (C = 64 tokens) in the WY form (same talk, WY and
 * four-step paragraphs): a gate kernel (chunk-local log-space cumsum, head
 * flags), a per-chunk kernel that inverts I + diag(beta) strictlower(K K^T)
 * without any exponentials (Gamma-extraction paragraph), optional intra-card
 * sequence parallelism (difference, compute-for-memory, auto-CP and
 * sliding-window paragraphs), and one fused kernel that forms U, runs the
 * chunk-to-chunk state recurrence and writes o.
 *
 * Layouts (all row-major, C order):
 *   q, k           [B, T, H, dk]   dtype (bf16 or fp32)
 *   v, o           [B, T, H, dv]   dtype
 *   g, beta        [B, T, H]       fp32 (g = log alpha <= 0, beta in [0, 1])
 *   initial_state,
 *   final_state    [N, H, dk, dv]  fp32; element [n][h][j][i] is S[i][j]
 *                                  (key index j outer, value index i inner)
 *   cu_seqlens     [N + 1]         int32, device memory; with it the batch is
 *                                  packed (B = 1, T = total tokens) and
 *                                  sequence n is tokens cu[n] .. cu[n+1]-1
 *
 * Ownership: the caller allocates every buffer (inputs, outputs, workspace)
 * and keeps them alive until the work on `stream` completes.  The library
 * allocates no device or host memory at run time, keeps no state between calls
 * besides per-device caches of device attributes, driver entry points and the
 * two copy streams of gdn_chunk_fwd_host (and the fixed scratch array of
 * gdn_chunk_fwd_static), and never synchronises the stream inside
 * gdn_chunk_fwd.
 *
 * Errors: every call returns a gdn_status and never aborts.  Argument errors
 * are found on the host before any launch.  Errors found on the device (a
 * malformed cu_seqlens, a bounded wait that ran out) are written to an error
 * word inside the workspace; gdn_chunk_fwd_check() reads it.
 *
 * Preconditions that are not checked: q and k rows are L2-normalised (the
 * sliding-window bound relies on it), g <= 0, 0 <= beta <= 1, all inputs
 * finite, and no two calls share a workspace concurrently.
 */
#ifndef GDN_GB300_H
#define GDN_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* cudaStream_t; NULL is the legacy default stream. */
typedef struct CUstream_st *gdn_stream_t;

typedef enum {
    GDN_OK = 0,
    GDN_ERR_INVALID_ARG = 1,   /* null pointer, bad size, misaligned buffer */
    GDN_ERR_UNSUPPORTED = 2,   /* shape/dtype/device the library does not handle */
    GDN_ERR_WORKSPACE = 3,     /* workspace smaller than gdn_chunk_fwd_workspace_size() */
    GDN_ERR_CUDA = 4,          /* a CUDA runtime/driver call failed */
    GDN_ERR_DEVICE_CHECK = 5,  /* the device found bad input (e.g. cu_seqlens) */
    GDN_ERR_TIMEOUT = 6        /* a bounded device-side wait ran out */
} gdn_status;

typedef enum { GDN_BF16 = 0, GDN_F32 = 1 } gdn_dtype;

/* Intra-card sequence parallelism (auto-CP paragraph): AUTO lets the planner
 * decide; OFF runs every (sequence, head) as one unit and is bitwise
 * deterministic; FORCE always splits sequences into segments. */
typedef enum { GDN_CP_AUTO = 0, GDN_CP_OFF = 1, GDN_CP_FORCE = 2 } gdn_cp_mode;

/* Which fused kernel runs: AUTO (and TC) pick the tcgen05 kernels for every
 * supported shape — kind::f16 for bf16 inputs, kind::tf32 for fp32 inputs
 * (fp32 operands read as tf32, fp32 accumulation), dk, dv in {32, 64, 128},
 * head sizes below 128 zero-padded to 128 inside the kernels, which is exact;
 * SIMT selects the CUDA-core kernel (fp32 arithmetic throughout; with fp32
 * inputs also the CUDA-core per-chunk inverse). */
typedef enum { GDN_KERNEL_AUTO = 0, GDN_KERNEL_TC = 1, GDN_KERNEL_SIMT = 2 } gdn_kernel;

typedef struct {
    int32_t cp_mode;            /* gdn_cp_mode */
    int32_t kernel;             /* gdn_kernel */
    int32_t chunks_per_segment; /* > 0 forces the segment length L (chunks) when CP is on */
    int32_t sliding;            /* 1 (default): heads with alpha != 1 restart from a
                                   look-back window; 0: every split head uses
                                   correction matrices */
    float sw_eps;               /* look-back tolerance: the window is long enough that
                                   prod(alpha) over it <= sw_eps (default 2^-24) */
    int32_t sm_count;           /* 0: query the device; > 0: plan for this many SMs */
    int32_t stages;             /* 0: the whole path; else a GDN_STAGE_* mask (stages not
                                   selected are skipped and their workspace outputs must
                                   already be there from an earlier call on the same
                                   problem and workspace) */
    int32_t debug_checks;       /* 0, or GDN_DEBUG_* bits (tests of the error paths) */
    void *prof_begin;           /* optional cudaEvent_t, recorded on `stream` right before
                                   the fused output pass is launched */
    void *prof_end;             /* optional cudaEvent_t, recorded right after it */
    int32_t qk_l2norm;          /* 1: the library scales every q and k row to unit L2 norm
                                   (gdn_qk_l2norm with eps 1e-6) into workspace copies
                                   before the pass; 0 (default): the caller's rows are
                                   used as they are (they should be unit-norm already) */
    int32_t inverse_overlap;    /* the tcgen05 path on equal sequences without a split, when
                                   the (sequence, head) units leave SMs idle: k > 0 lets the
                                   fused pass run the per-chunk inverse of the last k chunk
                                   columns (at most all) on those SMs while the other CTAs
                                   run the state recurrence (one cooperative launch; each
                                   such column is loaded only once all its units are in
                                   memory; the results are bitwise those of the separate
                                   inverse).  0 (default) and -1: off.  On a GB300 at
                                   B=4, T=8192, H=32 it moved the step by -6..+3 us (the
                                   24 idle SMs' inverse traffic slows the chain about as
                                   much as it hides), so it is not on by default */
    int32_t reserved[2];
} gdn_options;

/* GDN_DEBUG_TIMEOUT_PROBE: the tile producer of the tcgen05 fused pass signals
 * nothing, so every bounded wait of that pass runs out (about 2 s): the pass
 * records GDN_ERR_TIMEOUT, frees what it holds and returns, and the next call
 * on the same workspace runs normally.  It exists to test the timeout path
 * without faulting or hanging the GPU; the kind::tf32 and CUDA-core passes
 * ignore it. */
enum { GDN_DEBUG_TIMEOUT_PROBE = 1 };

enum {
    GDN_STAGE_PREP = 1,         /* sequence tables, gate kernel, device planner */
    GDN_STAGE_INVERSE = 2,      /* per-chunk inverse T' */
    GDN_STAGE_CORRECTION = 4,   /* correction pass and segment scan (when CP is on) */
    GDN_STAGE_FUSED = 8         /* fused output pass */
};

/* What the host planner decided for a problem (host-only, no GPU needed). */
typedef struct {
    int32_t kernel;             /* gdn_kernel actually used (TC or SIMT) */
    int32_t cp_enabled;         /* 1 when sequences may be split into segments */
    int32_t chunks_per_segment; /* segment length L in chunks */
    int32_t max_chunks;         /* upper bound on chunks over all sequences */
    int32_t max_items;          /* capacity of the fused-kernel work list */
    int32_t max_cp_slots;       /* capacity of the correction-matrix buffers */
    int32_t sm_count;           /* SMs the plan was made for */
    int32_t grid_fused;         /* CTAs of the persistent fused kernel */
    int32_t overlap_columns;    /* chunk columns whose inverse runs inside the fused pass
                                   (see gdn_options.inverse_overlap); 0: none */
    int32_t launches;           /* kernels one gdn_chunk_fwd call launches (the whole path:
                                   q/k normalisation, sequence prep, gate, planner, inverse,
                                   correction pass and scan, fused pass, as the plan needs) */
    size_t workspace_bytes;     /* bytes gdn_chunk_fwd needs */
} gdn_plan_info;

/* Byte offsets of the intermediate tensors inside the workspace, so tests and
 * tools can inspect them after a call (read them only after the stream syncs). */
typedef struct {
    size_t error_word;     /* int32: 0 or a gdn_status found on the device */
    size_t gate_cumsum;    /* fp32 [H, total_T]: chunk-local inclusive cumsum of g */
    size_t chunk_totals;   /* fp32 [H, max_chunks]: sum of g per chunk (chunks in sequence order) */
    size_t head_flags;     /* int32 [N, H]: 1 when some g != 0 (alpha not identically 1) */
    size_t tprime;         /* [H, total_T, 64] T' rows by token; bf16 for bf16 inputs, fp32 for fp32.
                              When the tcgen05 fused kernel runs (bf16) this holds
                              T' diag(c1) instead, c1_m = exp(G* - G_m) beta_m with G* the middle of
                              the chunk's gate cumsum range, or (Gamma ⊙ T') diag(beta) for a chunk
                              whose last cumsum is below -80 */
    size_t chunk_table;    /* int32x4 [max_chunks]: (seq, first token, length, chunk index in seq) */
    size_t num_chunks;     /* int32: chunks actually present */
    size_t items;          /* int32x8 [max_items]: fused-kernel work items (see gdn_work_item) */
    size_t num_items;      /* int32: [0] pass-2 items, [1] pass-1 items, [2] scan units */
    size_t total;
} gdn_workspace_layout;

/* One unit of fused-kernel work as the planner writes it. */
typedef struct {
    int32_t seq, head;
    int32_t c_begin, c_end;   /* chunks [c_begin, c_end) of the sequence produce output */
    int32_t c_start;          /* first chunk run (c_start <= c_begin); chunks before
                                 c_begin only advance the state (look-back) */
    int32_t flags;            /* GDN_ITEM_* bits */
    int32_t slot;             /* correction-buffer slot (CP) or -1 */
    int32_t pad;
} gdn_work_item;

enum {
    GDN_ITEM_OUTPUT = 1,        /* write o for chunks [c_begin, c_end) */
    GDN_ITEM_FROM_INITIAL = 2,  /* start from initial_state (or zero when it is NULL) */
    GDN_ITEM_FROM_ZERO = 4,     /* start from S = 0 */
    GDN_ITEM_FROM_IDENTITY = 8, /* start from S = I and use zero values (correction matrix) */
    GDN_ITEM_FROM_SLOT = 16,    /* start from the scanned segment start in `slot` */
    GDN_ITEM_WRITE_FINAL = 32,  /* write final_state */
    GDN_ITEM_WRITE_SLOT = 64,   /* write the end state to the S* buffer `slot` */
    GDN_ITEM_WRITE_M = 128      /* write the end state to the M buffer `slot` */
};

/* Fill *opts with the defaults (AUTO everywhere, sliding on, sw_eps 2^-24). */
void gdn_default_options(gdn_options *opts);

/*
 * Cost model of the auto-CP planner.  The intra-card sequence-parallel
 * paragraph of the FlashQLA talk "Qwen系列模型线性注意力高性能优化实践" models the
 * time of a split sequence as T = lambda1 L + lambda2 N / L (L chunks per
 * segment, N / L segments) with lambda measured on the hardware; the planner
 * here is the wave-aware form of that model and takes its lambdas from this
 * table, in microseconds on the target GPU with every SM busy:
 *   chunk_step_us  one chunk step of the fused output pass (lambda1, pass 2)
 *   state_step_us  one chunk step of a state-only correction item (lambda1, pass 1)
 *   scan_step_us   one segment step of the segment scan (lambda2)
 *   pass_us        the fixed cost of the correction pass and the scan launches
 * The library starts with values measured on a GB300; gdn_set_plan_costs()
 * replaces them for the whole process (NULL restores those defaults; a
 * non-finite, negative or zero step cost is GDN_ERR_INVALID_ARG) and
 * gdn_get_plan_costs() reads the current table.  The Python package's
 * `calibrate` module measures the table on the GPU at hand by timing this
 * library's own passes.  Plans made before a change keep the costs they were
 * made with; nothing else depends on the table (every plan is exact).
 */
typedef struct {
    float chunk_step_us;
    float state_step_us;
    float scan_step_us;
    float pass_us;
} gdn_plan_costs;

gdn_status gdn_set_plan_costs(const gdn_plan_costs *costs);
void gdn_get_plan_costs(gdn_plan_costs *costs);

/*
 * The enabling boundary of auto CP for batches of equal sequences: the least
 * sequence length, in chunks of 64 tokens, at which GDN_CP_AUTO splits
 * sequences when there are `units` = B x H (sequence, head) units on `sms`
 * SMs, under the current cost table; 0 when no length up to 2^20 chunks does
 * (always for units >= sms).  The talk's enabling-condition paragraph notes
 * that the boundary in the (B x H, length) plane is a curve rather than a
 * threshold on either axis: more units leave fewer idle SMs, so a longer
 * sequence is needed before splitting pays.  Host-only.
 */
int gdn_auto_cp_min_chunks(int units, int sms);

/* Host-only planning: which kernel, whether CP is on, the segment length and
 * the workspace size.  `total_T` is B*T for batched input or the packed token
 * count with cu_seqlens (then B must be 1 and n_seqs = N).  opts may be NULL. */
gdn_status gdn_plan_query(int B, int T, int H, int dk, int dv, int n_seqs, int varlen,
                          gdn_dtype dtype, const gdn_options *opts, gdn_plan_info *out);

/* Bytes of device workspace gdn_chunk_fwd needs for this problem (0 on bad
 * arguments).  `varlen` is 1 when cu_seqlens will be passed. */
size_t gdn_chunk_fwd_workspace_size(int B, int T, int H, int dk, int dv, int n_seqs, int varlen,
                                    gdn_dtype dtype, const gdn_options *opts);

/* Offsets of the intermediates inside the workspace for this problem. */
gdn_status gdn_workspace_query(int B, int T, int H, int dk, int dv, int n_seqs, int varlen,
                               gdn_dtype dtype, const gdn_options *opts, gdn_workspace_layout *out);

/*
 * The forward pass.  All pointers are device pointers (initial_state and
 * cu_seqlens may be NULL).  With cu_seqlens == NULL the batch is B sequences of
 * T tokens (n_seqs is ignored); otherwise B must be 1, T is the total token
 * count and n_seqs = N.  scale <= 0 selects dk^-0.5.  dk, dv in {32, 64, 128}.
 * q, k, v, o, g, beta, states and workspace must be 16-byte aligned.
 * The workspace must hold gdn_chunk_fwd_workspace_size() bytes; it needs no
 * initialisation.  Everything is enqueued on `stream`; nothing syncs.
 */
gdn_status gdn_chunk_fwd(const void *q, const void *k, const void *v,
                         const float *g, const float *beta,
                         const float *initial_state,
                         const int32_t *cu_seqlens, int n_seqs,
                         float scale,
                         int B, int T, int H, int dk, int dv, gdn_dtype dtype,
                         void *o, float *final_state,
                         void *workspace, size_t workspace_bytes,
                         const gdn_options *opts, gdn_stream_t stream);

/* Synchronises `stream`, then reads the device error word of `workspace`:
 * GDN_OK, GDN_ERR_DEVICE_CHECK (bad cu_seqlens) or GDN_ERR_TIMEOUT. */
gdn_status gdn_chunk_fwd_check(const void *workspace, gdn_stream_t stream);

/* Device bytes gdn_chunk_fwd_host needs as its staging buffer (inputs, outputs
 * and workspace together). */
size_t gdn_chunk_fwd_host_buffer_size(int B, int T, int H, int dk, int dv, int n_seqs, int varlen,
                                      int has_initial_state, gdn_dtype dtype, const gdn_options *opts);

/*
 * The same forward pass for inputs and outputs in HOST memory (pinned memory
 * makes the copies asynchronous).  The call copies the inputs into
 * `device_buffer` (gdn_chunk_fwd_host_buffer_size() bytes, caller-owned), runs
 * gdn_chunk_fwd on `stream`, copies o and final_state back, waits for all of
 * it and returns the device error status as gdn_chunk_fwd_check does.
 * cu_seqlens is a host array here.
 *
 * Above 64 MB of input the problem goes through in up to eight parts: groups
 * of whole sequences with about equal token counts or, when there are fewer
 * sequences than parts and the plan runs every (sequence, head) as one unit,
 * 64-token-aligned pieces of each sequence, each starting from the state the
 * previous piece left in the device buffer.  Part p+1 is copied in on a
 * library copy stream while the pass runs part p on `stream` and part p-1 is
 * copied out on a second library copy stream (both created once per device,
 * non-blocking; they first wait for the work already on `stream`).  Every part
 * keeps the whole problem's plan (CP on or off, the segment length), so the
 * result is the one gdn_chunk_fwd gives on the whole problem, bit for bit.
 */
gdn_status gdn_chunk_fwd_host(const void *q, const void *k, const void *v,
                              const float *g, const float *beta,
                              const float *initial_state,
                              const int32_t *cu_seqlens, int n_seqs,
                              float scale,
                              int B, int T, int H, int dk, int dv, gdn_dtype dtype,
                              void *o, float *final_state,
                              void *device_buffer, size_t device_buffer_bytes,
                              const gdn_options *opts, gdn_stream_t stream);

/*
 * Inter-card sequence parallelism (the talk's difference and compute-for-memory
 * paragraphs, and its timeline paragraph's "inter-card sequence parallelism":
 * the three steps of intra-card CP with the segments on different GPUs).  A
 * batch of sequences is split along time into R slices, one per rank; every
 * rank holds the same (sequence, head) units.  Step one, on every rank:
 *
 *   gdn_chunk_transition: for each (sequence, head) of the local slice, the
 *   affine map the slice applies to the state, S_end = S_start M + S*:
 *   S* is the slice's end state from S_start = 0 with the slice's values, and
 *   M (dk x dk) the end state from S_start = I with zero values, i.e. the
 *   product of the slice's token transitions alpha_t (I - beta_t k_t k_t^T).
 *
 * q is not read (the map does not depend on the queries).  k, v, g, beta,
 * cu_seqlens, B, T, H, dk, dv, dtype as for gdn_chunk_fwd.  Outputs (device,
 * fp32, 16-byte aligned): s_star [N, H, dk, dv] in the state layout of
 * final_state, m [N, H, dk, dk] in the same transposed layout
 * (m[n][h][b][a] = M[a][b]).  An empty sequence maps to S* = 0, M = I.  The
 * workspace holds gdn_chunk_transition_workspace_size() bytes.  Nothing syncs;
 * device-side errors (bad cu_seqlens, timeout) land in the workspace's error
 * word: read them with gdn_chunk_fwd_check(workspace, stream).
 *
 * Step two is an all-gather of (S*, M) over the ranks (the caller's
 * collective), step three gdn_state_scan below, step four gdn_chunk_fwd on the
 * local slice from the rank's start state.
 */
size_t gdn_chunk_transition_workspace_size(int B, int T, int H, int dk, int dv, int n_seqs, int varlen,
                                           gdn_dtype dtype);
gdn_status gdn_chunk_transition(const void *k, const void *v, const float *g, const float *beta,
                                const int32_t *cu_seqlens, int n_seqs,
                                int B, int T, int H, int dk, int dv, gdn_dtype dtype,
                                float *s_star, float *m,
                                void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/*
 * Start states of R consecutive slices of the same sequences from their maps:
 * s_start[0] = s0 (NULL: zero) and s_start[r + 1] = s_start[r] M_r + S*_r.
 * s_star [R, N, H, dk, dv], m [R, N, H, dk, dk] as gdn_chunk_transition writes
 * them (rank-major, e.g. the result of an all-gather), s0 [N, H, dk, dv] or
 * NULL, s_start [R, N, H, dk, dv]; device fp32, 16-byte aligned; s_start must
 * not overlap the inputs.  The last map (r = R - 1) is not used.  fp32
 * arithmetic, one CUDA kernel, nothing syncs.
 */
gdn_status gdn_state_scan(const float *s0, const float *s_star, const float *m, int R, int N, int H, int dk,
                          int dv, float *s_start, gdn_stream_t stream);

/*
 * The same walk for the gradient of the state, from the last slice down
 * (sequence parallelism in the backward pass: the results paragraph of the
 * talk has the backward split with the same sliding-window / correction
 * scheme).  With S_end = S_start M + S* per slice, the gradient of the loss
 * with respect to a slice's start state is that of its end state times M^T
 * plus the slice's own term ds_star (its backward run with a zero end
 * gradient), so
 *
 *   ds_end[R - 1] = ds_last (NULL: zero),
 *   ds_end[r] = ds_end[r + 1] M_{r+1}^T + ds_star[r + 1].
 *
 * Layouts, alignment and errors as gdn_state_scan (ds_star in the state
 * layout, m as gdn_chunk_transition writes it); ds_star[0] and m[0] are not
 * used.
 */
gdn_status gdn_state_grad_scan(const float *ds_last, const float *ds_star, const float *m, int R, int N, int H,
                               int dk, int dv, float *ds_end, gdn_stream_t stream);

/*
 * The same forward pass for callers that cannot allocate device memory while
 * they run: a server that hands all of HBM to its own pool at start-up and
 * forbids allocation on the request path, or a plugin that receives tensors
 * from a host framework and has no allocator.  The paper has no counterpart;
 * this is an addition of this library.
 *
 * Arguments are those of gdn_chunk_fwd without the workspace: the scratch is a
 * static device array of 64 MiB inside the library, which every GPU that loads
 * the library holds until the process exits.  A problem whose
 * gdn_chunk_fwd_workspace_size() exceeds 64 MiB is rejected with
 * GDN_ERR_WORKSPACE before anything is enqueued (gdn_last_error_detail() then
 * says how many bytes it needed).  opts->stages must be 0 (the whole pass).
 *
 * The first call on a device looks up the array's device address and caches
 * it (cudaGetSymbolAddress, no allocation); make that first call before any
 * stream capture.  With lazy module loading (the CUDA default) that first
 * call is also when the runtime loads the library's device code and reserves
 * the 64 MiB array on the device, so a caller whose pool takes the rest of
 * HBM at start-up must make one call (any size, e.g. an empty batch) before
 * the pool reserves its memory.  The cached address belongs to the device's
 * current primary context: after cudaDeviceReset() in the same process this
 * entry point must not be called again.  Apart from that first load the call
 * allocates nothing, host or device.
 *
 * Every call on a device shares the one array, which keeps the previous call's
 * contents; the call clears what must start at zero (the error word and the
 * work counters) on `stream` itself.  Calls whose GPU work overlaps (other
 * streams, other host threads) race on the array and give wrong results: order
 * them, e.g. on one stream.
 *
 * device_status: NULL makes the call synchronise `stream` and return the
 * device-side status as gdn_chunk_fwd_check() does.  Otherwise it is a 4-byte
 * aligned device int32 into which the call enqueues a copy of the device
 * status word (0, or a gdn_status) after the pass, and the call returns
 * without synchronising.
 */
gdn_status gdn_chunk_fwd_static(const void *q, const void *k, const void *v,
                                const float *g, const float *beta,
                                const float *initial_state,
                                const int32_t *cu_seqlens, int n_seqs,
                                float scale,
                                int B, int T, int H, int dk, int dv, gdn_dtype dtype,
                                void *o, float *final_state,
                                int32_t *device_status,
                                const gdn_options *opts, gdn_stream_t stream);

/*
 * L2 normalisation of q and k rows over the head dimension, the step in front
 * of the recurrence (the sliding-window paragraph of the FlashQLA talk
 * "Qwen系列模型线性注意力高性能优化实践" takes every key to have unit L2 norm):
 *
 *     x_hat[d] = x[d] / sqrt(sum_d' x[d']^2 + eps)
 *
 * with the sum in fp32 and one rounding to the output type.  q, k: device
 * pointers to `rows` rows of dk contiguous elements (dk in {32, 64, 128};
 * rows = tokens x heads for a [.., H, dk] tensor); either may be NULL, and
 * then its output pointer must be NULL too.  q_out / k_out receive the
 * normalised rows in the same layout and dtype; they may equal q / k (in
 * place).  All pointers 16-byte aligned.  eps <= 0 selects 1e-6.  Enqueued on
 * `stream`; nothing syncs.  gdn_chunk_fwd runs this pass itself, into copies
 * in its workspace, when opts->qk_l2norm is 1.
 * Errors: GDN_ERR_INVALID_ARG (sizes, dtype, alignment, a NULL pairing),
 * GDN_ERR_CUDA (launch failure; see gdn_last_error_detail()).
 */
gdn_status gdn_qk_l2norm(const void *q, const void *k, void *q_out, void *k_out,
                         int64_t rows, int dk, gdn_dtype dtype, float eps,
                         gdn_stream_t stream);

/*
 * Backward of gdn_qk_l2norm for one tensor: with n = sqrt(sum_d x_d^2 + eps)
 * and dy the gradient of x_hat = x / n,
 *
 *     dx = dy / n - x (x . dy) / n^3        (the Jacobian of x / n)
 *
 * in fp32.  x: `rows` rows of dk elements in `dtype` (the tensor that was
 * normalised); dy, dx: fp32 rows in the same layout (dx may equal dy).  All
 * pointers 16-byte aligned, non-NULL when rows > 0; dk in {32, 64, 128};
 * eps <= 0 selects 1e-6 (the forward's default).  Enqueued on `stream`.
 * Errors: GDN_ERR_INVALID_ARG (sizes, dtype, alignment, NULL), GDN_ERR_CUDA.
 */
gdn_status gdn_qk_l2norm_bwd(const void *x, const float *dy, float *dx, int64_t rows, int dk,
                             gdn_dtype dtype, float eps, gdn_stream_t stream);

/*
 * The backward pass: gradients of L = sum <o, d_o> + <final_state,
 * d_final_state> with respect to q, k, v, g, beta and initial_state, for the
 * forward pass gdn_chunk_fwd computes (the backward paragraph of the FlashQLA
 * talk "Qwen系列模型线性注意力高性能优化实践": chunk by chunk in the WY form,
 * the dA and dA^T terms merged).  The library recomputes the chunk start
 * states itself (a forward sweep), so the forward's outputs are not inputs.
 *
 * Inputs as gdn_chunk_fwd (q, k, v in `dtype`; g, beta, initial_state fp32;
 * initial_state and cu_seqlens may be NULL), plus
 *   d_o             [B, T, H, dv]   dtype, the gradient of o
 *   d_final_state   [N, H, dk, dv]  fp32 or NULL (zero)
 * Outputs, all fp32 and written in full (no accumulation into them):
 *   dq, dk          [B, T, H, dk]
 *   dv              [B, T, H, dv]
 *   dg, dbeta       [B, T, H]
 *   d_initial_state [N, H, dk, dv]  (may be NULL: not written)
 * All pointers are device pointers, 16-byte aligned.  The workspace must hold
 * gdn_chunk_bwd_workspace_size() bytes (no initialisation needed; it keeps the
 * chunk start states and the per-chunk intermediates).  Enqueued on `stream`;
 * nothing syncs.  The result does not depend on the launch order of CTAs.
 *
 * Kernels (gdn_set_backward_kernel): by default the tensor-core backward, two
 * tcgen05 kernels with fp32 operands read as tf32 and fp32 accumulation — a
 * chain kernel per (sequence, head) for the state and state-gradient
 * recurrences, dv and d_initial_state, then one CTA per (chunk, head) for dq,
 * dk, dg and dbeta; GDN_KERNEL_SIMT selects the CUDA-core kernel (fp32
 * products, one CTA per 32 value columns, head and sequence).
 * Errors: GDN_ERR_INVALID_ARG / GDN_ERR_UNSUPPORTED / GDN_ERR_WORKSPACE before
 * any launch; GDN_ERR_CUDA on a launch failure; a malformed cu_seqlens is
 * written to the workspace's error word, which gdn_chunk_bwd_check() reads.
 * Preconditions as gdn_chunk_fwd's; n_seqs (or B) at most 65535.
 */
size_t gdn_chunk_bwd_workspace_size(int B, int T, int H, int dk, int dv, int n_seqs, int varlen,
                                    gdn_dtype dtype);

gdn_status gdn_chunk_bwd(const void *q, const void *k, const void *v,
                         const float *g, const float *beta,
                         const float *initial_state,
                         const int32_t *cu_seqlens, int n_seqs,
                         float scale,
                         int B, int T, int H, int dk, int dv, gdn_dtype dtype,
                         const void *d_o, const float *d_final_state,
                         float *dq, float *dk_out, float *dv_out, float *dg, float *dbeta,
                         float *d_initial_state,
                         void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/*
 * The gradient of the initial state alone: d_initial_state of the backward
 * pass above, from d_o and d_final_state (the state-gradient recurrence run
 * from the last chunk back to the first; it needs neither v nor the initial
 * state, and writes nothing else).  The same tensor-core chain kernel as
 * gdn_chunk_bwd's default, so the result equals its d_initial_state bit for
 * bit.  The sequence-parallel backward takes each segment's local map from it.
 * Arguments, workspace (gdn_chunk_bwd_workspace_size) and errors as
 * gdn_chunk_bwd's; d_initial_state [N, H, dk, dv] fp32 must not be NULL.
 */
gdn_status gdn_chunk_state_grad(const void *q, const void *k, const float *g, const float *beta,
                                const int32_t *cu_seqlens, int n_seqs, float scale,
                                int B, int T, int H, int dk, int dv, gdn_dtype dtype,
                                const void *d_o, const float *d_final_state, float *d_initial_state,
                                void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/* Selects the kernels of later gdn_chunk_bwd calls in this process:
 * GDN_KERNEL_AUTO or GDN_KERNEL_TC (the tensor-core backward, the default) or
 * GDN_KERNEL_SIMT (the CUDA-core backward).  Both fit the same workspace size.
 * GDN_ERR_INVALID_ARG for another value. */
gdn_status gdn_set_backward_kernel(gdn_kernel kernel);
gdn_kernel gdn_get_backward_kernel(void);

/* Synchronises `stream` and reads the error word of a gdn_chunk_bwd
 * workspace: GDN_OK, GDN_ERR_DEVICE_CHECK (bad cu_seqlens) or GDN_ERR_TIMEOUT. */
gdn_status gdn_chunk_bwd_check(const void *workspace, gdn_stream_t stream);

/*
 * Layer operators: what a linear-attention layer computes around the
 * recurrence.  All of them run on `stream` without synchronising, keep nothing
 * between calls, and take buffers that the caller owns; data pointers need the
 * alignment of their element type only (16-byte aligned rows take the faster
 * path).  Activations are bf16 or fp32 (`dtype`), arithmetic and sums are
 * fp32, results are rounded once.  Strides count elements; the last axis is
 * contiguous.
 *
 * Operators on packed batches (cu_seqlens, int32 [n_seqs + 1] in device
 * memory, B = 1) take `device_status`: NULL, or a device int32 into which the
 * call writes 0, or GDN_ERR_DEVICE_CHECK for entries that do not start at 0,
 * decrease, or do not end at T.  The outputs are then unspecified; no access
 * leaves the given buffers.  Sequences may be empty.
 *
 * Single-token forms update a cached state in place.  With state_indices
 * (int32 [N] in device memory) row r uses state state_indices[r] of the
 * n_states there are; a row whose index is outside [0, n_states) is padding:
 * its output is zero and no state changes.  Without it row r uses state r.
 * Two rows of one call must not name the same state.
 *
 * Outputs and states overlap neither inputs nor one another: other threads may
 * still have to read what one writes (the convolution's neighbouring tokens, the
 * delta step's v).  The one exception is y at the address of a contiguous x in
 * gdn_layer_norm_fwd, gdn_causal_conv_step, gdn_selective_scan_fwd and
 * gdn_selective_scan_step (there also of dt or z): what writes an element is all
 * that reads it.
 */

/*
 * Layer norm over rows of D elements:
 *
 *     y = (x - mean) rstd w + b,  rstd = (var + eps)^-1/2,
 *
 * var the mean squared deviation.  x: `rows` rows, x_stride elements apart;
 * y: [rows, D]; weight, bias: [D] in w_dtype, either may be NULL (one, zero);
 * mean, rstd: fp32 [rows] outputs, either may be NULL.  eps >= 0, D at most 2^30.
 */
gdn_status gdn_layer_norm_fwd(const void *x, int64_t x_stride, const void *weight, const void *bias,
                              gdn_dtype w_dtype, float eps, int64_t rows, int D, gdn_dtype dtype, void *y,
                              float *mean, float *rstd, gdn_stream_t stream);

/*
 * Its backward pass from the forward's mean and rstd: with xh = (x - mean) rstd
 * and g = dy w,
 *
 *     dx = rstd (g - mean_d(g) - xh mean_d(g xh)),  dw = sum dy xh,  db = sum dy.
 *
 * dx [rows, D] in dtype; dweight, dbias fp32 [D], either may be NULL.  The
 * workspace (16-byte aligned, gdn_layer_norm_bwd_workspace_size() bytes, no
 * initialisation) is needed for dweight or dbias only.  The sums are added in
 * a fixed order: the same inputs give the same bits.
 */
size_t gdn_layer_norm_bwd_workspace_size(int64_t rows, int D);
gdn_status gdn_layer_norm_bwd(const void *dy, int64_t dy_stride, const void *x, int64_t x_stride, const float *mean,
                              const float *rstd, const void *weight, gdn_dtype w_dtype, int64_t rows, int D,
                              gdn_dtype dtype, void *dx, float *dweight, float *dbias, void *workspace,
                              size_t workspace_bytes, gdn_stream_t stream);

/*
 * Short causal depthwise convolution along each sequence,
 *
 *     u_t = bias + sum_{i < W} w_i x_{t - (W-1) + i},  y = silu ? u sigmoid(u) : u,
 *
 * W in {2, 3, 4}, T and D at most 2^30.  x: [B, T, D] with the given batch and
 * token strides;
 * weight: [D, W], bias: [D] or NULL, in w_dtype (fp32 or dtype); y: [B, T, D].
 * The inputs before a sequence's first token are the rows of initial_state
 * [n, W - 1, D] (dtype, oldest first; NULL: zero), n = B or n_seqs;
 * final_state (same layout, or NULL) receives the last W - 1 inputs, the
 * initial state's own rows among them where a sequence is shorter.
 */
gdn_status gdn_causal_conv_fwd(const void *x, int64_t x_batch_stride, int64_t x_token_stride, const void *weight,
                               const void *bias, gdn_dtype w_dtype, const void *initial_state,
                               const int32_t *cu_seqlens, int n_seqs, int B, int T, int D, int W, int silu,
                               gdn_dtype dtype, void *y, void *final_state, int32_t *device_status,
                               gdn_stream_t stream);

/*
 * Its backward pass: dx [B, T, D] (dtype), dweight [D, W] and dbias [D] (fp32,
 * either may be NULL), d_initial_state [n, W - 1, D] (dtype, may be NULL) from
 * dy and, where given, d_final_state (like final_state).  The workspace
 * (16-byte aligned, gdn_causal_conv_bwd_workspace_size() bytes) is needed for
 * dweight or dbias only.  The same inputs give the same bits.
 */
size_t gdn_causal_conv_bwd_workspace_size(int B, int T, int D, int W);
gdn_status gdn_causal_conv_bwd(const void *dy, int64_t dy_batch_stride, int64_t dy_token_stride, const void *x,
                               int64_t x_batch_stride, int64_t x_token_stride, const void *weight, const void *bias,
                               gdn_dtype w_dtype, const void *initial_state, const void *d_final_state,
                               const int32_t *cu_seqlens, int n_seqs, int B, int T, int D, int W, int silu,
                               gdn_dtype dtype, void *dx, float *dweight, float *dbias, void *d_initial_state,
                               int32_t *device_status, void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/*
 * One token of N sequences: x [N, D] (rows x_stride apart), y [N, D], state
 * [n_states, W - 1, D] updated in place (the oldest row leaves, x enters).
 * N at most 65535.
 */
gdn_status gdn_causal_conv_step(const void *x, int64_t x_stride, void *state, const int32_t *state_indices,
                                int n_states, const void *weight, const void *bias, gdn_dtype w_dtype, int N, int D,
                                int W, int silu, gdn_dtype dtype, void *y, gdn_stream_t stream);

/*
 * Selective state space scan with a diagonal transition: per channel d < D and
 * state index n < N of a sequence,
 *
 *     h_t[d][n] = exp(s_t[d] A[d][n]) h_{t-1}[d][n] + s_t[d] x_t[d] B_t[n],
 *     y_t[d] = (sum_n C_t[n] h_t[d][n] + D_skip[d] x_t[d]) silu(z_t[d]),
 *     s_t[d] = f(dt_t[d] + dt_bias[d]),  f softplus or the identity.
 *
 * x, dt, z: [B, T, D], B_, C_: [B, T, N] in dtype, shared by all channels,
 * each with its own batch and token strides; A fp32 [D, N], D_skip and dt_bias
 * fp32 [D]; initial_state fp32 [n, D, N], n = B or n_seqs.  z (no gate),
 * D_skip and dt_bias (zero), initial_state (zero) and cu_seqlens may be NULL.
 * N at most 64, B at most 65535, T at most 2^30, D at most 2^26.  s A <= 0 is
 * expected: a row is cut into segments, and where the product of exp(s A) over one
 * exceeds fp32's range, states and outputs are not the formula's (an infinity times
 * a zero state is not zero).  A step or x that is not finite makes its channel's
 * outputs non-finite from that token to the end of its sequence, and no other
 * channel's.
 */
typedef struct {
    const void *x, *dt, *z, *B_, *C_;
    const float *A, *D_skip, *dt_bias, *initial_state;
    const int32_t *cu_seqlens;
    int64_t x_batch_stride, x_token_stride, dt_batch_stride, dt_token_stride, z_batch_stride, z_token_stride;
    int64_t b_batch_stride, b_token_stride, c_batch_stride, c_token_stride;
    int32_t B, T, D, N, n_seqs, dt_softplus, dtype, reserved;
} gdn_scan_desc;

/* y [B, T, D] in dtype; final_state fp32 [n, D, N] or NULL.  The workspace is
 * 16-byte aligned and holds gdn_selective_scan_fwd_workspace_size() bytes. */
size_t gdn_selective_scan_fwd_workspace_size(int B, int T, int D, int N);
gdn_status gdn_selective_scan_fwd(const gdn_scan_desc *desc, void *y, float *final_state, int32_t *device_status,
                                  void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/*
 * Its backward pass, from dy [B, T, D] (dtype, with its strides) and
 * d_final_state (fp32 [n, D, N], or NULL): dx, ddt, dz [B, T, D] and dB, dC
 * [B, T, N] in dtype, contiguous (dz NULL without a gate); dA fp32 [D, N];
 * dD_skip, ddt_bias fp32 [D] and d_initial_state fp32 [n, D, N], each may be
 * NULL.  ddt is the gradient of dt before bias and softplus.  The states are
 * recomputed.  Workspace as above.  The same inputs give the same bits.
 */
size_t gdn_selective_scan_bwd_workspace_size(int B, int T, int D, int N);
gdn_status gdn_selective_scan_bwd(const gdn_scan_desc *desc, const void *dy, int64_t dy_batch_stride,
                                  int64_t dy_token_stride, const float *d_final_state, void *dx, void *ddt, float *dA,
                                  void *dB, void *dC, float *dD_skip, void *dz, float *ddt_bias,
                                  float *d_initial_state, int32_t *device_status, void *workspace,
                                  size_t workspace_bytes, gdn_stream_t stream);

/* One token of B sequences (desc->T = 1, initial_state and cu_seqlens unused):
 * y [B, D]; state fp32 [n_states, D, N] updated in place. */
gdn_status gdn_selective_scan_step(const gdn_scan_desc *desc, float *state, const int32_t *state_indices,
                                   int n_states, void *y, gdn_stream_t stream);

/*
 * One token of the gated delta rule (gdn_chunk_fwd's recurrence) for N
 * sequences: q, k [N, H, dk], v [N, H, dv] in dtype, the tokens' rows of H heads
 * q_stride (k_stride, v_stride) elements apart, so that slices of one projection
 * can be used as they lie; o [N, H, dv] in dtype, g, beta fp32 [N, H]; state fp32
 * [n_states, H, dk, dv] in the layout of final_state, 16-byte aligned, updated in
 * place.  dk, dv in {32, 64, 128}; scale <= 0 selects dk^-0.5; qk_l2norm = 1
 * scales the rows of q and k to unit L2 norm first (eps 1e-6).
 */
gdn_status gdn_delta_step(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                          int64_t v_stride, const float *g, const float *beta, float *state,
                          const int32_t *state_indices, int n_states, float scale, int qk_l2norm, int N, int H,
                          int dk, int dv, gdn_dtype dtype, void *o, gdn_stream_t stream);

/*
 * Block norm: what lies between two blocks of a layer, over rows of D elements,
 *
 *     n = y rstd_post w_post   (post_norm; else n = y),  rstd_post = (mean y^2 + eps)^-1/2,
 *     x = residual + scale n a(gate),                    a = SiLU or sigmoid,
 *     h = x rstd_pre w_pre     (pre_norm),               rstd_pre = (mean x^2 + eps)^-1/2.
 *
 * The rows are [outer][inner] (heads of a token are inner rows; inner = 1: plain
 * rows), outer inner < 2^31, with a stride for each level; outputs are contiguous.
 * gate, residual (no gate, no residual), the weights and scale ([D] in w_dtype, fp32 or
 * dtype; one) may be NULL.  x, h: [rows, D] in dtype; rstd_post, rstd_pre: fp32 [rows],
 * needed with their norm.  h and rstd_pre are of x before it is rounded.  x or h may be
 * the memory of y, gate or residual itself where that is contiguous.
 */
typedef enum { GDN_GATE_SILU = 0, GDN_GATE_SIGMOID = 1 } gdn_gate;
typedef struct {
    const void *y, *gate, *post_weight, *scale, *pre_weight;
    int64_t outer, inner, D;
    int64_t y_outer_stride, y_inner_stride, gate_outer_stride, gate_inner_stride;
    float eps;
    int32_t post_norm, pre_norm, gate_activation, dtype, w_dtype;
} gdn_block_norm_desc;

gdn_status gdn_block_norm_fwd(const gdn_block_norm_desc *desc, const void *residual, int64_t r_outer_stride,
                              int64_t r_inner_stride, void *x, void *h, float *rstd_post, float *rstd_pre,
                              gdn_stream_t stream);

/*
 * Its backward pass, from dx (the gradient of x beside h's; NULL: zero, with pre_norm
 * only), dh and x (with pre_norm; NULL else), and the forward pass's rstd: with g = dh
 * w_pre, xh = x rstd_pre, yh = y rstd_post,
 *
 *     d = dx + rstd_pre (g - xh mean(g xh)),   dresidual = d,   dgate = d scale n a'(gate),
 *     dy = rstd_post (e - yh mean(e yh)),      e = d scale a(gate) w_post,
 *     dpre_weight = sum dh xh,  dpost_weight = scale sum d a yh,  dscale = sum d a n.
 *
 * dy, dgate (with a gate), dresidual (may be NULL) in dtype, contiguous; the
 * parameters' gradients fp32 [D], each may be NULL.  The workspace (16-byte aligned,
 * gdn_block_norm_bwd_workspace_size() bytes) is needed for those only.  The same
 * inputs give the same bits.  dresidual or dy may be the memory of dx, dh or x, and
 * dgate that of gate.
 */
size_t gdn_block_norm_bwd_workspace_size(const gdn_block_norm_desc *desc);
gdn_status gdn_block_norm_bwd(const gdn_block_norm_desc *desc, const void *dx, int64_t dx_outer_stride,
                              int64_t dx_inner_stride, const void *dh, int64_t dh_outer_stride, int64_t dh_inner_stride,
                              const void *x, int64_t x_outer_stride, int64_t x_inner_stride, const float *rstd_post,
                              const float *rstd_pre, void *dy, void *dresidual, void *dgate, float *dpost_weight,
                              float *dscale, float *dpre_weight, void *workspace, size_t workspace_bytes,
                              gdn_stream_t stream);

/*
 * Gated feed-forward block over M rows:
 *
 *     g = x w_gate^T,  u = x w_up^T,  h = act(g) u,  y = h w_down^T,
 *
 * act SiLU, or GELU in its tanh form.  x: M rows of D, x_stride elements apart;
 * w_gate, w_up: [F, D], w_down: [D_out, F], all in dtype; y: [M, D_out]; gate, up:
 * [M, F], g and u for the backward pass, or both NULL.  bf16 (h is rounded to bf16
 * between the two products, whose sums are fp32) or fp32 (products of three bf16
 * terms a value, sums fp32: as exact as fp32 products).  A row that is not finite
 * makes its own outputs non-finite (with fp32 an infinity may give NaN, and a value
 * from 3.39e38 on counts as one).
 *
 * The workspace is 16-byte aligned and holds gdn_gated_ffn_fwd_workspace_size()
 * bytes, which depends on the sizes and on how x and the weights are aligned (0:
 * arguments that the call refuses); with fp32, or rows that are not 16-byte aligned,
 * it holds copies of x and of the weights.  M, D, F and D_out at most 2^24, the largest
 * tensor (x with its stride too) 2^38 elements.
 *
 * device_status: NULL, or a device int32 into which the call writes 0, or
 * GDN_ERR_TIMEOUT where a wait inside a kernel ran out.
 */
typedef enum { GDN_ACT_SILU = 0, GDN_ACT_GELU_TANH = 1 } gdn_activation;
typedef struct {
    const void *x, *w_gate, *w_up, *w_down;
    int64_t x_stride, M, D, F, D_out;
    int32_t activation, dtype;
} gdn_ffn_desc;

size_t gdn_gated_ffn_fwd_workspace_size(const gdn_ffn_desc *desc);
gdn_status gdn_gated_ffn_fwd(const gdn_ffn_desc *desc, void *y, void *gate, void *up, int32_t *device_status,
                             void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/*
 * Its backward pass, from dy (M rows of D_out, dy_stride elements apart) and the
 * forward pass's gate and up: with dh = dy w_down,
 *
 *     dg = dh u act'(g),  du = dh act(g),  dx = dg w_gate + du w_up,
 *     dw_gate = dg^T x,  dw_up = du^T x,  dw_down = dy^T h.
 *
 * dx [M, D] and the weights' gradients (laid out like the weights) in dtype, each
 * may be NULL; for bf16 dg, du and h are rounded to bf16 between the products.  The
 * same inputs give the same bits.  Workspace and device_status as above.
 */
size_t gdn_gated_ffn_bwd_workspace_size(const gdn_ffn_desc *desc, const void *dy, int64_t dy_stride);
gdn_status gdn_gated_ffn_bwd(const gdn_ffn_desc *desc, const void *dy, int64_t dy_stride, const void *gate,
                             const void *up, void *dx, void *dw_gate, void *dw_up, void *dw_down,
                             int32_t *device_status, void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/* Tests of the error path: 0, or GDN_DEBUG_TIMEOUT_PROBE (the products on tiles load
 * nothing, so that their bounded waits run out, about 2 s a launch, and the call reports
 * GDN_ERR_TIMEOUT), for the later calls of this host thread. */
gdn_status gdn_gated_ffn_debug(int debug_checks);

/*
 * How the block's products run (host only, no GPU needed), for tests and tools: few
 * tokens forward by kernels of their own, else each pass as two launches on tiles,
 * first = 0 (both projections; backward dh) and 1 (y; backward the gradients of x, w_gate,
 * w_up, w_down).  backward = 0 ignores dy.
 */
enum { GDN_FFN_NOTHING = 0, GDN_FFN_FEW = 1, GDN_FFN_TILES = 2 };
typedef struct {
    int32_t path;             /* GDN_FFN_*: no tokens, a few, or tiles (then the rest) */
    int32_t tile[2];          /* 0: pairs of CTAs of 256 x 256, 1: 128 x 256, 2: 128 x 128 */
    int32_t a_rows[2];        /* tiles of 128 x 128: rows of the first operand's boxes */
    int32_t products[2];
    int32_t parts[2][4];      /* of each product: 0: leaves at once, n > 0: as n parts of
                                 its sum, which another kernel adds */
} gdn_ffn_plan_info;
gdn_status gdn_gated_ffn_plan_query(const gdn_ffn_desc *desc, int backward, const void *dy, int64_t dy_stride,
                                    gdn_ffn_plan_info *info);

/* The CUDA error (and, for tensor-map encoding, the driver result) behind the
 * most recent GDN_ERR_CUDA returned on the calling host thread, as text such
 * as "launch fused_tc: cudaErrorInvalidValue"; after gdn_chunk_fwd_static
 * returns GDN_ERR_WORKSPACE, the scratch it would have needed; "" when there
 * was none. */
const char *gdn_last_error_detail(void);

/* Human-readable name of a status. */
const char *gdn_status_string(gdn_status status);

/* Library version string. */
const char *gdn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_GB300_H */
