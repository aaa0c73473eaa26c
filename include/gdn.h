/*
 * gdn.h -- C ABI of libgdn: Gated DeltaNet (GDN) chunked prefill, forward and
 * backward, on one AMD Instinct MI355X (gfx950).
 *
 * The operation. The FlashQLA pages describe a linear-attention kernel library
 * for the Gated Delta Network's chunked prefill (ollai.cn article, sections
 * "what it is" and "main features"): it takes q, k, v, a gate g and a write
 * strength beta, returns O and the final state, and accepts an optional
 * initial state and packed variable-length sequences via cu_seqlens
 * ("how to use"). It offers low-level forward / backward entry points
 * ("main features", two-level API). The pages print no formula; this library
 * computes the standard gated delta rule, per sequence and head,
 *
 *     S_t = exp(g_t) S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T
 *     o_t = scale * S_t q_t
 *
 * S is V x K (row i over the value dimension, column j over the key
 * dimension). The state enters as initial_state (zeros when NULL) and leaves
 * as final_state. g is a natural-log decay (exp(g_t) multiplies the state).
 * q and k are used as given (no normalisation inside).
 *
 * Layouts (all row-major, contiguous, device memory unless stated):
 *   q, k, dq, dk        [B, T, H, K]   element type desc->dtype
 *   v, o, d_o, dv       [B, T, H, V]   element type desc->dtype
 *   g, beta, dg, dbeta  [B, T, H]      fp32
 *   initial_state, final_state, d_final_state, d_initial_state
 *                       [N, H, V, K]   fp32, N = number of sequences
 *   With varlen (cu_seqlens != NULL) B must be 1, T is the packed token count
 *   and sequence n owns tokens [cu_seqlens[n], cu_seqlens[n+1]).
 *
 * How it runs (the split the pages describe in "technical principles" and
 * "core advantages"): a gate-cumsum + intra-chunk kernel writes the WY factors
 * w and u, an optional intra-card context-parallel (CP) preprocessing step
 * gives every sub-sequence its initial state, and an inter-chunk recurrence
 * kernel produces O and the final state. CP turns on by itself for small
 * batch x heads ("AutoCP"; the pages' thresholds, B*H <= 40 or B*H <= 56 with
 * seq_len >= 8192, were tuned for a 132-SM part: here the default turns CP on when
 * the recurrence would otherwise leave compute units idle, GDN_CP_PAGES keeps the
 * pages' rule) and picks per sub-sequence boundary either the exact correction or a
 * sliding-window warmup of a few chunks where the gate decay makes the warmup exact within
 * tolerance ("gate-driven" warmup, "core advantages").
 *
 * Ownership and errors: the caller allocates every buffer, including the
 * workspace, whose size the *_workspace_size calls return. The library
 * allocates no memory (gdn_chunk_fwd_noalloc's fixed scratch array is part of
 * the library's image, see there), keeps no pointer after a call returns, never
 * synchronises the host with the device and never aborts. All work is
 * enqueued on `stream` (a hipStream_t; NULL = the default stream). Outputs
 * are overwritten, never accumulated, and must not alias inputs. Argument
 * checks run on the host before any launch; a failed launch reports
 * GDN_ERR_HIP. Results are deterministic (no atomics).
 */
#ifndef GDN_H_
#define GDN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_ABI_VERSION 10

typedef enum gdn_status {
    GDN_OK = 0,
    GDN_ERR_INVALID_ARG = 1, /* null pointer, bad size, inconsistent cu_seqlens */
    GDN_ERR_UNSUPPORTED = 2, /* K or V not in {64,128}, chunk != 64, sizes beyond 32-bit grids */
    GDN_ERR_WORKSPACE = 3,   /* workspace NULL or smaller than required */
    GDN_ERR_HIP = 4          /* a HIP call or kernel launch failed */
} gdn_status;

typedef enum gdn_dtype {
    GDN_DTYPE_BF16 = 0, /* q,k,v,o and their gradients in bf16; fp32 accumulation and state */
    GDN_DTYPE_FP32 = 1  /* everything fp32 */
} gdn_dtype;

typedef enum gdn_cp_mode {
    GDN_CP_AUTO = 0,   /* CP when the recurrence would leave compute units idle without it: the
                          sequence-heads' row tiles fill at most half of its workgroup slots
                          and the longest sequence spans two sub-sequences of 16 chunks or
                          more; or, for packed sequences, when the longest one takes 1.5x
                          (and at least 64) the chunk steps per slot the batch needs, in
                          sub-sequences of half that (at least 32); a gate test at every
                          sub-sequence boundary picks warmup or exact there */
    GDN_CP_OFF = 1,    /* one serial pass per sequence-head */
    GDN_CP_ON = 2,     /* CP regardless of the shape rule; per-boundary gate test. Without
                          seg_chunks, a batch that already fills the slots takes sub-sequences
                          of half the chunk steps per slot it needs (at least 16) */
    GDN_CP_EXACT = 3,  /* CP, exact correction for every sequence-head */
    GDN_CP_WARMUP = 4, /* CP, warmup for every sequence-head (caller asserts fast decay) */
    GDN_CP_PAGES = 5   /* the pages' AutoCP thresholds, tuned for a 132-SM part: CP iff
                          N*H <= 40, or N*H <= 56 and the longest sequence >= 8192 tokens */
} gdn_cp_mode;

/* desc->flags: keeping the forward's intermediates for the backward of a training step.
 * GDN_FLAG_KEEP_FORWARD    gdn_chunk_fwd leaves in its workspace what the backward
 *                          recomputes otherwise: the chunk gate cumsums, w, u, T = (I+A)^-1,
 *                          the CP decisions, the sub-sequence entry states, every chunk's
 *                          entry state and Delta = U - W S^T (the forward workspace then
 *                          includes room for T, the states and Delta).
 * GDN_FLAG_REUSE_FORWARD   gdn_chunk_bwd starts from them instead of recomputing the
 *                          intra-chunk pass, the forward CP preprocessing and the chunk-state
 *                          pass. The caller
 *                          guarantees that the same workspace last held a KEEP_FORWARD
 *                          forward of the same inputs and descriptor (flags aside), with
 *                          no other call on it since except REUSE_FORWARD backwards. */
#define GDN_FLAG_KEEP_FORWARD 1
#define GDN_FLAG_REUSE_FORWARD 2

/* GDN_FLAG_QK_L2NORM: q and k are raw; the path scales every row of K values (one token,
 * one head) to x / sqrt(sum x^2 + 1e-6) and runs on those rows, the preprocessing the pages place
 * ahead of the fused kernels (edge.aivizor.me community post, its account of the chunked-prefill
 * pipeline) with the unit-norm q and k their workloads use. The kernels normalise the rows as
 * they stage them; the intra-chunk kernel writes the normalised k rows once for the later ones,
 * at the start of the workspace (T x H x K values in the input dtype more, in both layouts).
 * gdn_chunk_bwd then returns dq and dk with respect to the raw q and k:
 * dx = r (dxhat - xhat (xhat . dxhat)), r = (sum x^2 + 1e-6)^(-1/2). With
 * GDN_FLAG_REUSE_FORWARD the normalised k rows come from the kept forward, which must have had
 * this flag too. gdn_intra_chunk and gdn_cp_modes normalise k; gdn_recurrent_fwd normalises q
 * and k inside its kernel (fp32 rows, not rounded to the input dtype). */
#define GDN_FLAG_QK_L2NORM 4

/* GDN_FLAG_BWD_ADJOINT_PASS: gdn_chunk_bwd runs the reverse adjoint recurrence as a pass of its
 * own that stores every chunk's adjoint and dDelta for the per-chunk gradient kernel. By default,
 * at V = 128 in bf16 with CP on or a uniform batch, the per-chunk gradient kernel carries the
 * adjoint itself (one workgroup per sub-sequence and head walking its chunks in reverse), which
 * moves fewer bytes; the flag keeps the other path selectable, for comparison. Same results within
 * rounding. */
#define GDN_FLAG_BWD_ADJOINT_PASS 8

/* The fully fused forward: with CP off, bf16 inputs and no kept intermediates, gdn_chunk_fwd can run
 * the intra-chunk step and the recurrence in one kernel (one workgroup per sequence, head and row
 * tile, walking the chunks in order), so w, u and the gate cumsum never go to memory: 1,032 instead
 * of 2,320 bytes per token-head at K = V = 128. The pages name the fully fused design as the one
 * with less memory I/O at large batch (announcement post, on the two-kernel split). The plan picks it
 * where it measures faster (gdn_plan_info.fused_fwd); GDN_FLAG_FWD_FUSED asks for it wherever it is
 * supported, GDN_FLAG_FWD_SPLIT never. Same results within rounding. */
#define GDN_FLAG_FWD_FUSED 16
#define GDN_FLAG_FWD_SPLIT 32

/* Carrying the forward's CP results to the backward (a checkpoint of a few MB instead of the
 * intra-chunk intermediates): with CP on, the backward's chunk-state pass needs the same
 * sub-sequence entry states that the forward's CP preprocessing (decision, prepass, segment scan;
 * ollai.cn article, "technical principles") already produced. gdn_chunk_fwd writes its CP
 * decisions and those states to desc->cp_states when that pointer is set; gdn_chunk_bwd with
 * GDN_FLAG_REUSE_CP reads them from there instead of running the forward-direction
 * preprocessing again (it still recomputes the intra-chunk pass and decides the reverse
 * direction itself). The caller guarantees that a gdn_chunk_fwd of the same inputs and
 * descriptor (flags aside) last wrote the buffer. A GDN_FLAG_REUSE_FORWARD backward reads them
 * there too when the pointer is set (its forward wrote them there); any other backward leaves
 * the buffer alone. Without CP the flag does nothing and the buffer is not touched.
 * GDN_FLAG_REUSE_CP with CP on and desc->cp_states NULL returns GDN_ERR_INVALID_ARG. */
#define GDN_FLAG_REUSE_CP 64

/* Problem descriptor. Zero-initialise, then fill. */
typedef struct gdn_desc {
    int64_t B, T, H, K, V;          /* batch, tokens per row (packed total if varlen), heads, key dim, value dim */
    int32_t chunk;                  /* chunk length; must be 64 (0 = 64) */
    int32_t dtype;                  /* gdn_dtype */
    float scale;                    /* query scale applied to o (the rule above has none: pass 1.0) */
    int32_t num_seqs;               /* varlen: N (>= 1); ignored otherwise */
    const int32_t* cu_seqlens;      /* device [N+1] token offsets, or NULL (then N = B) */
    const int32_t* cu_seqlens_host; /* host copy of cu_seqlens; required with it (planning needs no sync) */
    int32_t cp_mode;                /* gdn_cp_mode */
    int32_t warmup_chunks;          /* warmup window in chunks, 1..16 (0 = 8) */
    int32_t seg_chunks;             /* CP sub-sequence length in chunks (0 = chosen from the CU count) */
    float warmup_eps;               /* warmup acceptance: exp(window gate sum) <= eps (0 = 1e-4 bf16, 1e-6 fp32) */
    int32_t num_cus;                /* compute units to plan for (0 = query the current device) */
    int32_t flags;                  /* GDN_FLAG_* (0 = none) */
    int32_t warmup_max_chunks;      /* longest warmup window a sequence-head may take when
                                       warmup_chunks do not meet the acceptance bound (AUTO, ON):
                                       warmup_chunks..warmup_chunks+63, or 0 = the sub-sequence
                                       length (at least warmup_chunks, at most warmup_chunks+63);
                                       equal to warmup_chunks keeps one fixed window */
    int32_t reserved[5];            /* must be zero */
    void* cp_states;                /* device buffer of gdn_plan_info.cp_states_bytes bytes, 256-byte
                                       aligned, or NULL: see GDN_FLAG_REUSE_CP (owned by the caller;
                                       gdn_recurrent_fwd requires NULL) */
} gdn_desc;

/* Host-side plan of a call (filled by gdn_plan; no device work). */
typedef struct gdn_plan_info {
    int32_t num_seqs;               /* N */
    int32_t cp_on;                  /* 1 if the call splits sequences into sub-sequences */
    int32_t seg_chunks;             /* chunks per sub-sequence (the last one may be shorter) */
    int32_t warmup_chunks;          /* warmup window W in chunks (the shortest one taken) */
    int32_t warmup_max_chunks;      /* longest warmup window a sequence-head may take */
    float warmup_eps;               /* warmup acceptance threshold */
    int32_t v_tiles;                /* value-row tiles per sequence-head in the recurrence kernel */
    int64_t max_len;                /* longest sequence, tokens */
    int64_t total_chunks;           /* sum over sequences of ceil(len / 64) */
    int64_t total_segments;         /* sum over sequences of sub-sequence counts */
    size_t fwd_workspace_bytes;
    size_t bwd_workspace_bytes;
    size_t cp_states_bytes;         /* size of desc->cp_states (CP decisions and sub-sequence entry
                                       states, fp32 [total_segments, H, V, K]); 0 when CP is off */
    int32_t fused_fwd;              /* 1 if gdn_chunk_fwd runs the fully fused forward */
    int32_t bwd_carried;            /* 1 if gdn_chunk_bwd's per-chunk kernel carries the adjoint
                                       (no separate adjoint pass) */
    int32_t reserved_out[2];
} gdn_plan_info;

/* ABI version (GDN_ABI_VERSION of the built library). */
int gdn_abi_version(void);

/* Static English text for a status code; never NULL. */
const char* gdn_status_string(gdn_status status);

/* Validate `desc` and fill `out` with the plan the calls below would use:
 * whether CP is on (AutoCP, "core advantages"; see gdn_cp_mode), sub-sequence
 * length, warmup window and workspace sizes. Host only: reads
 * cu_seqlens_host, never cu_seqlens; queries the device CU count only when
 * desc->num_cus == 0. */
gdn_status gdn_plan(const gdn_desc* desc, gdn_plan_info* out);

/* Workspace bytes that gdn_chunk_fwd needs for `desc`. */
gdn_status gdn_chunk_fwd_workspace_size(const gdn_desc* desc, size_t* bytes);

/* Forward (the pages' low-level fwd entry, "main features"): O and the final
 * state of the gated delta rule above.
 *   q, k, v, g, beta : inputs (layouts above)
 *   initial_state    : [N,H,V,K] fp32 or NULL (zeros)
 *   o                : output [B,T,H,V]
 *   final_state      : output [N,H,V,K] fp32, or NULL (not written)
 *   workspace        : device scratch of at least gdn_chunk_fwd_workspace_size bytes, 256-byte aligned
 *                      (with GDN_FLAG_KEEP_FORWARD, the one the backward will receive)
 *   stream           : hipStream_t (NULL = default stream)
 * Returns GDN_OK once all work is enqueued. */
gdn_status gdn_chunk_fwd(const gdn_desc* desc, const void* q, const void* k, const void* v,
                         const float* g, const float* beta, const float* initial_state,
                         void* o, float* final_state,
                         void* workspace, size_t workspace_bytes, void* stream);

/* For callers that cannot allocate device memory (code under HIP graph capture, serving loops
 * or harnesses that forbid hipMalloc): gdn_chunk_fwd with its workspace taken from a fixed
 * array inside the library, GDN_NOALLOC_SCRATCH_BYTES per GPU, which each GPU the call runs
 * on holds from the first call there until the process ends (that first call resolves the
 * array's address: make it once before capturing a graph). Same arguments, layouts and
 * results as gdn_chunk_fwd without the workspace; the caller still owns every input and
 * output. It allocates nothing.
 * Errors: a descriptor whose forward workspace (gdn_chunk_fwd_workspace_size) exceeds
 * GDN_NOALLOC_SCRATCH_BYTES returns GDN_ERR_WORKSPACE, and GDN_FLAG_KEEP_FORWARD or
 * GDN_FLAG_REUSE_FORWARD returns GDN_ERR_INVALID_ARG (kept intermediates would not outlive
 * the next call), both before any launch; otherwise as gdn_chunk_fwd.
 * Every call on one GPU shares that GPU's array, and the array keeps the last call's contents
 * (nothing in it needs to start at zero: every kernel writes what it reads in the same call).
 * Calls that overlap on one GPU (on different streams, or from several host threads) race on
 * the array: the caller serialises them. */
#define GDN_NOALLOC_SCRATCH_BYTES ((size_t)128 << 20)
gdn_status gdn_chunk_fwd_noalloc(const gdn_desc* desc, const void* q, const void* k, const void* v,
                                 const float* g, const float* beta, const float* initial_state,
                                 void* o, float* final_state, void* stream);

/* Workspace bytes that gdn_chunk_bwd needs for `desc`. */
gdn_status gdn_chunk_bwd_workspace_size(const gdn_desc* desc, size_t* bytes);

/* Backward (the pages' low-level bwd entry): gradients of
 * L = <d_o, O> + <d_final_state, final_state> with respect to every input.
 *   q, k, v, g, beta, initial_state : the forward's inputs (initial_state may be NULL)
 *   d_o             : [B,T,H,V] upstream gradient of O
 *   d_final_state   : [N,H,V,K] fp32 upstream gradient of the final state, or NULL (zeros)
 *   dq, dk, dv      : outputs, same layouts and dtype as q, k, v
 *   dg, dbeta       : outputs [B,T,H] fp32 (dg is with respect to the raw per-token g)
 *   d_initial_state : output [N,H,V,K] fp32, or NULL (not written)
 * The forward is recomputed inside, unless desc->flags has GDN_FLAG_REUSE_FORWARD (then the
 * intra-chunk pass and the forward CP preprocessing come from the workspace; see above) or
 * GDN_FLAG_REUSE_CP (then the forward CP preprocessing comes from desc->cp_states).
 * The reverse adjoint pass runs on a second stream of the library's (one per device, made on
 * the first call with the default priority), forked from `stream` and joined back to it
 * before the per-chunk gradients: work enqueued on `stream` afterwards sees every output.
 * Concurrent calls from several host threads are serialised while they enqueue. */
gdn_status gdn_chunk_bwd(const gdn_desc* desc, const void* q, const void* k, const void* v,
                         const float* g, const float* beta, const float* initial_state,
                         const void* d_o, const float* d_final_state,
                         void* dq, void* dk, void* dv, float* dg, float* dbeta,
                         float* d_initial_state,
                         void* workspace, size_t workspace_bytes, void* stream);

/* Recurrent form: the gated delta rule token by token from a given state, for decoding
 * after a prefill (the pages' interface continues a call from the previous one's state,
 * ollai.cn article, "how to use"). Every sequence b has desc->T tokens (T >= 0; a decoder
 * passes 1 or a few); no cu_seqlens, no CP, no workspace; desc->flags 0 or GDN_FLAG_QK_L2NORM
 * (raw q and k, normalised per token as in gdn_chunk_fwd).
 *   q, k [B,T,H,K]; v, o [B,T,H,V] (desc->dtype); g, beta [B,T,H] fp32 (layouts above)
 *   state_in  : [B,H,V,K] fp32 state entering the first token, or NULL (zeros); typically
 *               the final_state of gdn_chunk_fwd or of the previous call
 *   state_out : [B,H,V,K] fp32 state after the last token (required); may be state_in
 *               itself (updated in place)
 * One workgroup per (sequence, head) keeps its state in registers across the T tokens; the
 * state is read and written once per call. Same status codes as the calls above (K, V not
 * in {64,128}: GDN_ERR_UNSUPPORTED). */
gdn_status gdn_recurrent_fwd(const gdn_desc* desc, const void* q, const void* k, const void* v,
                             const float* g, const float* beta, const float* state_in,
                             float* state_out, void* o, void* stream);

/* Intra-chunk step alone (the first fused kernel): chunk-local cumulative gate
 * sum and the WY factors, for kernel-level checks. With gam the chunk-local
 * cumsum of g, A = strict_lower(diag(beta) (exp(gam_r - gam_j) k_r.k_j)) and
 * T = (I + A)^-1 per chunk:
 *   gam_out [B,T,H] fp32; w_out = T diag(beta exp(gam)) K  [B,T,H,K];
 *   u_out   = T diag(beta) V  [B,T,H,V]  (dtype desc->dtype).
 * Uses the forward workspace. */
gdn_status gdn_intra_chunk(const gdn_desc* desc, const void* k, const void* v,
                           const float* g, const float* beta,
                           float* gam_out, void* w_out, void* u_out,
                           void* workspace, size_t workspace_bytes, void* stream);

/* CP decision per sequence-head, as the forward would take it. The decision is made per
 * boundary (the start of every sub-sequence but a sequence's first): the warmup over the
 * shortest window from warmup_chunks to warmup_max_chunks chunks that meets the acceptance
 * bound there, else the exact correction ("gate-driven" warmup, ollai.cn article, "core
 * advantages"); the exact maps and the scan then run only across the exact boundaries.
 * modes_out [N, H] int32 (device): 0 = no split needed, 1 = every boundary takes the warmup,
 * 2 = every boundary takes the exact correction, 3 = both kinds (mixed).
 * Uses the forward workspace; runs the intra-chunk kernel to get the gates. */
gdn_status gdn_cp_modes(const gdn_desc* desc, const void* k, const void* v,
                        const float* g, const float* beta, int32_t* modes_out,
                        void* workspace, size_t workspace_bytes, void* stream);

/* The per-boundary CP decision itself (see gdn_cp_modes): fwd_windows [S, H] int32 (device),
 * S = gdn_plan_info.total_segments, row gs for the boundary at the start of global sub-sequence
 * gs (a sequence's sub-sequences are consecutive): the warmup window in chunks before it, 0 =
 * exact correction, -1 = no boundary (a sequence's first sub-sequence). rev_windows, if not
 * NULL, the same for the backward's adjoint pass (windows after each boundary). Uses the
 * forward workspace; runs the intra-chunk kernel to get the gates. */
gdn_status gdn_cp_windows(const gdn_desc* desc, const void* k, const void* v,
                          const float* g, const float* beta, int32_t* fwd_windows,
                          int32_t* rev_windows, void* workspace, size_t workspace_bytes,
                          void* stream);

/* ------------------------------------------------------------------------------------------
 * Operators that stand around the gated delta rule in a layer. Same conventions as above:
 * row-major contiguous device buffers of the caller, the caller's stream, argument checks before
 * any launch, no allocation, no host synchronisation, deterministic results, outputs overwritten.
 * Descriptors are zero-initialised, then filled; `reserved` must be zero. They take channels in
 * any number; rows whose length or buffers whose address do not fit 16-byte vectors are slower, no
 * more. Sizes beyond a 32-bit grid of threads return GDN_ERR_UNSUPPORTED.
 *
 * Sequences: without cu_seqlens, row b of [B, T, D] is sequence b (N = B). With cu_seqlens (device
 * int32 [N+1], not decreasing), B is 1 and sequence n owns tokens [cu_seqlens[n], cu_seqlens[n+1]);
 * tokens before cu_seqlens[0] and from cu_seqlens[N] on belong to no sequence: their inputs reach no
 * result, and their rows of the outputs (and of dx and dg) are left as they were, or receive zeros
 * with GDN_FLAG_ZERO_OUTSIDE. No host copy is needed. Offsets are read clamped into [0, T]: an array that
 * decreases gives unspecified values, never an access out of range.
 * An empty sequence passes its entering state on as its final state (and the final state's
 * gradient on as the entering state's). */
#define GDN_FLAG_ZERO_OUTSIDE 128

/* Gated scan: the recurrence with a gate per channel,
 *     h_t = exp(g_t) h_{t-1} + x_t,    h_0 = initial_state (zeros when NULL),
 * per sequence and channel; g is a natural-log decay (usually <= 0; -inf forgets). Gates above zero
 * are taken too, but the tokens are worked on in runs of up to 128, whose gates' products must stay
 * within fp32's range where a state other than zero enters the run (in the gradient: where a gradient
 * other than zero does, from behind). A product below the range counts as zero. */
typedef struct gdn_scan_desc {
    int64_t B, T, D;
    int32_t dtype;             /* gdn_dtype of x, h and their gradients */
    int32_t g_dtype;           /* gdn_dtype of g and dg: dtype's, or GDN_DTYPE_FP32 */
    int32_t num_seqs;          /* with cu_seqlens: N (>= 1); ignored otherwise */
    int32_t flags;             /* 0 or GDN_FLAG_ZERO_OUTSIDE */
    const int32_t* cu_seqlens; /* device [N+1], or NULL */
    int32_t reserved[4];       /* must be zero */
} gdn_scan_desc;

/* Bytes of the workspaces (256-byte aligned) and of the kept states. They do not depend on the
 * types; a packed call never needs more than the unpacked one of its B, T and D. */
gdn_status gdn_gated_scan_fwd_workspace_size(const gdn_scan_desc* desc, size_t* bytes);
gdn_status gdn_gated_scan_bwd_workspace_size(const gdn_scan_desc* desc, size_t* bytes);
gdn_status gdn_gated_scan_states_size(const gdn_scan_desc* desc, size_t* bytes);

/* Forward.
 *   x, h  [B,T,D] (dtype); g [B,T,D] (g_dtype); initial_state, final_state [N,D] fp32
 *   initial_state may be NULL (zeros); final_state may be NULL (not written) or initial_state
 *   itself (updated in place, for decoding)
 *   states: NULL, or a buffer of gdn_gated_scan_states_size bytes (256-byte aligned) that receives
 *   what gdn_gated_scan_bwd needs of the forward: the fp32 state entering every 64th token (nothing
 *   is written where a call is one tile of tokens and needs none)
 * A call of up to 16 tokens per row (decoding), or of a packed batch of up to 512 tokens and no more of
 * them than sequences, is one launch and needs no workspace. In the others a run of tokens waits on the
 * device for the state of the run before it; a wait that lasts about a second (which no call in working
 * order comes near) gives up, and leaves NaN from there to the sequence's end. */
gdn_status gdn_gated_scan_fwd(const gdn_scan_desc* desc, const void* x, const void* g,
                              const float* initial_state, void* h, float* final_state, void* states,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Gradients of <d_h, h> + <d_final_state, final_state>.
 *   d_h, dx [B,T,D] (dtype); dg [B,T,D] (g_dtype; with respect to the log-decay)
 *   d_final_state [N,D] fp32 or NULL (zeros); d_initial_state [N,D] fp32 or NULL (not written)
 *   states: what the forward of the same inputs wrote, or NULL (recomputed here) */
gdn_status gdn_gated_scan_bwd(const gdn_scan_desc* desc, const void* x, const void* g,
                              const float* initial_state, const void* d_h,
                              const float* d_final_state, const void* states, void* dx, void* dg,
                              float* d_initial_state, void* workspace, size_t workspace_bytes,
                              void* stream);

/* Short causal convolution, one filter of W taps per channel:
 *     z_t = bias + sum_j weight[:, j] x_{t-W+1+j},    y = z or silu(z),
 * the inputs before a sequence's first token being its initial_state (zeros when NULL). */
typedef enum gdn_activation {
    GDN_ACT_NONE = 0,
    GDN_ACT_SILU = 1,
    GDN_ACT_GELU_TANH = 2 /* the gated feed-forward block alone */
} gdn_activation;
typedef struct gdn_conv_desc {
    int64_t B, T, D;
    int32_t width;             /* W: 2, 3 or 4 taps */
    int32_t dtype;             /* gdn_dtype of x, y, the states and their gradients */
    int32_t w_dtype;           /* gdn_dtype of weight and bias: dtype's, or GDN_DTYPE_FP32 */
    int32_t activation;        /* gdn_activation */
    int32_t num_seqs;          /* with cu_seqlens: N (>= 1); ignored otherwise */
    int32_t flags;             /* 0 or GDN_FLAG_ZERO_OUTSIDE */
    const int32_t* cu_seqlens; /* device [N+1], or NULL */
    int32_t reserved[4];       /* must be zero */
} gdn_conv_desc;

gdn_status gdn_short_conv_bwd_workspace_size(const gdn_conv_desc* desc, size_t* bytes);

/* Forward.
 *   x, y [B,T,D]; weight [D,W]; bias [D] or NULL
 *   initial_state, final_state [N, W-1, D], oldest input first: the last W-1 inputs of a sequence,
 *   its initial_state in front of them where it is shorter. initial_state may be NULL (zeros);
 *   final_state may be NULL (not written), or initial_state itself where T <= GDN_CONV_INPLACE_T
 *   without cu_seqlens (updated in place, for decoding; otherwise GDN_ERR_INVALID_ARG) */
#define GDN_CONV_INPLACE_T 16
gdn_status gdn_short_conv_fwd(const gdn_conv_desc* desc, const void* x, const void* weight,
                              const void* bias, const void* initial_state, void* y,
                              void* final_state, void* stream);

/* Gradients of <d_y, y> + <d_final_state, final_state>; the forward is recomputed inside.
 *   d_y, dx [B,T,D]; dweight [D,W] fp32; dbias [D] fp32 or NULL (not written)
 *   d_final_state, d_initial_state [N, W-1, D] (dtype) or NULL (zeros; not written) */
gdn_status gdn_short_conv_bwd(const gdn_conv_desc* desc, const void* x, const void* weight,
                              const void* bias, const void* initial_state, const void* d_y,
                              const void* d_final_state, void* dx, float* dweight, float* dbias,
                              void* d_initial_state, void* workspace, size_t workspace_bytes,
                              void* stream);

/* RMS norm of rows of D values, the residual stream's addition in front:
 *     r = x + residual (rounded to dtype: what residual_out receives is what is normed),
 *     y = r weight / sqrt(mean(r^2) + eps).
 * With out_type GDN_OUT_E4M3, y holds 8-bit floats (OCP e4m3) and scale their fp32 scales, of a
 * whole row (scale_group 0; scale [rows]) or of every 128 columns (scale_group 128; scale
 * [rows, ceil(D/128)]): scale = max|y| / 448 (at least 2^-126), or 1 where every y is zero, and the
 * 8-bit value is y / scale to nearest even, formed from the fp32 y. A row with NaN or infinity in it gets what
 * the formulas give: NaN scales where a NaN is among their columns. */
typedef enum gdn_out_type { GDN_OUT_SAME = 0, GDN_OUT_E4M3 = 1 } gdn_out_type;
typedef struct gdn_rmsnorm_desc {
    int64_t rows, D;
    int32_t dtype;       /* gdn_dtype of x, residual, residual_out, y and their gradients */
    int32_t w_dtype;     /* gdn_dtype of weight: dtype's, or GDN_DTYPE_FP32 */
    int32_t out_type;    /* gdn_out_type (the backward ignores it) */
    int32_t scale_group; /* with GDN_OUT_E4M3: 0 (a row) or 128 columns per scale; else 0 */
    float eps;           /* >= 0 */
    int32_t flags;       /* must be zero */
    int32_t reserved[4]; /* must be zero */
} gdn_rmsnorm_desc;

/* Forward. residual and residual_out are both given or both NULL; residual_out may be x or residual
 * itself (in place). scale only with GDN_OUT_E4M3. Rows of fewer than 8 columns or more than 32,768
 * (in the gradient 16,384): at most 4,194,303 of them (GDN_ERR_UNSUPPORTED). */
gdn_status gdn_rmsnorm_fwd(const gdn_rmsnorm_desc* desc, const void* x, const void* residual,
                           const void* weight, void* y, float* scale, void* residual_out,
                           void* stream);

gdn_status gdn_rmsnorm_bwd_workspace_size(const gdn_rmsnorm_desc* desc, size_t* bytes);

/* Gradients of <d_y, y> + <d_residual, residual_out> (of the unquantised y), from r: residual_out,
 * or x where there was no residual.
 *   dx [rows, D]: the gradient of x and, being the same, of residual; d_residual or NULL (zeros)
 *   dweight [D] fp32, or NULL (not written) */
gdn_status gdn_rmsnorm_bwd(const gdn_rmsnorm_desc* desc, const void* r, const void* weight,
                           const void* d_y, const void* d_residual, void* dx, float* dweight,
                           void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------------------------
 * The products of a layer: quantisation to e4m3, the product of e4m3 matrices, and the gated
 * feed-forward block. Conventions as above; matrices of any size at any address of their type
 * (memory rows and addresses that are multiples of 16 bytes are faster).
 *
 * Quantised matrices hold 8-bit floats (OCP e4m3) beside fp32 scales; a value stands for e4m3 x
 * scale. A scale belongs to a row, to 128 columns of a row, or to 128 x 128 values (the last ones
 * of a row or column may be fewer): */
typedef enum gdn_scales {
    GDN_SCALE_ROW = 0,   /* [rows] */
    GDN_SCALE_GROUP = 1, /* [rows, ceil(cols/128)] (what gdn_rmsnorm_fwd writes with scale_group 128) */
    GDN_SCALE_BLOCK = 2  /* [ceil(rows/128), ceil(cols/128)] */
} gdn_scales;

/* Quantisation of x [rows, cols]: scale = max|x| / 448 over the values that share it (at least 2^-126;
 * 1 where all are zero), the 8-bit value is x / scale to nearest even. With transpose (not with
 * GDN_SCALE_ROW) q is [cols, rows], and the scales are those of that matrix: groups of 128 run along
 * x's rows. Values that share a scale with a NaN become NaN, beside an infinity the finite ones become 0.
 * A scale per row: at most 16,777,215 rows, 4,194,303 of more than 8,192 columns (GDN_ERR_UNSUPPORTED). */
typedef struct gdn_quant_desc {
    int64_t rows, cols;
    int32_t dtype;       /* gdn_dtype of x */
    int32_t scales;      /* gdn_scales */
    int32_t transpose;   /* 0 or 1 */
    int32_t flags;       /* must be zero */
    int32_t reserved[4]; /* must be zero */
} gdn_quant_desc;

gdn_status gdn_quant_e4m3(const gdn_quant_desc* desc, const void* x, void* q, float* scale, void* stream);

/* y = a b^T of quantised matrices a [M,K] and b [N,K], y [M,N] in out_dtype. desc->scales is the kind of
 * b's scales: GDN_SCALE_BLOCK or GDN_SCALE_GROUP with a_scale in groups [M, ceil(K/128)], GDN_SCALE_ROW
 * with a_scale [M]. The scaled sums are fp32, and so is the product of two scales that a sum is
 * multiplied by: below 2^-126 it loses bits, below 2^-149 the sum counts as 0 (values near 1e-17 in
 * both operands, or near 1e-32 in one beside 0.1 in the other). K may be 0 (y is 0, and no scale is read).
 *   GDN_DTYPE_FP32: products and sums as in fp32.
 *   GDN_DTYPE_BF16: by the 8-bit matrix instruction, at about twice the rate: it adds products in groups
 *   of eight (neighbours along K) aligned to the largest of them, and drops what lies about 2^-13 below
 *   it. On quantised activations and weights that is 1.5e-5 of the result in the 2-norm, a hundredth
 *   of the rounding to bf16. Where large products cancel it is more, up to all that is left: ask for
 *   GDN_FLAG_EXACT_SUMS, with which the products and sums are those of fp32 and rounded to bf16 at the
 *   end (the flag says nothing new for an output in fp32). */
#define GDN_FLAG_EXACT_SUMS 256
typedef struct gdn_matmul_desc {
    int64_t M, N, K;
    int32_t out_dtype;   /* gdn_dtype of y */
    int32_t scales;      /* gdn_scales of b */
    int32_t flags;       /* 0 or GDN_FLAG_EXACT_SUMS */
    int32_t reserved[5]; /* must be zero */
} gdn_matmul_desc;

gdn_status gdn_matmul_e4m3_workspace_size(const gdn_matmul_desc* desc, size_t* bytes);
gdn_status gdn_matmul_e4m3(const gdn_matmul_desc* desc, const void* a, const float* a_scale, const void* b,
                           const float* b_scale, void* y, void* workspace, size_t workspace_bytes,
                           void* stream);

/* Gated feed-forward block:
 *     gate = x w_gate^T,  up = x w_up^T,  h = act(gate) up,
 * act(z) = z sigmoid(z) (GDN_ACT_SILU) or z sigmoid(2 sqrt(2/pi) (z + 0.044715 z^3))
 * (GDN_ACT_GELU_TANH). gate and up are fp32 sums. */
typedef struct gdn_ffn_desc {
    int64_t rows, K, F;
    int32_t dtype;       /* gdn_dtype of x, the weights, h and their gradients (gdn_gated_ffn_e4m3: of h) */
    int32_t activation;  /* GDN_ACT_SILU or GDN_ACT_GELU_TANH */
    int32_t out_type;    /* gdn_out_type of h: GDN_OUT_E4M3 with gdn_gated_ffn_e4m3 alone */
    int32_t flags;       /* 0, or with gdn_gated_ffn_e4m3 GDN_FLAG_EXACT_SUMS, with gdn_gated_ffn_bwd GDN_FLAG_GRAD_PAIRS */
    int32_t reserved[4]; /* must be zero */
} gdn_ffn_desc;

/* Forward. x [rows,K]; w_gate, w_up [F,K]; h [rows,F]. pre: NULL, or [2,rows,F] fp32 that receives gate
 * and up for the backward. */
gdn_status gdn_gated_ffn_fwd_workspace_size(const gdn_ffn_desc* desc, size_t* bytes);
gdn_status gdn_gated_ffn_fwd(const gdn_ffn_desc* desc, const void* x, const void* w_gate, const void* w_up,
                             void* h, float* pre, void* workspace, size_t workspace_bytes, void* stream);

/* Gradients of <d_h, h>. pre: what the forward of the same inputs wrote, or NULL (gate and up are computed
 * again). The gradients of gate and up are rounded to dtype, the operands' type of the products behind, which in bf16
 * makes the results' error sqrt 2 times their own rounding; to a pair of bf16, which adds nothing to it, where rows F,
 * rows K or F K is below 65,536, and with GDN_FLAG_GRAD_PAIRS at any size (8,192 x 2,048 x 8,192: 1,040 us to 2,690).
 *   d_h [rows,F]; dx [rows,K] or NULL (not written); dw_gate, dw_up [F,K], both or neither */
#define GDN_FLAG_GRAD_PAIRS 512
gdn_status gdn_gated_ffn_bwd_workspace_size(const gdn_ffn_desc* desc, size_t* bytes);
gdn_status gdn_gated_ffn_bwd(const gdn_ffn_desc* desc, const void* x, const void* w_gate, const void* w_up,
                             const float* pre, const void* d_h, void* dx, void* dw_gate, void* dw_up,
                             void* workspace, size_t workspace_bytes, void* stream);

/* Forward on quantised x (GDN_SCALE_GROUP) and weights (GDN_SCALE_BLOCK). h [rows,F] in dtype (scale
 * NULL; a bf16 h by the 8-bit matrix instruction unless GDN_FLAG_EXACT_SUMS is set, see gdn_matmul_e4m3),
 * or with GDN_OUT_E4M3 quantised from its fp32 values, scale [rows, ceil(F/128)] (GDN_SCALE_GROUP; dtype is
 * then ignored). */
gdn_status gdn_gated_ffn_e4m3_workspace_size(const gdn_ffn_desc* desc, size_t* bytes);
gdn_status gdn_gated_ffn_e4m3(const gdn_ffn_desc* desc, const void* x, const float* x_scale,
                              const void* w_gate, const float* gate_scale, const void* w_up,
                              const float* up_scale, void* h, float* scale, void* workspace,
                              size_t workspace_bytes, void* stream);

/* Per-kernel timing, for measurement tools (off by default). While enabled, each kernel
 * launch of the calls above is bracketed by two HIP events recorded on the call's stream
 * (this adds a few microseconds per launch). gdn_profile_read waits for the recorded
 * events, writes up to max_entries per-kernel totals (kernel name, launches, total
 * milliseconds) and clears them; it returns the number of entries written, or -1 on a
 * HIP error. The state is process-wide and guarded by a mutex. */
typedef struct gdn_kernel_time {
    char name[32];
    int64_t launches;
    double total_ms;
} gdn_kernel_time;

gdn_status gdn_profile_enable(int enable);
int gdn_profile_read(gdn_kernel_time* out, int max_entries);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H_ */
