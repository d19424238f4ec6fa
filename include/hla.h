/*
 * hla.h -- C ABI of libhla.so: the Gated DeltaNet + HLA hot path on MI355X (gfx950).
 *
 * Sources, cited by page title and section:
 *   [HLA]  "HLA: Expressive Hybrid Linear Attention via Chunk-Wise Dynamic Mixing"
 *          (ai.info AI-summary page): Overview, Key Contributions, Methodology in Plain
 *          English paragraphs 1-4, Authors' abstract.
 *   [TR]   Tail-Replay abstract (second abstract on the thelatestinai.com page listed
 *          under the same HLA title).
 *   The per-token update is the gated delta rule of Gated DeltaNet, the affine update
 *   [HLA] Methodology paragraph 1 describes in words:
 *       S_t = alpha_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,   o_t = S_t q_t.
 *
 * Orientation and layouts (all tensors dense, row-major, no hidden padding):
 *   - The math state S is [dv, dk]; the library stores M = S^T as [dk, dv] float32.
 *   - A chunk's exact affine map ([HLA] Methodology paragraph 1) S -> S A_c + B_c is
 *     stored in the state orientation as the pair (At, Bc) with
 *         M_end = At @ M_start + Bc,   At = A_c^T [dk, dk],   Bc = B_c^T [dk, dv].
 *   - Per-token inputs: q, k [B, ld_T, H, dk]; v [B, ld_T, H, dv]; beta, alpha
 *     [B, ld_T, H] float32, with beta in [0, 1] and alpha in [0, 1] (alpha = 0 clears the
 *     state: the chunk kernels take log alpha clamped at float32's smallest normal).  Only tokens [0, T) of each batch row are read, so a suffix
 *     view (Tail-Replay) passes base pointers offset to the suffix start and ld_T = the
 *     allocated row length.
 *   - Chunk c covers tokens [c C, min((c + 1) C, T)); N = ceil(T / C); the last chunk may
 *     be partial and its transition is the product over its own tokens.
 *   - q, k, v, reps and the transitions use the call's dtype (float32 or bfloat16);
 *     states, outputs, gates and every accumulation are float32.
 *
 * Conventions for every entry point:
 *   - Pointers are device pointers unless marked "host".  Base pointers of tensors moved in
 *     16-byte vectors (q, k, v and reps of the prefill calls, transitions, states, chunk
 *     inits, caches and the workspace) must be 16-byte aligned; per-token scalars (beta,
 *     alpha), gates, counts, element-wise outputs (o) and the decode token vectors (bf16 ones
 *     too) need 4-byte alignment.  The caller allocates and owns every buffer, including the
 *     workspace; the library never allocates or frees device memory and keeps no pointer after
 *     return.
 *   - Calls only enqueue work on `stream`; nothing synchronises.  Calls that overlap on
 *     the same buffers race; calls on separate buffers are independent and reentrant.
 *   - Arguments are validated before anything is enqueued.  On an error the call returns a
 *     non-zero status and enqueues nothing.  A failed launch returns HLA_ERR_HIP.
 *     Asynchronous device faults surface at the caller's next synchronisation.
 *   - Every output element is overwritten, so results never depend on prior contents.
 */
#ifndef HLA_H_
#define HLA_H_

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define HLA_ABI_VERSION 7

typedef enum { HLA_F32 = 0, HLA_BF16 = 1 } hla_dtype_t;

typedef enum {
  HLA_OK = 0,
  HLA_ERR_NULL_ARG = 1,     /* a required pointer is NULL                              */
  HLA_ERR_BAD_SHAPE = 2,    /* a size is out of range or inconsistent                  */
  HLA_ERR_BAD_DTYPE = 3,    /* dtype is not HLA_F32 / HLA_BF16                         */
  HLA_ERR_WORKSPACE = 4,    /* workspace missing or smaller than hla_workspace_bytes() */
  HLA_ERR_HIP = 5,          /* a kernel launch failed                                  */
  HLA_ERR_UNSUPPORTED = 6,  /* a valid but unsupported combination of arguments        */
  HLA_ERR_ALIGN = 7,        /* a base pointer is not 16-byte aligned                   */
  HLA_ERR_INTERNAL = 8,     /* an unexpected host-side failure                         */
  HLA_ERR_SCRATCH_LIMIT = 9 /* a no-allocation call exceeds its fixed device scratch    */
} hla_status_t;

/* Problem sizes.  B batch rows, T tokens processed per row, H heads, ld_T >= T tokens
 * allocated per row; dk, dv in {64, 128}; C in {64, 128, 256} tokens per chunk (C > 64
 * needs dtype HLA_BF16, else HLA_ERR_UNSUPPORTED).  The kernels work on 64-token pieces;
 * a chunk of C tokens is C / 64 consecutive pieces, and its map is their composition. */
typedef struct {
  int64_t B, T, H, ld_T;
  int32_t dk, dv, C;
  int32_t dtype; /* hla_dtype_t */
} hla_dims_t;

/* Which entry point a workspace size is asked for (hla_workspace_bytes). */
typedef enum {
  HLA_FN_CHUNK_TRANSITIONS = 0,
  HLA_FN_GDN_PREFILL = 1,
  HLA_FN_ROUTE_MIX = 2,
  HLA_FN_WU_HANDOFF = 3, /* size of the optional wu buffer of hla_chunk_transitions and
                            hla_gdn_prefill: B H ceil(T / 64) 64 (dk + dv) bf16 values;
                            0 for float32, which takes no hand-off */
  HLA_FN_CHUNK_REPS = 4, /* workspace of hla_chunk_reps; n_rep = C / window */
  HLA_FN_COMPOSE_BACKWARD = 5, /* workspace of hla_compose_backward (one pass) */
  HLA_FN_PREFILL_BACKWARD = 6, /* workspace of hla_prefill_backward (one pass) */
  HLA_FN_CHUNK_BACKWARD = 7,   /* workspace of hla_chunk_backward */
  HLA_FN_COMPOSE_BACKWARD_MIN = 8, /* smallest workspace hla_compose_backward accepts */
  HLA_FN_PREFILL_BACKWARD_MIN = 9, /* smallest workspace hla_prefill_backward accepts */
  HLA_FN_GDN2_CHUNK_BACKWARD = 10, /* workspace of hla_gdn2_chunk_backward */
  HLA_FN_GDN2_PREFILL_BACKWARD = 11, /* workspace of hla_gdn2_prefill_backward (one pass) */
  HLA_FN_GDN2_PREFILL_BACKWARD_MIN = 12, /* smallest workspace hla_gdn2_prefill_backward accepts */
  HLA_FN_ROUTER_BACKWARD = 13,   /* workspace of hla_router_backward */
  HLA_FN_CHUNK_REPS_BACKWARD = 14 /* workspace of hla_chunk_reps_backward; n_rep says whether Wr
                                     is given (0: no, 1: yes) */
} hla_fn_t;

/*
 * hla_chunk_transitions -- the exact affine map of every chunk.
 * [HLA] Methodology paragraph 1 (affine maps compose, so a chunk is summarised exactly by
 * one affine map) and Key Contributions 2 (exact chunk-wise affine transitions).
 * Computed per (b, h, chunk) through the UT form of the chunk: the strictly lower matrix
 * diag(beta)(K K^T o decay) is inverted per chunk instead of running the token loop.
 *   k, v, beta, alpha : inputs as in the header notes (q is not needed).
 *   At [B, H, N, dk, dk], Bc [B, H, N, dk, dv] (out, dtype): M_end = At M_start + Bc.
 *   wu     (out, optional, bf16 only): a buffer of at least
 *           hla_workspace_bytes(HLA_FN_WU_HANDOFF) bytes (B H ceil(T / 64) 64 (dk + dv)
 *           bf16 values; the call has no size argument for it, so a smaller buffer is
 *           written past its end), or NULL.  Receives, for every 64-token piece, the
 *           UT-transformed keys and values W = X diag(beta gamma) K and U = X diag(beta) V
 *           (X the inverted strictly lower part plus identity) in the library's own
 *           fragment order, so that hla_gdn_prefill on the same inputs can take them
 *           instead of recomputing the inverse.  The layout is private to this library version.  A non-NULL wu
 *           with float32 inputs is HLA_ERR_UNSUPPORTED.
 *   ws, ws_bytes: workspace of at least hla_workspace_bytes(HLA_FN_CHUNK_TRANSITIONS)
 *           bytes (zero for C = 64; for C > 64 it holds the maps of the 64-token pieces,
 *           which are then composed C / 64 at a time: [HLA] Methodology paragraph 1).
 * Errors: HLA_ERR_NULL_ARG, HLA_ERR_BAD_SHAPE, HLA_ERR_BAD_DTYPE, HLA_ERR_ALIGN,
 *         HLA_ERR_WORKSPACE, HLA_ERR_UNSUPPORTED, HLA_ERR_HIP.
 */
hla_status_t hla_chunk_transitions(const hla_dims_t* d, const void* k, const void* v,
                                   const float* beta, const float* alpha, void* At, void* Bc,
                                   void* wu, void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * hla_gdn_prefill -- chunkwise Gated DeltaNet prefill.
 * [HLA] Methodology paragraph 1 (the per-token affine recurrence and its chunk form);
 * [TR] (state rebuild by replaying a suffix from a zero state: pass o = NULL).
 * Modes:
 *   native  (chunk_init == NULL): states run through the chunks in order starting from S0
 *           (NULL = zero state); o_t = S_t q_t; S_final = state after token T-1.
 *   routed  (chunk_init != NULL): chunk c starts from chunk_init[b, h, c] (the routed
 *           states of hla_route_mix; the current chunk has weight one, [HLA]
 *           Methodology paragraph 3); no state is carried between chunks.  S0 and S_final
 *           must be NULL.
 *   state-only (o == NULL): only S_final is produced; q may be NULL (Tail-Replay).
 *   q, k, v, beta, alpha : per-token inputs.
 *   S0         [B, H, dk, dv] float32 or NULL.
 *   chunk_init [B, H, N, dk, dv] float32 or NULL.
 *   wu         (optional, bf16 only): a buffer of hla_workspace_bytes(HLA_FN_WU_HANDOFF)
 *           bytes that hla_chunk_transitions filled from the same k, v, beta, alpha and
 *           dims, or NULL.  Given, the routed output pass reads W and U from it instead
 *           of recomputing them; results are identical.  The native bf16 prefill forms
 *           W and U inside its single pass and does not read it.
 *   o          [B, T, H, dv] float32 (out) or NULL.
 *   S_final    [B, H, dk, dv] float32 (out) or NULL.  At least one of o, S_final.
 *   ws, ws_bytes: workspace of at least hla_workspace_bytes(HLA_FN_GDN_PREFILL) bytes
 *           (none in routed mode with C = 64; in routed mode with C > 64 every chunk's
 *           64-token pieces start from states scanned from its routed state).  The
 *           native outputs do not depend on C: the prefill runs on 64-token pieces.
 * Native mode with bf16 inputs and outputs runs in two passes and never forms the chunk
 * maps (a state-only call scans the chunk maps instead): a parallel pass writes every
 * piece's UT products (-W, U^T, the log decays and (Q K^T) o decay: B H ceil(T / 64)
 * (128 (dk + dv) + 8448) bytes of the workspace), then one workgroup per (b, h, 32 state
 * columns) carries the state through the pieces in order, forming each piece's outputs
 * and next state on the way; no state goes through HBM.
 * Errors: as hla_chunk_transitions, plus HLA_ERR_WORKSPACE, HLA_ERR_UNSUPPORTED.
 */
hla_status_t hla_gdn_prefill(const hla_dims_t* d, const void* q, const void* k, const void* v,
                             const float* beta, const float* alpha, const float* S0,
                             const float* chunk_init, const void* wu, float* o, float* S_final,
                             void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * hla_gdn2_chunk_transitions, hla_gdn2_prefill -- the same two calls for the Gated
 * DeltaNet-2 recurrence.
 * [GDN2] the Gated DeltaNet-2 abstract (thelatestinai.com pages): channel-wise decay, a
 * channel-wise erase gate on the key side and a channel-wise write gate on the value side;
 * with one scalar for both gates it is Kimi Delta Attention, and with a scalar decay too,
 * Gated DeltaNet.  The formula taken here (the pages print none): with the math state S
 * [dv, dk], each token does
 *     S' = S diag(a_t),   S = S' - (S' k_t)(b_t o k_t)^T + (w_t o v_t) k_t^T,   o_t = S q_t.
 * Each token is affine in S, so each chunk is one exact affine map and hla_route_mix
 * composes these maps exactly as it composes Gated DeltaNet's ([HLA] Methodology
 * paragraph 1).
 *   a_decay [B, ld_T, H, dk], b_erase [B, ld_T, H, dk], w_write [B, ld_T, H, dv]: float32
 *           per-token gates (4-byte aligned) in place of beta and alpha.
 *   Every other argument, output, mode, workspace size and error is as for
 *           hla_chunk_transitions and hla_gdn_prefill, which have no wu argument here (the
 *           W | U hand-off belongs to Gated DeltaNet's UT form).
 * With bf16 inputs the chunk pass runs the chunkwise WY form on the matrix cores (every
 * per-channel decay factor it forms is taken against a reference token of its 16 x 16
 * block, and log a_t is floored at -11 per token); with float32 inputs it runs each
 * 64-token piece's tokens in float32 on the vector units.
 */
hla_status_t hla_gdn2_chunk_transitions(const hla_dims_t* d, const void* k, const void* v,
                                        const float* a_decay, const float* b_erase,
                                        const float* w_write, void* At, void* Bc, void* ws,
                                        size_t ws_bytes, hipStream_t stream);
hla_status_t hla_gdn2_prefill(const hla_dims_t* d, const void* q, const void* k, const void* v,
                              const float* a_decay, const float* b_erase, const float* w_write,
                              const float* S0, const float* chunk_init, float* o, float* S_final,
                              void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * hla_chunk_reps -- learned representatives of every chunk.
 * [HLA] Methodology paragraph 2: each chunk is cut into pooling windows of `window`
 * consecutive tokens; one-head self-attention runs inside every window over its keys
 * (scores scaled by 1/sqrt(dk), every token sees the whole window), the token outputs are
 * mean-pooled and a learned projection gives one representative per window.  The router's
 * learned query projection Wr is folded in: the output row is r' = Wr^T Wp pooled, so
 * hla_route_mix and hla_gdn_decode, which score the plain query q against r', compute
 * (Wr q) . (Wp pooled).  A window cut by the end of the sequence pools the tokens it has;
 * a window with no tokens gets a zero row.
 *   k      : [B, ld_T, H, dk] keys (dims d; dv is not used).
 *   window : 8, 16, 32 or 64 tokens (C / window representatives per chunk).
 *   Wq, Wk, Wv, Wp : [dk, dk] weights in the dims' dtype, row-major [out, in] (a row
 *           vector x maps to W x); head h's matrices start w_hstride elements after head
 *           h-1's (w_hstride = 0: one set shared by all heads; else >= dk*dk).
 *   Wr     : [dk, dk] query projection [out, in], same head stride, or NULL (identity).
 *   reps   : [B, N * (C / window), H, dk] (out, dtype): chunk j's representatives are rows
 *           [j n_rep, (j + 1) n_rep) with n_rep = C / window -- the reps argument of
 *           hla_route_mix with that n_rep and ld_R = N n_rep.
 *   ws, ws_bytes: workspace of at least hla_workspace_bytes(HLA_FN_CHUNK_REPS, d,
 *           C / window) bytes (float32 window means).
 * Errors: HLA_ERR_NULL_ARG, HLA_ERR_BAD_SHAPE (window, w_hstride), HLA_ERR_BAD_DTYPE,
 *         HLA_ERR_ALIGN (every pointer 16-byte aligned, head strides 16-byte multiples),
 *         HLA_ERR_WORKSPACE, HLA_ERR_UNSUPPORTED, HLA_ERR_HIP.
 */
hla_status_t hla_chunk_reps(const hla_dims_t* d, const void* k, int32_t window, const void* Wq,
                            const void* Wk, const void* Wv, const void* Wp, const void* Wr,
                            int64_t w_hstride, void* reps, void* ws, size_t ws_bytes,
                            hipStream_t stream);

/*
 * hla_chunk_reps_noalloc -- hla_chunk_reps for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid allocation).
 * Same arguments, kernels and results as hla_chunk_reps, without ws and ws_bytes: the
 * float32 window means live in a fixed device array of 32 MiB (HLA_REPS_SCRATCH_BYTES)
 * that the library holds on every GPU it runs on until the process ends; the call itself
 * allocates nothing.  It holds B H ceil(T / C) (C / window) dk float32 values, so at
 * dk = 128 up to 65536 (batch row, head, representative) rows.
 * Every call on a GPU shares that GPU's array: calls that overlap on one GPU (other
 * streams, other host threads) race and must be serialised by the caller.
 * Errors: as hla_chunk_reps, and HLA_ERR_SCRATCH_LIMIT (returned before anything reaches
 * the GPU) when the problem needs more than the fixed array.
 */
#define HLA_REPS_SCRATCH_BYTES ((size_t)32 << 20)
hla_status_t hla_chunk_reps_noalloc(const hla_dims_t* d, const void* k, int32_t window, const void* Wq,
                                    const void* Wk, const void* Wv, const void* Wp, const void* Wr,
                                    int64_t w_hstride, void* reps, hipStream_t stream);

/*
 * hla_route_mix -- HLA router gates and the gated composition of chunk transitions.
 * [HLA] Overview (log-mean-exp pooled routing gates), Methodology paragraphs 2-4,
 * Key Contributions 3 and the abstract (effective support):
 *   qbar_i   = mean of q over query chunk i's tokens;
 *   l_ij     = log( (1/n_rep) sum_r exp(qbar_i . r / sqrt(dk)) ) over chunk j's
 *              representatives r;  g_ij = sigmoid(l_ij) for j < i (independent gates);
 *   g_ii = 1 (current chunk), g_ij = 0 for j > i (future masked);
 *   mask_ij  = (j < i) and (g_ij >= tau)   [skip below tau without renormalisation,
 *              decided in float32];  ghat = g * mask;
 *   n_eff_i  = (sum_j ghat_ij)^2 / sum_j ghat_ij^2 over j < i (0 when all are skipped);
 *   S~_i     = chronological composition over j < i with mask_ij of
 *              M -> M + ghat_ij (At_j M + Bc_j - M), starting from S0 (NULL = zero).
 *   q          per-token queries (read only when gates_in == NULL).
 *   reps       [B, ld_R, H, dk] (dtype): chunk j's representatives are rows
 *              [j n_rep, (j + 1) n_rep); rows are read for j < N - 1 only, so
 *              ld_R >= (N - 1) n_rep.  Passing k with n_rep = C, ld_R = ld_T uses the
 *              chunk's raw keys.
 *   At, Bc     [B, H, N, dk, dk] / [B, H, N, dk, dv] (dtype), from hla_chunk_transitions.
 *   gates_in   [B, H, N, N] float32 caller gates (entries j < i are read) or NULL.
 *   gates      [B, H, N, N] float32 out (full matrix, diagonal 1, upper 0).
 *   mask       [B, H, N, N] uint8 out (1 = composed).
 *   active_idx [B, H, N, N] int32 out: ascending j with mask_ij, then -1.
 *   active_cnt [B, H, N] int32 out.   n_eff [B, H, N] float32 out or NULL.
 *   S_routed   [B, H, N, dk, dv] float32 out.
 *   ws, ws_bytes: workspace of at least hla_workspace_bytes(HLA_FN_ROUTE_MIX) bytes (the
 *              query-chunk means and, for bf16, reordered copies of At - I and of Bc for
 *              the composition).
 * Errors: as hla_gdn_prefill.
 */
hla_status_t hla_route_mix(const hla_dims_t* d, const void* q, const void* reps, int32_t n_rep,
                           int64_t ld_R, const void* At, const void* Bc, const float* S0,
                           const float* gates_in, float tau, float* gates, uint8_t* mask,
                           int32_t* active_idx, int32_t* active_cnt, float* n_eff,
                           float* S_routed, void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * hla_gdn_decode -- one single-token decode step for Bs sequences x H heads.
 * [HLA] Key Contributions 3 (dynamic autoregressive decoding) with Methodology
 * paragraphs 2-4.  Per (sequence b, head h):
 *   live chunk : S_cur (= M of the tokens since the last cached chunk) and its
 *                transition At_cur are extended by this token:
 *                M <- alpha (I - beta k k^T) M + beta k v^T,  At <- alpha (I - beta k k^T) At.
 *   gates      : g_j = sigmoid(log-mean-exp_r (q . r / sqrt(dk))) over cached chunk j's
 *                representatives, using the token's own q (or gates_in);
 *                ghat_j = g_j if g_j >= tau else 0.
 *   output     : o = (S~ A_cur + B_cur) q in math orientation, where S~ composes the
 *                gated cached chunks j < n_cache[b] from zero in time order.
 *   native     : At_cur == NULL: S_cur is the full-prefix state and o = S_cur^T q.
 *   q, k [Bs, H, dk], v [Bs, H, dv] (dtype); beta, alpha [Bs, H] float32.
 *   S_cur   [Bs, H, dk, dv] float32 in/out.   At_cur [Bs, H, dk, dk] float32 in/out or NULL.
 *   At_cache [Bs, H, n_cap, dk, dk], Bc_cache [Bs, H, n_cap, dk, dv] (dtype) in/out.
 *   reps_cache [Bs, H, n_cap, n_rep, dk] (dtype); may be NULL when gates_in is given.
 *   n_cache [Bs] int32 in/out (device): cached chunks per sequence; values above n_cap
 *           are clamped to n_cap.
 *   gates_in [Bs, H, n_cap] float32 or NULL;  gates_out [Bs, H, n_cap] float32 or NULL
 *           (entries j >= n_cache[b] are written as 0).
 *   o [Bs, H, dv] float32 out.
 *   commit: 1 = after the step append (At_cur, S_cur), cast to dtype, at slot n_cache[b],
 *           reset At_cur = I, S_cur = 0 and increment n_cache[b].  A full cache
 *           (n_cache[b] == n_cap) is left unchanged.  The caller writes that chunk's
 *           representatives.
 * Errors: HLA_ERR_NULL_ARG, HLA_ERR_BAD_SHAPE, HLA_ERR_BAD_DTYPE, HLA_ERR_ALIGN, HLA_ERR_HIP.
 */
hla_status_t hla_gdn_decode(int64_t Bs, int64_t H, int32_t dk, int32_t dv, int32_t dtype,
                            const void* q, const void* k, const void* v, const float* beta,
                            const float* alpha, float* S_cur, float* At_cur, void* At_cache,
                            void* Bc_cache, const void* reps_cache, int32_t n_rep,
                            int32_t* n_cache, int32_t n_cap, const float* gates_in, float tau,
                            float* o, float* gates_out, int32_t commit, hipStream_t stream);

/*
 * hla_gdn2_decode -- hla_gdn_decode for the Gated DeltaNet-2 recurrence ([GDN2] abstract):
 * a_decay, b_erase [Bs, H, dk] and w_write [Bs, H, dv] (float32, 4-byte aligned) replace
 * beta and alpha; the live chunk takes the token as in hla_gdn2_prefill,
 *     S_cur <- S_cur diag(a) (I - k (b o k)^T) + (w o v) k^T,   A_cur likewise with no write,
 * and the gates, the routed read over the cache and commit are hla_gdn_decode's.  Every
 * other argument and error is as for hla_gdn_decode.
 */
hla_status_t hla_gdn2_decode(int64_t Bs, int64_t H, int32_t dk, int32_t dv, int32_t dtype,
                             const void* q, const void* k, const void* v, const float* a_decay,
                             const float* b_erase, const float* w_write, float* S_cur,
                             float* At_cur, void* At_cache, void* Bc_cache, const void* reps_cache,
                             int32_t n_rep, int32_t* n_cache, int32_t n_cap, const float* gates_in,
                             float tau, float* o, float* gates_out, int32_t commit,
                             hipStream_t stream);

/*
 * The chunk cache in 8 bits: what a decoding program keeps of the prefix, per (sequence,
 * head), at about half the bytes of a bfloat16 cache, with a set of chunks of its own for
 * every head.  [HLA] Methodology paragraphs 1 and 2 (each chunk's exact affine map, scored by
 * its representatives).
 *   maps   [Bs, H, n_cap, dk + dv, dk]  8 bits, math orientation: rows 0 .. dk-1 hold A - I,
 *           rows dk .. dk+dv-1 hold B (S -> S A + B; A - I and not A, so that a chunk that
 *           changes little costs little precision and a skipped one none).
 *   reps   [Bs, H, n_cap, n_rep, dk]  8 bits: the representatives; NULL when n_rep is 0.
 *   scale  [Bs, H, n_cap, 4]  float32: the factors of A - I, of B and of the
 *           representatives, and 0.  The value of a stored number x is x * scale.
 *   order  [Bs, H, n_cap]  int32: the slot of every position in time; a permutation of
 *           0 .. n_cap-1, the positions from count on naming the free slots.  A slot out of
 *           range is read as the last one.
 *   count  [Bs, H]  int32: chunks held (positions 0 .. count-1), read as clamped to
 *           0 .. n_cap.
 *   weight [Bs, H, n_cap]  float32 by position: the sum of the gates that a chunk was read
 *           with, each taken within [0, 1]; or NULL, then nothing is accumulated.
 * Sizes: dk, dv in {64, 128}, 1 <= n_cap <= 1024, 0 <= n_rep <= 256.  maps, reps and scale are
 * 16-byte aligned, the others 4-byte.  Slots that no position below count names may hold
 * anything.  A call on a cache races with any other call that writes the same cache.
 */
typedef enum { HLA_CACHE_I8 = 0, HLA_CACHE_E4M3 = 1 } hla_cache8_format_t;
typedef struct {
  int64_t Bs, H;
  int32_t dk, dv, n_cap, n_rep;
  int32_t format; /* hla_cache8_format_t */
  void* maps;
  void* reps;
  float* scale;
  int32_t* order;
  int32_t* count;
  float* weight;
} hla_cache8_t;

/*
 * hla_cache8_append -- quantise chunks and append them to the cache.
 * Of each of X = A - I, X = B and X = the representatives of one chunk and head, with m the
 * largest |X| and Q = 127 (int8) or 448 (e4m3): scale = m (1 / Q), and X ((1 / m) Q) is rounded
 * to the nearest stored value, ties to even, every operation in float32; m < 2^-100 stores
 * zeros with scale 0.  An X with a NaN or an infinity stores zeros with scale NaN: a decode that
 * reads the chunk gives NaN (of representatives its gate is NaN, which is below every threshold).
 *   At [Bs, H, ld_src, dk, dk], Bc [Bs, H, ld_src, dk, dv] (dtype): maps as
 *           hla_chunk_transitions writes them, the first n_src of each row being complete
 *           chunks (0 <= n_src <= ld_src; a partial last chunk is not appended); or with
 *           n_src = ld_src = 1 the live chunk of a decode step (At_cur, S_cur).
 *   reps    [Bs, ld_R, H, dk] (dtype): source chunk i's representatives are rows
 *           [i n_rep, (i + 1) n_rep), ld_R >= n_src n_rep (hla_chunk_reps' output, or k with
 *           n_rep = C); ignored when the cache holds none.
 *   src     [Bs, H, ld_src] int32 or NULL: the source chunk of every appended one (clamped to
 *           0 .. n_src-1; NULL: chunk i is source chunk i).
 *   n_new   [Bs, H] int32 or NULL (n_src): chunks to append, clamped to 0 .. n_src and to the
 *           room left; the chunks past the room are dropped.
 *   weight_in [Bs, H, ld_src] float32 or NULL (zeros): the appended chunks' weights.
 *   reset   : 1 = the cache is emptied first (count 0, slots in order, weights 0).
 *   reset_live : 1 = the source maps of every chunk that was appended are set to A = I, B = 0
 *           (a live chunk begins again); needs HLA_F32 and src = NULL, else HLA_ERR_UNSUPPORTED.
 * Errors: HLA_ERR_NULL_ARG, HLA_ERR_BAD_SHAPE, HLA_ERR_BAD_DTYPE (dtype, format),
 *         HLA_ERR_ALIGN (At, Bc, reps 16 bytes), HLA_ERR_UNSUPPORTED, HLA_ERR_HIP.
 */
hla_status_t hla_cache8_append(const hla_cache8_t* c, int32_t dtype, int32_t n_src, int32_t ld_src,
                               void* At, void* Bc, const void* reps, int64_t ld_R, const int32_t* src,
                               const int32_t* n_new, const float* weight_in, int32_t reset,
                               int32_t reset_live, hipStream_t stream);

/*
 * hla_gdn_decode8, hla_gdn2_decode8 -- hla_gdn_decode and hla_gdn2_decode over the 8-bit
 * cache: the same live update, gates and composition, on the values the cache stands for
 * (float32 accumulation; the stored numbers enter exactly).
 *   q, k, v and the token gates, S_cur, At_cur (both required, updated in place), tau: as
 *           there, with Bs, H, dk and dv of the cache and every head's own count and order.
 *   gates_in  [Bs, H, n_cap] float32 by position or NULL (then n_rep >= 1).
 *   gates_out [Bs, H, n_cap] float32 or NULL: every held position's gate, 0 behind them.
 *   o         [Bs, H, dv] float32 out.
 *   The cache is read; its weight (if any) gains every held position's gate after the
 *   threshold.  A gate that is NaN is below every threshold.
 *   The vectors that meet the chunks are q (for the gates) and At_cur^T q as the chunks pass it
 *   on.  Over int8 chunks they enter as fixed point, to 2^-22 of the vector's largest magnitude (of
 *   the one before the last chunk, where that chunk shrank it), so that a row of a map that reads
 *   only the smallest elements sees them coarsely; they hold values below 2^127, and a larger one
 *   makes the gates, or o, NaN.  Over e4m3 chunks they enter as float32; a sum over values of 2^112
 *   and above may pass float32's range and is then not finite.
 *   ws, ws_bytes: workspace of at least hla_decode8_workspace_bytes() bytes, 16-byte aligned
 *           (0 but for few rows with a long cache, whose positions are cut into segments: then
 *           mostly a float32 dk x dk matrix a segment, the product of up to 64 neighbouring
 *           chunks' gated maps, which has to lie in float32's range; a call with gates_in may
 *           leave it unused).  It belongs to one call at a time.
 * Appending the live chunk is hla_cache8_append's (reset_live).
 * Errors: HLA_ERR_NULL_ARG, HLA_ERR_BAD_SHAPE, HLA_ERR_BAD_DTYPE, HLA_ERR_ALIGN,
 *         HLA_ERR_WORKSPACE, HLA_ERR_HIP.
 */
hla_status_t hla_gdn_decode8(const hla_cache8_t* c, int32_t dtype, const void* q, const void* k,
                             const void* v, const float* beta, const float* alpha, float* S_cur,
                             float* At_cur, const float* gates_in, float tau, float* o,
                             float* gates_out, void* ws, size_t ws_bytes, hipStream_t stream);
hla_status_t hla_gdn2_decode8(const hla_cache8_t* c, int32_t dtype, const void* q, const void* k,
                              const void* v, const float* a_decay, const float* b_erase,
                              const float* w_write, float* S_cur, float* At_cur,
                              const float* gates_in, float tau, float* o, float* gates_out, void* ws,
                              size_t ws_bytes, hipStream_t stream);
hla_status_t hla_decode8_workspace_bytes(const hla_cache8_t* c, size_t* out);

/*
 * hla_gate_weights -- the weight that a prefill's gates give every chunk: the sum of the gates
 * that the prompt's own later query chunks read it with, one for each query chunk (a decode step
 * adds one for each token: times C the two are in one unit).
 *     weight[b, h, j] = sum over j < i < n_b of g_ij [g_ij >= tau], g taken within [0, 1]
 *   gates    [B, H, N, N] float32 as hla_route_mix writes them (entries j < i count).
 *   n_chunks [B] int32 or NULL (N): valid chunks n_b, clamped to 0 .. N.
 *   weight   [B, H, N] float32 out (0 at and behind the last valid chunk).
 * Sums are float32 in a fixed order.
 * Errors: HLA_ERR_NULL_ARG, HLA_ERR_BAD_SHAPE (sizes, NaN tau), HLA_ERR_ALIGN, HLA_ERR_HIP.
 */
hla_status_t hla_gate_weights(int64_t B, int64_t H, int32_t N, const float* gates, const int32_t* n_chunks,
                              float tau, float* weight, hipStream_t stream);

/*
 * hla_evict_chunks -- cut every row's chunks to a budget by accumulated weight.
 * With n_h = count (clamped to 0 .. n) and m = max(n_h - budget, 0): of the positions
 * [0, n_h - n_recent) the m with the lowest weight leave (of equal weights the older first; NaN
 * is below every number); the others keep their order in time.
 *   weight [Bs, H, n], order [Bs, H, n] (NULL: position p is slot p), count [Bs, H]: as in the
 *           cache, or of a prompt's chunks (hla_gate_weights), whose `order_out` is then the
 *           src of hla_cache8_append.  1 <= n <= 16384; 0 <= n_recent <= budget.
 *   order_out  : the slots that stay, in time order, then those that left, then (unmoved) the
 *           positions from count on.   weight_out: likewise, 0 behind the chunks that stay.
 *   count_out  : min(count, budget).
 * Outputs may be the inputs of the same kind (in place); no other overlap.
 * Errors: HLA_ERR_NULL_ARG, HLA_ERR_BAD_SHAPE, HLA_ERR_ALIGN, HLA_ERR_HIP.
 */
hla_status_t hla_evict_chunks(int64_t Bs, int64_t H, int32_t n, const float* weight, const int32_t* order,
                              const int32_t* count, int32_t budget, int32_t n_recent, int32_t* order_out,
                              float* weight_out, int32_t* count_out, hipStream_t stream);

/*
 * hla_compose_backward -- reverse of the gated composition of hla_route_mix.
 * [HLA] Methodology paragraphs 1, 3 and 4.  Query chunk i's routed state is the chain
 *     M_j = M_{j-1} + g_ij (At_j - I) M_{j-1} + g_ij Bc_j    over active j < i, M = S0 first,
 * and given lambda = dL/dS~_i (stored orientation) the reverse of every step is
 *     dBc_j += g lambda_j,  dAt_j += g lambda_j M_{j-1}^T,
 *     dg_ij = <lambda_j, (At_j - I) M_{j-1} + Bc_j>,  lambda_{j-1} = lambda_j + g (At_j - I)^T lambda_j.
 * Skipped pairs (mask 0) pass lambda unchanged and get dg = 0 (the skip is a step function
 * of g with zero derivative).
 *   At, Bc     [B, H, N, dk, dk] / [B, H, N, dk, dv] (dtype), as given to hla_route_mix.
 *   gates, mask [B, H, N, N] float32 / uint8, as hla_route_mix wrote them (entries j < i
 *              are read).
 *   S0         [B, H, dk, dv] float32 or NULL (zero).
 *   dS_routed  [B, H, N, dk, dv] float32: upstream gradient of S_routed.
 *   dAt, dBc   out [B, H, N, dk, dk] / [B, H, N, dk, dv] float32.
 *   dgates     out [B, H, N, N] float32: dL/dg_ij for active j < i, 0 elsewhere.
 *   dS0        out [B, H, dk, dv] float32, or NULL.
 *   S_routed   out [B, H, N, dk, dv] float32 (the routed states, recomputed), or NULL.
 *   ws, ws_bytes: workspace: (At - I), its transpose and Bc reordered for the matrix
 *              cores, and slots for the state in front of an active step, (At_j - I) M
 *              + Bc_j and g lambda (dtype, dk x dv each) of the pairs whose step j lies in
 *              one segment of K consecutive history steps, plus float32 checkpoints of
 *              every chain's state at each segment boundary it crosses.  The call takes
 *              the longest segments the workspace holds and runs them last to first, each
 *              chain's steps of a segment replayed from its checkpoint.  With
 *              hla_workspace_bytes(HLA_FN_COMPOSE_BACKWARD) bytes K = N: one segment,
 *              every pair j < i has its slots (N (N - 1) / 2 per (b, h), so it grows as
 *              N^2) and there is no checkpoint.  Any size down to
 *              hla_workspace_bytes(HLA_FN_COMPOSE_BACKWARD_MIN) (the segment length that
 *              needs least, about K (N - 1) slots and N^2 / (2 K) checkpoints per (b, h))
 *              works too.  float32 maps: the checkpoints come from the call's own replay
 *              and results are bit-identical to one segment's; bf16 maps: they come from
 *              the bf16 composition of hla_route_mix (several chains share each staged
 *              map), whose rounding differs, and results agree to bf16 rounding.
 * Computation: bf16 (or float32) matrix-core products with float32 accumulation; sums in a
 * fixed order (deterministic).
 * Errors: HLA_ERR_NULL_ARG, HLA_ERR_BAD_SHAPE, HLA_ERR_BAD_DTYPE, HLA_ERR_ALIGN,
 * HLA_ERR_WORKSPACE, HLA_ERR_HIP.
 */
hla_status_t hla_compose_backward(const hla_dims_t* d, const void* At, const void* Bc,
                                  const float* gates, const uint8_t* mask, const float* S0,
                                  const float* dS_routed, float* dAt, float* dBc, float* dgates,
                                  float* dS0, float* S_routed, void* ws, size_t ws_bytes,
                                  hipStream_t stream);

/*
 * hla_chunk_backward -- reverse of the per-chunk work (64-token chunks, C = 64):
 *   outputs part: the routed outputs of hla_gdn_prefill with chunk_init (every chunk's
 *     tokens run by the gated delta rule from its own start state, o_t = S_t q_t);
 *   map part: the chunk maps (At, Bc) of hla_chunk_transitions ([HLA] Methodology
 *     paragraph 1: the product of the per-token linear parts, and the state from zero).
 * Every state column follows x <- alpha (x - beta k (k . x)) + beta k u on its own; the
 * reverse of one token with dx = dL/dx after it is b = k . dx, dv[col] += beta b,
 * dbeta += b (u - alpha k . x_prev), dalpha += dx . x_prev - beta (k . x_prev) b,
 * dk += beta u dx - alpha beta ((k . x_prev) dx + b x_prev), dx <- alpha (dx - beta k b).
 *   q, k, v, beta, alpha: as for hla_gdn_prefill (q is read by the outputs part only).
 *   chunk_init [B, H, N, dk, dv] float32 and dO [B, T, H, dv] float32: both or neither
 *              (outputs part).
 *   dAt [B, H, N, dk, dk], dBc [B, H, N, dk, dv] float32: both or neither (map part).
 *   dq, dk [B, T, H, dk], dv [B, T, H, dv], dbeta, dalpha [B, T, H]: float32 outputs, the
 *              sum of both parts (dq is zero without the outputs part).
 *   dchunk_init [B, H, N, dk, dv] float32 out (required with the outputs part).
 *   ws, ws_bytes: workspace of at least hla_workspace_bytes(HLA_FN_CHUNK_BACKWARD) bytes
 *              (per-workgroup partial sums).
 * Arithmetic is float32 throughout; partial sums are added in a fixed order.
 * Errors: HLA_ERR_NULL_ARG (no part, or a missing output), HLA_ERR_UNSUPPORTED (C != 64),
 * and as hla_gdn_prefill.
 */
hla_status_t hla_chunk_backward(const hla_dims_t* d, const void* q, const void* k, const void* v,
                                const float* beta, const float* alpha, const float* chunk_init,
                                const float* dO, const float* dAt, const float* dBc, float* dq,
                                float* dk, float* dv, float* dbeta, float* dalpha,
                                float* dchunk_init, void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * hla_prefill_backward -- gradients of the routed prefill (raw-key representatives, C = 64).
 * Given dO = dL/do for the outputs of hla_chunk_transitions + hla_route_mix (reps = k,
 * n_rep = 64) + hla_gdn_prefill with chunk_init = S_routed, the call recomputes that
 * forward and returns dL/d(q, k, v, beta, alpha), dL/dS0 and dL/dg for the history gates:
 *   the outputs part of hla_chunk_backward (dS~ and the chunk-local gradients);
 *   hla_compose_backward (dAt, dBc, dgates, dS0);
 *   the maps part of hla_chunk_backward;
 *   the router ([HLA] Overview, Methodology paragraph 2): dl_ij = dg_ij g_ij (1 - g_ij),
 *     p_ijr = softmax over chunk j's keys of qbar_i . k_r / sqrt(dk),
 *     dqbar_i = sum_j dl_ij sum_r p_ijr k_r / sqrt(dk) (spread as dqbar_i / n_i over chunk
 *     i's tokens), dk_r += sum_i dl_ij p_ijr qbar_i / sqrt(dk);
 * then the per-token sums.  The skip mask is a step function of g: a skipped pair passes
 * no gradient.  With gates_in the gates are the caller's: dgates is the gradient w.r.t.
 * them and the router takes no part.
 *   q, k, v, beta, alpha, S0, gates_in, tau: as for the forward calls.
 *   dO [B, T, H, dv] float32.
 *   dq, dk [B, T, H, dk], dv [B, T, H, dv], dbeta, dalpha [B, T, H]: float32 out.
 *   dS0 [B, H, dk, dv] float32 out or NULL;  dgates [B, H, N, N] float32 out or NULL.
 *   ws, ws_bytes: workspace; it holds the composition backward's per-pair states.  With
 *              hla_workspace_bytes(HLA_FN_PREFILL_BACKWARD) bytes (growing as N^2 dk dv
 *              per (b, h)) every chunk pair has its slots; any size down to
 *              hla_workspace_bytes(HLA_FN_PREFILL_BACKWARD_MIN) runs the composition's
 *              history steps in segments replayed from checkpoints, as for
 *              hla_compose_backward.
 * Errors: HLA_ERR_UNSUPPORTED (C != 64) and as hla_gdn_prefill.
 */
hla_status_t hla_prefill_backward(const hla_dims_t* d, const void* q, const void* k, const void* v,
                                  const float* beta, const float* alpha, const float* S0,
                                  const float* gates_in, float tau, const float* dO, float* dq,
                                  float* dk, float* dv, float* dbeta, float* dalpha, float* dS0,
                                  float* dgates, void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * hla_gdn2_chunk_backward, hla_gdn2_prefill_backward -- hla_chunk_backward and
 * hla_prefill_backward for the Gated DeltaNet-2 recurrence (the formula of
 * hla_gdn2_chunk_transitions: S' = S diag(a_t), S = S' - (S' k_t)(b_t o k_t)^T +
 * (w_t o v_t) k_t^T, o_t = S q_t; [GDN2] the Gated DeltaNet-2 abstract).  The per-token
 * gates a_decay, b_erase [B, ld_T, H, dk] and w_write [B, ld_T, H, dv] (float32) take the
 * place of alpha and beta, and their gradients da, db [B, T, H, dk] and dw [B, T, H, dv]
 * (float32 out) the place of dalpha and dbeta.  The reverse of a chunk runs token by token
 * per state column in float32, from the state in front of every 8-token block: per token
 *     du = k . dx,  dp = -(b o k) . dx,  dv[col] += w[col] du,  dw[col] += v[col] du,
 *     dk += dx o (u - b p) + dp x',  db += -p k o dx,  dx' = dx + dp k,  da += dx' o x,
 *     dx <- a o dx'
 * (x the column before the token, x' = a o x, p = k . x', u = w[col] v[col]).  The
 * routed prefill's router, composition and their reverses are those of
 * hla_prefill_backward, unchanged.  Every other argument, output, mode, workspace rule
 * (HLA_FN_GDN2_CHUNK_BACKWARD, HLA_FN_GDN2_PREFILL_BACKWARD, down to
 * HLA_FN_GDN2_PREFILL_BACKWARD_MIN with history segments) and error is as for the Gated
 * DeltaNet calls.
 */
hla_status_t hla_gdn2_chunk_backward(const hla_dims_t* d, const void* q, const void* k, const void* v,
                                     const float* a_decay, const float* b_erase, const float* w_write,
                                     const float* chunk_init, const float* dO, const float* dAt,
                                     const float* dBc, float* dq, float* dk, float* dv, float* da,
                                     float* db, float* dw, float* dchunk_init, void* ws,
                                     size_t ws_bytes, hipStream_t stream);
hla_status_t hla_gdn2_prefill_backward(const hla_dims_t* d, const void* q, const void* k, const void* v,
                                       const float* a_decay, const float* b_erase,
                                       const float* w_write, const float* S0, const float* gates_in,
                                       float tau, const float* dO, float* dq, float* dk, float* dv,
                                       float* da, float* db, float* dw, float* dS0, float* dgates,
                                       void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * hla_router_backward -- gradients of the history gates to the queries and to the
 * representatives (learned ones, or the raw keys), for callers that compose the learned-
 * representative backward themselves: hla_prefill_backward with the forward's gates as
 * gates_in returns dgates; this call takes them on to dq and dreps, and
 * hla_chunk_reps_backward takes dreps on to the keys and the pooler's weights.
 * [HLA] Overview, Methodology paragraph 2: with qbar_i the mean of q over chunk i,
 * s_ijr = qbar_i . r_{j n_rep + r} / sqrt(dk), g_ij = sigmoid(log-mean-exp_r s_ijr):
 *     dl_ij = dg_ij g_ij (1 - g_ij),  p_ijr = softmax_r s_ijr,
 *     dq_t = (1 / n_i) sum_{j<i} dl_ij sum_r p_ijr r_{j n_rep + r} / sqrt(dk)  (t in chunk i),
 *     dr_{j n_rep + r} = sum_{i>j} dl_ij p_ijr qbar_i / sqrt(dk).
 *   d      : dims (C = 64).
 *   q      : [B, ld_T, H, dk] (dtype);  reps: [B, ld_R, H, dk] (dtype), chunk j's rows
 *           [j n_rep, (j + 1) n_rep), 1 <= n_rep <= 64, ld_R >= (N - 1) n_rep.
 *   gates, dgates : [B, H, N, N] float32: the gates hla_route_mix wrote and their gradient
 *           (entries j < i are read; a skipped pair's gradient is zero).
 *   dq     : [B, T, H, dk] float32 out (the router's part of the query gradient).
 *   dreps  : [B, N n_rep, H, dk] float32 out (the last chunk's rows are zero).
 *   ws, ws_bytes : hla_workspace_bytes(HLA_FN_ROUTER_BACKWARD) bytes.
 * Errors: HLA_ERR_NULL_ARG, HLA_ERR_BAD_SHAPE (n_rep, ld_R), HLA_ERR_ALIGN (q, reps, ws
 *         16 bytes; the float32 arrays 4), HLA_ERR_WORKSPACE, HLA_ERR_UNSUPPORTED (C != 64),
 *         HLA_ERR_HIP.
 */
hla_status_t hla_router_backward(const hla_dims_t* d, const void* q, const void* reps, int32_t n_rep,
                                 int64_t ld_R, const float* gates, const float* dgates, float* dq,
                                 float* dreps, void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * hla_chunk_reps_backward -- reverse of hla_chunk_reps: from dreps, the gradient of every
 * representative row, the gradients of the keys and of the weights.
 * [HLA] Methodology paragraph 2 (the forward of hla_chunk_reps).  Per window of n >= 1
 * tokens X, with P the window's attention, c_s its column sums, m = (1/n) sum_s c_s V_s
 * and z = Wp m:
 *     dz = Wr dr (dr without Wr),  dWr += z dr^T,  dm = Wp^T dz,  dWp += dz m^T,
 *     dV_s = c_s dm / n,  e_s = V_s . dm / n,  dS_ts = P_ts (e_s - sum_s' P_ts' e_s'),
 *     dQ = dS K / sqrt(dk),  dK = dS^T Q / sqrt(dk),
 *     dX = dQ Wq + dK Wk + dV Wv,  dWq += dQ^T X,  dWk += dK^T X,  dWv += dV^T X;
 * an empty window passes nothing.  The weight gradients sum over every window of every
 * batch row (and head, with shared weights) in a fixed order.
 *   k, window, Wq, Wk, Wv, Wp, Wr, w_hstride : as for hla_chunk_reps (C a multiple of 64).
 *   dreps  : [B, N (C / window), H, dk] float32, rows as hla_chunk_reps writes them.
 *   dk     : [B, T, H, dk] float32 out.
 *   dWq, dWk, dWv, dWp : [Hw, dk, dk] float32 out, Hw = H (w_hstride != 0) or 1 (shared),
 *           each head's matrix dk * dk elements after the previous one.
 *   dWr    : same, out; required exactly when Wr is given.
 *   ws, ws_bytes : hla_workspace_bytes(HLA_FN_CHUNK_REPS_BACKWARD, d, Wr ? 1 : 0) bytes
 *           (dWq, dWk and dWv of every 8 consecutive 64-token tiles, and four dk-vectors per
 *           window).
 * Errors: as hla_chunk_reps, and HLA_ERR_UNSUPPORTED (C not a multiple of 64).
 */
hla_status_t hla_chunk_reps_backward(const hla_dims_t* d, const void* k, int32_t window, const void* Wq,
                                     const void* Wk, const void* Wv, const void* Wp, const void* Wr,
                                     int64_t w_hstride, const float* dreps, float* dk, float* dWq,
                                     float* dWk, float* dWv, float* dWp, float* dWr, void* ws,
                                     size_t ws_bytes, hipStream_t stream);

/*
 * Linear attention with a decay for each head: the additive recurrence without the delta rule's
 * erase, which hybrid models mix with it.  Per (batch row, head), M [dk, dv] in float32:
 *     M_t = exp(g_t) M_{t-1} + k_t v_t^T,     o_t = M_t^T q_t        (S = M^T in math orientation)
 *   q, k      [B, ld_T, Hk, dk], v [B, ld_T, H, dv] (dtype); Hk divides H, and value heads
 *             h = i H/Hk .. (i + 1) H/Hk - 1 share query and key head i.  q is not scaled.
 *   log_decay g <= 0, float32: [B, ld_T, H] (decay_per_head = 0) or [H] (1).  A decay below float32's
 *             smallest normal number (g below -87.33, -inf included) is zero and clears the state;
 *             so does the product of a piece's decays where it falls below.
 *   lens      [B] int32 or NULL (T): tokens of each row, clamped to 0 .. T.  Tokens behind a row's
 *             length are not read; outputs and gradients there are zero.  Where every row is full NULL is
 *             faster: with lengths, rows are cut into segments for a batch of which some end early.
 *   sizes     dk, dv 64 or 128; H <= 65536, B H < 2^23, T <= 2^35.
 * S_final may be S0's own buffer, and no other output may overlap an input or another output.
 * dtype is that of q, k, v, o and of their gradients; states, log_decay and their gradients are
 * float32.  Arithmetic: float32 sums, sums of log_decay in float64.  Over bf16 tensors what is float32
 * enters the matrix cores as bf16 terms: three (24 bits) where the result is float32, two (2^-16)
 * where it is rounded to bf16.  A number that is not finite spreads over its own piece (64 tokens of
 * bf16, 32 of float32), to earlier tokens of the piece too.  Sums have a fixed order: a call repeats
 * its bits.
 */
typedef struct {
  int64_t B, T, H, Hk, ld_T;
  int32_t dk, dv, dtype, decay_per_head;
} hla_la_dims_t;
typedef enum { HLA_LA_PREFILL = 0, HLA_LA_PREFILL_BACKWARD = 1 } hla_la_fn_t;

/*
 * hla_la_prefill -- the chunked form over a prompt.
 *   S0       [B, H, dk, dv] float32 or NULL (zero).
 *   o        [B, T, H, dv] (dtype, out) or NULL;  S_final [B, H, dk, dv] float32 (out) or NULL: the
 *            state behind every row's last token.  At least one; q may be NULL without o.
 *   ws       hla_la_workspace_bytes(HLA_LA_PREFILL) bytes: the states in front of the segments that
 *            long rows are cut into where there are few rows (0 otherwise).
 * Errors: HLA_ERR_NULL_ARG, HLA_ERR_BAD_SHAPE, HLA_ERR_BAD_DTYPE, HLA_ERR_ALIGN (log_decay and lens
 *         4 bytes, the others 16), HLA_ERR_WORKSPACE, HLA_ERR_HIP.
 */
hla_status_t hla_la_prefill(const hla_la_dims_t* d, const void* q, const void* k, const void* v,
                            const float* log_decay, const int32_t* lens, const float* S0, void* o,
                            float* S_final, void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * hla_la_prefill_backward -- gradients of hla_la_prefill, for dO = dL/do and dS_final = dL/dS_final.
 * With G_t = exp(g_{t+1}) G_{t+1} + q_t dO_t^T (dS_final behind the last token):
 *     dq_t = M_t dO_t,  dk_t = G_t v_t,  dv_t = G_t^T k_t,  dg_t = exp(g_t) <G_t, M_{t-1}>,
 *     dS0 = exp(g_1) G_1; shared heads' dq and dk and a head's one dg are sums.
 * dg is the gradient of log_decay; it is 0 where a decay clears the state.  It is formed from sums over
 * tokens: its error is that of a float32 sum of the magnitudes k_j . dk_j and q_j . dq_j over the tokens
 * in front of t's piece and in it, or behind and in it, whichever is less (so a token far from every loss
 * has an error as small as its gradient); dg of one decay a head is the sum of these values, with their errors.
 *   dO [B, T, H, dv] (dtype);  dS_final [B, H, dk, dv] float32 or NULL (zero).
 *   dq, dk [B, T, Hk, dk], dv [B, T, H, dv] (dtype, out);  dlog_decay [B, T, H] or [H] float32 (out);
 *   dS0 [B, H, dk, dv] float32 (out) or NULL.
 *   ws hla_la_workspace_bytes(HLA_LA_PREFILL_BACKWARD) bytes.
 * Errors: as hla_la_prefill.
 */
hla_status_t hla_la_prefill_backward(const hla_la_dims_t* d, const void* q, const void* k, const void* v,
                                     const float* log_decay, const int32_t* lens, const float* S0,
                                     const void* dO, const float* dS_final, void* dq, void* dk, void* dv,
                                     float* dlog_decay, float* dS0, void* ws, size_t ws_bytes,
                                     hipStream_t stream);
hla_status_t hla_la_workspace_bytes(int32_t fn, const hla_la_dims_t* d, size_t* out);

/*
 * hla_la_decode -- one token of Bs sequences: S [Bs, H, dk, dv] float32 is updated in place and read.
 *   q, k [Bs, Hk, dk], v [Bs, H, dv] (dtype, 4-byte aligned);  log_decay [Bs, H] or [H] float32;
 *   o [Bs, H, dv] (dtype, out, 4-byte aligned).  S is 16-byte aligned.
 * Errors: HLA_ERR_NULL_ARG, HLA_ERR_BAD_SHAPE, HLA_ERR_BAD_DTYPE, HLA_ERR_ALIGN, HLA_ERR_HIP.
 */
hla_status_t hla_la_decode(int64_t Bs, int64_t H, int64_t Hk, int32_t dk, int32_t dv, int32_t dtype,
                           const void* q, const void* k, const void* v, const float* log_decay,
                           int32_t decay_per_head, float* S, void* o, hipStream_t stream);

/*
 * Trees of drafted tokens (speculative decoding) over the state of hla_gdn_decode.  A sequence drafts
 * up to n <= 64 tokens that form a tree; node i continues its parent's state by the gated delta rule
 * (the live state for parent -1), and each is answered as hla_gdn_decode would answer it after its own
 * ancestors.  hla_gdn_tree_decode answers all nodes and changes nothing; hla_gdn_tree_accept lets the
 * path to an accepted node into the live state.
 *   parent [Bs, n] int32 (device): -1 <= parent[i] < i.  Any other value (as -2 for the places behind a
 *          smaller tree) marks node i absent, and so are the nodes below it: their inputs are not used,
 *          their outputs and gates are zero.
 *   q, k [Bs, n, H, dk], v [Bs, n, H, dv] (dtype);  beta, alpha [Bs, n, H] float32, alpha >= 0.
 *   S_cur, At_cur, At_cache, Bc_cache, reps_cache, n_rep, n_cache, n_cap, tau: as for hla_gdn_decode;
 *          n_cap <= 1024.  At_cur = NULL: no cache is read, what belongs to it (gates_in too) is not used,
 *          and there are no gates: gates_out must be NULL.
 * q, k, v, o and the caches and live matrices are 16-byte aligned, the others 4-byte.
 */

/*
 * hla_gdn_tree_decode
 *   gates_in  [Bs, n, H, n_cap] float32 or NULL (then n_rep >= 1): every node's own gates.
 *   o         [Bs, n, H, dv] float32 out.
 *   gates_out [Bs, n, H, n_cap] float32 out or NULL: the gates in front of the threshold, 0 from
 *             n_cache[b] on and at absent nodes.
 *   ws        hla_gdn_tree_workspace_bytes() bytes (0 without At_cur, n_cap = 0), 16-byte aligned, for one
 *             call at a time.
 * Every chunk that any node reads is read once for all of them.  A NaN gate is below every threshold.
 * float32 accumulation; over bf16 maps z enters as three bf16 terms (24 bits).
 * Errors: HLA_ERR_NULL_ARG, HLA_ERR_BAD_SHAPE (sizes, NaN tau), HLA_ERR_BAD_DTYPE, HLA_ERR_ALIGN,
 *         HLA_ERR_WORKSPACE, HLA_ERR_HIP.
 */
hla_status_t hla_gdn_tree_decode(int64_t Bs, int64_t H, int32_t n, int32_t dk, int32_t dv, int32_t dtype,
                                 const void* q, const void* k, const void* v, const float* beta,
                                 const float* alpha, const int32_t* parent, const float* S_cur,
                                 const float* At_cur, const void* At_cache, const void* Bc_cache,
                                 const void* reps_cache, int32_t n_rep, const int32_t* n_cache,
                                 int32_t n_cap, const float* gates_in, float tau, float* o,
                                 float* gates_out, void* ws, size_t ws_bytes, hipStream_t stream);
hla_status_t hla_gdn_tree_workspace_bytes(int64_t Bs, int64_t H, int32_t n, int32_t dk, int32_t dv,
                                          int32_t n_cap, size_t* out);

/*
 * hla_gdn_tree_accept
 *   node   [Bs] int32 (device): the accepted node, whose ancestors and itself enter S_cur (and At_cur)
 *          in order; an absent or out-of-range one (-1): none.
 *   commit [Bs] int32 (device) or NULL: where not 0, the live chunk is appended afterwards at slot
 *          n_cache[b] (cast to dtype), At_cur is reset to I and S_cur to 0 and n_cache[b] advances, as
 *          hla_gdn_decode's commit; a sequence whose cache is full is left as it is.  Needs At_cur and
 *          the cache.
 * Errors: HLA_ERR_NULL_ARG, HLA_ERR_BAD_SHAPE, HLA_ERR_BAD_DTYPE, HLA_ERR_ALIGN, HLA_ERR_HIP.
 */
hla_status_t hla_gdn_tree_accept(int64_t Bs, int64_t H, int32_t n, int32_t dk, int32_t dv, int32_t dtype,
                                 const void* k, const void* v, const float* beta, const float* alpha,
                                 const int32_t* parent, const int32_t* node, float* S_cur, float* At_cur,
                                 void* At_cache, void* Bc_cache, int32_t* n_cache, int32_t n_cap,
                                 const int32_t* commit, hipStream_t stream);

/* Workspace bytes that entry point `fn` needs for dims `d`; n_rep is the number of
 * representatives per chunk for HLA_FN_CHUNK_REPS (C / window; it must divide C), whether
 * Wr is given (0 or 1) for HLA_FN_CHUNK_REPS_BACKWARD, and ignored otherwise.  `out` is a
 * host pointer. */
hla_status_t hla_workspace_bytes(int32_t fn, const hla_dims_t* d, int32_t n_rep, size_t* out);

/* Kernel kinds that hla_timing_read() reports. */
typedef enum {
  HLA_KERNEL_CHUNK = 0,    /* per-chunk UT kernel (transitions, chunk outputs)        */
  HLA_KERNEL_SCAN = 1,     /* sequential chunk scan of the native prefill             */
  HLA_KERNEL_GATES = 2,    /* router: query-chunk means, gate scores, mask and lists  */
  HLA_KERNEL_COMPOSE = 3,  /* gated composition of chunk transitions                  */
  HLA_KERNEL_DECODE = 4,   /* single-token decode step                                */
  HLA_KERNEL_REPS = 5,     /* learned representatives: window attention and mean-pool */
  HLA_KERNEL_BWD_SAVE = 6,    /* backward: composition replay that keeps the step states */
  HLA_KERNEL_BWD_ADJOINT = 7, /* backward: adjoint sweep of every composition chain     */
  HLA_KERNEL_BWD_REDUCE = 8,  /* backward: per-history-chunk sums (dAt, dBc, gates, dS0)  */
  HLA_KERNEL_BWD_CHUNK = 9,   /* backward: per-chunk reverse token recurrence            */
  HLA_KERNEL_BWD_ROUTER = 10, /* backward: router gates to queries and keys              */
  HLA_KERNEL_PREFILL = 11,    /* one-pass native prefill (bf16): UT, outputs, state scan */
  HLA_KERNEL_BWD_REPS = 12,   /* backward: learned representatives (tiles and reduction)  */
  HLA_KERNEL_LA = 13,         /* linear attention: a prompt's passes, or one token        */
  HLA_KERNEL_BWD_LA = 14,     /* backward: linear attention, all passes of a call         */
  HLA_KERNEL_TREE = 15,       /* trees of drafted tokens: answering them, or accepting    */
  HLA_KERNEL_COUNT = 16
} hla_kernel_t;

/*
 * Optional per-kernel timing (profiling aid; off by default).  hla_timing_enable(1) clears
 * earlier records and starts bracketing every launch of the kernels above with two HIP
 * events recorded on that launch's own stream; hla_timing_enable(0) stops and clears.
 * hla_timing_read() waits for the recorded events of one kernel kind and returns the
 * summed elapsed milliseconds and the number of launches (host pointers).  These two
 * calls are the one exception to the no-global-state convention above: the switch and the
 * event records are process-global (host memory and HIP events, never device buffers), so
 * enable timing only while one thread issues work.  With timing off no entry point reads
 * or writes that state.
 */
hla_status_t hla_timing_enable(int32_t on);
hla_status_t hla_timing_read(int32_t which, double* total_ms, int64_t* launches);

/* Static description of a status code (never NULL). */
const char* hla_status_string(int32_t status);

/* HLA_ABI_VERSION of the loaded library. */
int32_t hla_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* HLA_H_ */
