/*
 * gdn.h -- C ABI of the chunked gated delta rule (GDN) prefill library for NVIDIA GB300
 * (sm_103a).
 *
 * The operation (FlashQLA pages: agentlenshq "GDN chunked prefill optimisation" and the
 * aisparkup "usage" section, which gives the high-level call
 * chunk_gated_delta_rule(q, k, v, g, beta, scale, initial_state, output_final_state,
 * cu_seqlens) -> (o, final_state) and the low-level forward/backward entry points):
 *
 *   per sequence, per v-head j (q/k head j / G, G = Hv / Hqk), state S_t in R^{V x K}:
 *     S_t = exp(g_t) S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T
 *     o_t = scale * S_t q_t
 *   S_0 = initial state (zero when absent); the final state is S after the last token.
 *
 * States cross this ABI transposed, as h = S^T stored [K][V] (row-major, V fastest).
 *
 * Tensor layouts (row-major, contiguous; "T_total" = B*T, or T when varlen):
 *   q, k      [T_total, Hqk, K]   dtype (bf16 or fp32)
 *   v, o, dO  [T_total, Hv,  V]   dtype
 *   g, beta   [T_total, Hv]       fp32   (g: natural-log decay, beta: write strength)
 *   h0, ht, dht, dh0  [N_seq, Hv, K, V]  fp32
 *   dq, dk    like q;  dv like v;  dg, dbeta like g (fp32)
 *
 * Conventions, for every entry point:
 *   - Pointers are DEVICE pointers unless the field says host.  Every device pointer must
 *     be 16-byte aligned (an argument that may be less aligned says so).  The caller owns all memory; the library never allocates, frees
 *     or synchronises.  Work is enqueued on `stream` (a cudaStream_t; NULL = legacy stream)
 *     and runs asynchronously.
 *   - Arguments are validated before anything is launched; on a non-OK status nothing has
 *     been written and gdn_last_error() (thread-local) says why.
 *   - Results are deterministic: repeated calls give bitwise-identical outputs.
 *   - K = V = 128 only (GDN_ERR_UNSUPPORTED otherwise).
 *   - Stream order holds as for any launch.  Inside a call, kernels overlap their
 *     predecessors' ends by programmatic dependent launch, each waiting for its predecessor
 *     (griddepcontrol.wait) before it reads anything that one wrote; the library's kernels
 *     signal their dependents early, so a caller's kernel launched right after a call WITH
 *     programmatic stream serialisation must itself wait (cudaGridDependencySynchronize)
 *     before it reads the call's outputs.  Ordinary launches, copies and events need nothing.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GDN_OK = 0,
    GDN_ERR_INVALID_ARG = 1,   /* bad shape, pointer, alignment or cu_seqlens */
    GDN_ERR_UNSUPPORTED = 2,   /* valid but not implemented (e.g. K != 128) */
    GDN_ERR_WORKSPACE = 3,     /* workspace missing or smaller than the *_workspace_size */
    GDN_ERR_CUDA = 4,          /* a CUDA launch or attribute call failed */
    GDN_ERR_TIMEOUT = 5,       /* a device-side wait gave up (gdn_device_status) */
    GDN_ERR_BOUNDS = 6         /* checked build: a store index fell outside its tensor (gdn_device_status) */
} gdn_status;

/* GDN_E4M3 (8 bits: 1 sign, 4 exponent, 3 mantissa bits, no infinities) only where an entry
 * point names it: a paged cache, the output of gdn_rmsnorm_fwd. */
typedef enum { GDN_BF16 = 0, GDN_FP32 = 1, GDN_E4M3 = 2 } gdn_dtype;

/* Intra-GPU context parallelism over chunk ranges (FlashQLA pages, "AutoCP" section: when
 * batch * heads leaves SMs idle, each sequence's chunks are split into segments). */
typedef enum {
    GDN_CP_AUTO = 0,    /* exact; the planner picks the segment length L: by default the L
                           that minimises a cost model of the launches on this GPU (waves of
                           one CTA per SM, chunk steps, fix-up steps); with cp_lambda > 0 the
                           pages' rule L = cp_lambda * sqrt(chunks) instead */
    GDN_CP_OFF = 1,     /* one segment per sequence: a plain serial chunk scan */
    GDN_CP_EXACT = 2,   /* segments of cp_segment_chunks chunks; transition fix-up, exact */
    GDN_CP_WARMUP = 3,  /* opt-in approximation: each segment starts warmup_chunks chunks
                           early from a zero state instead of the exact fix-up (FlashQLA
                           pages, "warm-up" paragraph: 6-8 chunks); NOT exact */
    GDN_CP_EXACT_FULL = 4 /* as GDN_CP_EXACT, with every segment's transition computed and
                           composed and every segment rerun from its entering state */
} gdn_cp_mode;

/* How the exact modes (AUTO, EXACT) skip work without changing the result.  Every chunk's
 * state transition X -> prod_t exp(g_t) (I - beta_t k_t k_t^T) X has 2-norm at most
 * B = exp(sum_t g_t) prod_t max(1, |1 - beta_t |k_t|^2|), computed per (chunk, v-head) from
 * the inputs (bf16 path).  Where the product of these bounds over a prefix of a segment falls
 * below 2^-126, the smallest normal fp32 number, whatever enters the segment changes the states
 * past that prefix by less than 2^-126 times its norm: the segment's transition is then not
 * computed (the fix-up takes the segment's state from zero as its result) and only the
 * prefix's outputs are recomputed from the true entering state.  Elsewhere the transition is
 * computed, composed and the whole segment rerun, as in GDN_CP_EXACT_FULL.  The fp32 test mode
 * always works as GDN_CP_EXACT_FULL. */

typedef struct gdn_problem {
    int32_t B;                        /* batch; must be 1 when cu_seqlens is given */
    int32_t T;                        /* tokens per sequence (total tokens when varlen) */
    int32_t Hqk;                      /* q/k heads */
    int32_t Hv;                       /* v heads; multiple of Hqk */
    int32_t K;                        /* key dim (128) */
    int32_t V;                        /* value dim (128) */
    int32_t dtype;                    /* gdn_dtype of q, k, v, o, dO, dq, dk, dv */
    float scale;                      /* output scale, finite and > 0 (GDN_ERR_INVALID_ARG
                                         otherwise); usually K^-0.5 */
    const int32_t* cu_seqlens;        /* device [num_seqs+1] or NULL (then B sequences of T) */
    const int32_t* cu_seqlens_host;   /* HOST copy with the same contents; required iff
                                         cu_seqlens != NULL (sizes the launch grids) */
    int32_t num_seqs;                 /* N_seq when varlen */
    int32_t cp_mode;                  /* gdn_cp_mode */
    int32_t cp_segment_chunks;        /* EXACT, EXACT_FULL, WARMUP: chunks per segment
                                         (0 = auto) */
    int32_t warmup_chunks;            /* WARMUP: warm-up chunks (0 = 8) */
    float cp_lambda;                  /* AUTO: lambda in L = lambda sqrt(N) (0 = cost model) */
} gdn_problem;

/* Bytes of device workspace gdn_chunk_fwd needs for *p (written to *bytes). */
gdn_status gdn_chunk_fwd_workspace_size(const gdn_problem* p, size_t* bytes);

/*
 * Forward (FlashQLA pages: the low-level forward of the aisparkup "usage" section; the
 * chunk-local prep, the chunk-serial state scan and the output stage of the agentlenshq
 * "GDN chunked prefill" section).
 *   h0  : initial states or NULL (zero).       o  : output, written for every token.
 *   ht  : final states or NULL (not returned).
 *   workspace: device scratch of at least gdn_chunk_fwd_workspace_size bytes (contents
 *   are overwritten; it may be reused across calls on the same stream).
 */
gdn_status gdn_chunk_fwd(const gdn_problem* p, const void* q, const void* k, const void* v,
                         const float* g, const float* beta, const float* h0, void* o,
                         float* ht, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of device workspace gdn_chunk_bwd needs for *p (written to *bytes). */
gdn_status gdn_chunk_bwd_workspace_size(const gdn_problem* p, size_t* bytes);

/*
 * Backward (FlashQLA pages, agentlenshq "backward pass" paragraph: the dv, dh-scan,
 * dq/dk/dw/dg and WY-backward steps).  Gradients of
 *   L = <o, dO> + <ht, dht>
 * with respect to q, k, v, g, beta and h0, for the forward defined above with the same
 * inputs.  The forward intermediates are recomputed from q, k, v, g, beta, h0.
 *   dht : NULL = zero.   dh0 : NULL = not returned.
 *   dq, dk are summed over the G v-heads that share each q/k head.
 *   Context parallelism in the backward is always exact (GDN_CP_WARMUP is treated as
 *   GDN_CP_EXACT here).
 */
gdn_status gdn_chunk_bwd(const gdn_problem* p, const void* q, const void* k, const void* v,
                         const float* g, const float* beta, const float* h0, const void* dO,
                         const float* dht, void* dq, void* dk, void* dv, float* dg,
                         float* dbeta, float* dh0, void* workspace, size_t workspace_bytes,
                         void* stream);

/* ------------------------------------------------------------------------------------
 * Low-level forward / backward pair with saved intermediates (FlashQLA pages, aisparkup
 * "usage" section: the low-level forward returns g, A, o, h and the final state, and the
 * backward is called separately).  The pages name the tuple but do not define its members;
 * this library reads them as
 *   g_cum : [T_total, Hv] fp32, gamma, the cumulative sum of g within each chunk (it restarts
 *           at every chunk start and at every sequence start);
 *   A     : [T_total, Hv, C] dtype, for every token its row of its chunk's
 *           T = (I + diag(beta) (K K^T * Dm))^-1 (unit lower triangular; Dm_ij =
 *           exp(gamma_i - gamma_j) for i > j, else 0); column i of a token's row refers to
 *           the chunk's i-th token, columns past the token's own position are 0;
 *   h     : [total_chunks, Hv, K, V] dtype, the state h = S^T entering every chunk, chunks
 *           numbered over all sequences in order (sequence s holds ceil(len_s / C) of them,
 *           its first one being h0, or 0).
 * C is the kernels' chunk size (64 for bf16, 32 in the fp32 test mode); gdn_chunk_layout
 * reports it and total_chunks.
 *
 * gdn_chunk_fwd_saved computes what gdn_chunk_fwd computes and also writes g_cum and A (when
 * non-NULL) and h (required).  It runs the backward's decomposition of the problem
 * (context parallelism is exact; GDN_CP_WARMUP is treated as GDN_CP_EXACT) and leaves in
 * the workspace the chunk records and segment transitions that the backward needs: the
 * workspace must hold gdn_chunk_bwd_workspace_size bytes.
 *
 * gdn_chunk_bwd_saved computes what gdn_chunk_bwd computes for the same inputs, without
 * recomputing the forward: it reads h and the workspace exactly as gdn_chunk_fwd_saved left
 * them for the same problem (the caller keeps both unchanged between the two calls, and
 * orders the calls, e.g. on one stream).  h0 is not needed (h holds it).  g_cum and A are
 * outputs only; the backward does not read them.
 * ------------------------------------------------------------------------------------ */
gdn_status gdn_chunk_layout(const gdn_problem* p, int32_t* chunk_size, int64_t* total_chunks);

gdn_status gdn_chunk_fwd_saved(const gdn_problem* p, const void* q, const void* k, const void* v,
                               const float* g, const float* beta, const float* h0, void* o,
                               float* ht, float* g_cum, void* A, void* h, void* workspace,
                               size_t workspace_bytes, void* stream);

gdn_status gdn_chunk_bwd_saved(const gdn_problem* p, const void* q, const void* k, const void* v,
                               const float* g, const float* beta, const void* h, const void* dO,
                               const float* dht, void* dq, void* dk, void* dv, float* dg,
                               float* dbeta, float* dh0, void* workspace, size_t workspace_bytes,
                               void* stream);

/* ------------------------------------------------------------------------------------
 * Fused prologue: the activations that turn a layer's raw projections into the inputs of
 * gdn_chunk_fwd, in one pass (read once, write once), and their reverse mode.  The FlashQLA
 * pages take q, k, g, beta as given (g a log-decay, beta a write strength, q and k the unit
 * keys of the delta rule) and do not say how they are formed; this library reads them as
 *   q = q_raw / sqrt(sum(q_raw^2) + 1e-6)  and  k likewise   (per token and q/k head, over K)
 *   g = -exp(A_log[j]) * softplus(a + dt_bias[j])           (per token and v-head j)
 *   beta = 1 / (1 + exp(-b))
 * with softplus(x) = log(1 + exp(x)) (x itself above 20).
 *
 * Shapes from *p (B, T or varlen total T, Hqk, Hv, K = 128, dtype; cu_seqlens unused):
 *   q_raw, k_raw, q, k, dq, dk, dq_raw, dk_raw   [T_total, Hqk, K]  dtype
 *   a, b, g, beta, dg, dbeta, da, db             [T_total, Hv]      fp32
 *   A_log, dt_bias, dA_log, ddt_bias             [Hv]               fp32
 * gdn_prologue_fwd may run in place (q == q_raw, k == k_raw, g == a, beta == b).
 * gdn_prologue_bwd takes dq, dk, dg, dbeta (the gradients gdn_chunk_bwd returns) and the
 * forward's raw inputs, and writes the gradients of L with respect to q_raw, k_raw, a, b,
 * A_log and dt_bias; dA_log and ddt_bias are sums over all tokens taken in a fixed order.
 * Its workspace (gdn_prologue_bwd_workspace_size bytes) holds per-head partial sums.
 * ------------------------------------------------------------------------------------ */
gdn_status gdn_prologue_fwd(const gdn_problem* p, const void* q_raw, const void* k_raw,
                            const float* a, const float* b, const float* A_log,
                            const float* dt_bias, void* q, void* k, float* g, float* beta,
                            void* stream);

gdn_status gdn_prologue_bwd_workspace_size(const gdn_problem* p, size_t* bytes);

gdn_status gdn_prologue_bwd(const gdn_problem* p, const void* q_raw, const void* k_raw,
                            const float* a, const float* b, const float* A_log,
                            const float* dt_bias, const void* dq, const void* dk,
                            const float* dg, const float* dbeta, void* dq_raw, void* dk_raw,
                            float* da, float* db, float* dA_log, float* ddt_bias,
                            void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------------------
 * Recurrent step: the gated delta rule one token after another, for decoding (one new token
 * per sequence, or the few drafted ones that a verification pass runs) from the states that a
 * prefill (gdn_chunk_fwd's ht) or an earlier step left.  Per sequence, v-head and token
 *     u = beta (v - e^g h^T k),   h <- e^g h + k u^T,   o = scale h^T q
 * which is the recurrence at the top of this file for h = S^T.  Arithmetic and states are fp32;
 * between a sequence's tokens the decay may be kept as a factor in [2^-20, 2^20] beside the state,
 * with u divided by it (to 2^-22 of u), multiplied out with the last token.
 *
 * The states live in pools [num_slots, Hv, K, V] fp32: sequence s reads slot slots[s] of
 * state_in (NULL: zero states) and writes the same slot of state_out (NULL: not returned).
 * state_out may be state_in (in place); the pools may not overlap otherwise.  Slots that no
 * sequence names are not touched.  A sequence whose slot lies outside [0, num_slots) (-1 for the
 * padding rows of a captured batch) reads and writes no state, and its o is 0.  No two
 * sequences of a call may name the same slot (their states would race).  A sequence without
 * tokens keeps its state (state_out gets a copy).
 *
 * With A_log and dt_bias given (both or neither), q and k are raw projections and g, beta the
 * pre-activations a, b of gdn_prologue_fwd, whose formulas are applied on the way in.
 *
 * cu_seqlens is read on the device alone, so a captured graph serves every split of
 * total_tokens; offsets outside [0, total_tokens] are clamped to it.  Tokens before the first
 * offset and from the last one on belong to no sequence: their o is left as it is, or set to 0
 * with clear_rest.  K = V = 128.
 * ------------------------------------------------------------------------------------ */
typedef struct gdn_step_problem {
    int32_t num_seqs;
    int32_t total_tokens;          /* rows of q, k, v, g, beta and o */
    int32_t Hqk, Hv, K, V;
    int32_t dtype;                 /* gdn_dtype of q, k, v and o (bf16 or fp32) */
    float scale;                   /* finite and > 0 */
    const int32_t* cu_seqlens;     /* device [num_seqs+1], or NULL: total_tokens / num_seqs each */
    const int32_t* slots;          /* device [num_seqs], or NULL: sequence s has slot s */
    int64_t num_slots;
    /* elements from one token's row to the next, 0 for contiguous rows; a row's heads and
     * features are contiguous.  Those of q, k, v are multiples of 16 bytes. */
    int64_t q_stride, k_stride, v_stride, g_stride, beta_stride;
    int32_t clear_rest;            /* not 0: o = 0 for tokens that no sequence covers */
} gdn_step_problem;

gdn_status gdn_recurrent_step(const gdn_step_problem* p, const void* q, const void* k,
                              const void* v, const float* g, const float* beta, /* g, beta: 4-byte aligned */
                              const float* A_log, const float* dt_bias, const float* state_in,
                              float* state_out, void* o, void* stream);

/* ------------------------------------------------------------------------------------
 * Attention of one new token per sequence over a paged key-value cache (the full-attention
 * layers of a model that interleaves them with gated-delta-rule layers).  Per sequence n and
 * query head h, with kv-head j = h / (Hq / Hkv) and the tokens t of [first, len),
 * len = seq_lens[n], first = max(0, len - window) (0 without a window):
 *     z_t = scale <q_h, k_t>,   o_h = sum_t softmax(z)_t v_t,   lse_h = log sum_t e^{z_t}
 * Token t of sequence n lies in slot t % page_size of page page_table[n][t / page_size].
 * lens count the new token: it attends to itself.
 *
 * k_new, v_new (both or neither): the new token's key and value, written by the call to
 * position len - 1 of the caches (divided by k_scale, v_scale and rounded to the cache's type;
 * in 8 bits clamped to +-448) and attended to as written.  No two sequences of such a call may
 * share the page of that position.
 * 8-bit caches hold k / k_scale[j] and v / v_scale[j]; NULL scales are 1.
 *
 * Scores, softmax statistics and sums are fp32.  With bf16 queries the weights e^{z - max} are
 * rounded to bf16 (8-bit caches: to fp16, as 2^14 e^{z - max}) for their product with v; the sum
 * that o is divided by, and lse, take them unrounded.  Under 8-bit caches a query value is the sum
 * of two 8-bit ones: exact down to 2^-9 of its row's largest, within 2^-18 of that one below.
 * Under fp32 caches nothing is rounded below fp32.
 *
 * A sequence of length 0 gets o = 0 and lse = -inf.  Whatever lies in slots outside
 * [first, len) is not used, NaN or not.  Page numbers outside [0, num_pages) are not read: the tokens of
 * such a page count as masked (and a new token there is not written); a length past
 * max_pages * page_size is cut to it (and its new token not written).
 *
 * Caches of any page size and strides; features contiguous; D = 64, 128 or 256.  Lengths, pages
 * and tables are read on the device alone, so a captured call serves other lengths; how the work
 * is divided follows from max_pages (a table no wider than the longest sequence may become is
 * best) and, on the device, from the lengths.  Partial results lie in the workspace (0 bytes where
 * none is needed) and are joined in a fixed order: the same lengths give the same bits.
 * ------------------------------------------------------------------------------------ */
typedef struct gdn_paged_problem {
    int32_t num_seqs;
    int32_t Hq, Hkv;               /* query heads, a multiple of the kv-heads */
    int32_t D;                     /* 64, 128 or 256 */
    int32_t dtype;                 /* gdn_dtype of q, k_new, v_new and o: bf16 or fp32 */
    int32_t cache_dtype;           /* bf16 or e4m3 with bf16 queries, fp32 with fp32 queries */
    float scale;                   /* finite and > 0 */
    int32_t window;                /* tokens attended to, 0 for all */
    int32_t page_size;             /* tokens per page */
    int32_t max_pages;             /* columns of page_table */
    int64_t num_pages;             /* pages in each cache */
    int64_t q_stride, new_stride;  /* elements between the rows of q, of k_new and v_new (0: contiguous) */
    int64_t table_stride;          /* elements between the rows of page_table (0: contiguous) */
    /* elements between pages, a page's tokens and a token's heads; multiples of 16 bytes */
    int64_t k_page_stride, k_token_stride, k_head_stride;
    int64_t v_page_stride, v_token_stride, v_head_stride;
} gdn_paged_problem;

gdn_status gdn_paged_attn_workspace_size(const gdn_paged_problem* p, size_t* bytes);

gdn_status gdn_paged_attn_decode(const gdn_paged_problem* p, const void* q, void* k_cache, void* v_cache,
                                 const int32_t* page_table, const int32_t* seq_lens, /* 4-byte aligned */
                                 const void* k_new, const void* v_new,
                                 const float* k_scale, const float* v_scale, /* [Hkv], 4-byte aligned */
                                 void* o, float* lse,  /* [num_seqs, Hq, D]; [num_seqs, Hq] or NULL */
                                 void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------------------
 * Root-mean-square norm with the residual's addition, optionally with an 8-bit output.  Per
 * row, with w = weight + weight_offset:
 *     s = x + residual (x itself without a residual),   r = 1 / sqrt(mean(s^2) + eps),
 *     y = r s w;   sum = s, rounded to dtype (y comes from the unrounded s)
 * With out_dtype GDN_E4M3, y / scale is rounded to nearest even in 8 bits, with one fp32 scale per
 * row (group = 0) or per `group` consecutive values of a row (y_scale [rows, dim / group]):
 *     scale = max(max |y| / 448, 2^-126)
 * Both quotients are products with reciprocals: the scale is within 2^-23 of max |y| / 448, and
 * y / scale within 2^-22 of itself before it is rounded, so that a value that near to the middle
 * between two 8-bit ones may get the other.
 * A row with infinities or NaN gets NaN in that row alone.
 * sum may be x or residual (in place), y of x's type may be x, where their rows are contiguous
 * like the output's; NULL sum: not returned.
 *
 * gdn_rmsnorm_bwd: the gradients of <y, dy> + <sum, dsum> (dsum NULL: 0) with respect to s
 * (x and residual alike) and to weight, for the s given:
 *     dx = r (w dy - n mean(w dy n)) + dsum with n = r s;   dweight = sum over rows of dy n
 * dweight is fp32, summed in a fixed order.  For an 8-bit y, dy is the gradient with respect to
 * y y_scale: the rounding passes it through.
 * dx may be dy or dsum (in place) where their rows are contiguous.
 *
 * Pointers and strides need only the alignment of their elements here; rows whose pointers and
 * strides are all multiples of 16 bytes run faster.
 * ------------------------------------------------------------------------------------ */
typedef struct gdn_norm_problem {
    int64_t rows;
    int32_t dim;
    int32_t dtype;                 /* gdn_dtype of x, residual, sum, dy, dsum, dx: bf16 or fp32 */
    int32_t weight_dtype;          /* bf16 or fp32 */
    int32_t out_dtype;             /* of y: dtype, or GDN_E4M3 */
    int32_t group;                 /* values to a scale; 0: a row; else divides dim */
    float eps;                     /* finite and >= 0 */
    float weight_offset;           /* 0, or 1 for weights that are kept as w - 1 */
    int64_t x_stride, residual_stride;  /* elements between rows (x_stride is s's in the backward), 0: dim */
    int64_t dy_stride, dsum_stride;
} gdn_norm_problem;

gdn_status gdn_rmsnorm_fwd(const gdn_norm_problem* p, const void* x, const void* residual,
                           const void* weight, void* y, float* y_scale, void* sum, void* stream);

gdn_status gdn_rmsnorm_bwd_workspace_size(const gdn_norm_problem* p, size_t* bytes);

gdn_status gdn_rmsnorm_bwd(const gdn_norm_problem* p, const void* s, const void* weight,
                           const void* dy, const void* dsum, void* dx, float* dweight,
                           void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------------------
 * Causal attention over whole prompts, and its gradient (the full-attention layers of a model that
 * interleaves them with gated-delta-rule layers).  Per sequence of Lq queries and Lk keys and query
 * head h, with kv-head j = h / (Hq / Hkv): query i stands at position i + Lk - Lq and attends to the
 * keys t of [max(0, position - window + 1), position] (from 0 without a window):
 *     z_it = scale <q_i, k_t>,   o_i = sum_t softmax(z_i)_t v_t,   lse_i = log sum_t e^{z_it}
 * Lk = Lq is a whole prompt; Lk > Lq its last part, the earlier keys given with it; with Lk < Lq the
 * first Lq - Lk queries see nothing.  A query that sees nothing gets o = 0, lse = -inf and no gradient.
 *
 *   q, o, dO, dq  [total_q, Hq, D]     k, v, dk, dv  [total_k, Hkv, D]     lse, dlse  [total_q, Hq] fp32
 * Sequences are packed: queries [cu_seqlens[n], cu_seqlens[n+1]), keys by cu_seqlens_k (NULL: by
 * cu_seqlens, with total_k = total_q); without cu_seqlens there are num_seqs of equal lengths.  Both are
 * read on the device alone, and cut to [0, total], so a captured call serves other lengths; sequences must
 * not overlap.  Nothing that this or a following entry point writes may overlap what it reads, unless it is the same
 * argument.  Rows that no sequence covers are left as they were (clear_rest = 0), or get o = 0, lse = -inf
 * and gradients of 0 (clear_rest = 1).  What lies there, NaN or not, is not used.
 *
 * gdn_prompt_attn_bwd: the gradients of <o, dO> + <lse, dlse> (dlse NULL: 0) with respect to q, k and v,
 * from the forward's o and lse; dk and dv are summed over the query heads that share a kv-head.  o_rest (bf16,
 * like o; NULL: none) is what rounding o left, itself rounded: with it <dO, o> has 16 bits of o instead of 8, and dq
 * and dk, whose terms all have that product in them, some 10 % less error.
 *
 * Scores, softmax statistics, sums and gradients are held in fp32.  With bf16 the weights e^{z - m} (m the
 * running maximum, or up to 8 log 2 below it) are rounded to bf16 for their product with v, while the sum
 * that o is divided by, and lse, take them unrounded; in the gradient, softmax(z) and the gradient of z are
 * rounded to bf16 for the products with dO, q and k.  With fp32 nothing is rounded below fp32.
 * A value v_t that is infinite or NaN reaches the queries that attend to t and no others.  In the gradient
 * such a value, or one in q, k, o or dO, may reach the other rows of its sequence within the same 128.
 * ------------------------------------------------------------------------------------ */
typedef struct gdn_prompt_problem {
    int32_t num_seqs;
    int32_t total_q, total_k;      /* rows of q and of k and v */
    int32_t Hq, Hkv;               /* query heads, a multiple of the kv-heads */
    int32_t D;                     /* 64, 128 or 256 */
    int32_t dtype;                 /* gdn_dtype of q, k, v, o and their gradients: bf16 or fp32 */
    float scale;                   /* finite and > 0 */
    int32_t window;                /* keys attended to, 0 for all */
    int32_t clear_rest;
    const int32_t* cu_seqlens;     /* device [num_seqs+1], or NULL; 4-byte aligned */
    const int32_t* cu_seqlens_k;
    /* elements from one token's row to the next, 0 for contiguous rows; a row's heads and features are
     * contiguous.  Multiples of 16 bytes. */
    int64_t q_stride, k_stride, v_stride;
} gdn_prompt_problem;

gdn_status gdn_prompt_attn_fwd(const gdn_prompt_problem* p, const void* q, const void* k, const void* v,
                               void* o, float* lse, void* o_rest, /* lse, o_rest NULL: not returned */
                               void* stream);

gdn_status gdn_prompt_attn_bwd_workspace_size(const gdn_prompt_problem* p, size_t* bytes);

gdn_status gdn_prompt_attn_bwd(const gdn_prompt_problem* p, const void* q, const void* k, const void* v,
                               const void* o, const float* lse, const void* o_rest, const void* dO,
                               const float* dlse, void* dq, void* dk, void* dv, void* workspace,
                               size_t workspace_bytes, void* stream);

/* Waits in the tensor-core kernels of the attention over prompts and of drafted trees are bounded like those
 * of the chunked rule (2 s; see "Device-side failure report"), but leave their mark in the library: this waits
 * for `stream` and returns GDN_OK, or GDN_ERR_TIMEOUT where a wait of such a call on the current device has given
 * up since it was last asked (that call's outputs are not valid).  Not to be called while a stream is captured. */
gdn_status gdn_attn_device_status(void* stream);

/* Test hook of that report: a wait that nothing ends gives up after limit_us microseconds (1 .. 1000000) and leaves the mark of
 * the kernels 0 (prompts forward), 1 (prompts backward), 2 (trees, bf16) or 3 (trees, 8 bits).  Asynchronous on `stream`. */
gdn_status gdn_debug_attn_wait_timeout(int32_t kernels, int32_t limit_us, void* stream);

/* ------------------------------------------------------------------------------------
 * Attention of a tree of drafted tokens over a paged key-value cache (their verification: all branches
 * in one call).  Sequence n has seq_lens[n] tokens in its pages, as in gdn_paged_attn_decode, but none of
 * the drafted ones, and up to T drafted tokens whose keys and values are k_new and v_new.  parents[n][t]
 * is the drafted token that t follows, below t; -1: t follows the cached tokens; anything else: there is
 * no token t (its o is 0, its lse -inf, and a token that follows it is none either).
 * Token t attends to the cached tokens, its ancestors and itself.  With a window it attends to positions above its own, seq_lens[n] +
 * (number of its ancestors), less window.
 * k_scale and v_scale are those of the cache; k_new and v_new are used as given.  Nothing is written to
 * the cache: the accepted tokens are by gdn_paged_cache_write.
 *
 * Types, scales, roundings, lengths past the table, page numbers out of range and slots without tokens: as
 * in gdn_paged_attn_decode, but that query values are not split under 8-bit caches (keys and values are widened to
 * bf16, exactly, and weights rounded to bf16), and that strides of bf16 and 8-bit caches are not 0 where there is more than
 * one page, token or head.  1 <= T <= 64.
 * ------------------------------------------------------------------------------------ */
typedef struct gdn_tree_problem {
    int32_t num_seqs;
    int32_t T;                     /* drafted tokens of a sequence, at most */
    int32_t Hq, Hkv, D;
    int32_t dtype, cache_dtype;
    float scale;
    int32_t window;
    int32_t page_size, max_pages;
    int64_t num_pages;
    int64_t q_stride, k_new_stride, v_new_stride; /* elements between tokens (0: contiguous), sequence n's at n T */
    int64_t table_stride;
    int64_t k_page_stride, k_token_stride, k_head_stride;
    int64_t v_page_stride, v_token_stride, v_head_stride;
} gdn_tree_problem;

gdn_status gdn_paged_attn_tree_workspace_size(const gdn_tree_problem* p, size_t* bytes);

gdn_status gdn_paged_attn_tree(const gdn_tree_problem* p, const void* q, const void* k_new, const void* v_new,
                               const void* k_cache, const void* v_cache, const int32_t* page_table,
                               const int32_t* seq_lens, const int32_t* parents, /* [num_seqs, T] */
                               const float* k_scale, const float* v_scale, void* o, /* [num_seqs, T, Hq, D] */
                               float* lse, /* [num_seqs, T, Hq] or NULL */
                               void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------------------
 * Keys and values into a paged cache.  For i < count, row rows[i] (i itself where rows is NULL) of k and v
 * goes to slot slots[i] % page_size of page slots[i] / page_size, as k / k_scale[j] and v / v_scale[j] rounded
 * to the cache's type (in 8 bits clamped to +-448, NaN kept; NULL scales: 1).  Slots outside
 * [0, num_pages page_size) and rows outside [0, num_rows) are skipped.  Two rows of a call may not have the
 * same slot: which values stay is not defined then.  Strides of the caches are not 0 where there is more than one
 * page, token or head.
 * ------------------------------------------------------------------------------------ */
typedef struct gdn_cache_problem {
    int64_t count, num_rows;
    int32_t Hkv, D;                /* D a multiple of 16 */
    int32_t dtype, cache_dtype;    /* as in gdn_paged_problem */
    int32_t page_size;
    int64_t num_pages;
    int64_t k_stride, v_stride;    /* elements between rows (0: contiguous); multiples of 16 bytes */
    int64_t k_page_stride, k_token_stride, k_head_stride;
    int64_t v_page_stride, v_token_stride, v_head_stride;
} gdn_cache_problem;

gdn_status gdn_paged_cache_write(const gdn_cache_problem* p, const void* k, const void* v, void* k_cache,
                                 void* v_cache, const int64_t* slots /* 8-byte aligned */, const int32_t* rows,
                                 const float* k_scale, const float* v_scale, void* stream);

/* ------------------------------------------------------------------------------------
 * Page tables on the device.  Row n of page_table [num_seqs, max_pages] lists the pages of sequence n, which
 * has seq_lens[n] tokens and thus ceil(seq_lens[n] / page_size) pages; free_pages[0 .. *num_free) are the
 * pages that no sequence has, a stack with its top at the end.  All of it is device memory, updated in place.
 *
 * gdn_page_table_extend makes room for new_lens[n] more tokens of every sequence.  In the sequences' order,
 * a sequence that needs m pages more takes the top m (its next column the topmost) and its length grows, if
 *   its length then fits the table's row, and
 *   m = 0, or the stack has as many pages as the sequences up to it need that fit their rows;
 * otherwise it is refused: its length and row stay.  Outputs: cu_seqlens [num_seqs+1], the sums of new_lens,
 * and slots [total]: for the new token cu_seqlens[n] + i of sequence n the slot page * page_size + offset of its position in
 * the cache, -1 where the sequence was refused and behind the last token.  Tokens behind `total` get no slot.
 *
 * gdn_page_table_trim cuts every sequence to keep_lens[n] tokens (longer ones stay as they are) and puts the
 * pages that it then does not need on the stack, the last sequence's first and of each the last column's
 * first, so that it undoes an extension.  0 gives up the sequence; the table's row is left as it was.
 * Pages that the stack has no place for (stack_size) are dropped.
 *
 * Negative lengths count as 0, and *num_free is cut to [0, stack_size]; a cached length past the table's row
 * counts as the row's.  Page numbers are copied as they are.  num_seqs <= 8192.  Integer work: exact.
 * ------------------------------------------------------------------------------------ */
typedef struct gdn_table_problem {
    int32_t num_seqs, max_pages, page_size;
    int32_t stack_size;            /* places in free_pages */
    int64_t total;                 /* places in slots */
    int64_t table_stride;          /* elements between rows of page_table (0: contiguous) */
} gdn_table_problem;

gdn_status gdn_page_table_extend(const gdn_table_problem* p, int32_t* page_table, int32_t* seq_lens,
                                 const int32_t* new_lens, int32_t* free_pages, int32_t* num_free,
                                 int64_t* slots, int32_t* cu_seqlens, void* stream);
gdn_status gdn_page_table_trim(const gdn_table_problem* p, const int32_t* page_table, int32_t* seq_lens,
                               const int32_t* keep_lens, int32_t* free_pages, int32_t* num_free, void* stream);

/* ------------------------------------------------------------------------------------
 * Per-kernel timing (instrumentation for benchmarks; not needed for computation).
 * While enabled, every kernel the library launches is bracketed by two CUDA events
 * recorded on the launching stream.  gdn_timing_collect waits for the recorded events
 * (it synchronises on them), sums the elapsed time per kernel name, writes up to
 * max_entries records, sets *n_entries to the number of distinct kernels, releases the
 * events and clears the record.  Not thread-safe: time one thread's calls at a time.
 * ------------------------------------------------------------------------------------ */
typedef struct gdn_kernel_time {
    char name[48];     /* kernel name, e.g. "fwd_phase_c" */
    int32_t launches;  /* launches recorded since the last collect */
    float total_ms;    /* summed event-to-event time of those launches */
} gdn_kernel_time;

gdn_status gdn_timing_enable(int32_t enable);
gdn_status gdn_timing_collect(gdn_kernel_time* out, int32_t max_entries, int32_t* n_entries);

/* ------------------------------------------------------------------------------------
 * Allocation-free forward.  The FlashQLA pages have no counterpart to this entry point: it
 * exists for callers that cannot allocate device memory themselves -- a runtime that has
 * handed all device memory to its own pool, a latency-critical loop where cudaMalloc or
 * cudaFree may synchronise the device, or a plug-in interface that passes only inputs and
 * outputs.  It computes exactly what gdn_chunk_fwd computes, with the same arguments minus
 * the workspace.
 *
 * Its scratch is one fixed device array of GDN_NOALLOC_SCRATCH_BYTES inside the library;
 * every GPU that loads the library holds that memory until the process exits.  Problems
 * whose gdn_chunk_fwd_workspace_size exceeds it are rejected with GDN_ERR_WORKSPACE and a
 * message (nothing is launched); fewer context-parallel segments (cp_mode /
 * cp_segment_chunks) shrink the need.  The call allocates nothing: no cudaMalloc, no
 * cudaFree, no allocating library routine.
 *
 * The first call on a device looks up the array's device address (cudaGetSymbolAddress,
 * with that device current); make that first call before any stream capture.  The lookup is
 * repeated when the device's context has changed since (e.g. after cudaDeviceReset, which
 * may load the array at another address), so such a call, too, belongs outside a capture.
 * All calls share the one array and it keeps the last call's contents (every byte a call
 * reads is written earlier by the same call), so calls whose GPU work overlaps -- on
 * different streams, or from different threads -- race on it and must be serialised by the
 * caller.
 *
 * gdn_noalloc_device_status is gdn_device_status for these calls: it waits for `stream` and
 * reads the error word that the calls keep at the start of the array (their device-side
 * failure report, see below).  gdn_noalloc_debug_wait_timeout is gdn_debug_wait_timeout on
 * that word (a test hook).
 * ------------------------------------------------------------------------------------ */
#define GDN_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)

gdn_status gdn_chunk_fwd_noalloc(const gdn_problem* p, const void* q, const void* k,
                                 const void* v, const float* g, const float* beta,
                                 const float* h0, void* o, float* ht, void* stream);

gdn_status gdn_noalloc_device_status(void* stream);

gdn_status gdn_noalloc_debug_wait_timeout(int32_t limit_us, void* stream);

/* ------------------------------------------------------------------------------------
 * Device-side failure report.  Every wait of the tensor-core kernels on an mbarrier (a TMA
 * copy landing, a tensor-core product completing, a warp role handing over) is bounded: after
 * 2 s of wall time it gives up, sets a bit in the call's error word -- the first 4 bytes of
 * its workspace, cleared by the first kernel of every gdn_chunk_fwd, gdn_chunk_bwd,
 * gdn_chunk_fwd_saved and gdn_chunk_bwd_saved call -- and the kernel winds down (issued copies
 * and products drained, tensor memory released) instead of hanging; the outputs of that call
 * are then not valid.
 *
 * gdn_device_status waits for `stream` (this call does synchronise), reads the error word of
 * `workspace` (the workspace of the call(s) just enqueued on that stream) and returns GDN_OK,
 * or GDN_ERR_TIMEOUT with the word's bits in gdn_last_error().  workspace: device pointer, at
 * least 4 bytes, 16-byte aligned.
 *
 * Checked builds of this library (compiled with -DGDN_CHECK; libgdn_check.so, for tests)
 * also test the element index of every output store of the bf16 path (o, dq, dk, dv, dg,
 * dbeta, gamma and the rows of T) against the tensor's extent; a store outside it is skipped
 * and sets bit 31 of the error word, and gdn_device_status then returns GDN_ERR_BOUNDS.
 * Release builds do not test and never set that bit.
 * ------------------------------------------------------------------------------------ */
gdn_status gdn_device_status(const void* workspace, void* stream);

/* Test hook of the planner (host only, no GPU work): the segmentation that gdn_chunk_fwd (and
 * gdn_chunk_bwd) would use for `p` on a GPU with `sms` multiprocessors -- chunks per
 * context-parallel segment and the number of segments over all sequences (one per sequence
 * when the planner does not split them).  GDN_ERR_INVALID_ARG for an invalid problem, NULL
 * outputs or sms <= 0. */
gdn_status gdn_debug_plan(const gdn_problem* p, int32_t sms, int32_t* chunks_per_segment,
                          int32_t* segments);

/* Test hook of the failure report: one block waits on an mbarrier that no thread ever
 * completes, gives up after limit_us microseconds (1 .. 1000000) and sets its bit in the error
 * word of `workspace` (only those 4 bytes are touched).  Asynchronous on `stream`. */
gdn_status gdn_debug_wait_timeout(void* workspace, int32_t limit_us, void* stream);

/* Message for the last non-OK status returned on this thread ("" if none). */
const char* gdn_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* GDN_H */
