/*
 * ds4hc.h -- C ABI of libds4hc.so, the MI355X (gfx950) implementation of the
 * DeepSeek-V4 hyper-connection (HC) op.
 *
 * The op, as the lucebox pages describe it:
 *   - lucebox PR #496 "feat(ds4): add DSpark speculative runtime +
 *     optimizations", PR body: a fused DS4 hyper-connection op
 *     (GGML_OP_DS4_HC) with a register-resident Sinkhorn kernel.
 *   - lucebox-hub PR #494 "fix(ds4): keep ROCmFPX generation byte-safe":
 *     "HC-pre" as a decode cost centre (comment with the timing breakdown);
 *     commit notes on the HC fn matvecs, hc_post and the GPU HC pre-mix;
 *     the comment on the Sinkhorn kernel specialised for NHC = 4; and the
 *     direct HC-pre API left out of that PR.
 *   - lucebox PR #507 "correct layer-split HC handoff and per-device state",
 *     Summary/Implementation: the full HC state flows between layers, the HC
 *     fn weights are held as F16 per device, and HC scratch must be per
 *     device (a shared scratch buffer was a bug there).
 *
 * Definitions (n = n_hc streams, d features, K = n*d, m = 2n + n*n):
 *   X[t]      state of token t: n streams x d features, row-major
 *             (flattened index k = i*d + c).
 *   r         = sqrt(sum_k X[t]_k^2 / K + rms_eps)
 *   z_j       = sum_k W[j][k] * X[t]_k / r + bias[j]             (fn matvec)
 *   pre_i     = 1/(1+exp(-z_i)),  post_i = 1/(1+exp(-z_{n+i}))  (gates)
 *   H         = Sinkhorn of Z[i][j] = z_{2n+i*n+j}: M = exp(Z - rowmax(Z)),
 *               then sinkhorn_iters x (divide rows by their sums, then
 *               columns by their sums).
 *   layer_in[c] = sum_i pre_i * X[i][c]                           (pre-mix)
 *   X'[i][c]    = sum_j H[i][j] * X[j][c] + post_i * layer_out[c]  (hc_post)
 *   coeffs[t] = pre[0..n) | post[0..n) | H row-major [n*n]  (m floats)
 *
 * Conventions for every entry point:
 *   - All array pointers are DEVICE pointers on the calling thread's current
 *     HIP device, dense row-major with the shapes given. Alignment: the
 *     state-typed arrays (X, X_out, layer_in, layer_out and their _share
 *     forms) and W must be 16-byte aligned, since the kernels move them in
 *     16-byte vectors; the float32 arrays (bias, coeffs, coeffs_prev, logits,
 *     partials, logits_res, H) and the workspace need 4-byte alignment only.
 *     A pointer that misses its alignment is DS4HC_ERR_INVALID_ARG.
 *   - The caller owns every buffer; the library allocates no device memory.
 *     Its only global state is a per-device cache of the compute-unit count
 *     (looked up on a device's first call, read-only after, atomically
 *     published), a thread-local slot holding the last HIP error text, and
 *     the fixed scratch array of ds4hc_post_pre_noalloc (below) with its
 *     per-device address cache. Every other entry point is re-entrant and
 *     thread-safe.
 *   - Work is enqueued on `stream` (0 = the default stream) and the call
 *     returns without waiting. Faults during execution surface at the
 *     caller's next synchronisation of that stream.
 *   - Arguments are validated on the host before any HIP call. A rejected
 *     call enqueues nothing.
 *   - State dtype (X, layer_in, layer_out, X_out): float32 or bfloat16.
 *     Coefficients, logits and bias are float32; W is IEEE float16.
 *     Arithmetic is float32 with one round-to-nearest-even at each store.
 *     The Sinkhorn normalises by multiplying with the hardware reciprocal
 *     of each row or column sum (within 1 ulp of 1/sum) rather than by a
 *     correctly rounded division, and clamps each entry of H to at most 1
 *     (a NaN stays NaN); H is within a few float32 ulps of the divided result.
 *   - Every path is deterministic: no floating-point atomics, fixed
 *     reduction orders. Repeated calls on equal inputs give equal bits.
 *   - T = 0 returns DS4HC_OK once the scalar arguments are valid, without
 *     looking at any pointer (zero-size buffers may be NULL); nothing runs.
 *   - Supported on the GPU: n_hc in {1, 2, 4}; d > 0 with d % 8 == 0;
 *     0 <= T <= 2^24; sinkhorn_iters in [0, 1000].
 */
#ifndef DS4HC_H
#define DS4HC_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DS4HC_ABI_VERSION 1

typedef enum {
    DS4HC_OK = 0,
    DS4HC_ERR_INVALID_ARG = 1, /* null/misaligned pointer, bad shape, small workspace, overlap */
    DS4HC_ERR_UNSUPPORTED = 2, /* valid for the op, not supported by this GPU library */
    DS4HC_ERR_HIP = 3          /* a HIP launch failed; see ds4hc_last_hip_error() */
} ds4hc_status;

typedef enum {
    DS4HC_F32 = 0,  /* state stored as IEEE float32 */
    DS4HC_BF16 = 1, /* state stored as bfloat16 (uint16 bit patterns) */
    DS4HC_F16 = 2   /* IEEE float16: the operators of an attention site only */
} ds4hc_dtype;

/* Operation constants. Defaults: rms_eps = 1e-6f, sinkhorn_iters = 20. */
typedef struct {
    int32_t n_hc;           /* streams n: 1, 2 or 4 on the GPU */
    int32_t d;              /* features per stream, d % 8 == 0 */
    float rms_eps;          /* added to the mean square inside the sqrt, >= 0 */
    int32_t sinkhorn_iters; /* row-then-column normalisation rounds, 0..1000 */
    uint32_t flags;         /* DS4HC_FLAG_* */
} ds4hc_params;

/* Every path is deterministic already; the flag is accepted and changes nothing. */
#define DS4HC_FLAG_DETERMINISTIC 1u
/* Force one kernel path (all compute the same op; forcing more than one is
 * invalid). The default for HC-pre and fused is the cheapest by a cost model
 * in T and the row length K = n * d, fitted to measured times of every path
 * (at d = 4096 float32: split-K through T = 519, the tile kernel above):
 *   ROWRES  one token per workgroup, row kept in registers, VALU matvec;
 *   TILE    persistent, one workgroup per CU striding over tiles of four
 *           tokens, rows kept in registers, MFMA matvec;
 *   SPLITK  partials over column chunks into the workspace (4 tokens per
 *           workgroup below T = 32, 16 from T = 32), then a combining
 *           kernel. */
#define DS4HC_FLAG_FORCE_ROWRES 2u
#define DS4HC_FLAG_FORCE_SPLITK 4u
#define DS4HC_FLAG_FORCE_TILE 8u

/*
 * ds4hc_pre -- HC-pre: RMS statistic, fn matvec, sigmoid gates, Sinkhorn and
 * the pre-mix ("HC-pre" and the GPU "HC pre-mix", lucebox-hub PR #494).
 *   X          [T, n, d]  state dtype       (read)
 *   W_f16      [m, n*d]   float16 bits      (read)
 *   bias       [m]        float32           (read)
 *   layer_in   [T, d]     state dtype       (written)
 *   coeffs     [T, m]     float32           (written: pre | post | H)
 *   logits_opt [T, m]     float32 or NULL   (written: raw z, for debugging)
 *   workspace  device scratch of at least ds4hc_workspace_bytes(p, T, dtype)
 *              bytes (may be NULL when that is 0); contents need not be set
 *              and are overwritten. Calls that share one workspace must be
 *              ordered on one stream.
 * Outputs must not overlap inputs or each other.
 */
ds4hc_status ds4hc_pre(const ds4hc_params *p, int64_t T, ds4hc_dtype dtype, const void *X,
                       const uint16_t *W_f16, const float *bias, void *layer_in, float *coeffs,
                       float *logits_opt, void *workspace, size_t workspace_bytes,
                       hipStream_t stream);

/*
 * ds4hc_sinkhorn -- the register-resident Sinkhorn micro-kernel alone (the
 * NHC = 4 template kernel of lucebox-hub PR #494's comment on its 95 us ->
 * 5.3 us fix), on arbitrary residual logits.
 *   logits_res [T, n, n] float32 (read), H [T, n, n] float32 (written).
 * n_hc in {1, 2, 4}; iters in [0, 1000]. H may not overlap logits_res.
 */
ds4hc_status ds4hc_sinkhorn(int64_t T, int32_t n_hc, int32_t iters, const float *logits_res,
                            float *H, hipStream_t stream);

/*
 * ds4hc_post -- hc_post (lucebox-hub PR #494 commit notes): the post update
 * X' = H.X + post (x) layer_out from coefficients written by ds4hc_pre.
 *   X [T, n, d] state (read), coeffs [T, m] float32 (read),
 *   layer_out [T, d] state (read), X_out [T, n, d] state (written).
 * X_out may be exactly X (in-place update); any other overlap is invalid.
 */
ds4hc_status ds4hc_post(const ds4hc_params *p, int64_t T, ds4hc_dtype dtype, const void *X,
                        const float *coeffs, const void *layer_out, void *X_out,
                        hipStream_t stream);

/*
 * ds4hc_fused -- the whole op (GGML_OP_DS4_HC of lucebox PR #496) in one
 * call, for a layer_out that does not depend on this call's layer_in.
 * Arguments as in ds4hc_pre and ds4hc_post; coeffs_opt may be NULL.
 * X_out may be exactly X; layer_in must not overlap X, X_out or layer_out.
 */
ds4hc_status ds4hc_fused(const ds4hc_params *p, int64_t T, ds4hc_dtype dtype, const void *X,
                         const uint16_t *W_f16, const float *bias, const void *layer_out,
                         void *layer_in, float *coeffs_opt, void *X_out, void *workspace,
                         size_t workspace_bytes, hipStream_t stream);

/* Workspace bytes ds4hc_pre / ds4hc_fused need for these arguments (0 when
 * the chosen path needs none). Pure function; 0 for invalid arguments. It takes
 * the state dtype because the path, and below T = 32 the split-K column-chunk
 * width (16 or 32 lanes x one 16-byte vector) and hence the number of partial
 * sums, depend on it. */
size_t ds4hc_workspace_bytes(const ds4hc_params *p, int64_t T, ds4hc_dtype dtype);

/*
 * ds4hc_post_pre -- one decode-chain step: the post update of site l followed
 * by HC-pre of site l+1, the two halves the pages run back to back on the GPU
 * with no host round trip between them ("hc_post" and "HC-pre", lucebox-hub
 * PR #494, comment on the GPU HC pre-mix and hc_post). With
 *   X' = H_l . X + post_l (x) layer_out_l            (coefficients from site l)
 * it writes X_out = X' and, for site l+1 on X' (as stored, in the state dtype):
 * layer_in = pre-mix, coeffs = pre | post | H, logits_opt = raw z.
 *   X            [T, n, d]  state dtype  (read)  state before site l's post
 *   coeffs_prev  [T, m]     float32      (read)  site l's coefficients
 *   layer_out    [T, d]     state dtype  (read)  site l's layer output
 *   W_f16_next   [m, n*d]   float16 bits (read)  site l+1's fn weight
 *   bias_next    [m]        float32      (read)
 *   X_out        [T, n, d]  state dtype  (written; may be exactly X)
 *   layer_in     [T, d]     state dtype  (written)
 *   coeffs       [T, m]     float32      (written; must not overlap coeffs_prev)
 *   workspace    >= ds4hc_post_pre_workspace_bytes(p, T, dtype) bytes
 * X' is bitwise what ds4hc_post writes. For T <= 160 (or DS4HC_FLAG_FORCE_SPLITK)
 * the state is read once: a split-K kernel over column chunks applies the post
 * update, stores X' and accumulates site l+1's partial projections, then a
 * combining kernel finishes site l+1. Otherwise it runs the post kernel, then
 * HC-pre on the path ds4hc_pre would take (or the forced one). Errors as for
 * ds4hc_fused.
 */
ds4hc_status ds4hc_post_pre(const ds4hc_params *p, int64_t T, ds4hc_dtype dtype, const void *X,
                            const float *coeffs_prev, const void *layer_out,
                            const uint16_t *W_f16_next, const float *bias_next, void *X_out,
                            void *layer_in, float *coeffs, float *logits_opt, void *workspace,
                            size_t workspace_bytes, hipStream_t stream);

/* Workspace bytes ds4hc_post_pre needs for these arguments (0 if none or invalid). */
size_t ds4hc_post_pre_workspace_bytes(const ds4hc_params *p, int64_t T, ds4hc_dtype dtype);

/*
 * ds4hc_post_pre_noalloc -- ds4hc_post_pre for callers that cannot allocate
 * device memory: code under HIP graph capture, tight serving loops, harnesses
 * that forbid hipMalloc. Same arguments, semantics, kernels and results (bit
 * for bit) as ds4hc_post_pre, without the workspace: the split-K partial sums
 * go to a file-scope device array of DS4HC_NOALLOC_SCRATCH_BYTES bytes that
 * every device the library runs on holds until the process ends. The call
 * allocates nothing; on a device's first call it looks up the array's device
 * address (hipGetSymbolAddress) and keeps it.
 * Limit: a call whose ds4hc_post_pre_workspace_bytes(p, T, dtype) exceeds
 * DS4HC_NOALLOC_SCRATCH_BYTES returns DS4HC_ERR_UNSUPPORTED and enqueues
 * nothing (n = 4: T * P * 100 bytes with P = ceil(d / (16 * V)) column chunks
 * where that is at most 64, else ceil(d / (32 * V)); V = 4 for float32 and 8
 * for bfloat16 state; d = 4096 float32 fits every T of the one-pass path).
 * All calls on one device share that device's array, and the kernels
 * overwrite every byte they read before reading it (nothing must start at
 * zero). Calls that overlap on one device race on the array: order them on
 * one stream.
 */
#define DS4HC_NOALLOC_SCRATCH_BYTES (2u << 20)
ds4hc_status ds4hc_post_pre_noalloc(const ds4hc_params *p, int64_t T, ds4hc_dtype dtype,
                                    const void *X, const float *coeffs_prev, const void *layer_out,
                                    const uint16_t *W_f16_next, const float *bias_next,
                                    void *X_out, void *layer_in, float *coeffs, float *logits_opt,
                                    hipStream_t stream);

/*
 * Split over d (one GPU's share of the columns of every stream; the exchange
 * point of a tensor-parallel split, shown on one GPU). The op's only coupling
 * across columns is the 2n + n^2 fn dot products and the sum of squares of
 * each token row, so a share can emit those partial sums, the shares exchange
 * them ([T, m + 1] floats per share: an all-gather), and each share finishes
 * its own columns. p->d is the share's width d_s (d_s % 8 == 0).
 *
 * ds4hc_partials -- per token, over the share's columns:
 *   partials[t][j] = sum_k W_share[j][k] x_share[k]  (j < m, unnormalised)
 *   partials[t][m] = sum_k x_share[k]^2
 *   X_share   [T, n, d_s]    state dtype   (read)
 *   W_share   [m, n * d_s]   float16 bits  (read) W's columns i*d + share, per stream i
 *   partials  [T, m + 1]     float32       (written)
 *   workspace >= ds4hc_partials_workspace_bytes(p, T, dtype) bytes (0 for
 *               T > 160: a streamed kernel, 16 tokens per workgroup, writes the
 *               partials directly; split-K chunks below, or when forced)
 */
ds4hc_status ds4hc_partials(const ds4hc_params *p, int64_t T, ds4hc_dtype dtype, const void *X_share,
                            const uint16_t *W_share, float *partials, void *workspace,
                            size_t workspace_bytes, hipStream_t stream);
size_t ds4hc_partials_workspace_bytes(const ds4hc_params *p, int64_t T, ds4hc_dtype dtype);

/*
 * ds4hc_combine -- sums the G shares' partials [G, T, m + 1] in share order
 * (deterministic; every share that combines the same partials gets bitwise the
 * same coefficients), then z = dots / r + bias with r over all n * d_total
 * columns, the gates, the Sinkhorn, and pass 2 on this share: layer_in_share
 * = pre-mix, X_out_share = H . X_share + post (x) layer_out_share (may be
 * exactly X_share). coeffs_opt [T, m] may be NULL. d_total >= p->d.
 */
ds4hc_status ds4hc_combine(const ds4hc_params *p, int32_t d_total, int64_t T, ds4hc_dtype dtype,
                           int32_t G, const float *partials, const float *bias, const void *X_share,
                           const void *layer_out_share, void *layer_in_share, float *coeffs_opt,
                           void *X_out_share, hipStream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Operators of an attention site: what runs between ds4hc_pre (which gives the
 * layer input) and ds4hc_post (which takes the layer output) besides the plain
 * projections. Attention keeps ONE shared vector a token: a latent of d_latent
 * elements, from which every head's key and value come by a fixed projection,
 * and a rotated key of 64 elements that all heads share.
 *
 *   ds4hc_rope            rotary positions of the queries' (or keys') rotated part
 *   ds4hc_latent_append   RMS-norm of the latents, rotation of the shared keys,
 *                         store into a paged cache
 *   ds4hc_latent_attn     absorbed form over that cache: queries are multiplied
 *                         into the latent space beforehand, keys and values are
 *                         the cached vectors themselves (decode, drafted chains
 *                         and trees, chunks of a prompt)
 *   ds4hc_latent_prefill  expanded form: keys and values a head, from a ragged
 *                         batch of prompts
 *
 * The conventions at the top hold, with these additions: strides count elements;
 * arrays of the 16-bit types and rows of strided arrays must start on 16-byte
 * boundaries (ds4hc_rope alone takes any element-aligned address and stride);
 * int32 and float32 arrays need 4-byte, int64, uint64 and float64 arrays 8-byte
 * alignment. The library allocates nothing and keeps nothing between calls. These
 * are operators of inference; of rotation the transpose is there (its gradient).
 *
 * What the device arrays of lengths and pages hold is not known to the host.
 * Every entry is checked in the kernel before it is used: cu_q and cu_k entries
 * are taken as clamped to [0, tokens] and a sequence that would end before it
 * starts as empty, kv_len as clamped to [0, max_pages * page_size], and tokens
 * of a page whose block_table entry is not in [0, n_pages) as not in the cache
 * (no query sees them, an append to them stores nothing). No value in them makes
 * a kernel read or write outside the arrays given. Sequences of one call that
 * overlap (cu_q that does not rise) write the shared rows in any order, and
 * ds4hc_latent_prefill, whose grid has room for N queries, may then leave others
 * unwritten.
 * ---------------------------------------------------------------------------
 */

/* Elements between two tokens and between two heads of a [tokens, heads, dim]
 * array whose innermost dimension is dense. Not negative. */
typedef struct {
    int64_t token;
    int64_t head;
} ds4hc_strides;

/* Pairs of a rotation are (2i, 2i + 1), or (i, i + dim / 2) with DS4HC_ROPE_HALF. */
#define DS4HC_ROPE_HALF 1u
/* Rotate by the negative angle (the transpose: undoes the rotation, and is its
 * gradient, up to amplitude^2). ds4hc_rope only. */
#define DS4HC_ROPE_INVERSE 2u

/*
 * ds4hc_rope -- rotary positions. For token t, head h, pair i, with the angle
 * a = positions[t] * inv_freq[i] formed in 64 bits:
 *   y0 = (x0 cos a - x1 sin a) * amplitude,  y1 = (x0 sin a + x1 cos a) * amplitude
 * in float32, one rounding at the store.
 *   x         [N, heads, dim] strided, any of the three dtypes (read). To rotate
 *             part of a head pass the address of that part and the strides of
 *             the whole. Strides may be 0 (a broadcast input).
 *   positions [N]       int64   (read; any sign)
 *   inv_freq  [dim / 2] float64 (read; radians a position)
 *   y         [N, heads, dim] strided, dtype of x (written: these elements only)
 * y may be exactly x with x's strides (in place); otherwise the two may not
 * overlap, as ranges from the first to the last element. Rows of y may not
 * overlap one another. dim is even, 2..512; heads 1..1024; N <= 2^24.
 */
ds4hc_status ds4hc_rope(int64_t N, int32_t heads, int32_t dim, ds4hc_dtype dtype, const void *x,
                        ds4hc_strides x_strides, const int64_t *positions, const double *inv_freq,
                        float amplitude, uint32_t flags, void *y, ds4hc_strides y_strides,
                        hipStream_t stream);

/*
 * ds4hc_rope_frequencies -- HOST function, fills the HOST arrays inv_freq
 * [dim / 2] and *amplitude for ds4hc_rope and ds4hc_latent_append:
 *   f_i = base^(-2i / dim)                                      (factor == 1)
 *   f_i / factor               (factor > 1, original_length == 0: interpolated)
 *   f_i ((1 - k_i) / factor + k_i)                (factor > 1, original_length > 0)
 * the last after Peng et al. 2023 ("YaRN: Efficient Context Window Extension of
 * Large Language Models"): pairs that make beta_fast turns or more over the trained
 * length stay as they are, those of beta_slow or fewer are stretched fully. With the
 * pair that makes b turns, pair(b) = dim ln(original_length / (2 pi b)) / (2 ln base),
 * lo = max(floor(pair(beta_fast)), 0), hi = min(ceil(pair(beta_slow)), dim - 1),
 *   k_i = 1 - clamp((i - lo) / max(hi - lo, 0.001), 0, 1),
 * and amplitude = 0.1 ln(factor) + 1 (1 in the other two cases). Between the ends
 * the ramp is linear in the pair's index, the form in common use, which trained
 * weights expect; the paper's own is linear in the turns (dim 64, length 4096,
 * factor 40: pair 16 keeps 0.55 of its frequency here, 0.20 there). hi may lie
 * behind the last pair, as it does for long trained lengths. base > 1,
 * factor >= 1, beta_fast >= beta_slow > 0 (looked at in the last case only).
 */
ds4hc_status ds4hc_rope_frequencies(int32_t dim, double base, double factor,
                                    int64_t original_length, double beta_fast, double beta_slow,
                                    double *inv_freq, float *amplitude);

/*
 * A paged cache of latent vectors, and the batch of sequences that a call
 * handles. The cache is [n_pages, page_size, d_latent + 64] of dtype, dense;
 * token j of sequence b lies in page block_table[b][j / page_size], at place
 * j % page_size. The call's tokens are ragged: sequence b has tokens
 * cu_q[b] .. cu_q[b + 1] - 1 of the call's N, and they are the LAST tokens of
 * its kv_len[b] tokens (token i of the call's q_len for b is token
 * kv_len[b] - q_len + i of the sequence). Tokens of the call behind the last
 * sequence have no effect and their outputs are left as they were; their inputs
 * may be read (all N rows must be there).
 */
typedef struct {
    ds4hc_dtype dtype;          /* DS4HC_BF16 or DS4HC_F16 */
    int32_t d_latent;           /* 128, 256 or 512 */
    int32_t d_rope;             /* 64 */
    int32_t page_size;          /* tokens a page: a power of two, 1..65536 */
    int64_t n_pages;            /* pages of the cache, >= 1; n_pages * page_size < 2^31 */
    int32_t n_seqs;             /* sequences B, 0..2^20 */
    int32_t max_pages;          /* entries of a row of block_table, >= 1;
                                   max_pages * page_size <= 2^30 */
    const int32_t *cu_q;        /* [B + 1] */
    const int32_t *kv_len;      /* [B], this call's tokens included */
    const int32_t *block_table; /* [B, max_pages] */
} ds4hc_paged_cache;

/*
 * ds4hc_latent_append -- for each token of the call, with kv = (c | r):
 *   c' = c / sqrt(mean(c^2) + rms_eps) * norm_weight   (c' = c if norm_weight is NULL)
 *   r' = r rotated as by ds4hc_rope
 * in float32, rounded once to the cache's dtype and stored at the token's place.
 * Places before token 0 of a sequence (q_len > kv_len) are passed over. The
 * sequences' pages that are written must differ from one another: of two tokens
 * with one place either may be kept, in parts.
 *   kv          [N, d_latent + 64], kv_stride elements between rows, src_dtype any
 *               of the three (read)
 *   positions   [N] int64, inv_freq [32] float64, amplitude, flags (DS4HC_ROPE_HALF)
 *   norm_weight [d_latent] float32 or NULL (read)
 *   cache       (written: the tokens' places only)
 */
ds4hc_status ds4hc_latent_append(const ds4hc_paged_cache *c, int64_t N, ds4hc_dtype src_dtype,
                                 const void *kv, int64_t kv_stride, const float *norm_weight,
                                 float rms_eps, const int64_t *positions, const double *inv_freq,
                                 float amplitude, uint32_t flags, void *cache, hipStream_t stream);

/*
 * ds4hc_latent_attn -- attention of the call's tokens over the cache, absorbed
 * form. For token t of sequence b, head h, over the cached tokens j that t sees:
 *   s_j = scale * (q_latent[t][h] . c_j + q_rope[t][h] . r_j)
 *   out[t][h] = sum_j softmax(s)_j c_j,   lse[t][h] = ln sum_j exp(s_j)
 * Token i of the call's q_len for b sees the cached tokens before the call's
 * own, j < kv_len[b] - q_len, and of the call's own:
 *   tree_mask NULL: its own place and those before it;
 *   otherwise those whose bit is set: bit d % 64 of word tree_mask[t][d / 64]
 *   stands for token d of the call's tokens for b (its own bit included: nothing
 *   is implied). Tokens d >= 64 * mask_words are seen by none.
 * A row that sees nothing gives out = 0 and lse = -infinity, and so does one all of
 * whose logits are -infinity. A NaN in a cached token, or an infinity in its latent,
 * makes the rows that see it not finite, in some of their elements at least. An
 * infinity in its rotated part gives an infinite logit: -infinity is a weight of 0,
 * +infinity makes the row not finite. Rows that do not see the token stay right.
 *   q_latent [N, heads, d_latent], q_rope [N, heads, 64] strided, c->dtype (read)
 *   cache    (read)
 *   tree_mask [N, mask_words] uint64 or NULL (read; mask_words 1..1024)
 *   out      [N, heads, d_latent] strided, c->dtype (written)
 *   lse_opt  [N, heads] float32 or NULL (written)
 *   workspace of ds4hc_latent_attn_workspace_bytes(c, N, heads) bytes, 16-byte
 *            aligned (may be NULL when that is 0); as for ds4hc_pre. It holds parts of
 *            sums of 512 row tiles, whatever the lengths, which the host does not know:
 *            with d_latent 512 34 MB up to 32 rows (tokens x heads) a sequence on
 *            average, 68 MB up to 64, 135 MB beyond.
 * Products are of the 16-bit inputs and sums, softmax statistics and the running
 * output float32; the softmax weights are rounded to the 16-bit type for the
 * second product, and divided by their sum as rounded (lse is of the sum before
 * that rounding). In float16 that rounding keeps its relative size down to 2^-20
 * of the row's largest weight and weights below 2^-31 of it become 0; in bfloat16
 * there is no such end. Logits are float32: beyond 2^24 their last place is more
 * than a unit, and rows with logits beyond 2^30 (float16: 2^27) may become NaN.
 * Every row goes through all of its sequence's cached tokens, also those that a
 * chunk's early tokens do not see: a prompt without a context (q_len = kv_len = 4096,
 * 128 heads: 5.9 ms) is for ds4hc_latent_prefill (0.76 ms, besides the projections).
 * scale > 0; heads 1..1024; N <= 2^24, N * heads <= 2^30.
 * Outputs may not overlap inputs or each other, as ranges from the first to the
 * last element; rows of out may not overlap one another.
 */
ds4hc_status ds4hc_latent_attn(const ds4hc_paged_cache *c, int64_t N, int32_t heads, float scale,
                               const void *q_latent, ds4hc_strides q_latent_strides,
                               const void *q_rope, ds4hc_strides q_rope_strides, const void *cache,
                               const uint64_t *tree_mask, int32_t mask_words, void *out,
                               ds4hc_strides out_strides, float *lse_opt, void *workspace,
                               size_t workspace_bytes, hipStream_t stream);

/* Workspace bytes ds4hc_latent_attn needs. Pure function of the host fields (the
 * device arrays are not looked at and may be NULL); 0 for invalid arguments. */
size_t ds4hc_latent_attn_workspace_bytes(const ds4hc_paged_cache *c, int64_t N, int32_t heads);

/* Every query sees every key of its sequence (the default is causal). */
#define DS4HC_ATTN_FULL 1u

/*
 * ds4hc_latent_prefill -- attention over expanded keys and values of a ragged
 * batch. Sequence b has queries cu_q[b] .. cu_q[b + 1] - 1 and keys cu_k[b] ..
 * cu_k[b + 1] - 1; its queries are the last of its tokens: query i sees key j if
 * j <= i + k_len - q_len (any j with DS4HC_ATTN_FULL). With q = (qn | qr):
 *   s_j = scale * (qn . kn_j + qr . kr_j),  out = sum_j softmax(s)_j v_j,
 *   lse = ln sum_j exp(s_j);  a row that sees nothing gives 0 and -infinity.
 *   q      [N, heads, 128 + 64] dense, dtype BF16 or F16 (read)
 *   kv     [S, heads, 128 + 128] dense: kn | v of each head (read)
 *   k_rope [S, 64], k_rope_stride elements between rows, shared by the heads (read)
 *   cu_q, cu_k [n_seqs + 1] int32 (read)
 *   out    [N, heads, 128] dense (written), lse_opt [N, heads] float32 or NULL (written)
 * Rows of out and lse behind the last sequence are left as they were. Keys and
 * values that are not finite touch no row that does not see them; of those that do,
 * a NaN or an infinite value makes elements not finite at least, and an infinite
 * key an infinite logit, as for ds4hc_latent_attn.
 * Rounding as for ds4hc_latent_attn. heads 1..1024, N and S <= 2^24,
 * N * heads <= 2^30, n_seqs <= 2^20.
 */
ds4hc_status ds4hc_latent_prefill(int64_t N, int64_t S, int32_t n_seqs, int32_t heads,
                                  ds4hc_dtype dtype, float scale, uint32_t flags, const void *q,
                                  const void *kv, const void *k_rope, int64_t k_rope_stride,
                                  const int32_t *cu_q, const int32_t *cu_k, void *out,
                                  float *lse_opt, hipStream_t stream);

/* Static, human-readable name of a status code. */
const char *ds4hc_status_string(ds4hc_status s);

/* Text of the last HIP error seen by a ds4hc call on this thread ("" if none). */
const char *ds4hc_last_hip_error(void);

/* DS4HC_ABI_VERSION of the loaded library. */
int ds4hc_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DS4HC_H */
