// latent_api.cpp -- the attention-site part of the C ABI declared in
// include/ds4hc.h: host-side argument validation and launch. As for the HC
// entry points, nothing touches the GPU until every argument has been checked,
// and no memory is allocated. What device arrays hold is checked in the kernels.
#include "ds4hc.h"

#include <math.h>

#include "api_common.hpp"
#include "latent_launch.hpp"

namespace {

using ds4hc::aligned;
using ds4hc::MAX_T;
using ds4hc::overlap;
using ds4hc::Range;

constexpr int MAX_HEADS = 1024;
constexpr int MAX_ROPE_DIM = 512;
constexpr int MAX_SEQS = 1 << 20;
constexpr int MAX_MASK_WORDS = 1024;
constexpr int64_t MAX_KV = int64_t(1) << 30;    // tokens of a sequence
constexpr int64_t MAX_ROWS = int64_t(1) << 30;  // tokens x heads of a call
constexpr int64_t MAX_STRIDE = int64_t(1) << 36;  // elements: offsets stay far inside 64 bits

int elem_bytes(ds4hc_dtype dt) { return dt == DS4HC_F32 ? 4 : 2; }
bool half_type(ds4hc_dtype dt) { return dt == DS4HC_BF16 || dt == DS4HC_F16; }
bool any_type(ds4hc_dtype dt) { return dt == DS4HC_F32 || half_type(dt); }
bool strides_ok(ds4hc_strides s) {
    return s.token >= 0 && s.head >= 0 && s.token <= MAX_STRIDE && s.head <= MAX_STRIDE;
}

// Bytes from the first to the last element of a strided [N, heads, dim] array.
uint64_t span(int64_t N, int heads, int dim, ds4hc_strides s, int eb) {
    return ((uint64_t)(N - 1) * s.token + (uint64_t)(heads - 1) * s.head + dim) * eb;
}

// Whether no two rows of a strided array share an element: tokens outside heads
// or heads outside tokens.
bool rows_apart(int64_t N, int heads, int dim, ds4hc_strides s) {
    const int64_t H = heads;
    const bool by_token = (H == 1 || s.head >= dim) && (N == 1 || s.token >= (H - 1) * s.head + dim);
    const bool by_head = (N == 1 || s.token >= dim) && (H == 1 || s.head >= (N - 1) * s.token + dim);
    return by_token || by_head;
}

// Rows on 16-byte boundaries: base and strides that are used.
bool rows_aligned16(const void *p, int64_t N, int heads, ds4hc_strides s, int eb) {
    return aligned(p, 16) && (N == 1 || s.token * eb % 16 == 0) && (heads == 1 || s.head * eb % 16 == 0);
}

ds4hc_status check_cache(const ds4hc_paged_cache *c, int64_t N) {
    if (!c || N < 0) return DS4HC_ERR_INVALID_ARG;
    if (!any_type(c->dtype)) return DS4HC_ERR_INVALID_ARG;
    if (c->d_latent <= 0 || c->d_rope < 0 || c->page_size <= 0 || c->n_pages <= 0 || c->n_seqs < 0 ||
        c->max_pages <= 0)
        return DS4HC_ERR_INVALID_ARG;
    if (c->page_size & (c->page_size - 1)) return DS4HC_ERR_INVALID_ARG;
    if (!half_type(c->dtype) || c->d_rope != ds4hc::LATENT_ROPE ||
        (c->d_latent != 128 && c->d_latent != 256 && c->d_latent != 512))
        return DS4HC_ERR_UNSUPPORTED;
    if (c->page_size > 65536 || c->n_seqs > MAX_SEQS || N > MAX_T || c->n_pages > (int64_t(1) << 31) - 1 ||
        c->n_pages * c->page_size >= (int64_t(1) << 31) || (int64_t)c->max_pages * c->page_size > MAX_KV)
        return DS4HC_ERR_UNSUPPORTED;
    return DS4HC_OK;
}

// The device arrays of the descriptor.
bool batch_arrays_ok(const ds4hc_paged_cache *c) {
    return c->cu_q && c->kv_len && c->block_table && aligned(c->cu_q, 4) && aligned(c->kv_len, 4) &&
           aligned(c->block_table, 4);
}

uint64_t cache_bytes(const ds4hc_paged_cache *c) {
    return (uint64_t)c->n_pages * c->page_size * (c->d_latent + c->d_rope) * 2;
}

ds4hc::Paged view(const ds4hc_paged_cache *c) {
    return {__builtin_ctz((unsigned)c->page_size), c->n_seqs, c->max_pages, c->n_pages,
            c->cu_q, c->kv_len, c->block_table};
}

ds4hc_status done(hipError_t e) { return e == hipSuccess ? DS4HC_OK : ds4hc::hip_fail(e); }

// Whether any of the outputs overlaps another output or an input.
template <int NI, int NO>
bool clash(const Range (&in)[NI], const Range (&out)[NO]) {
    for (int o = 0; o < NO; ++o) {
        for (int i = 0; i < NI; ++i)
            if (overlap(out[o], in[i])) return true;
        for (int q = o + 1; q < NO; ++q)
            if (overlap(out[o], out[q])) return true;
    }
    return false;
}

}  // namespace

extern "C" {

ds4hc_status ds4hc_rope(int64_t N, int32_t heads, int32_t dim, ds4hc_dtype dtype, const void *x,
                        ds4hc_strides xs, const int64_t *positions, const double *inv_freq,
                        float amplitude, uint32_t flags, void *y, ds4hc_strides ys,
                        hipStream_t stream) {
    if (N < 0 || heads < 1 || dim < 2 || dim % 2 || !any_type(dtype)) return DS4HC_ERR_INVALID_ARG;
    if (flags & ~(DS4HC_ROPE_HALF | DS4HC_ROPE_INVERSE)) return DS4HC_ERR_INVALID_ARG;
    if (!isfinite(amplitude) || !strides_ok(xs) || !strides_ok(ys)) return DS4HC_ERR_INVALID_ARG;
    if (heads > MAX_HEADS || dim > MAX_ROPE_DIM || N > MAX_T) return DS4HC_ERR_UNSUPPORTED;
    if (N == 0) return DS4HC_OK;
    const int eb = elem_bytes(dtype);
    if (!x || !y || !positions || !inv_freq) return DS4HC_ERR_INVALID_ARG;
    if (!aligned(x, eb) || !aligned(y, eb) || !aligned(positions, 8) || !aligned(inv_freq, 8))
        return DS4HC_ERR_INVALID_ARG;
    if (!rows_apart(N, heads, dim, ys)) return DS4HC_ERR_INVALID_ARG;
    const Range rx{x, span(N, heads, dim, xs, eb)}, ry{y, span(N, heads, dim, ys, eb)};
    const bool in_place = x == y && (N == 1 || xs.token == ys.token) && (heads == 1 || xs.head == ys.head);
    if (!in_place && overlap(rx, ry)) return DS4HC_ERR_INVALID_ARG;
    if (overlap(ry, Range{positions, (uint64_t)N * 8}) || overlap(ry, Range{inv_freq, (uint64_t)dim * 4}))
        return DS4HC_ERR_INVALID_ARG;
    const ds4hc::RopeArgs a{N, heads, dim, (int)dtype, x, xs.token, xs.head, positions, inv_freq, amplitude,
                            (flags & DS4HC_ROPE_HALF) != 0, (flags & DS4HC_ROPE_INVERSE) != 0,
                            y, ys.token, ys.head};
    return done(ds4hc::launch_rope(a, stream));
}

ds4hc_status ds4hc_rope_frequencies(int32_t dim, double base, double factor, int64_t original_length,
                                    double beta_fast, double beta_slow, double *inv_freq,
                                    float *amplitude) {
    if (dim < 2 || dim % 2 || !(base > 1.0) || !isfinite(base) || !(factor >= 1.0) || !isfinite(factor) ||
        original_length < 0 || !inv_freq || !amplitude)
        return DS4HC_ERR_INVALID_ARG;
    const bool ramp = factor > 1.0 && original_length > 0;
    if (ramp && (!(beta_slow > 0.0) || !(beta_fast >= beta_slow) || !isfinite(beta_fast)))
        return DS4HC_ERR_INVALID_ARG;
    if (dim > MAX_ROPE_DIM) return DS4HC_ERR_UNSUPPORTED;
    double lo = 0.0, hi = 0.0;
    if (ramp) {
        const double per = dim / (2.0 * log(base)), len = (double)original_length / (2.0 * M_PI);
        lo = fmax(floor(per * log(len / beta_fast)), 0.0);
        // behind the last pair (dim / 2 - 1) for long trained lengths: the ramp's slope is what
        // counts, and pairs that make more than beta_slow turns are not to be stretched fully
        hi = fmin(ceil(per * log(len / beta_slow)), dim - 1.0);
    }
    for (int i = 0; i < dim / 2; ++i) {
        const double f = pow(base, -2.0 * i / dim);
        const double kept = ramp ? 1.0 - fmin(fmax((i - lo) / fmax(hi - lo, 0.001), 0.0), 1.0) : 0.0;
        inv_freq[i] = f * ((1.0 - kept) / factor + kept);
    }
    *amplitude = ramp ? (float)(0.1 * log(factor) + 1.0) : 1.f;
    return DS4HC_OK;
}

ds4hc_status ds4hc_latent_append(const ds4hc_paged_cache *c, int64_t N, ds4hc_dtype src_dtype,
                                 const void *kv, int64_t kv_stride, const float *norm_weight,
                                 float rms_eps, const int64_t *positions, const double *inv_freq,
                                 float amplitude, uint32_t flags, void *cache, hipStream_t stream) {
    const ds4hc_status st = check_cache(c, N);
    if (st != DS4HC_OK) return st;
    if (!any_type(src_dtype) || (flags & ~DS4HC_ROPE_HALF) || !isfinite(amplitude) || !(rms_eps >= 0.f) ||
        !isfinite(rms_eps))
        return DS4HC_ERR_INVALID_ARG;
    const int D = c->d_latent + c->d_rope, eb = elem_bytes(src_dtype);
    if (kv_stride < D || kv_stride > MAX_STRIDE || kv_stride * eb % 16) return DS4HC_ERR_INVALID_ARG;
    if (N == 0 || c->n_seqs == 0) return DS4HC_OK;
    if (!batch_arrays_ok(c) || !kv || !positions || !inv_freq || !cache) return DS4HC_ERR_INVALID_ARG;
    if (!aligned(kv, 16) || !aligned(cache, 16) || !aligned(positions, 8) || !aligned(inv_freq, 8) ||
        (norm_weight && !aligned(norm_weight, 4)))
        return DS4HC_ERR_INVALID_ARG;
    const uint64_t B = (uint64_t)c->n_seqs;
    const Range in[] = {{kv, ((uint64_t)(N - 1) * kv_stride + D) * eb}, {norm_weight, (uint64_t)c->d_latent * 4},
                        {positions, (uint64_t)N * 8}, {inv_freq, (uint64_t)c->d_rope * 4},
                        {c->cu_q, (B + 1) * 4}, {c->kv_len, B * 4}, {c->block_table, B * c->max_pages * 4}};
    const Range out[] = {{cache, cache_bytes(c)}};
    if (clash(in, out)) return DS4HC_ERR_INVALID_ARG;
    const ds4hc::AppendArgs a{view(c), (int)c->dtype, c->d_latent, (int)src_dtype, N, kv, kv_stride, norm_weight,
                              rms_eps, positions, inv_freq, amplitude, (flags & DS4HC_ROPE_HALF) != 0, cache};
    return done(ds4hc::launch_append(a, stream));
}

ds4hc_status ds4hc_latent_attn(const ds4hc_paged_cache *c, int64_t N, int32_t heads, float scale,
                               const void *q_latent, ds4hc_strides ls, const void *q_rope,
                               ds4hc_strides rs, const void *cache, const uint64_t *tree_mask,
                               int32_t mask_words, void *out, ds4hc_strides os, float *lse_opt,
                               void *workspace, size_t workspace_bytes, hipStream_t stream) {
    const ds4hc_status st = check_cache(c, N);
    if (st != DS4HC_OK) return st;
    if (heads < 1 || !(scale > 0.f) || !isfinite(scale) || !strides_ok(ls) || !strides_ok(rs) || !strides_ok(os))
        return DS4HC_ERR_INVALID_ARG;
    if (tree_mask && mask_words < 1) return DS4HC_ERR_INVALID_ARG;
    if (heads > MAX_HEADS || N * heads > MAX_ROWS || (tree_mask && mask_words > MAX_MASK_WORDS))
        return DS4HC_ERR_UNSUPPORTED;
    if (N == 0 || c->n_seqs == 0) return DS4HC_OK;
    if (!batch_arrays_ok(c) || !q_latent || !q_rope || !cache || !out) return DS4HC_ERR_INVALID_ARG;
    if (!rows_aligned16(q_latent, N, heads, ls, 2) || !rows_aligned16(q_rope, N, heads, rs, 2) ||
        !rows_aligned16(out, N, heads, os, 2) || !aligned(cache, 16) || (lse_opt && !aligned(lse_opt, 4)) ||
        (tree_mask && !aligned(tree_mask, 8)) || (workspace && !aligned(workspace, 16)))
        return DS4HC_ERR_INVALID_ARG;
    if (!rows_apart(N, heads, c->d_latent, os)) return DS4HC_ERR_INVALID_ARG;
    const ds4hc::Paged v = view(c);
    const uint64_t need = ds4hc::attn_workspace_bytes(v, c->d_latent, heads, N);
    if (need > 0 && (!workspace || workspace_bytes < need)) return DS4HC_ERR_INVALID_ARG;
    const uint64_t B = (uint64_t)c->n_seqs;
    const Range in[] = {{q_latent, span(N, heads, c->d_latent, ls, 2)}, {q_rope, span(N, heads, c->d_rope, rs, 2)},
                        {cache, cache_bytes(c)}, {tree_mask, (uint64_t)N * (tree_mask ? mask_words : 0) * 8},
                        {c->cu_q, (B + 1) * 4}, {c->kv_len, B * 4}, {c->block_table, B * c->max_pages * 4}};
    const Range outs[] = {{out, span(N, heads, c->d_latent, os, 2)}, {lse_opt, (uint64_t)N * heads * 4},
                          {need ? workspace : nullptr, need}};
    if (clash(in, outs)) return DS4HC_ERR_INVALID_ARG;
    const ds4hc::AttnArgs a{v, (int)c->dtype, c->d_latent, heads, N, scale, q_latent, ls.token, ls.head,
                            q_rope, rs.token, rs.head, cache, tree_mask, tree_mask ? mask_words : 0, out, os.token,
                            os.head, lse_opt, workspace, 0};
    return done(ds4hc::launch_attn(a, stream));
}

size_t ds4hc_latent_attn_workspace_bytes(const ds4hc_paged_cache *c, int64_t N, int32_t heads) {
    if (check_cache(c, N) != DS4HC_OK || heads < 1 || heads > MAX_HEADS || N * heads > MAX_ROWS || N == 0 || c->n_seqs == 0) return 0;
    return (size_t)ds4hc::attn_workspace_bytes(view(c), c->d_latent, heads, N);
}

ds4hc_status ds4hc_latent_prefill(int64_t N, int64_t S, int32_t n_seqs, int32_t heads,
                                  ds4hc_dtype dtype, float scale, uint32_t flags, const void *q,
                                  const void *kv, const void *k_rope, int64_t k_rope_stride,
                                  const int32_t *cu_q, const int32_t *cu_k, void *out,
                                  float *lse_opt, hipStream_t stream) {
    if (N < 0 || S < 0 || n_seqs < 0 || heads < 1 || !any_type(dtype) || !(scale > 0.f) || !isfinite(scale))
        return DS4HC_ERR_INVALID_ARG;
    if (flags & ~DS4HC_ATTN_FULL) return DS4HC_ERR_INVALID_ARG;
    if (k_rope_stride < ds4hc::LATENT_ROPE || k_rope_stride > MAX_STRIDE || k_rope_stride % 8)
        return DS4HC_ERR_INVALID_ARG;
    if (!half_type(dtype) || heads > MAX_HEADS || N > MAX_T || S > MAX_T || n_seqs > MAX_SEQS ||
        N * heads > MAX_ROWS)
        return DS4HC_ERR_UNSUPPORTED;
    if (N == 0 || n_seqs == 0) return DS4HC_OK;
    // without keys (S = 0) every row sees nothing; kv and k_rope may then be NULL
    if (!q || !cu_q || !cu_k || !out || (S > 0 && (!kv || !k_rope))) return DS4HC_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(k_rope, 16) || !aligned(out, 16) || !aligned(cu_q, 4) ||
        !aligned(cu_k, 4) || (lse_opt && !aligned(lse_opt, 4)))
        return DS4HC_ERR_INVALID_ARG;
    const uint64_t R = (uint64_t)N * heads, B = (uint64_t)n_seqs;
    constexpr uint64_t DQ = ds4hc::PREFILL_NOPE + ds4hc::LATENT_ROPE, DKV = ds4hc::PREFILL_NOPE + ds4hc::PREFILL_VALUE;
    const Range in[] = {{q, R * DQ * 2}, {S ? kv : nullptr, (uint64_t)S * heads * DKV * 2},
                        {S ? k_rope : nullptr, S ? ((uint64_t)(S - 1) * k_rope_stride + ds4hc::LATENT_ROPE) * 2 : 0},
                        {cu_q, (B + 1) * 4}, {cu_k, (B + 1) * 4}};
    const Range outs[] = {{out, R * ds4hc::PREFILL_VALUE * 2}, {lse_opt, R * 4}};
    if (clash(in, outs)) return DS4HC_ERR_INVALID_ARG;
    const ds4hc::PrefillArgs a{N, S, n_seqs, heads, (int)dtype, scale, (flags & DS4HC_ATTN_FULL) != 0, q, kv, k_rope,
                               k_rope_stride, cu_q, cu_k, out, lse_opt};
    return done(ds4hc::launch_prefill(a, stream));
}

}  // extern "C"
