// serve_api.cpp -- the part of the C ABI declared in include/ds4hc.h that stands around the
// attention of drafted tokens: their verification, the moves of cached rows, and pages. Host-side
// argument validation and launch, as in the other two implementation files.
#include "ds4hc.h"

#include "api_common.hpp"
#include "serve_launch.hpp"

namespace {

using ds4hc::aligned;
using ds4hc::clash;
using ds4hc::MAX_T;
using ds4hc::Range;

constexpr int MAX_SEQS = 65535;  // a dimension of the grid
constexpr int MAX_VOCAB = 1 << 24;
constexpr int64_t MAX_KV = int64_t(1) << 30;  // tokens of a sequence
constexpr int64_t MAX_ITEMS = int64_t(1) << 20;
constexpr int64_t MAX_STRIDE = int64_t(1) << 36;  // offsets stay far inside 64 bits

ds4hc_status done(hipError_t e) { return e == hipSuccess ? DS4HC_OK : ds4hc::hip_fail(e); }
bool power_of_2(int v) { return v > 0 && (v & (v - 1)) == 0; }

ds4hc_status check_store(const ds4hc_page_store *s) {
    if (!s || s->layers < 1 || !power_of_2(s->page_size) || s->n_pages < 1 || s->row_bytes < 16 || s->row_bytes % 16)
        return DS4HC_ERR_INVALID_ARG;
    if (s->layers > 65535 || s->page_size > 65536 || s->n_pages > (int64_t(1) << 31) - 1 ||
        s->n_pages * s->page_size >= (int64_t(1) << 31) || s->row_bytes > 65536)
        return DS4HC_ERR_UNSUPPORTED;
    if (s->layers > 1) {
        if (s->layer_stride % 16 || s->layer_stride < s->n_pages * s->page_size * s->row_bytes) return DS4HC_ERR_INVALID_ARG;
        if (s->layer_stride > (int64_t(1) << 46)) return DS4HC_ERR_UNSUPPORTED;
    }
    return DS4HC_OK;
}

uint64_t store_bytes(const ds4hc_page_store *s) {
    return (uint64_t)(s->layers - 1) * s->layer_stride + (uint64_t)s->n_pages * s->page_size * s->row_bytes;
}

ds4hc::Store view(const ds4hc_page_store *s) {
    return {s->layers, __builtin_ctz((unsigned)s->page_size), s->n_pages, s->row_bytes, s->layers > 1 ? s->layer_stride : 0,
            static_cast<char *>(s->data)};
}

ds4hc_status check_pool(const ds4hc_page_pool *p, int64_t n) {
    if (!p || n < 0 || !power_of_2(p->page_size) || p->n_slots < 1 || p->max_pages < 1 || p->n_pages < 1)
        return DS4HC_ERR_INVALID_ARG;
    if (p->page_size > 65536 || p->n_slots > (1 << 20) || (int64_t)p->max_pages * p->page_size > MAX_KV ||
        p->n_pages > (1 << 28) || n > MAX_ITEMS)
        return DS4HC_ERR_UNSUPPORTED;
    return DS4HC_OK;
}

// The arrays that a resize and a fork have alike. `copies` of a fork: null.
ds4hc_status check_items(const ds4hc_page_pool *p, int64_t n, const int32_t *a, const int32_t *b, int32_t *copies, bool with_copies,
                         int32_t *status, void *ws, size_t ws_bytes) {
    if (!p->block_table || !p->kv_len || !p->refs || !a || !b || (with_copies && !copies) || !status || !ws) return DS4HC_ERR_INVALID_ARG;
    for (const void *q : {(const void *)p->block_table, (const void *)p->kv_len, (const void *)p->refs, (const void *)a, (const void *)b,
                          (const void *)copies, (const void *)status})
        if (!aligned(q, 4)) return DS4HC_ERR_INVALID_ARG;
    const uint64_t need = ds4hc::pages_workspace_bytes(p->n_slots, p->n_pages, n);
    if (!aligned(ws, 16) || ws_bytes < need) return DS4HC_ERR_INVALID_ARG;
    const Range in[] = {{a, (uint64_t)n * 4}, {b, (uint64_t)n * 4}};
    const Range out[] = {{p->block_table, (uint64_t)p->n_slots * p->max_pages * 4}, {p->kv_len, (uint64_t)p->n_slots * 4},
                         {p->refs, (uint64_t)p->n_pages * 4}, {copies, (uint64_t)n * 8}, {status, (uint64_t)n * 4}, {ws, need}};
    return clash(in, out) ? DS4HC_ERR_INVALID_ARG : DS4HC_OK;
}

}  // namespace

extern "C" {

size_t ds4hc_draft_verify_workspace_bytes(int32_t n_seqs, int32_t vocab) {
    if (n_seqs < 1 || n_seqs > MAX_SEQS || vocab < 1 || vocab > MAX_VOCAB) return 0;
    return (size_t)ds4hc::verify_workspace_bytes(n_seqs, vocab);
}

ds4hc_status ds4hc_draft_verify(int64_t N, int32_t n_seqs, int32_t vocab, const float *target, int64_t target_stride,
                                const float *draft, int64_t draft_stride, const int64_t *tokens, const int32_t *parents,
                                const int32_t *cu_q, const float *uniform, int32_t *path, int32_t *n_kept, int64_t *next,
                                void *workspace, size_t workspace_bytes, hipStream_t stream) {
    if (N < 0 || n_seqs < 0 || vocab < 1 || target_stride < vocab || target_stride > MAX_STRIDE ||
        (draft && (draft_stride < vocab || draft_stride > MAX_STRIDE)) || (draft && parents))
        return DS4HC_ERR_INVALID_ARG;
    if (N > MAX_T || n_seqs > MAX_SEQS || vocab > MAX_VOCAB) return DS4HC_ERR_UNSUPPORTED;
    if (n_seqs == 0) return DS4HC_OK;
    // without tokens (N = 0) every sequence is empty: n_kept 0, next -1
    if (!cu_q || !n_kept || !next || !workspace || (N > 0 && (!target || !tokens || !uniform || !path))) return DS4HC_ERR_INVALID_ARG;
    if (!aligned(target, 4) || !aligned(draft, 4) || !aligned(tokens, 8) || !aligned(parents, 4) || !aligned(cu_q, 4) ||
        !aligned(uniform, 4) || !aligned(path, 4) || !aligned(n_kept, 4) || !aligned(next, 8) || !aligned(workspace, 16))
        return DS4HC_ERR_INVALID_ARG;
    const uint64_t need = ds4hc::verify_workspace_bytes(n_seqs, vocab), B = (uint64_t)n_seqs;
    if (workspace_bytes < need) return DS4HC_ERR_INVALID_ARG;
    const uint64_t rows = N ? (uint64_t)(N - 1) : 0, on = N ? 1 : 0;
    const Range in[] = {{target, on * (rows * target_stride + vocab) * 4}, {draft, on * (rows * draft_stride + vocab) * 4},
                        {tokens, (uint64_t)N * 8}, {parents, (uint64_t)N * 4}, {cu_q, (B + 1) * 4}, {uniform, (uint64_t)N * 4}};
    const Range out[] = {{path, (uint64_t)N * 4}, {n_kept, B * 4}, {next, B * 8}, {workspace, need}};
    if (clash(in, out)) return DS4HC_ERR_INVALID_ARG;
    return done(ds4hc::launch_verify({N, n_seqs, vocab, target, target_stride, draft, draft_stride, tokens, parents, cu_q, uniform, path,
                                      n_kept, next, workspace, 0}, stream));
}

ds4hc_status ds4hc_cache_compact(const ds4hc_page_store *s, int64_t N, int32_t n_seqs, int32_t max_pages, const int32_t *cu_q,
                                 const int32_t *kv_len, const int32_t *block_table, const int32_t *keep, const int32_t *n_keep,
                                 hipStream_t stream) {
    const ds4hc_status st = check_store(s);
    if (st != DS4HC_OK) return st;
    if (N < 0 || n_seqs < 0 || max_pages < 1) return DS4HC_ERR_INVALID_ARG;
    if (N > MAX_T || n_seqs > MAX_SEQS || (int64_t)max_pages * s->page_size > MAX_KV) return DS4HC_ERR_UNSUPPORTED;
    if (N == 0 || n_seqs == 0) return DS4HC_OK;
    if (!s->data || !cu_q || !kv_len || !block_table || !keep || !n_keep || !aligned(s->data, 16)) return DS4HC_ERR_INVALID_ARG;
    for (const int32_t *q : {cu_q, kv_len, block_table, keep, n_keep})
        if (!aligned(q, 4)) return DS4HC_ERR_INVALID_ARG;
    const uint64_t B = (uint64_t)n_seqs;
    const Range in[] = {{cu_q, (B + 1) * 4}, {kv_len, B * 4}, {block_table, B * max_pages * 4}, {keep, (uint64_t)N * 4}, {n_keep, B * 4}};
    const Range out[] = {{s->data, store_bytes(s)}};
    if (clash(in, out)) return DS4HC_ERR_INVALID_ARG;
    return done(ds4hc::launch_compact({view(s), N, n_seqs, max_pages, cu_q, kv_len, block_table, keep, n_keep}, stream));
}

ds4hc_status ds4hc_pages_copy(const ds4hc_page_store *s, int64_t n, const int32_t *pairs, hipStream_t stream) {
    const ds4hc_status st = check_store(s);
    if (st != DS4HC_OK) return st;
    if (n < 0) return DS4HC_ERR_INVALID_ARG;
    if (n > MAX_ITEMS) return DS4HC_ERR_UNSUPPORTED;
    if (n == 0) return DS4HC_OK;
    if (!s->data || !pairs || !aligned(s->data, 16) || !aligned(pairs, 4)) return DS4HC_ERR_INVALID_ARG;
    const Range in[] = {{pairs, (uint64_t)n * 8}}, out[] = {{s->data, store_bytes(s)}};
    if (clash(in, out)) return DS4HC_ERR_INVALID_ARG;
    return done(ds4hc::launch_pages_copy(view(s), n, pairs, stream));
}

size_t ds4hc_pages_workspace_bytes(const ds4hc_page_pool *p, int64_t n) {
    if (check_pool(p, n) != DS4HC_OK || n == 0) return 0;
    return (size_t)ds4hc::pages_workspace_bytes(p->n_slots, p->n_pages, n);
}

ds4hc_status ds4hc_pages_resize(const ds4hc_page_pool *p, int64_t n, const int32_t *slots, const int32_t *lengths, int32_t *copies,
                                int32_t *status, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    ds4hc_status st = check_pool(p, n);
    if (st != DS4HC_OK || n == 0) return st;
    st = check_items(p, n, slots, lengths, copies, true, status, workspace, workspace_bytes);
    if (st != DS4HC_OK) return st;
    return done(ds4hc::launch_pages_resize({__builtin_ctz((unsigned)p->page_size), p->n_slots, p->max_pages, p->n_pages, p->block_table,
                                            p->kv_len, p->refs, (int)n, slots, lengths, copies, status, workspace}, stream));
}

ds4hc_status ds4hc_pages_fork(const ds4hc_page_pool *p, int64_t n, const int32_t *parents, const int32_t *children, int32_t *status,
                              void *workspace, size_t workspace_bytes, hipStream_t stream) {
    ds4hc_status st = check_pool(p, n);
    if (st != DS4HC_OK || n == 0) return st;
    st = check_items(p, n, parents, children, nullptr, false, status, workspace, workspace_bytes);
    if (st != DS4HC_OK) return st;
    return done(ds4hc::launch_pages_fork({__builtin_ctz((unsigned)p->page_size), p->n_slots, p->max_pages, p->n_pages, p->block_table,
                                          p->kv_len, p->refs, (int)n, children, parents, nullptr, status, workspace}, stream));
}

}  // extern "C"
