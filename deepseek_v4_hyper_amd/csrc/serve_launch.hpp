// serve_launch.hpp -- internal interface between the C ABI (serve_api.cpp) and the kernels around
// the attention of drafted tokens (draft_kernels.hip, page_kernels.hip). Arguments have been
// validated. Not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ds4hc {

struct VerifyArgs {
    int64_t N;
    int n_seqs, vocab;
    const float *target;
    int64_t target_stride;
    const float *draft;  // may be null
    int64_t draft_stride;
    const int64_t *tokens;
    const int32_t *parents;  // may be null
    const int32_t *cu_q;
    const float *uniform;
    int32_t *path, *n_kept;
    int64_t *next;
    void *ws;
    int chunk;  // elements of a row that a workgroup sums: launch_verify sets it
};
uint64_t verify_workspace_bytes(int n_seqs, int vocab);
hipError_t launch_verify(const VerifyArgs &a, hipStream_t s);

// Device view of a ds4hc_page_store.
struct Store {
    int layers, page_shift;
    int64_t n_pages, row_bytes, layer_stride;
    char *data;
};

struct CompactArgs {
    Store s;
    int64_t N;
    int n_seqs, max_pages;
    const int32_t *cu_q, *kv_len, *block_table, *keep, *n_keep;
};
hipError_t launch_compact(const CompactArgs &a, hipStream_t s);
hipError_t launch_pages_copy(const Store &st, int64_t n, const int32_t *pairs, hipStream_t s);

// Device view of a ds4hc_page_pool, and a call's items.
struct PoolArgs {
    int page_shift, n_slots, max_pages, n_pages;
    int32_t *block_table, *kv_len, *refs;
    int n;
    const int32_t *slots;    // of a fork: the children
    const int32_t *lengths;  // of a fork: the parents
    int32_t *copies, *status;
    void *ws;
};
uint64_t pages_workspace_bytes(int n_slots, int n_pages, int64_t n);
hipError_t launch_pages_resize(const PoolArgs &a, hipStream_t s);
hipError_t launch_pages_fork(const PoolArgs &a, hipStream_t s);

}  // namespace ds4hc
