// latent_launch.hpp -- internal interface between the C ABI (latent_api.cpp)
// and the kernels of an attention site (rope_kernels.hip, latent_attn.hip,
// latent_attn8.hip, latent_prefill.hip). Arguments have been validated. Not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ds4hc {

constexpr int LATENT_ROPE = 64;    // rotated part of a cached vector and of a head
constexpr int PREFILL_NOPE = 128;  // unrotated part of an expanded head
constexpr int PREFILL_VALUE = 128;

struct RopeArgs {
    int64_t N;
    int heads, dim, dt;
    const void *x;
    int64_t x_token, x_head;
    const int64_t *positions;
    const double *inv_freq;
    float amplitude;
    bool half, inverse;
    void *y;
    int64_t y_token, y_head;
};
hipError_t launch_rope(const RopeArgs &a, hipStream_t s);

// Device view of a ds4hc_paged_cache.
struct Paged {
    int page_shift;
    int n_seqs, max_pages;
    int64_t n_pages;
    const int32_t *cu_q, *kv_len, *block_table;
};

struct AppendArgs {
    Paged c;
    int dt, latent, src_dt;
    int64_t N;
    const void *kv;
    int64_t kv_stride;
    const float *norm_weight;  // may be null
    float rms_eps;
    const int64_t *positions;
    const double *inv_freq;
    float amplitude;
    bool half;
    void *cache;
    bool eight;  // a cache of 8-bit latents
};
hipError_t launch_append(const AppendArgs &a, hipStream_t s);

struct AttnArgs {
    Paged c;
    int dt, latent, heads;
    int64_t N;
    float scale;
    const void *ql;
    int64_t ql_token, ql_head;
    const void *qr;
    int64_t qr_token, qr_head;
    const void *cache;
    const uint64_t *tree_mask;  // may be null
    int mask_words;
    void *out;
    int64_t out_token, out_head;
    float *lse;  // may be null
    void *ws;
    int members;  // workgroups of a cluster: launch_attn sets it
};
uint64_t attn8_workspace_bytes(const Paged &c, int latent, int heads, int64_t N);
hipError_t launch_attn8(const AttnArgs &a, hipStream_t s);  // cache rows of 8-bit latents
uint64_t attn_workspace_bytes(const Paged &c, int latent, int heads, int64_t N);
hipError_t launch_attn(const AttnArgs &a, hipStream_t s);

struct PrefillArgs {
    int64_t N, S;
    int n_seqs, heads, dt;
    float scale;
    bool full;
    const void *q, *kv, *k_rope;
    int64_t k_rope_stride;
    const int32_t *cu_q, *cu_k;
    void *out;
    float *lse;  // may be null
};
hipError_t launch_prefill(const PrefillArgs &a, hipStream_t s);

}  // namespace ds4hc
