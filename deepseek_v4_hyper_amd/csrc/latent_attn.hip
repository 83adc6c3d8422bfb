// latent_attn.hip -- attention over the paged latent cache, absorbed form.
#include "latent_device.hpp"

namespace ds4hc {

namespace {

// Whether token i of a sequence's `few` call tokens (row t of the mask) sees
// token j of its `len` cached ones.
__device__ __forceinline__ bool attn_sees(const AttnArgs &a, int t, int i, int few, int len, int j) {
    const int d = j - (len - few);  // place among the call's tokens
    if (d < 0) return true;
    if (!a.tree_mask) return d <= i;
    return (d >> 6) < a.mask_words && ((a.tree_mask[(int64_t)t * a.mask_words + (d >> 6)] >> (d & 63)) & 1);
}

// Wave a (token, head): each lane holds LATENT / 64 elements of the latent query
// and the running output and one of the rotated query; one cached token at a time.
template <int DT, int LATENT>
__global__ __launch_bounds__(64) void attn_kernel(AttnArgs a) {
    constexpr int E = LATENT / 64, D = LATENT + LATENT_ROPE;
    const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x, n = (int)a.N;
    const int b = sequence_of(a.c.cu_q, a.c.n_seqs, n, t);
    if (b < 0) return;
    const int q0 = cu_at(a.c.cu_q, b, n), few = cu_at(a.c.cu_q, b + 1, n) - q0, len = kv_len_at(a.c, b);
    const elem_t<DT> *ql = static_cast<const elem_t<DT> *>(a.ql) + t * a.ql_token + h * a.ql_head;
    const elem_t<DT> *qr = static_cast<const elem_t<DT> *>(a.qr) + t * a.qr_token + h * a.qr_head;
    float q[E], acc[E];
    for (int e = 0; e < E; ++e) {
        q[e] = elem_load<DT>(ql + lane * E + e);
        acc[e] = 0.f;
    }
    const float q_rope = elem_load<DT>(qr + lane);
    float top = -INFINITY, total = 0.f;
    for (int j = 0; j < len; ++j) {
        if (!attn_sees(a, t, t - q0, few, len, j)) continue;
        const int64_t row = cache_row(a.c, b, j);
        if (row < 0) continue;
        const elem_t<DT> *x = static_cast<const elem_t<DT> *>(a.cache) + row * D;
        float v[E], s = q_rope * elem_load<DT>(x + LATENT + lane);
        for (int e = 0; e < E; ++e) {
            v[e] = elem_load<DT>(x + lane * E + e);
            s += q[e] * v[e];
        }
        for (int m = 32; m; m >>= 1) s += __shfl_xor(s, m);
        s *= a.scale;
        const float high = fmaxf(top, s), keep = top == high ? 1.f : expf(top - high);
        const float p = expf(s - high);
        total = total * keep + p;
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * keep + p * v[e];
        top = high;
    }
    elem_t<DT> *o = static_cast<elem_t<DT> *>(a.out) + t * a.out_token + h * a.out_head;
    for (int e = 0; e < E; ++e) o[lane * E + e] = elem_round<DT>(total == 0.f ? 0.f : acc[e] / total);
    if (a.lse && lane == 0) a.lse[(int64_t)t * a.heads + h] = total == 0.f ? -INFINITY : top + logf(total);
}

template <int DT>
hipError_t launch_attn_of(const AttnArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)a.N, (unsigned)a.heads);
    switch (a.latent) {
    case 128: return launch_kernel(attn_kernel<DT, 128>, grid, dim3(64), s, a);
    case 256: return launch_kernel(attn_kernel<DT, 256>, grid, dim3(64), s, a);
    default: return launch_kernel(attn_kernel<DT, 512>, grid, dim3(64), s, a);
    }
}

}  // namespace

uint64_t attn_workspace_bytes(const Paged &, int, int, int64_t) { return 0; }

hipError_t launch_attn(const AttnArgs &a, hipStream_t s) {
    return a.dt == DT_BF16 ? launch_attn_of<DT_BF16>(a, s) : launch_attn_of<DT_F16>(a, s);
}

}  // namespace ds4hc
