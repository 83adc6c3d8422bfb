// latent_prefill.hip -- attention over expanded keys and values of a ragged batch.
#include "latent_device.hpp"

namespace ds4hc {

namespace {

// Wave a (query, head): each lane holds 3 elements of the query and 2 of the
// running output; one key at a time.
template <int DT>
__global__ __launch_bounds__(64) void prefill_kernel(PrefillArgs a) {
    constexpr int DQ = PREFILL_NOPE + LATENT_ROPE, DKV = PREFILL_NOPE + PREFILL_VALUE;
    const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x, n = (int)a.N;
    const int b = sequence_of(a.cu_q, a.n_seqs, n, t);
    if (b < 0) return;
    const int q0 = cu_at(a.cu_q, b, n), few = cu_at(a.cu_q, b + 1, n) - q0;
    const int k0 = cu_at(a.cu_k, b, (int)a.S), len = max(cu_at(a.cu_k, b + 1, (int)a.S) - k0, 0);
    const int seen = a.full ? len : min(len, t - q0 + len - few + 1);
    const elem_t<DT> *q = static_cast<const elem_t<DT> *>(a.q) + ((int64_t)t * a.heads + h) * DQ;
    const float qa = elem_load<DT>(q + lane), qb = elem_load<DT>(q + 64 + lane), qr = elem_load<DT>(q + 128 + lane);
    float top = -INFINITY, total = 0.f, oa = 0.f, ob = 0.f;
    for (int j = 0; j < seen; ++j) {
        const elem_t<DT> *k = static_cast<const elem_t<DT> *>(a.kv) + ((int64_t)(k0 + j) * a.heads + h) * DKV;
        const elem_t<DT> *r = static_cast<const elem_t<DT> *>(a.k_rope) + (int64_t)(k0 + j) * a.k_rope_stride;
        float s = qa * elem_load<DT>(k + lane) + qb * elem_load<DT>(k + 64 + lane) + qr * elem_load<DT>(r + lane);
        for (int m = 32; m; m >>= 1) s += __shfl_xor(s, m);
        s *= a.scale;
        const float high = fmaxf(top, s), keep = top == high ? 1.f : expf(top - high);
        const float p = expf(s - high);
        total = total * keep + p;
        oa = oa * keep + p * elem_load<DT>(k + 128 + lane);
        ob = ob * keep + p * elem_load<DT>(k + 192 + lane);
        top = high;
    }
    elem_t<DT> *o = static_cast<elem_t<DT> *>(a.out) + ((int64_t)t * a.heads + h) * PREFILL_VALUE;
    o[lane] = elem_round<DT>(total == 0.f ? 0.f : oa / total);
    o[64 + lane] = elem_round<DT>(total == 0.f ? 0.f : ob / total);
    if (a.lse && lane == 0) a.lse[(int64_t)t * a.heads + h] = total == 0.f ? -INFINITY : top + logf(total);
}

}  // namespace

hipError_t launch_prefill(const PrefillArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)a.N, (unsigned)a.heads);
    return a.dt == DT_BF16 ? launch_kernel(prefill_kernel<DT_BF16>, grid, dim3(64), s, a)
                           : launch_kernel(prefill_kernel<DT_F16>, grid, dim3(64), s, a);
}

}  // namespace ds4hc
