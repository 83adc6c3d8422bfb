// rope_kernels.hip -- rotary positions, and the append of normed, rotated latent
// vectors to the paged cache.
#include "latent_device.hpp"

namespace ds4hc {

namespace {

// Thread a pair: grid (tokens, blocks of heads * pairs).
template <int DT>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a) {
    const int pairs = a.dim >> 1, item = blockIdx.y * 256 + threadIdx.x;
    if (item >= a.heads * pairs) return;
    const int64_t t = blockIdx.x;
    const int h = item / pairs, i = item - h * pairs;
    float c, s;
    rope_angle(a.positions[t], a.inv_freq[i], a.amplitude, c, s);
    if (a.inverse) s = -s;
    const int i0 = a.half ? i : 2 * i, i1 = a.half ? i + pairs : 2 * i + 1;
    const elem_t<DT> *x = static_cast<const elem_t<DT> *>(a.x) + t * a.x_token + h * a.x_head;
    elem_t<DT> *y = static_cast<elem_t<DT> *>(a.y) + t * a.y_token + h * a.y_head;
    const float x0 = elem_load<DT>(x + i0), x1 = elem_load<DT>(x + i1);
    y[i0] = elem_round<DT>(x0 * c - x1 * s);
    y[i1] = elem_round<DT>(x0 * s + x1 * c);
}

// Wave a token.
template <int SRC, int DT>
__global__ __launch_bounds__(64) void append_kernel(AppendArgs a) {
    const int t = blockIdx.x, lane = threadIdx.x, n = (int)a.N;
    const int b = sequence_of(a.c.cu_q, a.c.n_seqs, n, t);
    if (b < 0) return;
    const int q1 = cu_at(a.c.cu_q, b + 1, n), j = kv_len_at(a.c, b) - (q1 - t);
    if (j < 0) return;
    const int64_t row = cache_row(a.c, b, j);
    if (row < 0) return;
    const int D = a.latent + LATENT_ROPE;
    const elem_t<SRC> *x = static_cast<const elem_t<SRC> *>(a.kv) + (int64_t)t * a.kv_stride;
    elem_t<DT> *y = static_cast<elem_t<DT> *>(a.cache) + row * D;
    float inv = 1.f;
    if (a.norm_weight) {
        float ss = 0.f;
        for (int i = lane; i < a.latent; i += 64) {
            const float v = elem_load<SRC>(x + i);
            ss += v * v;
        }
        for (int m = 32; m; m >>= 1) ss += __shfl_xor(ss, m);
        inv = 1.f / sqrtf(ss / a.latent + a.rms_eps);
    }
    for (int i = lane; i < a.latent; i += 64) {
        const float v = elem_load<SRC>(x + i);
        y[i] = elem_round<DT>(a.norm_weight ? v * inv * a.norm_weight[i] : v);
    }
    if (lane < LATENT_ROPE / 2) {
        float c, s;
        rope_angle(a.positions[t], a.inv_freq[lane], a.amplitude, c, s);
        const int i0 = a.latent + (a.half ? lane : 2 * lane), i1 = a.half ? i0 + LATENT_ROPE / 2 : i0 + 1;
        const float x0 = elem_load<SRC>(x + i0), x1 = elem_load<SRC>(x + i1);
        y[i0] = elem_round<DT>(x0 * c - x1 * s);
        y[i1] = elem_round<DT>(x0 * s + x1 * c);
    }
}

}  // namespace

hipError_t launch_rope(const RopeArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)a.N, (unsigned)((a.heads * (a.dim / 2) + 255) / 256));
    switch (a.dt) {
    case DT_F32: return launch_kernel(rope_kernel<DT_F32>, grid, dim3(256), s, a);
    case DT_BF16: return launch_kernel(rope_kernel<DT_BF16>, grid, dim3(256), s, a);
    default: return launch_kernel(rope_kernel<DT_F16>, grid, dim3(256), s, a);
    }
}

template <int DT>
static hipError_t launch_append_to(const AppendArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)a.N);
    switch (a.src_dt) {
    case DT_F32: return launch_kernel(append_kernel<DT_F32, DT>, grid, dim3(64), s, a);
    case DT_BF16: return launch_kernel(append_kernel<DT_BF16, DT>, grid, dim3(64), s, a);
    default: return launch_kernel(append_kernel<DT_F16, DT>, grid, dim3(64), s, a);
    }
}

hipError_t launch_append(const AppendArgs &a, hipStream_t s) {
    return a.dt == DT_BF16 ? launch_append_to<DT_BF16>(a, s) : launch_append_to<DT_F16>(a, s);
}

}  // namespace ds4hc
