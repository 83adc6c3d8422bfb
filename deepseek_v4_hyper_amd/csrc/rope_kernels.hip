// rope_kernels.hip -- rotary positions, and the append of normed, rotated latent
// vectors to the paged cache. Both move each element once; what is computed beside
// that, an angle in 64 bits with its cosine and sine, is made once a token and pair
// and shared by the heads.
#include "latent_device.hpp"

namespace ds4hc {

namespace {

constexpr int THREADS = 256;
constexpr int MAX_PAIRS = 256;     // of a head: dim <= 512
constexpr int MAX_SPLITS = 64;     // workgroups a token at most
constexpr unsigned GRID_X = 1u << 20;  // tokens in x (a dispatch has fewer than 2^32 threads a dimension)

// 16 bytes of consecutive elements of one row, widened.
template <int DT> struct Vec {
    static constexpr int V = DT == DT_F32 ? 4 : 8;
    float f[V];
    __device__ __forceinline__ void load(const elem_t<DT> *p) {
        const u32x4_t w = *reinterpret_cast<const u32x4_t *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == DT_F32) f[i] = __uint_as_float(w[i]);
            else if constexpr (DT == DT_BF16) f[2 * i] = bf16_lo(w[i]), f[2 * i + 1] = bf16_hi(w[i]);
            else f[2 * i] = f16_lo(w[i]), f[2 * i + 1] = f16_hi(w[i]);
        }
    }
    __device__ __forceinline__ void store(elem_t<DT> *p) const {
        u32x4_t w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == DT_F32) w[i] = __float_as_uint(f[i]);
            else w[i] = pack2<DT>(f[2 * i], f[2 * i + 1]);
        }
        *reinterpret_cast<u32x4_t *>(p) = w;
    }
};

// Contracted by hand, and kept in float32 up to the store (not joined with a conversion to
// float16, which would round once instead of twice), so that every variant gives the same bits.
template <int DT> __device__ __forceinline__ void turn(float &x0, float &x1, float c, float s) {
    float y0 = fmaf(x0, c, -(x1 * s)), y1 = fmaf(x0, s, x1 * c);
    if constexpr (DT == DT_F16) asm("" : "+v"(y0), "+v"(y1));
    x0 = y0;
    x1 = y1;
}

// Bound by memory: 4096 tokens x 128 heads x 64, bf16, take 21.9 us (6.1 TB/s of 134 MB), 25.2 us
// a call in a chain of them; a few tokens 3.1 us, a launch. Simple pairs of 2-byte loads took 70 us.
// A workgroup some heads of one token: grid (tokens, splits of the heads, tokens / 2^20). The token's
// cosines and sines go to LDS first; then each thread turns 16 bytes at a time (VECTOR:
// rows on 16-byte boundaries, dim a multiple of what they hold; half layout: of twice that,
// 16 bytes of either half), or one pair.
template <int DT, bool HALF, bool VECTOR>
__global__ __launch_bounds__(THREADS) void rope_kernel(RopeArgs a) {
    __shared__ __align__(16) float cosine[MAX_PAIRS], sine[MAX_PAIRS];
    const int64_t t = (int64_t)blockIdx.z * GRID_X + blockIdx.x;
    if (t >= a.N) return;
    const int pairs = a.dim >> 1;
    const int64_t position = a.positions[t];
    for (int i = threadIdx.x; i < pairs; i += THREADS) {
        float c, s;
        rope_angle(position, a.inv_freq[i], a.amplitude, c, s);
        cosine[i] = c;
        sine[i] = a.inverse ? -s : s;
    }
    __syncthreads();
    constexpr int V = VECTOR ? Vec<DT>::V : 1;
    const int each = VECTOR ? (HALF ? pairs / V : a.dim / V) : pairs;  // pieces a head
    const elem_t<DT> *x = static_cast<const elem_t<DT> *>(a.x) + t * a.x_token;
    elem_t<DT> *y = static_cast<elem_t<DT> *>(a.y) + t * a.y_token;
    const int pieces = a.heads * each;
#pragma unroll 1  // (4: the same within 2 % for all types and layouts, 2 % slower for one head)
    for (int k = blockIdx.y * THREADS + threadIdx.x; k < pieces; k += gridDim.y * THREADS) {
        const int h = k / each, i = k - h * each;
        const elem_t<DT> *xh = x + h * a.x_head;
        elem_t<DT> *yh = y + h * a.y_head;
        if constexpr (!VECTOR) {
            const int i0 = HALF ? i : 2 * i, i1 = HALF ? i + pairs : 2 * i + 1;
            float x0 = elem_load<DT>(xh + i0), x1 = elem_load<DT>(xh + i1);
            turn<DT>(x0, x1, cosine[i], sine[i]);
            yh[i0] = elem_round<DT>(x0);
            yh[i1] = elem_round<DT>(x1);
        } else if constexpr (HALF) {
            Vec<DT> p, q;
            p.load(xh + i * V);
            q.load(xh + pairs + i * V);
#pragma unroll
            for (int e = 0; e < V; ++e) turn<DT>(p.f[e], q.f[e], cosine[i * V + e], sine[i * V + e]);
            p.store(yh + i * V);
            q.store(yh + pairs + i * V);
        } else {
            Vec<DT> p;
            p.load(xh + i * V);
#pragma unroll
            for (int e = 0; e < V / 2; ++e) turn<DT>(p.f[2 * e], p.f[2 * e + 1], cosine[i * (V / 2) + e], sine[i * (V / 2) + e]);
            p.store(yh + i * V);
        }
    }
}

// The sequence that token t of the call belongs to, -1 if there is none: the last one that
// starts at or before it, if it ends behind it (where cu rises, the only one that holds it).
// All lanes of a wave look at a sequence each.
__device__ __forceinline__ int sequence_by_wave(const int32_t *cu, int n_seqs, int n, int t) {
    const int lane = threadIdx.x & 63;
    int found = -1;
    for (int b0 = 0; b0 < n_seqs; b0 += 64) {
        const int b = b0 + lane;
        const bool in = b < n_seqs && cu_at(cu, b, n) <= t && cu_at(cu, b + 1, n) > t;
        const uint64_t who = __ballot(in);
        if (who) found = b0 + 63 - __builtin_clzll(who);
    }
    return found;
}

// Bound by memory, and in small calls by the chain of loads (sequence, length, page) before the
// first store, beside which the row's own loads run: 32 tokens 3.4 us; 4096 float32 rows of 576
// 5.5 us (16 MB, 2.9 TB/s).
// A wave a token: LATENT / 64 consecutive elements a lane, and a pair of the rope key for each
// of the first 32 lanes. The row is read once, kept in registers over the sum of its squares.
template <int SRC, int DT, int LATENT>
__global__ __launch_bounds__(64) void append_kernel(AppendArgs a) {
    constexpr int E = LATENT / 64, D = LATENT + LATENT_ROPE;
    const int t = blockIdx.x, lane = threadIdx.x, n = (int)a.N;
    // loads that do not wait for the token's place
    const elem_t<SRC> *x = static_cast<const elem_t<SRC> *>(a.kv) + (int64_t)t * a.kv_stride;
    float v[E];
    if constexpr (E * sizeof(elem_t<SRC>) % 16 == 0) {
        constexpr int V = Vec<SRC>::V;
#pragma unroll
        for (int i = 0; i < E / V; ++i) {
            Vec<SRC> w;
            w.load(x + lane * E + i * V);
#pragma unroll
            for (int e = 0; e < V; ++e) v[i * V + e] = w.f[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = elem_load<SRC>(x + lane * E + e);
    }
    const int i0 = a.half ? lane & 31 : 2 * (lane & 31), i1 = a.half ? i0 + LATENT_ROPE / 2 : i0 + 1;
    float x0 = elem_load<SRC>(x + LATENT + i0), x1 = elem_load<SRC>(x + LATENT + i1);
    float w[E];
    if (a.norm_weight)
#pragma unroll
        for (int e = 0; e < E; ++e) w[e] = a.norm_weight[lane * E + e];
    const int64_t position = a.positions[t];
    const double inv_freq = a.inv_freq[lane & 31];

    const int b = sequence_by_wave(a.c.cu_q, a.c.n_seqs, n, t);
    if (b < 0) return;
    const int j = kv_len_at(a.c, b) - (cu_at(a.c.cu_q, b + 1, n) - t);
    if (j < 0) return;
    const int64_t row = cache_row(a.c, b, j);
    if (row < 0) return;
    elem_t<DT> *y = static_cast<elem_t<DT> *>(a.cache) + row * D;
    if (a.norm_weight) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) ss += v[e] * v[e];
        for (int m = 32; m; m >>= 1) ss += __shfl_xor(ss, m);
        const float inv = 1.f / sqrtf(ss / LATENT + a.rms_eps);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] *= inv * w[e];
    }
    if constexpr (E == 8) {
        Vec<DT> o;
#pragma unroll
        for (int e = 0; e < E; ++e) o.f[e] = v[e];
        o.store(y + lane * E);
    } else {
#pragma unroll
        for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t *>(y + lane * E + e) = pack2<DT>(v[e], v[e + 1]);
    }
    if (lane < LATENT_ROPE / 2) {
        float c, s;
        rope_angle(position, inv_freq, a.amplitude, c, s);
        turn<DT>(x0, x1, c, s);
        if (a.half) {
            y[LATENT + i0] = elem_round<DT>(x0);
            y[LATENT + i1] = elem_round<DT>(x1);
        } else {
            *reinterpret_cast<uint32_t *>(y + LATENT + i0) = pack2<DT>(x0, x1);
        }
    }
}

template <int DT> hipError_t launch_rope_of(const RopeArgs &a, hipStream_t s) {
    constexpr int V = Vec<DT>::V, B = sizeof(elem_t<DT>);
    const bool rows16 = ((uintptr_t)a.x | (uintptr_t)a.y | (uintptr_t)((a.x_token | a.y_token | a.x_head | a.y_head) * B)) % 16 == 0;
    const bool vector = rows16 && a.dim % (a.half ? 2 * V : V) == 0;
    // a workgroup has four pieces a thread where the tokens alone fill the chip (they share the
    // token's cosines and sines, 32 or more of them in 64 bits), one where they do not. bf16, heads x
    // 64, four pieces and one: 128 heads, 256 tokens 4.4 and 4.0 us, 512 5.1 and 5.0, 1024 7.1 and 7.6,
    // 4096 22.8 and 23.4, 8192 45 and 56; 64 heads, 1024 tokens 4.8 and 5.0, 2048 6.9 and 7.5, 8192 22.6 and
    // 23.5; up to 32 heads (256 pieces) both are the same launch. float32, 128 heads, 1024 tokens 12.6 and 13.0,
    // 8192 111 and 115. Half layout: equal within 2 % but for 16-bit types at 8192 x 128, 55 and 48. Pairs in
    // place of 16 bytes, what rows on other boundaries get: 1024 x 128 11.3 and 16.5, 8192 x 128 94 and 157,
    // 8192 x 8 9.3 and 9.4, 8192 x 1 5.6 either way.
    const int pieces = a.heads * (a.dim / 2) / (vector ? (a.half ? V : V / 2) : 1);
    const int64_t by_token = a.N >= 1024 ? 4 : 1;
    const int64_t splits = (pieces + THREADS * by_token - 1) / (THREADS * by_token);
    const dim3 grid((unsigned)(a.N < GRID_X ? a.N : GRID_X), (unsigned)(splits < MAX_SPLITS ? splits : MAX_SPLITS), (unsigned)((a.N + GRID_X - 1) / GRID_X));
    if (a.half) return vector ? launch_kernel(rope_kernel<DT, true, true>, grid, dim3(THREADS), s, a)
                              : launch_kernel(rope_kernel<DT, true, false>, grid, dim3(THREADS), s, a);
    return vector ? launch_kernel(rope_kernel<DT, false, true>, grid, dim3(THREADS), s, a)
                  : launch_kernel(rope_kernel<DT, false, false>, grid, dim3(THREADS), s, a);
}

template <int SRC, int DT> hipError_t launch_append_of(const AppendArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)a.N);
    switch (a.latent) {
    case 128: return launch_kernel(append_kernel<SRC, DT, 128>, grid, dim3(64), s, a);
    case 256: return launch_kernel(append_kernel<SRC, DT, 256>, grid, dim3(64), s, a);
    default: return launch_kernel(append_kernel<SRC, DT, 512>, grid, dim3(64), s, a);
    }
}

template <int DT> hipError_t launch_append_to(const AppendArgs &a, hipStream_t s) {
    switch (a.src_dt) {
    case DT_F32: return launch_append_of<DT_F32, DT>(a, s);
    case DT_BF16: return launch_append_of<DT_BF16, DT>(a, s);
    default: return launch_append_of<DT_F16, DT>(a, s);
    }
}

}  // namespace

hipError_t launch_rope(const RopeArgs &a, hipStream_t s) {
    switch (a.dt) {
    case DT_F32: return launch_rope_of<DT_F32>(a, s);
    case DT_BF16: return launch_rope_of<DT_BF16>(a, s);
    default: return launch_rope_of<DT_F16>(a, s);
    }
}

hipError_t launch_append(const AppendArgs &a, hipStream_t s) {
    return a.dt == DT_BF16 ? launch_append_to<DT_BF16>(a, s) : launch_append_to<DT_F16>(a, s);
}

}  // namespace ds4hc
