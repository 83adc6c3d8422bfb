// latent_device.hpp -- device-side building blocks of the attention-site
// kernels: 16- and 32-bit element access, the ragged batch, the paged cache.
#pragma once

#include "hc_device.hpp"
#include "hc_launch.hpp"
#include "latent_launch.hpp"

namespace ds4hc {

enum : int { DT_F16 = 2 };

template <int DT> struct ElemOf { using type = uint16_t; };
template <> struct ElemOf<DT_F32> { using type = float; };
template <int DT> using elem_t = typename ElemOf<DT>::type;

template <int DT> __device__ __forceinline__ float elem_load(const elem_t<DT> *p) {
    if constexpr (DT == DT_F32) return *p;
    else if constexpr (DT == DT_BF16) return __uint_as_float((uint32_t)*p << 16);
    else return (float)__builtin_bit_cast(_Float16, *p);
}

// One rounding to nearest even.
template <int DT> __device__ __forceinline__ elem_t<DT> elem_round(float f) {
    if constexpr (DT == DT_F32) return f;
    else if constexpr (DT == DT_BF16) return (uint16_t)f32_to_bf16_bits(f);
    else return __builtin_bit_cast(uint16_t, (_Float16)f);
}

// cu[i] of a ragged batch, held inside the call's `n` tokens.
__device__ __forceinline__ int cu_at(const int32_t *cu, int i, int n) {
    const int v = cu[i];
    return v < 0 ? 0 : v > n ? n : v;
}

// Tokens of sequence b that the cache can hold at all.
__device__ __forceinline__ int kv_len_at(const Paged &c, int b) {
    const int v = c.kv_len[b], most = c.max_pages << c.page_shift;
    return v < 0 ? 0 : v > most ? most : v;
}

// Cache row of token j (0 <= j < max_pages << page_shift) of sequence b, -1 if
// its page is not in the cache.
__device__ __forceinline__ int64_t cache_row(const Paged &c, int b, int j) {
    const int page = c.block_table[(int64_t)b * c.max_pages + (j >> c.page_shift)];
    if (page < 0 || page >= c.n_pages) return -1;
    return ((int64_t)page << c.page_shift) + (j & ((1 << c.page_shift) - 1));
}

// The sequence that token t of the call belongs to: the last b with cu[b] <= t,
// if it ends behind t; -1 if there is none.
__device__ __forceinline__ int sequence_of(const int32_t *cu, int n_seqs, int n, int t) {
    int lo = 0, hi = n_seqs;  // cu[lo] <= t < cu[hi], as far as cu rises
    if (cu_at(cu, 0, n) > t || cu_at(cu, n_seqs, n) <= t) return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu_at(cu, mid, n) <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// cos and sin of position * inv_freq. The angle is formed and reduced to a part
// of a turn in 64 bits (a float32 angle of position 2^20 is off by 2^-5), the
// rest of it, at most half a turn, has 32 bits' precision.
__device__ __forceinline__ void rope_angle(int64_t position, double inv_freq, float amplitude,
                                           float &c, float &s) {
    double turns = (double)position * inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
    turns -= rint(turns);
    float sn, cs;
    sincospif((float)(2.0 * turns), &sn, &cs);
    c = cs * amplitude;
    s = sn * amplitude;
}

}  // namespace ds4hc
