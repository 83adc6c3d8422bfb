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

// A value that is the same in all lanes, loaded through the scalar cache. For arrays that
// no kernel of the library writes.
__device__ __forceinline__ int scalar_load(const int32_t *p, int64_t i) {
    return ((const __attribute__((address_space(4))) int32_t *)(uintptr_t)p)[i];
}

// Values that are the same in all lanes, into scalar registers.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
    return ((int64_t)uniform((int)(v >> 32)) << 32) | (uint32_t)uniform((int)v);
}

// The value, computed anew where it stands: keeps what is made of it from being kept in
// registers over a loop.
__device__ __forceinline__ uint32_t here(uint32_t v) {
    asm volatile("" : "+v"(v));
    return v;
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

// ------------------------------------------------------------------ matrix tiles

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef float acc4_t __attribute__((ext_vector_type(4)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));

#define DS4HC_LDS __attribute__((address_space(3)))
#define DS4HC_GLOBAL __attribute__((address_space(1)))

// C[16 x 16] += A[16 x 32] B[32 x 16]. Lane l holds row (A) or column (B) l % 16 and
// its 8 elements k = (l / 16) * 8 .. + 7; of C column l % 16, rows (l / 16) * 4 .. + 3.
template <int DT> __device__ __forceinline__ acc4_t mfma_k32(u32x4_t a, u32x4_t b, acc4_t c) {
    if constexpr (DT == DT_BF16) {
        typedef __bf16 v8 __attribute__((ext_vector_type(8)));
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
    } else {
        typedef _Float16 v8 __attribute__((ext_vector_type(8)));
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
    }
}

// The same with C in vector registers, whatever the kernel's other products use: where a
// kernel may have accumulation registers the compiler puts every builtin's C there, and a
// second set of results does not fit beside 256 running sums. The compiler does not know
// these as matrix instructions, so the wait states are written out: the s_nop before one
// (its operands may come from a vector instruction just before), mfma_results() before
// anything reads the results. Chains on one C need none.
template <int DT> __device__ __forceinline__ acc4_t mfma_k32_first_v(u32x4_t a, u32x4_t b) {
    acc4_t c;
    if constexpr (DT == DT_BF16) asm("s_nop 1\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, 0" : "=&v"(c) : "v"(a), "v"(b));
    else asm("s_nop 1\n\tv_mfma_f32_16x16x32_f16 %0, %1, %2, 0" : "=&v"(c) : "v"(a), "v"(b));
    return c;
}
template <int DT> __device__ __forceinline__ void mfma_k32_v(u32x4_t a, u32x4_t b, acc4_t &c) {
    if constexpr (DT == DT_BF16) asm("s_nop 1\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+&v"(c) : "v"(a), "v"(b));
    else asm("s_nop 1\n\tv_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+&v"(c) : "v"(a), "v"(b));
}
template <int N> __device__ __forceinline__ void mfma_results(acc4_t (&c)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("s_nop 15" : "+v"(c[i]));
    asm volatile("s_nop 15" : "+v"(c[N - 1]));
}

// Keeps running sums in accumulation registers over branches and loops in which vector
// instructions touch them too: without it the compiler carries them in vector registers
// and copies them all over and back for every tile.
__device__ __forceinline__ void pin_acc(acc4_t &c) { asm volatile("" : "+a"(c)); }

// C[16 x 16] += A[16 x 16] B[16 x 16]: 4 elements k = (l / 16) * 4 .. + 3 a lane.
template <int DT> __device__ __forceinline__ acc4_t mfma_k16(u32x2_t a, u32x2_t b, acc4_t c) {
    if constexpr (DT == DT_BF16) {
        return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s16x4_t, a), __builtin_bit_cast(s16x4_t, b), c,
                                                         0, 0, 0);
    } else {
        typedef _Float16 v4 __attribute__((ext_vector_type(4)));
        return __builtin_amdgcn_mfma_f32_16x16x16f16(__builtin_bit_cast(v4, a), __builtin_bit_cast(v4, b), c, 0, 0, 0);
    }
}

// Two float32 -> one word of two 16-bit values (a in the low half), each rounded to
// nearest even.
template <int DT> __device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (DT == DT_BF16) return f32x2_to_bf16x2_bits(a, b);
    else {
        typedef float f2_t __attribute__((ext_vector_type(2)));
        typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
        const f2_t f = {a, b};
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, h2_t));
    }
}

// Transposing LDS read of a 4 x 16 block of 16-bit values in each group of 16 lanes:
// lane l of a group gives the address of row l / 4, columns (l % 4) * 4 .. + 3, and gets
// column l, rows 0 .. 3.
__device__ __forceinline__ u32x2_t lds_read_tr(const DS4HC_LDS char *p) {
    return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((DS4HC_LDS s16x4_t *)p));
}

__device__ __forceinline__ u32x4_t lds_read16(const DS4HC_LDS char *p) {
    return *reinterpret_cast<const DS4HC_LDS u32x4_t *>(p);
}

// 16 bytes a lane from base + offset (the lane's own, in bytes) to LDS byte lds + 16 * lane
// (lds the same in all lanes). Nothing is returned in registers. The compiler does not count
// it among the wave's loads: wait_and_barrier() waits for it, before any lane reads the
// bytes, and until then other loads' waits are longer than they need be, never shorter.
// (The builtin's loads are counted, and every LDS read that may alias one of them then waits
// for all of them, the tiles ahead included.) The s_nop is the wait state that a load to LDS
// needs after a write of m0.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is reserved: nothing of the compiler's is kept in it
__device__ __forceinline__ void load_to_lds16(const char *base, uint32_t offset, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds), "v"(offset), "s"(base)
                 : "m0", "memory");
}

// The same from an address of each lane's own.
__device__ __forceinline__ void load_to_lds16(const char *from, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :
                 : "s"(lds), "v"(from)
                 : "m0", "memory");
}
#pragma clang diagnostic pop

// Byte address in LDS.
__device__ __forceinline__ uint32_t lds_address(const void *p) {
    return (uint32_t)(uintptr_t)(const DS4HC_LDS void *)p;
}

// Maximum and sum over the four lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ float max_over_groups(float x) {
    auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_over_groups(float x) {
    auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Whether a word of two 16-bit values holds one that is not finite.
template <int DT> __device__ __forceinline__ bool word_not_finite(uint32_t w) {
    constexpr uint32_t E = DT == DT_BF16 ? 0x7F80u : 0x7C00u;
    return (w & E) == E || (w & (E << 16)) == (E << 16);
}

// Waits until at most `VM` of this wave's vector-memory operations are in flight and its
// LDS operations are done, then for the workgroup's other waves.
template <int VM> __device__ __forceinline__ void wait_and_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(VM) : "memory");
}

}  // namespace ds4hc
