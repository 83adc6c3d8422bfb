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

// Values that are the same in all lanes, into scalar registers.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
    return ((int64_t)uniform((int)(v >> 32)) << 32) | (uint32_t)uniform((int)v);
}

// Lane `lane`'s value.
__device__ __forceinline__ int from_lane(int v, int lane) { return __builtin_amdgcn_ds_bpermute(lane << 2, v); }

// The value, computed anew where it stands: keeps what is made of it from being kept in
// registers over a loop.
__device__ __forceinline__ uint32_t here(uint32_t v) {
    asm volatile("" : "+v"(v));
    return v;
}

// The lane's number, made anew where it stands: two instructions in place of a register that
// is held, or spilled, over a loop.
__device__ __forceinline__ int lane_here() {
    int l;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
    return l;
}

// Cache row of token j (0 <= j < max_pages << page_shift) of sequence b, -1 if
// its page is not in the cache.
__device__ __forceinline__ int64_t cache_row(const Paged &c, int b, int j) {
    const int page = c.block_table[(int64_t)b * c.max_pages + (j >> c.page_shift)];
    if (page < 0 || page >= c.n_pages) return -1;
    return ((int64_t)page << c.page_shift) + (j & ((1 << c.page_shift) - 1));
}

// cos and sin of position * inv_freq. The angle is formed and reduced to a part
// of a turn in 64 bits (a float32 angle of position 2^20 is off by 2^-5). The
// functions are of its float32 part, and what that leaves, d, turns the pair by
// (1, d): at most 1.35 x 2^-24 off over 2^25 angles of positions to 10^6, 1.92
// without it, for 0.9 us of 27 for 65536 tokens of one head, 0.1 of 5.6 for 8192
// and no time with many heads. (64-bit functions, 0.50, add 5 us and 0.7.)
__device__ __forceinline__ void rope_angle(int64_t position, double inv_freq, float amplitude,
                                           float &c, float &s) {
    double turns = (double)position * inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
    turns -= rint(turns);
    const double half_turns = 2.0 * turns;
    const float rounded = (float)half_turns, d = (float)((half_turns - rounded) * 3.14159265358979323846);
    float sn, cs;
    sincospif(rounded, &sn, &cs);
    c = fmaf(-d, sn, cs) * amplitude;
    s = fmaf(d, cs, sn) * amplitude;
}

// ------------------------------------------------------------------ matrix tiles

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef float acc4_t __attribute__((ext_vector_type(4)));
typedef float acc16_t __attribute__((ext_vector_type(16)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));

#define DS4HC_LDS __attribute__((address_space(3)))

// C[32 x 32] += A[32 x 16] B[16 x 32]. Lane l holds row (A) or column (B) l % 32 and its 8
// elements k = (l / 32) * 8 .. + 7; of C column l % 32 and rows 8 (i / 4) + 4 (l / 32) + i % 4.
template <int DT> __device__ __forceinline__ acc16_t mfma32(u32x4_t a, u32x4_t b, acc16_t c) {
    if constexpr (DT == DT_BF16) {
        typedef __bf16 v8 __attribute__((ext_vector_type(8)));
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
    } else {
        typedef _Float16 v8 __attribute__((ext_vector_type(8)));
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
    }
}

// The same with C in vector registers, whatever the kernel's other products use: where a
// kernel may have accumulation registers the compiler puts every builtin's C there, and a
// second set of results does not fit beside 256 running sums. The compiler does not know
// these as matrix instructions, so the wait states are written out: the s_nop before one
// (its operands may come from a vector instruction just before), mfma_results() before
// anything reads the results. A chain on one C needs none.
template <int DT> __device__ __forceinline__ void mfma32_first_v(u32x4_t a, u32x4_t b, acc16_t &c) {
    if constexpr (DT == DT_BF16) asm("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, 0" : "=&v"(c) : "v"(a), "v"(b));
    else asm("s_nop 1\n\tv_mfma_f32_32x32x16_f16 %0, %1, %2, 0" : "=&v"(c) : "v"(a), "v"(b));
}
template <int DT> __device__ __forceinline__ void mfma32_v(u32x4_t a, u32x4_t b, acc16_t &c) {
    if constexpr (DT == DT_BF16) asm("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+&v"(c) : "v"(a), "v"(b));
    else asm("s_nop 1\n\tv_mfma_f32_32x32x16_f16 %0, %1, %2, %0" : "+&v"(c) : "v"(a), "v"(b));
}
// With B in accumulation registers, which such an instruction reads as well.
template <int DT> __device__ __forceinline__ void mfma32_first_va(u32x4_t a, u32x4_t b, acc16_t &c) {
    if constexpr (DT == DT_BF16) asm("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, 0" : "=&v"(c) : "v"(a), "a"(b));
    else asm("s_nop 1\n\tv_mfma_f32_32x32x16_f16 %0, %1, %2, 0" : "=&v"(c) : "v"(a), "a"(b));
}
template <int DT> __device__ __forceinline__ void mfma32_va(u32x4_t a, u32x4_t b, acc16_t &c) {
    if constexpr (DT == DT_BF16) asm("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+&v"(c) : "v"(a), "a"(b));
    else asm("s_nop 1\n\tv_mfma_f32_32x32x16_f16 %0, %1, %2, %0" : "+&v"(c) : "v"(a), "a"(b));
}
// (12 wait states from this instruction to a vector instruction that reads its result.)
__device__ __forceinline__ void mfma_results(acc16_t &c) { asm volatile("s_nop 13" : "+v"(c)); }

// Keeps running sums in accumulation registers over branches and loops in which vector
// instructions touch them too: without it the compiler carries them in vector registers
// and copies them all over and back for every tile.
__device__ __forceinline__ void pin_acc(acc16_t &c) { asm volatile("" : "+a"(c)); }

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

// Sum plus both 16-bit values of a word, in float32: what rounded weights are divided by, so that
// a row's weights sum to 1 as they were used (a row that sees one token gives its values without
// an error, and a rounding that many weights share cancels). The sum before the rounding is lse's.
template <int DT> __device__ __forceinline__ float add2_words(uint32_t w, float sum) {
    if constexpr (DT == DT_BF16) {
        typedef __bf16 b2_t __attribute__((ext_vector_type(2)));
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2_t, w), b2_t{(__bf16)1.f, (__bf16)1.f}, sum, false);
    } else {
        asm("v_fma_mix_f32 %0, %1, 1.0, %0 op_sel_hi:[1,0,0]\n\tv_fma_mix_f32 %0, %1, 1.0, %0 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "+v"(sum) : "v"(w));
        return sum;
    }
}

// Both 16-bit values of a word times a factor.
template <int DT> __device__ __forceinline__ uint32_t scale2_words(uint32_t w, float f) {
    if constexpr (DT == DT_BF16) return pack2<DT>(bf16_lo(w) * f, bf16_hi(w) * f);
    else return pack2<DT>(f16_lo(w) * f, f16_hi(w) * f);
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
// (lds the same in all lanes); nothing where `lanes` is 0 (it is that or all ones, and all
// lanes are active where this stands: a branch around each of the loads that run beside a
// tile's products would split them into small blocks). Nothing is returned in registers. The
// compiler does not count it among the wave's loads: wait_and_barrier() waits for it, before
// any lane reads the bytes, and until then other loads' waits are longer than they need be,
// never shorter. (The builtin's loads are counted, and every LDS read that may alias one of
// them then waits for all of them, those of the next tile included.) Wait states: a load to
// LDS needs one after a write of m0, and a load 5 after a vector instruction that wrote its
// scalar address (v_readlane may stand right before).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is reserved: nothing of the compiler's is kept in it
__device__ __forceinline__ void load_to_lds16(const char *base, uint32_t offset, uint32_t lds, uint64_t lanes) {
    asm volatile("s_mov_b32 m0, %0\n\ts_mov_b64 exec, %3\n\ts_nop 2\n\tglobal_load_lds_dwordx4 %1, %2\n\ts_mov_b64 exec, -1"
                 :
                 : "s"(lds), "v"(offset), "s"(base), "s"(lanes)
                 : "m0", "memory");
}
// The same from an address of each lane's own.
__device__ __forceinline__ void load_to_lds16(const char *from, uint32_t lds, uint64_t lanes) {
    asm volatile("s_mov_b32 m0, %0\n\ts_mov_b64 exec, %2\n\tglobal_load_lds_dwordx4 %1, off\n\ts_mov_b64 exec, -1"
                 :
                 : "s"(lds), "v"(from), "s"(lanes)
                 : "m0", "memory");
}
#pragma clang diagnostic pop

// Waits for the loads that the values come from: a wait that the compiler would otherwise
// place at their first use, inside a loop, where it would wait for the next tile as well.
__device__ __forceinline__ void loaded(u32x4_t &v) { asm volatile("" : "+v"(v)); }
// The same, and the values into accumulation registers.
__device__ __forceinline__ void loaded_acc(u32x4_t &v) { asm volatile("" : "+a"(v)); }
__device__ __forceinline__ void loaded(int &v) { asm volatile("" : "+v"(v)); }

// Byte address in LDS.
__device__ __forceinline__ uint32_t lds_address(const void *p) {
    return (uint32_t)(uintptr_t)(const DS4HC_LDS void *)p;
}

// Maximum and sum over lanes l and l ^ 32.
__device__ __forceinline__ float max_halves(float x) {
    auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float sum_halves(float x) {
    auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// Largest of three, and of a result's 16. (The compiler would first rewrite every value that
// comes out of an asm block, so that a NaN is quiet.)
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
__device__ __forceinline__ float max16(const acc16_t &s) {
    const float a = max3(s[0], s[1], s[2]), b = max3(s[3], s[4], s[5]), c = max3(s[6], s[7], s[8]);
    const float d = max3(s[9], s[10], s[11]), e = max3(s[12], s[13], s[14]);
    return max3(max3(a, b, c), max3(d, e, s[15]), s[15]);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// ------------------------------------------------------------------ softmax

constexpr float LN2 = 0.69314718055994530942f, LOG2E = 1.44269504088896340736f;
constexpr float LAZY = 8.f;  // the running maximum is raised only by more than this (in powers of 2)
// The largest weight is brought to (2^(LIFT - 1), 2^LIFT]. float16 has 5 bits of exponent: with
// the largest near 1, weights below 2^-14 would lose bits and those below 2^-25 vanish, which
// many of them together do not deserve (131072 tokens 17.5 below one that holds 99.5 % of the
// weight kept 0.39 % of 0.54). With 2^7, and 2^15 as the most that LAZY leaves, that begins 2^7 further
// down, at no instruction in the loop. bfloat16 has float32's exponents.
template <int DT> constexpr float LIFT = DT == DT_F16 ? 7.f : 0.f;

// ln of the sum of exponentials, from the exponent subtracted and the sum of the weights (before
// their rounding). LIFT is taken out first: the logarithm's error is relative to it.
template <int DT> __device__ __forceinline__ float row_lse(float top, float sum) {
    constexpr float UNIT = DT == DT_F16 ? 1.f / 128.f : 1.f;
    return sum == 0.f ? -INFINITY : ((top + LIFT<DT>) + __log2f(sum * UNIT)) * LN2;
}

// Not 0 if one of eight 16-bit values is not finite: an exponent of all ones carries into the
// sign's place when one is added to it.
template <int DT> __device__ __forceinline__ uint32_t not_finite_bits(u32x4_t w) {
    constexpr uint32_t ONE = DT == DT_BF16 ? 0x00800080u : 0x04000400u, REST = 0x7FFF7FFFu;
    return (((w.x & REST) + ONE) | ((w.y & REST) + ONE) | ((w.z & REST) + ONE) | ((w.w & REST) + ONE)) & ~REST;
}
template <int DT> __device__ __forceinline__ bool not_all_finite(u32x4_t w) { return not_finite_bits<DT>(w) != 0; }

// Waits until at most `VM` of this wave's vector-memory operations are in flight and its
// LDS operations are done, then for the workgroup's other waves.
template <int VM> __device__ __forceinline__ void wait_and_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(VM) : "memory");
}

}  // namespace ds4hc
