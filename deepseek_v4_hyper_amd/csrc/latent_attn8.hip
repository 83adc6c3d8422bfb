// latent_attn8.hip -- attention over the paged latent cache whose latents are held in 8 bits.
//
// Per query row (a token and a head) and cached row (c8 | r | s) of a sequence, with c = c8 2^(s - 127):
//   x = scale (ql . c + qr . r),  out = softmax(x) C.
// The work is split as for the 16-bit cache (latent_split.hpp): tiles of 64 tokens go to LDS as they
// are, 656 bytes a token in place of 1152, and every wave takes 32 query rows through them.
// A token's power of 2 scales its whole latent, so it goes into the logit's operand, and for the
// second product into the weight: out = sum_j p_j c8_j / sum_j p_j 2^(127 - s_j), p_j = w_j 2^(s_j - 127).
#include <type_traits>

#include "latent_split.hpp"

namespace ds4hc {

namespace {

template <int LATENT_, int ROW_WAVES_, int SETS_> struct Shape8 {
    static constexpr int LATENT = LATENT_, ROW_WAVES = ROW_WAVES_, SETS = SETS_;
    static constexpr int TOKENS = 64, BUFS = 2, STEPS = TOKENS / SETS / 32;
    static constexpr int WAVES = ROW_WAVES * SETS, THREADS = WAVES * 64;
    static constexpr int ROWS = ROW_WAVES * 32;
    static constexpr int ROW_BYTES = LATENT, CHUNKS = ROW_BYTES / 16;  // a token's latent in LDS
    static constexpr int ROPE_AT = TOKENS * ROW_BYTES, SCALE_AT = ROPE_AT + TOKENS * LATENT_ROPE * 2;
    static constexpr int TILE_BYTES = SCALE_AT + TOKENS * 16;
    static constexpr int ROWS_A_LOAD = 1024 / ROW_BYTES;
    static constexpr int OWN_LATENT = TOKENS / ROWS_A_LOAD / WAVES, OWN_ROPE = TOKENS / 8 / WAVES;
    static constexpr int LOADS = OWN_LATENT + OWN_ROPE + 1;  // of a wave and tile; the last, of the scales, is one wave's
    static constexpr int KLATENT = LATENT / 16, KSTEPS = KLATENT + LATENT_ROPE / 16, DBLOCKS = LATENT / 32;
    // of the output, that a wave finishes, and what it takes to store them (with two sets: to give them away)
    static constexpr int BLOCKS = DBLOCKS / SETS, BLOCK_BYTES = 16 * 64 * 4;
    static constexpr int END_BYTES = SETS == 1 ? WAVES * 32 * BLOCKS * 64 : WAVES * (BLOCKS * BLOCK_BYTES + 384);
    static constexpr int RING_BYTES = BUFS * TILE_BYTES > END_BYTES ? BUFS * TILE_BYTES : END_BYTES;
    static_assert(OWN_LATENT * ROWS_A_LOAD * WAVES == TOKENS && OWN_ROPE * 8 * WAVES == TOKENS, "the waves load alike");
};

// Swizzle: 16-byte chunk c of token row r lies at chunk c ^ swz8(r) of the row's place in LDS. A read of the
// first product takes the same chunk of 16 rows, 256 bytes: swz8 takes 16 values over 16 rows (rows of 128
// bytes: 8 over 8 pairs of rows). A transposing read takes 32 bytes of each of 8 rows, 0 .. 3 and 8 .. 11 or those
// 4 further on: swz8 without its lowest bit takes 8 values over them (of 128 bytes: 4 over their pairs).
template <int CHUNKS> __device__ __forceinline__ int swz8(int r) {
    if constexpr (CHUNKS >= 16) return (r & 3) << 1 | (r & 8) | ((r >> 2) & 1);
    else return (r & 2) | ((r >> 1) & 4) | ((r >> 2) & 1);
}
__device__ __forceinline__ int swz8_rope(int r) { return (r >> 1) & 7; }

// Scale bytes that the append writes; others but 255, which marks a token that is not finite, are taken
// as the nearest of these. With float16 operands all values are below its smallest number at 87 (448 x 2^-40),
// and half of the codes beyond its largest at 143.
constexpr int SCALE_NAN = 255;
template <int DT> __device__ __forceinline__ int scale_byte(uint32_t word) {
    constexpr int MIN = DT == DT_F16 ? 87 : 10, MAX = DT == DT_F16 ? 143 : 246;
    return min(max((int)(word & 255), MIN), MAX);
}
__device__ __forceinline__ bool scale_is_nan(uint32_t word) { return (word & 255) == SCALE_NAN; }
template <int DT> __device__ __forceinline__ float scale_of(uint32_t word) {
    return scale_is_nan(word) ? NAN : __uint_as_float((uint32_t)scale_byte<DT>(word) << 23);
}

// Four e4m3 values of each of two words, times a power of 2, as the 16-bit type. Exact in bfloat16, in float16 as
// far as its range goes.
template <int DT> __device__ __forceinline__ u32x4_t widen8(uint32_t a, uint32_t b, float scale) {
    u32x4_t w;
    if constexpr (DT == DT_BF16) {
        w.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, false));
        w.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, true));
        w.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, false));
        w.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, true));
    } else {
        w.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, scale, false));
        w.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, scale, true));
        w.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, scale, false));
        w.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, scale, true));
    }
    return w;
}

// Transposing LDS read of an 8 x 16 block of bytes in each group of 16 lanes: lane l of a group gives the
// address of row l / 2, columns (l % 2) * 8 .. + 7, and gets column l, rows 0 .. 7.
__device__ __forceinline__ u32x2_t lds_read_tr8(const DS4HC_LDS char *p) {
    typedef int i32x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr8_b64_v2i32((DS4HC_LDS i32x2_t *)p));
}

// Not 0 if one of 16 e4m3 values is NaN (all bits but the sign set; there are no infinities).
__device__ __forceinline__ uint32_t nan_bits8(u32x4_t w) {
    constexpr uint32_t REST = 0x7F7F7F7Fu, ONE = 0x01010101u;
    return (((w.x & REST) + ONE) | ((w.y & REST) + ONE) | ((w.z & REST) + ONE) | ((w.w & REST) + ONE)) & ~REST;
}

template <int DT, class S>
__global__ __launch_bounds__(S::THREADS, 1) void attn8_kernel(AttnArgs a) {
    __shared__ __align__(256) char ring[S::RING_BYTES];
    __shared__ uint32_t not_finite[2];
    __shared__ __align__(16) float units[S::WAVES][S::TOKENS];  // the tile's powers of 2, each wave's own copy
    __shared__ __align__(16) float powers[DT == DT_F16 ? S::WAVES : 1][S::TOKENS];  // their exponents
    const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
    const int row_wave = wave % S::ROW_WAVES, set = wave / S::ROW_WAVES;
    // clusters in the order of the work run on one XCD
    const int slot = blockIdx.x / XCDS, member = slot % a.members;
    const int cluster = (blockIdx.x % XCDS) * (WORKGROUPS / XCDS / a.members) + slot / a.members;

    int64_t share, off = 0;
    int b, extra;
    Seq sq{};
    const int64_t total = find_unit<S>(a, share, extra, cluster, b, off, sq);
    b = uniform(b);
    off = uniform(off);
    extra = uniform(extra);
    if (threadIdx.x == 0 && member == 0) {
        Header *head = static_cast<Header *>(a.ws);
        if (cluster == 0) head->share = share;
        Start at = {b, 0, 0, 0};
        if (b >= 0) {
            const int each = sq.kv_tiles + extra;
            at.batch = (int)(off / each);
            at.tile = max((int)(off - (int64_t)at.batch * each) - extra, 0);
        }
        head->start[cluster] = at;
    }
    if (b < 0) return;
    int64_t left = uniform(min(share, total - cluster * share));
    const float scale2 = a.scale * LOG2E;
    const char *cache = static_cast<const char *>(a.cache);
    constexpr int STRIDE = S::LATENT + LATENT_ROPE * 2 + 16;  // bytes of a cached row

    bool first_part = true;
    while (left > 0) {
        sq = {uniform(sq.q0), uniform(sq.few), uniform(sq.len), uniform(sq.row_tiles), uniform(sq.kv_tiles)};
        const int each = sq.kv_tiles + extra;  // units of a batch
        if (off >= (int64_t)sq.batches(a.members) * each) {  // next sequence (the units in all bound b)
            sq = sequence<S>(a, ++b);
            off = 0;
            continue;
        }
        const int q0 = sq.q0;
        const int batch = (int)(off / each), u0 = (int)(off - (int64_t)batch * each), u1 = u0 + (int)min((int64_t)(each - u0), left);
        const int t_first = max(u0 - extra, 0), n = max(u1 - extra, 0) - t_first;
        const int row_tile = batch * a.members + member;
        const bool part_of_first = first_part && t_first > 0;
        first_part = false;
        left -= u1 - u0;
        off += u1 - u0;
        if (n == 0 || row_tile >= sq.row_tiles) continue;
        const int n_rows = sq.few * a.heads;  // the host keeps N * heads below 2^31
        const int context = sq.len - sq.few;

        // ---- the lane's row: its query in registers. Lanes below 32 hold channels 32 j .. 32 j + 15 of each 32, in
        // steps 2 j and 2 j + 1, the others those behind: what a read of 16 bytes of a cached row gives.
        const int row0 = row_tile * S::ROWS + row_wave * 32;
        const int tok = min(row0 + (lane & 31), n_rows - 1) / a.heads;  // rows behind the last repeat it
        u32x4_t q[S::KSTEPS];
        auto load_queries = [&]() {
            const int head = min(row0 + (lane & 31), n_rows - 1) - tok * a.heads;
            const elem_t<DT> *ql = static_cast<const elem_t<DT> *>(a.ql) + (int64_t)(q0 + tok) * a.ql_token + head * a.ql_head + (lane >> 5) * 16;
            const elem_t<DT> *qr = static_cast<const elem_t<DT> *>(a.qr) + (int64_t)(q0 + tok) * a.qr_token + head * a.qr_head + (lane >> 5) * 8;
#pragma unroll
            for (int k = 0; k < S::KSTEPS; ++k)
                q[k] = *reinterpret_cast<const u32x4_t *>(k < S::KLATENT ? ql + (k >> 1) * 32 + (k & 1) * 8 : qr + (k - S::KLATENT) * 16);
#pragma unroll
            for (int k = 0; k < S::KSTEPS; ++k) loaded(q[k]);
        };
        float top = -INFINITY, from = 0.f;  // running maximum less LIFT (what is subtracted: 0 if there is none)
        float sum = 0.f;                    // of the weights
        acc16_t acc[S::DBLOCKS];
#pragma unroll
        for (int d = 0; d < S::DBLOCKS; ++d) {
            acc[d] = acc16_t{};
            pin_acc(acc[d]);
        }

        // Pages: lane e holds entry e of those of the next tiles, 1 << e_shift a tile, so that the
        // block table is read once for many tiles and its latency is not a tile's.
        const int e_shift = max(__builtin_ctz(S::TOKENS) - a.c.page_shift, 0);
        int pages = -1, pages_from = t_first - 64;
        // Cache rows of a tile's tokens, lane r that of token r (-1: not in the cache, or behind the end).
        auto look_up = [&](int tile) {
            if (tile >= t_first + n) return -1;
            if (tile - pages_from >= 64 >> e_shift) {
                pages_from = tile;
                const int e = lane_here(), in_tile = e >> e_shift;
                const int j = (tile + in_tile) * S::TOKENS + ((e - (in_tile << e_shift)) << a.c.page_shift);
                pages = -1;
                if (tile + in_tile < t_first + n && j < sq.len) pages = a.c.block_table[(int64_t)b * a.c.max_pages + (j >> a.c.page_shift)];
                if (pages >= a.c.n_pages) pages = -1;
                loaded(pages);
            }
            const int r = lane_here() & (S::TOKENS - 1), j = tile * S::TOKENS + r;
            const int page = from_lane(pages, ((tile - pages_from) << e_shift) + (e_shift ? r >> a.c.page_shift : 0));
            return page < 0 || j >= sq.len ? -1 : (page << a.c.page_shift) + (j & ((1 << a.c.page_shift) - 1));
        };
        // Tokens that are not there get the data of one that is (their places may hold anything, also NaN, which a
        // weight of 0 would not hide). Which tokens are there, a bit each:
        auto present = [&](int &rows) -> uint64_t {
            const uint64_t ok = __ballot(rows >= 0);
            const int one = __builtin_amdgcn_readlane(rows, __builtin_ctzll(ok | 1ull << 63));
            rows = rows >= 0 ? rows : one >= 0 ? one : 0;  // (none is there: row 0; nothing sees it)
            return ok;
        };
        // The wave's load number i of the tile to `buf`; lane r of `rows` has token r's cache row.
        auto load = [&](int i, int rows, uint32_t l, uint32_t buf, uint64_t lanes) {
            auto of_row = [&](int r) { return cache + (uint64_t)(uint32_t)from_lane(rows, r) * STRIDE; };
            if (i < S::OWN_LATENT) {
                const int r0 = (wave * S::OWN_LATENT + i) * S::ROWS_A_LOAD, r = r0 + l / S::CHUNKS, c = l % S::CHUNKS;
                load_to_lds16(of_row(r) + ((c ^ swz8<S::CHUNKS>(r)) << 4), buf + r0 * S::ROW_BYTES, lanes);
            } else if (i < S::OWN_LATENT + S::OWN_ROPE) {
                const int r0 = (wave * S::OWN_ROPE + i - S::OWN_LATENT) * 8, r = r0 + l / 8, c = l % 8;
                load_to_lds16(of_row(r) + S::LATENT + ((c ^ swz8_rope(r)) << 4), buf + S::ROPE_AT + r0 * 128, lanes);
            } else {
                load_to_lds16(of_row(l) + S::LATENT + LATENT_ROPE * 2, buf + S::SCALE_AT, (uint64_t)uniform((int64_t)(wave == 0 ? lanes : 0)));
            }
        };

        // Tile t (tokens `ok`) in LDS at `at`, and the loads of the next one, if there is one, beside it.
        auto tile = [&](int t, uint64_t ok, uint32_t at, int rows, uint32_t at_next) {
            DS4HC_LDS char *buf = (DS4HC_LDS char *)(uintptr_t)at;
            DS4HC_LDS uint32_t *scales = (DS4HC_LDS uint32_t *)(uintptr_t)(at + S::SCALE_AT);  // (token r's: element 4 r, its lowest byte)
            const int j0 = t * S::TOKENS;
            const bool masked = ok != ~0ull || j0 + S::TOKENS > (a.tree_mask ? context : context + 1);
            uint64_t bad = 0;  // tokens that hold a value that is not finite
            if (masked) {  // the same in all waves
                // Only what some rows see and others do not has to be looked at: the call's own tokens,
                // and the copies in place of tokens that are not there, if it is one of those they copy. (A
                // copy of a context token is seen, as that token, by all.) If none of the tile's tokens is
                // there, they copy the cache's first row, which may be nobody's and is seen by none.
                const int own = ok ? context - j0 : 0, copied = ok ? __builtin_ctzll(ok) : 0;
                const int lo = copied >= own ? 0 : own, hi = copied >= own ? S::TOKENS : min(S::TOKENS, sq.len - j0);
                if (threadIdx.x < 2) not_finite[threadIdx.x] = 0;
                wait_and_barrier<63>();
                for (int i = lo * S::CHUNKS + threadIdx.x; i < hi * S::CHUNKS; i += S::THREADS)
                    if (nan_bits8(lds_read16(buf + i * 16)) || scale_is_nan(scales[i / S::CHUNKS * 4]))
                        atomicOr(&not_finite[(i / S::CHUNKS) >> 5], 1u << ((i / S::CHUNKS) & 31));
                wait_and_barrier<63>();
                bad = ((uint64_t)uniform((int)not_finite[1]) << 32) | (uint32_t)uniform((int)not_finite[0]);
                if (bad) {  // zero in LDS, so that they meet no weight of 0; the rows that see them get NaN weights
                    for (int i = threadIdx.x; i < S::TOKENS * S::CHUNKS; i += S::THREADS)
                        if ((bad >> (i / S::CHUNKS)) & 1) {
                            const uint32_t zero = here(0);
                            *reinterpret_cast<DS4HC_LDS u32x4_t *>(buf + i * 16) = u32x4_t{zero, zero, zero, zero};
                            scales[i / S::CHUNKS * 4] = 127;
                        }
                    wait_and_barrier<63>();
                }
            }
            const int l = lane_here(), lr = l & 31, lh = l >> 5;
            units[wave][l] = scale_of<DT>(scales[l * 4]);
            if constexpr (DT == DT_F16) powers[wave][l] = scale_is_nan(scales[l * 4]) ? NAN : (float)(scale_byte<DT>(scales[l * 4]) - 127);
            // LDS offsets of this lane's reads for the first k step, rope step and block of the
            // output; the others' chunks differ in higher bits, which an xor reaches. Made anew for
            // every tile: there are no registers to keep them.
            const int t0 = set * S::STEPS * 32;  // first token of the wave
            const uint32_t k0 = (t0 + lr) * S::ROW_BYTES + ((lh ^ swz8<S::CHUNKS>(lr)) << 4);
            const uint32_t r0 = S::ROPE_AT + (t0 + lr) * 128 + ((lh ^ swz8_rope(lr)) << 4);
            const int vr = lh * 4 + ((l >> 1) & 3) + (l & 8);
            const uint32_t v0 = (t0 + vr) * S::ROW_BYTES + ((((l >> 4) & 1) ^ swz8<S::CHUNKS>(vr)) << 4) + (l & 1) * 8;

            // X^T = K Q^T of 32 tokens, the operands of the next products on their way; `between`
            // gives other work to the vector unit while the matrix unit is busy
            auto products_k = [&](int step, acc16_t &s, auto &&between) {
                const float unit_k = scale_of<DT>(scales[(t0 + step * 32 + lr) * 4]);
                auto read = [&](int j) { return lds_read16(buf + (k0 ^ ((j & 7) << 5)) + (j >> 3) * 256 + step * 32 * S::ROW_BYTES); };
                auto read_rope = [&](int j) { return lds_read16(buf + (r0 ^ (j << 5)) + step * 32 * 128); };
                constexpr int ROPE_STEPS = LATENT_ROPE / 16;
                u32x4_t x[2] = {read(0), read(1)}, r[ROPE_STEPS];
#pragma unroll
                for (int j = 0; j < S::KLATENT / 2; ++j) {
                    const u32x4_t now = x[j & 1];
                    if (j + 2 < S::KLATENT / 2) x[j & 1] = read(j + 2);
                    if (j >= S::KLATENT / 2 - ROPE_STEPS) r[j - S::KLATENT / 2 + ROPE_STEPS] = read_rope(j - S::KLATENT / 2 + ROPE_STEPS);
                    const u32x4_t w0 = widen8<DT>(now.x, now.y, unit_k), w1 = widen8<DT>(now.z, now.w, unit_k);
                    if (j == 0) mfma32_first_v<DT>(w0, q[0], s);
                    else mfma32_v<DT>(w0, q[2 * j], s);
                    between(2 * j);
                    mfma32_v<DT>(w1, q[2 * j + 1], s);
                    between(2 * j + 1);
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int j = 0; j < ROPE_STEPS; ++j) {
                    mfma32_v<DT>(r[j], q[S::KLATENT + j], s);
                    between(S::KLATENT + j);
                    __builtin_amdgcn_sched_barrier(0);
                }
            };
            // O^T += V^T P^T of 32 tokens; the order of the tokens is that of X^T's rows, for both operands
            constexpr int VAHEAD = 4;
            auto products_v = [&](int step, const u32x4_t (&p)[2], auto &&between) {
                auto read = [&](int i) {  // block i / 2, tokens 16 (i % 2) .. + 15
                    const int d = i / 2;
                    return lds_read_tr8(buf + (v0 ^ ((d & 7) << 5)) + (d >> 3) * 256 + (step * 32 + (i & 1) * 16) * S::ROW_BYTES);
                };
                u32x2_t v[VAHEAD];
#pragma unroll
                for (int i = 0; i < VAHEAD; ++i) v[i] = read(i);
#pragma unroll
                for (int i = 0; i < S::DBLOCKS * 2; ++i) {
                    const u32x4_t w = widen8<DT>(v[i % VAHEAD].x, v[i % VAHEAD].y, 1.f);
                    acc[i / 2] = mfma32<DT>(w, p[i & 1], acc[i / 2]);
                    if (i + VAHEAD < S::DBLOCKS * 2) v[i % VAHEAD] = read(i + VAHEAD);
                    between(i);
                    __builtin_amdgcn_sched_barrier(0);
                }
            };
            // Softmax of a step, in pieces. The mask, and the largest logit (of the lane's row).
            uint64_t sees = ~0ull;
            if (masked) sees = sees_of_tile(a, q0 + tok, tok, j0 - context) & ok;
            // (float16: of the logit in powers of 2 with the token's power, so that the weights that the second product
            // takes lie in float16's range whatever the powers are, and small ones are lost only beside larger ones)
            const int at_token = t0 + lh * 4;
            auto largest = [&](int step, acc16_t &s) {
                if constexpr (DT == DT_F16) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[i] = fmaf(s[i], scale2, powers[wave][at_token + step * 32 + 8 * (i / 4) + i % 4]);
                }
                if (masked) {
                    const int at0 = t0 + step * 32 + (lane_here() >> 5) * 4;
                    const uint32_t see = (uint32_t)(sees >> at0), nan = (uint32_t)((sees & bad) >> at0);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int r = 8 * (i / 4) + i % 4;
                        s[i] = (nan >> r) & 1 ? NAN : (see >> r) & 1 ? s[i] : -INFINITY;
                    }
                }
                const float high = max_halves(max16(s));
                return DT == DT_F16 ? high : high * scale2;
            };
            // A new running maximum, a whole number: see the kernel of the 16-bit cache.
            auto too_high = [&](float high) { return high - top > LAZY + LIFT<DT>; };
            auto raise = [&](float high) {
                const float was = top;
                top = fmaxf(top, ceilf(high) - LIFT<DT>);
                from = top == -INFINITY ? 0.f : top;
                const float keep = was == -INFINITY ? 0.f : exp2_fast(was - top);
                sum *= keep;
                if (__any(was != -INFINITY)) {  // (the first maximum: the sums are 0)
#pragma unroll
                    for (int d = 0; d < S::DBLOCKS; ++d) {
                        pin_acc(acc[d]);
                        acc[d] *= keep;
                        pin_acc(acc[d]);
                    }
                }
                return keep;
            };
            // Weights 2 i and 2 i + 1 times their tokens' powers of 2, rounded to the type that the second product takes.
            auto weight2 = [&](int step, const acc16_t &s, int i, u32x4_t (&p)[2]) {
                const float *u = &units[wave][at_token + step * 32 + 8 * (i / 2) + 2 * (i & 1)];
                if constexpr (DT == DT_F16) {
                    const float e0 = exp2_fast(s[2 * i] - from), e1 = exp2_fast(s[2 * i + 1] - from);
                    auto inverse = [](float power) { return __uint_as_float((254u << 23) - __float_as_uint(power)); };
                    sum = fmaf(e0, inverse(u[0]), sum);
                    sum = fmaf(e1, inverse(u[1]), sum);
                    p[i >> 2][i & 3] = pack2<DT>(e0, e1);
                } else {
                    const float e0 = exp2_fast(fmaf(s[2 * i], scale2, -from)), e1 = exp2_fast(fmaf(s[2 * i + 1], scale2, -from));
                    sum += e0;
                    sum += e1;
                    p[i >> 2][i & 3] = pack2<DT>(e0 * u[0], e1 * u[1]);
                }
            };
            constexpr int SLOTS = S::KSTEPS * S::STEPS + S::DBLOCKS * 2, LOAD_EVERY = SLOTS / S::LOADS;
            static_assert(LOAD_EVERY >= 1, "a place for each load");
            const uint64_t lanes = (uint64_t)uniform((int64_t)(t + 1 < t_first + n ? -1 : 0));
            auto load_some = [&](int i) {
                if (i % LOAD_EVERY == 0 && i / LOAD_EVERY < S::LOADS) load(i / LOAD_EVERY, rows, lane_here(), at_next, lanes);
            };
            acc16_t s;
            u32x4_t p[2];
            products_k(0, s, load_some);
            if constexpr (S::STEPS == 1) {
                mfma_results(s);
                const float high = largest(0, s);
                if (__any(too_high(high))) raise(high);
#pragma unroll
                for (int i = 0; i < 8; ++i) weight2(0, s, i, p);
                products_v(0, p, [&](int i) { load_some(S::KSTEPS + i); });
            } else {  // two steps, the softmax of each beside the products of the other, as far as can be
                acc16_t s1;
                u32x4_t p1[2];
                mfma_results(s);
                float high = largest(0, s);
                if (__any(too_high(high))) raise(high);
                products_k(1, s1, [&](int i) {
                    constexpr int EVERY = S::KSTEPS / 8;
                    load_some(S::KSTEPS + i);
                    if (i % EVERY == EVERY - 1 && i / EVERY < 8) weight2(0, s, i / EVERY, p);
                });
                mfma_results(s1);
                high = largest(1, s1);
                if (__any(too_high(high))) {
                    const float keep = raise(high);
#pragma unroll
                    for (int i = 0; i < 8; ++i) p[i >> 2][i & 3] = scale2_words<DT>(p[i >> 2][i & 3], keep);
                }
                products_v(0, p, [&](int i) {
                    constexpr int EVERY = S::DBLOCKS / 4;
                    load_some(2 * S::KSTEPS + i);
                    if (i % EVERY == EVERY - 1) weight2(1, s1, i / EVERY, p1);
                });
                products_v(1, p1, [](int) {});
            }
        };

        // ---- tiles: the next one's loads run beside this one's products. All waves are done with
        // tile t - 1 when they meet at the barrier of tile t, so its buffer takes tile t + 1.
        wait_and_barrier<63>();  // the last part's reads of the ring
        const uint32_t ring_at = lds_address(ring);
        int rows = look_up(t_first);
        uint64_t ok = present(rows);
#pragma unroll
        for (int i = 0; i < S::LOADS; ++i) load(i, rows, lane_here(), ring_at, ~0ull);
        load_queries();  // (waits for the first tile, too)
        int next = look_up(t_first + 1);
        for (int i = 0; i < n; ++i) {
            wait_and_barrier<0>();
            rows = next;
            const uint64_t ok_next = present(rows);
            next = look_up(t_first + i + 2);
            tile(t_first + i, ok, ring_at + (i & 1) * S::TILE_BYTES, rows, ring_at + ((i + 1) & 1) * S::TILE_BYTES);
            ok = ok_next;
        }

        // ---- the part's result
#pragma unroll
        for (int d = 0; d < S::DBLOCKS; ++d) pin_acc(acc[d]);
        const int l = lane_here(), lh = l >> 5, my_row = row0 + (l & 31), head = my_row - tok * a.heads;
        const bool whole = t_first == 0 && n == sq.kv_tiles, mine = my_row < n_rows;  // (a part's rows behind the last: never looked at)
        const int in = my_row - row_tile * S::ROWS;
        float *part = part_at<S>(a, cluster, part_of_first ? 0 : 1, member);
        float all = sum_halves(sum);
        // the blocks of the output that this wave finishes: all, or with two sets its half
        constexpr int BLOCKS = S::BLOCKS, BLOCK_BYTES = S::BLOCK_BYTES;
        acc16_t fin[BLOCKS];
        if constexpr (S::SETS == 1) {
#pragma unroll
            for (int d = 0; d < BLOCKS; ++d) fin[d] = acc[d];
            wait_and_barrier<63>();  // the last tile has been read by all
        } else {
            // each set gives the other one's half through LDS, and all is brought to the common maximum
            float *st = reinterpret_cast<float *>(ring + S::WAVES * BLOCKS * BLOCK_BYTES);  // maximum, sum [row waves][sets][32]
            char *give = ring + (row_wave * 2 + set) * BLOCKS * BLOCK_BYTES + l * 16, *take = ring + (row_wave * 2 + 1 - set) * BLOCKS * BLOCK_BYTES + l * 16;
            float *mine_st = st + (row_wave * 2 + set) * 96, *other_st = st + (row_wave * 2 + 1 - set) * 96;
            auto give_half = [&](auto from) {
#pragma unroll
                for (int d = 0; d < BLOCKS; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const acc16_t &v = acc[from.value + d];
                        *reinterpret_cast<acc4_t *>(give + (d * 4 + i) * 1024) = acc4_t{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
                    }
            };
            wait_and_barrier<63>();
            if (lh == 0) {
                mine_st[l] = top;
                mine_st[32 + l] = all;
            }
            if (set == 0) give_half(std::integral_constant<int, BLOCKS>{});
            else give_half(std::integral_constant<int, 0>{});
            wait_and_barrier<63>();
            const float other = other_st[l & 31], to = fmaxf(top, other);
            // (no logit that is a number, -infinity: the sums are 0 or NaN)
            const float keep = to == -INFINITY ? 1.f : exp2_fast(top - to), add = to == -INFINITY ? 1.f : exp2_fast(other - to);
            all = all * keep + other_st[32 + (l & 31)] * add;
            top = to;
            auto take_half = [&](auto from) {
#pragma unroll
                for (int d = 0; d < BLOCKS; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const acc4_t v = *reinterpret_cast<const acc4_t *>(take + (d * 4 + i) * 1024);
#pragma unroll
                        for (int e = 0; e < 4; ++e) fin[d][4 * i + e] = acc[from.value + d][4 * i + e] * keep + v[e] * add;
                    }
            };
            if (set == 0) take_half(std::integral_constant<int, 0>{});
            else take_half(std::integral_constant<int, BLOCKS>{});
        }
        const int block0 = (S::SETS - 1) * set * BLOCKS;
        if (whole) {
            const float inv = all == 0.f ? 0.f : 1.f / all;
            if (a.lse && set == 0 && lh == 0 && mine) a.lse[(int64_t)q0 * a.heads + my_row] = row_lse<DT>(top, all);
            // through LDS, to store whole rows: chunk c of row r at chunk c ^ (r % 16), in the wave's own place
            // (with two sets in what it has just read)
            constexpr int OUT_BYTES = BLOCKS * 64, PER = OUT_BYTES / 16, SPREAD = PER < 16 ? PER - 1 : 15;
            char *rows_at = ring + (S::SETS == 1 ? wave * 32 * OUT_BYTES : (row_wave * 2 + 1 - set) * BLOCKS * BLOCK_BYTES);
#pragma unroll
            for (int d = 0; d < BLOCKS; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<u32x2_t *>(rows_at + (l & 31) * OUT_BYTES + (((d * 4 + i) ^ (l & SPREAD)) << 4) + lh * 8) = u32x2_t{
                        pack2<DT>(fin[d][4 * i] * inv, fin[d][4 * i + 1] * inv), pack2<DT>(fin[d][4 * i + 2] * inv, fin[d][4 * i + 3] * inv)};
            const int64_t o = (int64_t)(q0 + tok) * a.out_token + head * a.out_head + block0 * 32;
            for (int i = 0; i < 32; i += 64 / PER) {
                const int r = i + l / PER, c = l % PER;
                const int64_t to = (int64_t)(uint32_t)from_lane((int)(uint32_t)o, r) | (int64_t)from_lane((int)(o >> 32), r) << 32;
                const u32x4_t v = *reinterpret_cast<const u32x4_t *>(rows_at + r * OUT_BYTES + ((c ^ (r & SPREAD)) << 4));
                if (row0 + r < n_rows) *reinterpret_cast<u32x4_t *>(static_cast<elem_t<DT> *>(a.out) + to + c * 8) = v;
            }
        } else {
            if (lh == 0 && set == 0) {
                part[S::ROWS * S::LATENT + in] = top;
                part[S::ROWS * (S::LATENT + 1) + in] = all;
                part[S::ROWS * (S::LATENT + 2) + in] = all;
            }
            float *o = part + ((row_wave * S::DBLOCKS + block0) * 256 + l) * 4;
#pragma unroll
            for (int d = 0; d < BLOCKS; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<acc4_t *>(o + (d * 4 + i) * 256) = acc4_t{fin[d][4 * i], fin[d][4 * i + 1], fin[d][4 * i + 2], fin[d][4 * i + 3]};
        }
    }
}

// How a call is run: tiles and clusters by the average rows of a sequence, as for the 16-bit cache.
struct Plan8 {
    int rows, members;
};

Plan8 plan8(const Paged &c, int heads, int64_t N) {
    const int64_t rows = (N * heads + c.n_seqs - 1) / c.n_seqs;
    if (rows <= 32) return {32, 1};
    if (rows <= 64) return {64, 1};
    return {128, rows <= 128 ? 1 : rows <= 256 ? 2 : 4};
}

template <int DT, class S> hipError_t run8(const AttnArgs &a, hipStream_t s) {
    const hipError_t e = launch_kernel(attn8_kernel<DT, S>, dim3(WORKGROUPS), dim3(S::THREADS), s, a);
    if (e != hipSuccess) return e;
    return launch_kernel(attn_join_kernel<DT, S>, dim3(WORKGROUPS / a.members - 1, a.members), dim3(JOIN_WAVES * 64), s, a);
}

template <int DT, int LATENT> hipError_t run8_rows(const AttnArgs &a, int rows, hipStream_t s) {
    switch (rows) {
    case 32: return run8<DT, Shape8<LATENT, 1, 2>>(a, s);
    case 64: return run8<DT, Shape8<LATENT, 2, 2>>(a, s);
    default: return run8<DT, Shape8<LATENT, 4, 1>>(a, s);
    }
}

template <int DT> hipError_t run8_latent(const AttnArgs &a, int rows, hipStream_t s) {
    switch (a.latent) {
    case 128: return run8_rows<DT, 128>(a, rows, s);
    case 256: return run8_rows<DT, 256>(a, rows, s);
    default: return run8_rows<DT, 512>(a, rows, s);
    }
}

}  // namespace

uint64_t attn8_workspace_bytes(const Paged &c, int latent, int heads, int64_t N) {
    return sizeof(Header) + 2ull * WORKGROUPS * plan8(c, heads, N).rows * (latent + 3) * sizeof(float);
}

hipError_t launch_attn8(const AttnArgs &args, hipStream_t s) {
    AttnArgs a = args;
    const Plan8 p = plan8(a.c, a.heads, a.N);
    a.members = p.members;
    return a.dt == DT_BF16 ? run8_latent<DT_BF16>(a, p.rows, s) : run8_latent<DT_F16>(a, p.rows, s);
}

}  // namespace ds4hc
