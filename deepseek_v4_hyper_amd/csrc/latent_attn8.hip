// latent_attn8.hip -- attention over the paged latent cache whose latents are held in 8 bits.
//
// Per query row (a token and a head) and cached row (c8 | r | s) of a sequence, with c = c8 2^(s - 127):
//   x = scale (ql . c + qr . r),  out = softmax(x) C.
// The work is split as for the 16-bit cache (latent_split.hpp): tiles of 64 tokens go to LDS as they
// are, 656 bytes a token in place of 1152, three of them, and every wave takes 32 query rows through them
// with its sums in its 256 accumulation registers. A wave widens what it reads to 16 bits, which is exact.
// A token's power of 2 scales its whole latent, so it goes into the logit's operand, and for the
// second product into the weight: out = sum_j p_j c8_j / sum_j p_j 2^(127 - s_j), p_j = w_j 2^(s_j - 127).
// What bounds it (by clock readings in a copy of the kernel): with all workgroups at work a tile takes 2.5 us with up to 32 rows
// a sequence, of which its bytes need 1.75 at 6 TB/s; with 64 rows 2.7, in float16 3.1, with 128 rows 4.5: instructions of the one
// wave a SIMD has registers for, in 64 tokens by 32 rows 1700 (512 of them widen), a third of which fit beside its 136
// products (4350 cycles of 9000). Beside its tiles a workgroup needs 12 to 13 us for a part of the sums: 1.5 to 2.4 to find its work,
// 1.3 to 1.9 to take it up, 3 to 3.4 for queries and the first page numbers, 0.6 to 2 until the first tile is there, 3.4 to 4.4
// to store the results. A second part (a third of the workgroups has one) costs 8 to 10 again: nothing of it runs beside tiles.
// Measured (latent 512, bf16, both kernels in a graph): 128 sequences of up to 8192 tokens x 16 heads 108 us (3.1 TB/s),
// 64 x 128 heads 113 us, 24 chains of 4 tokens over up to 4096 77 us, one token of 128
// heads over 131000 68 us, 512 tokens over 4096 594 us. The 16-bit cache: 64 x 128 heads 129, chains 103.
// Products of e4m3 values as they are (queries and weights as two such numbers) take the same time within 5 %: they need
// no widening but have to split the weights, and of 64 products the matrix unit keeps what lies within 2^-13 of the
// largest, which takes the error of lse from 1e-8 to 5e-6.
#include <type_traits>

#include "latent_split.hpp"

namespace ds4hc {

namespace {

template <int LATENT_, int ROW_WAVES_, int SETS_> struct Shape8 {
    static constexpr int LATENT = LATENT_, ROW_WAVES = ROW_WAVES_, SETS = SETS_;
    static constexpr int TOKENS = 64, BUFS = 3, STEPS = TOKENS / SETS / 32;
    // (EXTRA and the share that it may take: 4 and a half, 5 and a half, 5 and all take 24 calls of 1 to 256 sequences of up to
    // 8192 tokens, all tile shapes, 1.000, 0.997 and 1.006 of the time, single ones 0.96 to 1.05)
    static constexpr int EXTRA = 6, EXTRA_OF = 2;
    static constexpr int WAVES = ROW_WAVES * SETS, THREADS = WAVES * 64;
    static constexpr int ROWS = ROW_WAVES * 32;
    static constexpr int ROW_BYTES = LATENT, CHUNKS = ROW_BYTES / 16;  // a token's latent in LDS
    // a wave loads the tokens of its GROUPS groups of 16, which lie in one page each unless pages are smaller
    static constexpr int OWN = TOKENS / WAVES, GROUPS = OWN / 16;
    static constexpr int ROPE_AT = TOKENS * ROW_BYTES, SCALE_AT = ROPE_AT + TOKENS * LATENT_ROPE * 2;
    static constexpr int TILE_BYTES = SCALE_AT + TOKENS * 64;  // (scales: a group's 16 bytes a token, 1024 bytes on)
    static constexpr int ROWS_A_LOAD = 1024 / ROW_BYTES;
    static constexpr int LOADS_LATENT = 16 / ROWS_A_LOAD, LOADS_GROUP = LOADS_LATENT + 2 + 1, LOADS = GROUPS * LOADS_GROUP;  // of a wave and tile
    static constexpr int KLATENT = LATENT / 16, KSTEPS = KLATENT + LATENT_ROPE / 16, DBLOCKS = LATENT / 32;
    // of the output, that a wave finishes, and what it takes to store them (with two sets: to give them away)
    static constexpr int BLOCKS = DBLOCKS / SETS, BLOCK_BYTES = 16 * 64 * 4;
    static constexpr int END_BYTES = SETS == 1 ? WAVES * 32 * BLOCKS * 64 : WAVES * (BLOCKS * BLOCK_BYTES + 384);
    static constexpr int RING_BYTES = BUFS * TILE_BYTES > END_BYTES ? BUFS * TILE_BYTES : END_BYTES;
    // the queries, on their way to registers: behind the first tile, or (of 128 rows) where it will be
    static constexpr int QUERY_BYTES = LATENT * 2, QUERY_AT = SETS == 1 ? 0 : TILE_BYTES, QUERY_ROWS = 1024 / QUERY_BYTES;
    static constexpr int QUERY_LOADS = 32 / SETS / QUERY_ROWS;
    static_assert(GROUPS * 16 * WAVES == TOKENS && LOADS_LATENT * ROWS_A_LOAD == 16, "the waves load alike");
    static_assert(QUERY_AT + ROWS * QUERY_BYTES <= RING_BYTES, "the queries' place");
};

// f(0) .. f(N - 1), each with its number as a constant.
template <int... I, class F> __device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, F &&f) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F> __device__ __forceinline__ void for_each(F &&f) { each_of(std::make_integer_sequence<int, N>{}, f); }

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
// as the nearest of these. With float16 operands the ends may lie nearer: at 87 all values are below its smallest
// number (448 x 2^-40), at 152 all but zeros beyond its largest (2^-9 x 2^25).
constexpr int SCALE_NAN = 255;
template <int DT> __device__ __forceinline__ int scale_byte(uint32_t word) {
    constexpr int MIN = DT == DT_F16 ? 87 : 10, MAX = DT == DT_F16 ? 152 : 246;
    return min(max((int)(word & 255), MIN), MAX);
}
__device__ __forceinline__ bool scale_is_nan(uint32_t word) { return (word & 255) == SCALE_NAN; }
// In bfloat16 a weight times a power below 2^-63 may be rounded to few of its bits, or none: they end at 2^-133, and a latent
// of zeros has 2^-117. Such a token adds next to nothing to a row's values, but its weight counts in what divides them.
constexpr uint32_t SCALE_LOW = 64;
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

// 16 bytes a lane, at `voffset` + `soffset` from a buffer's base, to LDS byte lds + 16 * lane; zeros behind the buffer's
// end. Counted like load_to_lds16, of which it saves the address arithmetic of 64 bits. Wait states: one after
// a write of m0.
typedef uint32_t buffer_t __attribute__((ext_vector_type(4)));
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void buffer_to_lds16(uint32_t voffset, buffer_t buffer, int soffset, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(lds), "v"(voffset), "s"(buffer), "s"(soffset)
                 : "m0", "memory");
}
#pragma clang diagnostic pop

// LDS byte of token r's scale word in a tile.
template <class S> __device__ __forceinline__ uint32_t scale_at(int r) { return S::SCALE_AT + (r >> 4) * 1024 + (r & 15) * 16; }

// Not 0 if one of 16 e4m3 values is NaN (all bits but the sign set; there are no infinities).
__device__ __forceinline__ uint32_t nan_bits8(u32x4_t w) {
    constexpr uint32_t REST = 0x7F7F7F7Fu, ONE = 0x01010101u;
    return (((w.x & REST) + ONE) | ((w.y & REST) + ONE) | ((w.z & REST) + ONE) | ((w.w & REST) + ONE)) & ~REST;
}

// SMALL: pages of fewer than 16 tokens, whose rows are looked up one by one.
template <int DT, class S, bool SMALL>
__global__ __launch_bounds__(S::THREADS, 1) void attn8_kernel(AttnArgs a) {
    __shared__ __align__(256) char ring[S::RING_BYTES];
    __shared__ uint32_t not_finite[2];
    __shared__ __align__(16) u32x4_t rope_queries[S::WAVES][LATENT_ROPE / 16][64];  // (no registers are left for them)
    __shared__ __align__(16) float units[S::WAVES][S::TOKENS];  // the tile's powers of 2, each wave's own copy
    __shared__ __align__(16) float powers[DT == DT_F16 ? S::WAVES : 1][S::TOKENS];  // float16: their exponents
    __shared__ __align__(16) uint16_t inverses[DT == DT_BF16 ? S::WAVES : 1][S::TOKENS];  // bfloat16: one over them
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
            at.batch = (int)quotient(off, each);
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
        const int batch = (int)quotient(off, each), u0 = (int)(off - (int64_t)batch * each), u1 = u0 + (int)min((int64_t)(each - u0), left);
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
        u32x4_t q[S::KLATENT];
        // They come through LDS, by loads of whole lines: a lane's own 16 bytes of a row each, straight to registers, take the
        // texture unit 4 us longer. Chunk c of 16 bytes of row r lies at chunk c ^ (r % 16).
        const uint32_t ring_at = lds_address(ring);
        auto load_queries = [&]() {
            const int l = lane_here(), head = min(row0 + (l & 31), n_rows - 1) - tok * a.heads;
            const int64_t o = (int64_t)(q0 + tok) * a.ql_token + head * a.ql_head;
            const char *ql = static_cast<const char *>(a.ql);
            constexpr int CHUNKS = S::QUERY_BYTES / 16;
            const uint32_t first = S::SETS == 1 ? 0 : set * 16, to = (uint32_t)uniform((int)(ring_at + S::QUERY_AT + (row_wave * 32 + first) * S::QUERY_BYTES));
            for_each<S::QUERY_LOADS>([&](auto nth) {
                const uint32_t r = nth * S::QUERY_ROWS + l / CHUNKS, at = ((l % CHUNKS) ^ (r & 15)) << 4;
                const int64_t row = (int64_t)(uint32_t)from_lane((int)(uint32_t)o, first + r) | (int64_t)from_lane((int)(o >> 32), first + r) << 32;
                load_to_lds16(ql + row * 2 + at, to + nth * 1024, ~0ull);
            });
            const elem_t<DT> *qr = static_cast<const elem_t<DT> *>(a.qr) + (int64_t)(q0 + tok) * a.qr_token + head * a.qr_head + (l >> 5) * 8;
#pragma unroll
            for (int k = 0; k < LATENT_ROPE / 16; ++k)
                load_to_lds16(reinterpret_cast<const char *>(qr + k * 16), (uint32_t)uniform((int)lds_address(rope_queries[wave][k])), ~0ull);
        };
        auto read_queries = [&]() {
            const uint32_t l = lane_here(), x = ((l >> 5) * 2) ^ (l & 15);
            const DS4HC_LDS char *row = (const DS4HC_LDS char *)(uintptr_t)(ring_at + S::QUERY_AT + (row_wave * 32 + (l & 31)) * S::QUERY_BYTES);
#pragma unroll
            for (int k = 0; k < S::KLATENT; ++k) {
                const uint32_t c = (k >> 1) * 4 + (k & 1);  // (bit 1: the lane's half)
                q[k] = lds_read16(row + ((x ^ (c & 15)) << 4) + (c >> 4) * 256);
            }
#pragma unroll
            for (int k = 0; k < S::KLATENT; ++k) loaded(q[k]);
        };
        float top = -INFINITY, from = 0.f;  // running maximum less LIFT (what is subtracted: 0 if there is none)
        float sum = 0.f, used = 0.f;        // of the weights, and of the weights as they were rounded
        int least = 255, most = 0;          // float16: scale bytes so far
        uint32_t low = 255;                 // bfloat16: the lowest of the lane's tokens
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
        // Where a tile's tokens lie, and which of them are in the cache. A token that is not there takes a place in the
        // cache all the same (of its page, if that is there, else of page 0), whose bytes do not count.
        struct Where {
            int row;            // SMALL: of the lane's token
            int first[S::GROUPS];  // else: of the wave's groups
            uint64_t ok;
        };
        auto look_up = [&](int tile) {
            Where w = {};
            if (tile >= t_first + n) return w;
            if (tile - pages_from >= 64 >> e_shift) {
                pages_from = tile;
                const int e = lane_here(), in_tile = e >> e_shift;
                const int j = (tile + in_tile) * S::TOKENS + ((e - (in_tile << e_shift)) << a.c.page_shift);
                pages = -1;
                if (tile + in_tile < t_first + n && j < sq.len) pages = a.c.block_table[(int64_t)b * a.c.max_pages + (j >> a.c.page_shift)];
                if (pages >= a.c.n_pages) pages = -1;
                loaded(pages);
            }
            const int e0 = (tile - pages_from) << e_shift, in_page = (1 << a.c.page_shift) - 1, left_over = sq.len - tile * S::TOKENS;
            if constexpr (SMALL) {
                const int r = lane_here(), page = from_lane(pages, e0 + (r >> a.c.page_shift));
                w.row = (max(page, 0) << a.c.page_shift) + (r & in_page);
                w.ok = __ballot(page >= 0 && r < left_over);
            } else {
#pragma unroll
                for (int g = 0; g < S::GROUPS; ++g) {
                    const int o = wave * S::OWN + g * 16;
                    const int page = __builtin_amdgcn_readlane(pages, e0 + (e_shift ? o >> a.c.page_shift : 0));
                    w.first[g] = (max(page, 0) << a.c.page_shift) + ((tile * S::TOKENS + o) & in_page);
                }
                w.ok = ~0ull;
                const uint64_t there = __ballot(pages >= 0) >> e0;
                const int entries = 1 << e_shift, each = S::TOKENS >> e_shift;
                for (int k = 0; k < entries; ++k)
                    if (!((there >> k) & 1)) w.ok &= ~((~0ull >> (64 - each)) << (k * each));
                if (left_over < 64) w.ok &= (1ull << max(left_over, 0)) - 1;
            }
            return w;
        };
        // What a lane's places in the loads have alike: the chunk, swizzled, and the row, of the latents and of the rotated keys.
        struct Place {
            uint32_t chunk, row, rope_chunk, rope_row, scale;
            uint32_t to, to_rope, to_scale;  // the wave's places in LDS
        };
        auto place = [&](uint32_t buf) {
            const uint32_t l = lane_here();
            uint32_t to = buf + wave * (S::OWN * S::ROW_BYTES), to_rope = buf + S::ROPE_AT + wave * (S::OWN * 128), to_scale = buf + S::SCALE_AT + wave * (S::OWN * 64);
            asm volatile("" : "+s"(to), "+s"(to_rope), "+s"(to_scale));  // (not one register for every load)
            return Place{((l % S::CHUNKS) ^ swz8<S::CHUNKS>(l / S::CHUNKS)) << 4, l / S::CHUNKS * STRIDE, ((l % 8) ^ swz8_rope(l / 8)) << 4, l / 8 * STRIDE,
                         (l & 15) * STRIDE, to, to_rope, to_scale};
        };
        // The wave's load number i of the tile to LDS at `buf`. Rows of a group lie one behind another.
        auto load = [&](int i, const Where &w, const buffer_t (&buffers)[S::GROUPS], const Place &x) {
            const int g = i / S::LOADS_GROUP, k = i % S::LOADS_GROUP, r0 = wave * S::OWN + g * 16;
            const uint32_t to = k < S::LOADS_LATENT ? x.to + (g * 16 + k * S::ROWS_A_LOAD) * S::ROW_BYTES
                              : k < S::LOADS_LATENT + 2 ? x.to_rope + (g * 16 + (k - S::LOADS_LATENT) * 8) * 128 : x.to_scale + g * 1024;
            if constexpr (SMALL) {
                const uint32_t l = lane_here();
                auto of_row = [&](int r) { return cache + (uint64_t)(uint32_t)from_lane(w.row, r) * STRIDE; };
                if (k < S::LOADS_LATENT) {
                    const int r = r0 + k * S::ROWS_A_LOAD + l / S::CHUNKS, c = l % S::CHUNKS;
                    load_to_lds16(of_row(r) + ((c ^ swz8<S::CHUNKS>(r)) << 4), to, ~0ull);
                } else if (k < S::LOADS_LATENT + 2) {
                    const int at = r0 + (k - S::LOADS_LATENT) * 8, r = at + l / 8, c = l % 8;
                    load_to_lds16(of_row(r) + S::LATENT + ((c ^ swz8_rope(r)) << 4), to, ~0ull);
                } else {
                    load_to_lds16(of_row(r0 + (l & 15)) + S::LATENT + LATENT_ROPE * 2, to, ~0ull);
                }
            } else if (k < S::LOADS_LATENT) {
                buffer_to_lds16((x.chunk ^ (swz8<S::CHUNKS>(k * S::ROWS_A_LOAD) << 4)) + x.row, buffers[g], k * S::ROWS_A_LOAD * STRIDE, to);
            } else if (k < S::LOADS_LATENT + 2) {
                const int half = k - S::LOADS_LATENT;
                buffer_to_lds16((x.rope_chunk ^ (swz8_rope(half * 8) << 4)) + x.rope_row, buffers[g], half * 8 * STRIDE + S::LATENT, to);
            } else {
                buffer_to_lds16(x.scale, buffers[g], S::LATENT + LATENT_ROPE * 2, to);
            }
        };
        // The groups' rows as buffers; without an end where there is no tile to load.
        auto buffers_of = [&](const Where &w, bool any, buffer_t (&buffers)[S::GROUPS]) {
#pragma unroll
            for (int g = 0; g < S::GROUPS; ++g) {
                const uint64_t at = (uint64_t)cache + (uint64_t)(uint32_t)w.first[g] * STRIDE;
                buffers[g] = {(uint32_t)uniform((int)(uint32_t)at), (uint32_t)uniform((int)(at >> 32)), (uint32_t)uniform(any ? 16 * STRIDE : 0), 0x00020000u};
                // (a load may read scalar registers 5 wait states after the vector unit wrote them)
                asm volatile("s_nop 4" : "+s"(buffers[g]));
            }
        };

        // Tile t (tokens `ok`) in LDS at `at`, and the loads of the one BUFS - 1 further on, if there is one, beside it.
        auto tile = [&](int t, uint64_t ok, uint32_t at, const Where &next, uint32_t at_next) {
            DS4HC_LDS char *buf = (DS4HC_LDS char *)(uintptr_t)at;
            auto scale_of_token = [&](int r) -> DS4HC_LDS uint32_t & { return *(DS4HC_LDS uint32_t *)(buf + scale_at<S>(r)); };
            const int j0 = t * S::TOKENS;
            const bool masked = ok != ~0ull || j0 + S::TOKENS > (a.tree_mask ? context : context + 1);
            uint64_t bad = 0;  // tokens that hold a value that is not finite
            if (masked) {  // the same in all waves
                // Tokens that are not there become zeros, so that what lies in their places meets no weight of 0. Of
                // the others only what some rows see and others do not has to be looked at: the call's own tokens.
                const int lo = max(context - j0, 0), hi = min(S::TOKENS, sq.len - j0);
                auto clear = [&](int i) {
                    const uint32_t zero = here(0);
                    *reinterpret_cast<DS4HC_LDS u32x4_t *>(buf + i * 16) = u32x4_t{zero, zero, zero, zero};
                    if (i % S::CHUNKS == 0) scale_of_token(i / S::CHUNKS) = 127;
                };
                if (threadIdx.x < 2) not_finite[threadIdx.x] = 0;
                wait_and_barrier<63>();
                if (~ok)
                    for (int i = threadIdx.x; i < S::TOKENS * S::CHUNKS; i += S::THREADS)
                        if (!((ok >> (i / S::CHUNKS)) & 1)) clear(i);
                for (int i = lo * S::CHUNKS + threadIdx.x; i < hi * S::CHUNKS; i += S::THREADS)
                    if (((ok >> (i / S::CHUNKS)) & 1) && (nan_bits8(lds_read16(buf + i * 16)) || scale_is_nan(scale_of_token(i / S::CHUNKS))))
                        atomicOr(&not_finite[(i / S::CHUNKS) >> 5], 1u << ((i / S::CHUNKS) & 31));
                wait_and_barrier<63>();
                bad = ((uint64_t)uniform((int)not_finite[1]) << 32) | (uint32_t)uniform((int)not_finite[0]);
                if (bad) {  // zeros, too; the rows that see them get NaN weights
                    for (int i = threadIdx.x; i < S::TOKENS * S::CHUNKS; i += S::THREADS)
                        if ((bad >> (i / S::CHUNKS)) & 1) clear(i);
                    wait_and_barrier<63>();
                }
            }
            const int l = lane_here(), lr = l & 31, lh = l >> 5;
            const uint32_t own_scale = scale_of_token(l);
            units[wave][l] = scale_of<DT>(own_scale);
            if constexpr (DT == DT_BF16) {
                low = min(low, own_scale & 255);
                inverses[wave][l] = (uint16_t)((254 - scale_byte<DT>(own_scale)) << 7);
            }
            if constexpr (DT == DT_F16) {
                powers[wave][l] = scale_is_nan(own_scale) ? NAN : (float)(scale_byte<DT>(own_scale) - 127);
                const int byte = scale_byte<DT>(own_scale);
                const bool counts = (ok >> l) & 1 && !scale_is_nan(own_scale);
                if (__ballot(counts && (byte < least || byte > most))) {
                    int lo = counts ? byte : 255, hi = counts ? byte : 0;
                    for (int m = 32; m; m >>= 1) {
                        lo = min(lo, __shfl_xor(lo, m));
                        hi = max(hi, __shfl_xor(hi, m));
                    }
                    least = uniform(min(least, lo));
                    most = uniform(max(most, hi));
                }
            }
            // LDS offsets of this lane's reads for the first k step, rope step and block of the
            // output; the others' chunks differ in higher bits, which an xor reaches. Made anew for
            // every tile: there are no registers to keep them.
            const int t0 = set * S::STEPS * 32;  // first token of the wave
            const uint32_t k0 = (t0 + lr) * S::ROW_BYTES + ((lh ^ swz8<S::CHUNKS>(lr)) << 4);
            const uint32_t r0 = S::ROPE_AT + (t0 + lr) * 128 + ((lh ^ swz8_rope(lr)) << 4);
            const int vr = lh * 4 + ((l >> 1) & 3) + (l & 8);
            const uint32_t v0 = (t0 + vr) * S::ROW_BYTES + ((((l >> 4) & 1) ^ swz8<S::CHUNKS>(vr)) << 4) + (l & 1) * 8;

            // X^T = K Q^T of 32 tokens. A chain's first operands are read before it begins (begin_k), the others while it
            // runs; `between` gives other work to the vector unit while the matrix unit is busy.
            constexpr int ROPE_STEPS = LATENT_ROPE / 16;
            constexpr int SLOTS_K = S::KSTEPS, SLOTS_V = S::DBLOCKS * 2;  // places for other work
            constexpr int KREADS = S::LATENT / 32, KAHEAD = KREADS < 4 ? KREADS : 4;  // reads of 16 bytes a lane
            u32x4_t kx[KAHEAD];
            uint32_t scale_word;
            auto read_k = [&](int step, int i) {
                return lds_read16(buf + (k0 ^ ((i & 7) << 5)) + (i >> 3) * 256 + step * 32 * S::ROW_BYTES);
            };
            auto begin_k = [&](int step) {
                scale_word = scale_of_token(t0 + step * 32 + lr);
#pragma unroll
                for (int i = 0; i < KAHEAD; ++i) kx[i] = read_k(step, i);
            };
            auto products_k = [&](int step, acc16_t &s, auto &&between) {
                u32x4_t r[2], rq[2];
                auto read_rope = [&](int j) {
                    r[j & 1] = lds_read16(buf + (r0 ^ (j << 5)) + step * 32 * 128);
                    rq[j & 1] = rope_queries[wave][j][l];
                };
                const float unit_k = scale_of<DT>(scale_word);
                for_each<KREADS>([&](auto nth) {
                    constexpr int i = nth;
                    const u32x4_t now = kx[i % KAHEAD];
                    if (i + KAHEAD < KREADS) kx[i % KAHEAD] = read_k(step, i + KAHEAD);
                    if (i == KREADS - 1) read_rope(0), read_rope(1);
                    const u32x4_t w0 = widen8<DT>(now.x, now.y, unit_k), w1 = widen8<DT>(now.z, now.w, unit_k);
                    if (i == 0) mfma32_first_v<DT>(w0, q[0], s);
                    else mfma32_v<DT>(w0, q[2 * i], s);
                    between(2 * i);
                    mfma32_v<DT>(w1, q[2 * i + 1], s);
                    between(2 * i + 1);
                    __builtin_amdgcn_sched_barrier(0);
                });
                for_each<ROPE_STEPS>([&](auto nth) {
                    constexpr int j = nth;
                    mfma32_v<DT>(r[j & 1], rq[j & 1], s);
                    if (j + 2 < ROPE_STEPS) read_rope(j + 2);
                    between(SLOTS_K - ROPE_STEPS + j);
                    __builtin_amdgcn_sched_barrier(0);
                });
            };
            // O^T += V^T P^T of 32 tokens; the order of the tokens is that of X^T's rows, for both operands
            constexpr int VREADS = S::DBLOCKS * 2, VAHEAD = VREADS < 4 ? VREADS : 4;
            u32x2_t vx[VAHEAD];
            auto read_v = [&](int step, int i) {  // block i / 2, tokens 16 (i % 2) .. + 15
                const int d = i / 2;
                return lds_read_tr8(buf + (v0 ^ ((d & 7) << 5)) + (d >> 3) * 256 + (step * 32 + (i & 1) * 16) * S::ROW_BYTES);
            };
            auto begin_v = [&](int step) {
#pragma unroll
                for (int i = 0; i < VAHEAD; ++i) vx[i] = read_v(step, i);
            };
            auto products_v = [&](int step, const u32x4_t (&p)[2], auto &&between) {
                for_each<VREADS>([&](auto nth) {
                    constexpr int i = nth;
                    const u32x4_t a = widen8<DT>(vx[i % VAHEAD].x, vx[i % VAHEAD].y, 1.f);
                    acc[i / 2] = mfma32<DT>(a, p[i & 1], acc[i / 2]);
                    if (i + VAHEAD < VREADS) vx[i % VAHEAD] = read_v(step, i + VAHEAD);
                    between(i);
                    __builtin_amdgcn_sched_barrier(0);
                });
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
                used *= keep;
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
            // Weights 2 i and 2 i + 1 times their tokens' powers of 2, rounded to the type that the second product takes, and
            // what is left of the weights themselves after that: a row is divided by their sum.
            constexpr int PIECES = 8;
            acc4_t powers2[2];  // read ahead, and in bfloat16 one over them
            u32x2_t over[2];
            auto read_powers = [&](int step, int k) {
                powers2[k & 1] = *reinterpret_cast<const acc4_t *>(&units[wave][at_token + step * 32 + 8 * k]);
                if constexpr (DT == DT_BF16) over[k & 1] = *reinterpret_cast<const u32x2_t *>(&inverses[wave][at_token + step * 32 + 8 * k]);
            };
            auto weigh = [&](int step, const acc16_t &s, int i, u32x4_t (&p)[2]) {
                const float u[2] = {powers2[i / 2 & 1][2 * (i & 1)], powers2[i / 2 & 1][2 * (i & 1) + 1]};
                const uint32_t over2 = DT == DT_BF16 ? over[i / 2 & 1][i & 1] : 0;
                if ((i & 1) && i / 2 + 2 < 4) read_powers(step, i / 2 + 2);
                if constexpr (DT == DT_F16) {
                    const float e0 = exp2_fast(s[2 * i] - from), e1 = exp2_fast(s[2 * i + 1] - from);
                    auto inverse = [](float power) { return __uint_as_float((254u << 23) - __float_as_uint(power)); };
                    const float o0 = inverse(u[0]), o1 = inverse(u[1]);
                    sum = fmaf(e0, o0, sum);
                    sum = fmaf(e1, o1, sum);
                    const uint32_t both = pack2<DT>(e0, e1);
                    asm("v_fma_mix_f32 %0, %1, %2, %0 op_sel_hi:[1,0,0]\n\tv_fma_mix_f32 %0, %1, %3, %0 op_sel:[1,0,0] op_sel_hi:[1,0,0]"
                        : "+&v"(used)
                        : "v"(both), "v"(o0), "v"(o1));
                    p[i >> 2][i & 3] = both;
                } else {
                    typedef __bf16 b2_t __attribute__((ext_vector_type(2)));
                    const float e0 = exp2_fast(fmaf(s[2 * i], scale2, -from)), e1 = exp2_fast(fmaf(s[2 * i + 1], scale2, -from));
                    sum += e0;
                    sum += e1;
                    const uint32_t both = pack2<DT>(e0 * u[0], e1 * u[1]);
                    used = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2_t, both), __builtin_bit_cast(b2_t, over2), used, false);
                    p[i >> 2][i & 3] = both;
                }
            };
            constexpr int SLOTS = SLOTS_K * S::STEPS + SLOTS_V, LOAD_EVERY = SLOTS > S::LOADS ? SLOTS / S::LOADS : 1, LOADS_A_SLOT = (S::LOADS + SLOTS - 1) / SLOTS;
            buffer_t buffers[S::GROUPS];
            buffers_of(next, t + S::BUFS - 1 < t_first + n, buffers);
            const Place places = place(at_next);
            auto load_some = [&](int i) {
                if (i % LOAD_EVERY) return;
#pragma unroll
                for (int k = i / LOAD_EVERY * LOADS_A_SLOT; k < (i / LOAD_EVERY + 1) * LOADS_A_SLOT; ++k)
                    if (k < S::LOADS) load(k, next, buffers, places);
            };
            acc16_t s;
            u32x4_t p[2];
            begin_k(0);
            __builtin_amdgcn_sched_barrier(0);
            constexpr int LATE = SLOTS_K - ROPE_STEPS;  // the chain's latents have been read
            if constexpr (S::STEPS == 1) {
                products_k(0, s, [&](int i) {
                    load_some(i);
                    if (i == LATE) begin_v(0);
                    if (i == LATE + 1) read_powers(0, 0), read_powers(0, 1);
                });
                mfma_results(s);
                const float high = largest(0, s);
                if (__any(too_high(high))) raise(high);
#pragma unroll
                for (int i = 0; i < PIECES; ++i) weigh(0, s, i, p);
                products_v(0, p, [&](int i) { load_some(SLOTS_K + i); });
            } else {  // two steps, the softmax of each beside the products of the other, as far as can be
                acc16_t s1;
                u32x4_t p1[2];
                products_k(0, s, [&](int i) {
                    load_some(i);
                    if (i == LATE) begin_k(1);
                    if (i == LATE + 1) read_powers(0, 0), read_powers(0, 1);
                });
                mfma_results(s);
                float high = largest(0, s);
                if (__any(too_high(high))) raise(high);
                products_k(1, s1, [&](int i) {
                    load_some(SLOTS_K + i);
#pragma unroll
                    for (int k = i * PIECES / SLOTS_K; k < (i + 1) * PIECES / SLOTS_K; ++k) weigh(0, s, k, p);
                    if (i == LATE) begin_v(0);
                    if (i == SLOTS_K - 1) read_powers(1, 0), read_powers(1, 1);
                });
                mfma_results(s1);
                high = largest(1, s1);
                if (__any(too_high(high))) {
                    const float keep = raise(high);
#pragma unroll
                    for (int i = 0; i < 8; ++i) p[i >> 2][i & 3] = scale2_words<DT>(p[i >> 2][i & 3], keep);
                }
                products_v(0, p, [&](int i) {
                    load_some(2 * SLOTS_K + i);
#pragma unroll
                    for (int k = i * PIECES / SLOTS_V; k < (i + 1) * PIECES / SLOTS_V; ++k) weigh(1, s1, k, p1);
                });
                begin_v(1);
                products_v(1, p1, [](int) {});
            }
        };

        // ---- tiles: the loads of the next two run beside this one's products. All waves are done with
        // tile t - 1 when they meet at the barrier of tile t, so its buffer takes tile t + 2.
        static_assert(S::BUFS == 3, "two tiles on their way");
        wait_and_barrier<63>();  // the last part's reads of the ring
        load_queries();
        Where now = look_up(t_first), next = look_up(t_first + 1);
        if constexpr (S::SETS == 1) {
            wait_and_barrier<0>();
            read_queries();
            wait_and_barrier<63>();
        }
        buffer_t buffers[S::GROUPS];
        buffers_of(now, true, buffers);
#pragma unroll
        for (int i = 0; i < S::LOADS; ++i) load(i, now, buffers, place(ring_at));
        if constexpr (S::SETS == 2) {
            wait_and_barrier<S::LOADS>();  // the queries are there, of both sets
            read_queries();
            wait_and_barrier<63>();  // and read: their place is the second tile's
        }
        buffers_of(next, n > 1, buffers);
#pragma unroll
        for (int i = 0; i < S::LOADS; ++i) load(i, next, buffers, place(ring_at + S::TILE_BYTES));
        uint64_t ok = now.ok, ok_next = next.ok;
        uint32_t at = 0;
        for (int i = 0; i < n; ++i) {
            wait_and_barrier<S::LOADS>();  // only the next tile's loads are on their way
            const Where behind = look_up(t_first + i + 2);
            tile(t_first + i, ok, ring_at + at, behind, ring_at + (at >= S::TILE_BYTES ? at - S::TILE_BYTES : at + 2 * S::TILE_BYTES));
            at = at == 2 * S::TILE_BYTES ? 0 : at + S::TILE_BYTES;
            ok = ok_next;
            ok_next = behind.ok;
        }
        wait_and_barrier<0>();  // (those behind the last tile write zeros to LDS)

        // ---- the part's result
#pragma unroll
        for (int d = 0; d < S::DBLOCKS; ++d) pin_acc(acc[d]);
        const int l = lane_here(), lh = l >> 5, my_row = row0 + (l & 31), head = my_row - tok * a.heads;
        const bool whole = t_first == 0 && n == sq.kv_tiles, mine = my_row < n_rows;  // (a part's rows behind the last: never looked at)
        const int in = my_row - row_tile * S::ROWS;
        float *part = part_at<S>(a, cluster, part_of_first ? 0 : 1, member);
        // A token whose power is far below the others' (float16), or far below 1 (bfloat16), may keep nothing of a weight that
        // counts, so where they differ by more than 2^6, or one is below SCALE_LOW, the sum before the rounding is what divides.
        // (In bfloat16 leaving such tokens alone out of the rounded sum takes a second branch beside a tile's products, up to 1.4 %
        // of a call for up to 0.5.)
        if (DT == DT_F16 ? most - least > 6 : __any(low < SCALE_LOW)) used = sum;
        float all = sum_halves(sum), all_used = sum_halves(used);
        // the blocks of the output that this wave finishes: all, or with two sets its half
        constexpr int BLOCKS = S::BLOCKS, BLOCK_BYTES = S::BLOCK_BYTES;
        acc16_t fin[BLOCKS];
        if constexpr (S::SETS == 1) {
#pragma unroll
            for (int d = 0; d < BLOCKS; ++d) fin[d] = acc[d];
            wait_and_barrier<63>();  // the last tile has been read by all
        } else {
            // each set gives the other one's half through LDS, and all is brought to the common maximum
            float *st = reinterpret_cast<float *>(ring + S::WAVES * BLOCKS * BLOCK_BYTES);  // maximum, sums [row waves][sets][32]
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
                mine_st[64 + l] = all_used;
            }
            if (set == 0) give_half(std::integral_constant<int, BLOCKS>{});
            else give_half(std::integral_constant<int, 0>{});
            wait_and_barrier<63>();
            const float other = other_st[l & 31], to = fmaxf(top, other);
            // (no logit that is a number, -infinity: the sums are 0 or NaN)
            const float keep = to == -INFINITY ? 1.f : exp2_fast(top - to), add = to == -INFINITY ? 1.f : exp2_fast(other - to);
            all = all * keep + other_st[32 + (l & 31)] * add;
            all_used = all_used * keep + other_st[64 + (l & 31)] * add;
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
            const float inv = all_used == 0.f ? 0.f : 1.f / all_used;
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
                part[S::ROWS * (S::LATENT + 2) + in] = all_used;
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

// How a call is run, by the average rows of a sequence. Up to 64: a tile of them each. More, with latents of 512: tiles of 64
// rows in clusters of two, of which a cut leaves half the bytes of sums that it leaves of 128 rows; unless there are so many
// rows that most tiles are cut little, where 128 rows keep the matrix unit better fed. Of 128 rows, of 64, and of 64 in clusters
// of four (whole calls in a graph, us; 128 heads unless said): 8 trees of up to 40 tokens x 16 heads, float16, 76, 66 and 68, 24
// chains of up to 4 tokens 82, 77 and 82, 32 over up to 2048 83, 64 and 70, one token over 131000 78, 68 and 99, 64 x 1 over up to
// 8192 121, 113 and 186, 64 chains of up to 4 228, 235 and 263, 24 x up to 16 157, 157 and 166, 512 tokens over 4096 594, 680 and 682.
// Smaller latents have smaller sums: 256 rather 128 rows (64 x 1 72, 80 and 132; 24 chains 53, 57 and 63).
// Clusters of four read the cache once, but all of it waits for the slowest, and the caches serve the single ones as well.
struct Plan8 {
    int rows, members;
};

Plan8 plan8(const Paged &c, int latent, int heads, int64_t N) {
    const int64_t all = N * heads, rows = (all + c.n_seqs - 1) / c.n_seqs;
    if (rows <= 32) return {32, 1};
    if (rows <= 64) return {64, 1};
    if (latent == 512 && all < WORKGROUPS * 128) return {64, 2};
    return {128, 1};
}

template <int DT, class S> hipError_t run8(const AttnArgs &a, hipStream_t s) {
    const dim3 grid(WORKGROUPS), block(S::THREADS);
    const hipError_t e = a.c.page_shift >= 4 ? launch_kernel(attn8_kernel<DT, S, false>, grid, block, s, a) : launch_kernel(attn8_kernel<DT, S, true>, grid, block, s, a);
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
    return sizeof(Header) + 2ull * WORKGROUPS * plan8(c, latent, heads, N).rows * (latent + 3) * sizeof(float);
}

hipError_t launch_attn8(const AttnArgs &args, hipStream_t s) {
    AttnArgs a = args;
    const Plan8 p = plan8(a.c, a.latent, a.heads, a.N);
    a.members = p.members;
    return a.dt == DT_BF16 ? run8_latent<DT_BF16>(a, p.rows, s) : run8_latent<DT_F16>(a, p.rows, s);
}

}  // namespace ds4hc
