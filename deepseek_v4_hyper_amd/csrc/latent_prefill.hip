// latent_prefill.hip -- attention over expanded keys and values of a ragged batch.
//
// Per query row (a token, one head) and key of its sequence:
//   s = scale (qn . kn + qr . kr),  out = softmax(s) V.
// One pass over the keys with a running maximum and sum; both products on the matrix unit:
// 640 operations a (row, key), while a key's 640 bytes serve 128 rows. What bounds it, by counters
// (4096 tokens x 32 heads, 128 rows a workgroup, two waves a SIMD): a wave is on a tile for 4770
// cycles. 2000 it issues (302 vector instructions, 40 products among them, 58 of LDS, 85 scalar), 1420 it
// waits for its turn, 1340 for data, results and the other waves. The matrix unit is busy 1280 of
// them a wave, the vector unit 1180 besides, both at once 540. A workgroup alone on its CU takes 1.86 us a
// tile, two 2.68 for both. The clock falls from 2.4 to 1.94 GHz. 66 tiles one behind another in each of
// 512 places are 162 us; the rest of the call are places out of work: CUs are busy 83 % of its time
// (8192 tokens: 93 %, 4450 cycles). 4096 tokens x 32 heads, causal: 187-210 us, 860 TFLOP/s, without a
// mask 347 us, 990 TFLOP/s; 8192 tokens, causal: 686 us, 1.00 PFLOP/s; 4096 x 128 heads 755 us, 910.
#include "latent_device.hpp"

namespace ds4hc {

namespace {

constexpr int THREADS = 256, WAVES = 4;
constexpr int TOKENS = 64;                           // keys a tile
constexpr int KV_BYTES = (PREFILL_NOPE + PREFILL_VALUE) * 2, ROPE_BYTES = LATENT_ROPE * 2;
constexpr int ROPE_AT = TOKENS * KV_BYTES, TILE_BYTES = TOKENS * (KV_BYTES + ROPE_BYTES);
constexpr int DQ = PREFILL_NOPE + LATENT_ROPE;
constexpr int KNOPE = PREFILL_NOPE / 16, KSTEPS = DQ / 16, DBLOCKS = PREFILL_VALUE / 32;
constexpr int SORTED = 32;                           // sequences at most that are sorted by their keys
constexpr unsigned GRID_X = 1u << 20;                // workgroups in x (a dispatch has 2^32 threads a dimension)

// Tile shapes. The waves of a workgroup take 32 rows each, all of one head: 128 rows, or 64 in two
// sets of waves of which each takes half of a tile's keys, in steps of 32.
template <int SETS_> struct Rows {
    static constexpr int SETS = SETS_, WAVES_OF_SET = WAVES / SETS, ROWS = WAVES_OF_SET * 32, STEPS = TOKENS / SETS / 32;
};

// Swizzle of the 16-byte chunks of a token's row in LDS: 16 values over 16 rows, the upper 2
// bits 4 values over 4 rows (for the transposing reads, 64 bytes of 4 rows at a time).
__device__ __forceinline__ int swz(int r) { return ((r & 3) << 2) | ((r >> 2) & 3); }
__device__ __forceinline__ int swz_rope(int r) { return (r >> 1) & 7; }

// Row tile `nth` of the batch: its sequence and its first row there; -1 if there is none. A
// sequence's last row tile, which sees the most keys, comes first, and of up to 32 sequences the
// one with the most keys, so that the workgroups that start last have little to do (68 -> 57 us for
// six ragged prompts of up to 1500 tokens x 8 heads behind 700). Of more sequences each has a small
// share of the work, and sorting costs every workgroup more than that saves (48 of up to 300
// tokens x 8 heads: 36 us as they stand, 40 sorted).
template <int ROWS> __device__ __forceinline__ int find_tile(const PrefillArgs &a, int nth, int &row0) {
    const int lane = threadIdx.x & 63, B = a.n_seqs, n = (int)a.N, per = (B + 63) / 64;
    auto tiles = [&](int b) { return (max(cu_at(a.cu_q, b + 1, n) - cu_at(a.cu_q, b, n), 0) + ROWS - 1) / ROWS; };
    int mine = 0, which = lane;
    if (per == 1) {
        int keys = -1;
        if (lane < B) mine = tiles(lane);
        if (lane < B && B <= SORTED) {
            keys = max(cu_at(a.cu_k, lane + 1, (int)a.S) - cu_at(a.cu_k, lane, (int)a.S), 0);
        }
        if (B <= SORTED) {
            int place = 0;  // among the sequences, sorted
            for (int b = 0; b < B; ++b) {
                const int other = __builtin_amdgcn_readlane(keys, b);
                place += other > keys || (other == keys && b < lane);
            }
            if (lane >= B) place = lane;
            mine = __builtin_amdgcn_ds_permute(place << 2, mine);
            which = __builtin_amdgcn_ds_permute(place << 2, lane);
        }
    } else {
        for (int i = 0; i < per; ++i)
            if (lane * per + i < B) mine += tiles(lane * per + i);
    }
    int upto = mine;
    for (int m = 1; m < 64; m <<= 1) {
        const int o = __shfl_up(upto, m);
        if (lane >= m) upto += o;
    }
    const uint64_t in = __ballot(nth >= upto - mine && nth < upto);
    if (!in) return -1;
    const int who = __builtin_ctzll(in);
    int rest = nth - __builtin_amdgcn_readlane(upto - mine, who);
    if (per == 1) {
        row0 = (__builtin_amdgcn_readlane(mine, who) - 1 - rest) * ROWS;
        return __builtin_amdgcn_readlane(which, who);
    }
    for (int b = who * per; b < min(B, (who + 1) * per); ++b) {
        const int t = tiles(b);
        if (rest < t) {
            row0 = (t - 1 - rest) * ROWS;
            return b;
        }
        rest -= t;
    }
    return -1;
}

template <int DT, class S>
__global__ __launch_bounds__(THREADS, 2) void prefill_kernel(PrefillArgs a) {
    __shared__ __align__(256) char ring[2 * TILE_BYTES];  // two workgroups a CU fill its LDS
    const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
    const int row_wave = wave % S::WAVES_OF_SET, set = wave / S::WAVES_OF_SET;
    // heads are neighbours in the grid: with 8 of them or more an XCD keeps to its own heads' keys.
    const unsigned id = blockIdx.y * GRID_X + blockIdx.x;
    const int head = id % a.heads;
    int row0 = 0;
    const int b = uniform(find_tile<S::ROWS>(a, (int)(id / a.heads), row0));
    if (b < 0) return;
    row0 = uniform(row0);
    const int q0 = uniform(cu_at(a.cu_q, b, (int)a.N)), few = uniform(cu_at(a.cu_q, b + 1, (int)a.N)) - q0;
    const int k0 = uniform(cu_at(a.cu_k, b, (int)a.S)), len = max(uniform(cu_at(a.cu_k, b + 1, (int)a.S)) - k0, 0);
    // keys that row i sees: the first limit(i)
    const int before = len - few;  // may be negative
    auto limit = [&](int i) { return a.full ? len : max(min(len, i + before + 1), 0); };
    const int n = (limit(min(row0 + S::ROWS, few) - 1) + TOKENS - 1) / TOKENS;  // tiles
    const float scale2 = a.scale * LOG2E;
    const int my = row0 + row_wave * 32 + (lane & 31);

    float top = -INFINITY, from = 0.f;  // running maximum less LIFT (what is subtracted: 0 if there is none)
    float sum = 0.f, used = 0.f;        // sums of the weights and of the rounded weights
    acc16_t acc[DBLOCKS];
#pragma unroll
    for (int d = 0; d < DBLOCKS; ++d) {
        acc[d] = acc16_t{};
        pin_acc(acc[d]);
    }

    if (n > 0) {
        const int lim = limit(min(my, few - 1));  // rows behind the last repeat it
        const char *kv = static_cast<const char *>(a.kv) + ((int64_t)k0 * a.heads + head) * KV_BYTES;
        const char *kr = static_cast<const char *>(a.k_rope) + (int64_t)k0 * a.k_rope_stride * 2;
        const uint32_t kv_step = (uint32_t)a.heads * KV_BYTES;  // bytes between tokens, at most 2^19
        const uint64_t rope_step = (uint64_t)a.k_rope_stride * 2;
        constexpr int KV_LOADS = TOKENS * KV_BYTES / 1024 / WAVES, LOADS = KV_LOADS + TOKENS * ROPE_BYTES / 1024 / WAVES;
        // The wave's load number i of a tile: two tokens' keys and values, or 8 tokens' rope keys. Behind
        // the sequence's last token, `room` tokens on from the tile's first, that one is loaded again (what
        // lies there is another's, and may be NaN, which a weight of 0 would not hide). The tokens' part
        // of an offset and the lane's chunk have no bits in common, and both swizzles part into the
        // lane's share and load i's, so that three instructions make an offset.
        const int l0 = lane_here();
        const uint32_t row_off = (uint32_t)(wave * KV_LOADS * 2 + (l0 >> 5)) * kv_step, chunk0 = ((l0 & 31) ^ swz(l0 >> 5)) << 4;
        const int rope_row = wave * (LOADS - KV_LOADS) * 8 + (l0 >> 3);
        const uint32_t rope_chunk0 = ((l0 & 7) ^ swz_rope(l0 >> 3)) << 4;
        auto load = [&](int i, const char *kv_tile, const char *kr_tile, int room, uint32_t buf, uint64_t lanes) {
            if (i < KV_LOADS) {
                const uint32_t off = __builtin_elementwise_min(row_off + (uint32_t)i * 2 * kv_step, (uint32_t)room * kv_step);
                load_to_lds16(kv_tile, (chunk0 ^ (swz(i * 2) << 4)) + off, buf + (wave * KV_LOADS + i) * 2 * KV_BYTES, lanes);
            } else {
                const int nth = i - KV_LOADS;
                const uint64_t off = (uint64_t)(uint32_t)__builtin_elementwise_min(rope_row + nth * 8, room) * rope_step;
                load_to_lds16(kr_tile + off + (rope_chunk0 ^ (swz_rope(nth * 8) << 4)), buf + ROPE_AT + (wave * (LOADS - KV_LOADS) + nth) * 8 * ROPE_BYTES, lanes);
            }
        };
        static_assert(KV_LOADS % 8 == 0 && LOADS - KV_LOADS == 2, "a wave's first token has no part in its swizzle");
        const uint32_t ring_at = lds_address(ring);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) load(i, kv, kr, min(len - 1, TOKENS - 1), ring_at, ~0ull);
        u32x4_t q[KSTEPS];
        {
            const elem_t<DT> *from_q = static_cast<const elem_t<DT> *>(a.q) + ((int64_t)(q0 + min(my, few - 1)) * a.heads + head) * DQ + (lane >> 5) * 8;
#pragma unroll
            for (int k = 0; k < KSTEPS; ++k) q[k] = *reinterpret_cast<const u32x4_t *>(from_q + k * 16);
#pragma unroll
            for (int k = 0; k < KSTEPS; ++k) loaded_acc(q[k]);
        }

        // LDS offsets of this lane's reads for the first k step, rope step and block of values; the
        // others' chunks differ in higher bits, which an xor reaches
        const int lr = l0 & 31, lh = l0 >> 5;
        const uint32_t k_at = (set * 32 * (S::SETS - 1) + lr) * KV_BYTES + ((lh ^ swz(lr)) << 4);
        const uint32_t r_at = ROPE_AT + (set * 32 * (S::SETS - 1) + lr) * ROPE_BYTES + ((lh ^ swz_rope(lr)) << 4);
        const int vr = lh * 4 + ((l0 >> 2) & 3);
        const uint32_t v_at = (set * 32 * (S::SETS - 1) + vr) * KV_BYTES + PREFILL_NOPE * 2 + (((((l0 >> 4) & 1) << 1 | ((l0 >> 1) & 1)) ^ swz(vr)) << 4) + (l0 & 1) * 8;
        const uint32_t v8_at = (v_at ^ 32) + 8 * KV_BYTES;  // 8 rows on, swz differs in bit 1
        const int first_masked = limit(row0) / TOKENS;      // the first tile that some rows do not see whole

        auto tile = [&](int t, uint32_t at, uint32_t at_next) {
            DS4HC_LDS char *buf = (DS4HC_LDS char *)(uintptr_t)at;
            const int j0 = t * TOKENS;
            const bool masked = t >= first_masked;
            uint64_t bad = 0;  // tokens whose values are not all finite
            if (masked) {  // the same in all waves, and so is what they find
                const DS4HC_LDS char *at_values = buf + (lane_here() >> 4) * KV_BYTES + PREFILL_NOPE * 2 + (lane_here() & 15) * 16;
                uint32_t found = 0;
#pragma unroll 4
                for (int i = 0; i < TOKENS / 4; ++i) found |= not_finite_bits<DT>(lds_read16(at_values + i * 4 * KV_BYTES));
                if (__any(found != 0))  // rarely: which
                    for (int i = 0; i < TOKENS / 4; ++i) {
                        const uint64_t lanes = __ballot(not_finite_bits<DT>(lds_read16(at_values + i * 4 * KV_BYTES)) != 0);
                        for (int r = 0; r < 4; ++r) bad |= (uint64_t)((lanes >> (16 * r) & 0xFFFF) != 0) << (i * 4 + r);
                    }
                if (bad) {  // zero in LDS, so that they meet no weight of 0; the rows that see them get NaN weights
                    wait_and_barrier<63>();
                    for (int i = threadIdx.x; i < TOKENS * 16; i += THREADS)
                        if ((bad >> (i >> 4)) & 1) {
                            const uint32_t zero = here(0);
                            *reinterpret_cast<DS4HC_LDS u32x4_t *>(buf + (i >> 4) * KV_BYTES + PREFILL_NOPE * 2 + (i & 15) * 16) = u32x4_t{zero, zero, zero, zero};
                        }
                    wait_and_barrier<63>();
                }
            }
            // Reads of both products' left operands, AHEAD of them under way: S^T = K Q^T, and
            // O^T += V^T P^T with the tokens in the order of S^T's rows for both operands
            constexpr int AHEAD = 4, ALL_K = S::STEPS * KSTEPS, VSTEPS = S::STEPS * DBLOCKS * 2;
            auto read = [&](int n) {
                if (n < ALL_K) {
                    const int step = n / KSTEPS, k = n % KSTEPS;
                    return k < KNOPE ? lds_read16(buf + (k_at ^ (k << 5)) + step * 32 * KV_BYTES)
                                     : lds_read16(buf + (r_at ^ ((k - KNOPE) << 5)) + step * 32 * ROPE_BYTES);
                }
                const int i = n - ALL_K;  // block i % DBLOCKS, tokens 16 (i / DBLOCKS) .. + 15
                const uint32_t chunk = (i % DBLOCKS) << 6, off = (i / DBLOCKS) * 16 * KV_BYTES;
                const u32x2_t lo = lds_read_tr(buf + (v_at ^ chunk) + off), hi = lds_read_tr(buf + (v8_at ^ chunk) + off);
                return u32x4_t{lo.x, lo.y, hi.x, hi.y};
            };
            u32x4_t x[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) x[i] = read(i);
            // `between` gives other work to the vector unit while the matrix unit is busy
            auto products_k = [&](int step, acc16_t &s, auto &&between) {
#pragma unroll
                for (int i = 0; i < KSTEPS; ++i) {
                    const int n = step * KSTEPS + i;
                    if (i == 0) mfma32_first_va<DT>(x[n % AHEAD], q[i], s);
                    else mfma32_va<DT>(x[n % AHEAD], q[i], s);
                    x[n % AHEAD] = read(n + AHEAD);
                    between(i);
                    __builtin_amdgcn_sched_barrier(0);
                }
            };
            auto products_v = [&](const u32x4_t (&p)[2], const u32x4_t (&p1)[2], auto &&between) {
#pragma unroll
                for (int i = 0; i < VSTEPS; ++i) {
                    const int n = ALL_K + i;
                    acc[i % DBLOCKS] = mfma32<DT>(x[n % AHEAD], i < DBLOCKS * 2 ? p[i / DBLOCKS] : p1[i / DBLOCKS - 2], acc[i % DBLOCKS]);
                    if (i + AHEAD < VSTEPS) x[n % AHEAD] = read(n + AHEAD);
                    between(i);
                    __builtin_amdgcn_sched_barrier(0);
                }
            };
            // Softmax of a step, in pieces. The mask, and the largest logit (of the lane's row).
            auto largest = [&](int step, acc16_t &s) {
                if (masked) {
                    const int sees_n = lim - j0;
                    const uint64_t sees = sees_n >= 64 ? ~0ull : sees_n <= 0 ? 0 : (1ull << sees_n) - 1;
                    const int at0 = (step + set * (S::SETS - 1)) * 32 + (lane_here() >> 5) * 4;
                    const uint32_t see = (uint32_t)(sees >> at0), nan = (uint32_t)((sees & bad) >> at0);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int r = 8 * (i / 4) + i % 4;
                        s[i] = (nan >> r) & 1 ? NAN : (see >> r) & 1 ? s[i] : -INFINITY;
                    }
                }
                return max_halves(max16(s));
            };
            // A new running maximum. It is a whole number, so that what is there is scaled by a power of 2:
            // without rounding, but for weights that become float16's subnormal numbers (LIFT: half a step
            // of those is 2^-31 of the largest weight). Whether one is needed is looked at in one rounding,
            // so that no weight passes 2^(LAZY + LIFT) however far from 0 the logits lie.
            auto too_high = [&](float high) { return fmaf(high, scale2, -top) > LAZY + LIFT<DT>; };
            auto raise = [&](float high) {
                const float was = top;
                top = fmaxf(top, ceilf(high * scale2) - LIFT<DT>);
                from = top == -INFINITY ? 0.f : top;
                const float keep = was == -INFINITY ? 0.f : exp2_fast(was - top);
                sum *= keep;
                used *= keep;
                if (__any(was != -INFINITY)) {  // (the first maximum: the sums are 0)
#pragma unroll
                    for (int d = 0; d < DBLOCKS; ++d) {
                        pin_acc(acc[d]);
                        acc[d] *= keep;
                        pin_acc(acc[d]);
                    }
                }
                return keep;
            };
            // Weights 2 i and 2 i + 1, rounded to the type that the second product takes. (In two 16-bit
            // parts they would double that product, 40 % of all, to take the error of an output from
            // 1.3 times that of float32 weights to 1.)
            auto weight2 = [&](const acc16_t &s, int i, u32x4_t (&p)[2]) {
                const float e0 = exp2_fast(fmaf(s[2 * i], scale2, -from)), e1 = exp2_fast(fmaf(s[2 * i + 1], scale2, -from));
                sum += e0;
                sum += e1;
                uint32_t w = pack2<DT>(e0, e1);
                asm volatile("" : "+v"(w));  // here, beside the products, and not where it is first used
                p[i >> 2][i & 3] = w;
                used = add2_words<DT>(w, used);
            };
            const int t_next = min(t + 1, n - 1), room = min(len - 1 - t_next * TOKENS, TOKENS - 1);
            const char *kv_next = kv + (uint64_t)(uint32_t)t_next * ((uint64_t)kv_step * TOKENS), *kr_next = kr + (uint64_t)(uint32_t)t_next * (rope_step * TOKENS);
            const uint64_t lanes = (uint64_t)uniform((int64_t)(t + 1 < n ? -1 : 0));
            acc16_t s, s1;
            u32x4_t p[2], p1[2];
            if constexpr (S::STEPS == 2) {
                products_k(0, s, [&](int i) {
                    if (i % 2 == 0) load(i / 2, kv_next, kr_next, room, at_next, lanes);
                });
                mfma_results(s);
                float high = largest(0, s);
                if (__any(too_high(high))) raise(high);
                products_k(1, s1, [&](int i) {
                    if (i < 8) weight2(s, i, p);
                    if (i % 2 == 0 && KSTEPS / 2 + i / 2 < LOADS) load(KSTEPS / 2 + i / 2, kv_next, kr_next, room, at_next, lanes);
                });
                mfma_results(s1);
                high = largest(1, s1);
                if (__any(too_high(high))) {
                    const float keep = raise(high);
#pragma unroll
                    for (int i = 0; i < 8; ++i) p[i >> 2][i & 3] = scale2_words<DT>(p[i >> 2][i & 3], keep);
                }
                // (the last weights are needed from three quarters on)
                products_v(p, p1, [&](int i) {
                    if (i < 8 && i % 4 != 3) weight2(s1, i - i / 4, p1);
                    if (i == 8 || i == 9) weight2(s1, i - 2, p1);
                });
            } else {
                products_k(0, s, [&](int i) {
                    if (i < LOADS) load(i, kv_next, kr_next, room, at_next, lanes);
                });
                mfma_results(s);
                const float high = largest(0, s);
                if (__any(too_high(high))) raise(high);
#pragma unroll
                for (int i = 0; i < 4; ++i) weight2(s, i, p);
                products_v(p, p, [&](int i) {
                    if (i < 4) weight2(s, 4 + i, p);
                });
            }
        };

        // the next tile's loads run beside this one's products. All waves are done with tile t - 1 when
        // they meet at the barrier of tile t, so its buffer takes tile t + 1.
        for (int t = 0; t < n; ++t) {
            wait_and_barrier<0>();
            tile(t, ring_at + (t & 1) * TILE_BYTES, ring_at + ((t + 1) & 1) * TILE_BYTES);
        }
    }

    // ---- results
#pragma unroll
    for (int d = 0; d < DBLOCKS; ++d) pin_acc(acc[d]);
    const int l = lane_here(), lh = l >> 5;
    float all = sum_halves(sum), all_used = sum_halves(used);
    wait_and_barrier<63>();  // the last tile has been read by all
    if constexpr (S::SETS == 2) {
        // the second set's sums through LDS, brought to the common maximum
        constexpr int WAVE_BYTES = DBLOCKS * 16 * 64 * 4;
        static_assert(S::WAVES_OF_SET * (WAVE_BYTES + 384) <= 2 * TILE_BYTES, "a set's sums and statistics");
        float *st = reinterpret_cast<float *>(ring + S::WAVES_OF_SET * WAVE_BYTES);  // maximum, sums [row waves][32]
        if (set == 1) {
            if (lh == 0) {
                st[row_wave * 96 + l] = top;
                st[row_wave * 96 + 32 + l] = all;
                st[row_wave * 96 + 64 + l] = all_used;
            }
#pragma unroll
            for (int d = 0; d < DBLOCKS; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<acc4_t *>(ring + row_wave * WAVE_BYTES + ((d * 4 + i) * 64 + l) * 16) =
                        acc4_t{acc[d][4 * i], acc[d][4 * i + 1], acc[d][4 * i + 2], acc[d][4 * i + 3]};
        }
        wait_and_barrier<63>();
        if (set == 1) return;
        const float other = st[row_wave * 96 + (l & 31)], to = fmaxf(top, other);
        // (no logit that is a number, -infinity: the sums are 0 or NaN)
        const float keep = to == -INFINITY ? 1.f : exp2_fast(top - to), keep1 = to == -INFINITY ? 1.f : exp2_fast(other - to);
        all = all * keep + st[row_wave * 96 + 32 + (l & 31)] * keep1;
        all_used = all_used * keep + st[row_wave * 96 + 64 + (l & 31)] * keep1;
        top = to;
#pragma unroll
        for (int d = 0; d < DBLOCKS; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const acc4_t v = *reinterpret_cast<const acc4_t *>(ring + row_wave * WAVE_BYTES + ((d * 4 + i) * 64 + l) * 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[d][4 * i + e] = acc[d][4 * i + e] * keep + v[e] * keep1;
            }
    }
    const float inv = all_used == 0.f ? 0.f : 1.f / all_used;
    if (a.lse && lh == 0 && my < few) a.lse[(int64_t)(q0 + my) * a.heads + head] = row_lse<DT>(top, all);
    // through LDS, to store whole rows: chunk c of row r at chunk c ^ (r % 16). (A wave's own place; with
    // two sets it lies in what that wave has just read.)
    constexpr int OUT_BYTES = PREFILL_VALUE * 2;
    char *rows_at = ring + row_wave * 32 * OUT_BYTES * S::SETS;
#pragma unroll
    for (int d = 0; d < DBLOCKS; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<u32x2_t *>(rows_at + (l & 31) * OUT_BYTES + (((d * 4 + i) ^ (l & 15)) << 4) + lh * 8) = u32x2_t{
                pack2<DT>(acc[d][4 * i] * inv, acc[d][4 * i + 1] * inv), pack2<DT>(acc[d][4 * i + 2] * inv, acc[d][4 * i + 3] * inv)};
    char *out = static_cast<char *>(a.out) + ((int64_t)(q0 + row0 + row_wave * 32) * a.heads + head) * OUT_BYTES;
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        const int r = i + (l >> 4), c = l & 15;
        const u32x4_t v = *reinterpret_cast<const u32x4_t *>(rows_at + r * OUT_BYTES + ((c ^ (r & 15)) << 4));
        if (row0 + row_wave * 32 + r < few) *reinterpret_cast<u32x4_t *>(out + (int64_t)r * a.heads * OUT_BYTES + c * 16) = v;
    }
}

template <int DT, class S> hipError_t run(const PrefillArgs &a, hipStream_t s) {
    const int tiles = (int)(a.N / S::ROWS) + (int)(a.n_seqs < a.N ? a.n_seqs : a.N);  // at most
    const uint64_t groups = (uint64_t)tiles * (uint64_t)a.heads;  // at most 2^31: N * heads is at most 2^30
    const dim3 grid((unsigned)(groups < GRID_X ? groups : GRID_X), (unsigned)((groups + GRID_X - 1) / GRID_X));
    return launch_kernel(prefill_kernel<DT, S>, grid, dim3(THREADS), s, a);
}

// 64 rows a workgroup where 128 would leave places for workgroups empty (there are 512): twice the
// workgroups, each done with a tile of keys in 55 % of the time. 128 rows where they fill the card,
// since they load each key half as often. Measured, 64 against 128 rows: one prompt of 2048 tokens
// x 8 heads 38 and 54 us, x 24 heads 55 and 61, x 32 heads 72 and 66; 4096 x 12 91 and 106, x 16
// 120 and 117, x 32 234 and 209; six ragged prompts of up to 1000 tokens x 8 heads 31 and 33, x 16 49 and 45.
constexpr int64_t FEW_ROWS = 3 * 128 * 128;

template <int DT> hipError_t run_rows(const PrefillArgs &a, hipStream_t s) {
    return a.N * a.heads <= FEW_ROWS ? run<DT, Rows<2>>(a, s) : run<DT, Rows<1>>(a, s);
}

}  // namespace

hipError_t launch_prefill(const PrefillArgs &a, hipStream_t s) {
    return a.dt == DT_BF16 ? run_rows<DT_BF16>(a, s) : run_rows<DT_F16>(a, s);
}

}  // namespace ds4hc
