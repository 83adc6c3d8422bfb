// latent_attn.hip -- attention over the paged latent cache, absorbed form.
#include "latent_device.hpp"

namespace ds4hc {

namespace {

constexpr int GROUPS = 256;      // workgroups: one a CU (a tile ring fills most of its LDS)
constexpr int JOIN_BLOCKS = 1 << 20;  // of the second kernel's grid in x (a dispatch has 2^32 threads a dimension)
constexpr int MIN_SHARE = 2;     // tiles a workgroup takes at least
constexpr float LN2 = 0.69314718055994530942f, LOG2E = 1.44269504088896340736f;
constexpr float LAZY = 8.f;      // the running maximum is raised only by more than this (in powers of 2)

// Tile shapes. ROWS query rows (a row is a token and a head; all rows of a sequence share
// its keys) by TOKENS cached tokens, four waves. With `split` every wave has all the rows
// and a quarter of the tokens, otherwise a quarter of the rows and all the tokens.
template <int LATENT_, int NB_, bool SPLIT_> struct Shape {
    static constexpr int LATENT = LATENT_, NB = NB_;  // NB: blocks of 16 rows a wave
    static constexpr bool SPLIT = SPLIT_;
    static constexpr int D = LATENT + LATENT_ROPE;
    static constexpr int ROWS = SPLIT ? NB * 16 : NB * 64;
    static constexpr int TOKENS = SPLIT ? 64 : 32;
    static constexpr int KVB = SPLIT ? 1 : 2;          // blocks of 16 tokens a wave
    static constexpr int BUFS = SPLIT ? 2 : 4;
    static constexpr int ROW_BYTES = LATENT * 2;
    static constexpr int ROPE_AT = TOKENS * ROW_BYTES;
    static constexpr int TILE_BYTES = TOKENS * D * 2;
    static constexpr int WAVE_TOKENS = TOKENS / 4;     // tokens a wave loads
    static constexpr int ROWS_A_LOAD = 1024 / ROW_BYTES;
    static constexpr int LOADS = WAVE_TOKENS / ROWS_A_LOAD + WAVE_TOKENS / 8;  // a tile and wave
    static constexpr int KSTEPS = LATENT / 32, DBLOCKS = LATENT / 16;
};

// Swizzle: 16-byte chunk c of token row r lies at chunk c ^ swz(r) of the row's place in
// LDS. swz takes all 16 values over 16 rows and its upper 3 bits all 8 values over 8 rows,
// so 16 lanes that read one chunk of 16 rows, and 32 lanes that read 32 bytes of 8 rows,
// touch every bank once.
__device__ __forceinline__ int swz(int r) { return ((r & 7) << 1) | ((r >> 3) & 1); }
__device__ __forceinline__ int swz_rope(int r) { return (r >> 1) & 7; }

// ------------------------------------------------------------------ the split of the work
//
// The unit of work is a tile: TOKENS cached tokens of a sequence against one tile of its
// rows. Units are ordered by sequence, row tile, tokens; workgroup w takes the units
// [w * share, (w + 1) * share). Lengths are read on the device, so a captured call follows
// them. A (sequence, row tile) that lies in one workgroup's range is written by it; of one
// that is cut every workgroup writes its part of the sums to the workspace, and the second
// kernel joins the parts in order.

struct Seq {
    int few, len;        // tokens of the call, cached tokens
    int row_tiles, kv_tiles;
};

template <class S> __device__ __forceinline__ Seq sequence(const AttnArgs &a, int b) {
    Seq s;
    const int q0 = cu_at(a.c.cu_q, b, (int)a.N);
    s.few = max(cu_at(a.c.cu_q, b + 1, (int)a.N) - q0, 0);
    s.len = kv_len_at(a.c, b);
    s.row_tiles = (int)(((int64_t)s.few * a.heads + S::ROWS - 1) / S::ROWS);
    s.kv_tiles = max((s.len + S::TOKENS - 1) / S::TOKENS, 1);  // no token: one empty tile, to write the zeros
    return s;
}

// Sums over lanes 0 .. l.
__device__ __forceinline__ int64_t wave_prefix(int64_t v, int lane) {
    for (int m = 1; m < 64; m <<= 1) {
        const int64_t o = __shfl_up(v, m);
        if (lane >= m) v += o;
    }
    return v;
}

// Every wave finds by itself: the units in all, and (if `at` >= 0 and below that) the
// sequence that unit `at` belongs to and the unit's place in it.
template <class S>
__device__ __forceinline__ int64_t find_unit(const AttnArgs &a, int64_t &share, int64_t group, int &b_out, int64_t &off) {
    const int lane = threadIdx.x & 63, B = a.c.n_seqs, per = (B + 63) / 64;
    int64_t mine = 0;
    for (int i = 0; i < per; ++i) {
        const int b = lane * per + i;
        if (b < B) {
            const Seq s = sequence<S>(a, b);
            mine += (int64_t)s.row_tiles * s.kv_tiles;
        }
    }
    const int64_t upto = wave_prefix(mine, lane), total = __shfl(upto, 63);
    share = (total + GROUPS - 1) / GROUPS;
    if (share < MIN_SHARE) share = MIN_SHARE;
    const int64_t at = group * share;
    b_out = -1;
    if (at >= total) return total;
    const uint64_t in = __ballot(at >= upto - mine && at < upto);
    const int who = __builtin_ctzll(in);
    int64_t rest = at - __shfl(upto - mine, who);
    for (int b = who * per; b < min(B, (who + 1) * per); ++b) {
        const Seq s = sequence<S>(a, b);
        const int64_t w = (int64_t)s.row_tiles * s.kv_tiles;
        if (rest < w) {
            b_out = b;
            off = rest;
            break;
        }
        rest -= w;
    }
    return total;
}

// Place of a part in the workspace: sums [ROWS][LATENT], then maximum and sum [ROWS] each.
template <class S> constexpr int64_t part_floats() { return (int64_t)S::ROWS * (S::LATENT + 2); }

// ------------------------------------------------------------------ tiles

// Tokens of a tile that a row's token sees, one bit each, whether or not they are in the
// cache. `at`: the first one's place among the call's own tokens (negative: the context).
__device__ __forceinline__ uint64_t sees_of_tile(const AttnArgs &a, int t, int i, int at) {
    if (!a.tree_mask) return at > i ? 0 : at + 63 <= i ? ~0ull : (2ull << (i - at)) - 1;
    const uint64_t *m = a.tree_mask + (int64_t)t * a.mask_words;
    auto word = [&](int w) { return w < 0 ? ~0ull : w < a.mask_words ? m[w] : 0ull; };
    const int shift = at & 63;
    const uint64_t lo = word(at >> 6);
    return shift ? (lo >> shift) | (word((at >> 6) + 1) << (64 - shift)) : lo;
}

template <int DT, class S>
__global__ __launch_bounds__(256, 1) void attn_kernel(AttnArgs a) {
    __shared__ __align__(16) char ring[S::BUFS * S::TILE_BYTES];
    __shared__ uint32_t not_finite[2];
    constexpr int NB = S::NB, KVB = S::KVB;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, grp = lane >> 4;
    // neighbours in the order of the work on one XCD (workgroups go round the 8 XCDs)
    const int group = (blockIdx.x & 7) * (GROUPS / 8) + (blockIdx.x >> 3);

    int64_t share, off;
    int b;
    const int64_t total = find_unit<S>(a, share, group, b, off);
    if (b < 0) return;
    b = uniform(b);
    off = uniform(off);
    int64_t left = uniform(min(share, total - group * share));
    const float scale2 = a.scale * LOG2E;
    const char *cache = static_cast<const char *>(a.cache);

    // LDS byte offsets of this lane's reads inside a tile, for the first k step, rope step and
    // block of the output; the others' chunks differ in higher bits, which an xor reaches
    const int row0_in_tile = S::SPLIT ? wave * 16 : 0;  // first token of the wave's blocks
    const uint32_t k_at = (row0_in_tile + col) * S::ROW_BYTES + ((grp ^ swz(col)) << 4);
    const uint32_t r_at = S::ROPE_AT + (row0_in_tile + col) * 128 + ((grp ^ swz_rope(col)) << 4);
    const int vr = grp * 4 + (col >> 2);
    const uint32_t v_at = (row0_in_tile + vr) * S::ROW_BYTES + ((((col >> 1) & 1) ^ swz(vr)) << 4) + (col & 1) * 8;

    bool first_part = true;
    while (left > 0) {
        Seq sq = sequence<S>(a, b);
        sq = {uniform(sq.few), uniform(sq.len), uniform(sq.row_tiles), uniform(sq.kv_tiles)};
        const int64_t units = (int64_t)sq.row_tiles * sq.kv_tiles;
        if (off >= units) {  // next sequence (the units in all bound b)
            ++b;
            off = 0;
            continue;
        }
        const int q0 = uniform(cu_at(a.c.cu_q, b, (int)a.N));
        const int row_tile = (int)(off / sq.kv_tiles), t_first = (int)(off - (int64_t)row_tile * sq.kv_tiles);
        const int n = (int)min((int64_t)(sq.kv_tiles - t_first), left);
        const int n_rows = sq.few * a.heads;  // the host keeps N * heads below 2^31
        const int context = sq.len - sq.few;

        // ---- rows: queries in registers
        int tok[NB];
        u32x4_t q[NB][S::KSTEPS + 2];
        for (int nb = 0; nb < NB; ++nb) {
            const int64_t r64 = (int64_t)row_tile * S::ROWS + (S::SPLIT ? 0 : wave * NB * 16) + nb * 16 + col;
            const int r = (int)min(r64, (int64_t)n_rows - 1);  // rows behind the last repeat it
            tok[nb] = r / a.heads;
            const int h = r - tok[nb] * a.heads;
            const elem_t<DT> *ql = static_cast<const elem_t<DT> *>(a.ql) + (int64_t)(q0 + tok[nb]) * a.ql_token + h * a.ql_head;
            const elem_t<DT> *qr = static_cast<const elem_t<DT> *>(a.qr) + (int64_t)(q0 + tok[nb]) * a.qr_token + h * a.qr_head;
            for (int k = 0; k < S::KSTEPS; ++k) q[nb][k] = *reinterpret_cast<const u32x4_t *>(ql + k * 32 + grp * 8);
            for (int k = 0; k < 2; ++k) q[nb][S::KSTEPS + k] = *reinterpret_cast<const u32x4_t *>(qr + k * 32 + grp * 8);
        }
        float top[NB], sum[NB];
        acc4_t acc[S::DBLOCKS][NB];
        for (int nb = 0; nb < NB; ++nb) {
            top[nb] = -INFINITY;
            sum[nb] = 0.f;
            for (int d = 0; d < S::DBLOCKS; ++d) {
                acc[d][nb] = acc4_t{0.f, 0.f, 0.f, 0.f};
                pin_acc(acc[d][nb]);
            }
        }

        // Cache rows of a tile's tokens, lane r that of token r (-1: not in the cache, or behind the end).
        auto look_up = [&](int tile) {
            const int r = lane & (S::TOKENS - 1), j = tile * S::TOKENS + r;
            if (a.c.page_shift < 4) {  // pages of less than 16 tokens: a lookup a lane
                int64_t at = -1;
                if (tile < t_first + n && j < sq.len) at = cache_row(a.c, b, j);
                return (int)at;
            }
            constexpr int PAGES = S::TOKENS / 16;
            int page = -1;
            for (int i = 0; i < PAGES; ++i) {
                const int first = tile * S::TOKENS + i * 16;
                if (tile >= t_first + n || first >= sq.len) break;
                const int pg = scalar_load(a.c.block_table, (int64_t)b * a.c.max_pages + (first >> a.c.page_shift));
                if ((r >> 4) == i) page = pg;
            }
            if (j >= sq.len || page < 0 || page >= a.c.n_pages) return -1;
            return (page << a.c.page_shift) + (j & ((1 << a.c.page_shift) - 1));
        };
        // Issues a tile's loads. Tokens that are not there get the data of one that is (their
        // places may hold anything, also NaN, which a weight of 0 would not hide).
        auto issue = [&](int t, int rows, uint32_t buf) {
            if (t >= t_first + n) return;
            const uint64_t ok = __ballot(rows >= 0);
            // (a tile with no token that is there: row 0, never looked at; the waits count on its loads)
            rows = rows >= 0 ? rows : ok ? __shfl(rows, __builtin_ctzll(ok | 1ull << 63)) : 0;
            const uint32_t here_lane = here(lane);
            for (int i = 0; i < S::WAVE_TOKENS / S::ROWS_A_LOAD; ++i) {
                const int r0 = wave * S::WAVE_TOKENS + i * S::ROWS_A_LOAD;
                if constexpr (S::ROWS_A_LOAD == 1) {
                    const int at = __builtin_amdgcn_readlane(rows, r0);
                    load_to_lds16(cache + (int64_t)at * (S::D * 2), (here_lane ^ swz(r0)) * 16, buf + r0 * S::ROW_BYTES);
                } else {
                    constexpr int PER = 64 / S::ROWS_A_LOAD;  // lanes a row
                    const int r = r0 + here_lane / PER, at = __shfl(rows, r);
                    load_to_lds16(cache + (int64_t)at * (S::D * 2) + ((here_lane & (PER - 1)) ^ swz(r)) * 16,
                                  buf + r0 * S::ROW_BYTES);
                }
            }
            for (int i = 0; i < S::WAVE_TOKENS / 8; ++i) {
                const int r0 = wave * S::WAVE_TOKENS + i * 8, r = r0 + (here_lane >> 3), at = __shfl(rows, r);
                load_to_lds16(cache + (int64_t)at * (S::D * 2) + S::ROW_BYTES + (((here_lane & 7) ^ swz_rope(r)) << 4),
                              buf + S::ROPE_AT + r0 * 128);
            }
        };

        auto tile = [&](int t, int rows, uint32_t at) {
            DS4HC_LDS char *buf = (DS4HC_LDS char *)(uintptr_t)at;
            const uint64_t ok = __ballot(rows >= 0);
            if (!ok) return;
            const int j0 = t * S::TOKENS;
            const bool masked = ok != ~0ull || j0 + S::TOKENS > (a.tree_mask ? context : context + 1);
            uint64_t bad = 0;  // tokens that hold a value that is not finite
            if (masked) {  // uniform over the workgroup
                if (threadIdx.x < 2) not_finite[threadIdx.x] = 0;
                wait_and_barrier<63>();
                constexpr int CHUNKS = S::ROW_BYTES / 16;
                for (int i = threadIdx.x; i < S::TOKENS * CHUNKS; i += 256) {
                    const u32x4_t w = lds_read16(buf + i * 16);
                    if (word_not_finite<DT>(w.x) || word_not_finite<DT>(w.y) || word_not_finite<DT>(w.z) || word_not_finite<DT>(w.w))
                        atomicOr(&not_finite[(i / CHUNKS) >> 5], 1u << ((i / CHUNKS) & 31));
                }
                wait_and_barrier<63>();
                bad = ((uint64_t)uniform((int)not_finite[1]) << 32) | (uint32_t)uniform((int)not_finite[0]);
            }
            // S^T = K Q^T
            acc4_t s[KVB * NB];
            constexpr int STEPS = S::KSTEPS + 2, AHEAD = NB == 2 ? 3 : 4;
            const uint32_t k0 = here(k_at), r0 = here(r_at);
            auto read_k = [&](int k, int kb) {
                return k < S::KSTEPS ? lds_read16(buf + (k0 ^ ((k & 3) << 6)) + (k >> 2) * 256 + kb * 16 * S::ROW_BYTES)
                                     : lds_read16(buf + (r0 ^ ((k - S::KSTEPS) << 6)) + kb * 16 * 128);
            };
            u32x4_t x[AHEAD][KVB];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
#pragma unroll
                for (int kb = 0; kb < KVB; ++kb) x[k][kb] = read_k(k, kb);
#pragma unroll
            for (int k = 0; k < STEPS; ++k) {
                u32x4_t now[KVB];
#pragma unroll
                for (int kb = 0; kb < KVB; ++kb) {
                    now[kb] = x[k % AHEAD][kb];
                    if (k + AHEAD < STEPS) x[k % AHEAD][kb] = read_k(k + AHEAD, kb);
                }
#pragma unroll
                for (int kb = 0; kb < KVB; ++kb)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        if (k == 0) s[kb * NB + nb] = mfma_k32_first_v<DT>(now[kb], q[nb][k]);
                        else mfma_k32_v<DT>(now[kb], q[nb][k], s[kb * NB + nb]);
                    }
                __builtin_amdgcn_sched_barrier(0);
            }
            mfma_results(s);
            if (bad) {
                // values that are not finite: zero in LDS, so that they meet no weight of 0; the rows that see them get NaN weights
                wait_and_barrier<63>();
                constexpr int CHUNKS = S::ROW_BYTES / 16;
                for (int i = threadIdx.x; i < S::TOKENS * CHUNKS; i += 256) {
                    const int r = i / CHUNKS;
                    if ((bad >> r) & 1) *reinterpret_cast<DS4HC_LDS u32x4_t *>(buf + i * 16) = u32x4_t{0, 0, 0, 0};
                }
                wait_and_barrier<63>();
            }
            u32x2_t p[KVB][NB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                float x[KVB][4], high = -INFINITY;
                uint64_t sees = ~0ull, nan = 0;
                if (masked) {
                    sees = sees_of_tile(a, q0 + tok[nb], tok[nb], j0 - context) & ok;
                    nan = sees & bad;
                }
#pragma unroll
                for (int kb = 0; kb < KVB; ++kb)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[kb][i] = s[kb * NB + nb][i] * scale2;
                        if (masked) {
                            const int r = row0_in_tile + kb * 16 + grp * 4 + i;
                            x[kb][i] = (nan >> r) & 1 ? NAN : (sees >> r) & 1 ? x[kb][i] : -INFINITY;
                        }
                        high = fmaxf(high, x[kb][i]);
                    }
                high = max_over_groups(high);
                if (__any(high > top[nb] + LAZY)) {
                    const float to = fmaxf(top[nb], high);
                    const float keep = to == -INFINITY ? 0.f : exp2_fast(top[nb] - to);
                    top[nb] = to;
                    sum[nb] *= keep;
#pragma unroll
                    for (int d = 0; d < S::DBLOCKS; ++d) {
                        pin_acc(acc[d][nb]);
                        acc[d][nb] *= keep;
                        pin_acc(acc[d][nb]);
                    }
                }
                const float from = top[nb] == -INFINITY ? 0.f : top[nb];
#pragma unroll
                for (int kb = 0; kb < KVB; ++kb) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[kb][i] = exp2_fast(x[kb][i] - from);
                        sum[nb] += x[kb][i];
                    }
                    p[kb][nb] = u32x2_t{pack2<DT>(x[kb][0], x[kb][1]), pack2<DT>(x[kb][2], x[kb][3])};
                }
            }
            // O^T += V^T P^T; the order of the tokens in a step is that of S^T's rows, for both operands
            constexpr int VAHEAD = 8;
            const uint32_t v0 = here(v_at);
            auto read_v = [&](int d, int kb) { return lds_read_tr(buf + (v0 ^ ((d & 7) << 5)) + (d >> 3) * 256 + kb * 16 * S::ROW_BYTES); };
            u32x2_t v[VAHEAD][KVB];
#pragma unroll
            for (int d = 0; d < VAHEAD; ++d)
#pragma unroll
                for (int kb = 0; kb < KVB; ++kb) v[d][kb] = read_v(d, kb);
#pragma unroll
            for (int d = 0; d < S::DBLOCKS; ++d) {
                u32x2_t now[KVB];
#pragma unroll
                for (int kb = 0; kb < KVB; ++kb) {
                    now[kb] = v[d % VAHEAD][kb];
                    if (d + VAHEAD < S::DBLOCKS) v[d % VAHEAD][kb] = read_v(d + VAHEAD, kb);
                }
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    if constexpr (KVB == 2)
                        acc[d][nb] = mfma_k32<DT>(u32x4_t{now[0].x, now[0].y, now[KVB - 1].x, now[KVB - 1].y},
                                                  u32x4_t{p[0][nb].x, p[0][nb].y, p[KVB - 1][nb].x, p[KVB - 1][nb].y}, acc[d][nb]);
                    else
                        acc[d][nb] = mfma_k16<DT>(now[0], p[0][nb], acc[d][nb]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        };

        // ---- tiles: BUFS - 1 in flight. All waves are done with tile t - 1 when they meet at
        // the barrier of tile t, so its buffer takes tile t - 1 + BUFS.
        wait_and_barrier<0>();  // the last part's reads of the ring
        const uint32_t ring_at = lds_address(ring);
        int ahead[S::BUFS - 1];  // cache rows of the tiles in flight
#pragma unroll
        for (int i = 0; i < S::BUFS - 1; ++i) {
            ahead[i] = look_up(t_first + i);
            issue(t_first + i, ahead[i], ring_at + i * S::TILE_BYTES);
        }
        uint32_t buf = ring_at, free_buf = ring_at + (S::BUFS - 1) * S::TILE_BYTES;
        int next = look_up(t_first + S::BUFS - 1);
        for (int i = 0; i < n; ++i) {
            // loads of the tiles behind this one stay in flight
            if (S::BUFS > 2 && i + 2 < n) wait_and_barrier<2 * S::LOADS>();
            else if (S::BUFS > 2 && i + 1 < n) wait_and_barrier<S::LOADS>();
            else wait_and_barrier<0>();
            issue(t_first + i + S::BUFS - 1, next, free_buf);
            const int rows = ahead[0];
#pragma unroll
            for (int k = 0; k + 1 < S::BUFS - 1; ++k) ahead[k] = ahead[k + 1];
            ahead[S::BUFS - 2] = next;
            next = look_up(t_first + i + S::BUFS);
            tile(t_first + i, rows, buf);
            free_buf = buf;
            buf = buf + S::TILE_BYTES == ring_at + S::BUFS * S::TILE_BYTES ? ring_at : buf + S::TILE_BYTES;
        }

        // ---- the part's result
#pragma unroll
        for (int d = 0; d < S::DBLOCKS; ++d)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) pin_acc(acc[d][nb]);
        const bool whole = t_first == 0 && n == sq.kv_tiles;
        float *part = static_cast<float *>(a.ws) + (2 * (int64_t)group + (first_part && t_first > 0 ? 0 : 1)) * part_floats<S>();
        auto row_of = [&](int nb) { return row_tile * (int64_t)S::ROWS + (S::SPLIT ? 0 : wave * NB * 16) + nb * 16 + col; };
        // where the lane's row goes, and its statistics
        auto out_at = [&](int nb) {
            const int h = (int)row_of(nb) - tok[nb] * a.heads;
            return static_cast<elem_t<DT> *>(a.out) + (int64_t)(q0 + tok[nb]) * a.out_token + h * a.out_head;
        };
        auto part_at = [&](int nb) { return part + (row_of(nb) - row_tile * (int64_t)S::ROWS) * S::LATENT; };
        auto put_sums = [&](int nb, float t, float total_sum) {
            const int64_t r = row_of(nb);
            if (r >= n_rows) return;
            if (whole) {
                if (a.lse) a.lse[(int64_t)q0 * a.heads + r] = total_sum == 0.f ? -INFINITY : (t + __log2f(total_sum)) * LN2;
            } else {
                const int64_t in = r - row_tile * (int64_t)S::ROWS;
                part[S::ROWS * S::LATENT + in] = t;
                part[S::ROWS * (S::LATENT + 1) + in] = total_sum;
            }
        };
        // four elements of a row, as they are or divided by the sum
        auto put4 = [&](elem_t<DT> *o, acc4_t v, float inv) {
            *reinterpret_cast<u32x2_t *>(o) = u32x2_t{pack2<DT>(v[0] * inv, v[1] * inv), pack2<DT>(v[2] * inv, v[3] * inv)};
        };
        if constexpr (!S::SPLIT) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const float all = sum_over_groups(sum[nb]);
                if (grp == 0) put_sums(nb, top[nb], all);
                if (row_of(nb) < n_rows) {
                    if (whole) {
                        elem_t<DT> *o = out_at(nb) + grp * 4;
                        const float inv = all == 0.f ? 0.f : 1.f / all;
#pragma unroll
                        for (int d = 0; d < S::DBLOCKS; ++d) put4(o + d * 16, acc[d][nb], inv);
                    } else {
                        float *o = part_at(nb) + grp * 4;
#pragma unroll
                        for (int d = 0; d < S::DBLOCKS; ++d) *reinterpret_cast<acc4_t *>(o + d * 16) = acc[d][nb];
                    }
                }
            }
        } else {
            // the four waves' tokens: common maximum and sums through LDS, 16 rows at a time
            constexpr int HALF = 16 * S::LATENT * 4;  // a wave's sums of 16 rows
            static_assert(4 * HALF + 512 <= S::BUFS * S::TILE_BYTES, "four waves' sums and statistics");
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const float all = sum_over_groups(sum[nb]);
                float *st = reinterpret_cast<float *>(ring + 4 * HALF);  // [2][4][16]
                wait_and_barrier<0>();
                if (grp == 0) {
                    st[wave * 16 + col] = top[nb];
                    st[64 + wave * 16 + col] = all;
                }
                wait_and_barrier<0>();
                float to = -INFINITY;  // stays so where no logit is a number above it: sums are then 0 or NaN
                for (int w = 0; w < 4; ++w) to = fmaxf(to, st[w * 16 + col]);
                float total_sum = 0.f;
                for (int w = 0; w < 4; ++w)
                    total_sum += st[64 + w * 16 + col] * (to == -INFINITY ? 1.f : exp2_fast(st[w * 16 + col] - to));
                const float keep = to == -INFINITY ? 1.f : exp2_fast(top[nb] - to);
                char *mine = ring + wave * HALF;
#pragma unroll
                for (int d = 0; d < S::DBLOCKS; ++d)
                    *reinterpret_cast<acc4_t *>(mine + ((d * 4 + grp) * 16 + col) * 16) = acc[d][nb] * keep;
                wait_and_barrier<0>();
                if (wave == 0 && grp == 0) put_sums(nb, to, total_sum);
#pragma unroll
                for (int d = 0; d < S::DBLOCKS / 4; ++d) {
                    const int db = wave * (S::DBLOCKS / 4) + d, at = ((db * 4 + grp) * 16 + col) * 16;
                    acc4_t v = *reinterpret_cast<const acc4_t *>(ring + at);
#pragma unroll
                    for (int w = 1; w < 4; ++w) v += *reinterpret_cast<const acc4_t *>(ring + w * HALF + at);
                    if (row_of(nb) >= n_rows) continue;
                    if (whole) put4(out_at(nb) + db * 16 + grp * 4, v, total_sum == 0.f ? 0.f : 1.f / total_sum);
                    else *reinterpret_cast<acc4_t *>(part_at(nb) + db * 16 + grp * 4) = v;
                }
            }
        }
        first_part = false;
        left -= n;
        off += n;
    }
}

// Joins the parts of the row tiles that were cut: a wave a row.
template <int DT, class S>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t item = ((int64_t)blockIdx.y * JOIN_BLOCKS + blockIdx.x) * 4 + (threadIdx.x >> 6);  // token * heads + head
    if (item >= a.N * a.heads) return;
    const int t = (int)(item / a.heads), h = (int)(item - (int64_t)t * a.heads);
    const int B = a.c.n_seqs, per = (B + 63) / 64;
    const int b_of = sequence_of(a.c.cu_q, B, (int)a.N, t);
    if (b_of < 0) return;
    // units before this sequence, and in all
    int64_t mine = 0, before = 0;
    for (int i = 0; i < per; ++i) {
        const int b = lane * per + i;
        if (b < B) {
            const Seq s = sequence<S>(a, b);
            const int64_t w = (int64_t)s.row_tiles * s.kv_tiles;
            mine += w;
            if (b < b_of) before += w;
        }
    }
    for (int m = 32; m; m >>= 1) {
        mine += __shfl_xor(mine, m);
        before += __shfl_xor(before, m);
    }
    int64_t share = (mine + GROUPS - 1) / GROUPS;
    if (share < MIN_SHARE) share = MIN_SHARE;
    const Seq sq = sequence<S>(a, b_of);
    const int q0 = cu_at(a.c.cu_q, b_of, (int)a.N);
    const int64_t r = (int64_t)(t - q0) * a.heads + h;
    const int row_tile = (int)(r / S::ROWS), in = (int)(r - (int64_t)row_tile * S::ROWS);
    const int64_t u0 = before + (int64_t)row_tile * sq.kv_tiles, u1 = u0 + sq.kv_tiles;
    const int64_t g0 = u0 / share, g1 = (u1 - 1) / share;
    if (g0 == g1) return;  // written whole
    const float *ws = static_cast<const float *>(a.ws);
    auto part = [&](int64_t g) { return ws + (2 * g + (g == g0 ? 1 : 0)) * part_floats<S>(); };
    float to = -INFINITY;
    for (int64_t g = g0; g <= g1; ++g) to = fmaxf(to, part(g)[S::ROWS * S::LATENT + in]);
    constexpr int E = S::LATENT / 64;
    float acc[E], total = 0.f;
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int64_t g = g0; g <= g1; ++g) {
        const float *p = part(g);
        const float keep = to == -INFINITY ? 1.f : exp2_fast(p[S::ROWS * S::LATENT + in] - to);  // (1: sums of 0, or NaN)
        total += keep * p[S::ROWS * (S::LATENT + 1) + in];
        for (int e = 0; e < E; ++e) acc[e] += keep * p[(int64_t)in * S::LATENT + lane * E + e];
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    elem_t<DT> *o = static_cast<elem_t<DT> *>(a.out) + (int64_t)t * a.out_token + h * a.out_head + lane * E;
    for (int e = 0; e < E; ++e) o[e] = elem_round<DT>(acc[e] * inv);
    if (a.lse && lane == 0) a.lse[item] = total == 0.f ? -INFINITY : (to + __log2f(total)) * LN2;
}

template <int DT, class S> hipError_t run(const AttnArgs &a, hipStream_t s) {
    const hipError_t e = launch_kernel(attn_kernel<DT, S>, dim3(GROUPS), dim3(256), s, a);
    if (e != hipSuccess) return e;
    const unsigned blocks = (unsigned)((a.N * a.heads + 3) / 4);
    const dim3 grid(blocks < JOIN_BLOCKS ? blocks : JOIN_BLOCKS, (blocks + JOIN_BLOCKS - 1) / JOIN_BLOCKS);
    return launch_kernel(attn_join_kernel<DT, S>, grid, dim3(256), s, a);
}

// Rows of a tile: the rows a sequence has on average.
int tile_rows(const Paged &c, int heads, int64_t N) {
    const int64_t rows = (N * heads + c.n_seqs - 1) / c.n_seqs;
    return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
}

template <int DT, int LATENT> hipError_t run_rows(const AttnArgs &a, hipStream_t s) {
    switch (tile_rows(a.c, a.heads, a.N)) {
    case 16: return run<DT, Shape<LATENT, 1, true>>(a, s);
    case 32: return run<DT, Shape<LATENT, 2, true>>(a, s);
    case 64: return run<DT, Shape<LATENT, 1, false>>(a, s);
    default: return run<DT, Shape<LATENT, 2, false>>(a, s);
    }
}

template <int DT> hipError_t run_latent(const AttnArgs &a, hipStream_t s) {
    switch (a.latent) {
    case 128: return run_rows<DT, 128>(a, s);
    case 256: return run_rows<DT, 256>(a, s);
    default: return run_rows<DT, 512>(a, s);
    }
}

}  // namespace

uint64_t attn_workspace_bytes(const Paged &c, int latent, int heads, int64_t N) {
    return 2ull * GROUPS * tile_rows(c, heads, N) * (latent + 2) * sizeof(float);
}

hipError_t launch_attn(const AttnArgs &a, hipStream_t s) {
    return a.dt == DT_BF16 ? run_latent<DT_BF16>(a, s) : run_latent<DT_F16>(a, s);
}

}  // namespace ds4hc
