// latent_attn.hip -- attention over the paged latent cache, absorbed form.
//
// Per query row (a token and a head) and cached vector (c | r) of a sequence:
//   s = scale (ql . c + qr . r),  out = softmax(s) C,  with C the latents themselves.
// All rows of a sequence share its vectors, so a tile of cached tokens is loaded once,
// serves as keys and (read transposed) as values, and is used for as many rows as fit: with
// 128 heads 1088 * 2 operations a row against 1152 bytes a token, so that one token of 128
// heads stands where the card's rates of memory and of matrix products meet. A workgroup a CU
// takes 128 rows (32 a wave, their sums in its 256 accumulation registers) through tiles of 64
// tokens, two of them in LDS.
// This kernel with 1, 8, 16, 32 and 64 tiles a workgroup (one sequence, 128 heads): 30, 62, 97, 180
// and 409 us. That is 26 us beside the tiles (the batch's arrays, the page, the queries, the first
// tile's way to LDS; the part of the sums behind the last) and 4.4 a tile (4.3 TB/s), 5.2 and 7.2 where
// the cache is past 300 and 600 MB. Latent 256: 16 us and 2.8 a tile.
// Measured (latent 512, bf16, both kernels in a graph): 64 sequences of up to 8192 tokens x 128
// heads 140 us (106 and 26 us), one of 131000 tokens 82 us (59 and 20), 24 chains of 4 tokens
// over up to 4096 112 us (89 and 24), 512 tokens over 4096 556 us (985 TFLOP/s).
#include <type_traits>

#include "latent_device.hpp"

namespace ds4hc {

namespace {

constexpr int WORKGROUPS = 256;  // one a CU: the ring of tiles fills most of its LDS
constexpr int XCDS = 8;          // workgroup i runs on XCD i % 8
// tiles that a batch's queries and results cost as much as (0, 4, 8: 64 sequences of up to 8192 x 128
// heads 158, 143, 136 us; 24 chains over up to 4096 166, 110, 119; trees 89, 76, 78)
constexpr int EXTRA = 4;

// Tile shapes. ROWS query rows by TOKENS cached tokens; ROW_WAVES waves side by side in the
// rows, 32 each, times SETS sets of waves that take TOKENS / SETS of the tokens each, in
// steps of 32.
template <int LATENT_, int ROW_WAVES_, int SETS_> struct Shape {
    static constexpr int LATENT = LATENT_, ROW_WAVES = ROW_WAVES_, SETS = SETS_;
    static constexpr int TOKENS = 64, BUFS = 2, STEPS = TOKENS / SETS / 32;
    static constexpr int WAVES = ROW_WAVES * SETS, THREADS = WAVES * 64;
    static constexpr int D = LATENT + LATENT_ROPE;
    static constexpr int ROWS = ROW_WAVES * 32;
    static constexpr int ROW_BYTES = LATENT * 2;
    static constexpr int ROPE_AT = TOKENS * ROW_BYTES;
    static constexpr int TILE_BYTES = TOKENS * D * 2;
    static constexpr int ROWS_A_LOAD = 1024 / ROW_BYTES;
    static constexpr int LATENT_LOADS = TOKENS / ROWS_A_LOAD, ROPE_LOADS = TOKENS / 8;  // a tile
    static constexpr int KLATENT = LATENT / 16, KSTEPS = KLATENT + LATENT_ROPE / 16, DBLOCKS = LATENT / 32;
    static_assert(LATENT_LOADS % WAVES == 0 && ROPE_LOADS % WAVES == 0, "the waves load alike");
};

// Swizzle: 16-byte chunk c of token row r lies at chunk c ^ swz(r) of the row's place in
// LDS. swz takes all 16 values over 16 rows (a lane each reads the same chunk of 16 rows),
// and its upper 2 bits all 4 values over 4 rows (a transposing read takes 64 bytes of 4 rows
// at a time).
__device__ __forceinline__ int swz(int r) { return ((r & 3) << 2) | ((r >> 2) & 3); }
__device__ __forceinline__ int swz_rope(int r) { return (r >> 1) & 7; }

// ------------------------------------------------------------------ the split of the work
//
// `members` workgroups of one XCD form a cluster: they take the same cached tokens at the
// same time (one reads them from HBM, the others from the XCD's L2), each for a row tile of
// its own. The unit of the clusters' work is a tile of cached tokens against `members` row
// tiles; what a (sequence, batch of row tiles) costs besides its tiles (queries, results) is
// counted as `extra` units before them. Units are ordered by sequence, batch, tokens, and
// cluster c takes the units [c * share, (c + 1) * share). Lengths are read on the device, so a
// captured call follows them. A batch whose tiles lie in one cluster's range is written by it;
// of one that is cut each cluster writes its part of the sums to the workspace, and the second
// kernel joins the parts in order.
//
// Workspace: share, then where each cluster starts (for the second kernel), then a place for
// each part: sums in the order of the lanes that hold them ([row wave][LATENT / 8][64 lanes] of
// 4 elements, so that stores and loads are of whole lines), maxima, sums of the weights and of the
// rounded weights [ROWS].

struct Start {
    int b, batch, tile, pad;  // sequence (-1: the cluster has nothing to do), batch, first tile of its range
};
struct Header {
    int64_t share, pad;
    Start start[WORKGROUPS];
};

struct Seq {
    int q0, few, len;    // first token of the call, tokens of the call, cached tokens
    int row_tiles, kv_tiles;
    __device__ __forceinline__ int batches(int members) const { return (row_tiles + members - 1) / members; }
};

template <class S> __device__ __forceinline__ Seq sequence(const AttnArgs &a, int b) {
    Seq s;
    s.q0 = cu_at(a.c.cu_q, b, (int)a.N);
    s.few = max(cu_at(a.c.cu_q, b + 1, (int)a.N) - s.q0, 0);
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

template <class S> __host__ __device__ constexpr int64_t part_floats() { return (int64_t)S::ROWS * (S::LATENT + 3); }
template <class S> __device__ __forceinline__ float *part_at(const AttnArgs &a, int64_t cluster, int second, int member) {
    return reinterpret_cast<float *>(static_cast<Header *>(a.ws) + 1) + ((2 * cluster + second) * a.members + member) * part_floats<S>();
}

__device__ __forceinline__ int64_t wave_sum(int64_t v) {
    for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
    return v;
}

// Every wave finds by itself: the units in all, the share of a cluster and the extra units of a
// batch, and (b < 0 if there is none) the sequence that the cluster's first unit belongs to and
// its place there.
template <class S>
__device__ __forceinline__ int64_t find_unit(const AttnArgs &a, int64_t &share, int &extra, int64_t cluster, int &b_out, int64_t &off, Seq &at_b) {
    const int lane = threadIdx.x & 63, B = a.c.n_seqs, per = (B + 63) / 64;
    int64_t tiles = 0, batches = 0;
    Seq s{};
    for (int i = 0; i < per; ++i) {
        const int b = lane * per + i;
        if (b < B) {
            s = sequence<S>(a, b);
            batches += s.batches(a.members);
            tiles += (int64_t)s.batches(a.members) * s.kv_tiles;
        }
    }
    const int clusters = WORKGROUPS / a.members;
    extra = (int)min(wave_sum(tiles) / clusters / 4, (int64_t)EXTRA);  // (none where a share is a few tiles)
    const int64_t mine = tiles + batches * extra, upto = wave_prefix(mine, lane), total = __shfl(upto, 63);
    share = (total + clusters - 1) / clusters;
    if (share < 1) share = 1;
    const int64_t at = cluster * share;
    b_out = -1;
    if (at >= total) return total;
    const int who = __builtin_ctzll(__ballot(at >= upto - mine && at < upto));
    int64_t rest = at - __shfl(upto - mine, who);
    if (per == 1) {  // the lane's own sequence
        b_out = who;
        off = rest;
        auto of = [&](int v) { return __builtin_amdgcn_readlane(v, who); };
        at_b = {of(s.q0), of(s.few), of(s.len), of(s.row_tiles), of(s.kv_tiles)};
        return total;
    }
    for (int b = who * per; b < min(B, (who + 1) * per); ++b) {
        s = sequence<S>(a, b);
        const int64_t w = (int64_t)s.batches(a.members) * (s.kv_tiles + extra);
        if (rest < w) {
            b_out = b;
            off = rest;
            at_b = s;
            break;
        }
        rest -= w;
    }
    return total;
}

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
__global__ __launch_bounds__(S::THREADS, 1) void attn_kernel(AttnArgs a) {
    __shared__ __align__(256) char ring[S::BUFS * S::TILE_BYTES];
    __shared__ uint32_t not_finite[2];
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

        // ---- the lane's row: its query in registers
        const int row0 = row_tile * S::ROWS + row_wave * 32;
        const int tok = min(row0 + (lane & 31), n_rows - 1) / a.heads;  // rows behind the last repeat it
        u32x4_t q[S::KSTEPS];
        auto load_queries = [&]() {
            const int head = min(row0 + (lane & 31), n_rows - 1) - tok * a.heads;
            const elem_t<DT> *ql = static_cast<const elem_t<DT> *>(a.ql) + (int64_t)(q0 + tok) * a.ql_token + head * a.ql_head;
            const elem_t<DT> *qr = static_cast<const elem_t<DT> *>(a.qr) + (int64_t)(q0 + tok) * a.qr_token + head * a.qr_head;
#pragma unroll
            for (int k = 0; k < S::KSTEPS; ++k)
                q[k] = *reinterpret_cast<const u32x4_t *>((k < S::KLATENT ? ql + k * 16 : qr + (k - S::KLATENT) * 16) + (lane >> 5) * 8);
#pragma unroll
            for (int k = 0; k < S::KSTEPS; ++k) loaded(q[k]);
        };
        float top = -INFINITY, from = 0.f;  // running maximum less LIFT (what is subtracted: 0 if there is none)
        float sum = 0.f, used = 0.f;        // sums of the weights and of the rounded weights
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
        // A tile's loads. Tokens that are not there get the data of one that is (their places may
        // hold anything, also NaN, which a weight of 0 would not hide). Which tokens are there, a bit each:
        auto present = [&](int &rows) -> uint64_t {
            const uint64_t ok = __ballot(rows >= 0);
            const int one = __builtin_amdgcn_readlane(rows, __builtin_ctzll(ok | 1ull << 63));
            rows = rows >= 0 ? rows : one >= 0 ? one : 0;  // (none is there: row 0; nothing sees it)
            return ok;
        };
        // The wave's load number i of the tile; `from`: lane r's is the address of token r.
        constexpr int OWN_LATENT = S::LATENT_LOADS / S::WAVES, LOADS = OWN_LATENT + S::ROPE_LOADS / S::WAVES;
        constexpr int OWN_ROWS = S::TOKENS / S::WAVES;  // 16 or 32: swz of a row is that of its number in the wave
        static_assert(OWN_ROWS % 16 == 0, "the waves' rows swizzle alike");
        auto load = [&](int i, uint64_t from, uint32_t lane16, uint32_t buf, uint64_t lanes) {
            auto of_row = [&](int r) {
                return (uint64_t)(uint32_t)from_lane((int)(uint32_t)from, r) | (uint64_t)(uint32_t)from_lane((int)(from >> 32), r) << 32;
            };
            if (i < OWN_LATENT) {
                const int own = i * S::ROWS_A_LOAD, r0 = wave * OWN_ROWS + own;
                if constexpr (S::ROWS_A_LOAD == 1) {
                    const uint64_t at = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)from, r0) |
                                        (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(from >> 32), r0) << 32;
                    load_to_lds16((const char *)at, lane16 ^ (swz(own) << 4), buf + r0 * S::ROW_BYTES, lanes);
                } else {
                    constexpr int PER = 64 / S::ROWS_A_LOAD;  // lanes a row
                    const int r = r0 + lane16 / (16 * PER);
                    load_to_lds16((const char *)of_row(r) + ((lane16 & (16 * PER - 16)) ^ (swz(r) << 4)), buf + r0 * S::ROW_BYTES, lanes);
                }
            } else {
                const int r0 = (wave * (LOADS - OWN_LATENT) + i - OWN_LATENT) * 8, r = r0 + (lane16 >> 7);
                load_to_lds16((const char *)of_row(r) + S::ROW_BYTES + ((lane16 & 112) ^ (swz_rope(r) << 4)), buf + S::ROPE_AT + r0 * 128,
                              lanes);
            }
        };
        auto address = [&](int row) { return (uint64_t)cache + (uint64_t)(uint32_t)row * (S::D * 2); };
        auto load_all = [&](int rows, uint32_t buf) {
#pragma unroll
            for (int i = 0; i < LOADS; ++i) load(i, address(rows), lane_here() * 16, buf, ~0ull);
        };

        // Tile t (tokens `ok`) in LDS at `at`, and the loads of the next one, if there is one, beside it.
        auto tile = [&](int t, uint64_t ok, uint32_t at, int rows, uint32_t at_next) {
            DS4HC_LDS char *buf = (DS4HC_LDS char *)(uintptr_t)at;
            const int j0 = t * S::TOKENS;
            const bool masked = ok != ~0ull || j0 + S::TOKENS > (a.tree_mask ? context : context + 1);
            uint64_t bad = 0;  // tokens that hold a value that is not finite
            if (masked) {  // the same in all waves
                // Only what some rows see and others do not has to be looked at: the call's own tokens,
                // and the copies in place of tokens that are not there, if it is one of those they copy. (A
                // copy of a context token is seen, as that token, by all.) If none of the tile's tokens is
                // there, they copy the cache's first row, which may be nobody's and is seen by none.
                constexpr int CHUNKS = S::ROW_BYTES / 16;
                const int own = ok ? context - j0 : 0, copied = ok ? __builtin_ctzll(ok) : 0;
                const int lo = copied >= own ? 0 : own, hi = copied >= own ? S::TOKENS : min(S::TOKENS, sq.len - j0);
                if (threadIdx.x < 2) not_finite[threadIdx.x] = 0;
                wait_and_barrier<63>();
                for (int i = lo * CHUNKS + threadIdx.x; i < hi * CHUNKS; i += S::THREADS)
                    if (not_all_finite<DT>(lds_read16(buf + i * 16))) atomicOr(&not_finite[(i / CHUNKS) >> 5], 1u << ((i / CHUNKS) & 31));
                wait_and_barrier<63>();
                bad = ((uint64_t)uniform((int)not_finite[1]) << 32) | (uint32_t)uniform((int)not_finite[0]);
                if (bad) {  // zero in LDS, so that they meet no weight of 0; the rows that see them get NaN weights
                    for (int i = threadIdx.x; i < S::TOKENS * CHUNKS; i += S::THREADS)
                        if ((bad >> (i / CHUNKS)) & 1) {
                            const uint32_t zero = here(0);
                            *reinterpret_cast<DS4HC_LDS u32x4_t *>(buf + i * 16) = u32x4_t{zero, zero, zero, zero};
                        }
                    wait_and_barrier<63>();
                }
            }
            // LDS offsets of this lane's reads for the first k step, rope step and block of the
            // output; the others' chunks differ in higher bits, which an xor reaches. Made anew for
            // every tile: there are no registers to keep them.
            const int l = lane_here(), lr = l & 31, lh = l >> 5;
            const int t0 = set * S::STEPS * 32;  // first token of the wave
            const uint32_t k0 = (t0 + lr) * S::ROW_BYTES + ((lh ^ swz(lr)) << 4);
            const uint32_t r0 = S::ROPE_AT + (t0 + lr) * 128 + ((lh ^ swz_rope(lr)) << 4);
            const int vr = lh * 4 + ((l >> 2) & 3);
            const uint32_t v0 = (t0 + vr) * S::ROW_BYTES + (((((l >> 4) & 1) << 1 | ((l >> 1) & 1)) ^ swz(vr)) << 4) + (l & 1) * 8;
            const uint32_t v8 = (v0 ^ 32) + 8 * S::ROW_BYTES;  // 8 rows on, swz differs in bit 1

            // S^T = K Q^T of 32 tokens, the operands of the next products on their way; `between`
            // gives other work to the vector unit while the matrix unit is busy
            constexpr int AHEAD = 3;
            auto products_k = [&](int step, acc16_t &s, auto &&between) {
                // (steps in an order that uses one offset up before the next)
                auto nth = [](int i) { return i < S::KLATENT ? i % (S::KLATENT / 8) * 8 + i / (S::KLATENT / 8) : i; };
                auto read = [&](int i) {
                    const int k = nth(i);
                    return k < S::KLATENT ? lds_read16(buf + (k0 ^ ((k & 7) << 5)) + (k >> 3) * 256 + step * 32 * S::ROW_BYTES)
                                          : lds_read16(buf + (r0 ^ ((k - S::KLATENT) << 5)) + step * 32 * 128);
                };
                u32x4_t x[AHEAD];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) x[i] = read(i);
#pragma unroll
                for (int i = 0; i < S::KSTEPS; ++i) {
                    const u32x4_t now = x[i % AHEAD];
                    if (i == 0) mfma32_first_v<DT>(now, q[nth(i)], s);
                    else mfma32_v<DT>(now, q[nth(i)], s);
                    if (i + AHEAD < S::KSTEPS) x[i % AHEAD] = read(i + AHEAD);
                    between(i);
                    __builtin_amdgcn_sched_barrier(0);
                }
            };
            // O^T += V^T P^T of 32 tokens; the order of the tokens is that of S^T's rows, for both operands
            constexpr int VAHEAD = 4;
            auto products_v = [&](int step, const u32x4_t (&p)[2], auto &&between) {
                auto read = [&](int i) {  // block i / 2 in the order nth(), tokens 16 (i % 2) .. + 15
                    const int d = i / 2 % (S::DBLOCKS / 4) * 4 + i / 2 / (S::DBLOCKS / 4);
                    const uint32_t chunk = (d & 3) << 6, off = (d >> 2) * 256 + (step * 32 + (i & 1) * 16) * S::ROW_BYTES;
                    const u32x2_t lo = lds_read_tr(buf + (v0 ^ chunk) + off), hi = lds_read_tr(buf + (v8 ^ chunk) + off);
                    return u32x4_t{lo.x, lo.y, hi.x, hi.y};
                };
                u32x4_t v[VAHEAD];
#pragma unroll
                for (int i = 0; i < VAHEAD; ++i) v[i] = read(i);
#pragma unroll
                for (int i = 0; i < S::DBLOCKS * 2; ++i) {
                    const int d = i / 2 % (S::DBLOCKS / 4) * 4 + i / 2 / (S::DBLOCKS / 4);
                    acc[d] = mfma32<DT>(v[i % VAHEAD], p[i & 1], acc[d]);
                    if (i + VAHEAD < S::DBLOCKS * 2) v[i % VAHEAD] = read(i + VAHEAD);
                    between(i);
                    __builtin_amdgcn_sched_barrier(0);
                }
            };
            // Softmax of a step, in pieces. The mask, and the largest logit (of the lane's row).
            uint64_t sees = ~0ull;
            if (masked) sees = sees_of_tile(a, q0 + tok, tok, j0 - context) & ok;
            auto largest = [&](int step, acc16_t &s) {
                if (masked) {
                    const int at0 = t0 + step * 32 + (lane_here() >> 5) * 4;
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
                    for (int d = 0; d < S::DBLOCKS; ++d) {
                        pin_acc(acc[d]);
                        acc[d] *= keep;
                        pin_acc(acc[d]);
                    }
                }
                return keep;
            };
            // Weights 2 i and 2 i + 1, rounded to the type that the second product takes. (In two 16-bit
            // parts they would double that product, half of all, to take the error of an output from
            // 1.25 times that of float32 weights to 1.)
            auto weight2 = [&](const acc16_t &s, int i, u32x4_t (&p)[2]) {
                const float e0 = exp2_fast(fmaf(s[2 * i], scale2, -from)), e1 = exp2_fast(fmaf(s[2 * i + 1], scale2, -from));
                sum += e0;
                sum += e1;
                p[i >> 2][i & 3] = pack2<DT>(e0, e1);
                used = add2_words<DT>(p[i >> 2][i & 3], used);
            };
            // the next tile's loads, spread over the products (all but a second step's last): issued
            // faster than one in some 34 cycles a CU they hold the waves up
            constexpr int SLOTS = S::KSTEPS * S::STEPS + S::DBLOCKS * 2, LOAD_EVERY = SLOTS / LOADS;
            static_assert(LOAD_EVERY >= 1, "a place for each load");
            const uint64_t lanes = (uint64_t)uniform((int64_t)(t + 1 < t_first + n ? -1 : 0));
            const uint64_t from = address(rows);
            const uint32_t lane16 = lane_here() * 16;
            auto load_some = [&](int i) {
                if (i % LOAD_EVERY == 0 && i / LOAD_EVERY < LOADS) load(i / LOAD_EVERY, from, lane16, at_next, lanes);
            };
            acc16_t s;
            u32x4_t p[2];
            products_k(0, s, load_some);
            if constexpr (S::STEPS == 1) {
                mfma_results(s);
                const float high = largest(0, s);
                if (__any(too_high(high))) raise(high);
#pragma unroll
                for (int i = 0; i < 8; ++i) weight2(s, i, p);
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
                    if (i % EVERY == EVERY - 1 && i / EVERY < 8) weight2(s, i / EVERY, p);
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
                    if (i % EVERY == EVERY - 1) weight2(s1, i / EVERY, p1);
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
        load_all(rows, ring_at);
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
        float all = sum_halves(sum), all_used = sum_halves(used);
        // the blocks of the output that this wave finishes: all, or with two sets its half
        constexpr int BLOCKS = S::DBLOCKS / S::SETS, BLOCK_BYTES = 16 * 64 * 4;
        acc16_t fin[BLOCKS];
        if constexpr (S::SETS == 1) {
#pragma unroll
            for (int d = 0; d < BLOCKS; ++d) fin[d] = acc[d];
            wait_and_barrier<63>();  // the last tile has been read by all
        } else {
            // each set gives the other one's half through LDS, and all is brought to the common maximum
            static_assert(S::WAVES * (BLOCKS * BLOCK_BYTES + 384) <= S::BUFS * S::TILE_BYTES, "the halves and statistics");
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

// Joins the parts of the batches that were cut. Workgroup (c, member) stands at the border
// between clusters c and c + 1. If the border cuts a batch into P parts, its P - 1 borders share
// the work out among themselves, so that one long sequence keeps all workgroups busy, too. A
// piece of the work is C chunks of 8 elements for 32 rows: one wave's, or several waves' that take
// the parts in turn if there are more waves than pieces. Of tiles of 64 rows and more, where there
// are 8 pieces or more a workgroup, they are 8 chunks wide, so that a wave writes whole 128-byte lines
// of the output (of which several XCDs would write parts). With fewer pieces the parts are many, and
// more waves count; of fewer rows the output is small. Whole calls, 8 chunks and 1: 64 sequences of
// 128 heads 138 and 152 us, 24 chains of 4 tokens 112 and 123, 8 sequences of up to 500 42 and 52;
// one token of 128 heads over 131000 103 and 82; 64 sequences of 16 heads 86 and 84, one over 100
// tokens 23.7 and 22.2. (Two workgroups a border, 8 waves for 16, and 8 parts in flight for 4 changed
// nothing beyond 2 %.)
constexpr int JOIN_WAVES = 16;  // waves a workgroup

template <int DT, class S, int C>
__device__ __forceinline__ void join_pieces(const AttnArgs &a, int q0, int before, int borders, int rows, int row_tile, int member,
                                            float (*shared)[7][64]) {
    constexpr int ALL = S::LATENT / 8, CHUNKS = ALL / C;  // chunks, pieces a group of 32 rows
    const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
    const int parts = borders + 1, c0 = (int)blockIdx.x - before;  // first part: of cluster c0
    const int pieces = (rows + 31) / 32 * CHUNKS;
    const int mine = before < pieces ? (pieces - before - 1) / borders + 1 : 0;  // pieces before, before + borders, ...
    int waves = 1;  // a piece
    while (waves * 2 * mine <= JOIN_WAVES && waves * 2 <= parts) waves *= 2;
    const int sub = wave % waves, at_once = JOIN_WAVES / waves;
    const float *first = part_at<S>(a, c0, 1, member), *second = part_at<S>(a, c0 + 1, 0, member);
    const int64_t step = 2 * a.members * part_floats<S>();
    for (int k0 = 0; k0 < mine; k0 += at_once) {
        const int k = k0 + wave / waves;
        const bool real = k < mine;
        const int piece = real ? before + k * borders : 0, group = piece / CHUNKS, chunk = piece % CHUNKS * C;
        const int in = group * 32 + (lane & 31);
        float top = -INFINITY, total = 0.f, used = 0.f;
        acc4_t acc[C];
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] = acc4_t{0.f, 0.f, 0.f, 0.f};
        // brings what there is and a part to the larger maximum (-infinity: no logit that is a number; sums of 0, or NaN)
        auto factors = [&](float t, float &keep, float &add) {
            const float to = fmaxf(top, t);
            keep = to == -INFINITY ? 1.f : exp2_fast(top - to);
            add = to == -INFINITY ? 1.f : exp2_fast(t - to);
            top = to;
        };
        constexpr int AT_ONCE = C == 1 ? 4 : 2;  // parts whose loads are in flight together
        for (int i0 = sub; i0 < parts; i0 += AT_ONCE * waves) {
            float t[AT_ONCE], w[AT_ONCE], n[AT_ONCE];
            acc4_t v[AT_ONCE][C];
#pragma unroll
            for (int u = 0; u < AT_ONCE; ++u) {
                const int i = min(i0 + u * waves, parts - 1);
                const float *p = i == 0 ? first : second + (i - 1) * step;
                t[u] = p[S::ROWS * S::LATENT + in];
                w[u] = p[S::ROWS * (S::LATENT + 1) + in];
                n[u] = p[S::ROWS * (S::LATENT + 2) + in];
#pragma unroll
                for (int c = 0; c < C; ++c) v[u][c] = *reinterpret_cast<const acc4_t *>(p + ((group * ALL + chunk + c) * 64 + lane) * 4);
            }
#pragma unroll
            for (int u = 0; u < AT_ONCE; ++u)
                if (i0 + u * waves < parts) {
                    float keep, add;
                    factors(t[u], keep, add);
                    total = total * keep + w[u] * add;
                    used = used * keep + n[u] * add;
#pragma unroll
                    for (int c = 0; c < C; ++c) acc[c] = acc[c] * keep + v[u][c] * add;
                }
        }
        if (waves > 1) {  // (the same for all waves)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                __syncthreads();
                shared[wave][0][lane] = top;
                shared[wave][1][lane] = total;
                shared[wave][2][lane] = used;
                for (int e = 0; e < 4; ++e) shared[wave][3 + e][lane] = acc[c][e];
                __syncthreads();
                if (sub > 0) continue;
                // the maximum of all, then the sums (the first wave's statistics are its own until the last chunk)
                float to = top, sums = 0.f, sums_used = 0.f;
                for (int w = wave + 1; w < wave + waves; ++w) to = fmaxf(to, shared[w][0][lane]);
                acc4_t v = {0.f, 0.f, 0.f, 0.f};
                for (int w = wave; w < wave + waves; ++w) {
                    const float add = to == -INFINITY ? 1.f : exp2_fast(shared[w][0][lane] - to);
                    sums += shared[w][1][lane] * add;
                    sums_used += shared[w][2][lane] * add;
                    v += acc4_t{shared[w][3][lane], shared[w][4][lane], shared[w][5][lane], shared[w][6][lane]} * add;
                }
                acc[c] = v;
                if (c == C - 1) {
                    top = to;
                    total = sums;
                    used = sums_used;
                }
            }
        }
        if (sub == 0 && real && in < rows) {
            const int r = row_tile * S::ROWS + in, t = q0 + r / a.heads, h = r % a.heads;
            const float inv = used == 0.f ? 0.f : 1.f / used;
            elem_t<DT> *o = static_cast<elem_t<DT> *>(a.out) + (int64_t)t * a.out_token + h * a.out_head + chunk * 8 + (lane >> 5) * 4;
#pragma unroll
            for (int c = 0; c < C; ++c)
                *reinterpret_cast<u32x2_t *>(o + c * 8) = u32x2_t{pack2<DT>(acc[c][0] * inv, acc[c][1] * inv), pack2<DT>(acc[c][2] * inv, acc[c][3] * inv)};
            if (a.lse && chunk == 0 && lane < 32) a.lse[(int64_t)t * a.heads + h] = row_lse<DT>(top, total);
        }
    }
}

template <int DT, class S>
__global__ __launch_bounds__(JOIN_WAVES * 64) void attn_join_kernel(AttnArgs a) {
    __shared__ float shared[JOIN_WAVES][7][64];
    const Header *header = static_cast<const Header *>(a.ws);
    const int64_t share = uniform(header->share);
    const Start at = header->start[blockIdx.x + 1];
    if (at.b < 0 || at.tile == 0) return;  // no work behind the border, or it cuts nothing
    const Seq sq = sequence<S>(a, at.b);
    const int member = blockIdx.y, row_tile = at.batch * a.members + member;
    if (row_tile >= sq.row_tiles) return;
    // borders of this batch before this one, and behind it
    const int before = uniform((int)((at.tile - 1) / share)), behind = uniform((int)((sq.kv_tiles - at.tile - 1) / share));
    const int borders = before + behind + 1;
    const int rows = uniform(min(S::ROWS, sq.few * a.heads - row_tile * S::ROWS));
    if constexpr (S::ROWS >= 64)
        if ((rows + 31) / 32 * (S::LATENT / 64) >= 8 * borders) {
            join_pieces<DT, S, 8>(a, sq.q0, before, borders, rows, row_tile, member, shared);
            return;
        }
    join_pieces<DT, S, 1>(a, sq.q0, before, borders, rows, row_tile, member, shared);
}

// How a call is run. A tile has the rows that a sequence has on average, at most 128; sequences
// of several row tiles give them to a cluster of workgroups that load the same tokens. Measured
// (latent 512), tiles of 32, 64 and 128 rows: 64 sequences x 16 rows 90, 96, 111 us; x 64 rows 141,
// 110, 125; x 128 rows 230, 152, 139. Clusters of 1, 2 and 4 tiles of 128: 24 sequences x 512 rows
// 120, 110, 109 us; 8 x up to 640 79, 76, 75; 128 rows a sequence, one tile, 139, 170, 270; a chunk
// of 65536 rows 558, 554, 564. (One sequence of 128 rows alone is 5 % faster in two tiles of 64.)
// The average is all that the host knows. It serves unlike sequences badly: 64 of one token x 128
// heads take 150 us, a chunk of 512 tokens 556, both in one call 873, since each single token's
// row tile gets a cluster of four.
struct Plan {
    int rows, members;
};

Plan plan(const Paged &c, int heads, int64_t N) {
    const int64_t rows = (N * heads + c.n_seqs - 1) / c.n_seqs;
    if (rows <= 32) return {32, 1};
    if (rows <= 64) return {64, 1};
    return {128, rows <= 128 ? 1 : rows <= 256 ? 2 : 4};
}

template <int LATENT> using Rows32 = Shape<LATENT, 1, 2>;
template <int LATENT> using Rows64 = Shape<LATENT, 2, 2>;
template <int LATENT> using Rows128 = Shape<LATENT, 4, 1>;

template <int DT, class S> hipError_t run(const AttnArgs &a, hipStream_t s) {
    const hipError_t e = launch_kernel(attn_kernel<DT, S>, dim3(WORKGROUPS), dim3(S::THREADS), s, a);
    if (e != hipSuccess) return e;
    return launch_kernel(attn_join_kernel<DT, S>, dim3(WORKGROUPS / a.members - 1, a.members), dim3(JOIN_WAVES * 64), s, a);
}

template <int DT, int LATENT> hipError_t run_rows(const AttnArgs &a, int rows, hipStream_t s) {
    switch (rows) {
    case 32: return run<DT, Rows32<LATENT>>(a, s);
    case 64: return run<DT, Rows64<LATENT>>(a, s);
    default: return run<DT, Rows128<LATENT>>(a, s);
    }
}

template <int DT> hipError_t run_latent(const AttnArgs &a, int rows, hipStream_t s) {
    switch (a.latent) {
    case 128: return run_rows<DT, 128>(a, rows, s);
    case 256: return run_rows<DT, 256>(a, rows, s);
    default: return run_rows<DT, 512>(a, rows, s);
    }
}

}  // namespace

uint64_t attn_workspace_bytes(const Paged &c, int latent, int heads, int64_t N) {
    return sizeof(Header) + 2ull * WORKGROUPS * plan(c, heads, N).rows * (latent + 3) * sizeof(float);
}

hipError_t launch_attn(const AttnArgs &args, hipStream_t s) {
    AttnArgs a = args;
    const Plan p = plan(a.c, a.heads, a.N);
    a.members = p.members;
    return a.dt == DT_BF16 ? run_latent<DT_BF16>(a, p.rows, s) : run_latent<DT_F16>(a, p.rows, s);
}

}  // namespace ds4hc
