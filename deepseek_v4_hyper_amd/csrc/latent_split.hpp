// latent_split.hpp -- how attention over a paged latent cache is split over workgroups, and the
// joining of what is cut: shared by the kernels of the 16-bit (latent_attn.hip) and of the 8-bit
// cache (latent_attn8.hip). S is a kernel's tile shape: S::ROWS query rows by S::TOKENS tokens, S::LATENT, and
// S::EXTRA, the tiles that a batch's queries and results cost as much as, but at most 1 / S::EXTRA_OF of a share.
#pragma once

#include "latent_device.hpp"

namespace ds4hc {

namespace {

constexpr int WORKGROUPS = 256;  // one a CU: the ring of tiles fills most of its LDS
constexpr int XCDS = 8;          // workgroup i runs on XCD i % 8

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

// a / b, of which a hardly ever needs 64 bits (the same in all lanes).
__device__ __forceinline__ int64_t quotient(int64_t a, int b) {
    return (uint64_t)a >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

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
    const int clusters = WORKGROUPS / a.members, shift = __builtin_ctz(clusters);  // (a power of 2: 64-bit divisions take their time)
    extra = (int)min((wave_sum(tiles) >> shift) / S::EXTRA_OF, (int64_t)S::EXTRA);  // (none where a share is a few tiles)
    const int64_t mine = tiles + batches * extra, upto = wave_prefix(mine, lane), total = __shfl(upto, 63);
    share = (total + clusters - 1) >> shift;
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

}  // namespace

}  // namespace ds4hc
