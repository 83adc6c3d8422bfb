// draft_kernels.hip -- which drafted tokens are kept, and the token that follows them.
//
// Only one row of each distribution is summed over the vocabulary for a sequence, that of the last
// token kept: whether a token is accepted takes single elements. Everything is in 64 bits: the sums of
// a vocabulary's float32 weights decide between neighbours whose borders lie 1e-5 of the total apart and less,
// and one in a hundred of 32-bit sums would choose another.
#include "ds4hc.h"

#include "latent_device.hpp"
#include "serve_launch.hpp"

namespace ds4hc {

namespace {

constexpr int NODES = DS4HC_VERIFY_MAX_TOKENS;  // of a sequence
constexpr int WIDE = 256, WAVES = WIDE / 64, LAST = 1024;  // threads of a workgroup: of the sums, of the choice
constexpr int CHUNK_STEP = 1024, CHUNK_MOST = 16384;       // elements of a workgroup, a quarter of them a wave
constexpr int GOAL = 1024;   // workgroups that sum

// What the first kernel leaves for the second: of each sequence, then of each (sequence, wave's part of the row).
struct Reached {
    int node;    // last token kept, -1: the sequence has none
    int ends;    // its children have all been rejected, or (chain with draft) its child: weights are what is left
    int pad[2];
};
struct Sums {
    double left, all;  // of what is left of p, and of p
};

int chunks_of(int vocab, int chunk) { return (vocab + chunk - 1) / chunk; }
int chunk_of(int n_seqs, int vocab) {
    const int64_t each = ((int64_t)vocab * n_seqs + GOAL - 1) / GOAL;
    const int64_t chunk = (each + CHUNK_STEP - 1) / CHUNK_STEP * CHUNK_STEP;
    return (int)(chunk < CHUNK_STEP ? CHUNK_STEP : chunk > CHUNK_MOST ? CHUNK_MOST : chunk);
}

__device__ __forceinline__ Reached *reached_at(const VerifyArgs &a) { return static_cast<Reached *>(a.ws); }
__device__ __forceinline__ Sums *sums_at(const VerifyArgs &a) { return reinterpret_cast<Sums *>(reached_at(a) + a.n_seqs); }

// A weight: what is negative or not finite counts as 0.
__device__ __forceinline__ float weight(float p) { return p > 0.f && p < INFINITY ? p : 0.f; }
__device__ __forceinline__ double number(float u) { return u > 0.f ? (double)fminf(u, 0x1.fffffep-1f) : 0.0; }

__device__ __forceinline__ double wave_sum(double v) {
    for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
    return v;
}

// Marks of the rejected tokens among the elements [first, first + count) of a row, a bit each.
template <int THREADS>
__device__ __forceinline__ bool mark_rejected(const VerifyArgs &a, int t0, int few, int node, int first, int count, uint32_t *marks) {
    __shared__ int any;
    for (int i = threadIdx.x; i < (count + 31) / 32; i += THREADS) marks[i] = 0;
    if (threadIdx.x == 0) any = 0;
    __syncthreads();
    for (int i = node + 1 + (int)threadIdx.x; i < few; i += THREADS) {
        const int parent = a.parents ? a.parents[t0 + i] : i - 1;
        const int64_t x = a.tokens[t0 + i] - first;
        if (parent == node && x >= 0 && x < count) {
            atomicOr(&marks[x >> 5], 1u << (x & 31));
            any = 1;
        }
    }
    __syncthreads();
    return any != 0;
}

// One element of what is left of a row, after the root's distribution p and, of a chain with draft that ended
// early, less q.
__device__ __forceinline__ double left_of(float p, float q, bool less) {
    return less ? fmax((double)weight(p) - (double)weight(q), 0.0) : (double)weight(p);
}

// Grid (chunks, sequences). Every workgroup of a sequence finds its path by itself, from single elements
// of the rows, and sums its chunk of the row that the path ends at; the first one writes the path.
// 64 chains of up to 5 tokens over 100003: 12.0 us, 4.3 TB/s; of which some 4 are the chain of loads before the rows'
// (offsets, tokens, elements). Half of the loads in flight, and a sum a workgroup in place of one a wave: 16.3.
__global__ __launch_bounds__(WIDE) void verify_sums_kernel(VerifyArgs a) {
    __shared__ int parent[NODES], on_path[NODES];
    __shared__ float at_token[NODES], uniform_of[NODES];
    __shared__ int64_t token_of[NODES];
    __shared__ uint32_t marks[CHUNK_MOST / 32];
    __shared__ int shared_node, shared_kept;
    const int b = blockIdx.y, chunk = blockIdx.x, n = (int)a.N, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int t0 = cu_at(a.cu_q, b, n), all_tokens = max(cu_at(a.cu_q, b + 1, n) - t0, 0), few = min(all_tokens, NODES);
    if (few == 0) {
        if (chunk == 0 && threadIdx.x == 0) {
            a.n_kept[b] = 0;
            reached_at(a)[b] = {-1, 0, {0, 0}};
        }
        return;
    }
    // single elements: of each token, at the row of its parent. A chain with draft: whether it would be accepted.
    if (threadIdx.x == 0) {
        parent[0] = -1;
        on_path[0] = 0;
    }
    for (int i = 1 + threadIdx.x; i < few; i += WIDE) {
        int up = a.parents ? a.parents[t0 + i] : i - 1;
        if (up < 0 || up >= i) up = -1;
        const int64_t x = a.tokens[t0 + i];
        const bool inside = up >= 0 && x >= 0 && x < a.vocab;
        const float u = a.uniform[t0 + i], p = inside ? weight(a.target[(int64_t)(t0 + up) * a.target_stride + x]) : 0.f;
        parent[i] = up;
        token_of[i] = x;
        at_token[i] = p;
        uniform_of[i] = u;
        if (a.draft) {
            const float q = inside ? weight(a.draft[(int64_t)(t0 + up) * a.draft_stride + x]) : 0.f;
            on_path[i] = p > 0.f && number(u) * (double)q < (double)p;
        }
    }
    __syncthreads();
    if (wave == 0) {
        int node = 0, kept = 1;
        if (a.draft) {
            for (int i0 = 1; i0 < few; i0 += 64) {  // the first that is not accepted
                const int i = i0 + lane;
                const uint64_t no = __ballot(i >= few || !on_path[i < few ? i : 0]);
                if (no) {
                    node = i0 + __builtin_ctzll(no) - 1;
                    break;
                }
                node = i0 + 63;
            }
            kept = node + 1;
        } else {
            // level by level: the children of the node in their order, a lane each
            for (bool down = true; down;) {
                down = false;
                double mass = 1.0;
                int next = -1;
                for (int i0 = (node + 1) & ~63; i0 < few && next < 0; i0 += 64) {
                    const int i = i0 + lane;
                    uint64_t children = __ballot(i < few && i > node && parent[i < few ? i : 0] == node);
                    while (children) {
                        const int c = i0 + __builtin_ctzll(children);
                        children &= children - 1;
                        // (the same token among the children before it: tried already)
                        bool again = false;
                        for (int j0 = node + 1; j0 < c && !again; j0 += 64) {
                            const int j = j0 + lane;
                            again = __any(j < c && parent[j < c ? j : 0] == node && token_of[j < c ? j : c] == token_of[c]);
                        }
                        if (again) continue;
                        const double p = at_token[c];
                        if (p > 0.0 && number(uniform_of[c]) * mass < p) {
                            next = c;
                            break;
                        }
                        mass -= p;
                    }
                }
                if (next >= 0) {
                    node = next;
                    ++kept;
                    down = true;
                }
            }
        }
        if (lane == 0) {
            shared_node = node;
            shared_kept = kept;
        }
    }
    __syncthreads();
    const int node = shared_node, kept = shared_kept;
    const bool less = a.draft && node + 1 < few;
    if (chunk == 0) {
        // the path: of a chain 0 .. node, of a tree the ancestors, written from the end
        for (int i = threadIdx.x; i < all_tokens; i += WIDE)
            if (i >= kept) a.path[t0 + i] = -1;
            else if (a.draft) a.path[t0 + i] = i;
        if (threadIdx.x == 0) {
            if (!a.draft)
                for (int i = kept - 1, at = node; i >= 0; --i, at = parent[at]) a.path[t0 + i] = at;
            a.n_kept[b] = kept;
            reached_at(a)[b] = {node, less ? 1 : 0, {0, 0}};
        }
    }
    const int first = chunk * a.chunk, count = min(a.chunk, a.vocab - first);
    const bool marked = !a.draft && mark_rejected<WIDE>(a, t0, few, node, first, count, marks);
    const float *p = a.target + (int64_t)(t0 + node) * a.target_stride + first;
    const float *q = less ? a.draft + (int64_t)(t0 + node) * a.draft_stride + first : p;
    // a wave a quarter of the chunk, 8 loads of each row in flight
    const int part = a.chunk / WAVES, end = min((wave + 1) * part, count);
    double left = 0.0, all = 0.0;
    constexpr int AT_ONCE = 8;
    for (int i0 = wave * part + lane; i0 < end; i0 += 64 * AT_ONCE) {
        float w[AT_ONCE], v[AT_ONCE];
#pragma unroll
        for (int e = 0; e < AT_ONCE; ++e) {
            const int i = min(i0 + e * 64, end - 1);
            w[e] = p[i];
            v[e] = less ? q[i] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < AT_ONCE; ++e) {
            const int i = i0 + e * 64;
            if (i < end) {
                all += (double)weight(w[e]);
                left += marked && (marks[i >> 5] >> (i & 31)) & 1 ? 0.0 : left_of(w[e], v[e], less);
            }
        }
    }
    left = wave_sum(left);
    all = wave_sum(all);
    if (lane == 0) sums_at(a)[((int64_t)b * gridDim.x + chunk) * WAVES + wave] = {left, all};
}

// A workgroup a sequence: the part in which the sum passes the number, then the element. 5.4 us, a chain of latencies;
// with one thread's look at the sums, and four times the elements behind it, 9.8.
__global__ __launch_bounds__(LAST) void verify_choose_kernel(VerifyArgs a, int parts) {
    constexpr int PART_MOST = CHUNK_MOST / WAVES;
    __shared__ uint32_t marks[PART_MOST / 32];
    __shared__ double before[LAST / 64 + 1], goal, base;
    __shared__ int chosen, in_part, least, use_all;
    const int b = blockIdx.x, n = (int)a.N, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Reached r = reached_at(a)[b];
    if (r.node < 0) {
        if (threadIdx.x == 0) a.next[b] = -1;
        return;
    }
    const int t0 = cu_at(a.cu_q, b, n), few = min(cu_at(a.cu_q, b + 1, n) - t0, NODES);
    if (wave == 0) {
        const Sums *sums = sums_at(a) + (int64_t)b * parts;
        const float u = a.uniform[t0];
        // lane by lane, 64 parts at a time; `left` and `all` are the sums before them
        auto upto = [&](double v) {
            for (int m = 1; m < 64; m <<= 1) {
                const double o = __shfl_up(v, m);
                if (lane >= m) v += o;
            }
            return v;
        };
        double left = 0.0, all = 0.0;
        for (int c0 = 0; c0 < parts; c0 += 64) {
            const Sums s = c0 + lane < parts ? sums[c0 + lane] : Sums{0.0, 0.0};
            left += __shfl(upto(s.left), 63);
            all += __shfl(upto(s.all), 63);
        }
        const bool every = !(left > 0.0);
        const double to = number(u) * (every ? all : left);
        // the first part whose end is above the goal; if rounding leaves none, the last that has any weight
        int found = -1;
        double sum = 0.0, at = 0.0;
        for (int c0 = 0; c0 < parts; c0 += 64) {
            const Sums s = c0 + lane < parts ? sums[c0 + lane] : Sums{0.0, 0.0};
            const double v = every ? s.all : s.left, end = sum + upto(v);
            const uint64_t some = __ballot(v > 0.0), over = __ballot(v > 0.0 && end > to);
            if (some) {
                const int who = over ? __builtin_ctzll(over) : 63 - __builtin_clzll(some);
                found = c0 + who;
                at = __shfl(end, who) - __shfl(v, who);
            }
            if (over) break;
            sum = __shfl(end, 63);
        }
        if (lane == 0) {
            use_all = every;
            goal = to;
            in_part = found;
            base = at;
            chosen = INT_MAX;
            least = -1;
        }
    }
    __syncthreads();
    if (in_part < 0) {  // no weight at all
        if (threadIdx.x == 0) a.next[b] = -1;
        return;
    }
    const int part = a.chunk / WAVES, first = in_part / WAVES * a.chunk + in_part % WAVES * part, count = min(part, a.vocab - first);
    const bool less = r.ends && !use_all;
    const bool marked = !a.draft && !use_all && mark_rejected<LAST>(a, t0, few, r.node, first, count, marks);
    const float *p = a.target + (int64_t)(t0 + r.node) * a.target_stride + first;
    const float *q = less ? a.draft + (int64_t)(t0 + r.node) * a.draft_stride + first : p;
    // a thread some elements one behind another
    constexpr int MOST = PART_MOST / LAST;
    const int each = (part + LAST - 1) / LAST, i0 = threadIdx.x * each;
    double w[MOST], mine = 0.0;
#pragma unroll
    for (int e = 0; e < MOST; ++e) {
        const int i = i0 + e;
        w[e] = 0.0;
        if (e < each && i < count && !(marked && (marks[i >> 5] >> (i & 31)) & 1)) w[e] = left_of(p[i], less ? q[i] : 0.f, less);
        mine += w[e];
    }
    double upto = mine;  // inclusive, over the wave's lanes
    for (int m = 1; m < 64; m <<= 1) {
        const double o = __shfl_up(upto, m);
        if (lane >= m) upto += o;
    }
    if (lane == 63) before[wave + 1] = upto;
    __syncthreads();
    if (threadIdx.x == 0) {
        before[0] = base;
        for (int i = 1; i <= LAST / 64; ++i) before[i] += before[i - 1];
    }
    __syncthreads();
    double sum = before[wave] + (upto - mine);
    int hit = INT_MAX, last = -1;  // the first element of this thread with which the sum passes the goal, and its last with a weight
#pragma unroll
    for (int e = 0; e < MOST; ++e)
        if (w[e] > 0.0) {
            sum += w[e];
            last = i0 + e;
            if (sum > goal && hit == INT_MAX) hit = i0 + e;
        }
    const uint64_t hits = __ballot(hit != INT_MAX);
    if (hits && lane == __builtin_ctzll(hits)) atomicMin(&chosen, hit);
    __syncthreads();
    if (chosen == INT_MAX && last >= 0) atomicMax(&least, last);  // (rounding left none: the part's last)
    __syncthreads();
    if (threadIdx.x == 0) a.next[b] = first + (chosen != INT_MAX ? chosen : least);
}

}  // namespace

uint64_t verify_workspace_bytes(int n_seqs, int vocab) {
    return (uint64_t)n_seqs * (sizeof(Reached) + (uint64_t)chunks_of(vocab, chunk_of(n_seqs, vocab)) * WAVES * sizeof(Sums));
}

hipError_t launch_verify(const VerifyArgs &args, hipStream_t s) {
    VerifyArgs a = args;
    a.chunk = chunk_of(a.n_seqs, a.vocab);
    const int chunks = chunks_of(a.vocab, a.chunk);
    const hipError_t e = launch_kernel(verify_sums_kernel, dim3((unsigned)chunks, (unsigned)a.n_seqs), dim3(WIDE), s, a);
    if (e != hipSuccess) return e;
    return launch_kernel(verify_choose_kernel, dim3((unsigned)a.n_seqs), dim3(LAST), s, a, chunks * WAVES);
}

}  // namespace ds4hc
