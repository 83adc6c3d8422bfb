// page_kernels.hip -- pages of paged caches: who has which (taking, sharing and giving back), and the
// moves of whole pages and of single rows.
#include "ds4hc.h"

#include "latent_device.hpp"
#include "serve_launch.hpp"

namespace ds4hc {

namespace {

// ------------------------------------------------------------------ rows and pages

constexpr int THREADS = 256;
constexpr int AT_ONCE = 8;  // rows in flight

// A thread takes the same 16 bytes of every row of a sequence, in one layer, and moves them in the order of
// the kept tokens: `keep` rises and entries that do not lie behind their targets are passed over, so what it reads was
// written by none of its own earlier moves, and nobody else touches its bytes. AT_ONCE loads are
// issued before their stores. Grid (layers x columns, sequences). 64 sequences, up to 8 rows of 656 bytes in 43 layers:
// 5.0 us, 3.3 TB/s; one sequence and layer 2.6 us.
__global__ __launch_bounds__(THREADS) void compact_kernel(CompactArgs a) {
    __shared__ int from[64], to[64];
    const int b = blockIdx.y, n = (int)a.N;
    const int t0 = cu_at(a.cu_q, b, n), few = max(cu_at(a.cu_q, b + 1, n) - t0, 0), kept = min(a.n_keep[b], few);
    const Paged view = {a.s.page_shift, a.n_seqs, a.max_pages, a.s.n_pages, a.cu_q, a.kv_len, a.block_table};
    const int base = kv_len_at(view, b) - few, most = a.max_pages << a.s.page_shift;
    const int columns = (int)(a.s.row_bytes / 16), at = blockIdx.x * THREADS + threadIdx.x, layer = at / columns;
    const bool real = layer < a.s.layers;
    char *data = a.s.data + (real ? layer : 0) * a.s.layer_stride + (int64_t)(at - layer * columns) * 16;
    auto place = [&](int i) { return base + i < 0 || base + i >= most ? -1 : (int)cache_row(view, b, base + i); };
    for (int i0 = 0; i0 < kept; i0 += 64) {
        __syncthreads();
        if (threadIdx.x < 64) {
            const int i = i0 + threadIdx.x;
            int source = -1, target = -1;
            if (i < kept) {
                const int k = a.keep[t0 + i];
                if (k > i && k < few) {
                    source = place(k);
                    target = place(i);
                }
            }
            from[threadIdx.x] = target < 0 ? -1 : source;
            to[threadIdx.x] = target;
        }
        __syncthreads();
        if (!real) continue;
        for (int i = 0; i < min(64, kept - i0); i += AT_ONCE) {
            u32x4_t v[AT_ONCE];
#pragma unroll
            for (int e = 0; e < AT_ONCE; ++e)
                if (from[i + e] >= 0) v[e] = *reinterpret_cast<const u32x4_t *>(data + (int64_t)from[i + e] * a.s.row_bytes);
#pragma unroll
            for (int e = 0; e < AT_ONCE; ++e)
                if (from[i + e] >= 0) *reinterpret_cast<u32x4_t *>(data + (int64_t)to[i + e] * a.s.row_bytes) = v[e];
        }
    }
}

// Grid (pieces of a page, layers, pairs); a workgroup a piece of COPY bytes. 64 pages of 42 KB in 43 layers: 36 us, 6.4 TB/s
// (part of what is read is still in the last cache).
constexpr int COPY = THREADS * 16 * 4;
__global__ __launch_bounds__(THREADS) void copy_kernel(Store s, int n, const int32_t *pairs) {
    const int64_t page_bytes = s.row_bytes << s.page_shift;
    for (int i = blockIdx.z; i < n; i += gridDim.z) {
        const int from = pairs[2 * i], to = pairs[2 * i + 1];
        if (from < 0 || from >= s.n_pages || to < 0 || to >= s.n_pages || from == to) continue;
        char *data = s.data + blockIdx.y * s.layer_stride;
        for (int64_t at = (int64_t)blockIdx.x * COPY + threadIdx.x * 16; at < page_bytes; at += (int64_t)gridDim.x * COPY) {
            u32x4_t v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (at + e * THREADS * 16 < page_bytes) v[e] = *reinterpret_cast<const u32x4_t *>(data + from * page_bytes + at + e * THREADS * 16);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (at + e * THREADS * 16 < page_bytes) *reinterpret_cast<u32x4_t *>(data + to * page_bytes + at + e * THREADS * 16) = v[e];
        }
    }
}

// ------------------------------------------------------------------ the pool

// Two kernels: the first, one workgroup, finds what each item needs and the free pages in ascending order; the
// second writes tables and counts, all items side by side. Counts change by whole-number atomics alone, in the
// second kernel, so that results do not depend on an order. 64 slots with up to 128 pages each, of 65536: 12.0 and
// 4.0 us where pages are taken, 3.5 and 3.1 where none are: chains of latencies, and the counts, which one workgroup reads from the
// first page on until it has found as many free ones as are needed (a call that takes one behind 2^14 used pages 12 us, 2^16 26,
// 2^18 81, 2^20 318; none 4.9 whatever the pool). (Both in one kernel, a wave an item: 16 slots with 16 pages 7.2 for 8.4 us, 64 with 16
// 11.3 for 9.1, 256 with 128 37 for 14.)
constexpr int DECIDE = 1024, WAVES = DECIDE / 64;
constexpr int SCAN = 16;  // pages a lane: 1024 a wave, 16384 a step of the workgroup

struct Item {
    int had, has;  // pages before and after; has -1: DS4HC_PAGES_INVALID (fork: has is the pages to share)
    int first;     // its first page's number among those that are taken
    int own;       // it gets its last page anew
};

// Workspace: free pages found, [n] items, [n_slots] the first item of a slot, free pages in ascending order.
struct Space {
    int *found;
    Item *items;
    int *owner, *free;
};
__device__ __forceinline__ Space space(const PoolArgs &a) {
    char *p = static_cast<char *>(a.ws);
    Item *items = reinterpret_cast<Item *>(p + 16);
    int *owner = reinterpret_cast<int *>(items + a.n);
    return {reinterpret_cast<int *>(p), items, owner, owner + a.n_slots};
}

// Loads that see other threads' atomics of this kernel.
__device__ __forceinline__ int load_fresh(const int *p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// Sum over threads before this one, and over all.
__device__ __forceinline__ int64_t block_prefix(int64_t v, int64_t *shared, int64_t &total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t upto = v;
    for (int m = 1; m < 64; m <<= 1) {
        const int64_t o = __shfl_up(upto, m);
        if (lane >= m) upto += o;
    }
    __syncthreads();
    if (lane == 63) shared[wave] = upto;
    __syncthreads();
    int64_t before = 0;
    total = 0;
    for (int w = 0; w < WAVES; ++w) {
        if (w < wave) before += shared[w];
        total += shared[w];
    }
    return before + upto - v;
}

// Whether item i is the first that names slot `s`. Of up to DECIDE items the slots stand in a table in LDS, each at the first
// free place from its hash on; of more each slot's first item in the workspace. (Through the workspace a call waits for
// three round trips more.)
constexpr int PLACES = 2 * DECIDE;
struct First {
    int slot[PLACES], item[PLACES];
};
__device__ __forceinline__ int place_of(int s) { return (int)((uint32_t)s * 2654435769u >> 21); }
static_assert(PLACES == 1 << 11, "the hash's bits");

__device__ __forceinline__ void find_firsts(const PoolArgs &a, int *owner, First &f) {
    if (a.n <= DECIDE) {
        for (int i = threadIdx.x; i < PLACES; i += DECIDE) {
            f.slot[i] = -1;
            f.item[i] = INT_MAX;
        }
        __syncthreads();
        const int i = threadIdx.x, s = i < a.n ? a.slots[i] : -1;
        if (s >= 0 && s < a.n_slots)
            for (int at = place_of(s);; at = (at + 1) % PLACES) {  // (at most DECIDE of the places are taken)
                const int was = atomicCAS(&f.slot[at], -1, s);
                if (was == -1 || was == s) {
                    atomicMin(&f.item[at], i);
                    break;
                }
            }
    } else {
        for (int i = threadIdx.x; i < a.n; i += DECIDE) {
            const int s = a.slots[i];
            if (s >= 0 && s < a.n_slots) __hip_atomic_store(&owner[s], INT_MAX, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < a.n; i += DECIDE) {
            const int s = a.slots[i];
            if (s >= 0 && s < a.n_slots) atomicMin(&owner[s], i);
        }
    }
    __syncthreads();
}
__device__ __forceinline__ bool is_first(const PoolArgs &a, const int *owner, const First &f, int s, int i) {
    if (a.n > DECIDE) return load_fresh(&owner[s]) == i;
    int at = place_of(s);
    while (f.slot[at] != s) at = (at + 1) % PLACES;
    return f.item[at] == i;
}

__device__ __forceinline__ int length_at(const PoolArgs &a, int slot) {
    return min(max(a.kv_len[slot], 0), a.max_pages << a.page_shift);
}
__device__ __forceinline__ int pages_of(const PoolArgs &a, int length) { return (length + (1 << a.page_shift) - 1) >> a.page_shift; }

__global__ __launch_bounds__(DECIDE) void resize_decide_kernel(PoolArgs a) {
    __shared__ int64_t shared[WAVES];
    __shared__ First firsts;
    const Space ws = space(a);
    find_firsts(a, ws.owner, firsts);
    int64_t need = 0;  // of all items so far
    for (int i0 = 0; i0 < a.n; i0 += DECIDE) {
        const int i = i0 + threadIdx.x;
        Item item = {0, -1, 0, 0};
        int mine = 0;
        if (i < a.n) {
            const int s = a.slots[i], length = a.lengths[i];
            if (s >= 0 && s < a.n_slots && length >= 0 && length <= a.max_pages << a.page_shift && is_first(a, ws.owner, firsts, s, i)) {
                const int old = length_at(a, s);
                item.had = pages_of(a, old);
                item.has = pages_of(a, length);
                if (length > old && (old & ((1 << a.page_shift) - 1))) {
                    const int last = a.block_table[(int64_t)s * a.max_pages + item.had - 1];
                    item.own = last >= 0 && last < a.n_pages && a.refs[last] > 1;
                }
                mine = max(item.has - item.had, 0) + item.own;
            }
        }
        int64_t total;
        const int64_t first = need + block_prefix(mine, shared, total);
        item.first = (int)min(first, (int64_t)INT_MAX);
        if (i < a.n) ws.items[i] = item;
        need += total;
    }
    // free pages until there are enough
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t found = 0;
    for (int p0 = 0; p0 < a.n_pages && found < need; p0 += DECIDE * SCAN) {
        const int base = p0 + wave * 64 * SCAN + lane;
        uint64_t free[SCAN];
        int count = 0;
#pragma unroll
        for (int k = 0; k < SCAN; ++k) {
            const int p = base + k * 64;
            free[k] = __ballot(p < a.n_pages && a.refs[p < a.n_pages ? p : 0] == 0);
            count += __builtin_popcountll(free[k]);
        }
        int64_t total;
        int64_t at = found + block_prefix(lane == 0 ? count : 0, shared, total);
        at = __shfl(at, 0);
#pragma unroll
        for (int k = 0; k < SCAN; ++k) {
            const int64_t r = at + __builtin_popcountll(free[k] & ((1ull << lane) - 1));
            if ((free[k] >> lane) & 1 && r < need) ws.free[r] = base + k * 64;
            at += __builtin_popcountll(free[k]);
        }
        found += total;
    }
    if (threadIdx.x == 0) *ws.found = (int)min(found, need);
}

// Grid (items, pieces of a row of the table).
__global__ __launch_bounds__(THREADS) void resize_apply_kernel(PoolArgs a) {
    const int i = blockIdx.x, at = blockIdx.y * THREADS + threadIdx.x, step = gridDim.y * THREADS;
    const Space ws = space(a);
    const Item item = ws.items[i];
    const int grows = max(item.has - item.had, 0);
    const bool too_few = (int64_t)item.first + grows + item.own > *ws.found && grows + item.own > 0;
    const int state = item.has < 0 ? DS4HC_PAGES_INVALID : too_few ? DS4HC_PAGES_SHORT : DS4HC_PAGES_DONE;
    int from = -1, to = -1;
    if (state == DS4HC_PAGES_DONE) {
        const int slot = a.slots[i];
        int32_t *row = a.block_table + (int64_t)slot * a.max_pages;
        if (at == 0) {
            if (item.own) {
                from = row[item.had - 1];
                to = ws.free[item.first];
                row[item.had - 1] = to;
                a.refs[to] = 1;
                atomicSub(&a.refs[from], 1);
            }
            a.kv_len[slot] = a.lengths[i];
        }
        for (int e = item.had + at; e < item.has; e += step) {
            const int page = ws.free[item.first + item.own + e - item.had];
            row[e] = page;
            a.refs[page] = 1;
        }
        for (int e = item.has + at; e < item.had; e += step) {
            const int page = row[e];
            row[e] = -1;
            if (page >= 0 && page < a.n_pages) atomicSub(&a.refs[page], 1);
        }
    }
    if (at == 0) {
        a.copies[2 * i] = from;
        a.copies[2 * i + 1] = to;
        a.status[i] = state;
    }
}

__global__ __launch_bounds__(DECIDE) void fork_decide_kernel(PoolArgs a) {
    __shared__ First firsts;
    const Space ws = space(a);
    find_firsts(a, ws.owner, firsts);
    for (int i = threadIdx.x; i < a.n; i += DECIDE) {
        const int child = a.slots[i], parent = a.lengths[i];
        Item item = {0, -1, 0, 0};
        if (child >= 0 && child < a.n_slots && parent >= 0 && parent < a.n_slots && child != parent && is_first(a, ws.owner, firsts, child, i) &&
            a.kv_len[child] == 0) {
            item.had = length_at(a, parent);
            item.has = pages_of(a, item.had);
        }
        ws.items[i] = item;
    }
}

__global__ __launch_bounds__(THREADS) void fork_apply_kernel(PoolArgs a) {
    const int i = blockIdx.x, at = blockIdx.y * THREADS + threadIdx.x, step = gridDim.y * THREADS;
    const Item item = space(a).items[i];
    if (item.has >= 0) {
        const int32_t *from = a.block_table + (int64_t)a.lengths[i] * a.max_pages;
        int32_t *to = a.block_table + (int64_t)a.slots[i] * a.max_pages;
        for (int e = at; e < item.has; e += step) {
            const int page = from[e];
            to[e] = page;
            if (page >= 0 && page < a.n_pages) atomicAdd(&a.refs[page], 1);
        }
        if (at == 0) a.kv_len[a.slots[i]] = item.had;
    }
    if (at == 0) a.status[i] = item.has < 0 ? DS4HC_PAGES_INVALID : DS4HC_PAGES_DONE;
}

// Workgroups a row of the table.
unsigned row_pieces(const PoolArgs &a) {
    const int64_t pieces = ((int64_t)a.max_pages + THREADS - 1) / THREADS;
    return (unsigned)(pieces < 16 ? pieces : 16);
}

}  // namespace

hipError_t launch_compact(const CompactArgs &a, hipStream_t s) {
    const int64_t threads = (int64_t)a.s.layers * (a.s.row_bytes / 16);
    return launch_kernel(compact_kernel, dim3((unsigned)((threads + THREADS - 1) / THREADS), (unsigned)a.n_seqs), dim3(THREADS), s, a);
}

hipError_t launch_pages_copy(const Store &st, int64_t n, const int32_t *pairs, hipStream_t s) {
    const int64_t pieces = ((st.row_bytes << st.page_shift) + COPY - 1) / COPY;
    const dim3 grid((unsigned)(pieces < 1024 ? pieces : 1024), (unsigned)st.layers, (unsigned)(n < 32768 ? n : 32768));
    return launch_kernel(copy_kernel, grid, dim3(THREADS), s, st, (int)n, pairs);
}

uint64_t pages_workspace_bytes(int n_slots, int n_pages, int64_t n) {
    return 16 + (uint64_t)n * sizeof(Item) + ((uint64_t)n_slots + n_pages) * sizeof(int);
}

hipError_t launch_pages_resize(const PoolArgs &a, hipStream_t s) {
    const hipError_t e = launch_kernel(resize_decide_kernel, dim3(1), dim3(DECIDE), s, a);
    if (e != hipSuccess) return e;
    return launch_kernel(resize_apply_kernel, dim3((unsigned)a.n, row_pieces(a)), dim3(THREADS), s, a);
}

hipError_t launch_pages_fork(const PoolArgs &a, hipStream_t s) {
    const hipError_t e = launch_kernel(fork_decide_kernel, dim3(1), dim3(DECIDE), s, a);
    if (e != hipSuccess) return e;
    return launch_kernel(fork_apply_kernel, dim3((unsigned)a.n, row_pieces(a)), dim3(THREADS), s, a);
}

}  // namespace ds4hc
