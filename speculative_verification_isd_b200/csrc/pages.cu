// Page bookkeeping of the paged KV cache between steps: a new batch made of
// an old one (requests continued, forked, moved to other slots or dropped),
// and compaction, which gives the bump allocator the dropped pages back.
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "launch.h"
#include "plan.h"

namespace isd {

namespace {

constexpr int kPageThreads = 256;
constexpr int kCopies = 8;     // 16-byte loads in flight per thread of a fork's copy
constexpr int kForkPools = 4;  // pools of one copy

struct ForkArgs {
    int B, R, P, num_pages, max_pages, n_pools;
    size_t row_bytes, page_bytes;  // one token's K (or V) rows; one page of a pool
    const int32_t* parent;
    const int32_t* reserve;  // or null: no room asked for
    const int32_t* kv_len;
    const int32_t* pages_used;
    const int32_t* page_table;
    const int32_t* next_free;
    int32_t* next_kv_len;
    int32_t* next_pages_used;
    int32_t* next_table;
    int32_t* next_free_out;
    int32_t* err_flag;
};

// What child r takes over: `have` columns of its parent's row, `need` columns
// in all (need - have new pages), and whether it is the parent's first child.
struct Child {
    int par, kv, have, need;
    bool first;
    int fault;  // an ISD_FLAG_* bit: the slot is left empty
};

ISD_DEVINL Child child_of(const ForkArgs& a, const int* first_of, int r) {
    Child c = {-1, 0, 0, 0, false, 0};
    const int par = a.parent[r];
    if (par == -1) return c;
    if (par < 0 || par >= a.B) {
        c.fault = ISD_FLAG_PARENT_OOB;
        return c;
    }
    const int kv = a.kv_len[par], used = a.pages_used[par];
    const int more = a.reserve ? a.reserve[r] : 0;
    const bool first = first_of[par] == r;
    const long long want = ((long long)kv + more + a.P - 1) / a.P;
    const int whole = kv / a.P, cover = (int)(((long long)kv + a.P - 1) / a.P);
    if (kv < 0 || more < 0 || used < cover || used > a.max_pages || want > a.max_pages) {
        c.fault = ISD_FLAG_CAPACITY;
        return c;
    }
    c.par = par;
    c.kv = kv;
    c.first = first;
    c.have = first ? used : whole;
    c.need = max((int)want, first ? used : cover);
    return c;
}

// Exclusive scan over the CTA; returns the total.
template <int THREADS, typename T>
ISD_DEVINL T block_scan(T v, T& before, T* part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const T u = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += u;
    }
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    T base = 0, total = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) base += part[w];
        total += part[w];
    }
    __syncthreads();
    before = base + incl - v;
    return total;
}

// Every CTA works out all children's new pages (a scan in slot order), then
// takes its share: the state and table row of some children, and of the
// part-filled pages' copies some (child, group of pools) pairs.
//
// A copy is latency: a child's rows of one pool are 2 to 30 KB.  So the pairs,
// whose bytes go from none to a page's, are dealt out in turn (a grid of (child,
// share of the pools) left the CTAs of the longest tail running alone: 18.6
// against 16.2 us for 45 slots and 72 pools), and a thread has kCopies loads in flight
// over the pools of a pair.
__global__ void __launch_bounds__(kPageThreads, 3) fork_kernel(const __grid_constant__ ForkArgs a,
                                                               const __grid_constant__ PoolList pools) {
    extern __shared__ int first_of[];  // [B]: the first child of each request
    int* page_of = first_of + a.B;     // [R]: each child's first new page, or -1 where it cannot be made
    __shared__ long long part[kPageThreads / 32];
    __shared__ int s_end;
    for (int b = threadIdx.x; b < a.B; b += kPageThreads) first_of[b] = a.R;
    if (threadIdx.x == 0) s_end = max(*a.next_free, 0);
    __syncthreads();
    for (int i = threadIdx.x; i < a.R; i += kPageThreads) {
        const int p = a.parent[i];
        if (p >= 0 && p < a.B) atomicMin(&first_of[p], i);
    }
    __syncthreads();
    long long run = max(*a.next_free, 0);
    for (int i0 = 0; i0 < a.R; i0 += kPageThreads) {
        const int i = i0 + (int)threadIdx.x;
        const Child c = i < a.R ? child_of(a, first_of, i) : Child{-1, 0, 0, 0, false, 0};
        const long long add = c.need - c.have;
        long long before;
        const long long sum = block_scan<kPageThreads>(add, before, part);
        const long long base = run + before;
        // a child past the pool's end gets no pages, nor does any after it that needs some
        const bool fits = add == 0 || base + add <= a.num_pages;
        if (i < a.R) page_of[i] = fits ? (int)min(base, (long long)a.num_pages) : -1;
        if (add > 0 && fits) atomicMax(&s_end, (int)(base + add));
        run += sum;
    }
    __syncthreads();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.next_free_out = s_end;
    auto child = [&](int r) {
        const Child c = child_of(a, first_of, r);
        return page_of[r] < 0 ? Child{-1, 0, 0, 0, false, ISD_FLAG_CAPACITY} : c;
    };
    for (int r = blockIdx.x; r < a.R; r += gridDim.x) {
        const Child c = child(r);
        const int base = page_of[r];
        if (threadIdx.x == 0) {
            if (c.fault) raise_flag(a.err_flag, c.fault);
            a.next_kv_len[r] = c.kv;
            a.next_pages_used[r] = c.need;
        }
        for (int j = threadIdx.x; j < a.max_pages; j += kPageThreads) {
            int id = -1;
            if (j < c.have) {
                id = a.page_table[(size_t)c.par * a.max_pages + j];
                if (id < 0 || id >= a.num_pages) raise_flag(a.err_flag, ISD_FLAG_PAGE_OOB);
            } else if (j < c.need) {
                id = base + (j - c.have);
            }
            a.next_table[(size_t)r * a.max_pages + j] = id;
        }
    }
    // the part-filled pages: the rows before kv_len go to the child's own page
    const int groups = (a.n_pools + kForkPools - 1) / kForkPools;
    for (long long w = blockIdx.x; w < (long long)a.R * groups; w += gridDim.x) {
        const int r = (int)(w / groups), p0 = (int)(w - (long long)r * groups) * kForkPools;
        const Child c = child(r);
        const int tail = c.par >= 0 && !c.first ? c.kv % a.P : 0;
        if (tail == 0) continue;
        const int src = a.page_table[(size_t)c.par * a.max_pages + c.have];
        if (src < 0 || src >= a.num_pages) {
            if (p0 == 0 && threadIdx.x == 0) raise_flag(a.err_flag, ISD_FLAG_PAGE_OOB);
            continue;
        }
        const size_t from = (size_t)src * a.page_bytes, to = (size_t)page_of[r] * a.page_bytes;
        const size_t vecs = (size_t)tail * a.row_bytes / 16, all = min(kForkPools, a.n_pools - p0) * vecs;
        for (size_t i0 = threadIdx.x; i0 < all; i0 += kCopies * kPageThreads) {
            uint4 v[kCopies];
            uint4* dst[kCopies];
#pragma unroll
            for (int u = 0; u < kCopies; ++u) {
                const size_t i = i0 + u * kPageThreads;
                if (i >= all) break;
                int p = 0;  // pool i / vecs of the group
#pragma unroll
                for (int k = 1; k < kForkPools; ++k) p += i >= k * vecs;
                char* pool = static_cast<char*>(pools.p[p0 + p]);
                v[u] = reinterpret_cast<const uint4*>(pool + from)[i - p * vecs];
                dst[u] = reinterpret_cast<uint4*>(pool + to) + (i - p * vecs);
            }
#pragma unroll
            for (int u = 0; u < kCopies; ++u)
                if (i0 + u * kPageThreads < all) *dst[u] = v[u];
        }
    }
}

struct CompactArgs {
    int B, num_pages, max_pages, n_pools;
    size_t page_bytes;
    const int32_t* pages_used;
    const int32_t* page_table;
    int32_t* next_table;
    int32_t* next_free_out;
    uint32_t* live;  // bitmap of the pages in use
    int32_t* moves;  // number of pages that move, then their old and new places
    int32_t* err_flag;
};

// Compaction, by the size of the bookkeeping: up to kSmallPages pages and
// kSmallCells table cells one CTA does all of it with the bitmap in shared
// memory (plan_small_kernel: 2 launches in all); beyond, mark, plan and place
// are kernels of their own (5 with the bitmap's clearing).  A compaction by the
// small way took 8.7 us against 12.3 with a table of 8 x 26 cells, and 45.2
// against 38.0 with 64 x 1001.
constexpr int kSmallPages = 1 << 20, kSmallCells = 1 << 14, kSmallThreads = 1024;

// One CTA per request: marks its pages.
__global__ void __launch_bounds__(kPageThreads) mark_kernel(const __grid_constant__ CompactArgs a) {
    const int b = blockIdx.x;
    int used = a.pages_used[b];
    if (used < 0 || used > a.max_pages) {
        if (threadIdx.x == 0) raise_flag(a.err_flag, ISD_FLAG_CAPACITY);
        used = min(max(used, 0), a.max_pages);
    }
    for (int j = threadIdx.x; j < used; j += kPageThreads) {
        const int id = a.page_table[(size_t)b * a.max_pages + j];
        if (id < 0 || id >= a.num_pages) raise_flag(a.err_flag, ISD_FLAG_PAGE_OOB);
        else atomicOr(&a.live[id >> 5], 1u << (id & 31));
    }
}

// L pages are in use; the k-th used page at or past L moves to the k-th free
// place before L.  One CTA writes the list of moves.
template <int THREADS>
ISD_DEVINL int list_moves(const CompactArgs& a, const uint32_t* live, int* part) {
    const int words = (a.num_pages - 1) / 32 + 1;
    int count = 0;
    for (int w0 = 0; w0 < words; w0 += THREADS) {
        const int w = w0 + (int)threadIdx.x;
        int before;
        count += block_scan<THREADS>(w < words ? __popc(live[w]) : 0, before, part);
    }
    int holes = 0, movers = 0;
    int32_t* src = a.moves + 1;
    int32_t* dst = src + a.num_pages;
    for (int w0 = 0; w0 < words; w0 += THREADS) {
        const int w = w0 + (int)threadIdx.x;
        const uint32_t bits = w < words ? live[w] : 0;
        // pages of this word that lie before / from L on
        const int below = min(max(count - 32 * w, 0), 32);
        const uint32_t low = below == 32 ? 0xffffffffu : ((1u << below) - 1);
        uint32_t h = w < words ? ~bits & low : 0, m = bits & ~low;
        int hb, mb;
        const int ht = block_scan<THREADS>(__popc(h), hb, part), mt = block_scan<THREADS>(__popc(m), mb, part);
        for (int k = holes + hb; h; h &= h - 1) dst[k++] = 32 * w + __ffs(h) - 1;
        for (int k = movers + mb; m; m &= m - 1) src[k++] = 32 * w + __ffs(m) - 1;
        holes += ht;
        movers += mt;
    }
    if (threadIdx.x == 0) {
        a.moves[0] = movers;
        *a.next_free_out = count;
    }
    return movers;
}

__global__ void __launch_bounds__(kSmallThreads) plan_kernel(const __grid_constant__ CompactArgs a) {
    __shared__ int part[kSmallThreads / 32];
    list_moves<kSmallThreads>(a, a.live, part);
}

// Marking, listing and placing by one CTA.
__global__ void __launch_bounds__(kSmallThreads) plan_small_kernel(const __grid_constant__ CompactArgs a) {
    extern __shared__ uint32_t live[];
    __shared__ int part[kSmallThreads / 32];
    pdl_trigger();
    const int words = (a.num_pages - 1) / 32 + 1, cells = a.B * a.max_pages;
    for (int w = threadIdx.x; w < words; w += kSmallThreads) live[w] = 0;
    for (int b = threadIdx.x; b < a.B; b += kSmallThreads) {
        const int used = a.pages_used[b];
        if (used < 0 || used > a.max_pages) raise_flag(a.err_flag, ISD_FLAG_CAPACITY);
    }
    __syncthreads();
#pragma unroll 4
    for (int e = threadIdx.x; e < cells; e += kSmallThreads) {
        const int b = e / a.max_pages, j = e - b * a.max_pages;
        const int id = a.page_table[e];
        if (j >= a.pages_used[b]) continue;
        if (id < 0 || id >= a.num_pages) raise_flag(a.err_flag, ISD_FLAG_PAGE_OOB);
        else atomicOr(&live[id >> 5], 1u << (id & 31));
    }
    __syncthreads();
    const int n = list_moves<kSmallThreads>(a, live, part);
    __syncthreads();
    const int32_t* src = a.moves + 1;
    const int32_t* dst = src + a.num_pages;
    int32_t* to = a.moves + 1 + 2 * (size_t)a.num_pages;
    for (int i = threadIdx.x; i < n; i += kSmallThreads) to[src[i]] = dst[i];
}

// New place of every page that moves, by its old one.
__global__ void __launch_bounds__(kPageThreads) place_kernel(const __grid_constant__ CompactArgs a) {
    const int n = a.moves[0];
    const int32_t* src = a.moves + 1;
    const int32_t* dst = src + a.num_pages;
    int32_t* to = a.moves + 1 + 2 * (size_t)a.num_pages;
    for (int i = blockIdx.x * kPageThreads + threadIdx.x; i < n; i += gridDim.x * kPageThreads) to[src[i]] = dst[i];
}

constexpr int kMoves = 4;  // 16-byte loads in flight per thread
// The moves of the pools (grid.y), as one long list of 16-byte vectors with
// kMoves loads in flight per thread, and (with `tables`) the page tables.  Bound
// by memory: 2.15 GB of 32 KB pages in 348 us, 0.94 of a copy's rate.
__global__ void __launch_bounds__(kPageThreads) move_kernel(const __grid_constant__ CompactArgs a,
                                                            const __grid_constant__ PoolList pools, int tables) {
    pdl_wait();
    const int n = a.moves[0];
    const int32_t* src = a.moves + 1;
    const int32_t* dst = src + a.num_pages;
    const int32_t* to = a.moves + 1 + 2 * (size_t)a.num_pages;
    const int live = *a.next_free_out;
    if (tables) {
        for (int b = blockIdx.y * gridDim.x + blockIdx.x; b < a.B; b += gridDim.x * gridDim.y) {
            const int used = min(max(a.pages_used[b], 0), a.max_pages);
            for (int j = threadIdx.x; j < a.max_pages; j += kPageThreads) {
                int id = -1;
                if (j < used) {
                    id = a.page_table[(size_t)b * a.max_pages + j];
                    if (id >= live && id < a.num_pages) id = to[id];
                }
                a.next_table[(size_t)b * a.max_pages + j] = id;
            }
        }
    }
    if ((int)blockIdx.y >= a.n_pools) return;
    const uint32_t vecs = (uint32_t)(a.page_bytes / 16);  // of a page; a page of 64 GB is no pool's
    const unsigned long long all = (unsigned long long)n * vecs, step = (unsigned long long)gridDim.x * kPageThreads;
    char* pool = static_cast<char*>(pools.p[blockIdx.y]);
    for (unsigned long long i0 = (unsigned long long)blockIdx.x * kPageThreads + threadIdx.x; i0 < all; i0 += kMoves * step) {
        uint4 v[kMoves];
        uint4* dest[kMoves];
#pragma unroll
        for (int u = 0; u < kMoves; ++u) {
            const unsigned long long i = i0 + u * step;
            if (i >= all) break;
            const uint32_t k = all >> 32 ? (uint32_t)(i / vecs) : (uint32_t)i / vecs;
            const size_t x = i - (unsigned long long)k * vecs;
            v[u] = reinterpret_cast<const uint4*>(pool + (size_t)src[k] * a.page_bytes)[x];
            dest[u] = reinterpret_cast<uint4*>(pool + (size_t)dst[k] * a.page_bytes) + x;
        }
#pragma unroll
        for (int u = 0; u < kMoves; ++u)
            if (i0 + u * step < all) *dest[u] = v[u];
    }
}

}  // namespace

cudaError_t launch_fork(const isd_dims* d, int R, const int32_t* parent, const int32_t* reserve,
                        const int32_t* kv_len, const int32_t* pages_used, const int32_t* page_table,
                        const int32_t* next_free, int n_pools, uint16_t* const* pools,
                        int32_t* next_kv_len, int32_t* next_pages_used, int32_t* next_table,
                        int32_t* next_free_out, int32_t* err_flag, cudaStream_t st) {
    ForkArgs a;
    a.B = d->B;
    a.R = R;
    a.P = d->page_size;
    a.num_pages = d->num_pages;
    a.max_pages = d->max_pages_per_req;
    a.n_pools = 0;
    a.row_bytes = (size_t)d->Hkv * d->D * 2;
    a.page_bytes = a.row_bytes * d->page_size;
    a.parent = parent;
    a.reserve = reserve;
    a.kv_len = kv_len;
    a.pages_used = pages_used;
    a.page_table = page_table;
    a.next_free = next_free;
    a.next_kv_len = next_kv_len;
    a.next_pages_used = next_pages_used;
    a.next_table = next_table;
    a.next_free_out = next_free_out;
    a.err_flag = err_flag;
    for (int p0 = 0; p0 == 0 || p0 < n_pools; p0 += kPoolsPerLaunch) {
        PoolList list;
        a.n_pools = n_pools - p0 < kPoolsPerLaunch ? n_pools - p0 : kPoolsPerLaunch;
        for (int i = 0; i < a.n_pools; ++i) list.p[i] = pools[p0 + i];
        const long long jobs = (long long)R * std::max(1, (a.n_pools + kForkPools - 1) / kForkPools);
        const int grid = (int)std::min(jobs, 3ll * persistent_grid());  // as many as run at once
        const cudaError_t e = launch_kernel(false, fork_kernel, dim3(grid), dim3(kPageThreads),
                                            ((size_t)d->B + R) * 4, st, a, list);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_compact(const isd_dims* d, const int32_t* pages_used, const int32_t* page_table,
                           int n_pools, uint16_t* const* pools, int32_t* next_table,
                           int32_t* next_free_out, void* ws, int32_t* err_flag, cudaStream_t st) {
    CompactArgs a;
    a.B = d->B;
    a.num_pages = d->num_pages;
    a.max_pages = d->max_pages_per_req;
    a.page_bytes = (size_t)d->page_size * d->Hkv * d->D * 2;
    a.pages_used = pages_used;
    a.page_table = page_table;
    a.next_table = next_table;
    a.next_free_out = next_free_out;
    const size_t bitmap = page_bitmap_bytes(d->num_pages);
    a.live = static_cast<uint32_t*>(ws);
    a.moves = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + align_up(bitmap, 256));
    a.err_flag = err_flag;
    const bool small = d->num_pages <= kSmallPages && (long long)d->B * d->max_pages_per_req <= kSmallCells;
    cudaError_t e;
    if (small) {
        static unsigned long long configured = 0;  // bit per device
        int dev = 0;
        e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
        if (!(configured >> dev & 1ull)) {
            e = cudaFuncSetAttribute(plan_small_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmallPages / 8);
            if (e != cudaSuccess) return e;
            configured |= 1ull << dev;
        }
        e = launch_kernel(false, plan_small_kernel, dim3(1), dim3(kSmallThreads), bitmap, st, a);
        if (e != cudaSuccess) return e;
    } else {
        e = cudaMemsetAsync(a.live, 0, bitmap, st);
        if (e != cudaSuccess) return e;
        e = launch_kernel(false, mark_kernel, dim3(d->B), dim3(kPageThreads), 0, st, a);
        if (e != cudaSuccess) return e;
        e = launch_kernel(false, plan_kernel, dim3(1), dim3(kSmallThreads), 0, st, a);
        if (e != cudaSuccess) return e;
        e = launch_kernel(false, place_kernel, dim3(persistent_grid()), dim3(kPageThreads), 0, st, a);
        if (e != cudaSuccess) return e;
    }
    for (int p0 = 0; p0 == 0 || p0 < n_pools; p0 += kPoolsPerLaunch) {
        PoolList list;
        a.n_pools = n_pools - p0 < kPoolsPerLaunch ? n_pools - p0 : kPoolsPerLaunch;
        for (int i = 0; i < a.n_pools; ++i) list.p[i] = pools[p0 + i];
        const int rows = a.n_pools > 0 ? a.n_pools : 1;
        e = launch_kernel(small && p0 == 0, move_kernel, dim3((8 * persistent_grid() + rows - 1) / rows, rows),
                          dim3(kPageThreads), 0, st, a, list, p0 == 0 ? 1 : 0);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace isd
