// Page bookkeeping of the 4-bit K/V cache: copy, reserve, fork, free, compact.
//
// Who gets which page is decided by one workgroup (prefix sums over the
// requests and over the free pages, both in order, so that the outcome does
// not depend on timing); the bulk -- pages, table rows, counts -- is moved by
// a second launch over many workgroups, from the lists that the first left
// in the workspace.  Counts are changed by integer atomics, whose order does
// not show.
#include "qmm_kv.hpp"

namespace qmm {
namespace kv {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kPlan = 1024;   // threads of a planning workgroup
constexpr int kMove = 256;    // threads of a moving one
constexpr int kPiece = 4;     // 16-byte loads in flight of each of them

// Exclusive prefix sum over the workgroup; every thread gets the total.
template <class T>
__device__ __forceinline__ T block_scan(T v, T* total, T* lds) {
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    T x = v;
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
        const T y = __shfl_up(x, m);
        if (lane >= m) x += y;
    }
    if (lane == 63) lds[wave] = x;
    __syncthreads();
    T before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPlan / 64; ++w) {
        const T t = lds[w];
        before += w < wave ? t : 0;
        all += t;
    }
    __syncthreads();
    *total = all;
    return before + x - v;
}

struct Pool {
    u32x4_t* p;
    int64_t pages, page16;  // 16-byte pieces of a page in one layer
    int layers;
};

// One workgroup's share of moving `count` pages in every layer: pieces of
// kMove * kPiece * 16 bytes.  Bound by memory: 460 pages of 8 layers (543 MB
// read and written) 101 us, 5.4 TB/s; three pages of one layer 3.0 us, which is
// the launch and two dependent reads.
__device__ void move_pages(const Pool& pool, const int32_t* src, const int32_t* dst, int64_t count, int64_t first,
                           int64_t step) {
    const int64_t pieces = (pool.page16 + kMove * kPiece - 1) / (kMove * kPiece);
    const int64_t items = count * pool.layers * pieces;
    for (int64_t it = first; it < items; it += step) {
        const int64_t piece = it % pieces, ml = it / pieces;
        const int64_t layer = ml % pool.layers, m = ml / pool.layers;
        const int64_t s = src[m], d = dst[m];
        if (s < 0 || d < 0 || s >= pool.pages || d >= pool.pages || s == d) continue;
        const u32x4_t* from = pool.p + (layer * pool.pages + s) * pool.page16;
        u32x4_t* to = pool.p + (layer * pool.pages + d) * pool.page16;
        const int64_t at = piece * (kMove * kPiece) + threadIdx.x;
        u32x4_t v[kPiece];
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
            if (at + i * kMove < pool.page16) v[i] = __builtin_nontemporal_load(from + at + i * kMove);
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
            if (at + i * kMove < pool.page16) __builtin_nontemporal_store(v[i], to + at + i * kMove);
    }
}

__global__ __launch_bounds__(kMove) void copy_kernel(Pool pool, const int32_t* __restrict__ src,
                                                     const int32_t* __restrict__ dst, int64_t n) {
    move_pages(pool, src, dst, n, blockIdx.x, gridDim.x);
}

// Gives the lowest free pages, in order, to the requests whose needs have the
// exclusive prefix sums `before` [n], `total` in all: take(request, which of
// its pages, page).  Returns how many pages were given.
template <class Take>
__device__ int allocate(const int32_t* refs, int64_t pages, const int32_t* before, int64_t n, int total, int* lds,
                        Take take) {
    int found = 0;
    for (int64_t base = 0; base < pages && found < total; base += kPlan) {
        const int64_t p = base + threadIdx.x;
        const int free = p < pages && refs[p] == 0;
        int here;
        const int rank = found + block_scan(free, &here, lds);
        if (free && rank < total) {
            // the last request whose pages begin at or before this rank
            int64_t lo = 0, hi = n;
            while (hi - lo > 1) {
                const int64_t mid = (lo + hi) / 2;
                if (before[mid] <= rank) lo = mid; else hi = mid;
            }
            take(lo, rank - before[lo], static_cast<int32_t>(p));
        }
        found += here;
    }
    return found < total ? found : total;
}

// Plan of a reservation, all of it: workspace before[n], need[n], col[n].
// Needs are summed in 64 bits and kept cut to pages + 1: a request that far
// back is refused whatever its number is.
__global__ __launch_bounds__(kPlan) void reserve_kernel(int32_t* __restrict__ tables, int64_t width,
                                                        int32_t* __restrict__ lens, int32_t* __restrict__ refs,
                                                        int64_t pages, int64_t seqs, int page_shift,
                                                        const int32_t* __restrict__ add, int32_t* __restrict__ ok,
                                                        int32_t* ws) {
    __shared__ int lds[kPlan / 64];
    __shared__ int64_t lds64[kPlan / 64];
    __shared__ int granted;
    int32_t* before = ws;
    int32_t* need = ws + seqs;
    int32_t* col = ws + 2 * seqs;
    const int64_t page = int64_t{1} << page_shift;
    if (threadIdx.x == 0) granted = 0;
    // free pages in all
    int free_pages = 0;
    for (int64_t base = 0; base < pages; base += kPlan) {
        const int64_t p = base + threadIdx.x;
        int here;
        block_scan(static_cast<int>(p < pages && refs[p] == 0), &here, lds);
        free_pages += here;
    }
    int64_t sum = 0;
    for (int64_t base = 0; base < seqs; base += kPlan) {
        const int64_t s = base + threadIdx.x;
        int64_t lack = 0, c = 0;
        bool sound = false;
        if (s < seqs) {
            const int64_t len = lens[s], more = add[s];
            sound = len >= 0 && more >= 0 && len + more <= width * page;
            if (sound) {
                const int64_t want = (len + more + page - 1) >> page_shift;
                c = (len + page - 1) >> page_shift;
                while (c < want && tables[s * width + c] >= 0) ++c;  // held already (the length was cut back)
                lack = want - c;
            }
        }
        int64_t all;
        const int64_t at = sum + block_scan(lack, &all, lds64);
        sum += all;
        if (s < seqs) {
            const bool get = sound && at + lack <= free_pages;
            before[s] = static_cast<int32_t>(at <= pages ? at : pages + 1);
            need[s] = sound && (lack == 0 || get) ? static_cast<int32_t>(lack) : -1;
            col[s] = static_cast<int32_t>(c);
            if (get && lack > 0) atomicMax(&granted, static_cast<int>(at + lack));
        }
    }
    __syncthreads();
    allocate(refs, pages, before, seqs, granted, lds, [&](int64_t s, int which, int32_t p) {
        tables[s * width + col[s] + which] = p;
        refs[p] = 1;
    });
    __syncthreads();
    for (int64_t s = threadIdx.x; s < seqs; s += kPlan) {
        const bool get = need[s] >= 0;
        ok[s] = get;
        if (get) lens[s] += add[s];
    }
}

// Plan of a fork (64 new sequences, 1500 pages: 4.9 us, one workgroup's chain
// of reads, prefix sums and stores): workspace before[n], from[n], to[n] (page to copy and its
// place; to < 0: none).  Sets lens of the new sequences and counts of the new
// pages; fork_apply fills the rows, counts the shared pages and copies.
__global__ __launch_bounds__(kPlan) void fork_plan_kernel(const int32_t* __restrict__ tables, int64_t width,
                                                          int32_t* __restrict__ lens, int32_t* __restrict__ refs,
                                                          int64_t pages, int64_t seqs, int page_shift,
                                                          const int32_t* __restrict__ src,
                                                          const int32_t* __restrict__ dst, int64_t n,
                                                          int32_t* __restrict__ ok, int32_t* ws) {
    __shared__ int lds[kPlan / 64];
    int32_t* before = ws;
    int32_t* from = ws + n;
    int32_t* to = ws + 2 * n;
    const int64_t page = int64_t{1} << page_shift;
    int total = 0;
    for (int64_t base = 0; base < n; base += kPlan) {
        const int64_t i = base + threadIdx.x;
        int need = 0;
        if (i < n) {
            const int64_t s = src[i], d = dst[i];
            bool sound = s >= 0 && s < seqs && d >= 0 && d < seqs && s != d;
            int32_t last = -1;
            if (sound) {
                const int64_t len = lens[s];
                sound = len >= 0 && len <= width * page;
                if (sound && len % page != 0) {
                    last = tables[s * width + (len >> page_shift)];
                    sound = last >= 0 && last < pages;
                    need = sound;
                }
            }
            ok[i] = sound;
            from[i] = last;
            to[i] = -1;
        }
        int all;
        const int at = total + block_scan(need, &all, lds);
        if (i < n) before[i] = at;
        total += all;
    }
    __syncthreads();
    // (requests that need nothing share their prefix with the next that does: that one is the last of them)
    const int given = allocate(refs, pages, before, n, total, lds, [&](int64_t i, int, int32_t p) {
        to[i] = p;
        refs[p] = 1;
    });
    __syncthreads();
    for (int64_t i = threadIdx.x; i < n; i += kPlan) {
        if (!ok[i]) {
            from[i] = -1;
        } else if (from[i] >= 0 && before[i] >= given) {
            ok[i] = 0;
            from[i] = -1;
        }
        const int64_t d = dst[i];
        if (d >= 0 && d < seqs && d != src[i]) lens[d] = ok[i] ? lens[src[i]] : 0;
    }
}

// 64 sequences forked in 8 layers, 75.5 MB: 13 to 15 us, 5 to 5.8 TB/s.
__global__ __launch_bounds__(kMove) void fork_apply_kernel(Pool pool, int32_t* __restrict__ tables, int64_t width,
                                                           const int32_t* __restrict__ lens, int32_t* __restrict__ refs,
                                                           int64_t seqs, int page_shift,
                                                           const int32_t* __restrict__ src,
                                                           const int32_t* __restrict__ dst, int64_t n,
                                                           const int32_t* __restrict__ ok,
                                                           const int32_t* __restrict__ ws, int64_t row_blocks) {
    const int32_t* from = ws + n;
    const int32_t* to = ws + 2 * n;
    if (blockIdx.x >= row_blocks) {
        move_pages(pool, from, to, n, blockIdx.x - row_blocks, gridDim.x - row_blocks);
        return;
    }
    for (int64_t i = blockIdx.x; i < n; i += row_blocks) {
        const int64_t s = src[i], d = dst[i];
        if (d < 0 || d >= seqs || s == d) continue;
        const bool get = ok[i] != 0;
        const int64_t whole = get ? lens[s] >> page_shift : 0;
        for (int64_t c = threadIdx.x; c < width; c += kMove) {
            int32_t p = -1;
            if (c < whole) {
                p = tables[s * width + c];
                if (p >= 0 && p < pool.pages) atomicAdd(&refs[p], 1);
            } else if (get && c == whole) {
                p = to[i];
            }
            tables[d * width + c] = p;
        }
    }
}

__global__ __launch_bounds__(kMove) void free_kernel(int32_t* __restrict__ tables, int64_t width,
                                                     int32_t* __restrict__ lens, int32_t* __restrict__ refs,
                                                     int64_t pages, int64_t seqs, const int32_t* __restrict__ which,
                                                     int64_t n) {
    for (int64_t i = blockIdx.x; i < n; i += gridDim.x) {
        const int64_t s = which[i];
        if (s < 0 || s >= seqs) continue;
        for (int64_t c = threadIdx.x; c < width; c += kMove) {
            // exchanged, so that a sequence named twice gives its pages up once
            const int32_t p = atomicExch(&tables[s * width + c], -1);
            if (p >= 0 && p < pages) atomicSub(&refs[p], 1);
        }
        if (threadIdx.x == 0) lens[s] = 0;
    }
}

// Plan of a compaction (2049 pages: 8.8 us, three prefix sums over them, one
// after the other): workspace count, from[half], to[half], place[pages]
// (where each page goes).
__global__ __launch_bounds__(kPlan) void compact_plan_kernel(const int32_t* refs, int64_t pages, int32_t* refs_out,
                                                             int32_t* __restrict__ live_out, int32_t* ws) {
    __shared__ int lds[kPlan / 64];
    const int64_t half = pages / 2 + 1;
    int32_t* from = ws + 1;
    int32_t* to = from + half;
    int32_t* place = to + half;
    int live = 0;
    for (int64_t base = 0; base < pages; base += kPlan) {
        const int64_t p = base + threadIdx.x;
        int here;
        block_scan(static_cast<int>(p < pages && refs[p] > 0), &here, lds);
        live += here;
    }
    int movers = 0, holes = 0;
    for (int64_t base = 0; base < pages; base += kPlan) {
        const int64_t p = base + threadIdx.x;
        const int32_t r = p < pages ? refs[p] : 0;
        const int mover = p < pages && p >= live && r > 0, hole = p < live && r <= 0;
        int here;
        const int m = movers + block_scan(mover, &here, lds);
        movers += here;
        const int h = holes + block_scan(hole, &here, lds);
        holes += here;
        if (mover) from[m] = static_cast<int32_t>(p);
        if (hole) to[h] = static_cast<int32_t>(p);
        if (p < pages) place[p] = static_cast<int32_t>(p);
    }
    if (threadIdx.x == 0) {
        ws[0] = movers;
        live_out[0] = live;
    }
    __syncthreads();
    // counts of what moves first (they are read at or above `live`, written below it) ...
    for (int64_t i = threadIdx.x; i < movers; i += kPlan) {
        place[from[i]] = to[i];
        refs_out[to[i]] = refs[from[i]];
    }
    __syncthreads();
    // ... then the rest: live pages that stay, and none at or above `live`
    for (int64_t p = threadIdx.x; p < pages; p += kPlan) {
        if (p >= live) refs_out[p] = 0;
        else if (refs != refs_out && refs[p] > 0) refs_out[p] = refs[p];
    }
}

__global__ __launch_bounds__(kMove) void compact_apply_kernel(Pool pool, const int32_t* tables, int32_t* tables_out,
                                                              int64_t entries, const int32_t* __restrict__ ws,
                                                              int64_t table_blocks) {
    const int64_t half = pool.pages / 2 + 1;
    const int32_t* from = ws + 1;
    const int32_t* to = from + half;
    const int32_t* place = to + half;
    if (blockIdx.x >= table_blocks) {
        move_pages(pool, from, to, ws[0], blockIdx.x - table_blocks, gridDim.x - table_blocks);
        return;
    }
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kMove + threadIdx.x; i < entries; i += table_blocks * kMove) {
        const int32_t p = tables[i];
        tables_out[i] = p >= 0 && p < pool.pages ? place[p] : -1;
    }
}

Pool pool_of(const qmm_kv_cache& c) {
    const Record rec(c.page_size, c.head_dim, c.group_size);
    return Pool{static_cast<u32x4_t*>(c.pool), c.pages, static_cast<int64_t>(rec.words()) / 4 * c.kv_heads, c.layers};
}

// Workgroups for moving `count` pages: one a piece, up to a chip full.
int64_t move_blocks(const Pool& p, int64_t count) {
    const int64_t pieces = (p.page16 + kMove * kPiece - 1) / (kMove * kPiece);
    const int64_t items = count * p.layers * pieces;
    return items < 8192 ? (items > 0 ? items : 1) : 8192;
}

int shift_of(const qmm_kv_cache& c) { return __builtin_ctz(static_cast<unsigned>(c.page_size)); }

}  // namespace

int64_t pages_workspace(const qmm_kv_cache& c, int64_t n) {
    const int64_t ints = n > 0 ? 3 * n : 1 + 2 * (c.pages / 2 + 1) + c.pages;
    return (ints * 4 + 15) / 16 * 16;
}

hipError_t launch_copy_pages(const qmm_kv_cache& c, const int32_t* src, const int32_t* dst, int64_t n,
                             hipStream_t st) {
    const Pool p = pool_of(c);
    hipLaunchKernelGGL(copy_kernel, dim3(static_cast<unsigned>(move_blocks(p, n))), dim3(kMove), 0, st, p, src, dst,
                       n);
    return hipGetLastError();
}

hipError_t launch_reserve(const qmm_kv_cache& c, const PageArgs& a, const int32_t* add, int32_t* ok) {
    hipLaunchKernelGGL(reserve_kernel, dim3(1), dim3(kPlan), 0, a.stream, a.tables, a.width, a.lens, a.refs, c.pages,
                       a.seqs, shift_of(c), add, ok, a.workspace);
    return hipGetLastError();
}

hipError_t launch_fork(const qmm_kv_cache& c, const PageArgs& a, const int32_t* src, const int32_t* dst, int64_t n,
                       int32_t* ok) {
    hipLaunchKernelGGL(fork_plan_kernel, dim3(1), dim3(kPlan), 0, a.stream, a.tables, a.width, a.lens, a.refs, c.pages,
                       a.seqs, shift_of(c), src, dst, n, ok, a.workspace);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const Pool p = pool_of(c);
    const int64_t rows = n < 1024 ? n : 1024;
    hipLaunchKernelGGL(fork_apply_kernel, dim3(static_cast<unsigned>(rows + move_blocks(p, n))), dim3(kMove), 0,
                       a.stream, p, a.tables, a.width, a.lens, a.refs, a.seqs, shift_of(c), src, dst, n, ok,
                       a.workspace, rows);
    return hipGetLastError();
}

hipError_t launch_free(const qmm_kv_cache& c, const PageArgs& a, const int32_t* which, int64_t n) {
    hipLaunchKernelGGL(free_kernel, dim3(static_cast<unsigned>(n < 8192 ? n : 8192)), dim3(kMove), 0, a.stream,
                       a.tables, a.width, a.lens, a.refs, c.pages, a.seqs, which, n);
    return hipGetLastError();
}

hipError_t launch_compact(const qmm_kv_cache& c, const PageArgs& a, int32_t* tables_out, int32_t* refs_out,
                          int32_t* live_out) {
    hipLaunchKernelGGL(compact_plan_kernel, dim3(1), dim3(kPlan), 0, a.stream, a.refs, c.pages, refs_out, live_out,
                       a.workspace);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const Pool p = pool_of(c);
    const int64_t entries = a.seqs * a.width;
    int64_t tb = (entries + kMove - 1) / kMove;
    tb = tb < 1024 ? tb : 1024;
    hipLaunchKernelGGL(compact_apply_kernel, dim3(static_cast<unsigned>(tb + move_blocks(p, c.pages / 2))),
                       dim3(kMove), 0, a.stream, p, a.tables, tables_out, entries, a.workspace, tb);
    return hipGetLastError();
}

}  // namespace kv
}  // namespace qmm
