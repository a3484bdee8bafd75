// Geometry and launch arguments of the paged 4-bit K/V cache (formats: qmm.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmm.h"

namespace qmm {
namespace kv {

// Words and word offsets of one record (one page of one layer and head).
struct Record {
    int code, sb;  // words of the codes / of the scales and biases of K (V the same)
    __host__ __device__ constexpr Record(int page, int dim, int gs) : code(page * dim / 8), sb(page * (dim / gs)) {}
    __host__ __device__ constexpr int k_codes() const { return 0; }
    __host__ __device__ constexpr int v_codes() const { return code; }
    __host__ __device__ constexpr int k_sb() const { return 2 * code; }
    __host__ __device__ constexpr int v_sb() const { return 2 * code + sb; }
    __host__ __device__ constexpr int words() const { return 2 * code + 2 * sb; }
};

// What the kernels that walk over sequences share.
struct Seqs {
    uint32_t* pool;          // the layer's first record
    const int32_t* tables;   // [seqs][width]
    const int32_t* lens;     // [seqs]
    const int32_t* starts;   // [seqs + 1] or null
    int64_t width, rows, pages;
    int seqs, max_new, kv_heads, page_shift;
};

// New tokens of sequence b: first row, how many, and the position of the
// first; clamped so that every row lies in [0, rows).
struct NewTokens {
    int64_t row0;
    int n, pos0;
};
__device__ __forceinline__ NewTokens new_tokens(const Seqs& s, int b) {
    NewTokens t;
    int64_t first, last;
    if (s.starts != nullptr) {
        first = s.starts[b];
        last = s.starts[b + 1];
    } else {
        first = static_cast<int64_t>(b) * s.max_new;
        last = first + s.max_new;
    }
    if (first < 0 || last > s.rows || last <= first) last = first = 0;
    t.row0 = first;
    t.n = static_cast<int>(last - first < s.max_new ? last - first : s.max_new);
    const int len = s.lens[b];
    t.pos0 = (len > 0 ? len : 0) - t.n;
    return t;
}

// Page of position pos of sequence b, or -1.
__device__ __forceinline__ int64_t page_of(const Seqs& s, int b, int pos) {
    if (pos < 0) return -1;
    const int col = pos >> s.page_shift;
    if (col >= s.width) return -1;
    const int p = s.tables[static_cast<int64_t>(b) * s.width + col];
    return p >= 0 && p < s.pages ? p : -1;
}

struct Rows {  // a [rows][heads][dim] operand
    const void* p;
    int64_t stride_row, stride_head;
};

hipError_t launch_append(const qmm_kv_cache& c, const Seqs& s, Rows k, Rows v, hipStream_t st);
hipError_t launch_read(const qmm_kv_cache& c, const Seqs& s, void* k, void* v, hipStream_t st);

struct AttendArgs {
    Seqs s;
    Rows q;
    int heads;
    float scale;
    const int64_t* mask;
    void* out;
    float* lse;
    void* workspace;
    int64_t max_len;
    int window, sinks;  // window 0: none
    hipStream_t stream;
};
int64_t attend_workspace(const qmm_kv_cache& c, int64_t seqs, int64_t max_new, int64_t rows, int64_t heads,
                         int64_t max_len, int window, int sinks);
hipError_t launch_attend(const qmm_kv_cache& c, const AttendArgs& a);

struct PageArgs {
    int32_t* tables;
    int32_t* lens;
    int32_t* refs;
    int64_t seqs, width;
    int32_t* workspace;
    hipStream_t stream;
};
int64_t pages_workspace(const qmm_kv_cache& c, int64_t n);
hipError_t launch_copy_pages(const qmm_kv_cache& c, const int32_t* src, const int32_t* dst, int64_t n, hipStream_t st);
hipError_t launch_reserve(const qmm_kv_cache& c, const PageArgs& a, const int32_t* add, int32_t* ok);
hipError_t launch_fork(const qmm_kv_cache& c, const PageArgs& a, const int32_t* src, const int32_t* dst, int64_t n,
                       int32_t* ok);
hipError_t launch_free(const qmm_kv_cache& c, const PageArgs& a, const int32_t* which, int64_t n);
hipError_t launch_compact(const qmm_kv_cache& c, const PageArgs& a, int32_t* tables_out, int32_t* refs_out,
                          int32_t* live_out);

}  // namespace kv
}  // namespace qmm
