// extern "C" boundary of the paged 4-bit K/V cache: argument validation and
// launches on the caller's stream.  Declarations and contracts: qmm.h.
#include <initializer_list>

#include "qmm_kv.hpp"

namespace {

using namespace qmm::kv;

int hip_status(hipError_t e) { return e == hipSuccess ? QMM_OK : QMM_ERR_HIP; }

bool off(const void* p, unsigned align) { return (reinterpret_cast<uintptr_t>(p) & (align - 1)) != 0; }

int check_ptrs(std::initializer_list<const void*> ps, unsigned align) {
    for (const void* p : ps)
        if (p == nullptr) return QMM_ERR_INVALID_ARG;
    for (const void* p : ps)
        if (off(p, align)) return QMM_ERR_MISALIGNED;
    return QMM_OK;
}

int check_geometry(const qmm_kv_cache* c) {
    if (c == nullptr || c->pages < 0) return QMM_ERR_INVALID_ARG;
    if (c->dt != QMM_F16 && c->dt != QMM_BF16) return QMM_ERR_UNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return QMM_ERR_UNSUPPORTED;
    if (c->group_size != 32 && c->group_size != 64 && c->group_size != 128) return QMM_ERR_UNSUPPORTED;
    if (c->group_size > c->head_dim) return QMM_ERR_UNSUPPORTED;
    if (c->page_size != 32 && c->page_size != 64 && c->page_size != 128 && c->page_size != 256)
        return QMM_ERR_UNSUPPORTED;
    if (c->kv_heads < 1 || c->kv_heads > 65535 || c->layers < 1 || c->layers > 65535) return QMM_ERR_UNSUPPORTED;
    if (c->pages > (int64_t{1} << 30)) return QMM_ERR_UNSUPPORTED;
    return QMM_OK;
}

// Tokens that a table's row may have room for: positions, and those that a
// kernel's loops look ahead to, are 32-bit.
constexpr int64_t kMostTokens = int64_t{1} << 30;

int64_t record_words(const qmm_kv_cache& c) { return Record(c.page_size, c.head_dim, c.group_size).words(); }

// What every call over sequences checks; *s is filled where it returns
// QMM_OK.
int check_seqs(const qmm_kv_cache* c, int layer, int64_t seqs, int64_t max_new, int64_t rows, const int32_t* tables,
               int64_t width, const int32_t* lens, const int32_t* starts, Seqs* s) {
    if (const int st = check_geometry(c); st != QMM_OK) return st;
    if (layer < 0 || layer >= c->layers || seqs < 0 || max_new < 0 || rows < 0 || width < 0) return QMM_ERR_INVALID_ARG;
    if (seqs > INT32_MAX / 64 || max_new > INT32_MAX / 2 || rows > INT32_MAX ||
        width > kMostTokens / c->page_size || max_new > INT32_MAX / c->kv_heads)
        return QMM_ERR_UNSUPPORTED;
    if (starts == nullptr && rows != seqs * max_new) return QMM_ERR_INVALID_ARG;
    if (starts != nullptr && rows > seqs * max_new) return QMM_ERR_INVALID_ARG;
    s->seqs = static_cast<int>(seqs);
    s->max_new = static_cast<int>(max_new);
    s->rows = rows;
    s->width = width;
    s->pages = c->pages;
    s->kv_heads = c->kv_heads;
    s->page_shift = __builtin_ctz(static_cast<unsigned>(c->page_size));
    s->tables = tables;
    s->lens = lens;
    s->starts = starts;
    if (rows == 0) return QMM_OK;
    // a pool or a table without entries may be NULL: nothing is read from it
    if (const int st = check_ptrs({lens}, 4); st != QMM_OK) return st;
    if (width > 0)
        if (const int st = check_ptrs({tables}, 4); st != QMM_OK) return st;
    if (starts != nullptr && off(starts, 4)) return QMM_ERR_MISALIGNED;
    if (c->pages > 0)
        if (const int st = check_ptrs({c->pool}, 16); st != QMM_OK) return st;
    s->pool = static_cast<uint32_t*>(c->pool) + layer * c->pages * c->kv_heads * record_words(*c);
    return QMM_OK;
}

int check_rows(const void* p, int64_t stride_row, int64_t stride_head) {
    if (stride_row < 0 || stride_head < 0) return QMM_ERR_INVALID_ARG;
    if (const int st = check_ptrs({p}, 16); st != QMM_OK) return st;
    if (stride_row % 8 != 0 || stride_head % 8 != 0) return QMM_ERR_MISALIGNED;
    return QMM_OK;
}

int check_heads(const qmm_kv_cache* c, int64_t max_new, int64_t heads) {
    if (heads < 1 || heads > INT32_MAX / 1024 || heads % c->kv_heads != 0 || max_new > 64) return QMM_ERR_UNSUPPORTED;
    return QMM_OK;
}

int check_workspace(const void* ws, int64_t bytes, int64_t need) {
    if (need < 0) return static_cast<int>(need);
    if (need == 0) return QMM_OK;
    if (ws == nullptr || bytes < need) return QMM_ERR_INVALID_ARG;
    return off(ws, 16) ? QMM_ERR_MISALIGNED : QMM_OK;
}

int check_pages(const qmm_kv_cache* c, int64_t seqs, const int32_t* tables, int64_t width, const int32_t* lens,
                const int32_t* refs) {
    if (const int st = check_geometry(c); st != QMM_OK) return st;
    if (seqs < 0 || width < 0) return QMM_ERR_INVALID_ARG;
    if (seqs > INT32_MAX / 64 || width > kMostTokens / c->page_size) return QMM_ERR_UNSUPPORTED;
    if (seqs > 0 && lens != nullptr && off(lens, 4)) return QMM_ERR_MISALIGNED;
    if (seqs > 0 && width > 0)
        if (const int st = check_ptrs({tables}, 4); st != QMM_OK) return st;
    if (c->pages > 0)
        if (const int st = check_ptrs({refs}, 4); st != QMM_OK) return st;
    return QMM_OK;
}

}  // namespace

extern "C" {

int64_t qmm_kv_record_bytes(const qmm_kv_cache* cache) {
    if (const int st = check_geometry(cache); st != QMM_OK) return st;
    return 4 * record_words(*cache);
}

int qmm_kv_append(const qmm_kv_cache* cache, int layer, int64_t seqs, int64_t max_new, int64_t rows,
                  const int32_t* tables, int64_t table_width, const int32_t* lens, const int32_t* starts,
                  const void* k, int64_t k_stride_row, int64_t k_stride_head, const void* v, int64_t v_stride_row,
                  int64_t v_stride_head, void* stream) {
    Seqs s{};
    int st = check_seqs(cache, layer, seqs, max_new, rows, tables, table_width, lens, starts, &s);
    if (st != QMM_OK || rows == 0) return st;
    if ((st = check_rows(k, k_stride_row, k_stride_head)) != QMM_OK) return st;
    if ((st = check_rows(v, v_stride_row, v_stride_head)) != QMM_OK) return st;
    if (table_width == 0 || cache->pages == 0) return QMM_OK;
    return hip_status(launch_append(*cache, s, Rows{k, k_stride_row, k_stride_head},
                                    Rows{v, v_stride_row, v_stride_head}, static_cast<hipStream_t>(stream)));
}

int qmm_kv_read(const qmm_kv_cache* cache, int layer, int64_t seqs, int64_t max_new, int64_t rows,
                const int32_t* tables, int64_t table_width, const int32_t* lens, const int32_t* starts, void* k,
                void* v, void* stream) {
    Seqs s{};
    int st = check_seqs(cache, layer, seqs, max_new, rows, tables, table_width, lens, starts, &s);
    if (st != QMM_OK || rows == 0) return st;
    if ((st = check_ptrs({k, v}, 16)) != QMM_OK) return st;
    return hip_status(launch_read(*cache, s, k, v, static_cast<hipStream_t>(stream)));
}

// (a window beyond the longest sequence is none)
static int clamped(int64_t n) { return static_cast<int>(n < kMostTokens ? n : kMostTokens); }

static int64_t attend_space(const qmm_kv_cache* cache, int64_t seqs, int64_t max_new, int64_t rows, int64_t heads,
                            int64_t max_len, int window, int sinks) {
    if (const int st = check_geometry(cache); st != QMM_OK) return st;
    if (seqs < 0 || max_new < 0 || rows < 0 || max_len < 1) return QMM_ERR_INVALID_ARG;
    if (seqs > INT32_MAX / 64 || rows > INT32_MAX || max_len > INT32_MAX) return QMM_ERR_UNSUPPORTED;
    if (const int st = check_heads(cache, max_new, heads); st != QMM_OK) return st;
    if (rows == 0 || max_new == 0) return 0;
    return attend_workspace(*cache, seqs, max_new, rows, heads, max_len, window, sinks);
}

int64_t qmm_kv_attend_workspace_bytes(const qmm_kv_cache* cache, int64_t seqs, int64_t max_new, int64_t rows,
                                      int64_t heads, int64_t max_len) {
    return attend_space(cache, seqs, max_new, rows, heads, max_len, 0, 0);
}

int64_t qmm_kv_attend_window_workspace_bytes(const qmm_kv_cache* cache, int64_t seqs, int64_t max_new, int64_t rows,
                                             int64_t heads, int64_t max_len, int64_t window, int64_t sinks) {
    if (window < 1 || sinks < 0) return QMM_ERR_INVALID_ARG;
    return attend_space(cache, seqs, max_new, rows, heads, max_len, clamped(window), clamped(sinks));
}

static int attend(const qmm_kv_cache* cache, int layer, int64_t seqs, int64_t max_new, int64_t rows,
                  const int32_t* tables, int64_t table_width, const int32_t* lens, const int32_t* starts,
                  const void* q, int64_t q_stride_row, int64_t q_stride_head, int64_t heads, float scale,
                  const int64_t* mask, void* out, float* lse, int64_t max_len, void* workspace,
                  int64_t workspace_bytes, int window, int sinks, void* stream) {
    Seqs s{};
    int st = check_seqs(cache, layer, seqs, max_new, rows, tables, table_width, lens, starts, &s);
    if (st != QMM_OK) return st;
    if ((st = check_heads(cache, max_new, heads)) != QMM_OK) return st;
    if (max_len < 1) return QMM_ERR_INVALID_ARG;
    if (max_len > INT32_MAX) return QMM_ERR_UNSUPPORTED;
    if (rows == 0) return QMM_OK;
    if ((st = check_rows(q, q_stride_row, q_stride_head)) != QMM_OK) return st;
    if ((st = check_ptrs({out}, 16)) != QMM_OK) return st;
    if (off(mask, 8) || off(lse, 4)) return QMM_ERR_MISALIGNED;
    st = check_workspace(workspace, workspace_bytes,
                         attend_workspace(*cache, seqs, max_new, rows, heads, max_len, window, sinks));
    if (st != QMM_OK) return st;
    return hip_status(launch_attend(
        *cache, AttendArgs{s, Rows{q, q_stride_row, q_stride_head}, static_cast<int>(heads), scale, mask, out, lse,
                           workspace, max_len, window, sinks, static_cast<hipStream_t>(stream)}));
}

int qmm_kv_attend(const qmm_kv_cache* cache, int layer, int64_t seqs, int64_t max_new, int64_t rows,
                  const int32_t* tables, int64_t table_width, const int32_t* lens, const int32_t* starts,
                  const void* q, int64_t q_stride_row, int64_t q_stride_head, int64_t heads, float scale,
                  const int64_t* mask, void* out, float* lse, int64_t max_len, void* workspace,
                  int64_t workspace_bytes, void* stream) {
    return attend(cache, layer, seqs, max_new, rows, tables, table_width, lens, starts, q, q_stride_row, q_stride_head,
                  heads, scale, mask, out, lse, max_len, workspace, workspace_bytes, 0, 0, stream);
}

int qmm_kv_attend_window(const qmm_kv_cache* cache, int layer, int64_t seqs, int64_t max_new, int64_t rows,
                         const int32_t* tables, int64_t table_width, const int32_t* lens, const int32_t* starts,
                         const void* q, int64_t q_stride_row, int64_t q_stride_head, int64_t heads, float scale,
                         const int64_t* mask, int64_t window, int64_t sinks, void* out, float* lse, int64_t max_len,
                         void* workspace, int64_t workspace_bytes, void* stream) {
    if (window < 1 || sinks < 0) return QMM_ERR_INVALID_ARG;
    return attend(cache, layer, seqs, max_new, rows, tables, table_width, lens, starts, q, q_stride_row, q_stride_head,
                  heads, scale, mask, out, lse, max_len, workspace, workspace_bytes, clamped(window), clamped(sinks), stream);
}

int64_t qmm_kv_pages_workspace_bytes(const qmm_kv_cache* cache, int64_t n) {
    if (const int st = check_geometry(cache); st != QMM_OK) return st;
    if (n < 0) return QMM_ERR_INVALID_ARG;
    if (n > INT32_MAX / 64) return QMM_ERR_UNSUPPORTED;
    return pages_workspace(*cache, n);
}

int qmm_kv_copy_pages(const qmm_kv_cache* cache, const int32_t* src, const int32_t* dst, int64_t n, void* stream) {
    if (const int st = check_geometry(cache); st != QMM_OK) return st;
    if (n < 0) return QMM_ERR_INVALID_ARG;
    if (n > INT32_MAX / 64) return QMM_ERR_UNSUPPORTED;
    if (n == 0 || cache->pages == 0) return QMM_OK;
    if (const int st = check_ptrs({src, dst}, 4); st != QMM_OK) return st;
    if (const int st = check_ptrs({cache->pool}, 16); st != QMM_OK) return st;
    return hip_status(launch_copy_pages(*cache, src, dst, n, static_cast<hipStream_t>(stream)));
}

int qmm_kv_reserve(const qmm_kv_cache* cache, int64_t seqs, int32_t* tables, int64_t table_width, int32_t* lens,
                   int32_t* refs, const int32_t* add, int32_t* ok, void* workspace, int64_t workspace_bytes,
                   void* stream) {
    int st = check_pages(cache, seqs, tables, table_width, lens, refs);
    if (st != QMM_OK || seqs == 0) return st;
    if ((st = check_ptrs({lens, add, ok}, 4)) != QMM_OK) return st;
    if ((st = check_workspace(workspace, workspace_bytes, pages_workspace(*cache, seqs))) != QMM_OK) return st;
    const PageArgs a{tables, lens, refs, seqs, table_width, static_cast<int32_t*>(workspace),
                     static_cast<hipStream_t>(stream)};
    return hip_status(launch_reserve(*cache, a, add, ok));
}

int qmm_kv_fork(const qmm_kv_cache* cache, int64_t seqs, int32_t* tables, int64_t table_width, int32_t* lens,
                int32_t* refs, const int32_t* src, const int32_t* dst, int64_t n, int32_t* ok, void* workspace,
                int64_t workspace_bytes, void* stream) {
    int st = check_pages(cache, seqs, tables, table_width, lens, refs);
    if (st != QMM_OK) return st;
    if (n < 0) return QMM_ERR_INVALID_ARG;
    if (n > INT32_MAX / 64) return QMM_ERR_UNSUPPORTED;
    if (n == 0) return QMM_OK;
    if ((st = check_ptrs({src, dst, ok}, 4)) != QMM_OK) return st;
    if (seqs > 0 && (st = check_ptrs({lens}, 4)) != QMM_OK) return st;
    if (cache->pages > 0 && (st = check_ptrs({cache->pool}, 16)) != QMM_OK) return st;
    if ((st = check_workspace(workspace, workspace_bytes, pages_workspace(*cache, n))) != QMM_OK) return st;
    const PageArgs a{tables, lens, refs, seqs, table_width, static_cast<int32_t*>(workspace),
                     static_cast<hipStream_t>(stream)};
    return hip_status(launch_fork(*cache, a, src, dst, n, ok));
}

int qmm_kv_free(const qmm_kv_cache* cache, int64_t seqs, int32_t* tables, int64_t table_width, int32_t* lens,
                int32_t* refs, const int32_t* which, int64_t n, void* stream) {
    int st = check_pages(cache, seqs, tables, table_width, lens, refs);
    if (st != QMM_OK) return st;
    if (n < 0) return QMM_ERR_INVALID_ARG;
    if (n > INT32_MAX / 64) return QMM_ERR_UNSUPPORTED;
    if (n == 0 || seqs == 0) return QMM_OK;
    if ((st = check_ptrs({which, lens}, 4)) != QMM_OK) return st;
    const PageArgs a{tables, lens, refs, seqs, table_width, nullptr, static_cast<hipStream_t>(stream)};
    return hip_status(launch_free(*cache, a, which, n));
}

int qmm_kv_compact(const qmm_kv_cache* cache, int64_t seqs, const int32_t* tables, int64_t table_width,
                   const int32_t* refs, int32_t* tables_out, int32_t* refs_out, int32_t* live_out, void* workspace,
                   int64_t workspace_bytes, void* stream) {
    int st = check_pages(cache, seqs, tables, table_width, nullptr, refs);
    if (st != QMM_OK) return st;
    if ((st = check_ptrs({live_out}, 4)) != QMM_OK) return st;
    if (seqs > 0 && table_width > 0 && (st = check_ptrs({tables_out}, 4)) != QMM_OK) return st;
    if (cache->pages > 0) {
        if ((st = check_ptrs({refs_out}, 4)) != QMM_OK) return st;
        if ((st = check_ptrs({cache->pool}, 16)) != QMM_OK) return st;
    }
    if ((st = check_workspace(workspace, workspace_bytes, pages_workspace(*cache, 0))) != QMM_OK) return st;
    const PageArgs a{const_cast<int32_t*>(tables), nullptr, const_cast<int32_t*>(refs), seqs, table_width,
                     static_cast<int32_t*>(workspace), static_cast<hipStream_t>(stream)};
    return hip_status(launch_compact(*cache, a, tables_out, refs_out, live_out));
}

}  // extern "C"
