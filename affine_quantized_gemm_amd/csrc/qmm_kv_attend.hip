// Attention over the paged 4-bit K/V cache: how a call is cut, and its launch.
#include "qmm_kv_attend.hpp"

namespace qmm {
namespace kv {

template <> AttendFn attend_fn<DT_F16, 64>(int, int);
template <> AttendFn attend_fn<DT_F16, 128>(int, int);
template <> AttendFn attend_fn<DT_F16, 256>(int, int);
template <> AttendFn attend_fn<DT_BF16, 64>(int, int);
template <> AttendFn attend_fn<DT_BF16, 128>(int, int);
template <> AttendFn attend_fn<DT_BF16, 256>(int, int);

namespace {

struct AttendPlan {
    int row_tiles, row_groups, splits, chunk;
};

// Tokens are split until the workgroups fill the chip (two for each of 256
// CUs), in parts of 128 tokens (a step for each wavefront) at least.
AttendPlan plan_of(const qmm_kv_cache& c, int64_t seqs, int64_t max_new, int64_t heads, int64_t max_len) {
    AttendPlan p;
    const int64_t rows = max_new * (heads / c.kv_heads);
    p.row_tiles = rows <= 16 ? 1 : 2;
    p.row_groups = static_cast<int>((rows + 16 * p.row_tiles - 1) / (16 * p.row_tiles));
    const int64_t units = seqs * c.kv_heads * p.row_groups;
    int64_t splits = (512 + units - 1) / units;
    const int64_t most = (max_len + 127) / 128;
    splits = splits < most ? splits : most;
    const int64_t chunk = ((max_len + splits - 1) / splits + 127) / 128 * 128;
    p.splits = static_cast<int>((max_len + chunk - 1) / chunk);
    p.chunk = static_cast<int>(chunk < INT32_MAX / 2 ? chunk : INT32_MAX / 2);
    return p;
}

}  // namespace

int64_t attend_workspace(const qmm_kv_cache& c, int64_t seqs, int64_t max_new, int64_t, int64_t heads,
                         int64_t max_len) {
    const AttendPlan p = plan_of(c, seqs, max_new, heads, max_len);
    if (p.splits == 1) return 0;
    return (seqs * max_new * heads * p.splits * (c.head_dim + 2) * 4 + 15) / 16 * 16;
}

hipError_t launch_attend(const qmm_kv_cache& c, const AttendArgs& a) {
    const AttendPlan p = plan_of(c, a.s.seqs, a.s.max_new, a.heads, a.max_len);
    AttendParams k{};
    k.s = a.s;
    k.q = static_cast<const uint16_t*>(a.q.p);
    k.q_row = a.q.stride_row;
    k.q_head = a.q.stride_head;
    k.heads = a.heads;
    k.group = a.heads / c.kv_heads;
    k.row_groups = p.row_groups;
    k.splits = p.splits;
    k.chunk = p.chunk;
    k.scale = a.scale;
    k.mask = a.mask;
    k.out = static_cast<uint16_t*>(a.out);
    k.lse = a.lse;
    k.part = static_cast<float*>(a.workspace);
    const int64_t units = static_cast<int64_t>(a.s.seqs) * c.kv_heads * p.splits;
    const int64_t blocks = (units + 7) / 8 * 8 * p.row_groups;
    if (blocks > INT32_MAX || static_cast<int64_t>(a.s.seqs) * a.s.max_new * a.heads > INT32_MAX) return hipErrorInvalidValue;
    AttendFn fn = nullptr;
    const bool half = c.dt == QMM_F16;
    switch (c.head_dim) {
        case 64: fn = half ? attend_fn<DT_F16, 64>(c.group_size, p.row_tiles) : attend_fn<DT_BF16, 64>(c.group_size, p.row_tiles); break;
        case 128: fn = half ? attend_fn<DT_F16, 128>(c.group_size, p.row_tiles) : attend_fn<DT_BF16, 128>(c.group_size, p.row_tiles); break;
        case 256: fn = half ? attend_fn<DT_F16, 256>(c.group_size, p.row_tiles) : attend_fn<DT_BF16, 256>(c.group_size, p.row_tiles); break;
        default: break;
    }
    return fn != nullptr ? fn(k, blocks, a.stream) : hipErrorInvalidValue;
}

}  // namespace kv
}  // namespace qmm
