// Attention over the paged 4-bit K/V cache: how a call is cut, and its launch.
#include "qmm_kv_attend.hpp"

namespace qmm {
namespace kv {

template <> AttendFn attend_fn<DT_F16, 64, false>(int);
template <> AttendFn attend_fn<DT_F16, 64, true>(int);
template <> AttendFn attend_fn<DT_F16, 128, false>(int);
template <> AttendFn attend_fn<DT_F16, 128, true>(int);
template <> AttendFn attend_fn<DT_F16, 256, false>(int);
template <> AttendFn attend_fn<DT_F16, 256, true>(int);
template <> AttendFn attend_fn<DT_BF16, 64, false>(int);
template <> AttendFn attend_fn<DT_BF16, 64, true>(int);
template <> AttendFn attend_fn<DT_BF16, 128, false>(int);
template <> AttendFn attend_fn<DT_BF16, 128, true>(int);
template <> AttendFn attend_fn<DT_BF16, 256, false>(int);
template <> AttendFn attend_fn<DT_BF16, 256, true>(int);

namespace {

struct AttendPlan {
    int row_tiles, row_groups, parts;
    bool by_rows;
    int64_t bytes;
};

// By tokens, with two tiles of rows a wavefront (heads of 256 have the
// registers for one), or where there are more tiles by rows, a workgroup a
// sequence.  By rows costs the tokens of a sequence one after another, by
// tokens a start, a meeting of its wavefronts and an end for every two tiles:
// over sequences, kv heads and pairs of tiles, as multiples of the
// workgroups that the chip runs at a time, those weigh as
// 512 * multiple > max_len + 384.  Measured (us of a call, by rows / by tokens,
// 64 rows of 4 heads of 128): multiple 1/16, 512 tokens 21.5 / 15.5; 1, 128
// 11.3 / 13.4 and 512 22.3 / 16.6; 2, 128 12.2 / 24.1, 512 23.0 / 30.4 and
// 1024 37.1 / 37.6; 4, 1024 45.5 / 71.6 and 4096 175 / 185.  64 rows of 32
// heads, 4 sequences of 16k 639 / 117.
// Parts for the workgroups that fill the chip over the kv heads and row
// groups; where the sequences are that many, or short, or too many to plan,
// one part each.
AttendPlan plan_of(const qmm_kv_cache& c, int64_t seqs, int64_t max_new, int64_t heads, int64_t max_len) {
    AttendPlan p;
    const int64_t tiles = (max_new * (heads / c.kv_heads) + 15) / 16;
    const int64_t most_tiles = c.head_dim == 256 ? 1 : 2;
    const int64_t units = seqs * c.kv_heads * ((tiles + most_tiles - 1) / most_tiles);
    p.by_rows = tiles > most_tiles && max_len + 384 <= 512 * units / attend_workgroups(static_cast<int>(most_tiles));
    p.row_tiles = tiles == 1 || most_tiles == 1 || (p.by_rows && tiles <= 4) ? 1 : 2;
    const int per = attend_tiles(p.row_tiles, p.by_rows);
    p.row_groups = static_cast<int>((tiles + per - 1) / per);
    const int64_t each = static_cast<int64_t>(c.kv_heads) * p.row_groups;
    int64_t parts = attend_workgroups(p.row_tiles) / each;
    const int64_t most = seqs * ((max_len + kChunk - 1) / kChunk);
    parts = parts < most ? parts : most;
    if (p.by_rows || parts <= seqs || seqs > 64 * kPlanLanes) parts = seqs;
    p.parts = static_cast<int>(parts);
    // (sequences are cut only where seqs * each < workgroups: the counters fit their fixed place)
    static_assert(4 * kDoneStride * attend_workgroups(1) <= QMM_KV_ATTEND_ZEROED_BYTES, "a counter for each");
    p.bytes = parts > seqs ? QMM_KV_ATTEND_ZEROED_BYTES + parts * each * part_floats(c.head_dim, p.row_tiles) * 4 : 0;
    return p;
}

// Tokens that the rows of a sequence may see, up to whole steps at both ends.
int64_t seen_len(int64_t max_new, int64_t max_len, int window, int sinks) {
    const int64_t most = static_cast<int64_t>(window) + sinks + max_new + 96;
    return window > 0 && most < max_len ? most : max_len;
}

template <bool WINDOW>
AttendFn attend_of(const qmm_kv_cache& c) {
    const bool half = c.dt == QMM_F16;
    switch (c.head_dim) {
        case 64: return half ? attend_fn<DT_F16, 64, WINDOW>(c.group_size) : attend_fn<DT_BF16, 64, WINDOW>(c.group_size);
        case 128: return half ? attend_fn<DT_F16, 128, WINDOW>(c.group_size) : attend_fn<DT_BF16, 128, WINDOW>(c.group_size);
        case 256: return half ? attend_fn<DT_F16, 256, WINDOW>(c.group_size) : attend_fn<DT_BF16, 256, WINDOW>(c.group_size);
        default: return nullptr;
    }
}

}  // namespace

int64_t attend_workspace(const qmm_kv_cache& c, int64_t seqs, int64_t max_new, int64_t, int64_t heads,
                         int64_t max_len, int window, int sinks) {
    return plan_of(c, seqs, max_new, heads, seen_len(max_new, max_len, window, sinks)).bytes;
}

hipError_t launch_attend(const qmm_kv_cache& c, const AttendArgs& a) {
    const AttendPlan p = plan_of(c, a.s.seqs, a.s.max_new, a.heads, seen_len(a.s.max_new, a.max_len, a.window, a.sinks));
    AttendParams k{};
    k.s = a.s;
    k.q = static_cast<const uint16_t*>(a.q.p);
    k.q_row = a.q.stride_row;
    k.q_head = a.q.stride_head;
    k.heads = a.heads;
    k.group = a.heads / c.kv_heads;
    k.parts = p.parts;
    k.scale = a.scale;
    k.window = a.window;
    k.sinks = a.sinks;
    k.mask = a.mask;
    k.out = static_cast<uint16_t*>(a.out);
    k.lse = a.lse;
    k.done = static_cast<uint32_t*>(a.workspace);
    k.sums = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + QMM_KV_ATTEND_ZEROED_BYTES);
    const int64_t blocks = (static_cast<int64_t>(p.parts) * c.kv_heads + 7) / 8 * 8;
    if (blocks > INT32_MAX || p.row_groups > 65535) return hipErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(p.row_groups));
    const AttendFn fn = a.window > 0 ? attend_of<true>(c) : attend_of<false>(c);
    return fn != nullptr ? fn(k, p.row_tiles, p.by_rows, grid, a.stream) : hipErrorInvalidValue;
}

}  // namespace kv
}  // namespace qmm
