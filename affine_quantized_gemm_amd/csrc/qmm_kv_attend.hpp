// Attention over the paged 4-bit K/V cache on the matrix cores (gfx950).
//
// Mathematics.  With codes c, scale s and bias b of token t and group g (of
// GS consecutive d), k_hat = s c + b, a score is
//   S[t, row] = sum_g s_K[t, g] (sum_{d in g} q[row, d] c[t, d])  +  b_K[t, g] (sum_{d in g} q[row, d]),
// so the first product runs on the codes themselves and its result is scaled
// per token and group; with p = 2^(S - R),
//   O[row, d] = sum_t (p s_V[t, g]) (c[t, d] - 7.5)  +  sum_t p (b_V[t, g] + 7.5 s_V[t, g])
// takes the second product's operand P' = p s_V, one per group, to codes
// again.  Nothing is ever dequantized, and what remains besides the codes --
// biases of K against sums of q, sums of p b and p s -- are small products
// of the stored scales and biases as they are, on the matrix cores as well:
// the vector ALUs are its busiest unit.  The codes are centred because P' is
// rounded to 11 bits: its error is then weighed by |c - 7.5|, about the size of
// the values, and not by c; the centring itself is -7.5 sum_t P', a product
// with a constant.
//
// References.  Each row has an R: 6 below its largest score where it was set,
// rounded up, and moved (what is summed so far scaled) when a score passes it
// by 11.  P' is an fp16 operand, with 11 bits between 2^-14 and 2^16 and fewer
// below, so each row and group has an exponent e besides, P' = 2^e p s: 0 if
// the group's largest p s where R was set is in 2^-4..2^10, else what brings
// it to about 2^3; moved when a P' passes 2^15.  R and e come from the tokens
// that the row sees and from nothing else, so that no other token, row or
// group has a part in a result, whatever its size.
// As long as the scales of V lie in 2^-9..2^4 all e are 0, and most steps do
// not know of them.  A wavefront that meets others starts its tokens anew in
// the form that does (32 sequences of 1k..4k: 49 us instead of 25, 64 rows over
// 16k 310 instead of 120).  To know them in every step is one more instruction
// for every probability and group, 32 of 320 with two tiles; to change over in
// the middle takes the registers of two forms, and a spilled one is a wait for
// the next tokens (verify rows 69 us and more instead of 41).
//
// Codes as operands.  A 4-bit code in the low bits of an fp16 is the
// subnormal number c 2^-24 (in bits 4..7: 16 c 2^-24), which the matrix core
// multiplies exactly.  But it cuts the products of a sum off at a distance
// from the largest one's exponent, and all subnormals have -14: up to 2^-18 of
// P' is lost from every even code's product, downwards.  So what these sums
// are centred by is summed in the same form, over the codes 8..15, and loses
// as much.  (Without, the average of 16k tokens is 1e-4 of itself off, half of
// fp16's rounding.)  The scores' sums lose what depends on the row's q alone,
// found with the codes 8..15 again once for a row and given back with the biases
// (the logarithms of the sums were 1e-6 of themselves off, now 1e-7 to 7e-7).
// Unpacking a word of 8 codes takes four ands and a shift, no conversion and
// no offset to take away again.  The factors 2^24 go into the scores' scale and
// the last step; the 16 of the odd codes into the d order of Q (q / 16) and
// into the last step.  Q is scaled per row by a power of two into fp16's
// range, for bf16 too, so there is one form for both types.
//
// Layout of v_mfma_f32_16x16x32_f16: lane l = 16 j + i supplies A[i][8 j + e]
// and B[8 j + e][i], e = 0..7, and receives D[4 j + r][i], r = 0..3.
//   * Scores are formed as S^T = K Q^T: A = 16 tokens, B = 16 rows.  A lane
//     then holds, for row i, the tokens 4 j + r.
//   * Two such tiles (32 tokens) are the 32 k-slots of the second product
//     O^T = V^T P^T with slot 8 j + e <- token 4 j + e of the first tile, and
//     of the second for e >= 4: P' is in place without any exchange of lanes,
//     and everything that belongs to a row (R, sums) is one value a lane.
// The cache record keeps K codes so that a lane's words of a token are one
// 16-byte piece, and V codes with two neighbouring tokens in the halves of a
// word, so that a masked word is two k-slots.
#pragma once

#include <type_traits>

#include "qmm_device.hpp"
#include "qmm_internal.hpp"
#include "qmm_kv.hpp"
#include "qmm_kv_window.hpp"
#include "qmm_mfma_frag.hpp"

namespace qmm {
namespace kv {

constexpr int kAttendSlots = 2;   // steps of a wavefront in LDS: one read, the others on their way
constexpr float kFar = -3.0e38f;

// How a workgroup's wavefronts share the work.  By tokens: all have the same
// one or two row tiles, take the part's steps in turn and add up at the end
// (one tile: 4 wavefronts, for shorter parts; two: 8, half as many parts to
// put together).  By rows, where there are several tiles: 4 wavefronts have
// one or two tiles of their own each and all the tokens of a sequence, and
// nothing to add.
constexpr int attend_waves(int row_tiles, bool by_rows) { return row_tiles == 2 && !by_rows ? 8 : 4; }
// Rows of a workgroup, in tiles.
constexpr int attend_tiles(int row_tiles, bool by_rows) { return by_rows ? 4 * row_tiles : row_tiles; }
// Wavefronts a SIMD that the registers are to leave room for.
constexpr int attend_occupancy(int dim, int row_tiles) { return dim == 256 || row_tiles == 2 ? 2 : 3; }
// Workgroups that a call is cut into at most: 8 wavefronts a CU.
constexpr int attend_workgroups(int row_tiles) { return 2048 / attend_waves(row_tiles, false); }

// The tokens of a sequence are cut into parts of whole chunks, one workgroup
// a part.
constexpr int kChunk = 128;
constexpr int kDoneStride = 32;  // counters lie in lines of their own: device-wide atomics on one line queue up
constexpr int kPlanLanes = 4;  // sequences a lane holds while the cut is planned: up to 256 are cut

struct AttendParams {
    Seqs s;
    const uint16_t* q;
    int64_t q_row, q_head;
    int heads;
    uint32_t group;         // heads of one kv head
    int parts;              // parts of all sequences together, at most
    float scale;
    const int64_t* mask;
    uint16_t* out;
    float* lse;
    // where sequences are cut: how many parts of (sequence, row group, head) are done, and the parts' sums
    uint32_t* done;         // [seqs][row_groups][kv_heads], kDoneStride apart, 0 before and after the call
    float* sums;            // [parts][row_groups][kv_heads][part_floats]
    int window, sinks;      // (forms with a window)
};

// Floats of one part's sums: rows of D values, then (R, l, -, -) of each row.
constexpr int part_floats(int dim, int row_tiles) { return 16 * row_tiles * (dim + 4); }

namespace {

using mf::Frag;
using mf::float4_t;
using mf::swap16;
using mf::swap32;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Over the four lanes that share i (j = 0..3).
__device__ __forceinline__ float max_j(float v) {
    uint32_t a = __builtin_bit_cast(uint32_t, v), b = a;
    swap32(a, b);
    v = fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
    a = b = __builtin_bit_cast(uint32_t, v);
    swap16(a, b);
    return fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}
__device__ __forceinline__ float sum_j(float v) {
    uint32_t a = __builtin_bit_cast(uint32_t, v), b = a;
    swap32(a, b);
    v = __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
    a = b = __builtin_bit_cast(uint32_t, v);
    swap16(a, b);
    return __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
}

// Half h (0: low) of a word as fp32.
template <int DT>
__device__ __forceinline__ float half_f32(uint32_t w, int h) {
    if constexpr (DT == DT_F16) {
        return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(h ? w >> 16 : w & 0xFFFFu)));
    } else {
        return __builtin_bit_cast(float, h ? w & 0xFFFF0000u : w << 16);
    }
}

// LDS byte address of a pointer into it, the same in every lane.
__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return __builtin_amdgcn_readfirstlane(
        static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) char*)p)));
}

// Two fp32 values -> fp16 halves, to nearest.  (Toward zero would be biased:
// over 131071 tokens the code part of the sum then no longer cancels the bias
// part, 1.3 % of the result off.)
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    typedef float float2_t __attribute__((ext_vector_type(2)));
    typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((float2_t{lo, hi}), half2_t));
}

// A word of 8 codes -> codes (0, 4), 16 x (1, 5), (2, 6), 16 x (3, 7), times 2^-24.
__device__ __forceinline__ Frag codes8(uint32_t w) {
    Frag f;
    const uint32_t t = w >> 8;
    f.v[0] = w & 0x000F000Fu;
    f.v[1] = w & 0x00F000F0u;
    f.v[2] = t & 0x000F000Fu;
    f.v[3] = t & 0x00F000F0u;
    return f;
}

template <int N>
__device__ __forceinline__ void load_words(const uint32_t* p, uint32_t (&w)[N]) {
    if constexpr (N == 2) {
        const uint2 a = *reinterpret_cast<const uint2*>(p);
        w[0] = a.x; w[1] = a.y;
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 a = reinterpret_cast<const uint4*>(p)[i];
            w[4 * i] = a.x; w[4 * i + 1] = a.y; w[4 * i + 2] = a.z; w[4 * i + 3] = a.w;
        }
    }
}

// Values to and from memory that other XCDs' workgroups read and write in the
// same launch: through the device's point of coherence (the XCDs' L2 caches
// are not coherent with each other), as device-scope atomics go, but 16 bytes
// at a time.  `at` is a byte offset from the workspace's sums.  (The 8-byte
// load builtin of this compiler loads 4.)
constexpr int kDeviceScope = 16;  // the sc1 bit of a buffer instruction
using Shared = __amdgpu_buffer_rsrc_t;
__device__ __forceinline__ Shared shared_of(float* p) {
    return __builtin_amdgcn_make_buffer_rsrc(p, 0, -1, 0x00027000);
}
__device__ __forceinline__ void store_shared(Shared r, uint32_t at, float4_t v) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(mf::u32x4_t, v), r, at, 0, kDeviceScope);
}
__device__ __forceinline__ float4_t load_shared(Shared r, uint32_t at) {
    return __builtin_bit_cast(float4_t, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, kDeviceScope));
}

// Sum over the wavefront, in every lane.
__device__ __forceinline__ int wave_sum(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x128, 0xf, 0xf, true);  // rotations within 16 lanes: by 8, 4, 2, 1
    v += __builtin_amdgcn_update_dpp(0, v, 0x124, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x122, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x121, 0xf, 0xf, true);
    uint32_t a = v, b = v;
    swap16(a, b);
    a = b = a + b;
    swap32(a, b);
    return static_cast<int>(a + b);
}

// Which part of which sequence the unit-th workgroup (of a head and row
// group) takes: chunks [first, first + chunks) of sequence b, part `part` of
// `parts`; b < 0: none.
struct Part {
    int b, part, parts, first, chunks, slot0;  // slot0: number of the sequence's first part
};

// Every sequence gets ceil(chunks / T) parts with the least T (up to where
// the search stops) for which they are at most `parts` together: all
// workgroups then take about T chunks whatever the lengths are.  Each
// workgroup finds the cut by itself from the lengths, 64 a register.
template <bool WINDOW>
__device__ __forceinline__ Part find_part(const Seqs& s, int unit, int parts, int lane, int window, int sinks, bool masked) {
    Part p;
    p.part = 0;
    p.parts = 1;
    p.first = 0;
    p.slot0 = unit;
    p.b = unit < s.seqs ? unit : -1;
    p.chunks = INT32_MAX / kChunk;
    if (parts <= s.seqs) return p;  // one part each
    const int64_t cap = s.width << s.page_shift;
    int c[kPlanLanes];
    uint32_t total = 0;  // (2^8 sequences of up to 2^23 chunks)
#pragma unroll
    for (int k = 0; k < kPlanLanes; ++k) {
        const int b = 64 * k + lane;
        c[k] = 0;
        if (64 * k < s.seqs && b < s.seqs) {
            int64_t len = s.lens[b];
            if constexpr (WINDOW) {
                const NewTokens nt = new_tokens(s, b);
                len = window_of(nt.pos0, nt.n, cap, window, sinks, masked).len;
            }
            c[k] = static_cast<int>(((len < cap ? len : cap) + kChunk - 1) / kChunk);
            c[k] = c[k] > 0 ? c[k] : 1;
        }
        total += c[k];
    }
    total = static_cast<uint32_t>(wave_sum(static_cast<int>(total)));
    // (divisions by T through its fp32 reciprocal: all workgroups do the same, which is all that counts)
    auto parts_at = [&](int k, float inv) {
        return c[k] == 0 ? 0 : static_cast<int>((static_cast<float>(c[k]) - 0.5f) * inv) + 1;
    };
    auto fits = [&](int t) {
        const float inv = 1.0f / static_cast<float>(t);
        int n = 0;
#pragma unroll
        for (int k = 0; k < kPlanLanes; ++k) n += parts_at(k, inv);
        return __builtin_amdgcn_readfirstlane(wave_sum(n)) <= parts;
    };
    const uint32_t sum = __builtin_amdgcn_readfirstlane(total);
    // sum / parts <= T, and with T = sum / (parts - seqs) there surely are enough
    int lo = static_cast<int>((sum + parts - 1) / static_cast<uint32_t>(parts));
    int hi = static_cast<int>(sum / static_cast<uint32_t>(parts - s.seqs)) + 1;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (fits(mid)) hi = mid; else lo = mid + 1;
    }
    const float inv = 1.0f / static_cast<float>(lo);
    // the sequence whose parts hold number `unit`
    int before = 0;
    p.b = -1;
#pragma unroll
    for (int k = 0; k < kPlanLanes; ++k) {
        if (64 * k >= s.seqs) break;
        const int mine = parts_at(k, inv);
        int upto = mine;  // parts of this lane's sequence and those before it
#pragma unroll
        for (int m = 1; m < 64; m *= 2) {
            const int y = __shfl_up(upto, m);
            upto += lane >= m ? y : 0;
        }
        const uint64_t past = __ballot(before + upto <= unit);  // sequences all of whose parts come before
        if (past != ~uint64_t{0}) {
            const int l = __builtin_ctzll(~past);
            const int n = __builtin_amdgcn_readlane(mine, l);
            if (64 * k + l < s.seqs && n > 0) {
                p.b = 64 * k + l;
                p.parts = n;
                p.slot0 = before + __builtin_amdgcn_readlane(upto, l) - n;
                p.part = unit - p.slot0;
                const uint32_t chunks = __builtin_amdgcn_readlane(c[k], l);
                p.chunks = static_cast<int>((chunks + n - 1) / static_cast<uint32_t>(n));
                p.first = p.part * p.chunks;
            }
            break;
        }
        before += __builtin_amdgcn_readlane(upto, 63);
    }
    return p;
}

// One step is 32 tokens, a run in each part of a record.  A wavefront brings
// it into a slot of LDS of its own, parts in the record's order, with direct
// global-to-LDS loads of 16 bytes a lane (consecutive lanes, whole lines; no
// registers held), and reads it from there in operand order: its pieces of K
// and V lie lane by lane, a token's scales are the same for 16 lanes.
template <int D, int GS>
struct Slot {
    static constexpr int S = D / 32, G = D / GS;
    static constexpr int kCodes = 4 * D;               // words of 32 tokens' codes
    static constexpr int kSb = 32 * G;                 // words of their scales and biases
    static constexpr int kV = kCodes, kKs = 2 * kCodes, kVs = 2 * kCodes + kSb;
    static constexpr int kWords = 2 * kCodes + 2 * kSb;
    static constexpr int kCodeLoads = D / 64;          // 1 KiB each, for K and for V
    static constexpr int kSbLoads = G == 8 ? 2 : 1;    // 16 G lanes of 16 bytes
    static constexpr int kLoads = 2 * kCodeLoads + kSbLoads;
};

// Starts the loads of the step at `slot` tokens into record rec.
template <int D, int GS, bool NT>
__device__ __forceinline__ void load_step(const uint32_t* rec, const Record& r, int slot, int lane, uint32_t lds) {
    using L = Slot<D, GS>;
    constexpr int G = L::G;
#pragma unroll
    for (int c = 0; c < L::kCodeLoads; ++c)
        mf::dma16<NT>(rec + r.k_codes() + slot * (D / 8), 1024 * c + 16 * lane, lds + 1024 * c);
#pragma unroll
    for (int c = 0; c < L::kCodeLoads; ++c)
        mf::dma16<NT>(rec + r.v_codes() + slot * (D / 8), 1024 * c + 16 * lane, lds + 4 * L::kV + 1024 * c);
    if constexpr (G == 8) {
        mf::dma16<NT>(rec + r.k_sb() + slot * G, 16 * lane, lds + 4 * L::kKs);
        mf::dma16<NT>(rec + r.v_sb() + slot * G, 16 * lane, lds + 4 * L::kVs);
    } else {
        // K's in the first 8 G lanes, V's in the next
        const uint32_t at = lane < 8 * G ? 16 * lane : 16 * lane + 4 * (r.v_sb() - r.k_sb()) - 128 * G;
        if (lane < 16 * G) mf::dma16<NT>(rec + r.k_sb() + slot * G, at, lds + 4 * L::kKs);
    }
}

// An operand of a value per group and lane (16 i, 4 j lanes), and its product:
// 4 slots a lane are enough for up to 4 groups, and take half the registers.
template <int G>
struct Sums {
    uint32_t v[G == 8 ? 4 : 2];
};
template <int DT, int G>
__device__ __forceinline__ float4_t mfma_sums(const Sums<G>& a, const Sums<G>& b) {
    const float4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (G == 8) {
        return mf::mfma<DT>(__builtin_bit_cast(Frag, a), __builtin_bit_cast(Frag, b), zero);
    } else if constexpr (DT == DT_F16) {
        typedef _Float16 half4_t __attribute__((ext_vector_type(4)));
        return __builtin_amdgcn_mfma_f32_16x16x16f16(__builtin_bit_cast(half4_t, a), __builtin_bit_cast(half4_t, b), zero, 0, 0, 0);
    } else {
        typedef short short4_t __attribute__((ext_vector_type(4)));
        return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(short4_t, a), __builtin_bit_cast(short4_t, b), zero, 0, 0, 0);
    }
}

// Heads of 256 in groups of 32: the Q operands lie in LDS behind the slots, a
// lane's 16 bytes of each side by side (8 KiB a wavefront).  Their registers
// would have to be spilled, and a wait for a spilled one is a wait for the next
// step's tokens as well.
template <int D, int GS>
constexpr bool kQInLds = D / GS == 8;

// State of one tile of 16 rows.
template <int D, int GS>
struct RowTile {
    static constexpr int S = D / 32, G = D / GS, NT = D / 16;
    Frag q[S];        // Q^T operand
    Sums<G> qs;       // sums of the groups' q, times kQsUnit, in three pieces: group g of lane j, piece j; j = 3: what is lost
    float cs;         // score -> log2 units
    float ref, l;     // R; this lane's share of the sum of p
    float4_t zb;      // sums p b (rows 0..7: group; 7: of p alone, where there are fewer) and p s (rows 8..15)
    float zp;         // 8 groups: this lane's share of the sum of p as zb has it
    float4_t z[G];    // lanes j = 0, 1: sum P'; 2, 3: 4 j + r times it, as a code
    float4_t o[NT];
};

// The new tokens (bits) that a row sees under a window: it keeps the last
// `window` of the tokens it sees and those before position `sinks`.  low: the
// first token before the new ones that it sees, from there (0 or less).
__device__ __forceinline__ uint64_t window_bits(uint64_t bits, const NewTokens& nt, int window, int sinks, int& low) {
    // (bits that name no token do not count)
    if (nt.n < 64) bits &= (uint64_t{1} << nt.n) - 1;
    const int pos0 = nt.pos0;
    if (pos0 < 0) bits = pos0 > -64 ? bits >> -pos0 << -pos0 : 0;
    const int count = __builtin_popcountll(bits);
    low = count < window ? count - window : 0;
    uint64_t last = bits;
    for (int n = count - window; n > 0; --n) last &= last - 1;  // (at most 63 rounds)
    const int first = sinks - pos0;  // new tokens that are sinks
    const uint64_t firsts = first <= 0 ? 0 : first >= 64 ? ~uint64_t{0} : (uint64_t{1} << first) - 1;
    return last | (bits & firsts);
}

// What only some steps need of a row, in LDS.
struct __attribute__((aligned(16))) RowInfo {
    uint32_t seen[2];  // bits: new tokens that the row sees
    uint32_t exps[2];  // e of each group, a byte each
};
static_assert(sizeof(RowInfo) == 16, "behind the slots in LDS");

// Unit of the sums of q as an operand.  Scores are in units of 2^-24 q; fp16
// cannot hold the sums' low bits there (2^-25 would be half a unit of a q
// scaled to 2^15), so they are brought to 2^-9 and their product scaled.
template <int DT>
constexpr float kQsUnit = DT == DT_F16 ? 0x1p-9f : 0x1p-24f;

// Scores may pass R by 11, and scales be up to 2^4 where e is 0, so that P' stays
// below 2^15.
constexpr float kScoreRoom = 11.0f, kScaleRoom = 0x1p4f;
constexpr int kMostSize = 15;
constexpr float kFarScore = 0x1p20f;
// What fp32 sums of p b and p s are to stay below, log2 (bf16 values may be of any size).
constexpr float kMostSum = 100.0f;
// e where the row saw no scale but 0 in the group yet.
constexpr int kNoExp = 127;

__device__ __forceinline__ int exp_of(const RowInfo& info, int g) {
    return static_cast<int>(info.exps[g / 4] << (24 - 8 * (g % 4))) >> 24;
}
// 0 where there is none.
__device__ __forceinline__ int factor_of(const RowInfo& info, int g) {
    const int e = exp_of(info, g);
    return e == kNoExp ? 0 : e;
}
// A difference of references as an exponent.
__device__ __forceinline__ int exp_int(float x) { return static_cast<int>(fminf(fmaxf(x, -300.0f), 300.0f)); }

// 1 as DT, twice.
template <int DT>
constexpr uint32_t kOnes = DT == DT_F16 ? 0x3C003C00u : 0x3F803F80u;

// One value as DT's bits, nearest.
template <int DT>
__device__ __forceinline__ uint32_t bits_of(float f) {
    return DtOps<DT>::rne(f);
}
// Two values as DT's halves, nearest.
template <int DT>
__device__ __forceinline__ uint32_t pack_dt(float lo, float hi) {
    typedef float float2_t __attribute__((ext_vector_type(2)));
    if constexpr (DT == DT_F16) {
        return pack_f16(lo, hi);
    } else {
        typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((float2_t{lo, hi}), bf16x2_t));
    }
}

// Row tile's Q from its words w: values of row i, d = 32 s + 8 j + e.
template <int DT, int D, int GS>
__device__ __forceinline__ void make_q(RowTile<D, GS>& t, const uint32_t (&w)[D / 32][4], float scale, int i, int j) {
    constexpr int S = D / 32, G = D / GS;
    float f[S][8];
    float top = 0.0f;
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f[s][e] = half_f32<DT>(w[s][e / 2], e & 1);
            top = fmaxf(top, fabsf(f[s][e]));
        }
    }
    top = max_j(top);
    // 2^k: the row's largest value comes to [2^14, 2^15)
    int k = top > 0.0f ? 15 - __builtin_amdgcn_frexp_expf(top) : 0;
    k = k < -90 ? -90 : k > 120 ? 120 : k;
    // (odd d meet codes that count 16 times)
    const float up[2] = {__builtin_ldexpf(scale < 0.0f ? -1.0f : 1.0f, k), __builtin_ldexpf(scale < 0.0f ? -1.0f : 1.0f, k - 4)};
    float sums[G];
#pragma unroll
    for (int g = 0; g < G; ++g) sums[g] = 0.0f;
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[32 * s / GS] += f[s][e];
#pragma unroll
        for (int e = 0; e < 4; ++e) t.q[s].v[e] = pack_f16(f[s][e] * up[e & 1], f[s][e + 4] * up[e & 1]);
    }
    t.qs = Sums<G>{};
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const float sum = sum_j(sums[g]) * up[0], x = sum * kQsUnit<DT>;
        // three pieces of 11 or 8 bits, exact up to 2^-24 of x (fp16: 2^-25, 2^-31 of the row's largest q)
        const uint32_t h0 = bits_of<DT>(x);
        const float r1 = x - DtOps<DT>::to_f32(static_cast<uint16_t>(h0));
        const uint32_t h1 = bits_of<DT>(r1);
        const uint32_t h2 = bits_of<DT>(r1 - DtOps<DT>::to_f32(static_cast<uint16_t>(h1)));
        // what the codes' products with this q lose to the cut (rows of codes 8..15, against 11.5 times the sum)
        const Frag codes = codes8(0x11111111u * (8 + i % 8));
        float4_t cut = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = g * (GS / 32); s < (g + 1) * (GS / 32); ++s) cut = mf::mfma<DT_F16>(codes, t.q[s], cut);
        const float lost = 0x1p-24f * 11.5f * sum - 0.0625f * sum_j(cut[0] + cut[1] + cut[2] + cut[3]);
        const uint32_t h = j == 0 ? h0 : j == 1 ? h1 : j == 2 ? h2 : bits_of<DT>(lost * (0x1p24f * kQsUnit<DT>));
        t.qs.v[g / 2] |= h << (16 * (g & 1));
    }
    // log2(e) * |scale| * 2^24 / 2^k
    t.cs = __builtin_ldexpf(fabsf(scale) * 1.44269504088896f, 24 - k);
}

// Zero the halves of token pairs (0, 1) and (2, 3) of a bundle that has n tokens.
__device__ __forceinline__ void keep_tokens(uint32_t& w01, uint32_t& w23, int n) {
    w01 &= n >= 2 ? ~0u : n == 1 ? 0xFFFFu : 0u;
    w23 &= n >= 4 ? ~0u : n == 3 ? 0xFFFFu : 0u;
}

// Two halves, 0 for those that are infinite or NaN.
template <int DT>
__device__ __forceinline__ uint32_t finite_halves(uint32_t w) {
    constexpr uint32_t top = DT == DT_F16 ? 0x7C00u : 0x7F80u;
    if ((w & top) == top) w &= 0xFFFF0000u;
    if (((w >> 16) & top) == top) w &= 0xFFFFu;
    return w;
}

// Issue priority of the wavefront.  The matrix products go first, so that a
// SIMD's two wavefronts do not do their softmax at the same time; between
// them the younger wavefront (`late`) goes first, which otherwise falls behind
// and is left without another to hide its waits.  (64 rows over 16k tokens
// 121 us, 128 without; 32 sequences of 1k..4k 25.4, 27.4; verify rows over 8k
// 41.5, 42.7.)
__device__ __forceinline__ void priority_products() { __builtin_amdgcn_s_setprio(2); }
__device__ __forceinline__ void priority_rest(bool late) {
    if (late) __builtin_amdgcn_s_setprio(1);
    else __builtin_amdgcn_s_setprio(0);
}

// A step is 32 tokens against the row tiles, in two halves.  EDGE: `first` is
// the place of the step's first token among the new ones (negative: before
// them), `left` how many tokens of the step there are (slots past them may hold
// anything: their scales and biases of V are taken as 0).

// The pair (for 8 groups: pairs n = 0, 1) of V's scales that a lane looks at for
// the step; `none` stands for tokens past the end.
template <int D, int GS, bool EDGE>
__device__ __forceinline__ uint32_t scale_pair(const uint32_t* x, int lane, int n, int left, uint32_t none) {
    using L = Slot<D, GS>;
    constexpr int G = L::G;
    const int at = (lane + 64 * n) % (16 * G);  // (bundle, group), pair
    uint32_t w = x[L::kVs + (at >> 1) * 4 + (at & 1)];
    if constexpr (EDGE) {
        const int tokens = left - (at >> 1) / G * 4 - 2 * (at & 1);
        const uint32_t keep = tokens >= 2 ? ~0u : tokens == 1 ? 0xFFFFu : 0u;
        w = (w & keep) | (none & ~keep);
    }
    return w;
}

// WINDOW: sinks, counted as first; lows: what window_bits found for each row.
// The scores, in units 1 / cs; see: which tokens the lane's row sees (EDGE);
// most: the lane's largest of those.  Returns whether a reference may have to
// be moved, or a scale is one that e of 0 have no room for.
template <int DT, int D, int GS, int RT, bool EDGE, bool WINDOW>
__device__ __forceinline__ bool step_scores(const uint32_t* x, const RowTile<D, GS> (&rows)[RT], const RowInfo* info, const int* lows,
                                            const Frag* q, float (&sc)[RT][2][4], bool (&see)[RT][2][4], float (&most)[RT], int lane,
                                            int first, int sinks, int left, bool late) {
    using L = Slot<D, GS>;
    constexpr int S = D / 32, G = D / GS;
    const int i = lane % 16, j = lane / 16;
    const float4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};

    float big = 0.0f;
#pragma unroll
    for (int n = 0; n < (G == 8 ? 2 : 1); ++n) {
        const uint32_t w = scale_pair<D, GS, EDGE>(x, lane, n, left, 0);
        big = fmaxf(big, fmaxf(half_f32<DT>(w, 0), half_f32<DT>(w, 1)));
    }

    priority_products();
    // scores of all row tiles: sum_g b (sum of q) and s (what the codes' products lose) from the matrix core, + s (codes . q)
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        uint32_t k[S];
        load_words<S>(x + t * (L::kCodes / 2) + (4 * i + j) * S, k);
        Sums<G> kb{};
        const uint16_t* hb = reinterpret_cast<const uint16_t*>(x + L::kKs) + ((4 * t + i / 4) * G) * 8 + (j < 3 ? 4 : 0) + i % 4;
#pragma unroll
        for (int g = 0; g < G; ++g) kb.v[g / 2] |= static_cast<uint32_t>(hb[8 * g]) << (16 * (g & 1));
        float4_t acc[RT];
#pragma unroll
        for (int u = 0; u < RT; ++u) acc[u] = mfma_sums<DT>(kb, rows[u].qs);
#pragma unroll
        for (int u = 0; u < RT; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) sc[u][t][r] = DT == DT_F16 ? acc[u][r] * (0x1p-24f / kQsUnit<DT>) : acc[u][r];
        constexpr int GB = G == 8 ? 4 : G;  // (8 groups: four at a time, for the registers)
#pragma unroll
        for (int g0 = 0; g0 < G; g0 += GB) {
            float4_t p[RT][GB];
#pragma unroll
            for (int s = g0 * GS / 32; s < (g0 + GB) * GS / 32; ++s) {
                const Frag a = codes8(k[s]);
                const int g = 32 * s / GS - g0;
#pragma unroll
                for (int u = 0; u < RT; ++u) {
                    Frag b = rows[u].q[s];
                    if constexpr (kQInLds<D, GS>) load_words<4>(q[64 * s + lane].v, b.v);
                    if (32 * s % GS == 0) p[u][g] = mf::mfma<DT_F16>(a, b, zero);
                    else p[u][g] = mf::mfma<DT_F16>(a, b, p[u][g]);
                }
            }
#pragma unroll
            for (int g = 0; g < GB; ++g) {
                uint32_t w[2];
                load_words<2>(x + L::kKs + ((4 * t + j) * G + g0 + g) * 4, w);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float ks = half_f32<DT>(w[r / 2], r & 1);
#pragma unroll
                    for (int u = 0; u < RT; ++u) sc[u][t][r] = __builtin_fmaf(ks, p[u][g][r], sc[u][t][r]);
                }
            }
            if constexpr (GB < G) __builtin_amdgcn_sched_barrier(0);
        }
    }
    priority_rest(late);
    bool move = big >= kScaleRoom;
#pragma unroll
    for (int u = 0; u < RT; ++u) {
        float mx = kFar;
        uint64_t bits = 0;
        if constexpr (EDGE) bits = info[16 * u + i].seen[0] | static_cast<uint64_t>(info[16 * u + i].seen[1]) << 32;
        int low = 0;
        if constexpr (EDGE && WINDOW) low = lows[16 * u + i];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                see[u][t][r] = true;
                if constexpr (EDGE) {
                    const int at = 16 * t + 4 * j + r, n = first + at;
                    if constexpr (WINDOW)
                        see[u][t][r] = at < left && (n < 0 ? n >= low || n < sinks : ((bits >> (n & 63)) & 1) != 0);
                    else
                        see[u][t][r] = at < left && (n < 0 || ((bits >> (n & 63)) & 1) != 0);
                }
                mx = fmaxf(mx, see[u][t][r] ? sc[u][t][r] : kFar);
            }
        most[u] = mx;
        move = move || mx * rows[u].cs > rows[u].ref + kScoreRoom;
    }
    return move;
}

// Whether all scales of the step lie in 2^-9..2^4: e that are 0 then stay so;
// and no score is one that p_of minds.
// (A row's largest p where R was just moved is in 2^5..2^6, so its largest p s
// lies in 2^-4..2^10; else p s is below 2^15.)
template <int DT, int D, int GS, int RT, bool EDGE>
__device__ __forceinline__ bool is_calm(const uint32_t* x, const RowTile<D, GS> (&rows)[RT], const float (&most)[RT],
                                        int lane, int left) {
    constexpr int G = D / GS;
    bool calm = true;
#pragma unroll
    for (int u = 0; u < RT; ++u) calm = calm && (most[u] == kFar || fabsf(most[u] * rows[u].cs) < kFarScore);
#pragma unroll
    for (int n = 0; n < (G == 8 ? 2 : 1); ++n) {
        const uint32_t w = scale_pair<D, GS, EDGE>(x, lane, n, left, kOnes<DT>);
#pragma unroll
        for (int h = 0; h < 2; ++h) calm = calm && half_f32<DT>(w, h) >= 0x1p-9f && half_f32<DT>(w, h) < kScaleRoom;
    }
    return __all(calm);
}

// p of a score.  Beyond 2^21 a score is rounded as R was: exactly, the product
// may lie more above R than fp16 holds.
template <bool FAR>
__device__ __forceinline__ float p_of(float score, float cs, float ref) {
#pragma clang fp contract(off)
    float x = __builtin_fmaf(score, cs, -ref);
    if constexpr (FAR) {
        const float rounded = score * cs;
        x = fabsf(ref) < 2.0f * kFarScore ? x : rounded - ref;  // (an R of the fast form is always below)
    }
    return exp2_fast(x);
}

// R of a row whose largest score in the step is `high`.
__device__ __forceinline__ float moved_ref(float from, float high) {
    return high - from > kScoreRoom ? __builtin_ceilf(high) - 6.0f : from;
}

// Moves R in a calm step, where all sums of a row scale alike.
template <int D, int GS, int RT>
__device__ __forceinline__ void move_calm(RowTile<D, GS> (&rows)[RT], const float (&most)[RT]) {
    constexpr int G = D / GS, NT = D / 16;
#pragma unroll
    for (int u = 0; u < RT; ++u) {
        const float ref = moved_ref(rows[u].ref, max_j(most[u] > kFar ? most[u] * rows[u].cs : -__builtin_inff()));
        const float f = __builtin_ldexpf(1.0f, exp_int(rows[u].ref - ref));
        rows[u].ref = ref;
        rows[u].l *= f;
#pragma unroll
        for (int r = 0; r < 4; ++r) rows[u].zb[r] *= f;
        if constexpr (G == 8) rows[u].zp *= f;
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int r = 0; r < 4; ++r) rows[u].z[g][r] *= f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) rows[u].o[n][r] *= f;
    }
}

// Moves R and the e of one tile as the step's scores and scales ask for.  What
// they become depends on what the row sees and on nothing else.
template <int DT, int D, int GS>
__device__ __forceinline__ void move_exact(const uint32_t* x, RowTile<D, GS>& t, RowInfo* info, const float (&sc)[2][4],
                                           const bool (&see)[2][4], float most, int lane, int left) {
    using L = Slot<D, GS>;
    constexpr int G = D / GS;
    const int i = lane % 16, j = lane / 16;
    RowInfo mine = info[i];
    const float from = t.ref;
    t.ref = moved_ref(from, max_j(most > kFar ? most * t.cs : -__builtin_inff()));
    if constexpr (DT == DT_BF16) {
        // p times the token's largest bias or 8 scales is to stay below 2^kMostSum: the sums are fp32's (fp16's cannot pass it)
        float size[2][4], all = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int r = 0; r < 4; ++r) size[h][r] = 0.0f;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                uint32_t w[4];
                load_words<4>(x + L::kVs + ((4 * h + j) * G + g) * 4, w);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float s = half_f32<DT>(finite_halves<DT>(w[r / 2]), r & 1), b = half_f32<DT>(finite_halves<DT>(w[2 + r / 2]), r & 1);
                    size[h][r] = fmaxf(size[h][r], fmaxf(0.125f * fabsf(b), s));
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (!see[h][r]) size[h][r] = 0.0f;
                all = fmaxf(all, size[h][r]);
            }
        }
        if (__any(all > 0x1p64f)) {
            float high = -__builtin_inff();
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (size[h][r] > 0x1p64f) high = fmaxf(high, __builtin_fmaf(sc[h][r], t.cs, __builtin_amdgcn_logf(size[h][r]) + (3.0f - kMostSum)));
            t.ref = fmaxf(t.ref, __builtin_ceilf(max_j(high)));
        }
    }
    const bool up = t.ref != from;
    const int raised = exp_int(t.ref - from);
    t.l = __builtin_ldexpf(t.l, -raised);
#pragma unroll
    for (int r = 0; r < 4; ++r) t.zb[r] = __builtin_ldexpf(t.zb[r], -raised);
    if constexpr (G == 8) t.zp = __builtin_ldexpf(t.zp, -raised);
    float p[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            p[h][r] = see[h][r] ? p_of<true>(sc[h][r], t.cs, t.ref) : 0.0f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        // the largest p s of the row and group (infinite scales count as none)
        float ps = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t w[2];
            load_words<2>(x + L::kVs + ((4 * h + j) * G + g) * 4, w);
            keep_tokens(w[0], w[1], left - (16 * h + 4 * j));
            w[0] = finite_halves<DT>(w[0]);
            w[1] = finite_halves<DT>(w[1]);
#pragma unroll
            for (int r = 0; r < 4; ++r) ps = fmaxf(ps, p[h][r] * half_f32<DT>(w[r / 2], r & 1));
        }
        ps = max_j(ps);
        const int size = __builtin_amdgcn_frexp_expf(ps);  // 2^(size - 1) <= ps < 2^size
        const bool none = from == kFar || exp_of(mine, g) == kNoExp;
        const int kept = exp_of(mine, g) + raised;  // with P' as it was
        int to = none ? kNoExp : kept < 100 ? kept : 100;
        if (ps > 0.0f && (up || none || size + kept > kMostSize)) {
            to = size > 10 || size < -3 ? 3 - size : 0;
            if (!none && to > 0) to = to < kept ? to : kept > 0 ? kept : 0;  // (the row saw larger ones before)
            to = to < -126 ? -126 : to > 100 ? 100 : to;
        }
        const int scaled = none ? 0 : to - kept;
#pragma unroll
        for (int r = 0; r < 4; ++r) t.z[g][r] = __builtin_ldexpf(t.z[g][r], scaled);
#pragma unroll
        for (int n = g * (GS / 16); n < (g + 1) * (GS / 16); ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) t.o[n][r] = __builtin_ldexpf(t.o[n][r], scaled);
        const int at = 8 * (g % 4);
        mine.exps[g / 4] = (mine.exps[g / 4] & ~(0xFFu << at)) | (static_cast<uint32_t>(to & 0xFF) << at);
        __builtin_amdgcn_sched_barrier(0);
    }
    if (j == 0) info[i] = mine;
}

// p from the scores, its sums, P' and the second product.  PLAIN: all e are 0.
template <int DT, int D, int GS, int RT, bool EDGE, bool PLAIN>
__device__ __forceinline__ void step_values(const uint32_t* x, RowTile<D, GS> (&rows)[RT], const RowInfo* info,
                                            float (&sc)[RT][2][4], const bool (&see)[RT][2][4], int lane, int left,
                                            bool late) {
    using L = Slot<D, GS>;
    constexpr int S = D / 32, G = D / GS, C = D / 64;
    const int i = lane % 16, j = lane / 16;
    // p, its sum, and p as an operand
    Frag p16[RT];
#pragma unroll
    for (int u = 0; u < RT; ++u) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float p = p_of<!PLAIN>(sc[u][t][r], rows[u].cs, rows[u].ref);
                if constexpr (EDGE) p = see[u][t][r] ? p : 0.0f;
                sc[u][t][r] = p;
                rows[u].l += p;
            }
            p16[u].v[2 * t] = pack_dt<DT>(sc[u][t][0], sc[u][t][1]);
            p16[u].v[2 * t + 1] = pack_dt<DT>(sc[u][t][2], sc[u][t][3]);
        }
    }
    // sums of p b and p s, raw scales and biases as the operand: row i < 8 is
    // the bias of group i mod G, row 8 + i its scale.  p is rounded to the type
    // here (8 bits for bf16), so the sum of the same rounded p is kept beside
    // them (row 7, a group's double where G < 8): the mean of the middles
    // b + 7.5 s is theirs over that, and the rounding is weighed by what they
    // differ by, not by what they are.  Rows may not see a token whose values are infinite or
    // NaN: its scale and bias are left out here, and the rows that do see it
    // have them from P' (a bias is finite where the scale is).
    {
        Frag sb;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            uint32_t w[2];
            load_words<2>(x + L::kVs + ((4 * t + j) * G + i % G) * 4 + (i < 8 ? 2 : 0), w);
            if constexpr (EDGE) {
                keep_tokens(w[0], w[1], left - (16 * t + 4 * j));
                w[0] = finite_halves<DT>(w[0]);
                w[1] = finite_halves<DT>(w[1]);
            }
            sb.v[2 * t] = G < 8 && i == 7 ? kOnes<DT> : w[0];
            sb.v[2 * t + 1] = G < 8 && i == 7 ? kOnes<DT> : w[1];
        }
#pragma unroll
        for (int u = 0; u < RT; ++u) rows[u].zb = mf::mfma<DT>(sb, p16[u], rows[u].zb);
        if constexpr (G == 8)
#pragma unroll
            for (int u = 0; u < RT; ++u)
#pragma unroll
                for (int k = 0; k < 4; ++k) rows[u].zp += half_f32<DT>(p16[u].v[k], 0) + half_f32<DT>(p16[u].v[k], 1);
    }
    priority_products();
    // P' and the second product: tile n = 4 c + q of 16 d, from nibble q of the words of quad c
    // (rows 0..7 of the constant: 1, rows 8..15: the codes 8..15)
    Frag ones;
    ones.v[0] = ones.v[1] = ones.v[2] = ones.v[3] = i < 8 ? 0x3C003C00u : 0x00010001u * i;
    uint32_t v[2][S];
#pragma unroll
    for (int t = 0; t < 2; ++t) load_words<S>(x + L::kV + t * (L::kCodes / 2) + 16 * S * j + S * i, v[t]);
#pragma unroll
    for (int g = 0; g < G; ++g) {
        Frag pp[RT];
        if constexpr (!PLAIN) {  // p by this group's 2^e, from the one before's (what falls below fp32 is 2^-26 of the largest p)
#pragma unroll
            for (int u = 0; u < RT; ++u) {
                const RowInfo& mine = info[16 * u + i];
                const int by = factor_of(mine, g) - (g > 0 ? factor_of(mine, g - 1) : 0);
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) sc[u][t][r] = __builtin_ldexpf(sc[u][t][r], by);
            }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            uint32_t w[2];
            load_words<2>(x + L::kVs + ((4 * t + j) * G + g) * 4, w);
            if constexpr (EDGE) keep_tokens(w[0], w[1], left - (16 * t + 4 * j));
            float s[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) s[r] = half_f32<DT>(w[r / 2], r & 1);
#pragma unroll
            for (int u = 0; u < RT; ++u) {
                float ps[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    ps[r] = sc[u][t][r] * s[r];
                    if constexpr (EDGE) ps[r] = see[u][t][r] ? ps[r] : 0.0f;  // (s may be infinite)
                }
                pp[u].v[2 * t] = pack_f16(ps[0], ps[1]);
                pp[u].v[2 * t + 1] = pack_f16(ps[2], ps[3]);
            }
        }
#pragma unroll
        for (int u = 0; u < RT; ++u) rows[u].z[g] = mf::mfma<DT_F16>(ones, pp[u], rows[u].z[g]);
#pragma unroll
        for (int n = g * (GS / 16); n < (g + 1) * (GS / 16); ++n) {
            const int c = n / 4, q = n % 4;
            Frag a;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t w = v[k / 2][(k & 1) * C + c];
                a.v[k] = (q < 2 ? w : w >> 8) & ((q & 1) ? 0x00F000F0u : 0x000F000Fu);
            }
#pragma unroll
            for (int u = 0; u < RT; ++u) rows[u].o[n] = mf::mfma<DT_F16>(a, pp[u], rows[u].o[n]);
        }
    }
    priority_rest(late);
}

// Puts the sums of `parts` parts, the first at byte `at0` and `stride` bytes
// apart, together for `valid` rows.  An item is four values of a row,
// consecutive threads take consecutive items; where items are fewer than
// threads, `share` groups of threads take every share-th part and meet in
// LDS.  A thread has the values of NI items * NP parts in flight, for the
// latency of a read from another XCD's stores is what this costs: 64 parts of
// 4 rows about 4 us.  (A launch of its own for it would cost as much again.)
template <int D, int RT, int W, int NI, int NP, class Finish>
__device__ __forceinline__ void join_parts(Shared sums, uint32_t at0, uint32_t stride, int parts, int valid,
                                           float* lds, Finish finish) {
    constexpr int Q4 = D / 4, kThreads = 64 * W;
    const int items = valid * Q4;
    int share = 1;
    while (2 * share * items <= kThreads && share < 8) share *= 2;
    const int per = kThreads / share, mine = threadIdx.x / per;  // (per: a power of two, at least items where share > 1)
    for (int it0 = threadIdx.x % per; it0 < items; it0 += NI * per) {
        float ref[NI], l[NI], o[NI][4];
#pragma unroll
        for (int n = 0; n < NI; ++n) {
            ref[n] = kFar;
            l[n] = o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
        }
        for (int k0 = mine; k0 < parts; k0 += share * NP) {
            float2 s[NI][NP];
            float4_t v[NI][NP];
#pragma unroll
            for (int n = 0; n < NI; ++n)
#pragma unroll
                for (int m = 0; m < NP; ++m) {
                    // (no branch around a load, which would wait for it: past the end the last one again)
                    const int it = it0 + n * per < items ? it0 + n * per : items - 1;
                    const int k = k0 + m * share < parts ? k0 + m * share : parts - 1;
                    const uint32_t at = at0 + k * stride;
                    const float4_t rl = load_shared(sums, at + 4 * (16 * RT * D + 4 * (it / Q4)));
                    s[n][m] = make_float2(rl[0], rl[1]);
                    v[n][m] = load_shared(sums, at + 16 * it);
                }
#pragma unroll
            for (int n = 0; n < NI; ++n)
#pragma unroll
                for (int m = 0; m < NP; ++m)
                    if (k0 + m * share >= parts) s[n][m] = make_float2(kFar, 0.0f);
#pragma unroll
            for (int n = 0; n < NI; ++n) {
                float top = ref[n];
#pragma unroll
                for (int m = 0; m < NP; ++m) top = fmaxf(top, s[n][m].x);
                const float f0 = exp2_fast(ref[n] - top);
                l[n] *= f0;
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][e] *= f0;
#pragma unroll
                for (int m = 0; m < NP; ++m) {
                    const float f = s[n][m].y != 0.0f ? exp2_fast(s[n][m].x - top) : 0.0f;
                    l[n] = __builtin_fmaf(f, s[n][m].y, l[n]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[n][e] = __builtin_fmaf(f, v[n][m][e], o[n][e]);
                }
                ref[n] = top;
            }
        }
        if (share == 1) {
#pragma unroll
            for (int n = 0; n < NI; ++n) {
                const int it = it0 + n * per;
                if (it < items) finish(it / Q4, it % Q4 * 4, o[n], ref[n], l[n]);
            }
        } else {  // one item a thread: items <= per
            float* p = lds + (mine * per + it0) * 6;
            p[0] = ref[0];
            p[1] = l[0];
#pragma unroll
            for (int e = 0; e < 4; ++e) p[2 + e] = o[0][e];
        }
    }
    if (share > 1) {
        __syncthreads();
        if (static_cast<int>(threadIdx.x) < items) {
            float ref = kFar, l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int k = 0; k < share; ++k) ref = fmaxf(ref, lds[(k * per + threadIdx.x) * 6]);
            for (int k = 0; k < share; ++k) {
                const float* p = lds + (k * per + threadIdx.x) * 6;
                const float f = exp2_fast(p[0] - ref);
                l = __builtin_fmaf(f, p[1], l);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = __builtin_fmaf(f, p[2 + e], o[e]);
            }
            finish(threadIdx.x / Q4, threadIdx.x % Q4 * 4, o, ref, l);
        }
    }
}

}  // namespace

// One workgroup: one part of one sequence and kv head against the rows of row
// group blockIdx.y (row = new token * group + head within the group).
//
// Measured (bf16 or fp16, 32 heads, 8 kv heads of 128, groups of 64 unless
// said): one token over 777 tokens 10.1 us, 32 sequences of 1k..4k 25.3 us
// (3.8 TB/s; 13.7 us of reading), 16 sequences of 4..6 rows over 8k 41.7 us
// (3.6 TB/s; 21.6), one token over 131071 30.7 us (4.6 TB/s; 20.6), 64 rows of
// 4 sequences over 16k 121 us (542 TFLOP/s; 54; 111 in a row of calls); 8 trees
// of 13 rows, 16 heads of 64, up to 2k 12.6 us.  With a window: of 4096 and 4
// sinks, one token at 131071, 13.9 us; of 1023 and 4, 16 sequences of 4..6 rows
// near 8k, 22 us; of 4096 and 64, 64 rows of 4 sequences near 16k, 48 us (366
// TFLOP/s; 14; 43 in a row of calls): an eighth to a sixth more than over as many
// tokens without one (qmm_kv_window.hpp).  A call starts (lengths, plan,
// q, page ids, first tokens) in 3 to 4 us and joins its parts in about 4;
// between them one row tile is bound by its reads (6 TB/s over 131071 tokens).
// With two no unit is full: vector ALUs 52 % busy (verify rows) and 63 % (64
// rows), matrix cores 18 % and 28 %; of the wavefronts' time, two a SIMD,
// 49 % and 51 % goes to instructions, 30 % and 23 % to waits for data, 21 %
// and 26 % to waits for a unit.
template <int DT, int D, int GS, int RT, bool ROWS, bool NT_LOADS, bool WINDOW>
__global__ __launch_bounds__(64 * attend_waves(RT, ROWS), attend_occupancy(D, RT)) void attend_kernel(AttendParams a) {
    constexpr int kAttendWaves = attend_waves(RT, ROWS), kTiles = attend_tiles(RT, ROWS);
    using L = Slot<D, GS>;
    constexpr int G = D / GS, NT = D / 16;
    constexpr int DC = D < 128 ? D : 128;      // values a row that go through LDS at a time
    constexpr int kRow = DC + 4;               // floats of a row there
    extern __shared__ __align__(16) uint32_t lds[];
    // the slots; at the end the wavefronts' sums
    float (*buf)[16 * kRow] = reinterpret_cast<float (*)[16 * kRow]>(lds);
    float (*stat)[RT][16][2] = reinterpret_cast<float (*)[RT][16][2]>(lds + kAttendWaves * 16 * kRow);
    const int lane = threadIdx.x % 64, i = lane % 16, j = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);

    // heads fastest; workgroups that read the same tokens (row groups, blockIdx.y) are a multiple of 8 apart: one XCD
    const uint32_t unit = blockIdx.x / static_cast<uint32_t>(a.s.kv_heads);
    const int head = static_cast<int>(blockIdx.x - unit * a.s.kv_heads), rg = blockIdx.y;
    const Part part = find_part<WINDOW>(a.s, static_cast<int>(unit), a.parts, lane, a.window, a.sinks, a.mask != nullptr);
    const int b = part.b;
    if (b < 0) return;
    const NewTokens nt = new_tokens(a.s, b);
    const int count = nt.n * static_cast<int>(a.group);
    const int base_row = rg * 16 * kTiles;
    if (base_row >= count) return;
    const int wave_row = base_row + (ROWS ? wave * 16 * RT : 0);  // the wavefront's first
    const int64_t cap = a.s.width << a.s.page_shift;
    Window win{};
    if constexpr (WINDOW) win = window_of(nt.pos0, nt.n, cap, a.window, a.sinks, a.mask != nullptr);
    const int len = WINDOW ? win.len : static_cast<int>(nt.pos0 + nt.n < cap ? nt.pos0 + nt.n : cap);
    // (positions are counted in the window's order up to where the record, or the place among the new tokens, counts)
    auto real = [&](int t) { return WINDOW ? win.real(t) : t; };
    const int t0 = part.first * kChunk;
    const int t1 = len - t0 > part.chunks * kChunk ? t0 + part.chunks * kChunk : len;

    const Record rec(1 << a.s.page_shift, D, GS);
    const int mask_slot = (1 << a.s.page_shift) - 1;
    // page ids of 64 columns of the table, one a lane
    int ids, col0;
    auto load_ids = [&](int col) {
        col0 = col;
        const int64_t c = col + lane;
        ids = c < a.s.width ? a.s.tables[static_cast<int64_t>(b) * a.s.width + c] : -1;
        if (ids >= a.s.pages) ids = -1;
    };
    load_ids(real(t0) >> a.s.page_shift);
    auto page_at = [&](int t) -> int {
        const int col = t >> a.s.page_shift;
        if (WINDOW ? static_cast<unsigned>(col - col0) >= 64 : col >= col0 + 64) load_ids(col);
        return __builtin_amdgcn_readlane(ids, col - col0);
    };
    // the rows of q, asked for together with the page ids; worked on while the first tokens come
    uint32_t qw[RT][D / 32][4];
    uint64_t bits[RT];
#pragma unroll
    for (int u = 0; u < RT; ++u) {
        const int row = wave_row + 16 * u + i;
        const bool have = row < count;
        const int tok = have ? static_cast<uint32_t>(row) / a.group : 0;
        const uint16_t* q = a.q + (nt.row0 + tok) * a.q_row +
                            (static_cast<int64_t>(head) * a.group + (have ? row - tok * static_cast<int>(a.group) : 0)) * a.q_head + 8 * j;
#pragma unroll
        for (int s = 0; s < D / 32; ++s) {
            load_words<4>(reinterpret_cast<const uint32_t*>(q + 32 * s), qw[u][s]);  // (no row: the first one's)
#pragma unroll
            for (int e = 0; e < 4; ++e) qw[u][s][e] = have ? qw[u][s][e] : 0;
        }
        bits[u] = !have ? 0 : a.mask != nullptr ? static_cast<uint64_t>(a.mask[nt.row0 + tok]) : ~uint64_t{0} >> (63 - tok);
        // (waited for here: behind the token loads the wait would be for those as well)
#pragma unroll
        for (int s = 0; s < D / 32; ++s)
            asm volatile("" : "+v"(qw[u][s][0]), "+v"(qw[u][s][1]), "+v"(qw[u][s][2]), "+v"(qw[u][s][3]));
        asm volatile("" : "+v"(bits[u]));
    }
    uint32_t* ring = lds + wave * (kAttendSlots * L::kWords);
    RowInfo* info = reinterpret_cast<RowInfo*>(lds + kAttendWaves * kAttendSlots * L::kWords) + wave * 16 * RT;
    Frag* q_lds = reinterpret_cast<Frag*>(lds + kAttendWaves * (kAttendSlots * L::kWords + 64 * RT)) + wave * 2 * D;
    int* lows = reinterpret_cast<int*>(lds) + kAttendWaves * (kAttendSlots * L::kWords + 64 * RT + (kQInLds<D, GS> ? 8 * D : 0)) + wave * 16 * RT;
    const uint32_t ring_at = lds_address(ring);
    constexpr int kStride = ROWS ? 32 : 32 * kAttendWaves;
    // a wavefront without rows (by rows) takes no steps
    const int t_first = ROWS ? (wave_row < count ? t0 : t1) : t0 + 32 * wave;
    // starts the loads of the step at token t; whether there are any
    auto fetch = [&](int t, int slot) -> bool {
        if (t >= t1) return false;
        const int at = real(t);
        const int page = page_at(at);
        if (page < 0) return false;
        const uint32_t* r = a.s.pool + (static_cast<int64_t>(page) * a.s.kv_heads + head) * rec.words();
        load_step<D, GS, NT_LOADS>(r, rec, at & mask_slot, lane, ring_at + 4 * slot * L::kWords);
        return true;
    };
    // steps in flight: slot n % kAttendSlots holds step n, `there` whether it has a page (bit 0: the next)
    unsigned there = 0;
    int slot = 0, t = t_first;
    auto start = [&] {
        there = 0;
        slot = 0;
        t = t_first;
#pragma unroll
        for (int n = 0; n < kAttendSlots - 1; ++n)
            there |= fetch(t_first + n * kStride, n) ? 1u << n : 0u;
    };
    start();
    RowTile<D, GS> rows[RT];
#pragma unroll
    for (int u = 0; u < RT; ++u) {
        make_q<DT, D, GS>(rows[u], qw[u], a.scale, i, j);
        if constexpr (kQInLds<D, GS>) {
#pragma unroll
            for (int s = 0; s < D / 32; ++s) q_lds[64 * s + lane] = rows[u].q[s];
        }
        if constexpr (WINDOW) {
            int low;
            bits[u] = window_bits(bits[u], nt, a.window, a.sinks, low);
            if (j == 0) lows[16 * u + i] = low;
        }
        if (j == 0) info[16 * u + i] = RowInfo{{static_cast<uint32_t>(bits[u]), static_cast<uint32_t>(bits[u] >> 32)}, {0, 0}};
    }
    auto clear = [&] {
#pragma unroll
        for (int u = 0; u < RT; ++u) {
            rows[u].ref = wave_row + 16 * u + i < count ? kFar : 0.0f;
            rows[u].l = 0.0f;
            rows[u].zp = 0.0f;
            rows[u].zb = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int g = 0; g < G; ++g) rows[u].z[g] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int n = 0; n < NT; ++n) rows[u].o[n] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
        }
    };
    clear();

    // the second of the wavefronts, or workgroups, that share a SIMD
    const bool late = kAttendWaves == 8 ? wave >= 4 : (blockIdx.x & 256) != 0;
    priority_rest(late);
    // starts the loads of the step after the one at t and waits for that one's; whether there is any
    auto begin = [&]() -> bool {
        // the slot that the step before this one was read from
        const int free_slot = slot == 0 ? kAttendSlots - 1 : slot - 1;
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        there |= fetch(t + (kAttendSlots - 1) * kStride, free_slot) ? 1u << (kAttendSlots - 1) : 0u;
        const bool have = there & 1;
        there >>= 1;
        if (have) {
            // this step's loads are done when only those of the steps after it are left
            const int after = __builtin_popcount(there);
            if (after == 0) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            else if (after == 1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(L::kLoads) : "memory");
            else asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * L::kLoads) : "memory");
        }
        return have;
    };
    auto next = [&] {
        slot = slot == kAttendSlots - 1 ? 0 : slot + 1;
        t += kStride;
    };
    int calm = 1;
    // the lane, and where registers are short, one that nothing worked out from it is kept for from step to step
    auto step_lane = [&]() -> int {
        int here = lane;
        if constexpr (RT * G >= 8) asm volatile("" : "+v"(here));
        return here;
    };
    auto turn = [&](auto edge) {
        constexpr bool EDGE = decltype(edge)::value;
        if (begin()) {
            const uint32_t* x = ring + slot * L::kWords;
            float sc[RT][2][4], most[RT];
            bool see[RT][2][4];
            const int here = step_lane();
            if (__any(step_scores<DT, D, GS, RT, EDGE, WINDOW>(x, rows, info, lows, q_lds, sc, see, most, here, real(t) - nt.pos0,
                                                               a.sinks - nt.pos0, t1 - t, late))) {
                if (is_calm<DT, D, GS, RT, EDGE>(x, rows, most, here, t1 - t)) move_calm(rows, most);
                else calm = 0;
            }
            if (calm != 0) step_values<DT, D, GS, RT, EDGE, true>(x, rows, info, sc, see, here, t1 - t, late);
        }
        next();
    };
    // tokens that every row sees, then the new ones and the end
    const int all_seen = WINDOW ? win.all : nt.pos0, seen = all_seen < t1 ? all_seen : t1;
    while (calm != 0 && t + 32 <= seen) turn(std::false_type{});
    while (calm != 0 && t < t1) turn(std::true_type{});
    if constexpr (DT == DT_BF16) {
        bool small = true;
#pragma unroll
        for (int u = 0; u < RT; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) small = small && fabsf(rows[u].zb[r]) < 0x1p99f;
        if (!__all(small)) calm = 0;
    }
    if (calm == 0) {
        // some values are of another size: all over, by the form that can tell
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");  // (no slot is written or read any more)
        load_ids(real(t0) >> a.s.page_shift);
        clear();
        start();
        while (t < t1) {
            if (begin()) {
                const uint32_t* x = ring + slot * L::kWords;
                float sc[RT][2][4], most[RT];
                bool see[RT][2][4];
                step_scores<DT, D, GS, RT, true, WINDOW>(x, rows, info, lows, q_lds, sc, see, most, lane, real(t) - nt.pos0,
                                                         a.sinks - nt.pos0, t1 - t, late);
#pragma unroll
                for (int u = 0; u < RT; ++u)
                    move_exact<DT, D, GS>(x, rows[u], info + 16 * u, sc[u], see[u], most[u], lane, t1 - t);
                step_values<DT, D, GS, RT, true, false>(x, rows, info, sc, see, lane, t1 - t, late);
            }
            next();
        }
    }
    int exps[RT][G];
#pragma unroll
    for (int u = 0; u < RT; ++u)
#pragma unroll
        for (int g = 0; g < G; ++g) exps[u][g] = factor_of(info[16 * u + i], g);
    if constexpr (!ROWS) __syncthreads();  // the slots become the sums' buffer

    // one set of sums: R and l first
    float middle[RT][G], centre[RT][G][2];
#pragma unroll
    for (int u = 0; u < RT; ++u) {
        rows[u].l = sum_j(rows[u].l);
        // l over the sum of the rounded p (row 7 of zb: lanes j = 1)
        const float rounded = G == 8 ? sum_j(rows[u].zp) : __shfl(rows[u].zb[3], i + 16);
        const float whole = rows[u].l / (rounded != 0.0f ? rounded : 1.0f);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            // sum p (b + 7.5 s) of group g, to p that add up to l: rows g and 8 + g of zb, in the lanes j = g / 4 and 2 + g / 4
            middle[u][g] = whole * (__shfl(rows[u].zb[g % 4], i + 16 * (g / 4)) + 7.5f * __shfl(rows[u].zb[g % 4], i + 16 * (2 + g / 4)));
            // what the sums of codes are centred by: odd codes by 7.5 sum P',
            // even ones by the mean of 8..15 times it, less 4 of it (2^-24 each)
            const float4_t z = rows[u].z[g];
            const float codes = z[0] + z[1] + z[2] + z[3], one = __shfl(z[0], i);
            centre[u][g][0] = 0.125f * (__shfl(codes, i + 32) + __shfl(codes, i + 48)) - 0x1p-22f * one;
            centre[u][g][1] = (7.5f * 0x1p-20f) * one;
        }
        if (!ROWS && j == 0) {
            stat[wave][u][i][0] = rows[u].l != 0.0f ? rows[u].ref : kFar;
            stat[wave][u][i][1] = rows[u].l;
        }
    }
    if constexpr (!ROWS) __syncthreads();
    uint32_t* done = a.done + kDoneStride * ((static_cast<int64_t>(b) * gridDim.y + rg) * a.s.kv_heads + head);
    const Shared sums = shared_of(a.sums);
    auto sums_at = [&](int slot) -> uint32_t {  // (all parts' sums are some tens of MB)
        return ((static_cast<uint32_t>(slot) * gridDim.y + rg) * a.s.kv_heads + head) * (4 * part_floats(D, RT));
    };
    constexpr int PER = DC * 16 / (64 * kAttendWaves) > 4 ? DC * 16 / (64 * kAttendWaves) : 4;
    const int oi = threadIdx.x / (DC / PER) % 16, dd = threadIdx.x % (DC / PER) * PER;
    // one row's values, normalized and rounded
    auto out_at = [&](int row) {
        const int tok = static_cast<uint32_t>(row) / a.group;
        return (nt.row0 + tok) * a.heads + static_cast<int64_t>(head) * a.group + row - tok * static_cast<int>(a.group);
    };
    auto put = [&](int64_t at, int d, const float* o, float inv) {
        uint32_t w[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
            w[e] = static_cast<uint32_t>(DtOps<DT>::rne(o[2 * e] * inv)) |
                   (static_cast<uint32_t>(DtOps<DT>::rne(o[2 * e + 1] * inv)) << 16);
        *reinterpret_cast<uint2*>(a.out + at * D + d) = make_uint2(w[0], w[1]);
    };
    auto put_lse = [&](int64_t at, float ref, float l) {
        if (a.lse != nullptr)
            a.lse[at] = l != 0.0f ? 0.693147180559945f * (ref + __builtin_amdgcn_logf(l)) : -__builtin_inff();
    };
    // value 16 n + 4 j + r of a row, from its three sums
    auto value = [&](int u, int n, int r) {
        const int g = 16 * n / GS;
        return __builtin_ldexpf(rows[u].o[n][r] - centre[u][g][n & 1], ((n & 1) ? 20 : 24) - exps[u][g]) + middle[u][g];
    };
    if constexpr (ROWS) {
#pragma unroll
        for (int u = 0; u < RT; ++u) {
            const int row = wave_row + 16 * u + i;
            if (row >= count) continue;
            const float l = rows[u].l, inv = l != 0.0f ? 1.0f / l : 0.0f;
            const int64_t at = out_at(row);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float o[4] = {value(u, n, 0), value(u, n, 1), value(u, n, 2), value(u, n, 3)};
                put(at, 16 * n + 4 * j, o, inv);
            }
            if (j == 0) put_lse(at, rows[u].ref, l);
        }
        return;  // (a sequence is one part)
    } else {
#pragma unroll
        for (int u = 0; u < RT; ++u) {
            float ref = kFar;
#pragma unroll
            for (int w = 0; w < kAttendWaves; ++w) ref = fmaxf(ref, stat[w][u][i][0]);
            // (a wavefront that saw nothing has l = 0 and sums of 0; an l that is NaN is to show)
            const float f = rows[u].l != 0.0f ? exp2_fast(rows[u].ref - ref) : 0.0f;
            const int out_row = base_row + 16 * u + oi;
#pragma unroll
            for (int d0 = 0; d0 < D; d0 += DC) {
#pragma unroll
                for (int n = d0 / 16; n < (d0 + DC) / 16; ++n) {
                    float4_t v;
#pragma unroll
                    for (int r = 0; r < 4; ++r) v[r] = f * value(u, n, r);
                    *reinterpret_cast<float4_t*>(&buf[wave][i * kRow + 16 * n - d0 + 4 * j]) = v;
                }
                __syncthreads();
                // a thread takes PER values of a row
                float o[PER];
#pragma unroll
                for (int e = 0; e < PER; ++e) o[e] = 0.0f;
#pragma unroll
                for (int w = 0; w < kAttendWaves; ++w)
#pragma unroll
                    for (int e = 0; e < PER; e += 4) {
                        const float4_t v = *reinterpret_cast<const float4_t*>(&buf[w][oi * kRow + dd + e]);
#pragma unroll
                        for (int k = 0; k < 4; ++k) o[e + k] += v[k];
                    }
                float big = kFar, l = 0.0f;
#pragma unroll
                for (int w = 0; w < kAttendWaves; ++w) big = fmaxf(big, stat[w][u][oi][0]);
#pragma unroll
                for (int w = 0; w < kAttendWaves; ++w)
                    l += stat[w][u][oi][1] != 0.0f ? stat[w][u][oi][1] * exp2_fast(stat[w][u][oi][0] - big) : 0.0f;
                if (out_row < count && threadIdx.x < 16 * DC / PER) {
                    if (part.parts == 1) {
                        const int64_t at = out_at(out_row);
#pragma unroll
                        for (int e = 0; e < PER; e += 4) put(at, d0 + dd + e, o + e, l != 0.0f ? 1.0f / l : 0.0f);
                        if (d0 == 0 && dd == 0) put_lse(at, big, l);
                    } else {
                        const uint32_t at = sums_at(part.slot0 + part.part);
#pragma unroll
                        for (int e = 0; e < PER; e += 4)
                            store_shared(sums, at + 4 * ((16 * u + oi) * D + d0 + dd + e), float4_t{o[e], o[e + 1], o[e + 2], o[e + 3]});
                        if (d0 == 0 && dd == 0)
                            store_shared(sums, at + 4 * (16 * RT * D + 4 * (16 * u + oi)), float4_t{l != 0.0f ? big : kFar, l, 0.0f, 0.0f});
                    }
                }
                __syncthreads();
            }
        }
    }
    if (part.parts == 1) return;

    // The workgroup that finds all other parts done puts them together.  Each
    // thread's stores are waited for (they are then at the point of
    // coherence) before the barrier, the count after it.  (Ordinary stores
    // behind a device fence write back and drop the whole L2 for every
    // workgroup: 75 us more for 512 of them.)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();  // (also: no slot is read or written any more)
    uint32_t* flag = lds;
    if (threadIdx.x == 0) {
        const uint32_t n = __hip_atomic_fetch_add(done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        flag[0] = n;
        // the last one leaves the counter as it was found
        if (n == static_cast<uint32_t>(part.parts) - 1)
            __hip_atomic_store(done, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (flag[0] != static_cast<uint32_t>(part.parts) - 1) return;
    const int left = count - base_row, valid = left < 16 * RT ? left : 16 * RT;
    const uint32_t at0 = sums_at(part.slot0), stride = 4 * gridDim.y * a.s.kv_heads * part_floats(D, RT);
    auto finish = [&](int row, int d, const float* o, float ref, float l) {
        const int64_t at = out_at(base_row + row);
        put(at, d, o, l != 0.0f ? 1.0f / l : 0.0f);
        if (d == 0) put_lse(at, ref, l);
    };
    // few parts: more items (four values of a row) of a thread in flight
    float* meet = reinterpret_cast<float*>(lds) + 64;  // beyond the flag
    constexpr int W = kAttendWaves;
    if (part.parts <= 2) join_parts<D, RT, W, 4, 2>(sums, at0, stride, part.parts, valid, meet, finish);
    else if (part.parts <= 4) join_parts<D, RT, W, 3, 4>(sums, at0, stride, part.parts, valid, meet, finish);
    else join_parts<D, RT, W, 1, 12>(sums, at0, stride, part.parts, valid, meet, finish);
}

template <int DT, int D, int GS, int RT, bool ROWS, bool NT_LOADS, bool WINDOW>
hipError_t launch_attend_kernel(const AttendParams& p, dim3 grid, hipStream_t st) {
    constexpr int W = attend_waves(RT, ROWS);
    constexpr int kRow = (D < 128 ? D : 128) + 4;
    constexpr int slots = 4 * W * (kAttendSlots * Slot<D, GS>::kWords + 64 * RT) + (kQInLds<D, GS> ? 32 * W * D : 0) +
                          (WINDOW ? 4 * W * 16 * RT : 0);
    constexpr int sums = 4 * W * (16 * kRow + RT * 16 * 2);
    constexpr int bytes = slots > sums ? slots : sums;
    if constexpr (bytes > 64 * 1024) {
        static std::atomic<uint64_t> raised{0};
        const hipError_t e =
            raise_lds_limit(reinterpret_cast<const void*>(&attend_kernel<DT, D, GS, RT, ROWS, NT_LOADS, WINDOW>), raised);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((attend_kernel<DT, D, GS, RT, ROWS, NT_LOADS, WINDOW>), grid, dim3(64 * W), bytes, st, p);
    return hipGetLastError();
}

// Tokens that workgroups of several row groups read stay in L2; others are
// streamed past it (one token over 131071: 30.7 us, kept 35.1).  Heads of 256,
// four row groups, 4096 tokens: 64 sequences of 4 heads 195 us, streamed 216, 16
// of 8 heads 84 and 96; of 64 sequences of 8 heads, 604 MB, 448 and 422.  Heads
// of 128, eight row groups over 16k: either way 120.
template <int DT, int D, int GS, bool WINDOW>
hipError_t run_attend(const AttendParams& p, int row_tiles, bool by_rows, dim3 grid, hipStream_t st) {
    if constexpr (D <= 128) {
        if (row_tiles == 2 && by_rows) return launch_attend_kernel<DT, D, GS, 2, true, false, WINDOW>(p, grid, st);
        if (row_tiles == 2 && grid.y > 1) return launch_attend_kernel<DT, D, GS, 2, false, false, WINDOW>(p, grid, st);
        if (row_tiles == 2) return launch_attend_kernel<DT, D, GS, 2, false, true, WINDOW>(p, grid, st);
    }
    if (by_rows) return launch_attend_kernel<DT, D, GS, 1, true, false, WINDOW>(p, grid, st);
    if constexpr (D == 256)
        if (grid.y > 1) return launch_attend_kernel<DT, D, GS, 1, false, false, WINDOW>(p, grid, st);
    return launch_attend_kernel<DT, D, GS, 1, false, true, WINDOW>(p, grid, st);
}

// One translation unit per type and head size, with a window and without.
using AttendFn = hipError_t (*)(const AttendParams&, int row_tiles, bool by_rows, dim3, hipStream_t);
template <int DT, int D, bool WINDOW>
AttendFn attend_fn(int gs);

}  // namespace kv
}  // namespace qmm

#define QMM_KV_ATTEND_UNIT(DTV, DV, WINDOWV)                           \
    namespace qmm {                                                    \
    namespace kv {                                                     \
    template <>                                                        \
    AttendFn attend_fn<DTV, DV, WINDOWV>(int gs) {                     \
        if (gs == 32) return run_attend<DTV, DV, 32, WINDOWV>;         \
        if (gs == 64) return run_attend<DTV, DV, 64, WINDOWV>;         \
        if constexpr (DV >= 128)                                       \
            if (gs == 128) return run_attend<DTV, DV, 128, WINDOWV>;   \
        return nullptr;                                                \
    }                                                                  \
    }                                                                  \
    }
