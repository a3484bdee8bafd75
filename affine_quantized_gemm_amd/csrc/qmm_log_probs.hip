// Log probabilities of given tokens, entropy and the likeliest tokens of rows
// of logits, and the gradient (gfx950).
//
// Mathematics.  With z = scale * logit, in base 2 (c = scale log2 e) and
// against a reference m, the row's largest logit so far,
//   t = c (logit - m),  L = sum 2^t,  W = sum t 2^t,
//   lse = scale m + ln 2 log2 L,  H = ln 2 (log2 L - W / L),
// in one pass: a lane keeps m, L and W of what it has seen and scales L and W
// when its m moves (W then takes L times the move besides).  t of a barred
// token (-infinity) is cut at -10^4, so that its product with 2^t is 0.
//
// The likeliest tokens: a logit's 16 bits as an ordered number and its column
// make a key without equals (of equal logits the lowest column is first), so
// the selection is exact and has one answer.  A wavefront keeps the keys of
// the `top` best of its columns, one a lane; a slice of 1024 columns is looked
// at closer only where a lane's largest passes the last one of the wavefront's
// keys, that of another wavefront of the workgroup, and the least of the four
// wavefronts' (top / 4)-th.  A few such lanes' values
// are put in one by one (a comparison, a count of lanes and a shift by a lane).
// Of a slice with many no more is collected, in LDS, than what is at or above
// the top-th of the lanes' largest: at most 16 values of `top` lanes, whatever
// the values are.  (1000 rows of 152k, fp16 and bf16: none likeliest 63 and 60
// us, 1 79 and 78, 5 114 and 101, 20 half barred 112, all there 127 and 120, 48
// 136 and 151, 63 168 and 207, 64 463 and 633.  The 20 half barred took 163 us
// without the first way and the others' keys, 128 without their (top / 4)-th.)
// Of 64 likeliest the 64 lanes' largest bound nothing: a wavefront collects all
// 1024 values of its first slice and ranks each among all of them, which is the
// 290 to 430 us between 63 and 64.  Besides that the vector units' work a logit
// bounds it (the exponential, t's cut and the two sums; with 20 likeliest they
// are busy 72 % of the time): 60 us of it.  The bf16 form has 132 registers,
// three wavefronts a SIMD; fp16's 120 leave room for four.
//
// A row is one workgroup's, or cut into parts of whole slices where rows are
// few; the workgroup that is last to finish a row joins the parts.
//
// gradient, with g_n of the given tokens' log probabilities, g_H of the
// entropy, g_l of lse:
//   d[v] = scale (sum_n g_n [v = t_n] + p_v (g_l - sum_n g_n - g_H (ln p_v + H))).
#include "qmm.h"
#include "qmm_device.hpp"
#include "qmm_mfma_frag.hpp"
#include "qmm_rows.hpp"

namespace qmm {
namespace {

using mf::swap16;
using mf::swap32;

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kVecs = 2;                        // 16-byte pieces of a lane in a slice
constexpr int kSlice = 64 * kVecs;              // pieces
constexpr int kMostTop = QMM_LOG_PROBS_MOST_TOP;
constexpr int kMostParts = 64;                  // a lane each when they are joined
// Workgroups that rows are cut for (152k logits, one likeliest, bf16; with 512:
// 300 rows 36 us and 43, 6 rows 11.0 with 8 likeliest either way, but 28 rows 17
// and 13, 64 rows 21 and 16, where the joining of twice the parts costs more
// than the emptier chip).
constexpr int kBlocks = 1024;
constexpr int kDoneStride = 32;                 // counters in lines of their own
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
// What exponents are cut at where they multiply a power that is 0 there: far
// beyond fp32's least, and small enough for finite products with sums of any
// length and with incoming gradients.
constexpr float kFarBelow = -1e4f;
constexpr int kNothing = -32768;                // below every ordered logit that is a number
// Lanes whose values are put in one by one (1000 rows, 20 likeliest, fp16 and
// bf16: 2 to 8 lanes 104 to 107 us and 120 to 122, 16 109 and 124, none 114 and 147).
constexpr int kFewLanes = 6;

// 64-bit words of a part: m and L, W, then its keys.
constexpr int part_words(int top) { return 2 + top; }
static_assert(QMM_LOG_PROBS_ZEROED_BYTES >= 4 * kDoneStride * kBlocks / 2, "rows that are cut: at most half of the workgroups");
static_assert(QMM_LOG_PROBS_WORKSPACE_BYTES >= QMM_LOG_PROBS_ZEROED_BYTES + kBlocks * 8 * part_words(kMostTop), "every part");

struct Params {
    LogProbsArgs a;
    float c;
    int parts;
    int64_t part_vecs;   // 16-byte pieces of a part, a multiple of kSlice
    uint32_t* done;      // [rows], kDoneStride apart, 0 before and after
    uint64_t* sums;      // [rows][parts][part_words]
};

// The ordered numbers of a word's two logits: their bits, negative ones turned
// round (-0 becomes 0, which it is equal to).
__device__ __forceinline__ uint32_t ordered2(uint32_t w) {
    typedef short short2_t __attribute__((ext_vector_type(2)));
    const short2_t x = __builtin_bit_cast(short2_t, w);
    const short2_t s = x >> 15;
    return __builtin_bit_cast(uint32_t, static_cast<short2_t>((x ^ (s & static_cast<short2_t>(0x7FFF))) - s));
}
template <int DT>
__device__ __forceinline__ float ordered_f32(int o) {
    return DtOps<DT>::to_f32(static_cast<uint16_t>(o < 0 ? (o - 1) ^ 0x7FFF : o));
}
// Over the wavefront, in every lane.
template <class F>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, F f) {
    v = f(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, 0x128, 0xf, 0xf, true)));  // rotations within 16 lanes
    v = f(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, 0x124, 0xf, 0xf, true)));
    v = f(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, 0x122, 0xf, 0xf, true)));
    v = f(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, 0x121, 0xf, 0xf, true)));
    uint32_t a = v, b = v;
    swap16(a, b);
    a = b = f(a, b);
    swap32(a, b);
    return f(a, b);
}
__device__ __forceinline__ float wave_max(float v) {
    return __builtin_bit_cast(float, wave_reduce(__builtin_bit_cast(uint32_t, v), [](uint32_t a, uint32_t b) {
        return __builtin_bit_cast(uint32_t, fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)));
    }));
}
__device__ __forceinline__ float wave_sum(float v) {
    return __builtin_bit_cast(float, wave_reduce(__builtin_bit_cast(uint32_t, v), [](uint32_t a, uint32_t b) {
        return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
    }));
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    return wave_reduce(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

// m, L and W of some columns; empty: -infinity, 0, 0.
struct Sums {
    float m, l, w;
};
// m as a reference: a row of which nothing is left has none.  (It is taken from
// the logit before the product: with c m, rounded, logits of 10^30 would be as
// far above it as that rounding.)
__device__ __forceinline__ float reference(float m) { return m == -__builtin_inff() ? 0.0f : m; }

// Brought to the reference of a larger m.
__device__ __forceinline__ void move(Sums& s, float m, float c) {
    const float d = s.l != 0.0f ? (reference(s.m) - reference(m)) * c : 0.0f;  // (l NaN: stays so)
    const float f = __builtin_amdgcn_exp2f(d);
    // (d is at most 0; -infinity where bf16 logits lie further apart than fp32's largest)
    s.w = f * __builtin_fmaf(s.l, fmaxf(d, kFarBelow), s.w);
    s.l *= f;
    s.m = m;
}
__device__ __forceinline__ Sums wave_join(Sums s, float c) {
    // (fmaxf passes over NaN; L is NaN where there was one)
    move(s, wave_max(s.m), c);
    s.l = wave_sum(s.l);
    s.w = wave_sum(s.w);
    return s;
}

// Keys: the ordered logit above 2^15, then the columns from the last down.
__device__ __forceinline__ uint64_t key_of(int o, uint32_t col) {
    return static_cast<uint64_t>(static_cast<uint32_t>(o + 32768)) << 32 | (0xFFFFFFFFu - col);
}
__device__ __forceinline__ int key_ordered(uint64_t k) { return static_cast<int>(k >> 32) - 32768; }
__device__ __forceinline__ uint32_t key_column(uint64_t k) { return 0xFFFFFFFFu - static_cast<uint32_t>(k); }

__device__ __forceinline__ int64_t token_at(const void* t, bool wide, int64_t i) {
    return wide ? static_cast<const int64_t*>(t)[i] : static_cast<const int32_t*>(t)[i];
}

// Device-scope: other XCDs read what is stored.
__device__ __forceinline__ void put_shared(uint64_t* p, uint64_t v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t get_shared(const uint64_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t two(float a, float b) {
    return static_cast<uint64_t>(__builtin_bit_cast(uint32_t, b)) << 32 | __builtin_bit_cast(uint32_t, a);
}

// A wavefront's LDS: `top` kept keys, what a slice adds (at most 8 kVecs of
// `top` lanes), and the next kept ones.
constexpr int wave_keys(int top) { return top * (2 + 8 * kVecs); }

// What a wavefront's lanes have written to LDS, the others read after this.
__device__ __forceinline__ void lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

struct Piece {
    uint32_t w[4];
};
// What lanes load where a row has no whole piece.
__device__ const uint4 kNoPiece = {0, 0, 0, 0};
// The largest of a lane's logits.
template <int DT>
__device__ __forceinline__ float largest(const Piece (&q)[kVecs]) {
    if constexpr (DT == DT_F16) {
        typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
        half2_t m = __builtin_bit_cast(half2_t, q[0].w[0]);
#pragma unroll
        for (int n = 0; n < kVecs; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) m = __builtin_elementwise_max(m, __builtin_bit_cast(half2_t, q[n].w[e]));
        return fmaxf(static_cast<float>(m[0]), static_cast<float>(m[1]));
    } else {
        float m = -__builtin_inff();
#pragma unroll
        for (int n = 0; n < kVecs; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) m = fmaxf(m, fmaxf(low_f32<DT>(q[n].w[e]), high_f32<DT>(q[n].w[e])));
        return m;
    }
}

// From the lane before (the first lane: 0).
__device__ __forceinline__ uint32_t shift_lane(uint32_t v) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x138, 0xf, 0xf, false));
}

template <int DT, bool TOP>
__global__ __launch_bounds__(kThreads) void log_probs_kernel(Params p) {
    extern __shared__ __align__(16) uint64_t lds[];
    __shared__ Sums joined[kWaves];
    __shared__ int counts[kWaves];
    __shared__ uint32_t last_flag;
    // what `top` columns have been found at or above: the largest of the wavefronts' last keys' values, and the least of
    // their ceil(top / 4)-th ones' (a third of the values that pass the former alone)
    __shared__ int shared_least;
    __shared__ __align__(16) int shared_part[kWaves];
    if constexpr (TOP) {
        if (threadIdx.x < kWaves) shared_part[threadIdx.x] = shared_least = kNothing;
        __syncthreads();
    }
    const LogProbsArgs& a = p.a;
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int top = a.top, part_of = (top + kWaves - 1) / kWaves;
    const int64_t row = blockIdx.x / static_cast<uint32_t>(p.parts);
    const int part = blockIdx.x - static_cast<uint32_t>(row) * p.parts;
    const uint16_t* const z = static_cast<const uint16_t*>(a.logits) + row * a.stride;
    const float c = p.c;

    // the given tokens' logits, on their way to the end
    int64_t token = -1;
    float given = 0.0f;
    if (static_cast<int>(threadIdx.x) < a.given) {
        token = token_at(a.tokens, a.tokens64, row * a.given + threadIdx.x);
        if (token < 0 || token >= a.vocab) token = -1;
        else given = DtOps<DT>::to_f32(z[token]);
    }

    // the row in 16-byte pieces from the last 16-byte boundary before it: piece v holds columns 8 v - shift ..
    const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(z) & 15) / 2);
    const int64_t vecs = (a.vocab + shift + 7) / 8;
    const int64_t v_end = (part + 1) * p.part_vecs < vecs ? (part + 1) * p.part_vecs : vecs;
    // Loads are issued for every slice, without a branch (one makes the waits for others wait for everything): of the
    // row's nearest whole piece where a lane has none; those lanes' columns follow one by one when the slice is looked at.
    const int64_t whole0 = shift > 0 ? 1 : 0, whole1 = (a.vocab + shift) / 8;  // whole pieces from, to
    const bool tiny = whole1 <= whole0;
    const uint16_t* const pieces = tiny ? reinterpret_cast<const uint16_t*>(&kNoPiece) : z - shift;
    auto load = [&](Piece (&q)[kVecs], int64_t v0) {
#pragma unroll
        for (int n = 0; n < kVecs; ++n) {
            int64_t v = v0 + 64 * n + lane;
            v = v < whole1 ? v : whole1 - 1;
            v = tiny ? 0 : v > whole0 ? v : whole0;
            const mf::u32x4_t u = __builtin_nontemporal_load(reinterpret_cast<const mf::u32x4_t*>(pieces + 8 * v));
#pragma unroll
            for (int e = 0; e < 4; ++e) q[n].w[e] = u[e];
        }
    };
    auto mend = [&](Piece (&q)[kVecs], int64_t v0) {
#pragma unroll
        for (int n = 0; n < kVecs; ++n) {
            const int64_t v = v0 + 64 * n + lane, col = 8 * v - shift;
            if (v >= whole0 && v < whole1 && v < v_end) continue;
            // (columns outside the row or the part are barred)
            constexpr uint32_t none = DT == DT_F16 ? 0xFC00u : 0xFF80u;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t h[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int64_t at = col + 2 * e + k;
                    h[k] = v < v_end && at >= 0 && at < a.vocab ? z[at] : none;
                }
                q[n].w[e] = h[0] | h[1] << 16;
            }
        }
    };

    uint64_t* const keys = lds + wave * wave_keys(top);
    int have = 0;             // kept keys: lane i has the i-th best
    uint64_t mine = 0;
    int least = kNothing - 1; // a later column has to be above it
    Sums s{-__builtin_inff(), 0.0f, 0.0f};
    int64_t v0 = part * p.part_vecs + static_cast<int64_t>(wave) * kSlice;
    auto look = [&](Piece (&q)[kVecs]) {
        const bool inner = v0 >= whole0 && v0 + kSlice <= whole1 && v0 + kSlice <= v_end;
        if (!inner) mend(q, v0);
        // the lane's largest (passes over NaN, which show in the sums)
        const float big = largest<DT>(q);
        if (big > s.m) move(s, big, c);
        const float ref = reference(s.m);
#pragma unroll
        for (int n = 0; n < kVecs; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x[2] = {low_f32<DT>(q[n].w[e]), high_f32<DT>(q[n].w[e])};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float t = (x[k] - ref) * c;
                    const float f = __builtin_amdgcn_exp2f(t);
                    s.l += f;
                    s.w = __builtin_fmaf(f, fmaxf(t, kFarBelow), s.w);
                }
            }
        if constexpr (TOP) {
            // what a value has to pass: later columns the wavefront's own last key, any column the others' last value
            int others = __hip_atomic_load(&shared_part[0], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
#pragma unroll
            for (int w = 1; w < kWaves; ++w) {
                const int x = __hip_atomic_load(&shared_part[w], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
                others = x < others ? x : others;
            }
            const int most = __hip_atomic_load(&shared_least, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
            others = __builtin_amdgcn_readfirstlane(most > others ? most : others);
            const int pass = least >= others ? least : others - 1;
            const uint64_t over = pass < kNothing ? ~uint64_t{0} : __ballot(big > ordered_f32<DT>(pass) || (pass == others - 1 && big >= ordered_f32<DT>(others)));
            if (over != 0) {
                // the lane's keys within the slice: ordered logit, then columns from the last down; 0: not looked at
                uint32_t own[kVecs][4][2], best = 0;
                const int64_t first = 8 * v0 - shift;
#pragma unroll
                for (int n = 0; n < kVecs; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t o = ordered2(q[n].w[e]);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int x = k ? static_cast<int>(o) >> 16 : static_cast<int16_t>(o);
                            const int at = 512 * n + 8 * lane + 2 * e + k;
                            bool in = x > pass;
                            if (!inner) in = in && first + at >= 0 && first + at < a.vocab && v0 + 64 * n + lane < v_end;
                            own[n][e][k] = in ? static_cast<uint32_t>(x + 32768) << 16 | (0xFFFFu - at) : 0;
                            best = own[n][e][k] > best ? own[n][e][k] : best;
                        }
                    }
                const uint32_t columns = static_cast<uint32_t>(first);
                auto whole = [&](uint32_t k) { return key_of(static_cast<int>(k >> 16) - 32768, columns + (0xFFFFu - (k & 0xFFFFu))); };
                uint64_t some = __ballot(best != 0);
                if (__popcll(some) <= kFewLanes) {
                    while (some != 0) {
                        const int l = __builtin_ctzll(some);
                        const uint32_t k = __builtin_amdgcn_readlane(best, l);
                        const uint64_t key = whole(k);
                        // those before it stay, the others move on by a lane
                        const bool before = mine > key;
                        const uint32_t hi = shift_lane(static_cast<uint32_t>(mine >> 32)), lo = shift_lane(static_cast<uint32_t>(mine));
                        const int place = __popcll(__ballot(before));
                        if (!before) mine = lane == place ? key : static_cast<uint64_t>(hi) << 32 | lo;
                        if (lane >= top) mine = 0;
                        have = have < top ? have + 1 : top;
                        best = 0;
#pragma unroll
                        for (int n = 0; n < kVecs; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    own[n][e][h] = own[n][e][h] == k ? 0 : own[n][e][h];
                                    best = own[n][e][h] > best ? own[n][e][h] : best;
                                }
                        some = __ballot(best != 0);
                    }
                } else if (some != 0) {
                    // the top-th of the lanes' best
                    uint32_t from = 1;
                    if (__popcll(some) <= top) {
                    } else if (top <= 8) {
                        from = ~0u;  // (a key is smaller: its column is below 1024)
                        for (int k = 0; k < top; ++k) from = wave_max_u32(best < from ? best : 0);
                        from = __builtin_amdgcn_readfirstlane(from);
                    } else {
                        int rank = 0;
#pragma unroll 8
                        for (int k = 0; k < 64; ++k) rank += static_cast<uint32_t>(__builtin_amdgcn_readlane(best, k)) > best;
                        const uint64_t at = __ballot(rank == top - 1 && best != 0);
                        from = __builtin_amdgcn_readlane(best, __builtin_ctzll(at));
                    }
                    if (lane < have) keys[lane] = mine;
                    int n_keys = have;
#pragma unroll
                    for (int n = 0; n < kVecs; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const bool take = own[n][e][k] >= from;
                                const uint64_t taken = __ballot(take);
                                if (taken != 0) {
                                    if (take) keys[n_keys + __popcll(taken & ((uint64_t{1} << lane) - 1))] = whole(own[n][e][k]);
                                    n_keys += __popcll(taken);
                                }
                            }
                    lds_order();
                    // each key's place among them all; the first `top` stay
                    uint64_t* const fresh = keys + wave_keys(top) - top;
                    for (int k0 = 0; k0 < n_keys; k0 += 64) {
                        const uint64_t key = k0 + lane < n_keys ? keys[k0 + lane] : 0;
                        int place = 0;
#pragma unroll 8
                        for (int k = 0; k < n_keys; ++k) place += keys[k] > key;
                        if (k0 + lane < n_keys && place < top) fresh[place] = key;
                    }
                    lds_order();
                    have = n_keys < top ? n_keys : top;
                    mine = lane < have ? fresh[lane] : 0;
                    lds_order();
                }
                if (have >= part_of) {
                    const int part_least = static_cast<int>(__builtin_amdgcn_readlane(static_cast<uint32_t>(mine >> 32), part_of - 1)) - 32768;
                    if (lane == 0) __hip_atomic_store(&shared_part[wave], part_least, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
                }
                if (have == top) {
                    least = static_cast<int>(__builtin_amdgcn_readlane(static_cast<uint32_t>(mine >> 32), top - 1)) - 32768;
                    if (lane == 0) __hip_atomic_fetch_max(&shared_least, least, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
                }
            }
        }
    };
    // two slices on their way; one is taken out of its registers before the next is asked for
    Piece even[kVecs], odd[kVecs];
    load(even, v0);
    load(odd, v0 + kWaves * kSlice);
    auto turn = [&](Piece (&q)[kVecs]) {
        Piece now[kVecs];
#pragma unroll
        for (int n = 0; n < kVecs; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                now[n].w[e] = q[n].w[e];
                asm volatile("" : "+v"(now[n].w[e]));
            }
        load(q, v0 + 2 * kWaves * kSlice);
        look(now);
        v0 += kWaves * kSlice;
    };
    while (v0 < v_end) {
        turn(even);
        if (v0 >= v_end) break;
        turn(odd);
    }

    // the wavefronts' sums and keys together
    s = wave_join(s, c);
    if (TOP && lane < have) keys[lane] = mine;
    if (lane == 0) {
        joined[wave] = s;
        counts[wave] = have;
    }
    __syncthreads();
    s = joined[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) {
        Sums o = joined[w];
        const float m = fmaxf(s.m, o.m);
        move(s, m, c);
        move(o, m, c);
        s.l += o.l;
        s.w += o.w;
    }
    uint64_t* const best = lds + kWaves * wave_keys(top);  // [top] of the workgroup
    if constexpr (TOP) {
        for (int i = threadIdx.x; i < top; i += kThreads) best[i] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < kWaves * top; i += kThreads) {
            const int w = i / top, n = i - w * top;
            if (n < counts[w]) {
                const uint64_t key = lds[w * wave_keys(top) + n];
                int place = n;  // (its own wavefront's are in order)
                for (int u = 0; u < kWaves; ++u)
                    if (u != w)
#pragma unroll 8
                        for (int k = 0; k < counts[u]; ++k) place += lds[u * wave_keys(top) + k] > key;
                if (place < top) best[place] = key;
            }
        }
        __syncthreads();
    }

    if (p.parts > 1) {
        uint64_t* const mine = p.sums + blockIdx.x * static_cast<int64_t>(part_words(top));
        if (threadIdx.x == 0) {
            put_shared(mine, two(s.m, s.l));
            put_shared(mine + 1, two(s.w, 0.0f));
        }
        if constexpr (TOP)
            for (int i = threadIdx.x; i < top; i += kThreads) put_shared(mine + 2 + i, best[i]);
        // every thread's stores have reached the device's point of coherence before the count
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (threadIdx.x == 0) {
            uint32_t* const done = p.done + row * kDoneStride;
            const uint32_t n = __hip_atomic_fetch_add(done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (n == static_cast<uint32_t>(p.parts) - 1) __hip_atomic_store(done, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            last_flag = n;
        }
        __syncthreads();
        if (last_flag != static_cast<uint32_t>(p.parts) - 1) return;
        const uint64_t* const all = p.sums + row * p.parts * static_cast<int64_t>(part_words(top));
        Sums o{-__builtin_inff(), 0.0f, 0.0f};
        if (lane < p.parts) {  // (every wavefront does the same)
            const uint64_t ml = get_shared(all + lane * part_words(top)), w = get_shared(all + lane * part_words(top) + 1);
            o.m = __builtin_bit_cast(float, static_cast<uint32_t>(ml));
            o.l = __builtin_bit_cast(float, static_cast<uint32_t>(ml >> 32));
            o.w = __builtin_bit_cast(float, static_cast<uint32_t>(w));
        }
        s = wave_join(o, c);
        if constexpr (TOP) {
            // the parts' keys into LDS, then the best of the parts' first ones, `top` times
            for (int i = threadIdx.x; i < p.parts * top; i += kThreads) {
                const int u = i / top;
                lds[i] = get_shared(all + u * part_words(top) + 2 + (i - u * top));
            }
            __syncthreads();
            uint64_t winner = 0;
            if (wave == 0) {
                int at = 0;
                uint64_t head = lane < p.parts ? lds[lane * top] : 0;
                for (int i = 0; i < top; ++i) {
                    const uint32_t hi = wave_max_u32(static_cast<uint32_t>(head >> 32));
                    const uint32_t lo = wave_max_u32(static_cast<uint32_t>(head >> 32) == hi ? static_cast<uint32_t>(head) : 0);
                    const uint64_t k = static_cast<uint64_t>(hi) << 32 | lo;
                    if (lane == i) winner = k;
                    if (head == k && k != 0) {
                        ++at;
                        head = at < top ? lds[lane * top + at] : 0;
                    }
                }
            }
            __syncthreads();
            if (wave == 0 && lane < top) lds[lane] = winner;
            __syncthreads();
        }
    }
    const uint64_t* const chosen = p.parts > 1 ? lds : best;

    // NaN among the logits, or +infinity: NaN.  Nothing but -infinity: no probabilities.
    const bool none = s.m == -__builtin_inff() && s.l == s.l;
    const float log2_l = __builtin_amdgcn_logf(s.l), ref = reference(s.m);
    const bool bad = !(s.l == s.l) || s.m == __builtin_inff();
    const float nan = __builtin_nanf("");
    const float lse = bad ? nan : none ? -__builtin_inff() : __builtin_fmaf(ref, a.scale, kLn2 * log2_l);
    // (halves: bf16 logits may lie further apart than fp32's largest)
    auto log_p = [&](float x) {
        return bad ? nan : none || x == -__builtin_inff() ? -__builtin_inff() : kLn2 * __builtin_fmaf(0.5f * x - 0.5f * ref, 2.0f * c, -log2_l);
    };
    if (threadIdx.x == 0) {
        a.lse[row] = lse;
        a.entropy[row] = bad ? nan : none ? 0.0f : kLn2 * (log2_l - s.w / s.l);
    }
    if (static_cast<int>(threadIdx.x) < a.given) a.token_lp[row * a.given + threadIdx.x] = token < 0 ? 0.0f : log_p(given);
    if constexpr (TOP) {
        if (static_cast<int>(threadIdx.x) < top) {
            const uint64_t k = chosen[threadIdx.x];
            const int64_t at = row * top + threadIdx.x;
            a.top_values[at] = log_p(ordered_f32<DT>(key_ordered(k)));
            a.top_ids[at] = bad ? int64_t{-1} : static_cast<int64_t>(key_column(k));
        }
    }
}

// One thread takes 8 columns; a workgroup kGradVecs pieces of one row a thread.
constexpr int kGradVecs = 2;

template <int DT>
__global__ __launch_bounds__(kThreads) void log_probs_grad_kernel(LogProbsGradArgs a, uint32_t blocks_row) {
    const int64_t row = blockIdx.x / blocks_row;
    const uint32_t block = blockIdx.x - static_cast<uint32_t>(row) * blocks_row;
    const uint16_t* const z = static_cast<const uint16_t*>(a.logits) + row * a.stride;
    uint16_t* const d = static_cast<uint16_t*>(a.out) + row * a.out_stride;
    const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(z) & 15) / 2);
    const bool alike = ((reinterpret_cast<uintptr_t>(z) ^ reinterpret_cast<uintptr_t>(d)) & 15) == 0;
    const int64_t v0 = static_cast<int64_t>(block) * (kGradVecs * kThreads) + threadIdx.x;
    mf::u32x4_t q[kGradVecs];
    bool whole[kGradVecs];
#pragma unroll
    for (int n = 0; n < kGradVecs; ++n) {
        const int64_t col = 8 * (v0 + n * kThreads) - shift;
        whole[n] = col >= 0 && col + 8 <= a.vocab;
        if (whole[n]) {
            q[n] = __builtin_nontemporal_load(reinterpret_cast<const mf::u32x4_t*>(z + col));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t at = col + 2 * e;
                q[n][e] = (at >= 0 && at < a.vocab ? z[at] : 0u) | (at + 1 >= 0 && at + 1 < a.vocab ? static_cast<uint32_t>(z[at + 1]) << 16 : 0u);
            }
        }
    }
    const float lse = a.lse[row];
    const float gh = a.grad_entropy != nullptr ? a.grad_entropy[row] : 0.0f;
    const float h = gh != 0.0f ? a.entropy[row] : 0.0f;
    float g = a.grad_lse != nullptr ? a.grad_lse[row] : 0.0f;
    if (a.grad_tokens != nullptr)
        for (int n = 0; n < a.given; ++n) {
            const int64_t t = token_at(a.tokens, a.tokens64, row * a.given + n);
            if (t >= 0 && t < a.vocab) g -= a.grad_tokens[row * a.given + n];
        }
    const bool none = lse == -__builtin_inff();  // (a row without probabilities has no gradient)
    const float plus = g - gh * h;
#pragma unroll
    for (int n = 0; n < kGradVecs; ++n) {
        const int64_t col = 8 * (v0 + n * kThreads) - shift;
        if (col >= a.vocab) continue;
        float y[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x[2] = {low_f32<DT>(q[n][e]), high_f32<DT>(q[n][e])};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float lp = __builtin_fmaf(x[k], a.scale, -lse);
                const float pv = __builtin_amdgcn_exp2f(lp * kLog2e);
                y[2 * e + k] = none ? 0.0f : pv * __builtin_fmaf(-gh, fmaxf(lp, kFarBelow), plus);
                if (lse != lse) y[2 * e + k] = lse;
            }
        }
        if (a.grad_tokens != nullptr && !none)
            for (int k = 0; k < a.given; ++k) {
                const int64_t t = token_at(a.tokens, a.tokens64, row * a.given + k);
                const int64_t at = t - col;
                if (t >= 0 && t < a.vocab && at >= 0 && at < 8) {
                    const float gt = a.grad_tokens[row * a.given + k];
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] += e == at ? gt : 0.0f;
                }
            }
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = pack2<DT>(a.scale * y[2 * e], a.scale * y[2 * e + 1]);
        if (whole[n] && alike) {
            __builtin_nontemporal_store(mf::u32x4_t{w[0], w[1], w[2], w[3]}, reinterpret_cast<mf::u32x4_t*>(d + col));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (col + e >= 0 && col + e < a.vocab) d[col + e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
        }
    }
}

constexpr int64_t kMostBlocks = UINT32_MAX / kThreads;  // of a launch: a grid's threads are 32 bits

const void* after(const void* p, int64_t bytes) { return p != nullptr ? static_cast<const char*>(p) + bytes : nullptr; }

}  // namespace

// Parts of a row: for about kBlocks workgroups, each wavefront with a slice
// at least (the first piece may lie before the row: one more).
int log_probs_parts(int64_t rows, int64_t vocab) {
    const int64_t slices = ((vocab + 7) / 8 + 1 + kSlice - 1) / kSlice;
    int64_t parts = rows > 0 ? kBlocks / rows : 1;
    parts = parts < kMostParts ? parts : kMostParts;
    const int64_t most = (slices + kWaves - 1) / kWaves;
    parts = parts < most ? parts : most;
    return parts > 1 ? static_cast<int>(parts) : 1;
}

hipError_t launch_log_probs(int dt, const LogProbsArgs& a, hipStream_t st) {
    Params p{};
    p.a = a;
    p.c = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
    p.parts = log_probs_parts(a.rows, a.vocab);
    const int64_t slices = ((a.vocab + 7) / 8 + 1 + kSlice - 1) / kSlice;
    p.part_vecs = (slices + p.parts - 1) / p.parts * kSlice;
    p.done = static_cast<uint32_t*>(a.workspace);
    p.sums = reinterpret_cast<uint64_t*>(static_cast<char*>(a.workspace) + QMM_LOG_PROBS_ZEROED_BYTES);
    int64_t words = static_cast<int64_t>(kWaves) * wave_keys(a.top) + a.top;
    if (p.parts > 1 && words < static_cast<int64_t>(p.parts) * a.top) words = static_cast<int64_t>(p.parts) * a.top;
    const unsigned bytes = static_cast<unsigned>(8 * words);
    for (int64_t row = 0; row < a.rows; row += kMostBlocks) {
        const int64_t n = a.rows - row < kMostBlocks ? a.rows - row : kMostBlocks;
        // (rows that are cut are few)
        const dim3 grid(static_cast<unsigned>(n * p.parts));
        p.a = a;
        p.a.logits = static_cast<const uint16_t*>(a.logits) + row * a.stride;
        p.a.tokens = after(a.tokens, row * a.given * (a.tokens64 ? 8 : 4));
        p.a.lse = a.lse + row;
        p.a.entropy = a.entropy + row;
        if (a.given > 0) p.a.token_lp = a.token_lp + row * a.given;
        if (a.top > 0) {
            p.a.top_values = a.top_values + row * a.top;
            p.a.top_ids = a.top_ids + row * a.top;
        }
        if (dt == DT_F16) {
            if (a.top > 0) hipLaunchKernelGGL((log_probs_kernel<DT_F16, true>), grid, dim3(kThreads), bytes, st, p);
            else hipLaunchKernelGGL((log_probs_kernel<DT_F16, false>), grid, dim3(kThreads), bytes, st, p);
        } else {
            if (a.top > 0) hipLaunchKernelGGL((log_probs_kernel<DT_BF16, true>), grid, dim3(kThreads), bytes, st, p);
            else hipLaunchKernelGGL((log_probs_kernel<DT_BF16, false>), grid, dim3(kThreads), bytes, st, p);
        }
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_log_probs_grad(int dt, const LogProbsGradArgs& a, hipStream_t st) {
    const int64_t vecs = (a.vocab + 7) / 8 + 1;
    const int64_t blocks_row = (vecs + kGradVecs * kThreads - 1) / (kGradVecs * kThreads);
    const int64_t most = kMostBlocks / blocks_row;
    for (int64_t row = 0; row < a.rows; row += most) {
        const int64_t n = a.rows - row < most ? a.rows - row : most;
        const dim3 grid(static_cast<unsigned>(blocks_row * n));
        LogProbsGradArgs p = a;
        p.logits = static_cast<const uint16_t*>(a.logits) + row * a.stride;
        p.tokens = after(a.tokens, row * a.given * (a.tokens64 ? 8 : 4));
        p.lse = a.lse + row;
        if (a.entropy != nullptr) p.entropy = a.entropy + row;
        if (a.grad_tokens != nullptr) p.grad_tokens = a.grad_tokens + row * a.given;
        if (a.grad_entropy != nullptr) p.grad_entropy = a.grad_entropy + row;
        if (a.grad_lse != nullptr) p.grad_lse = a.grad_lse + row;
        p.out = static_cast<uint16_t*>(a.out) + row * a.out_stride;
        if (dt == DT_F16)
            hipLaunchKernelGGL((log_probs_grad_kernel<DT_F16>), grid, dim3(kThreads), 0, st, p, static_cast<uint32_t>(blocks_row));
        else
            hipLaunchKernelGGL((log_probs_grad_kernel<DT_BF16>), grid, dim3(kThreads), 0, st, p, static_cast<uint32_t>(blocks_row));
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace qmm
