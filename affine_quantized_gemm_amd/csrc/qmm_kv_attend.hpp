// Attention over the paged 4-bit K/V cache on the matrix cores (gfx950).
//
// Mathematics.  With codes c, scale s and bias b of token t and group g (of
// GS consecutive d), k_hat = s c + b, a score is
//   S[t, row] = sum_g s_K[t, g] (sum_{d in g} q[row, d] c[t, d])  +  b_K[t, g] (sum_{d in g} q[row, d]),
// so the first product runs on the codes themselves and its result is scaled
// per token and group; with p = 2^(S - R),
//   O[row, d] = sum_t (p s_V[t, g]) (c[t, d] - 8)  +  sum_t p (b_V[t, g] + 8 s_V[t, g])
// takes the second product's operand P' = p s_V, one per group, to codes
// again.  Nothing is ever dequantized.  The codes are centred because P' is
// rounded to 11 bits: its error is then weighed by |c - 8|, about the size of
// the values, and not by c; the centring itself is -8 sum_t P', a product
// with ones on the matrix core.  R = M + E is a running reference: M follows
// the scores' maximum and E the exponent of the largest s_V, so that P' stays
// near 1 whatever the values' size.  Both are moved (and everything summed so
// far scaled) only when a score passes M by 8, or a scale 2^E by 2^7.
//
// Codes as operands.  A 4-bit code in the low bits of an fp16 is the
// subnormal number c 2^-24 (in bits 4..7: 16 c 2^-24), which the matrix core
// multiplies exactly: unpacking a word of 8 codes takes four ands and a
// shift, no conversion and no offset to take away again.  The factors 2^24
// go into the scores' scale and the last step; the 16 of the odd codes into
// the d order of Q (q / 16) and into the last step.  Q is scaled per row by a
// power of two into fp16's range, for bf16 too, so there is one form for
// both types.
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

#include "qmm_device.hpp"
#include "qmm_internal.hpp"
#include "qmm_kv.hpp"
#include "qmm_mfma_frag.hpp"

namespace qmm {
namespace kv {

constexpr int kAttendWaves = 4;
constexpr int kAttendSlots = 2;   // steps of a wavefront in LDS: one read, the others on their way
constexpr float kFar = -3.0e38f;

// Wavefronts a SIMD that the registers are to leave room for.
constexpr int attend_occupancy(int dim, int row_tiles) { return dim == 256 ? 1 : row_tiles == 1 ? 3 : 2; }

struct AttendParams {
    Seqs s;
    const uint16_t* q;
    int64_t q_row, q_head;
    int heads, group;       // heads of one kv head
    int row_groups;         // row tiles a sequence needs at most / RT
    int splits;             // parts a sequence is cut into at most
    int chunk;              // tokens a part (a multiple of 32), more where the sequence is longer than planned
    float scale;
    const int64_t* mask;
    uint16_t* out;
    float* lse;
    float* part;            // [seqs][kv_heads][splits][max_new * group][D + 2]
};

// How sequence b is cut: tokens, tokens a part.
struct Cut {
    int len, chunk;
};
__device__ __forceinline__ Cut cut_of(const AttendParams& a, const NewTokens& t) {
    const int64_t cap = a.s.width << a.s.page_shift;
    const int64_t end = static_cast<int64_t>(t.pos0) + t.n;
    Cut c;
    c.len = static_cast<int>(end < cap ? end : cap);
    int chunk = a.chunk;
    if (c.len > static_cast<int64_t>(chunk) * a.splits) {
        const int each = (c.len + a.splits - 1) / a.splits;
        chunk = (each + 31) / 32 * 32;
    }
    c.chunk = chunk;
    return c;
}

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

// Two fp32 values -> fp16 halves.  Nearest for fp16 outputs; toward zero (one
// instruction) for bf16 ones, whose 8 bits do not see the 11th.
template <int DT>
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    if constexpr (DT == DT_F16) {
        const uint32_t a = __builtin_bit_cast(uint16_t, static_cast<_Float16>(lo));
        const uint32_t b = __builtin_bit_cast(uint16_t, static_cast<_Float16>(hi));
        return a | (b << 16);
    } else {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(lo, hi));
    }
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

// State of one tile of 16 rows.
template <int D, int GS>
struct RowTile {
    static constexpr int S = D / 32, G = D / GS, NT = D / 16;
    Frag q[S];        // Q^T operand
    float qs[G];      // sum of the group's q, times 2^-24
    float cs;         // score -> log2 units
    float m, l;       // M; this lane's share of the sum of p
    float bias[G];    // this lane's share of sum p (b + 8 s)
    float4_t z[G];    // sum P'
    float4_t o[NT];
    uint64_t bits;    // new tokens that the row sees
};

// Loads row tile's Q: values of row i, d = 32 s + 8 j + e.
template <int DT, int D, int GS>
__device__ __forceinline__ void load_q(RowTile<D, GS>& t, const uint16_t* q, bool have, float scale) {
    constexpr int S = D / 32, G = D / GS;
    float f[S][8];
    float top = 0.0f;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        uint32_t w[4] = {0, 0, 0, 0};
        if (have) load_words<4>(reinterpret_cast<const uint32_t*>(q + 32 * s), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f[s][e] = half_f32<DT>(w[e / 2], e & 1);
            top = fmaxf(top, fabsf(f[s][e]));
        }
    }
    top = max_j(top);
    // 2^k: the row's largest value comes to [2^9, 2^10); its smallest that
    // still counts, 2^-24 of that, is then a normal number also after q / 16
    int k = top > 0.0f ? 9 - __builtin_amdgcn_frexp_expf(top) + 1 : 0;
    k = k < -90 ? -90 : k > 120 ? 120 : k;
    const float up = __builtin_ldexpf(scale < 0.0f ? -1.0f : 1.0f, k);
#pragma unroll
    for (int g = 0; g < G; ++g) t.qs[g] = 0.0f;
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f[s][e] *= up;
            t.qs[32 * s / GS] += f[s][e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float m = (e & 1) ? 0.0625f : 1.0f;
            t.q[s].v[e] = pack_f16<DT_F16>(f[s][e] * m, f[s][e + 4] * m);
        }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) t.qs[g] = sum_j(t.qs[g]) * 0x1p-24f;
    // log2(e) * |scale| * 2^24 / 2^k
    t.cs = __builtin_ldexpf(fabsf(scale) * 1.44269504088896f, 24 - k);
}

// One step: 32 tokens against the row tiles.  EDGE: `first` is the place of
// the step's first token among the new ones (negative: before them), `left`
// how many tokens of the step there are.
template <int DT, int D, int GS, int RT, bool EDGE>
__device__ __forceinline__ void step(const uint32_t* x, RowTile<D, GS> (&rows)[RT], float& ref_e, int lane,
                                     int first, int left) {
    using L = Slot<D, GS>;
    constexpr int S = D / 32, G = D / GS, NT = D / 16, C = D / 64;
    const int j = lane / 16;
    uint32_t vs[2][G][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int g = 0; g < G; ++g) load_words<4>(x + L::kVs + ((4 * t + j) * G + g) * 4, vs[t][g]);
    if constexpr (EDGE) {
        // slots past the end may hold anything: their scales and biases of V become 0
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int n = left - (16 * t + 4 * j);
            const uint32_t m01 = n >= 2 ? ~0u : n == 1 ? 0xFFFFu : 0u;
            const uint32_t m23 = n >= 4 ? ~0u : n == 3 ? 0xFFFFu : 0u;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                vs[t][g][0] &= m01;
                vs[t][g][1] &= m23;
                vs[t][g][2] &= m01;
                vs[t][g][3] &= m23;
            }
        }
    }
    // the largest scale of V among this lane's tokens, against 2^(E + 7)
    float big = 0.0f;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int r = 0; r < 4; ++r) big = fmaxf(big, half_f32<DT>(vs[t][g][r / 2], r & 1));

    // scores of all row tiles: sum_g s (codes . q) + b (sum of q)
    float sc[RT][2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        float4_t p[RT][G];
        uint32_t k[S];
        load_words<S>(x + t * (L::kCodes / 2) + (4 * (lane % 16) + j) * S, k);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const Frag a = codes8(k[s]);
#pragma unroll
            for (int u = 0; u < RT; ++u) {
                const int g = 32 * s / GS;
                const float4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
                p[u][g] = mf::mfma<DT_F16>(a, rows[u].q[s], 32 * s % GS == 0 ? zero : p[u][g]);
            }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            uint32_t w[4];
            load_words<4>(x + L::kKs + ((4 * t + j) * G + g) * 4, w);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float ks = half_f32<DT>(w[r / 2], r & 1);
                const float kb = half_f32<DT>(w[2 + r / 2], r & 1);
#pragma unroll
                for (int u = 0; u < RT; ++u) {
                    const float before = g == 0 ? kb * rows[u].qs[0] : __builtin_fmaf(kb, rows[u].qs[g], sc[u][t][r]);
                    sc[u][t][r] = __builtin_fmaf(ks, p[u][g][r], before);
                }
            }
        }
    }
    bool see[RT][2][4];
    float top[RT];
    bool move = big > exp2_fast(ref_e + 7.0f);
#pragma unroll
    for (int u = 0; u < RT; ++u) {
        float mx = kFar;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                see[u][t][r] = true;
                if constexpr (EDGE) {
                    const int at = 16 * t + 4 * j + r, n = first + at;
                    see[u][t][r] = at < left && (n < 0 || ((rows[u].bits >> (n & 63)) & 1) != 0);
                }
                mx = fmaxf(mx, see[u][t][r] ? sc[u][t][r] : kFar);
            }
        top[u] = mx * rows[u].cs;
        move = move || top[u] > rows[u].m + 8.0f;
    }
    if (__any(move)) {
        const float old_e = ref_e;
        const float all = max_j(big);
        if (all > 0.0f) ref_e = fmaxf(ref_e, fminf(static_cast<float>(__builtin_amdgcn_frexp_expf(all)), 100.0f));
#pragma unroll
        for (int u = 0; u < RT; ++u) {
            const float m = fmaxf(rows[u].m, max_j(top[u]));
            const float f = exp2_fast(rows[u].m - m + (old_e - ref_e));
            rows[u].m = m;
            rows[u].l *= f;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                rows[u].bias[g] *= f;
#pragma unroll
                for (int r = 0; r < 4; ++r) rows[u].z[g][r] *= f;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r) rows[u].o[n][r] *= f;
        }
    }
    // p, its sum, P' and the bias sums
    Frag pp[RT][G];
#pragma unroll
    for (int u = 0; u < RT; ++u) {
        const float ref = rows[u].m + ref_e;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            float p[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                p[r] = exp2_fast(__builtin_fmaf(sc[u][t][r], rows[u].cs, -ref));
                if constexpr (EDGE) p[r] = see[u][t][r] ? p[r] : 0.0f;
                rows[u].l += p[r];
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                float s[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    s[r] = half_f32<DT>(vs[t][g][r / 2], r & 1);
                    const float mid = __builtin_fmaf(8.0f, s[r], half_f32<DT>(vs[t][g][2 + r / 2], r & 1));
                    rows[u].bias[g] = __builtin_fmaf(p[r], mid, rows[u].bias[g]);
                }
                pp[u][g].v[2 * t] = pack_f16<DT>(p[0] * s[0], p[1] * s[1]);
                pp[u][g].v[2 * t + 1] = pack_f16<DT>(p[2] * s[2], p[3] * s[3]);
            }
        }
        Frag ones;
        ones.v[0] = ones.v[1] = ones.v[2] = ones.v[3] = 0x3C003C00u;
#pragma unroll
        for (int g = 0; g < G; ++g) rows[u].z[g] = mf::mfma<DT_F16>(ones, pp[u][g], rows[u].z[g]);
    }
    // the second product: tile n = 4 c + q of 16 d, from nibble q of the words of quad c
    uint32_t v[2][S];
#pragma unroll
    for (int t = 0; t < 2; ++t) load_words<S>(x + L::kV + t * (L::kCodes / 2) + 16 * S * j + S * (lane % 16), v[t]);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        uint32_t w[4] = {v[0][c], v[0][C + c], v[1][c], v[1][C + c]};
        uint32_t h[4] = {w[0] >> 8, w[1] >> 8, w[2] >> 8, w[3] >> 8};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            Frag a;
#pragma unroll
            for (int k = 0; k < 4; ++k) a.v[k] = (q < 2 ? w[k] : h[k]) & ((q & 1) ? 0x00F000F0u : 0x000F000Fu);
            const int n = 4 * c + q;
#pragma unroll
            for (int u = 0; u < RT; ++u) rows[u].o[n] = mf::mfma<DT_F16>(a, pp[u][16 * n / GS], rows[u].o[n]);
        }
    }
}

}  // namespace

// One workgroup: one part of one sequence and kv head against RT tiles of 16
// rows (row = new token * group + head within the group).  Its four
// wavefronts take the part's steps of 32 tokens in turn, each with sums of
// its own, which are put together through LDS at the end.
template <int DT, int D, int GS, int RT, bool NT_LOADS>
__global__ __launch_bounds__(64 * kAttendWaves, attend_occupancy(D, RT)) void attend_kernel(AttendParams a) {
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

    // workgroups that read the same tokens (row groups) have ids 8 apart: one XCD
    const int64_t id = blockIdx.x;
    const int64_t unit = id / (8 * a.row_groups) * 8 + id % 8;
    const int rg = static_cast<int>(id / 8 % a.row_groups);
    const int head = static_cast<int>(unit % a.s.kv_heads);
    const int64_t bp = unit / a.s.kv_heads;
    const int part = static_cast<int>(bp % a.splits);
    const int64_t b64 = bp / a.splits;
    if (b64 >= a.s.seqs) return;
    const int b = static_cast<int>(b64);
    const NewTokens nt = new_tokens(a.s, b);
    const int count = nt.n * a.group;
    if (rg * 16 * RT >= count) return;
    const Cut cut = cut_of(a, nt);
    const int t0 = part * cut.chunk;
    if (t0 >= cut.len && part > 0) return;
    const int t1 = t0 + cut.chunk < cut.len ? t0 + cut.chunk : cut.len;
    const bool whole = cut.len <= cut.chunk;

    RowTile<D, GS> rows[RT];
#pragma unroll
    for (int u = 0; u < RT; ++u) {
        const int row = (rg * RT + u) * 16 + i;
        const bool have = row < count;
        const int tok = have ? row / a.group : 0;
        const uint16_t* q = a.q + (nt.row0 + tok) * a.q_row +
                            (static_cast<int64_t>(head) * a.group + (have ? row % a.group : 0)) * a.q_head + 8 * j;
        load_q<DT, D, GS>(rows[u], q, have, a.scale);
        rows[u].bits = !have ? 0 : a.mask != nullptr ? static_cast<uint64_t>(a.mask[nt.row0 + tok]) : ~uint64_t{0} >> (63 - tok);
        rows[u].m = kFar;
        rows[u].l = 0.0f;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            rows[u].bias[g] = 0.0f;
            rows[u].z[g] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) rows[u].o[n] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
    float ref_e = -100.0f;

    const Record rec(1 << a.s.page_shift, D, GS);
    const int mask_slot = (1 << a.s.page_shift) - 1;
    // page ids of 64 columns of the table, one a lane
    int ids = -1, col0 = -64;
    auto page_at = [&](int t) -> int {
        const int col = t >> a.s.page_shift;
        if (col >= col0 + 64) {
            col0 = col;
            const int64_t c = col + lane;
            ids = c < a.s.width ? a.s.tables[static_cast<int64_t>(b) * a.s.width + c] : -1;
            if (ids >= a.s.pages) ids = -1;
        }
        return __builtin_amdgcn_readlane(ids, col - col0);
    };
    uint32_t* ring = lds + wave * (kAttendSlots * L::kWords);
    const uint32_t ring_at = lds_address(ring);
    constexpr int kStride = 32 * kAttendWaves;
    // starts the loads of the step at token t; whether there are any
    auto fetch = [&](int t, int slot) -> bool {
        if (t >= t1) return false;
        const int page = page_at(t);
        if (page < 0) return false;
        const uint32_t* r = a.s.pool + (static_cast<int64_t>(page) * a.s.kv_heads + head) * rec.words();
        load_step<D, GS, NT_LOADS>(r, rec, t & mask_slot, lane, ring_at + 4 * slot * L::kWords);
        return true;
    };
    // steps in flight: slot n % kAttendSlots holds step n, `there` whether it has a page (bit 0: the next)
    unsigned there = 0;
#pragma unroll
    for (int n = 0; n < kAttendSlots - 1; ++n)
        there |= fetch(t0 + 32 * wave + n * kStride, n) ? 1u << n : 0u;
    int slot = 0;
    for (int t = t0 + 32 * wave; t < t1; t += kStride) {
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
            const uint32_t* x = ring + slot * L::kWords;
            if (t + 32 > nt.pos0)
                step<DT, D, GS, RT, true>(x, rows, ref_e, lane, t - nt.pos0, t1 - t);
            else
                step<DT, D, GS, RT, false>(x, rows, ref_e, lane, 0, 0);
        }
        slot = slot == kAttendSlots - 1 ? 0 : slot + 1;
    }
    __syncthreads();  // the slots become the sums' buffer

    // one set of sums: R and l first
#pragma unroll
    for (int u = 0; u < RT; ++u) {
        rows[u].l = sum_j(rows[u].l);
#pragma unroll
        for (int g = 0; g < G; ++g) rows[u].bias[g] = sum_j(rows[u].bias[g]);
        if (j == 0) {
            stat[wave][u][i][0] = rows[u].l > 0.0f ? rows[u].m + ref_e : kFar;
            stat[wave][u][i][1] = rows[u].l;
        }
    }
    __syncthreads();
    const int64_t part_row = ((static_cast<int64_t>(b) * a.s.kv_heads + head) * a.splits + part) * a.s.max_new * a.group;
#pragma unroll
    for (int u = 0; u < RT; ++u) {
        float ref = kFar;
#pragma unroll
        for (int w = 0; w < kAttendWaves; ++w) ref = fmaxf(ref, stat[w][u][i][0]);
        // (a wavefront that saw nothing has l = 0 and sums of 0)
        const float f = rows[u].l > 0.0f ? exp2_fast(rows[u].m + ref_e - ref) : 0.0f;
        const int out_row = (rg * RT + u) * 16 + threadIdx.x / 16;
#pragma unroll
        for (int d0 = 0; d0 < D; d0 += DC) {
#pragma unroll
            for (int n = d0 / 16; n < (d0 + DC) / 16; ++n) {
                const int g = 16 * n / GS;
                const float up = (n & 1) ? 0x1p20f : 0x1p24f;
                float4_t v;
#pragma unroll
                for (int r2 = 0; r2 < 4; ++r2)
                    v[r2] = f * (__builtin_fmaf(rows[u].o[n][r2], up, rows[u].bias[g]) - 8.0f * rows[u].z[g][r2]);
                *reinterpret_cast<float4_t*>(&buf[wave][i * kRow + 16 * n - d0 + 4 * j]) = v;
            }
            __syncthreads();
            // thread: row threadIdx / 16, DC / 16 values
            constexpr int PER = DC / 16;
            const int oi = threadIdx.x / 16, dd = (threadIdx.x % 16) * PER;
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
                l += stat[w][u][oi][1] > 0.0f ? stat[w][u][oi][1] * exp2_fast(stat[w][u][oi][0] - big) : 0.0f;
            if (out_row < count) {
                if (whole) {
                    const int tok = out_row / a.group;
                    const int64_t orow = (nt.row0 + tok) * a.heads + static_cast<int64_t>(head) * a.group + out_row % a.group;
                    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
                    uint32_t w[PER / 2];
#pragma unroll
                    for (int e = 0; e < PER / 2; ++e)
                        w[e] = static_cast<uint32_t>(DtOps<DT>::rne(o[2 * e] * inv)) |
                               (static_cast<uint32_t>(DtOps<DT>::rne(o[2 * e + 1] * inv)) << 16);
                    uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + orow * D + d0 + dd);
#pragma unroll
                    for (int e = 0; e < PER / 2; e += 2) *reinterpret_cast<uint2*>(dst + e) = make_uint2(w[e], w[e + 1]);
                    if (a.lse != nullptr && d0 == 0 && threadIdx.x % 16 == 0)
                        a.lse[orow] = l > 0.0f ? 0.693147180559945f * (big + __builtin_amdgcn_logf(l)) : -__builtin_inff();
                } else {
                    float* dst = a.part + (part_row + out_row) * (D + 2);
#pragma unroll
                    for (int e = 0; e < PER; e += 2) *reinterpret_cast<float2*>(dst + 2 + d0 + dd + e) = make_float2(o[e], o[e + 1]);
                    if (d0 == 0 && threadIdx.x % 16 == 0) *reinterpret_cast<float2*>(dst) = make_float2(l > 0.0f ? big : kFar, l);
                }
            }
            __syncthreads();
        }
    }
}

// The parts of sequences that were cut, put together: one wavefront a row.
template <int DT, int D>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendParams a) {
    constexpr int PER = D / 64;
    const int lane = threadIdx.x % 64;
    const int per_seq = a.s.max_new * a.heads;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / 64;
    const int64_t b64 = id / per_seq;
    if (b64 >= a.s.seqs) return;
    const int b = static_cast<int>(b64);
    const NewTokens nt = new_tokens(a.s, b);
    const int at = static_cast<int>(id % per_seq);
    const int head = at / (a.s.max_new * a.group), row = at % (a.s.max_new * a.group);
    if (row >= nt.n * a.group) return;
    const Cut cut = cut_of(a, nt);
    if (cut.len <= cut.chunk) return;
    const int parts = (cut.len + cut.chunk - 1) / cut.chunk;
    const int64_t stride = static_cast<int64_t>(a.s.max_new) * a.group * (D + 2);
    const float* p = a.part + ((static_cast<int64_t>(b) * a.s.kv_heads + head) * a.splits * a.s.max_new * a.group + row) * (D + 2);
    float ref = kFar;
    for (int k = lane; k < parts; k += 64) ref = fmaxf(ref, p[k * stride]);
#pragma unroll
    for (int m = 1; m < 64; m *= 2) ref = fmaxf(ref, __shfl_xor(ref, m));
    float l = 0.0f, o[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] = 0.0f;
    for (int k = 0; k < parts; ++k) {
        const float* c = p + k * stride;
        const float f = c[1] > 0.0f ? exp2_fast(c[0] - ref) : 0.0f;
        l += f * c[1];
#pragma unroll
        for (int e = 0; e < PER; ++e) o[e] += f * c[2 + lane * PER + e];
    }
    const int64_t orow = (nt.row0 + row / a.group) * a.heads + static_cast<int64_t>(head) * a.group + row % a.group;
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int e = 0; e < PER; ++e) a.out[orow * D + lane * PER + e] = DtOps<DT>::rne(o[e] * inv);
    if (a.lse != nullptr && lane == 0)
        a.lse[orow] = l > 0.0f ? 0.693147180559945f * (ref + __builtin_amdgcn_logf(l)) : -__builtin_inff();
}

template <int DT, int D, int GS, int RT, bool NT_LOADS>
hipError_t launch_attend_kernel(const AttendParams& p, int64_t blocks, hipStream_t st) {
    constexpr int kRow = (D < 128 ? D : 128) + 4;
    constexpr int slots = 4 * kAttendWaves * kAttendSlots * Slot<D, GS>::kWords;
    constexpr int sums = 4 * kAttendWaves * (16 * kRow + RT * 16 * 2);
    constexpr int bytes = slots > sums ? slots : sums;
    if constexpr (bytes > 64 * 1024) {
        static std::atomic<uint64_t> raised{0};
        const hipError_t e =
            raise_lds_limit(reinterpret_cast<const void*>(&attend_kernel<DT, D, GS, RT, NT_LOADS>), raised);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((attend_kernel<DT, D, GS, RT, NT_LOADS>), dim3(static_cast<unsigned>(blocks)),
                       dim3(64 * kAttendWaves), bytes, st, p);
    return hipGetLastError();
}

template <int DT, int D, int GS, int RT>
hipError_t run_attend(const AttendParams& p, int64_t blocks, hipStream_t st) {
    // tokens that several workgroups read stay in L2
    hipError_t e;
    if constexpr (RT == 1)
        e = launch_attend_kernel<DT, D, GS, RT, true>(p, blocks, st);
    else
        e = p.row_groups == 1 ? launch_attend_kernel<DT, D, GS, RT, true>(p, blocks, st)
                              : launch_attend_kernel<DT, D, GS, RT, false>(p, blocks, st);
    if (e != hipSuccess || p.splits == 1) return e;
    const int64_t rows = static_cast<int64_t>(p.s.seqs) * p.s.max_new * p.heads;
    hipLaunchKernelGGL((attend_join_kernel<DT, D>), dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(256), 0, st, p);
    return hipGetLastError();
}

// One translation unit per type and head size.
using AttendFn = hipError_t (*)(const AttendParams&, int64_t, hipStream_t);
template <int DT, int D>
AttendFn attend_fn(int gs, int row_tiles);

}  // namespace kv
}  // namespace qmm

// Instantiates attend_fn<DT, D> (two row tiles at most 16 rows apart share a wavefront).
#define QMM_KV_ATTEND_UNIT(DTV, DV)                                                       \
    namespace qmm {                                                                       \
    namespace kv {                                                                        \
    template <>                                                                           \
    AttendFn attend_fn<DTV, DV>(int gs, int row_tiles) {                                  \
        if (gs == 32) return row_tiles == 1 ? run_attend<DTV, DV, 32, 1> : run_attend<DTV, DV, 32, 2>; \
        if (gs == 64) return row_tiles == 1 ? run_attend<DTV, DV, 64, 1> : run_attend<DTV, DV, 64, 2>; \
        if constexpr (DV >= 128)                                                          \
            if (gs == 128) return row_tiles == 1 ? run_attend<DTV, DV, 128, 1> : run_attend<DTV, DV, 128, 2>; \
        return nullptr;                                                                   \
    }                                                                                     \
    }                                                                                     \
    }
