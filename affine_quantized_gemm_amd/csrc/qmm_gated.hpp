// Gated block on quantized weights (gfx950): h = act(x Wg^T) * (x Wu^T) with
// W = [Wg; Wu] quantized along K, both products, the activation and the
// product of the two in one kernel; with a gradient of h in its place the
// gradients of the two products, [dh u act'(g), dh act(g)].
//
// Mathematics.  As in the other products (qmm_mfma_frag.hpp): the matrix cores
// multiply x with q + off, codes as exact fp16 / bf16 numbers, and
//   sum_k x w = sum_u s_u P_u + (b_u - off s_u) X_u
// over groups u, P_u = sum x (q + off), X_u = sum x.  All offsets of a format
// are alike here, so the second term is one fp32 matrix step (16x16x4) for
// four groups, exact to fp32.  Both products stay in fp32 through the
// activation; h is rounded once.
//
// Split.  A wavefront owns 16 columns of the gate and the same 16 of the other
// product (their x operand is read once for both, and both values of an output
// end in the same lane), RT tiles of 16 rows, and a share of K: superblocks of
// 128 bytes of codes a row (6-bit: 96), a KS-th of them.  A workgroup is W
// wavefronts, KS shares of K for W / KS column tiles.  x goes through LDS in
// chunks (rows padded by 16 bytes: 16 rows' pieces then lie in different
// banks), its groups' sums beside it.
//
// Loads.  A matrix operand has the 16 columns on neighbouring lanes: loaded so,
// every lane's 16 bytes are an access of their own to the vector cache (8.3
// million of them for 66 MB: 26 us whatever the split).  So a wavefront loads
// its rows' codes as whole lines into registers, two superblocks ahead, and
// turns them in an LDS slot of its own; the scales and biases of the 2 x 16
// rows come with one load, an array on each quarter of the lanes.
//
// Measured (4 bits, groups of 64, unless said): 5 rows, 1024 to 2 x 2048, 5.0
// us (start, one superblock or two, join; 0.3 of reading); 6 rows, 4096 to 2 x
// 14336, 19.5 us (3.4 TB/s; 9.4 of reading).  There 224 workgroups of 16
// wavefronts at 127 registers and 136 KB of LDS fill a CU each, 32 CUs are left
// empty, and a wavefront takes 4 superblocks in all, two of them on their way
// and each turned in LDS: 43 % of the wavefronts' time is waiting for data or a
// barrier, 36 % for a unit.  (The register kernel of the plain product reads the
// same bytes as two products of 14336 columns in 16.3 us.)  64 rows, 6 bits,
// groups of 128, the same widths, 54 us (278 TFLOP/s; 13.4 of reading): x of 64
// rows goes through LDS in 8 chunks with two barriers around each, and two
// wavefronts a SIMD, 207 registers, turn and widen the codes in between; vector
// units busy 36 % of the time, matrix cores 10 %, 37 % of LDS's busy cycles are
// conflicts.  With a gradient, 37 rows, 4 bits, 39.5 us (30 %, 16 %, 28 %).
#pragma once

#include "qmm_device.hpp"
#include "qmm_internal.hpp"
#include "qmm_mfma_frag.hpp"
#include "qmm_rows.hpp"

namespace qmm {
namespace gated {

using mf::float4_t;
using mf::Frag;

// Wavefronts of a workgroup: the registers of one row tile leave room for four
// a SIMD; where those make few workgroups, four (5 rows, 1024 to 2 x 2048: 8.3
// us with 16).
constexpr int waves_of(int rt, bool few) { return few ? 4 : rt == 1 ? 16 : 8; }
constexpr int super_of(int bits) { return bits == 4 ? 256 : 128; }      // codes of a superblock
constexpr int super_bytes(int bits) { return super_of(bits) * bits / 8; }
constexpr int row_stride(int bits) { return super_bytes(bits) + 16; }   // of a slot
// Bytes of a wavefront's LDS: 2 x 16 rows of codes, then their scales and
// biases; at a tile's end its share of the sums.
constexpr int slot_bytes(int bits, int gs, int rt) {
    const int groups = super_of(bits) / gs, slot = 32 * row_stride(bits) + 128 * (groups > 1 ? groups : 2), sums = 2048 * rt;
    return slot > sums ? slot : sums;
}
constexpr int kLds = 158 * 1024;
constexpr int sums_of(int rt) { return 16 * rt + 4; }                   // floats of a group's sums of x
// 16-byte pieces of x that a thread has on their way; with several row tiles, whose x goes through LDS in many chunks,
// the whole next chunk (the loads behind the weights' took as long as the products: 64 rows 41 us).
constexpr int pieces_of(int rt) { return rt == 1 ? 4 : 8; }

struct GatedParams {
    const uint16_t* x;
    const uint32_t* wq;
    const uint16_t* scales;
    const uint16_t* biases;
    const uint16_t* grad;
    uint16_t* out;
    float* d;         // with grad: the two gradients in fp32 as well, [M][2F]
    int M, act;
    int64_t F, K;
    int words;        // uint32 of a weight row
    int groups;       // of a weight row
    int chunk;        // codes of x in LDS at a time, a power of two: superblocks of all shares
    int chunks;
    int supers;       // superblocks of K
    int per;          // of a share, an even number where workgroups have several tiles; share s has those from s * per on
    int steps_shift;  // a chunk of x has 1 << steps_shift steps of each share
    int piece_shift;  // and 1 << piece_shift pieces of 16 bytes a row
    int ks_shift;     // KS = 1 << ks_shift
    int tiles;        // column tile groups of the grid: ceil(F / (16 * W / KS))
};

namespace {

enum { ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2, ACT_RELU = 3 };

// act(a) and act'(a).
struct Act {
    float value, slope;
};
__device__ __forceinline__ Act activation(int act, float a) {
    constexpr float log2e = 1.44269504088896341f;
    Act r;
    if (act == ACT_SILU) {
        // (a far below 0: exp is infinite, s and r 0; an infinite a gives NaN where it meets that 0)
        const float s = 1.0f / (1.0f + __builtin_amdgcn_exp2f(-a * log2e));
        r.value = a * s;
        r.slope = s * (1.0f + a * (1.0f - s));
    } else if (act == ACT_RELU) {
        // (NaN stays NaN)
        r.value = a > 0.0f ? a : a != a ? a : 0.0f;
        r.slope = a > 0.0f ? 1.0f : a != a ? a : 0.0f;
    } else if (act == ACT_GELU) {
        // half erfc of -a / sqrt 2: exact also where it is small
        const float phi = 0.5f * erfcf(-a * 0.707106781186547524f);
        r.value = a * phi;
        r.slope = phi + a * 0.398942280401432678f * __builtin_amdgcn_exp2f(-0.5f * log2e * a * a);
    } else {
        // 0.5 (1 + tanh t) = 1 / (1 + exp(-2 t)), t = sqrt(2 / pi) (a + 0.044715 a^3)
        constexpr float r2 = 1.59576912160573071f;
        const float a2 = fminf(a * a, 1e18f);  // (s is 0 or 1 long before)
        const float s = 1.0f / (1.0f + __builtin_amdgcn_exp2f(-log2e * r2 * a * (1.0f + 0.044715f * a2)));
        r.value = a * s;
        r.slope = s + a * s * (1.0f - s) * r2 * (1.0f + 0.134145f * a2);
    }
    return r;
}

// One superblock of 2 x 16 rows on its way: whole lines of codes, and this
// quarter's array of scales or biases (gate's scales, gate's biases, the
// other's scales, the other's biases) of row i.
template <int BITS, int GS>
struct Super {
    static constexpr int LOADS = 4;                          // of 16 bytes a lane (6-bit: the last 32 lanes of every second one repeat)
    static constexpr int GP = super_of(BITS) / GS, GW = GP > 1 ? GP / 2 : 1;
    mf::u32x4_t w[LOADS];
    uint32_t sb[GW];
};

// GP 16-bit values as words.
template <int GP, int GW>
__device__ __forceinline__ void load_halves(const char* p, uint32_t (&d)[GW]) {
    if constexpr (GP == 1) d[0] = *reinterpret_cast<const uint16_t*>(p);
    else mf::load_words<GW>(reinterpret_cast<const uint16_t*>(p), d);
}

// sum + the two halves of a word.
template <int DT>
__device__ __forceinline__ float half_sum(uint32_t w, float one, float sum) {
    if constexpr (DT == DT_F16) {
        sum = __builtin_fmaf(low_f32<DT>(w), one, sum);
        return __builtin_fmaf(high_f32<DT>(w), one, sum);
    } else {
        typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, w), __builtin_bit_cast(bf16x2_t, 0x3F803F80u), sum, false);
    }
}

// Sum over 4, 8 or 16 neighbouring lanes, in each of them.
template <int N>
__device__ __forceinline__ float lanes_sum(float v) {
    auto add = [](float a, int b) { return a + __builtin_bit_cast(float, b); };
    auto bits = [](float a) { return __builtin_bit_cast(int, a); };
    v = add(v, __builtin_amdgcn_update_dpp(0, bits(v), 0xB1, 0xf, 0xf, true));   // lane ^ 1
    v = add(v, __builtin_amdgcn_update_dpp(0, bits(v), 0x4E, 0xf, 0xf, true));   // lane ^ 2
    if constexpr (N >= 8) v = add(v, __builtin_amdgcn_update_dpp(0, bits(v), 0x141, 0xf, 0xf, true));   // mirrored in 8
    if constexpr (N >= 16) v = add(v, __builtin_amdgcn_update_dpp(0, bits(v), 0x140, 0xf, 0xf, true));  // mirrored in 16
    return v;
}

}  // namespace

// VEC: superblocks are whole and their scales one aligned load; without it
// each is looked at by itself, clamped into the row (what lies past it meets
// an x of 0).
template <int DT, int BITS, int GS, int RT, bool FEW, bool VEC>
__global__ __launch_bounds__(64 * waves_of(RT, FEW), RT == 1 ? 4 : 2) void gated_kernel(GatedParams p) {
    using F = mf::Fmt<DT, BITS, GS>;
    using S = Super<BITS, GS>;
    constexpr int W = waves_of(RT, FEW), kThreads = 64 * W, kSuper = super_of(BITS);
    constexpr int NB = kSuper / F::KBLK, GP = S::GP, GW = S::GW, SEGW = F::SEG_WORDS, STEPS = F::STEPS;
    constexpr int ROW = super_bytes(BITS), STRIDE = row_stride(BITS), PIECES = ROW / 16;
    static_assert(NB == 2 && 16 * PIECES <= 128, "a superblock");
    constexpr bool UNI = DT == DT_F16 && BITS == 4;
    constexpr float OFF = DT == DT_F16 ? 1024.0f : BITS == 8 ? 0.0f : 128.0f;
    extern __shared__ __align__(16) char lds[];
    const int lane = threadIdx.x % 64, i = lane % 16, j = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int KS = 1 << p.ks_shift, CT = W >> p.ks_shift;
    const int ks = wave & (KS - 1), ct = wave >> p.ks_shift;
    const int row0 = blockIdx.y * 16 * RT;
    const int rows = p.M - row0 < 16 * RT ? p.M - row0 : 16 * RT;
    const int x_stride = 2 * p.chunk + 16;                 // bytes of a row of x in LDS
    constexpr int SLOT = slot_bytes(BITS, GS, RT);
    char* const slot = lds + wave * SLOT;                  // [32][STRIDE] codes, then [4][16][GP] scales and biases
    char* const slot_sb = slot + 32 * STRIDE;
    char* const x_lds = lds + W * SLOT;
    float* const sums = reinterpret_cast<float*>(x_lds + rows * x_stride);  // [chunk's groups][sum_stride], a row's in place
    constexpr int sum_stride = sums_of(RT);
    constexpr int kPieces = pieces_of(RT);
    const mf::UnpackConsts consts = mf::unpack_consts<DT>();

    // ---- x: pieces of 8 values, neighbouring threads on neighbouring pieces of a row ----
    // A row of a chunk is a power of two of pieces, at most the threads: a thread has the same place in every `pass`-th row
    // from row `r0` on, and its addresses are one offset and uniform steps.  (With a division and 64-bit addresses for every
    // piece, and the sums by conversions and adds, this was 70 vector instructions a piece: 64 rows 45 us, of which a
    // third was that.)
    const int pass = kThreads >> p.piece_shift;
    struct XPlace {
        int r0, at;  // first row, piece of it
        int k;       // code within the chunk's shares
    };
    auto x_place = [&]() -> XPlace {
        // (from the thread's number anew each time: else kept in registers throughout)
        int tid = threadIdx.x;
        asm volatile("" : "+v"(tid));
        XPlace x;
        x.r0 = tid >> p.piece_shift;
        x.at = tid & ((1 << p.piece_shift) - 1);
        // superblock `local` of the chunk is step local % steps (of the chunk's) of share local / steps
        const int local = x.at / (kSuper / 8);
        x.k = ((local >> p.steps_shift) * p.per + (local & ((1 << p.steps_shift) - 1))) * kSuper + 8 * (x.at % (kSuper / 8));
        return x;
    };
    // (not 1 to the compiler: a product with it takes halves of a word as they are)
    float one = 1.0f;
    asm volatile("" : "+s"(one));
    // thread's pieces n0, n0 + 1, .. of chunk c
    auto fetch_x = [&](int c, int n0, uint4 (&xs)[kPieces]) {
        const XPlace x = x_place();
        const int k = (c << p.steps_shift) * kSuper;
        const char* const base = reinterpret_cast<const char*>(p.x + static_cast<int64_t>(row0) * p.K + k);
        const uint32_t off = 2 * (x.r0 * static_cast<uint32_t>(p.K) + x.k);
#pragma unroll
        for (int m = 0; m < kPieces; ++m) {
            xs[m] = make_uint4(0, 0, 0, 0);
            if (x.r0 + (n0 + m) * pass < rows && x.k + k < p.K)
                xs[m] = *reinterpret_cast<const uint4*>(base + static_cast<int64_t>((n0 + m) * pass) * (2 * p.K) + off);
        }
    };
    auto store_x = [&](int n0, const uint4 (&xs)[kPieces]) {
        const XPlace x = x_place();
        char* const to = x_lds + x.r0 * x_stride + 16 * x.at;
        float* const sum_to = sums + x.at / (GS / 8) * sum_stride + x.r0;
#pragma unroll
        for (int m = 0; m < kPieces; ++m) {
            if ((n0 + m) * pass >= rows) break;
            const uint4 u = xs[m];
            float sum = lanes_sum<GS / 8>(half_sum<DT>(u.x, one, half_sum<DT>(u.y, one, 0.0f)) + half_sum<DT>(u.z, one, half_sum<DT>(u.w, one, 0.0f)));
            if (x.r0 + (n0 + m) * pass < rows) {
                const Frag f = mf::x_frag<BITS, DT>(u);
                *reinterpret_cast<uint4*>(to + (n0 + m) * pass * x_stride) = make_uint4(f.v[0], f.v[1], f.v[2], f.v[3]);
                if (x.at % (GS / 8) == 0) sum_to[(n0 + m) * pass] = sum;
            }
        }
    };

    // ---- weights: uniform bases, and a lane's offsets fixed for the kernel ----
    const int64_t row_bytes = 4 * static_cast<int64_t>(p.words), group_bytes = 2 * static_cast<int64_t>(p.groups);
    const int last_row = p.F < 16 ? static_cast<int>(p.F) - 1 : 15;
    // load q: matrix q / 2, pieces 64 (q % 2) + lane of its 16 rows (row-major)
    uint32_t w_off[2], slot_at[2];
    int piece[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const int at = 64 * n + lane < 16 * PIECES ? 64 * n + lane : 16 * PIECES - 1, r = at / PIECES;
        piece[n] = 16 * (at % PIECES);
        w_off[n] = (r < last_row ? r : last_row) * static_cast<uint32_t>(row_bytes) + (VEC ? piece[n] : 0);
        slot_at[n] = r * STRIDE + piece[n];
    }
    const char* const sb_lane = reinterpret_cast<const char*>(j & 1 ? p.biases : p.scales) + ((j >> 1) * p.F + (i < last_row ? i : last_row)) * group_bytes;
    // first column of the wavefront's tile: the last one is moved back to end with the columns (their values come out alike)
    auto first_col = [&](int tile) {
        const int64_t n = (static_cast<int64_t>(tile) * CT + ct) * 16;
        return n + 16 <= p.F ? n : p.F > 16 ? p.F - 16 : 0;
    };
    auto load = [&](S& buf, int64_t col, int sb) {
#pragma unroll
        for (int q = 0; q < S::LOADS; ++q) {
            const char* const base = reinterpret_cast<const char*>(p.wq) + ((q / 2) * p.F + col) * row_bytes;
            if constexpr (VEC) {
                buf.w[q] = __builtin_nontemporal_load(reinterpret_cast<const mf::u32x4_t*>(base + static_cast<int64_t>(sb) * ROW + w_off[q % 2]));
            } else {
                const uint32_t in = sb * ROW + piece[q % 2], most = static_cast<uint32_t>(row_bytes) - 16;
                buf.w[q] = *reinterpret_cast<const mf::u32x4_t*>(base + (w_off[q % 2] + (in < most ? in : most)));
            }
        }
        const char* const from = sb_lane + col * group_bytes;
        if constexpr (VEC) {
            load_halves<GP>(from + sb * (2 * GP), buf.sb);
        } else {
#pragma unroll
            for (int g = 0; g < GW; ++g) {
                const int g0 = sb * GP + 2 * g, last = p.groups - 1;
                const uint16_t* const v = reinterpret_cast<const uint16_t*>(from);
                buf.sb[g] = v[g0 < last ? g0 : last] | static_cast<uint32_t>(v[g0 + 1 < last ? g0 + 1 : last]) << 16;
            }
        }
    };
    auto turn = [&](const S& buf) {
#pragma unroll
        for (int q = 0; q < S::LOADS; ++q) *reinterpret_cast<mf::u32x4_t*>(slot + (q / 2) * (16 * STRIDE) + slot_at[q % 2]) = buf.w[q];
        uint32_t* const at = reinterpret_cast<uint32_t*>(slot_sb + lane * (4 * GW));
        if constexpr (GW == 4) *reinterpret_cast<uint4*>(at) = make_uint4(buf.sb[0], buf.sb[1], buf.sb[2], buf.sb[3]);
        else if constexpr (GW == 2) *reinterpret_cast<uint2*>(at) = make_uint2(buf.sb[0], buf.sb[1]);
        else *at = buf.sb[0];
    };

    float4_t acc[2][RT];
    auto clear = [&] {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < RT; ++t) acc[h][t] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    };
    // natural place in a k-block of the 8 codes of step s and lane quarter q: place(s, 0) + place(0, q)
    auto place = [](int s, int q) { return F::src_lane(s, q) * F::SEG + F::src_slot(s, q) * 8; };
    // this lane's row of each tile in LDS (rows past the last one: the last one, never stored)
    int x_row[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int r = 16 * t + i < rows ? 16 * t + i : rows - 1;
        x_row[t] = r * x_stride + 2 * place(0, j);
    }
    // takes one of four halves of two words as fp32 (bf16), or into a word's low half
    constexpr int QUARTERS = GP < 4 ? GP : 4;  // that have a group
    const uint32_t quarter = j & (QUARTERS - 1);
    const uint32_t pick = DT == DT_BF16 ? (2 * quarter + 1) << 24 | (2 * quarter) << 16 | 0x0C0Cu : 0x0C0C0000u | (2 * quarter + 1) << 8 | 2 * quarter;
    auto picked = [&](const uint32_t (&w)[GW], int n) {
        const uint32_t h = __builtin_amdgcn_perm(w[(2 * n + 1) % GW], w[2 * n % GW], pick);
        return DT == DT_BF16 ? __builtin_bit_cast(float, h) : low_f32<DT_F16>(h);
    };
    const char* const codes = slot + i * STRIDE + j * (4 * SEGW);
    const uint32_t* const row_sb = reinterpret_cast<const uint32_t*>(slot_sb + i * (4 * GW));
    auto multiply = [&](int at) {  // at: superblock within the chunk
        const char* const x0 = x_lds + at * (2 * kSuper);
        uint32_t sc[2][GW], bi[2][GW];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int g = 0; g < GW; ++g) {
                sc[h][g] = row_sb[(2 * h) * (16 * GW) + g];
                bi[h][g] = row_sb[(2 * h + 1) * (16 * GW) + g];
            }
        float4_t P[2][RT];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            __builtin_amdgcn_sched_barrier(0);
            Frag w[2][STEPS];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t seg[SEGW];
                const uint32_t* const from = reinterpret_cast<const uint32_t*>(codes + h * (16 * STRIDE) + nb * (F::KBLK * BITS / 8));
                if constexpr (SEGW == 4) {
                    const uint4 v = *reinterpret_cast<const uint4*>(from);
                    seg[0] = v.x; seg[1] = v.y; seg[2] = v.z; seg[3] = v.w;
                } else {
#pragma unroll
                    for (int e = 0; e < SEGW; ++e) seg[e] = from[e];
                }
                mf::segment_frags<DT, BITS, GS, SEGW, STEPS, UNI>(seg, w[h], consts);
            }
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int step = nb * STEPS + s;                       // of the superblock
                const bool first = 32 * step % GS == 0, last = 32 * (step + 1) % GS == 0;
                const int g = 32 * step / GS;
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const uint4 u = *reinterpret_cast<const uint4*>(x0 + x_row[t] + 2 * (F::KBLK * nb + place(s, 0)));
                    const Frag a{{u.x, u.y, u.z, u.w}};
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        P[h][t] = mf::mfma<DT>(a, w[h][s], first ? float4_t{0.0f, 0.0f, 0.0f, 0.0f} : P[h][t]);
                }
                if (last) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float v = (g & 1) ? high_f32<DT>(sc[h][g / 2]) : low_f32<DT>(sc[h][g / 2]);
#pragma unroll
                        for (int t = 0; t < RT; ++t)
#pragma unroll
                            for (int r = 0; r < 4; ++r) acc[h][t][r] = __builtin_fmaf(v, P[h][t][r], acc[h][t][r]);
                    }
                }
            }
        }
        // biases and offsets against the groups' sums of x
        if constexpr (GP == 1) {
            // one group: on the vector ALUs (a matrix step would be three quarters empty)
            const float* const from = sums + at * sum_stride + 4 * j;
            float cb[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) cb[h] = __builtin_fmaf(-OFF, low_f32<DT>(sc[h][0]), low_f32<DT>(bi[h][0]));
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const float4_t x4 = *reinterpret_cast<const float4_t*>(from + 16 * t);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[h][t][r] = __builtin_fmaf(cb[h], x4[r], acc[h][t][r]);
            }
        } else {
            // lane quarter j takes group 4 n + j
#pragma unroll
            for (int n = 0; n < (GP + 3) / 4; ++n) {
                float cb[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    cb[h] = __builtin_fmaf(-OFF, picked(sc[h], n), picked(bi[h], n));
                    if (QUARTERS < 4 && j >= QUARTERS) cb[h] = 0.0f;
                }
                const float* const from = sums + (at * GP + 4 * n + static_cast<int>(quarter)) * sum_stride + i;
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    // (rows past the last one may hold anything: their results are not stored)
                    const float xsum = from[16 * t];
#pragma unroll
                    for (int h = 0; h < 2; ++h) acc[h][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(xsum, cb[h], acc[h][t], 0, 0, 0);
                }
            }
        }
    };

    auto end_tile = [&](int at_tile) {
        const int64_t col = first_col(at_tile) + i, from = (static_cast<int64_t>(at_tile) * CT + ct) * 16;
        auto finish = [&](int t, int r, float gate, float up) {
            const int row = 16 * t + 4 * j + r;
            if (row >= rows || col >= p.F || col < from) return;
            const Act v = activation(p.act, gate);
            const int64_t m = row0 + row;
            if (p.grad == nullptr) {
                p.out[m * p.F + col] = static_cast<uint16_t>(pack2<DT>(v.value * up, 0.0f));
            } else {
                const float d = DtOps<DT>::to_f32(p.grad[m * p.F + col]), dg = d * up * v.slope, du = d * v.value;
                const int64_t at = m * 2 * p.F + col;
                p.out[at] = static_cast<uint16_t>(pack2<DT>(dg, 0.0f));
                p.out[at + p.F] = static_cast<uint16_t>(pack2<DT>(du, 0.0f));
                p.d[at] = dg;
                p.d[at + p.F] = du;
            }
        };
        // the shares of K meet in the wavefronts' slots, [2][RT][4][64] each; the KS wavefronts of a tile take values in turn
        auto part = [&](int w) { return reinterpret_cast<float*>(lds + w * SLOT) + lane; };
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) part(wave)[64 * ((h * RT + t) * 4 + r)] = acc[h][t][r];
        __syncthreads();
#pragma unroll 1
        for (int v = ks; v < 4 * RT; v += KS) {
            float two[2] = {0.0f, 0.0f};
#pragma unroll 4
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int h = 0; h < 2; ++h) two[h] += part(ct * KS + s)[64 * (h * RT * 4 + v)];
            finish(v / 4, v % 4, two[0], two[1]);
        }
        __syncthreads();
    };

    // The wavefront's steps: its share of the superblocks, p.per of them, of each of the workgroup's tiles in turn (ones
    // past K multiply nothing).
    const int stride = gridDim.x;
    // loads are issued for every step, past the last one and past K too (the tile's first bytes again): a load under a
    // branch makes the waits for all others wait for everything
    S buf[2];
    int ahead_tile = blockIdx.x, ahead = 0;   // to be asked for next
    if (ahead_tile >= p.tiles) return;
    auto ask = [&](S& to, int tile) {
        const int sb = ks * p.per + ahead;
        const bool there = ahead_tile < p.tiles && sb < p.supers;
        load(to, first_col(there ? ahead_tile : tile), there ? sb : 0);
        if (++ahead == p.per) {
            ahead = 0;
            ahead_tile += stride;
        }
    };
    // x is asked for before any weights (behind them it comes when the first 2 W superblocks have, 6 us of a workgroup's
    // 18), and the second superblocks when it is there
    uint4 xs[kPieces];
    int chunk = 0;  // in LDS; RT > 1: the one after it is in xs
    auto restage = [&](int c) {
        if constexpr (RT > 1) {
            store_x(0, xs);
            __syncthreads();
            fetch_x(c + 1 < p.chunks ? c + 1 : 0, 0, xs);
        } else {
#pragma unroll 1
                for (int n = 0; n * pass < rows; n += kPieces) {
                fetch_x(c, n, xs);
                store_x(n, xs);
            }
            __syncthreads();
        }
        chunk = c;
    };
    fetch_x(0, 0, xs);
    __builtin_amdgcn_s_barrier();
    ask(buf[0], blockIdx.x);
    store_x(0, xs);
#pragma unroll 1
    for (int n = kPieces; n * pass < rows; n += kPieces) {
        fetch_x(0, n, xs);
        store_x(n, xs);
    }
    __syncthreads();
    ask(buf[1], blockIdx.x);
    if (RT > 1 && p.chunks > 1) fetch_x(1, 0, xs);
    for (int tile = blockIdx.x; tile < p.tiles; tile += stride) {
        clear();
        if (chunk != 0) restage(0);  // (a tile ends with a barrier)
        int at = 0;                  // step within the chunk of x
        auto take = [&](S& now, int step) {
            if (at == 1 << p.steps_shift) {
                __syncthreads();     // the chunk before is not read any more
                restage(chunk + 1);
                at = 0;
            }
            turn(now);
            ask(now, tile);
            if (ks * p.per + step < p.supers) multiply((ks << p.steps_shift) + at);
            ++at;
        };
#pragma unroll 1
        for (int step = 0; step < p.per; step += 2) {
            take(buf[0], step);
            if (step + 1 < p.per) take(buf[1], step + 1);
        }
        end_tile(tile);
    }
}

// Bytes of LDS: the wavefronts' slots, x and its groups' sums.
inline int lds_bytes(int bits, int gs, int rt, int waves, int rows, int chunk) {
    return waves * slot_bytes(bits, gs, rt) + rows * (2 * chunk + 16) + 4 * (chunk / gs) * sums_of(rt);
}

template <int DT, int BITS, int GS, int RT, bool FEW, bool VEC>
hipError_t launch(const GatedParams& p, dim3 grid, int bytes, hipStream_t st) {
    if (bytes > 64 * 1024) {
        static std::atomic<uint64_t> raised{0};
        const hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(&gated_kernel<DT, BITS, GS, RT, FEW, VEC>), raised);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((gated_kernel<DT, BITS, GS, RT, FEW, VEC>), grid, dim3(64 * waves_of(RT, FEW)), bytes, st, p);
    return hipGetLastError();
}

template <int DT, int BITS, int GS>
hipError_t run(const GatedParams& p, int rt, bool few, bool vec, dim3 grid, int bytes, hipStream_t st) {
    if (!vec) return few ? launch<DT, BITS, GS, 1, true, false>(p, grid, bytes, st) : launch<DT, BITS, GS, 1, false, false>(p, grid, bytes, st);
    if (rt == 1) return few ? launch<DT, BITS, GS, 1, true, true>(p, grid, bytes, st) : launch<DT, BITS, GS, 1, false, true>(p, grid, bytes, st);
    if (rt == 2) return launch<DT, BITS, GS, 2, false, true>(p, grid, bytes, st);
    return launch<DT, BITS, GS, 4, false, true>(p, grid, bytes, st);
}

// One translation unit per type and code width.
using GatedFn = hipError_t (*)(const GatedParams&, int rt, bool few, bool vec, dim3, int, hipStream_t);
template <int DT, int BITS>
GatedFn gated_fn(int gs);

}  // namespace gated
}  // namespace qmm

#define QMM_GATED_UNIT(DTV, BITSV)                            \
    namespace qmm {                                           \
    namespace gated {                                         \
    template <>                                               \
    GatedFn gated_fn<DTV, BITSV>(int gs) {                    \
        if (gs == 32) return run<DTV, BITSV, 32>;             \
        if (gs == 64) return run<DTV, BITSV, 64>;             \
        return gs == 128 ? run<DTV, BITSV, 128> : nullptr;    \
    }                                                         \
    }                                                         \
    }
