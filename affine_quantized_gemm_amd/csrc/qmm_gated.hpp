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
// 256 codes, every KS-th one.  A workgroup is 8 wavefronts, KS shares of K for
// 8 / KS column tiles.  x goes through LDS in chunks (rows padded by 16 bytes:
// 16 rows' pieces then lie in different banks), its groups' sums beside it;
// weights go straight to registers, one superblock ahead.
#pragma once

#include "qmm_device.hpp"
#include "qmm_internal.hpp"
#include "qmm_mfma_frag.hpp"
#include "qmm_rows.hpp"

namespace qmm {
namespace gated {

using mf::float4_t;
using mf::Frag;

constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kSuper = 256;              // codes of a superblock
constexpr int kChunkBytes = 64 * 1024;   // of x in LDS at a time, at most
constexpr int kAhead = 4;                // 16-byte pieces of x that a thread has on their way

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
    int chunk;        // codes of x in LDS at a time, a multiple of kSuper * KS
    int chunks;
    int supers;       // superblocks of K
    int ks_shift;     // KS = 1 << ks_shift
    int tiles;        // column tile groups of the grid: ceil(F / (16 * 8 / KS))
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
        // (a far below 0: exp is infinite, s and r 0; infinite times 0 does not arise, a is finite)
        const float s = 1.0f / (1.0f + __builtin_amdgcn_exp2f(-a * log2e));
        r.value = a * s;
        r.slope = s * (1.0f + a * (1.0f - s));
    } else if (act == ACT_RELU) {
        r.value = fmaxf(a, 0.0f);
        r.slope = a > 0.0f ? 1.0f : 0.0f;
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

// One superblock of a column's row as it comes from memory.
template <int DT, int BITS, int GS>
struct Super {
    using F = mf::Fmt<DT, BITS, GS>;
    static constexpr int NB = kSuper / F::KBLK, GP = kSuper / GS, GW = GP / 2;
    uint32_t w[NB][F::SEG_WORDS];
    uint32_t s[GW], b[GW];  // scales and biases of its groups, two a word
};

template <int N>
__device__ __forceinline__ void load_scales(const uint16_t* p, uint32_t (&d)[N]) {
    mf::load_words<N>(p, d);
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

// VEC: K is a multiple of 256, so that superblocks are whole and their scales
// one aligned load; without it each is looked at by itself, clamped into the
// row (what lies past it meets an x of 0).
template <int DT, int BITS, int GS, int RT, bool VEC>
__global__ __launch_bounds__(kThreads, RT == 1 ? 4 : 2) void gated_kernel(GatedParams p) {
    using F = mf::Fmt<DT, BITS, GS>;
    using S = Super<DT, BITS, GS>;
    constexpr int NB = S::NB, GP = S::GP, GW = S::GW, SEGW = F::SEG_WORDS, STEPS = F::STEPS;
    constexpr bool UNI = DT == DT_F16 && BITS == 4;
    constexpr float OFF = DT == DT_F16 ? 1024.0f : BITS == 8 ? 0.0f : 128.0f;
    extern __shared__ __align__(16) char lds[];
    const int lane = threadIdx.x % 64, i = lane % 16, j = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int KS = 1 << p.ks_shift, CT = kWaves >> p.ks_shift;
    const int ks = wave & (KS - 1), ct = wave >> p.ks_shift;
    const int row0 = blockIdx.y * 16 * RT;
    const int rows = p.M - row0 < 16 * RT ? p.M - row0 : 16 * RT;
    const int x_stride = 2 * p.chunk + 16;                 // bytes of a row of x in LDS
    const int chunk_groups = p.chunk / GS;
    char* const x_lds = lds;
    float* const sums = reinterpret_cast<float*>(lds + rows * x_stride);  // [rows][chunk_groups + 1]
    const int sum_stride = chunk_groups + 1;
    const mf::UnpackConsts consts = mf::unpack_consts<DT>();

    // ---- x: pieces of 8 values, neighbouring threads on neighbouring pieces of a row ----
    const int row_pieces = p.chunk / 8, pieces = rows * row_pieces;
    auto stage_x = [&](int c) {
#pragma unroll 1
        for (int n = 0; n * kThreads < pieces; n += kAhead) {
            uint4 xs[kAhead];
            int r[kAhead], at[kAhead];
#pragma unroll
            for (int m = 0; m < kAhead; ++m) {
                const int q = threadIdx.x + (n + m) * kThreads;
                r[m] = q / row_pieces;
                at[m] = q - r[m] * row_pieces;
                const int64_t k = static_cast<int64_t>(c) * p.chunk + 8 * at[m];
                xs[m] = make_uint4(0, 0, 0, 0);
                if (q < pieces && k < p.K) xs[m] = *reinterpret_cast<const uint4*>(p.x + (row0 + r[m]) * p.K + k);
            }
#pragma unroll
            for (int m = 0; m < kAhead; ++m) {
                const uint4 u = xs[m];
                float sum = (low_f32<DT>(u.x) + high_f32<DT>(u.x)) + (low_f32<DT>(u.y) + high_f32<DT>(u.y)) +
                            ((low_f32<DT>(u.z) + high_f32<DT>(u.z)) + (low_f32<DT>(u.w) + high_f32<DT>(u.w)));
                sum = lanes_sum<GS / 8>(sum);
                if (static_cast<int>(threadIdx.x) + (n + m) * kThreads < pieces) {
                    const Frag f = mf::x_frag<BITS, DT>(u);
                    *reinterpret_cast<uint4*>(x_lds + r[m] * x_stride + 16 * at[m]) = make_uint4(f.v[0], f.v[1], f.v[2], f.v[3]);
                    if (at[m] % (GS / 8) == 0) sums[r[m] * sum_stride + at[m] / (GS / 8)] = sum;
                }
            }
        }
    };

    // ---- weights ----
    const int64_t row_groups = p.groups;
    auto load = [&](S (&buf)[2], int tile, int sb) {
        const int64_t col0 = (static_cast<int64_t>(tile) * CT + ct) * 16;
        const int64_t col = col0 + i < p.F ? col0 + i : p.F - 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t row = h * p.F + col;
            const uint32_t* w = p.wq + row * p.words;
            const uint16_t* sc = p.scales + row * row_groups;
            const uint16_t* bi = p.biases + row * row_groups;
            if constexpr (VEC) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                    mf::load_segment<BITS, SEGW, true>(w + (sb * (kSuper / 32) * BITS) + nb * (F::KBLK * BITS / 32) + j * SEGW, buf[h].w[nb]);
                load_scales(sc + sb * GP, buf[h].s);
                load_scales(bi + sb * GP, buf[h].b);
            } else {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    int at = sb * (kSuper / 32) * BITS + nb * (F::KBLK * BITS / 32) + j * SEGW;
                    at = at < p.words - SEGW ? at : p.words - SEGW;
                    mf::load_segment<BITS, SEGW, false>(w + at, buf[h].w[nb]);
                }
#pragma unroll
                for (int g = 0; g < GW; ++g) {
                    const int g0 = sb * GP + 2 * g, last = p.groups - 1;
                    const int a0 = g0 < last ? g0 : last, a1 = g0 + 1 < last ? g0 + 1 : last;
                    buf[h].s[g] = sc[a0] | static_cast<uint32_t>(sc[a1]) << 16;
                    buf[h].b[g] = bi[a0] | static_cast<uint32_t>(bi[a1]) << 16;
                }
            }
        }
    };

    float4_t acc[2][RT];
    auto clear = [&] {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < RT; ++t) acc[h][t] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    };
    // this lane's row of each tile in LDS (rows past the last one: the last one, never stored)
    int x_row[RT], sum_row[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int r = 16 * t + i < rows ? 16 * t + i : rows - 1;
        x_row[t] = r * x_stride;
        sum_row[t] = r * sum_stride;
    }
    auto multiply = [&](S (&buf)[2], int place) {  // place: superblock within the chunk
        const char* const x0 = x_lds + place * (2 * kSuper);
        float4_t P[2][RT];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            __builtin_amdgcn_sched_barrier(0);
            Frag w[2][STEPS];
#pragma unroll
            for (int h = 0; h < 2; ++h) mf::segment_frags<DT, BITS, GS, SEGW, STEPS, UNI>(buf[h].w[nb], w[h], consts);
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                // natural place of the step's 8 codes of this lane
                const int in = j == 0 ? F::src_lane(s, 0) * F::SEG + F::src_slot(s, 0) * 8
                             : j == 1 ? F::src_lane(s, 1) * F::SEG + F::src_slot(s, 1) * 8
                             : j == 2 ? F::src_lane(s, 2) * F::SEG + F::src_slot(s, 2) * 8
                                      : F::src_lane(s, 3) * F::SEG + F::src_slot(s, 3) * 8;
                const int step = nb * STEPS + s;                       // of the superblock: 8 in all
                const bool first = 32 * step % GS == 0, last = 32 * (step + 1) % GS == 0;
                const int g = 32 * step / GS;
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const uint4 u = *reinterpret_cast<const uint4*>(x0 + x_row[t] + 2 * (F::KBLK * nb + in));
                    const Frag a{{u.x, u.y, u.z, u.w}};
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        P[h][t] = mf::mfma<DT>(a, w[h][s], first ? float4_t{0.0f, 0.0f, 0.0f, 0.0f} : P[h][t]);
                }
                if (last) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float sc = (g & 1) ? high_f32<DT>(buf[h].s[g / 2]) : low_f32<DT>(buf[h].s[g / 2]);
#pragma unroll
                        for (int t = 0; t < RT; ++t)
#pragma unroll
                            for (int r = 0; r < 4; ++r) acc[h][t][r] = __builtin_fmaf(sc, P[h][t][r], acc[h][t][r]);
                    }
                }
            }
        }
        // biases and offsets against the groups' sums of x: lane quarter j takes group 4 n + j
#pragma unroll
        for (int n = 0; n < (GP + 3) / 4; ++n) {
            float cb[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t sw = GP > 2 && (j & 2) ? buf[h].s[(2 * n + 1) % GW] : buf[h].s[(2 * n) % GW];
                const uint32_t bw = GP > 2 && (j & 2) ? buf[h].b[(2 * n + 1) % GW] : buf[h].b[(2 * n) % GW];
                const float s = (j & 1) ? high_f32<DT>(sw) : low_f32<DT>(sw), b = (j & 1) ? high_f32<DT>(bw) : low_f32<DT>(bw);
                cb[h] = __builtin_fmaf(-OFF, s, b);
                if (GP == 2 && j >= 2) cb[h] = 0.0f;
            }
            const int g = place * GP + (GP == 2 ? (j & 1) : 4 * n + j);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const float xsum = sums[sum_row[t] + g];
#pragma unroll
                for (int h = 0; h < 2; ++h) acc[h][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(xsum, cb[h], acc[h][t], 0, 0, 0);
            }
        }
    };

    const int per_chunk = p.chunk / kSuper;
    S buf[2][2];
    int tile = blockIdx.x;
    // the wavefront's superblocks, chunk by chunk and tile by tile; buf holds the one that is next
    if (tile < p.tiles && ks < p.supers) load(buf[0], tile, ks);
    bool staged = false;
    for (; tile < p.tiles; tile += gridDim.x) {
        clear();
        for (int c = 0; c < p.chunks; ++c) {
            if (!staged || p.chunks > 1) {
                __syncthreads();  // the chunk before is not read any more
                stage_x(c);
                __syncthreads();
                staged = true;
            }
            const int first = c * per_chunk, end = first + per_chunk < p.supers ? first + per_chunk : p.supers;
            auto next_of = [&](int sb, int& t2) {  // the wavefront's superblock after sb
                t2 = tile;
                if (sb + KS < p.supers) return sb + KS;
                t2 = tile + gridDim.x;
                return ks;
            };
            for (int sb = first + ks; sb < end; sb += 2 * KS) {
                int t2;
                int nx = next_of(sb, t2);
                if (t2 < p.tiles) load(buf[1], t2, nx);
                multiply(buf[0], sb - first);
                if (sb + KS < end) {
                    nx = next_of(sb + KS, t2);
                    if (t2 < p.tiles) load(buf[0], t2, nx);
                    multiply(buf[1], sb + KS - first);
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) buf[0][h] = buf[1][h];
                }
            }
        }
        const int64_t col = (static_cast<int64_t>(tile) * CT + ct) * 16 + i;
        auto finish = [&](int t, int r, float gate, float up) {
            const int row = 16 * t + 4 * j + r;
            if (row >= rows || col >= p.F) return;
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
        // the shares of K meet in LDS, behind x or, where that is brought again, in its place:
        // [wave][2][RT][4][64]; the KS wavefronts of a tile take values in turn
        float* const part = p.chunks > 1 ? reinterpret_cast<float*>(lds) : sums + ((rows * sum_stride + 3) & ~3);
        if (p.chunks > 1) __syncthreads();
        constexpr int kVals = 2 * RT * 4;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) part[(wave * kVals + (h * RT + t) * 4 + r) * 64 + lane] = acc[h][t][r];
        __syncthreads();
#pragma unroll 1
        for (int v = ks; v < 4 * RT; v += KS) {
            float two[2] = {0.0f, 0.0f};
#pragma unroll 1
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int h = 0; h < 2; ++h) two[h] += part[((ct * KS + s) * kVals + h * RT * 4 + v) * 64 + lane];
            finish(v / 4, v % 4, two[0], two[1]);
        }
        __syncthreads();
    }
}

// Bytes of LDS: x, its groups' sums, the shares of K.
inline int lds_bytes(int rows, int chunk, int chunks, int gs, int rt) {
    const int x = rows * (2 * chunk + 16) + 4 * ((rows * (chunk / gs + 1) + 3) & ~3);
    const int part = 4 * kWaves * 2 * rt * 4 * 64;
    return chunks > 1 ? (x > part ? x : part) : x + part;
}

template <int DT, int BITS, int GS, int RT, bool VEC>
hipError_t launch(const GatedParams& p, dim3 grid, int bytes, hipStream_t st) {
    if (bytes > 64 * 1024) {
        static std::atomic<uint64_t> raised{0};
        const hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(&gated_kernel<DT, BITS, GS, RT, VEC>), raised);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((gated_kernel<DT, BITS, GS, RT, VEC>), grid, dim3(kThreads), bytes, st, p);
    return hipGetLastError();
}

template <int DT, int BITS, int GS>
hipError_t run(const GatedParams& p, int rt, bool vec, dim3 grid, int bytes, hipStream_t st) {
    if (!vec) return launch<DT, BITS, GS, 1, false>(p, grid, bytes, st);
    if (rt == 1) return launch<DT, BITS, GS, 1, true>(p, grid, bytes, st);
    if (rt == 2) return launch<DT, BITS, GS, 2, true>(p, grid, bytes, st);
    return launch<DT, BITS, GS, 4, true>(p, grid, bytes, st);
}

// One translation unit per type and code width.
using GatedFn = hipError_t (*)(const GatedParams&, int rt, bool vec, dim3, int, hipStream_t);
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
