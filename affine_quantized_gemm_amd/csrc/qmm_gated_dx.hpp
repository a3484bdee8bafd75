// Gradient of the gated block for x (gfx950): y[M, K] = d[M, N] . W[N, K] with
// d the gradients of the two products in fp32 (N = 2F rows of W) and W
// quantized along K: the sum runs down the rows of W, over which its scales
// change, so they go to the other operand,
//   y[m, k] = sum_n (d[m, n] s[n, g]) (q[n, k] + off) + sum_n d[m, n] (b[n, g] - off s[n, g])
// for the columns k of group g.  The first sum is on the matrix cores: codes
// with a small offset (16 + q, 64 + q, or q itself of 8 bits) are exact in
// bf16, and t = d s is two bf16 numbers, its upper half and what is left,
// together within 2^-16 of t, whatever its size and whatever the type.  (One
// rounding of d to the type, as the two gradients are returned, is as large as
// the result's own: grad_x 1.4 times as far off.)  The second is one value a
// group, on the vector ALUs.
//
// Split.  A workgroup owns 256 columns and a slice of N; a wavefront 64 of the
// columns, so that t is formed once for four column tiles (two with groups of
// 32), and every second 64 rows of a chunk of 128.  A chunk's codes (6-bit ones
// widened to bytes), scales, biases and d lie in LDS, the next one's in
// registers; ds_read_b64_tr_b4 and _b8 turn rows of codes into matrix operands
// (the layouts are those that the non-transposed product uses).  Slices' sums
// are added in order by a second kernel.
//
// Measured (37 rows, 28672 x 4096, 4 bits, groups of 64): 46 us and 4.7 for the
// slices' sums (9.4 us of reading, 14 us of matrix work for the two pieces: t's
// forming and cutting, once a row, row tile and 64 columns, and the barriers
// between chunks; one workgroup of 512 threads a CU; vector units busy 48 % of
// the time, matrix cores 18 %).  It is not its loads: with
// two chunks on their way it took 51 us, with a slice's workgroups on one die 47.
#pragma once

#include <type_traits>

#include "qmm_device.hpp"
#include "qmm_internal.hpp"
#include "qmm_mfma_frag.hpp"
#include "qmm_rows.hpp"

namespace qmm {
namespace gated {

constexpr int kDxThreads = 512;
constexpr int kDxCols = 256;   // columns of a workgroup
constexpr int kDxRows = 128;   // rows of W in a chunk

struct DxParams {
    const float* d;        // [M][N]
    const uint32_t* wq;
    const uint16_t* scales;
    const uint16_t* biases;
    uint16_t* y;           // one slice: [M][K]
    float* part;           // several: [slices][M][K]
    int M;
    int64_t N, K;
    int64_t slice;         // rows of W of a slice, a multiple of kDxRows
};

namespace {

using mf::float4_t;
using mf::Frag;

template <int BITS>
struct DxFmt {
    static constexpr int CB = BITS == 4 ? 4 : 8;                  // bits of a code in LDS
    static constexpr int RP = kDxCols * CB / 8;                   // bytes of a row there
    static constexpr float OFF = BITS == 4 ? 16.0f : BITS == 6 ? 64.0f : 0.0f;
    static constexpr int UNIT_WORDS = BITS == 6 ? 3 : 4;          // what a thread loads: 32, 16 or 16 codes
    static constexpr int UNIT = UNIT_WORDS * 32 / BITS;
    static constexpr int UNITS = kDxCols / UNIT;                  // of a row
    static constexpr int PER = kDxRows * UNITS / kDxThreads;      // of a thread
};

// Place of 16-byte piece c of row r, spread over the banks for the transposed reads of neighbouring rows.
__device__ __forceinline__ int dx_place(int r, int c, int row_bytes) { return r * row_bytes + 16 * (c ^ (r & 7)); }

// Codes of 8 rows of one column (nibbles of w0, or bytes of w0 and w1) as bf16 q + OFF, rows in the order 0, 4, 1, 5, 2, 6, 3, 7.
template <int BITS>
__device__ __forceinline__ Frag dx_codes(uint32_t w0, uint32_t w1) {
    Frag f;
    if constexpr (BITS == 4) {
        f.v[0] = ((w0 << 3) & 0x00780078u) | 0x41804180u;
        f.v[1] = ((w0 >> 1) & 0x00780078u) | 0x41804180u;
        f.v[2] = ((w0 >> 5) & 0x00780078u) | 0x41804180u;
        f.v[3] = ((w0 >> 9) & 0x00780078u) | 0x41804180u;
    } else if constexpr (BITS == 6) {
        // bytes e of w0 and w1 into the halves, one bit up
        f.v[0] = (__builtin_amdgcn_perm(w1, w0, 0x0C040C00u) << 1) | 0x42804280u;
        f.v[1] = (__builtin_amdgcn_perm(w1, w0, 0x0C050C01u) << 1) | 0x42804280u;
        f.v[2] = (__builtin_amdgcn_perm(w1, w0, 0x0C060C02u) << 1) | 0x42804280u;
        f.v[3] = (__builtin_amdgcn_perm(w1, w0, 0x0C070C03u) << 1) | 0x42804280u;
    } else {
        // (an integer below 256 is exactly the top half of its fp32 value)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t a = __builtin_bit_cast(uint32_t, static_cast<float>((w0 >> (8 * e)) & 0xFFu));
            const uint32_t b = __builtin_bit_cast(uint32_t, static_cast<float>((w1 >> (8 * e)) & 0xFFu));
            f.v[e] = __builtin_amdgcn_perm(b, a, 0x07060302u);
        }
    }
    return f;
}

// t as two bf16 numbers: its upper half, and the rest to nearest; rows in the codes' order.
__device__ __forceinline__ void dx_split(const float (&t)[8], Frag& hi, Frag& lo) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t a = __builtin_bit_cast(uint32_t, t[e]), b = __builtin_bit_cast(uint32_t, t[e + 4]);
        hi.v[e] = __builtin_amdgcn_perm(b, a, 0x07060302u);
        lo.v[e] = pack2<DT_BF16>(t[e] - __builtin_bit_cast(float, a & 0xFFFF0000u), t[e + 4] - __builtin_bit_cast(float, b & 0xFFFF0000u));
    }
}

__device__ __forceinline__ float dx_sum_quarters(float v) {
    uint32_t a = __builtin_bit_cast(uint32_t, v), b = a;
    mf::swap32(a, b);
    v = __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
    a = b = __builtin_bit_cast(uint32_t, v);
    mf::swap16(a, b);
    return __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
}

}  // namespace

constexpr int dx_d_stride() { return kDxRows + 4; }  // floats: 16 rows' pieces in different banks

// Bytes of LDS: codes, d, scales and biases; at the end the second half's sums.
inline int dx_lds_bytes(int bits, int gs, int rt) {
    const int chunk = kDxRows * kDxCols * (bits == 4 ? 4 : 8) / 8 + 4 * 16 * rt * dx_d_stride() + 4 * kDxRows * (kDxCols / gs);
    const int sums = 4 * 4 * 64 * 16 * rt;
    return chunk > sums ? chunk : sums;
}

template <int DT, int BITS, int GS, int RT, bool PART>
__global__ __launch_bounds__(kDxThreads, 2) void gated_dx_kernel(DxParams p) {
    using F = DxFmt<BITS>;
    constexpr int NG = 64 / GS > 1 ? 2 : 1;                  // groups of a wavefront's columns
    constexpr int GB = kDxCols / GS;                         // of the workgroup's
    constexpr int DP = (16 * RT * kDxRows / 4 + kDxThreads - 1) / kDxThreads;  // 16-byte pieces of d a thread
    constexpr int SP = (kDxRows * GB + kDxThreads - 1) / kDxThreads;
    extern __shared__ __align__(16) char lds[];
    char* const w_lds = lds;
    float* const d_lds = reinterpret_cast<float*>(lds + kDxRows * F::RP);
    uint16_t* const s_lds = reinterpret_cast<uint16_t*>(d_lds + 16 * RT * dx_d_stride());  // [GB][kDxRows]
    uint16_t* const b_lds = s_lds + GB * kDxRows;
    const int tid = threadIdx.x, lane = tid % 64, i = lane % 16, j = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int cg = wave & 3, half = wave >> 2;
    const int64_t n_cols0 = static_cast<int64_t>(blockIdx.x) * kDxCols;
    const int cols = p.K - n_cols0 < kDxCols ? static_cast<int>(p.K - n_cols0) : kDxCols;  // a multiple of 64
    const int64_t lo = static_cast<int64_t>(blockIdx.y) * p.slice, hi = lo + p.slice < p.N ? lo + p.slice : p.N;
    const int64_t groups = p.K / GS, g0 = n_cols0 / GS;
    const int group_last = static_cast<int>(groups - 1 - g0 < GB - 1 ? groups - 1 - g0 : GB - 1);
    const int64_t row_words = p.K * BITS / 32;

    struct Chunk {
        uint32_t w[F::PER][F::UNIT_WORDS];
        float4_t d[DP];
        uint32_t s[SP], b[SP];
    };
    // what lies past the slice, the rows or the columns is read from a valid place; d, scales and biases of it become 0
    auto fetch = [&](int64_t n0, Chunk& c) {
#pragma unroll
        for (int u = 0; u < F::PER; ++u) {
            const int at = tid + u * kDxThreads, r = at / F::UNITS, k = at % F::UNITS * F::UNIT;
            const int64_t row = n0 + r < hi ? n0 + r : hi - 1;
            const uint32_t* q = p.wq + row * row_words + (n_cols0 + (k < cols ? k : 0)) / 32 * BITS + (k < cols ? k % 32 * BITS / 32 : 0);
            mf::load_segment<BITS, F::UNIT_WORDS, false>(q, c.w[u]);
        }
#pragma unroll
        for (int u = 0; u < DP; ++u) {
            const int at = tid + u * kDxThreads, m = at / (kDxRows / 4), n = at % (kDxRows / 4) * 4;
            // (slices and N are multiples of 32: a piece is whole or past the end)
            const int64_t col = n0 + n < hi ? n0 + n : lo;
            c.d[u] = *reinterpret_cast<const float4_t*>(p.d + static_cast<int64_t>(m < p.M ? m : p.M - 1) * p.N + col);
        }
#pragma unroll
        for (int u = 0; u < SP; ++u) {
            const int at = (tid + u * kDxThreads) % (kDxRows * GB), r = at / GB, g = at % GB;
            const int64_t from = (n0 + r < hi ? n0 + r : hi - 1) * groups + g0 + (g < group_last ? g : group_last);
            c.s[u] = p.scales[from];
            c.b[u] = p.biases[from];
        }
    };
    auto stage = [&](int64_t n0, const Chunk& c) {
#pragma unroll
        for (int u = 0; u < F::PER; ++u) {
            const int at = tid + u * kDxThreads, r = at / F::UNITS, unit = at % F::UNITS;
            uint4 v;
            if constexpr (BITS == 6) {
                const uint32_t q[4] = {c.w[u][0], __builtin_amdgcn_alignbit(c.w[u][1], c.w[u][0], 24),
                                       __builtin_amdgcn_alignbit(c.w[u][2], c.w[u][1], 16), c.w[u][2] >> 8};
                uint32_t b[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    b[e] = (q[e] & 63u) | (q[e] << 2 & 0x3F00u) | (q[e] << 4 & 0x3F0000u) | (q[e] << 6 & 0x3F000000u);
                v = make_uint4(b[0], b[1], b[2], b[3]);
            } else {
                v = make_uint4(c.w[u][0], c.w[u][1], c.w[u][2], c.w[u][3]);
            }
            *reinterpret_cast<uint4*>(w_lds + dx_place(r, unit, F::RP)) = v;
        }
        const float4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < DP; ++u) {
            const int at = tid + u * kDxThreads, m = at / (kDxRows / 4), n = at % (kDxRows / 4) * 4;
            if (m < 16 * RT) *reinterpret_cast<float4_t*>(d_lds + m * dx_d_stride() + n) = n0 + n < hi ? c.d[u] : zero;
        }
#pragma unroll
        for (int u = 0; u < SP; ++u) {
            const int at = tid + u * kDxThreads, r = at / GB, g = at % GB;
            if (at < kDxRows * GB) {
                s_lds[g * kDxRows + r] = static_cast<uint16_t>(n0 + r < hi ? c.s[u] : 0);
                b_lds[g * kDxRows + r] = static_cast<uint16_t>(n0 + r < hi ? c.b[u] : 0);
            }
        }
    };

    float4_t acc[4][RT];
    float z[RT][NG];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
#pragma unroll
        for (int n = 0; n < 4; ++n) acc[n][t] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int g = 0; g < NG; ++g) z[t][g] = 0.0f;
    }
    const bool live = 64 * cg < cols;
    auto compute = [&] {
        typedef int v2i_t __attribute__((ext_vector_type(2)));
        auto turned = [&](int r, int off) {
            auto* at = reinterpret_cast<__attribute__((address_space(3))) v2i_t*>(
                reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)(w_lds)) + r * F::RP + off);
            if constexpr (BITS == 4) return __builtin_amdgcn_ds_read_tr4_b64_v2i32(at);
            else return __builtin_amdgcn_ds_read_tr8_b64_v2i32(at);
        };
        v2i_t words[4];
        if constexpr (BITS == 4) {  // 64 rows at a time: word st has rows 8 st .. of the quarter's 16
            const int r = 64 * half + 16 * j + i;
#pragma unroll
            for (int n = 0; n < 4; ++n) words[n] = turned(r, 16 * ((2 * cg + n / 2) ^ (r & 7)) + 8 * (n & 1));
        }
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            // the 8 rows of this lane
            const int row = BITS == 4 ? 64 * half + 16 * j + 8 * st : 64 * half + 32 * st + 8 * j;
            Frag w[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                if constexpr (BITS == 4) {
                    w[n] = dx_codes<4>(static_cast<uint32_t>(words[n][st]), 0u);
                } else {
                    const int r = row + (i >> 1);
                    const v2i_t v = turned(r, 16 * ((4 * cg + n) ^ (r & 7)) + 8 * (i & 1));
                    w[n] = dx_codes<BITS>(static_cast<uint32_t>(v[0]), static_cast<uint32_t>(v[1]));
                }
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const int group = 64 * cg / GS + g;
                float s[8], b[8];
                const uint4 su = *reinterpret_cast<const uint4*>(s_lds + group * kDxRows + row);
                const uint4 bu = *reinterpret_cast<const uint4*>(b_lds + group * kDxRows + row);
                const uint32_t sw[4] = {su.x, su.y, su.z, su.w}, bw[4] = {bu.x, bu.y, bu.z, bu.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    s[e] = e & 1 ? high_f32<DT>(sw[e / 2]) : low_f32<DT>(sw[e / 2]);
                    b[e] = __builtin_fmaf(-F::OFF, s[e], e & 1 ? high_f32<DT>(bw[e / 2]) : low_f32<DT>(bw[e / 2]));
                }
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const float4_t* const from = reinterpret_cast<const float4_t*>(d_lds + (16 * t + i) * dx_d_stride() + row);
                    const float4_t d0 = from[0], d1 = from[1];
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float d = e < 4 ? d0[e] : d1[e - 4];
                        z[t][g] = __builtin_fmaf(d, b[e], z[t][g]);
                        v[e] = d * s[e];
                    }
                    Frag up, rest;
                    dx_split(v, up, rest);
#pragma unroll
                    for (int n = g * 4 / NG; n < (g + 1) * 4 / NG; ++n) {
                        acc[n][t] = mf::mfma<DT_BF16>(up, w[n], acc[n][t]);
                        acc[n][t] = mf::mfma<DT_BF16>(rest, w[n], acc[n][t]);
                    }
                }
            }
        }
    };

    Chunk next;
    fetch(lo, next);
    for (int64_t n0 = lo; n0 < hi; n0 += kDxRows) {
        __syncthreads();  // the chunk before is not read any more
        stage(n0, next);
        __syncthreads();
        if (n0 + kDxRows < hi) fetch(n0 + kDxRows, next);
        if (live) compute();
    }

    // a group's value to all its columns: from row i of the quarters to rows 4 j + r
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const float sum = dx_sum_quarters(z[t][g]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float mine = __shfl(sum, 4 * j + r);
#pragma unroll
                for (int n = g * 4 / NG; n < (g + 1) * 4 / NG; ++n) acc[n][t][r] += mine;
            }
        }
    // the two halves of the rows
    __syncthreads();
    float* const other = reinterpret_cast<float*>(lds) + cg * (64 * 16 * RT) + lane;
    if (half == 1) {
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) other[64 * ((n * RT + t) * 4 + r)] = acc[n][t][r];
    }
    __syncthreads();
    if (half == 1 || !live) return;
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int m = 16 * t + 4 * j + r;
                if (m >= p.M) continue;
                const float v = acc[n][t][r] + other[64 * ((n * RT + t) * 4 + r)];
                const int64_t at = static_cast<int64_t>(m) * p.K + n_cols0 + 64 * cg + 16 * n + i;
                if constexpr (PART) p.part[static_cast<int64_t>(blockIdx.y) * p.M * p.K + at] = v;
                else p.y[at] = static_cast<uint16_t>(pack2<DT>(v, 0.0f));
            }
}

template <int DT, int BITS, int GS, int RT>
hipError_t launch_dx(const DxParams& p, dim3 grid, hipStream_t st) {
    const int bytes = dx_lds_bytes(BITS, GS, RT);
    auto go = [&](auto part) -> hipError_t {
        constexpr bool PART = decltype(part)::value;
        if (bytes > 64 * 1024) {
            static std::atomic<uint64_t> raised{0};
            const hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(&gated_dx_kernel<DT, BITS, GS, RT, PART>), raised);
            if (e != hipSuccess) return e;
        }
        hipLaunchKernelGGL((gated_dx_kernel<DT, BITS, GS, RT, PART>), grid, dim3(kDxThreads), bytes, st, p);
        return hipGetLastError();
    };
    return grid.y > 1 ? go(std::true_type{}) : go(std::false_type{});
}

template <int DT, int BITS, int GS>
hipError_t run_dx(const DxParams& p, int rt, dim3 grid, hipStream_t st) {
    if (rt == 1) return launch_dx<DT, BITS, GS, 1>(p, grid, st);
    if (rt == 2) return launch_dx<DT, BITS, GS, 2>(p, grid, st);
    if (rt == 3) return launch_dx<DT, BITS, GS, 3>(p, grid, st);
    return launch_dx<DT, BITS, GS, 4>(p, grid, st);
}

using DxFn = hipError_t (*)(const DxParams&, int rt, dim3, hipStream_t);
template <int DT, int BITS>
DxFn dx_fn(int gs);

}  // namespace gated
}  // namespace qmm

#define QMM_GATED_DX_UNIT(DTV, BITSV)                         \
    namespace qmm {                                           \
    namespace gated {                                         \
    template <>                                               \
    DxFn dx_fn<DTV, BITSV>(int gs) {                          \
        if (gs == 32) return run_dx<DTV, BITSV, 32>;          \
        if (gs == 64) return run_dx<DTV, BITSV, 64>;          \
        return gs == 128 ? run_dx<DTV, BITSV, 128> : nullptr; \
    }                                                         \
    }                                                         \
    }
