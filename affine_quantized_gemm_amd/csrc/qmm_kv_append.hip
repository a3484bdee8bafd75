// Appending to the paged 4-bit K/V cache and reading it back.
//
// Per token, kv head and group of GS consecutive values the quantizer of
// qmm_quant.hip at 4 bits, step for step (IEEE fp32, explicit rounding):
//   lo = min, hi = max (a zero minimum is +0),
//   s  = round_up_dt(fl32(fl32(hi - lo) / 15)),  b = lo,
//   q  = s == 0 ? 0 : clamp(rint(fl32(fl32(x - b) / s)), 0, 15);
// back: RNE_dt(fma(s, q, b)).
//
// Appending gives one wavefront a bundle: the four tokens 4u..4u+3 of a page,
// of one kv head.  That is the unit in which the record keeps V codes
// and scales, so a wavefront writes whole 16-byte runs where all four tokens
// are new, and no two wavefronts ever write the same 16 bits: a token's codes
// of V are half-words of their own, and neighbours' slots are left alone.
// Lane 16 t + c holds token t's values [c D/16, (c + 1) D/16): whole rows are
// read with 8..32 bytes a lane, and a group is a run of 16 GS / D lanes.
#include "qmm_device.hpp"
#include "qmm_kv.hpp"

namespace qmm {
namespace kv {
namespace {

constexpr int kWaves = 4;

// Unit `id` of the grid: sequence, bundle among those its new tokens touch,
// kv head.  Heads fastest: neighbouring wavefronts read neighbouring memory.
struct Unit {
    NewTokens t;
    int head, bundle;  // bundle: position / 4
    int64_t page;      // -1: nothing here
};
__device__ __forceinline__ Unit unit_of(const Seqs& s, int64_t id, int64_t units, int bundles) {
    Unit u;
    u.page = -1;
    if (id >= units) return u;
    u.head = static_cast<int>(id % s.kv_heads);
    const int64_t sb = id / s.kv_heads;
    const int b = static_cast<int>(sb / bundles);
    u.t = new_tokens(s, b);
    if (u.t.n <= 0) return u;
    // positions before 0 hold nothing: the first bundle is that of position 0
    const int first = u.t.pos0 > 0 ? u.t.pos0 : 0;
    u.bundle = (first >> 2) + static_cast<int>(sb % bundles);
    if (4 * static_cast<int64_t>(u.bundle) >= static_cast<int64_t>(u.t.pos0) + u.t.n) return u;
    u.page = page_of(s, b, 4 * u.bundle);
    return u;
}

// Bundles that n consecutive positions can touch.
__host__ int bundles_of(int64_t n) { return static_cast<int>((n + 2) / 4 + 1); }

template <int N>
__device__ __forceinline__ void load_values(const uint16_t* p, uint16_t (&v)[N]) {
    uint32_t w[N / 2];
    if constexpr (N == 4) {
        const uint2 a = *reinterpret_cast<const uint2*>(p);
        w[0] = a.x; w[1] = a.y;
    } else {
#pragma unroll
        for (int i = 0; i < N / 8; ++i) {
            const uint4 a = reinterpret_cast<const uint4*>(p)[i];
            w[4 * i] = a.x; w[4 * i + 1] = a.y; w[4 * i + 2] = a.z; w[4 * i + 3] = a.w;
        }
    }
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        v[2 * i] = static_cast<uint16_t>(w[i] & 0xFFFFu);
        v[2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
    }
}

template <int N>
__device__ __forceinline__ void store_values(uint16_t* p, const uint16_t (&v)[N]) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = static_cast<uint32_t>(v[2 * i]) | (static_cast<uint32_t>(v[2 * i + 1]) << 16);
    if constexpr (N == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < N / 8; ++i)
            reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
}

// One operand's N values a lane -> codes; writes the scale and bias of each
// group (sb: the bundle's first group, 8 half-words a group).
template <int DT, int D, int GS>
__device__ __forceinline__ void quantize_lane(const uint16_t (&v)[D / 16], uint32_t (&q)[D / 16], uint16_t* sb,
                                              int tok, int c, bool live) {
    constexpr int N = D / 16;
    constexpr int LANES = GS / N;  // lanes of a group
    float f[N];
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = DtOps<DT>::to_f32(v[i]);
    float lo = f[0], hi = f[0];
#pragma unroll
    for (int i = 1; i < N; ++i) {
        lo = fminf(lo, f[i]);
        hi = fmaxf(hi, f[i]);
    }
#pragma unroll
    for (int m = 1; m < LANES; m *= 2) {
        lo = fminf(lo, __shfl_xor(lo, m));
        hi = fmaxf(hi, __shfl_xor(hi, m));
    }
    lo = __fadd_rn(lo, 0.0f);
    const float s32 = __fdiv_rn(__fsub_rn(hi, lo), 15.0f);
    const uint16_t s_bits = round_up_nonneg<DT>(s32);
    const float s = DtOps<DT>::to_f32(s_bits);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        q[i] = 0u;
        if (s != 0.0f) {
            const float t = __fdiv_rn(__fsub_rn(f[i], lo), s);
            q[i] = static_cast<uint32_t>(fminf(fmaxf(rintf(t), 0.0f), 15.0f));
        }
    }
    if (live && c % LANES == 0) {
        uint16_t* p = sb + (c / LANES) * 8 + tok;
        p[0] = s_bits;
        p[4] = DtOps<DT>::rne(lo);
    }
}

// K codes of a lane: a token's row is words (j, s) of values 32 s + 8 j + e.
template <int D>
__device__ __forceinline__ void store_k(uint32_t* row, const uint32_t (&q)[D / 16], int c) {
    constexpr int S = D / 32;
    if constexpr (D == 64) {  // half a word: values 4 c ..
        uint32_t h = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) h |= q[e] << (4 * e);
        const int w = c / 2;
        reinterpret_cast<uint16_t*>(row + (w % 4) * S + w / 4)[c & 1] = static_cast<uint16_t>(h);
    } else {
#pragma unroll
        for (int k = 0; k < D / 128; ++k) {
            uint32_t h = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) h |= q[8 * k + e] << (4 * e);
            const int w = c * (D / 128) + k;
            row[(w % 4) * S + w / 4] = h;
        }
    }
}

template <int DT, int D, int GS>
__global__ __launch_bounds__(64 * kWaves) void append_kernel(Seqs s, int64_t units, int bundles,
                                                             const uint16_t* __restrict__ k, int64_t k_row,
                                                             int64_t k_head, const uint16_t* __restrict__ v,
                                                             int64_t v_row, int64_t v_head) {
    constexpr int N = D / 16, C = D / 64, G = D / GS;
    __shared__ uint8_t codes[kWaves][4][D];
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const int tok = lane / 16, c = lane % 16;
    const int page_size = 1 << s.page_shift;
    const Record rec(page_size, D, GS);
    // every wavefront of the workgroup makes the same number of turns
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * kWaves; base < units;
         base += static_cast<int64_t>(gridDim.x) * kWaves) {
        const Unit u = unit_of(s, base + wave, units, bundles);
        const bool have = u.page >= 0;
        uint32_t* r = nullptr;
        int slot = 0, live_bits = 0;
        uint32_t qv[N];
        if (have) {
            r = s.pool + (u.page * s.kv_heads + u.head) * rec.words();
            slot = (4 * u.bundle) & (page_size - 1);
            const int i = 4 * u.bundle + tok - u.t.pos0;  // place among the new tokens
            const bool live = i >= 0 && i < u.t.n;
            const int64_t row = u.t.row0 + i;
            uint16_t kv[N], vv[N];
#pragma unroll
            for (int e = 0; e < N; ++e) kv[e] = vv[e] = 0;
            if (live) {
                load_values<N>(k + row * k_row + u.head * k_head + c * N, kv);
                load_values<N>(v + row * v_row + u.head * v_head + c * N, vv);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int it = 4 * u.bundle + t - u.t.pos0;
                live_bits |= (it >= 0 && it < u.t.n) ? 1 << t : 0;
            }
            uint32_t qk[N];
            const int sb = (slot / 4) * G * 4;  // words of the bundles before
            quantize_lane<DT, D, GS>(kv, qk, reinterpret_cast<uint16_t*>(r + rec.k_sb() + sb), tok, c, live);
            quantize_lane<DT, D, GS>(vv, qv, reinterpret_cast<uint16_t*>(r + rec.v_sb() + sb), tok, c, live);
            if (live) store_k<D>(r + rec.k_codes() + (slot + tok) * (D / 8), qk, c);
#pragma unroll
            for (int e = 0; e < N; ++e) codes[wave][tok][c * N + e] = static_cast<uint8_t>(qv[e]);
        }
        __syncthreads();
        if (have) {
            // V codes: word (i, p, cc) of the bundle
            uint32_t* dst = r + rec.v_codes() + (slot / 4) * (32 * C);
#pragma unroll
            for (int w0 = 0; w0 < 32 * C; w0 += 64) {
                const int w = w0 + lane;
                if (w < 32 * C) {
                    const int i = w / (2 * C), p = (w / C) % 2, cc = w % C;
                    uint32_t h[2];
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        h[half] = 0;
#pragma unroll
                        for (int n = 0; n < 4; ++n)
                            h[half] |= static_cast<uint32_t>(codes[wave][2 * p + half][64 * cc + 16 * n + i]) << (4 * n);
                    }
                    const int both = (live_bits >> (2 * p)) & 3;
                    if (both == 3) {
                        dst[w] = h[0] | (h[1] << 16);
                    } else if (both != 0) {
                        reinterpret_cast<uint16_t*>(dst + w)[both >> 1] = static_cast<uint16_t>(h[both >> 1]);
                    }
                }
            }
        }
        __syncthreads();  // the codes are read before the next turn's are written
    }
}

// Four rows of a sequence and one kv head a wavefront: lane 16 t + c writes
// values [c D/16, (c + 1) D/16) of row 4 x + t.
template <int DT, int D, int GS>
__global__ __launch_bounds__(64 * kWaves) void read_kernel(Seqs s, int64_t units, int quads,
                                                           uint16_t* __restrict__ k, uint16_t* __restrict__ v) {
    constexpr int N = D / 16, C = D / 64, G = D / GS, S = D / 32;
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const int c = lane % 16;
    const int page_size = 1 << s.page_shift;
    const Record rec(page_size, D, GS);
    for (int64_t id = static_cast<int64_t>(blockIdx.x) * kWaves + wave; id < units;
         id += static_cast<int64_t>(gridDim.x) * kWaves) {
        const int head = static_cast<int>(id % s.kv_heads);
        const int64_t sq = id / s.kv_heads;
        const int b = static_cast<int>(sq / quads);
        const NewTokens t = new_tokens(s, b);
        const int i = 4 * static_cast<int>(sq % quads) + lane / 16;
        if (i >= t.n) continue;
        const int pos = t.pos0 + i;
        const int64_t page = page_of(s, b, pos);
        const int slot = pos & (page_size - 1), tok = slot % 4;
        const uint32_t* r = s.pool + (page * s.kv_heads + head) * rec.words();  // used where page >= 0
        const int64_t at = ((t.row0 + i) * s.kv_heads + head) * D + c * N;
        const int sb = ((slot / 4) * G + c * N / GS) * 8 + tok;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            uint16_t o[N];
#pragma unroll
            for (int e = 0; e < N; ++e) o[e] = 0;
            if (page >= 0) {
                const uint16_t* q = reinterpret_cast<const uint16_t*>(r + (part ? rec.v_sb() : rec.k_sb())) + sb;
                const float sc = DtOps<DT>::to_f32(q[0]), bi = DtOps<DT>::to_f32(q[4]);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const int d = c * N + e;
                    uint32_t code;
                    if (part == 0) {
                        const int w = d / 8;
                        code = r[rec.k_codes() + slot * (D / 8) + (w % 4) * S + w / 4] >> (4 * (d % 8));
                    } else {
                        const int w = ((d % 16) * 2 + tok / 2) * C + d / 64;
                        code = r[rec.v_codes() + (slot / 4) * (32 * C) + w] >> (4 * ((d % 64) / 16) + 16 * (tok & 1));
                    }
                    o[e] = DtOps<DT>::rne(__fmaf_rn(sc, static_cast<float>(code & 15u), bi));
                }
            }
            store_values<N>((part ? v : k) + at, o);
        }
    }
}

unsigned grid_of(int64_t units) {
    const int64_t blocks = (units + kWaves - 1) / kWaves;
    return static_cast<unsigned>(blocks < (1 << 22) ? blocks : 1 << 22);
}

template <int DT, int D, int GS>
hipError_t append_t(const Seqs& s, Rows k, Rows v, hipStream_t st) {
    const int bundles = bundles_of(s.max_new);
    const int64_t units = static_cast<int64_t>(s.seqs) * bundles * s.kv_heads;
    hipLaunchKernelGGL((append_kernel<DT, D, GS>), dim3(grid_of(units)), dim3(64 * kWaves), 0, st, s, units, bundles,
                       static_cast<const uint16_t*>(k.p), k.stride_row, k.stride_head,
                       static_cast<const uint16_t*>(v.p), v.stride_row, v.stride_head);
    return hipGetLastError();
}

template <int DT, int D, int GS>
hipError_t read_t(const Seqs& s, void* k, void* v, hipStream_t st) {
    const int quads = s.max_new / 4 + (s.max_new % 4 != 0);
    const int64_t units = static_cast<int64_t>(s.seqs) * quads * s.kv_heads;
    hipLaunchKernelGGL((read_kernel<DT, D, GS>), dim3(grid_of(units)), dim3(64 * kWaves), 0, st, s, units, quads,
                       static_cast<uint16_t*>(k), static_cast<uint16_t*>(v));
    return hipGetLastError();
}

}  // namespace

#define QMM_KV_SWITCH(c, CALL)                                                        \
    switch ((c).dt * 10000 + (c).head_dim / 64 * 1000 + (c).group_size) {              \
        case 1032: return CALL(0, 64, 32);     case 1064: return CALL(0, 64, 64);      \
        case 2032: return CALL(0, 128, 32);    case 2064: return CALL(0, 128, 64);     \
        case 2128: return CALL(0, 128, 128);   case 4032: return CALL(0, 256, 32);     \
        case 4064: return CALL(0, 256, 64);    case 4128: return CALL(0, 256, 128);    \
        case 11032: return CALL(1, 64, 32);    case 11064: return CALL(1, 64, 64);     \
        case 12032: return CALL(1, 128, 32);   case 12064: return CALL(1, 128, 64);    \
        case 12128: return CALL(1, 128, 128);  case 14032: return CALL(1, 256, 32);    \
        case 14064: return CALL(1, 256, 64);   case 14128: return CALL(1, 256, 128);   \
        default: return hipErrorInvalidValue;                                         \
    }

hipError_t launch_append(const qmm_kv_cache& c, const Seqs& s, Rows k, Rows v, hipStream_t st) {
#define ACALL(T, D, G) append_t<T, D, G>(s, k, v, st)
    QMM_KV_SWITCH(c, ACALL)
#undef ACALL
}

hipError_t launch_read(const qmm_kv_cache& c, const Seqs& s, void* k, void* v, hipStream_t st) {
#define RCALL(T, D, G) read_t<T, D, G>(s, k, v, st)
    QMM_KV_SWITCH(c, RCALL)
#undef RCALL
}

}  // namespace kv
}  // namespace qmm
