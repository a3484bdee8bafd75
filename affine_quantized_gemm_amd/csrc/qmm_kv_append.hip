// Appending to the paged 4-bit K/V cache and reading it back.
//
// Per token, kv head and group of GS consecutive values the quantizer of
// qmm_quant.hip at 4 bits, step for step (IEEE fp32, explicit rounding):
//   lo = min, hi = max (a zero minimum is +0),
//   s  = round_up_dt(fl32(fl32(hi - lo) / 15)),  b = lo,
//   q  = s == 0 ? 0 : clamp(rint(fl32(fl32(x - b) / s)), 0, 15);
// back: RNE_dt(fma(s, q, b)).  Only for NaN it differs: a group that holds one
// gets NaN for s and b (the weights' quantizer leaves it out of min and max and
// gives it code 0), so that what a model computed wrongly is not read back as
// a number.
//
// Both kernels give one wavefront a bundle: the four tokens 4u..4u+3 of a
// page, of one kv head.  That is the unit in which the record keeps V codes
// and scales, so a wavefront writes whole 16-byte runs where all four tokens
// are new, and no two wavefronts ever write the same 16 bits: a token's codes
// of V are half-words of their own, and neighbours' slots are left alone.
// Lane 16 t + c holds token t's values [c D/16, (c + 1) D/16): whole rows are
// read with 8..32 bytes a lane, and a group is a run of 16 GS / D lanes.  The
// V codes, which the record keeps across rows, change places through LDS.
#include "qmm_device.hpp"
#include "qmm_kv.hpp"

namespace qmm {
namespace kv {
namespace {

constexpr int kWaves = 4;  // the bundles of 16 tokens

// A wavefront's unit: a bundle that the new tokens of sequence b touch, and a
// kv head.  A workgroup has the four bundles of 16 aligned tokens of one head,
// so that their scales, a line of the record, are written by one XCD.
struct Unit {
    NewTokens t;
    int head, bundle;  // bundle: position / 4, rounded down
    bool any;          // there are new tokens in it
};
__device__ __forceinline__ Unit unit_of(const Seqs& s, int b, int wave) {
    Unit u;
    const uint32_t at = blockIdx.x / static_cast<uint32_t>(s.kv_heads);
    u.head = static_cast<int>(blockIdx.x - at * s.kv_heads);
    u.t = new_tokens(s, b);
    u.bundle = ((u.t.pos0 >> 4) + static_cast<int>(at)) * 4 + wave;
    u.any = u.t.n > 0 && 4 * static_cast<int64_t>(u.bundle) < static_cast<int64_t>(u.t.pos0) + u.t.n;
    return u;
}

// The runs of 16 aligned positions that n consecutive ones can touch, for
// every head.
dim3 grid_of(const Seqs& s) {
    return dim3(static_cast<unsigned>(((static_cast<int64_t>(s.max_new) + 14) / 16 + 1) * s.kv_heads),
                static_cast<unsigned>(s.seqs < 65535 ? s.seqs : 65535));
}

// Place of (token t, value d) in a bundle's codes in LDS, a byte each: the
// four codes of a half-word side by side.
template <int D>
__device__ __forceinline__ int code_at(int t, int d) {
    return ((t * (D / 64) + d / 64) * 16 + d % 16) * 4 + d % 64 / 16;
}

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

// The smaller and the larger of two, NaN where one of them is.
__device__ __forceinline__ float low_of(float a, float b) { return __builtin_elementwise_minimum(a, b); }
__device__ __forceinline__ float high_of(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// Minimum and maximum over runs of LANES lanes (2..16), by exchanges within 16
// lanes: with the neighbour, the other pair, the other half of 8 (mirrored,
// its lanes are alike by then), the other 8.
template <int CTRL>
__device__ __forceinline__ float from_lane(float v) {
    const int x = __builtin_bit_cast(int, v);
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(x, x, CTRL, 0xf, 0xf, false));
}
template <int LANES>
__device__ __forceinline__ void group_min_max(float& lo, float& hi) {
    if constexpr (LANES >= 2) { lo = low_of(lo, from_lane<0xB1>(lo)); hi = high_of(hi, from_lane<0xB1>(hi)); }
    if constexpr (LANES >= 4) { lo = low_of(lo, from_lane<0x4E>(lo)); hi = high_of(hi, from_lane<0x4E>(hi)); }
    if constexpr (LANES >= 8) { lo = low_of(lo, from_lane<0x141>(lo)); hi = high_of(hi, from_lane<0x141>(hi)); }
    if constexpr (LANES >= 16) { lo = low_of(lo, from_lane<0x140>(lo)); hi = high_of(hi, from_lane<0x140>(hi)); }
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
        lo = low_of(lo, f[i]);
        hi = high_of(hi, f[i]);
    }
    group_min_max<LANES>(lo, hi);
    lo = __fadd_rn(lo, 0.0f);
    const float s32 = __fdiv_rn(__fsub_rn(hi, lo), 15.0f);
    const uint16_t s_bits = round_up_nonneg<DT>(s32);
    const float s = DtOps<DT>::to_f32(s_bits);
    // q = rint(fl32((x - lo) / s)), at most 15 as s >= (hi - lo) / 15.  The
    // division is only carried out where its result could round otherwise
    // than the product with 1 / s: that is off by less than 2^-21 of at most
    // 15.1, so within 2^-16 of a half.
    const float inv = __builtin_amdgcn_rcpf(s);
    float a[N], t[N];
    float far = 0.0f;  // largest distance from a whole number
#pragma unroll
    for (int i = 0; i < N; ++i) {
        a[i] = __fsub_rn(f[i], lo);
        const float p = a[i] * inv;
        t[i] = rintf(p);
        far = fmaxf(far, fabsf(p - t[i]));
    }
    // (s = 0, or so small that 1 / s is infinite: the distances are no numbers)
    if (!(inv < __builtin_inff() && far < 0.5f - 0x1p-16f)) {
#pragma unroll
        for (int i = 0; i < N; ++i) t[i] = s != 0.0f ? rintf(__fdiv_rn(a[i], s)) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        q[i] = static_cast<uint32_t>(__builtin_amdgcn_fmed3f(t[i], 0.0f, 15.0f));  // (of NaN: the least of the others)
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

// 4 prompts of 1801..2047 tokens, 8 heads of 128 (fp16, 40 MB) 15.1 us, 2.7
// TB/s; neither memory nor the vector ALUs (47 % busy, 406 instructions a
// wavefront of 4 tokens) are full: of the wavefronts' time 20 % goes to instructions,
// 44 % to waits for data and barriers, 37 % to waits for a unit.  64 tokens of 64
// sequences 4.7 us, 4..6 rows of 16 sequences (heads of 256) 5.3: a launch and two
// dependent reads (length, page).
template <int DT, int D, int GS>
__global__ __launch_bounds__(64 * kWaves) void append_kernel(Seqs s, const uint16_t* __restrict__ k,
                                                             int64_t k_row, int64_t k_head,
                                                             const uint16_t* __restrict__ v, int64_t v_row,
                                                             int64_t v_head) {
    constexpr int N = D / 16, C = D / 64, G = D / GS;
    __shared__ __align__(16) uint8_t codes[kWaves][4 * D];
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const int tok = lane / 16, c = lane % 16;
    const int page_size = 1 << s.page_shift;
    const Record rec(page_size, D, GS);
    for (int b = blockIdx.y; b < s.seqs; b += gridDim.y) {
        const Unit u = unit_of(s, b, wave);
        const bool any = u.any;
        const int i = 4 * u.bundle + tok - u.t.pos0;  // place among the new tokens
        const bool live = any && i >= 0 && i < u.t.n;
        uint16_t kv[N], vv[N];
#pragma unroll
        for (int e = 0; e < N; ++e) kv[e] = vv[e] = 0;
        if (live) {
            const int64_t row = u.t.row0 + i;
            load_values<N>(k + row * k_row + u.head * k_head + c * N, kv);
            load_values<N>(v + row * v_row + u.head * v_head + c * N, vv);
        }
        const int64_t page = any ? page_of(s, b, 4 * u.bundle) : -1;
        uint32_t* r = s.pool + (page * s.kv_heads + u.head) * rec.words();  // used where page >= 0
        const int slot = (4 * u.bundle) & (page_size - 1);
        if (page >= 0) {
            uint32_t q[N];
            const int sb = (slot / 4) * G * 4;  // words of the bundles before
            quantize_lane<DT, D, GS>(kv, q, reinterpret_cast<uint16_t*>(r + rec.k_sb() + sb), tok, c, live);
            if (live) store_k<D>(r + rec.k_codes() + (slot + tok) * (D / 8), q, c);
            quantize_lane<DT, D, GS>(vv, q, reinterpret_cast<uint16_t*>(r + rec.v_sb() + sb), tok, c, live);
#pragma unroll
            for (int e = 0; e < N; ++e) codes[wave][code_at<D>(tok, c * N + e)] = static_cast<uint8_t>(q[e]);
        }
        __syncthreads();
        if (page >= 0) {
            // V codes: word (i, p, cc) of the bundle
            uint32_t* dst = r + rec.v_codes() + (slot / 4) * (32 * C);
            const int first = u.t.pos0 - 4 * u.bundle, last = first + u.t.n;  // new tokens of the bundle: [first, last)
#pragma unroll
            for (int w0 = 0; w0 < 32 * C; w0 += 64) {
                const int w = w0 + lane;
                if (w < 32 * C) {
                    const int p = (w / C) % 2, at = code_at<D>(2 * p, 64 * (w % C) + w / (2 * C));
                    uint32_t h[2];
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        // four codes, a byte each, to four nibbles
                        uint32_t x = *reinterpret_cast<const uint32_t*>(&codes[wave][at + half * D]);
                        x |= x >> 4;
                        h[half] = (x & 0xFFu) | ((x >> 8) & 0xFF00u);
                    }
                    const bool lo = 2 * p >= first && 2 * p < last, hi = 2 * p + 1 >= first && 2 * p + 1 < last;
                    if (lo && hi) dst[w] = h[0] | (h[1] << 16);
                    else if (lo || hi) reinterpret_cast<uint16_t*>(dst + w)[hi ? 1 : 0] = static_cast<uint16_t>(hi ? h[1] : h[0]);
                }
            }
        }
        __syncthreads();  // the codes are read before the next sequence's are written
    }
}

// The way back: the same prompts 10.8 us, 3.7 TB/s; the small calls 3.6 and 3.8.
template <int DT, int D, int GS>
__global__ __launch_bounds__(64 * kWaves) void read_kernel(Seqs s, uint16_t* __restrict__ k,
                                                           uint16_t* __restrict__ v) {
    constexpr int N = D / 16, C = D / 64, G = D / GS, S = D / 32, KW = D / 128 ? D / 128 : 1;
    __shared__ uint32_t vw[kWaves][32 * C];
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const int tok = lane / 16, c = lane % 16;
    const int page_size = 1 << s.page_shift;
    const Record rec(page_size, D, GS);
    for (int b = blockIdx.y; b < s.seqs; b += gridDim.y) {
        const Unit u = unit_of(s, b, wave);
        const bool any = u.any;
        const int64_t page = any ? page_of(s, b, 4 * u.bundle) : -1;
        const uint32_t* r = s.pool + (page * s.kv_heads + u.head) * rec.words();  // used where page >= 0
        const int slot = (4 * u.bundle) & (page_size - 1);
        float sc[2] = {0.0f, 0.0f}, bi[2] = {0.0f, 0.0f};
        uint32_t kw[KW];
#pragma unroll
        for (int x = 0; x < KW; ++x) kw[x] = 0;
        if (page >= 0) {
            const int sb = ((slot / 4) * G + c * N / GS) * 8 + tok;
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                const uint16_t* q = reinterpret_cast<const uint16_t*>(r + (part ? rec.v_sb() : rec.k_sb())) + sb;
                sc[part] = DtOps<DT>::to_f32(q[0]);
                bi[part] = DtOps<DT>::to_f32(q[4]);
            }
#pragma unroll
            for (int x = 0; x < KW; ++x) {
                const int w = c * N / 8 + x;
                kw[x] = r[rec.k_codes() + (slot + tok) * (D / 8) + (w % 4) * S + w / 4];
            }
            const uint32_t* src = r + rec.v_codes() + (slot / 4) * (32 * C);
#pragma unroll
            for (int w0 = 0; w0 < 32 * C; w0 += 64)
                if (w0 + lane < 32 * C) vw[wave][w0 + lane] = src[w0 + lane];
        }
        __syncthreads();
        const int i = 4 * u.bundle + tok - u.t.pos0;
        if (any && i >= 0 && i < u.t.n) {
            const int64_t at = ((u.t.row0 + i) * s.kv_heads + u.head) * D + c * N;
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                uint16_t o[N];
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const int d = c * N + e;
                    uint32_t code = 0;
                    if (part == 0) code = kw[e / 8] >> (D == 64 ? 16 * (c & 1) + 4 * e : 4 * (e % 8));
                    else if (page >= 0)
                        code = vw[wave][((d % 16) * 2 + tok / 2) * C + d / 64] >> (4 * ((d % 64) / 16) + 16 * (tok & 1));
                    o[e] = DtOps<DT>::rne(__fmaf_rn(sc[part], static_cast<float>(code & 15u), bi[part]));
                }
                store_values<N>((part ? v : k) + at, o);
            }
        }
        __syncthreads();
    }
}

template <int DT, int D, int GS>
hipError_t append_t(const Seqs& s, Rows k, Rows v, hipStream_t st) {
    hipLaunchKernelGGL((append_kernel<DT, D, GS>), grid_of(s), dim3(64 * kWaves), 0, st, s,
                       static_cast<const uint16_t*>(k.p), k.stride_row,
                       k.stride_head, static_cast<const uint16_t*>(v.p), v.stride_row, v.stride_head);
    return hipGetLastError();
}

template <int DT, int D, int GS>
hipError_t read_t(const Seqs& s, void* k, void* v, hipStream_t st) {
    hipLaunchKernelGGL((read_kernel<DT, D, GS>), grid_of(s), dim3(64 * kWaves), 0, st, s,
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
