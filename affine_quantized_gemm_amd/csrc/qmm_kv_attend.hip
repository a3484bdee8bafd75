// Attention over the paged 4-bit K/V cache: the plain kernel.
//
// One workgroup a (row, head): 256 threads take 256 tokens at a time, one
// score each; the running maximum and sum of the softmax are kept in fp32,
// and threads then take one value d each over the tile's probabilities.
#include "qmm_device.hpp"
#include "qmm_kv.hpp"

namespace qmm {
namespace kv {
namespace {

constexpr int kT = 256;

template <int DT>
__global__ __launch_bounds__(kT) void attend_kernel(Seqs s, int D, int GS, const uint16_t* __restrict__ q,
                                                    int64_t q_row, int64_t q_head, int heads, float scale,
                                                    const int64_t* __restrict__ mask, uint16_t* __restrict__ out,
                                                    float* __restrict__ lse) {
    __shared__ float qs[256], ps[kT];
    __shared__ float red[4];
    __shared__ int64_t pg[kT];
    const int tid = threadIdx.x;
    const int h = blockIdx.x % heads;
    const int64_t bi = blockIdx.x / heads;
    const int b = static_cast<int>(bi / s.max_new), i = static_cast<int>(bi % s.max_new);
    const NewTokens t = new_tokens(s, b);
    if (i >= t.n) return;
    const int kh = h / (heads / s.kv_heads);
    const int page = 1 << s.page_shift;
    const Record rec(page, D, GS);
    const int G = D / GS, S = D / 32, C = D / 64;
    const int64_t row = t.row0 + i;
    for (int d = tid; d < D; d += kT) qs[d] = DtOps<DT>::to_f32(q[row * q_row + h * q_head + d]);
    __syncthreads();
    const int64_t cap = s.width << s.page_shift;
    int64_t len = static_cast<int64_t>(t.pos0) + t.n;
    if (len > cap) len = cap;
    const uint64_t bits = mask ? static_cast<uint64_t>(mask[row]) : ~uint64_t{0} >> (63 - i);
    float m = -__builtin_inff(), l = 0.f, o = 0.f;
    for (int64_t base = 0; base < len; base += kT) {
        const int64_t pos = base + tid;
        float sc = -__builtin_inff();
        int64_t p = -1;
        if (pos < len) {
            const int64_t j = pos - t.pos0;
            if (j < 0 || ((bits >> j) & 1)) p = page_of(s, b, static_cast<int>(pos));
        }
        pg[tid] = p;
        if (p >= 0) {
            const uint32_t* r = s.pool + (p * s.kv_heads + kh) * rec.words();
            const int slot = static_cast<int>(pos) & (page - 1);
            const uint16_t* sb = reinterpret_cast<const uint16_t*>(r + rec.k_sb()) + (slot / 4) * G * 8 + slot % 4;
            float acc = 0.f;
            for (int w = 0; w < D / 8; ++w) {
                const uint32_t word = r[rec.k_codes() + slot * (D / 8) + (w % 4) * S + w / 4];
                const int g = 8 * w / GS;
                const float ks = DtOps<DT>::to_f32(sb[g * 8]), kb = DtOps<DT>::to_f32(sb[g * 8 + 4]);
                for (int e = 0; e < 8; ++e)
                    acc += qs[8 * w + e] * (ks * static_cast<float>((word >> (4 * e)) & 15u) + kb);
            }
            sc = acc * scale;
        }
        float top = sc;
        for (int x = 1; x < 64; x *= 2) top = fmaxf(top, __shfl_xor(top, x));
        if (tid % 64 == 0) red[tid / 64] = top;
        __syncthreads();
        top = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
        const float pr = sc > -__builtin_inff() ? expf(sc - top) : 0.f;
        const float keep = m > -__builtin_inff() ? expf(m - top) : 0.f;
        ps[tid] = pr;
        float sum = pr;
        for (int x = 1; x < 64; x *= 2) sum += __shfl_xor(sum, x);
        __syncthreads();
        if (tid % 64 == 0) red[tid / 64] = sum;
        __syncthreads();
        l = l * keep + red[0] + red[1] + red[2] + red[3];
        m = top;
        o *= keep;
        if (tid < D) {
            const int d = tid;
            for (int x = 0; x < kT; ++x) {
                if (pg[x] < 0) continue;
                const uint32_t* r = s.pool + (pg[x] * s.kv_heads + kh) * rec.words();
                const int slot = static_cast<int>(base + x) & (page - 1), tok = slot % 4;
                const uint16_t* sb = reinterpret_cast<const uint16_t*>(r + rec.v_sb()) + ((slot / 4) * G + d / GS) * 8 + tok;
                const uint32_t word = r[rec.v_codes() + (slot / 4) * (32 * C) + ((d % 16) * 2 + tok / 2) * C + d / 64];
                const uint32_t code = (word >> (4 * ((d % 64) / 16) + 16 * (tok & 1))) & 15u;
                o += ps[x] * (DtOps<DT>::to_f32(sb[0]) * static_cast<float>(code) + DtOps<DT>::to_f32(sb[4]));
            }
        }
        __syncthreads();
    }
    if (tid < D) out[(row * heads + h) * D + tid] = DtOps<DT>::rne(l > 0.f ? o / l : 0.f);
    if (lse != nullptr && tid == 0) lse[row * heads + h] = l > 0.f ? m + logf(l) : -__builtin_inff();
}

}  // namespace

int64_t attend_workspace(const qmm_kv_cache&, int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_attend(const qmm_kv_cache& c, const AttendArgs& a) {
    const int64_t blocks = static_cast<int64_t>(a.s.seqs) * a.s.max_new * a.heads;
    if (blocks > INT32_MAX) return hipErrorInvalidValue;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kT), 0, a.stream, a.s, c.head_dim,
                           c.group_size, static_cast<const uint16_t*>(a.q.p), a.q.stride_row, a.q.stride_head,
                           a.heads, a.scale, a.mask, static_cast<uint16_t*>(a.out), a.lse);
        return hipGetLastError();
    };
    return c.dt == QMM_F16 ? go(attend_kernel<DT_F16>) : go(attend_kernel<DT_BF16>);
}

}  // namespace kv
}  // namespace qmm
