// Rotary positions on one to four axes (gfx950).
//
// Pair p of a head of row r is turned by angle = pos[axis(p)][r] * freq[p]:
//   (a, b) -> scale (a cos - b sin, b cos + a sin),
// inverse by minus the angle, which is the transposed map, so also the
// gradient's.  An angle of a far position has lost everything below 2 pi in
// fp32 (position 10^6 is 0.06 off), so revolutions pos * freq / (2 pi) are
// formed in fp64 and only what is left of them after the whole ones goes to
// fp32; the products and sums are fp32, rounded once.
//
// The angles are the same for all heads: a workgroup forms those of its rows
// once, one thread a pair, and keeps cos and sin in LDS; then a thread turns
// eight pairs at a time, two 16-byte loads and stores.  (8191 rows, 40 heads of
// 128, three axes: 34 us, 4.9 TB/s read and written, a copy's rate; 28 rows 3.6
// us, the chain of position, angle, table, value.)
#include "qmm_device.hpp"
#include "qmm_rows.hpp"

namespace qmm {
namespace {

constexpr int kThreads = 256;
constexpr int kTable = 1024;  // pairs' cos and sin in LDS: 8 KiB
constexpr int kAhead = 4;     // items of a thread on their way

struct RotaryParams {
    RotaryArgs a;
    int per;              // items of a head: 8 pairs each, then 8 unturned values each
    uint32_t per_magic, heads_magic;
    int row_block, head_block;
};

// n / d for n d < 2^32, with magic = ceil(2^32 / d); d = 1 has no such magic.
__device__ __forceinline__ uint32_t divide(uint32_t n, uint32_t d, uint32_t magic) {
    return d == 1 ? n : __umulhi(n, magic);
}

template <int DT, bool ADJACENT>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryParams p) {
    __shared__ float2 table[kTable];
    const RotaryArgs& a = p.a;
    const int half = a.half;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.row_block;
    const int rows = a.rows - row0 < p.row_block ? static_cast<int>(a.rows - row0) : p.row_block;
    const int head0 = blockIdx.y * p.head_block;
    const int heads = a.heads - head0 < p.head_block ? a.heads - head0 : p.head_block;
    // (items are counted with head_block heads a row; a last block that has fewer passes over the others')
    const uint32_t all = static_cast<uint32_t>(rows) * p.head_block * p.per;

    struct Place {
        int row, head, v;
        int64_t in, out;  // of the head
    };
    auto place = [&](uint32_t item) {
        const uint32_t slot = divide(item, p.per, p.per_magic);
        const uint32_t row = divide(slot, p.head_block, p.heads_magic);
        Place q;
        q.row = row;
        q.head = slot - row * p.head_block;
        q.v = item - slot * p.per;
        const int64_t r = row0 + row, h = head0 + q.head;
        q.in = r * a.x_row + h * a.x_head;
        q.out = r * a.out_row + h * a.out_head;
        return q;
    };
    const int nv = half / 8;
    uint4 lo[kAhead], hi[kAhead];
    Place at[kAhead];
    bool have[kAhead];
    auto fetch = [&](uint32_t first) {
#pragma unroll
        for (int n = 0; n < kAhead; ++n) {
            const uint32_t item = first + n * kThreads;
            at[n] = place(item < all ? item : 0);
            have[n] = item < all && at[n].head < heads;
            if (have[n]) {
                const uint16_t* x = static_cast<const uint16_t*>(a.x) + at[n].in;
                const int v = at[n].v;
                if (v >= nv) {
                    lo[n] = *reinterpret_cast<const uint4*>(x + 2 * half + 8 * (v - nv));
                } else if constexpr (ADJACENT) {
                    lo[n] = *reinterpret_cast<const uint4*>(x + 16 * v);
                    hi[n] = *reinterpret_cast<const uint4*>(x + 16 * v + 8);
                } else {
                    lo[n] = *reinterpret_cast<const uint4*>(x + 8 * v);
                    hi[n] = *reinterpret_cast<const uint4*>(x + half + 8 * v);
                }
            }
        }
    };
    fetch(threadIdx.x);  // on their way while the angles are formed

    for (int k = threadIdx.x; k < rows * half; k += kThreads) {
        const int row = k / half, pair = k - row * half;
        const int axis = (pair >= a.cut[0]) + (pair >= a.cut[1]) + (pair >= a.cut[2]);
        const int64_t where = axis * a.pos_axis + row0 + row;
        const double pos = a.pos64 ? static_cast<double>(static_cast<const int64_t*>(a.pos)[where])
                                   : static_cast<double>(static_cast<const int32_t*>(a.pos)[where]);
        const double turns = pos * (static_cast<double>(a.freq[pair]) * 0.15915494309189533577);
        float s, c;
        sincospif(2.0f * static_cast<float>(turns - rint(turns)), &s, &c);
        table[k] = make_float2(c * a.scale, (a.inverse ? -s : s) * a.scale);
    }
    __syncthreads();

    for (uint32_t first = threadIdx.x; first < all; first += kAhead * kThreads) {
#pragma unroll
        for (int n = 0; n < kAhead; ++n) {
            if (!have[n]) continue;
            uint16_t* out = static_cast<uint16_t*>(a.out) + at[n].out;
            const int v = at[n].v;
            if (v >= nv) {
                *reinterpret_cast<uint4*>(out + 2 * half + 8 * (v - nv)) = lo[n];
                continue;
            }
            const float2* t = table + at[n].row * half + 8 * v;
            const uint32_t l[4] = {lo[n].x, lo[n].y, lo[n].z, lo[n].w}, h[4] = {hi[n].x, hi[n].y, hi[n].z, hi[n].w};
            uint32_t y[4], z[4];
            if constexpr (ADJACENT) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float a0 = low_f32<DT>(l[e]), b0 = high_f32<DT>(l[e]), a1 = low_f32<DT>(h[e]), b1 = high_f32<DT>(h[e]);
                    y[e] = pack2<DT>(a0 * t[e].x - b0 * t[e].y, b0 * t[e].x + a0 * t[e].y);
                    z[e] = pack2<DT>(a1 * t[4 + e].x - b1 * t[4 + e].y, b1 * t[4 + e].x + a1 * t[4 + e].y);
                }
                *reinterpret_cast<uint4*>(out + 16 * v) = make_uint4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<uint4*>(out + 16 * v + 8) = make_uint4(z[0], z[1], z[2], z[3]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float a0 = low_f32<DT>(l[e]), a1 = high_f32<DT>(l[e]), b0 = low_f32<DT>(h[e]), b1 = high_f32<DT>(h[e]);
                    const float2 t0 = t[2 * e], t1 = t[2 * e + 1];
                    y[e] = pack2<DT>(a0 * t0.x - b0 * t0.y, a1 * t1.x - b1 * t1.y);
                    z[e] = pack2<DT>(b0 * t0.x + a0 * t0.y, b1 * t1.x + a1 * t1.y);
                }
                *reinterpret_cast<uint4*>(out + 8 * v) = make_uint4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<uint4*>(out + half + 8 * v) = make_uint4(z[0], z[1], z[2], z[3]);
            }
        }
        if (first + kAhead * kThreads < all) fetch(first + kAhead * kThreads);
    }
}

uint32_t magic_of(int d) { return d > 1 ? static_cast<uint32_t>(((uint64_t{1} << 32) + d - 1) / d) : 0; }

}  // namespace

hipError_t launch_rotary(int dt, const RotaryArgs& a, hipStream_t st) {
    RotaryParams p{};
    p.a = a;
    p.per = a.half / 8 + (a.dim - 2 * a.half) / 8;
    // rows whose angles make one a thread; then heads, up to where the grid still has two workgroups a CU
    p.row_block = a.half >= kThreads ? 1 : kThreads / a.half;
    const int64_t row_blocks = (a.rows + p.row_block - 1) / p.row_block;
    int hb = (kThreads + p.row_block * p.per - 1) / (p.row_block * p.per);
    while (hb < a.heads && hb < 64 && row_blocks * ((a.heads + 2 * hb - 1) / (2 * hb)) >= 512) hb *= 2;
    p.head_block = hb < a.heads ? hb : a.heads;
    p.per_magic = magic_of(p.per);
    p.heads_magic = magic_of(p.head_block);
    const int64_t head_blocks = (a.heads + p.head_block - 1) / p.head_block;
    if (head_blocks > 65535) return hipErrorInvalidValue;
    const int64_t most = UINT32_MAX / kThreads * static_cast<int64_t>(p.row_block);  // rows of a launch: a grid's threads are 32 bits on an axis
    for (int64_t row = 0; row < a.rows; row += most) {
        p.a.rows = a.rows - row < most ? a.rows - row : most;
        p.a.x = static_cast<const uint16_t*>(a.x) + row * a.x_row;
        p.a.out = static_cast<uint16_t*>(a.out) + row * a.out_row;
        p.a.pos = static_cast<const char*>(a.pos) + row * (a.pos64 ? 8 : 4);
        const dim3 grid(static_cast<unsigned>((p.a.rows + p.row_block - 1) / p.row_block), static_cast<unsigned>(head_blocks));
        if (dt == DT_F16) {
            if (a.adjacent) hipLaunchKernelGGL((rotary_kernel<DT_F16, true>), grid, dim3(kThreads), 0, st, p);
            else hipLaunchKernelGGL((rotary_kernel<DT_F16, false>), grid, dim3(kThreads), 0, st, p);
        } else {
            if (a.adjacent) hipLaunchKernelGGL((rotary_kernel<DT_BF16, true>), grid, dim3(kThreads), 0, st, p);
            else hipLaunchKernelGGL((rotary_kernel<DT_BF16, false>), grid, dim3(kThreads), 0, st, p);
        }
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace qmm
