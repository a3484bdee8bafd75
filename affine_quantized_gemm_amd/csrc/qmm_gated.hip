// Gated block on quantized weights: how a call is split, and its launch.
#include "qmm_gated.hpp"
#include "qmm_gated_dx.hpp"

namespace qmm {
namespace gated {

template <> GatedFn gated_fn<DT_F16, 4>(int);
template <> GatedFn gated_fn<DT_F16, 6>(int);
template <> GatedFn gated_fn<DT_F16, 8>(int);
template <> GatedFn gated_fn<DT_BF16, 4>(int);
template <> GatedFn gated_fn<DT_BF16, 6>(int);
template <> GatedFn gated_fn<DT_BF16, 8>(int);
template <> DxFn dx_fn<DT_F16, 4>(int);
template <> DxFn dx_fn<DT_F16, 6>(int);
template <> DxFn dx_fn<DT_F16, 8>(int);
template <> DxFn dx_fn<DT_BF16, 4>(int);
template <> DxFn dx_fn<DT_BF16, 6>(int);
template <> DxFn dx_fn<DT_BF16, 8>(int);

namespace {

__global__ __launch_bounds__(256) void gated_dx_zero_kernel(uint4* y, int64_t n) {
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (at < n) y[at] = make_uint4(0, 0, 0, 0);
}

}  // namespace
}  // namespace gated

hipError_t launch_gated(const GatedArgs& a) {
    using namespace gated;
    GatedParams p{};
    p.x = static_cast<const uint16_t*>(a.x);
    p.wq = a.wq;
    p.scales = static_cast<const uint16_t*>(a.scales);
    p.biases = static_cast<const uint16_t*>(a.biases);
    p.grad = static_cast<const uint16_t*>(a.grad);
    p.out = static_cast<uint16_t*>(a.out);
    p.d = a.d;
    p.M = static_cast<int>(a.M);
    p.act = a.act;
    p.F = a.F;
    p.K = a.K;
    p.words = static_cast<int>(a.K * a.bits / 32);
    p.groups = static_cast<int>(a.K / a.gs);
    const int super = super_of(a.bits);
    p.supers = static_cast<int>((a.K + super - 1) / super);
    // Row tiles: a workgroup widens the codes once for all of its tiles, its other row blocks do it again.  4096 to 2 x
    // 14336, us with one, two and four tiles: 4 bits (bf16, groups of 64) 16 rows 21 23 29, 17 rows 32 24 30, 32 rows 32 27
    // 33, 33 rows 56 41 36, 64 rows 57 41 41; 6 bits (fp16, groups of 128) 16 rows 36 38 40, 17 rows 56 38 41, 33 rows 97 64
    // 47, 64 rows 96 62 52; 8 bits alike.
    // K not of whole superblocks: one tile and loads that are looked at one by one.  2 x 8192 columns, beside the next whole
    // K: 4 bits, groups of 64, 6 rows of 2880 14.0 us and of 2816 11.7, 64 rows 24.9 and 31.2; groups of 32 (11 registers
    // spilled) 6 rows of 896 8.9 and of 1024 6.7, of 1152 13.5 and of 1280 8.7, 64 rows of 896 18.2 and of 1024 16.6; 6 bits,
    // 64 rows of 1088 17.7 and of 1152 17.2; 8 bits, 64 rows of 2880 29.5 and of 2816 26.0.  (The row blocks' second and
    // later readings come from L2.)
    const bool vec = a.K % super == 0;
    const int rt = !vec || a.M <= 16 ? 1 : a.M <= 32 ? 2 : 4;
    const int row_blocks = static_cast<int>((a.M + 16 * rt - 1) / (16 * rt));
    const int rows = static_cast<int>(a.M < 16 * rt ? a.M : 16 * rt);
    const int64_t tiles16 = (a.F + 15) / 16;
    // the wavefronts that all superblocks would keep busy, one each, are few
    const bool few = rt == 1 && tiles16 * row_blocks * (p.supers < 16 ? p.supers : 16) <= 128 * 16;
    const int waves = waves_of(rt, few);
    // superblocks of x that LDS holds beside the slots
    int most = (kLds - waves * slot_bytes(a.bits, a.gs, rt) - 16 * rows) / (2 * super * rows + 4 * (super / a.gs) * sums_of(rt));
    int held = 64 * waves * 8 / super;  // a row's pieces are at most the threads
    if (rt > 1) {                       // and a chunk passes through their registers
        const int all = pieces_of(rt) * 64 * waves * 8 / (rows * super);
        held = all < held ? all : held;
    }
    most = held < most ? held : most;
    // shares of K (x of all of them goes through LDS together) for as many workgroups as the chip holds at a time
    const int64_t hold = 256;
    while ((2 << p.ks_shift) <= waves && (2 << p.ks_shift) <= most && (1 << p.ks_shift) < p.supers &&
           (tiles16 << (p.ks_shift + 1)) * row_blocks <= hold * waves)
        ++p.ks_shift;
    const int ks = 1 << p.ks_shift;
    const int64_t tiles = (tiles16 * ks + waves - 1) / waves;
    if (tiles > INT32_MAX / 2) return hipErrorInvalidValue;
    p.tiles = static_cast<int>(tiles);
    // a multiple of 8, so that the row blocks of a column share an XCD's L2
    const int64_t grid_x = tiles < hold ? (tiles + 7) / 8 * 8 : hold;
    p.per = (p.supers + ks - 1) / ks;
    if (tiles > grid_x) p.per += p.per % 2;
    while ((1 << p.steps_shift) < p.per && (2 << p.steps_shift) * ks <= most) ++p.steps_shift;
    p.chunk = super * ks << p.steps_shift;
    p.piece_shift = __builtin_ctz(p.chunk / 8);
    p.chunks = (p.per + (1 << p.steps_shift) - 1) >> p.steps_shift;
    const int bytes = lds_bytes(a.bits, a.gs, rt, waves, rows, p.chunk);
    const dim3 grid(static_cast<unsigned>(grid_x), static_cast<unsigned>(row_blocks));
    GatedFn fn = nullptr;
    const bool half = a.dt == DT_F16;
    switch (a.bits) {
        case 4: fn = half ? gated_fn<DT_F16, 4>(a.gs) : gated_fn<DT_BF16, 4>(a.gs); break;
        case 6: fn = half ? gated_fn<DT_F16, 6>(a.gs) : gated_fn<DT_BF16, 6>(a.gs); break;
        case 8: fn = half ? gated_fn<DT_F16, 8>(a.gs) : gated_fn<DT_BF16, 8>(a.gs); break;
        default: break;
    }
    return fn != nullptr ? fn(p, rt, few, vec, grid, bytes, a.stream) : hipErrorInvalidValue;
}

// Slices for the workgroups that the chip holds at a time: two a CU with one
// row tile, else one.  (4 bits, 4096 to 2 x 14336, the whole call in us with 128,
// 256, 512 and 1024 workgroups: 6 rows 68 49 48 52, 16 rows 70 52 51 56, 17 rows
// 87 62 64 73, 37 rows 116 84 91 107, 64 rows 140 101 113 135.)
GatedDxPlan gated_dx_plan(int64_t M, int64_t F, int64_t K) {
    using namespace gated;
    const int64_t blocks = (K + kDxCols - 1) / kDxCols, chunks = (2 * F + kDxRows - 1) / kDxRows;
    int64_t slices = (M <= 16 ? 512 : 256) / blocks;
    slices = slices < 1 ? 1 : slices < chunks ? slices : chunks;
    const int64_t slice = (chunks + slices - 1) / slices * kDxRows;
    return {static_cast<int>((2 * F + slice - 1) / slice), slice};
}

hipError_t launch_gated_dx(const GatedArgs& a, void* y, float* part) {
    using namespace gated;
    const GatedDxPlan plan = gated_dx_plan(a.M, a.F, a.K);
    DxParams p{};
    p.d = a.d;
    p.wq = a.wq;
    p.scales = static_cast<const uint16_t*>(a.scales);
    p.biases = static_cast<const uint16_t*>(a.biases);
    p.y = static_cast<uint16_t*>(y);
    p.part = part;
    p.M = static_cast<int>(a.M);
    p.N = 2 * a.F;
    p.K = a.K;
    p.slice = plan.slice;
    const dim3 grid(static_cast<unsigned>((a.K + kDxCols - 1) / kDxCols), static_cast<unsigned>(plan.slices));
    DxFn fn = nullptr;
    const bool half = a.dt == DT_F16;
    switch (a.bits) {
        case 4: fn = half ? dx_fn<DT_F16, 4>(a.gs) : dx_fn<DT_BF16, 4>(a.gs); break;
        case 6: fn = half ? dx_fn<DT_F16, 6>(a.gs) : dx_fn<DT_BF16, 6>(a.gs); break;
        case 8: fn = half ? dx_fn<DT_F16, 8>(a.gs) : dx_fn<DT_BF16, 8>(a.gs); break;
        default: break;
    }
    if (fn == nullptr) return hipErrorInvalidValue;
    const hipError_t e = fn(p, static_cast<int>((a.M + 15) / 16), grid, a.stream);
    if (e != hipSuccess || plan.slices == 1) return e;
    return launch_reduce_partials(a.dt, part, y, plan.slices, a.M * a.K, a.stream);
}

hipError_t launch_gated_dx_zero(void* y, int64_t n, hipStream_t st) {
    const dim3 grid(static_cast<unsigned>((n / 8 + 255) / 256));
    hipLaunchKernelGGL(gated::gated_dx_zero_kernel, grid, dim3(256), 0, st, static_cast<uint4*>(y), n / 8);
    return hipGetLastError();
}

}  // namespace qmm
