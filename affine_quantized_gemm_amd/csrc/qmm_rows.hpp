// What the operators on rows share: rotary positions, log probabilities, the
// gated block (arguments, validated by the boundary; conversions).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmm_device.hpp"

namespace qmm {

// The halves of a word as fp32.
template <int DT>
__device__ __forceinline__ float low_f32(uint32_t w) {
    if constexpr (DT == DT_F16) return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(w)));
    else return __builtin_bit_cast(float, w << 16);
}
template <int DT>
__device__ __forceinline__ float high_f32(uint32_t w) {
    if constexpr (DT == DT_F16) return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(w >> 16)));
    else return __builtin_bit_cast(float, w & 0xFFFF0000u);
}
// Two values rounded to nearest (even); NaN stays NaN.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    typedef float float2_t __attribute__((ext_vector_type(2)));
    if constexpr (DT == DT_F16) {
        typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((float2_t{lo, hi}), half2_t));
    } else {
        typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((float2_t{lo, hi}), bf16x2_t));
    }
}

struct RotaryArgs {
    const void* x;
    int64_t x_row, x_head;
    void* out;
    int64_t out_row, out_head;
    int64_t rows;
    int heads, dim, half;  // half: turned pairs of a head
    bool adjacent, inverse, pos64;
    float scale;
    const void* pos;       // [axes][rows], the axes pos_axis apart
    int64_t pos_axis;
    int cut[3];            // first pair of the second, third and fourth axis
    const float* freq;     // [half]
};
hipError_t launch_rotary(int dt, const RotaryArgs& a, hipStream_t st);

struct LogProbsArgs {
    const void* logits;
    int64_t stride, rows, vocab;
    float scale;
    const void* tokens;    // [rows][given] or null
    bool tokens64;
    int given, top;
    float* lse;
    float* entropy;
    float* token_lp;       // [rows][given]
    float* top_values;     // [rows][top]
    int64_t* top_ids;
    void* workspace;
};
int log_probs_parts(int64_t rows, int64_t vocab);
hipError_t launch_log_probs(int dt, const LogProbsArgs& a, hipStream_t st);

struct LogProbsGradArgs {
    const void* logits;
    int64_t stride, rows, vocab;
    float scale;
    const void* tokens;
    bool tokens64;
    int given;
    const float* lse;
    const float* entropy;      // null without grad_entropy
    const float* grad_tokens;  // [rows][given] or null
    const float* grad_entropy;
    const float* grad_lse;
    void* out;
    int64_t out_stride;
};
hipError_t launch_log_probs_grad(int dt, const LogProbsGradArgs& a, hipStream_t st);

struct GatedArgs {
    int dt, bits, gs, act;
    int64_t M, F, K;
    const void* x;
    const uint32_t* wq;    // [2F] rows: the gate's, then the other product's
    const void* scales;
    const void* biases;
    const void* grad;      // [M][F] or null
    void* out;             // [M][F]; with grad [M][2F]
    float* d;              // with grad: the same in fp32
    hipStream_t stream;
};
hipError_t launch_gated(const GatedArgs& a);
// y [M][K] = d [M][2F] . W, sums of slices in part where there are several.
struct GatedDxPlan {
    int slices;
    int64_t slice;         // rows of W
};
GatedDxPlan gated_dx_plan(int64_t M, int64_t F, int64_t K);
hipError_t launch_gated_dx(const GatedArgs& a, void* y, float* part);
// n zeros of 2 bytes, a multiple of 8.
hipError_t launch_gated_dx_zero(void* y, int64_t n, hipStream_t st);

}  // namespace qmm
