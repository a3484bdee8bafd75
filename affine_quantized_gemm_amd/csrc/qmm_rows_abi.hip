// extern "C" boundary of the gated block, rotary positions and log
// probabilities: argument validation and launches on the caller's stream.
// Declarations and contracts: qmm.h.
#include <cmath>
#include <initializer_list>

#include "qmm.h"
#include "qmm_internal.hpp"
#include "qmm_rows.hpp"

namespace {

int hip_status(hipError_t e) { return e == hipSuccess ? QMM_OK : QMM_ERR_HIP; }

bool off(const void* p, unsigned align) { return (reinterpret_cast<uintptr_t>(p) & (align - 1)) != 0; }

int check_ptrs(std::initializer_list<const void*> ps, unsigned align) {
    for (const void* p : ps)
        if (p == nullptr) return QMM_ERR_INVALID_ARG;
    for (const void* p : ps)
        if (off(p, align)) return QMM_ERR_MISALIGNED;
    return QMM_OK;
}

bool known_dt(int dt) { return dt == QMM_F16 || dt == QMM_BF16; }

int check_gated(int dt, int bits, int gs, int64_t M, int64_t F, int64_t K) {
    if (M < 0 || F < 0 || K < 0) return QMM_ERR_INVALID_ARG;
    if (!known_dt(dt)) return QMM_ERR_UNSUPPORTED;
    if (bits != 4 && bits != 6 && bits != 8) return QMM_ERR_UNSUPPORTED;
    if (gs != 32 && gs != 64 && gs != 128) return QMM_ERR_UNSUPPORTED;
    if (K < 64 || K % 64 != 0 || K % gs != 0) return QMM_ERR_UNSUPPORTED;
    // (offsets within x and within 16 rows of weights are 32-bit)
    if (F > INT32_MAX / 2 || K > (1 << 24) || M > 64) return QMM_ERR_UNSUPPORTED;
    return QMM_OK;
}

bool known_act(int act) {
    return act == QMM_ACT_SILU || act == QMM_ACT_GELU || act == QMM_ACT_GELU_TANH || act == QMM_ACT_RELU;
}

// Whether all places (r, h, 0..dim) of an output lie apart.
bool apart(int64_t rows, int64_t heads, int64_t dim, int64_t row, int64_t head) {
    if (rows == 1) return heads == 1 || head >= dim;
    if (heads == 1) return row >= dim;
    return (head >= dim && row / heads >= head) || (row >= dim && head / rows >= row) ||
           (head >= dim && row >= (heads - 1) * head + dim) || (row >= dim && head >= (rows - 1) * row + dim);
}

}  // namespace

extern "C" {

int qmm_gated(int dt, int bits, int group_size, int act, int64_t M, int64_t F, int64_t K, const void* x,
              const uint32_t* wq, const void* scales, const void* biases, void* h, void* stream) {
    int st = check_gated(dt, bits, group_size, M, F, K);
    if (st != QMM_OK) return st;
    if (!known_act(act)) return QMM_ERR_UNSUPPORTED;
    if (M == 0 || F == 0) return QMM_OK;
    if ((st = check_ptrs({x, wq, scales, biases, h}, 16)) != QMM_OK) return st;
    const qmm::GatedArgs a{dt, bits, group_size, act, M, F, K, x, wq, scales, biases, nullptr, h, nullptr, static_cast<hipStream_t>(stream)};
    return hip_status(qmm::launch_gated(a));
}

int64_t qmm_gated_backward_workspace_bytes(int dt, int bits, int group_size, int64_t M, int64_t F, int64_t K) {
    if (const int st = check_gated(dt, bits, group_size, M, F, K); st != QMM_OK) return st;
    if (F % 16 != 0) return QMM_ERR_UNSUPPORTED;
    if (M == 0 || F == 0) return 0;
    const int slices = qmm::gated_dx_plan(M, F, K).slices;
    return 4 * M * (2 * F + (slices > 1 ? slices * K : 0));
}

int qmm_gated_backward(int dt, int bits, int group_size, int act, int64_t M, int64_t F, int64_t K, const void* x,
                       const uint32_t* wq, const void* scales, const void* biases, const void* grad,
                       void* grad_gate_up, void* grad_x, void* workspace, int64_t workspace_bytes, void* stream) {
    const int64_t need = qmm_gated_backward_workspace_bytes(dt, bits, group_size, M, F, K);
    if (need < 0) return static_cast<int>(need);
    if (!known_act(act)) return QMM_ERR_UNSUPPORTED;
    if (workspace_bytes < 0) return QMM_ERR_INVALID_ARG;
    if (M == 0) return QMM_OK;
    int st;
    if (F == 0) {  // a sum of nothing
        if ((st = check_ptrs({grad_x}, 16)) != QMM_OK) return st;
        return hip_status(qmm::launch_gated_dx_zero(grad_x, M * K, static_cast<hipStream_t>(stream)));
    }
    if ((st = check_ptrs({x, wq, scales, biases, grad, grad_gate_up, grad_x}, 16)) != QMM_OK) return st;
    if (workspace == nullptr || workspace_bytes < need) return QMM_ERR_INVALID_ARG;
    if (off(workspace, 16)) return QMM_ERR_MISALIGNED;
    // the workspace: the two gradients in fp32, then the sums of grad_x's slices
    float* const d = static_cast<float*>(workspace);
    const qmm::GatedArgs a{dt, bits, group_size, act, M, F, K, x, wq, scales, biases, grad, grad_gate_up, d, static_cast<hipStream_t>(stream)};
    if ((st = hip_status(qmm::launch_gated(a))) != QMM_OK) return st;
    return hip_status(qmm::launch_gated_dx(a, grad_x, d + M * 2 * F));
}

int qmm_rotary(int dt, int64_t rows, int64_t heads, int64_t head_dim, int64_t rotary_dim, int pairs, int inverse,
               float scale, const void* x, int64_t x_stride_row, int64_t x_stride_head, const void* positions,
               int positions_64, int64_t position_stride, int axes, const int32_t* sections, const float* freq,
               void* out, int64_t out_stride_row, int64_t out_stride_head, void* stream) {
    if (rows < 0 || heads < 0 || x_stride_row < 0 || x_stride_head < 0 || out_stride_row < 0 || out_stride_head < 0 ||
        position_stride < 0)
        return QMM_ERR_INVALID_ARG;
    if (!known_dt(dt) || (pairs != QMM_PAIRS_HALVES && pairs != QMM_PAIRS_ADJACENT)) return QMM_ERR_UNSUPPORTED;
    if (head_dim < 16 || head_dim > 1024 || head_dim % 8 != 0) return QMM_ERR_UNSUPPORTED;
    if (rotary_dim < 16 || rotary_dim > head_dim || rotary_dim % 16 != 0) return QMM_ERR_UNSUPPORTED;
    if (axes < 1 || axes > 4 || heads > INT32_MAX / 1024 || rows > INT32_MAX) return QMM_ERR_UNSUPPORTED;
    if (sections == nullptr && axes > 1) return QMM_ERR_INVALID_ARG;
    qmm::RotaryArgs a{};
    const int64_t half = rotary_dim / 2;
    int64_t at = 0;
    for (int n = 0; n < 3; ++n) a.cut[n] = INT32_MAX;  // (no pair lies there)
    for (int n = 0; n < axes && sections != nullptr; ++n) {
        if (sections[n] < 0) return QMM_ERR_INVALID_ARG;
        at += sections[n];
        if (n < axes - 1) a.cut[n] = static_cast<int>(at < half ? at : half);
    }
    if (sections != nullptr && at != half) return QMM_ERR_INVALID_ARG;
    if (rows == 0 || heads == 0) return QMM_OK;
    int st = check_ptrs({x, out}, 16);
    if (st != QMM_OK) return st;
    if (((x_stride_row | x_stride_head | out_stride_row | out_stride_head) & 7) != 0) return QMM_ERR_MISALIGNED;
    if ((st = check_ptrs({freq}, 4)) != QMM_OK) return st;
    if ((st = check_ptrs({positions}, positions_64 ? 8 : 4)) != QMM_OK) return st;
    if (!apart(rows, heads, head_dim, out_stride_row, out_stride_head)) return QMM_ERR_INVALID_ARG;
    a.x = x;
    a.x_row = x_stride_row;
    a.x_head = x_stride_head;
    a.out = out;
    a.out_row = out_stride_row;
    a.out_head = out_stride_head;
    a.rows = rows;
    a.heads = static_cast<int>(heads);
    a.dim = static_cast<int>(head_dim);
    a.half = static_cast<int>(half);
    a.adjacent = pairs == QMM_PAIRS_ADJACENT;
    a.inverse = inverse != 0;
    a.pos64 = positions_64 != 0;
    a.scale = scale;
    a.pos = positions;
    a.pos_axis = position_stride;
    a.freq = freq;
    return hip_status(qmm::launch_rotary(dt, a, static_cast<hipStream_t>(stream)));
}

// (columns are 32-bit numbers; rows of more than a launch holds go in several)
static int check_logits(int dt, int64_t rows, int64_t vocab, float scale, int64_t stride, int64_t given) {
    if (rows < 0 || vocab < 0 || stride < 0 || given < 0) return QMM_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || scale <= 0.0f) return QMM_ERR_INVALID_ARG;
    // (within these, logits further apart than fp32's largest leave a probability of 0, and the scale in base 2 is finite)
    if (scale < 0x1p-100f || scale > 0x1p100f) return QMM_ERR_UNSUPPORTED;
    if (!known_dt(dt) || given > 64 || rows > INT32_MAX || vocab > INT32_MAX - 1024) return QMM_ERR_UNSUPPORTED;
    return QMM_OK;
}

int qmm_log_probs_needs_workspace(int64_t rows, int64_t vocab) {
    if (rows < 0 || vocab < 0) return QMM_ERR_INVALID_ARG;
    if (rows > INT32_MAX || vocab > INT32_MAX - 1024) return QMM_ERR_UNSUPPORTED;
    return qmm::log_probs_parts(rows, vocab) > 1 ? 1 : 0;
}

int qmm_log_probs(int dt, int64_t rows, int64_t vocab, float scale, const void* logits, int64_t stride,
                  const void* tokens, int tokens_64, int64_t given, int64_t top, float* lse, float* entropy,
                  float* token_logprobs, float* top_logprobs, int64_t* top_ids, void* workspace,
                  int64_t workspace_bytes, void* stream) {
    int st = check_logits(dt, rows, vocab, scale, stride, given);
    if (st != QMM_OK) return st;
    if (top < 0 || workspace_bytes < 0) return QMM_ERR_INVALID_ARG;
    if (top > QMM_LOG_PROBS_MOST_TOP || top > vocab) return QMM_ERR_UNSUPPORTED;
    if (rows == 0) return QMM_OK;
    if (vocab == 0) return QMM_ERR_UNSUPPORTED;
    if ((st = check_ptrs({logits}, 2)) != QMM_OK) return st;
    if ((st = check_ptrs({lse, entropy}, 4)) != QMM_OK) return st;
    if (given > 0) {
        if ((st = check_ptrs({tokens}, tokens_64 ? 8 : 4)) != QMM_OK) return st;
        if ((st = check_ptrs({token_logprobs}, 4)) != QMM_OK) return st;
    }
    if (top > 0) {
        if ((st = check_ptrs({top_logprobs}, 4)) != QMM_OK) return st;
        if ((st = check_ptrs({top_ids}, 8)) != QMM_OK) return st;
    }
    if (qmm::log_probs_parts(rows, vocab) > 1) {
        if (workspace == nullptr || workspace_bytes < QMM_LOG_PROBS_WORKSPACE_BYTES) return QMM_ERR_INVALID_ARG;
        if (off(workspace, 16)) return QMM_ERR_MISALIGNED;
    }
    const qmm::LogProbsArgs a{logits, stride, rows, vocab, scale, tokens, tokens_64 != 0, static_cast<int>(given),
                              static_cast<int>(top), lse, entropy, token_logprobs, top_logprobs, top_ids, workspace};
    return hip_status(qmm::launch_log_probs(dt, a, static_cast<hipStream_t>(stream)));
}

int qmm_log_probs_backward(int dt, int64_t rows, int64_t vocab, float scale, const void* logits, int64_t stride,
                           const void* tokens, int tokens_64, int64_t given, const float* lse, const float* entropy,
                           const float* grad_tokens, const float* grad_entropy, const float* grad_lse, void* out,
                           int64_t out_stride, void* stream) {
    int st = check_logits(dt, rows, vocab, scale, stride, given);
    if (st != QMM_OK) return st;
    if (out_stride < 0 || (rows > 1 && out_stride < vocab)) return QMM_ERR_INVALID_ARG;
    if (rows == 0 || vocab == 0) return QMM_OK;
    if ((st = check_ptrs({logits, out}, 2)) != QMM_OK) return st;
    if ((st = check_ptrs({lse}, 4)) != QMM_OK) return st;
    if (grad_entropy != nullptr && (st = check_ptrs({entropy, grad_entropy}, 4)) != QMM_OK) return st;
    if (off(grad_lse, 4)) return QMM_ERR_MISALIGNED;
    if (given > 0 && grad_tokens != nullptr) {
        if ((st = check_ptrs({tokens}, tokens_64 ? 8 : 4)) != QMM_OK) return st;
        if (off(grad_tokens, 4)) return QMM_ERR_MISALIGNED;
    }
    const qmm::LogProbsGradArgs a{logits, stride, rows, vocab, scale, tokens, tokens_64 != 0, static_cast<int>(given), lse,
                                  entropy, grad_tokens, grad_entropy, grad_lse, out, out_stride};
    return hip_status(qmm::launch_log_probs_grad(dt, a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
