// Gated block on quantized weights: bf16, 8-bit codes.
#include "qmm_gated.hpp"
QMM_GATED_UNIT(qmm::DT_BF16, 8)
