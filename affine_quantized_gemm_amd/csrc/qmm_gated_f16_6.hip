// Gated block on quantized weights: fp16, 6-bit codes.
#include "qmm_gated.hpp"
QMM_GATED_UNIT(qmm::DT_F16, 6)
