// Gradient of the gated block for x: bf16, 8-bit codes.
#include "qmm_gated_dx.hpp"
QMM_GATED_DX_UNIT(qmm::DT_BF16, 8)
