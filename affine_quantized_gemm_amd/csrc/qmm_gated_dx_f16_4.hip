// Gradient of the gated block for x: fp16, 4-bit codes.
#include "qmm_gated_dx.hpp"
QMM_GATED_DX_UNIT(qmm::DT_F16, 4)
