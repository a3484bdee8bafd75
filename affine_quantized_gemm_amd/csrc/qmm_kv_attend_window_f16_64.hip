// Attention over a window of the 4-bit cache: f16, head size 64.
#include "qmm_kv_attend.hpp"
QMM_KV_ATTEND_UNIT(qmm::DT_F16, 64, true)
