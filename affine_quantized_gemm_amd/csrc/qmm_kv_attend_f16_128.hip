// Attention over the 4-bit cache: f16, head size 128.
#include "qmm_kv_attend.hpp"
QMM_KV_ATTEND_UNIT(qmm::DT_F16, 128, false)
