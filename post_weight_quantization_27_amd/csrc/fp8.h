// Shared by the e4m3 kernels (fp8_quant.hip, fp8_mm.hip).
#pragma once

#include "pwq_internal.h"
#include "pwq_common.h"

namespace pwq {

constexpr int F8_B = 128;                  // values of a token, rows and columns of weights per scale
constexpr float F8_TOP = 448.f;            // the largest e4m3 value
constexpr float F8_TINY = 0x1p-120f;       // float32 scales below this count as 0

}  // namespace pwq
