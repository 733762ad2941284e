// The INT8 product of up to kFewRows rows (gemm_i8_few.hip), with the results of
// launch_gemm_i8 for OutKind::BF16 and F32.
#pragma once

#include "common.hpp"

namespace convrot {

constexpr int64_t kFewRows = 16;
hipError_t launch_gemm_i8_few(const int8_t *qx, const int8_t *qw, const float *sx,
                              const float *sw, const float *bias, void *Y, bool f32, int64_t M,
                              int64_t N, int64_t K, hipStream_t stream);

} // namespace convrot
