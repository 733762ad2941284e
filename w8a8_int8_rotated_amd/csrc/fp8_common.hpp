// Pieces shared by the FP8 kernels (fp8.hip, gemm_fp8.hip): operand types and the
// conversion of e4m3 codes.
#pragma once

#include "common.hpp"

namespace convrot {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// 8 e4m3 codes as bf16, exactly.
__device__ __forceinline__ v8bf bf16_of_codes(int lo, int hi)
{
    const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return (v8bf){a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

} // namespace
} // namespace convrot
