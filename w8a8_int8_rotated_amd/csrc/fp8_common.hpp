// Pieces shared by the FP8 kernels: operand types, the conversion of e4m3 codes and
// the quantisation of a block.
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

constexpr float kMaxE4M3 = 448.0f;

// The block's scale and the factor its values are multiplied with.  A scale
// below 2^-126 would have no finite reciprocal.  amax is never NaN (fmaxf
// drops NaNs); an infinite one gives an infinite scale and a zero factor, and
// codes of NaN for the infinities.
__device__ __forceinline__ void block_scale(float amax, bool pow2, float &s, float &inv)
{
    s = fmaxf(__fdiv_rn(amax, kMaxE4M3), 1.1754943508222875e-38f);
    if (pow2) {
        const uint32_t u = __float_as_uint(s);
        s = __uint_as_float((u & 0x7fffffu) ? (u & 0x7f800000u) + 0x800000u : u);
    }
    inv = __fdiv_rn(1.0f, s);
    if (!(amax > 0.0f)) s = inv = 0.0f;
}

// Four fp32 -> e4m3 codes (round to nearest even; |v| <= 448 up to the rounding
// of the factor, which the conversion rounds back to 448).
__device__ __forceinline__ int cvt_e4m3x4(float a, float b, float c, float d)
{
    int q = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return __builtin_amdgcn_cvt_pk_fp8_f32(c, d, q, true);
}

__device__ __forceinline__ float max8(const uint4 &u)
{
    const float a = fmaxf(fmaxf(fabsf(bf16_lo(u.x)), fabsf(bf16_hi(u.x))),
                          fmaxf(fabsf(bf16_lo(u.y)), fabsf(bf16_hi(u.y))));
    const float b = fmaxf(fmaxf(fabsf(bf16_lo(u.z)), fabsf(bf16_hi(u.z))),
                          fmaxf(fabsf(bf16_lo(u.w)), fabsf(bf16_hi(u.w))));
    return fmaxf(a, b);
}

// The e4m3 codes of 8 bf16 values times inv.
__device__ __forceinline__ int2 codes8(const uint4 &u, float inv)
{
    return make_int2(cvt_e4m3x4(__fmul_rn(bf16_lo(u.x), inv), __fmul_rn(bf16_hi(u.x), inv),
                                __fmul_rn(bf16_lo(u.y), inv), __fmul_rn(bf16_hi(u.y), inv)),
                     cvt_e4m3x4(__fmul_rn(bf16_lo(u.z), inv), __fmul_rn(bf16_hi(u.z), inv),
                                __fmul_rn(bf16_lo(u.w), inv), __fmul_rn(bf16_hi(u.w), inv)));
}

// Max over aligned groups of 16 lanes.
__device__ __forceinline__ float max16(float v)
{
#define CR_DPP_MAX(CTRL)                                                                          \
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true)))
    CR_DPP_MAX(0xB1);
    CR_DPP_MAX(0x4E);
    CR_DPP_MAX(0x141);
    CR_DPP_MAX(0x140);
#undef CR_DPP_MAX
    return v;
}

} // namespace
} // namespace convrot
