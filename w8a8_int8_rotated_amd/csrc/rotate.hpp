// The rotation of a row's blocks in registers and its INT8 codes, shared by the
// kernels that rotate and quantise (rotquant.hip, add_norm.hip).  rotquant.hip's
// first comment explains the lanes' layout, the sign tracking and the rounding.
#pragma once

#include "common.hpp"

namespace convrot {
namespace {

constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23

__device__ __forceinline__ int chunk_of_lane(int i)
{
    int c = 0;
    if (i & 1) c ^= 1;
    if (i & 2) c ^= 2;
    if (i & 4) c ^= 7;
    if (i & 8) c ^= 12;
    if (i & 16) c ^= 16;
    return c;
}

// One cross-lane butterfly stage on the 8 registers of a chunk.  The leading
// s_nop covers the VALU-write -> DPP-read hazard of whatever precedes.
#define CR_DPP_STAGE(CTRL, v, c)                                              \
    asm volatile("s_nop 1\n\t"                                                \
                 "v_fmac_f32_dpp %0, %0, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t" \
                 "v_fmac_f32_dpp %1, %1, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t" \
                 "v_fmac_f32_dpp %2, %2, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t" \
                 "v_fmac_f32_dpp %3, %3, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t" \
                 "v_fmac_f32_dpp %4, %4, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t" \
                 "v_fmac_f32_dpp %5, %5, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t" \
                 "v_fmac_f32_dpp %6, %6, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t" \
                 "v_fmac_f32_dpp %7, %7, %8 " CTRL " row_mask:0xf bank_mask:0xf"   \
                 : "+v"(v[0]), "+v"(v[1]), "+v"(v[2]), "+v"(v[3]),             \
                   "+v"(v[4]), "+v"(v[5]), "+v"(v[6]), "+v"(v[7])              \
                 : "v"(c))

template <int STAGE>
__device__ __forceinline__ void cross_stage(float (&v)[8], float c)
{
    if constexpr (STAGE == 0) {
        CR_DPP_STAGE("quad_perm:[1,0,3,2]", v, c);
    } else if constexpr (STAGE == 1) {
        CR_DPP_STAGE("quad_perm:[2,3,0,1]", v, c);
    } else if constexpr (STAGE == 2) {
        CR_DPP_STAGE("row_half_mirror", v, c);
    } else if constexpr (STAGE == 3) {
        CR_DPP_STAGE("row_mirror", v, c);
    } else {
        static_assert(STAGE == 4, "b <= 256");
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float p = __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(v[j]), 0x401F));
            v[j] = __builtin_fmaf(p, c, v[j]);
        }
    }
}

// Butterflies h = 1, 2, 4 inside one lane's chunk (ascending).
__device__ __forceinline__ void inlane_fwht8(float (&v)[8])
{
#pragma unroll
    for (int h = 1; h < 8; h *= 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if ((i & h) == 0) {
                float a = v[i], c = v[i + h];
                v[i] = __fadd_rn(a, c);
                v[i + h] = __fsub_rn(a, c);
            }
        }
    }
}

// d = s + (s of the lane holding the partner chunk of stage STAGE), for the
// regular rotation's pair sums.  fp32 addition is commutative, so both lanes
// of a pair get the same bits.
#define CR_DPP_ADD(CTRL, d, s)                                                \
    asm volatile("s_nop 1\n\t"                                                \
                 "v_add_f32_dpp %0, %8, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t" \
                 "v_add_f32_dpp %1, %9, %9 " CTRL " row_mask:0xf bank_mask:0xf\n\t" \
                 "v_add_f32_dpp %2, %10, %10 " CTRL " row_mask:0xf bank_mask:0xf\n\t" \
                 "v_add_f32_dpp %3, %11, %11 " CTRL " row_mask:0xf bank_mask:0xf\n\t" \
                 "v_add_f32_dpp %4, %12, %12 " CTRL " row_mask:0xf bank_mask:0xf\n\t" \
                 "v_add_f32_dpp %5, %13, %13 " CTRL " row_mask:0xf bank_mask:0xf\n\t" \
                 "v_add_f32_dpp %6, %14, %14 " CTRL " row_mask:0xf bank_mask:0xf\n\t" \
                 "v_add_f32_dpp %7, %15, %15 " CTRL " row_mask:0xf bank_mask:0xf"   \
                 : "=&v"(d[0]), "=&v"(d[1]), "=&v"(d[2]), "=&v"(d[3]),         \
                   "=&v"(d[4]), "=&v"(d[5]), "=&v"(d[6]), "=&v"(d[7])          \
                 : "v"(s[0]), "v"(s[1]), "v"(s[2]), "v"(s[3]),                 \
                   "v"(s[4]), "v"(s[5]), "v"(s[6]), "v"(s[7]))

template <int STAGE>
__device__ __forceinline__ void partner_add(float (&d)[8], const float (&s)[8])
{
    if constexpr (STAGE == 0) {
        CR_DPP_ADD("quad_perm:[1,0,3,2]", d, s);
    } else if constexpr (STAGE == 1) {
        CR_DPP_ADD("quad_perm:[2,3,0,1]", d, s);
    } else if constexpr (STAGE == 2) {
        CR_DPP_ADD("row_half_mirror", d, s);
    } else if constexpr (STAGE == 3) {
        CR_DPP_ADD("row_mirror", d, s);
    } else {
        static_assert(STAGE == 4, "b <= 256");
#pragma unroll
        for (int j = 0; j < 8; ++j)
            d[j] = __fadd_rn(s[j], __int_as_float(__builtin_amdgcn_ds_swizzle(
                                       __float_as_int(s[j]), 0x401F)));
    }
}

// The regular rotation of one chunk: H_4 = J - 2I along every base-4 digit
// of the in-block index, lowest digit first (the Rung-Omega README's
// H_256 = H_4 (x) H_4 (x) H_4 (x) H_4, and its order-64 counterpart).  A group
// (v0, v1, v2, v3) of one digit becomes S - 2 v_j with S = (v0 + v1) + (v2 +
// v3).  Digit 0 lies inside the lane; digit 1 pairs elements e, e + 4 of the
// lane and of the chunk across chunk bit 0; digit d >= 2 is chunk bits
// 2d - 3 and 2d - 2, whose partner lanes are the Sylvester stages' DPP
// patterns.  2 v_j is exact, so each output is one rounding of S - 2 v_j.
template <int B>
__device__ __forceinline__ void rotate_regular(float (&v)[8])
{
#pragma unroll
    for (int g = 0; g < 8; g += 4) {
        const float S = __fadd_rn(__fadd_rn(v[g], v[g + 1]), __fadd_rn(v[g + 2], v[g + 3]));
#pragma unroll
        for (int j = 0; j < 4; ++j) v[g + j] = __fsub_rn(S, 2.0f * v[g + j]);
    }
    {
        float p[8], S[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p[i] = __fadd_rn(v[i], v[i + 4]);
            p[i + 4] = p[i];
        }
        partner_add<0>(S, p);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __fsub_rn(S[j], 2.0f * v[j]);
    }
    {
        float a[8], S[8];
        partner_add<1>(a, v);
        partner_add<2>(S, a);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __fsub_rn(S[j], 2.0f * v[j]);
    }
    if constexpr (B == 256) {
        float a[8], S[8];
        partner_add<3>(a, v);
        partner_add<4>(S, a);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __fsub_rn(S[j], 2.0f * v[j]);
    }
}

// Rotation kinds: 0 = Sylvester blocks (butterflies with the sign trick),
// 1 = regular H_4 Kronecker blocks (B = 64 or 256).
template <int B, int ROT, int NSTAGE>
__device__ __forceinline__ void rotate_chunk(float (&v)[8], const float (&csign)[NSTAGE])
{
    if constexpr (ROT == 1) {
        static_assert(B == 64 || B == 256, "regular blocks are powers of 4");
        rotate_regular<B>(v);
    } else {
        inlane_fwht8(v);
        cross_stage<0>(v, csign[0]);
        cross_stage<1>(v, csign[1]);
        cross_stage<2>(v, csign[2]);
        if constexpr (NSTAGE > 3) cross_stage<3>(v, csign[3]);
        if constexpr (NSTAGE > 4) cross_stage<4>(v, csign[4]);
    }
}

// buffer resource word 3: raw (untyped) 32-bit data format, no swizzle
constexpr int kRsrcWord3 = 0x00020000;

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));

// One row as a buffer resource of `bytes` bytes: loads past the end read as
// zero and stores past the end are dropped, so a partial last step needs no
// per-lane branches.  A row beyond M gets an empty range.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_rsrc(const void *base, int bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, bytes,
                                             kRsrcWord3);
}

__device__ __forceinline__ uint32_t code_bits(float v, float inv)
{
    return __float_as_uint(__fadd_rn(__fmul_rn(v, inv), kMagic));
}

__device__ __forceinline__ uint2 quantise_chunk(const float (&v)[8], float inv)
{
    uint32_t c0 = code_bits(v[0], inv), c1 = code_bits(v[1], inv);
    uint32_t c2 = code_bits(v[2], inv), c3 = code_bits(v[3], inv);
    uint32_t c4 = code_bits(v[4], inv), c5 = code_bits(v[5], inv);
    uint32_t c6 = code_bits(v[6], inv), c7 = code_bits(v[7], inv);
    // v_perm_b32: pick the low byte of each code into one dword.
    uint32_t p01 = __builtin_amdgcn_perm(c1, c0, 0x0c0c0400u);
    uint32_t p23 = __builtin_amdgcn_perm(c3, c2, 0x0c0c0400u);
    uint32_t p45 = __builtin_amdgcn_perm(c5, c4, 0x0c0c0400u);
    uint32_t p67 = __builtin_amdgcn_perm(c7, c6, 0x0c0c0400u);
    uint2 r;
    r.x = __builtin_amdgcn_perm(p23, p01, 0x05040100u);
    r.y = __builtin_amdgcn_perm(p67, p45, 0x05040100u);
    return r;
}

} // namespace
} // namespace convrot
