// What the files of the C ABI share: checks of shapes, descriptors and pointers, workspace
// carving, and the calls that convrot_api.hip defines for all of them.
#pragma once

#include "convrot.h"
#include "common.hpp"

#include <cmath>
#include <cstdint>

namespace convrot {

// A HIP error kept for convrot_last_hip_error, as a status.
int hip_status(hipError_t e);
// With CONVROT_LOG=1 the main entry points also print their name, shape and status to stderr.
void log_call(const char *name, int64_t M, int64_t N, int64_t K, int rc);
// A product of codes with the plain epilogue.
hipError_t product_i8(const int8_t *qx, const float *sx, int64_t M, const convrot_weights *W,
                      const float *bias, void *Y, int y_dtype, hipStream_t s);

} // namespace convrot

namespace {

using convrot::hip_status;
using convrot::log_call;
using convrot::product_i8;

constexpr int64_t kMaxK = 65536;
constexpr int64_t kI32Bound = (int64_t)1 << 31;
constexpr size_t kAlign = 256;

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool valid_block(int b) { return b == 64 || b == 128 || b == 256; }

// Rotation kinds (convrot_weights.flags, convrot_rotate_quantize flags): the
// Sylvester blocks, or CONVROT_ROT_REGULAR, the H_4 Kronecker blocks, which
// exist for b = 64 and 256 only.
bool valid_rotation(uint32_t rot, int b)
{
    if (rot == 0) return true;
    return rot == CONVROT_ROT_REGULAR && (b == 64 || b == 256);
}

bool is_regular(const convrot_weights *W) { return (W->flags & CONVROT_ROT_REGULAR) != 0; }
uint32_t rotation_of(const convrot_weights *W) { return (uint32_t)W->flags & CONVROT_ROT_REGULAR; }
bool is_swiglu_pairs(const convrot_weights *W)
{
    return ((uint32_t)W->flags & CONVROT_SWIGLU_PAIRS) != 0;
}

// fp32 1/sqrt(b), rounded once from double.
float inv_sqrt_block(int b) { return (float)(1.0 / std::sqrt((double)b)); }

// Shape rules shared by every projection (K inputs, N outputs, block b).
int check_linear_shape(int64_t N, int64_t K, int block)
{
    if (N <= 0 || K <= 0 || !valid_block(block) || K % block != 0) return CONVROT_EINVAL;
    // N is bounded before the product, so it cannot overflow
    if (K % 128 != 0 || N % 16 != 0 || K > kMaxK || N >= kI32Bound || N * K >= kI32Bound)
        return CONVROT_EUNSUPPORTED;
    return CONVROT_OK;
}

// A prepared descriptor.  `pairs`: whether the weight must (true) or must not
// (false) hold interleaved SwiGLU gate/up rows; a mismatch is ELAYOUT, since
// the outputs of such a weight are not the columns of a plain linear.
int check_weights(const convrot_weights *W, bool pairs = false)
{
    if (!W) return CONVROT_EINVAL;
    if (W->magic != CONVROT_WEIGHTS_MAGIC || W->version != CONVROT_WEIGHTS_VERSION)
        return CONVROT_ELAYOUT;
    if (!W->codes || !W->scale) return CONVROT_EINVAL;
    if (!aligned16(W->codes) || !aligned16(W->scale)) return CONVROT_EALIGN;
    int rc = check_linear_shape(W->N, W->K, W->block);
    const uint32_t extra = (uint32_t)W->flags & ~(CONVROT_ROT_REGULAR | CONVROT_SWIGLU_PAIRS);
    if (rc == CONVROT_OK &&
        (extra != 0 || !valid_rotation(rotation_of(W), W->block) || is_swiglu_pairs(W) != pairs ||
         (pairs && W->N % 32 != 0)))
        return CONVROT_ELAYOUT;
    return rc == CONVROT_EINVAL ? CONVROT_ELAYOUT : rc;
}

// M rows of K: the K-tiled codes hold padded_rows(M) rows, and every byte
// offset the kernels form must fit in 32 bits.
int check_rows(int64_t M, int64_t K)
{
    if (M < 0) return CONVROT_EINVAL;
    // K <= 65536 here; M is bounded before padding and product
    if (M >= kI32Bound || convrot::padded_rows(M) * K >= kI32Bound) return CONVROT_EUNSUPPORTED;
    return CONVROT_OK;
}

int check_out_dtype(int y_dtype)
{
    return (y_dtype == CONVROT_BF16 || y_dtype == CONVROT_F32) ? CONVROT_OK : CONVROT_EUNSUPPORTED;
}

convrot::OutKind out_kind(int y_dtype)
{
    return y_dtype == CONVROT_F32 ? convrot::OutKind::F32 : convrot::OutKind::BF16;
}

// Bump allocator over a caller workspace.
struct Carve {
    char *base;
    size_t used = 0;
    explicit Carve(void *p) : base(static_cast<char *>(p)) {}
    void *take(size_t bytes)
    {
        void *p = base ? base + used : nullptr;
        used += round_up(bytes, kAlign);
        return p;
    }
};

size_t codes_bytes(int64_t M, int64_t K)
{
    return round_up((size_t)convrot::padded_rows(M) * (size_t)K, kAlign);
}
size_t scales_bytes(int64_t M) { return round_up((size_t)M * 4u, kAlign); }

// activation scales [K / 128, Mp]
size_t fp8_row_scales_bytes(int64_t M, int64_t K)
{
    return round_up((size_t)convrot::padded_rows(M) * (size_t)(K / 128) * 4u, kAlign);
}

bool valid_fp8_scales(int kind)
{
    return kind == CONVROT_FP8_SCALE_F32 || kind == CONVROT_FP8_SCALE_POW2;
}

int check_fp8_weights(const convrot_fp8_weights *W)
{
    if (!W) return CONVROT_EINVAL;
    if (W->magic != CONVROT_FP8_MAGIC || W->version != CONVROT_FP8_VERSION ||
        !valid_fp8_scales(W->scales) || W->reserved != 0)
        return CONVROT_ELAYOUT;
    if (!W->codes || !W->scale) return CONVROT_EINVAL;
    if (!aligned16(W->codes) || !aligned16(W->scale)) return CONVROT_EALIGN;
    const int rc = check_linear_shape(W->N, W->K, 128);
    return rc == CONVROT_EINVAL ? CONVROT_ELAYOUT : rc;
}

int check_eps(float eps) { return eps > 0.0f && std::isfinite(eps) ? CONVROT_OK : CONVROT_EINVAL; }

} // namespace
