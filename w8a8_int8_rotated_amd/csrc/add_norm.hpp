// Launches of the residual's addition with the RMS norm (add_norm.hip).  Arguments
// were validated by the API layer.
#pragma once

#include "common.hpp"

namespace convrot {

// h = x + r rounded to r's type (without r: h = x, not written);
// n = h rsqrt(mean h^2 + eps) w, out as rows y, as the INT8 codes of the rotated row
// or as e4m3 codes.  All matrices [M, K], dense.
struct AddNorm {
    const void *x, *r;             // r null: no addition
    const float *w;                // [K], null: ones
    void *h;                       // r's type; null without r
    void *y;                       // ROWS
    uint8_t *q;                    // ROTATED_I8, FP8: K-tiled codes and their scales
    float *s;
    int64_t M;
    int K;
    float eps;
    bool x_f32, r_f32, y_f32;      // r_f32 where x_f32
    int block;                     // ROTATED_I8
    bool regular;
    float inv_sqrt_b;
    bool pow2;                     // FP8
};
enum class NormOut { ROWS, ROTATED_I8, FP8 };
constexpr int64_t kMaxNormK = 32768;
hipError_t launch_add_norm(NormOut out, const AddNorm &a, hipStream_t stream);

// From g, the gradient of n, and gh, the one that reaches h otherwise (null: none):
// dh, its bf16 copy dx (or null) and dw (or null; then no partial sums).
struct AddNormGrad {
    const void *g, *h, *gh;        // gh of h's type
    const float *w;
    void *dh, *dx;
    float *dw, *partial;           // partial: add_norm_partial_rows(M, K) rows of K
    int64_t M;
    int K;
    float eps;
    bool g_f32, h_f32;
};
int64_t add_norm_partial_rows(int64_t M, int64_t K);
hipError_t launch_add_norm_grad(const AddNormGrad &a, hipStream_t stream);

} // namespace convrot
