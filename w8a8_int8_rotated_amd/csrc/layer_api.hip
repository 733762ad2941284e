// C ABI of the residual's addition with the RMS norm and of the mixture-of-experts layer:
// argument validation, workspace carving and launch sequencing.
#include "add_norm.hpp"
#include "api_common.hpp"
#include "moe.hpp"

namespace {

// Whether an output may stand where an input does: in its place, or apart from it.
bool overlaps(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && na > 0 && nb > 0 && x < y + nb && y < x + na;
}
bool in_place_or_apart(const void *a, size_t na, const void *b, size_t nb)
{
    return (a == b && na == nb) || !overlaps(a, na, b, nb);
}

// Whether everything a call writes is apart from all that it reads and from each other.
struct Extent {
    const void *p;
    size_t n;
};
template <int O, int I>
bool apart(const Extent (&out)[O], const Extent (&in)[I])
{
    for (int i = 0; i < O; ++i) {
        for (const Extent &e : in)
            if (overlaps(out[i].p, out[i].n, e.p, e.n)) return false;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i].p, out[i].n, out[j].p, out[j].n)) return false;
    }
    return true;
}

} // namespace

extern "C" {

// ---------------------------------------------------------------------------
// The residual's addition and the RMS norm.
// ---------------------------------------------------------------------------

static bool is_float_dtype(int t) { return t == CONVROT_F32 || t == CONVROT_BF16; }
static size_t dtype_bytes(int t) { return t == CONVROT_F32 ? 4u : 2u; }

// Rows and channels of a norm; every byte count formed from them fits 64 bits.
static int check_norm_shape(int64_t M, int64_t K, float eps)
{
    if (M < 0 || K <= 0) return CONVROT_EINVAL;
    if (M >= kI32Bound || K > convrot::kMaxNormK || K % 8 != 0) return CONVROT_EUNSUPPORTED;
    return check_eps(eps);
}

// The arguments the forward calls share, checked and gathered.  M > 0 or nothing but
// the shape is looked at.
static int add_norm_args(const void *x, int x_dtype, const void *residual, int res_dtype,
                         const float *w, float eps, int64_t M, int64_t K, void *residual_out,
                         convrot::AddNorm *a)
{
    int rc = check_norm_shape(M, K, eps);
    if (rc != CONVROT_OK) return rc;
    const bool add = residual != nullptr;
    if (add != (residual_out != nullptr)) return CONVROT_EINVAL;
    if (!is_float_dtype(x_dtype) || (add && !is_float_dtype(res_dtype)))
        return CONVROT_EUNSUPPORTED;
    if (add && x_dtype == CONVROT_F32 && res_dtype != CONVROT_F32) return CONVROT_EUNSUPPORTED;
    *a = {};
    a->x = x;
    a->r = residual;
    a->w = w;
    a->h = residual_out;
    a->M = M;
    a->K = (int)K;
    a->eps = eps;
    a->x_f32 = x_dtype == CONVROT_F32;
    a->r_f32 = add ? res_dtype == CONVROT_F32 : a->x_f32;
    if (M == 0) return CONVROT_OK;
    if (!x) return CONVROT_EINVAL;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(w) || !aligned16(residual_out))
        return CONVROT_EALIGN;
    const size_t n = (size_t)M * (size_t)K, nx = n * dtype_bytes(x_dtype);
    if (add) {
        const size_t nr = n * dtype_bytes(res_dtype);
        if (!in_place_or_apart(residual_out, nr, residual, nr) ||
            !in_place_or_apart(residual_out, nr, x, nx) ||
            overlaps(residual_out, nr, w, (size_t)K * 4u))
            return CONVROT_EINVAL;
    }
    return CONVROT_OK;
}

// An output of n bytes apart from the inputs and from residual_out.
static bool apart_from_norm(const convrot::AddNorm &a, const void *out, size_t n)
{
    const size_t e = (size_t)a.M * (size_t)a.K;
    const size_t nr = e * (a.r_f32 ? 4u : 2u);
    return !overlaps(out, n, a.x, e * (a.x_f32 ? 4u : 2u)) && !overlaps(out, n, a.r, nr) &&
           !overlaps(out, n, a.h, nr) && !overlaps(out, n, a.w, (size_t)a.K * 4u);
}

int convrot_add_rms_norm_forward(const void *x, int x_dtype, const void *residual, int res_dtype,
                                 const float *w, float eps, int64_t M, int64_t K,
                                 void *residual_out, void *y, int y_dtype, void *stream)
{
    convrot::AddNorm a;
    int rc = add_norm_args(x, x_dtype, residual, res_dtype, w, eps, M, K, residual_out, &a);
    if (rc != CONVROT_OK) return rc;
    if ((rc = check_out_dtype(y_dtype)) != CONVROT_OK) return rc;
    if (M == 0) return CONVROT_OK;
    if (!y) return CONVROT_EINVAL;
    if (!aligned16(y)) return CONVROT_EALIGN;
    const size_t n = (size_t)M * (size_t)K, ny = n * dtype_bytes(y_dtype);
    const size_t nr = n * (a.r_f32 ? 4u : 2u);
    if (!in_place_or_apart(y, ny, x, n * dtype_bytes(x_dtype)) ||
        !in_place_or_apart(y, ny, residual, nr) || overlaps(y, ny, residual_out, nr) ||
        overlaps(y, ny, w, (size_t)K * 4u))
        return CONVROT_EINVAL;
    a.y = y;
    a.y_f32 = y_dtype == CONVROT_F32;
    return hip_status(convrot::launch_add_norm(convrot::NormOut::ROWS, a,
                                               static_cast<hipStream_t>(stream)));
}

int convrot_add_rms_norm_rotate_quantize(const void *x, int x_dtype, const void *residual,
                                         int res_dtype, const float *w, float eps, int64_t M,
                                         int64_t K, int block, uint32_t flags,
                                         void *residual_out, int8_t *q, float *s, void *stream)
{
    convrot::AddNorm a;
    int rc = add_norm_args(x, x_dtype, residual, res_dtype, w, eps, M, K, residual_out, &a);
    if (rc != CONVROT_OK) return rc;
    if ((flags & ~CONVROT_ROT_REGULAR) != 0) return CONVROT_EUNSUPPORTED;
    if (!valid_block(block) || K % block != 0 || !valid_rotation(flags, block))
        return CONVROT_EINVAL;
    if (K % 128 != 0 || check_rows(M, K) != CONVROT_OK) return CONVROT_EUNSUPPORTED;
    if (M == 0) return CONVROT_OK;
    if (!q || !s) return CONVROT_EINVAL;
    if (!aligned16(q) || !aligned16(s)) return CONVROT_EALIGN;
    const size_t nq = codes_bytes(M, K), ns = (size_t)M * 4u;
    if (!apart_from_norm(a, q, nq) || !apart_from_norm(a, s, ns) || overlaps(q, nq, s, ns))
        return CONVROT_EINVAL;
    a.q = reinterpret_cast<uint8_t *>(q);
    a.s = s;
    a.block = block;
    a.regular = flags != 0;
    a.inv_sqrt_b = inv_sqrt_block(block);
    return hip_status(convrot::launch_add_norm(convrot::NormOut::ROTATED_I8, a,
                                               static_cast<hipStream_t>(stream)));
}

int convrot_add_rms_norm_fp8_quantize(const void *x, int x_dtype, const void *residual,
                                      int res_dtype, const float *w, float eps, int64_t M,
                                      int64_t K, int scales, void *residual_out, uint8_t *q,
                                      float *s, void *stream)
{
    convrot::AddNorm a;
    int rc = add_norm_args(x, x_dtype, residual, res_dtype, w, eps, M, K, residual_out, &a);
    if (rc != CONVROT_OK) return rc;
    if (!valid_fp8_scales(scales) || K % 128 != 0) return CONVROT_EINVAL;
    if (check_rows(M, K) != CONVROT_OK) return CONVROT_EUNSUPPORTED;
    if (M == 0) return CONVROT_OK;
    if (!q || !s) return CONVROT_EINVAL;
    if (!aligned16(q) || !aligned16(s)) return CONVROT_EALIGN;
    const size_t nq = codes_bytes(M, K), ns = fp8_row_scales_bytes(M, K);
    if (!apart_from_norm(a, q, nq) || !apart_from_norm(a, s, ns) || overlaps(q, nq, s, ns))
        return CONVROT_EINVAL;
    a.q = q;
    a.s = s;
    a.pow2 = scales == CONVROT_FP8_SCALE_POW2;
    return hip_status(convrot::launch_add_norm(convrot::NormOut::FP8, a,
                                               static_cast<hipStream_t>(stream)));
}

size_t convrot_fp8_norm_linear_workspace_bytes(int64_t M, int64_t K, int64_t N)
{
    if (check_linear_shape(N, K, 128) != CONVROT_OK || check_rows(M, K) != CONVROT_OK) return 0;
    return codes_bytes(M, K) + fp8_row_scales_bytes(M, K);
}

// What both paths check before anything is launched (W was checked): its outputs N, codes and
// scales.  Y may stand in the place of x or of the residual, which the first launch reads.
static int norm_linear_check(const convrot::AddNorm &a, int64_t N, const Extent &codes,
                             const Extent &scale, const float *bias, const void *Y, int y_dtype,
                             const void *ws, size_t ws_bytes, size_t need)
{
    int rc = check_rows(a.M, a.K);
    if (rc != CONVROT_OK) return rc;
    if ((rc = check_out_dtype(y_dtype)) != CONVROT_OK) return rc;
    if (a.M == 0) return CONVROT_OK;
    if (!Y) return CONVROT_EINVAL;
    if (!aligned16(Y) || !aligned16(bias) || !aligned16(ws)) return CONVROT_EALIGN;
    if (!ws || ws_bytes < need) return CONVROT_EWORKSPACE;
    const size_t e = (size_t)a.M * (size_t)a.K, nx = e * (a.x_f32 ? 4u : 2u),
                 nr = e * (a.r_f32 ? 4u : 2u),
                 ny = (size_t)a.M * (size_t)N * dtype_bytes(y_dtype);
    const Extent out[] = {{a.h, nr}, {Y, ny}, {ws, need}},
                 in[] = {{a.w, (size_t)a.K * 4u}, {bias, (size_t)N * 4u}, codes, scale};
    return apart(out, in) && in_place_or_apart(Y, ny, a.x, nx) && in_place_or_apart(Y, ny, a.r, nr) &&
                   !overlaps(ws, need, a.x, nx) && !overlaps(ws, need, a.r, nr)
               ? CONVROT_OK : CONVROT_EINVAL;
}

static int norm_linear_impl(const void *x, int x_dtype, const void *residual, int res_dtype,
                            const float *w, float eps, int64_t M, const convrot_weights *W,
                            const float *bias, void *residual_out, void *Y, int y_dtype, void *ws,
                            size_t ws_bytes, void *stream)
{
    int rc = check_weights(W);
    if (rc != CONVROT_OK) return rc;
    convrot::AddNorm a;
    rc = add_norm_args(x, x_dtype, residual, res_dtype, w, eps, M, W->K, residual_out, &a);
    if (rc == CONVROT_OK)
        rc = norm_linear_check(a, W->N,
                               {W->codes, convrot_weights_packed_bytes(W->N, W->K, W->block)},
                               {W->scale, (size_t)W->N * 4u}, bias, Y, y_dtype, ws, ws_bytes,
                               convrot_linear_workspace_bytes(M, W->K, W->N, W->block));
    if (rc != CONVROT_OK || M == 0) return rc;
    Carve c(ws);
    a.q = static_cast<uint8_t *>(c.take(codes_bytes(M, W->K)));
    a.s = static_cast<float *>(c.take((size_t)M * 4u));
    a.block = W->block;
    a.regular = is_regular(W);
    a.inv_sqrt_b = inv_sqrt_block(W->block);
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e = convrot::launch_add_norm(convrot::NormOut::ROTATED_I8, a, st);
    if (e == hipSuccess)
        e = product_i8(reinterpret_cast<const int8_t *>(a.q), a.s, M, W, bias, Y, y_dtype, st);
    return hip_status(e);
}

int convrot_norm_linear_forward(const void *x, int x_dtype, const void *residual, int res_dtype,
                                const float *w, float eps, int64_t M, const convrot_weights *W,
                                const float *bias, void *residual_out, void *Y, int y_dtype,
                                void *ws, size_t ws_bytes, void *stream)
{
    const int rc = norm_linear_impl(x, x_dtype, residual, res_dtype, w, eps, M, W, bias,
                                    residual_out, Y, y_dtype, ws, ws_bytes, stream);
    log_call("convrot_norm_linear_forward", M, W ? W->N : 0, W ? W->K : 0, rc);
    return rc;
}

static int fp8_norm_linear_impl(const void *x, int x_dtype, const void *residual, int res_dtype,
                                const float *w, float eps, int64_t M,
                                const convrot_fp8_weights *W, const float *bias,
                                void *residual_out, void *Y, int y_dtype, void *ws,
                                size_t ws_bytes, void *stream)
{
    int rc = check_fp8_weights(W);
    if (rc != CONVROT_OK) return rc;
    convrot::AddNorm a;
    rc = add_norm_args(x, x_dtype, residual, res_dtype, w, eps, M, W->K, residual_out, &a);
    if (rc == CONVROT_OK)
        rc = norm_linear_check(a, W->N, {W->codes, convrot_fp8_packed_bytes(W->N, W->K)},
                               {W->scale, convrot_fp8_scale_bytes(W->N, W->K)}, bias, Y, y_dtype,
                               ws, ws_bytes,
                               convrot_fp8_norm_linear_workspace_bytes(M, W->K, W->N));
    if (rc != CONVROT_OK || M == 0) return rc;
    Carve c(ws);
    a.q = static_cast<uint8_t *>(c.take(codes_bytes(M, W->K)));
    a.s = static_cast<float *>(c.take(fp8_row_scales_bytes(M, W->K)));
    a.pow2 = W->scales == CONVROT_FP8_SCALE_POW2;
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e = convrot::launch_add_norm(convrot::NormOut::FP8, a, st);
    if (e == hipSuccess) {
        const convrot::Fp8Gemm g = {nullptr, a.q, a.s, W->codes, W->scale, bias, Y, M, W->N, W->K,
                                    a.pow2, y_dtype == CONVROT_F32};
        e = convrot::launch_fp8_gemm(g, st);
    }
    return hip_status(e);
}

int convrot_fp8_norm_linear_forward(const void *x, int x_dtype, const void *residual,
                                    int res_dtype, const float *w, float eps, int64_t M,
                                    const convrot_fp8_weights *W, const float *bias,
                                    void *residual_out, void *Y, int y_dtype, void *ws,
                                    size_t ws_bytes, void *stream)
{
    const int rc = fp8_norm_linear_impl(x, x_dtype, residual, res_dtype, w, eps, M, W, bias,
                                        residual_out, Y, y_dtype, ws, ws_bytes, stream);
    log_call("convrot_fp8_norm_linear_forward", M, W ? W->N : 0, W ? W->K : 0, rc);
    return rc;
}

size_t convrot_add_rms_norm_workspace_bytes(int64_t M, int64_t K)
{
    if (check_norm_shape(M, K, 1.0f) != CONVROT_OK) return 0;
    return round_up((size_t)convrot::add_norm_partial_rows(M, K) * (size_t)K * 4u, kAlign);
}

int convrot_add_rms_norm_backward(const void *g, int g_dtype, const void *h, int h_dtype,
                                  const void *g_h, const float *w, float eps, int64_t M, int64_t K,
                                  void *dh, void *dx, float *dw, void *ws, size_t ws_bytes,
                                  void *stream)
{
    const int rc = check_norm_shape(M, K, eps);
    if (rc != CONVROT_OK) return rc;
    if (!is_float_dtype(g_dtype) || !is_float_dtype(h_dtype)) return CONVROT_EUNSUPPORTED;
    if (dx && h_dtype != CONVROT_F32) return CONVROT_EINVAL;
    if (M == 0 && !dw) return CONVROT_OK;
    if (M > 0 && (!g || !h || !dh)) return CONVROT_EINVAL;
    const void *const all[] = {g, h, g_h, w, dh, dx, dw, ws};
    for (const void *p : all)
        if (!aligned16(p)) return CONVROT_EALIGN;
    const size_t n = (size_t)M * (size_t)K, ng = n * dtype_bytes(g_dtype),
                 nh = n * dtype_bytes(h_dtype), nk = (size_t)K * 4u;
    const struct { const void *p; size_t n; } in[] = {{g, ng}, {h, nh}, {g_h, nh}};
    for (const auto &i : in)
        if (!in_place_or_apart(dh, nh, i.p, i.n) || !in_place_or_apart(dx, 2 * n, i.p, i.n) ||
            overlaps(dw, nk, i.p, i.n))
            return CONVROT_EINVAL;
    if (overlaps(dh, nh, dx, 2 * n) || overlaps(dh, nh, dw, nk) || overlaps(dx, 2 * n, dw, nk) ||
        overlaps(w, nk, dh, nh) || overlaps(w, nk, dx, 2 * n) || overlaps(w, nk, dw, nk))
        return CONVROT_EINVAL;
    const size_t need = dw ? convrot_add_rms_norm_workspace_bytes(M, K) : 0;
    if (need > 0 && (!ws || ws_bytes < need)) return CONVROT_EWORKSPACE;
    const Extent scratch[] = {{ws, need}},
                 rest[] = {{g, ng}, {h, nh}, {g_h, nh}, {w, nk}, {dh, nh}, {dx, 2 * n}, {dw, nk}};
    if (!apart(scratch, rest)) return CONVROT_EINVAL;
    const convrot::AddNormGrad a = {g, h, g_h, w, dh, dx, dw, static_cast<float *>(ws), M, (int)K,
                                    eps, g_dtype == CONVROT_F32, h_dtype == CONVROT_F32};
    return hip_status(convrot::launch_add_norm_grad(a, static_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------------------------
// The mixture-of-experts layer.
// ---------------------------------------------------------------------------

static bool moe_shape(int64_t n, int64_t R, int64_t C)
{
    return n >= 1 && n <= CONVROT_MOE_MAX_EXPERTS + CONVROT_MOE_MAX_SHARED && R > 0 && C > 0 &&
           R <= 2 * kMaxK && C <= kMaxK && R % 128 == 0 && C % 128 == 0 && R * C < kI32Bound;
}

size_t convrot_moe_packed_bytes(int64_t n, int64_t R, int64_t C)
{
    return moe_shape(n, R, C) ? (size_t)n * (size_t)R * (size_t)C : 0;
}

size_t convrot_moe_scale_bytes(int64_t n, int64_t R, int64_t C)
{
    return moe_shape(n, R, C) ? (size_t)n * (size_t)(R / 128) * (size_t)(C / 128) * 4u : 0;
}

// The caller's part of a descriptor.
static int check_moe_shape(const convrot_moe_weights *W)
{
    if (W->experts < 1 || W->shared < 0 || W->K <= 0 || W->F <= 0) return CONVROT_EINVAL;
    if (W->experts > CONVROT_MOE_MAX_EXPERTS || W->shared > CONVROT_MOE_MAX_SHARED ||
        W->K > kMaxK || W->F > kMaxK || W->K % 128 != 0 || W->F % 128 != 0 ||
        2 * W->F * W->K >= kI32Bound)
        return CONVROT_EUNSUPPORTED;
    if (!W->gate_up || !W->gate_up_scale || !W->down || !W->down_scale) return CONVROT_EINVAL;
    return aligned16(W->gate_up) && aligned16(W->gate_up_scale) && aligned16(W->down) &&
                   aligned16(W->down_scale) ? CONVROT_OK : CONVROT_EALIGN;
}

static int check_moe_weights(const convrot_moe_weights *W)
{
    if (!W) return CONVROT_EINVAL;
    if (W->magic != CONVROT_MOE_MAGIC || W->version != CONVROT_MOE_VERSION) return CONVROT_ELAYOUT;
    return check_moe_shape(W);
}

// n experts' [R, C] weights, one after another.
static hipError_t moe_pack(const void *W, int w_dtype, const float *src_scale, bool pow2, int64_t n,
                           int64_t R, int64_t C, uint8_t *codes, float *scale, hipStream_t s)
{
    const int64_t each = R * C, sc = (R / 128) * (C / 128);
    hipError_t e = hipSuccess;
    for (int64_t i = 0; i < n && e == hipSuccess; ++i) {
        if (w_dtype == CONVROT_F8E4M3)
            e = convrot::launch_tile_codes(static_cast<const int8_t *>(W) + i * each, false,
                                           reinterpret_cast<int8_t *>(codes + i * each), R, C, s);
        else
            e = convrot::launch_fp8_block_weights(
                static_cast<const char *>(W) + i * each * (int64_t)dtype_bytes(w_dtype),
                w_dtype == CONVROT_F32 ? convrot::InType::F32 : convrot::InType::BF16, R, C, pow2,
                codes + i * each, scale + i * sc, s);
    }
    if (e == hipSuccess && w_dtype == CONVROT_F8E4M3)
        e = hipMemcpyAsync(scale, src_scale, (size_t)(n * sc) * 4u, hipMemcpyDeviceToDevice, s);
    return e;
}

int convrot_moe_prepare_weights(const void *W_gate_up, const void *W_down, int w_dtype,
                                const float *src_scale_gate_up, const float *src_scale_down,
                                int scales, convrot_moe_weights *out, void *stream)
{
    if (!W_gate_up || !W_down || !out) return CONVROT_EINVAL;
    int rc = check_moe_shape(out);
    if (rc != CONVROT_OK) return rc;
    if (w_dtype != CONVROT_F32 && w_dtype != CONVROT_BF16 && w_dtype != CONVROT_F8E4M3)
        return CONVROT_EUNSUPPORTED;
    const bool import = w_dtype == CONVROT_F8E4M3;
    if (import != (src_scale_gate_up != nullptr) || import != (src_scale_down != nullptr) ||
        (!import && !valid_fp8_scales(scales)))
        return CONVROT_EINVAL;
    if (!aligned16(W_gate_up) || !aligned16(W_down) || !aligned16(src_scale_gate_up) ||
        !aligned16(src_scale_down))
        return CONVROT_EALIGN;
    const int64_t n = (int64_t)out->experts + out->shared;
    const bool pow2 = scales == CONVROT_FP8_SCALE_POW2;
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = moe_pack(W_gate_up, w_dtype, src_scale_gate_up, pow2, n, 2 * out->F, out->K,
                            out->gate_up, out->gate_up_scale, s);
    if (e == hipSuccess)
        e = moe_pack(W_down, w_dtype, src_scale_down, pow2, n, out->K, out->F, out->down,
                     out->down_scale, s);
    rc = hip_status(e);
    if (rc != CONVROT_OK) return rc;
    out->magic = CONVROT_MOE_MAGIC;
    out->version = CONVROT_MOE_VERSION;
    return CONVROT_OK;
}

static bool valid_top_k(const convrot_moe_weights *W, int top_k)
{
    return top_k >= 1 && top_k <= W->experts && top_k <= CONVROT_MOE_MAX_TOP_K;
}

size_t convrot_moe_workspace_bytes(int64_t T, const convrot_moe_weights *W, int top_k)
{
    if (T <= 0 || check_moe_weights(W) != CONVROT_OK || !valid_top_k(W, top_k)) return 0;
    return convrot::moe_workspace_bytes((int)(T < convrot::kMoeTokens ? T : convrot::kMoeTokens),
                                        W->experts, W->shared, top_k, (int)W->K, (int)W->F);
}

static int moe_forward_impl(const void *X, int64_t T, const void *router, int router_dtype,
                            const float *router_bias, const convrot_moe_weights *W, int top_k,
                            int score, uint32_t flags, float scale, void *Y, int y_dtype,
                            int32_t *ids, float *weights, void *ws, size_t ws_bytes, void *stream)
{
    int rc = check_moe_weights(W);
    if (rc != CONVROT_OK) return rc;
    if (T < 0) return CONVROT_EINVAL;
    if (T >= kI32Bound || !is_float_dtype(router_dtype) || !is_float_dtype(y_dtype) ||
        (flags & ~CONVROT_MOE_RENORMALIZE) != 0)
        return CONVROT_EUNSUPPORTED;
    if (!valid_top_k(W, top_k) || !std::isfinite(scale) ||
        (score != CONVROT_MOE_SCORE_SOFTMAX && score != CONVROT_MOE_SCORE_SIGMOID))
        return CONVROT_EINVAL;
    if (T == 0) return CONVROT_OK;
    if (!X || !router || !Y || !ids || !weights) return CONVROT_EINVAL;
    const void *const all[] = {X, router, router_bias, Y, ids, weights, ws};
    for (const void *p : all)
        if (!aligned16(p)) return CONVROT_EALIGN;
    const size_t n = (size_t)T * (size_t)W->K, nk = (size_t)T * (size_t)top_k * 4u;
    const size_t need = convrot_moe_workspace_bytes(T, W, top_k);
    const int64_t experts = (int64_t)W->experts + W->shared;
    const Extent out[] = {{Y, n * dtype_bytes(y_dtype)}, {ids, nk}, {weights, nk}, {ws, need}},
                 in[] = {{X, n * 2u},
                         {router, (size_t)W->experts * (size_t)W->K * dtype_bytes(router_dtype)},
                         {router_bias, (size_t)W->experts * 4u},
                         {W->gate_up, convrot_moe_packed_bytes(experts, 2 * W->F, W->K)},
                         {W->gate_up_scale, convrot_moe_scale_bytes(experts, 2 * W->F, W->K)},
                         {W->down, convrot_moe_packed_bytes(experts, W->K, W->F)},
                         {W->down_scale, convrot_moe_scale_bytes(experts, W->K, W->F)}};
    if (!apart(out, in)) return CONVROT_EINVAL;
    if (!ws || ws_bytes < need) return CONVROT_EWORKSPACE;

    convrot::Moe m = {};
    m.router = router;
    m.bias = router_bias;
    m.gate_up = W->gate_up;
    m.down = W->down;
    m.gate_up_scale = W->gate_up_scale;
    m.down_scale = W->down_scale;
    m.E = W->experts;
    m.S = W->shared;
    m.top_k = top_k;
    m.K = (int)W->K;
    m.F = (int)W->F;
    m.router_f32 = router_dtype == CONVROT_F32;
    m.sigmoid = score == CONVROT_MOE_SCORE_SIGMOID;
    m.renormalize = (flags & CONVROT_MOE_RENORMALIZE) != 0;
    m.y_f32 = y_dtype == CONVROT_F32;
    m.factor = (double)scale;
    m.ws = ws;
    hipError_t e = hipSuccess;
    for (int64_t t = 0; t < T && e == hipSuccess; t += convrot::kMoeTokens) {
        m.T = (int)(T - t < convrot::kMoeTokens ? T - t : convrot::kMoeTokens);
        m.x = static_cast<const uint16_t *>(X) + t * W->K;
        m.y = static_cast<char *>(Y) + t * W->K * (int64_t)dtype_bytes(y_dtype);
        m.ids = ids + t * top_k;
        m.weights = weights + t * top_k;
        e = convrot::launch_moe(m, static_cast<hipStream_t>(stream));
    }
    return hip_status(e);
}

int convrot_moe_forward(const void *X, int64_t T, const void *router, int router_dtype,
                        const float *router_bias, const convrot_moe_weights *W, int top_k,
                        int score, uint32_t flags, float scale, void *Y, int y_dtype, int32_t *ids,
                        float *weights, void *ws, size_t ws_bytes, void *stream)
{
    const int rc = moe_forward_impl(X, T, router, router_dtype, router_bias, W, top_k, score,
                                    flags, scale, Y, y_dtype, ids, weights, ws, ws_bytes, stream);
    log_call("convrot_moe_forward", T, W ? W->F : 0, W ? W->K : 0, rc);
    return rc;
}

} // extern "C"
