/* Drives the host code of the residual addition with the RMS norm and of the mixture of
 * experts under AddressSanitizer and UndefinedBehaviorSanitizer: every sizing query and
 * every validating path over a grid of extents up to INT64_MAX, with calls that must
 * return before anything is launched. */
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "convrot.h"

static int failed = 0, checks = 0;
#define CHECK(x)                                                                     \
    do {                                                                             \
        ++checks;                                                                    \
        if (!(x)) {                                                                  \
            ++failed;                                                                \
            printf("line %d: %s\n", __LINE__, #x);                                   \
        }                                                                            \
    } while (0)

static const int64_t EXT[] = {INT64_MIN, -1, 0, 1, 7, 16, 127, 128, 1000, 38656, 65536, 65664,
                              (int64_t)1 << 20, ((int64_t)1 << 31) - 16, (int64_t)1 << 31,
                              (int64_t)1 << 32, (int64_t)1 << 62, INT64_MAX};
#define NEXT ((int)(sizeof EXT / sizeof *EXT))
/* addresses: aligned and far apart, and one that is not aligned */
static void *at(int i) { return (void *)((uintptr_t)(i + 1) << 56); }
static void *const BAD = (void *)0x1002;

int main(void)
{
    convrot_weights w;
    memset(&w, 0, sizeof w);
    w.magic = CONVROT_WEIGHTS_MAGIC;
    w.version = CONVROT_WEIGHTS_VERSION;
    w.N = 1536, w.K = 512, w.block = 128, w.codes = at(9), w.scale = at(10);
    convrot_fp8_weights f = {CONVROT_FP8_MAGIC, CONVROT_FP8_VERSION, 1536, 512, 0, 0, at(9), at(10)};
    convrot_moe_weights e = {CONVROT_MOE_MAGIC, CONVROT_MOE_VERSION, 8, 1, 512, 256,
                             at(9), at(10), at(11), at(12)};

    for (int i = 0; i < NEXT; ++i)
        for (int j = 0; j < NEXT; ++j) {
            const int64_t a = EXT[i], b = EXT[j];
            const size_t need = convrot_add_rms_norm_workspace_bytes(a, b);
            CHECK(need == 0 || (a > 0 && b > 0));
            /* a pointer that is not aligned: refused, or nothing to do */
            int rc = convrot_add_rms_norm_forward(BAD, CONVROT_BF16, at(1), CONVROT_F32, at(2), 1e-6f,
                                                  a, b, at(3), at(4), CONVROT_BF16, NULL);
            CHECK(rc != CONVROT_OK || a == 0);
            rc = convrot_add_rms_norm_rotate_quantize(BAD, CONVROT_BF16, NULL, 0, NULL, 1e-6f, a, b,
                                                      128, 0, NULL, at(3), at(4), NULL);
            CHECK(rc != CONVROT_OK || a == 0);
            rc = convrot_add_rms_norm_rotate_quantize(at(0), CONVROT_BF16, at(1), CONVROT_BF16, NULL,
                                                      1e-6f, a, b, 64, CONVROT_ROT_REGULAR, at(2),
                                                      at(3), BAD, NULL);
            CHECK(rc != CONVROT_OK || a == 0);
            rc = convrot_add_rms_norm_fp8_quantize(at(0), CONVROT_F32, at(1), CONVROT_F32, NULL,
                                                   1e-6f, a, b, CONVROT_FP8_SCALE_POW2, at(2), BAD,
                                                   at(4), NULL);
            CHECK(rc != CONVROT_OK || a == 0);
            rc = convrot_add_rms_norm_forward(at(0), CONVROT_F32, at(1), CONVROT_F32, at(2), 1e-6f,
                                              a, b, at(1), at(1), CONVROT_F32, NULL);
            CHECK(rc != CONVROT_OK || a == 0);
            rc = convrot_add_rms_norm_backward(at(0), CONVROT_BF16, at(1), CONVROT_F32, at(2), at(3),
                                               1e-6f, a, b, at(4), at(5), at(6), BAD, SIZE_MAX, NULL);
            CHECK(rc != CONVROT_OK);
            rc = convrot_add_rms_norm_backward(at(0), CONVROT_BF16, at(1), CONVROT_F32, at(2), at(3),
                                               1e-6f, a, b, at(4), at(5), at(6), at(7),
                                               need ? need - 1 : 0, NULL);
            CHECK(rc != CONVROT_OK);
            /* a descriptor of any shape, rows that are not aligned */
            convrot_weights v = w;
            v.N = a, v.K = b;
            CHECK(convrot_norm_linear_forward(BAD, CONVROT_BF16, NULL, 0, NULL, 1e-6f, 40, &v, NULL,
                                              NULL, at(3), CONVROT_BF16, at(4), SIZE_MAX,
                                              NULL) != CONVROT_OK);
            convrot_fp8_weights d = f;
            d.N = a, d.K = b;
            CHECK(convrot_fp8_norm_linear_forward(at(0), CONVROT_BF16, at(1), CONVROT_F32, NULL,
                                                  1e-6f, 40, &d, BAD, at(2), at(3), CONVROT_F32,
                                                  at(4), SIZE_MAX, NULL) != CONVROT_OK);
            CHECK(convrot_norm_linear_forward(at(0), CONVROT_BF16, at(1), CONVROT_F32, NULL, 1e-6f,
                                              a, &w, NULL, at(2), BAD, CONVROT_BF16, at(4),
                                              SIZE_MAX, NULL) != CONVROT_OK || a == 0);
            for (int k = 0; k < NEXT; ++k)
                (void)convrot_fp8_norm_linear_workspace_bytes(EXT[k], a, b);
            /* experts */
            for (int n = -1; n < 600; n += 97) {
                const size_t p = convrot_moe_packed_bytes(n, a, b);
                CHECK(p == 0 || (n > 0 && a > 0 && b > 0 && p < ((size_t)1 << 41)));
                CHECK((convrot_moe_scale_bytes(n, a, b) == 0) == (p == 0));
            }
            (void)convrot_moe_packed_bytes(a, b, 128);
            (void)convrot_moe_scale_bytes(a, 128, b);
            convrot_moe_weights m = e;
            m.K = a, m.F = b;
            (void)convrot_moe_workspace_bytes(64, &m, 8);
            (void)convrot_moe_workspace_bytes(INT64_MAX, &m, 8);
            CHECK(convrot_moe_workspace_bytes(a, &e, (int)b) == 0 ||
                  (a > 0 && (int)b >= 1 && (int)b <= 8));
            CHECK(convrot_moe_forward(at(0), 5, at(1), CONVROT_F32, NULL, &m, 2, 0, 0, 1.0f, BAD,
                                      CONVROT_F32, at(3), at(4), at(5), SIZE_MAX,
                                      NULL) != CONVROT_OK);
            rc = convrot_moe_forward(at(0), a, at(1), CONVROT_BF16, at(2), &e, 2, 1, 1, 2.5f, at(3),
                                     CONVROT_BF16, BAD, at(5), at(6), SIZE_MAX, NULL);
            CHECK(rc != CONVROT_OK || a == 0);
            m.magic = 0;
            m.down = NULL;
            CHECK(convrot_moe_prepare_weights(at(0), at(1), CONVROT_BF16, NULL, NULL, 0, &m,
                                              NULL) != CONVROT_OK);
            CHECK(m.magic == 0);
        }
    const size_t ws = convrot_moe_workspace_bytes(7, &e, 2);
    CHECK(ws > 0 && convrot_moe_workspace_bytes(64, &e, 2) == convrot_moe_workspace_bytes(65, &e, 2));
    CHECK(convrot_moe_forward(at(0), 7, at(1), CONVROT_F32, NULL, &e, 2, 0, 0, 1.0f, at(2), CONVROT_F32,
                              at(3), at(4), at(5), ws - 1, NULL) == CONVROT_EWORKSPACE);
    printf("%d checks, %d failed checks\n", checks, failed);
    return failed != 0;
}
