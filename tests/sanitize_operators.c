/* Drives the host code of the FP8 linear, the rotary positions, the Q/K norms
 * and the QKV entries under AddressSanitizer and UndefinedBehaviorSanitizer:
 * every sizing query and every validating path over a grid of extents up to
 * INT64_MAX, with calls that must return before anything is launched. */
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
static void *const P = (void *)0x1000;
static void *const BAD = (void *)0x1002;

int main(void)
{
    convrot_fp8_weights f = {CONVROT_FP8_MAGIC, CONVROT_FP8_VERSION, 1536, 512, 0, 0, P, P};
    convrot_weights w;
    memset(&w, 0, sizeof w);
    w.magic = CONVROT_WEIGHTS_MAGIC;
    w.version = CONVROT_WEIGHTS_VERSION;
    w.N = 1536, w.K = 512, w.block = 128, w.codes = P, w.scale = P;
    convrot_rope r = {CONVROT_ROPE_MAGIC, CONVROT_ROPE_VERSION, 3, 128, 128, 0, P, P};

    for (int i = 0; i < NEXT; ++i)
        for (int j = 0; j < NEXT; ++j) {
            const int64_t a = EXT[i], b = EXT[j];
            const size_t bytes = convrot_fp8_packed_bytes(a, b);
            CHECK(bytes == 0 || (a > 0 && b > 0 && bytes < ((size_t)1 << 31)));
            CHECK((convrot_fp8_scale_bytes(a, b) == 0) == (bytes == 0));
            for (int k = 0; k < NEXT; ++k) (void)convrot_fp8_linear_workspace_bytes(EXT[k], a, b);
            (void)convrot_fp8_prepare_workspace_bytes(a, b, CONVROT_F32, CONVROT_IN_MAJOR);
            /* no codes: refused whatever the shape */
            convrot_fp8_weights o = {0, 0, 0, 0, 0, 0, NULL, P};
            CHECK(convrot_fp8_prepare_weights(P, CONVROT_F32, 0, NULL, a, b, &o, P, SIZE_MAX,
                                              NULL) == CONVROT_EINVAL);
            /* a shape whose pointers are bad: refused, or nothing to do */
            int rc = convrot_fp8_quantize(BAD, a, b, 0, P, P, NULL);
            CHECK(rc != CONVROT_OK || a == 0);
            convrot_fp8_weights d = f;
            d.N = a, d.K = b;
            rc = convrot_fp8_linear_forward(BAD, 40, &d, NULL, P, CONVROT_BF16, P, SIZE_MAX, NULL);
            CHECK(rc != CONVROT_OK);
            rc = convrot_fp8_linear_forward(BAD, a, &f, NULL, P, CONVROT_F32, P, SIZE_MAX, NULL);
            CHECK(rc != CONVROT_OK || a == 0);
            rc = convrot_fp8_gemm_dequant(BAD, P, a, &f, NULL, P, CONVROT_F32, NULL);
            CHECK(rc != CONVROT_OK || a == 0);

            /* batch a, tokens b: queries whose data is missing or misaligned */
            const int none = a == 0 || b == 0;
            for (int s = 0; s < NEXT; ++s) {
                convrot_heads x = {BAD, 4, 0, EXT[s], EXT[s], EXT[s]}, y = {P, 4, 0, 512, 512, 128};
                CHECK(convrot_rope_forward(a, b, CONVROT_BF16, &x, &y, NULL, NULL, &r, P,
                                           CONVROT_I32, 0, 0, NULL) != CONVROT_OK);
                CHECK(convrot_qk_norm_rope_forward(a, b, CONVROT_F32, &x, &y, NULL, NULL, NULL,
                                                   NULL, 1e-6f, &r, P, CONVROT_F32,
                                                   EXT[s] < 0 ? 0 : EXT[s], NULL) != CONVROT_OK);
                CHECK(convrot_qk_norm_rope_backward(a, b, CONVROT_F32, &y, &x, &y, NULL, P, NULL,
                                                    NULL, NULL, NULL, NULL, 1e-6f, &r, P,
                                                    CONVROT_F32, 0, P, SIZE_MAX, NULL) !=
                      CONVROT_OK);
            }
            for (int h = -1; h < 70000; h += 23333)
                for (int d8 = -8; d8 <= 520; d8 += 132)
                    (void)convrot_qk_norm_rope_workspace_bytes(a, b, h, 1, d8);
            /* the QKV entries: misaligned outputs */
            rc = convrot_qkv_forward(P, a, b, &w, NULL, 8, 2, NULL, NULL, 1e-6f, &r, P,
                                     CONVROT_I32, 0, BAD, CONVROT_BF16, P, SIZE_MAX, NULL);
            CHECK(rc != CONVROT_OK || none);
            rc = convrot_fp8_qkv_forward(P, a, b, &f, NULL, 8, 2, NULL, NULL, 1e-6f, &r, P,
                                         CONVROT_I32, 0, BAD, CONVROT_F32, P, SIZE_MAX, NULL);
            CHECK(rc != CONVROT_OK || none);
        }
    /* head counts whose products leave 32 bits */
    CHECK(convrot_qkv_forward(P, 1, 4, &w, NULL, INT32_MAX, INT32_MAX, NULL, NULL, 1e-6f, &r, P,
                              CONVROT_I32, 0, P, CONVROT_BF16, P, SIZE_MAX,
                              NULL) == CONVROT_ELAYOUT);
    const int32_t huge[4] = {INT32_MAX - 1, INT32_MAX - 1, INT32_MAX - 1, INT32_MAX - 1};
    convrot_rope o = {0, 0, 0, 0, 0, 0, P, P};
    for (int axes = -1; axes <= 5; ++axes)
        CHECK(convrot_rope_prepare(huge, axes, INT32_MAX, 1e4, 0, 0, &o, NULL) != CONVROT_OK);
    printf("%d checks, %d failed checks\n", checks, failed);
    return failed != 0;
}
