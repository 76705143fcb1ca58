/* Host-side checks of the norm's, the adapters' and the clipping's argument
 * validation and size queries, built with AddressSanitizer and
 * UndefinedBehaviorSanitizer (host code only) by tests/test_sanitize_ops_cpu.py.
 * Every call here is rejected, or is a pure size query, before any HIP call;
 * the pointers are fake addresses the library never dereferences, but for the
 * host arrays of bfly_grad_clip, which are real and of the exact length. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "bfly.h"

static int failures = 0;
#define EXPECT(cond)                                                         \
    do {                                                                     \
        if (!(cond)) {                                                       \
            fprintf(stderr, "%s:%d: expected %s\n", __FILE__, __LINE__, #cond); \
            ++failures;                                                      \
        }                                                                    \
    } while (0)

#define P(a) ((void*)(uintptr_t)(a))
#define F(a) ((float*)(uintptr_t)(a))

static const int64_t rows[] = {INT64_MAX, INT64_MIN, -1, (int64_t)1 << 62, ((int64_t)1 << 46) + 1};
static const int32_t sizes[] = {INT32_MIN, -1, 0, 7, 16385, 1 << 30, INT32_MAX};

int main(void)
{
    const size_t big = SIZE_MAX;
    for (size_t i = 0; i < sizeof(rows) / sizeof(rows[0]); ++i) {
        EXPECT(bfly_rmsnorm_backward_workspace_bytes(rows[i], 4096) == 0);
        EXPECT(bfly_lora_matmul_workspace_bytes(rows[i], 256, 512, 16) == 0);
        EXPECT(bfly_rmsnorm(P(0x10000), BFLY_BF16, NULL, NULL, NULL, BFLY_F32, P(0x20000), BFLY_F32,
                            NULL, NULL, NULL, rows[i], 4096, 1e-5f, BFLY_Q8_INT8, 4096, NULL) !=
               BFLY_OK);
        EXPECT(bfly_rmsnorm_backward(P(0x10000), BFLY_BF16, NULL, BFLY_F32, F(0x20000), P(0x30000),
                                     NULL, P(0x40000), BFLY_BF16, F(0x50000), rows[i], 4096,
                                     P(0x60000), big, NULL) != BFLY_OK);
        EXPECT(bfly_lora_matmul(P(0x10000), BFLY_BF16, P(0x20000), P(0x30000), P(0x40000),
                                F(0x50000), NULL, BFLY_F32, P(0x60000), BFLY_F32, rows[i], 256, 512,
                                4, 16, P(0x70000), big, NULL) != BFLY_OK);
    }
    for (size_t i = 0; i < sizeof(sizes) / sizeof(sizes[0]); ++i) {
        const int32_t v = sizes[i];
        EXPECT(bfly_lora_matmul_workspace_bytes(4, 256, 512, v) == 0);
        EXPECT(bfly_lora_matmul_workspace_bytes(4, 256, v, 16) == 0 || v == (1 << 30));
        EXPECT(bfly_rmsnorm(P(0x10000), BFLY_BF16, NULL, NULL, NULL, BFLY_F32, P(0x20000), BFLY_F32,
                            P(0x30000), P(0x40000), NULL, 4, 4096, 1e-5f, BFLY_Q8_INT8, v, NULL) ==
               BFLY_ERR_QUANT);
        EXPECT(bfly_rmsnorm(P(0x10000), (bfly_dtype)(v | 2), NULL, NULL, NULL, BFLY_F32, P(0x20000),
                            BFLY_F32, NULL, NULL, NULL, 4, 4096, 1e-5f, BFLY_Q8_INT8, 64, NULL) ==
               BFLY_ERR_DTYPE);
        EXPECT(bfly_rmsnorm(P(0x10000), BFLY_F32, NULL, NULL, NULL, BFLY_F32, NULL, BFLY_F32,
                            P(0x30000), P(0x40000), NULL, 4, 4096, 1e-5f, (bfly_q8)(v | 2), 64,
                            NULL) == BFLY_ERR_QUANT);
        EXPECT(bfly_lora_matmul(P(0x10000), BFLY_BF16, P(0x20000), P(0x30000), P(0x40000),
                                F(0x50000), NULL, BFLY_F32, P(0x60000), BFLY_F32, 4, 256, 512, 4, v,
                                P(0x70000), big, NULL) != BFLY_OK);
        if (v < 1)
            EXPECT(bfly_grad_clip(v < 0 ? v : -1, NULL, NULL, NULL, NULL, 1.f, F(0x10000),
                                  P(0x20000), big, NULL) == BFLY_ERR_SIZE);
    }
    /* sizes that grow with the rows */
    size_t last = 0;
    for (int64_t r = 1; r <= ((int64_t)1 << 23); r *= 2) {
        const size_t now = bfly_lora_matmul_workspace_bytes(r, 4096, 4096, 64);
        EXPECT(now > 0);
        if (r >= 16384) {
            EXPECT(now >= last);
            last = now;
        }
    }
    /* host arrays of exactly `count` entries; the last one is what is refused */
    enum { N = 1000 };
    const void** grads = malloc(N * sizeof(*grads));
    int64_t* numels = malloc(N * sizeof(*numels));
    int32_t* dtypes = malloc(N * sizeof(*dtypes));
    for (int i = 0; i < N; ++i) {
        grads[i] = P(0x100000 + 64 * i);
        numels[i] = i % 7;
        dtypes[i] = i & 1;
    }
#define CLIP(ws) bfly_grad_clip(N, grads, (void* const*)grads, numels, dtypes, 1.f, F(0x10000), P(0x20000), ws, NULL)
    EXPECT(CLIP(bfly_grad_clip_workspace_bytes(N) - 1) == BFLY_ERR_WORKSPACE);
    numels[N - 1] = INT64_MAX;
    EXPECT(CLIP(big) == BFLY_ERR_UNSUPPORTED);
    numels[N - 1] = -5;
    EXPECT(CLIP(big) == BFLY_ERR_SIZE);
    numels[N - 1] = 5;
    dtypes[N - 1] = 9;
    EXPECT(CLIP(big) == BFLY_ERR_DTYPE);
    dtypes[N - 1] = 1;
    grads[N - 1] = P(0x100001);
    EXPECT(CLIP(big) == BFLY_ERR_ALIGN);
    grads[N - 1] = NULL;
    EXPECT(CLIP(big) == BFLY_ERR_NULL);
    EXPECT(bfly_grad_clip(0, NULL, NULL, NULL, NULL, NAN, F(0x10000), P(0x20000), big, NULL) ==
           BFLY_ERR_SIZE);
    free(grads);
    free(numels);
    free(dtypes);
    if (failures) {
        fprintf(stderr, "%d failed checks\n", failures);
        return 1;
    }
    printf("ops_san: all checks passed\n");
    return 0;
}
