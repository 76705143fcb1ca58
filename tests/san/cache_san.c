/* Host-side checks of the cache calls' argument validation and size query,
 * built with AddressSanitizer and UndefinedBehaviorSanitizer (host code only)
 * by tests/test_sanitize_cache_cpu.py.  Every call here is rejected, or is a
 * pure size query, before any HIP call; the pointers are fake addresses the
 * library never dereferences. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>

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
#define S(a) ((uint16_t*)(uintptr_t)(a))
#define I(a) ((int32_t*)(uintptr_t)(a))
#define F(a) ((float*)(uintptr_t)(a))

static const int64_t wide[] = {INT64_MAX, INT64_MIN, -1, (int64_t)1 << 62, ((int64_t)1 << 46) + 1};
static const int32_t sizes[] = {INT32_MIN, -1, 0, 7, 1 << 30, INT32_MAX};

static bfly_status rows(int write, int64_t ks, int64_t vs, int64_t tokens, int32_t pages,
                        int32_t kv, int32_t page, int32_t d, int32_t dt, int32_t fmt)
{
    /* slots are misaligned: no call gets past the checks */
    return write ? bfly_cache_write(P(0x10000), ks, P(0x20000), vs, (bfly_dtype)dt, I(0x30002), tokens,
                                    P(0x40000), P(0x50000), S(0x60000), S(0x70000), pages, kv, page,
                                    d, (bfly_kv)fmt, NULL)
                 : bfly_cache_read(P(0x40000), P(0x50000), S(0x60000), S(0x70000), I(0x30002), tokens,
                                   P(0x10000), ks, P(0x20000), vs, (bfly_dtype)dt, pages, kv, page, d,
                                   (bfly_kv)fmt, NULL);
}

static bfly_status attend(int64_t qs, int32_t width, int64_t n, int32_t heads, int32_t pages,
                          int32_t kv, int32_t page, int32_t d, int32_t fmt, float scale,
                          int32_t most, int32_t window, size_t bytes)
{
    return bfly_cache_attention(P(0x10000), qs, BFLY_BF16, P(0x20000), P(0x30000), S(0x40000),
                                S(0x50000), I(0x60002), width, I(0x70000), P(0x80000), BFLY_BF16,
                                F(0x90000), n, heads, pages, kv, page, d, (bfly_kv)fmt, scale, most,
                                window, P(0xA0000), bytes, NULL);
}

int main(void)
{
    for (int w = 0; w < 2; ++w) {
        EXPECT(rows(w, 1024, 1024, 4, 10, 8, 16, 128, 1, 1) == BFLY_ERR_ALIGN);
        for (size_t i = 0; i < sizeof(wide) / sizeof(wide[0]); ++i) {
            const int64_t v = wide[i];
            EXPECT(rows(w, v, 1024, 4, 10, 8, 16, 128, 1, 1) != BFLY_OK);
            EXPECT(rows(w, 1024, v, 4, 10, 8, 16, 128, 1, 1) != BFLY_OK);
            EXPECT(rows(w, 1024, 1024, v, 10, 8, 16, 128, 1, 1) != BFLY_OK);
        }
        for (size_t i = 0; i < sizeof(sizes) / sizeof(sizes[0]); ++i) {
            const int32_t v = sizes[i];
            EXPECT(rows(w, 1024, 1024, 4, v, 8, 16, 128, 1, 1) != BFLY_OK);
            EXPECT(rows(w, 1024, 1024, 4, 10, v, 16, 128, 1, 1) != BFLY_OK);
            EXPECT(rows(w, 1024, 1024, 4, 10, 8, v, 128, 1, 1) != BFLY_OK);
            EXPECT(rows(w, 1024, 1024, 4, 10, 8, 16, v, 1, 1) != BFLY_OK);
            EXPECT(rows(w, 1024, 1024, 4, 10, 8, 16, 128, v | 2, 1) == BFLY_ERR_DTYPE);
            EXPECT(rows(w, 1024, 1024, 4, 10, 8, 16, 128, 1, v | 4) == BFLY_ERR_QUANT);
        }
    }
    EXPECT(attend(4096, 8, 4, 32, 10, 8, 16, 128, 1, 0.1f, 128, 0, SIZE_MAX) == BFLY_ERR_ALIGN);
    for (size_t i = 0; i < sizeof(wide) / sizeof(wide[0]); ++i) {
        const int64_t v = wide[i];
        EXPECT(bfly_cache_attention_workspace_bytes(v, 32, 8, 128, 100000) == 0);
        EXPECT(attend(v, 8, 4, 32, 10, 8, 16, 128, 1, 0.1f, 128, 0, SIZE_MAX) != BFLY_OK);
        EXPECT(attend(4096, 8, v, 32, 10, 8, 16, 128, 1, 0.1f, 128, 0, SIZE_MAX) != BFLY_OK);
    }
    for (size_t i = 0; i < sizeof(sizes) / sizeof(sizes[0]); ++i) {
        const int32_t v = sizes[i];
        EXPECT(bfly_cache_attention_workspace_bytes(4, v, 8, 128, 100000) == 0);
        EXPECT(bfly_cache_attention_workspace_bytes(4, 32, v, 128, 100000) == 0);
        EXPECT(bfly_cache_attention_workspace_bytes(4, 32, 8, v, 100000) == 0);
        EXPECT(bfly_cache_attention_workspace_bytes(4, 32, 8, 128, v) == 0 || v == (1 << 30));
        EXPECT(attend(4096, v, 4, 32, 10, 8, 16, 128, 1, 0.1f, 128, 0, SIZE_MAX) != BFLY_OK);
        EXPECT(attend(1 << 30, 8, 4, v, 10, 8, 16, 128, 1, 0.1f, 128, 0, SIZE_MAX) != BFLY_OK);
        EXPECT(attend(4096, 8, 4, 32, v, 8, 16, 128, 1, 0.1f, 128, 0, SIZE_MAX) != BFLY_OK);
        EXPECT(attend(4096, 8, 4, 32, 10, v, 16, 128, 1, 0.1f, 128, 0, SIZE_MAX) != BFLY_OK);
        EXPECT(attend(4096, 8, 4, 32, 10, 8, v, 128, 1, 0.1f, 128, 0, SIZE_MAX) != BFLY_OK);
        EXPECT(attend(4096, 8, 4, 32, 10, 8, 16, v, 1, 0.1f, 128, 0, SIZE_MAX) != BFLY_OK);
        EXPECT(attend(4096, 8, 4, 32, 10, 8, 16, 128, v | 4, 0.1f, 128, 0, SIZE_MAX) ==
               BFLY_ERR_QUANT);
        EXPECT(attend(4096, INT32_MAX, 4, 32, 10, 8, 65536, 128, 1, 0.1f, v, 0, SIZE_MAX) != BFLY_OK);
        EXPECT(attend(4096, 8, 4, 32, 10, 8, 16, 128, 1, 0.1f, 128, v, SIZE_MAX) != BFLY_OK);
    }
    EXPECT(attend(4096, 8, 4, 32, 10, 8, 16, 128, 1, NAN, 128, 0, SIZE_MAX) == BFLY_ERR_SIZE);
    EXPECT(attend(4096, 8, 4, 32, 10, 8, 16, 128, 1, INFINITY, 128, 0, SIZE_MAX) == BFLY_ERR_SIZE);
    EXPECT(attend(4096, 1 << 26, 1 << 20, 32, 10, 8, 16, 128, 1, 0.1f, 1 << 30, 0, 0) != BFLY_OK);
    EXPECT(bfly_cache_attention_workspace_bytes(255, 65536, 4096, 256, 1 << 30) > 0);
    if (failures) return 1;
    puts("all checks passed");
    return 0;
}
