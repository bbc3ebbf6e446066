/*
 * Driver for the sanitizer build of the library's host layer, row operators
 * (test infrastructure; no GPU needed, no kernel is launched): every host-side
 * path of the embedding, norm and distillation entry points that ends before a
 * launch, with sizes at and past their limits and products that pass 64 bits.
 * Stand-in device pointers point into one small heap buffer, so any host read
 * or write through them past its end stops the run. Each call's status is
 * compared with the one the header documents.
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "../../include/qlora_amd.h"

static int g_fail = 0;

#define EXPECT(call, want)                                                          \
    do {                                                                            \
        const long long got_ = (long long)(call);                                   \
        if (got_ != (long long)(want)) {                                            \
            fprintf(stderr, "line %d: %s = %lld, expected %lld\n", __LINE__, #call, \
                    got_, (long long)(want));                                       \
            g_fail = 1;                                                             \
        }                                                                           \
    } while (0)

#define MAX64 INT64_MAX
#define F32 QLORA_DTYPE_F32
#define BF16 QLORA_DTYPE_BF16
#define I32 QLORA_DTYPE_I32
#define I64 QLORA_DTYPE_I64

static unsigned char* p; /* 4 KiB, 256-byte aligned: never read by a valid path */

static void queries(void) {
    static const int64_t bad[] = {-1, INT64_MIN, MAX64, (int64_t)1 << 40};
    for (int i = 0; i < 4; ++i) {
        EXPECT(qlora_embed_bwd_workspace_bytes(bad[i], 8), 0);
        EXPECT(qlora_embed_bwd_workspace_bytes(8, bad[i]), 0);
        EXPECT(qlora_norm_bwd_workspace_bytes(bad[i], 8), 0);
        EXPECT(qlora_norm_bwd_workspace_bytes(8, bad[i]), 0);
        EXPECT(qlora_distill_fwd_workspace_bytes(bad[i], 8), 0);
        EXPECT(qlora_distill_fwd_workspace_bytes(8, bad[i]), 0);
    }
    if (qlora_embed_bwd_workspace_bytes(QLORA_MAX_SORTED, 1 << 24) < ((size_t)1 << 40)) g_fail = 1;
    if (qlora_norm_bwd_workspace_bytes(QLORA_MAX_ROWS, QLORA_MAX_NORM_WIDTH) == 0) g_fail = 1;
    if (qlora_distill_fwd_workspace_bytes(QLORA_MAX_ROWS, INT32_MAX - 1) == 0) g_fail = 1;
    for (int64_t M = 0; M <= QLORA_MAX_SORTED; M = M * 3 + 1)
        for (int64_t n = 1; n <= QLORA_MAX_NORM_WIDTH; n = n * 5 + 2) {
            const size_t a = qlora_embed_bwd_workspace_bytes(M, n);
            const size_t b = qlora_norm_bwd_workspace_bytes(M, n);
            if ((M == 0) != (a == 0) || (M == 0) != (b == 0)) g_fail = 1;
        }
}

static void embed(void) {
    EXPECT(qlora_embed_fwd(p, 8, BF16, 10, 8, p, I64, 0, 1.0f, p, 8, F32, 0), QLORA_OK);
    EXPECT(qlora_embed_fwd(p, 8, BF16, 10, 8, p, I64, -1, 1.0f, p, 8, F32, 0), QLORA_ERR_INVALID_ARG);
    EXPECT(qlora_embed_fwd(p, 8, BF16, 10, 8, p, I64, 4, NAN, p, 8, F32, 0), QLORA_ERR_INVALID_ARG);
    EXPECT(qlora_embed_fwd(p, MAX64, BF16, 10, 8, p, I64, 4, 1.0f, p, 8, F32, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_embed_fwd(p, 8, BF16, 10, 8, p, I64, 4, 1.0f, p, MAX64, F32, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_embed_fwd(p, 8, BF16, MAX64, MAX64, p, I64, 4, 1.0f, p, 8, F32, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_embed_fwd(p, 8, BF16, 10, 8, p, I64, MAX64, 1.0f, p, 8, F32, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_embed_fwd(p, 8, 7, 10, 8, p, I64, 4, 1.0f, p, 8, F32, 0), QLORA_ERR_DTYPE);
    EXPECT(qlora_embed_fwd(0, 8, BF16, 10, 8, p, I64, 4, 1.0f, p, 8, F32, 0), QLORA_ERR_INVALID_ARG);
    EXPECT(qlora_embed_fwd(p + 1, 8, BF16, 10, 8, p, I64, 4, 1.0f, p, 8, F32, 0), QLORA_ERR_ALIGN);
    const size_t need = qlora_embed_bwd_workspace_bytes(4, 8);
    EXPECT(qlora_embed_bwd(p, 8, BF16, p, I32, 4, 10, 8, 1.0f, p, F32, 0, p, need - 1, 0),
           QLORA_ERR_WORKSPACE);
    EXPECT(qlora_embed_bwd(p, 8, BF16, p, I32, 4, 10, 8, 1.0f, p, F32, 0, 0, need, 0),
           QLORA_ERR_WORKSPACE);
    EXPECT(qlora_embed_bwd(p, 8, BF16, p, I32, MAX64, 10, 8, 1.0f, p, F32, 0, p, need, 0),
           QLORA_ERR_SHAPE);
    EXPECT(qlora_embed_bwd(0, 8, BF16, 0, I32, 0, 10, 8, 1.0f, p, F32, 1, 0, 0, 0), QLORA_OK);
    EXPECT(qlora_embed_bwd(p, 8, BF16, p, I32, 4, 10, 8, 1.0f, p + 2, F32, 0, p, need, 0),
           QLORA_ERR_ALIGN);
}

static void norm(void) {
    EXPECT(qlora_norm_fwd(p, 8, F32, 0, 8, 0, 0, 0, F32, 1e-5f, p, 8, F32, 0, 0), QLORA_OK);
    EXPECT(qlora_norm_fwd(p, 8, F32, 4, 8, 2, 0, 0, F32, 1e-5f, p, 8, F32, 0, 0), QLORA_ERR_INVALID_ARG);
    EXPECT(qlora_norm_fwd(p, 8, F32, 4, 8, 1, 0, 0, F32, -1.0f, p, 8, F32, 0, 0), QLORA_ERR_INVALID_ARG);
    EXPECT(qlora_norm_fwd(p, MAX64, F32, 4, 8, 1, 0, 0, F32, 0.0f, p, 8, F32, 0, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_norm_fwd(p, 8, F32, MAX64, 8, 1, 0, 0, F32, 0.0f, p, 8, F32, 0, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_norm_fwd(p, 8, F32, 4, 8, 1, p + 1, 0, BF16, 0.0f, p, 8, F32, 0, 0), QLORA_ERR_ALIGN);
    const size_t need = qlora_norm_bwd_workspace_bytes(4, 8);
    EXPECT(qlora_norm_bwd(p, 8, F32, p, 8, F32, 4, 8, 0, 0, F32, 0.0f, 0, p, 8, F32, p, 0, F32, p,
                          need - 1, 0), QLORA_ERR_WORKSPACE);
    EXPECT(qlora_norm_bwd(p, 8, F32, p, 8, F32, 4, 8, 0, 0, F32, 0.0f, 0, 0, 8, F32, 0, 0, F32, 0, 0, 0),
           QLORA_OK);
    EXPECT(qlora_norm_bwd(p, 8, F32, p, 8, F32, 4, 8, 0, 0, F32, 0.0f, 0, p, 7, F32, 0, 0, F32, 0, 0, 0),
           QLORA_ERR_SHAPE);
    EXPECT(qlora_norm_bwd(p, 8, F32, p, 8, F32, 4, 8, 0, 0, F32, 0.0f, 0, p, 8, 9, 0, 0, F32, 0, 0, 0),
           QLORA_ERR_DTYPE);
    EXPECT(qlora_norm_bwd(0, 8, F32, p, 8, F32, 4, 8, 0, 0, F32, 0.0f, 0, p, 8, F32, 0, 0, F32, 0, 0, 0),
           QLORA_ERR_INVALID_ARG);
}

static void distill(void) {
    EXPECT(qlora_distill_fwd(p, 9, BF16, 0, 9, p, I32, p, F32, 2, 1.0f, (float*)p, 0, 0, 0, 0), QLORA_OK);
    EXPECT(qlora_distill_fwd(p, 9, BF16, 4, 9, p, I32, p, F32, 2, INFINITY, (float*)p, 0, 0, 0, 0),
           QLORA_ERR_INVALID_ARG);
    EXPECT(qlora_distill_fwd(p, 9, BF16, 4, 9, p, I32, p, F32, QLORA_MAX_TOP + 1, 1.0f, (float*)p, 0, 0, 0, 0),
           QLORA_ERR_SHAPE);
    EXPECT(qlora_distill_fwd(p, MAX64, BF16, MAX64, MAX64, p, I32, p, F32, 2, 1.0f, (float*)p, 0, 0, 0, 0),
           QLORA_ERR_SHAPE);
    EXPECT(qlora_distill_fwd(p, 1 << 20, BF16, 4, 1 << 20, p, I32, p, F32, 2, 1.0f, (float*)p, 0, 0, 0, 0),
           QLORA_ERR_WORKSPACE);
    EXPECT(qlora_distill_fwd(p, 9, BF16, 4, 9, p, F32, p, F32, 2, 1.0f, (float*)p, 0, 0, 0, 0), QLORA_ERR_DTYPE);
    EXPECT(qlora_distill_bwd(p, 9, BF16, 4, 9, p, I32, p, F32, 2, 1.0f, 0, (float*)p, p, 9, F32, 0),
           QLORA_ERR_INVALID_ARG);
    EXPECT(qlora_distill_bwd(p, 9, BF16, 4, 9, p, I32, p, F32, 2, 1.0f, (float*)p, (float*)p, p, 8, F32, 0),
           QLORA_ERR_SHAPE);
    EXPECT(qlora_distill_bwd(p, 9, BF16, 4, 9, p, I32, p, F32, 2, 1.0f, (float*)p, (float*)p, p + 2, 9,
                             F32, 0), QLORA_ERR_ALIGN);
    EXPECT(qlora_distill_bwd(p, 9, BF16, 0, 9, 0, I32, 0, F32, 2, 1.0f, 0, 0, 0, 9, F32, 0), QLORA_OK);
}

int main(void) {
    unsigned char* raw = malloc(4096 + 256);
    if (!raw) return 2;
    p = (unsigned char*)(((uintptr_t)raw + 255) & ~(uintptr_t)255);
    queries();
    embed();
    norm();
    distill();
    free(raw);
    if (g_fail) return 1;
    printf("row operators: every status as documented\n");
    return 0;
}
