/*
 * Driver for the sanitizer build of the library's host layer, the operators
 * that close a training step (test infrastructure; no GPU needed, no kernel is
 * launched): every host-side path of their entry points that ends before a
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
#define E4M3 QLORA_DTYPE_E4M3
#define I64 QLORA_DTYPE_I64

static unsigned char* p; /* 4 KiB, 256-byte aligned: never read by a valid path */

static void add_norm(void) {
    EXPECT(qlora_add_norm_fwd(p, 8, F32, p, 8, F32, 0, 8, 0, 0, 0, F32, 0.0f, p, 8, p, 8, E4M3, 0, 0, 0),
           QLORA_OK);
    EXPECT(qlora_add_norm_fwd(p, MAX64, F32, p, 8, F32, 4, 8, 0, 0, 0, F32, 0.0f, p, 8, p, 8, F32, 0, 0, 0),
           QLORA_ERR_SHAPE);
    EXPECT(qlora_add_norm_fwd(p, 8, F32, p, MAX64, F32, 4, 8, 0, 0, 0, F32, 0.0f, p, 8, p, 8, F32, 0, 0, 0),
           QLORA_ERR_SHAPE);
    EXPECT(qlora_add_norm_fwd(p, 8, F32, p, 8, F32, MAX64, 8, 0, 0, 0, F32, 0.0f, p, 8, p, 8, F32, 0, 0, 0),
           QLORA_ERR_SHAPE);
    EXPECT(qlora_add_norm_fwd(p, 8, F32, 0, 8, 77, 4, 8, 0, 0, 0, F32, 0.0f, 0, 8, p, 8, F32, 0, 0, 0),
           QLORA_ERR_INVALID_ARG); /* y over x */
    EXPECT(qlora_add_norm_fwd(p, 8, F32, p, 8, 77, 4, 8, 0, 0, 0, F32, 0.0f, p, 8, p, 8, F32, 0, 0, 0),
           QLORA_ERR_DTYPE);
    EXPECT(qlora_add_norm_fwd(p, 8, F32, p, 8, F32, 4, 8, 0, 0, 0, F32, NAN, p, 8, p, 8, F32, 0, 0, 0),
           QLORA_ERR_INVALID_ARG);
    EXPECT(qlora_add_norm_bwd(p, 8, F32, p, MAX64, p, 8, F32, 4, 8, 0, 0, F32, 0.0f, 0, p, 8, F32, p, 0, F32, p,
                              4096, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_add_norm_bwd(p, 8, F32, p, 8, p, 8, F32, 4, 8, 0, 0, F32, 0.0f, 0, p, 8, F32, p, 0, F32, p, 1, 0),
           QLORA_ERR_WORKSPACE);
    EXPECT(qlora_add_norm_bwd(p, 8, F32, p, 8, p, 8, F32, 0, 8, 0, 0, F32, 0.0f, 0, p, 8, F32, 0, 0, F32, 0, 0, 0),
           QLORA_OK);
}

static void head(void) {
    static const int64_t bad[] = {-1, INT64_MIN, MAX64, (int64_t)1 << 40};
    for (int i = 0; i < 4; ++i)
        for (int copy = 0; copy < 2; ++copy) {
            EXPECT(qlora_head_loss_fwd_workspace_bytes(bad[i], 8, 8, copy), 0);
            EXPECT(qlora_head_loss_fwd_workspace_bytes(8, bad[i], 8, copy), 0);
            EXPECT(qlora_head_loss_fwd_workspace_bytes(8, 8, bad[i], copy), 0);
            EXPECT(qlora_head_loss_bwd_workspace_bytes(bad[i], 8, 8, copy, F32, F32), 0);
            EXPECT(qlora_head_loss_bwd_workspace_bytes(8, bad[i], 8, copy, F32, F32), 0);
            EXPECT(qlora_head_loss_bwd_workspace_bytes(8, 8, bad[i], copy, F32, F32), 0);
        }
    for (int64_t M = 1; M <= QLORA_MAX_SORTED; M = M * 3 + 1)
        for (int64_t V = 1; V <= (int64_t)1 << 24; V = V * 7 + 3)
            for (int64_t K = 1; K <= QLORA_MAX_HEAD_WIDTH; K = K * 5 + 2) {
                const size_t a = qlora_head_loss_fwd_workspace_bytes(M, V, K, 0);
                const size_t b = qlora_head_loss_fwd_workspace_bytes(M, V, K, 1);
                const size_t c = qlora_head_loss_bwd_workspace_bytes(M, V, K, 0, BF16, -1);
                const size_t d = qlora_head_loss_bwd_workspace_bytes(M, V, K, 1, F32, F32);
                if (V > ((int64_t)1 << 40) / K) continue;
                if (a == 0 || b < a || c == 0 || d == 0) g_fail = 1;
            }
    if (qlora_head_loss_fwd_workspace_bytes(QLORA_MAX_SORTED, INT32_MAX - 1, 512, 1) == 0) g_fail = 1;
    if (qlora_head_loss_bwd_workspace_bytes(QLORA_MAX_SORTED, INT32_MAX - 1, 512, 1, F32, F32) == 0) g_fail = 1;
    uint16_t* h = (uint16_t*)p;
    float* f = (float*)p;
    EXPECT(qlora_head_loss_fwd(h, 8, h, 8, 0, 9, 8, 0, I64, 1.0f, 0, 0, 0, 0, 0), QLORA_OK);
    EXPECT(qlora_head_loss_fwd(h, MAX64, h, 8, 4, 9, 8, p, I64, 1.0f, f, 0, p, 4096, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_head_loss_fwd(h, 8, h, MAX64, 4, 9, 8, p, I64, 1.0f, f, 0, p, 4096, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_head_loss_fwd(h, 8, h, 8, MAX64, MAX64, MAX64, p, I64, 1.0f, f, 0, p, 4096, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_head_loss_fwd(h, 8, h, 8, 4, 9, 8, p, I64, INFINITY, f, 0, p, 4096, 0), QLORA_ERR_INVALID_ARG);
    EXPECT(qlora_head_loss_fwd(h, 8, h, 8, 4, 9, 8, p, F32, 1.0f, f, 0, p, 4096, 0), QLORA_ERR_DTYPE);
    EXPECT(qlora_head_loss_fwd(h, 8, h, 8, 4, 9, 8, p, I64, 1.0f, f, 0, p, 1, 0), QLORA_ERR_WORKSPACE);
    EXPECT(qlora_head_loss_fwd(h, 8, h, 8, 4, 9, 8, p, I64, 1.0f, f, 0, p, 4096, 0), QLORA_ERR_INVALID_ARG);
    EXPECT(qlora_head_loss_bwd(h, 8, h, 8, 4, 9, 8, p, I64, 1.0f, f, f, p, MAX64, F32, 0, F32, 0, p, 4096, 0),
           QLORA_ERR_SHAPE);
    EXPECT(qlora_head_loss_bwd(h, 8, h, 8, 4, 9, 8, p, I64, 1.0f, f, f, p, 8, F32, 0, F32, 0, p, 4096, 0),
           QLORA_ERR_WORKSPACE);
    EXPECT(qlora_head_loss_bwd(h, 8, h, 8, 4, 9, 8, p, I64, 1.0f, f, f, 0, 8, F32, 0, F32, 0, p, 4096, 0),
           QLORA_OK);
    EXPECT(qlora_head_loss_bwd(h, 8, h, 8, 0, 9, 8, 0, I64, 1.0f, 0, 0, p, 8, F32, p, F32, 1, 0, 0, 0), QLORA_OK);
}

static void clip(void) {
    qlora_tensor* t = calloc(3000, sizeof *t);
    if (!t) exit(2);
    for (int i = 0; i < 3000; ++i) {
        t[i].data = p + 4 * (i % 1000);
        t[i].n = i % 7 == 6 ? 0 : 1;
        t[i].dtype = i & 1 ? BF16 : F32;
    }
    /* every size of the list, exactly allocated: reads past it stop the run */
    for (int n = 1; n <= 3000; n += 271) {
        qlora_tensor* u = malloc((size_t)n * sizeof *u);
        if (!u) exit(2);
        for (int i = 0; i < n; ++i) u[i] = t[i];
        const size_t bytes = qlora_tensor_table_bytes(u, n);
        void* table = aligned_alloc(16, bytes ? bytes : 16);
        EXPECT(qlora_tensor_table(u, n, table, bytes), QLORA_OK);
        EXPECT(qlora_tensor_table(u, n, table, bytes ? bytes - 1 : 0), bytes ? QLORA_ERR_WORKSPACE : QLORA_OK);
        EXPECT(qlora_grad_norm(u, n, 0, 1.0f, (float*)p, p, 1, 0), QLORA_ERR_WORKSPACE);
        EXPECT(qlora_grad_scale(u, 0, n, 0, 0, (float*)p, 0), QLORA_ERR_INVALID_ARG); /* the factor */
        EXPECT(qlora_grad_scale(u, t + 1, n < 2999 ? n : 2999, 0, 0, (float*)p, 0), QLORA_ERR_DTYPE);
        free(table);
        free(u);
    }
    t[0].n = MAX64;
    EXPECT(qlora_grad_norm(t, 1, 0, 1.0f, (float*)p, p, 1, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_tensor_table_bytes(t, 1), 0);
    t[0].n = INT64_MIN;
    EXPECT(qlora_grad_norm(t, 1, 0, 1.0f, (float*)p, p, 1, 0), QLORA_ERR_INVALID_ARG);
    t[0].n = (int64_t)1 << 40;
    t[1].n = (int64_t)1 << 40;
    EXPECT(qlora_grad_scale(t, 0, 2, 0, 0, (float*)p, 0), QLORA_ERR_SHAPE);
    EXPECT(qlora_grad_norm_workspace_bytes(t, MAX64), 0);
    EXPECT(qlora_grad_norm(0, 0, 0, -1.0f, (float*)p, 0, 0, 0), QLORA_ERR_INVALID_ARG);
    EXPECT(qlora_adamw_step_scaled((float*)p, p, F32, (float*)p, (float*)p, (float*)p, 0, 0, 1e-3, 0.9, 0.99, 1e-8,
                                   0.0, 1, 0), QLORA_OK);
    EXPECT(qlora_adamw_step_scaled((float*)p, p, F32, 0, (float*)p, (float*)p, 0, 8, 1e-3, 0.9, 0.99, 1e-8, 0.0, 1,
                                   0), QLORA_ERR_INVALID_ARG);
    free(t);
}

int main(void) {
    unsigned char* raw = malloc(4096 + 256);
    if (!raw) return 2;
    p = (unsigned char*)(((uintptr_t)raw + 255) & ~(uintptr_t)255);
    add_norm();
    head();
    clip();
    free(raw);
    if (g_fail) return 1;
    printf("the close of a step: every status as documented\n");
    return 0;
}
