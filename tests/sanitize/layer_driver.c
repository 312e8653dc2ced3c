/* Host validation of the layer's operators (include/ssd_layer.h) under AddressSanitizer and
 * UndefinedBehaviorSanitizer (host code only; no GPU is touched: every call below is refused before
 * anything is launched, or is a pure host query).  Exits 0 when every status is the expected one. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "ssd_layer.h"

static int fails = 0;
#define EXPECT(expr, want)                                                           \
    do {                                                                             \
        long got_ = (long)(expr);                                                    \
        if (got_ != (long)(want)) {                                                  \
            fprintf(stderr, "line %d: %s = %ld, expected %ld\n", __LINE__, #expr,    \
                    got_, (long)(want));                                             \
            ++fails;                                                                 \
        }                                                                            \
    } while (0)

int main(void) {
    void* F = (void*)0x100000; /* never dereferenced */
    const void* mis = (const void*)0x100004;
    float* f = (float*)F;
    const int32_t* cu = (const int32_t*)F;
    const size_t big = (size_t)1 << 60;

    /* workspace queries over a grid of sizes, the largest ones included */
    size_t total = 0;
    const int64_t toks[] = {INT64_MIN, 0, 1, 63, 1025, 100000, INT32_MAX - 127, INT32_MAX, INT64_MAX};
    for (int act = -1; act < 3; ++act)
        for (int d = 32; d <= 256; d *= 2)
            for (int t = 0; t < 9; ++t)
                for (int H = 1; H <= 65536; H *= 16)
                    for (int kind = 0; kind < 3; ++kind) {
                        ssd_gdelta p = {1, toks[t], H, 1, d, 128, act, 1.f, 0, 0, 0, 0, 0, 0, 0, 0, 0};
                        total += ssd_gdelta_workspace_bytes(&p, 1, kind) & 0xffff;
                        total += ssd_gdelta_workspace_bytes(&p, 1 << 24, kind) & 0xffff;
                        total += ssd_gdelta_workspace_bytes(&p, INT32_MAX, kind) & 0xffff;
                        total += ssd_gdelta_workspace_bytes(&p, INT32_MIN, kind) & 0xffff;
                        p.batch = toks[t];
                        total += ssd_gdelta_workspace_bytes(&p, 7, kind) & 0xffff;
                    }
    for (int t = 0; t < 9; ++t)
        for (int C = 0; C <= (1 << 21); C = C * 2 + 1) {
            ssd_block n = {toks[t], C, SSD_BF16, SSD_F32, 1, 1, SSD_GATE_SILU, 0, 1.f, 1e-5f, 0, 0, 0, 0, 0, 0, 0, 0};
            total += ssd_block_norm_workspace_bytes(&n) & 0xffff;
        }
    EXPECT(ssd_gdelta_workspace_bytes(NULL, 1, SSD_WS_FORWARD), 0);
    EXPECT(ssd_block_norm_workspace_bytes(NULL), 0);
    printf("workspace sum %zu\n", total);

    ssd_gdelta p = {1, 1000, 8, 2, 128, 64, SSD_BF16, 1.f, 0, 0, 0, 0, 0, 0, 0, 0, 0};
    EXPECT(ssd_gdelta_fwd(NULL, 1, F, F, F, f, f, cu, NULL, F, NULL, F, big, NULL), SSD_ERR_NULL);
    EXPECT(ssd_gdelta_fwd(&p, 1, F, F, F, f, NULL, cu, NULL, F, NULL, F, big, NULL), SSD_ERR_NULL);
    EXPECT(ssd_gdelta_fwd(&p, 2, F, F, F, f, f, NULL, NULL, F, NULL, F, big, NULL), SSD_ERR_SEGMENTS);
    EXPECT(ssd_gdelta_fwd(&p, 1, mis, F, F, f, f, cu, NULL, F, NULL, F, big, NULL), SSD_ERR_ALIGN);
    EXPECT(ssd_gdelta_fwd(&p, 1, F, F, F, f, f, cu, NULL, F, NULL, NULL, big, NULL), SSD_ERR_WORKSPACE);
    EXPECT(ssd_gdelta_fwd(&p, 1, F, F, F, f, f, cu, NULL, F, NULL, F, 16, NULL), SSD_ERR_WORKSPACE);
    EXPECT(ssd_gdelta_bwd(&p, 3, F, F, F, f, f, cu, F, NULL, NULL, F, F, NULL, f, f, NULL, F, big, NULL),
           SSD_ERR_NULL);
    EXPECT(ssd_gdelta_bwd(&p, 3, F, F, F, f, f, cu, F, NULL, NULL, F, F, F, f, f, NULL, F, 16, NULL),
           SSD_ERR_WORKSPACE);
    EXPECT(ssd_gdelta_step(&p, F, F, F, f, f, NULL, 0, NULL, f, F, NULL), SSD_ERR_SHAPE);
    const int64_t strides[] = {INT64_MIN, -8, 4, 1 << 22, INT64_MAX};
    for (int i = 0; i < 5; ++i) {
        p.q_stride = strides[i];
        EXPECT(ssd_gdelta_fwd(&p, 1, F, F, F, f, f, cu, NULL, F, NULL, F, big, NULL), SSD_ERR_SHAPE);
        p.q_stride = 0, p.beta_stride = strides[i];
        EXPECT(ssd_gdelta_fwd(&p, 1, F, F, F, f, f, cu, NULL, F, NULL, F, big, NULL), SSD_ERR_SHAPE);
        p.beta_stride = 0;
    }
    p.batch = p.seqlen = INT32_MAX;
    EXPECT(ssd_gdelta_step(&p, F, F, F, f, f, cu, 1, NULL, f, F, NULL), SSD_ERR_SHAPE);

    ssd_block n = {8, 512, SSD_BF16, SSD_F32, 1, 1, SSD_GATE_SILU, 0, 1.f, 1e-5f, 0, 0, 0, 0, 0, 0, 0, 0};
    EXPECT(ssd_block_norm_fwd(&n, F, F, NULL, NULL, f, NULL, f, NULL, F, F, NULL), SSD_ERR_NULL);
    EXPECT(ssd_block_norm_fwd(&n, F, F, F, NULL, NULL, NULL, f, NULL, F, F, NULL), SSD_ERR_NULL);
    EXPECT(ssd_block_norm_bwd(&n, F, F, F, NULL, f, NULL, f, F, F, F, F, F, f, f, NULL, f, NULL, F, 8, NULL),
           SSD_ERR_WORKSPACE);
    n.eps = NAN;
    EXPECT(ssd_block_norm_fwd(&n, F, F, F, NULL, f, NULL, f, NULL, F, F, NULL), SSD_ERR_SHAPE);
    n.eps = 1e-5f;
    n.rows = INT64_MAX;
    EXPECT(ssd_block_norm_fwd(&n, F, F, F, NULL, f, NULL, f, NULL, F, F, NULL), SSD_ERR_SHAPE);
    n.rows = 8;
    n.dz_stride = INT64_MAX;
    EXPECT(ssd_block_norm_bwd(&n, F, F, F, NULL, f, NULL, f, F, F, F, F, F, f, f, NULL, f, NULL, F, big, NULL),
           SSD_ERR_SHAPE);
    n.dz_stride = 0;
    n.channels = INT32_MAX;
    EXPECT(ssd_block_norm_fwd(&n, F, F, F, NULL, f, NULL, f, NULL, F, F, NULL), SSD_ERR_UNSUPPORTED);

    ssd_rope_problem r = {1, 100, 4, 2, 64, 64, SSD_BF16, SSD_ROPE_HALF, 1.f, 0, 0, 0, 0};
    const double* w = (const double*)F;
    EXPECT(ssd_rope(&r, F, NULL, w, NULL, NULL, 1, 0, F, F, NULL), SSD_ERR_NULL);
    EXPECT(ssd_rope(&r, F, F, NULL, NULL, NULL, 1, 0, F, F, NULL), SSD_ERR_NULL);
    r.rotdim = 63;
    EXPECT(ssd_rope(&r, F, F, w, NULL, NULL, 1, 0, F, F, NULL), SSD_ERR_SHAPE);
    r.rotdim = 64, r.headdim = INT32_MAX;
    EXPECT(ssd_rope(&r, F, F, w, NULL, NULL, 1, 0, F, F, NULL), SSD_ERR_UNSUPPORTED);
    r.headdim = 64, r.batch = r.seqlen = INT64_MAX;
    EXPECT(ssd_rope(&r, F, F, w, NULL, NULL, 1, 0, F, F, NULL), SSD_ERR_SHAPE);
    printf("%d failed checks\n", fails);
    return fails != 0;
}
