/* Host validation of the operators around the scan (include/ssd_mixer.h) under
 * AddressSanitizer and UndefinedBehaviorSanitizer (host code only; no GPU is touched: every
 * call below is refused before anything is launched, or is a pure host query).  Exits 0 when
 * every status is the expected one. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "ssd_mixer.h"

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
    const int32_t* cu = (const int32_t*)0x100000;
    const size_t big = (size_t)1 << 46;

    /* workspace queries over a grid of sizes, the largest ones included */
    size_t total = 0;
    const int64_t toks[] = {1, 63, 1025, 100000, INT32_MAX - 127, INT32_MAX, INT64_MAX};
    for (int act = -1; act < 3; ++act)
        for (int d = 32; d <= 256; d *= 2)
            for (int t = 0; t < 7; ++t)
                for (int H = 1; H <= 65536; H *= 16)
                    for (int kind = 0; kind < 3; ++kind) {
                        ssd_linattn p = {1, toks[t], H, 1, d, 128, act, 1.f, 0, 0, 0, 0, 0, 0, 0};
                        total += ssd_linattn_workspace_bytes(&p, 1, kind) & 0xffff;
                        total += ssd_linattn_workspace_bytes(&p, 1 << 24, kind) & 0xffff;
                        total += ssd_linattn_workspace_bytes(&p, INT32_MAX, kind) & 0xffff;
                        p.batch = toks[t];
                        total += ssd_linattn_workspace_bytes(&p, 7, kind) & 0xffff;
                    }
    for (int C = 1; C <= (1 << 21); C = C * 2 + 1)
        for (int G = 1; G <= C; G = G * 3 + 1) {
            ssd_norm n = {(int64_t)1 << 20, C, G, SSD_BF16, SSD_NORM_BEFORE, 1, 1e-5f, 0, 0, 0, 0, 0};
            total += ssd_norm_workspace_bytes(&n) & 0xffff;
        }
    printf("workspace sum %zu\n", total);

    ssd_linattn p = {1, 1000, 8, 2, 128, 64, SSD_BF16, 1.f, 0, 0, 0, 0, 0, 0, 0};
    const float* f = (const float*)F;
    EXPECT(ssd_linattn_fwd(NULL, 1, F, F, F, f, cu, NULL, F, NULL, F, big, NULL), SSD_ERR_NULL);
    EXPECT(ssd_linattn_fwd(&p, 1, F, F, F, f, cu, NULL, NULL, NULL, F, big, NULL), SSD_ERR_NULL);
    EXPECT(ssd_linattn_fwd(&p, 2, F, F, F, f, NULL, NULL, F, NULL, F, big, NULL), SSD_ERR_SEGMENTS);
    EXPECT(ssd_linattn_fwd(&p, 1, mis, F, F, f, cu, NULL, F, NULL, F, big, NULL), SSD_ERR_ALIGN);
    EXPECT(ssd_linattn_fwd(&p, 1, F, F, F, f, cu, NULL, F, NULL, NULL, big, NULL), SSD_ERR_WORKSPACE);
    EXPECT(ssd_linattn_bwd(&p, 3, F, F, F, f, cu, F, NULL, NULL, F, F, NULL, NULL, F, big, NULL),
           SSD_ERR_NULL);
    EXPECT(ssd_linattn_bwd(&p, 3, F, F, F, f, cu, F, NULL, NULL, F, F, F, NULL, F, 16, NULL),
           SSD_ERR_WORKSPACE);
    EXPECT(ssd_linattn_step(&p, F, F, F, f, NULL, 0, NULL, (float*)F, F, NULL), SSD_ERR_SHAPE);
    p.q_stride = INT64_MAX;
    EXPECT(ssd_linattn_fwd(&p, 1, F, F, F, f, cu, NULL, F, NULL, F, big, NULL), SSD_ERR_SHAPE);
    p.q_stride = INT64_MIN;
    EXPECT(ssd_linattn_fwd(&p, 1, F, F, F, f, cu, NULL, F, NULL, F, big, NULL), SSD_ERR_SHAPE);
    p.q_stride = 0;
    p.batch = p.seqlen = INT32_MAX;
    EXPECT(ssd_linattn_step(&p, F, F, F, f, cu, 1, NULL, (float*)F, F, NULL), SSD_ERR_SHAPE);

    ssd_problem s = {4, 1, 8, 64, 128, 2, 64, 4, SSD_BF16, 1e-3f, 0.1f};
    EXPECT(ssd_token_step(&s, F, f, F, f, f, f, NULL, 4, NULL, F, 4, (float*)F, F, NULL), SSD_ERR_NULL);
    EXPECT(ssd_token_step(&s, F, f, F, f, f, f, NULL, 4, cu, F, 3, (float*)F, F, NULL), SSD_ERR_SHAPE);
    s.seqlen = INT64_MAX;
    EXPECT(ssd_token_step(&s, F, f, F, f, f, f, cu, 4, cu, F, INT32_MAX, (float*)F, F, NULL),
           SSD_ERR_SHAPE);
    s.seqlen = 1;
    s.batch = INT64_MAX;
    EXPECT(ssd_token_step(&s, F, f, F, f, f, f, cu, 4, cu, F, 4, (float*)F, F, NULL), SSD_ERR_SHAPE);

    ssd_norm n = {8, 512, 4, SSD_BF16, SSD_NORM_BEFORE, 0, 1e-5f, 0, 0, 0, 0, 0};
    EXPECT(ssd_norm_fwd(&n, F, NULL, f, NULL, F, NULL), SSD_ERR_NULL);
    EXPECT(ssd_norm_bwd(&n, F, F, f, NULL, F, F, F, (float*)F, NULL, F, 8, NULL), SSD_ERR_WORKSPACE);
    n.eps = NAN;
    EXPECT(ssd_norm_fwd(&n, F, F, f, NULL, F, NULL), SSD_ERR_SHAPE);
    n.eps = 1e-5f;
    n.rows = INT64_MAX;
    EXPECT(ssd_norm_fwd(&n, F, F, f, NULL, F, NULL), SSD_ERR_SHAPE);
    n.rows = 8;
    n.dz_stride = INT64_MAX;
    EXPECT(ssd_norm_fwd(&n, F, F, f, NULL, F, NULL), SSD_ERR_SHAPE);
    printf("%d failed checks\n", fails);
    return fails != 0;
}
