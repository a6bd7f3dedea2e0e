/* Sizes at the ends of what gdn_linattn.h allows, for the host code of its entry points
 * built with AddressSanitizer and UndefinedBehaviorSanitizer: sums of sizes must not pass
 * their types.  No GPU is needed: no call here gets as far as a launch. */
#include <stdint.h>
#include <stdio.h>

#include "gdn_linattn.h"

static int failures = 0;
#define EXPECT(cond)                                              \
    do {                                                          \
        if (!(cond)) {                                            \
            ++failures;                                           \
            printf("line %d: %s (%s)\n", __LINE__, #cond, gdn_last_error()); \
        }                                                         \
    } while (0)

/* The workspace of one beam of V logits: a key for each of K per slice, slices of 2,048 logits or more. */
static void beam_vocabulary(int32_t V, int32_t K, int32_t dtype) {
    gdn_beam_desc d = {1, 1, V, K, dtype, V};
    size_t n = 0;
    EXPECT(gdn_beam_workspace_size(&d, &n) == GDN_OK);
    EXPECT(n >= (size_t)K * 8 && n <= ((size_t)V / 2048 + 1) * ((size_t)K * 8 + 8) + 512);
}

#define P(i) ((void *)(uintptr_t)((1ULL << 40) + (uint64_t)(i) * (1ULL << 36)))

/* Rows times a stride that no buffer can have (2^70 elements) are refused before they are multiplied. */
static void far_rows(int64_t stride) {
    gdn_qk_rope_desc r = {0x7fffffffLL, 4, 2, 128, 64, 0, GDN_F32, stride, 256, 1e-6f, 0.f};
    EXPECT(gdn_qk_norm_rope(&r, P(0), P(1), P(2), P(3), P(4), P(5), P(6), P(7), NULL) == GDN_ERR_INVALID_ARG);
    r.q_stride = 512;
    r.k_stride = stride;
    EXPECT(gdn_qk_norm_rope(&r, P(0), P(1), P(2), P(3), P(4), P(5), P(6), P(7), NULL) == GDN_ERR_INVALID_ARG);
    gdn_beam_desc b = {0x7fffffffLL / 64, 64, 100, 8, GDN_F32, stride};
    size_t n = 0;
    EXPECT(gdn_beam_workspace_size(&b, &n) == GDN_ERR_INVALID_ARG);
    EXPECT(gdn_beam_select(&b, P(0), P(1), P(2), P(3), P(4), P(5), (size_t)1 << 60, NULL) == GDN_ERR_INVALID_ARG);
}

/* No sequences: nothing to plan, whatever the number of tokens or heads.  States past 4e15 elements are refused. */
static void few_and_many_sequences(int32_t dtype, int32_t gate) {
    size_t n = 0;
    gdn_desc d = {0, 0x7fffffffffffffffLL, 16, 128, 128, dtype, gate, 1.0f, 0};
    EXPECT(gdn_linattn_workspace_size(&d, 0, &n) == GDN_OK && n >= 4 && n <= 4096);
    EXPECT(gdn_linattn_chunk_fwd(&d, NULL, NULL, NULL, NULL, NULL, NULL, 0, 0, NULL, NULL, NULL, NULL, 0, NULL) == GDN_OK);
    d.T = 0;
    d.H = 1LL << 61;
    EXPECT(gdn_linattn_workspace_size(&d, 0, &n) == GDN_OK && n >= 4 && n <= 4096);
    d.B = 1;
    EXPECT(gdn_linattn_workspace_size(&d, 1, &n) == GDN_ERR_INVALID_ARG);
    EXPECT(gdn_linattn_chunk_fwd(&d, NULL, NULL, NULL, NULL, NULL, NULL, 0, 0, NULL, P(0), NULL, P(1), (size_t)1 << 60,
                                 NULL) == GDN_ERR_INVALID_ARG);
    d.T = 1;
    d.H = 30000000000000LL;
    EXPECT(gdn_linattn_workspace_size(&d, 0x7fffffff, &n) == GDN_ERR_INVALID_ARG);
}

int main(void) {
    for (int32_t dt = 0; dt < 2; ++dt)
        for (int32_t gate = 0; gate < 3; gate += 2) few_and_many_sequences(dt, gate);

    far_rows(1LL << 40);
    far_rows(1LL << 34);
    far_rows(1LL << 62);
    far_rows(0x7ffffffffffffff0LL);

    for (int32_t under = 0; under < 20000; under += 331)
        for (int32_t K = 1; K <= 64; K += 21)
            for (int32_t dt = 0; dt < 2; ++dt) beam_vocabulary(0x7fffffff - under, K, dt);
    printf("%d failures\n", failures);
    return failures != 0;
}
