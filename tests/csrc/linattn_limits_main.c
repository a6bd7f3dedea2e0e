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

int main(void) {
    for (int32_t under = 0; under < 20000; under += 331)
        for (int32_t K = 1; K <= 64; K += 21)
            for (int32_t dt = 0; dt < 2; ++dt) beam_vocabulary(0x7fffffff - under, K, dt);
    printf("%d failures\n", failures);
    return failures != 0;
}
