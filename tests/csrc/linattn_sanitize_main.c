/* Test driver for the host code of the entry points in gdn_linattn.h, built with
 * AddressSanitizer and UndefinedBehaviorSanitizer: sizes that they must plan, and
 * arguments that they must refuse before anything reaches the device.  No GPU is
 * needed: no call here gets as far as a launch. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "gdn_linattn.h"

static int failures = 0;
#define EXPECT(call, want)                                                                    \
    do {                                                                                      \
        const gdn_status got_ = (call);                                                       \
        if (got_ != (want)) {                                                                 \
            ++failures;                                                                       \
            printf("line %d: %s -> %d, want %d (%s)\n", __LINE__, #call, (int)got_, (int)(want), \
                   gdn_last_error());                                                         \
        }                                                                                     \
    } while (0)

#define P(i) ((void *)(uintptr_t)((1ULL << 40) + (uint64_t)(i) * (1ULL << 36)))
#define F(i) ((float *)P(i))
#define I(i) ((int32_t *)P(i))

int main(void) {
    size_t n = 0, last;
    const size_t big = (size_t)1 << 40;
    const int64_t Ts[] = {0, 1, 63, 64, 65, 4096, 262144, 1 << 20, 0x7fffffffLL};
    const int64_t Hs[] = {1, 3, 16, 64, 1000};
    for (int dt = 0; dt < 2; ++dt)
        for (int gate = 0; gate < 3; gate += 2)
            for (int i = 0; i < 9; ++i)
                for (int j = 0; j < 5; ++j)
                    for (int64_t B = 1; B <= 64; B *= 4) {
                        gdn_desc d = {B, Ts[i], Hs[j], 128, 128, dt, gate, 1.0f, 0};
                        if (i == 8 && (B > 1 || j > 0)) continue;
                        EXPECT(gdn_linattn_workspace_size(&d, (int32_t)B, &n), GDN_OK);
                        last = n;
                        d.gate = 2 - gate; /* the size covers both gate kinds */
                        EXPECT(gdn_linattn_workspace_size(&d, (int32_t)B, &n), GDN_OK);
                        if (n != last) ++failures;
                        EXPECT(gdn_linattn_workspace_size(&d, 100000, &n), GDN_OK);
                    }
    gdn_desc d = {2, 130, 4, 128, 128, GDN_BF16, GDN_GATE_CONST, 1.0f, 2}, bad;
    EXPECT(gdn_linattn_workspace_size(&d, 2, NULL), GDN_ERR_INVALID_ARG);
    EXPECT(gdn_linattn_workspace_size(NULL, 2, &n), GDN_ERR_INVALID_ARG);
    EXPECT(gdn_linattn_workspace_size(&d, -1, &n), GDN_ERR_INVALID_ARG);
    bad = d; bad.gate = GDN_GATE_CHANNEL;
    EXPECT(gdn_linattn_workspace_size(&bad, 2, &n), GDN_ERR_UNSUPPORTED);
    bad = d; bad.gate = 3;
    EXPECT(gdn_linattn_workspace_size(&bad, 2, &n), GDN_ERR_INVALID_ARG);
    bad = d; bad.hk = 3;
    EXPECT(gdn_linattn_workspace_size(&bad, 2, &n), GDN_ERR_INVALID_ARG);
    bad = d; bad.dk = 96;
    EXPECT(gdn_linattn_workspace_size(&bad, 2, &n), GDN_ERR_UNSUPPORTED);

#define CHUNK(dp, out, fin, snaps, cu, seqs, stride, ws, bytes) \
    gdn_linattn_chunk_fwd(dp, P(0), P(1), P(2), F(3), F(4), cu, seqs, stride, out, fin, snaps, ws, bytes, NULL)
    EXPECT(CHUNK(NULL, P(5), F(6), NULL, NULL, 0, 0, P(7), big), GDN_ERR_INVALID_ARG);
    EXPECT(CHUNK(&d, P(5), F(6), NULL, NULL, 0, 0, NULL, big), GDN_ERR_WORKSPACE);
    EXPECT(CHUNK(&d, P(5), F(6), NULL, NULL, 0, 0, (char *)P(7) + 16, big), GDN_ERR_WORKSPACE);
    EXPECT(CHUNK(&d, P(5), F(6), NULL, NULL, 0, 0, P(7), 16), GDN_ERR_WORKSPACE);
    EXPECT(CHUNK(&d, P(2), F(6), NULL, NULL, 0, 0, P(7), big), GDN_ERR_INVALID_ARG);
    EXPECT(CHUNK(&d, P(5), F(5), NULL, NULL, 0, 0, P(7), big), GDN_ERR_INVALID_ARG);
    EXPECT(CHUNK(&d, P(5), F(6), NULL, NULL, 0, 64, P(7), big), GDN_ERR_INVALID_ARG);
    EXPECT(CHUNK(&d, P(5), F(6), F(8), NULL, 0, 65, P(7), big), GDN_ERR_INVALID_ARG);
    EXPECT(CHUNK(&d, P(5), F(6), NULL, I(9), 2, 0, P(7), big), GDN_ERR_INVALID_ARG); /* packed: B == 1 */
    EXPECT(CHUNK(&d, (char *)P(5) + 2, F(6), NULL, NULL, 0, 0, P(7), big), GDN_ERR_INVALID_ARG);
    bad = d; bad.B = 1LL << 20; bad.T = 1LL << 20;
    EXPECT(CHUNK(&bad, P(5), F(6), NULL, NULL, 0, 0, P(7), big), GDN_ERR_UNSUPPORTED);
    bad = d; bad.B = 0;
    EXPECT(CHUNK(&bad, P(5), F(6), NULL, NULL, 0, 0, P(7), big), GDN_OK);

    EXPECT(gdn_linattn_decode_step(&d, P(0), P(1), P(2), F(3), F(4), P(5), NULL), GDN_ERR_INVALID_ARG); /* T != 1 */
    bad = d; bad.T = 1;
    EXPECT(gdn_linattn_decode_step(&bad, P(0), P(1), P(2), F(3), NULL, P(5), NULL), GDN_ERR_INVALID_ARG);
    EXPECT(gdn_linattn_decode_step(&bad, P(0), P(1), P(2), F(3), F(4), P(4), NULL), GDN_ERR_INVALID_ARG);
    bad.B = 0;
    EXPECT(gdn_linattn_decode_step(&bad, P(0), P(1), P(2), F(3), F(4), P(5), NULL), GDN_OK);

    gdn_qk_rope_desc r = {100, 4, 2, 128, 64, 0, GDN_BF16, 512, 256, 1e-6f, 0.f}, rb;
#define ROPE(dp, q, qo, ko) gdn_qk_norm_rope(dp, q, P(1), I(2), F(3), F(4), F(5), qo, ko, NULL)
    EXPECT(ROPE(NULL, P(0), P(6), P(7)), GDN_ERR_INVALID_ARG);
    EXPECT(ROPE(&r, P(0), P(6), P(6)), GDN_ERR_INVALID_ARG);
    EXPECT(ROPE(&r, P(0), P(1), P(7)), GDN_ERR_INVALID_ARG);
    EXPECT(ROPE(&r, P(0), NULL, P(7)), GDN_ERR_INVALID_ARG);
    rb = r; rb.q_stride = 500;
    EXPECT(ROPE(&rb, P(0), P(6), P(7)), GDN_ERR_INVALID_ARG);
    rb = r; rb.q_stride = 1024; /* in place needs dense rows */
    EXPECT(ROPE(&rb, P(0), P(0), P(7)), GDN_ERR_INVALID_ARG);
    rb = r; rb.rot = 72;
    EXPECT(ROPE(&rb, P(0), P(6), P(7)), GDN_ERR_UNSUPPORTED);
    rb = r; rb.head_dim = 80;
    EXPECT(ROPE(&rb, P(0), P(6), P(7)), GDN_ERR_UNSUPPORTED);
    rb = r; rb.eps = NAN;
    EXPECT(ROPE(&rb, P(0), P(6), P(7)), GDN_ERR_INVALID_ARG);
    rb = r; rb.rows = 1LL << 40; rb.q_stride = rb.k_stride = 1LL << 40;
    EXPECT(ROPE(&rb, P(0), P(6), P(7)), GDN_ERR_UNSUPPORTED);

    gdn_beam_desc b = {3, 4, 1000, 8, GDN_F32, 1000}, bb;
    for (int W = 1; W <= 64; W += 7)
        for (int V = 1; V < 2000000; V = 3 * V + 1)
            for (int K = 1; K <= 64 && K <= W * V; K += 9) {
                gdn_beam_desc x = {5, W, V, K, W & 1, V};
                EXPECT(gdn_beam_workspace_size(&x, &n), GDN_OK);
                if (n == 0 || n % 256) ++failures;
            }
    EXPECT(gdn_beam_workspace_size(&b, NULL), GDN_ERR_INVALID_ARG);
#define BEAM(dp, so, po, ws, bytes) gdn_beam_select(dp, P(0), F(1), so, po, I(4), ws, bytes, NULL)
    EXPECT(BEAM(NULL, F(2), I(3), P(5), big), GDN_ERR_INVALID_ARG);
    EXPECT(BEAM(&b, F(1), I(3), P(5), big), GDN_ERR_INVALID_ARG);
    EXPECT(BEAM(&b, F(2), I(2), P(5), big), GDN_ERR_INVALID_ARG);
    EXPECT(BEAM(&b, F(2), I(3), P(5), 8), GDN_ERR_WORKSPACE);
    EXPECT(BEAM(&b, F(2), I(3), NULL, big), GDN_ERR_WORKSPACE);
    bb = b; bb.K = 65;
    EXPECT(BEAM(&bb, F(2), I(3), P(5), big), GDN_ERR_INVALID_ARG);
    bb = b; bb.W = 1; bb.V = 4; bb.K = 5;
    EXPECT(BEAM(&bb, F(2), I(3), P(5), big), GDN_ERR_INVALID_ARG);
    bb = b; bb.W = 64; bb.V = 0x7fffffff; bb.row_stride = 0x7fffffff;
    EXPECT(BEAM(&bb, F(2), I(3), P(5), big), GDN_ERR_UNSUPPORTED);
    bb = b; bb.row_stride = 999;
    EXPECT(BEAM(&bb, F(2), I(3), P(5), big), GDN_ERR_INVALID_ARG);
    bb = b; bb.B = 0;
    EXPECT(BEAM(&bb, F(2), I(3), P(5), big), GDN_OK);

    EXPECT(gdn_state_reorder(P(0), I(1), -1, 4, 64, NULL), GDN_ERR_INVALID_ARG);
    EXPECT(gdn_state_reorder(P(0), I(1), 2, 65, 64, NULL), GDN_ERR_INVALID_ARG);
    EXPECT(gdn_state_reorder(P(0), I(1), 2, 4, 60, NULL), GDN_ERR_INVALID_ARG);
    EXPECT(gdn_state_reorder(P(0), I(0), 2, 4, 64, NULL), GDN_ERR_INVALID_ARG);
    EXPECT(gdn_state_reorder(P(0), NULL, 2, 4, 64, NULL), GDN_ERR_INVALID_ARG);
    EXPECT(gdn_state_reorder(P(0), I(1), 1LL << 40, 64, 64, NULL), GDN_ERR_UNSUPPORTED);
    EXPECT(gdn_state_reorder(NULL, NULL, 0, 4, 64, NULL), GDN_OK);
    printf("%d failures\n", failures);
    return failures != 0;
}
