// Chunkwise linear attention with a decay for each head on the 5th-generation tensor
// cores (tcgen05, TMEM, TMA): bf16 q/k/v, d_k = d_v = 128, fp32 state.  The algebra is at
// the top of linattn.cuh; chunks have 64 tokens.  Per chunk the output kernel forms, with
// fp32 accumulators in TMEM and the 128 value channels as MMA rows,
//
//     QK  = Q K^T                     64 x 64 (a 128-row product, its upper half unused)
//     D1  = S0 Q^T                    128 x 64: what the state before the chunk gives
//     D2  = V^T P^T                   128 x 64: what the chunk's own tokens give
//     dS  = (V w)^T K                 128 x 128: the state's increment
//
// with P_ij = scale 2^{G_i - G_j} QK_ij for j <= i and w_j = 2^{G - G_j}, then
// o_i = scale 2^{G_i} D1_i + D2_i and S = 2^G S0 + dS.
//
// Rounding.  P and the copy of S0 that D1 multiplies are rounded to bf16, once each,
// like the output they go into.  The state itself keeps fp32: V w is split into three
// bf16 terms (8 + 8 + 8 bits: the whole fp32 product) whose products with K add up in the
// fp32 accumulator, at the price of two more 128 x 128 x 64 products per chunk; one bf16
// term would leave the state with 2^-9 relative error.
//
// Nothing in a chunk but D1 waits for the chunk before it, so the roles run
// ahead of one another, joined by mbarriers:
//   warps 0-7    hold the state (two threads per row, 64 columns each): S0 as the bf16
//                A operand in TMEM, S = 2^G S0 + dS, and the outputs
//   warps 8-11   the gates' sums, the three terms of V w (shared memory, in the V
//                tile's own swizzled layout), P
//   warp 12      TMA loads, three chunks deep (48 KB each)
//   warp 13      issues the MMAs
// One block per SM: 201 KB of shared memory, all 512 TMEM columns.
//
// A chunk moves 64 KB (q, k, v, out): 1.5 us of an SM's share of the HBM bandwidth; its MMAs
// take about 1400 cycles (0.75 us).
#include <cudaTypedefs.h>
#include <string.h>

#include <mutex>

#include "linattn.cuh"
#include "sm100.cuh"

namespace gdn {
namespace lin {
namespace {

using namespace sm100;

constexpr int C = kChunk;  // 64 tokens per chunk
constexpr int D = 128;     // d_k = d_v
static_assert(C == 64, "tile layouts");

__device__ __forceinline__ uint8_t *align1024(unsigned char *p) {
    return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}
__device__ __forceinline__ void flag_error(int *err, int code) {
    if (err) atomicCAS(err, 0, code);
}

// A wait by a whole warp: given up by all of its lanes or by none.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

// 4 x 4 transpose of bf16 values among the 4 lanes of a quad: lane j holds row j as two
// packed pairs (low half first) and afterwards column j.
__device__ __forceinline__ void quad_transpose(uint32_t &p01, uint32_t &p23, int lane) {
    const bool b1 = lane & 2, b0 = lane & 1;
    const uint32_t r = __shfl_xor_sync(0xffffffffu, b1 ? p01 : p23, 2);
    const uint32_t a = b1 ? r : p01, b = b1 ? p23 : r;
    const uint32_t x = __shfl_xor_sync(0xffffffffu, __byte_perm(a, b, b0 ? 0x5410u : 0x7632u), 1);
    p01 = __byte_perm(a, x, b0 ? 0x3254u : 0x5410u);
    p23 = __byte_perm(b, x, b0 ? 0x3276u : 0x7610u);
}

// The gates of a chunk's 64 tokens, two per lane (tokens 2 l, 2 l + 1), in log2 units:
// G their prefix sums, after the sums of what follows them, total the sum of all.
__device__ __forceinline__ void scan_gates(float g0, float g1, int lane, float2 &G, float2 &after, float &total) {
    const float pair = g0 + g1;
    float up = pair, down = pair;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float a = __shfl_up_sync(0xffffffffu, up, o), b = __shfl_down_sync(0xffffffffu, down, o);
        if (lane >= o) up += a;
        if (lane + o < 32) down += b;
    }
    const float before = __shfl_up_sync(0xffffffffu, up, 1), behind = __shfl_down_sync(0xffffffffu, down, 1);
    G.x = (lane > 0 ? before : 0.f) + g0;
    G.y = up;
    after.y = lane < 31 ? behind : 0.f;
    after.x = after.y + g1;
    total = __shfl_sync(0xffffffffu, up, 31);
}

// Eight bf16 values times w as three bf16 terms each, x = t0 + t1 + t2 to fp32 precision.
__device__ __forceinline__ void split_terms(const uint4 &src, float w, uint4 (&t)[3]) {
    const uint32_t in[4] = {src.x, src.y, src.z, src.w};
    uint32_t o[3][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 x = __fmul2_rn(make_float2(__uint_as_float(in[i] << 16), __uint_as_float(in[i] & 0xffff0000u)),
                              make_float2(w, w));
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            o[k][i] = pack_bf16(x.x, x.y);
            if (k < 2)
                x = __fadd2_rn(x, make_float2(-__uint_as_float(o[k][i] << 16), -__uint_as_float(o[k][i] & 0xffff0000u)));
        }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) t[k] = make_uint4(o[k][0], o[k][1], o[k][2], o[k][3]);
}

// ===========================================================================
// Output kernel
// ===========================================================================
// A stage: [Q, channels 0-63][K, 0-63][Q, 64-127][K, 64-127][V, 0-63][V, 64-127], each 64
// token rows of 128 bytes (128-byte swizzle); K follows Q so that the 128-row A operand of
// QK stays inside the stage.
constexpr uint32_t kStQ = 0, kStK = 8192, kStV = 32768, kHalfQK = 16384, kHalfV = 8192, kStage = 49152;
constexpr int kStages = 3;
constexpr uint32_t kOffT = kStages * kStage;   // the three terms of V w, 16 KB each
constexpr uint32_t kOffP = kOffT + 3 * 16384;  // P, 64 rows of 128 bytes
constexpr uint32_t kOutSmem = kOffP + 8192 + 1024;
constexpr uint32_t kTmQK = 0, kTmD1 = 64, kTmD2 = 192, kTmS = 320, kTmA = 448;  // D1, D2: two buffers each
constexpr int kOutThreads = 14 * 32;
constexpr int kRing = 4;

struct __align__(16) Factors {  // (read four at a time)
    float G[C], f[C], w[C], e[C];  // prefix sums; 2^{R - G}; decay to the chunk's end; scale * decay from its start
    float2 decay;                  // of the chunk
    float ref;                     // R; NaN: the chunk's decay spans too much for one reference
};
struct OutBars {
    uint64_t full[kStages], empty[kStages];
    uint64_t qk, ds, o;       // products done
    uint64_t state, terms, p; // operands ready: S0 in TMEM, V w, P
    uint64_t drain;
};

__global__ void __launch_bounds__(kOutThreads, 1)
gdn_linattn_tc(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
               const __grid_constant__ CUtensorMap mv, const Args a, const bool fixed) {
    extern __shared__ unsigned char smem_raw[];
    uint8_t *sm = align1024(smem_raw);
    __shared__ OutBars bars;
    __shared__ Factors ring[kRing];
    __shared__ uint32_t tmem_base;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t h = blockIdx.x % a.H;
    Slot s;
    if (!locate<false>(a, blockIdx.x / a.H, s)) return;
    if (!in_bounds(s.start >= 0 && s.start + s.len <= a.rows && s.n < a.N && h < a.H, a.status)) return;
    const int nch = (int)((s.len + C - 1) / C);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        mbar_init(&bars.qk, 1);
        mbar_init(&bars.ds, 1);
        mbar_init(&bars.o, 1);
        mbar_init(&bars.state, 256);
        mbar_init(&bars.terms, 128);
        mbar_init(&bars.p, 128);
        mbar_init(&bars.drain, 1);
        fence_mbar_init();
    }
    if (warp == 13) {
        tmem_alloc(&tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_base;
    bool ok = true;
    int issued = 0;  // (warp 12) chunks whose loads are issued

    if (warp < 8) {
        // ------------------------------------------------------------------
        // The state and the outputs: value channel v, key channels [64 hf, 64 hf + 64) of
        // the state, tokens [32 hf, 32 hf + 32) of the outputs.
        // ------------------------------------------------------------------
        const int qd = warp & 3, hf = warp >> 2, v = qd * 32 + lane;
        const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
        const int64_t srow = (int64_t)v * D + 64 * hf;
        const float *from = s.nseg > 1 ? a.states + (s.ss * a.H + h) * (int64_t)(D * D)
                                       : (a.h0 ? a.h0 + (s.n * a.H + h) * (int64_t)(D * D) : nullptr);
        float S[64];
        if (from) {
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
                const float4 t = *reinterpret_cast<const float4 *>(from + srow + c);
                S[c] = t.x; S[c + 1] = t.y; S[c + 2] = t.z; S[c + 3] = t.w;
            }
        } else {
#pragma unroll
            for (int c = 0; c < 64; ++c) S[c] = 0.f;
        }
        auto publish = [&] {  // S0 as bf16 pairs: this thread's 32 columns of the A operand
            uint32_t w[16];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = pack_bf16(S[32 * q + 2 * e], S[32 * q + 2 * e + 1]);
                tmem_st16u(tm + lane_off + kTmA + 32 * hf + 16 * q, w);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&bars.state);
        };
        publish();
        const int32_t kc = a.n_snap > 0 ? (int32_t)(a.snap_stride / C) : 0;  // chunks between snapshots
        const int64_t c0 = s.pos / C;
        int32_t snap_left = kc > 0 ? kc - (int32_t)(c0 % kc) : 0;
        int64_t snap_idx = kc > 0 ? c0 / kc : 0;
        const int j4 = lane & 3;
        const int64_t tstride = a.H * D;
        __nv_bfloat16 *op = static_cast<__nv_bfloat16 *>(a.out) + ((s.start + 32 * hf + j4) * a.H + h) * D + (v - j4);
        for (int c = 0; c < nch && ok; ++c, op += C * tstride) {
            const uint32_t par = c & 1;
            const Factors &fac = ring[c % kRing];
            ok = warp_wait(&bars.terms, par);  // (the factors were written before)
            ok = ok && warp_wait(&bars.ds, par);
            if (!ok) break;
            tc_fence_after();
            const float2 d = fac.decay;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float x[16];
                tmem_ld16(tm + lane_off + kTmS + 64 * hf + 16 * q, x);
                tmem_wait_ld();
#pragma unroll
                for (int t = 0; t < 16; t += 2) {
                    const float2 s0 = make_float2(S[16 * q + t], S[16 * q + t + 1]);
                    const float2 lo = __ffma2_rn(make_float2(d.y, d.y), s0, make_float2(x[t], x[t + 1]));
                    const float2 r = __ffma2_rn(make_float2(d.x, d.x), s0, lo);
                    S[16 * q + t] = r.x;
                    S[16 * q + t + 1] = r.y;
                }
            }
            publish();  // of the next chunk (this chunk's D1 is done: it was issued before dS)
            if (kc > 0 && --snap_left == 0) {
                snap_left = kc;
                // a snapshot is whole chunks from the sequence's start
                if (snap_idx < a.n_snap) {
                    float *dst = a.snaps + ((s.n * a.n_snap + snap_idx) * a.H + h) * (int64_t)(D * D) + srow;
#pragma unroll
                    for (int cc = 0; cc < 64; cc += 4)
                        *reinterpret_cast<float4 *>(dst + cc) = make_float4(S[cc], S[cc + 1], S[cc + 2], S[cc + 3]);
                }
                ++snap_idx;
            }
            ok = warp_wait(&bars.o, par);
            if (!ok) break;
            tc_fence_after();
            const int L = (int)(s.len - (int64_t)c * C < C ? s.len - (int64_t)c * C : C);
            const float4 *e4 = reinterpret_cast<const float4 *>(fac.e + 32 * hf);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float x[16], y[16];
                tmem_ld16(tm + lane_off + kTmD1 + 64 * par + 32 * hf + 16 * q, x);
                tmem_ld16(tm + lane_off + kTmD2 + 64 * par + 32 * hf + 16 * q, y);
                tmem_wait_ld();
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const float4 e = e4[4 * q + b];
                    const float2 r01 = __ffma2_rn(make_float2(x[4 * b], x[4 * b + 1]), make_float2(e.x, e.y),
                                                  make_float2(y[4 * b], y[4 * b + 1]));
                    const float2 r23 = __ffma2_rn(make_float2(x[4 * b + 2], x[4 * b + 3]), make_float2(e.z, e.w),
                                                  make_float2(y[4 * b + 2], y[4 * b + 3]));
                    // four tokens of this channel -> four channels of one token
                    uint32_t p01 = pack_bf16(r01.x, r01.y), p23 = pack_bf16(r23.x, r23.y);
                    quad_transpose(p01, p23, lane);
                    const int t = 16 * q + 4 * b;
                    if (32 * hf + t + j4 < L) *reinterpret_cast<uint2 *>(op + t * tstride) = make_uint2(p01, p23);
                }
            }
        }
        if (ok && a.final_state && s.j == s.nseg - 1) {
            float *dst = a.final_state + (s.n * a.H + h) * (int64_t)(D * D) + srow;
#pragma unroll
            for (int c = 0; c < 64; c += 4)
                *reinterpret_cast<float4 *>(dst + c) = make_float4(S[c], S[c + 1], S[c + 2], S[c + 3]);
        }
    } else if (warp < 12) {
        // ------------------------------------------------------------------
        // Gates, V w and P.  P's 64 rows belong to the first two warps (rows 32 w ..), of
        // which the second has twice the work: the V w tile is dealt out the other way.
        // ------------------------------------------------------------------
        const int w = warp - 8, t128 = tid - 256;
        const int part0 = w == 0 ? 0 : (w == 1 ? 8 : (w == 2 ? 12 : 22)), parts = w == 0 ? 8 : (w == 1 ? 4 : 10);
        const float gh = fixed ? a.g[h] * kLog2e : 0.f;
        auto load_gate = [&](int c) {
            const int64_t t = (int64_t)c * C + 2 * lane;
            float2 g = make_float2(0.f, 0.f);
            if (t < s.len) g.x = fixed ? gh : a.g[(s.start + t) * a.H + h] * kLog2e;
            if (t + 1 < s.len) g.y = fixed ? gh : a.g[(s.start + t + 1) * a.H + h] * kLog2e;
            return g;
        };
        float2 g = make_float2(0.f, 0.f), fixed_decay = make_float2(0.f, 0.f);
        if (w == 0 && nch > 0) {
            g = load_gate(0);
            if (fixed) fixed_decay = exp2_pair((double)a.g[h] * 1.4426950408889634074 * C);
        }
        uint8_t *T = sm + kOffT, *P = sm + kOffP;
        // the blocks above the diagonal stay zero
        if (w == 0)
            for (int j = 4; j < 8; ++j)
                *reinterpret_cast<uint4 *>(P + sw128_offset(lane, j)) = make_uint4(0u, 0u, 0u, 0u);
        for (int c = 0; c < nch && ok; ++c) {
            const int stage = c % kStages;
            const uint32_t par = c & 1;
            uint8_t *st = sm + stage * kStage;
            Factors &fac = ring[c % kRing];
            const int L = (int)(s.len - (int64_t)c * C < C ? s.len - (int64_t)c * C : C);
            if (w == 0) {
                float2 G, after;
                float total;
                scan_gates(g.x, g.y, lane, G, after, total);
                // One reference R in the middle keeps both factors of 2^{G_i - G_j} inside 2^+-60.
                const float ref = total > -120.f ? 0.5f * total : __int_as_float(0x7fc00000);
                *reinterpret_cast<float2 *>(&fac.G[2 * lane]) = G;
                *reinterpret_cast<float2 *>(&fac.f[2 * lane]) = make_float2(ex2(ref - G.x), ex2(ref - G.y));
                *reinterpret_cast<float2 *>(&fac.w[2 * lane]) = make_float2(ex2(after.x), ex2(after.y));
                *reinterpret_cast<float2 *>(&fac.e[2 * lane]) = make_float2(a.scale * ex2(G.x), a.scale * ex2(G.y));
                if (lane == 0) {
                    fac.ref = ref;
                    fac.decay = !fixed ? make_float2(ex2(total), 0.f)
                                       : (L == C ? fixed_decay : exp2_pair((double)a.g[h] * 1.4426950408889634074 * L));
                }
                if (c + 1 < nch) g = load_gate(c + 1);
            }
            named_bar_sync(1, 128);
            ok = warp_wait(&bars.full[stage], (c / kStages) & 1);
            // the terms' buffer: the previous chunk's dS has read it
            if (c > 0) ok = ok && warp_wait(&bars.ds, par ^ 1);
            if (!ok) break;
            if (L < C) {  // rows behind the sequence: whatever lies there stays out of the sums
                for (int i = t128; i < 64 * 8; i += 128) {
                    const uint32_t at = (uint32_t)i * 16;
                    if ((i >> 3) >= L) {
                        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4 *>(st + kStK + at) = z;
                        *reinterpret_cast<uint4 *>(st + kStK + kHalfQK + at) = z;
                        *reinterpret_cast<uint4 *>(st + kStV + at) = z;
                        *reinterpret_cast<uint4 *>(st + kStV + kHalfV + at) = z;
                    }
                }
            }
#pragma unroll 2
            for (int i = 0; i < parts; ++i) {
                const uint32_t at = (uint32_t)((part0 + i) * 32 + lane) * 16;  // 16-byte piece of the V tile
                const int row = (at >> 7) & 63;
                uint4 t[3];
                if (row < L) {
                    split_terms(*reinterpret_cast<const uint4 *>(st + kStV + at), fac.w[row], t);
                } else {
#pragma unroll
                    for (int k = 0; k < 3; ++k) t[k] = make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int k = 0; k < 3; ++k) *reinterpret_cast<uint4 *>(T + k * 16384 + at) = t[k];
            }
            fence_async_smem();
            mbar_arrive(&bars.terms);
            if (c > 0) ok = warp_wait(&bars.o, par ^ 1);  // P's buffer: the previous chunk's D2 has read it
            ok = ok && warp_wait(&bars.qk, par);
            if (!ok) break;
            tc_fence_after();
            if (w < 2) {
                const int i = 32 * w + lane;
                const float ref = fac.ref, Gi = fac.G[i];
                const bool one_ref = ref == ref;
                const float ei = a.scale * ex2(one_ref ? Gi - ref : 0.f);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (q > 2 * w + 1) break;
                    float x[16];
                    tmem_ld16(tm + ((uint32_t)(w * 32) << 16) + kTmQK + 16 * q, x);
                    tmem_wait_ld();
                    uint32_t o[8];
                    if (one_ref) {
                        const float4 *f4 = reinterpret_cast<const float4 *>(fac.f + 16 * q);
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            const float4 f = f4[b];
                            const float ff[4] = {f.x, f.y, f.z, f.w};
                            float y[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) y[e] = 16 * q + 4 * b + e <= i ? (x[4 * b + e] * ei) * ff[e] : 0.f;
                            o[2 * b] = pack_bf16(y[0], y[1]);
                            o[2 * b + 1] = pack_bf16(y[2], y[3]);
                        }
                    } else {
                        const float4 *G4 = reinterpret_cast<const float4 *>(fac.G + 16 * q);
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            const float4 G = G4[b];
                            const float gg[4] = {G.x, G.y, G.z, G.w};
                            float y[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                y[e] = 16 * q + 4 * b + e <= i ? x[4 * b + e] * (ei * ex2(Gi - gg[e])) : 0.f;
                            o[2 * b] = pack_bf16(y[0], y[1]);
                            o[2 * b + 1] = pack_bf16(y[2], y[3]);
                        }
                    }
                    *reinterpret_cast<uint4 *>(P + sw128_offset(i, 2 * q)) = make_uint4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint4 *>(P + sw128_offset(i, 2 * q + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
                }
            }
            tc_fence_before();
            fence_async_smem();
            mbar_arrive(&bars.p);
        }
    } else if (warp == 12) {
        // ------------------------------------------------------------------
        // Loads
        // ------------------------------------------------------------------
        if (lane == 0) {
            prefetch_tmap(&mq);
            prefetch_tmap(&mk);
            prefetch_tmap(&mv);
            const int32_t hq = (int32_t)(h / (a.H / a.Hk)), hv = (int32_t)h;
            for (int c = 0; c < nch; ++c) {
                const int stage = c % kStages;
                if (c >= kStages && !(ok = mbar_wait(&bars.empty[stage], ((c / kStages) & 1) ^ 1))) break;
                uint8_t *st = sm + stage * kStage;
                uint64_t *bar = &bars.full[stage];
                const int32_t row = (int32_t)(s.start + (int64_t)c * C);
                mbar_arrive_expect_tx(bar, kStage);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    tma_load_3d(st + kStQ + i * kHalfQK, &mq, 64 * i, hq, row, bar);
                    tma_load_3d(st + kStK + i * kHalfQK, &mk, 64 * i, hq, row, bar);
                    tma_load_3d(st + kStV + i * kHalfV, &mv, 64 * i, hv, row, bar);
                }
                issued = c + 1;
            }
        }
        ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
    } else {
        // ------------------------------------------------------------------
        // MMAs
        // ------------------------------------------------------------------
        const uint32_t base = smem_u32(sm);
        auto issue_qk = [&](int c) {
            const uint32_t st = base + (c % kStages) * kStage;
            const uint64_t aq = sdesc_sw128(st + kStQ, 16, 1024), bk = sdesc_sw128(st + kStK, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                const uint64_t at = (uint64_t)(((kk >> 2) * kHalfQK + (kk & 3) * 32) >> 4);
                mma_bf16_ss(tm + kTmQK, aq + at, bk + at, idesc_bf16(128, 64, 0, 0), kk > 0);
            }
            mma_commit_warp(&bars.qk);
        };
        if (nch > 0) {
            ok = warp_wait(&bars.full[0], 0);
            if (ok) issue_qk(0);
        }
        for (int c = 0; c < nch && ok; ++c) {
            const int stage = c % kStages;
            const uint32_t par = c & 1, st = base + stage * kStage;
            ok = warp_wait(&bars.state, par);
            if (!ok) break;
            tc_fence_after();
            {  // D1 (its buffer and dS's are free: the state of chunk c was published after their last reads)
                const uint64_t bq = sdesc_sw128(st + kStQ, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_bf16_ts(tm + kTmD1 + 64 * par, tm + kTmA + kk * 8,
                                bq + (uint64_t)(((kk >> 2) * kHalfQK + (kk & 3) * 32) >> 4), idesc_bf16(128, 64, 0, 0),
                                kk > 0);
            }
            ok = warp_wait(&bars.terms, par);
            if (!ok) break;
            tc_fence_after();
            {  // dS
                const uint64_t bk = sdesc_sw128(st + kStK, kHalfQK, 1024);
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    const uint64_t at = sdesc_sw128(base + kOffT + k * 16384, kHalfV, 1024);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_bf16_ss(tm + kTmS, at + (uint64_t)((kk * 2048) >> 4), bk + (uint64_t)((kk * 2048) >> 4),
                                    idesc_bf16(128, 128, 1, 1), k > 0 || kk > 0);
                }
                mma_commit_warp(&bars.ds);
            }
            ok = warp_wait(&bars.p, par);
            if (!ok) break;
            tc_fence_after();
            {  // D2
                const uint64_t av = sdesc_sw128(st + kStV, kHalfV, 1024), bp = sdesc_sw128(base + kOffP, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_bf16_ss(tm + kTmD2 + 64 * par, av + (uint64_t)((kk * 2048) >> 4), bp + (uint64_t)((kk * 32) >> 4),
                                idesc_bf16(128, 64, 1, 0), kk > 0);
                mma_commit_warp(&bars.o);
                mma_commit_warp(&bars.empty[stage]);
            }
            if (c + 1 < nch) {
                ok = warp_wait(&bars.full[(c + 1) % kStages], ((c + 1) / kStages) & 1);
                if (ok) issue_qk(c + 1);
            }
        }
    }
    __syncwarp();
    if (!ok) {
        // A wait gave up: record it.  Every other role's next wait gives up too (it waits,
        // directly or not, for this one), so all of them get here.
        if (lane == 0) flag_error(a.status, GDN_DEV_TIMEOUT_SCAN);
        if (warp == 12 && lane == 0)
            for (int j = issued > kStages ? issued - kStages : 0; j < issued; ++j)
                mbar_wait(&bars.full[j % kStages], (j / kStages) & 1);
        if (warp == 13) {
            mma_commit_warp(&bars.drain);
            warp_wait(&bars.drain, 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 13) tmem_dealloc(tm, 512);
}

// ===========================================================================
// State kernel: U of a segment (not its sequence's last) and its decay
// ===========================================================================
// Backwards from the segment's end, so that a token's weight is the sum of the gates after
// it and the products add up in TMEM without a rescale; it stops where nothing earlier
// reaches the end.  Warps 0-7: gates and V w (two buffers); warp 8: loads and MMAs.
constexpr uint32_t kSsK = 0, kSsV = 16384, kSsStage = 32768;
constexpr int kSsStages = 3;
constexpr uint32_t kSsOffT = kSsStages * kSsStage, kSsTerms = 3 * 16384;
constexpr uint32_t kStateSmem = kSsOffT + 2 * kSsTerms + 1024;
constexpr int kStateThreads = 9 * 32;

struct StateBars {
    uint64_t full[kSsStages], terms[2], ds[2], drain;
};

__global__ void __launch_bounds__(kStateThreads, 1)
gdn_linattn_state_tc(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const Args a,
                     const bool fixed) {
    extern __shared__ unsigned char smem_raw[];
    uint8_t *sm = align1024(smem_raw);
    __shared__ StateBars bars;
    __shared__ uint32_t tmem_base;
    __shared__ int s_last;  // index of the last chunk to add, once known
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t h = blockIdx.x % a.H;
    Slot s;
    if (!locate<true>(a, blockIdx.x / a.H, s) || s.nseg < 2 || s.j == s.nseg - 1) return;
    if (!in_bounds(s.start >= 0 && s.start + s.len <= a.rows && s.n < a.N && s.ss < a.sslots && s.len % C == 0, a.status))
        return;
    const int nch = (int)(s.len / C);
    if (tid == 0) {
        for (int i = 0; i < kSsStages; ++i) mbar_init(&bars.full[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.terms[i], 256);
            mbar_init(&bars.ds[i], 1);
        }
        mbar_init(&bars.drain, 1);
        s_last = nch - 1;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(&tmem_base, 128);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_base;
    bool ok = true;
    int issued = 0, waited = 0;  // (warp 8) loads
    if (warp < 8) {
        const float gh = fixed ? a.g[h] * kLog2e : 0.f;
        auto load_gate = [&](int i) {  // chunk i from the segment's end
            if (fixed) return make_float2(gh, gh);
            const float *p = a.g + (s.start + (int64_t)(nch - 1 - i) * C + 2 * lane) * a.H + h;
            return make_float2(p[0] * kLog2e, p[a.H] * kLog2e);
        };
        float2 g = load_gate(0);
        float after_chunk = 0.f;
        const int row = tid >> 3;  // the V rows of this thread: row and row + 32
        int i = 0;
        for (; i < nch; ++i) {
            const int stage = i % kSsStages, buf = i & 1;
            const uint8_t *V = sm + stage * kSsStage + kSsV;
            uint8_t *T = sm + kSsOffT + buf * kSsTerms;
            float2 G, after;
            float total;
            scan_gates(g.x, g.y, lane, G, after, total);
            const float w0 = ex2(after.x + after_chunk), w1 = ex2(after.y + after_chunk);
            float wr[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = row + 32 * k;
                const float x = __shfl_sync(0xffffffffu, w0, r >> 1), y = __shfl_sync(0xffffffffu, w1, r >> 1);
                wr[k] = r & 1 ? y : x;
            }
            after_chunk += total;
            const bool last = i == nch - 1 || after_chunk <= kDead;  // (the same in every warp)
            if (!last) g = load_gate(i + 1);
            ok = warp_wait(&bars.full[stage], (i / kSsStages) & 1);
            if (i >= 2) ok = ok && warp_wait(&bars.ds[buf], ((i >> 1) & 1) ^ 1);
            if (!ok) break;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t at = (uint32_t)(tid + 256 * k) * 16;
                uint4 t[3];
                split_terms(*reinterpret_cast<const uint4 *>(V + at), wr[k & 1], t);
#pragma unroll
                for (int m = 0; m < 3; ++m) *reinterpret_cast<uint4 *>(T + m * 16384 + at) = t[m];
            }
            if (last && tid == 0) s_last = i;
            fence_async_smem();
            mbar_arrive(&bars.terms[buf]);
            if (last) break;
        }
        if (ok) {
            ok = warp_wait(&bars.ds[i & 1], (i >> 1) & 1);  // the last chunk's products, and all before
            tc_fence_after();
        }
        if (ok) {
            const int qd = warp & 3, hf = warp >> 2, v = qd * 32 + lane;
            float *U = a.states + (s.ss * a.H + h) * (int64_t)(D * D) + (int64_t)v * D + 64 * hf;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float x[16];
                tmem_ld16(tm + ((uint32_t)(qd * 32) << 16) + 64 * hf + 16 * q, x);
                tmem_wait_ld();
#pragma unroll
                for (int t = 0; t < 16; t += 4)
                    *reinterpret_cast<float4 *>(U + 16 * q + t) = make_float4(x[t], x[t + 1], x[t + 2], x[t + 3]);
            }
            // the segment's decay (once it is past kDead, how far past does not matter)
            if (tid == 0)
                a.tot[s.ss * a.H + h] = fixed ? (double)a.g[h] * 1.4426950408889634074 * (double)s.len : (double)after_chunk;
        }
    } else {
        const uint32_t base = smem_u32(sm);
        const int32_t hq = (int32_t)(h / (a.H / a.Hk)), hv = (int32_t)h;
        auto load = [&](int i) {
            const int stage = i % kSsStages;
            if (lane == 0) {
                uint8_t *st = sm + stage * kSsStage;
                uint64_t *bar = &bars.full[stage];
                const int32_t r = (int32_t)(s.start + (int64_t)(nch - 1 - i) * C);
                mbar_arrive_expect_tx(bar, kSsStage);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    tma_load_3d(st + kSsK + k * 8192, &mk, 64 * k, hq, r, bar);
                    tma_load_3d(st + kSsV + k * 8192, &mv, 64 * k, hv, r, bar);
                }
            }
            issued = i + 1;
        };
        for (int i = 0; i < 2 && i < nch; ++i) load(i);
        for (int i = 0; i < nch; ++i) {
            const int stage = i % kSsStages, buf = i & 1;
            ok = warp_wait(&bars.full[stage], (i / kSsStages) & 1);
            if (!ok) break;
            waited = i + 1;
            ok = warp_wait(&bars.terms[buf], (i >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint64_t bk = sdesc_sw128(base + stage * kSsStage + kSsK, 8192, 1024);
#pragma unroll
            for (int m = 0; m < 3; ++m) {
                const uint64_t at = sdesc_sw128(base + kSsOffT + buf * kSsTerms + m * 16384, 8192, 1024);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_bf16_ss(tm, at + (uint64_t)((kk * 2048) >> 4), bk + (uint64_t)((kk * 2048) >> 4),
                                idesc_bf16(128, 128, 1, 1), i > 0 || m > 0 || kk > 0);
            }
            mma_commit_warp(&bars.ds[buf]);
            if (*(volatile int *)&s_last == i) break;
            if (i + 2 < nch) {  // into the stage of chunk i - 1
                if (i >= 1) ok = warp_wait(&bars.ds[buf ^ 1], ((i - 1) >> 1) & 1);
                if (!ok) break;
                load(i + 2);
            }
        }
    }
    __syncwarp();
    if (!ok) {
        if (lane == 0) flag_error(a.status, GDN_DEV_TIMEOUT_PREP);
        if (warp == 8) {
            mma_commit_warp(&bars.drain);
            warp_wait(&bars.drain, 0);
        }
    }
    if (warp == 8)  // loads still in flight (chunks that the early end left out)
        for (int j = waited; j < issued; ++j) warp_wait(&bars.full[j % kSsStages], (j / kSsStages) & 1);
    tc_fence_before();
    __syncthreads();
    if (warp == 8) tmem_dealloc(tm, 128);
}

// ===========================================================================
// Host side
// ===========================================================================
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        cudaDriverEntryPointQueryResult q;
        void *p = nullptr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// A (rows, H, 128) bf16 tensor in tiles of 64 tokens x 64 channels of one head, 128-byte swizzle.
gdn_status make_map(CUtensorMap *m, const void *base, int64_t rows, int64_t H) {
    auto enc = tensor_map_encoder();
    if (!enc) return fail(GDN_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)H * D * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)C}, es[3] = {1, 1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(GDN_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return GDN_OK;
}

}  // namespace

gdn_status launch_tc(const Plan &p, const Args &a, cudaStream_t s) {
    const int64_t grid = p.slots * p.H, sgrid = p.sslots * p.H;
    if (grid > 0x7fffffffLL || sgrid > 0x7fffffffLL) return fail(GDN_ERR_UNSUPPORTED, "grid too large");
    CUtensorMap mq, mk, mv;
    memset(&mq, 0, sizeof mq);
    memset(&mk, 0, sizeof mk);
    memset(&mv, 0, sizeof mv);
    gdn_status st = GDN_OK;
    if (p.rows > 0) {
        if ((st = make_map(&mq, a.q, p.rows, a.Hk)) != GDN_OK) return st;
        if ((st = make_map(&mk, a.k, p.rows, a.Hk)) != GDN_OK) return st;
        if ((st = make_map(&mv, a.v, p.rows, p.H)) != GDN_OK) return st;
    }
    static const cudaError_t attr = [] {
        const cudaError_t e = cudaFuncSetAttribute(gdn_linattn_tc, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kOutSmem);
        return e != cudaSuccess ? e
                                : cudaFuncSetAttribute(gdn_linattn_state_tc, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       (int)kStateSmem);
    }();
    if (attr != cudaSuccess) return fail(GDN_ERR_CUDA, "kernel attributes: %s", cudaGetErrorString(attr));
    if (sgrid > 0) {
        {
            log_launch("gdn_linattn_state_tc", dim3((unsigned)sgrid), dim3(kStateThreads), kStateSmem);
            LaunchScope ls("gdn_linattn_state_tc", s);
            gdn_linattn_state_tc<<<(unsigned)sgrid, kStateThreads, kStateSmem, s>>>(mk, mv, a, p.fixed_gate);
        }
        if ((st = check_launch("gdn_linattn_state_tc")) != GDN_OK) return st;
        if ((st = launch_combine(p, a, s)) != GDN_OK) return st;
    }
    {
        log_launch("gdn_linattn_tc", dim3((unsigned)grid), dim3(kOutThreads), kOutSmem);
        LaunchScope ls("gdn_linattn_tc", s);
        gdn_linattn_tc<<<(unsigned)grid, kOutThreads, kOutSmem, s>>>(mq, mk, mv, a, p.fixed_gate);
    }
    return check_launch("gdn_linattn_tc");
}

}  // namespace lin
}  // namespace gdn
