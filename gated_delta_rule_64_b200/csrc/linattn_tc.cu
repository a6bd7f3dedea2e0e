// Chunkwise linear attention with a decay for each head on the 5th-generation tensor
// cores (tcgen05, TMEM, TMA): bf16 q/k/v, d_k = d_v = 128, fp32 state.  The algebra is at
// the top of linattn.cuh; chunks have 64 tokens.  Per chunk the output kernel forms, with
// fp32 accumulators in TMEM and the 128 value channels as MMA rows,
//
//     QK  = Q K^T                     64 x 64
//     O   = S0 Q^T + V^T P^T          128 x 64 (one accumulator)
//     dS  = (V w)^T K                 128 x 128: the state's increment
//
// with w_j = 2^{G - G_j}, P_ij = 2^{-m - G_j} QK_ij for j <= i and 2^{-m} S0 in the place of S0;
// then o_i = scale 2^{m + G_i} O_i and S = 2^G S0 + dS.  m, half of the chunk's decay rounded to
// a whole number, keeps the factors within 2^60 of 1 for decays down to 2^-120 (and so the
// sums of q k v in range up to 2^67), and as a power of two it rounds nothing.  Where the decay
// is below that, m = 0 and P_ij = scale 2^{G_i - G_j} QK_ij, and the Q that S0 multiplies is
// scaled by scale 2^{G_i} in place (one more rounding to bf16, of that product only): slower, so
// only for those (taken from 2^-60 on, by one head of sixteen with a fixed decay, it held up a
// sequence of 262,144 tokens: 940 us in this kernel against 820).
//
// Rounding.  P and the copy of S0 that Q multiplies are rounded to bf16, once each,
// like the output they go into.  The state itself keeps fp32: V w is split into three
// bf16 terms (8 + 8 + 8 bits: the whole fp32 product) whose products with K add up in the
// fp32 accumulator, at the price of two more 128 x 128 x 64 products per chunk; one bf16
// term would leave the state with 2^-9 relative error.
//
// The roles run ahead of one another, joined by mbarriers:
//   warps 0-7    hold the state (two threads per row, 64 columns each): S = 2^G S0 + dS, its
//                bf16 copy as the A operand of S0 Q^T in TMEM; they turn O into token rows
//   warps 8-11   the three terms of V w, 32 value channels a warp, as the A operand of dS in
//                TMEM (two buffers): transposed on the way from shared memory (ldmatrix)
//                into the fragment layout that a 16-lane TMEM store takes
//   warps 12-15  P, 16 query tokens a warp (a 64-row product leaves 16 rows in each TMEM
//                quarter), through the fragment layout too: TMEM to stmatrix
//   warp 16      issues the MMAs of dS, warp 17 those of QK and O: a wait of one does not hold
//                up the other's products (one warp for all of them left the tensor pipe idle
//                half of the time, at about 200 cycles a wait)
//   warp 18      stores the outputs
//   warp 19      TMA loads (three stages of 48 KB) and the factors that come from the gates
// One block per SM: 208 KB of shared memory, all 512 TMEM columns.
//
// The loops of the roles are kept short on purpose: every scheduler runs a warp of each, and
// with them unrolled (about 40 KB of code) the instruction caches, not the tensor pipe, set
// the pace: 2.9 us a chunk, 0.36 instructions issued per cycle and scheduler.
//
// A chunk moves 64 KB (q, k, v, out): 1.5 us of an SM's share of the HBM bandwidth.  Its MMAs
// take about 1500 cycles (measured alone: 37 cycles for 128 x 64 x 16 with A in TMEM, 54 with
// A in shared memory, 69 for 128 x 128 x 16).  Measured: one sequence of 262,144 tokens and 16
// heads, 800 us at 1,965 MHz (1.8 us a chunk and SM, 5.4 TB/s); a call in a steady loop, which the
// power cap holds at 1,410 MHz, takes 1,100 us instead of 930, so a chunk's chain of products and
// the warps' work between them set the pace, not HBM.  4 sequences of 4,096 tokens, 64 us (128
// blocks of 32 chunks, and the start).
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

// Fragments: a 16 x 8k block over a warp, lane l holding rows l / 4 and l / 4 + 8.
// Store of 16 TMEM lanes: repeat n covers columns 4 n .. 4 n + 3, lane l's word of column
// 4 n + l % 4 of row l / 4 in r[2 n], of row l / 4 + 8 in r[2 n + 1].
// Over 8 columns.
__device__ __forceinline__ void tmem_st_frag8(uint32_t taddr, const uint32_t (&r)[4]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3])
                 : "memory");
}
// Load of 16 TMEM lanes: lane l holds columns 8 n + 2 (l % 4), + 1 of row l / 4 in
// x[4 n], x[4 n + 1], of row l / 4 + 8 in x[4 n + 2], x[4 n + 3].  Over 16 columns,
__device__ __forceinline__ void tmem_ld_frag16(uint32_t taddr, float (&x)[8]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r[i]);
}
// over 32 columns.
__device__ __forceinline__ void tmem_ld_frag32(uint32_t taddr, float (&x)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(r[i]);
}
// Four 8 x 8 b16 matrices, transposed: lanes 8 m .. 8 m + 7 give the row addresses of
// matrix m; lane l receives (column l / 4, rows 2 (l % 4), + 1) of it in r[m].
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void stsm_x4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

__device__ __forceinline__ void stsm_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}

// 32 lanes x 32 columns, 32 consecutive columns per thread.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&x)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(r[i]);
}
// Asynchronous copy of one float to shared memory (zero where `on` is false: nothing is read).
__device__ __forceinline__ void async_copy4(float *dst, const float *src, bool on) {
    const int bytes = on ? 4 : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Registers per thread of the calling warpgroup from here on.
template <int N> __device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Four MMAs of a K loop in one go, by one elected lane: operands A_STEP / B_STEP apart (bytes / 16
// of a shared-memory operand, columns of one in TMEM); the first adds to D if `add`, the
// others always.  (The issuing warp shares its scheduler with four busy ones, so the
// instructions around each MMA count: with an election and a predicate of its own for
// every MMA the warp needed about 80 cycles each.)
template <int A_STEP, int B_STEP>
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p, q, t;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "setp.ne.b32 q, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "add.u32 a1, %1, %5;\n\tadd.u32 a2, %1, 2 * %5;\n\tadd.u32 a3, %1, 3 * %5;\n\t"
        "add.u64 b1, %2, %6;\n\tadd.u64 b2, %2, 2 * %6;\n\tadd.u64 b3, %2, 3 * %6;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, q;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add), "n"(A_STEP), "n"(B_STEP)
        : "memory");
}
template <int A_STEP, int B_STEP>
__device__ __forceinline__ void mma4_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p, q, t;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "setp.ne.b32 q, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "add.u64 a1, %1, %5;\n\tadd.u64 a2, %1, 2 * %5;\n\tadd.u64 a3, %1, 3 * %5;\n\t"
        "add.u64 b1, %2, %6;\n\tadd.u64 b2, %2, 2 * %6;\n\tadd.u64 b3, %2, 3 * %6;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, q;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add), "n"(A_STEP), "n"(B_STEP)
        : "memory");
}

// Two bf16 values (low half first) times their weights, cut into three bf16 pairs whose sum is the
// fp32 product exactly: 24 significant bits are eight, eight and eight, each cut off.
__device__ __forceinline__ void split_terms(uint32_t v, float2 w, uint32_t &t0, uint32_t &t1, uint32_t &t2) {
    const float2 x = __fmul2_rn(make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)), w);
    const uint32_t x0 = __float_as_uint(x.x), x1 = __float_as_uint(x.y);
    t0 = __byte_perm(x0, x1, 0x7632);
    const float2 y = __fadd2_rn(x, make_float2(-__uint_as_float(x0 & 0xffff0000u), -__uint_as_float(x1 & 0xffff0000u)));
    const uint32_t y0 = __float_as_uint(y.x), y1 = __float_as_uint(y.y);
    t1 = __byte_perm(y0, y1, 0x7632);
    const float2 z = __fadd2_rn(y, make_float2(-__uint_as_float(y0 & 0xffff0000u), -__uint_as_float(y1 & 0xffff0000u)));
    t2 = __byte_perm(__float_as_uint(z.x), __float_as_uint(z.y), 0x7632);
}

// The three terms of V w for 16 value channels and 16 tokens, in the fragment layout of the
// TMEM stores.  addr: this lane's row for ldmatrix, of the matrices (tokens, channels) = (0-7,
// 0-7), (0-7, 8-15), (8-15, 0-7), (8-15, 8-15); w: the tokens' weights.
__device__ __forceinline__ void channel_terms(uint32_t addr, const float *w, int lane, uint32_t (&t0)[4], uint32_t (&t1)[4],
                                              uint32_t (&t2)[4]) {
    uint32_t r[4];
    ldsm_x4_trans(addr, r);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const float2 f = *reinterpret_cast<const float2 *>(w + 8 * m + 2 * (lane & 3));
#pragma unroll
        for (int e = 0; e < 2; ++e) split_terms(r[2 * m + e], f, t0[2 * m + e], t1[2 * m + e], t2[2 * m + e]);
    }
}
// That lane's row address for tokens `first` .. of a V half tile (64 channels) and the channels
// from 16-byte piece `piece` on (first: a multiple of 8).
__device__ __forceinline__ uint32_t terms_address(uint32_t half, int piece, int first, int lane) {
    const int row = first + (lane & 7) + ((lane >> 4) << 3), p = piece + ((lane >> 3) & 1);
    return half + (uint32_t)row * 128u + (((uint32_t)p ^ (uint32_t)(row & 7)) << 4);
}

// ===========================================================================
// Output kernel
// ===========================================================================
// A stage: [Q, channels 0-63][K, 0-63][Q, 64-127][K, 64-127][V, 0-63][V, 64-127], each 64
// token rows of 128 bytes (128-byte swizzle).
constexpr uint32_t kStQ = 0, kStK = 8192, kStV = 32768, kHalfQK = 16384, kHalfV = 8192, kStage = 49152;
constexpr int kStages = 3;
constexpr uint32_t kOffP = kStages * kStage;   // P, 64 rows of 128 bytes; two buffers
constexpr uint32_t kOffO = kOffP + 2 * 8192;   // outputs, two halves of 64 rows of 128 bytes; two buffers
constexpr uint32_t kOutSmem = kOffO + 2 * 16384 + 1024;
// TMEM columns: QK, O, dS, S0 (bf16 pairs), the three terms (bf16 pairs, 32 columns each; two buffers)
constexpr uint32_t kTmQK = 0, kTmO = 64, kTmS = 128, kTmA = 256, kTmT = 320;
constexpr int kOutThreads = 20 * 32;
constexpr int kRing = 8;  // chunks' gate factors
constexpr int kGateAhead = 6;
// Registers per thread: 96 at launch (20 warps); the warps of the state take what P and the last
// four give up, 2 * 136 + 96 + 56 + 56 = 5 * 96.
constexpr int kRegState = 136, kRegP = 56, kRegRest = 56;
static_assert(2 * kRegState + 96 + kRegP + kRegRest <= 5 * 96, "no more than the block was launched with");

constexpr float kFarDecay = -120.f;  // log2 of a chunk's decay

struct __align__(16) Factors {
    // per token: prefix sum G; 2^{-m - G}; decay to the chunk's end; what O is multiplied by
    float G[C], f[C], w[C], e[C];
    float2 decay;  // of the chunk
    __nv_bfloat162 shift;  // 2^{-m}, twice
    int far;       // the chunk's decay is below kFarDecay
};
// A barrier that one side may complete again before the other side has looked (terms and P are
// written up to a chunk ahead, ds and o are waited for two chunks later) is one of a pair,
// for even and odd chunks.
struct OutBars {
    uint64_t full[kStages], empty[kStages], fac[kRing];
    uint64_t out_full[2], out_empty[2];
    uint64_t qk, ds[2], o[2];                       // products done
    uint64_t state, terms[2], p[2], ds_read, qk_read;  // S0, V w and P ready; dS and QK read
    uint64_t drain[2];
};

__global__ void __launch_bounds__(kOutThreads, 1)
gdn_linattn_tc(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
               const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo, const Args a,
               const bool fixed) {
    extern __shared__ unsigned char smem_raw[];
    uint8_t *sm = align1024(smem_raw);
    __shared__ OutBars bars;
    __shared__ Factors ring[kRing];
    __shared__ __align__(8) float gate_ring[kRing][C];  // gates as they are read, kGateAhead chunks ahead
    __shared__ uint32_t tmem_base;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t h = blockIdx.x % a.H;
    // (kept in shared memory: a role reads of it what it needs when it needs it)
    __shared__ Slot s;
    {
        Slot found;
        if (!locate<false>(a, blockIdx.x / a.H, found) ||
            !in_bounds(found.start >= 0 && found.start + found.len <= a.rows && found.n < a.N && h < a.H, a.status)) {
            wait_for_previous();
            return;
        }
        if (tid == 0) s = found;
        __syncthreads();
    }
    // Roles that wait for the state's warps give up after a while, so none may start long before
    // these can: a state kernel ends within a block's time, the combine kernel, which goes over all
    // sequences, need not.
    if (!a.chained) wait_for_previous();
    const int len = (int)s.len, nch = (len + C - 1) / C;
    const int cut = len % C ? nch - 1 : -1;  // the chunk with rows behind the segment, if any
    constexpr int kIssuerS = 16, kIssuerO = 17, kStorer = 18, kLoader = 19;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bars.full[i], 1 + 32);  // the loads, and the chunk's factors
            mbar_init(&bars.empty[i], 2);      // both issuing warps
        }
        for (int i = 0; i < kRing; ++i) mbar_init(&bars.fac[i], 32);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.ds[i], 1);
            mbar_init(&bars.o[i], 1);
            mbar_init(&bars.terms[i], 128);
            mbar_init(&bars.p[i], 128);
            mbar_init(&bars.out_full[i], 256);
            mbar_init(&bars.out_empty[i], 1);
        }
        mbar_init(&bars.qk, 1);
        mbar_init(&bars.state, 256);
        mbar_init(&bars.ds_read, 256);
        mbar_init(&bars.qk_read, 128);
        mbar_init(&bars.drain[0], 1);
        mbar_init(&bars.drain[1], 1);
        fence_mbar_init();
    }
    if (warp == kIssuerS) {
        tmem_alloc(&tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_base;
    bool ok = true;
    int issued = 0;  // (loader) chunks whose loads are issued
    if (warp >= kIssuerS) fewer_registers<kRegRest>();  // (the four warps together)

    if (warp < 8) {
        // ------------------------------------------------------------------
        // The state and the outputs: value channel v, key channels [64 hf, 64 hf + 64) of
        // the state, tokens [32 hf, 32 hf + 32) of the outputs.
        // ------------------------------------------------------------------
        more_registers<kRegState>();
        const int qd = warp & 3, hf = warp >> 2, v = qd * 32 + lane;
        const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
        const int64_t srow = (int64_t)v * D + 64 * hf;
        float S[64];
#pragma unroll
        for (int c = 0; c < 64; ++c) S[c] = 0.f;
        wait_for_previous();  // (only here: the other roles need nothing that the state kernel wrote)
        start_state(a, s, h, (int64_t)(D * D), [&](float2 f, const float *src) {
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
                const float4 t = *reinterpret_cast<const float4 *>(src + srow + c);
                S[c] = fmaf(f.x, t.x, fmaf(f.y, t.x, S[c]));
                S[c + 1] = fmaf(f.x, t.y, fmaf(f.y, t.y, S[c + 1]));
                S[c + 2] = fmaf(f.x, t.z, fmaf(f.y, t.z, S[c + 2]));
                S[c + 3] = fmaf(f.x, t.w, fmaf(f.y, t.w, S[c + 3]));
            }
        });
        auto publish = [&](__nv_bfloat162 f) {  // 2^{-m} S0 as bf16 pairs: this thread's 32 columns of the A operand
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t y = pack_bf16(S[16 * q + 2 * e], S[16 * q + 2 * e + 1]);
                    const __nv_bfloat162 z = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&y), f);  // (exact)
                    w[e] = *reinterpret_cast<const uint32_t *>(&z);
                }
                tmem_st8u(tm + lane_off + kTmA + 32 * hf + 8 * q, w);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&bars.state);
        };
        if (nch > 0) {
            ok = warp_wait(&bars.fac[0], 0);
            if (ok) publish(ring[0].shift);
        }
        const int32_t kc = a.n_snap > 0 ? (int32_t)(a.snap_stride / C) : 0;  // chunks between snapshots
        const int64_t c0 = s.pos / C;
        int32_t snap_left = kc > 0 ? kc - (int32_t)(c0 % kc) : 0;
        int64_t snap_idx = kc > 0 ? c0 / kc : 0;
        // this lane's row of a stmatrix: tokens (0-7 | 8-15) x channels (0-7 | 8-15) of a block
        const int orow = 32 * hf + (lane & 7) + ((lane >> 4) << 3), opiece = (4 * qd & 7) + ((lane >> 3) & 1);
        const uint32_t obase = smem_u32(sm + kOffO) + (uint32_t)(qd >> 1) * 8192u;
        for (int c = 0; c < nch && ok; ++c) {
            const uint32_t par = (c >> 1) & 1;
            const Factors &fac = ring[c % kRing];
            if (c + 1 < nch) ok = warp_wait(&bars.fac[(c + 1) % kRing], ((c + 1) / kRing) & 1);  // (for its m)
            ok = ok && warp_wait(&bars.ds[c & 1], par);
            if (!ok) break;
            tc_fence_after();
            const float2 d = fac.decay;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float x[32];
                tmem_ld32(tm + lane_off + kTmS + 64 * hf + 32 * q, x);
                tmem_wait_ld();
                if (d.y != 0.f)  // (a fixed decay, or one close to 1: in two floats)
#pragma unroll
                    for (int t = 0; t < 32; ++t) x[t] = fmaf(d.y, S[32 * q + t], x[t]);
#pragma unroll
                for (int t = 0; t < 32; t += 2) {
                    const float2 r = __ffma2_rn(make_float2(d.x, d.x), make_float2(S[32 * q + t], S[32 * q + t + 1]),
                                                make_float2(x[t], x[t + 1]));
                    S[32 * q + t] = r.x;
                    S[32 * q + t + 1] = r.y;
                }
            }
            tc_fence_before();
            mbar_arrive(&bars.ds_read);
            ok = warp_wait(&bars.o[c & 1], par);
            if (!ok) break;
            tc_fence_after();
            float x[2][16];
#pragma unroll
            for (int m = 0; m < 2; ++m)
                tmem_ld_frag32(tm + lane_off + ((uint32_t)(16 * m) << 16) + kTmO + 32 * hf, x[m]);
            tmem_wait_ld();
            if (c + 1 < nch) publish(ring[(c + 1) % kRing].shift);  // S of the next chunk; O is read too
            // o = scale 2^G O, rounded, turned from channel rows to token rows
            if (c > 1) ok = warp_wait(&bars.out_empty[c & 1], par ^ 1);
            if (!ok) break;
            const uint32_t ob = obase + (c & 1) * 16384;
#pragma unroll
            for (int n = 0; n < 4; n += 2) {
                const float2 e0 = *reinterpret_cast<const float2 *>(fac.e + 32 * hf + 8 * n + 2 * (lane & 3));
                const float2 e1 = *reinterpret_cast<const float2 *>(fac.e + 32 * hf + 8 * n + 8 + 2 * (lane & 3));
#pragma unroll
                for (int m = 0; m < 2; ++m) {  // channels 16 m ..
                    const float *y = x[m] + 4 * n;
                    stsm_x4_trans(ob + (uint32_t)(orow + 8 * n) * 128u + (((uint32_t)(opiece + 2 * m) ^ (uint32_t)(orow & 7)) << 4),
                                  pack_bf16(y[0] * e0.x, y[1] * e0.y), pack_bf16(y[2] * e0.x, y[3] * e0.y),
                                  pack_bf16(y[4] * e1.x, y[5] * e1.y), pack_bf16(y[6] * e1.x, y[7] * e1.y));
                }
            }
            fence_async_smem();
            mbar_arrive(&bars.out_full[c & 1]);
            if (kc > 0 && --snap_left == 0) {
                snap_left = kc;
                if (snap_idx < a.n_snap) {
                    float *dst = a.snaps + ((s.n * a.n_snap + snap_idx) * a.H + h) * (int64_t)(D * D) + srow;
#pragma unroll
                    for (int cc = 0; cc < 64; cc += 4)
                        *reinterpret_cast<float4 *>(dst + cc) = make_float4(S[cc], S[cc + 1], S[cc + 2], S[cc + 3]);
                }
                ++snap_idx;
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
        // The terms of V w: value channels 32 (warp - 8) .. + 31.
        // ------------------------------------------------------------------
        const int w = warp - 8;
        const uint32_t to = tm + ((uint32_t)(w * 32) << 16) + kTmT;
        for (int c = 0; c < nch && ok; ++c) {
            const int stage = c % kStages;
            uint8_t *st = sm + stage * kStage;
            const Factors &fac = ring[c % kRing];
            ok = warp_wait(&bars.full[stage], (c / kStages) & 1);  // (the factors too)
            if (!ok) break;
            if (c == cut) {
                // Rows behind the sequence: whatever lies there stays out of the sums.  A warp clears
                // the channels of V that it reads itself and a quarter of K, which only products
                // that wait for the terms of all four warps read: no barrier among the four, at which
                // three would stay if a wait of the fourth gave up.
                const uint32_t z = (uint32_t)(w >> 1) * kHalfV;  // (halves of K are twice as far apart)
                for (int i = lane; i < 64 * 4; i += 32) {
                    const int row = i >> 2, p = (w & 1) * 4 + (i & 3);
                    if (row < len % C) continue;
                    const uint32_t at = row * 128 + ((p ^ (row & 7)) << 4);
                    *reinterpret_cast<uint4 *>(st + kStV + z + at) = make_uint4(0u, 0u, 0u, 0u);
                    *reinterpret_cast<uint4 *>(st + kStK + 2 * z + at) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_async_smem();
                __syncwarp();
            }
            if (c > 1) ok = warp_wait(&bars.ds[c & 1], ((c >> 1) & 1) ^ 1);  // dS of chunk c - 2 has read this buffer
            if (!ok) break;
            tc_fence_after();
            const uint32_t from = terms_address(smem_u32(st + kStV) + (uint32_t)(w >> 1) * kHalfV, 0, 0, lane);
            const int piece = (w & 1) * 4;
#pragma unroll 4
            for (int i = 0; i < 8; ++i) {  // 16 channels x 16 tokens each
                const int m = i >> 2, n = i & 3;
                uint32_t t0[4], t1[4], t2[4];
                // (the piece's bits are turned by the row's: exclusive or)
                channel_terms((from ^ (uint32_t)((piece + 2 * m) << 4)) + n * 2048u, fac.w + 16 * n, lane, t0, t1, t2);
                const uint32_t at = to + (c & 1) * 96 + ((uint32_t)(16 * m) << 16) + 8 * n;
                tmem_st_frag8(at, t0);
                tmem_st_frag8(at + 32, t1);
                tmem_st_frag8(at + 64, t2);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&bars.terms[c & 1]);
        }
    } else if (warp < kIssuerS) {
        // ------------------------------------------------------------------
        // P: query tokens 16 w .. 16 w + 15, of which a lane holds two (i0, i0 + 8).
        // ------------------------------------------------------------------
        fewer_registers<kRegP>();
        const int w = warp - 12, i0 = 16 * w + (lane >> 2), j0 = 2 * (lane & 3);
        uint8_t *P = sm + kOffP;
        // this lane's row of a stmatrix: matrices (tokens 0-7, keys 0-7), (8-15, 0-7), (0-7, 8-15),
        // (8-15, 8-15) of a block
        const int prow = 16 * w + (lane & 15);
        const uint32_t paddr = smem_u32(P) + (uint32_t)prow * 128u + (((uint32_t)(lane >> 4) ^ (uint32_t)(prow & 7)) << 4);
        for (int i = lane; i < 2 * 16 * 8; i += 32)  // the blocks above the diagonal stay zero
            *reinterpret_cast<uint4 *>(P + (i >> 7) * 8192 + (16 * w + ((i >> 3) & 15)) * 128 + (i & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
        __syncwarp();
        for (int c = 0; c < nch && ok; ++c) {
            const Factors &fac = ring[c % kRing];
            ok = warp_wait(&bars.fac[c % kRing], (c / kRing) & 1);
            ok = ok && warp_wait(&bars.qk, c & 1);
            if (c > 1) ok = ok && warp_wait(&bars.o[c & 1], ((c >> 1) & 1) ^ 1);  // O of chunk c - 2 has read this buffer
            if (!ok) break;
            tc_fence_after();
            const bool far = fac.far;
#pragma unroll 1
            for (int n = 0; n <= w; ++n) {  // 16 keys each
                float x[8];
                tmem_ld_frag16(tm + ((uint32_t)(w * 32) << 16) + kTmQK + 16 * n, x);
                tmem_wait_ld();
                float2 f[4];  // factors of keys j, j + 1 and j + 8, j + 9: for token i0, then for i0 + 8
                if (!far) {
                    f[0] = f[1] = *reinterpret_cast<const float2 *>(fac.f + 16 * n + j0);
                    f[2] = f[3] = *reinterpret_cast<const float2 *>(fac.f + 16 * n + 8 + j0);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float Gi = fac.G[i0 + 8 * (e & 1)];
                        const float2 Gj = *reinterpret_cast<const float2 *>(fac.G + 16 * n + 8 * (e >> 1) + j0);
                        f[e] = make_float2(a.scale * ex2(Gi - Gj.x), a.scale * ex2(Gi - Gj.y));
                    }
                }
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float2 p = __fmul2_rn(make_float2(x[2 * e], x[2 * e + 1]), f[e]);
                    const int i = i0 + 8 * (e & 1), j = 16 * n + 8 * (e >> 1) + j0;
                    if (j > i) p.x = 0.f;
                    if (j + 1 > i) p.y = 0.f;
                    o[e] = pack_bf16(p.x, p.y);
                }
                stsm_x4((paddr ^ (uint32_t)(n << 5)) + (c & 1) * 8192, o[0], o[1], o[2], o[3]);
            }
            tc_fence_before();
            mbar_arrive(&bars.qk_read);
            if (far) {  // Q by scale 2^G, in place (QK is done with it)
                uint8_t *Q = sm + (c % kStages) * kStage + kStQ;
                for (int i = lane; i < 16 * 16; i += 32) {
                    const int row = 16 * w + (i >> 4);
                    uint4 *q = reinterpret_cast<uint4 *>(Q + ((i >> 3) & 1) * kHalfQK + row * 128 + (i & 7) * 16);
                    const float f = a.scale * ex2(fac.G[row]);
                    uint4 t = *q;
                    uint32_t *u = &t.x;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        u[e] = pack_bf16(f * __uint_as_float(u[e] << 16), f * __uint_as_float(u[e] & 0xffff0000u));
                    *q = t;
                }
            }
            fence_async_smem();
            mbar_arrive(&bars.p[c & 1]);
        }
    } else if (warp == kIssuerS) {
        // ------------------------------------------------------------------
        // MMAs of dS
        // ------------------------------------------------------------------
        const uint32_t base = smem_u32(sm);
        for (int c = 0; c < nch; ++c) {
            const uint32_t par = c & 1;
            if (c > 0) ok = warp_wait(&bars.ds_read, par ^ 1);
            ok = ok && warp_wait(&bars.terms[par], (c >> 1) & 1);  // (K has arrived with V)
            if (!ok) break;
            tc_fence_after();
            const uint64_t bk = sdesc_sw128(base + (c % kStages) * kStage + kStK, kHalfQK, 1024);
            const uint32_t t = tm + kTmT + 96 * par;
#pragma unroll
            for (int k = 0; k < 3; ++k) mma4_ts<8, 128>(tm + kTmS, t + 32 * k, bk, idesc_bf16(128, 128, 0, 1), k > 0);
            mma_commit_warp(&bars.ds[par]);
            mma_commit_warp(&bars.empty[c % kStages]);
        }
    } else if (warp == kIssuerO) {
        // ------------------------------------------------------------------
        // MMAs of QK, a chunk ahead, and of O
        // ------------------------------------------------------------------
        const uint32_t base = smem_u32(sm);
        for (int c = -1; c < nch; ++c) {
            const uint32_t par = c & 1;
            if (c + 1 < nch) {
                const int stage = (c + 1) % kStages;
                ok = warp_wait(&bars.full[stage], ((c + 1) / kStages) & 1);
                if (c >= 0) ok = ok && warp_wait(&bars.qk_read, par);
                if (!ok) break;
                tc_fence_after();
                const uint32_t st = base + stage * kStage;
                const uint64_t aq = sdesc_sw128(st + kStQ, 16, 1024), bk = sdesc_sw128(st + kStK, 16, 1024);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    mma4_ss<2, 2>(tm + kTmQK, aq + i * (kHalfQK >> 4), bk + i * (kHalfQK >> 4), idesc_bf16(64, 64, 0, 0), i);
                mma_commit_warp(&bars.qk);
            }
            if (c < 0) continue;
            ok = warp_wait(&bars.state, par);  // S0 in place, the previous chunk's O read
            ok = ok && warp_wait(&bars.p[par], (c >> 1) & 1);
            // (a last chunk's rows behind the sequence have to be cleared, as they are before its terms)
            if (c == cut) ok = ok && warp_wait(&bars.terms[par], (c >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t st = base + (c % kStages) * kStage;
            const uint64_t bq = sdesc_sw128(st + kStQ, 16, 1024);
            const uint64_t av = sdesc_sw128(st + kStV, kHalfV, 1024), bp = sdesc_sw128(base + kOffP + par * 8192, 16, 1024);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                mma4_ts<8, 2>(tm + kTmO, tm + kTmA + 32 * i, bq + i * (kHalfQK >> 4), idesc_bf16(128, 64, 0, 0), i);
            mma4_ss<128, 2>(tm + kTmO, av, bp, idesc_bf16(128, 64, 1, 0), 1);
            mma_commit_warp(&bars.o[par]);
            mma_commit_warp(&bars.empty[c % kStages]);
        }
    } else if (warp == kStorer) {
        const int32_t hv = (int32_t)h;
        for (int c = 0; c < nch && ok; ++c) {
            ok = warp_wait(&bars.out_full[c & 1], (c >> 1) & 1);
            if (!ok) break;
            const uint8_t *o = sm + kOffO + (c & 1) * 16384;
            const int64_t row = s.start + (int64_t)c * C;
            if (c != cut) {
                if (lane == 0) {
                    tma_store_3d(&mo, o, 0, hv, (int32_t)row);
                    tma_store_3d(&mo, o + 8192, 64, hv, (int32_t)row);
                    bulk_commit();
                    bulk_wait_read();
                    mbar_arrive(&bars.out_empty[c & 1]);
                }
            } else {  // rows behind the sequence stay as they are
                __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(a.out) + (row * a.H + h) * D;
                for (int i = lane; i < len % C * 16; i += 32) {
                    const int t = i >> 4, p = i & 15;
                    *reinterpret_cast<uint4 *>(to + t * a.H * D + 8 * p) =
                        *reinterpret_cast<const uint4 *>(o + (p >> 3) * 8192 + sw128_offset(t, p & 7));
                }
            }
            __syncwarp();
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    } else {
        // ------------------------------------------------------------------
        // Loads, and the gates' factors, two tokens per lane
        // ------------------------------------------------------------------
        const int32_t hq = (int32_t)(h / (a.H / a.Hk)), hv = (int32_t)h;
        if (lane == 0 && nch > 0) {
            prefetch_tmap(&mq);
            prefetch_tmap(&mk);
            prefetch_tmap(&mv);
        }
        // (a call without tokens may come without gates: a segment without chunks reads none)
        const float gh = fixed && nch > 0 ? gate2(a.g[h]) : 0.f;
        // A head's gates lie H floats apart, a memory sector each: they are asked for early.
        const float *gates = a.g + (fixed ? 0 : s.start * a.H + h);
        auto ask_gates = [&](int c) {
            if (c < nch && !fixed) {
                const int t = c * C + 2 * lane;
                const float *p = gates + (int64_t)t * a.H;
                async_copy4(&gate_ring[c % kRing][2 * lane], t < len ? p : a.g, t < len);
                async_copy4(&gate_ring[c % kRing][2 * lane + 1], t + 1 < len ? p + a.H : a.g, t + 1 < len);
            }
            async_commit();  // (a group per chunk, empty or not)
        };
        for (int c = 0; c < kGateAhead; ++c) ask_gates(c);
        const float2 fixed_decay = fixed && nch > 0 ? exp2_pair(gate2_exact(a.g[h]) * C) : make_float2(0.f, 0.f);
        for (int c = 0; c < nch; ++c) {
            const int stage = c % kStages;
            if (c >= kStages) ok = warp_wait(&bars.empty[stage], ((c / kStages) & 1) ^ 1);
            if (!ok) break;
            if (lane == 0) {
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
            }
            issued = c + 1;
            __syncwarp();
            // The factors' slot: O of chunk c - 3 is formed, so O of chunk c - 4 was read, and the
            // slot's last readers (chunk c - 8) are done.
            ask_gates(c + kGateAhead);
            async_wait<kGateAhead>();  // (a lane reads what it copied itself)
            const int left = len - c * C;
            float2 g = *reinterpret_cast<const float2 *>(&gate_ring[c % kRing][2 * lane]);
            g = fixed ? make_float2(2 * lane < left ? gh : 0.f, 2 * lane + 1 < left ? gh : 0.f)
                      : make_float2(gate2(g.x), gate2(g.y));
            Factors &fac = ring[c % kRing];
            float2 G, after;
            float total;
            scan_gates(g.x, g.y, lane, G, after, total);
            const bool far = !(total > kFarDecay);
            *reinterpret_cast<float2 *>(&fac.G[2 * lane]) = G;
            const float m = far ? 0.f : rintf(-0.5f * total);
            *reinterpret_cast<float2 *>(&fac.f[2 * lane]) = make_float2(ex2(-m - G.x), ex2(-m - G.y));
            *reinterpret_cast<float2 *>(&fac.w[2 * lane]) = make_float2(ex2(after.x), ex2(after.y));
            *reinterpret_cast<float2 *>(&fac.e[2 * lane]) =
                far ? make_float2(1.f, 1.f) : make_float2(a.scale * ex2(m + G.x), a.scale * ex2(m + G.y));
            if (lane == 0) {
                fac.far = far;
                fac.shift = __float2bfloat162_rn(ex2(-m));
                fac.decay = !fixed ? exp2_pair_f32(total)
                                   : (left >= C ? fixed_decay
                                                : exp2_pair(gate2_exact(a.g[h]) * (double)left));
            }
            mbar_arrive(&bars.fac[c % kRing]);
            mbar_arrive(&bars.full[stage]);
        }
    }
    __syncwarp();
    if (!ok) {
        // A wait gave up: record it.  Every other role's next wait gives up too (it waits,
        // directly or not, for this one), so all of them get here.
        if (lane == 0) flag_error(a.status, GDN_DEV_TIMEOUT_SCAN);
        if (warp == kLoader)  // loads and MMAs still in flight
            for (int j = issued > kStages ? issued - kStages : 0; j < issued; ++j)
                warp_wait(&bars.full[j % kStages], (j / kStages) & 1);
        if (warp == kIssuerS || warp == kIssuerO) {
            mma_commit_warp(&bars.drain[warp - kIssuerS]);
            warp_wait(&bars.drain[warp - kIssuerS], 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kIssuerS) tmem_dealloc(tm, 512);
}

// ===========================================================================
// State kernel: what a part of a segment (not its sequence's last) adds to the state
// at the segment's end
// ===========================================================================
// Backwards from the part's end: a token's weight is the sum of the gates after it, so the
// products add up without a rescale, and the kernel stops where nothing earlier reaches the
// segment's end.  The products of kGroup chunks add up in TMEM; the tensor cores cut off what does
// not fit an accumulator's 24 bits, always towards zero, so a long sum there comes out short
// (2^-24 or so of it with every 16 tokens and term: 5e-5 of the state after 14,600 tokens that do not
// fade).  The groups are added in registers, rounded to nearest: the warps of the terms
// read one of two accumulators while the next group goes into the other.
// A segment is cut into parts so that the heads whose state lasts do not hold up the rest: their
// parts run side by side, and a part behind which the decay has left nothing ends at once.
// The weights of the whole part are formed first, 1024 tokens at a time by warps 0-15; then
// these make the terms of V w (32 value channels and 16 tokens a warp, two buffers in TMEM),
// warp 16 issues the MMAs and warp 17 the loads.  One block per SM (448 of 512 TMEM columns).
// Measured: 129 us for 262,144 tokens of 16 heads with fixed decays (the heads whose state
// lasts read all of k and v; 124 us with one accumulator for all chunks), 19 us for 4 x 4,096
// tokens of 16 heads (bound by its start, the gates and a few chunks).
constexpr uint32_t kSsK = 0, kSsV = 16384, kSsStage = 32768;
constexpr int kSsStages = 4;
constexpr uint32_t kSsOffW = kSsStages * kSsStage;  // the part's weights, newest token last
constexpr uint32_t kTmU = 0, kTmUT = 256;  // two accumulators, the terms
constexpr int kGroup = 4;                  // chunks of an accumulator (two or more)
constexpr int kTermWarps = 16, kTermThreads = kTermWarps * 32;
constexpr int kStateThreads = (kTermWarps + 2) * 32;
constexpr int kSpan = 2 * kTermThreads;  // tokens of a step of the scan

struct StateBars {
    uint64_t full[kSsStages], empty[kSsStages], terms[2], ds[2], drain;
};

// Weights of the tokens [begin, end) of a segment, from the end backwards: wts[t - begin] = 2^{after +
// gates behind t} for one head; stops after the step that brings the sum to kDead.
// Returns the sum at the first token weighed, and in `first` that token.  The whole block
// calls it; the first kTermThreads threads take two tokens each.
__device__ __forceinline__ float part_weights(const Args &a, const Slot &s, int64_t h, int64_t begin, int64_t end, float after,
                                              float *wts, float *s_sum, int64_t &first) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int64_t t1 = end;
    for (; t1 > begin && after > kDead; t1 -= kSpan) {
        const int64_t t = t1 - kSpan + 2 * tid;  // this thread's tokens t, t + 1 (the last thread's are the newest)
        float2 g = make_float2(0.f, 0.f);
        if (tid < kTermThreads) {
            if (t >= begin) g.x = gate2(a.g[(s.start + t) * a.H + h]);
            if (t + 1 >= begin) g.y = gate2(a.g[(s.start + t + 1) * a.H + h]);
        }
        float sum = g.x + g.y;  // of this lane and the lanes above it
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float x = __shfl_down_sync(0xffffffffu, sum, o);
            if (lane + o < 32) sum += x;
        }
        __syncthreads();
        if (warp < kTermWarps && lane == 0) s_sum[warp] = sum;
        __syncthreads();
        float behind = after, all = 0.f;  // what follows this warp's tokens
#pragma unroll
        for (int w = kTermWarps - 1; w >= 0; --w) {
            if (w > warp) behind += s_sum[w];
            all += s_sum[w];
        }
        if (wts && tid < kTermThreads) {
            const float above = __shfl_down_sync(0xffffffffu, sum, 1);
            const float b1 = behind + (lane < 31 ? above : 0.f);
            if (t >= begin) wts[t - begin] = ex2(b1 + g.y);
            if (t + 1 >= begin) wts[t + 1 - begin] = ex2(b1);
        }
        after += all;
    }
    first = t1 > begin ? t1 : begin;
    return after;
}

__global__ void __launch_bounds__(kStateThreads, 1)
gdn_linattn_state_tc(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const Args a,
                     const bool fixed) {
    extern __shared__ unsigned char smem_raw[];
    uint8_t *sm = align1024(smem_raw);
    float *wts = reinterpret_cast<float *>(sm + kSsOffW);
    __shared__ StateBars bars;
    __shared__ uint32_t tmem_base;
    __shared__ float s_sum[kTermWarps];
    constexpr int kIssuer = kTermWarps, kLoader = kTermWarps + 1;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t h = blockIdx.x % a.H, unit = blockIdx.x / a.H;
    let_next_start();
    // (the newest parts of all segments first: the blocks that find nothing to do come last)
    const int64_t part = a.parts - 1 - unit / a.sslots;
    Slot s;
    if (!locate<true>(a, unit % a.sslots, s) || s.nseg < 2 || s.j == s.nseg - 1) return;
    if (!in_bounds(s.start >= 0 && s.start + s.len <= a.rows && s.n < a.N && s.ss < a.sslots && s.len % C == 0, a.status))
        return;
    const int64_t begin = part * a.part_len;  // of the part, in the segment
    const int64_t end = begin + a.part_len < s.len ? begin + a.part_len : s.len;
    // the decay from the part's end to the segment's
    const double g64 = fixed ? gate2_exact(a.g[h]) : 0.0;
    int64_t first = 0;
    const float gap = fixed ? (float)(g64 * (double)(s.len - end))
                            : part_weights(a, s, h, end, s.len, 0.f, nullptr, s_sum, first);
    const int64_t at = (s.ss * a.parts + part) * a.H + h;
    const bool alive = end > begin && gap > kDead;
    if (tid == 0) {
        a.alive[at] = alive ? 1 : 0;
        if (part == 0 && !alive) a.tot[s.ss * a.H + h] = (double)gap;
    }
    if (!alive) return;
    const int most = (int)((end - begin) / C);
    if (tid == 0) {
        for (int i = 0; i < kSsStages; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.terms[i], kTermThreads);
            mbar_init(&bars.ds[i], 1);
        }
        mbar_init(&bars.drain, 1);
        fence_mbar_init();
    }
    if (warp == kIssuer) {
        tmem_alloc(&tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int issued = 0;  // (loader) chunks whose loads are issued
    auto load = [&](int i) {  // chunk i from the part's end
        if (lane == 0) {
            uint8_t *st = sm + (i % kSsStages) * kSsStage;
            uint64_t *bar = &bars.full[i % kSsStages];
            const int32_t r = (int32_t)(s.start + end - (int64_t)(i + 1) * C);
            const int32_t hq = (int32_t)(h / (a.H / a.Hk)), hv = (int32_t)h;
            mbar_arrive_expect_tx(bar, kSsStage);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                tma_load_3d(st + kSsK + k * 8192, &mk, 64 * k, hq, r, bar);
                tma_load_3d(st + kSsV + k * 8192, &mv, 64 * k, hv, r, bar);
            }
        }
        issued = i + 1;
        __syncwarp();
    };
    if (warp == kLoader)  // (on their way while the weights are formed)
        for (int i = 0; i < kSsStages && i < most; ++i) load(i);
    float reach;  // sum of the gates from the first chunk that is added on
    if (fixed) {
        // 2^{gap + g (tokens behind)}; nothing before the token where that is below 2^kDead
        const double live = g64 < 0.0 ? ((double)kDead - (double)gap) / g64 : 1e18;
        const int64_t keep = live < (double)(end - begin) ? (int64_t)live + 1 : end - begin;
        first = (end - keep) / C * C;
        first = first > begin ? first : begin;
        const float g2 = (float)g64;
        for (int64_t t = first + tid; t < end; t += kStateThreads) wts[t - begin] = ex2(gap + g2 * (float)(end - 1 - t));
        reach = 0.f;
    } else {
        reach = part_weights(a, s, h, begin, end, gap, wts, s_sum, first);
    }
    __syncthreads();
    // chunks to add, from the part's end: all those whose newest token still weighs something (at
    // least one)
    int skip = (int)((first - begin) / C);
    while (skip < most - 1 && wts[skip * C + C - 1] == 0.f) ++skip;
    const int nch = most - skip;
    const uint32_t tm = tmem_base;
    bool ok = true;
    if (warp < kTermWarps) {
        const int qd = warp & 3, tq = warp >> 2;  // channels 32 qd .., tokens 16 tq ..
        const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
        const uint32_t from = terms_address(smem_u32(sm + kSsV) + (uint32_t)(qd >> 1) * 8192u, (qd & 1) * 4, 16 * tq, lane);
        float U[32];  // row 32 qd + lane, columns 32 tq ..
#pragma unroll
        for (int e = 0; e < 32; ++e) U[e] = 0.f;
        int groups = 0;  // added
        auto add_group = [&] {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float x[16];
                tmem_ld16(tm + lane_off + kTmU + 128 * (groups & 1) + 32 * tq + 16 * q, x);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float2 y = __fadd2_rn(make_float2(U[16 * q + e], U[16 * q + e + 1]), make_float2(x[e], x[e + 1]));
                    U[16 * q + e] = y.x;
                    U[16 * q + e + 1] = y.y;
                }
            }
            ++groups;
        };
        for (int i = 0; i < nch; ++i) {
            const int stage = i % kSsStages;
            const float *w = wts + (most - 1 - i) * C + 16 * tq;
            ok = warp_wait(&bars.full[stage], (i / kSsStages) & 1);
            if (i >= 2) ok = ok && warp_wait(&bars.ds[i & 1], ((i >> 1) & 1) ^ 1);  // chunk i - 2 has used this buffer
            if (!ok) break;
            tc_fence_after();
            // (its accumulator is written again a group later, after the terms that this warp makes below)
            if (i >= 2 && (i - 1) % kGroup == 0) add_group();
#pragma unroll
            for (int m = 0; m < 2; ++m) {  // 16 channels x 16 tokens each
                uint32_t t0[4], t1[4], t2[4];
                channel_terms((from + stage * kSsStage) ^ (uint32_t)(m << 5), w, lane, t0, t1, t2);
                const uint32_t to = tm + lane_off + ((uint32_t)(16 * m) << 16) + kTmUT + 96 * (i & 1) + 8 * tq;
                tmem_st_frag8(to, t0);
                tmem_st_frag8(to + 32, t1);
                tmem_st_frag8(to + 64, t2);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&bars.terms[i & 1]);
        }
        if (ok) {
            ok = warp_wait(&bars.ds[(nch - 1) & 1], ((nch - 1) >> 1) & 1);  // the last chunk's products, and all before
            tc_fence_after();
        }
        if (ok) {
            while (groups * kGroup < nch) add_group();  // (one or two)
            float *to = a.states + at * (int64_t)(D * D) + (int64_t)(qd * 32 + lane) * D + 32 * tq;
#pragma unroll
            for (int e = 0; e < 32; e += 4) *reinterpret_cast<float4 *>(to + e) = make_float4(U[e], U[e + 1], U[e + 2], U[e + 3]);
            // the segment's decay (once it is past kDead, how far past does not matter)
            if (part == 0 && tid == 0) a.tot[s.ss * a.H + h] = fixed ? g64 * (double)s.len : (double)reach;
        }
    } else if (warp == kIssuer) {
        const uint32_t base = smem_u32(sm);
        for (int i = 0; i < nch; ++i) {
            ok = warp_wait(&bars.terms[i & 1], (i >> 1) & 1);  // (K has arrived with V)
            if (!ok) break;
            tc_fence_after();
            const uint64_t bk = sdesc_sw128(base + (i % kSsStages) * kSsStage + kSsK, 8192, 1024);
            const uint32_t t = tm + kTmUT + 96 * (i & 1);
#pragma unroll
            for (int m = 0; m < 3; ++m)
                mma4_ts<8, 128>(tm + kTmU + 128 * (i / kGroup & 1), t + 32 * m, bk, idesc_bf16(128, 128, 0, 1),
                                i % kGroup > 0 || m > 0);
            mma_commit_warp(&bars.ds[i & 1]);
            mma_commit_warp(&bars.empty[i % kSsStages]);
        }
    } else {
        for (int i = kSsStages; i < nch; ++i) {
            ok = warp_wait(&bars.empty[i % kSsStages], ((i / kSsStages) & 1) ^ 1);
            if (!ok) break;
            load(i);
        }
    }
    __syncwarp();
    if (!ok) {
        if (lane == 0) flag_error(a.status, GDN_DEV_TIMEOUT_PREP);
        if (warp == kIssuer) {
            mma_commit_warp(&bars.drain);
            warp_wait(&bars.drain, 0);
        }
    }
    if (warp == kLoader)  // loads that nobody has waited for: chunks left out, or all the last ones after a failed wait
        for (int j = issued > kSsStages ? issued - kSsStages : 0; j < issued; ++j)
            if (!ok || j >= nch) warp_wait(&bars.full[j % kSsStages], (j / kSsStages) & 1);
    tc_fence_before();
    __syncthreads();
    if (warp == kIssuer) tmem_dealloc(tm, 512);
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
    const int64_t grid = p.slots * p.H, sgrid = p.sslots * p.parts * p.H;
    if (grid > 0x7fffffffLL || sgrid > 0x7fffffffLL) return fail(GDN_ERR_UNSUPPORTED, "grid too large");
    CUtensorMap mq, mk, mv, mo;
    memset(&mq, 0, sizeof mq);
    memset(&mk, 0, sizeof mk);
    memset(&mv, 0, sizeof mv);
    memset(&mo, 0, sizeof mo);
    gdn_status st = GDN_OK;
    if (p.rows > 0) {
        if ((st = make_map(&mq, a.q, p.rows, a.Hk)) != GDN_OK) return st;
        if ((st = make_map(&mk, a.k, p.rows, a.Hk)) != GDN_OK) return st;
        if ((st = make_map(&mv, a.v, p.rows, p.H)) != GDN_OK) return st;
        if ((st = make_map(&mo, a.out, p.rows, p.H)) != GDN_OK) return st;
    }
    const size_t state_smem = kSsOffW + (size_t)p.part_len * sizeof(float) + 1024;
    static std::atomic<uint64_t> out_done{0}, state_done{0};
    if ((st = allow_smem((const void *)gdn_linattn_tc, kOutSmem, out_done)) != GDN_OK) return st;
    if ((st = allow_smem((const void *)gdn_linattn_state_tc, kSsOffW + kMaxPart * sizeof(float) + 1024, state_done)) != GDN_OK)
        return st;
    if (sgrid > 0) {
        {
            log_launch("gdn_linattn_state_tc", dim3((unsigned)sgrid), dim3(kStateThreads), state_smem);
            LaunchScope ls("gdn_linattn_state_tc", s);
            gdn_linattn_state_tc<<<(unsigned)sgrid, kStateThreads, state_smem, s>>>(mk, mv, a, p.fixed_gate);
        }
        if ((st = check_launch("gdn_linattn_state_tc")) != GDN_OK) return st;
        if (!a.chained && (st = launch_combine(p, a, s)) != GDN_OK) return st;
    }
    {
        log_launch("gdn_linattn_tc", dim3((unsigned)grid), dim3(kOutThreads), kOutSmem);
        LaunchScope ls("gdn_linattn_tc", s);
        launch_kernel(gdn_linattn_tc, dim3((unsigned)grid), dim3(kOutThreads), kOutSmem, s, sgrid > 0, mq, mk, mv, mo, a,
                      p.fixed_gate);
    }
    return check_launch("gdn_linattn_tc");
}

}  // namespace lin
}  // namespace gdn
