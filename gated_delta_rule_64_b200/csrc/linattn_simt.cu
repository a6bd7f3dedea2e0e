// Chunkwise linear attention with a decay for each head, on the CUDA cores: fp32
// inputs, and bf16 inputs of head widths the tensor-core path does not take.  Also the
// combine kernel, which both paths share.  The algebra is at the top of linattn.cuh.
//
// One block works on 32 state rows (value channels) of one segment and head, which
// stay in shared memory in fp32 for the whole segment, in chunks of 32 tokens: the
// scores Q K^T (32 x 32) of a chunk are formed by each of the d_v / 32 blocks that share
// a head, a third of the multiply-adds at d_k = 128, in exchange for four times
// as many blocks.  All sums are fp32.  The decays into and out of a chunk are sums of just
// the gates they cover; those between two tokens of a chunk are differences of prefix
// sums, held in 64 bits, since a gate that erases the state (-1e4, say) would leave
// nothing of its neighbours in fp32.
//
// Bound by latency: a chunk's three products follow one another with a barrier between,
// 256 threads a block.  Measured: 256 fp32 tokens of 2 heads, 64 wide, in four segments: 17 us
// in the output kernel, 12 us in the state kernel, which overlap at the ends (23 us a call).
#include "linattn.cuh"
#include "sm100.cuh"

namespace gdn {
namespace lin {
namespace {

using sm100::ex2;

constexpr int kC = 32;        // tokens per chunk
constexpr int kRows = 32;     // state rows per block
constexpr int kThreads = 256;

// Gate g of token row `row` and head h, in log2 units.
__device__ __forceinline__ float gate_of(const Args &a, bool fixed, int64_t row, int64_t h) {
    return gate2(a.g[fixed ? h : row * a.H + h]);
}

// Inclusive prefix sum over the warp, and the sum of what follows the lane.
template <typename Sum>
__device__ __forceinline__ void warp_scans(float x, int lane, Sum &prefix, float &after) {
    prefix = x;
    after = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sum p = __shfl_up_sync(0xffffffffu, prefix, o);
        const float s = __shfl_down_sync(0xffffffffu, after, o);
        if (lane >= o) prefix += p;
        if (lane + o < 32) after += s;
    }
    const float s = __shfl_down_sync(0xffffffffu, after, 1);
    after = lane < 31 ? s : 0.f;
}

// Two partial sums of a dot product, four more values (two multiply-adds an instruction).
__device__ __forceinline__ void dot4(const float4 &a, const float4 &b, float2 &c) {
    c = __ffma2_rn(make_float2(a.x, a.y), make_float2(b.x, b.y), c);
    c = __ffma2_rn(make_float2(a.z, a.w), make_float2(b.z, b.w), c);
}

// Four consecutive values: as they lie in memory (16-byte aligned fp32, 8-byte aligned bf16), as fp32.
template <typename Tin> struct Raw4;
template <> struct Raw4<float> { typedef float4 type; };
template <> struct Raw4<__nv_bfloat16> { typedef uint2 type; };
__device__ __forceinline__ float4 widen(const float4 &x) { return x; }
__device__ __forceinline__ float4 widen(const uint2 &w) {
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }

// A chunk's rows of W values, this thread's share: read ahead into registers, then put into
// shared rows of LD floats.  Rows from len on are zeros, and not read.
template <int W, int LD, typename Tin>
struct Rows {
    static constexpr int N = kC * (W / 4) / kThreads;
    static_assert(N * kThreads == kC * (W / 4), "whole pieces");
    typename Raw4<Tin>::type x[N];
    __device__ __forceinline__ void read(const Tin *src, int64_t ld, int64_t len) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = threadIdx.x + i * kThreads, r = e / (W / 4), c = e % (W / 4) * 4;
            x[i] = {};
            if (r < len) x[i] = *reinterpret_cast<const typename Raw4<Tin>::type *>(src + r * ld + c);
        }
    }
    __device__ __forceinline__ void put(float *dst) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = threadIdx.x + i * kThreads, r = e / (W / 4), c = e % (W / 4) * 4;
            *reinterpret_cast<float4 *>(dst + r * LD + c) = widen(x[i]);
        }
    }
};

template <int DK>
struct Smem {
    static constexpr int LK = DK + 4, LV = kRows + 4, LP = kC + 1;  // padded rows: no bank conflicts
    float q[kC * LK], k[kC * LK], S[kRows * LK], v[kC * LV], P[kC * LP];
    double G[kC];               // per token: prefix sum of the gates
    float w[kC], e[kC];         // decay to the chunk's end; scale * decay from its start
    float2 decay;               // of the whole chunk
};

// Outputs of one segment, head and 32 value channels, from the segment's start state.
template <int DK, typename Tin>
__global__ void __launch_bounds__(kThreads) gdn_linattn_simt(const Args a, int64_t dv, bool fixed) {
    extern __shared__ float4 smem_raw[];
    using Sm = Smem<DK>;
    Sm &sm = *reinterpret_cast<Sm *>(smem_raw);
    constexpr int LK = Sm::LK, LV = Sm::LV, LP = Sm::LP;
    constexpr int TR = DK / 32;  // state rows of a thread, four columns each
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slices = (int)(dv / kRows);
    const int64_t id = blockIdx.x;
    const int64_t h = id / slices % a.H;
    const int r0 = (int)(id % slices) * kRows;
    Slot s;
    if (!locate<false>(a, id / slices / a.H, s)) {
        wait_for_previous();
        return;
    }
    const int64_t hq = h / (a.H / a.Hk);
    const Tin *q = static_cast<const Tin *>(a.q) + (s.start * a.Hk + hq) * DK;
    const Tin *k = static_cast<const Tin *>(a.k) + (s.start * a.Hk + hq) * DK;
    const Tin *v = static_cast<const Tin *>(a.v) + (s.start * a.H + h) * dv + r0;
    Tin *out = static_cast<Tin *>(a.out) + (s.start * a.H + h) * dv + r0;
    const int64_t ldk = a.Hk * DK, ldv = a.H * dv;
    // this thread's part of the state: rows sr .. sr + TR - 1, columns sc .. sc + 3
    const int sc = tid % (DK / 4) * 4, sr = tid / (DK / 4) * TR;
    Rows<DK, LK, Tin> qn, kn;  // the next chunk's, on their way while the current one is worked on
    Rows<kRows, LV, Tin> vn;
    float gn = 0.f;
    auto ahead = [&](int64_t t0) {
        qn.read(q + t0 * ldk, ldk, s.len - t0);
        kn.read(k + t0 * ldk, ldk, s.len - t0);
        vn.read(v + t0 * ldv, ldv, s.len - t0);
        gn = warp == 0 && t0 + lane < s.len ? gate_of(a, fixed, s.start + t0 + lane, h) : 0.f;
    };
    if (s.len > 0) ahead(0);
    wait_for_previous();
    {
        float4 x[TR] = {};
        start_state(a, s, h, dv * DK, [&](float2 f, const float *src) {
#pragma unroll
            for (int i = 0; i < TR; ++i) {
                const float4 y = load4(src + (int64_t)(r0 + sr + i) * DK + sc);
                x[i].x = fmaf(f.x, y.x, fmaf(f.y, y.x, x[i].x));
                x[i].y = fmaf(f.x, y.y, fmaf(f.y, y.y, x[i].y));
                x[i].z = fmaf(f.x, y.z, fmaf(f.y, y.z, x[i].z));
                x[i].w = fmaf(f.x, y.w, fmaf(f.y, y.w, x[i].w));
            }
        });
#pragma unroll
        for (int i = 0; i < TR; ++i) *reinterpret_cast<float4 *>(sm.S + (sr + i) * LK + sc) = x[i];
    }
    for (int64_t t0 = 0; t0 < s.len; t0 += kC) {
        const int L = (int)(s.len - t0 < kC ? s.len - t0 : kC);
        __syncthreads();  // the previous chunk is done with the tiles
        qn.put(sm.q);
        kn.put(sm.k);
        vn.put(sm.v);
        const float g = gn;
        if (t0 + kC < s.len) ahead(t0 + kC);
        if (warp == 0) {
            double G;
            float after;
            warp_scans(g, lane, G, after);
            sm.G[lane] = G;
            sm.w[lane] = ex2(after);
            sm.e[lane] = a.scale * ex2((float)G);
            // the chunk's decay: a fixed gate's product in 64 bits, a token gate's sum
            if (lane == 31) sm.decay = exp2_pair(fixed ? gate2_exact(a.g[h]) * L : G);
        }
        __syncthreads();
        // scores: this thread's tokens i = ti, ti + 16 against j = tj, tj + 16
        const int tj = lane & 15, ti = warp * 2 + (lane >> 4);
        {
            float2 acc[2][2] = {};
#pragma unroll 8
            for (int c = 0; c < DK; c += 4) {
                const float4 q0 = load4(sm.q + ti * LK + c), q1 = load4(sm.q + (ti + 16) * LK + c);
                const float4 k0 = load4(sm.k + tj * LK + c), k1 = load4(sm.k + (tj + 16) * LK + c);
                dot4(q0, k0, acc[0][0]);
                dot4(q0, k1, acc[0][1]);
                dot4(q1, k0, acc[1][0]);
                dot4(q1, k1, acc[1][1]);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int i = ti + 16 * x, j = tj + 16 * y;
                    sm.P[i * LP + j] = j <= i ? a.scale * ex2((float)(sm.G[i] - sm.G[j])) * (acc[x][y].x + acc[x][y].y) : 0.f;
                }
        }
        __syncthreads();
        // outputs: tokens ti, ti + 16, channels tj, tj + 16
        {
            float2 part[2][2] = {};
#pragma unroll 8
            for (int c = 0; c < DK; c += 4) {
                const float4 q0 = load4(sm.q + ti * LK + c), q1 = load4(sm.q + (ti + 16) * LK + c);
                const float4 s0 = load4(sm.S + tj * LK + c), s1 = load4(sm.S + (tj + 16) * LK + c);
                dot4(q0, s0, part[0][0]);
                dot4(q0, s1, part[0][1]);
                dot4(q1, s0, part[1][0]);
                dot4(q1, s1, part[1][1]);
            }
            float2 sum[2];  // token x: channels tj, tj + 16
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float e = sm.e[ti + 16 * x];
                sum[x] = make_float2(e * (part[x][0].x + part[x][0].y), e * (part[x][1].x + part[x][1].y));
            }
#pragma unroll 8
            for (int j = 0; j < kC; ++j) {  // (rows from L on are zeros)
                const float2 vv = make_float2(sm.v[j * LV + tj], sm.v[j * LV + tj + 16]);
                const float p0 = sm.P[ti * LP + j], p1 = sm.P[(ti + 16) * LP + j];
                sum[0] = __ffma2_rn(make_float2(p0, p0), vv, sum[0]);
                sum[1] = __ffma2_rn(make_float2(p1, p1), vv, sum[1]);
            }
            const float acc[2][2] = {{sum[0].x, sum[0].y}, {sum[1].x, sum[1].y}};
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    if (ti + 16 * x < L) out[(t0 + ti + 16 * x) * ldv + tj + 16 * y] = from_f32<Tin>(acc[x][y]);
        }
        __syncthreads();
        // S = 2^G S + sum_j w_j v_j k_j^T
        {
            float2 acc[TR][2] = {};
#pragma unroll 8
            for (int j = 0; j < kC; ++j) {
                const float4 kk = load4(sm.k + j * LK + sc);
                const float w = sm.w[j];
#pragma unroll
                for (int i = 0; i < TR; ++i) {
                    const float x = w * sm.v[j * LV + sr + i];
                    acc[i][0] = __ffma2_rn(make_float2(x, x), make_float2(kk.x, kk.y), acc[i][0]);
                    acc[i][1] = __ffma2_rn(make_float2(x, x), make_float2(kk.z, kk.w), acc[i][1]);
                }
            }
            const float2 d = sm.decay;
            const int64_t done = s.pos + t0 + L;  // tokens of the sequence so far
            const bool snap = a.n_snap > 0 && done % a.snap_stride == 0;
#pragma unroll
            for (int i = 0; i < TR; ++i) {
                float4 *p = reinterpret_cast<float4 *>(sm.S + (sr + i) * LK + sc);
                float4 x = *p;
                x.x = fmaf(d.x, x.x, fmaf(d.y, x.x, acc[i][0].x));
                x.y = fmaf(d.x, x.y, fmaf(d.y, x.y, acc[i][0].y));
                x.z = fmaf(d.x, x.z, fmaf(d.y, x.z, acc[i][1].x));
                x.w = fmaf(d.x, x.w, fmaf(d.y, x.w, acc[i][1].y));
                *p = x;
                if (snap)
                    *reinterpret_cast<float4 *>(
                        a.snaps + (((s.n * a.n_snap + done / a.snap_stride - 1) * a.H + h) * dv + r0 + sr + i) * DK + sc) = x;
            }
        }
    }
    if (a.final_state && s.j == s.nseg - 1) {  // (each thread stores what it alone wrote)
        float *to = a.final_state + (s.n * a.H + h) * dv * DK;
#pragma unroll
        for (int i = 0; i < TR; ++i)
            *reinterpret_cast<float4 *>(to + (int64_t)(r0 + sr + i) * DK + sc) =
                *reinterpret_cast<const float4 *>(sm.S + (sr + i) * LK + sc);
    }
}

// U of one segment (not its sequence's last), head and 32 value channels, and the
// segment's decay.  From the last chunk backwards, so that every weight is the sum of
// the gates after its token; it ends where nothing before could reach the segment's end.
template <int DK, typename Tin>
__global__ void __launch_bounds__(kThreads) gdn_linattn_state_simt(const Args a, int64_t dv, bool fixed) {
    constexpr int LK = DK + 4, LV = kRows + 4, TR = DK / 32;
    __shared__ __align__(16) float ks[kC * LK];
    __shared__ __align__(16) float vs[kC * LV];
    __shared__ float ws[kC];
    __shared__ float s_total;
    let_next_start();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slices = (int)(dv / kRows);
    const int64_t id = blockIdx.x;
    const int64_t h = id / slices % a.H;
    const int r0 = (int)(id % slices) * kRows;
    Slot s;
    if (!locate<true>(a, id / slices / a.H, s) || s.nseg < 2 || s.j == s.nseg - 1) return;
    const int64_t hq = h / (a.H / a.Hk);
    const Tin *k = static_cast<const Tin *>(a.k) + (s.start * a.Hk + hq) * DK;
    const Tin *v = static_cast<const Tin *>(a.v) + (s.start * a.H + h) * dv + r0;
    const int64_t ldk = a.Hk * DK, ldv = a.H * dv;
    const int sc = tid % (DK / 4) * 4, sr = tid / (DK / 4) * TR;
    float2 acc[TR][2] = {};
    // Sum of the gates after the chunk, in 64 bits: alike gates would round alike in all of thousands of
    // chunks (1.9e-5 of the state after 4,220 of them).
    double after_chunk = 0.0;
    Rows<DK, LK, Tin> kn;     // the chunk before, on its way
    Rows<kRows, LV, Tin> vn;
    float gn = 0.f;
    auto ahead = [&](int64_t t0) {
        kn.read(k + t0 * ldk, ldk, kC);
        vn.read(v + t0 * ldv, ldv, kC);
        if (warp == 0) gn = gate_of(a, fixed, s.start + t0 + lane, h);
    };
    ahead(s.len - kC);
    for (int64_t t0 = s.len - kC; t0 >= 0 && after_chunk > (double)kDead; t0 -= kC) {  // (segments here are whole chunks)
        __syncthreads();
        kn.put(ks);
        vn.put(vs);
        const float g = gn;
        if (t0 >= kC) ahead(t0 - kC);
        if (warp == 0) {
            float G, after;
            warp_scans(g, lane, G, after);
            ws[lane] = ex2((float)(after_chunk + (double)after));
            if (lane == 31) s_total = G;
        }
        __syncthreads();
        after_chunk += (double)s_total;
#pragma unroll 8
        for (int j = 0; j < kC; ++j) {
            const float4 kk = load4(ks + j * LK + sc);
            const float w = ws[j];
#pragma unroll
            for (int i = 0; i < TR; ++i) {
                const float x = w * vs[j * LV + sr + i];
                acc[i][0] = __ffma2_rn(make_float2(x, x), make_float2(kk.x, kk.y), acc[i][0]);
                acc[i][1] = __ffma2_rn(make_float2(x, x), make_float2(kk.z, kk.w), acc[i][1]);
            }
        }
    }
    float *U = a.states + (s.ss * a.H + h) * dv * DK;
#pragma unroll
    for (int i = 0; i < TR; ++i)
        *reinterpret_cast<float4 *>(U + (int64_t)(r0 + sr + i) * DK + sc) =
            make_float4(acc[i][0].x, acc[i][0].y, acc[i][1].x, acc[i][1].y);
    // the segment's decay (once it is past kDead, how far past does not matter)
    if (r0 == 0 && tid == 0) {
        a.alive[s.ss * a.H + h] = 1;
        a.tot[s.ss * a.H + h] = fixed ? gate2_exact(a.g[h]) * (double)s.len : after_chunk;
    }
}

// Start states of the segments of one sequence and head, each in the place of its first
// part's U: S_{j+1} = 2^{tot_j} S_j + sum of the parts' U_j.  A thread chains four
// elements.  What decides which U are read, and the decays, are fetched 32 segments at a
// time by the whole block; the next segment's U are in flight while the current one is
// added.
constexpr int kCombThreads = 256, kCombSegs = 32, kCombParts = 8;
__global__ void __launch_bounds__(kCombThreads) gdn_linattn_combine(const Args a, int64_t elems) {
    __shared__ float2 s_decay[kCombSegs];
    __shared__ uint32_t s_alive[kCombSegs];  // a bit per part (of the first kCombParts)
    const int64_t h = blockIdx.y, e = ((int64_t)blockIdx.z * kCombThreads + threadIdx.x) * 4;
    const int tid = threadIdx.x, parts = (int)a.parts;
    let_next_start();
    wait_for_previous();
    for (int64_t n = blockIdx.x; n < a.N; n += gridDim.x) {
        int64_t start, len;
        seq_bounds(a.cu, n, a.T, a.rows, start, len);
        int64_t nseg;
        segment_length(a, len, nseg);
        const int64_t ss = state_base(a, n);
        if (nseg < 2 || ss + nseg > a.sslots) continue;
        float *states = a.states + (ss * parts * a.H + h) * elems + e;
        float4 S = a.h0 ? *reinterpret_cast<const float4 *>(a.h0 + (n * a.H + h) * elems + e) : make_float4(0.f, 0.f, 0.f, 0.f);
        for (int64_t j0 = 0; j0 + 1 < nseg; j0 += kCombSegs) {
            const int m = (int)(nseg - 1 - j0 < kCombSegs ? nseg - 1 - j0 : kCombSegs);
            __syncthreads();
            if (tid < m) s_alive[tid] = 0;
            __syncthreads();
            for (int i = tid; i < m * parts; i += kCombThreads)
                if (a.alive[((ss + j0) * parts + i) * a.H + h]) atomicOr(&s_alive[i / parts], 1u << (i % parts));
            if (tid < m) s_decay[tid] = exp2_pair(a.tot[(ss + j0 + tid) * a.H + h]);
            __syncthreads();
            auto added = [&](int j) {
                float4 x[kCombParts], u = make_float4(0.f, 0.f, 0.f, 0.f);
                const uint32_t bits = s_alive[j];
#pragma unroll
                for (int i = 0; i < kCombParts; ++i)
                    x[i] = bits >> i & 1 ? *reinterpret_cast<const float4 *>(states + ((j0 + j) * parts + i) * a.H * elems)
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < kCombParts; ++i) {
                    u.x += x[i].x; u.y += x[i].y; u.z += x[i].z; u.w += x[i].w;
                }
                for (int i = kCombParts; i < parts; ++i)  // (very long segments)
                    if (bits >> i & 1) {
                        const float4 y = *reinterpret_cast<const float4 *>(states + ((j0 + j) * parts + i) * a.H * elems);
                        u.x += y.x; u.y += y.y; u.z += y.z; u.w += y.w;
                    }
                return u;
            };
            float4 u = added(0);
            for (int j = 0; j < m; ++j) {
                const float4 next = j + 1 < m ? added(j + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
                const float2 d = s_decay[j];
                *reinterpret_cast<float4 *>(states + (j0 + j) * parts * a.H * elems) = S;
                S.x = fmaf(d.x, S.x, fmaf(d.y, S.x, u.x));
                S.y = fmaf(d.x, S.y, fmaf(d.y, S.y, u.y));
                S.z = fmaf(d.x, S.z, fmaf(d.y, S.z, u.z));
                S.w = fmaf(d.x, S.w, fmaf(d.y, S.w, u.w));
                u = next;
            }
        }
        *reinterpret_cast<float4 *>(states + (nseg - 1) * parts * a.H * elems) = S;
    }
}

template <int DK, typename Tin>
gdn_status launch_dk(const Plan &p, const Args &a, cudaStream_t s) {
    const int64_t slices = p.dv / kRows, grid = p.slots * p.H * slices, sgrid = p.sslots * p.H * slices;
    if (grid > 0x7fffffffLL || sgrid > 0x7fffffffLL) return fail(GDN_ERR_UNSUPPORTED, "grid too large");
    constexpr size_t smem = sizeof(Smem<DK>);
    static std::atomic<uint64_t> smem_done{0};
    gdn_status st = allow_smem((const void *)gdn_linattn_simt<DK, Tin>, smem, smem_done);
    if (st != GDN_OK) return st;
    if (sgrid > 0) {
        {
            log_launch("gdn_linattn_state_simt", dim3((unsigned)sgrid), dim3(kThreads), 0);
            LaunchScope ls("gdn_linattn_state_simt", s);
            gdn_linattn_state_simt<DK, Tin><<<(unsigned)sgrid, kThreads, 0, s>>>(a, p.dv, p.fixed_gate);
        }
        if ((st = check_launch("gdn_linattn_state_simt")) != GDN_OK) return st;
        if (!a.chained && (st = launch_combine(p, a, s)) != GDN_OK) return st;
    }
    {
        log_launch("gdn_linattn_simt", dim3((unsigned)grid), dim3(kThreads), smem);
        LaunchScope ls("gdn_linattn_simt", s);
        launch_kernel(gdn_linattn_simt<DK, Tin>, dim3((unsigned)grid), dim3(kThreads), smem, s, sgrid > 0, a, p.dv,
                      p.fixed_gate);
    }
    return check_launch("gdn_linattn_simt");
}

}  // namespace

gdn_status launch_combine(const Plan &p, const Args &a, cudaStream_t s) {
    if (p.H > 65535) return fail(GDN_ERR_UNSUPPORTED, "more than 65535 heads");
    const int64_t elems = p.dv * p.dk;
    const dim3 grid((unsigned)(p.N < 64 ? p.N : 64), (unsigned)p.H,
                    (unsigned)((elems + 4 * kCombThreads - 1) / (4 * kCombThreads)));
    log_launch("gdn_linattn_combine", grid, dim3(kCombThreads), 0);
    LaunchScope ls("gdn_linattn_combine", s);
    launch_kernel(gdn_linattn_combine, grid, dim3(kCombThreads), 0, s, true, a, elems);
    return check_launch("gdn_linattn_combine");
}

gdn_status launch_simt(const Plan &p, const Args &a, int dtype, cudaStream_t s) {
    if (dtype == GDN_BF16)
        return p.dk == 128 ? launch_dk<128, __nv_bfloat16>(p, a, s) : launch_dk<64, __nv_bfloat16>(p, a, s);
    return p.dk == 128 ? launch_dk<128, float>(p, a, s) : launch_dk<64, float>(p, a, s);
}

}  // namespace lin
}  // namespace gdn
