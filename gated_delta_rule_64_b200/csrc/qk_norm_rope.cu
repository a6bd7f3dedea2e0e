// Norm of every query and key head and the position rotation, in one pass.
//
// Every value is read once and written once (4 bytes a value in bf16); bound by the latency of
// HBM at 32 warps per SM, so three heads of each group are on their way (with two: 56 us; fp32,
// of twice the bytes, keeps its registers with six blocks per SM).  Measured: 16,384 tokens of
// 16 + 16 heads, 128 wide, 54 us, 269 MB at 5.0 TB/s (0.76 of a plain copy).  A group of lanes holds one head of one token, two quads of
// four channels a lane.  Where channels i and
// i + rot / 2 rotate together, the quads of a lane are such partners, so the rotation needs
// no exchange between lanes; the unrotated channels behind them, and the neighbours 2 i,
// 2 i + 1 of the interleaved form, come as two adjacent quads.  (With eight consecutive
// channels a lane and the partner fetched from another lane the prompt shape below took
// 117 us.)  A group stays with one token, so its cosines and sines, and the weights, are
// read into registers once for all of the token's heads.
//
// The angles depend on the token alone: a block works on all heads of a few tokens and forms
// them once, in shared memory, while its first loads are in flight.  An angle is
// position * inv_freq in 64 bits, reduced to a fraction of a turn before it is rounded to
// fp32: at position 2^31 the fraction is still good to 2^-22 of a turn.
#include "linattn.cuh"

namespace gdn {
namespace lin {
namespace {

constexpr int kThreads = 128;

struct Quad {
    float2 a, b;
};
__device__ __forceinline__ uint4 load_quad(const float *p) { return __ldcs(reinterpret_cast<const uint4 *>(p)); }
__device__ __forceinline__ uint2 load_quad(const __nv_bfloat16 *p) { return __ldcs(reinterpret_cast<const uint2 *>(p)); }
__device__ __forceinline__ Quad unpack(const uint4 &w) {
    return {make_float2(__uint_as_float(w.x), __uint_as_float(w.y)), make_float2(__uint_as_float(w.z), __uint_as_float(w.w))};
}
__device__ __forceinline__ Quad unpack(const uint2 &w) {
    return {make_float2(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u)),
            make_float2(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u))};
}
__device__ __forceinline__ void store_quad(float *p, const Quad &x) {
    *reinterpret_cast<float4 *>(p) = make_float4(x.a.x, x.a.y, x.b.x, x.b.y);
}
__device__ __forceinline__ void store_quad(__nv_bfloat16 *p, const Quad &x) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(x.a.x, x.a.y), hi = __floats2bfloat162_rn(x.b.x, x.b.y);
    *reinterpret_cast<uint2 *>(p) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ Quad scale(const Quad &x, const Quad &w) { return {mul2(x.a, w.a), mul2(x.b, w.b)}; }

template <typename Tin> struct Raw;
template <> struct Raw<float> { typedef uint4 type; };
template <> struct Raw<__nv_bfloat16> { typedef uint2 type; };

struct RopeArgs {
    const void *q, *k;
    const int32_t *pos;
    const float *inv_freq, *qw, *kw;
    void *q_out, *k_out;
    int64_t rows, q_stride, k_stride;
    int hq, hk, rot, tokens;  // tokens: per block, a power of two
    int half_bits;            // 2^half_bits >= rot / 2
    int step_bits;            // 2^step_bits groups of lanes share a token
    bool interleaved;
    float eps, offset;
};

template <int D, typename Tin, bool INTER>
__global__ void __launch_bounds__(kThreads, sizeof(Tin) == 2 ? 8 : 6) gdn_qk_norm_rope_kernel(const RopeArgs a) {
    constexpr int kGroup = D / 8;               // lanes of a head
    constexpr int kGroups = kThreads / kGroup;  // of a block; as many tokens at most
    __shared__ __align__(16) float s_cos[kGroups * D / 2], s_sin[kGroups * D / 2];
    const int tid = threadIdx.x, sub = tid % kGroup, group = tid / kGroup;
    const int64_t row0 = (int64_t)blockIdx.x * a.tokens;
    const int tokens = (int)(a.rows - row0 < a.tokens ? a.rows - row0 : a.tokens);
    const int half = a.rot / 2;
    // this lane's quads: channels c0 .. c0 + 3 and c1 .. c1 + 3
    const bool partners = !INTER && 4 * sub < half;
    const int c0 = INTER ? 8 * sub : (partners ? 4 * sub : a.rot + 8 * (sub - half / 4));
    const int c1 = partners ? c0 + half : c0 + 4;
    // this group's token and heads: h0, h0 + step, ...
    const int sb = a.step_bits, step = 1 << sb, t = group >> sb, h0 = group & (step - 1);
    const bool live = t < tokens;
    const int64_t row = row0 + (live ? t : 0);

    typedef typename Raw<Tin>::type raw;
    const int64_t qo = (int64_t)h0 * D;
    const Tin *q = static_cast<const Tin *>(a.q) + row * a.q_stride + qo, *k = static_cast<const Tin *>(a.k) + row * a.k_stride + qo;
    const int nq = live ? (a.hq - h0 + step - 1) >> sb : 0, nk = live ? (a.hk - h0 + step - 1) >> sb : 0;  // (0 past the last head)
    raw x0 = {}, x1 = {}, y0 = {}, y1 = {}, z0 = {}, z1 = {};
    if (nq > 0) {  // in flight while the angles are formed
        x0 = load_quad(q + c0);
        x1 = load_quad(q + c1);
    }
    if (nq > 1) {
        y0 = load_quad(q + step * D + c0);
        y1 = load_quad(q + step * D + c1);
    }
    if (nq > 2) {
        z0 = load_quad(q + 2 * step * D + c0);
        z1 = load_quad(q + 2 * step * D + c1);
    }
    if (half > 0) {  // a thread takes one frequency, of every (128 / width)-th token
        const int i = tid & ((1 << a.half_bits) - 1), stride = kThreads >> a.half_bits;
        if (i < half) {
            const double f = (double)a.inv_freq[i] * 0.15915494309189533577;
            for (int u = tid >> a.half_bits; u < tokens; u += stride) {
                const double turn = (double)a.pos[row0 + u] * f;
                sincospif((float)(2.0 * (turn - rint(turn))), &s_sin[u * half + i], &s_cos[u * half + i]);
            }
        }
    }
    __syncthreads();
    Quad cs = {make_float2(1.f, 1.f), make_float2(1.f, 1.f)}, sn = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    if (live && (INTER ? c0 < a.rot : partners)) {  // (interleaved: the lane's four pairs in order)
        const int i = t * half + (INTER ? c0 / 2 : c0);
        cs = unpack(*reinterpret_cast<const uint4 *>(s_cos + i));
        sn = unpack(*reinterpret_cast<const uint4 *>(s_sin + i));
    }
    auto weight = [&](const float *w, int c) {
        return w ? Quad{make_float2(a.offset + w[c], a.offset + w[c + 1]), make_float2(a.offset + w[c + 2], a.offset + w[c + 3])}
                 : Quad{make_float2(1.f, 1.f), make_float2(1.f, 1.f)};
    };
    // `n` heads of this group, of `most` that any group of the warp has (the shuffles are warp-wide);
    // x, y and z hold the first three.  With the weights taken into the angles (w cos, w sin) a pair of
    // partners is two multiply-adds each, and the norm one product at the end.
    auto run = [&](const Tin *src, Tin *dst, int n, int most, const float *wp) {
        const Quad w0 = weight(wp, c0), w1 = weight(wp, c1);
        const Quad cp = scale(w0, cs), cr = scale(w1, cs), sp = scale(w0, sn);
        const Quad sr = {make_float2(-w1.a.x * sn.a.x, -w1.a.y * sn.a.y), make_float2(-w1.b.x * sn.b.x, -w1.b.y * sn.b.y)};
        const Tin *ahead = src + 3 * step * D;
        for (int i = 0; i < most; ++i) {
            const Quad p = unpack(x0), r = unpack(x1);
            x0 = y0;
            x1 = y1;
            y0 = z0;
            y1 = z1;
            if (i + 3 < n) {
                z0 = load_quad(ahead + c0);
                z1 = load_quad(ahead + c1);
            }
            ahead += step * D;
            float2 s2 = mul2(p.a, p.a);
            s2 = fma2(p.b, p.b, s2);
            s2 = fma2(r.a, r.a, s2);
            s2 = fma2(r.b, r.b, s2);
            float ss = s2.x + s2.y;
#pragma unroll
            for (int o = kGroup / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float f = rsqrtf(ss * (1.f / D) + a.eps);
            const float2 ff = make_float2(f, f);
            Quad u, v;
            if (INTER) {
                auto turn = [](float2 x, float2 w, float c, float s) {
                    const float lo = x.x * w.x, hi = x.y * w.y;
                    return make_float2(lo * c - hi * s, hi * c + lo * s);
                };
                u = {turn(p.a, w0.a, cs.a.x, sn.a.x), turn(p.b, w0.b, cs.a.y, sn.a.y)};
                v = {turn(r.a, w1.a, cs.b.x, sn.b.x), turn(r.b, w1.b, cs.b.y, sn.b.y)};
            } else {
                u = {fma2(p.a, cp.a, mul2(r.a, sr.a)), fma2(p.b, cp.b, mul2(r.b, sr.b))};
                v = {fma2(r.a, cr.a, mul2(p.a, sp.a)), fma2(r.b, cr.b, mul2(p.b, sp.b))};
            }
            if (i < n) {
                store_quad(dst + c0, Quad{mul2(u.a, ff), mul2(u.b, ff)});
                store_quad(dst + c1, Quad{mul2(v.a, ff), mul2(v.b, ff)});
            }
            dst += step * D;
        }
    };
    run(q, static_cast<Tin *>(a.q_out) + row * a.hq * D + qo, nq, (a.hq + step - 1) >> sb, a.qw);
    if (a.hk > 0) {
        if (nk > 0) {
            x0 = load_quad(k + c0);
            x1 = load_quad(k + c1);
        }
        if (nk > 1) {
            y0 = load_quad(k + step * D + c0);
            y1 = load_quad(k + step * D + c1);
        }
        if (nk > 2) {
            z0 = load_quad(k + 2 * step * D + c0);
            z1 = load_quad(k + 2 * step * D + c1);
        }
        run(k, static_cast<Tin *>(a.k_out) + row * a.hk * D + qo, nk, (a.hk + step - 1) >> sb, a.kw);
    }
}

template <int D>
gdn_status launch_d(const gdn_qk_rope_desc &d, RopeArgs &a, cudaStream_t s) {
    // Tokens of a block: eight heads to a group of lanes (the angles and weights are then a
    // small part of its work: four heads or sixteen take 60 and 59 us), fewer where
    // the tokens would not fill the GPU twice.
    constexpr int kGroups = kThreads / (D / 8);
    const int heads = a.hq + a.hk;
    int tokens = 1;
    while (2 * tokens <= kGroups && tokens * heads < 8 * kGroups && d.rows / (2 * tokens) >= 296) tokens *= 2;
    a.tokens = tokens;
    for (a.step_bits = 0; (tokens << a.step_bits) < kGroups; ++a.step_bits) {
    }
    const unsigned grid = (unsigned)((d.rows + tokens - 1) / tokens);
    LaunchScope ls("gdn_qk_norm_rope_kernel", s);
    auto kern = d.dtype == GDN_BF16 ? (a.interleaved ? gdn_qk_norm_rope_kernel<D, __nv_bfloat16, true>
                                                     : gdn_qk_norm_rope_kernel<D, __nv_bfloat16, false>)
                                    : (a.interleaved ? gdn_qk_norm_rope_kernel<D, float, true>
                                                     : gdn_qk_norm_rope_kernel<D, float, false>);
    kern<<<grid, kThreads, 0, s>>>(a);
    return check_launch("gdn_qk_norm_rope_kernel");
}

}  // namespace

gdn_status launch_qk_norm_rope(const gdn_qk_rope_desc &d, const void *q, const void *k, const int32_t *pos,
                               const float *inv_freq, const float *qw, const float *kw, void *q_out, void *k_out,
                               cudaStream_t s) {
    RopeArgs a{q, k, pos, inv_freq, qw, kw, q_out, k_out, d.rows, d.q_stride, d.k_stride, d.hq, d.hk, d.rot, 1, 0, 0,
               d.interleaved != 0, d.eps, d.weight_offset};
    while ((1 << a.half_bits) < d.rot / 2) ++a.half_bits;
    return d.head_dim == 64 ? launch_d<64>(d, a, s) : d.head_dim == 128 ? launch_d<128>(d, a, s) : launch_d<256>(d, a, s);
}

}  // namespace lin
}  // namespace gdn
