// Norm of every query and key head and the position rotation, in one pass.
//
// Bound by HBM bandwidth: every value is read once and written once (4 bytes a value
// in bf16), and by the instructions around that: about 60 per 512 bytes read.  A group of lanes
// holds one head of one token, two quads of four channels a lane.  Where channels i and
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

constexpr int kThreads = 256;

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
    bool interleaved;
    float eps, offset;
};

template <int D, typename Tin>
__global__ void __launch_bounds__(kThreads, 4) gdn_qk_norm_rope_kernel(const RopeArgs a) {
    constexpr int kGroup = D / 8;               // lanes of a head
    constexpr int kGroups = kThreads / kGroup;  // of a block; as many tokens at most
    __shared__ __align__(16) float s_cos[kGroups * D / 2], s_sin[kGroups * D / 2];
    const int tid = threadIdx.x, sub = tid % kGroup, group = tid / kGroup;
    const int64_t row0 = (int64_t)blockIdx.x * a.tokens;
    const int tokens = (int)(a.rows - row0 < a.tokens ? a.rows - row0 : a.tokens);
    const int heads = a.hq + a.hk, half = a.rot / 2;
    // this lane's quads: channels c0 .. c0 + 3 and c1 .. c1 + 3
    const bool partners = !a.interleaved && 4 * sub < half;
    const int c0 = partners ? 4 * sub : (a.interleaved ? 8 * sub : a.rot + 8 * (sub - half / 4));
    const int c1 = partners ? c0 + half : c0 + 4;
    // this group's token and heads: h0, h0 + step, ...
    const int step = kGroups / a.tokens, t = group / step, h0 = group % step;
    const bool live = t < tokens;
    const int64_t row = row0 + (live ? t : 0);
    const Tin *q = static_cast<const Tin *>(a.q) + row * a.q_stride, *k = static_cast<const Tin *>(a.k) + row * a.k_stride;
    Tin *qo = static_cast<Tin *>(a.q_out) + row * a.hq * D, *ko = static_cast<Tin *>(a.k_out) + row * a.hk * D;

    typedef typename Raw<Tin>::type raw;
    raw x0 = {}, x1 = {}, y0 = {}, y1 = {};
    auto load = [&](int h, raw &lo, raw &hi) {
        if (live && h < heads) {
            const Tin *p = h < a.hq ? q + h * D : k + (h - a.hq) * D;
            lo = load_quad(p + c0);
            hi = load_quad(p + c1);
        }
    };
    load(h0, x0, x1);  // in flight while the angles are formed
    load(h0 + step, y0, y1);
    for (int i = tid; i < tokens * half; i += kThreads) {
        const double turn = (double)a.pos[row0 + i / half] * (double)a.inv_freq[i % half] * 0.15915494309189533577;
        sincospif((float)(2.0 * (turn - rint(turn))), &s_sin[i], &s_cos[i]);
    }
    auto weight = [&](const float *w, int c) {
        return w ? Quad{make_float2(a.offset + w[c], a.offset + w[c + 1]), make_float2(a.offset + w[c + 2], a.offset + w[c + 3])}
                 : Quad{make_float2(1.f, 1.f), make_float2(1.f, 1.f)};
    };
    Quad w0 = weight(a.qw, c0), w1 = weight(a.qw, c1);
    __syncthreads();
    Quad cos4 = {make_float2(1.f, 1.f), make_float2(1.f, 1.f)}, sin4 = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    // (interleaved: the lane's four angles belong to its channel pairs in order)
    const bool turns = live && (a.interleaved ? c0 < a.rot : partners);
    if (turns) {
        const int i = t * half + (a.interleaved ? c0 / 2 : c0);
        cos4 = unpack(*reinterpret_cast<const uint4 *>(s_cos + i));
        sin4 = unpack(*reinterpret_cast<const uint4 *>(s_sin + i));
    }
    bool keys = false;  // the weights are the keys'
    // every lane of a warp goes round equally often (the shuffles are warp-wide)
    for (int h = h0, n = (heads + step - 1) / step; n > 0; --n, h += step) {
        const raw r0 = x0, r1 = x1;
        x0 = y0;
        x1 = y1;
        load(h + 2 * step, y0, y1);
        Quad p = unpack(r0), r = unpack(r1);
        float2 s2 = mul2(p.a, p.a);
        s2 = fma2(p.b, p.b, s2);
        s2 = fma2(r.a, r.a, s2);
        s2 = fma2(r.b, r.b, s2);
        float ss = s2.x + s2.y;
#pragma unroll
        for (int o = kGroup / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float rs = rsqrtf(ss * (1.f / D) + a.eps);
        if (!live || h >= heads) continue;
        if (h >= a.hq && !keys) {
            keys = true;
            w0 = weight(a.kw, c0);
            w1 = weight(a.kw, c1);
        }
        const Quad rs4 = {make_float2(rs, rs), make_float2(rs, rs)};
        p = scale(scale(p, rs4), w0);
        r = scale(scale(r, rs4), w1);
        if (turns) {
            if (partners) {
                const Quad ps = scale(p, sin4), rsn = scale(r, Quad{make_float2(-sin4.a.x, -sin4.a.y), make_float2(-sin4.b.x, -sin4.b.y)});
                p = {fma2(p.a, cos4.a, rsn.a), fma2(p.b, cos4.b, rsn.b)};
                r = {fma2(r.a, cos4.a, ps.a), fma2(r.b, cos4.b, ps.b)};
            } else {
                auto turn = [](float2 x, float c, float s) { return make_float2(x.x * c - x.y * s, x.y * c + x.x * s); };
                p = {turn(p.a, cos4.a.x, sin4.a.x), turn(p.b, cos4.a.y, sin4.a.y)};
                r = {turn(r.a, cos4.b.x, sin4.b.x), turn(r.b, cos4.b.y, sin4.b.y)};
            }
        }
        Tin *o = h < a.hq ? qo + h * D : ko + (h - a.hq) * D;
        store_quad(o + c0, p);
        store_quad(o + c1, r);
    }
}

template <int D>
gdn_status launch_d(const gdn_qk_rope_desc &d, RopeArgs &a, cudaStream_t s) {
    // Tokens of a block: eight heads to a group of lanes (the angles and weights are then a
    // small part of its work), fewer where the tokens would not fill the GPU twice.
    constexpr int kGroups = kThreads / (D / 8);
    const int heads = a.hq + a.hk;
    int tokens = 1;
    while (2 * tokens <= kGroups && tokens * heads < 8 * kGroups && d.rows / (2 * tokens) >= 296) tokens *= 2;
    a.tokens = tokens;
    const unsigned grid = (unsigned)((d.rows + tokens - 1) / tokens);
    LaunchScope ls("gdn_qk_norm_rope_kernel", s);
    if (d.dtype == GDN_BF16)
        gdn_qk_norm_rope_kernel<D, __nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
    else
        gdn_qk_norm_rope_kernel<D, float><<<grid, kThreads, 0, s>>>(a);
    return check_launch("gdn_qk_norm_rope_kernel");
}

}  // namespace

gdn_status launch_qk_norm_rope(const gdn_qk_rope_desc &d, const void *q, const void *k, const int32_t *pos,
                               const float *inv_freq, const float *qw, const float *kw, void *q_out, void *k_out,
                               cudaStream_t s) {
    RopeArgs a{q, k, pos, inv_freq, qw, kw, q_out, k_out, d.rows, d.q_stride, d.k_stride, d.hq, d.hk, d.rot, 1,
               d.interleaved != 0, d.eps, d.weight_offset};
    return d.head_dim == 64 ? launch_d<64>(d, a, s) : d.head_dim == 128 ? launch_d<128>(d, a, s) : launch_d<256>(d, a, s);
}

}  // namespace lin
}  // namespace gdn
