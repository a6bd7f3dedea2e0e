// Norm of every query and key head and the position rotation, in one pass.
//
// Bound by HBM bandwidth: every value is read once and written once (4 bytes a value
// in bf16), the rest is a few multiply-adds.  A group of lanes holds one head of one
// token (E consecutive channels a lane, 16 bytes or two times 16), so the mean square
// is a shuffle reduction inside the group and the rotation's partner channel, rot / 2
// away, is in another lane of it at the same place.  The angles depend on the token
// alone: a block works on all heads of a few tokens and forms the cosines and sines
// once, in shared memory, while its first loads are in flight.  An angle
// is position * inv_freq in 64 bits, reduced to a fraction of a turn before it is
// rounded to fp32: at position 2^31 the fraction is still good to 2^-22 of a turn.
#include "linattn.cuh"

namespace gdn {
namespace lin {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;  // tokens of a block

template <typename Tin, int E>
struct Lane;  // E consecutive values of a lane, as they lie in memory
template <> struct Lane<__nv_bfloat16, 8> {
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { w = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&x)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <int E> struct Lane<float, E> {
    float4 w[E / 4];
    __device__ __forceinline__ void load(const float *p) {
#pragma unroll
        for (int i = 0; i < E / 4; ++i) w[i] = __ldcs(reinterpret_cast<const float4 *>(p) + i);
    }
    __device__ __forceinline__ void get(float (&x)[E]) const {
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
            x[4 * i] = w[i].x; x[4 * i + 1] = w[i].y; x[4 * i + 2] = w[i].z; x[4 * i + 3] = w[i].w;
        }
    }
    static __device__ __forceinline__ void store(float *p, const float (&x)[E]) {
#pragma unroll
        for (int i = 0; i < E / 4; ++i)
            reinterpret_cast<float4 *>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    }
};

struct RopeArgs {
    const void *q, *k;
    const int32_t *pos;
    const float *inv_freq, *qw, *kw;
    void *q_out, *k_out;
    int64_t rows, q_stride, k_stride;
    int hq, hk, rot, tokens;  // tokens: per block
    bool interleaved;
    float eps, offset;
};

template <int D, typename Tin>
__global__ void __launch_bounds__(kThreads) gdn_qk_norm_rope_kernel(const RopeArgs a) {
    constexpr int kVec = 16 / (int)sizeof(Tin);
    constexpr int E = D / 32 > kVec ? D / 32 : kVec;  // channels of a lane
    constexpr int kGroup = D / E;                     // lanes of a head
    constexpr int kGroups = kThreads / kGroup;
    __shared__ float2 cs[kMaxTokens * D / 2];
    const int tid = threadIdx.x, sub = tid % kGroup, group = tid / kGroup;
    const int64_t row0 = (int64_t)blockIdx.x * a.tokens;
    const int tokens = (int)(a.rows - row0 < a.tokens ? a.rows - row0 : a.tokens);
    const int heads = a.hq + a.hk, items = tokens * heads, half = a.rot / 2;

    auto source = [&](int item) {
        const int t = item / heads, h = item % heads;
        const int64_t row = row0 + t;
        return h < a.hq ? static_cast<const Tin *>(a.q) + row * a.q_stride + (int64_t)h * D + sub * E
                        : static_cast<const Tin *>(a.k) + row * a.k_stride + (int64_t)(h - a.hq) * D + sub * E;
    };
    Lane<Tin, E> cur, next;
    if (group < items) cur.load(source(group));  // in flight while the angles are formed
    for (int i = tid; i < tokens * half; i += kThreads) {
        const double turn = (double)a.pos[row0 + i / half] * (double)a.inv_freq[i % half] * 0.15915494309189533577;
        float s, c;
        sincospif((float)(2.0 * (turn - rint(turn))), &s, &c);
        cs[i] = make_float2(c, s);
    }
    __syncthreads();
    // every lane of a warp makes the same number of turns (the shuffles are warp-wide)
    const int turns = (items + kGroups - 1) / kGroups;
    for (int n = 0; n < turns; ++n) {
        const int item = n * kGroups + group;
        const bool on = item < items;
        if (item + kGroups < items) next.load(source(item + kGroups));
        float x[E];
        if (on) {
            cur.get(x);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) x[i] = 0.f;
        }
        const int t = on ? item / heads : 0, h = on ? item % heads : 0;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = kGroup / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(ss * (1.f / D) + a.eps);
        const float *w = h < a.hq ? a.qw : a.kw;
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] *= r;
        if (w) {
#pragma unroll
            for (int i = 0; i < E; i += 4) {
                const float4 wv = make_float4(w[sub * E + i], w[sub * E + i + 1], w[sub * E + i + 2], w[sub * E + i + 3]);
                x[i] *= a.offset + wv.x;
                x[i + 1] *= a.offset + wv.y;
                x[i + 2] *= a.offset + wv.z;
                x[i + 3] *= a.offset + wv.w;
            }
        }
        if (half > 0) {
            const int c0 = sub * E;  // this lane's first channel
            if (a.interleaved) {
                if (c0 < a.rot) {
                    const float2 *f = cs + t * half + c0 / 2;
#pragma unroll
                    for (int i = 0; i < E; i += 2) {
                        const float2 z = f[i / 2];
                        const float lo = x[i], hi = x[i + 1];
                        x[i] = lo * z.x - hi * z.y;
                        x[i + 1] = hi * z.x + lo * z.y;
                    }
                }
            } else {
                const bool low = c0 < half, rotated = c0 < a.rot;
                const int step = half / E;  // lanes to the partner channel
                const int from = (int)(threadIdx.x & 31) + (rotated ? (low ? step : -step) : 0);
                const float2 *f = cs + t * half + (low ? c0 : (rotated ? c0 - half : 0));
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const float other = __shfl_sync(0xffffffffu, x[i], from);
                    if (rotated) {
                        const float2 z = f[i];
                        x[i] = low ? x[i] * z.x - other * z.y : x[i] * z.x + other * z.y;
                    }
                }
            }
        }
        if (on) {
            const int64_t row = row0 + t;
            Tin *to = h < a.hq ? static_cast<Tin *>(a.q_out) + (row * a.hq + h) * (int64_t)D
                               : static_cast<Tin *>(a.k_out) + (row * a.hk + h - a.hq) * (int64_t)D;
            Lane<Tin, E>::store(to + sub * E, x);
        }
        cur = next;
    }
}

template <int D>
gdn_status launch_d(const gdn_qk_rope_desc &d, RopeArgs &a, cudaStream_t s) {
    // tokens of a block: about 64 heads, so that the angles of a token with few heads
    // do not cost a block of their own; one where the tokens do not fill the GPU twice
    const int heads = a.hq + a.hk;
    int64_t tokens = 64 / heads < 1 ? 1 : (64 / heads > kMaxTokens ? kMaxTokens : 64 / heads);
    if (d.rows / tokens < 296) tokens = d.rows / 296 > 1 ? d.rows / 296 : 1;
    a.tokens = (int)tokens;
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
