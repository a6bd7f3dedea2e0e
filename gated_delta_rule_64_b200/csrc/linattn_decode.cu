// One token of linear attention with a decay for each head, state in place:
//     z_i = sum_c S_ic q_c,  o_i = alpha z_i + v_i (k . q),  S'_ic = alpha S_ic + v_i k_c
// (q scaled).  The d_v x d_k fp32 state is read once and written once; everything else
// is a few hundred bytes per head, so the kernel is bound by HBM bandwidth.  Rows are
// independent: the layout is that of the delta rule's decode (a warp per eight rows, a
// lane per d_k / 32 columns, the eight rows' sums reduce-scattered over the warp), without
// its correction of v, so the new state does not wait for a reduction.  Measured: 256
// sequences of 32 heads, 128 x 128: 184 us, 1.08 GB at 5.9 TB/s (0.90 of a plain copy).
#include "decode_rows.cuh"
#include "linattn.cuh"

namespace gdn {
namespace lin {
namespace {

using dec::kRowsPerWarp;
using dec::kWarps;

template <int DK, int DV, typename Tin>
__global__ void __launch_bounds__(kWarps * 32)
gdn_linattn_decode_kernel(const Tin *__restrict__ q, const Tin *__restrict__ k, const Tin *__restrict__ v,
                          const float *__restrict__ g, float *__restrict__ state, Tin *__restrict__ out, int64_t H,
                          int64_t Hk, float scale, bool fixed) {
    constexpr int VEC = DK / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t unit = blockIdx.x, b = unit / H, h = unit % H;
    const int row0 = ((int)blockIdx.y * kWarps + warp) * kRowsPerWarp;
    float *S = state + (unit * DV + row0) * (int64_t)DK + lane * VEC;
    float s[kRowsPerWarp][VEC];
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) dec::Vec4<VEC>::ld(S + (int64_t)r * DK, s[r]);
    const int64_t tq = (b * Hk + h / (H / Hk)) * DK + lane * VEC;
    float kr[VEC], qr[VEC], kq = 0.f;
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
        kr[c] = to_f32<Tin>(k[tq + c]);
        qr[c] = scale * to_f32<Tin>(q[tq + c]);
        kq = fmaf(kr[c], qr[c], kq);
    }
    const float a = expf(g[fixed ? h : unit]);
    const float vl = lane < 8 ? to_f32<Tin>(v[unit * DV + row0 + lane]) : 0.f;
    kq = dec::warp_sum(kq);
    float zp[kRowsPerWarp];
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) {
        const float vr = __shfl_sync(0xffffffffu, vl, r);
        float z = 0.f;
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            z = fmaf(s[r][c], qr[c], z);
            s[r][c] = fmaf(a, s[r][c], vr * kr[c]);
        }
        zp[r] = z;
        dec::Vec4<VEC>::st(S + (int64_t)r * DK, s[r]);
    }
    const float z = dec::reduce8(zp, lane);
    const int R = (lane >> 2) & 7;
    const float vR = __shfl_sync(0xffffffffu, vl, R);
    if ((lane & 3) == 0) out[unit * DV + row0 + R] = from_f32<Tin>(fmaf(a, z, vR * kq));
}

template <int DK, int DV, typename Tin>
gdn_status launch_dkv(const gdn_desc &d, const void *q, const void *k, const void *v, const float *g, float *state,
                      void *out, cudaStream_t s) {
    const int64_t units = d.B * d.H;
    if (units > 0x7fffffffLL) return fail(GDN_ERR_UNSUPPORTED, "too many (sequence, head) pairs");
    const dim3 grid((unsigned)units, (unsigned)(DV / (kWarps * kRowsPerWarp))), block(kWarps * 32);
    LaunchScope ls("gdn_linattn_decode_kernel", s);
    gdn_linattn_decode_kernel<DK, DV, Tin><<<grid, block, 0, s>>>(
        (const Tin *)q, (const Tin *)k, (const Tin *)v, g, state, (Tin *)out, d.H, qk_heads(d), d.scale,
        d.gate == GDN_GATE_CONST);
    return check_launch("gdn_linattn_decode_kernel");
}

template <typename Tin>
gdn_status launch_t(const gdn_desc &d, const void *q, const void *k, const void *v, const float *g, float *state,
                    void *out, cudaStream_t s) {
    if (d.dk == 128)
        return d.dv == 128 ? launch_dkv<128, 128, Tin>(d, q, k, v, g, state, out, s)
                           : launch_dkv<128, 64, Tin>(d, q, k, v, g, state, out, s);
    return d.dv == 128 ? launch_dkv<64, 128, Tin>(d, q, k, v, g, state, out, s)
                       : launch_dkv<64, 64, Tin>(d, q, k, v, g, state, out, s);
}

}  // namespace

gdn_status launch_decode(const gdn_desc &d, const void *q, const void *k, const void *v, const float *g, float *state,
                         void *out, cudaStream_t s) {
    return d.dtype == GDN_BF16 ? launch_t<__nv_bfloat16>(d, q, k, v, g, state, out, s)
                               : launch_t<float>(d, q, k, v, g, state, out, s);
}

}  // namespace lin
}  // namespace gdn
