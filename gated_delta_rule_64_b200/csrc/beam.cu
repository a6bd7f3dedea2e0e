// One step of beam search over recurrent states: the selection over beams and
// vocabulary, and the reordering of the states.
//
// Selection.  Two kernels, one pass over the logits.  A block of the first reads a
// slice of one beam's logits into registers, with 16-byte loads, and leaves the slice's
// maximum, its sum of exponentials and its K best logits (a beam's order is its logits'
// order: the beam's score and normaliser add the same to all of them).  A block of the second
// joins a request's slices: the normaliser of each beam in 64 bits, the scores of the
// W * slices * K candidates, and the K best of those.
//
// The K best of a slice.  Every thread's best is known after the pass over its registers; the
// K-th best T of the 256 thread bests (a binary search over the bits of its key by
// one warp) is a lower bound of the slice's K-th best, and only the K threads whose best
// is at least T can hold values above it.  Those values, at least K and on random logits
// little more, go to shared memory, where each one's rank is the number of better
// ones.  Keys are (value, lowest index first), all different, so ties need no care.
//
// Reordering.  A thread owns 16 bytes of every beam's row of one request: it reads the
// parents' bytes of all beams that change, then writes them, so the move is in place
// without a second buffer and rows that stay are neither read nor written.
#include "linattn.cuh"

namespace gdn {
namespace lin {
namespace {

constexpr int kThreads = 256;
constexpr int kEach = 32;                     // logits of a thread
constexpr int kSlice = kThreads * kEach;      // logits of a block
constexpr int kMaxK = 64;

// A value's bits, ordered as unsigned integers; NaN counts as -infinity.
__device__ __forceinline__ uint32_t order_bits(float x) {
    if (x != x) x = -INFINITY;
    if (x == 0.f) x = 0.f;  // -0 and 0 are equal
    const uint32_t u = __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

template <typename Tin> __device__ __forceinline__ float as_float(Tin x) { return to_f32<Tin>(x); }

// Partial results of a slice: maximum and sum of exponentials below it, then K keys.
struct SliceHead {
    float max, sum;
};

// The K-th largest of the 256 keys in `best` (all different but for zeros, of which any
// number may stand for threads without a value), by one warp: each lane holds eight.
__device__ __forceinline__ unsigned long long kth_of_256(const unsigned long long *best, int K, int lane) {
    unsigned long long x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = best[lane + 32 * i];
    unsigned long long t = 0;
    for (int bit = 63; bit >= 0; --bit) {
        const unsigned long long c = t | (1ull << bit);
        int n = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) n += __popc(__ballot_sync(0xffffffffu, x[i] >= c));
        if (n >= K) t = c;
        if (n == K) break;  // exactly K at or above c: a bound as good as the K-th itself
    }
    return t;
}

template <typename Tin>
__global__ void __launch_bounds__(kThreads)
gdn_beam_slices(const Tin *__restrict__ logits, int64_t row_stride, int V, int K, int nsl, SliceHead *__restrict__ heads,
                unsigned long long *__restrict__ keys) {
    __shared__ unsigned long long best[kThreads];
    __shared__ unsigned long long found[kMaxK * kEach];
    __shared__ float red_m[kThreads / 32], red_s[kThreads / 32];
    __shared__ unsigned long long s_bound;
    __shared__ int s_count;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / nsl;
    const int sl = (int)(blockIdx.x % nsl), i0 = sl * kSlice;
    const Tin *p = logits + row * row_stride;
    constexpr int kVec = 16 / (int)sizeof(Tin);
    const bool wide = ((uintptr_t)(p + i0) & 15) == 0;
    // logit e of this thread: index i0 + (e / kVec) * 256 kVec + tid * kVec + e % kVec
    float x[kEach];
    auto index_of = [&](int e) { return i0 + (e / kVec) * (kThreads * kVec) + tid * kVec + e % kVec; };
#pragma unroll
    for (int c = 0; c < kEach / kVec; ++c) {
        const int i = index_of(c * kVec);
        if (wide && i + kVec <= V) {
            const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(p + i));
            const Tin *t = reinterpret_cast<const Tin *>(&w);
#pragma unroll
            for (int e = 0; e < kVec; ++e) x[c * kVec + e] = as_float<Tin>(t[e]);
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) x[c * kVec + e] = i + e < V ? as_float<Tin>(p[i + e]) : -INFINITY;
        }
    }
    if (tid == 0) s_count = 0;
    // the thread's best (lowest index among equals), its maximum with NaN seen
    unsigned long long mine = 0;
    float m = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        nan |= x[e] != x[e];
        m = fmaxf(m, x[e]);
    }
    auto key_of = [&](int e) {
        const int i = index_of(e);
        return i < V ? ((unsigned long long)order_bits(x[e]) << 32) | (uint32_t)~i : 0ull;
    };
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const unsigned long long kx = key_of(e);
        mine = kx > mine ? kx : mine;
    }
    best[tid] = mine;
    // maximum of the block, then the sum of 2^((x - max) log2 e)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) red_m[warp] = m;
    const bool any_nan = __syncthreads_or(nan);
    m = red_m[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) m = fmaxf(m, red_m[w]);
    float sum = 0.f;
    if (m > -INFINITY) {
#pragma unroll
        for (int e = 0; e < kEach; ++e) sum += x[e] > -INFINITY ? exp2f((x[e] - m) * kLog2e) : 0.f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) red_s[warp] = sum;
    if (warp == 0) {
        const unsigned long long t = kth_of_256(best, K, lane);
        if (lane == 0) s_bound = t;
    }
    __syncthreads();
    if (tid == 0) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) t += red_s[w];
        heads[blockIdx.x] = SliceHead{any_nan ? NAN : m, t};
    }
    const unsigned long long bound = s_bound > 0 ? s_bound : 1;
    if (mine >= bound) {  // at most K threads
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const unsigned long long kx = key_of(e);
            if (kx >= bound) found[atomicAdd(&s_count, 1)] = kx;
        }
    }
    __syncthreads();
    const int n = s_count;
    unsigned long long *to = keys + (int64_t)blockIdx.x * K;
    for (int i = tid; i < n; i += kThreads) {
        const unsigned long long kx = found[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += found[j] > kx;
        if (rank < K) to[rank] = kx;
    }
    for (int i = n + tid; i < K; i += kThreads) to[i] = 0;  // fewer values than K
}

// Joins the slices of one request.
struct Cand {
    double score;
    int flat;
    __device__ __forceinline__ bool better(const Cand &o) const {
        return score > o.score || (score == o.score && flat < o.flat);
    }
};

__global__ void __launch_bounds__(kThreads)
gdn_beam_join(const float *__restrict__ scores, int W, int V, int K, int nsl, const SliceHead *__restrict__ heads,
              const unsigned long long *__restrict__ keys, float *__restrict__ out_scores,
              int32_t *__restrict__ out_parent, int32_t *__restrict__ out_token) {
    __shared__ double s_add[64];    // a beam's score minus its normaliser (not finite: all its scores are -infinity)
    __shared__ Cand s_best[kThreads];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t b = blockIdx.x;
    for (int w = warp; w < W; w += kThreads / 32) {
        const SliceHead *hd = heads + (b * W + w) * nsl;
        float m = -INFINITY;
        bool nan = false;
        for (int i = lane; i < nsl; i += 32) {
            nan |= hd[i].max != hd[i].max;
            m = fmaxf(m, hd[i].max);
        }
        nan = __any_sync(0xffffffffu, nan);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        double sum = 0.0;
        for (int i = lane; i < nsl; i += 32)
            if (hd[i].max > -INFINITY) sum += (double)hd[i].sum * exp((double)hd[i].max - (double)m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) {
            const double add = (scores ? (double)scores[b * W + w] : 0.0) - ((double)m + log(sum));
            s_add[w] = nan ? (double)NAN : add;
        }
    }
    __syncthreads();
    const int n = W * nsl * K;
    const unsigned long long *ks = keys + b * n;
    // candidates in order, best first: K rounds of the best one below the last
    auto cand_of = [&](int i) {
        const int w = i / (nsl * K), r = i - w * nsl * K;
        const double add = s_add[w];
        if (!(fabs(add) < INFINITY)) return r < K && r < V ? Cand{-INFINITY, w * V + r} : Cand{-INFINITY, 0x7fffffff};
        const unsigned long long kx = ks[i];
        if (kx == 0) return Cand{-INFINITY, 0x7fffffff};
        return Cand{add + (double)value_of((uint32_t)(kx >> 32)), w * V + (int)~(uint32_t)kx};
    };
    Cand last{INFINITY, -1};
    for (int r = 0; r < K; ++r) {
        Cand mine{-INFINITY, 0x7fffffff};
        for (int i = tid; i < n; i += kThreads) {
            const Cand c = cand_of(i);
            if (c.flat != 0x7fffffff && last.better(c) && c.better(mine)) mine = c;
        }
        s_best[tid] = mine;
        __syncthreads();
        for (int o = kThreads / 2; o > 0; o >>= 1) {
            if (tid < o && s_best[tid + o].better(s_best[tid])) s_best[tid] = s_best[tid + o];
            __syncthreads();
        }
        last = s_best[0];
        if (tid == 0) {
            out_scores[b * K + r] = (float)last.score;
            out_parent[b * K + r] = last.flat / V;
            out_token[b * K + r] = last.flat % V;
        }
        __syncthreads();
    }
}

// WMAX: rows held in registers.
template <int WMAX>
__global__ void __launch_bounds__(kThreads)
gdn_state_reorder_kernel(uint4 *__restrict__ state, const int32_t *__restrict__ parent, int W, int64_t cols) {
    __shared__ int s_parent[WMAX];
    const int64_t b = blockIdx.y;
    if (threadIdx.x < W) {
        const int p = parent[b * W + threadIdx.x];
        s_parent[threadIdx.x] = p >= 0 && p < W ? p : (int)threadIdx.x;
    }
    __syncthreads();
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= cols) return;
    uint4 *base = state + b * W * cols + c;
    uint4 x[WMAX];
#pragma unroll
    for (int w = 0; w < WMAX; ++w)
        if (w < W && s_parent[w] != w) x[w] = base[s_parent[w] * cols];
#pragma unroll
    for (int w = 0; w < WMAX; ++w)
        if (w < W && s_parent[w] != w) base[w * cols] = x[w];
}

int slices(const gdn_beam_desc &d) { return (d.V + kSlice - 1) / kSlice; }

}  // namespace

size_t beam_workspace(const gdn_beam_desc &d) {
    const size_t n = (size_t)d.B * d.W * slices(d);
    return (n * sizeof(SliceHead) + 255) / 256 * 256 + (n * d.K * sizeof(unsigned long long) + 255) / 256 * 256;
}

gdn_status launch_beam_select(const gdn_beam_desc &d, const void *logits, const float *scores, float *out_scores,
                              int32_t *out_parent, int32_t *out_token, void *ws, cudaStream_t s) {
    const int nsl = slices(d);
    const int64_t n = d.B * d.W * nsl;
    if (n > 0x7fffffffLL) return fail(GDN_ERR_UNSUPPORTED, "grid too large");
    SliceHead *heads = static_cast<SliceHead *>(ws);
    auto *keys = reinterpret_cast<unsigned long long *>(static_cast<char *>(ws) + ((size_t)n * sizeof(SliceHead) + 255) / 256 * 256);
    {
        LaunchScope ls("gdn_beam_slices", s);
        if (d.dtype == GDN_BF16)
            gdn_beam_slices<__nv_bfloat16><<<(unsigned)n, kThreads, 0, s>>>((const __nv_bfloat16 *)logits, d.row_stride,
                                                                          d.V, d.K, nsl, heads, keys);
        else
            gdn_beam_slices<float><<<(unsigned)n, kThreads, 0, s>>>((const float *)logits, d.row_stride, d.V, d.K, nsl,
                                                                    heads, keys);
    }
    gdn_status st = check_launch("gdn_beam_slices");
    if (st != GDN_OK) return st;
    {
        LaunchScope ls("gdn_beam_join", s);
        gdn_beam_join<<<(unsigned)d.B, kThreads, 0, s>>>(scores, d.W, d.V, d.K, nsl, heads, keys, out_scores, out_parent,
                                                        out_token);
    }
    return check_launch("gdn_beam_join");
}

gdn_status launch_state_reorder(void *state, const int32_t *parent, int64_t B, int W, size_t row_bytes, cudaStream_t s) {
    const int64_t cols = (int64_t)(row_bytes / 16), blocks = (cols + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffLL) return fail(GDN_ERR_UNSUPPORTED, "rows too long");
    LaunchScope ls("gdn_state_reorder_kernel", s);
    uint4 *p = static_cast<uint4 *>(state);
    for (int64_t b0 = 0; b0 < B; b0 += 65535) {
        const int64_t nb = B - b0 < 65535 ? B - b0 : 65535;
        const dim3 grid((unsigned)blocks, (unsigned)nb);
        uint4 *q = p + b0 * W * cols;
        const int32_t *pp = parent + b0 * W;
        if (W <= 4) gdn_state_reorder_kernel<4><<<grid, kThreads, 0, s>>>(q, pp, W, cols);
        else if (W <= 8) gdn_state_reorder_kernel<8><<<grid, kThreads, 0, s>>>(q, pp, W, cols);
        else if (W <= 16) gdn_state_reorder_kernel<16><<<grid, kThreads, 0, s>>>(q, pp, W, cols);
        else if (W <= 32) gdn_state_reorder_kernel<32><<<grid, kThreads, 0, s>>>(q, pp, W, cols);
        else gdn_state_reorder_kernel<64><<<grid, kThreads, 0, s>>>(q, pp, W, cols);
    }
    return check_launch("gdn_state_reorder_kernel");
}

}  // namespace lin
}  // namespace gdn
