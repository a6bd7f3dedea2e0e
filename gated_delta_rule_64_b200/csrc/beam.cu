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
// The K best, in both.  Every thread knows its best value; each of the eight warps finds the
// R-th best of its 32, R = ceil(K / 8) (a few rounds of a warp-wide maximum).  At least
// 8 R >= K values reach the least of those eight, T, so nothing below T can be among the K
// best, and on random values little more than K reach it: they go to shared memory, where
// each one's rank is the number of better ones.  Values are compared by their order bits and
// then by index, lowest first.  Where too many reach T (long runs of equal values) the slice
// falls back on the K-th best of the threads' (value, index) pairs, of which at most K
// threads have one, and the join on K rounds of a block-wide maximum.
//
// Measured: 32 requests of 8 beams, 128,009 bf16 logits, K = 16: 34 us.  The first kernel takes
// 25 us (the 66 MB alone are 10 us of HBM): each block's chain of load, maximum, bound and search,
// and its instructions.  The second takes 14 us, a chain of dependent steps by 32 blocks, its
// start hidden behind the first.
//
// Reordering.  A thread owns 16 bytes of every beam's row of one request: it reads the
// parents' bytes of all beams that change, then writes them, so the move is in place
// without a second buffer and rows that stay are neither read nor written.  Measured: 256 states
// of 2 MB, most of which change: 127 to 134 us, 0.80 GB at 5.9 to 6.3 TB/s (0.91 to 0.96 of a plain copy).
#include "linattn.cuh"
#include "sm100.cuh"

namespace gdn {
namespace lin {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxK = 64;

// A value's bits, ordered as unsigned integers; NaN counts as -infinity.
__device__ __forceinline__ uint32_t order_bits(float x) {
    if (x != x) x = -INFINITY;
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);  // -0 and 0 are equal
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

// Partial results of a slice: maximum and sum of exponentials below it, then K keys.
struct SliceHead {
    float max, sum;
};

// The r-th largest of the warp's 32 values (0: fewer than r are above 0).
__device__ __forceinline__ uint32_t rth_of_warp(uint32_t x, int r, int lane) {
    uint32_t m = 0;
    for (int i = 0; i < r; ++i) {
        m = __reduce_max_sync(0xffffffffu, x);
        if (lane == __ffs(__ballot_sync(0xffffffffu, x == m)) - 1) x = 0;
    }
    return m;
}

// The K-th largest of the 256 keys in `best` (all different but for zeros, of which any
// number may stand for threads without a value), by one warp: each lane holds eight.
__device__ __noinline__ unsigned long long kth_of_256(const unsigned long long *best, int K, int lane) {
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

template <typename Tin, int EACH>
__global__ void __launch_bounds__(kThreads)
gdn_beam_slices(const Tin *__restrict__ logits, int64_t row_stride, uint32_t V, int K, int nsl, SliceHead *__restrict__ heads,
                unsigned long long *__restrict__ keys) {
    constexpr int kCap = 256;  // values at or above the bound before the fallback
    __shared__ unsigned long long best[kThreads];
    __shared__ unsigned long long found[kMaxK * EACH > kCap ? kMaxK * EACH : kCap];
    __shared__ float red_m[kWarps], red_s[kWarps];
    __shared__ uint32_t red_t[kWarps];
    __shared__ unsigned long long s_bound;
    __shared__ int s_count;
    let_next_start();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / nsl;
    // (indices are unsigned: those of a last slice may pass the vocabulary, and 2^31, by a slice)
    const uint32_t i0 = blockIdx.x % (uint32_t)nsl * (uint32_t)(kThreads * EACH);
    const Tin *p = logits + row * row_stride;
    constexpr int kVec = 16 / (int)sizeof(Tin);
    const bool wide = ((uintptr_t)(p + i0) & 15) == 0;
    // logit e of this thread: index i0 + (e / kVec) * 256 kVec + tid * kVec + e % kVec, kept as it
    // lies in memory (bf16: half the registers, so more blocks per SM)
    uint4 raw[EACH / kVec];
    auto x = [&](int e) {
        const uint4 &w = raw[e / kVec];
        if (kVec == 4) {
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
            return __uint_as_float(u[e % 4]);
        }
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        return __uint_as_float(e & 1 ? u[(e % 8) / 2] & 0xffff0000u : u[(e % 8) / 2] << 16);
    };
    auto index_of = [&](int e) { return i0 + (uint32_t)((e / kVec) * (kThreads * kVec) + tid * kVec + e % kVec); };
    constexpr uint32_t kLow = kVec == 4 ? 0xff800000u : 0xff80ff80u;  // -infinity
#pragma unroll
    for (int c = 0; c < EACH / kVec; ++c) {
        const uint32_t i = index_of(c * kVec);
        if (wide && i + kVec <= V) {
            raw[c] = __ldcs(reinterpret_cast<const uint4 *>(p + i));
        } else {
            uint32_t u[4] = {kLow, kLow, kLow, kLow};
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                if (i + e < V) {
                    if (kVec == 4)
                        u[e] = reinterpret_cast<const uint32_t *>(p)[i + e];
                    else
                        u[e / 2] = e & 1 ? (u[e / 2] & 0xffffu) | (uint32_t)reinterpret_cast<const uint16_t *>(p)[i + e] << 16
                                         : (u[e / 2] & 0xffff0000u) | reinterpret_cast<const uint16_t *>(p)[i + e];
                }
            raw[c] = make_uint4(u[0], u[1], u[2], u[3]);
        }
    }
    if (tid == 0) s_count = 0;
    // the thread's maximum and its sum of 2^((x - max) log2 e); a NaN makes the sum NaN
    float m;
    if (kVec == 4) {
        m = x(0);
#pragma unroll
        for (int e = 1; e < EACH; ++e) m = fmaxf(m, x(e));
    } else {  // two at a time
        const __nv_bfloat162 *y = reinterpret_cast<const __nv_bfloat162 *>(raw);
        __nv_bfloat162 m2 = y[0];
#pragma unroll
        for (int e = 1; e < EACH / 2; ++e) m2 = __hmax2(m2, y[e]);
        m = fmaxf(__low2float(m2), __high2float(m2));
    }
    // (x - max before the factor: the type's lowest value times log2 e would overflow)
    const float base = m > -INFINITY ? m : 0.f;
    float2 sum2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int e = 0; e < EACH; e += 2) {
        const float2 y = __fmul2_rn(__fadd2_rn(make_float2(x(e), x(e + 1)), make_float2(-base, -base)),
                                    make_float2(kLog2e, kLog2e));
        sum2 = __fadd2_rn(sum2, make_float2(sm100::ex2(y.x), sm100::ex2(y.y)));
    }
    float sum = sum2.x + sum2.y;
    // (a thread behind the vocabulary has nothing, not even -infinity)
    const uint32_t top = index_of(0) < V ? order_bits(m) : 0u;
    // (a last slice may leave whole warps without a logit: the others' share grows)
    const int left = (int)(V - i0), busy = left >= kThreads * kVec ? kWarps : (left + 32 * kVec - 1) / (32 * kVec);
    const uint32_t t = rth_of_warp(top, (K + busy - 1) / busy, lane);
    float wm = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, o));
    sum *= m > -INFINITY ? sm100::ex2((m - wm) * kLog2e) : 1.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
        red_m[warp] = wm;
        red_s[warp] = sum;
        red_t[warp] = t;
    }
    __syncthreads();
    uint32_t bound = red_t[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w)
        if (w < busy) bound = min(bound, red_t[w]);
    auto key_at = [&](uint32_t i) { return ((unsigned long long)order_bits(to_f32<Tin>(p[i])) << 32) | ~i; };
    if (top >= bound && top > 0) {
        // which of this thread's logits reach the bound (few threads have any): a bit each, then
        // those are read once more
        const float least = bound > 0 ? value_of(bound) : -INFINITY;  // (0: a warp with fewer than its share)
        // fp32: bit e for logit e; bf16: bit e for logit 2 e, bit 16 + e for 2 e + 1, of 32 logits
        constexpr int kPart = EACH < 32 ? EACH : 32;
        auto logit_of = [](int bit) { return kVec == 4 ? bit : 2 * (bit & 15) + (bit >> 4); };
#pragma unroll
        for (int e0 = 0; e0 < EACH; e0 += kPart) {
            uint32_t bits = 0;
            if (kVec == 4) {
#pragma unroll
                for (int e = 0; e < kPart; ++e) bits |= x(e0 + e) >= least ? 1u << e : 0u;
            } else {  // (the bound is one of the values: exact in bf16)
                const __nv_bfloat162 *y = reinterpret_cast<const __nv_bfloat162 *>(raw) + e0 / 2;
                const __nv_bfloat162 l2 = __float2bfloat162_rn(least);
#pragma unroll
                for (int e = 0; e < kPart / 2; ++e) bits |= __hge2_mask(y[e], l2) & (0x00010001u << e);
            }
            if (left < kThreads * EACH)
                for (uint32_t rest = bits; rest; rest &= rest - 1) {
                    const int bit = __ffs(rest) - 1;
                    if (index_of(e0 + logit_of(bit)) >= V) bits &= ~(1u << bit);
                }
            if (bits) {
                int at = atomicAdd(&s_count, __popc(bits));
                for (; bits; bits &= bits - 1, ++at)
                    if (at < kCap) found[at] = key_at(index_of(e0 + logit_of(__ffs(bits) - 1)));
            }
        }
    }
    if (warp == kWarps - 1) {  // the slice's maximum and sum, a warp's part per lane
        const float wm8 = lane < kWarps ? red_m[lane] : -INFINITY;
        float bm = wm8;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, o));
        double all = 0.0;
        if (lane < kWarps)
            all = wm8 > -INFINITY ? (double)red_s[lane] * (double)exp2f((wm8 - bm) * kLog2e) : (double)red_s[lane];
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        if (lane == 0) heads[blockIdx.x] = SliceHead{bm, (float)all};
    }
    __syncthreads();
    int n = s_count;
    if (n > kCap) {  // (the same for the whole block; the logits are read again)
        unsigned long long mine = 0;
#pragma unroll 1
        for (int e = 0; e < EACH; ++e) {
            const uint32_t i = index_of(e);
            const unsigned long long kx = i < V ? key_at(i) : 0ull;
            mine = kx > mine ? kx : mine;
        }
        best[tid] = mine;
        __syncthreads();
        if (tid == 0) s_count = 0;
        if (warp == 0) {
            const unsigned long long k = kth_of_256(best, K, lane);
            if (lane == 0) s_bound = k > 0 ? k : 1;
        }
        __syncthreads();
        if (mine >= s_bound) {  // at most K threads
#pragma unroll 1
            for (int e = 0; e < EACH; ++e) {
                const uint32_t i = index_of(e);
                const unsigned long long kx = i < V ? key_at(i) : 0ull;
                if (kx >= s_bound) found[atomicAdd(&s_count, 1)] = kx;
            }
        }
        __syncthreads();
        n = s_count;
    }
    unsigned long long *to = keys + (int64_t)blockIdx.x * K;
    for (int i = tid; i < n; i += kThreads) {
        const unsigned long long kx = found[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += found[j] > kx;
        if (rank < K) to[rank] = kx;
    }
    for (int i = n + tid; i < K; i += kThreads) to[i] = 0;  // fewer values than K
}

// A continuation; none: flat = kNone.
constexpr int kNone = 0x7fffffff;
struct Cand {
    double score;
    int flat;
    __device__ __forceinline__ bool better(const Cand &o) const {
        return score > o.score || (score == o.score && flat < o.flat);
    }
};
// A score's order bits, of which more is better, as those of a float above.
__device__ __forceinline__ unsigned long long order_bits(double x) {
    const unsigned long long u = (unsigned long long)__double_as_longlong(x == 0.0 ? 0.0 : x);
    return u >> 63 ? ~u : u | (1ull << 63);
}

// Joins the slices of one request.  A beam's candidates belong to `lanes` threads.  They are
// sifted in fp32 (the multiprocessor's 64-bit units would take most of the kernel's time):
// with |error| <= err, at least K scores are `bound` - err or more, so the K best are among
// those whose fp32 value is bound - 2 err or more.
__global__ void __launch_bounds__(kThreads)
gdn_beam_join(const float *__restrict__ scores, int W, int V, int K, int nsl, int lanes, const SliceHead *__restrict__ heads,
              const unsigned long long *__restrict__ keys, float *__restrict__ out_scores,
              int32_t *__restrict__ out_parent, int32_t *__restrict__ out_token) {
    constexpr int kCap = 512;
    __shared__ double s_add[64];  // a beam's score minus its normaliser (not finite: all its scores are -infinity)
    __shared__ unsigned long long s_key[kCap];
    __shared__ int s_flat[kCap];
    __shared__ Cand s_best[kThreads];
    __shared__ uint32_t red_t[kWarps];
    __shared__ float red_a[kWarps];
    __shared__ int s_count;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t b = blockIdx.x;
    if (tid == 0) s_count = 0;
    wait_for_previous();
    for (int w = warp; w < W; w += kWarps) {
        const SliceHead *hd = heads + (b * W + w) * nsl;
        float m = -INFINITY;
        for (int i = lane; i < nsl; i += 32) m = fmaxf(m, hd[i].max);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        double sum = 0.0;
        for (int i = lane; i < nsl; i += 32) {
            const SliceHead x = hd[i];  // (a slice of -infinities has the sum 0, one with a NaN has NaN)
            sum += x.max > -INFINITY ? (double)x.sum * exp((double)x.max - (double)m) : (double)x.sum;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) s_add[w] = (scores ? (double)scores[b * W + w] : 0.0) - ((double)m + log(sum));
    }
    __syncthreads();
    const int per = nsl * K, n = W * per;
    const unsigned long long *ks = keys + b * n;
    // (neighbouring threads have different beams: a warp's best are then a sample of all)
    const int w = tid % (kThreads / lanes), l = tid / (kThreads / lanes);
    const double add = w < W ? s_add[w] : 0.0;
    const float add32 = (float)add;
    const bool dead = !(fabs(add) < INFINITY);
    const unsigned long long *mine = ks + (int64_t)w * per;
    // fp32 value of candidate r of this beam; of a beam whose scores are all -infinity the
    // candidates are its first K tokens
    auto approx = [&](int r, bool &any) {
        if (dead) {
            any = r < K && r < V;
            return -INFINITY;
        }
        const unsigned long long kx = mine[r];
        any = kx != 0;
        return add32 + value_of((uint32_t)(kx >> 32));
    };
    // turn k takes candidates k lanes .. + lanes - 1, shifted from turn to turn: each slice's keys
    // are sorted, and a thread should not meet the same places only
    const int turns = (per + lanes - 1) / lanes;
    auto place = [&](int k) { return k * lanes + ((l + 5 * k) & (lanes - 1)); };
    uint32_t top = 0;
    if (w < W) {
#pragma unroll 4
        for (int k = 0; k < turns; ++k) {
            const int r = place(k);
            if (r >= per) continue;
            bool any;
            const float x = approx(r, any);
            if (any) top = max(top, order_bits(x));
        }
    }
    const uint32_t t = rth_of_warp(top, (K + kWarps - 1) / kWarps, lane);
    float most = w < W && !dead ? fabsf(add32) : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    if (lane == 0) {
        red_t[warp] = t;
        red_a[warp] = most;
    }
    __syncthreads();
    uint32_t bits = red_t[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) {
        bits = min(bits, red_t[i]);
        most = fmaxf(most, red_a[i]);
    }
    most = fmaxf(most, red_a[0]);
    // (0: a warp with fewer candidates than its share: all of them are wanted)
    const float bound = bits > 0 ? value_of(bits) : -INFINITY;
    float least = bound - 4.8e-7f * (most + fabsf(bound));  // 2 err, err <= 2^-22 of the terms
    if (!(least > -INFINITY)) least = -INFINITY;            // (terms past the range: nothing is sifted out)
    if (w < W) {
#pragma unroll 4
        for (int k = 0; k < turns; ++k) {
            const int r = place(k);
            if (r >= per) continue;
            bool any;
            const float x = approx(r, any);
            if (any && !(x < least)) {  // (a NaN, an infinite term less one, is kept)
                const int at = atomicAdd(&s_count, 1);
                if (at < kCap) {
                    const unsigned long long kx = dead ? 0ull : mine[r];
                    s_key[at] = order_bits(dead ? -(double)INFINITY : add + (double)value_of((uint32_t)(kx >> 32)));
                    s_flat[at] = w * V + (dead ? r : (int)~(uint32_t)kx);
                }
            }
        }
    }
    __syncthreads();
    const int found = s_count;
    auto put = [&](int r, double score, int flat) {
        out_scores[b * K + r] = (float)score;
        out_parent[b * K + r] = flat / V;
        out_token[b * K + r] = flat % V;
    };
    if (found <= kCap) {  // (the same for the whole block)
        for (int i = tid; i < found; i += kThreads) {
            const unsigned long long key = s_key[i];
            const int flat = s_flat[i];
            int rank = 0;
#pragma unroll 4
            for (int j = 0; j < found; ++j) rank += s_key[j] > key || (s_key[j] == key && s_flat[j] < flat);
            if (rank < K) {
                const unsigned long long u = key >> 63 ? key ^ (1ull << 63) : ~key;
                put(rank, __longlong_as_double((long long)u), flat);
            }
        }
        return;
    }
    auto cand_of = [&](int i) {
        const int v = i / per, r = i - v * per;
        const double s = s_add[v];
        if (!(fabs(s) < INFINITY)) return Cand{-INFINITY, r < K && r < V ? v * V + r : kNone};
        const unsigned long long kx = ks[i];
        return kx ? Cand{s + (double)value_of((uint32_t)(kx >> 32)), v * V + (int)~(uint32_t)kx} : Cand{-INFINITY, kNone};
    };
    Cand last{INFINITY, -1};
    for (int r = 0; r < K; ++r) {  // the best one below the last, K times
        Cand c0{-INFINITY, kNone};
        for (int i = tid; i < n; i += kThreads) {
            const Cand c = cand_of(i);
            if (c.flat != kNone && last.better(c) && c.better(c0)) c0 = c;
        }
        s_best[tid] = c0;
        __syncthreads();
        for (int o = kThreads / 2; o > 0; o >>= 1) {
            if (tid < o && s_best[tid + o].better(s_best[tid])) s_best[tid] = s_best[tid + o];
            __syncthreads();
        }
        last = s_best[0];
        if (tid == 0) put(r, last.score, last.flat);
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

// Slices of a beam with `each` logits a thread.
int64_t slices_of(int64_t V, int each) { return (V + kThreads * each - 1) / (kThreads * each); }

// Logits of a thread: 32, or 8 where slices of 8192 would leave SMs without one (4 beams of
// 32,000: 23 us a call with 16 blocks, 19 with 64; 8.3 us of those are the kernels' in a captured
// graph), or 64 in bf16
// where that still gives every SM four blocks (256 beams of 128,009: 35 us a call against 39, of
// which the join, with half the candidates, gives two).
int each(const gdn_beam_desc &d) {
    const int64_t rows = d.B * d.W;
    auto blocks = [&](int e) { return rows * slices_of(d.V, e); };
    if (d.dtype == GDN_BF16 && blocks(64) >= 4 * 148) return 64;
    return blocks(32) >= 148 ? 32 : 8;
}
int slices(const gdn_beam_desc &d) { return (int)slices_of(d.V, each(d)); }

template <typename Tin>
void launch_slices(const gdn_beam_desc &d, const void *logits, int nsl, SliceHead *heads, unsigned long long *keys,
                   cudaStream_t s) {
    constexpr int kMost = sizeof(Tin) == 2 ? 64 : 32;
    const int e = each(d);
    auto kern = e == 8 ? gdn_beam_slices<Tin, 8> : e == 32 ? gdn_beam_slices<Tin, 32> : gdn_beam_slices<Tin, kMost>;
    kern<<<(unsigned)(d.B * d.W * nsl), kThreads, 0, s>>>((const Tin *)logits, d.row_stride, (uint32_t)d.V, d.K, nsl, heads, keys);
}

}  // namespace

size_t beam_workspace(const gdn_beam_desc &d) {
    const size_t n = (size_t)d.B * d.W * slices(d);
    return (n * sizeof(SliceHead) + 255) / 256 * 256 + (n * d.K * sizeof(unsigned long long) + 255) / 256 * 256;
}

gdn_status launch_beam_select(const gdn_beam_desc &d, const void *logits, const float *scores, float *out_scores,
                              int32_t *out_parent, int32_t *out_token, void *ws, cudaStream_t s) {
    const int nsl = slices(d);
    const int64_t n = d.B * d.W * nsl;
    if (n > 0x7fffffffLL || (int64_t)d.W * nsl * d.K > 0x7fffffffLL) return fail(GDN_ERR_UNSUPPORTED, "grid too large");
    SliceHead *heads = static_cast<SliceHead *>(ws);
    auto *keys = reinterpret_cast<unsigned long long *>(static_cast<char *>(ws) + ((size_t)n * sizeof(SliceHead) + 255) / 256 * 256);
    {
        LaunchScope ls("gdn_beam_slices", s);
        if (d.dtype == GDN_BF16)
            launch_slices<__nv_bfloat16>(d, logits, nsl, heads, keys, s);
        else
            launch_slices<float>(d, logits, nsl, heads, keys, s);
    }
    gdn_status st = check_launch("gdn_beam_slices");
    if (st != GDN_OK) return st;
    {
        LaunchScope ls("gdn_beam_join", s);
        int lanes = kThreads;
        while (lanes * d.W > kThreads) lanes /= 2;
        launch_kernel(gdn_beam_join, dim3((unsigned)d.B), dim3(kThreads), 0, s, true, scores, d.W, d.V, d.K, nsl, lanes,
                      heads, keys, out_scores, out_parent, out_token);
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
