// Linear attention with a decay for each head: what its kernels share.
//
//     S_t = alpha_t S_{t-1} + v_t k_t^T,   o_t = S_t (scale q_t)
//
// Chunkwise form.  For a chunk of L tokens with start state S0, G_i = sum_{j <= i} g_j
// (log2 units throughout the kernels) and G = G_L:
//     o_i = scale 2^{G_i} S0 q_i + sum_{j <= i} scale 2^{G_i - G_j} (q_i . k_j) v_j
//     S   = 2^G S0 + sum_j 2^{G - G_j} v_j k_j^T
// Every exponent is <= 0.  Nothing but the d_v x d_k state passes from chunk to chunk,
// and its update is a plain sum: a segment of chunks contributes
// U = sum_j 2^{(decay from j to the segment's end)} v_j k_j^T whatever state it starts
// from.  So a long sequence is cut into segments of `seg` tokens: the state kernel
// forms every segment's U (all segments but each sequence's last, from its end
// backwards until nothing reaches the end any more; in one or more parts, whose U add up),
// and the output kernel runs all segments side by side, each from
//     S_g = U_{g-1} + 2^{G_{g-1}} (U_{g-2} + 2^{G_{g-2}} ( .. )):
// its blocks add that up themselves, newest first, until the decay has left nothing.  Where
// many segments could take part (kMostChained) the combine kernel chains the start
// states S_{g+1} = 2^{G_g} S_g + U_g first.  Sequences of one segment need the output kernel
// alone.
#pragma once

#include <atomic>

#include "chunk_common.cuh"
#include "gdn_internal.cuh"
#include "gdn_linattn.h"

namespace gdn {
namespace lin {

constexpr float kLog2e = 1.4426950408889634f;
// A decay below 2^-150 gives exactly zero in fp32 (the kernels flush from 2^-126 on).
constexpr float kDead = -150.f;

// A gate in log2 units.  At 2^kDead and below nothing is left of anything, so lower gates (the
// type's lowest value, -infinity) are taken as that: sums over a chunk stay finite and keep
// the gates beside them.
constexpr float kErase = -152.f;
__device__ __forceinline__ float gate2(float g) {
    const float x = g * kLog2e;
    return x < kErase ? kErase : x;
}
__device__ __forceinline__ double gate2_exact(float g) {
    const double x = (double)g * 1.4426950408889634074;
    return x < (double)kErase ? (double)kErase : x;
}

struct Plan {
    int64_t N, rows, T, H, Hk, dk, dv;
    bool packed, tc, fixed_gate;
    bool chained;    // the output kernel's blocks add up their start states
    int64_t seg;     // tokens per segment, a multiple of 64
    int64_t G;       // fixed-length sequences: segments per sequence (>= 1)
    int64_t slots;   // segments in all (packed: an upper bound)
    int64_t sslots;  // segments of sequences that have more than one (packed: an upper bound; 0: none has)
    int64_t parts, part_len;  // blocks of the state kernel per segment, and their tokens
    size_t off_status, off_tot, off_alive, off_state, total;
};
constexpr int64_t kMostChained = 128;  // U that a block of the output kernel adds up at most
constexpr int64_t kMaxPart = 16384;  // tokens of a part (their weights lie in shared memory)
constexpr int64_t kMostParts = 32;   // of a segment (the combine kernel keeps a bit for each)
Plan make_plan(const gdn_desc &d, int64_t num_seqs, bool packed);

struct Args {
    const void *q, *k, *v;
    const float *g, *h0;
    const int32_t *cu;
    int64_t T, N, rows, H, Hk, seg, G, slots, sslots, parts, part_len;
    float scale;
    bool chained;  // (not where the final state replaces the initial one that other blocks still read)
    int64_t snap_stride, n_snap;
    void *out;
    float *final_state, *snaps;
    double *tot;     // [sslots][H] decay of a segment, log2 units
    int32_t *alive;  // [sslots][parts][H] 1: the part's U was formed (0: it is zero)
    float *states;   // [sslots][parts][H][d_v][d_k]: U of a part; part 0: then the segment's start state
    int *status;
};

// A segment: the j-th of the nseg of sequence n, token rows [start, start + len), `pos`
// tokens into the sequence; ss is its place in the workspace (nseg > 1 only).
//
// Two numberings find it.  `slots` counts every segment (the output kernel's blocks):
// packed sequence n owns the slots from cu[n] / seg + n on.  They are enough, since
// floor(b/s) - floor(a/s) + 1 >= ceil((b - a)/s), and an empty sequence has one.  `sslots`
// counts the segments of sequences longer than one segment only (the state kernel's
// blocks and the workspace): from floor(2 cu[n] / seg) on, enough since
// floor(2 len / seg) >= ceil(len / seg) for len > seg.
struct Slot {
    int64_t n, j, nseg, start, pos, len, ss;
};
__device__ __forceinline__ int64_t clamped_cu(const Args &a, int64_t n) {
    const int64_t c = a.cu[n];
    return c < 0 ? 0 : (c > a.rows ? a.rows : c);
}
__device__ __forceinline__ int64_t state_base(const Args &a, int64_t n) {
    return a.cu ? 2 * clamped_cu(a, n) / a.seg : n * a.G;
}
// Tokens per segment of a sequence of `len` tokens, and how many segments it has: packed
// sequences are cut into equal segments of `seg` tokens or fewer (blocks of one length leave
// less of the GPU idle at the end than full ones and remainders: eight sequences of 1 to 16,023
// tokens and 32 heads took 405 us in both kernels, 425 before, in one process; from one to the next
// a call takes 390 to 500).
__device__ __forceinline__ int64_t segment_length(const Args &a, int64_t len, int64_t &nseg) {
    if (len <= 0) {
        nseg = 1;
        return a.seg;
    }
    nseg = (len + a.seg - 1) / a.seg;
    if (!a.cu || nseg == 1) return a.seg;
    const int64_t e = ((len + nseg - 1) / nseg + kChunk - 1) / kChunk * kChunk;
    nseg = (len + e - 1) / e;
    return e;
}
// (The whole block calls it, with the same slot.)
template <bool STATE>
__device__ __forceinline__ bool locate(const Args &a, int64_t slot, Slot &s) {
    int64_t base;
    if (a.cu) {
        auto base_of = [&](int64_t n) { return STATE ? state_base(a, n) : clamped_cu(a, n) / a.seg + n; };
        int64_t lo = 0, hi = a.N;  // the last sequence whose first slot is not past `slot`
        if (a.N <= blockDim.x) {   // a thread looks at one sequence: one trip to memory
            lo = __syncthreads_count(threadIdx.x < a.N && base_of(threadIdx.x) <= slot) - 1;
            if (lo < 0) return false;
        } else {
            while (hi - lo > 1) {
                const int64_t mid = (lo + hi) / 2;
                if (base_of(mid) <= slot) lo = mid; else hi = mid;
            }
        }
        s.n = lo;
        base = base_of(lo);
    } else {
        s.n = slot / a.G;
        base = s.n * a.G;
    }
    s.j = slot - base;
    if (s.n >= a.N || s.j < 0) return false;
    int64_t start, len;
    seq_bounds(a.cu, s.n, a.T, a.rows, start, len);
    const int64_t seg = segment_length(a, len, s.nseg);
    if (s.j >= s.nseg) return false;
    s.pos = s.j * seg;
    s.start = start + s.pos;
    s.len = len - s.pos < seg ? len - s.pos : seg;
    s.ss = state_base(a, s.n) + s.j;
    return s.nseg == 1 || s.ss < a.sslots;  // (wrong offsets stay inside the workspace)
}

// 2^x for a decay x <= 0 in 64 bits as two floats: a fixed decay close to 1, applied
// once a chunk over a very long sequence, must not carry the same rounding every time.
__device__ __forceinline__ float2 exp2_pair(double x) {
    const double e = exp2(x);
    const float hi = (float)e;
    return make_float2(hi, (float)(e - (double)hi));
}

// The same for the sum x <= 0 of a chunk's gates in 32 bits: two floats where the state keeps most of itself
// from chunk to chunk, and one where a rounding of 2^-24 a chunk, the same one every time if the
// gates are alike, is forgotten after a dozen chunks.
__device__ __forceinline__ float2 exp2_pair_f32(float x) {
    if (!(x > -0.125f)) return make_float2(exp2f(x), 0.f);
    const float m = expm1f(x * 0.693147180559945f), hi = 1.f + m;
    return make_float2(hi, m - (hi - 1.f));  // (both differences are exact)
}

// The kernels of a call overlap at their ends: each lets the next one start (early), and the
// next one waits for it before it touches what it wrote, in every block, so that the stream's
// order holds for what follows the call.  The first kernel of a call is launched as usual.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Dynamic shared memory above 48 KB for `kernel` on the current device, once a device (`done`: a bit
// for each).
inline gdn_status allow_smem(const void *kernel, size_t bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (e == cudaSuccess && (dev > 63 || !(done.load() & bit))) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e == cudaSuccess && dev <= 63) done.fetch_or(bit);
    }
    return e == cudaSuccess ? GDN_OK : fail(GDN_ERR_CUDA, "kernel attributes: %s", cudaGetErrorString(e));
}

template <typename... P, typename... A>
cudaError_t launch_kernel(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, bool after_previous,
                          A... args) {
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = block;
    c.dynamicSmemBytes = smem;
    c.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &attr;
    c.numAttrs = after_previous ? 1 : 0;
    return cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
}

// Start state of segment `s` of head h, `elems` values per state: `take(f, src)` is called for
// every state of `elems` floats at src that has a part in it, times f (two floats), by
// every thread that calls this.
template <typename Take>
__device__ __forceinline__ void start_state(const Args &a, const Slot &s, int64_t h, int64_t elems, Take take) {
    if (s.nseg > 1 && !a.chained) return take(make_float2(1.f, 0.f), a.states + (s.ss * a.parts * a.H + h) * elems);
    double decay = 0.0;  // log2, from the end of segment j to the start of this one
    for (int64_t j = s.j - 1; j >= 0; --j) {
        const float2 f = exp2_pair(decay);
        if (f.x == 0.f) return;
        const int64_t ss = s.ss - s.j + j;
        for (int64_t i = 0; i < a.parts; ++i)
            if (a.alive[(ss * a.parts + i) * a.H + h]) take(f, a.states + ((ss * a.parts + i) * a.H + h) * elems);
        decay += a.tot[ss * a.H + h];
    }
    const float2 f = s.j == 0 ? make_float2(1.f, 0.f) : exp2_pair(decay);
    if (a.h0 && f.x != 0.f) take(f, a.h0 + (s.n * a.H + h) * elems);
}

gdn_status launch_simt(const Plan &p, const Args &a, int dtype, cudaStream_t s);
gdn_status launch_tc(const Plan &p, const Args &a, cudaStream_t s);
gdn_status launch_combine(const Plan &p, const Args &a, cudaStream_t s);
gdn_status launch_decode(const gdn_desc &d, const void *q, const void *k, const void *v, const float *g, float *state,
                         void *out, cudaStream_t s);
gdn_status launch_qk_norm_rope(const gdn_qk_rope_desc &d, const void *q, const void *k, const int32_t *pos,
                               const float *inv_freq, const float *qw, const float *kw, void *q_out, void *k_out,
                               cudaStream_t s);
size_t beam_workspace(const gdn_beam_desc &d);
gdn_status launch_beam_select(const gdn_beam_desc &d, const void *logits, const float *scores, float *out_scores,
                              int32_t *out_parent, int32_t *out_token, void *ws, cudaStream_t s);
gdn_status launch_state_reorder(void *state, const int32_t *parent, int64_t B, int W, size_t row_bytes, cudaStream_t s);

}  // namespace lin
}  // namespace gdn
