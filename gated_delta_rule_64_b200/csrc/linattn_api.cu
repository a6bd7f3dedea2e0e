// C-ABI entry points of gdn_linattn.h: argument checks, the split of long sequences
// into segments, and launches.
#include <math.h>

#include "api_checks.cuh"
#include "linattn.cuh"

namespace gdn {
namespace lin {

static gdn_status check_lin_desc(const gdn_desc *d) {
    if (!d) return fail(GDN_ERR_INVALID_ARG, "descriptor is NULL");
    if (d->gate == GDN_GATE_CHANNEL)
        return fail(GDN_ERR_UNSUPPORTED, "linear attention takes a gate per head (GDN_GATE_HEAD or GDN_GATE_CONST)");
    gdn_desc c = *d;
    if (c.gate == GDN_GATE_CONST) c.gate = GDN_GATE_HEAD;
    return check_desc(&c);
}

// N states in elements, and the blocks that work on them, stay well inside int64 (check_desc
// bounds what has tokens).
static bool states_fit(const gdn_desc &d, int64_t N) {
    return (double)N * (double)d.H * (double)(d.dk * d.dv) <= 4.0e15;
}

// Tokens per segment (a multiple of 64; at least the longest possible sequence: no
// split).  `units` blocks work on one segment of one sequence, `wide` blocks run at once.
//
// The cost of a split is counted in chunk steps of a block: a block's start (state in,
// pipeline filled) is worth about kStart, the two extra launches about kLaunch, and the
// state kernel, which stops where the decay has left nothing, about a quarter of the
// segments' chunks.  Packed sequences: their lengths are on the device, so a segment is
// a third of a block's fair share of all tokens (the tail of uneven blocks stays within
// a third), at least 16 chunks.
// A chunk step of the CUDA-core kernels is five times as long, so for these the start and the
// launches weigh less: 256 fp32 tokens of 2 heads took 42 us in one segment, 30 us in four.
static int64_t choose_seg(int64_t N, int64_t units, int64_t T, int64_t rows, bool packed, int64_t wide, bool tc) {
    const double kStart = tc ? 4.0 : 0.5, kLaunch = tc ? 6.0 : 0.75;
    const int64_t kLeast = tc ? 4 : 1;
    if (packed) {
        const int64_t share = (rows * units / kChunk) / (3 * wide);
        const int64_t seg = (share > 16 ? share : 16) * kChunk;
        return seg < rows ? seg : ((rows + kChunk - 1) / kChunk + 1) * kChunk;
    }
    const int64_t nch = T > 0 ? (T + kChunk - 1) / kChunk : 1;
    auto waves = [wide](int64_t blocks) { return (double)((blocks + wide - 1) / wide); };
    int64_t best = nch;
    double best_cost = waves(N * units) * ((double)nch + kStart);
    // (more than 16 waves of blocks are never better)
    for (int64_t G = 2; G <= nch && (G == 2 || N * units * G <= 16 * wide); ++G) {
        const int64_t seg = (nch + G - 1) / G;
        if (seg < kLeast) break;
        const int64_t Gr = (nch + seg - 1) / seg;  // no empty segments
        if (Gr < 2) continue;
        const double cost = waves(N * units * Gr) * ((double)seg + kStart) + kLaunch +
                            waves(N * units * (Gr - 1)) * (0.25 * (double)seg + kStart);
        if (cost < best_cost) {
            best_cost = cost;
            best = seg;
        }
    }
    return best * kChunk;
}

Plan make_plan(const gdn_desc &d, int64_t num_seqs, bool packed) {
    Plan p{};
    p.N = num_seqs;
    p.T = d.T;
    p.rows = d.B * d.T;
    p.H = d.H;
    p.Hk = qk_heads(d);
    p.dk = d.dk;
    p.dv = d.dv;
    p.packed = packed;
    p.fixed_gate = d.gate == GDN_GATE_CONST;
    // bf16 with 128-wide heads on the tensor cores, whose kernels are laid out for that width, all
    // else on the CUDA cores.  4 sequences of 4,096 tokens and 16 heads: 78 us there; here 490 us
    // with 64-wide bf16 heads, 770 (keys) and 890 (values) with one side 128 wide, 520 and 1,410
    // with 64- and 128-wide fp32 heads (of which each operand would take three bf16 terms).
    p.tc = d.dtype == GDN_BF16 && d.dk == 128 && d.dv == 128;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) {
        cudaGetLastError();  // (no device: sizes are planned for the GPU this library is built for)
        sms = 148;
    }
    const int64_t units = p.tc ? p.H : p.H * (p.dv / 32), wide = p.tc ? sms : 2 * sms;
    p.seg = choose_seg(p.N, units, d.T, p.rows, packed, wide, p.tc);
    // (a bound that only sequences of half a million tokens in one segment meet)
    if (p.tc && p.seg > kMaxPart * kMostParts) p.seg = kMaxPart * kMostParts;
    if (packed) {
        p.G = 0;
        p.slots = p.rows / p.seg + p.N;
        p.sslots = p.rows > p.seg ? 2 * p.rows / p.seg + 1 : 0;
    } else {
        p.G = d.T > 0 ? (d.T + p.seg - 1) / p.seg : 1;
        p.slots = p.N * p.G;
        p.sslots = p.G > 1 ? p.slots : 0;
    }
    // Parts of a segment's state (tensor cores), of four chunks or more and kMaxPart tokens or
    // fewer.  With a fixed gate a block sees at once whether its part reaches the segment's
    // end, and heads whose state lasts work side by side: four parts (262,144 tokens of 16
    // heads, state and output kernel: 186 + 796 us with one part, 126 + 802 with four, 118 +
    // 822 with eight, which the output kernel's blocks have to add up).  With a gate per token
    // it has to add up the gates behind its part first, 3 us even where it then has nothing to
    // do, at one block per SM: about two blocks per SM in all (4 x 4,096 tokens of 16 heads: 32
    // us with eight parts, 19 with two).  The CUDA-core state kernel takes a segment whole (it
    // has d_v / 32 blocks for it already).
    const int64_t chunks = p.seg / kChunk, least = (p.seg + kMaxPart - 1) / kMaxPart;
    int64_t parts = p.fixed_gate ? 4 : (p.sslots > 0 ? 2 * sms / (p.sslots * p.H) : 1);
    if (parts > 8) parts = 8;
    if (parts > chunks / 4) parts = chunks / 4;
    if (parts < least) parts = least;
    p.parts = p.tc && parts > 1 ? parts : 1;
    p.part_len = (chunks + p.parts - 1) / p.parts * kChunk;
    p.chained = (packed ? (p.rows + p.seg - 1) / p.seg : p.G) * p.parts <= kMostChained;
    size_t off = 0;
    p.off_status = off;
    off += kStatusBytes;
    p.off_tot = off;
    off = align_up(off + sizeof(double) * (size_t)p.sslots * p.H, 256);
    p.off_alive = off;
    off = align_up(off + sizeof(int32_t) * (size_t)p.sslots * p.parts * p.H, 256);
    p.off_state = off;
    off += sizeof(float) * (size_t)p.sslots * p.parts * p.H * p.dv * p.dk;
    p.total = align_up(off, 256);
    return p;
}

}  // namespace lin
}  // namespace gdn

using namespace gdn;
using namespace gdn::lin;

extern "C" {

gdn_status gdn_linattn_workspace_size(const gdn_desc *d, int32_t num_seqs, size_t *bytes) {
    clear_error();
    gdn_status st = check_lin_desc(d);
    if (st != GDN_OK) return st;
    if (!bytes) return fail(GDN_ERR_INVALID_ARG, "bytes is NULL");
    if (num_seqs < 0) return fail(GDN_ERR_INVALID_ARG, "num_seqs < 0");
    if (!states_fit(*d, num_seqs)) return fail(GDN_ERR_INVALID_ARG, "problem too large");
    if (num_seqs == 0) {  // (nothing to plan: T may be anything)
        *bytes = kStatusBytes;
        return GDN_OK;
    }
    // either gate kind; packed, and fixed-length where the number of sequences allows it
    size_t total = 0;
    for (int i = 0; i < 4; ++i) {
        gdn_desc c = *d;
        c.gate = i & 1 ? (int32_t)GDN_GATE_CONST : (int32_t)GDN_GATE_HEAD;
        if (i & 2 ? num_seqs != d->B : d->B != 1) continue;
        const size_t n = lin::make_plan(c, num_seqs, !(i & 2)).total;
        total = n > total ? n : total;
    }
    *bytes = total > kStatusBytes ? total : kStatusBytes;
    return GDN_OK;
}

gdn_status gdn_linattn_chunk_fwd(const gdn_desc *d, const void *q, const void *k, const void *v,
                                 const float *log_gate, const float *initial_state, const int32_t *cu_seqlens,
                                 int32_t num_seqs, int64_t snapshot_stride, void *out, float *final_state,
                                 float *snapshots, void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
    clear_error();
    gdn_status st = check_lin_desc(d);
    if (st != GDN_OK) return st;
    const bool packed = cu_seqlens != nullptr;
    if (packed) {
        if (d->B != 1) return fail(GDN_ERR_INVALID_ARG, "packed sequences need B == 1");
        if (num_seqs < 0) return fail(GDN_ERR_INVALID_ARG, "num_seqs < 0");
        if (!aligned4(cu_seqlens)) return fail(GDN_ERR_INVALID_ARG, "cu_seqlens misaligned");
        if (snapshot_stride != 0)
            return fail(GDN_ERR_UNSUPPORTED, "snapshots are only supported without cu_seqlens");
    }
    const int64_t N = packed ? num_seqs : d->B;
    if (snapshot_stride < 0 || snapshot_stride % kChunk != 0)
        return fail(GDN_ERR_INVALID_ARG, "snapshot_stride must be 0 or a positive multiple of 64");
    const int64_t n_snap = snapshot_stride > 0 ? d->T / snapshot_stride : 0;
    if (!states_fit(*d, N)) return fail(GDN_ERR_INVALID_ARG, "problem too large");
    const int64_t rows = d->B * d->T;
    if (rows > 0x7fffffffLL) return fail(GDN_ERR_UNSUPPORTED, "more than 2^31 - 1 token rows");
    const size_t el = d->dtype == GDN_F32 ? 4 : 2;
    const size_t qk_bytes = (size_t)rows * qk_heads(*d) * d->dk * el, v_bytes = (size_t)rows * d->H * d->dv * el;
    const size_t g_bytes = (d->gate == GDN_GATE_CONST ? 1 : (size_t)rows) * d->H * 4;
    const size_t st_bytes = (size_t)N * d->H * d->dv * d->dk * 4;
    const size_t snap_bytes = (size_t)N * n_snap * d->H * d->dv * d->dk * 4;
    if (rows > 0) {
        if (!q || !k || !v || !log_gate || !out)
            return fail(GDN_ERR_INVALID_ARG, "q, k, v, log_gate and out are required");
        if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out))
            return fail(GDN_ERR_INVALID_ARG, "q, k, v and out must be 16-byte aligned");
        if (!aligned4(log_gate)) return fail(GDN_ERR_INVALID_ARG, "log_gate must be 4-byte aligned");
    }
    if ((initial_state && !aligned16(initial_state)) || (final_state && !aligned16(final_state)) ||
        (snapshots && !aligned16(snapshots)))
        return fail(GDN_ERR_INVALID_ARG, "state pointers must be 16-byte aligned");
    if (n_snap > 0 && !snapshots) return fail(GDN_ERR_INVALID_ARG, "snapshots buffer is required");
    if (N == 0) return GDN_OK;
    const lin::Plan p = lin::make_plan(*d, N, packed);
    if (!workspace) return fail(GDN_ERR_WORKSPACE, "workspace is NULL (need %zu bytes)", p.total);
    if (((uintptr_t)workspace & 255u) != 0) return fail(GDN_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    if (workspace_bytes < p.total)
        return fail(GDN_ERR_WORKSPACE, "workspace has %zu bytes, need %zu", workspace_bytes, p.total);
    // every buffer written against every buffer that the call reads or writes (the
    // final state may be the initial state itself)
    const Range w[] = {range_of(out, out ? v_bytes : 0), range_of(final_state, final_state ? st_bytes : 0),
                       range_of(snapshots, n_snap > 0 ? snap_bytes : 0), range_of(workspace, p.total)};
    const Range r[] = {range_of(q, qk_bytes), range_of(k, qk_bytes), range_of(v, v_bytes), range_of(log_gate, g_bytes),
                       range_of(cu_seqlens, packed ? (size_t)(N + 1) * 4 : 0),
                       range_of(initial_state, initial_state ? st_bytes : 0)};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 6; ++j)
            if (overlaps(w[i], r[j]) && !(i == 1 && j == 5 && final_state == initial_state))
                return fail(GDN_ERR_INVALID_ARG, "out, final_state, snapshots or the workspace overlaps an input");
        for (int j = i + 1; j < 4; ++j)
            if (overlaps(w[i], w[j]))
                return fail(GDN_ERR_INVALID_ARG, "out, final_state, snapshots and the workspace must not overlap");
    }
    lin::Args a{};
    char *ws = static_cast<char *>(workspace);
    a.status = reinterpret_cast<int *>(ws + p.off_status);
    const cudaError_t e = cudaMemsetAsync(a.status, 0, sizeof(int32_t), (cudaStream_t)stream);
    if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "status word: %s", cudaGetErrorString(e));
    a.q = q; a.k = k; a.v = v; a.g = log_gate; a.h0 = initial_state;
    a.cu = cu_seqlens;
    a.T = d->T;
    a.N = N;
    a.rows = rows;
    a.H = d->H;
    a.Hk = qk_heads(*d);
    a.seg = p.seg;
    a.G = p.G;
    a.slots = p.slots;
    a.sslots = p.sslots;
    a.parts = p.parts;
    a.part_len = p.part_len;
    // (blocks that add up their start states read the initial state while others may already write
    // the final one)
    a.chained = p.chained && !(final_state && final_state == initial_state);
    a.scale = d->scale;
    a.snap_stride = snapshot_stride;
    a.n_snap = n_snap;
    a.out = out;
    a.final_state = final_state;
    a.snaps = snapshots;
    a.tot = reinterpret_cast<double *>(ws + p.off_tot);
    a.alive = reinterpret_cast<int32_t *>(ws + p.off_alive);
    a.states = reinterpret_cast<float *>(ws + p.off_state);
    return p.tc ? launch_tc(p, a, (cudaStream_t)stream) : launch_simt(p, a, d->dtype, (cudaStream_t)stream);
}

gdn_status gdn_linattn_decode_step(const gdn_desc *d, const void *q, const void *k, const void *v,
                                   const float *log_gate, float *state, void *out, gdn_stream_t stream) {
    clear_error();
    gdn_status st = check_lin_desc(d);
    if (st != GDN_OK) return st;
    if (d->T != 1) return fail(GDN_ERR_INVALID_ARG, "decode needs T == 1 (got %lld)", (long long)d->T);
    if (d->B == 0) return GDN_OK;
    if (!q || !k || !v || !log_gate || !state || !out)
        return fail(GDN_ERR_INVALID_ARG, "all decode pointers are required");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(state) || !aligned16(out))
        return fail(GDN_ERR_INVALID_ARG, "q, k, v, state and out must be 16-byte aligned");
    if (!aligned4(log_gate)) return fail(GDN_ERR_INVALID_ARG, "log_gate must be 4-byte aligned");
    const size_t el = d->dtype == GDN_F32 ? 4 : 2, qk = (size_t)d->B * qk_heads(*d) * d->dk * el;
    const Range ro = range_of(out, (size_t)d->B * d->H * d->dv * el);
    const Range rs = range_of(state, (size_t)d->B * d->H * d->dv * d->dk * 4);
    const Range ins[] = {range_of(q, qk), range_of(k, qk), range_of(v, (size_t)d->B * d->H * d->dv * el),
                         range_of(log_gate, (size_t)(d->gate == GDN_GATE_CONST ? 1 : d->B) * d->H * 4)};
    if (overlaps(ro, rs)) return fail(GDN_ERR_INVALID_ARG, "out overlaps state");
    for (const Range &x : ins)
        if (overlaps(ro, x) || overlaps(rs, x)) return fail(GDN_ERR_INVALID_ARG, "out or state overlaps an input");
    return lin::launch_decode(*d, q, k, v, log_gate, state, out, (cudaStream_t)stream);
}

gdn_status gdn_qk_norm_rope(const gdn_qk_rope_desc *d, const void *q, const void *k, const int32_t *positions,
                            const float *inv_freq, const float *q_weight, const float *k_weight, void *q_out,
                            void *k_out, gdn_stream_t stream) {
    clear_error();
    if (!d) return fail(GDN_ERR_INVALID_ARG, "descriptor is NULL");
    if (d->rows < 0 || d->hq < 1 || d->hk < 0)
        return fail(GDN_ERR_INVALID_ARG, "need rows >= 0, hq >= 1, hk >= 0 (got %lld, %d, %d)", (long long)d->rows,
                    d->hq, d->hk);
    if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256)
        return fail(GDN_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256 (got %d)", d->head_dim);
    if (d->rot < 0 || d->rot > d->head_dim || d->rot % 16 != 0)
        return fail(GDN_ERR_UNSUPPORTED, "rot must be a multiple of 16 up to head_dim (got %d)", d->rot);
    if (d->dtype != GDN_F32 && d->dtype != GDN_BF16) return fail(GDN_ERR_INVALID_ARG, "unknown dtype %d", d->dtype);
    if (d->interleaved != 0 && d->interleaved != 1) return fail(GDN_ERR_INVALID_ARG, "interleaved must be 0 or 1");
    if (!(d->eps >= 0.f) || !isfinite(d->eps) || !isfinite(d->weight_offset))
        return fail(GDN_ERR_INVALID_ARG, "eps must be finite and >= 0, weight_offset finite");
    const int64_t el = d->dtype == GDN_F32 ? 4 : 2, vec = 16 / el;
    const int64_t qrow = (int64_t)d->hq * d->head_dim, krow = (int64_t)d->hk * d->head_dim;
    if (d->hq > (1 << 20) || d->hk > (1 << 20) || d->rows > 0x7fffffffLL)
        return fail(GDN_ERR_UNSUPPORTED, "more than 2^31 - 1 tokens or 2^20 heads");
    if (d->rows == 0) return GDN_OK;
    if (d->q_stride < qrow || d->q_stride % vec != 0 || (d->hk > 0 && (d->k_stride < krow || d->k_stride % vec != 0)))
        return fail(GDN_ERR_INVALID_ARG, "strides must hold a token's heads and be multiples of 16 bytes");
    // (offsets in elements and bytes stay well inside int64, as in check_desc)
    if ((double)d->rows * (double)d->q_stride > 4.0e15 || (d->hk > 0 && (double)d->rows * (double)d->k_stride > 4.0e15))
        return fail(GDN_ERR_INVALID_ARG, "stride too large");
    if (!q || !q_out || (d->hk > 0 && (!k || !k_out)) || (d->rot > 0 && (!positions || !inv_freq)))
        return fail(GDN_ERR_INVALID_ARG, "q, k, their outputs, and (with rot > 0) positions and inv_freq are required");
    if (!aligned16(q) || !aligned16(q_out) || (d->hk > 0 && (!aligned16(k) || !aligned16(k_out))))
        return fail(GDN_ERR_INVALID_ARG, "q, k and the outputs must be 16-byte aligned");
    if (!aligned4(positions) || !aligned4(inv_freq) || !aligned4(q_weight) || !aligned4(k_weight))
        return fail(GDN_ERR_INVALID_ARG, "positions, inv_freq and the weights must be 4-byte aligned");
    const bool has_k = d->hk > 0;
    const auto strided = [&](const void *p, int64_t stride, int64_t row) {
        return range_of(p, (size_t)(((d->rows - 1) * stride + row) * el));
    };
    const Range w[] = {range_of(q_out, (size_t)(d->rows * qrow * el)),
                       range_of(k_out, has_k ? (size_t)(d->rows * krow * el) : 0)};
    const Range r[] = {strided(q, d->q_stride, qrow),
                       has_k ? strided(k, d->k_stride, krow) : range_of(nullptr, 0),
                       range_of(positions, d->rot > 0 ? (size_t)d->rows * 4 : 0),
                       range_of(inv_freq, (size_t)d->rot * 2),
                       range_of(q_weight, q_weight ? (size_t)d->head_dim * 4 : 0),
                       range_of(k_weight, k_weight && has_k ? (size_t)d->head_dim * 4 : 0)};
    const bool same[2] = {q_out == q && d->q_stride == qrow, has_k && k_out == k && d->k_stride == krow};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 6; ++j)
            if (overlaps(w[i], r[j]) && !(i == j && same[i]))
                return fail(GDN_ERR_INVALID_ARG, "an output overlaps an input (in place needs dense rows)");
    if (overlaps(w[0], w[1])) return fail(GDN_ERR_INVALID_ARG, "outputs overlap");
    return lin::launch_qk_norm_rope(*d, q, k, positions, inv_freq, q_weight, k_weight, q_out, k_out,
                                    (cudaStream_t)stream);
}

static gdn_status check_beam_desc(const gdn_beam_desc *d) {
    if (!d) return fail(GDN_ERR_INVALID_ARG, "descriptor is NULL");
    if (d->B < 0 || d->W < 1 || d->W > 64 || d->V < 1)
        return fail(GDN_ERR_INVALID_ARG, "need B >= 0, 1 <= W <= 64, V >= 1 (got %lld, %d, %d)", (long long)d->B, d->W,
                    d->V);
    const int64_t wv = (int64_t)d->W * d->V;
    if (wv > 0x7fffffffLL) return fail(GDN_ERR_UNSUPPORTED, "W * V must be below 2^31");
    if (d->K < 1 || d->K > 64 || d->K > wv)
        return fail(GDN_ERR_INVALID_ARG, "need 1 <= K <= min(64, W V) (got %d)", d->K);
    if (d->dtype != GDN_F32 && d->dtype != GDN_BF16) return fail(GDN_ERR_INVALID_ARG, "unknown dtype %d", d->dtype);
    if (d->row_stride < d->V) return fail(GDN_ERR_INVALID_ARG, "row_stride must be at least V");
    if (d->B > 0x7fffffffLL / d->W) return fail(GDN_ERR_UNSUPPORTED, "more than 2^31 - 1 beams");
    if (d->row_stride > (1LL << 40) || (double)d->B * d->W * (double)d->row_stride > 4.0e15)
        return fail(GDN_ERR_INVALID_ARG, "row_stride too large");
    return GDN_OK;
}

gdn_status gdn_beam_workspace_size(const gdn_beam_desc *d, size_t *bytes) {
    clear_error();
    gdn_status st = check_beam_desc(d);
    if (st != GDN_OK) return st;
    if (!bytes) return fail(GDN_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = lin::beam_workspace(*d);
    return GDN_OK;
}

gdn_status gdn_beam_select(const gdn_beam_desc *d, const void *logits, const float *scores, float *out_scores,
                           int32_t *out_parent, int32_t *out_token, void *workspace, size_t workspace_bytes,
                           gdn_stream_t stream) {
    clear_error();
    gdn_status st = check_beam_desc(d);
    if (st != GDN_OK) return st;
    if (d->B == 0) return GDN_OK;
    if (!logits || !out_scores || !out_parent || !out_token)
        return fail(GDN_ERR_INVALID_ARG, "logits and the three outputs are required");
    const size_t el = d->dtype == GDN_F32 ? 4 : 2;
    if ((uintptr_t)logits % el || !aligned4(scores) || !aligned4(out_scores) || !aligned4(out_parent) ||
        !aligned4(out_token))
        return fail(GDN_ERR_INVALID_ARG, "logits: element-aligned; scores and outputs: 4-byte aligned");
    const size_t need = lin::beam_workspace(*d);
    if (!workspace) return fail(GDN_ERR_WORKSPACE, "workspace is NULL (need %zu bytes)", need);
    if (((uintptr_t)workspace & 255u) != 0) return fail(GDN_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    if (workspace_bytes < need)
        return fail(GDN_ERR_WORKSPACE, "workspace has %zu bytes, need %zu", workspace_bytes, need);
    const size_t rows = (size_t)d->B * d->W, ob = (size_t)d->B * d->K * 4;
    const Range w[] = {range_of(out_scores, ob), range_of(out_parent, ob), range_of(out_token, ob),
                       range_of(workspace, need)};
    const Range r[] = {range_of(logits, ((rows - 1) * (size_t)d->row_stride + d->V) * el),
                       range_of(scores, scores ? rows * 4 : 0)};
    for (int i = 0; i < 4; ++i) {
        for (const Range &x : r)
            if (overlaps(w[i], x)) return fail(GDN_ERR_INVALID_ARG, "an output or the workspace overlaps an input");
        for (int j = i + 1; j < 4; ++j)
            if (overlaps(w[i], w[j])) return fail(GDN_ERR_INVALID_ARG, "outputs and the workspace must not overlap");
    }
    return lin::launch_beam_select(*d, logits, scores, out_scores, out_parent, out_token, workspace,
                                   (cudaStream_t)stream);
}

gdn_status gdn_state_reorder(void *state, const int32_t *parent, int64_t B, int32_t W, size_t row_bytes,
                             gdn_stream_t stream) {
    clear_error();
    if (B < 0 || W < 1 || W > 64) return fail(GDN_ERR_INVALID_ARG, "need B >= 0, 1 <= W <= 64");
    if (row_bytes % 16 != 0) return fail(GDN_ERR_INVALID_ARG, "row_bytes must be a multiple of 16");
    if (B > 0x7fffffffLL / W || row_bytes > (size_t(1) << 40)) return fail(GDN_ERR_UNSUPPORTED, "too many rows or bytes");
    if ((double)B * W * (double)row_bytes > 9.0e18) return fail(GDN_ERR_INVALID_ARG, "problem too large");
    if (B == 0 || row_bytes == 0) return GDN_OK;
    if (!state || !parent) return fail(GDN_ERR_INVALID_ARG, "state and parent are required");
    if (!aligned16(state) || !aligned4(parent))
        return fail(GDN_ERR_INVALID_ARG, "state must be 16-byte aligned, parent 4-byte");
    if (overlaps(range_of(state, (size_t)B * W * row_bytes), range_of(parent, (size_t)B * W * 4)))
        return fail(GDN_ERR_INVALID_ARG, "parent lies inside the state");
    return lin::launch_state_reorder(state, parent, B, W, row_bytes, (cudaStream_t)stream);
}

}  // extern "C"
