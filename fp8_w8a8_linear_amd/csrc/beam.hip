// Beam search beside the mixer: the best continuations of each group's beams (nhm_beam_select)
// and the recurrent states moved to the beams' slots (nhm_beam_reorder).
//
// Selection: score(b, v) = cum[b] + x[b, v] - lse[b]. One kernel forms each row's lse, a second
// picks each group's best continuations one after another.
#include <math.h>

#include "nhm_device.h"
#include "nhm_internal.h"

namespace nhm {

// A logit as the selection reads it: NaN counts as -inf.
__device__ __forceinline__ float load_logit(const BeamArgs& g, int64_t row, int64_t v) {
    const float x = g.logits_f32 ? g.logits_f32[row * g.ld + v] : bf16_to_f32(g.logits_bf16[row * g.ld + v]);
    return x == x ? x : -INFINITY;
}
// x - top with the convention that the top's own entries (infinite ones too) give 0
__device__ __forceinline__ float below_top(float x, float top) { return x == top ? 0.f : x - top; }

constexpr int kBeamThreads = 256;

// top[row] and log(sum exp(x - top)) [row]
__global__ __launch_bounds__(kBeamThreads) void beam_rows_kernel(const BeamArgs g) {
    __shared__ float s_top[kBeamThreads];
    __shared__ double s_sum[kBeamThreads];
    const int64_t row = blockIdx.x;
    const int t = threadIdx.x;
    float top = -INFINITY;
    for (int64_t v = t; v < g.vocab; v += kBeamThreads) top = fmaxf(top, load_logit(g, row, v));
    s_top[t] = top;
    __syncthreads();
    for (int i = 0; i < kBeamThreads; ++i) top = fmaxf(top, s_top[i]);
    double sum = 0.0;
    for (int64_t v = t; v < g.vocab; v += kBeamThreads) sum += (double)expf(below_top(load_logit(g, row, v), top));
    s_sum[t] = sum;
    __syncthreads();
    if (t == 0) {
        sum = 0.0;
        for (int i = 0; i < kBeamThreads; ++i) sum += s_sum[i];
        g.row_top[row] = top;
        g.row_log[row] = log(sum);
    }
}

__global__ __launch_bounds__(kBeamThreads) void beam_pick_kernel(const BeamArgs g) {
    __shared__ double s_best[kBeamThreads];
    __shared__ int64_t s_at[kBeamThreads];
    const int64_t grp = blockIdx.x;
    const int t = threadIdx.x;
    const int64_t all = (int64_t)g.n_beams * g.vocab;
    double last = INFINITY;       // the previous pick: the next one comes after it in the order
    int64_t last_at = -1;
    for (int c = 0; c < g.n_cand; ++c) {
        double best = -INFINITY;
        int64_t at = -1;
        for (int64_t f = t; f < all; f += kBeamThreads) {
            const int b = (int)(f / g.vocab);
            const int64_t v = f - b * g.vocab, row = grp * g.n_beams + b;
            const double cum = g.cum[row];
            double s;
            if (g.finished && g.finished[row] != 0) {
                s = v == g.eos ? cum : -INFINITY;
            } else {
                const float x = load_logit(g, row, v);
                s = x == -INFINITY ? -INFINITY : cum + ((double)below_top(x, g.row_top[row]) - g.row_log[row]);
            }
            if (!(s > -INFINITY)) continue;
            if (!(s < last || (s == last && f > last_at))) continue;
            if (s > best) { best = s; at = f; }      // f ascends: the first of equals stays
        }
        s_best[t] = best;
        s_at[t] = at;
        __syncthreads();
        for (int i = 0; i < kBeamThreads; ++i)
            if (s_at[i] >= 0 && (at < 0 || s_best[i] > best || (s_best[i] == best && s_at[i] < at))) {
                best = s_best[i];
                at = s_at[i];
            }
        __syncthreads();
        last = best;
        last_at = at;
        if (t == 0) {
            const int64_t o = grp * g.n_cand + c;
            g.scores[o] = (float)best;
            g.parents[o] = at < 0 ? -1 : (int32_t)(at / g.vocab);
            g.tokens[o] = at < 0 ? -1 : (int32_t)(at % g.vocab);
        }
        if (at < 0) last = -INFINITY;                // no more: every later place stays empty
    }
}

size_t beam_ws_bytes(int64_t rows, int64_t, int32_t) { return align_up((size_t)rows * (sizeof(double) + sizeof(float)), 256); }

nhm_status launch_beam_select(BeamArgs g, void* ws, hipStream_t st) {
    const int64_t rows = g.n_groups * g.n_beams;
    g.row_log = static_cast<double*>(ws);
    g.row_top = reinterpret_cast<float*>(g.row_log + rows);
    beam_rows_kernel<<<dim3((unsigned)rows), dim3(kBeamThreads), 0, st>>>(g);
    count_launch(Kern::kBeamRows, rows);
    nhm_status s = check_launch("beam rows");
    if (s != NHM_OK) return s;
    beam_pick_kernel<<<dim3((unsigned)g.n_groups), dim3(kBeamThreads), 0, st>>>(g);
    count_launch(Kern::kBeamPick, g.n_groups);
    return check_launch("beam pick");
}

// ---------------------------------------------------------------- state reorder
//
// The first child of a parent keeps the parent's row where it is, so only the further children's
// rows move, into rows that no beam continues: no row is both read and written, the copies need
// no order and no second buffer, and the bytes are those of the rows that must exist twice.
// Every workgroup derives its group's slots itself (n_beams <= 32 entries, one lane each) and
// copies one piece of one layer's row for every beam of the group that has a copy to receive.

constexpr int kReorderThreads = 256;
constexpr int kReorderPiece = 64 * 1024;    // bytes of a row per workgroup

__global__ __launch_bounds__(kReorderThreads) void beam_reorder_kernel(const ReorderArgs g) {
    __shared__ int s_src[32], s_dst[32];
    const int t = threadIdx.x;
    const int64_t grp = blockIdx.y;
    const int K = g.n_beams;
    if (t < 64) {   // one wave: lane j is beam j
        const int64_t o = grp * K + t;
        const int par = t < K ? g.parents[o] : -1;
        const int slot = t < K ? g.slots[o] : -1;
        const bool has = par >= 0 && par < K;
        // first: no earlier beam continues the same parent; used: some beam continues this one
        bool first = has, used = false;
        for (int j = 0; j < K; ++j) {
            const int pj = __shfl(has ? par : -1, j);
            if (j < t && has && pj == par) first = false;
            if (pj == t) used = true;
        }
        const uint64_t lanes = (uint64_t(1) << K) - 1;      // K <= 32
        const uint64_t later = __ballot(t < K && !first) & lanes, freed = __ballot(t < K && !used) & lanes;
        const uint64_t below = (uint64_t(1) << t) - 1;
        // the beam whose slot this one takes: its parent, or the i-th freed one for the i-th later beam
        int from = has ? par : 0;
        if (!first) {
            int i = __popcll(later & below);
            uint64_t f = freed;
            while (i-- > 0) f &= f - 1;
            from = f ? __ffsll((unsigned long long)f) - 1 : 0;
        }
        const int mine = __shfl(slot, from);
        const int src = __shfl(slot, has ? par : 0);
        if (t < K) {
            const bool copy = has && !first && src >= 0 && src < g.n_slots && mine >= 0 && mine < g.n_slots;
            s_src[t] = copy ? src : -1;
            s_dst[t] = mine;
            if (blockIdx.x == 0 && blockIdx.z == 0) g.new_slots[o] = mine;
        }
    }
    __syncthreads();
    const int64_t off = (int64_t)blockIdx.x * kReorderPiece;   // within the layer's row: state, then window
    for (int j = 0; j < K; ++j) {
        if (s_src[j] < 0) continue;
        const int64_t src = s_src[j], dst = s_dst[j];
        for (int64_t b = off + t * 16; b < off + kReorderPiece && b < g.ssm_bytes + g.conv_bytes; b += kReorderThreads * 16) {
            const bool win = b >= g.ssm_bytes;
            char* pool = static_cast<char*>(win ? g.pools[blockIdx.z].conv : g.pools[blockIdx.z].ssm);
            const int64_t row = win ? g.conv_bytes : g.ssm_bytes, at = win ? b - g.ssm_bytes : b;
            *reinterpret_cast<uint4*>(pool + dst * row + at) = *reinterpret_cast<const uint4*>(pool + src * row + at);
        }
    }
}

nhm_status launch_beam_reorder(const ReorderArgs& g, int64_t n_groups, int32_t n_layers, hipStream_t st) {
    const unsigned pieces = (unsigned)((g.ssm_bytes + g.conv_bytes + kReorderPiece - 1) / kReorderPiece);
    for (int64_t g0 = 0; g0 < n_groups; g0 += 65535) {    // the grid's y extent
        ReorderArgs p = g;
        p.parents += g0 * g.n_beams;
        p.slots += g0 * g.n_beams;
        p.new_slots += g0 * g.n_beams;
        const int64_t ng = n_groups - g0 < 65535 ? n_groups - g0 : 65535;
        beam_reorder_kernel<<<dim3(pieces, (unsigned)ng, (unsigned)n_layers), dim3(kReorderThreads), 0, st>>>(p);
    }
    count_launch(Kern::kBeamReorder, n_groups);
    return check_launch("beam reorder");
}

}  // namespace nhm
