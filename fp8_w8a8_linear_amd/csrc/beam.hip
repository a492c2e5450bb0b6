// Beam search beside the mixer: the best continuations of each group's beams (nhm_beam_select)
// and the recurrent states moved to the beams' slots (nhm_beam_reorder).
#include <math.h>

#include "nhm_internal.h"
#include "select_device.h"

namespace nhm {

// ---------------------------------------------------------------- selection
//
// score(b, v) = cum[b] + x[b, v] - lse[b], lse = log(sum_v exp(x)). Within a row the order of the
// scores is the order of the logits, so one pass over the logits is enough: a wave walks a strip
// of a row and keeps, beside the running maximum and sum of the softmax, the strip's n_cand
// largest logits. A second kernel joins each row's strips into its lse and picks each group's best
// from the strips' lists. The pass is bound by bytes: 512 rows of 131,072 bf16 logits take 32 us, in which
// memory hands over 167 MB (5.2 TB/s): the logits' 134 MB and the lines of the cells that are read again. The picking
// takes 11 us, a chain of latencies (64 workgroups; one alone takes 6.6 us).
//
// A lane's share of a 2,048-logit piece is a cell of 32; the pass keeps each cell's maximum in LDS.
// After a span of 8 pieces the n_cand-th largest of the 64 lanes' maxima is a bar that at least
// n_cand logits reach, and so (once there are n_cand entries) is the list's last used entry: only
// cells that reach the bar, about n_cand of 512, are read again, two at a time with a lane per logit.
// The logits that enter collect in LDS until 64 of them are sorted and merged into the list, which
// is sorted with one entry per lane. Any number of entering logits is handled: equal and ascending
// rows cost time, not correctness.
// An earlier form looked for entering logits in every piece as it passed: 583 vector instructions
// per piece against about 200, 41 us for those 512 rows.

// The groups' list entries: score, then flat index.
struct GroupKey {
    double score;
    uint32_t flat;
    template <typename F>
    __device__ __forceinline__ GroupKey each(F f) const {
        const uint64_t u = __builtin_bit_cast(uint64_t, score);
        return GroupKey{__builtin_bit_cast(double, (uint64_t)f((uint32_t)(u >> 32)) << 32 | f((uint32_t)u)), f(flat)};
    }
};
__device__ __forceinline__ bool better(const GroupKey& a, const GroupKey& b) {
    return a.score > b.score || (a.score == b.score && a.flat < b.flat);
}

constexpr int kStripWaves = 4;      // waves per workgroup, each on its own

template <bool F32>
__global__ __launch_bounds__(kStripWaves * 64, F32 ? 3 : 4) void beam_strip_kernel(const BeamArgs g) {
    __shared__ StripLds s_lds[kStripWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t id = (int64_t)blockIdx.x * kStripWaves + wave;
    const int64_t row = id / g.n_strips;
    const int strip = (int)(id - row * g.n_strips);
    if (row >= g.n_groups * g.n_beams) return;
    if (g.finished && g.finished[row] != 0) return;          // its logits are not used
    constexpr int kSize = F32 ? 4 : 2;
    const char* const base = (F32 ? reinterpret_cast<const char*>(g.logits_f32)
                                  : reinterpret_cast<const char*>(g.logits_bf16)) + row * g.ld * kSize;

    StripBest<F32> best{&s_lds[wave], g.n_cand};
    float* const cmax = s_lds[wave].max;
    float top = -INFINITY;          // this lane's largest logit and sum of exp(x - top)
    double sum = 0.0;

    const int64_t p_beg = (int64_t)strip * g.strip_pieces * kPiece;
    const int64_t p_end = min(p_beg + (int64_t)g.strip_pieces * kPiece, g.vocab);
    Piece<F32> cur;
    cur.load(base, p_beg, g.vocab, lane);
    for (int64_t span = p_beg; span < p_end; span += kSpan * kPiece) {
        const int pieces = (int)min((int64_t)kSpan, (p_end - span + kPiece - 1) / kPiece);
        float span_max = -INFINITY;
        for (int q = 0; q < pieces; ++q) {
            const int64_t p = span + (int64_t)q * kPiece;
            float x[32], mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = cur.get(i);
#pragma unroll
            for (int i = 0; i < 32; ++i) asm volatile("" : "+v"(x[i]));
            // the next piece on its way while this one, now in x, is worked on (issued ahead of the
            // unpacking it was waited for at once, at the join behind its branch)
            if (p + kPiece < p_end) cur.load(base, p + kPiece, g.vocab, lane);
#pragma unroll
            for (int i = 0; i < 32; i += 2) mx = max3(mx, x[i], x[i + 1]);
            float now = fmaxf(top, mx);
            float ref = now > -INFINITY ? now : 0.f;
            float part = 0.f;        // 32 terms in f32, the strip's sum in f64
#pragma unroll
            for (int i = 0; i < 32; i += 8) {                // eight at a time: no sum waits for its exponential
                float e[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) e[j] = __builtin_amdgcn_exp2f((x[i + j] - ref) * kLog2e);
                __builtin_amdgcn_sched_barrier(0);
                part += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
            }
            // The maximum passes over quiet NaN and the sum does not, and inf - inf is NaN: a piece with
            // either is cleaned and taken again. Other pieces pay two comparisons for it.
            if (__ballot(part != part || mx != mx)) {
                mx = -INFINITY;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    asm volatile("" : "+v"(x[i]));           // not to be done ahead of the branch
                    x[i] = clean_logit(x[i]);
                    mx = fmaxf(mx, x[i]);
                }
                now = fmaxf(top, mx);
                ref = now > -INFINITY ? now : 0.f;
                part = 0.f;
#pragma unroll
                for (int i = 0; i < 32; ++i)                 // +inf entries share the probability
                    part += now < INFINITY ? __builtin_amdgcn_exp2f((x[i] - ref) * kLog2e) : x[i] == INFINITY ? 1.f : 0.f;
            }
            const float keep = top == now ? 1.f : __builtin_amdgcn_exp2f((top - ref) * kLog2e);   // 0 from -inf
            sum = sum * (double)keep + (double)part;
            top = now;
            cmax[q * 64 + lane] = mx;
            span_max = fmaxf(span_max, mx);
        }

        best.look(base, span, pieces, p_end, span_max, lane);
    }
    const float all_top = wave_max(top);
    sum = wave_sum_f64(top == all_top ? sum : sum * (double)__expf(top - all_top));
    if (lane < g.n_cand) g.strip_keys[id * g.n_cand + lane] = best.list.v;
    if (lane == 0) {
        g.strip_top[id] = all_top;
        g.strip_sum[id] = sum;
    }
}

// One workgroup per group: each row's lse from its strips, then the best continuations. Each lane
// takes a strip's sorted list, kPlaces entries at a time. The n_cand-th of 64 lists' best entries is a
// bar for the others; what reaches it collects and is merged as in the strips, and once none of the
// last entries read does, the rest of the lists is left.
constexpr int kPickWaves = 8, kPlaces = 8;
constexpr int64_t kPickGroups = int64_t(1) << 22;   // groups per launch: a launch holds fewer than 2^32 threads

__global__ __launch_bounds__(kPickWaves * 64) void beam_pick_kernel(const BeamArgs g) {
    __shared__ double s_lse[32];                    // each beam's log(sum exp(x - top)) (finished: not used)
    __shared__ float s_top[32];
    __shared__ GroupKey s_new[kPickWaves][128];
    __shared__ GroupKey s_list[kPickWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row0 = (int64_t)blockIdx.x * g.n_beams;
    const int S = g.n_strips, K = g.n_beams, all = K * S;
    // entries of places c .. c + kPlaces - 1 of strip i of the group (0: none)
    auto load = [&](int i, int c, uint64_t (&e)[kPlaces]) {
        const bool on = i < all && !(g.finished && g.finished[row0 + i / S] != 0);
        const uint64_t* src = g.strip_keys + (row0 * S + i) * g.n_cand + c;
#pragma unroll
        for (int j = 0; j < kPlaces; ++j) e[j] = on && c + j < g.n_cand ? src[j] : 0;
    };
    uint64_t e[kPlaces];
    load(wave * 64 + lane, 0, e);                   // in flight while the sums are joined
    for (int b = wave; b < K; b += kPickWaves) {
        if (g.finished && g.finished[row0 + b] != 0) continue;
        const int64_t id0 = (row0 + b) * S;
        float t0 = lane < S ? g.strip_top[id0 + lane] : -INFINITY;
        const double s0 = lane < S ? g.strip_sum[id0 + lane] : 0.0;
        float top = t0;
        for (int s = lane + 64; s < S; s += 64) top = fmaxf(top, g.strip_top[id0 + s]);
        top = wave_max(top);
        double sum = t0 > -INFINITY ? s0 * (t0 == top ? 1.0 : exp((double)t0 - (double)top)) : 0.0;
        for (int s = lane + 64; s < S; s += 64) {
            const float t = g.strip_top[id0 + s];
            if (t > -INFINITY) sum += g.strip_sum[id0 + s] * (t == top ? 1.0 : exp((double)t - (double)top));
        }
        sum = wave_sum_f64(sum);
        if (lane == 0) {
            s_top[b] = top;
            s_lse[b] = log(sum);
        }
    }
    __syncthreads();

    const GroupKey none{-INFINITY, 0xffffffffu};
    GroupKey list = none, last = none;
    double bar = -INFINITY;                         // n_cand scores are known to reach it
    int pending = 0;
    bool first = true;
    GroupKey* const buf = s_new[wave];
    auto flush = [&](int n) {
        wave_lds_order();
        GroupKey k = lane < n ? buf[lane] : none;
        sort64(k, lane);
        if (first) list = k;
        else merge64(list, k, lane);
        first = false;
        last = list.each([&](uint32_t w) { return (uint32_t)__shfl((int)w, g.n_cand - 1); });
    };
    for (int i0 = wave * 64; i0 < all; i0 += kPickWaves * 64) {
        const int i = i0 + lane, b = i < all ? i / S : 0;
        const double cum = g.cum[row0 + b];
        const float top = s_top[b];
        const double lse = s_lse[b];
        const bool fin = g.finished && g.finished[row0 + b] != 0;
        const uint32_t flat0 = (uint32_t)(b * g.vocab);
        for (int c = 0; c < g.n_cand; c += kPlaces) {
            if (i0 != wave * 64 || c != 0) load(i, c, e);
            bool more = false;
#pragma unroll
            for (int j = 0; j < kPlaces; ++j) {
                GroupKey k = none;
                if (e[j] != 0) {
                    // x - top first: +inf entries score cum - log(their number). cum + (x - top) is
                    // exact in f64 for f32 values within 29 bits of each other, so equal rows
                    // whose scores tie do so bit for bit, whatever lse's last bits are
                    const float x = unordered((uint32_t)(e[j] >> 32));
                    const double d = x == top ? 0.0 : (double)x - (double)top;
                    k = GroupKey{(cum + d) - lse, flat0 + (uint32_t)~(uint32_t)e[j]};
                } else if (fin && c + j == 0 && i < all && i == b * S) {
                    k = GroupKey{cum, flat0 + (uint32_t)g.eos};      // a finished beam's one continuation
                }
                if (c == 0 && j == 0) {
                    // the n_cand-th of these 64 lists' best, rounded down to f32, is a bar
                    float f = (float)k.score;
                    if ((double)f > k.score) f = unordered(ordered(f) - 1);
                    BarKey h{k.score > -INFINITY ? ordered(f) : 0};
                    sort64(h, lane);
                    const uint32_t t = take(h.v, g.n_cand - 1);
                    if (t != 0) bar = fmax(bar, (double)unordered(t));
                }
                const bool in = k.score > -INFINITY && k.score >= bar && better(k, last);
                const uint64_t m = __ballot(in);
                if (j == kPlaces - 1) more = m != 0;
                if (m == 0) continue;
                if (in) buf[pending + lanes_below(m)] = k;
                pending += __popcll(m);
                if (pending >= 64) {
                    flush(64);
                    pending -= 64;
                    if (lane < pending) buf[lane] = buf[64 + lane];
                    wave_lds_order();
                }
            }
            if (!more) break;        // the lists are sorted: what follows is no better
        }
    }
    if (pending > 0) flush(pending);
    // the waves' lists in pairs; waves past the last strip hold none
    int half = kPickWaves / 2;
    while (half > 0 && half * 64 >= all) half >>= 1;
    for (; half > 0; half >>= 1) {
        if (wave >= half && wave < 2 * half) s_list[wave][lane] = list;
        __syncthreads();
        if (wave < half) merge64(list, s_list[wave + half][lane], lane);
    }
    if (wave == 0 && lane < g.n_cand) {
        const int64_t o = (int64_t)blockIdx.x * g.n_cand + lane;
        const bool empty = list.flat == 0xffffffffu;
        g.scores[o] = (float)list.score;
        g.parents[o] = empty ? -1 : (int32_t)(list.flat / (uint32_t)g.vocab);
        g.tokens[o] = empty ? -1 : (int32_t)(list.flat % (uint32_t)g.vocab);
    }
}

// Strips per row: enough waves to fill the chip (4,096: 16 per CU), none shorter than a piece.
static void beam_strips(int64_t rows, int64_t vocab, int* strips, int* pieces) {
    const int64_t all = (vocab + kPiece - 1) / kPiece;
    int64_t s = rows > 0 ? (4096 + rows - 1) / rows : 1;
    s = s > 256 ? 256 : s;
    s = s > all ? all : s;
    *pieces = (int)((all + s - 1) / s);
    *strips = (int)((all + *pieces - 1) / *pieces);
}

struct BeamWs { size_t keys, sum, top, total; };
static BeamWs beam_ws(int64_t rows, int64_t vocab, int32_t n_cand) {
    int strips, pieces;
    beam_strips(rows, vocab, &strips, &pieces);
    const size_t n = (size_t)rows * strips;
    BeamWs w;
    w.keys = 0;
    w.sum = align_up(n * n_cand * sizeof(uint64_t), 256);
    w.top = w.sum + align_up(n * sizeof(double), 256);
    w.total = w.top + align_up(n * sizeof(float), 256);
    return w;
}
size_t beam_ws_bytes(int64_t rows, int64_t vocab, int32_t n_cand) { return beam_ws(rows, vocab, n_cand).total; }

nhm_status launch_beam_select(BeamArgs g, void* ws, hipStream_t st) {
    const int64_t rows = g.n_groups * g.n_beams;
    beam_strips(rows, g.vocab, &g.n_strips, &g.strip_pieces);
    const BeamWs w = beam_ws(rows, g.vocab, g.n_cand);
    char* const b = static_cast<char*>(ws);
    g.strip_keys = reinterpret_cast<uint64_t*>(b + w.keys);
    g.strip_sum = reinterpret_cast<double*>(b + w.sum);
    g.strip_top = reinterpret_cast<float*>(b + w.top);
    const dim3 grid((unsigned)((rows * g.n_strips + kStripWaves - 1) / kStripWaves));
    if (g.logits_f32) beam_strip_kernel<true><<<grid, dim3(kStripWaves * 64), 0, st>>>(g);
    else beam_strip_kernel<false><<<grid, dim3(kStripWaves * 64), 0, st>>>(g);
    count_launch(Kern::kBeamRows, rows);
    nhm_status s = check_launch("beam strips");
    if (s != NHM_OK) return s;
    for (int64_t g0 = 0; g0 < g.n_groups; g0 += kPickGroups) {
        BeamArgs p = g;
        const int64_t row0 = g0 * g.n_beams, id0 = row0 * g.n_strips;
        p.cum += row0;
        if (p.finished) p.finished += row0;
        p.strip_keys += id0 * g.n_cand;
        p.strip_sum += id0;
        p.strip_top += id0;
        p.scores += g0 * g.n_cand;
        p.parents += g0 * g.n_cand;
        p.tokens += g0 * g.n_cand;
        const int64_t ng = g.n_groups - g0 < kPickGroups ? g.n_groups - g0 : kPickGroups;
        beam_pick_kernel<<<dim3((unsigned)ng), dim3(kPickWaves * 64), 0, st>>>(p);
    }
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
// Bound by the copied bytes: 23 layers' f32 states of 12 beams, 0.59 GB read and as much written, 210 us (5.6 TB/s).

constexpr int kReorderThreads = 256;
constexpr int kReorderLoads = 4;                                        // 16-byte loads in flight per thread
constexpr int kReorderPiece = kReorderThreads * 16 * kReorderLoads;      // bytes of a row per workgroup

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
            const int pj = __builtin_amdgcn_readlane(has ? par : -1, j);
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
    const int64_t end = g.ssm_bytes + g.conv_bytes;
    char* const ssm = static_cast<char*>(g.pools[blockIdx.z].ssm);
    char* const conv = reinterpret_cast<char*>(g.pools[blockIdx.z].conv);
    for (int j = 0; j < K; ++j) {
        if (s_src[j] < 0) continue;
        const int64_t src = s_src[j], dst = s_dst[j];
        // straight-line loads (a piece past the row's end reads its last 16 bytes again), so that
        // all of them are in flight before the first store waits
        v4u v[kReorderLoads];
        char* to[kReorderLoads];
#pragma unroll
        for (int u = 0; u < kReorderLoads; ++u) {
            const int64_t b = min(off + (u * kReorderThreads + t) * 16, end - 16);
            const bool win = b >= g.ssm_bytes;
            char* const pool = win ? conv : ssm;
            const int64_t row = win ? g.conv_bytes : g.ssm_bytes, at = win ? b - g.ssm_bytes : b;
            v[u] = *reinterpret_cast<const v4u*>(pool + src * row + at);
            to[u] = pool + dst * row + at;
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < kReorderLoads; ++u)
            if (off + (u * kReorderThreads + t) * 16 < end) *reinterpret_cast<v4u*>(to[u]) = v[u];
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
