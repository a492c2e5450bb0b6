// Scoring of tokens (nhm_token_logprobs): of each row of logits the given token's log probability and
// rank, the entropy, and the best alternatives.
//
// With top = max x, S = sum exp(x - top), M = sum exp(x - top) (x - top) (no term of which is positive):
//   log p(v) = (x_v - top) - log S,  H = log S - M / S,  rank = 1 + #{v before the token, by logit, then index}
// One pass over the logits: a wave walks a strip of a row and keeps the running top, S, M, the count and
// the strip's best logits (as the beam selection does); a second kernel joins a row's strips. Bound by bytes where rows are
// many (1,021 x 131,072 bf16, 268 MB: 55 us without alternatives, 4.9 TB/s, 71 with five, for the cells read again and their sorting); one row
// takes 7.2 us without and 15.8 with 20 alternatives, two launches of latency chains.
#include <math.h>

#include "nhm_internal.h"
#include "select_device.h"

namespace nhm {

constexpr double kLn2 = 0.69314718055994530942;
constexpr int kScoreWaves = 4;      // waves per workgroup, each on its own

// The largest float below x, so that v > below(x) is v >= x (-0 counts as +0); x is not -inf.
__device__ __forceinline__ float below(float x) {
    const uint32_t o = ordered(x) - 1;
    return unordered(o == 0x7fffffffu ? o - 1 : o);
}

template <bool F32, bool kTop>
__global__ __launch_bounds__(kScoreWaves * 64, F32 ? 3 : 4) void score_strip_kernel(const ScoreArgs g) {
    __shared__ StripLds s_lds[kTop ? kScoreWaves : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t id = (int64_t)blockIdx.x * kScoreWaves + wave;
    const int64_t row = id / g.n_strips;
    const int strip = (int)(id - row * g.n_strips);
    if (row >= g.rows) return;
    constexpr int kSize = F32 ? 4 : 2, E = Piece<F32>::E;
    const char* const base = static_cast<const char*>(g.logits) + row * g.ld * kSize;
    const int64_t p_beg = (int64_t)strip * g.strip_pieces * kPiece;
    const int64_t p_end = min(p_beg + (int64_t)g.strip_pieces * kPiece, g.vocab);
    Piece<F32> cur;
    cur.load(base, p_beg, g.vocab, lane);

    const int64_t token = g.tokens ? g.tokens[row] : -1;
    const bool asked = token >= 0 && token < g.vocab;
    float xt = INFINITY;            // the token's logit: entries above it come before it, equal ones by index
    if (asked) xt = clean_logit(F32 ? *reinterpret_cast<const float*>(base + token * 4)
                                    : bf16_to_f32(*reinterpret_cast<const uint16_t*>(base + token * 2)));
    // what an entry ahead of the token must exceed (-inf, and NaN, tie with a token at -inf: the join adds them)
    const float over = xt == -INFINITY ? INFINITY : below(xt);
    uint32_t count = 0;
    float top = -INFINITY;          // this lane's largest logit, sum of exp(x - top) and of that times log2(e) (x - top)
    double sum = 0.0, mom = 0.0;
    StripBest<F32> best{&s_lds[kTop ? wave : 0], g.n_top};

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
            if (p + kPiece < p_end) cur.load(base, p + kPiece, g.vocab, lane);
#pragma unroll
            for (int i = 0; i < 32; i += 2) mx = maximum3(mx, x[i], x[i + 1]);
            // A piece with a NaN is cleaned and its maxima taken again (1,021 x 131,072 with one in every piece 72 us for 67). The terms below
            // do not show one: their bound takes it to 0.
            if (__ballot(mx != mx)) {
                mx = -INFINITY;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    asm volatile("" : "+v"(x[i]));
                    x[i] = clean_logit(x[i]);
                    mx = fmaxf(mx, x[i]);
                }
            }
            const float now = fmaxf(top, mx), ref = now > -INFINITY ? now : 0.f;
            float part = 0.f, pmom = 0.f;                    // 32 terms in f32, the strip's sums in f64
#pragma unroll
            for (int i = 0; i < 32; i += 8) {                // eight at a time: no sum waits for its exponential
                float d[8], e[8];
                // the bound takes -inf, and NaN, to a term of zero in both sums
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] = fmaxf((x[i + j] - ref) * kLog2e, -1e4f);
#pragma unroll
                for (int j = 0; j < 8; ++j) e[j] = __builtin_amdgcn_exp2f(d[j]);
                __builtin_amdgcn_sched_barrier(0);
                part += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
#pragma unroll
                for (int j = 0; j < 8; ++j) pmom = fmaf(e[j], d[j], pmom);
            }
            if (__ballot(now == INFINITY)) {                 // +inf entries share the probability
                if (now == INFINITY) {
                    part = pmom = 0.f;
#pragma unroll
                    for (int i = 0; i < 32; ++i) part += x[i] == INFINITY ? 1.f : 0.f;
                }
            }
            if (top != now) {
                const double keep = top == -INFINITY || now == INFINITY ? 0.0 : (double)__builtin_amdgcn_exp2f((top - now) * kLog2e);
                mom = keep > 0.0 ? keep * (mom + (double)((top - now) * kLog2e) * sum) : 0.0;
                sum *= keep;
                top = now;
            }
            sum += (double)part;
            mom += (double)pmom;
            // entries before the token
            if (p + kPiece <= token || p > token) {          // the whole piece on one side
                const float thr = p > token ? xt : over;
#pragma unroll
                for (int i = 0; i < 32; ++i) count += __popcll(__ballot(x[i] > thr));
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const int64_t at = p + ((i / E) * 64 + lane) * E + i % E;
                    count += __popcll(__ballot(x[i] > (at < token ? over : xt)));
                }
            }
            if constexpr (kTop) {
                s_lds[wave].max[q * 64 + lane] = mx;
                span_max = fmaxf(span_max, mx);
            }
        }
        if constexpr (kTop) best.look(base, span, pieces, p_end, span_max, lane);
    }
    const float all = wave_max(top);
    if (top != all) {
        const double keep = top == -INFINITY || all == INFINITY ? 0.0 : (double)__builtin_amdgcn_exp2f((top - all) * kLog2e);
        mom = keep > 0.0 ? keep * (mom + (double)((top - all) * kLog2e) * sum) : 0.0;
        sum *= keep;
    }
    sum = wave_sum_f64(sum);
    mom = wave_sum_f64(mom);
    if constexpr (kTop)
        if (lane < g.n_top) g.strip_keys[id * g.n_top + lane] = best.list.v;
    if (lane == 0) g.strips[id] = ScoreStrip{sum, mom, all, count};
}

// One workgroup per row: of one wave where the strips are few, else wave 0 forms the sums while the others merge
// the strips' lists (a row of 131,072 with 20 alternatives: 15.8 us, with eight waves that all did both 18.8).
constexpr int kJoinWaves = 16;

__global__ __launch_bounds__(kJoinWaves * 64) void score_join_kernel(const ScoreArgs g) {
    __shared__ StripKey s_list[kJoinWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int64_t row = blockIdx.x;
    const int S = g.n_strips;
    StripKey list{0};
    double top = 0.0, lse = 0.0;         // wave 0: the row's largest logit, and log of the sum beside it
    if (wave == 0) {
        const ScoreStrip* const st = g.strips + row * S;
        const int64_t token = g.tokens ? g.tokens[row] : -1;
        const bool asked = token >= 0 && token < g.vocab;
        const int64_t at = row * g.ld + (asked ? token : 0);
        const float x = clean_logit(g.f32 ? static_cast<const float*>(g.logits)[at] : bf16_to_f32(static_cast<const uint16_t*>(g.logits)[at]));
        float topf = -INFINITY;
        for (int s = lane; s < S; s += 64) topf = fmaxf(topf, st[s].top);
        topf = wave_max(topf);
        top = topf;
        double sum = 0.0, mom = 0.0;
        uint32_t count = 0;
        for (int s = lane; s < S; s += 64) {
            const ScoreStrip v = st[s];
            count += v.count;
            if (v.top == topf) {
                sum += v.sum;
                mom += v.mom;
            } else if (v.top > -INFINITY && topf < INFINITY) {
                const double d = (double)v.top - top, keep = exp(d);
                sum += keep * v.sum;
                mom += keep * (v.mom + d * (1.0 / kLn2) * v.sum);
            }
        }
        sum = wave_sum_f64(sum);
        mom = wave_sum_f64(mom);
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) count += __shfl_xor(count, o);
        const bool none = topf == -INFINITY;              // nothing is possible
        lse = none ? 0.0 : log(sum);
        if (lane == 0) {
            if (g.logprobs) g.logprobs[row] = !asked ? 0.f : x == -INFINITY ? -INFINITY : (float)((x == topf ? 0.0 : (double)x - top) - lse);
            // all the entries ahead of a token at -inf come before it
            if (g.ranks) g.ranks[row] = asked ? (int32_t)(count + 1 + (x == -INFINITY ? (uint32_t)token : 0u)) : 0;
            if (g.entropy) g.entropy[row] = none ? 0.f : (float)(lse - kLn2 * (mom / sum));
        }
    }
    if (g.n_top == 0) return;
    const uint64_t* const keys = g.strip_keys + row * S * g.n_top;
    const int step = waves > 1 ? waves - 1 : 1, s0 = waves > 1 ? wave - 1 : 0;
    if (s0 >= 0)
        for (int s = s0; s < S; s += step) {
            const StripKey k{lane < g.n_top ? keys[(int64_t)s * g.n_top + lane] : 0};
            if (s == s0) list = k;
            else merge64(list, k, lane);
        }
    for (int half = waves / 2; half > 0; half >>= 1) {
        if (wave >= half && wave < 2 * half) s_list[wave][lane] = list;
        __syncthreads();
        if (wave < half) merge64(list, s_list[wave + half][lane], lane);
    }
    if (wave == 0 && lane < g.n_top) {
        const int64_t o = row * g.n_top + lane;
        const float x = unordered((uint32_t)(list.v >> 32));
        // beside +inf entries the finite ones have no probability
        const double lp = list.v == 0 ? -INFINITY : ((double)x == top ? 0.0 : (double)x - top) - lse;
        g.top_tokens[o] = lp > -INFINITY ? (int32_t)~(uint32_t)list.v : -1;
        g.top_logprobs[o] = (float)lp;
    }
}

// Strips per row: enough waves to fill the chip (4,096: 16 per CU), none shorter than a piece.
static void score_strips(int64_t rows, int64_t vocab, int* strips, int* pieces) {
    const int64_t all = (vocab + kPiece - 1) / kPiece;
    int64_t s = rows > 0 ? (4096 + rows - 1) / rows : 1;
    s = s > 256 ? 256 : s;
    s = s > all ? all : s;
    *pieces = (int)((all + s - 1) / s);
    *strips = (int)((all + *pieces - 1) / *pieces);
}

size_t score_ws_bytes(int64_t rows, int64_t vocab, int32_t n_top) {
    int strips, pieces;
    score_strips(rows, vocab, &strips, &pieces);
    const size_t n = (size_t)rows * strips;
    return align_up(n * sizeof(ScoreStrip), 256) + align_up(n * n_top * sizeof(uint64_t), 256);
}

nhm_status launch_score(ScoreArgs g, void* ws, hipStream_t st) {
    score_strips(g.rows, g.vocab, &g.n_strips, &g.strip_pieces);
    const size_t n = (size_t)g.rows * g.n_strips;
    g.strips = static_cast<ScoreStrip*>(ws);
    g.strip_keys = reinterpret_cast<uint64_t*>(static_cast<char*>(ws) + align_up(n * sizeof(ScoreStrip), 256));
    const dim3 grid((unsigned)((n + kScoreWaves - 1) / kScoreWaves)), block(kScoreWaves * 64);
    if (g.f32) {
        if (g.n_top > 0) score_strip_kernel<true, true><<<grid, block, 0, st>>>(g);
        else score_strip_kernel<true, false><<<grid, block, 0, st>>>(g);
    } else {
        if (g.n_top > 0) score_strip_kernel<false, true><<<grid, block, 0, st>>>(g);
        else score_strip_kernel<false, false><<<grid, block, 0, st>>>(g);
    }
    count_launch(Kern::kScoreRows, g.rows);
    const nhm_status s = check_launch("token scores");
    if (s != NHM_OK) return s;
    // one launch: fewer than 2^24 rows of one wave are fewer than 2^30 threads (more than 8 strips, for which a row takes 16
    // waves, have only calls of at most 511 rows)
    const int waves = g.n_top > 0 && g.n_strips > 8 ? kJoinWaves : 1;
    score_join_kernel<<<dim3((unsigned)g.rows), dim3(waves * 64), 0, st>>>(g);
    count_launch(Kern::kScoreJoin, g.rows);
    return check_launch("token scores' join");
}

}  // namespace nhm
