// Beam search beside the mixer: the best continuations of each group's beams (nhm_beam_select)
// and the recurrent states moved to the beams' slots (nhm_beam_reorder).
#include <math.h>

#include "nhm_device.h"
#include "nhm_internal.h"

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

// x as the selection reads it: NaN counts as -inf.
__device__ __forceinline__ float clean_logit(float x) { return x == x ? x : -INFINITY; }

// The value of lane ^ M, by lane moves in the VALU (an LDS permute takes a round trip per step):
// within quads, then mirrored halves of a row of 16 (xor 7, undone by xor 3), a rotation by 8, and
// the swaps of rows and of halves of the wave.
template <int M>
__device__ __forceinline__ uint32_t lane_xor(uint32_t v) {
    if constexpr (M == 1) return __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, true);
    if constexpr (M == 2) return __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, true);
    if constexpr (M == 4) {
        const uint32_t m = __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, true);
        return __builtin_amdgcn_update_dpp(0, m, 0x1B, 0xF, 0xF, true);
    }
    if constexpr (M == 8) return __builtin_amdgcn_update_dpp(0, v, 0x128, 0xF, 0xF, true);
    if constexpr (M == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);   // even rows twice, odd rows twice
        return threadIdx.x & 16 ? r[0] : r[1];
    }
    if constexpr (M == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return threadIdx.x & 32 ? r[0] : r[1];
    }
}
// The value of lane 63 - lane.
__device__ __forceinline__ uint32_t lane_flip(uint32_t v) {
    return lane_xor<32>(lane_xor<16>(__builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, true)));   // row_mirror
}
__device__ __forceinline__ float wave_max(float v) {
    auto step = [&](uint32_t o) { v = fmaxf(v, __uint_as_float(o)); };
    step(lane_xor<1>(__float_as_uint(v)));
    step(lane_xor<2>(__float_as_uint(v)));
    step(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x141, 0xF, 0xF, true));
    step(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x140, 0xF, 0xF, true));
    step(lane_xor<16>(__float_as_uint(v)));
    step(lane_xor<32>(__float_as_uint(v)));
    return v;
}
__device__ __forceinline__ uint32_t take(uint32_t v, int src) { return (uint32_t)__builtin_amdgcn_readlane((int)v, src); }

// max3: quiet NaN passed over; a signalling one comes out as NaN.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
__device__ __forceinline__ double wave_sum_f64(double v) {
    auto step = [&](auto move) {
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        v += __builtin_bit_cast(double, (uint64_t)move((uint32_t)(u >> 32)) << 32 | move((uint32_t)u));
    };
    step([](uint32_t w) { return lane_xor<1>(w); });
    step([](uint32_t w) { return lane_xor<2>(w); });
    step([](uint32_t w) { return lane_xor<4>(w); });
    step([](uint32_t w) { return lane_xor<8>(w); });
    step([](uint32_t w) { return lane_xor<16>(w); });
    step([](uint32_t w) { return lane_xor<32>(w); });
    return v;
}

// Entries of the lists. Strips: ordered logit bits over the complement of the index (larger is
// better; 0: none). Groups: score, then flat index. each() applies a lane move to every word.
struct StripKey {
    uint64_t v;
    template <typename F>
    __device__ __forceinline__ StripKey each(F f) const {
        return StripKey{(uint64_t)f((uint32_t)(v >> 32)) << 32 | f((uint32_t)v)};
    }
};
__device__ __forceinline__ bool better(const StripKey& a, const StripKey& b) { return a.v > b.v; }

struct BarKey {      // an ordered logit alone
    uint32_t v;
    template <typename F>
    __device__ __forceinline__ BarKey each(F f) const { return BarKey{f(v)}; }
};
__device__ __forceinline__ bool better(const BarKey& a, const BarKey& b) { return a.v > b.v; }

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

// One exchange over lanes J apart; lanes with a clear bit K of their number end with the better one
// in the lower lane.
template <int K, int J, typename T>
__device__ __forceinline__ void exchange(T& v, int lane) {
    const T o = v.each([](uint32_t w) { return lane_xor<J>(w); });
    const bool want = ((lane & J) == 0) == ((lane & K) == 0);
    if (want == better(o, v)) v = o;
}
// The wave's 64 entries sorted, best in lane 0 (bitonic).
template <int K, int J, typename T>
__device__ __forceinline__ void halve(T& v, int lane) {
    exchange<K, J>(v, lane);
    if constexpr (J > 1) halve<K, J / 2>(v, lane);
}
template <typename T>
__device__ __forceinline__ void sort64(T& v, int lane) {
    halve<2, 1>(v, lane);
    halve<4, 2>(v, lane);
    halve<8, 4>(v, lane);
    halve<16, 8>(v, lane);
    halve<32, 16>(v, lane);
    halve<64, 32>(v, lane);
}
// The 64 best of two sorted lists, sorted: the better of entry i and entry 63 - i of the other
// list are those 64, in an order that halves into place.
template <typename T>
__device__ __forceinline__ void merge64(T& list, const T& sorted, int lane) {
    const T o = sorted.each([](uint32_t w) { return lane_flip(w); });
    if (better(o, list)) list = o;
    halve<64, 32>(list, lane);
}

__device__ __forceinline__ uint32_t lanes_below(uint64_t mask) {
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// Float order as unsigned order (-0 counted as +0); and back.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}

constexpr int kPiece = 2048;        // logits a wave takes at a time, 32 per lane
constexpr int kStripWaves = 4;      // waves per workgroup, each on its own

// 16 bytes from an address aligned to the element only, in one load (the hardware takes it).
struct __attribute__((packed, aligned(2))) Loose16 { uint32_t w[4]; };

// One lane's 32 logits of the piece at element p0: vector u of E elements at p0 + (64 u + lane) E.
// The layout follows the element's index, not its address, so equal rows have equal sums wherever
// they lie (and scores that tie do so bit for bit).
template <bool F32>
struct Piece {
    static constexpr int E = F32 ? 4 : 8, NV = 32 / E;
    v4u raw[NV];
    __device__ __forceinline__ void load(const char* row, int64_t p0, int64_t vocab, int lane) {
        if (p0 + kPiece <= vocab) {                          // the same branch for the whole wave
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                const Loose16 v = *reinterpret_cast<const Loose16*>(row + (p0 + (u * 64 + lane) * E) * (F32 ? 4 : 2));
                raw[u] = v4u{v.w[0], v.w[1], v.w[2], v.w[3]};
            }
            return;
        }
#pragma unroll
        for (int u = 0; u < NV; ++u) {                       // the row's last piece: its own logits only, element by element
            const int64_t p = p0 + (u * 64 + lane) * E;
            constexpr uint32_t kNone = F32 ? 0xff800000u : 0xff80ff80u;    // -inf
            uint32_t w[4] = {kNone, kNone, kNone, kNone};
            if (p + E <= vocab) {
                const Loose16 v = *reinterpret_cast<const Loose16*>(row + p * (F32 ? 4 : 2));
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = v.w[j];
            } else if (p < vocab) {
#pragma unroll
                for (int j = 0; j < E; ++j)
                    if (p + j < vocab) {
                        if constexpr (F32) w[j] = *reinterpret_cast<const uint32_t*>(row + (p + j) * 4);
                        else {
                            const uint32_t h = *reinterpret_cast<const uint16_t*>(row + (p + j) * 2);
                            w[j >> 1] = j & 1 ? (w[j >> 1] & 0xffffu) | h << 16 : (w[j >> 1] & 0xffff0000u) | h;
                        }
                    }
            }
            raw[u] = v4u{w[0], w[1], w[2], w[3]};
        }
    }
    __device__ __forceinline__ float get(int i) const {   // i a constant: element i % E of vector i / E
        const int j = i % E;
        if constexpr (F32) return __uint_as_float(raw[i / E][j]);
        else return __uint_as_float(j & 1 ? raw[i / E][j >> 1] & 0xffff0000u : raw[i / E][j >> 1] << 16);
    }
};

constexpr int kSpan = 8;            // pieces between two looks at the cells' maxima
constexpr int kCells = 8;           // cells a half-wave reads at once
constexpr float kLog2e = 1.44269504088896341f;

template <bool F32>
__global__ __launch_bounds__(kStripWaves * 64, F32 ? 3 : 4) void beam_strip_kernel(const BeamArgs g) {
    __shared__ StripKey s_new[kStripWaves][64 * (kCells + 1)];
    __shared__ float s_max[kStripWaves][kSpan * 64];         // the cells' maxima
    __shared__ uint16_t s_cell[kStripWaves][kSpan * 64];     // the cells to read again
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t id = (int64_t)blockIdx.x * kStripWaves + wave;
    const int64_t row = id / g.n_strips;
    const int strip = (int)(id - row * g.n_strips);
    if (row >= g.n_groups * g.n_beams) return;
    if (g.finished && g.finished[row] != 0) return;          // its logits are not used
    constexpr int kSize = F32 ? 4 : 2, E = Piece<F32>::E;
    const char* const base = (F32 ? reinterpret_cast<const char*>(g.logits_f32)
                                  : reinterpret_cast<const char*>(g.logits_bf16)) + row * g.ld * kSize;

    StripKey list{0};               // lane i: the strip's i-th best so far
    float last = -INFINITY;         // what a logit has to beat: a bar that n_cand logits reach (-inf: none
    uint32_t last_at = 0xffffffffu; // yet), and the index below which an equal one still does
    int pending = 0;                // entries waiting in LDS
    StripKey* const buf = s_new[wave];
    float* const cmax = s_max[wave];
    uint16_t* const cells = s_cell[wave];
    float top = -INFINITY;          // this lane's largest logit and sum of exp(x - top)
    double sum = 0.0;
    auto flush = [&](int n) {       // the last n (<= 64) waiting entries into the list
        wave_lds_order();
        pending -= n;
        StripKey k{lane < n ? buf[pending + lane].v : 0};
        wave_lds_order();
        sort64(k, lane);
        merge64(list, k, lane);
        const uint64_t t = (uint64_t)take((uint32_t)(list.v >> 32), g.n_cand - 1) << 32 | take((uint32_t)list.v, g.n_cand - 1);
        if (t != 0) {
            last = unordered((uint32_t)(t >> 32));
            last_at = ~(uint32_t)t;
        }
    };

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

        BarKey k{span_max > -INFINITY ? ordered(span_max) : 0};
        sort64(k, lane);
        const uint32_t t = take(k.v, g.n_cand - 1);
        if (t != 0 && unordered(t) > last) {     // as many lanes' maxima reach it; equal ones still enter
            last = unordered(t);
            last_at = 0xffffffffu;
        }
        const float bar = fmaxf(last, -3.402823466e38f);     // -inf never enters
        wave_lds_order();
        int n_cells = 0;
        for (int q = 0; q < pieces; ++q) {
            const bool in = cmax[q * 64 + lane] >= bar;
            const uint64_t m = __ballot(in);
            if (in) cells[n_cells + lanes_below(m)] = (uint16_t)(q * 64 + lane);
            n_cells += __popcll(m);
        }
        wave_lds_order();
        for (int c0 = 0; c0 < n_cells; c0 += 2 * kCells) {
            float v[kCells];
            uint32_t idx[kCells];
#pragma unroll
            for (int s = 0; s < kCells; ++s) {
                const int c = c0 + 2 * s + (lane >> 5);
                v[s] = -INFINITY;
                idx[s] = 0;
                if (c < n_cells) {
                    const int cell = cells[c], i = lane & 31;
                    const int64_t at0 = span + (int64_t)(cell >> 6) * kPiece + (cell & 63) * E;     // its first logit
                    const int64_t at = at0 + (i / E) * 64 * E + i % E;
                    const float cm = cmax[cell];
                    // a cell that no longer reaches the list is not read
                    if ((cm > last || (cm == last && (uint32_t)at0 < last_at)) && at < p_end) {
                        v[s] = F32 ? *reinterpret_cast<const float*>(base + at * 4)
                                   : bf16_to_f32(*reinterpret_cast<const uint16_t*>(base + at * 2));
                        idx[s] = (uint32_t)at;
                    }
                }
            }
#pragma unroll
            for (int s = 0; s < kCells; ++s) {
                const float x = clean_logit(v[s]);
                const bool in = x > -INFINITY && (x > last || (x == last && idx[s] < last_at));
                const uint64_t m = __ballot(in);
                if (in) buf[pending + lanes_below(m)].v = (uint64_t)ordered(x) << 32 | (uint32_t)~idx[s];
                pending += __popcll(m);
            }
            while (pending >= 64) flush(64);
        }
        if (pending > 0) flush(pending);
        wave_lds_order();
    }
    const float all_top = wave_max(top);
    sum = wave_sum_f64(top == all_top ? sum : sum * (double)__expf(top - all_top));
    if (lane < g.n_cand) g.strip_keys[id * g.n_cand + lane] = list.v;
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
