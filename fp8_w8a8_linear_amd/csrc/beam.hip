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
// from the strips' lists. The pass is bound by the logits' bytes; 512 rows of 131,072 bf16 logits.
//
// A wave's list is sorted, one entry per lane. A logit enters it only if it beats the list's last
// used entry, so after the first piece of a strip almost every piece is dismissed by one
// comparison of each lane's maximum; the others collect in LDS until 64 of them (or the strip's
// end) are sorted and merged in. Before the first piece the n_cand-th largest of the 64 lane maxima
// stands in for that entry: at least n_cand logits of the piece reach it.
// Any number of entering logits is handled (ascending rows merge all the time): only speed depends
// on the data.

// x as the selection reads it: NaN counts as -inf.
__device__ __forceinline__ float clean_logit(float x) { return x == x ? x : -INFINITY; }

template <typename K>
__device__ __forceinline__ K lane_xor(const K& v, int mask);
template <typename K>
__device__ __forceinline__ K lane_get(const K& v, int src);

// Entries of the lists. Strips: ordered logit bits over the complement of the index (larger is
// better; 0: none). Groups: score, then flat index.
typedef uint64_t StripKey;
template <>
__device__ __forceinline__ StripKey lane_xor(const StripKey& v, int mask) {
    return (uint64_t)(uint32_t)__shfl_xor((int)(v >> 32), mask) << 32 | (uint32_t)__shfl_xor((int)(uint32_t)v, mask);
}
template <>
__device__ __forceinline__ StripKey lane_get(const StripKey& v, int src) {
    return (uint64_t)(uint32_t)__shfl((int)(v >> 32), src) << 32 | (uint32_t)__shfl((int)(uint32_t)v, src);
}
__device__ __forceinline__ bool better(const StripKey& a, const StripKey& b) { return a > b; }

struct GroupKey { double score; uint32_t flat; };
template <>
__device__ __forceinline__ GroupKey lane_xor(const GroupKey& v, int mask) {
    return GroupKey{__shfl_xor(v.score, mask), (uint32_t)__shfl_xor((int)v.flat, mask)};
}
template <>
__device__ __forceinline__ GroupKey lane_get(const GroupKey& v, int src) {
    return GroupKey{__shfl(v.score, src), (uint32_t)__shfl((int)v.flat, src)};
}
__device__ __forceinline__ bool better(const GroupKey& a, const GroupKey& b) {
    return a.score > b.score || (a.score == b.score && a.flat < b.flat);
}

// The wave's 64 entries sorted, best in lane 0 (bitonic).
template <typename K>
__device__ __forceinline__ void sort64(K& v, int lane) {
#pragma unroll
    for (int k = 2; k <= 64; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j > 0; j >>= 1) {
            const K o = lane_xor(v, j);
            const bool want = ((lane & j) == 0) == ((lane & k) == 0);   // this lane keeps the better one
            if (want == better(o, v)) v = o;
        }
}
// The 64 best of two sorted lists, sorted: the better of entry i and entry 63 - i of the other
// list are those 64, in an order that halves into place.
template <typename K>
__device__ __forceinline__ void merge64(K& list, const K& sorted, int lane) {
    const K o = lane_get(sorted, 63 - lane);
    if (better(o, list)) list = o;
#pragma unroll
    for (int j = 32; j > 0; j >>= 1) {
        const K p = lane_xor(list, j);
        if (((lane & j) == 0) == better(p, list)) list = p;
    }
}

// Between a wave's LDS writes and its reads of other lanes' entries: LDS serves a wave's accesses
// in order, this keeps the compiler from moving them past each other.
__device__ __forceinline__ void wave_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
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
    uint4 raw[NV];
    __device__ __forceinline__ void load(const char* row, int64_t p0, int64_t vocab, int lane) {
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int64_t p = p0 + (u * 64 + lane) * E;
            constexpr uint32_t kNone = F32 ? 0xff800000u : 0xff80ff80u;    // -inf
            uint32_t w[4] = {kNone, kNone, kNone, kNone};
            if (p + E <= vocab) {
                const Loose16 v = *reinterpret_cast<const Loose16*>(row + p * (F32 ? 4 : 2));
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = v.w[j];
            } else if (p < vocab) {                      // the row's last vector: its own elements only
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
            raw[u] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    __device__ __forceinline__ float get(int i) const {   // i a constant: element i % E of vector i / E
        const uint4 v = raw[i / E];
        const int j = i % E;
        const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
        if constexpr (F32) return clean_logit(__uint_as_float(w4[j]));
        else return clean_logit(bf16_to_f32(j & 1 ? w4[j >> 1] >> 16 : w4[j >> 1] & 0xffffu));
    }
};

template <bool F32>
__global__ __launch_bounds__(kStripWaves * 64) void beam_strip_kernel(const BeamArgs g) {
    __shared__ StripKey s_new[kStripWaves][128];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t id = (int64_t)blockIdx.x * kStripWaves + wave;
    const int64_t row = id / g.n_strips;
    const int strip = (int)(id - row * g.n_strips);
    if (row >= g.n_groups * g.n_beams) return;
    if (g.finished && g.finished[row] != 0) return;          // its logits are not used
    constexpr int kSize = F32 ? 4 : 2, E = Piece<F32>::E;
    const char* const base = (F32 ? reinterpret_cast<const char*>(g.logits_f32)
                                  : reinterpret_cast<const char*>(g.logits_bf16)) + row * g.ld * kSize;

    StripKey list = 0;              // lane i: the strip's i-th best so far
    float last = -INFINITY;         // the n_cand-th best's logit and index (none yet)
    uint32_t last_at = 0;
    int pending = 0;                // entries waiting in LDS
    StripKey* const buf = s_new[wave];
    float top = -INFINITY;
    double sum = 0.0;               // this lane's sum of exp(x - top)
    auto flush = [&](int n) {       // the first n (<= 64) waiting entries into the list
        wave_lds_order();
        StripKey k = lane < n ? buf[lane] : 0;
        sort64(k, lane);
        merge64(list, k, lane);
        const StripKey t = lane_get(list, g.n_cand - 1);
        if (t != 0) {
            last = unordered((uint32_t)(t >> 32));
            last_at = ~(uint32_t)t;
        }
    };

    const int64_t p_beg = (int64_t)strip * g.strip_pieces * kPiece;
    const int64_t p_end = min(p_beg + (int64_t)g.strip_pieces * kPiece, g.vocab);
    Piece<F32> cur, nxt;
    cur.load(base, p_beg, g.vocab, lane);
    for (int64_t p = p_beg; p < p_end; p += kPiece) {
        if (p + kPiece < p_end) nxt.load(base, p + kPiece, g.vocab, lane);
        float x[32], mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            x[i] = cur.get(i);
            mx = fmaxf(mx, x[i]);
        }
        float piece_top = mx;
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) piece_top = fmaxf(piece_top, __shfl_xor(piece_top, d));
        if (piece_top > -INFINITY) {
            if (piece_top > top) {
                sum *= (double)__expf(top - piece_top);      // 0 from -inf
                top = piece_top;
            }
            float part = 0.f;        // 32 terms in f32, the strip's sum in f64
            if (top < INFINITY) {
#pragma unroll
                for (int i = 0; i < 32; ++i) part += __builtin_amdgcn_exp2f((x[i] - top) * 1.44269504088896341f);
            } else {                 // +inf entries share the probability
#pragma unroll
                for (int i = 0; i < 32; ++i) part += x[i] == INFINITY ? 1.0f : 0.0f;
            }
            sum += (double)part;

            float least = last;      // entries below it cannot be among the n_cand best
            if (last == -INFINITY) {
                StripKey k = mx > -INFINITY ? (uint64_t)ordered(mx) << 32 : 0;
                sort64(k, lane);
                k = lane_get(k, g.n_cand - 1);
                if (k != 0) least = unordered((uint32_t)(k >> 32));
            }
            if (__ballot(mx >= least && mx > -INFINITY)) {
                uint32_t hits = 0;
#pragma unroll
                for (int i = 0; i < 32; ++i) hits |= (x[i] >= least && x[i] > -INFINITY ? 1u : 0u) << i;
                while (__ballot(hits != 0)) {
                    // each lane's next one, read again (an index into registers would have to be a constant)
                    bool in = hits != 0;
                    StripKey k = 0;
                    if (in) {
                        const int i = __ffs((int)hits) - 1;
                        hits &= hits - 1;
                        const int64_t pos = p + ((i / E) * 64 + lane) * E + i % E;
                        const char* at = base + pos * kSize;
                        const float v = clean_logit(F32 ? *reinterpret_cast<const float*>(at)
                                                        : bf16_to_f32(*reinterpret_cast<const uint16_t*>(at)));
                        const uint32_t idx = (uint32_t)pos;
                        in = v > last || (v == last && idx < last_at);
                        k = (uint64_t)ordered(v) << 32 | (uint32_t)~idx;
                    }
                    const uint64_t m = __ballot(in);
                    if (in) buf[pending + lanes_below(m)] = k;
                    pending += __popcll(m);
                    if (pending >= 64) {
                        flush(64);
                        pending -= 64;
                        if (lane < pending) buf[lane] = buf[64 + lane];
                        wave_lds_order();
                    }
                }
            }
        }
        cur = nxt;
    }
    if (pending > 0) flush(pending);
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
    if (lane < g.n_cand) g.strip_keys[id * g.n_cand + lane] = list;
    if (lane == 0) {
        g.strip_top[id] = top;
        g.strip_sum[id] = sum;
    }
}

// One workgroup per group: each row's lse from its strips, then the best continuations. The strips'
// lists are sorted, so they are walked by place: first every strip's best, then every strip's
// second best, until at some place none of them beats the list's last used entry.
constexpr int kPickWaves = 4;

__global__ __launch_bounds__(kPickWaves * 64) void beam_pick_kernel(const BeamArgs g) {
    __shared__ double s_lse[32];                    // each beam's log(sum exp(x - top)) (finished: not used)
    __shared__ float s_top[32];
    __shared__ GroupKey s_new[kPickWaves][128];
    __shared__ GroupKey s_list[kPickWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row0 = (int64_t)blockIdx.x * g.n_beams;
    const int S = g.n_strips, K = g.n_beams;
    for (int b = wave; b < K; b += kPickWaves) {
        if (g.finished && g.finished[row0 + b] != 0) continue;
        const int64_t id0 = (row0 + b) * S;
        float top = -INFINITY;
        for (int s = lane; s < S; s += 64) top = fmaxf(top, g.strip_top[id0 + s]);
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
        double sum = 0.0;
        for (int s = lane; s < S; s += 64) {
            const float t = g.strip_top[id0 + s];
            if (t > -INFINITY) sum += g.strip_sum[id0 + s] * (t == top ? 1.0 : exp((double)t - (double)top));
        }
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
        if (lane == 0) {
            s_top[b] = top;
            s_lse[b] = log(sum);
        }
    }
    __syncthreads();

    GroupKey list{-INFINITY, 0xffffffffu};
    GroupKey last{-INFINITY, 0xffffffffu};
    int pending = 0;
    GroupKey* const buf = s_new[wave];
    auto flush = [&](int n) {
        wave_lds_order();
        GroupKey k = lane < n ? buf[lane] : GroupKey{-INFINITY, 0xffffffffu};
        sort64(k, lane);
        merge64(list, k, lane);
        last = lane_get(list, g.n_cand - 1);
    };
    const int all = K * S;
    for (int place = 0; place < g.n_cand; ++place) {
        bool any = false;
        for (int i0 = wave * 64; i0 < all; i0 += kPickWaves * 64) {
            const int i = i0 + lane;
            GroupKey k{-INFINITY, 0xffffffffu};
            if (i < all) {
                const int b = i / S, s = i - b * S;
                if (g.finished && g.finished[row0 + b] != 0) {
                    if (s == 0 && place == 0) k = GroupKey{(double)g.cum[row0 + b], (uint32_t)(b * g.vocab + g.eos)};
                } else {
                    const StripKey e = g.strip_keys[((row0 + b) * S + s) * g.n_cand + place];
                    if (e != 0) {
                        // x - top first: +inf entries score cum - log(their number). cum + (x - top) is
                        // exact in f64 for f32 values within 29 bits of each other, so equal rows
                        // whose scores tie do so bit for bit, whatever lse's last bits are
                        const float x = unordered((uint32_t)(e >> 32)), top = s_top[b];
                        const double d = x == top ? 0.0 : (double)x - (double)top;
                        k = GroupKey{((double)g.cum[row0 + b] + d) - s_lse[b], (uint32_t)(b * g.vocab + (uint32_t)~(uint32_t)e)};
                    }
                }
            }
            const bool in = k.score > -INFINITY && better(k, last);
            const uint64_t m = __ballot(in);
            if (m == 0) continue;
            any = true;
            if (in) buf[pending + lanes_below(m)] = k;
            pending += __popcll(m);
            if (pending >= 64) {
                flush(64);
                pending -= 64;
                if (lane < pending) buf[lane] = buf[64 + lane];
                wave_lds_order();
            }
        }
        if (!any) break;
        if (pending > 0) {
            flush(pending);
            pending = 0;
        }
    }
    s_list[wave][lane] = list;
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int w = 1; w < kPickWaves; ++w) merge64(list, s_list[w][lane], lane);
    if (lane < g.n_cand) {
        const int64_t o = (int64_t)blockIdx.x * g.n_cand + lane;
        const bool none = list.flat == 0xffffffffu;
        g.scores[o] = (float)list.score;
        g.parents[o] = none ? -1 : (int32_t)(list.flat / (uint32_t)g.vocab);
        g.tokens[o] = none ? -1 : (int32_t)(list.flat % (uint32_t)g.vocab);
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
    w.sum = align_up(n * n_cand * sizeof(StripKey), 256);
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
    beam_pick_kernel<<<dim3((unsigned)g.n_groups), dim3(kPickWaves * 64), 0, st>>>(g);
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
