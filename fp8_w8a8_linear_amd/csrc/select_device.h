// Sorted lists over a wave's lanes and the walk over a row of logits: what the beam selection and the
// scoring of tokens share.
#pragma once

#include <math.h>

#include "nhm_device.h"

namespace nhm {

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

// max3: quiet NaN passed over; a signalling one comes out as a quiet one, which the next max3 passes over together with
// what was in front of it, so that a chain of them does not show it.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
// maximum3: NaN where any of the three is one, quiet or signalling, so that a chain of them ends as NaN.
__device__ __forceinline__ float maximum3(float a, float b, float c) {
    float r;
    asm("v_maximum3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
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
// better; 0: none). each() applies a lane move to every word.
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

struct StripLds {                       // a wave's own
    StripKey fresh[64 * (kCells + 1)];  // entries waiting for the list
    float max[kSpan * 64];              // the cells' maxima
    uint16_t cell[kSpan * 64];          // the cells to read again
};

// The n largest logits of the strip a wave walks (n <= 64), found from the cells' maxima of a span.
template <bool F32>
struct StripBest {
    StripLds* lds;
    int n;
    StripKey list{0};               // lane i: the strip's i-th best so far
    float last = -INFINITY;         // what a logit has to beat: a bar that n logits reach (-inf: none
    uint32_t last_at = 0xffffffffu; // yet), and the index below which an equal one still does
    int pending = 0;                // entries waiting in LDS

    __device__ __forceinline__ void flush(int count, int lane) {   // the last count (<= 64) waiting entries into the list
        wave_lds_order();
        pending -= count;
        StripKey k{lane < count ? lds->fresh[pending + lane].v : 0};
        wave_lds_order();
        sort64(k, lane);
        if (__ballot(list.v != 0) == 0) list = k;     // the first ones
        else merge64(list, k, lane);
        const uint64_t t = (uint64_t)take((uint32_t)(list.v >> 32), n - 1) << 32 | take((uint32_t)list.v, n - 1);
        if (t != 0) {
            last = unordered((uint32_t)(t >> 32));
            last_at = ~(uint32_t)t;
        }
    }

    // The span of `pieces` pieces from element `span` on (of a strip that ends at p_end), whose cells' maxima are in
    // lds->max; span_max: the largest of this lane's.
    __device__ __forceinline__ void look(const char* base, int64_t span, int pieces, int64_t p_end, float span_max, int lane) {
        constexpr int E = Piece<F32>::E;
        StripKey* const buf = lds->fresh;
        float* const cmax = lds->max;
        uint16_t* const cells = lds->cell;
        BarKey k{span_max > -INFINITY ? ordered(span_max) : 0};
        sort64(k, lane);
        const uint32_t t = take(k.v, n - 1);
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
            while (pending >= 64) flush(64, lane);
        }
        if (pending > 0) flush(pending, lane);
        wave_lds_order();
    }
};

}  // namespace nhm
