// The adapters' part of a projection's epilogue: t B_e^T added to a wave's f32 result tiles.
//
// The tiles' lanes hold one token (row) each, in every MFMA layout used here: the weight rows are
// the A operand, the tokens the B operand's columns. So each lane keeps the product only where its own
// token has the adapter at hand, and the tile is taken once per adapter among its tokens (once in
// a batch of long runs). Selecting lanes instead of zeroing t keeps other adapters' infinities and
// NaN out of a token's row. The second operand is t in two or three bf16 parts, whose products
// with bf16 B are exact and summed in f32.
#pragma once

#include "nhm_device.h"
#include "nhm_internal.h"

namespace nhm {

// The adapter of row i, -1 for none.
__device__ __forceinline__ int lora_row(const LoraEpi& e, int64_t i, int64_t m) {
    const int a = i < m ? e.row_adapter[i] : -1;
    return a < e.n_adapters ? a : -1;
}

// 16 bytes (8 ranks) at a byte offset of a uniform base, zeros where !on.
__device__ __forceinline__ bf16x8 lora_load(const char* base, uint32_t off, bool on) {
    v4u v = {0u, 0u, 0u, 0u};
    if (on) v = *reinterpret_cast<const v4u*>(base + off);
    return __builtin_bit_cast(bf16x8, v);
}
// Adapter cur's features from n0 on (uniform): feature n0 + i at byte lora_b_off(e, i, n0, n), the last
// feature of the weight standing in for those past it (they are not stored).
__device__ __forceinline__ const char* lora_b_base(const LoraEpi& e, int cur, int64_t n0, int64_t n) {
    return reinterpret_cast<const char*>(e.b + ((int64_t)cur * n + n0) * e.rank);
}
__device__ __forceinline__ uint32_t lora_b_off(const LoraEpi& e, int i, int64_t n0, int64_t n) {
    const int64_t last = n - 1 - n0;       // negative for a tile part past the weight: one feature back and further
    return (uint32_t)((i < last ? i : last) * e.rank * 2);
}

// Runs f(cur) once for each distinct adapter among N ids per lane (negative: none), in order of
// first appearance. cur is uniform over the wave.
template <int N, typename F>
__device__ __forceinline__ void lora_each(const int (&id)[N], F f) {
    uint64_t todo[N];
#pragma unroll
    for (int j = 0; j < N; ++j) todo[j] = __ballot(id[j] >= 0);
    for (;;) {
        int cur = -1;
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (cur < 0 && todo[j]) cur = __builtin_amdgcn_readlane(id[j], __builtin_ctzll(todo[j]));
        if (cur < 0) break;
#pragma unroll
        for (int j = 0; j < N; ++j) todo[j] &= ~__ballot(id[j] == cur);
        f(cur);
    }
}

// 16 x 16 tiles: acc[i][j] register r of lane l is feature n0 + 16 i + 4 (l / 16) + r of row
// m0 + 16 j + l % 16. Nothing happens where the tiles lie past the weight or the rows.
template <int TN, int TM>
__device__ __forceinline__ void lora_add16(v4f (&acc)[TN][TM], const LoraEpi& e, int64_t m0, int64_t m, int64_t n0,
                                           int64_t n, int lane) {
    if (n0 >= n || m0 >= m) return;
    const int r16 = lane & 15, q8 = 8 * (lane >> 4);
    const char* const tb = reinterpret_cast<const char*>(e.t + m0 * e.parts * e.rp);
    const uint32_t tpart = (uint32_t)e.rp * 2;
    int id[TM];
    uint32_t toff[TM], boff[TN];
#pragma unroll
    for (int j = 0; j < TM; ++j) {
        const int64_t row = m0 + 16 * j + r16;
        id[j] = lora_row(e, row, m);
        toff[j] = (uint32_t)((row < m ? row : m - 1) - m0) * e.parts * tpart + q8 * 2;
    }
#pragma unroll
    for (int i = 0; i < TN; ++i) boff[i] = lora_b_off(e, 16 * i + r16, n0, n) + q8 * 2;
    lora_each(id, [&](int cur) {
        const char* const bb = lora_b_base(e, cur, n0, n);
        v4f x[TN][TM];
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j) x[i][j] = acc[i][j];
        for (int s = 0; s < e.rp; s += 32) {
            bf16x8 bf[TN];
#pragma unroll
            for (int i = 0; i < TN; ++i) bf[i] = lora_load(bb, boff[i] + s * 2, s + q8 < e.rank);
            for (int p = 0; p < e.parts; ++p) {
                bf16x8 tf[TM];
#pragma unroll
                for (int j = 0; j < TM; ++j) tf[j] = lora_load(tb, toff[j] + p * tpart + s * 2, true);
#pragma unroll
                for (int j = 0; j < TM; ++j)
#pragma unroll
                    for (int i = 0; i < TN; ++i) x[i][j] = mfma_bf16(bf[i], tf[j], x[i][j]);
            }
        }
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][j][r] = id[j] == cur ? x[i][j][r] : acc[i][j][r];
    });
}

}  // namespace nhm
