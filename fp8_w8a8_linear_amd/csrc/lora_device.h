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
// Adapter cur's features from n0 < n on (uniform): feature n0 + i at byte lora_b_off(e, i, n0, n), the last
// feature of the weight standing in for those past it (they are not stored).
__device__ __forceinline__ const char* lora_b_base(const LoraEpi& e, int cur, int64_t n0, int64_t n) {
    return reinterpret_cast<const char*>(e.b + ((int64_t)cur * n + n0) * e.rank);
}
__device__ __forceinline__ uint32_t lora_b_off(const LoraEpi& e, int i, int64_t n0, int64_t n) {
    const int64_t last = n - 1 - n0;
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

}  // namespace nhm
