// The low-rank product of many requests' adapters, t = scale x A_e^T (nhm_fp8_linear_lora), and in the
// same pass over x the e4m3 codes the projection reads. The projection's own kernels add
// t B_e^T in their epilogues (lora_device.h).
//
// Matrix instructions with 16 ranks as the A operand and 16 rows of x as the B operand. A
// workgroup owns 16 kRows rows and 16 kRanks ranks over all of k, kWaves / kRows waves to each 16
// rows, which take the 32-wide k-steps round robin, several in flight; their sums meet in LDS
// in wave order. Rows in a tile may have any adapters: the tile is taken once per distinct
// adapter, and each time only its rows are stored, so another adapter's values reach nobody
// else. What it must read is x and the used adapters' A; in decode both are small and latency
// bounds it, in a long prefill x's bytes do.
#include "nhm_device.h"
#include "nhm_internal.h"

namespace nhm {

// Eight values of x at p: bf16 as they are, e4m3 codes converted (exact).
__device__ __forceinline__ bf16x8 x8(const uint16_t* p) { return __builtin_bit_cast(bf16x8, *reinterpret_cast<const v4u*>(p)); }
__device__ __forceinline__ bf16x8 x8(const uint8_t* p) {
    const uint2 c = *reinterpret_cast<const uint2*>(p);
    return e4m3x8_to_bf16(c.x, c.y);
}

// The codes of eight bf16 values, as nhm_fp8_quantize_static forms them.
__device__ __forceinline__ void store_codes(uint8_t* q, const bf16x8& v, float s, float rs, bool fast) {
    const v4u u = __builtin_bit_cast(v4u, v);
    const uint4 in = make_uint4(u[0], u[1], u[2], u[3]);
    uint2 c;
    if (fast && __builtin_amdgcn_ballot_w64(bf16x8_special(in) != 0u) == 0) c = quant_bf16x8_fast(in, s, rs);
    else c = quant_bf16x8(in, s);
    *reinterpret_cast<uint2*>(q) = c;
}

constexpr int kUnroll = 4;   // k-steps whose loads are in flight together

// X: uint16_t (bf16) or uint8_t (codes). gridDim: (row tiles, rank groups, shares of the distinct
// adapters of a tile).
template <typename X, int kWaves, int kRows, int kRanks>
__global__ __launch_bounds__(kWaves * 64) void lora_down_kernel(const LoraDownArgs g) {
    constexpr int KW = kWaves / kRows;       // waves that share a row tile's k
    __shared__ v4f s_part[kRows][KW][kRanks][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rt = wave / KW, kw = wave % KW;
    const int r16 = lane & 15, q8 = 8 * (lane >> 4);
    const int64_t row = ((int64_t)blockIdx.x * kRows + rt) * 16 + r16;
    const int64_t src = row < g.m ? row : g.m - 1;
    const X* const xr = (sizeof(X) == 2 ? reinterpret_cast<const X*>(g.x) : reinterpret_cast<const X*>(g.x_codes)) + src * g.ld_x;
    const int rank0 = blockIdx.y * 16 * kRanks;
    int id = row < g.m ? g.row_adapter[row] : -1;
    if (id >= g.n_adapters) id = -1;
    const int steps = (int)((g.k + 31) / 32);
    const bool quant = sizeof(X) == 2 && g.q && blockIdx.y == 0 && blockIdx.z == 0;
    const float s = *g.a_scale;
    const bool fast = fast_scale(s);
    const float rs = quant ? __fdiv_rn(1.0f, s) : 0.f;

    // One pass over this wave's steps: the codes if asked, and the products with adapter cur (>= 0).
    v4f acc[kRanks];
    auto pass = [&](int cur, bool codes) {
#pragma unroll
        for (int j = 0; j < kRanks; ++j) acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
        const uint16_t* ar[kRanks];
#pragma unroll
        for (int j = 0; j < kRanks; ++j) {
            const int r = rank0 + 16 * j + r16;
            ar[j] = g.a + ((int64_t)(cur < 0 ? 0 : cur) * g.rank + (r < g.rank ? r : g.rank - 1)) * g.k;
        }
        for (int s0 = kw; s0 < steps; s0 += KW * kUnroll) {
            bf16x8 xv[kUnroll], av[kUnroll][kRanks];
            bool in[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int64_t kk = (int64_t)(s0 + u * KW) * 32 + q8;
                in[u] = kk < g.k;                               // steps past k read the row's start and count as zeros
                xv[u] = x8(xr + (in[u] ? kk : 0));
                if (cur >= 0) {
#pragma unroll
                    for (int j = 0; j < kRanks; ++j) av[u][j] = x8(ar[j] + (in[u] ? kk : 0));
                }
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (codes && in[u] && row < g.m) store_codes(g.q + row * g.k + (int64_t)(s0 + u * KW) * 32 + q8, xv[u], s, rs, fast);
                if (cur >= 0) {
                    const bf16x8 zero = __builtin_bit_cast(bf16x8, v4u{0u, 0u, 0u, 0u});
                    const bf16x8 xz = in[u] ? xv[u] : zero;
#pragma unroll
                    for (int j = 0; j < kRanks; ++j) acc[j] = mfma_bf16(in[u] ? av[u][j] : zero, xz, acc[j]);
                }
            }
        }
    };

    // The distinct adapters among the workgroup's rows: every wave of a row tile sees the same ones,
    // waves of other row tiles go through empty turns so that the barriers match.
    __shared__ int s_turns[kRows];
    uint64_t todo = __ballot(id >= 0) & 0xffffu;
    int turns = 0;
    for (uint64_t left = todo; left; ++turns) {
        const int cur = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        left &= ~__ballot(id == cur);
    }
    int most = turns;
    if constexpr (kRows > 1) {
        if (lane == 0 && kw == 0) s_turns[rt] = turns;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRows; ++i) most = max(most, s_turns[i]);
    }
    bool codes = quant;
    for (int turn = 0; turn < most; ++turn) {
        int cur = -1;
        if (todo) {
            cur = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
            todo &= ~__ballot(id == cur);
        }
        if (turn % gridDim.z != blockIdx.z) continue;
        if (cur >= 0 || codes) pass(cur, codes);
        codes = false;
#pragma unroll
        for (int j = 0; j < kRanks; ++j) s_part[rt][kw][j][lane] = acc[j];
        __syncthreads();
        // this row tile's waves finish its rank tiles in turn
        for (int j = kw; j < kRanks && cur >= 0; j += KW) {
            v4f d = s_part[rt][0][j][lane];
#pragma unroll
            for (int w = 1; w < KW; ++w) d += s_part[rt][w][j][lane];
            const int r0 = rank0 + 16 * j + 4 * (lane >> 4);         // d[r] is rank r0 + r of the row
            if (id != cur || r0 >= g.rp) continue;
            const float sc = (g.scale ? g.scale[cur] : 1.0f) * (sizeof(X) == 1 ? s : 1.0f);
            float v[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = r0 + r < g.rank ? d[r] * sc : 0.f;
            for (int p = 0; p < g.parts; ++p) {
                const uint32_t lo = f32x2_to_bf16x2(v[0], v[1]), hi = f32x2_to_bf16x2(v[2], v[3]);
                *reinterpret_cast<uint2*>(g.t + (row * g.parts + p) * g.rp + r0) = make_uint2(lo, hi);
                const uint32_t h[4] = {lo & 0xffffu, lo >> 16, hi & 0xffffu, hi >> 16};
#pragma unroll
                for (int r = 0; r < 4; ++r)      // what this part leaves (nothing of an infinity or NaN)
                    v[r] = (h[r] & 0x7f80u) == 0x7f80u ? 0.f : v[r] - bf16_to_f32(h[r]);
            }
        }
        __syncthreads();
    }
    if (codes && (blockIdx.z == 0)) pass(-1, true);      // no row here has an adapter
}

template <typename X>
static void launch_down(const LoraDownArgs& g, hipStream_t st) {
    const int64_t tiles = (g.m + 15) / 16;
    const unsigned groups = (unsigned)(g.rp / 16);
    if (tiles >= 512) {
        lora_down_kernel<X, 8, 4, 4><<<dim3((unsigned)((tiles + 3) / 4), (groups + 3) / 4), dim3(512), 0, st>>>(g);
        return;
    }
    int64_t z = 1024 / (tiles * groups);
    z = z < 1 ? 1 : z > 16 ? 16 : z;
    lora_down_kernel<X, 16, 1, 1><<<dim3((unsigned)tiles, groups, (unsigned)z), dim3(1024), 0, st>>>(g);
}

nhm_status launch_lora_down(const LoraDownArgs& g, hipStream_t st) {
    if (g.x) launch_down<uint16_t>(g, st);
    else launch_down<uint8_t>(g, st);
    count_launch(Kern::kLoraDown, g.m);
    return check_launch("lora down");
}

}  // namespace nhm
