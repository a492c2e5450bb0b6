// The low-rank product of many requests' adapters, t = scale x A_e^T (nhm_fp8_linear_lora), and in the
// same pass over x the e4m3 codes the projection reads. The projection's own kernels add
// t B_e^T in their epilogues (lora_device.h).
//
// Matrix instructions with 16 ranks as the A operand and 16 rows of x as the B operand. Rows in a
// tile may have any adapters: the tile is taken once per distinct adapter, and each time only its rows
// are stored, so another adapter's values reach nobody else. What it must read is x and the used
// adapters' A, and with a bf16 x it writes the codes.
//  * Few rows: latency and the bytes a CU is handed bound it. A workgroup owns 16 rows and 4 to 16 ranks over all of
//    k, 16 waves that take the 64-wide k-steps round robin with all their loads in flight (up to k = 4,096 one
//    round), and a share of the tile's distinct adapters, of whose rows alone it reads x.
//  * Many rows (8,192 or more fill half of the chip): latency bounds it, 135 MB in 48 us (2.8 TB/s), as 131 KB of
//    LDS and 356 registers leave one workgroup, a wave per SIMD, to a CU. A workgroup owns 64 rows and up to 64 ranks,
//    4 waves that each take whole 64 x 64 k-steps, so that x and A enter the CU once, the next
//    step's operands on their way while one is multiplied. Loads take whole lines, which turn into operands in
//    a wave-private piece of LDS (with the few rows' deal instead 60 us for 48).
// The waves' sums meet in LDS and are added in wave order. With few rows a lane's share of a 64-wide k-step is
// 16 consecutive values (two matrix instructions' worth; any deal of k to lanes will do that is the same
// for both operands), so that the first of its two loads asks for whole 128-byte lines.
// k = 2,688, codes formed: one row of rank 16 4.1 us (an empty launch 2.6), 8 rows with an adapter each of rank 64
// 5.3, 477 rows of rank 24 8.4, 15,360 rows of rank 64 48.
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
__device__ __forceinline__ uint2 codes8(const bf16x8& v, float s, float rs, bool fast) {
    const v4u u = __builtin_bit_cast(v4u, v);
    const uint4 in = make_uint4(u[0], u[1], u[2], u[3]);
    if (fast && __builtin_amdgcn_ballot_w64(bf16x8_special(in) != 0u) == 0) return quant_bf16x8_fast(in, s, rs);
    return quant_bf16x8(in, s);
}

// Ranks r0 .. r0 + 3 of a row (d, unscaled) into its parts.
__device__ __forceinline__ void store_parts(const LoraDownArgs& g, int64_t row, int r0, const v4f& d, float sc) {
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

// X: uint16_t (bf16) or uint8_t (codes).
template <typename X>
__device__ __forceinline__ const X* x_rows(const LoraDownArgs& g) {
    if constexpr (sizeof(X) == 2) return g.x;
    else return g.x_codes;
}

// ---------------------------------------------------------------- few rows

constexpr int kFewWaves = 16, kFewSteps = 4;   // k-steps of a wave whose loads are in flight together

// gridDim: (row tiles, rank groups, shares + extra): blockIdx.z < shares takes every shares-th
// distinct adapter of the tile; the workgroups past that form the tile's codes, one or a few vectors a
// thread (in the same workgroups as the products they made the code long and the launch slow: 9.2 us
// for 8 rows).
template <typename X>
__global__ __launch_bounds__(kFewWaves * 64) void lora_down_few_kernel(const LoraDownArgs g, int shares, int ranks) {
    __shared__ v4f s_part[kFewWaves][64];
    const int64_t tile0 = (int64_t)blockIdx.x * 16;
    if constexpr (sizeof(X) == 2) {
        if ((int)blockIdx.z >= shares) {
            const int per_row = (int)(g.k / 8);
            const int total = (int)min((int64_t)16, g.m - tile0) * per_row;
            const float s = *g.a_scale;
            const float rs = __fdiv_rn(1.0f, s);
            const bool fast = fast_scale(s);
            const int stride = (int)(gridDim.z - shares) * gridDim.y * kFewWaves * 64;
            for (int v = ((blockIdx.z - shares) * gridDim.y + blockIdx.y) * kFewWaves * 64 + threadIdx.x; v < total; v += stride) {
                const int64_t row = tile0 + v / per_row, c = (int64_t)(v % per_row) * 8;
                *reinterpret_cast<uint2*>(g.q + row * g.k + c) = codes8(x8(g.x + row * g.ld_x + c), s, rs, fast);
            }
            return;
        }
    }
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, q16 = 16 * (lane >> 4);
    const int64_t row = tile0 + r16;
    const int64_t src = row < g.m ? row : g.m - 1;
    int id = g.row_adapter[src];
    const X* const xr = x_rows<X>(g) + src * g.ld_x;
    const int steps = (int)((g.k + 63) / 64);
    const int r = blockIdx.y * ranks + r16;                      // this lane's rank of A
    const bool on = r16 < ranks && r < g.rank;
    const bf16x8 zero = __builtin_bit_cast(bf16x8, v4u{0u, 0u, 0u, 0u});
    if (row >= g.m || id >= g.n_adapters) id = -1;
    uint64_t todo = __ballot(id >= 0) & 0xffffu;
    for (int turn = 0; todo; ++turn) {
        const int cur = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
        todo &= ~__ballot(id == cur);
        if (turn % shares != (int)blockIdx.z) continue;
        // the scales through the scalar cache, and no branch that would wait for them
        typedef const __attribute__((address_space(4))) float* scalar_f32;
        const float s = *reinterpret_cast<scalar_f32>(reinterpret_cast<uintptr_t>(g.a_scale));
        const float se = *reinterpret_cast<scalar_f32>(reinterpret_cast<uintptr_t>(g.scale ? g.scale + cur : g.a_scale));
        v4f acc = {0.f, 0.f, 0.f, 0.f};
        const uint16_t* const ar = g.a + ((int64_t)cur * g.rank + r) * g.k;
        for (int s0 = wave; s0 < steps; s0 += kFewWaves * kFewSteps) {
            bf16x8 xv[kFewSteps][2], av[kFewSteps][2];
#pragma unroll
            for (int u = 0; u < kFewSteps; ++u) {
                const int kk = (s0 + u * kFewWaves) * 64 + q16;      // 16 divides k: all of a lane's 16 or none
#pragma unroll
                for (int h = 0; h < 2; ++h) xv[u][h] = av[u][h] = zero;
                if (kk < g.k && on) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) av[u][h] = x8(ar + kk + 8 * h);
                }
                if (kk < g.k && id == cur) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) xv[u][h] = x8(xr + kk + 8 * h);
                }
            }
#pragma unroll
            for (int u = 0; u < kFewSteps; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h) acc = mfma_bf16(av[u][h], xv[u][h], acc);
        }
        s_part[wave][lane] = acc;
        __syncthreads();
        if (wave == 0) {
            v4f d = s_part[0][lane];
#pragma unroll
            for (int w = 1; w < kFewWaves; ++w) d += s_part[w][lane];
            const float sc = (g.scale ? se : 1.0f) * (sizeof(X) == 1 ? s : 1.0f);
            const int r0 = 4 * (lane >> 4);
            if (id == cur && r0 < ranks) store_parts(g, row, blockIdx.y * ranks + r0, d, sc);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- many rows

constexpr int kManyWaves = 4, kManyRows = 4;   // row tiles of 16 per workgroup

// NR: 16-rank tiles per workgroup. gridDim: (64-row tiles, groups of 16 NR ranks).
template <typename X, int NR>
__global__ __launch_bounds__(kManyWaves * 64) void lora_down_many_kernel(const LoraDownArgs g) {
    __shared__ v4f s_part[kManyWaves][kManyRows * NR][64];
    __shared__ __attribute__((aligned(16))) uint8_t s_tr[kManyWaves][(kManyRows + NR) * 16 * 128];   // a wave's step
    constexpr bool kCodes = sizeof(X) == 1;        // x is given as codes
    constexpr int kXLoads = kCodes ? kManyRows : 2 * kManyRows;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, q = lane >> 4;
    const int64_t row0 = (int64_t)blockIdx.x * (16 * kManyRows);
    const int rank0 = blockIdx.y * 16 * NR;
    const float s = *g.a_scale;
    const bool fast = fast_scale(s);
    const float rs = __fdiv_rn(1.0f, s);
    int id[kManyRows];
#pragma unroll
    for (int i = 0; i < kManyRows; ++i) {
        const int64_t row = row0 + 16 * i + r16;
        id[i] = row < g.m ? g.row_adapter[row] : -1;
        if (id[i] >= g.n_adapters) id[i] = -1;
    }
    // A load of bf16 values takes whole 128-byte lines of 8 rows: lane l row l / 8 and the chunk of 8 values that
    // swz128 places at slot l % 8; one of codes 64 bytes of 16 rows: row l / 4 and 16 values.
    const int lr = lane >> 3, slot = lane & 7, cr = lane >> 2, cc = lane & 3;
    auto chunk = [&](int u) { return slot ^ lr ^ (u & 1); };       // of 8-row unit u
    const X* xr[kXLoads];
#pragma unroll
    for (int u = 0; u < kXLoads; ++u) {
        const int64_t row = row0 + (kCodes ? 16 * u + cr : 8 * u + lr);
        xr[u] = x_rows<X>(g) + (row < g.m ? row : g.m - 1) * g.ld_x + (kCodes ? 16 * cc : 8 * chunk(u));
    }
    const int full = (int)(g.k / 64);              // whole 64-wide steps; a part of one may follow
    const int steps = (int)((g.k + 63) / 64);
    const v4u zero = {0u, 0u, 0u, 0u};
    bool codes = !kCodes && g.q && blockIdx.y == 0;
    uint8_t* const tx = s_tr[wave];
    uint8_t* const ta = tx + kManyRows * 16 * 128;

    struct Ops { v4u x[kXLoads], a[2 * NR]; };
    v4f acc[kManyRows][NR];
    auto pass = [&](int cur, bool with_codes) {
        const uint16_t* ar[2 * NR];
#pragma unroll
        for (int v = 0; v < 2 * NR; ++v) {
            const int r = rank0 + 8 * v + lr;
            ar[v] = g.a + ((int64_t)(cur < 0 ? 0 : cur) * g.rank + (r < g.rank ? r : g.rank - 1)) * g.k + 8 * chunk(v);
        }
#pragma unroll
        for (int i = 0; i < kManyRows; ++i)
#pragma unroll
            for (int j = 0; j < NR; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
        // a step past the last whole one reads that again and is not used: loads under a branch would
        // all be waited for at the next use of any
        auto load = [&](Ops& o, int step) {
            const int kk = min(step, full - 1) * 64;
#pragma unroll
            for (int u = 0; u < kXLoads; ++u) o.x[u] = *reinterpret_cast<const v4u*>(xr[u] + kk);
#pragma unroll
            for (int v = 0; v < 2 * NR; ++v) o.a[v] = *reinterpret_cast<const v4u*>(ar[v] + kk);
        };
        auto use = [&](const Ops& o, int step) {
            const int kk = step * 64;
            if constexpr (!kCodes) {
                if (with_codes) {
#pragma unroll
                    for (int u = 0; u < kXLoads; ++u) {
                        const int64_t row = row0 + 8 * u + lr;
                        const int at = kk + 8 * chunk(u);
                        const uint2 c = codes8(__builtin_bit_cast(bf16x8, o.x[u]), s, rs, fast);
                        if (at < g.k && row < g.m) *reinterpret_cast<uint2*>(g.q + row * g.k + at) = c;
                    }
                }
            }
            if (cur >= 0) {
#pragma unroll
                for (int u = 0; u < kXLoads; ++u) {
                    if constexpr (kCodes) {
                        *reinterpret_cast<v4u*>(tx + swz128(16 * u + cr, 2 * cc)) =
                            __builtin_bit_cast(v4u, e4m3x8_to_bf16(o.x[u][0], o.x[u][1]));
                        *reinterpret_cast<v4u*>(tx + swz128(16 * u + cr, 2 * cc + 1)) =
                            __builtin_bit_cast(v4u, e4m3x8_to_bf16(o.x[u][2], o.x[u][3]));
                    } else {
                        *reinterpret_cast<v4u*>(tx + (8 * u + lr) * 128 + slot * 16) = o.x[u];
                    }
                }
#pragma unroll
                for (int v = 0; v < 2 * NR; ++v) *reinterpret_cast<v4u*>(ta + (8 * v + lr) * 128 + slot * 16) = o.a[v];
                wave_lds_order();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    bf16x8 xf[kManyRows], af[NR];
#pragma unroll
                    for (int i = 0; i < kManyRows; ++i)
                        xf[i] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const v4u*>(tx + swz128(16 * i + r16, q + 4 * h)));
#pragma unroll
                    for (int j = 0; j < NR; ++j)
                        af[j] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const v4u*>(ta + swz128(16 * j + r16, q + 4 * h)));
#pragma unroll
                    for (int i = 0; i < kManyRows; ++i)
#pragma unroll
                        for (int j = 0; j < NR; ++j) acc[i][j] = mfma_bf16(af[j], xf[i], acc[i][j]);
                }
                wave_lds_order();
            }
        };
        Ops o0, o1;
        if (full > 0) {
            load(o0, wave);
            for (int st = wave; st < full; st += 2 * kManyWaves) {
                load(o1, st + kManyWaves);
                use(o0, st);
                load(o0, st + 2 * kManyWaves);
                if (st + kManyWaves < full) use(o1, st + kManyWaves);
            }
        }
        if (full < steps && wave == full % kManyWaves) {     // the rest of a k that 64 does not divide (16 does)
            const int kk = full * 64;
#pragma unroll
            for (int u = 0; u < kXLoads; ++u)
                o0.x[u] = kk + (kCodes ? 16 * cc : 8 * chunk(u)) < g.k ? *reinterpret_cast<const v4u*>(xr[u] + kk) : zero;
#pragma unroll
            for (int v = 0; v < 2 * NR; ++v) o0.a[v] = kk + 8 * chunk(v) < g.k ? *reinterpret_cast<const v4u*>(ar[v] + kk) : zero;
            use(o0, full);
        }
    };

    uint64_t todo[kManyRows];
#pragma unroll
    for (int i = 0; i < kManyRows; ++i) todo[i] = __ballot(id[i] >= 0) & 0xffffu;
    for (;;) {
        int cur = -1;
#pragma unroll
        for (int i = 0; i < kManyRows; ++i)
            if (cur < 0 && todo[i]) cur = __builtin_amdgcn_readlane(id[i], __builtin_ctzll(todo[i]));
        if (cur < 0) break;
#pragma unroll
        for (int i = 0; i < kManyRows; ++i) todo[i] &= ~__ballot(id[i] == cur);
        pass(cur, codes);
        codes = false;
        const float sc = (g.scale ? g.scale[cur] : 1.0f) * (sizeof(X) == 1 ? s : 1.0f);
#pragma unroll
        for (int i = 0; i < kManyRows; ++i)
#pragma unroll
            for (int j = 0; j < NR; ++j) s_part[wave][i * NR + j][lane] = acc[i][j];
        __syncthreads();
        for (int t = wave; t < kManyRows * NR; t += kManyWaves) {
            v4f d = s_part[0][t][lane];
#pragma unroll
            for (int w = 1; w < kManyWaves; ++w) d += s_part[w][t][lane];
            const int64_t row = row0 + 16 * (t / NR) + r16;
            const int r0 = rank0 + 16 * (t % NR) + 4 * (lane >> 4);
            int mine = -1;
#pragma unroll
            for (int i = 0; i < kManyRows; ++i) mine = i == t / NR ? id[i] : mine;
            if (mine == cur && r0 < g.rp) store_parts(g, row, r0, d, sc);
        }
        __syncthreads();
    }
    if (codes) pass(-1, true);      // no row here has an adapter
}

template <typename X>
static void launch_down(const LoraDownArgs& g, hipStream_t st) {
    const int64_t tiles = (g.m + 15) / 16;
    if (tiles >= 512) {
        const dim3 grid((unsigned)((tiles + kManyRows - 1) / kManyRows), (unsigned)((g.rp + 63) / 64));
        if (g.rp == 32) lora_down_many_kernel<X, 2><<<grid, dim3(kManyWaves * 64), 0, st>>>(g);
        else lora_down_many_kernel<X, 4><<<grid, dim3(kManyWaves * 64), 0, st>>>(g);
        return;
    }
    // Fewer ranks per workgroup while there are CUs for them (up to an adapter per row): 16, 8 and 4 ranks, us with
    // the projection: 8 rows of rank 64 17.0, 16.3, 15.9, 61 rows of rank 32 26.2, 25.0, 28.6.
    const int ranks = g.m * (g.rp / 4) <= 256 ? 4 : g.m * (g.rp / 8) <= 512 ? 8 : 16;
    const unsigned groups = (unsigned)(g.rp / ranks);
    int64_t z = 1024 / (tiles * groups);
    z = z < 1 ? 1 : z > 16 ? 16 : z;
    // a vector of eight codes per thread, up to as many workgroups again
    const int64_t vecs = sizeof(X) == 2 && g.q ? (g.k / 8 * 16 + kFewWaves * 64 - 1) / (kFewWaves * 64) : 0;
    int64_t extra = (vecs + groups - 1) / groups;
    extra = extra > z ? z : extra;
    lora_down_few_kernel<X><<<dim3((unsigned)tiles, groups, (unsigned)(z + extra)), dim3(kFewWaves * 64), 0, st>>>(g, (int)z, ranks);
}

nhm_status launch_lora_down(const LoraDownArgs& g, hipStream_t st) {
    if (g.x) launch_down<uint16_t>(g, st);
    else launch_down<uint8_t>(g, st);
    count_launch(Kern::kLoraDown, g.m);
    return check_launch("lora down");
}

}  // namespace nhm
