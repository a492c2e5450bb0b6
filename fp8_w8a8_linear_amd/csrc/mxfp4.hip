// MXFP4: quantisation, the values codes stand for, and the projection of MXFP4 activations by an
// MXFP4 weight (nhm_layer.h).
//
// A row's 32 consecutive elements are a block: e2m1 codes c (two a byte, the lower index in the low
// nibble) under one e8m0 scale code s, worth c 2^(s - 127). The matrix instruction takes both:
// it multiplies 32 products of a block pair by 2^(sa + sw - 254). Measured on MI355X, its sums of up to
// 128 products are within 2^-24 of sum |a w| of the exact ones, scales 2^50 apart among them: what is
// summed is summed in f32.
#include <type_traits>

#include "nhm_device.h"
#include "nhm_internal.h"

namespace nhm {

// ---------------------------------------------------------------- quantisation
//
// Four lanes hold a block, eight elements each: the largest magnitude by two lane moves, the scale its
// power of two over four, and the hardware's conversion (to nearest, ties to even, saturating at 6: checked
// on every bf16 pattern). Bound by bytes: 15,360 x 4,096 bf16 31 us (159 MB, 5.1 TB/s).

// Largest magnitude of the block's four lanes, as float bits (ordered as integers; NaN above infinity).
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));
}

// Scale code of a block whose largest magnitude is `amax` (bits): floor(log2) - 2, as an e8m0 code; 255 (NaN) where the
// block holds an infinity or NaN. Subnormal magnitudes (2^-127 and below) and small normal ones take code 0.
__device__ __forceinline__ uint32_t mx_scale(uint32_t amax) {
    const uint32_t e = amax >> 23;
    return e == 255 ? 255u : e > 2 ? e - 2 : 0u;
}

// Eight floats to eight codes under scale code s.
__device__ __forceinline__ uint32_t mx_codes(const float (&f)[8], uint32_t s) {
    if (s == 255) return 0u;
    // the conversion divides by the scale; both sides times 2^64 where the scale is small, so that it is a normal float
    const float up = s < 64 ? 0x1p64f : 1.0f;
    const float sc = __uint_as_float((s < 64 ? s + 64 : s) << 23);
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[0] * up, f[1] * up, sc, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[2] * up, f[3] * up, sc, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[4] * up, f[5] * up, sc, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[6] * up, f[7] * up, sc, 3);
}

template <bool kF32>
__device__ __forceinline__ void load8(const char* p, float (&f)[8]) {
    if constexpr (kF32) {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        unpack8(*reinterpret_cast<const uint4*>(p), f);
    }
}

template <bool kF32>
__global__ __launch_bounds__(256) void mx_quant_kernel(const MxQuantArgs a) {
    const int per = (int)(a.cols / 8);      // pieces of a row
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.rows * per; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / per;
        const int c = (int)(i - row * per) * 8;
        float f[8];
        load8<kF32>(static_cast<const char*>(a.x) + (row * a.ld_x + c) * (kF32 ? 4 : 2), f);
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7fffffffu);
        const uint32_t s = mx_scale(quad_max(m));
        *reinterpret_cast<uint32_t*>(a.codes + row * a.ld_codes + c / 2) = mx_codes(f, s);
        if ((c & 31) == 0) {
            if (a.packed) {
                // byte (c / 32) % 4 of dword (c / 128, row); the last block also clears what its dword has left
                uint8_t* const d = reinterpret_cast<uint8_t*>(a.packed + (int64_t)(c / 128) * a.rows + row);
                d[c / 32 % 4] = (uint8_t)s;
                if (c + 32 == a.cols)
                    for (int p = c / 32 % 4 + 1; p < 4; ++p) d[p] = 0;
            } else {
                a.scales[row * a.ld_scales + c / 32] = (uint8_t)s;
            }
        }
    }
}

static unsigned mx_blocks(int64_t pieces) {
    const int64_t b = (pieces + 255) / 256;
    return (unsigned)(b < 65536 ? b : 65536);
}

nhm_status launch_mx_quant(const MxQuantArgs& a, bool f32, hipStream_t st) {
    if (f32) mx_quant_kernel<true><<<dim3(mx_blocks(a.rows * (a.cols / 8))), dim3(256), 0, st>>>(a);
    else mx_quant_kernel<false><<<dim3(mx_blocks(a.rows * (a.cols / 8))), dim3(256), 0, st>>>(a);
    count_launch(Kern::kMxQuant, a.rows);
    return check_launch("mxfp4 quantize");
}

// ---------------------------------------------------------------- the codes' values
//
// Eight values to a thread, 16 bytes. Bound by bytes: 15,360 x 4,096 34 us (159 MB, 4.6 TB/s).

// The bf16 value of a code under a scale code (not 255): exact, but past the largest finite bf16, which is infinity.
__device__ __forceinline__ float mx_value(uint32_t c, uint32_t s) {
    const uint32_t m = c & 7u;
    // 2^-1, 1, 2 and 4 times 1 or 1.5; code 1 is 0.5, code 0 is 0
    const float mag = m < 2 ? 0.5f * (float)m : __uint_as_float((126u + (m >> 1)) << 23 | (m & 1u) << 22);
    const float v = c & 8u ? -mag : mag;
    return s < 2 ? v * __uint_as_float((s + 64) << 23) * 0x1p-64f : v * __uint_as_float(s << 23);
}

__global__ __launch_bounds__(256) void mx_dequant_kernel(const MxDequantArgs a) {
    const int per = (int)(a.cols / 8);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.rows * per; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / per;
        const int c = (int)(i - row * per) * 8;
        const uint32_t q = *reinterpret_cast<const uint32_t*>(a.codes + row * a.ld_codes + c / 2);
        const uint32_t s = a.scales[row * a.ld_scales + c / 32];
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = s == 255 ? __uint_as_float(0x7fc00000u) : mx_value(q >> (4 * j) & 15u, s);
        *reinterpret_cast<uint4*>(a.out + row * a.ld_out + c) =
            make_uint4(f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]), f32x2_to_bf16x2(f[4], f[5]),
                       f32x2_to_bf16x2(f[6], f[7]));
    }
}

nhm_status launch_mx_dequant(const MxDequantArgs& a, hipStream_t st) {
    mx_dequant_kernel<<<dim3(mx_blocks(a.rows * (a.cols / 8))), dim3(256), 0, st>>>(a);
    count_launch(Kern::kMxDequant, a.rows);
    return check_launch("mxfp4 dequantize");
}

// ---------------------------------------------------------------- projection

constexpr uint32_t kPast = 0x80000000u;     // past every buffer range used here (< 2^31 bytes)

__device__ __forceinline__ __amdgpu_buffer_rsrc_t mx_buffer(const void* p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}

// 16x16x128 on e2m1: byte S of each scale register.
template <int S>
__device__ __forceinline__ v4f mfma_mx16(const v4u& a, const v4u& b, const v4f& c, uint32_t sa, uint32_t sb) {
    v8i x{}, y{};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] = (int)a[i];
        y[i] = (int)b[i];
    }
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, S, (int)sa, S, (int)sb);
}

// Few rows: a workgroup of eight waves takes 16 features, each wave a share of k, in steps of 256: lane (r, q) holds the 32 bytes
// of row r that start 32 q into the step's 128-byte line, two blocks, and their two scale codes. The waves' sums are added in LDS
// in wave order. TM: 16-row tiles of the activations. kQuant: the activations are bf16, and every workgroup quantises them
// into LDS, behind its first loads of the weight. Bound by latency and the weight's bytes: 1 row x 10,304 x 2,688 4.4 us (14.7 MB,
// 3.3 TB/s), 61 rows 9.9 to 10.7. (Loading a step or two ahead of the products made the call up to half again as long.)
constexpr int kMxWaves = 8;

template <int TM, bool kQuant>
__global__ __launch_bounds__(kMxWaves * 64) void mx_rows_kernel(const MxGemmArgs g) {
    __shared__ v4f s_sum[kMxWaves][TM][64];
    extern __shared__ __attribute__((aligned(16))) uint8_t s_a[];      // kQuant: codes [m, 128 steps], behind them scale codes [m, 8 steps]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane & 15, q = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int64_t kb = g.k / 2, ks = g.k / 32;       // bytes of codes and of scales in a weight row
    const int steps = (int)((g.k + 255) / 256);
    const auto wrs = mx_buffer(g.w, g.n * kb), wss = mx_buffer(g.w_scale, g.n * g.ld_ws);
    const int64_t wr = n0 + r16;
    const uint32_t woff = wr < g.n ? (uint32_t)(wr * kb) : kPast, wsoff = wr < g.n ? (uint32_t)(wr * g.ld_ws) : kPast;
    const auto ars = mx_buffer(g.a, kQuant ? 0 : g.m * g.ld_a), ass = mx_buffer(g.a_scale, kQuant ? 0 : g.m * g.ld_as);
    uint32_t aoff[TM], asoff[TM];
#pragma unroll
    for (int j = 0; j < TM; ++j) {
        const int64_t row = 16 * j + r16;
        aoff[j] = row < g.m ? (uint32_t)(row * g.ld_a) : kPast;
        asoff[j] = row < g.m ? (uint32_t)(row * g.ld_as) : kPast;
    }
    auto load16 = [&](const __amdgpu_buffer_rsrc_t& rs, uint32_t off, uint32_t at) {
        return __builtin_amdgcn_raw_buffer_load_b128(rs, at < kb ? off + at : kPast, 0, 0);
    };
    // two scale codes; past the row 2^-127, of zeros. In one load where every row's pairs are whole (half the requests: 64 x 2,688 x
    // 4,096 9.0 us, with two 11.0)
    const bool pairs = ks % 2 == 0 && ((reinterpret_cast<uintptr_t>(g.w_scale) | reinterpret_cast<uintptr_t>(g.a_scale)) & 1) == 0;
    auto load2 = [&](const __amdgpu_buffer_rsrc_t& rs, uint32_t off, uint32_t at) -> uint32_t {
        if (pairs) return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, at < ks ? off + at : kPast, 0, 0);
        const uint32_t lo = __builtin_amdgcn_raw_buffer_load_b8(rs, at < ks ? off + at : kPast, 0, 0);
        const uint32_t hi = __builtin_amdgcn_raw_buffer_load_b8(rs, at + 1 < ks ? off + at + 1 : kPast, 0, 0);
        return lo | hi << 8;
    };
    struct Step { v4u w0, w1, a0[TM], a1[TM]; uint32_t ws, as[TM]; };
    auto load = [&](Step& x, int s) {                // a step past the last is all zeros
        const uint32_t cb = (uint32_t)s * 128 + 32 * q, sb = (uint32_t)s * 8 + 2 * q;
        x.w0 = load16(wrs, woff, cb);
        x.w1 = load16(wrs, woff, cb + 16);
        x.ws = load2(wss, wsoff, sb);
        if constexpr (!kQuant)
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                x.a0[j] = load16(ars, aoff[j], cb);
                x.a1[j] = load16(ars, aoff[j], cb + 16);
                x.as[j] = load2(ass, asoff[j], sb);
            }
    };
    Step x;
    if constexpr (kQuant) {
        load(x, wave);
        // as mx_quant_kernel, zeros up to whole steps
        for (int i = threadIdx.x; i < (int)g.m * steps * 32; i += kMxWaves * 64) {
            const int row = i / (steps * 32), c = i % (steps * 32) * 8;
            uint32_t s = 0, codes = 0;
            if (c < g.k) {
                float f[8];
                load8<false>(reinterpret_cast<const char*>(g.a_bf16 + row * g.ld_bf16 + c), f);
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7fffffffu);
                s = mx_scale(quad_max(m));
                codes = mx_codes(f, s);
            }
            *reinterpret_cast<uint32_t*>(s_a + row * (steps * 128) + c / 2) = codes;
            if ((c & 31) == 0) s_a[(int)g.m * (steps * 128) + row * (steps * 8) + c / 32] = (uint8_t)s;
        }
        __syncthreads();
    }
    v4f acc[TM];
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
    auto use = [&](Step& x, int s) {
        if constexpr (kQuant) {
            const int row = min(r16, (int)g.m - 1);         // (rows past the last are not stored)
            const uint8_t* const c = s_a + row * (steps * 128) + s * 128 + 32 * q;
            x.a0[0] = *reinterpret_cast<const v4u*>(c);
            x.a1[0] = *reinterpret_cast<const v4u*>(c + 16);
            x.as[0] = *reinterpret_cast<const uint16_t*>(s_a + (int)g.m * (steps * 128) + row * (steps * 8) + s * 8 + 2 * q);
        }
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            acc[j] = mfma_mx16<0>(x.w0, x.a0[j], acc[j], x.ws, x.as[j]);
            acc[j] = mfma_mx16<1>(x.w1, x.a1[j], acc[j], x.ws, x.as[j]);
        }
    };
    for (int s = wave; s < steps; s += kMxWaves) {
        if (!kQuant || s != wave) load(x, s);
        use(x, s);
    }
#pragma unroll
    for (int j = 0; j < TM; ++j) s_sum[wave][j][lane] = acc[j];
    __syncthreads();
    for (int j = wave; j < TM; j += kMxWaves) {
        v4f x = s_sum[0][j][lane];
#pragma unroll
        for (int o = 1; o < kMxWaves; ++o) x += s_sum[o][j][lane];
        const int64_t row = 16 * j + r16, nb = n0 + 4 * q;     // four consecutive features of one row
        if (row >= g.m) continue;
        if (g.out_f32) {
            float* o = g.out_f32 + row * g.ld_out + nb;
            if (g.vec_out && nb + 4 <= g.n) *reinterpret_cast<v4f*>(o) = x;
            else
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (nb + r < g.n) o[r] = x[r];
        } else {
            uint16_t* o = g.out + row * g.ld_out + nb;
            if (g.vec_out && nb + 4 <= g.n) *reinterpret_cast<uint2*>(o) = make_uint2(f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]));
            else
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (nb + r < g.n) o[r] = (uint16_t)f32_to_bf16(x[r]);
        }
    }
}

// ---------------------------------------------------------------- tiles
//
// Many rows: a workgroup computes TN features x TM rows, its NWN x NWM waves TN / NWN x TM / NWM each, by the 32x32x64 matrix
// instruction. Slices of k, KB bytes of codes of every row, stream into a ring of LDS stages by direct loads; the operands of
// the next stage are read while the current one's products run. The scale codes travel as dwords, four blocks of a row, one
// dword (KB = 64) or two (KB = 128) to a row and stage, packed so that a load's 64 rows are 256 bytes in a row: from rows of
// scale codes every dword is a request of its own, and half of all requests to L2 were theirs.
// A lane's half of a stage's row is KB / 2 bytes, KB / 32 blocks, whose scale codes are adjacent bytes: with 128 byte
// slices a dword of its own, which the matrix instruction takes bytes of.
//
// 15,360 x 10,304 x 2,688: 265 to 300 us by the clock that the power leaves (2.8 to 3.2 PFLOP/s of codes). No unit is busy all the time:
// the matrix units 45 %, LDS with the operands' reads 21 % (no bank conflicts), and the way from L2 into LDS about a fifth (7.0 MB to a
// CU, at 133 bytes a ns at most). What is left is what each stage's wait and barrier keep from overlapping, not taken apart further.
// f32 outputs, on the 128 x 128 tile: 353 to 398 us, the matrix units 33 % busy, LDS 19 %. 477 x 2,688 x 4,096: 12 us, a workgroup's
// own chain of 16 stages, of which the ring of two has one on its way while one is used. Taking the activations' scale codes
// as rows, without the launch that packs them (2 us), is no faster from 96 to 15,360 rows.

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));

__device__ __forceinline__ i32x4 mx_desc(const void* base, int64_t bytes) {
    const uint64_t b = reinterpret_cast<uint64_t>(base);
    return i32x4{(int)(uint32_t)b, (int)((uint32_t)(b >> 32) & 0xffffu), (int)bytes, 0x00020000};
}

// kBytes (16 or 4) per lane from byte offset voff + soff of the buffer into LDS at lds + kBytes * lane (an offset past the
// range writes zeros; soff itself must lie within it: the hardware compares voff with the range less soff). As asm, so that the compiler does not hold every later LDS read behind it; the kernel waits for these
// loads itself, and the wait states ahead of the load stand here: one after the write of M0, five after a vector instruction
// that wrote a register of the descriptor.
template <int kBytes>
__device__ __forceinline__ void dma(const i32x4& rs, const uint8_t* lds, uint32_t voff, uint32_t soff) {
    const uint32_t m0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)lds;
    if constexpr (kBytes == 16)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(m0), "v"(voff), "s"(rs), "s"(soff)
                     : "memory", "m0");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"s"(m0), "v"(voff), "s"(rs), "s"(soff)
                     : "memory", "m0");
}

template <int S>
__device__ __forceinline__ v16f mfma_mx32(const v4u& a, const v4u& b, const v16f& c, uint32_t sa, uint32_t sb) {
    v8i x{}, y{};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] = (int)a[i];
        y[i] = (int)b[i];
    }
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, S, (int)sa, S, (int)sb);
}

// 16-byte chunk c of row r of a stage: 16 rows read at one chunk cover all LDS banks.
template <int KB>
__device__ __forceinline__ int mx_slot(int row, int c) {
    if constexpr (KB == 64) return row * 64 + ((c ^ (((row >> 1) ^ (row >> 2)) & 3)) << 4);
    else return swz128(row, c);
}

template <int TN, int TM, int NWN, int NWM, int KB, int RING, bool f32>
__global__ __launch_bounds__(64 * NWN * NWM) void mx_tile_kernel(const MxGemmArgs g) {
    constexpr int kWaves = NWN * NWM, kRows = TN + TM, kNI = TN / NWN / 32, kNJ = TM / NWM / 32;
    constexpr int kCodes = kRows * KB, kPlanes = KB / 64, kStage = kCodes + kPlanes * kRows * 4;
    constexpr int kBlockRows = 1024 / KB, kBlocks = kRows / kBlockRows, kLoads = kBlocks / kWaves;   // 1 KB a load
    constexpr int kScales = kPlanes * kRows / 64, kScaleLoads = (kScales + kWaves - 1) / kWaves;      // 64 dwords a load
    constexpr int kAll = kLoads + kScaleLoads, kSteps = KB / 32;
    static_assert(TN % (kBlockRows * kWaves) == 0 && TM % (kBlockRows * kWaves) == 0 && kBlockRows * kWaves % 16 == 0 &&
                  TN % 64 == 0 && TM % 64 == 0, "whole loads");
    static_assert(RING >= 2 && (RING - 2) * kAll + (f32 ? 4 : 2) * kNI * kNJ < 64 && (RING - 1) * kAll < 64, "ring depth and the vmcnt field");
    // With two waves to a matrix unit the loads go out between the products, ahead of which they hold the units up; with one,
    // ahead of them.
    constexpr bool kEarly = kWaves <= 4;
    constexpr int kSpare = kScales % kWaves ? 256 : 0;      // where the waves without a scale load put zeros
    __shared__ __attribute__((aligned(16))) uint8_t smem[RING * kStage + kSpare];
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wn = wave / NWM, wm = wave % NWM, r32 = lane & 31, q = lane >> 5;

    // Blocks go to the 8 XCDs round robin; each XCD takes a contiguous share of the tiles, its workgroups tile by tile in
    // turn, in an order that walks 8 row tiles per feature tile: the tiles it works on at once share operands through its L2.
    const int ntn = (int)((g.n + TN - 1) / TN), ntm = (int)((g.m + TM - 1) / TM), total = ntn * ntm;
    const int xcd = blockIdx.x & 7, share = gridDim.x >> 3;
    const int tile_end = (xcd + 1) * (total >> 3) + min(xcd + 1, total & 7);
    int tile = xcd * (total >> 3) + min(xcd, total & 7) + (int)(blockIdx.x >> 3);
    auto origin = [&](int j, int& m0, int& n0) {
        const int grp = j / (8 * ntn), in_grp = j - grp * 8 * ntn, gms = min(8, ntm - grp * 8);
        m0 = (grp * 8 + in_grp % gms) * TM;
        n0 = in_grp / gms * TN;
    };

    const int kb = (int)(g.k / 2), ks4 = (int)((g.k / 32 + 3) / 4), nk = (kb + KB - 1) / KB;
    const i32x4 wrs = mx_desc(g.w, g.n * kb), ars = mx_desc(g.a, (g.m - 1) * g.ld_a + kb);    // not past the last row's end
    const i32x4 wss = mx_desc(g.w_packed, g.n * ks4 * 4), ass = mx_desc(g.a_packed, g.m * ks4 * 4);
    // The loads go ahead of the products, into the next tile too: lt, ls are the tile and stage that they are at. Load i of
    // a wave is block wave + i kWaves of the stage, so that every wave's are of the weight first, then of the activations, in
    // rows a multiple of 16 apart, whose chunks have the same slots. No lane needs a check: rows past an operand lie past its
    // buffer and are zeros, and what a row's last stage takes from behind the row counts nothing, since both operands' scale
    // codes there are 0 (the products are below 2^-240).
    constexpr int kPer = KB / 16, kWLoads = TN / kBlockRows / kWaves, kRowStep = kBlockRows * kWaves;
    const int lrow = wave * kBlockRows + lane / kPer;
    const int lchunk = 16 * (KB == 64 ? (lane % kPer) ^ (((lrow >> 1) ^ (lrow >> 2)) & 3) : (lane % kPer) ^ (lrow & 7) ^ ((lrow >> 3) & 1));
    uint32_t wbase, abase, sbase[kScaleLoads];      // this lane's source offsets at k = 0
    int lt = tile, ls = 0;
    auto set_bases = [&]() {
        int m0, n0;
        origin(min(lt, total - 1), m0, n0);
        const bool more = lt < tile_end;            // else nothing but zeros
        wbase = more ? (uint32_t)(n0 + lrow) * (uint32_t)kb + lchunk : kPast;
        abase = more ? (uint32_t)(m0 + lrow) * (uint32_t)g.ld_a + lchunk : kPast;
#pragma unroll
        for (int i = 0; i < kScaleLoads; ++i) {
            const int blk = wave + i * kWaves, row = blk % (kRows / 64) * 64 + lane, plane = blk / (kRows / 64);
            const bool isw = row < TN;
            const int at = isw ? n0 + row : m0 + row - TN, rows = (int)(isw ? g.n : g.m);
            sbase[i] = more && blk < kScales && at < rows ? (uint32_t)(plane * rows + at) * 4 : kPast;
        }
    };
    // the next stage of the loads into a slot: load i of the wave's kAll, and what follows the last
    auto load = [&](int slot, int i) {
        uint8_t* const sb = smem + slot * kStage;
        if (i < kLoads) {
            uint8_t* const to = sb + (wave + i * kWaves) * 1024;
            if (i < kWLoads) dma<16>(wrs, to, wbase + (uint32_t)(i * kRowStep) * (uint32_t)kb, (uint32_t)(ls * KB));
            else dma<16>(ars, to, abase + (uint32_t)((i - kWLoads) * kRowStep) * (uint32_t)g.ld_a, (uint32_t)(ls * KB));
        } else {
            const int blk = wave + (i - kLoads) * kWaves;
            const bool isw = blk % (kRows / 64) * 64 < TN;
            uint8_t* const to = kSpare != 0 && blk >= kScales ? smem + RING * kStage : sb + kCodes + blk * 256;
            dma<4>(isw ? wss : ass, to, sbase[i - kLoads] + (uint32_t)(ls * kPlanes) * (uint32_t)(isw ? g.n : g.m) * 4u, 0u);
        }
    };
    auto advance = [&]() {
        if (++ls == nk) {
            ls = 0;
            lt += share;
            set_bases();
        }
    };
    struct Ops { v4u w[kNI], a[kNJ]; };
    struct Scales { uint32_t w[kNI], a[kNJ]; };
    // rows 16 apart have the same slots: addresses are those of the wave's first rows and constants
    int at[kSteps];
#pragma unroll
    for (int u = 0; u < kSteps; ++u) at[u] = mx_slot<KB>(r32, q * kSteps + u);
    const int wrow = wn * (TN / NWN), arow = TN + wm * (TM / NWM);
    const int sat = kCodes + (kPlanes == 2 ? (q * kRows + r32) * 4 : r32 * 4 + 2 * q);
    auto read = [&](int slot, int u, Ops& o) {
        const uint8_t* const p = smem + slot * kStage + at[u];
#pragma unroll
        for (int i = 0; i < kNI; ++i) o.w[i] = *reinterpret_cast<const v4u*>(p + (wrow + 32 * i) * KB);
#pragma unroll
        for (int j = 0; j < kNJ; ++j) o.a[j] = *reinterpret_cast<const v4u*>(p + (arow + 32 * j) * KB);
    };
    auto read_scales = [&](int slot, Scales& o) {
        const uint8_t* const p = smem + slot * kStage + sat;
        auto one = [&](int row) {
            if constexpr (kPlanes == 2) return *reinterpret_cast<const uint32_t*>(p + row * 4);
            else return (uint32_t)*reinterpret_cast<const uint16_t*>(p + row * 4);
        };
#pragma unroll
        for (int i = 0; i < kNI; ++i) o.w[i] = one(wrow + 32 * i);
#pragma unroll
        for (int j = 0; j < kNJ; ++j) o.a[j] = one(arow + 32 * j);
    };
    v16f acc[kNI][kNJ];
    Ops ops[2];
    Scales sc, sc_next;
    // then(n) behind the n-th product
    auto multiply = [&](auto u, auto then) {
        constexpr int U = decltype(u)::value;
#pragma unroll
        for (int i = 0; i < kNI; ++i)
#pragma unroll
            for (int j = 0; j < kNJ; ++j) {
                acc[i][j] = mfma_mx32<U>(ops[U & 1].w[i], ops[U & 1].a[j], acc[i][j], sc.w[i], sc.a[j]);
                then(i * kNJ + j);
            }
    };

    // stores of a finished tile: straight from the registers, so that the ring keeps filling. A fixed number of them, by
    // offsets in the tile (out of range for rows and features past the output), which the waits below count.
    // acc[i][j] register r: feature 32 i + 8 (r / 4) + 4 q + r % 4 of row 32 j + r32 of the wave's tile.
    constexpr int kStores = (f32 ? 4 : 2) * kNI * kNJ;
    const bool vec = g.vec_tile;
    auto store = [&](int m0, int n0) {
        const int nw = n0 + wrow, mw = m0 + arow - TN;
        if (vec) {
            const int size = f32 ? 4 : 2;
            char* const base = (f32 ? reinterpret_cast<char*>(g.out_f32) : reinterpret_cast<char*>(g.out)) + ((int64_t)m0 * g.ld_out + n0) * size;
            const auto rs = __builtin_amdgcn_make_buffer_rsrc(base, (short)0, 0x7fffffff, 0x00020000);
#pragma unroll
            for (int j = 0; j < kNJ; ++j) {
                const uint32_t row = (uint32_t)(arow - TN + 32 * j + r32) * (uint32_t)(g.ld_out * size);
                const bool in = mw + 32 * j + r32 < g.m;
#pragma unroll
                for (int i = 0; i < kNI; ++i) {
                    const v16f& c = acc[i][j];
                    if constexpr (f32) {
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            const int nb = 32 * i + 8 * b + 4 * q;
                            const v4f v = {c[4 * b], c[4 * b + 1], c[4 * b + 2], c[4 * b + 3]};
                            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, v), rs,
                                                                   in && nw + nb < g.n ? row + (wrow + nb) * 4 : kPast, 0, 0);
                        }
                    } else {
                        // a lane has four consecutive features of a row; two lanes' halves change places for eight
#pragma unroll
                        for (int b = 0; b < 4; b += 2) {
                            const auto lo = __builtin_amdgcn_permlane32_swap(f32x2_to_bf16x2(c[4 * b], c[4 * b + 1]),
                                                                             f32x2_to_bf16x2(c[4 * b + 4], c[4 * b + 5]), false, false);
                            const auto hi = __builtin_amdgcn_permlane32_swap(f32x2_to_bf16x2(c[4 * b + 2], c[4 * b + 3]),
                                                                             f32x2_to_bf16x2(c[4 * b + 6], c[4 * b + 7]), false, false);
                            const int nb = 32 * i + 8 * (b + q);
                            __builtin_amdgcn_raw_buffer_store_b128(v4u{lo[0], hi[0], lo[1], hi[1]}, rs,
                                                                   in && nw + nb < g.n ? row + (wrow + nb) * 2 : kPast, 0, 0);
                        }
                    }
                }
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < kNI; ++i)
#pragma unroll
            for (int j = 0; j < kNJ; ++j) {
                const int64_t row = mw + 32 * j + r32;
                if (row >= g.m) continue;
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int64_t nn = nw + 32 * i + 8 * (r / 4) + 4 * q + r % 4;
                    if (nn >= g.n) continue;
                    if (f32) g.out_f32[row * g.ld_out + nn] = acc[i][j][r];
                    else g.out[row * g.ld_out + nn] = (uint16_t)f32_to_bf16(acc[i][j][r]);
                }
            }
        wait_vmcnt<0>();
    };

    set_bases();
#pragma unroll
    for (int s = 0; s < RING; ++s) {
#pragma unroll
        for (int i = 0; i < kAll; ++i) load(s, i);
        advance();
    }
    wait_vmcnt<(RING - 1) * kAll>();
    __syncthreads();
    read(0, 0, ops[0]);
    read_scales(0, sc);
    // Of a stage, 64 of k at a time: the next step's operands are read while this one's products run. Ahead of the last
    // step's products the next stage has landed (this thread's loads, then everyone's) and everyone has this stage's last
    // operands in registers: its slot is refilled. Loads and stores return in order: for the first stages behind a tile's
    // stores these are younger than the stage waited for.
    int slot = 0, since = RING;
    for (; tile < tile_end; tile += share) {
        int m0, n0;
        origin(tile, m0, n0);
#pragma unroll
        for (int i = 0; i < kNI; ++i)
#pragma unroll
            for (int j = 0; j < kNJ; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
        for (int s = 0; s < nk; ++s) {
            const int next = slot + 1 == RING ? 0 : slot + 1;
            auto inner = [&](auto u) {
                constexpr int U = decltype(u)::value;
                if constexpr (U + 1 < kSteps) {
                    read(slot, U + 1, ops[(U + 1) & 1]);
                    __builtin_amdgcn_sched_barrier(0);
                    multiply(u, [](int) {});
                    __builtin_amdgcn_sched_barrier(0);
                }
            };
            inner(std::integral_constant<int, 0>());
            inner(std::integral_constant<int, 1>());
            inner(std::integral_constant<int, 2>());
            if (since > RING - 2) wait_vmcnt<(RING - 2) * kAll>();
            else wait_vmcnt<(RING - 2) * kAll + kStores>();
            ++since;
            __syncthreads();         // waits for the LDS reads too
            if constexpr (kEarly)
#pragma unroll
                for (int i = 0; i < kAll; ++i) load(slot, i);
            read(next, 0, ops[0]);
            read_scales(next, sc_next);
            __builtin_amdgcn_sched_barrier(0);
            constexpr int kProducts = kNI * kNJ, kEach = (kAll + kProducts - 1) / kProducts;
            multiply(std::integral_constant<int, kSteps - 1>(), [&](int n) {
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < kEach; ++i)
                    if (!kEarly && n * kEach + i < kAll) load(slot, n * kEach + i);
                __builtin_amdgcn_sched_barrier(0);
            });
            advance();
            sc = sc_next;
            slot = next;
        }
        store(m0, n0);
        since = vec ? 0 : RING;
    }
    wait_vmcnt<0>();                // the loads past the last tile
}

__global__ __launch_bounds__(256) void mx_pack_kernel(const uint8_t* scales, int rows, int ks, uint32_t* packed) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int row = (int)(i % rows), j = (int)(i / rows);
    if (4 * j >= ks) return;
    uint32_t v = 0;
#pragma unroll
    for (int p = 0; p < 4; ++p)
        if (4 * j + p < ks) v |= (uint32_t)scales[(int64_t)row * ks + 4 * j + p] << (8 * p);
    packed[i] = v;
}

nhm_status launch_mx_pack(const uint8_t* scales, int64_t rows, int64_t k, uint32_t* packed, hipStream_t st) {
    const int64_t words = mx_packed_words(rows, k);
    mx_pack_kernel<<<dim3((unsigned)((words + 255) / 256)), dim3(256), 0, st>>>(scales, (int)rows, (int)(k / 32), packed);
    count_launch(Kern::kMxPack, rows);
    return check_launch("mxfp4 scales");
}

// More tiles than the chip holds workgroups of follow one another in the same workgroups, whose loads then run ahead into the
// next tile.
template <int TN, int TM, int NWN, int NWM, int KB, int RING>
static void launch_tile(MxGemmArgs g, const MxTile& t, hipStream_t st) {
    const int64_t tiles = (g.n + TN - 1) / TN * ((g.m + TM - 1) / TM), most = 256 * t.per_cu;
    const int64_t blocks = tiles < most ? (tiles + 7) / 8 * 8 : most;
    // stores of 16 bytes at 32-bit offsets within a tile
    const int64_t size = g.out_f32 ? 4 : 2;
    const uintptr_t out = g.out_f32 ? reinterpret_cast<uintptr_t>(g.out_f32) : reinterpret_cast<uintptr_t>(g.out);
    g.vec_tile = out % 16 == 0 && g.ld_out * size % 16 == 0 && g.n * size % 16 == 0 && g.ld_out * size * TM < (int64_t(1) << 31);
    if (TN * TM < 256 * 256 && g.out_f32) mx_tile_kernel<TN, TM, NWN, NWM, KB, RING, TN * TM < 256 * 256><<<dim3((unsigned)blocks), dim3(64 * NWN * NWM), 0, st>>>(g);
    else mx_tile_kernel<TN, TM, NWN, NWM, KB, RING, false><<<dim3((unsigned)blocks), dim3(64 * NWN * NWM), 0, st>>>(g);
}

bool mx_tiled(int64_t m) { return m > 64; }

nhm_status launch_mx_gemm(const MxGemmArgs& g, hipStream_t st) {
    if (!mx_tiled(g.m)) {
        const dim3 grid((unsigned)((g.n + 15) / 16)), block(kMxWaves * 64);
        if (g.a_bf16) mx_rows_kernel<1, true><<<grid, block, (size_t)g.m * ((g.k + 255) / 256) * 136, st>>>(g);
        else if (g.m <= 16) mx_rows_kernel<1, false><<<grid, block, 0, st>>>(g);
        else if (g.m <= 32) mx_rows_kernel<2, false><<<grid, block, 0, st>>>(g);
        else mx_rows_kernel<4, false><<<grid, block, 0, st>>>(g);
        count_launch(Kern::kMxRows, g.m);
        return check_launch("mxfp4 linear");
    }
    const MxTile t = mx_tile(g.m, g.n, g.out_f32 != nullptr);
    if (t.tn == 256) launch_tile<256, 256, 2, 4, 64, 4>(g, t, st);
    else if (t.tm == 128) launch_tile<128, 128, 2, 2, 128, 2>(g, t, st);
    else if (t.tn == 128) launch_tile<128, 64, 2, 2, 128, 2>(g, t, st);
    else launch_tile<64, 64, 2, 2, 128, 2>(g, t, st);
    count_launch(Kern::kMxTile, g.m);
    return check_launch("mxfp4 linear");
}

}  // namespace nhm
