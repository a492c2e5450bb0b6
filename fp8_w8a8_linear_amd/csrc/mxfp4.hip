// MXFP4: quantisation, the values codes stand for, and the projection of MXFP4 activations by an
// MXFP4 weight (nhm_layer.h).
//
// A row's 32 consecutive elements are a block: e2m1 codes c (two a byte, the lower index in the low
// nibble) under one e8m0 scale code s, worth c 2^(s - 127). The matrix instruction takes both:
// it multiplies 32 products of a block pair by 2^(sa + sw - 254). Measured on MI355X, its sums of up to
// 128 products are within 2^-24 of sum |a w| of the exact ones, scales 2^50 apart among them: what is
// summed is summed in f32.
#include "nhm_device.h"
#include "nhm_internal.h"

namespace nhm {

// ---------------------------------------------------------------- quantisation
//
// Four lanes hold a block, eight elements each: the largest magnitude by two lane moves, the scale its
// power of two over four, and the hardware's conversion (to nearest, ties to even, saturating at 6: checked
// on every bf16 pattern). Bound by bytes.

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
        if ((c & 31) == 0) a.scales[row * a.ld_scales + c / 32] = (uint8_t)s;
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
// in wave order. TM: 16-row tiles of the activations.
constexpr int kMxWaves = 8;

template <int TM>
__global__ __launch_bounds__(kMxWaves * 64) void mx_rows_kernel(const MxGemmArgs g) {
    __shared__ v4f s_sum[kMxWaves][TM][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane & 15, q = lane >> 4;
    const unsigned tiles = (unsigned)((g.n + 15) / 16);
    const int64_t n0 = (int64_t)(blockIdx.x % tiles) * 16, m0 = (int64_t)(blockIdx.x / tiles) * (16 * TM);
    const int64_t kb = g.k / 2, ks = g.k / 32;       // bytes of codes and of scales in a weight row
    const auto wrs = mx_buffer(g.w, g.n * kb), wss = mx_buffer(g.w_scale, g.n * ks);
    const auto ars = mx_buffer(g.a, g.m * g.ld_a), ass = mx_buffer(g.a_scale, g.m * g.ld_as);
    const int64_t wr = n0 + r16;
    const uint32_t woff = wr < g.n ? (uint32_t)(wr * kb) : kPast, wsoff = wr < g.n ? (uint32_t)(wr * ks) : kPast;
    uint32_t aoff[TM], asoff[TM];
#pragma unroll
    for (int j = 0; j < TM; ++j) {
        const int64_t row = m0 + 16 * j + r16;
        aoff[j] = row < g.m ? (uint32_t)(row * g.ld_a) : kPast;
        asoff[j] = row < g.m ? (uint32_t)(row * g.ld_as) : kPast;
    }
    auto load16 = [&](const __amdgpu_buffer_rsrc_t& rs, uint32_t off, uint32_t at) {
        return __builtin_amdgcn_raw_buffer_load_b128(rs, at < kb ? off + at : kPast, 0, 0);
    };
    auto load2 = [&](const __amdgpu_buffer_rsrc_t& rs, uint32_t off, uint32_t at) {      // past the row: scale 2^-127 of zeros
        const uint32_t lo = __builtin_amdgcn_raw_buffer_load_b8(rs, at < ks ? off + at : kPast, 0, 0);
        const uint32_t hi = __builtin_amdgcn_raw_buffer_load_b8(rs, at + 1 < ks ? off + at + 1 : kPast, 0, 0);
        return lo | hi << 8;
    };
    v4f acc[TM];
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
    const int steps = (int)((g.k + 255) / 256);
#pragma unroll 2
    for (int s = wave; s < steps; s += kMxWaves) {
        const uint32_t cb = (uint32_t)s * 128 + 32 * q, sb = (uint32_t)s * 8 + 2 * q;
        const v4u w0 = load16(wrs, woff, cb), w1 = load16(wrs, woff, cb + 16);
        const uint32_t ws = load2(wss, wsoff, sb);
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            const v4u a0 = load16(ars, aoff[j], cb), a1 = load16(ars, aoff[j], cb + 16);
            const uint32_t as = load2(ass, asoff[j], sb);
            acc[j] = mfma_mx16<0>(w0, a0, acc[j], ws, as);
            acc[j] = mfma_mx16<1>(w1, a1, acc[j], ws, as);
        }
    }
#pragma unroll
    for (int j = 0; j < TM; ++j) s_sum[wave][j][lane] = acc[j];
    __syncthreads();
    for (int j = wave; j < TM; j += kMxWaves) {
        v4f x = s_sum[0][j][lane];
#pragma unroll
        for (int o = 1; o < kMxWaves; ++o) x += s_sum[o][j][lane];
        const int64_t row = m0 + 16 * j + r16, nb = n0 + 4 * q;     // four consecutive features of one row
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

nhm_status launch_mx_gemm(const MxGemmArgs& g, hipStream_t st) {
    auto rows = [&](int tm) { return dim3((unsigned)((g.n + 15) / 16 * ((g.m + 16 * tm - 1) / (16 * tm)))); };
    if (g.m <= 16) mx_rows_kernel<1><<<rows(1), dim3(kMxWaves * 64), 0, st>>>(g);
    else if (g.m <= 32) mx_rows_kernel<2><<<rows(2), dim3(kMxWaves * 64), 0, st>>>(g);
    else mx_rows_kernel<4><<<rows(4), dim3(kMxWaves * 64), 0, st>>>(g);
    count_launch(Kern::kMxRows, g.m);
    return check_launch("mxfp4 linear");
}

}  // namespace nhm
