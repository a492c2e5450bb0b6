// The selective state space scan with its short causal convolution (nhm_layer.h), for prompts and
// for single tokens.
//
// conv:  u_t = f(b + sum_j w_j x_{t - W + 1 + j}), f = silu or the identity
// scan:  dt = softplus(dt_raw + dt_bias), A = -exp(A_log)
//        h_t[n] = exp(dt_t A[n]) h_{t-1}[n] + dt_t u_t B_t[n]
//        y_t = (sum_n C_t[n] h_t[n] + D u_t) silu(z_t)
// for every channel, with a decay for each channel and state: no two channels share a decay, so that
// there is no chunked matrix form (as the mixer's scan has), and each state is a recurrence over time.
#include <type_traits>

#include "nhm_device.h"
#include "nhm_internal.h"

namespace nhm {

constexpr float kLog2e = 1.44269504088896341f;

// softplus(x) = max(x, 0) + log1p(e), e = exp(-|x|) in (0, 1], and log1p(e) = 2 atanh(s), s = e / (2 + e) <= 1/3. atanh(s) / s =
// 1 + s^2 / 3 + s^4 / 5 ... by the polynomial in s^2 <= 1/9 that meets it at the five Chebyshev nodes, within 2^-26.9 of the value.
__device__ __forceinline__ float softplus_poly(float x) {
    const float e = __builtin_amdgcn_exp2f(-fabsf(x) * kLog2e);
    const float s = e * __builtin_amdgcn_rcpf(2.0f + e), q = s * s;
    float p = fmaf(q, 2 * 0.1407889f, 2 * 0.13982579f);
    p = fmaf(q, p, 2 * 0.20012298f);
    p = fmaf(q, p, 2 * 0.3333316f);
    p = fmaf(q, p, 2.0f);
    return fmaf(s, p, fmaxf(x, 0.0f));
}

// A log2(e) of a state, finite where A is not, so that a step of 0 (as past a sequence's end) keeps any state.
__device__ __forceinline__ float decay_rate(float A_log) {
    const float r = -expf(A_log) * kLog2e;
    return r < -3.402823466e38f ? -3.402823466e38f : r;
}

__device__ __forceinline__ bool has_slot(int slot, int n_slots) { return slot >= 0 && slot < n_slots; }

// ---------------------------------------------------------------- scan of prompts
//
// A lane holds one state of one channel (R of them where d_state > 16): 16 lanes are a channel, a wave is four, a
// workgroup of four waves 16. Tokens are staged 16 to 64 at a time, loads one such block ahead: a thread takes four
// channels of a token, forms dt and dt u, and leaves them, u and z in LDS by channel, as it does B and C by state, widened to f32;
// the lanes read four tokens of theirs at once. (Lane moves inside the multiplications halve their rate: 8.4 cycles
// against 4.5.) A token then costs mul, exp2, mul, fma, mul per state, and the sum over the channel's lanes: 16 tokens' products
// are summed together, each step keeping half of the tokens in half of the lanes, so that the lane of state n ends with
// token n's sum, which it finishes and leaves in LDS, from where the workgroup stores 32 bytes of a row at a time. The lanes of
// a channel are those of equal bits 2 and 3: the steps over bits 5 and 4 are swaps of two registers' halves and an add; where a
// lane has one state the states are swapped ahead of the first step, whose products then are its sum (378 us without that).
//
// Bound by the vector units: 15,360 tokens in 4 sequences x 4,096 channels x 16 states 355 us (508 MB, 1.4 TB/s), 9.1
// instructions for a token in a wave, the units busy 87 % of the time. Few tokens take the longest sequence's own chain (512 x
// 4,096 24 us, 4,096 147), and a start of 5 us again where the workgroups, three to a CU by their LDS, do not all fit at once
// (524 tokens in 6 sequences x 2,688, 260 the longest, 22 us). Eight lanes to a channel of two states each save a sixth of
// the instructions and take 320 us in place of 356 for 16 sequences of 960, but 646 in place of 432 for 4 of 8,192 to 1,024 (both
// as first written, before the chunks and the wide rows), whose few waves then wait for each other's results. More states take more
// sums to a lane, two where d_state is up to 32 and four past that: 15,360 x 4,096 x 32 540 to 570 us (14.9 instructions a token and wave),
// x 64 1,056 to 1,071 (25.8).

template <int kCtrl>
__device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), kCtrl, 0xF, 0xF, true));
}
__device__ __forceinline__ int lane_state(int lane) { return (lane >> 4) * 4 + (lane & 3); }
__device__ __forceinline__ int lane_channel(int lane) { return (lane >> 2) & 3; }

// The sums over a channel's lanes of two registers, the first's in the lanes with a clear bit 5 (or 4), the second's in the others.
__device__ __forceinline__ float swap32_sum(float a, float b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float swap16_sum(float a, float b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// The lane of state n: the sum over its channel of token n's products, from a[i]: the products' sums over bit 5, of token i in
// the lanes with a clear bit 5, of token i + 8 in the others.
__device__ __forceinline__ float channel_sums(const float (&a)[8], int lane) {
    const bool b1 = lane & 2, b0 = lane & 1;
    float b[4], c[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = swap16_sum(a[i], a[i + 4]);
#pragma unroll
    for (int i = 0; i < 2; ++i) c[i] = (b1 ? b[i + 2] : b[i]) + dpp<0x4E>(b1 ? b[i] : b[i + 2]);    // xor 2
    return (b0 ? c[1] : c[0]) + dpp<0xB1>(b0 ? c[0] : c[1]);                                        // xor 1
}

// Rows t0 .. end - 1 of a bf16 tensor of row stride ld behind a buffer descriptor: offsets from row t0, rows past the end read
// as zeros and are not written. Offsets of up to 80 rows stay within 31 bits for ld <= kMaxScanLd.
constexpr uint32_t kPastRow = 0x80000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_from(const uint16_t* p, int64_t ld, int64_t t0, int64_t end) {
    const int64_t bytes = (end - t0) * ld * 2;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p + t0 * ld), (short)0, (int)min(bytes, (int64_t)0x7fffffff), 0x00020000);
}

constexpr int kScanWaves = 4, kScanChannels = 4 * kScanWaves;   // channels of a workgroup

// kMode 0: the whole of a sequence. Of a sequence cut into chunks of a.chunk tokens: kMode 1 leaves each
// chunk's end state from zero (the first chunk's: from the initial state, which it also copies) and its sum of dt
// in the workspace, kMode 2 forms the state entering its chunk from those and does the rest.
template <int R, int kMode>
__global__ __launch_bounds__(kScanWaves * 64) void scan_prefill_kernel(const ScanPrefillArgs a) {
    constexpr int kBlock = R == 1 ? 64 : R == 2 ? 32 : 16;      // tokens staged at a time
    constexpr int kTiles = kBlock / 16, kRowsN = 16 * R;
    constexpr bool kOut = kMode != 1;
    __shared__ __attribute__((aligned(16))) float s_bc[2][2][kRowsN][kBlock + 4];   // odd multiples of 16 bytes a row
    __shared__ __attribute__((aligned(16))) float s_dt[2][2][kScanChannels][kBlock + 4];   // dt and dt u
    __shared__ uint32_t s_uz[kOut ? 2 : 1][kScanChannels][kBlock + 4];                      // u and z
    __shared__ __attribute__((aligned(8))) uint16_t s_y[kOut ? 2 : 1][kBlock][kScanChannels + 4];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, l16 = lane_state(lane), chan = lane_channel(lane);
    // Units of four workgroups, whose channels share 128-byte lines, follow one another on one XCD (block b runs
    // on XCD b % 8): the lines come from memory once. The last units, past the sequences, zero the rows behind them.
    const int lines = (a.dim + 4 * kScanChannels - 1) / (4 * kScanChannels);
    const int64_t j = blockIdx.x >> 3;
    const int64_t unit = (j >> 2) * 8 + (blockIdx.x & 7);
    const int64_t sc = unit / lines;                            // sequence, and chunk of it
    const int chunks = kMode == 0 ? 1 : a.n_chunks;
    const int seq = (int)(sc / chunks), chunk = (int)(sc % chunks);
    const int ch0 = ((int)(unit % lines) * 4 + (int)(j & 3)) * kScanChannels;
    if (seq > a.n_seqs || ch0 >= a.dim) return;
    const int ch = ch0 + wave * 4 + chan;
    const bool on = ch < a.dim;
    const int chc = on ? ch : a.dim - 1;
    if (seq == a.n_seqs) {
        if constexpr (kOut) {
            if (chunk == 0)
                for (int64_t i = (a.n_seqs > 0 ? a.cu_seqlens[a.n_seqs] : 0) + l16; i < a.n_tokens; i += 16)
                    if (on) a.out[i * a.ld_out + ch] = 0;
        }
        return;
    }
    const int64_t first = a.cu_seqlens[seq], last = a.cu_seqlens[seq + 1];
    const int64_t beg = kMode == 0 ? first : first + (int64_t)chunk * a.chunk;
    const int64_t end = kMode == 0 ? last : min(last, beg + a.chunk);
    if (kMode != 0 && beg >= end && chunk > 0) return;
    const int slot = a.slot_idx[seq];
    const bool held = has_slot(slot, a.n_slots);
    const int64_t state0 = ((int64_t)(held ? slot : 0) * a.dim + chc) * a.d_state;

    float A2[R], h[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int n = l16 + 16 * r;
        const bool in = n < a.d_state;
        A2[r] = in ? decay_rate(a.A_log[(int64_t)chc * a.d_state + n]) : 0.f;
        h[r] = 0.f;
        if (in && (kMode == 0 || (kMode == 1 && chunk == 0)) && held && a.has_initial[seq] != 0)
            h[r] = a.pool_bf16 ? bf16_to_f32(a.pool_bf16[state0 + n]) : a.pool[state0 + n];
    }
    // workspace: per sequence and chunk boundary a state (entry 0: the initial one), per chunk the sum of dt
    auto ws_state = [&](int c) { return a.ws_state + (((int64_t)seq * (a.n_chunks + 1) + c) * a.dim + chc) * a.d_state; };
    if constexpr (kMode == 1) {
        if (chunk == 0 && on)
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (l16 + 16 * r < a.d_state) ws_state(0)[l16 + 16 * r] = h[r];
    }
    if constexpr (kMode == 2) {
        // entry 1 holds the state behind the first chunk, the later ones what their chunk adds; eight at a time, so that the
        // loads do not wait for each other
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (l16 + 16 * r < a.d_state) h[r] = ws_state(min(chunk, 1))[l16 + 16 * r];
        for (int c0 = 2; c0 <= chunk; c0 += 8) {
            float keep[8], add[R][8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = min(c0 + i, chunk);
                keep[i] = a.ws_dt[((int64_t)seq * a.n_chunks + c - 1) * a.dim + chc];
#pragma unroll
                for (int r = 0; r < R; ++r) add[r][i] = l16 + 16 * r < a.d_state ? ws_state(c)[l16 + 16 * r] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c0 + i <= chunk)
#pragma unroll
                    for (int r = 0; r < R; ++r) h[r] = fmaf(__builtin_amdgcn_exp2f(keep[i] * A2[r]), h[r], add[r][i]);
        }
    }
    const float Dc = a.D ? a.D[chc] : 0.f;

    // A block's loads: thread (token lt, quad lq) takes four channels' u, dt and z of a token, 8 bytes of a row of which the
    // workgroup takes 32, and four states' B and C of token tb, at offsets from the block's first token that stay the same; a
    // block's rows end where the sequence does (zeros past that).
    constexpr int kQuads = kRowsN / 4;
    const int lt = t >> 2, lq = t & 3, tb = t / kQuads, qb = t % kQuads;
    const bool in = ch0 + 4 * lq < a.dim && lt < kBlock, bin = 4 * qb < a.d_state;
    auto offset = [](bool v, int row, int64_t ld, int col) { return v ? (uint32_t)(row * (int)ld + col) * 2 : kPastRow; };
    const uint32_t uoff = offset(in, lt, a.ld_u, ch0 + 4 * lq), doff = offset(in, lt, a.ld_dt, ch0 + 4 * lq), zoff = offset(in, lt, a.ld_z, ch0 + 4 * lq),
                   ooff = offset(in, lt, a.ld_out, ch0 + 4 * lq), boff = offset(bin, tb, a.ld_b, 4 * qb), coff = offset(bin, tb, a.ld_c, 4 * qb);
    float bias[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) bias[c] = a.dt_bias && in ? a.dt_bias[ch0 + 4 * lq + c] : 0.f;
    typedef uint32_t v2u __attribute__((ext_vector_type(2)));
    v2u ru{}, rd{}, rz{}, rb{}, rc{};
    auto load = [&](int64_t t0) {
        ru = __builtin_amdgcn_raw_buffer_load_b64(rows_from(a.u, a.ld_u, t0, end), uoff, 0, 0);
        rd = __builtin_amdgcn_raw_buffer_load_b64(rows_from(a.dt, a.ld_dt, t0, end), doff, 0, 0);
        rb = __builtin_amdgcn_raw_buffer_load_b64(rows_from(a.B, a.ld_b, t0, end), boff, 0, 0);
        if constexpr (kOut) {
            rc = __builtin_amdgcn_raw_buffer_load_b64(rows_from(a.C, a.ld_c, t0, end), coff, 0, 0);
            if (a.z) rz = __builtin_amdgcn_raw_buffer_load_b64(rows_from(a.z, a.ld_z, t0, end), zoff, 0, 0);
        }
    };
    auto half = [](const v2u& v, int c) { return c & 1 ? v[c >> 1] >> 16 : v[c >> 1] & 0xffffu; };
    // a block's outputs, whole rows of the workgroup, once everyone has passed the barrier behind it
    auto store = [&](int64_t t0, int buf) {
        if (lt < kBlock)
            __builtin_amdgcn_raw_buffer_store_b64(*reinterpret_cast<const v2u*>(&s_y[buf][lt][4 * lq]), rows_from(a.out, a.ld_out, t0, end), ooff, 0, 0);
    };
    float dt_sum[4] = {0.f, 0.f, 0.f, 0.f};
    if (beg < end) load(beg);
    int buf = 0;
    for (int64_t t0 = beg; t0 < end; t0 += kBlock) {
        // Past the sequence's end (and d_state) B is zero and dt too: the state stays.
        const int left = (int)min(end - t0, (int64_t)kBlock);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s_bc[buf][0][4 * qb + j][tb] = bf16_to_f32(half(rb, j));
            if (kOut) s_bc[buf][1][4 * qb + j][tb] = bf16_to_f32(half(rc, j));
        }
        if (lt < kBlock)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float d = lt < left ? softplus_poly(bf16_to_f32(half(rd, c)) + bias[c]) : 0.f;
                s_dt[buf][0][4 * lq + c][lt] = d;
                s_dt[buf][1][4 * lq + c][lt] = d * bf16_to_f32(half(ru, c));
                if (kOut) s_uz[buf][4 * lq + c][lt] = half(ru, c) | half(rz, c) << 16;
                if (kMode == 1) dt_sum[c] += d;
            }
        __syncthreads();     // this block is in LDS, and everyone is done with the one before the last
        if (t0 + kBlock < end) load(t0 + kBlock);
        if (kOut && t0 > beg) store(t0 - kBlock, buf ^ 1);
        auto tile = [&](int i) {
            v4f dts[2][4], bc[kOut ? 2 : 1][R][4], cs[2][2];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
#pragma unroll
                for (int m = 0; m < 2; ++m) dts[m][k] = *reinterpret_cast<const v4f*>(&s_dt[buf][m][4 * wave + chan][16 * i + 4 * k]);
#pragma unroll
                for (int m = 0; m < (kOut && R > 1 ? 2 : 1); ++m)
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        bc[m][r][k] = *reinterpret_cast<const v4f*>(&s_bc[buf][m][l16 + 16 * r][16 * i + 4 * k]);
            }
            if constexpr (kOut && R == 1)
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        cs[m][k] = *reinterpret_cast<const v4f*>(&s_bc[buf][1][(l16 & 7) + 8 * m][16 * i + (lane & 32) / 4 + 4 * k]);
            float p[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float e = __builtin_amdgcn_exp2f(dts[0][k >> 2][k & 3] * A2[r]);
                    h[r] = fmaf(e, h[r], dts[1][k >> 2][k & 3] * bc[0][r][k >> 2][k & 3]);
                    if constexpr (kOut && R == 1) p[k] = h[0];
                    else if constexpr (kOut) p[k] = r == 0 ? h[r] * bc[1][r][k >> 2][k & 3] : fmaf(h[r], bc[1][r][k >> 2][k & 3], p[k]);
                }
            }
            if constexpr (kOut) {
                float a8[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if constexpr (R == 1) {
                        // the states change lanes before their products, C read as they lie then: 24 instructions in place of 32
                        const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(p[k]), __float_as_uint(p[k + 8]), false, false);
                        a8[k] = fmaf(__uint_as_float(x[1]), cs[1][k >> 2][k & 3], __uint_as_float(x[0]) * cs[0][k >> 2][k & 3]);
                    } else {
                        a8[k] = swap32_sum(p[k], p[k + 8]);
                    }
                }
                const uint32_t uz = s_uz[buf][4 * wave + chan][16 * i + l16];
                float y = fmaf(Dc, bf16_to_f32(uz & 0xffffu), channel_sums(a8, lane));
                if (a.z) y *= silu(bf16_to_f32(uz >> 16));
                s_y[buf][16 * i + l16][4 * wave + chan] = (uint16_t)f32_to_bf16(y);
            }
        };
        if (left == kBlock) {        // no branch between the tiles: their latencies overlap
#pragma unroll
            for (int i = 0; i < kTiles; ++i) tile(i);
        } else {
#pragma unroll
            for (int i = 0; i < kTiles; ++i)
                if (16 * i < left) tile(i);
        }
        buf ^= 1;
    }
    if (kOut && beg < end) {
        __syncthreads();
        store(beg + (end - 1 - beg) / kBlock * kBlock, buf ^ 1);
    }
    if constexpr (kMode == 1) {
        if (beg < end && on) {
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (l16 + 16 * r < a.d_state) ws_state(chunk + 1)[l16 + 16 * r] = h[r];
        }
        if (beg < end) {         // the chunk's sum of dt of each channel: over the tokens' threads of the workgroup
            __syncthreads();     // everyone is done with the last block
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (lt < kBlock) s_dt[0][0][4 * lq + c][lt] = dt_sum[c];
            __syncthreads();
            float sum = 0.f;
            for (int i = l16; i < kBlock; i += 16) sum += s_dt[0][0][4 * wave + chan][i];
            sum = swap32_sum(sum, sum);
            sum = swap16_sum(sum, sum);
            sum += dpp<0x4E>(sum);
            sum += dpp<0xB1>(sum);
            if (l16 == 0 && on) a.ws_dt[((int64_t)seq * a.n_chunks + chunk) * a.dim + ch] = sum;
        }
    } else {
        if (end == last && held && on)      // the sequence's last chunk (an empty sequence's only one)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int n = l16 + 16 * r;
                if (n >= a.d_state) continue;
                if (a.pool_bf16) a.pool_bf16[state0 + n] = (uint16_t)f32_to_bf16(h[r]);
                else a.pool[state0 + n] = h[r];
            }
    }
}

template <int R>
static void launch_scan_r(const ScanPrefillArgs& a, hipStream_t st) {
    const int64_t lines = (a.dim + 4 * kScanChannels - 1) / (4 * kScanChannels);
    auto grid = [&](int64_t per_seq) { return dim3((unsigned)(((a.n_seqs + 1) * per_seq * lines + 7) / 8 * 32)); };
    if (a.n_chunks <= 1) {
        scan_prefill_kernel<R, 0><<<grid(1), dim3(kScanWaves * 64), 0, st>>>(a);
        return;
    }
    scan_prefill_kernel<R, 1><<<grid(a.n_chunks), dim3(kScanWaves * 64), 0, st>>>(a);
    scan_prefill_kernel<R, 2><<<grid(a.n_chunks), dim3(kScanWaves * 64), 0, st>>>(a);
}

// Where sequences x channels do not fill the chip, sequences are cut into chunks of at least 128 tokens, up to 64 of them, for
// about 1,024 workgroups, at the price of forming the decays twice. us, whole and cut: 4,096 tokens x 4,096 channels (4
// chunks) 155 and 166, x 2,048 (8) 151 and 88, x 1,024 152 and 50, x 64 149 and 18; 15,360 x 512 547 and 94; 256 x 256
// (2 of 128 tokens) 13.5 and 14.4, 1,024 x 1,024 41 and 19. The host knows the sequences' number and not their lengths: one of
// 15,000 tokens beside 31 of 11, x 4,096 channels, is not cut and takes its own chain, 520 us.
ScanSplit scan_split(int64_t dim, int64_t n_tokens, int64_t n_seqs) {
    const ScanSplit whole{1, n_tokens > 0 ? n_tokens : 1};
    const int64_t groups = (n_seqs > 0 ? n_seqs : 1) * ((dim + 15) / 16);
    const int64_t s = 1024 / groups < 64 ? 1024 / groups : 64;
    if (s < 6) return whole;
    int64_t chunk = ((n_tokens + s - 1) / s + 63) / 64 * 64;
    chunk = chunk < 128 ? 128 : chunk;
    const int64_t n = (n_tokens + chunk - 1) / chunk;
    return n < 4 ? whole : ScanSplit{n, chunk};
}

size_t scan_ws_bytes(int64_t dim, int32_t d_state, int64_t n_tokens, int64_t n_seqs) {
    const ScanSplit s = scan_split(dim, n_tokens, n_seqs);
    if (s.n_chunks <= 1) return 0;
    return align_up((size_t)n_seqs * (s.n_chunks + 1) * dim * d_state * 4, 256) + align_up((size_t)n_seqs * s.n_chunks * dim * 4, 256);
}

nhm_status launch_scan_prefill(ScanPrefillArgs a, void* ws, hipStream_t st) {
    const ScanSplit s = scan_split(a.dim, a.n_tokens, a.n_seqs);
    a.n_chunks = (int)s.n_chunks;
    a.chunk = s.chunk;
    a.ws_state = static_cast<float*>(ws);
    a.ws_dt = a.ws_state ? reinterpret_cast<float*>(static_cast<char*>(ws) + align_up((size_t)a.n_seqs * (s.n_chunks + 1) * a.dim * a.d_state * 4, 256)) : nullptr;
    if (a.d_state <= 16) launch_scan_r<1>(a, st);
    else if (a.d_state <= 32) launch_scan_r<2>(a, st);
    else launch_scan_r<4>(a, st);
    count_launch(Kern::kScanPrefill, a.n_tokens);
    return check_launch("selective scan prefill");
}

// ---------------------------------------------------------------- scan of single tokens
//
// Four states of a channel to a lane, 16 bytes of an f32 pool's row; kLanes lanes are a channel. Bound by the
// states' bytes, read and written once, where there are many rows; 8 rows x 4,096 channels x 16 states take 3.9 us, a chain of loads.
template <int kLanes>
__global__ __launch_bounds__(256) void scan_decode_kernel(const ScanDecodeArgs a) {
    constexpr int kPer = 256 / kLanes;      // channels of a workgroup
    const int t = threadIdx.x, s4 = (t % kLanes) * 4, ch = blockIdx.x * kPer + t / kLanes;
    const int64_t row = blockIdx.y;
    if (ch >= a.dim) return;                // whole groups of lanes
    const int slot = a.slot_idx[row];
    if (!has_slot(slot, a.n_slots)) {
        if (s4 == 0) a.out[row * a.ld_out + ch] = 0;
        return;
    }
    const bool in = s4 < a.d_state;
    const int64_t at = ((int64_t)slot * a.dim + ch) * a.d_state + (in ? s4 : 0);
    float h[4];
    if (a.pool_bf16) {
        const uint2 v = *reinterpret_cast<const uint2*>(a.pool_bf16 + at);
        h[0] = bf16_to_f32(v.x & 0xffffu); h[1] = bf16_to_f32(v.x >> 16);
        h[2] = bf16_to_f32(v.y & 0xffffu); h[3] = bf16_to_f32(v.y >> 16);
    } else {
        const v4f v = *reinterpret_cast<const v4f*>(a.pool + at);
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = v[k];
    }
    const v4f al = *reinterpret_cast<const v4f*>(a.A_log + (int64_t)ch * a.d_state + (in ? s4 : 0));
    float B[4], C[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        B[k] = bf16_to_f32(a.B[row * a.ld_b + (in ? s4 + k : 0)]);
        C[k] = bf16_to_f32(a.C[row * a.ld_c + (in ? s4 + k : 0)]);
    }
    const float u = bf16_to_f32(a.u[row * a.ld_u + ch]);
    const float dt = softplus_poly(bf16_to_f32(a.dt[row * a.ld_dt + ch]) + (a.dt_bias ? a.dt_bias[ch] : 0.f));
    float y = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        h[k] = fmaf(__builtin_amdgcn_exp2f(dt * decay_rate(al[k])), h[k], dt * u * B[k]);
        y = fmaf(h[k], C[k], y);
    }
    if (in) {
        if (a.pool_bf16) *reinterpret_cast<uint2*>(a.pool_bf16 + at) = make_uint2(f32x2_to_bf16x2(h[0], h[1]), f32x2_to_bf16x2(h[2], h[3]));
        else *reinterpret_cast<v4f*>(a.pool + at) = v4f{h[0], h[1], h[2], h[3]};
    } else {
        y = 0.f;
    }
    if constexpr (kLanes >= 2) y += dpp<0xB1>(y);
    if constexpr (kLanes >= 4) y += dpp<0x4E>(y);
    if constexpr (kLanes >= 8) y += dpp<0x141>(y);
    if constexpr (kLanes >= 16) y += dpp<0x128>(y);
    if (s4 == 0) {
        y = fmaf(a.D ? a.D[ch] : 0.f, u, y);
        if (a.z) y *= silu(bf16_to_f32(a.z[row * a.ld_z + ch]));
        a.out[row * a.ld_out + ch] = (uint16_t)f32_to_bf16(y);
    }
}

nhm_status launch_scan_decode(const ScanDecodeArgs& g, int32_t batch, hipStream_t st) {
    auto go = [&](auto lanes) {
        constexpr int kLanes = decltype(lanes)::value, kPer = 256 / kLanes;
        for (int32_t r0 = 0; r0 < batch; r0 += 65535) {      // the grid's y extent
            ScanDecodeArgs a = g;
            a.slot_idx += r0;
            a.u += r0 * a.ld_u; a.dt += r0 * a.ld_dt; a.B += r0 * a.ld_b; a.C += r0 * a.ld_c; a.out += r0 * a.ld_out;
            if (a.z) a.z += r0 * a.ld_z;
            const unsigned rows = (unsigned)(batch - r0 < 65535 ? batch - r0 : 65535);
            scan_decode_kernel<kLanes><<<dim3((unsigned)((a.dim + kPer - 1) / kPer), rows), dim3(256), 0, st>>>(a);
        }
    };
    if (g.d_state <= 4) go(std::integral_constant<int, 1>());
    else if (g.d_state <= 8) go(std::integral_constant<int, 2>());
    else if (g.d_state <= 16) go(std::integral_constant<int, 4>());
    else if (g.d_state <= 32) go(std::integral_constant<int, 8>());
    else go(std::integral_constant<int, 16>());
    count_launch(Kern::kScanDecode, batch);
    return check_launch("selective scan decode");
}

// ---------------------------------------------------------------- convolution
//
// A thread takes eight channels. Bound by bytes: x read and u written once (15,360 tokens x 4,096 44 to 46 us, 252 MB at 5.4 TB/s, and
// 16 MB more: each thread also writes the zero row that a window may be taken from to private memory). 1,920 sequences of 8 tokens, whose
// tokens follow one another in a thread, 95 us for 346 MB. 8 single tokens 2.9 us, a chain of loads.

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]), f32x2_to_bf16x2(f[4], f[5]), f32x2_to_bf16x2(f[6], f[7]));
}

// This thread's taps and bias.
template <int W>
struct Taps {
    float w[W][8], b[8];
    __device__ __forceinline__ void load(const ConvArgs& a, int c) {
        uint32_t raw[4 * W];                  // 8 channels x W taps in memory order
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const uint4 v = reinterpret_cast<const uint4*>(a.w + (int64_t)c * W)[i];
            raw[4 * i] = v.x; raw[4 * i + 1] = v.y; raw[4 * i + 2] = v.z; raw[4 * i + 3] = v.w;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int k = 0; k < W; ++k) {
                const int e = j * W + k;
                w[k][j] = bf16_to_f32(e & 1 ? raw[e >> 1] >> 16 : raw[e >> 1] & 0xffffu);
            }
        if (a.b) unpack8(*reinterpret_cast<const uint4*>(a.b + c), b);
        else
#pragma unroll
            for (int j = 0; j < 8; ++j) b[j] = 0.f;
    }
    // rows: the W rows that end with the token, oldest first
    __device__ __forceinline__ uint4 apply(const uint4 (&rows)[W], bool act) const {
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = b[j];
#pragma unroll
        for (int k = 0; k < W; ++k) {
            float x[8];
            unpack8(rows[k], x);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = fmaf(w[k][j], x[j], y[j]);
        }
        if (act)
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = silu(y[j]);
        return pack8(y);
    }
};

constexpr int kConvTokens = 8;      // tokens of a wave's run

// A wave takes 512 channels of a run of tokens. The first W - 1 tokens of a sequence need its window, which the
// call replaces: those tokens and the new window are the business of the wave whose run holds the sequence's
// first token (an empty sequence's place), so that one thread reads and writes a window's channels. A run's
// first tokens that belong to an earlier run's sequence head are left to that run's wave.
template <int W>
__global__ __launch_bounds__(256) void conv_prefill_kernel(const ConvArgs a) {
    constexpr int H = W - 1;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const unsigned across = (a.dim + 511) / 512;             // workgroups over the channels
    const int64_t t0 = ((int64_t)(blockIdx.x / across) * 4 + wave) * kConvTokens;
    const int c = (blockIdx.x % across * 64 + lane) * 8;
    const int n = a.n_seqs;
    if (t0 > a.n_tokens) return;
    // s: sequences that start before t0; the last of them (with a token there) is the one t0 may lie in
    int s = 0;
    for (int i0 = 0; i0 < n; i0 += 64) {
        const bool before = i0 + lane < n && a.cu_seqlens[i0 + lane] < t0;
        const int got = __popcll(__ballot(before));
        s += got;
        if (got < 64) break;
    }
    if (c >= a.dim) return;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    Taps<W> taps;
    taps.load(a, c);
    const int64_t stop = n > 0 ? a.cu_seqlens[n] : 0;
    const int64_t run_end = min(t0 + kConvTokens, a.n_tokens);
    auto row = [&](int64_t t) { return *reinterpret_cast<const uint4*>(a.x + t * a.ld_x + c); };
    auto put = [&](int64_t t, uint4 v) { *reinterpret_cast<uint4*>(a.out + t * a.ld_out + c) = v; };

    int64_t t = t0;
    if (s > 0) {     // the sequence that goes on in this run, from its W-th token on
        const int64_t first = a.cu_seqlens[s - 1], next = a.cu_seqlens[s];
        t = max(t0, first + H);
        const int64_t e = min(run_end, next);
        if (t < e) {
            uint4 x[kConvTokens + H];
#pragma unroll
            for (int i = 0; i < kConvTokens + H; ++i) x[i] = t + i - H < e ? row(t + i - H) : zero;
#pragma unroll
            for (int i = 0; i < kConvTokens; ++i) {
                uint4 r[W];
#pragma unroll
                for (int k = 0; k < W; ++k) r[k] = x[i + k];
                if (t + i < e) put(t + i, taps.apply(r, a.silu));
            }
        }
    }
    // sequences that start in this run
    for (; s < n; ++s) {
        const int64_t first = a.cu_seqlens[s], next = a.cu_seqlens[s + 1];
        if (first >= t0 + kConvTokens) break;
        const int slot = a.slot_idx[s];
        const bool held = has_slot(slot, a.n_slots);
        uint16_t* const win = a.pool + (int64_t)(held ? slot : 0) * H * a.dim + c;
        uint4 r[W];
#pragma unroll
        for (int k = 0; k < H; ++k)
            r[k] = held && a.has_initial[s] != 0 ? *reinterpret_cast<const uint4*>(win + (int64_t)k * a.dim) : zero;
        // its tokens of this run, and its first W - 1 wherever they lie
        const int64_t e = min(next, max(run_end, first + H));
        const int64_t tail = next - H;          // the new window's rows: from the token tail on
        uint4 keep[H];
#pragma unroll
        for (int k = 0; k < H; ++k) {
            // row k of the window behind the sequence: token tail + k, or an older row of the old window
            const int64_t p = tail + k - first;
            uint4 v = zero;
#pragma unroll
            for (int o = 0; o < H; ++o)
                if (p < 0 && p + H == o) v = r[o];
            if (p >= 0) v = row(tail + k);
            keep[k] = v;
        }
        for (int64_t i = first; i < e; ++i) {
            r[H] = row(i);
            put(i, taps.apply(r, a.silu));
#pragma unroll
            for (int k = 0; k < H; ++k) r[k] = r[k + 1];
        }
        if (held)
#pragma unroll
            for (int k = 0; k < H; ++k) *reinterpret_cast<uint4*>(win + (int64_t)k * a.dim) = keep[k];
    }
    // rows behind the last sequence
    for (int64_t i = max(t0, stop); i < run_end; ++i) put(i, zero);
}

template <int W>
__global__ __launch_bounds__(64) void conv_decode_kernel(const ConvArgs a) {
    constexpr int H = W - 1;
    const int c = (blockIdx.x * 64 + threadIdx.x) * 8;
    const int64_t t = blockIdx.y;
    if (c >= a.dim) return;
    const int slot = a.slot_idx[t];
    uint16_t* const o = a.out + t * a.ld_out + c;
    if (!has_slot(slot, a.n_slots)) {
        *reinterpret_cast<uint4*>(o) = make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    uint16_t* const win = a.pool + (int64_t)slot * H * a.dim + c;
    uint4 r[W];
#pragma unroll
    for (int k = 0; k < H; ++k) r[k] = *reinterpret_cast<const uint4*>(win + (int64_t)k * a.dim);
    r[H] = *reinterpret_cast<const uint4*>(a.x + t * a.ld_x + c);
    Taps<W> taps;
    taps.load(a, c);
    *reinterpret_cast<uint4*>(o) = taps.apply(r, a.silu);
#pragma unroll
    for (int k = 0; k < H; ++k) *reinterpret_cast<uint4*>(win + (int64_t)k * a.dim) = r[k + 1];
}

nhm_status launch_conv_prefill(const ConvArgs& a, int32_t width, hipStream_t st) {
    // one run more than the tokens fill: empty sequences at the end have their place there
    const int64_t runs = a.n_tokens / kConvTokens + 1, per = (runs + 3) / 4;
    const dim3 grid((unsigned)((a.dim + 511) / 512 * per));
    if (width == 2) conv_prefill_kernel<2><<<grid, dim3(256), 0, st>>>(a);
    else if (width == 3) conv_prefill_kernel<3><<<grid, dim3(256), 0, st>>>(a);
    else conv_prefill_kernel<4><<<grid, dim3(256), 0, st>>>(a);
    count_launch(Kern::kConvPrefill, a.n_tokens);
    return check_launch("causal conv prefill");
}

nhm_status launch_conv_decode(const ConvArgs& g, int32_t width, int32_t batch, hipStream_t st) {
    for (int32_t r0 = 0; r0 < batch; r0 += 65535) {      // the grid's y extent
        ConvArgs a = g;
        a.slot_idx += r0;
        a.x += r0 * a.ld_x;
        a.out += r0 * a.ld_out;
        const dim3 grid((unsigned)((a.dim + 511) / 512), (unsigned)(batch - r0 < 65535 ? batch - r0 : 65535));
        if (width == 2) conv_decode_kernel<2><<<grid, dim3(64), 0, st>>>(a);
        else if (width == 3) conv_decode_kernel<3><<<grid, dim3(64), 0, st>>>(a);
        else conv_decode_kernel<4><<<grid, dim3(64), 0, st>>>(a);
    }
    count_launch(Kern::kConvDecode, batch);
    return check_launch("causal conv decode");
}

}  // namespace nhm
