// Host-side declarations shared by the libnhm translation units (not part of the ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/nhm.h"
#include "../../include/nhm_serving.h"

namespace nhm {

// Records a failure detail for nhm_last_error() and returns the status.
nhm_status fail(nhm_status s, const char* fmt, ...);

// Returns NHM_ERR_HIP (with the runtime's message) if the last launch failed.
nhm_status check_launch(const char* what);

// Empties the calling thread's failure detail (nhm_last_error), as every entry point does first.
void clear_error();

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Path-taken counters (nhm_dispatch_counters): one per kernel the library launches, counting
// launches and the rows (tokens, or chunks for the scan kernels) they covered. Host-side,
// atomic; a launch recorded into a HIP graph counts once, at capture.
enum class Kern : int {
    kQuantVec8, kQuantScalar, kDequantChannel, kGemv, kRing192x128, kRing192x128Exact, kRing256x128,
    kRing256x128Exact, kRing256x256, kRing256x256Exact, kPanel64x128, kPanel64x128Exact, kTile128,
    kTile128Exact, kSplitkReduce, kDecodeSsm, kGnormQuant, kClear, kConvFwd, kSsdState, kSsdPass, kSsdOut,
    kLoraDown, kLoraRows, kLoraRowsExact, kBeamRows, kBeamPick, kBeamReorder, kBatchPlan, kCount
};
void count_launch(Kern k, int64_t rows);

// ---- host checks and the projection shared by the entry points (api.hip)
nhm_status check_geometry(const nhm_geometry* g);
void fill_layout(const nhm_geometry* g, nhm_layout* l);
// Every check of nhm_fp8_linear_ex's arguments; need: workspace bytes the call cannot do without.
nhm_status linear_check(const void* a, nhm_dtype a_type, int64_t m, int64_t ld_a, const nhm_fp8_weight* w,
                        const void* out, nhm_dtype out_type, int64_t ld_out, const void* ws, size_t ws_bytes,
                        size_t need);
// The weight-streaming GEMV serves m <= 16 (k up to 16384, weights under 2 GiB: its buffer
// descriptors take 32-bit offsets); the tiled GEMM the rest.
inline bool use_gemv(int64_t m, int64_t n, int64_t k) { return m <= 16 && k <= 16384 && n * k < (int64_t(1) << 31); }
// Index step of the weight scale: per channel (w_scale[n]) or one scale for every channel.
inline int ws_step(const nhm_fp8_weight& w) { return w.w_scale_per_tensor ? 0 : 1; }
// bytes of the e4m3 copy of a bf16 activation
size_t linear_codes_ws(int64_t m, int64_t k, nhm_dtype t);
// One projection on an e4m3 activation [m, lda]; out_f32 non-null: f32 output instead of out.
// part / part_bytes: scratch for the GEMM's split-k partials (nullptr: no split).
// exact: every product summed in f32 on the tiled path too (the GEMV always is).
// out_q: also the e4m3 codes of the bf16 output under *q_scale (GEMV path only; callers of the
// tiled path quantize its output themselves).
nhm_status project(const uint8_t* a, int64_t lda, int64_t m, const nhm_fp8_weight& w, uint16_t* out, int64_t ld_out,
                   hipStream_t st, float* out_f32 = nullptr, float* part = nullptr, size_t part_bytes = 0,
                   bool exact = false, uint8_t* out_q = nullptr, int64_t ld_q = 0, const float* q_scale = nullptr);

// The mixer's projections done by the caller: nhm_mixer_decode and nhm_mixer_prefill with a hook in place
// of a projection call it where they would quantize and project themselves. extra: workspace bytes
// past the call's own, which the hooks get as `ws`.
struct ProjectionHooks {
    // block input [m, hidden] bf16 -> its codes q and the in_proj output zx; clear_n words at clear (if any) zeroed
    nhm_status (*in_proj)(const ProjectionHooks& h, const uint16_t* hidden, int64_t m, uint8_t* q, uint16_t* zx,
                          uint32_t* clear, int clear_n, char* ws, hipStream_t st) = nullptr;
    // norm output [m, d_inner] bf16 and its codes q -> block output
    nhm_status (*out_proj)(const ProjectionHooks& h, const uint16_t* norm, const uint8_t* q, int64_t m, uint16_t* out,
                           char* ws, hipStream_t st) = nullptr;
    size_t extra = 0;
    const nhm_mixer_params* p = nullptr;
    const nhm_lora* lora_in = nullptr;
    const nhm_lora* lora_out = nullptr;
    const int32_t* row_adapter = nullptr;
    bool decode = false;
};
nhm_status mixer_decode_call(const nhm_mixer_params* p, const uint16_t* hidden, const uint8_t* hidden_q, int32_t batch,
                             const int32_t* slot_idx, void* ssm_pool, nhm_dtype ssm_type, uint16_t* conv_pool,
                             int32_t n_slots, uint16_t* out, uint8_t* out_q, const float* out_q_scale, void* ws,
                             size_t ws_bytes, void* stream, bool noalloc, const ProjectionHooks* hooks = nullptr);
nhm_status mixer_prefill_call(const nhm_mixer_params* p, const uint16_t* hidden, int64_t n_tokens,
                              const int32_t* cu_seqlens, int32_t n_seqs, const int32_t* slot_idx,
                              const int32_t* has_initial, int32_t chunk, void* ssm_pool, nhm_dtype ssm_type,
                              uint16_t* conv_pool, int32_t n_slots, uint16_t* out, void* ws, size_t ws_bytes,
                              void* stream, const ProjectionHooks* hooks = nullptr);

// ---- activation quant (quant.hip)
void launch_quantize(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld_x, const float* scale,
                     uint8_t* q, int64_t ld_q, hipStream_t st);

// n 32-bit words set to zero (quant.hip)
void launch_clear(uint32_t* p, int n, hipStream_t st);

// per-channel e4m3 -> bf16 weight dequant (quant.hip); cols a multiple of 16, 16-byte rows
void launch_dequant_channel(const uint8_t* w, int64_t rows, int64_t cols, int64_t ld_w, const float* w_scale,
                            uint16_t* out, int64_t ld_out, hipStream_t st);

// ---- weight-streaming GEMV for m <= 16 (gemv.hip)

// out[m, n] = bf16(sum_k a[m,k] w[n,k] * a_scale * w_scale[n]); a is e4m3 [m, lda], stored to
// out[m * ld_out + n]; with out_f32 the unrounded f32 result goes to out_f32[m * ld_out + n]
// instead. out_q (bf16 output only): also E4M3(out / *q_scale) at out_q[m * ld_q + n].
// clear (optional): clear_n 32-bit words set to zero by the launch (side work of workgroup 0).
// ws_step: 1 for a weight scale per output channel, 0 for one scale (w_scale[0]) for all.
nhm_status launch_gemv(const uint8_t* a, int64_t lda, int m, const uint8_t* w, const float* w_scale,
                       const float* a_scale, int64_t n, int64_t k, uint16_t* out, int64_t ld_out, hipStream_t st,
                       float* out_f32 = nullptr, uint8_t* out_q = nullptr, int64_t ld_q = 0,
                       const float* q_scale = nullptr, uint32_t* clear = nullptr, int clear_n = 0, int ws_step = 1);

// ---- tiled MFMA GEMM for larger m (gemm.hip)
// part (16-byte aligned, part_bytes >= gemm_part_bytes(m, n, k)): scratch for the split-k
// partials of the shapes that take a split (m <= 640 with too few ring tiles); without it
// those shapes run unsplit.
size_t gemm_part_bytes(int64_t m, int64_t n, int64_t k);
// exact: every product summed in f32 (codes converted to bf16, bf16 MFMA) instead of the e4m3
// MFMA's coarser 128-product reductions.
nhm_status launch_gemm(const uint8_t* a, int64_t lda, int64_t m, const uint8_t* w, const float* w_scale,
                       const float* a_scale, int64_t n, int64_t k, uint16_t* out, int64_t ld_out,
                       hipStream_t st, float* out_f32 = nullptr, float* part = nullptr, size_t part_bytes = 0,
                       bool exact = false, int ws_step = 1);

// ---- decode SSM state update (decode.hip)
// The kernel also runs the causal conv + SiLU of the channels it reads (the head's x, the
// group's B and C) from the pre-conv projection and the carried window, stores them to
// xbc_conv, and shifts the windows of the head's x channels; the B and C channels' windows
// (read by every head of the group) are shifted by the gated-norm kernel that follows.
struct DecodeSsmArgs {
    const int32_t* slot_idx;
    float* ssm_pool;           // f32 state pool, or nullptr with ssm_pool_bf16
    uint16_t* ssm_pool_bf16;   // bf16 state pool (widened on load, rounded on store), or nullptr
    const uint16_t* zxbcdt;    // [m, d_in_proj]
    uint16_t* xbc_conv;        // [m, conv_dim] conv + SiLU output
    uint16_t* conv_pool;       // [S, W-1, conv_dim]
    const uint16_t* conv_w;    // [conv_dim, W]
    const uint16_t* conv_b;    // [conv_dim]
    const float* A_log;
    const float* D;
    const float* dt_bias;
    uint16_t* y;               // [m, d_inner]
    int32_t n_heads, n_groups, d_in_proj, conv_dim, d_inner, xbc_off, dt_off, b_off, c_off;
    // fused gated norm (cnt != nullptr): the last of a group's head workgroups to finish also
    // computes the group's gated RMSNorm and its e4m3 codes and shifts the group's B and C conv
    // windows; cnt holds one counter per (row, group), zero at launch
    uint32_t* cnt = nullptr;
    const uint16_t* norm_w = nullptr;   // [d_inner]
    const float* out_a_scale = nullptr;
    float eps = 0.f;
    int32_t z_off = 0;
    uint16_t* norm = nullptr;           // [m, d_inner]
    uint8_t* q_out = nullptr;           // [m, d_inner]
};
nhm_status launch_decode_ssm(const DecodeSsmArgs& a, int m, hipStream_t st);

// ---- gated group RMSNorm + out_proj quant (norm.hip)
struct GnormArgs {
    int64_t T;
    int32_t n_groups, d_inner, d_in_proj, z_off;
    float eps;
    const uint16_t* y;         // [T, d_inner]
    const uint16_t* zxbcdt;    // [T, d_in_proj] (z columns)
    const uint16_t* norm_w;    // [d_inner]
    const float* out_a_scale;  // [1]
    uint16_t* norm;            // [T, d_inner] bf16 norm output (nullptr: not kept)
    uint8_t* q_out;            // [T, d_inner]
    // decode: shift the B and C channels' conv windows of each token's slot (slot_idx ==
    // nullptr: none). Row 2 takes the pre-conv value from zxbcdt.
    const int32_t* slot_idx = nullptr;
    uint16_t* conv_pool = nullptr;   // [S, W-1, conv_dim]
    int32_t conv_dim = 0, xbc_off = 0, b_off = 0, c_off = 0, d_state = 0;
    const int32_t* n_real = nullptr;   // prefill: tokens of all sequences (device); zeros from there to T
};
nhm_status launch_gnorm_quant(const GnormArgs& a, hipStream_t st);

// ---- prefill pieces (prefill.hip)
struct PrefillArgs {
    int64_t T;
    int32_t n_seqs, chunk, max_chunks, n_heads, n_groups, d_in_proj, conv_dim, d_inner;
    int32_t z_off, xbc_off, dt_off, b_off, c_off;
    float eps;
    const int32_t* cu_seqlens;
    const int32_t* slot_idx;
    const int32_t* has_initial;
    float* ssm_pool;           // f32 state pool, or nullptr with ssm_pool_bf16
    uint16_t* ssm_pool_bf16;   // bf16 state pool (widened on load, rounded on store), or nullptr
    uint16_t* conv_pool;
    const uint16_t* conv_w;
    const uint16_t* conv_b;
    const float* A_log;
    const float* D;
    const float* dt_bias;
    const uint16_t* norm_w;
    const float* out_a_scale;
    uint16_t* zxbcdt;         // [T, d_in_proj]
    uint16_t* xbc_conv;       // [T, conv_dim]
    int32_t* chunk_info;      // [max_chunks, 4]: seq, tok0, len, index in seq
    int32_t* seq_chunk0;      // [n_seqs + 1]
    float* chunk_cs;          // [max_chunks, n_heads, chunk]  cumulative log-decay
    float* chunk_dt;          // [max_chunks, n_heads, chunk]
    float* chunk_state;       // [max_chunks, n_heads, 64, 128]
    uint16_t* y;              // [T, d_inner]
    uint16_t* norm;           // [T, d_inner] (nullptr: not kept)
    uint8_t* q_out;           // [T, d_inner]
};
// conv + chunk plan in one launch, then the chunked scan and the gated norm + quant, in
// stream order.
nhm_status launch_prefill_mid(const PrefillArgs& a, hipStream_t st);

// SSD chunk kernels on the bf16 MFMA (ssd.hip): per (chunk, head) dt, cumulative
// log-decay and the chunk's own state; then, after the state pass, the outputs.
void launch_ssd_state(const PrefillArgs& a, hipStream_t st);
void launch_ssd_out(const PrefillArgs& a, hipStream_t st);

// ---- low-rank adapters (lora.hip, and the projections' epilogues in gemv.hip and gemm.hip)

// The low-rank product t = scale x A_e^T enters the second product as bf16 parts that add up to
// it: parts 0, 1 (, 2) of row i at t[(i * parts + part) * rp], rp = 32, 64 or 128, the
// first that holds the rank, zeros past it. Rows without an adapter hold nothing.
constexpr int kLoraMaxRank = 128;
inline int lora_rp(int rank) { return rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

// What a projection's epilogue needs to add t B_e^T to its f32 result before it is rounded.
struct LoraEpi {
    const uint16_t* t = nullptr;            // [m, parts, rp]
    const uint16_t* b = nullptr;            // bf16 [n_adapters, n, rank]
    const int32_t* row_adapter = nullptr;   // [m]
    int32_t n_adapters = 0, rank = 0, rp = 0, parts = 0;
};

struct LoraDownArgs {
    const uint16_t* x;         // bf16 [m, ld_x], or nullptr with x_codes
    const uint8_t* x_codes;    // e4m3 [m, ld_x], worth code * *a_scale
    int64_t ld_x, m, k;
    const float* a_scale;      // [1]
    uint8_t* q;                // non-null (bf16 input): also the codes E4M3(x / *a_scale) [m, k]
    const uint16_t* a;         // bf16 [n_adapters, rank, k]
    const float* scale;        // [n_adapters] or nullptr
    int32_t n_adapters, rank, rp, parts;
    const int32_t* row_adapter;   // [m]
    uint16_t* t;               // [m, parts, rp]
};
nhm_status launch_lora_down(const LoraDownArgs& g, hipStream_t st);

// The projections with the adapters' part (the same kernels and choices as without, no split over k).
nhm_status launch_gemv_lora(const uint8_t* a, int64_t lda, int m, const uint8_t* w, const float* w_scale,
                            const float* a_scale, int64_t n, int64_t k, uint16_t* out, int64_t ld_out, hipStream_t st,
                            float* out_f32, int ws_step, const LoraEpi& lora, uint32_t* clear = nullptr,
                            int clear_n = 0);
nhm_status launch_gemm_lora(const uint8_t* a, int64_t lda, int64_t m, const uint8_t* w, const float* w_scale,
                            const float* a_scale, int64_t n, int64_t k, uint16_t* out, int64_t ld_out, hipStream_t st,
                            float* out_f32, bool exact, int ws_step, const LoraEpi& lora);

// ---- beam search (beam.hip)
struct BeamArgs {
    const uint16_t* logits_bf16;   // [n_groups * n_beams, ld], or nullptr with logits_f32
    const float* logits_f32;
    int64_t ld, n_groups;
    int32_t n_beams;
    int64_t vocab;
    const float* cum;              // [n_groups, n_beams]
    const int32_t* finished;       // [n_groups, n_beams] or nullptr
    int32_t eos, n_cand;
    float* scores;                 // [n_groups, n_cand]
    int32_t* parents;
    int32_t* tokens;
    // workspace: per strip (a run of a row) its n_cand best entries, sum of exp(x - top) and top
    uint64_t* strip_keys;          // [rows, n_strips, n_cand]
    double* strip_sum;             // [rows, n_strips]
    float* strip_top;
    int32_t n_strips, strip_pieces;
};
size_t beam_ws_bytes(int64_t rows, int64_t vocab, int32_t n_cand);
nhm_status launch_beam_select(BeamArgs g, void* ws, hipStream_t st);

constexpr int kMaxStatePools = 64;
struct ReorderArgs {
    nhm_state_pool pools[kMaxStatePools];
    const int32_t* parents;
    const int32_t* slots;
    int32_t* new_slots;
    int32_t n_beams, n_slots;
    int64_t ssm_bytes, conv_bytes;   // of one row; multiples of 16
};
nhm_status launch_beam_reorder(const ReorderArgs& g, int64_t n_groups, int32_t n_layers, hipStream_t st);

// ---- batch plan (plan.hip)
constexpr int kMaxPlanSeqs = 8192;
struct PlanArgs {
    const int32_t* lengths;
    const int32_t* past;        // or nullptr
    const int32_t* adapters;    // or nullptr
    int32_t n_seqs;
    int64_t n_tokens;
    int32_t* cu_seqlens;
    int32_t* has_initial;
    int32_t* token_seq;         // each of the three may be nullptr
    int32_t* token_pos;
    int32_t* token_adapter;
};
nhm_status launch_batch_plan(const PlanArgs& g, hipStream_t st);

}  // namespace nhm
