/*
 * nhm_layer.h -- C ABI of libnhm's operators for a selective-scan layer in 4 bits, beside the mixer
 * of nhm.h: MXFP4 quantisation and projections, the short causal convolution and the selective
 * state space scan (a decay for each channel and state) for prompts and for single tokens, and the scoring of
 * tokens from logits. They run on the mixer's batches: packed sequences by cu_seqlens, states in pools by
 * slot (nhm_batch_plan of nhm_serving.h makes the index tensors).
 *
 * The conventions of nhm.h hold for every call: caller-owned memory, host validation before
 * anything is enqueued, a status and nhm_last_error() instead of exceptions, work enqueued on
 * the given stream only, no synchronization, no allocation, legal inside HIP graph capture.
 * The stream must belong to the current device, and so must the tensors. Two calls that can
 * run at the same time need workspaces of their own, captured or not. Outputs must not overlap inputs (state
 * pools, updated in place, are both).
 * Results are deterministic: no call's result depends on the order of atomics.
 */
#ifndef NHM_LAYER_H
#define NHM_LAYER_H

#include "nhm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- MXFP4 */

/* OCP MXFP4: each row's 32 consecutive elements are a block with one scale code s (e8m0, worth 2^(s - 127); 255 is
 * NaN) and 32 element codes (e2m1: sign, then 0, 0.5, 1, 1.5, 2, 3, 4, 6), two a byte, the element of the lower index
 * in the low four bits. A value is that of its code times that of its scale; all of a NaN scale's are NaN. */

/* codes and scales of x:
 *   s = clamp(floor(log2(max |x|)) - 2, -127, 127) + 127 over the block (0 for a block of zeros)
 *   code = e2m1 nearest to x / 2^(s - 127), ties to the even code, magnitudes past 6 to 6; the sign of zero kept
 * A block that holds an infinity or NaN gets scale code 255 and codes 0.
 *   x       (device) [rows, ld_x] of type NHM_BF16 or NHM_F32, 16-byte aligned rows
 *   codes   (device) [rows, ld_codes] bytes, 4-byte aligned, ld_codes >= cols / 2, ld_codes % 4 == 0
 *   scales  (device) [rows, ld_scales], ld_scales >= cols / 32
 * cols must be a multiple of 32. rows == 0 or cols == 0 is a valid no-op.
 * Errors: NHM_ERR_NULL, NHM_ERR_SHAPE, NHM_ERR_ALIGN, NHM_ERR_UNSUPPORTED (type), NHM_ERR_HIP. */
NHM_API nhm_status nhm_mxfp4_quantize(const void* x, nhm_dtype type, int64_t rows, int64_t cols, int64_t ld_x,
                                      uint8_t* codes, int64_t ld_codes, uint8_t* scales, int64_t ld_scales,
                                      void* stream);

/* The values as bf16 (exact; those past the largest finite bf16 are infinities).
 *   codes, scales as nhm_mxfp4_quantize writes them;  out (device) bf16 [rows, ld_out], 16-byte aligned rows */
NHM_API nhm_status nhm_mxfp4_dequantize(const uint8_t* codes, int64_t ld_codes, const uint8_t* scales,
                                        int64_t ld_scales, int64_t rows, int64_t cols, uint16_t* out, int64_t ld_out,
                                        void* stream);

/* One projection's weight, in the [out, in] orientation (device pointers, host struct). */
typedef struct nhm_mxfp4_weight {
    const uint8_t* w;      /* (device) codes [n, k / 2], 16-byte aligned     */
    const uint8_t* scale;  /* (device) scale codes [n, k / 32]               */
    int64_t n;             /* output features                                */
    int64_t k;             /* input features, k % 32 == 0                    */
    const uint32_t* packed_scale; /* (device) nhm_mxfp4_pack_scales of scale, or NULL: packed
                              in the workspace by every call of more than 64 rows   */
} nhm_mxfp4_weight;

/* A weight's scale codes in the order in which the kernels for many rows take them, made once where the weight is
 * loaded: dword [j, row] of packed [ceil(k / 128), n] holds the codes of the row's blocks 4 j .. 4 j + 3, the first in the
 * low byte, 0 past the row. packed: (device, 4-byte aligned) nhm_mxfp4_packed_scale_bytes(n, k) bytes.
 * Errors: NHM_ERR_NULL, NHM_ERR_SHAPE, NHM_ERR_ALIGN, NHM_ERR_UNSUPPORTED (2 GiB or more), NHM_ERR_HIP. */
NHM_API size_t nhm_mxfp4_packed_scale_bytes(int64_t n, int64_t k);
NHM_API nhm_status nhm_mxfp4_pack_scales(const uint8_t* scale, int64_t n, int64_t k, uint32_t* packed, void* stream);

/* Workspace bytes of nhm_mxfp4_linear (0 for m, n or k <= 0): the codes and scales of a bf16 input, and past 64 rows the
 * packed scales of both operands. */
NHM_API size_t nhm_mxfp4_linear_workspace_bytes(int64_t m, int64_t n, int64_t k, nhm_dtype a_type);

/* out[i, j] = sum_k val(a[i, k]) val(w[j, k]), summed in f32 (within 2^-24 of sum |a w| per 128 products), rounded
 * once to bf16, or not for an f32 output.
 *   a        a_type NHM_BF16: (device) bf16 [m, ld_a], 16-byte aligned rows, quantized as by nhm_mxfp4_quantize;
 *            a_type NHM_MXFP4: (device) codes [m, ld_a] bytes, ld_a >= k / 2, 16-byte aligned rows
 *   a_scale  (device) scale codes [m, k / 32] of an MXFP4 input (NULL with bf16)
 *   out      (device) [m, ld_out] of out_type NHM_BF16 or NHM_F32, ld_out >= n, aligned to its element size
 *   ws       (device, 256-byte aligned) nhm_mxfp4_linear_workspace_bytes(...) bytes (may be 0: NULL)
 * m == 0 is a valid no-op. The result of a row does not depend on the other rows' values.
 * Operands of 2 GiB or more (of codes) are NHM_ERR_UNSUPPORTED, and so are more than 2^27 - 16 features
 * with at most 64 rows.
 * Errors: NHM_ERR_NULL, NHM_ERR_SHAPE, NHM_ERR_ALIGN, NHM_ERR_UNSUPPORTED, NHM_ERR_WORKSPACE, NHM_ERR_HIP. */
NHM_API nhm_status nhm_mxfp4_linear(const void* a, nhm_dtype a_type, const uint8_t* a_scale, int64_t m, int64_t ld_a,
                                    const nhm_mxfp4_weight* w, void* out, nhm_dtype out_type, int64_t ld_out, void* ws,
                                    size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------- short causal convolution */

/* Depthwise causal convolution over each sequence's tokens, a window of the width - 1 rows before the call carried
 * in a pool:  out_t = f(b + sum_j w[:, j] x_{t - width + 1 + j}),  f = silu where silu != 0, else the identity;
 * summed in f32, rounded once.
 *   x         (device) bf16 [n_tokens or batch, ld_x], 16-byte aligned rows
 *   w, b      (device) bf16 [dim, width] and [dim] (or NULL: 0), 16-byte aligned
 *   conv_pool (device) bf16 [n_slots, width - 1, dim], oldest row first, 16-byte aligned; updated in place
 *   out       (device) bf16 [.., ld_out], 16-byte aligned rows
 * dim % 8 == 0, width 2 .. 4. A slot outside [0, n_slots) is none. Decode: such a row is padding, its output zero.
 * Prefill: sequence i owns tokens cu_seqlens[i] .. cu_seqlens[i + 1] - 1 (contract as for nhm_mixer_prefill); it starts
 * from its slot's window where has_initial[i] != 0, else (and without a slot) from zeros, and leaves its last
 * rows there (a fresh empty sequence: zeros). Rows behind the last sequence are zero.
 * Contract: slots that are one are distinct within the call.
 * Errors: NHM_ERR_NULL, NHM_ERR_SHAPE, NHM_ERR_ALIGN, NHM_ERR_UNSUPPORTED, NHM_ERR_HIP. */
NHM_API nhm_status nhm_causal_conv_decode(const uint16_t* x, int64_t ld_x, const uint16_t* w, const uint16_t* b,
                                          int32_t dim, int32_t width, int32_t silu, int32_t batch,
                                          const int32_t* slot_idx, uint16_t* conv_pool, int32_t n_slots, uint16_t* out,
                                          int64_t ld_out, void* stream);
NHM_API nhm_status nhm_causal_conv_prefill(const uint16_t* x, int64_t ld_x, int64_t n_tokens, const uint16_t* w,
                                           const uint16_t* b, int32_t dim, int32_t width, int32_t silu,
                                           const int32_t* cu_seqlens, int32_t n_seqs, const int32_t* slot_idx,
                                           const int32_t* has_initial, uint16_t* conv_pool, int32_t n_slots,
                                           uint16_t* out, int64_t ld_out, void* stream);

/* ---------------------------------------------------------------- selective scan */

/* One layer's scan parameters (device pointers, host struct). */
typedef struct nhm_scan_params {
    const float* A_log;    /* f32 [dim, d_state], 16-byte aligned; A = -exp(A_log)      */
    const float* D;        /* f32 [dim] skip weight, or NULL: 0                         */
    const float* dt_bias;  /* f32 [dim], or NULL: 0; dt = softplus(dt_raw + dt_bias)    */
    int32_t dim;           /* channels, a multiple of 8                                 */
    int32_t d_state;       /* states of a channel, 4 .. 64, a multiple of 4             */
} nhm_scan_params;

/* For every channel c and state n:
 *   h_t[c, n] = exp(dt_t[c] A[c, n]) h_{t-1}[c, n] + dt_t[c] u_t[c] B_t[n]
 *   out_t[c] = (sum_n C_t[n] h_t[c, n] + D[c] u_t[c]) silu(z_t[c])      (without silu(z) where z is NULL)
 * in f32, out rounded once; a bf16 pool's states are widened when read and rounded when written, as the mixer's.
 *   u, dt, z, out (device) bf16 [n_tokens or batch, ld_*], dim columns; 2-byte aligned: slices of wider
 *                 rows (a projection's output) are taken as they are; row strides of at most 2^23
 *   B, C          (device) bf16 [.., ld_*], d_state columns, shared by the channels; likewise
 *   ssm_pool      (device) f32 or bf16 (ssm_type) [n_slots, dim, d_state], 16-byte aligned; updated in place
 *   ws            (device, 256-byte aligned) nhm_selective_scan_prefill_workspace_bytes(...) bytes (may be 0: NULL)
 * From a token on whose u is not finite, or whose dt_raw + dt_bias is NaN or +inf, its channel's outputs of that sequence are
 * infinite or NaN (which of them may differ between the two forms); other channels and sequences do not depend on it.
 * A dt_raw + dt_bias of -inf is a step of 0, as softplus has it: with a finite u the state stays as it is.
 * Slots, cu_seqlens, has_initial, padding and the rows behind the last sequence: as for the convolution above.
 * Errors: NHM_ERR_NULL, NHM_ERR_SHAPE, NHM_ERR_ALIGN, NHM_ERR_UNSUPPORTED, NHM_ERR_WORKSPACE, NHM_ERR_HIP. */
NHM_API nhm_status nhm_selective_scan_decode(const nhm_scan_params* p, const uint16_t* u, int64_t ld_u,
                                             const uint16_t* dt, int64_t ld_dt, const uint16_t* B, int64_t ld_b,
                                             const uint16_t* C, int64_t ld_c, const uint16_t* z, int64_t ld_z,
                                             int32_t batch, const int32_t* slot_idx, void* ssm_pool, nhm_dtype ssm_type,
                                             int32_t n_slots, uint16_t* out, int64_t ld_out, void* stream);
NHM_API size_t nhm_selective_scan_prefill_workspace_bytes(int32_t dim, int32_t d_state, int64_t n_tokens, int32_t n_seqs);
NHM_API nhm_status nhm_selective_scan_prefill(const nhm_scan_params* p, const uint16_t* u, int64_t ld_u,
                                              const uint16_t* dt, int64_t ld_dt, const uint16_t* B, int64_t ld_b,
                                              const uint16_t* C, int64_t ld_c, const uint16_t* z, int64_t ld_z,
                                              int64_t n_tokens, const int32_t* cu_seqlens, int32_t n_seqs,
                                              const int32_t* slot_idx, const int32_t* has_initial, void* ssm_pool,
                                              nhm_dtype ssm_type, int32_t n_slots, uint16_t* out, int64_t ld_out,
                                              void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------- scoring of tokens */

/* Workspace bytes of nhm_token_logprobs (0 for arguments outside its limits). */
NHM_API size_t nhm_token_logprobs_workspace_bytes(int64_t rows, int64_t vocab, int32_t n_top);

/* Of each row of logits, with p = softmax(logits[i]):
 *   logprobs[i] = log p(tokens[i])
 *   ranks[i]    = the token's place, from 1, in the row's order: by logit, highest first, equal ones by index, lowest first
 *   entropy[i]  = -sum_v p(v) log p(v), in nats
 *   top_logprobs[i, :], top_tokens[i, :] = the n_top first entries of that order
 * Sums are of f32 terms in f64. A NaN logit counts as -inf; where a row holds +inf, its +inf entries share the
 * probability. Entries without probability (-inf, and every other beside +inf) have log probability -inf, and places that they
 * would take among the first get token -1 and log probability -inf. A row of -inf has entropy 0.
 *   logits  (device) [rows, ld] of type NHM_BF16 or NHM_F32, ld >= vocab
 *   tokens  (device) int32 [rows], or NULL: none. A value outside [0, vocab) is none: log probability 0, rank 0
 *   logprobs, ranks, entropy (device) f32, int32, f32 [rows]; each may be NULL
 *   top_logprobs, top_tokens (device) f32, int32 [rows, n_top]; not used where n_top == 0
 * Limits: n_top 0 .. 64, vocab 1 .. 2^24, rows < 2^24. rows == 0 is a valid no-op.
 * Errors: NHM_ERR_NULL, NHM_ERR_SHAPE, NHM_ERR_ALIGN, NHM_ERR_UNSUPPORTED (a limit or the type), NHM_ERR_WORKSPACE,
 * NHM_ERR_HIP. */
NHM_API nhm_status nhm_token_logprobs(const void* logits, nhm_dtype type, int64_t ld, int64_t rows, int64_t vocab,
                                      const int32_t* tokens, int32_t n_top, float* logprobs, int32_t* ranks,
                                      float* entropy, float* top_logprobs, int32_t* top_tokens, void* ws,
                                      size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* NHM_LAYER_H */
