/*
 * nhm_serving.h -- C ABI of libnhm's serving operators: what a server of many requests runs
 * beside the mixer of nhm.h. The adapters of many requests beside a shared projection, beam
 * search's selection and the reordering of the recurrent states it asks for, and the index
 * tensors of a batch built on the GPU from request lengths.
 *
 * The conventions of nhm.h hold for every call: caller-owned memory, host validation before
 * anything is enqueued, a status and nhm_last_error() instead of exceptions, work enqueued on
 * the given stream only, no synchronization, no allocation, legal inside HIP graph capture.
 * The stream must belong to the current device, and so must the tensors. Two calls that can
 * run at the same time need workspaces of their own, captured or not.
 * Results are deterministic: no call's result depends on the order of atomics.
 */
#ifndef NHM_SERVING_H
#define NHM_SERVING_H

#include "nhm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- low-rank adapters */

/* A set of low-rank adapters of one projection [n, k] (device pointers, host struct): adapter
 * e adds scale[e] * B_e (A_e x) to the projection of x. Adapters of smaller rank are padded
 * with zero rows of A or zero columns of B. */
typedef struct nhm_lora {
    const uint16_t* a;     /* (device) bf16 [n_adapters, rank, k], 16-byte aligned      */
    const uint16_t* b;     /* (device) bf16 [n_adapters, n, rank], 16-byte aligned      */
    const float* scale;    /* (device) f32 [n_adapters], or NULL: 1 for every adapter   */
    int32_t n_adapters;    /* >= 1                                                      */
    int32_t rank;          /* 8 .. 128, a multiple of 8                                 */
} nhm_lora;

/* Workspace bytes of nhm_fp8_linear_lora (0 for m <= 0, n <= 0, k <= 0 or an unsupported rank). */
NHM_API size_t nhm_fp8_linear_lora_workspace_bytes(int64_t m, int64_t n, int64_t k, nhm_dtype a_type, int32_t rank);

/* One projection shared by every row, and each row's own adapter beside it:
 *   out[i, :] = (a_q[i] W^T) a_scale w_scale + scale[e] (x[i] A_e^T) B_e^T,  e = row_adapter[i]
 * with x[i] the row as given: the bf16 values, or val(code) * a_scale for an e4m3 input. The
 * projection is that of nhm_fp8_linear_ex (exact == 0) or nhm_fp8_linear_exact (exact != 0),
 * without the split over k. The low-rank product x A_e^T is summed in f32 and enters the second
 * product as a sum of bf16 parts (two for a bf16 output, three for f32: 2^-17 and 2^-25 of the
 * value), the projection and the adapter's part are added in f32, and the sum is rounded once.
 *   a, a_type, m, ld_a, w, out, out_type, ld_out   as for nhm_fp8_linear_ex
 *   row_adapter (device) int32 [m]: the row's adapter; a value outside [0, n_adapters) is no
 *               adapter, and the row's result is the projection's alone, bit for bit. Rows in any
 *               order; rows of one adapter next to each other cost least
 *   ws          (device, 256-byte aligned) nhm_fp8_linear_lora_workspace_bytes(...) bytes
 * A row reads its own adapter only: values of other adapters, NaN and infinities among them,
 * do not reach it. m == 0 is a valid no-op.
 * Errors: those of nhm_fp8_linear_ex; NHM_ERR_UNSUPPORTED for a rank outside the list above,
 * NHM_ERR_SHAPE for n_adapters < 1, NHM_ERR_WORKSPACE for a missing or short ws. */
NHM_API nhm_status nhm_fp8_linear_lora(const void* a, nhm_dtype a_type, int64_t m, int64_t ld_a,
                                       const nhm_fp8_weight* w, const nhm_lora* lora, const int32_t* row_adapter,
                                       void* out, nhm_dtype out_type, int64_t ld_out, int32_t exact, void* ws,
                                       size_t ws_bytes, void* stream);

/* nhm_mixer_decode_ex and nhm_mixer_prefill_ex with adapters beside the projections: lora_in of in_proj
 * (n = d_in_proj, k = hidden) on the block input, lora_out of out_proj (n = hidden, k = d_inner) on the
 * bf16 gated norm output. Either may be NULL: that projection runs as without. row_adapter (device) int32
 * [batch] or [n_tokens] as for nhm_fp8_linear_lora (nhm_batch_plan's token_adapter is one), the same
 * for both sets, which may differ in rank and number. in_proj sums every product in f32, out_proj as in
 * the calls without adapters; where those split out_proj over k, these do not.
 * A padded decode row (negative slot) and a prefill row behind the last sequence have a zero norm output, so
 * their output stays zero with any finite adapter. ws: the layout calls below, with the larger rank of the two sets.
 * Errors: those of the calls without adapters and of nhm_fp8_linear_lora. */
NHM_API nhm_status nhm_mixer_decode_lora_ws_layout(const nhm_geometry* g, int32_t batch, int32_t rank,
                                                   nhm_ws_layout* out);
NHM_API nhm_status nhm_mixer_decode_lora(const nhm_mixer_params* p, const nhm_lora* lora_in, const nhm_lora* lora_out,
                                         const int32_t* row_adapter, const uint16_t* hidden, int32_t batch,
                                         const int32_t* slot_idx, void* ssm_pool, nhm_dtype ssm_type,
                                         uint16_t* conv_pool, int32_t n_slots, uint16_t* out, void* ws, size_t ws_bytes,
                                         void* stream);
NHM_API nhm_status nhm_mixer_prefill_lora_ws_layout(const nhm_geometry* g, int64_t n_tokens, int32_t n_seqs,
                                                    int32_t chunk, int32_t rank, nhm_ws_layout* out);
NHM_API nhm_status nhm_mixer_prefill_lora(const nhm_mixer_params* p, const nhm_lora* lora_in, const nhm_lora* lora_out,
                                          const int32_t* row_adapter, const uint16_t* hidden, int64_t n_tokens,
                                          const int32_t* cu_seqlens, int32_t n_seqs, const int32_t* slot_idx,
                                          const int32_t* has_initial, int32_t chunk, void* ssm_pool,
                                          nhm_dtype ssm_type, uint16_t* conv_pool, int32_t n_slots, uint16_t* out,
                                          void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------- beam search */

/* Workspace bytes of nhm_beam_select (0 for arguments outside its limits). */
NHM_API size_t nhm_beam_select_workspace_bytes(int64_t n_groups, int32_t n_beams, int64_t vocab, int32_t n_cand);

/* The n_cand best continuations of each group's beams:
 *   score(b, v) = cum[g, b] + logits[g, b, v] - log(sum_v exp(logits[g, b, v]))
 * ordered by score, highest first, equal scores by beam and then token, lowest first. Scores are
 * formed and compared in f64 (the sum of the exponentials from f32 terms) and returned in f32.
 * A NaN logit counts as -inf; where a row holds +inf, its +inf entries share the probability.
 * Of one beam's continuations whose logits differ too little for their f64 scores to differ, those
 * of the larger logits are kept.
 * Continuations whose score is -inf or NaN are none: places they would take get score -inf,
 * parent -1 and token -1.
 *   logits    (device) [n_groups * n_beams, ld] of type NHM_BF16 or NHM_F32, ld >= vocab
 *   cum       (device) f32 [n_groups, n_beams]: the beams' scores so far (-inf: an unused beam)
 *   finished  (device) int32 [n_groups, n_beams] or NULL: a non-zero entry marks a finished beam,
 *             whose one continuation is the token eos at score cum; its logits are not used
 *   eos       the end token, in [0, vocab) (not used without finished)
 *   scores    (device) f32 [n_groups, n_cand]
 *   parents   (device) int32 [n_groups, n_cand]: the continued beam within its group
 *   tokens    (device) int32 [n_groups, n_cand]
 * Limits: n_beams 1 .. 32, n_cand 1 .. 64, vocab 1 .. 2^24, n_groups * n_beams < 2^24.
 * n_groups == 0 is a valid no-op.
 * Errors: NHM_ERR_NULL, NHM_ERR_SHAPE, NHM_ERR_ALIGN, NHM_ERR_UNSUPPORTED (a limit or the type),
 * NHM_ERR_WORKSPACE, NHM_ERR_HIP. */
NHM_API nhm_status nhm_beam_select(const void* logits, nhm_dtype type, int64_t ld, int64_t n_groups, int32_t n_beams,
                                   int64_t vocab, const float* cum, const int32_t* finished, int32_t eos,
                                   int32_t n_cand, float* scores, int32_t* parents, int32_t* tokens, void* ws,
                                   size_t ws_bytes, void* stream);

/* One layer's state pools (device), as nhm_mixer_decode takes them. */
typedef struct nhm_state_pool {
    void* ssm;             /* f32 or bf16 [n_slots, n_heads, head_dim, d_state], 16-byte aligned */
    uint16_t* conv;        /* bf16 [n_slots, conv_width - 1, conv_dim], 16-byte aligned          */
} nhm_state_pool;

/* The slots of each group's beams after a selection, and the states moved to match, for every
 * layer at once. New beam j of a group continues beam parents[g, j]. The first beam (lowest j)
 * that continues a parent takes the parent's slot, whose rows stay in place; the other beams
 * get, in order of j, the slots of the beams that none continues, in ascending order of beam,
 * and those of them with a parent get a copy of its rows there. new_slots is thus a permutation
 * of slots within each group, and rows of slots outside the group are not touched.
 *   parents    (device) int32 [n_groups, n_beams]; a value outside [0, n_beams) is no parent:
 *              that beam's slot holds whatever its rows held
 *   slots      (device) int32 [n_groups, n_beams]. Contract: non-negative entries are distinct
 *              over the call. An entry outside [0, n_slots) marks an absent row, which is neither
 *              read nor written
 *   pools      (host) [n_layers] device pointers, 1 .. 64 layers
 *   new_slots  (device) int32 [n_groups, n_beams]; must not overlap parents or slots
 * Limits: n_beams 1 .. 32, n_groups * n_beams <= 2^24. n_groups == 0 is a valid no-op.
 * Errors: NHM_ERR_NULL, NHM_ERR_SHAPE, NHM_ERR_ALIGN, NHM_ERR_UNSUPPORTED, NHM_ERR_HIP. */
NHM_API nhm_status nhm_beam_reorder(const nhm_geometry* g, const int32_t* parents, const int32_t* slots,
                                    int64_t n_groups, int32_t n_beams, const nhm_state_pool* pools, int32_t n_layers,
                                    nhm_dtype ssm_type, int32_t n_slots, int32_t* new_slots, void* stream);

/* ---------------------------------------------------------------- batch plan */

/* The index tensors of a packed batch, from the requests' lengths on the GPU:
 *   cu_seqlens[0] = 0, cu_seqlens[i + 1] = cu_seqlens[i] + lengths[i]
 *   has_initial[i] = past[i] > 0
 * and for token t of sequence i (cu_seqlens[i] <= t < cu_seqlens[i + 1]):
 *   token_seq[t] = i, token_pos[t] = past[i] + t - cu_seqlens[i], token_adapter[t] = adapters[i]
 * Tokens from the last sequence's end up to n_tokens get -1 in all three. Sequences end at
 * n_tokens at the latest: where the lengths add up to more, cu_seqlens holds n_tokens from there
 * on. A negative length counts as 0.
 *   lengths       (device) int32 [n_seqs]: this batch's tokens of each sequence
 *   past          (device) int32 [n_seqs] or NULL (0): tokens that its state holds already
 *   adapters      (device) int32 [n_seqs] or NULL (-1): its adapter (nhm_fp8_linear_lora)
 *   cu_seqlens    (device) int32 [n_seqs + 1]
 *   has_initial   (device) int32 [n_seqs]
 *   token_seq, token_pos, token_adapter (device) int32 [n_tokens], each may be NULL
 * Outputs must not overlap inputs. Limits: n_seqs 0 .. 8192, n_tokens 0 .. 2^31 - 1.
 * Errors: NHM_ERR_NULL, NHM_ERR_SHAPE, NHM_ERR_ALIGN, NHM_ERR_UNSUPPORTED, NHM_ERR_HIP. */
NHM_API nhm_status nhm_batch_plan(const int32_t* lengths, const int32_t* past, const int32_t* adapters, int32_t n_seqs,
                                  int64_t n_tokens, int32_t* cu_seqlens, int32_t* has_initial, int32_t* token_seq,
                                  int32_t* token_pos, int32_t* token_adapter, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* NHM_SERVING_H */
