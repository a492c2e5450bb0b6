// Entry points of the serving operators (nhm_serving.h): host validation and launch order.
#include <limits.h>

#include "nhm_internal.h"

using namespace nhm;

namespace {

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool rank_ok(int32_t rank) { return rank >= 8 && rank <= kLoraMaxRank && rank % 8 == 0; }

// Regions of the adapter call's workspace: the activation codes of a bf16 input, the low-rank product.
struct LoraWs { size_t t, total; };
LoraWs lora_ws(int64_t m, int64_t k, nhm_dtype a_type, int32_t rank) {
    LoraWs w{};
    w.t = align_up(linear_codes_ws(m, k, a_type), 256);
    w.total = w.t + align_up((size_t)m * 3 * lora_rp(rank) * sizeof(uint16_t), 256);
    return w;
}

nhm_status check_lora(const nhm_lora* l) {
    if (!l) return fail(NHM_ERR_NULL, "lora is NULL");
    if (!l->a || !l->b) return fail(NHM_ERR_NULL, "lora: a or b is NULL");
    if (l->n_adapters < 1) return fail(NHM_ERR_SHAPE, "lora: n_adapters %d must be positive", l->n_adapters);
    if (!rank_ok(l->rank)) return fail(NHM_ERR_UNSUPPORTED, "lora: rank %d: a multiple of 8 in 8 .. 128", l->rank);
    if (!aligned(l->a, 16) || !aligned(l->b, 16) || !aligned(l->scale, 4))
        return fail(NHM_ERR_ALIGN, "lora: a and b must be 16-byte aligned, scale 4-byte aligned");
    return NHM_OK;
}

// ---- the mixer's projections with adapters

// The low-rank product's workspace of m rows, bf16 outputs.
size_t mixer_t_bytes(int64_t m, int32_t rank) { return align_up((size_t)m * 2 * lora_rp(rank) * sizeof(uint16_t), 256); }

LoraDownArgs down_args(const ProjectionHooks& h, const nhm_lora* l, const uint16_t* x, int64_t m, const nhm_fp8_weight& w,
                       uint8_t* q, char* ws) {
    LoraDownArgs g{};
    g.x = x;
    g.ld_x = w.k;
    g.m = m; g.k = w.k;
    g.a_scale = w.a_scale;
    g.q = q;
    g.a = l->a; g.scale = l->scale;
    g.n_adapters = l->n_adapters; g.rank = l->rank;
    g.rp = lora_rp(l->rank);
    g.parts = 2;
    g.row_adapter = h.row_adapter;
    g.t = reinterpret_cast<uint16_t*>(ws);
    return g;
}

// One projection of m rows: up to 32 decode rows 16 at a time on the GEMV, as the mixer's own, else one call.
nhm_status project_rows(const LoraDownArgs& d, const nhm_lora* l, const nhm_fp8_weight& w, const uint8_t* q, uint16_t* out,
                        bool decode, bool exact, uint32_t* clear, int clear_n, hipStream_t st) {
    const LoraEpi e{d.t, l->b, d.row_adapter, d.n_adapters, d.rank, d.rp, d.parts};
    const int64_t m = d.m;
    if (decode ? m <= 32 && use_gemv(16, w.n, w.k) : use_gemv(m, w.n, w.k)) {
        for (int64_t r0 = 0; r0 < m; r0 += 16) {
            LoraEpi er = e;
            er.t += r0 * e.parts * e.rp;
            er.row_adapter += r0;
            const nhm_status s = launch_gemv_lora(q + r0 * w.k, w.k, (int)(m - r0 < 16 ? m - r0 : 16), w.w, w.w_scale,
                                                  w.a_scale, w.n, w.k, out + r0 * w.n, w.n, st, nullptr, ws_step(w), er,
                                                  r0 == 0 ? clear : nullptr, r0 == 0 ? clear_n : 0);
            if (s != NHM_OK) return s;
        }
        return NHM_OK;
    }
    if (clear && clear_n > 0) launch_clear(clear, clear_n, st);
    return launch_gemm_lora(q, w.k, m, w.w, w.w_scale, w.a_scale, w.n, w.k, out, w.n, st, nullptr, exact, ws_step(w), e);
}

nhm_status hook_in(const ProjectionHooks& h, const uint16_t* hidden, int64_t m, uint8_t* q, uint16_t* zx, uint32_t* clear,
                   int clear_n, char* ws, hipStream_t st) {
    const LoraDownArgs d = down_args(h, h.lora_in, hidden, m, h.p->in_proj, q, ws);
    const nhm_status s = launch_lora_down(d, st);
    // every product summed in f32, as the mixer's own in_proj
    return s != NHM_OK ? s : project_rows(d, h.lora_in, h.p->in_proj, q, zx, h.decode, true, clear, clear_n, st);
}

nhm_status hook_out(const ProjectionHooks& h, const uint16_t* norm, const uint8_t* q, int64_t m, uint16_t* out, char* ws,
                    hipStream_t st) {
    const LoraDownArgs d = down_args(h, h.lora_out, norm, m, h.p->out_proj, nullptr, ws);
    const nhm_status s = launch_lora_down(d, st);
    return s != NHM_OK ? s : project_rows(d, h.lora_out, h.p->out_proj, q, out, h.decode, false, nullptr, 0, st);
}

// Checks the adapters of a mixer call and fills in its hooks (either set of adapters may be NULL).
nhm_status mixer_hooks(ProjectionHooks& h, const nhm_mixer_params* p, const nhm_lora* in, const nhm_lora* out,
                       const int32_t* row_adapter, int64_t m, bool decode) {
    if (!p) return fail(NHM_ERR_NULL, "params is NULL");
    h.p = p;
    h.row_adapter = row_adapter;
    h.decode = decode;
    for (int i = 0; i < 2; ++i) {
        const nhm_lora* l = i == 0 ? in : out;
        if (!l) continue;
        const int64_t n = i == 0 ? p->in_proj.n : p->out_proj.n;
        const nhm_status s = check_lora(l);
        if (s != NHM_OK) return s;
        if (n >= (int64_t(1) << 30) / l->rank)
            return fail(NHM_ERR_UNSUPPORTED, "lora: an adapter's b of 2 GiB or more");
        const size_t t = mixer_t_bytes(m, l->rank);
        h.extra = h.extra > t ? h.extra : t;
    }
    if ((in || out) && m > 0) {
        if (!row_adapter) return fail(NHM_ERR_NULL, "row_adapter is NULL");
        if (!aligned(row_adapter, 4)) return fail(NHM_ERR_ALIGN, "row_adapter must be 4-byte aligned");
    }
    h.lora_in = in;
    h.lora_out = out;
    h.in_proj = in ? hook_in : nullptr;
    h.out_proj = out ? hook_out : nullptr;
    return NHM_OK;
}

constexpr int kMaxBeams = 32, kMaxCand = 64;
constexpr int64_t kMaxVocab = int64_t(1) << 24, kMaxRows = int64_t(1) << 24;

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

}  // namespace

extern "C" {

size_t nhm_fp8_linear_lora_workspace_bytes(int64_t m, int64_t n, int64_t k, nhm_dtype a_type, int32_t rank) {
    if (m <= 0 || n <= 0 || k <= 0 || !rank_ok(rank)) return 0;
    return lora_ws(m, k, a_type, rank).total;
}

nhm_status nhm_fp8_linear_lora(const void* a, nhm_dtype a_type, int64_t m, int64_t ld_a, const nhm_fp8_weight* w,
                               const nhm_lora* lora, const int32_t* row_adapter, void* out, nhm_dtype out_type,
                               int64_t ld_out, int32_t exact, void* ws, size_t ws_bytes, void* stream) {
    clear_error();
    nhm_status s = check_lora(lora);
    if (s != NHM_OK) return s;
    const size_t need = w && m > 0 && w->n > 0 && w->k > 0 ? lora_ws(m, w->k, a_type, lora->rank).total : 0;
    s = linear_check(a, a_type, m, ld_a, w, out, out_type, ld_out, ws, ws_bytes, need);
    if (s != NHM_OK || m == 0) return s;
    if (m > INT_MAX) return fail(NHM_ERR_SHAPE, "m %lld out of range", (long long)m);
    if (!row_adapter) return fail(NHM_ERR_NULL, "row_adapter is NULL");
    if (!aligned(row_adapter, 4)) return fail(NHM_ERR_ALIGN, "row_adapter must be 4-byte aligned");
    if (w->n >= (int64_t(1) << 30) / lora->rank)       // 32-bit byte offsets within one adapter's B
        return fail(NHM_ERR_UNSUPPORTED, "lora: an adapter's b of 2 GiB or more");
    hipStream_t st = (hipStream_t)stream;
    const LoraWs l = lora_ws(m, w->k, a_type, lora->rank);
    char* wsb = static_cast<char*>(ws);
    const bool bf16 = a_type == NHM_BF16;
    const uint8_t* q = bf16 ? reinterpret_cast<uint8_t*>(wsb) : static_cast<const uint8_t*>(a);
    const int64_t ld_q = bf16 ? w->k : ld_a;
    LoraDownArgs g{};
    g.x = bf16 ? static_cast<const uint16_t*>(a) : nullptr;
    g.x_codes = bf16 ? nullptr : q;
    g.ld_x = ld_a;
    g.m = m; g.k = w->k;
    g.a_scale = w->a_scale;
    g.q = bf16 ? reinterpret_cast<uint8_t*>(wsb) : nullptr;
    g.a = lora->a; g.scale = lora->scale;
    g.n_adapters = lora->n_adapters; g.rank = lora->rank;
    g.rp = lora_rp(lora->rank);
    g.parts = out_type == NHM_F32 ? 3 : 2;
    g.row_adapter = row_adapter;
    g.t = reinterpret_cast<uint16_t*>(wsb + l.t);
    if ((s = launch_lora_down(g, st)) != NHM_OK) return s;
    const LoraEpi epi{g.t, lora->b, row_adapter, g.n_adapters, g.rank, g.rp, g.parts};
    uint16_t* ob = out_type == NHM_BF16 ? static_cast<uint16_t*>(out) : nullptr;
    float* of = out_type == NHM_F32 ? static_cast<float*>(out) : nullptr;
    if (use_gemv(m, w->n, w->k))
        return launch_gemv_lora(q, ld_q, (int)m, w->w, w->w_scale, w->a_scale, w->n, w->k, ob, ld_out, st, of, ws_step(*w), epi);
    return launch_gemm_lora(q, ld_q, m, w->w, w->w_scale, w->a_scale, w->n, w->k, ob, ld_out, st, of, exact != 0, ws_step(*w),
                            epi);
}

nhm_status nhm_mixer_decode_lora_ws_layout(const nhm_geometry* g, int32_t batch, int32_t rank, nhm_ws_layout* out) {
    const nhm_status s = nhm_mixer_decode_ws_layout(g, batch, out);
    if (s != NHM_OK) return s;
    if (!rank_ok(rank)) return fail(NHM_ERR_UNSUPPORTED, "lora: rank %d: a multiple of 8 in 8 .. 128", rank);
    out->total += mixer_t_bytes(batch, rank);
    return NHM_OK;
}

nhm_status nhm_mixer_prefill_lora_ws_layout(const nhm_geometry* g, int64_t n_tokens, int32_t n_seqs, int32_t chunk,
                                            int32_t rank, nhm_ws_layout* out) {
    const nhm_status s = nhm_mixer_prefill_ws_layout(g, n_tokens, n_seqs, chunk, out);
    if (s != NHM_OK) return s;
    if (!rank_ok(rank)) return fail(NHM_ERR_UNSUPPORTED, "lora: rank %d: a multiple of 8 in 8 .. 128", rank);
    out->total += mixer_t_bytes(n_tokens, rank);
    return NHM_OK;
}

nhm_status nhm_mixer_decode_lora(const nhm_mixer_params* p, const nhm_lora* lora_in, const nhm_lora* lora_out,
                                 const int32_t* row_adapter, const uint16_t* hidden, int32_t batch,
                                 const int32_t* slot_idx, void* ssm_pool, nhm_dtype ssm_type, uint16_t* conv_pool,
                                 int32_t n_slots, uint16_t* out, void* ws, size_t ws_bytes, void* stream) {
    clear_error();
    ProjectionHooks h;
    const nhm_status s = mixer_hooks(h, p, lora_in, lora_out, row_adapter, batch < 0 ? 0 : batch, true);
    if (s != NHM_OK) return s;
    return mixer_decode_call(p, hidden, nullptr, batch, slot_idx, ssm_pool, ssm_type, conv_pool, n_slots, out, nullptr,
                             nullptr, ws, ws_bytes, stream, false, &h);
}

nhm_status nhm_mixer_prefill_lora(const nhm_mixer_params* p, const nhm_lora* lora_in, const nhm_lora* lora_out,
                                  const int32_t* row_adapter, const uint16_t* hidden, int64_t n_tokens,
                                  const int32_t* cu_seqlens, int32_t n_seqs, const int32_t* slot_idx,
                                  const int32_t* has_initial, int32_t chunk, void* ssm_pool, nhm_dtype ssm_type,
                                  uint16_t* conv_pool, int32_t n_slots, uint16_t* out, void* ws, size_t ws_bytes,
                                  void* stream) {
    clear_error();
    if (n_tokens > INT_MAX) return fail(NHM_ERR_SHAPE, "n_tokens %lld out of range", (long long)n_tokens);
    ProjectionHooks h;
    const nhm_status s = mixer_hooks(h, p, lora_in, lora_out, row_adapter, n_tokens < 0 ? 0 : n_tokens, false);
    if (s != NHM_OK) return s;
    return mixer_prefill_call(p, hidden, n_tokens, cu_seqlens, n_seqs, slot_idx, has_initial, chunk, ssm_pool, ssm_type,
                              conv_pool, n_slots, out, ws, ws_bytes, stream, &h);
}

size_t nhm_beam_select_workspace_bytes(int64_t n_groups, int32_t n_beams, int64_t vocab, int32_t n_cand) {
    if (n_groups <= 0 || n_beams < 1 || n_beams > kMaxBeams || vocab < 1 || vocab > kMaxVocab || n_cand < 1 ||
        n_cand > kMaxCand || n_groups > (kMaxRows - 1) / n_beams)
        return 0;
    return beam_ws_bytes(n_groups * n_beams, vocab, n_cand);
}

nhm_status nhm_beam_select(const void* logits, nhm_dtype type, int64_t ld, int64_t n_groups, int32_t n_beams,
                           int64_t vocab, const float* cum, const int32_t* finished, int32_t eos, int32_t n_cand,
                           float* scores, int32_t* parents, int32_t* tokens, void* ws, size_t ws_bytes, void* stream) {
    clear_error();
    if (type != NHM_BF16 && type != NHM_F32) return fail(NHM_ERR_UNSUPPORTED, "logits dtype %d: bf16 or f32", (int)type);
    if (n_groups < 0 || vocab < 1 || n_cand < 1 || n_beams < 1 || ld < vocab)
        return fail(NHM_ERR_SHAPE, "groups %lld, beams %d, vocab %lld (ld %lld), candidates %d out of range",
                    (long long)n_groups, n_beams, (long long)vocab, (long long)ld, n_cand);
    if (n_beams > kMaxBeams || n_cand > kMaxCand || vocab > kMaxVocab || n_groups > (kMaxRows - 1) / n_beams)
        return fail(NHM_ERR_UNSUPPORTED, "at most %d beams, %d candidates, a vocabulary of 2^24 and fewer than 2^24 rows",
                    kMaxBeams, kMaxCand);
    if (n_groups == 0) return NHM_OK;
    if (!logits || !cum || !scores || !parents || !tokens)
        return fail(NHM_ERR_NULL, "logits, cum, scores, parents or tokens is NULL");
    if (finished && (eos < 0 || eos >= vocab)) return fail(NHM_ERR_SHAPE, "eos %d outside the vocabulary", eos);
    if (!aligned(logits, type == NHM_F32 ? 4 : 2) || !aligned(cum, 4) || !aligned(finished, 4) || !aligned(scores, 4) ||
        !aligned(parents, 4) || !aligned(tokens, 4))
        return fail(NHM_ERR_ALIGN, "every tensor must be aligned to its element size");
    const size_t need = beam_ws_bytes(n_groups * n_beams, vocab, n_cand);
    if (!ws || ws_bytes < need)
        return fail(NHM_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? ws_bytes : (size_t)0);
    if (!aligned(ws, 256)) return fail(NHM_ERR_ALIGN, "ws must be 256-byte aligned");
    BeamArgs g{};
    g.logits_bf16 = type == NHM_BF16 ? static_cast<const uint16_t*>(logits) : nullptr;
    g.logits_f32 = type == NHM_F32 ? static_cast<const float*>(logits) : nullptr;
    g.ld = ld; g.n_groups = n_groups; g.n_beams = n_beams; g.vocab = vocab;
    g.cum = cum; g.finished = finished; g.eos = eos; g.n_cand = n_cand;
    g.scores = scores; g.parents = parents; g.tokens = tokens;
    return launch_beam_select(g, ws, (hipStream_t)stream);
}

nhm_status nhm_beam_reorder(const nhm_geometry* geo, const int32_t* parents, const int32_t* slots, int64_t n_groups,
                            int32_t n_beams, const nhm_state_pool* pools, int32_t n_layers, nhm_dtype ssm_type,
                            int32_t n_slots, int32_t* new_slots, void* stream) {
    clear_error();
    nhm_status s = check_geometry(geo);
    if (s != NHM_OK) return s;
    if (ssm_type != NHM_F32 && ssm_type != NHM_BF16)
        return fail(NHM_ERR_UNSUPPORTED, "SSM state dtype %d: f32 or bf16", (int)ssm_type);
    if (n_groups < 0 || n_beams < 1 || n_layers < 1 || n_slots < 1)
        return fail(NHM_ERR_SHAPE, "groups %lld, beams %d, layers %d, slots %d out of range", (long long)n_groups, n_beams,
                    n_layers, n_slots);
    if (n_beams > kMaxBeams || n_layers > kMaxStatePools || n_groups > kMaxRows / n_beams)
        return fail(NHM_ERR_UNSUPPORTED, "at most %d beams, %d layers and 2^24 rows", kMaxBeams, kMaxStatePools);
    if (n_groups == 0) return NHM_OK;
    if (!parents || !slots || !pools || !new_slots) return fail(NHM_ERR_NULL, "parents, slots, pools or new_slots is NULL");
    if (!aligned(parents, 4) || !aligned(slots, 4) || !aligned(new_slots, 4))
        return fail(NHM_ERR_ALIGN, "parents, slots and new_slots must be 4-byte aligned");
    const size_t nb = (size_t)n_groups * n_beams * 4;
    if (overlap(new_slots, nb, parents, nb) || overlap(new_slots, nb, slots, nb))
        return fail(NHM_ERR_UNSUPPORTED, "new_slots must not overlap parents or slots");
    nhm_layout l;
    fill_layout(geo, &l);
    ReorderArgs g{};
    for (int32_t i = 0; i < n_layers; ++i) {
        if (!pools[i].ssm || !pools[i].conv) return fail(NHM_ERR_NULL, "layer %d: a pool is NULL", i);
        if (!aligned(pools[i].ssm, 16) || !aligned(pools[i].conv, 16))
            return fail(NHM_ERR_ALIGN, "layer %d: pools must be 16-byte aligned", i);
        g.pools[i] = pools[i];
    }
    g.parents = parents; g.slots = slots; g.new_slots = new_slots;
    g.n_beams = n_beams; g.n_slots = n_slots;
    g.ssm_bytes = (int64_t)geo->n_heads * geo->head_dim * geo->d_state * (ssm_type == NHM_F32 ? 4 : 2);
    g.conv_bytes = (int64_t)(geo->conv_width - 1) * l.conv_dim * 2;
    return launch_beam_reorder(g, n_groups, n_layers, (hipStream_t)stream);
}

nhm_status nhm_batch_plan(const int32_t* lengths, const int32_t* past, const int32_t* adapters, int32_t n_seqs,
                          int64_t n_tokens, int32_t* cu_seqlens, int32_t* has_initial, int32_t* token_seq,
                          int32_t* token_pos, int32_t* token_adapter, void* stream) {
    clear_error();
    if (n_seqs < 0 || n_tokens < 0 || n_tokens > INT_MAX)
        return fail(NHM_ERR_SHAPE, "n_seqs %d or n_tokens %lld out of range", n_seqs, (long long)n_tokens);
    if (n_seqs > kMaxPlanSeqs) return fail(NHM_ERR_UNSUPPORTED, "%d sequences: at most %d", n_seqs, kMaxPlanSeqs);
    if (!cu_seqlens || (n_seqs > 0 && (!lengths || !has_initial)))
        return fail(NHM_ERR_NULL, "lengths, cu_seqlens or has_initial is NULL");
    if (!aligned(lengths, 4) || !aligned(past, 4) || !aligned(adapters, 4) || !aligned(cu_seqlens, 4) ||
        !aligned(has_initial, 4) || !aligned(token_seq, 4) || !aligned(token_pos, 4) || !aligned(token_adapter, 4))
        return fail(NHM_ERR_ALIGN, "every tensor must be 4-byte aligned");
    const PlanArgs g{lengths, past, adapters, n_seqs, n_tokens, cu_seqlens, has_initial, token_seq, token_pos, token_adapter};
    return launch_batch_plan(g, (hipStream_t)stream);
}

}  // extern "C"
