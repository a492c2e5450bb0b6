// Entry points of the operators of a selective-scan layer in 4 bits (nhm_layer.h): host validation and
// launch order.
#include <limits.h>

#include "nhm_internal.h"

using namespace nhm;

namespace {

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool rows16(const void* p, int64_t ld_bytes) { return aligned(p, 16) && ld_bytes % 16 == 0; }

// A launch holds fewer than 2^32 threads.
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 1;
constexpr int64_t kMaxLd = int64_t(1) << 40;           // row strides: offsets stay within 63 bits
constexpr int64_t kMaxOperand = int64_t(1) << 31;      // bytes behind a buffer descriptor
constexpr int64_t kMaxScanLd = int64_t(1) << 23;       // 80 rows of bf16 within 31 bits
constexpr int64_t kMaxVocab = int64_t(1) << 24, kMaxRows = int64_t(1) << 24;
constexpr int kMaxTop = 64;

// Codes of a bf16 activation and its scales, as rows or packed for the tile kernels (an MXFP4 input's packed scales
// alone), and on the tile kernels room for the weight's packed scales where the caller has none. Nothing where the rows
// kernel quantises the activation itself.
struct MxWs { size_t scales, weight, total; };
MxWs mx_ws(int64_t m, int64_t n, int64_t k, nhm_dtype t) {
    MxWs w{0, 0, 0};
    const bool tiled = mx_tiled(m);
    if (t == NHM_BF16 && mx_rows_quantise(m, k)) return w;
    if (t == NHM_BF16) w.scales = align_up((size_t)m * (k / 2), 256);
    w.weight = w.scales;
    if (tiled) w.weight += align_up((size_t)mx_packed_words(m, k) * 4, 256);
    else if (t == NHM_BF16) w.weight += align_up((size_t)m * (k / 32), 256);
    w.total = w.weight + (tiled ? align_up((size_t)mx_packed_words(n, k) * 4, 256) : 0);
    return w;
}

nhm_status check_conv(const uint16_t* x, int64_t ld_x, int64_t rows, const uint16_t* w, const uint16_t* b, int32_t dim,
                      int32_t width, const int32_t* slot_idx, const uint16_t* pool, int32_t n_slots, const uint16_t* out,
                      int64_t ld_out) {
    if (rows < 0 || rows > INT_MAX || dim < 1 || n_slots < 1 || ld_x < dim || ld_out < dim || ld_x > kMaxLd || ld_out > kMaxLd)
        return fail(NHM_ERR_SHAPE, "conv: rows %lld, dim %d (ld %lld, %lld) or slots %d out of range", (long long)rows, dim,
                    (long long)ld_x, (long long)ld_out, n_slots);
    if (width < 2 || width > 4 || dim % 8 != 0)
        return fail(NHM_ERR_UNSUPPORTED, "conv: width %d (2 .. 4) and dim %d (a multiple of 8)", width, dim);
    if (!w || !pool || !slot_idx || (rows > 0 && (!x || !out)))
        return fail(NHM_ERR_NULL, "conv: x, w, slot_idx, conv_pool or out is NULL");
    if ((rows > 0 && (!rows16(x, ld_x * 2) || !rows16(out, ld_out * 2))) || !aligned(w, 16) || !aligned(b, 16) ||
        !aligned(pool, 16) || !aligned(slot_idx, 4))
        return fail(NHM_ERR_ALIGN, "conv: x, out (rows too), w, b and conv_pool must be 16-byte aligned");
    return NHM_OK;
}

ConvArgs conv_args(const uint16_t* x, int64_t ld_x, const uint16_t* w, const uint16_t* b, int32_t dim, int32_t silu,
                   const int32_t* slot_idx, uint16_t* pool, int32_t n_slots, uint16_t* out, int64_t ld_out) {
    ConvArgs a{};
    a.x = x; a.ld_x = ld_x;
    a.w = w; a.b = b; a.dim = dim;
    a.silu = silu != 0;
    a.slot_idx = slot_idx; a.pool = pool; a.n_slots = n_slots;
    a.out = out; a.ld_out = ld_out;
    return a;
}

// Checks what both forms of the scan share and fills in their arguments.
nhm_status scan_args(ScanDecodeArgs& a, const nhm_scan_params* p, const uint16_t* u, int64_t ld_u, const uint16_t* dt,
                     int64_t ld_dt, const uint16_t* B, int64_t ld_b, const uint16_t* C, int64_t ld_c, const uint16_t* z,
                     int64_t ld_z, int64_t rows, const int32_t* slot_idx, void* pool, nhm_dtype type, int32_t n_slots,
                     uint16_t* out, int64_t ld_out) {
    if (!p) return fail(NHM_ERR_NULL, "scan: params is NULL");
    if (type != NHM_F32 && type != NHM_BF16) return fail(NHM_ERR_UNSUPPORTED, "scan: state dtype %d: f32 or bf16", (int)type);
    if (rows < 0 || rows > INT_MAX || n_slots < 1 || p->dim < 1 || p->d_state < 1)
        return fail(NHM_ERR_SHAPE, "scan: rows %lld, dim %d, d_state %d or slots %d out of range", (long long)rows, p->dim,
                    p->d_state, n_slots);
    if (p->dim % 8 != 0 || p->d_state % 4 != 0 || p->d_state > 64)
        return fail(NHM_ERR_UNSUPPORTED, "scan: dim %d (a multiple of 8) and d_state %d (a multiple of 4, at most 64)", p->dim,
                    p->d_state);
    const int64_t lds[6] = {ld_u, ld_dt, ld_b, ld_c, z ? ld_z : p->dim, ld_out};
    for (int i = 0; i < 6; ++i)
        if (lds[i] < (i == 2 || i == 3 ? p->d_state : p->dim) || lds[i] > kMaxLd)
            return fail(NHM_ERR_SHAPE, "scan: a leading dimension of %lld is out of range", (long long)lds[i]);
    for (int i = 0; i < 6; ++i)
        if (lds[i] > kMaxScanLd) return fail(NHM_ERR_UNSUPPORTED, "scan: a leading dimension of more than 2^23");
    if (!p->A_log || !pool || !slot_idx || (rows > 0 && (!u || !dt || !B || !C || !out)))
        return fail(NHM_ERR_NULL, "scan: A_log, u, dt, B, C, slot_idx, ssm_pool or out is NULL");
    if (!aligned(p->A_log, 16) || !aligned(pool, 16) || !aligned(p->D, 4) || !aligned(p->dt_bias, 4) || !aligned(slot_idx, 4) ||
        !aligned(u, 2) || !aligned(dt, 2) || !aligned(B, 2) || !aligned(C, 2) || !aligned(z, 2) || !aligned(out, 2))
        return fail(NHM_ERR_ALIGN, "scan: A_log and ssm_pool must be 16-byte aligned, other tensors to their element size");
    a.u = u; a.dt = dt; a.B = B; a.C = C; a.z = z;
    a.ld_u = ld_u; a.ld_dt = ld_dt; a.ld_b = ld_b; a.ld_c = ld_c; a.ld_z = z ? ld_z : 0;
    a.A_log = p->A_log; a.D = p->D; a.dt_bias = p->dt_bias;
    a.dim = p->dim; a.d_state = p->d_state; a.n_slots = n_slots;
    a.slot_idx = slot_idx;
    a.pool = type == NHM_F32 ? static_cast<float*>(pool) : nullptr;
    a.pool_bf16 = type == NHM_BF16 ? static_cast<uint16_t*>(pool) : nullptr;
    a.out = out; a.ld_out = ld_out;
    return NHM_OK;
}

nhm_status check_seqs(const int32_t* cu_seqlens, int32_t n_seqs, const int32_t* slot_idx, const int32_t* has_initial,
                      int64_t n_tokens) {
    if (n_seqs < 0) return fail(NHM_ERR_SHAPE, "n_seqs %d out of range", n_seqs);
    if (n_seqs > 0 && (!cu_seqlens || !slot_idx || !has_initial))
        return fail(NHM_ERR_NULL, "cu_seqlens, slot_idx or has_initial is NULL");
    if (!aligned(cu_seqlens, 4) || !aligned(slot_idx, 4) || !aligned(has_initial, 4))
        return fail(NHM_ERR_ALIGN, "cu_seqlens, slot_idx and has_initial must be 4-byte aligned");
    return NHM_OK;
}

}  // namespace

extern "C" {

nhm_status nhm_mxfp4_quantize(const void* x, nhm_dtype type, int64_t rows, int64_t cols, int64_t ld_x, uint8_t* codes,
                              int64_t ld_codes, uint8_t* scales, int64_t ld_scales, void* stream) {
    clear_error();
    if (type != NHM_BF16 && type != NHM_F32) return fail(NHM_ERR_UNSUPPORTED, "mxfp4: input dtype %d: bf16 or f32", (int)type);
    if (rows < 0 || rows > INT_MAX || cols < 0 || cols > INT_MAX || cols % 32 != 0 || ld_x < cols || ld_codes < cols / 2 ||
        ld_scales < cols / 32 || ld_x > kMaxLd || ld_codes > kMaxLd || ld_scales > kMaxLd)
        return fail(NHM_ERR_SHAPE, "mxfp4: [%lld, %lld] (a multiple of 32; ld %lld, %lld, %lld) out of range", (long long)rows,
                    (long long)cols, (long long)ld_x, (long long)ld_codes, (long long)ld_scales);
    if (rows == 0 || cols == 0) return NHM_OK;
    if (!x || !codes || !scales) return fail(NHM_ERR_NULL, "mxfp4: x, codes or scales is NULL");
    if (!rows16(x, ld_x * (type == NHM_F32 ? 4 : 2)) || !aligned(codes, 4) || ld_codes % 4 != 0)
        return fail(NHM_ERR_ALIGN, "mxfp4: rows of x must be 16-byte aligned, rows of codes 4-byte aligned");
    return launch_mx_quant(MxQuantArgs{x, rows, cols, ld_x, codes, ld_codes, scales, ld_scales}, type == NHM_F32,
                           (hipStream_t)stream);
}

nhm_status nhm_mxfp4_dequantize(const uint8_t* codes, int64_t ld_codes, const uint8_t* scales, int64_t ld_scales,
                                int64_t rows, int64_t cols, uint16_t* out, int64_t ld_out, void* stream) {
    clear_error();
    if (rows < 0 || rows > INT_MAX || cols < 0 || cols > INT_MAX || cols % 32 != 0 || ld_out < cols || ld_codes < cols / 2 ||
        ld_scales < cols / 32 || ld_out > kMaxLd || ld_codes > kMaxLd || ld_scales > kMaxLd)
        return fail(NHM_ERR_SHAPE, "mxfp4: [%lld, %lld] (a multiple of 32; ld %lld, %lld, %lld) out of range", (long long)rows,
                    (long long)cols, (long long)ld_codes, (long long)ld_scales, (long long)ld_out);
    if (rows == 0 || cols == 0) return NHM_OK;
    if (!codes || !scales || !out) return fail(NHM_ERR_NULL, "mxfp4: codes, scales or out is NULL");
    if (!rows16(out, ld_out * 2) || !aligned(codes, 4) || ld_codes % 4 != 0)
        return fail(NHM_ERR_ALIGN, "mxfp4: rows of out must be 16-byte aligned, rows of codes 4-byte aligned");
    return launch_mx_dequant(MxDequantArgs{codes, ld_codes, scales, ld_scales, rows, cols, out, ld_out}, (hipStream_t)stream);
}

size_t nhm_mxfp4_linear_workspace_bytes(int64_t m, int64_t n, int64_t k, nhm_dtype a_type) {
    if (m <= 0 || n <= 0 || k <= 0 || m > INT_MAX || n > INT_MAX || k > INT_MAX) return 0;
    return mx_ws(m, n, k, a_type).total;
}

nhm_status nhm_mxfp4_linear(const void* a, nhm_dtype a_type, const uint8_t* a_scale, int64_t m, int64_t ld_a,
                            const nhm_mxfp4_weight* w, void* out, nhm_dtype out_type, int64_t ld_out, void* ws,
                            size_t ws_bytes, void* stream) {
    clear_error();
    if (!w) return fail(NHM_ERR_NULL, "mxfp4: weight is NULL");
    if (a_type != NHM_BF16 && a_type != NHM_MXFP4)
        return fail(NHM_ERR_UNSUPPORTED, "mxfp4: activation dtype %d: bf16 or MXFP4", (int)a_type);
    if (out_type != NHM_BF16 && out_type != NHM_F32)
        return fail(NHM_ERR_UNSUPPORTED, "mxfp4: output dtype %d: bf16 or f32", (int)out_type);
    const bool bf16 = a_type == NHM_BF16;
    if (m < 0 || m > INT_MAX || w->n < 1 || w->n > INT_MAX || w->k < 1 || w->k > INT_MAX || w->k % 32 != 0 ||
        ld_a < (bf16 ? w->k : w->k / 2) || ld_out < w->n || ld_a > kMaxLd || ld_out > kMaxLd)
        return fail(NHM_ERR_SHAPE, "mxfp4: m %lld, n %lld, k %lld (a multiple of 32; ld %lld, %lld) out of range", (long long)m,
                    (long long)w->n, (long long)w->k, (long long)ld_a, (long long)ld_out);
    if (m == 0) return NHM_OK;
    if (!aligned(w->packed_scale, 4)) return fail(NHM_ERR_ALIGN, "mxfp4: the weight's packed scales must be 4-byte aligned");
    if (!a || !w->w || !w->scale || !out || (!bf16 && !a_scale))
        return fail(NHM_ERR_NULL, "mxfp4: a, a_scale, the weight's codes or scales, or out is NULL");
    if (!rows16(a, ld_a * (bf16 ? 2 : 1)) || !aligned(w->w, 16) || !aligned(out, out_type == NHM_F32 ? 4 : 2))
        return fail(NHM_ERR_ALIGN, "mxfp4: rows of a and the weight's codes must be 16-byte aligned, out to its element size");
    const int64_t ld_q = bf16 ? w->k / 2 : ld_a;
    if (w->n > (kMaxOperand - 1) / (w->k / 2) || m > (kMaxOperand - 1) / ld_q)
        return fail(NHM_ERR_UNSUPPORTED, "mxfp4: an operand of 2 GiB or more");
    // up to 64 rows: workgroups of 512 threads take 16 features each
    if (!mx_tiled(m) && (w->n + 15) / 16 > kMaxThreads / 512)
        return fail(NHM_ERR_UNSUPPORTED, "mxfp4: %lld features are more than a launch holds", (long long)w->n);
    const MxWs l = mx_ws(m, w->n, w->k, a_type);
    if (l.total > 0 && (!ws || ws_bytes < l.total))
        return fail(NHM_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", l.total, ws ? ws_bytes : (size_t)0);
    if (l.total > 0 && !aligned(ws, 256)) return fail(NHM_ERR_ALIGN, "ws must be 256-byte aligned");
    hipStream_t st = (hipStream_t)stream;
    MxGemmArgs g{};
    g.a = static_cast<const uint8_t*>(a); g.ld_a = ld_q;
    g.a_scale = a_scale; g.ld_as = w->k / 32;
    g.m = m; g.n = w->n; g.k = w->k;
    g.w = w->w; g.w_scale = w->scale; g.ld_ws = w->k / 32;
    g.out = out_type == NHM_BF16 ? static_cast<uint16_t*>(out) : nullptr;
    g.out_f32 = out_type == NHM_F32 ? static_cast<float*>(out) : nullptr;
    g.ld_out = ld_out;
    const size_t four = out_type == NHM_F32 ? 16 : 8;
    g.vec_out = aligned(out, four) && ld_out % 4 == 0;
    uint8_t* const wsb = static_cast<uint8_t*>(ws);
    uint32_t* const packed = mx_tiled(m) ? reinterpret_cast<uint32_t*>(wsb + l.scales) : nullptr;
    nhm_status s = NHM_OK;
    if (bf16 && mx_rows_quantise(m, w->k)) {
        g.a_bf16 = static_cast<const uint16_t*>(a);
        g.ld_bf16 = ld_a;
    } else if (bf16) {
        MxQuantArgs q{a, m, w->k, ld_a, wsb, ld_q, wsb + l.scales, w->k / 32};
        q.packed = packed;
        s = launch_mx_quant(q, false, st);
        g.a = wsb;
        g.a_scale = wsb + l.scales;
    } else if (packed) {
        s = launch_mx_pack(a_scale, m, w->k, packed, st);
    }
    if (s != NHM_OK) return s;
    g.a_packed = packed;
    g.w_packed = w->packed_scale;
    if (packed && !w->packed_scale) {
        uint32_t* const wp = reinterpret_cast<uint32_t*>(wsb + l.weight);
        if ((s = launch_mx_pack(w->scale, w->n, w->k, wp, st)) != NHM_OK) return s;
        g.w_packed = wp;
    }
    return launch_mx_gemm(g, st);
}

size_t nhm_mxfp4_packed_scale_bytes(int64_t n, int64_t k) {
    if (n <= 0 || k <= 0 || n > INT_MAX || k > INT_MAX || k % 32 != 0) return 0;
    return (size_t)mx_packed_words(n, k) * 4;
}

nhm_status nhm_mxfp4_pack_scales(const uint8_t* scale, int64_t n, int64_t k, uint32_t* packed, void* stream) {
    clear_error();
    if (n < 0 || k < 0 || n > INT_MAX || k > INT_MAX || k % 32 != 0)
        return fail(NHM_ERR_SHAPE, "mxfp4: scales of [%lld, %lld] (a multiple of 32) out of range", (long long)n, (long long)k);
    if (n == 0 || k == 0) return NHM_OK;
    if (!scale || !packed) return fail(NHM_ERR_NULL, "mxfp4: scale or packed is NULL");
    if (!aligned(packed, 4)) return fail(NHM_ERR_ALIGN, "mxfp4: packed must be 4-byte aligned");
    if (mx_packed_words(n, k) >= kMaxOperand / 4) return fail(NHM_ERR_UNSUPPORTED, "mxfp4: scales of 2 GiB or more");
    return launch_mx_pack(scale, n, k, packed, (hipStream_t)stream);
}

nhm_status nhm_causal_conv_decode(const uint16_t* x, int64_t ld_x, const uint16_t* w, const uint16_t* b, int32_t dim,
                                  int32_t width, int32_t silu, int32_t batch, const int32_t* slot_idx,
                                  uint16_t* conv_pool, int32_t n_slots, uint16_t* out, int64_t ld_out, void* stream) {
    clear_error();
    const nhm_status s = check_conv(x, ld_x, batch, w, b, dim, width, slot_idx, conv_pool, n_slots, out, ld_out);
    if (s != NHM_OK || batch == 0) return s;
    return launch_conv_decode(conv_args(x, ld_x, w, b, dim, silu, slot_idx, conv_pool, n_slots, out, ld_out), width, batch,
                              (hipStream_t)stream);
}

nhm_status nhm_causal_conv_prefill(const uint16_t* x, int64_t ld_x, int64_t n_tokens, const uint16_t* w, const uint16_t* b,
                                   int32_t dim, int32_t width, int32_t silu, const int32_t* cu_seqlens, int32_t n_seqs,
                                   const int32_t* slot_idx, const int32_t* has_initial, uint16_t* conv_pool,
                                   int32_t n_slots, uint16_t* out, int64_t ld_out, void* stream) {
    clear_error();
    nhm_status s = check_seqs(cu_seqlens, n_seqs, slot_idx, has_initial, n_tokens);
    if (s != NHM_OK) return s;
    if (n_tokens == 0 && n_seqs == 0) return NHM_OK;
    // without sequences (a batch of padding alone) there are no slots to name
    s = check_conv(x, ld_x, n_tokens, w, b, dim, width, n_seqs > 0 ? slot_idx : reinterpret_cast<const int32_t*>(conv_pool), conv_pool,
                   n_slots, out, ld_out);
    if (s != NHM_OK) return s;
    if ((n_tokens / 8 + 4) * (((int64_t)dim + 511) / 512) > kMaxThreads / 64)
        return fail(NHM_ERR_UNSUPPORTED, "conv: %lld tokens of %d channels are more than a launch holds", (long long)n_tokens, dim);
    ConvArgs a = conv_args(x, ld_x, w, b, dim, silu, slot_idx, conv_pool, n_slots, out, ld_out);
    a.n_tokens = n_tokens; a.n_seqs = n_seqs;
    a.cu_seqlens = cu_seqlens; a.has_initial = has_initial;
    return launch_conv_prefill(a, width, (hipStream_t)stream);
}

nhm_status nhm_selective_scan_decode(const nhm_scan_params* p, const uint16_t* u, int64_t ld_u, const uint16_t* dt,
                                     int64_t ld_dt, const uint16_t* B, int64_t ld_b, const uint16_t* C, int64_t ld_c,
                                     const uint16_t* z, int64_t ld_z, int32_t batch, const int32_t* slot_idx,
                                     void* ssm_pool, nhm_dtype ssm_type, int32_t n_slots, uint16_t* out, int64_t ld_out,
                                     void* stream) {
    clear_error();
    ScanDecodeArgs a{};
    const nhm_status s = scan_args(a, p, u, ld_u, dt, ld_dt, B, ld_b, C, ld_c, z, ld_z, batch, slot_idx, ssm_pool, ssm_type, n_slots,
                                   out, ld_out);
    if (s != NHM_OK || batch == 0) return s;
    return launch_scan_decode(a, batch, (hipStream_t)stream);
}

size_t nhm_selective_scan_prefill_workspace_bytes(int32_t dim, int32_t d_state, int64_t n_tokens, int32_t n_seqs) {
    if (dim <= 0 || d_state <= 0 || n_tokens <= 0 || n_seqs <= 0 || n_tokens > INT_MAX) return 0;
    return scan_ws_bytes(dim, d_state, n_tokens, n_seqs);
}

nhm_status nhm_selective_scan_prefill(const nhm_scan_params* p, const uint16_t* u, int64_t ld_u, const uint16_t* dt,
                                      int64_t ld_dt, const uint16_t* B, int64_t ld_b, const uint16_t* C, int64_t ld_c,
                                      const uint16_t* z, int64_t ld_z, int64_t n_tokens, const int32_t* cu_seqlens,
                                      int32_t n_seqs, const int32_t* slot_idx, const int32_t* has_initial, void* ssm_pool,
                                      nhm_dtype ssm_type, int32_t n_slots, uint16_t* out, int64_t ld_out, void* ws,
                                      size_t ws_bytes, void* stream) {
    clear_error();
    nhm_status s = check_seqs(cu_seqlens, n_seqs, slot_idx, has_initial, n_tokens);
    if (s != NHM_OK) return s;
    if (n_tokens == 0 && n_seqs == 0) return NHM_OK;
    ScanPrefillArgs a{};
    s = scan_args(a, p, u, ld_u, dt, ld_dt, B, ld_b, C, ld_c, z, ld_z, n_tokens,
                  n_seqs > 0 ? slot_idx : static_cast<const int32_t*>(ssm_pool), ssm_pool, ssm_type, n_slots, out, ld_out);
    if (s != NHM_OK) return s;
    const ScanSplit sp = scan_split(p->dim, n_tokens, n_seqs);
    // workgroups of 256 threads: 16 channels of a chunk each, rounded up to units of 8 x 4
    if (((int64_t)n_seqs + 1) * sp.n_chunks > (kMaxThreads / 256 - 32) / (((int64_t)p->dim + 63) / 64 * 4))
        return fail(NHM_ERR_UNSUPPORTED, "scan: %d sequences of %d channels are more than a launch holds", n_seqs, p->dim);
    const size_t need = nhm_selective_scan_prefill_workspace_bytes(p->dim, p->d_state, n_tokens, n_seqs);
    if (need > 0 && (!ws || ws_bytes < need))
        return fail(NHM_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? ws_bytes : (size_t)0);
    if (need > 0 && !aligned(ws, 256)) return fail(NHM_ERR_ALIGN, "ws must be 256-byte aligned");
    a.n_tokens = n_tokens; a.n_seqs = n_seqs;
    a.cu_seqlens = cu_seqlens; a.has_initial = has_initial;
    return launch_scan_prefill(a, need > 0 ? ws : nullptr, (hipStream_t)stream);
}

size_t nhm_token_logprobs_workspace_bytes(int64_t rows, int64_t vocab, int32_t n_top) {
    if (rows <= 0 || rows >= kMaxRows || vocab < 1 || vocab > kMaxVocab || n_top < 0 || n_top > kMaxTop) return 0;
    return score_ws_bytes(rows, vocab, n_top);
}

nhm_status nhm_token_logprobs(const void* logits, nhm_dtype type, int64_t ld, int64_t rows, int64_t vocab,
                              const int32_t* tokens, int32_t n_top, float* logprobs, int32_t* ranks, float* entropy,
                              float* top_logprobs, int32_t* top_tokens, void* ws, size_t ws_bytes, void* stream) {
    clear_error();
    if (type != NHM_BF16 && type != NHM_F32) return fail(NHM_ERR_UNSUPPORTED, "logits dtype %d: bf16 or f32", (int)type);
    if (rows < 0 || vocab < 1 || n_top < 0 || ld < vocab || ld > kMaxLd)
        return fail(NHM_ERR_SHAPE, "rows %lld, vocab %lld (ld %lld) or n_top %d out of range", (long long)rows, (long long)vocab,
                    (long long)ld, n_top);
    if (n_top > kMaxTop || vocab > kMaxVocab || rows >= kMaxRows)
        return fail(NHM_ERR_UNSUPPORTED, "at most %d alternatives, a vocabulary of 2^24 and fewer than 2^24 rows", kMaxTop);
    if (rows == 0) return NHM_OK;
    if (!logits || (n_top > 0 && (!top_logprobs || !top_tokens)))
        return fail(NHM_ERR_NULL, "logits, top_logprobs or top_tokens is NULL");
    if (!aligned(logits, type == NHM_F32 ? 4 : 2) || !aligned(tokens, 4) || !aligned(logprobs, 4) || !aligned(ranks, 4) ||
        !aligned(entropy, 4) || !aligned(top_logprobs, 4) || !aligned(top_tokens, 4))
        return fail(NHM_ERR_ALIGN, "every tensor must be aligned to its element size");
    const size_t need = score_ws_bytes(rows, vocab, n_top);
    if (!ws || ws_bytes < need)
        return fail(NHM_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? ws_bytes : (size_t)0);
    if (!aligned(ws, 256)) return fail(NHM_ERR_ALIGN, "ws must be 256-byte aligned");
    ScoreArgs g{};
    g.logits = logits; g.f32 = type == NHM_F32;
    g.ld = ld; g.rows = rows; g.vocab = vocab;
    g.tokens = tokens; g.n_top = n_top;
    g.logprobs = logprobs; g.ranks = ranks; g.entropy = entropy;
    g.top_logprobs = top_logprobs; g.top_tokens = top_tokens;
    return launch_score(g, ws, (hipStream_t)stream);
}

}  // extern "C"
