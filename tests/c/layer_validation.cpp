// Host-only driver for an AddressSanitizer / UndefinedBehaviorSanitizer build of the layer operators'
// validation (csrc/layer.hip). Every call below fails validation before anything is enqueued, is an
// empty call or a pure host query, so no GPU is needed; the kernel launchers are replaced by stubs that
// abort if reached.
#include <limits.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <hip/hip_runtime.h>

#include "../../fp8_w8a8_linear_amd/csrc/nhm_internal.h"   // the launchers' declarations

namespace nhm {
static char g_err[512];
nhm_status fail(nhm_status s, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof(g_err), fmt, ap);
    va_end(ap);
    return s;
}
void clear_error() { g_err[0] = 0; }
[[noreturn]] static void reached(const char* f) {
    fprintf(stderr, "kernel launcher %s reached from a call that should have failed validation\n", f);
    abort();
}
nhm_status launch_conv_prefill(const ConvArgs&, int32_t, hipStream_t) { reached("launch_conv_prefill"); }
nhm_status launch_conv_decode(const ConvArgs&, int32_t, int32_t, hipStream_t) { reached("launch_conv_decode"); }
nhm_status launch_scan_decode(const ScanDecodeArgs&, int32_t, hipStream_t) { reached("launch_scan_decode"); }
ScanSplit scan_split(int64_t, int64_t, int64_t) { return ScanSplit{4, 64}; }
size_t scan_ws_bytes(int64_t dim, int32_t n, int64_t, int64_t seqs) { return (size_t)dim * n * seqs * 4; }
nhm_status launch_scan_prefill(ScanPrefillArgs, void*, hipStream_t) { reached("launch_scan_prefill"); }
nhm_status launch_mx_quant(const MxQuantArgs&, bool, hipStream_t) { reached("launch_mx_quant"); }
nhm_status launch_mx_dequant(const MxDequantArgs&, hipStream_t) { reached("launch_mx_dequant"); }
bool mx_tiled(int64_t m) { return m > 64; }
nhm_status launch_mx_pack(const uint8_t*, int64_t, int64_t, uint32_t*, hipStream_t) { reached("launch_mx_pack"); }
nhm_status launch_mx_gemm(const MxGemmArgs&, hipStream_t) { reached("launch_mx_gemm"); }
size_t score_ws_bytes(int64_t rows, int64_t, int32_t) { return (size_t)rows * 16; }
nhm_status launch_score(ScoreArgs, void*, hipStream_t) { reached("launch_score"); }
}  // namespace nhm

static int failures = 0;
#define EXPECT(call, want)                                                                        \
    do {                                                                                          \
        const int got_ = (int)(call);                                                             \
        if (got_ != (int)(want)) {                                                                \
            fprintf(stderr, "line %d: %s -> %d, expected %d (%s)\n", __LINE__, #call, got_, (int)(want), \
                    nhm::g_err);                                                                  \
            ++failures;                                                                           \
        }                                                                                         \
    } while (0)

template <typename T>
static T* P(uintptr_t v) { return reinterpret_cast<T*>(v); }

int main() {
    const int64_t extremes[] = {INT64_MIN, -1, INT64_MAX, INT64_MAX - 31, (int64_t(1) << 40) + 32};
    uint16_t* const H = P<uint16_t>(0x10000);
    uint8_t* const Q = P<uint8_t>(0x20000);
    int32_t* const I = P<int32_t>(0x30000);
    float* const F = P<float>(0x40000);
    void* const WS = P<void>(0x50000);
    // MXFP4
    for (int64_t v : extremes) {
        EXPECT(nhm_mxfp4_quantize(H, NHM_BF16, v, 64, 64, Q, 32, Q, 2, nullptr), NHM_ERR_SHAPE);
        EXPECT(nhm_mxfp4_quantize(H, NHM_BF16, 4, v, INT64_MAX, Q, INT64_MAX, Q, INT64_MAX, nullptr), NHM_ERR_SHAPE);
        EXPECT(nhm_mxfp4_dequantize(Q, 32, Q, 2, v, 64, H, 64, nullptr), NHM_ERR_SHAPE);
        if (v > 0) EXPECT(nhm_mxfp4_quantize(H, NHM_BF16, 4, 64, v, Q, 32, Q, 2, nullptr), NHM_ERR_SHAPE);
        nhm_mxfp4_weight w = {Q, Q, v, 64, nullptr};
        EXPECT(nhm_mxfp4_linear(H, NHM_BF16, nullptr, 4, 64, &w, H, NHM_BF16, INT64_MAX, WS, SIZE_MAX, nullptr), NHM_ERR_SHAPE);
        w = nhm_mxfp4_weight{Q, Q, 64, v, nullptr};
        EXPECT(nhm_mxfp4_linear(H, NHM_BF16, nullptr, 4, INT64_MAX, &w, H, NHM_BF16, 64, WS, SIZE_MAX, nullptr), NHM_ERR_SHAPE);
        w = nhm_mxfp4_weight{Q, Q, 64, 64, nullptr};
        EXPECT(nhm_mxfp4_linear(H, NHM_BF16, nullptr, v, 64, &w, H, NHM_BF16, 64, WS, SIZE_MAX, nullptr), NHM_ERR_SHAPE);
        nhm_mxfp4_linear_workspace_bytes(v, v, v, NHM_BF16);
        EXPECT(nhm_mxfp4_pack_scales(Q, v, 64, P<uint32_t>(0x60000), nullptr), NHM_ERR_SHAPE);
        EXPECT(nhm_mxfp4_pack_scales(Q, 64, v, P<uint32_t>(0x60000), nullptr), NHM_ERR_SHAPE);
        EXPECT(nhm_mxfp4_packed_scale_bytes(v, 64), 0);
    }
    const nhm_mxfp4_weight w = {Q, Q, 64, 64, nullptr};
    EXPECT(nhm_mxfp4_linear(H, (nhm_dtype)INT_MIN, nullptr, 4, 64, &w, H, NHM_BF16, 64, WS, SIZE_MAX, nullptr), NHM_ERR_UNSUPPORTED);
    EXPECT(nhm_mxfp4_linear(H, NHM_BF16, nullptr, 4, 64, &w, H, (nhm_dtype)77, 64, WS, SIZE_MAX, nullptr), NHM_ERR_UNSUPPORTED);
    EXPECT(nhm_mxfp4_linear(H, NHM_BF16, nullptr, INT_MAX, 64, &w, H, NHM_BF16, 64, WS, SIZE_MAX, nullptr), NHM_ERR_UNSUPPORTED);
    EXPECT(nhm_mxfp4_linear(H, NHM_BF16, nullptr, 0, 64, &w, nullptr, NHM_BF16, 64, nullptr, 0, nullptr), NHM_OK);
    // convolution and scan
    for (int64_t v : extremes) {
        EXPECT(nhm_causal_conv_prefill(H, 64, v, H, H, 64, 4, 1, I, 2, I, I, H, 4, H, 64, nullptr), NHM_ERR_SHAPE);
        if (v > 64 || v < 0) EXPECT(nhm_causal_conv_decode(H, v, H, H, 64, 4, 1, 2, I, H, 4, H, 64, nullptr), NHM_ERR_SHAPE);
        const nhm_scan_params p = {F, F, F, 64, 16};
        EXPECT(nhm_selective_scan_prefill(&p, H, 64, H, 64, H, 16, H, 16, H, 64, v, I, 2, I, I, F, NHM_F32, 4, H, 64, WS, SIZE_MAX,
                                          nullptr), NHM_ERR_SHAPE);
        EXPECT(nhm_selective_scan_decode(&p, H, v, H, 64, H, 16, H, 16, H, 64, 2, I, F, NHM_F32, 4, H, 64, nullptr), NHM_ERR_SHAPE);
        nhm_selective_scan_prefill_workspace_bytes(64, 16, v, 2);
    }
    const nhm_scan_params wide = {F, F, F, INT_MAX - 7, 64};
    EXPECT(nhm_selective_scan_prefill(&wide, H, INT_MAX, H, INT_MAX, H, 64, H, 64, nullptr, 0, 8, I, INT_MAX, I, I, F, NHM_F32, 4, H,
                                      INT_MAX, WS, SIZE_MAX, nullptr), NHM_ERR_UNSUPPORTED);
    EXPECT(nhm_causal_conv_prefill(H, INT_MAX - 7, INT_MAX, H, H, INT_MAX - 7, 4, 1, I, INT_MAX, I, I, H, 4, H, INT_MAX - 7, nullptr),
           NHM_ERR_UNSUPPORTED);
    EXPECT(nhm_causal_conv_prefill(H, int64_t(1) << 31, INT_MAX, H, H, INT_MAX - 7, 4, 1, I, INT_MAX, I, I, H, 4, H, int64_t(1) << 31,
                                   nullptr), NHM_ERR_UNSUPPORTED);
    // scores
    for (int64_t v : extremes) {
        EXPECT(nhm_token_logprobs(H, NHM_BF16, INT64_MAX, v, 100, I, 0, F, I, F, F, I, WS, SIZE_MAX, nullptr), NHM_ERR_SHAPE);
        EXPECT(nhm_token_logprobs(H, NHM_BF16, 100, v, 100, I, 0, F, I, F, F, I, WS, SIZE_MAX, nullptr), v < 0 ? NHM_ERR_SHAPE : NHM_ERR_UNSUPPORTED);
        if (v > 0) EXPECT(nhm_token_logprobs(H, NHM_BF16, int64_t(1) << 40, 4, v, I, 0, F, I, F, F, I, WS, SIZE_MAX, nullptr), NHM_ERR_SHAPE);
        nhm_token_logprobs_workspace_bytes(v, v, 5);
    }
    EXPECT(nhm_token_logprobs(H, NHM_BF16, 100, 4, 100, I, INT_MAX, F, I, F, F, I, WS, SIZE_MAX, nullptr), NHM_ERR_UNSUPPORTED);
    EXPECT(nhm_token_logprobs(H, NHM_BF16, 100, 4, 100, I, INT_MIN, F, I, F, F, I, WS, SIZE_MAX, nullptr), NHM_ERR_SHAPE);
    if (failures == 0) printf("layer validation ok\n");
    return failures ? 1 : 0;
}
