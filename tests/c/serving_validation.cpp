// Host-only driver for an AddressSanitizer / UndefinedBehaviorSanitizer build of the serving
// operators' validation (csrc/serving.hip with csrc/api.hip). Every call below fails validation
// before anything is enqueued, is an empty call or a pure host query, so no GPU is needed; the
// kernel launchers of the other translation units are replaced by stubs that abort if reached.
#include <limits.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <hip/hip_runtime.h>

#include "../../fp8_w8a8_linear_amd/csrc/nhm_internal.h"   // the launchers' declarations

namespace nhm {
[[noreturn]] static void reached(const char* f) {
    fprintf(stderr, "kernel launcher %s reached from a call that should have failed validation\n", f);
    abort();
}
void launch_quantize(const uint16_t*, int64_t, int64_t, int64_t, const float*, uint8_t*, int64_t, hipStream_t) {
    reached("launch_quantize");
}
void launch_dequant_channel(const uint8_t*, int64_t, int64_t, int64_t, const float*, uint16_t*, int64_t, hipStream_t) {
    reached("launch_dequant_channel");
}
nhm_status launch_gemv(const uint8_t*, int64_t, int, const uint8_t*, const float*, const float*, int64_t, int64_t,
                       uint16_t*, int64_t, hipStream_t, float*, uint8_t*, int64_t, const float*, uint32_t*, int, int) {
    reached("launch_gemv");
}
size_t gemm_part_bytes(int64_t, int64_t, int64_t) { return 0; }
nhm_status launch_gemm(const uint8_t*, int64_t, int64_t, const uint8_t*, const float*, const float*, int64_t, int64_t,
                       uint16_t*, int64_t, hipStream_t, float*, float*, size_t, bool, int) {
    reached("launch_gemm");
}
nhm_status launch_decode_ssm(const DecodeSsmArgs&, int, hipStream_t) { reached("launch_decode_ssm"); }
void launch_clear(uint32_t*, int, hipStream_t) { reached("launch_clear"); }
nhm_status launch_gnorm_quant(const GnormArgs&, hipStream_t) { reached("launch_gnorm_quant"); }
nhm_status launch_prefill_mid(const PrefillArgs&, hipStream_t) { reached("launch_prefill_mid"); }
nhm_status launch_lora_down(const LoraDownArgs&, hipStream_t) { reached("launch_lora_down"); }
nhm_status launch_gemv_lora(const uint8_t*, int64_t, int, const uint8_t*, const float*, const float*, int64_t, int64_t,
                            uint16_t*, int64_t, hipStream_t, float*, int, const LoraEpi&, uint32_t*, int) {
    reached("launch_gemv_lora");
}
nhm_status launch_gemm_lora(const uint8_t*, int64_t, int64_t, const uint8_t*, const float*, const float*, int64_t, int64_t,
                            uint16_t*, int64_t, hipStream_t, float*, bool, int, const LoraEpi&) {
    reached("launch_gemm_lora");
}
size_t beam_ws_bytes(int64_t rows, int64_t, int32_t) { return (size_t)rows * 16; }
nhm_status launch_beam_select(BeamArgs, void*, hipStream_t) { reached("launch_beam_select"); }
nhm_status launch_beam_reorder(const ReorderArgs&, int64_t, int32_t, hipStream_t) { reached("launch_beam_reorder"); }
nhm_status launch_batch_plan(const PlanArgs&, hipStream_t) { reached("launch_batch_plan"); }
}  // namespace nhm

static int failures = 0;
#define EXPECT(call, want)                                                                        \
    do {                                                                                          \
        const int got_ = (int)(call);                                                             \
        if (got_ != (int)(want)) {                                                                \
            fprintf(stderr, "line %d: %s -> %d, expected %d (%s)\n", __LINE__, #call, got_, (int)(want), \
                    nhm_last_error());                                                            \
            ++failures;                                                                           \
        }                                                                                         \
    } while (0)

template <typename T>
static T* P(uintptr_t v) { return reinterpret_cast<T*>(v); }

int main() {
    // adapters
    const nhm_fp8_weight w = {P<uint8_t>(0x1000), P<float>(0x2000), P<float>(0x3000), 64, 128, 0};
    const nhm_lora l = {P<uint16_t>(0x4000), P<uint16_t>(0x5000), nullptr, 4, 16};
    const size_t need = nhm_fp8_linear_lora_workspace_bytes(32, 64, 128, NHM_BF16, 16);
    EXPECT(need > 0, 1);
    EXPECT(nhm_fp8_linear_lora_workspace_bytes(INT64_MIN, 64, 128, NHM_BF16, 16), 0);
    auto lora = [&](int64_t m, const nhm_fp8_weight* wp, const nhm_lora* lp, void* ws, size_t wsb, nhm_dtype t = NHM_BF16) {
        return nhm_fp8_linear_lora(P<void>(0x10000), t, m, 128, wp, lp, P<int32_t>(0x6000), P<void>(0x20000), NHM_BF16, 64,
                                   0, ws, wsb, nullptr);
    };
    EXPECT(lora(0, &w, &l, nullptr, 0), NHM_OK);
    EXPECT(lora(32, nullptr, &l, P<void>(0x40000), need), NHM_ERR_NULL);
    EXPECT(lora(32, &w, nullptr, P<void>(0x40000), need), NHM_ERR_NULL);
    EXPECT(lora(32, &w, &l, P<void>(0x40000), need - 1), NHM_ERR_WORKSPACE);
    EXPECT(lora(32, &w, &l, P<void>(0x40010), need), NHM_ERR_ALIGN);
    EXPECT(lora(-5, &w, &l, P<void>(0x40000), need), NHM_ERR_SHAPE);
    EXPECT(lora(32, &w, &l, P<void>(0x40000), need, (nhm_dtype)-77), NHM_ERR_UNSUPPORTED);
    nhm_fp8_weight bad = w;
    bad.k = -16;
    EXPECT(lora(32, &bad, &l, P<void>(0x40000), need), NHM_ERR_SHAPE);
    bad.k = INT64_MAX;
    EXPECT(lora(32, &bad, &l, P<void>(0x40000), need), NHM_ERR_SHAPE);
    nhm_lora lb = l;
    lb.rank = INT_MIN;
    EXPECT(lora(32, &w, &lb, P<void>(0x40000), need), NHM_ERR_UNSUPPORTED);
    lb = l;
    lb.n_adapters = INT_MIN;
    EXPECT(lora(32, &w, &lb, P<void>(0x40000), need), NHM_ERR_SHAPE);

    // the mixer with adapters
    {
        const nhm_geometry geo = {2688, 64, 64, 128, 8, 4, 1e-5f};
        nhm_mixer_params mp = {geo, {P<uint8_t>(0x1000), P<float>(0x2000), P<float>(0x3000), 10304, 2688, 0},
                               {P<uint8_t>(0x1000), P<float>(0x2000), P<float>(0x3000), 2688, 4096, 0},
                               P<uint16_t>(0x4000), P<uint16_t>(0x5000), P<uint16_t>(0x6000), P<float>(0x7000),
                               P<float>(0x8000), P<float>(0x9000)};
        nhm_ws_layout lay;
        EXPECT(nhm_mixer_decode_lora_ws_layout(&geo, 8, 16, &lay), NHM_OK);
        const size_t dec = lay.total;
        EXPECT(nhm_mixer_prefill_lora_ws_layout(&geo, 512, 2, 128, 16, &lay), NHM_OK);
        const size_t pre = lay.total;
        EXPECT(nhm_mixer_decode_lora_ws_layout(&geo, 8, INT_MIN, &lay), NHM_ERR_UNSUPPORTED);
        EXPECT(nhm_mixer_decode_lora_ws_layout(nullptr, 8, 16, &lay), NHM_ERR_NULL);
        EXPECT(nhm_mixer_prefill_lora_ws_layout(&geo, 512, 2, 128, INT_MAX, &lay), NHM_ERR_UNSUPPORTED);
        auto decode = [&](const nhm_lora* in, const nhm_lora* out, int32_t batch, size_t wsb, const int32_t* ids) {
            return nhm_mixer_decode_lora(&mp, in, out, ids, P<uint16_t>(0x10000), batch, P<int32_t>(0x20000),
                                         P<void>(0x30000), NHM_F32, P<uint16_t>(0x40000), 16, P<uint16_t>(0x50000),
                                         P<void>(0x60000), wsb, nullptr);
        };
        auto prefill = [&](const nhm_lora* in, const nhm_lora* out, int64_t T, size_t wsb) {
            return nhm_mixer_prefill_lora(&mp, in, out, P<int32_t>(0x70000), P<uint16_t>(0x10000), T, P<int32_t>(0x80000), 2,
                                          P<int32_t>(0x20000), P<int32_t>(0x90000), 128, P<void>(0x30000), NHM_F32,
                                          P<uint16_t>(0x40000), 16, P<uint16_t>(0x50000), P<void>(0x60000), wsb, nullptr);
        };
        EXPECT(decode(&l, &l, 0, 0, nullptr), NHM_OK);
        EXPECT(decode(&l, &l, 8, dec - 1, P<int32_t>(0x70000)), NHM_ERR_WORKSPACE);
        EXPECT(decode(&l, &l, 8, dec, nullptr), NHM_ERR_NULL);
        EXPECT(decode(&l, &l, 8, dec, P<int32_t>(0x70001)), NHM_ERR_ALIGN);
        EXPECT(decode(&l, &l, INT_MIN, dec, P<int32_t>(0x70000)), NHM_ERR_SHAPE);
        EXPECT(decode(&l, &l, INT_MAX, dec, P<int32_t>(0x70000)) != NHM_OK, 1);
        EXPECT(decode(nullptr, &lb, 8, dec, P<int32_t>(0x70000)), NHM_ERR_SHAPE);
        EXPECT(prefill(&l, &l, 512, pre - 1), NHM_ERR_WORKSPACE);
        EXPECT(prefill(&l, &l, INT64_MAX, SIZE_MAX), NHM_ERR_SHAPE);
        EXPECT(prefill(&l, &l, INT64_MIN, SIZE_MAX), NHM_ERR_SHAPE);
        mp.in_proj.n = INT64_MAX;
        EXPECT(decode(&l, nullptr, 8, dec, P<int32_t>(0x70000)), NHM_ERR_UNSUPPORTED);
        mp.in_proj.n = INT64_MIN;
        EXPECT(decode(&l, nullptr, 8, dec, P<int32_t>(0x70000)), NHM_ERR_SHAPE);
    }

    // selection
    auto select = [&](nhm_dtype t, int64_t ld, int64_t G, int32_t K, int64_t V, int32_t n, void* ws, size_t wsb) {
        return nhm_beam_select(P<void>(0x1000), t, ld, G, K, V, P<float>(0x2000), nullptr, 0, n, P<float>(0x3000),
                               P<int32_t>(0x4000), P<int32_t>(0x5000), ws, wsb, nullptr);
    };
    EXPECT(nhm_beam_select_workspace_bytes(2, 4, 1000, 8) > 0, 1);
    EXPECT(nhm_beam_select_workspace_bytes(INT64_MAX, 4, 1000, 8), 0);
    EXPECT(nhm_beam_select_workspace_bytes(2, 4, INT64_MAX, 8), 0);
    EXPECT(select(NHM_F32, 1000, 0, 4, 1000, 8, nullptr, 0), NHM_OK);
    EXPECT(select(NHM_F32, INT64_MAX, 2, 4, INT64_MAX, 8, P<void>(0x40000), SIZE_MAX), NHM_ERR_UNSUPPORTED);
    EXPECT(select(NHM_F32, 1000, INT64_MAX, 4, 1000, 8, P<void>(0x40000), SIZE_MAX), NHM_ERR_UNSUPPORTED);
    EXPECT(select(NHM_F32, 1000, 2, INT_MIN, 1000, 8, P<void>(0x40000), SIZE_MAX), NHM_ERR_SHAPE);
    EXPECT(select(NHM_F32, 1000, 2, 4, 1000, 8, P<void>(0x40000), 1), NHM_ERR_WORKSPACE);
    EXPECT(select((nhm_dtype)INT_MAX, 1000, 2, 4, 1000, 8, P<void>(0x40000), SIZE_MAX), NHM_ERR_UNSUPPORTED);

    // reorder
    nhm_geometry g = {2688, 64, 64, 128, 8, 4, 1e-5f};
    nhm_state_pool pools[65];
    for (auto& p : pools) p = nhm_state_pool{P<void>(0x100000), P<uint16_t>(0x200000)};
    auto reorder = [&](int64_t G, int32_t K, int32_t layers, int32_t* out, int32_t S = 16) {
        return nhm_beam_reorder(&g, P<int32_t>(0x1000), P<int32_t>(0x2000), G, K, pools, layers, NHM_F32, S, out, nullptr);
    };
    EXPECT(reorder(0, 4, 2, P<int32_t>(0x3000)), NHM_OK);
    EXPECT(reorder(2, 4, 65, P<int32_t>(0x3000)), NHM_ERR_UNSUPPORTED);
    EXPECT(reorder(INT64_MAX, 4, 2, P<int32_t>(0x3000)), NHM_ERR_UNSUPPORTED);
    EXPECT(reorder(2, 4, INT_MIN, P<int32_t>(0x3000)), NHM_ERR_SHAPE);
    EXPECT(reorder(2, 4, 2, P<int32_t>(0x201c)), NHM_ERR_UNSUPPORTED);
    EXPECT(reorder(2, 4, 2, P<int32_t>(0x3000), 0), NHM_ERR_SHAPE);
    pools[63].conv = nullptr;
    EXPECT(reorder(2, 4, 64, P<int32_t>(0x3000)), NHM_ERR_NULL);

    // plan
    EXPECT(nhm_batch_plan(nullptr, nullptr, nullptr, 4, 10, P<int32_t>(0x1000), P<int32_t>(0x2000), nullptr, nullptr, nullptr,
                          nullptr), NHM_ERR_NULL);
    EXPECT(nhm_batch_plan(P<int32_t>(0x1000), nullptr, nullptr, INT_MAX, 10, P<int32_t>(0x2000), P<int32_t>(0x3000), nullptr,
                          nullptr, nullptr, nullptr), NHM_ERR_UNSUPPORTED);
    EXPECT(nhm_batch_plan(P<int32_t>(0x1000), nullptr, nullptr, 4, INT64_MIN, P<int32_t>(0x2000), P<int32_t>(0x3000), nullptr,
                          nullptr, nullptr, nullptr), NHM_ERR_SHAPE);
    if (failures) return 1;
    printf("serving validation ok\n");
    return 0;
}
