// Low-rank adapters of many requests beside a shared W8A8 projection:
//   out[i, j] = base[i, j] + scale[e] sum_r (sum_k x[i, k] A_e[r, k]) B_e[j, r],  e = row_adapter[i]
// Two kernels: the low-rank product t = scale x A_e^T, then the adapter's part added to the f32
// projection and the sum rounded once.
#include "nhm_device.h"
#include "nhm_internal.h"

namespace nhm {

// t[i, r]: one wave per (row, rank), lanes over k.
__global__ __launch_bounds__(256) void lora_down_kernel(const LoraArgs g) {
    const int lane = threadIdx.x & 63;
    const int64_t i = blockIdx.x;
    const int r = blockIdx.y * 4 + (threadIdx.x >> 6);
    if (r >= g.rank) return;
    const int e = g.row_adapter[i];
    float sum = 0.f;
    if (e >= 0 && e < g.n_adapters) {
        const uint16_t* ar = g.a + ((int64_t)e * g.rank + r) * g.k;
        for (int64_t k = lane; k < g.k; k += 64) {
            const float x = g.x_codes ? e4m3_value(g.x_codes[i * g.ld_x + k]) * *g.a_scale
                                      : bf16_to_f32(g.x[i * g.ld_x + k]);
            sum = fmaf(x, bf16_to_f32(ar[k]), sum);
        }
        sum = wave_sum(sum) * (g.scale ? g.scale[e] : 1.0f);
    }
    if (lane == 0) g.t[i * g.rank + r] = sum;
}

// out = round(base + t B_e^T): one thread per output.
__global__ __launch_bounds__(256) void lora_up_kernel(const LoraArgs g) {
    const int64_t i = blockIdx.y, j = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (j >= g.n) return;
    const int e = g.row_adapter[i];
    float v = g.base[i * g.n + j];
    if (e >= 0 && e < g.n_adapters) {
        const uint16_t* br = g.b + ((int64_t)e * g.n + j) * g.rank;
        float sum = 0.f;
        for (int r = 0; r < g.rank; ++r) sum = fmaf(g.t[i * g.rank + r], bf16_to_f32(br[r]), sum);
        v += sum;
    }
    if (g.out_f32) g.out_f32[i * g.ld_out + j] = v;
    else g.out[i * g.ld_out + j] = (uint16_t)f32_to_bf16(v);
}

nhm_status launch_lora_down(const LoraArgs& g, hipStream_t st) {
    lora_down_kernel<<<dim3((unsigned)g.m, (unsigned)((g.rank + 3) / 4)), dim3(256), 0, st>>>(g);
    count_launch(Kern::kLoraDown, g.m);
    return check_launch("lora down");
}

nhm_status launch_lora_up(const LoraArgs& g, hipStream_t st) {
    for (int64_t r0 = 0; r0 < g.m; r0 += 65535) {    // the grid's y extent
        LoraArgs p = g;
        p.m = g.m - r0 < 65535 ? g.m - r0 : 65535;
        p.row_adapter += r0;
        p.base += r0 * g.n;
        p.t += r0 * g.rank;
        if (p.out_f32) p.out_f32 += r0 * g.ld_out;
        else p.out += r0 * g.ld_out;
        lora_up_kernel<<<dim3((unsigned)((g.n + 255) / 256), (unsigned)p.m), dim3(256), 0, st>>>(p);
    }
    count_launch(Kern::kLoraUp, g.m);
    return check_launch("lora up");
}

}  // namespace nhm
