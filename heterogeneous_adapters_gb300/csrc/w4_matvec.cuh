// y = x W^T with 4-bit weights and group scales, for up to 256 rows of x.
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"
#include "lora_w4.h"

namespace lora {

constexpr int kW4Warps = 8;
constexpr int kW4Rows = 8;     // rows of x a warp holds sums of at a time

struct W4Params {
    lora_w4_problem prob[LORA_W4_MAX_PROBLEMS];
    int32_t first[LORA_W4_MAX_PROBLEMS + 1];   // first block of each problem
    int32_t nprob;
    int32_t T;
    uint32_t* err;
};

// One warp per output column and eight rows: the lanes split K in words of eight codes.
__global__ void __launch_bounds__(kW4Warps * 32) w4_matvec_kernel(const __grid_constant__ W4Params p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int i = 0;
    while (i + 1 < p.nprob && (int)blockIdx.x >= p.first[i + 1]) ++i;
    const lora_w4_problem& pr = p.prob[i];
    const int n = ((int)blockIdx.x - p.first[i]) * kW4Warps + warp;
    if (n >= pr.N) return;
    const uint32_t* codes = reinterpret_cast<const uint32_t*>(pr.codes) + (int64_t)n * (pr.K / 8);
    const __nv_bfloat16* x = reinterpret_cast<const __nv_bfloat16*>(pr.x);
    for (int t0 = blockIdx.y * kW4Rows; t0 < min(p.T, (int)(blockIdx.y + 1) * kW4Rows); t0 += kW4Rows) {
        float acc[kW4Rows] = {};
        for (int k8 = lane; k8 < pr.K / 8; k8 += 32) {
            const uint32_t w = codes[k8];
            const int g = k8 * 8 / pr.group;
            const float s = __half2float(reinterpret_cast<const __half*>(pr.scales)[(int64_t)g * pr.N + n]);
            int z = 8;
            if (pr.zeros) z = reinterpret_cast<const uint8_t*>(pr.zeros)[(int64_t)g * (pr.N / 2) + n / 2] >> (n & 1) * 4 & 15;
#pragma unroll
            for (int r = 0; r < kW4Rows; ++r) {
                if (t0 + r >= p.T) continue;
                float xv[8], sum = 0.f;
                unpack8(ld16(x + (t0 + r) * pr.ldx + k8 * 8), xv);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum += xv[j] * (float)((int)(w >> 4 * j & 15) - z);
                acc[r] += s * sum;
            }
        }
#pragma unroll
        for (int r = 0; r < kW4Rows; ++r) {
            for (int o = 16; o; o >>= 1) acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], o);
            if (lane == 0 && t0 + r < p.T)
                reinterpret_cast<__nv_bfloat16*>(pr.y)[(t0 + r) * pr.ldy + n] = __float2bfloat16_rn(acc[r]);
        }
    }
}

}  // namespace lora
