// Causal attention of a batch's rows over the 4-bit cache.
#pragma once
#include "kv_layout.cuh"

namespace lora {

struct AttendParams {
    KvView v;
    const __nv_bfloat16* q;
    __nv_bfloat16* out;
    float* lse;
    int64_t ldq, ldo;
    int32_t q_heads;
    float scale;
};

constexpr int kAttendThreads = 128;

// One CTA per (row, query head): 128 tokens at a time, a thread a token for the scores and
// a thread a dimension for the output; running maximum and sum in fp32.
template <int D, int G>
__global__ void __launch_bounds__(kAttendThreads) kv_attend_kernel(const __grid_constant__ AttendParams p) {
    constexpr int kTileBytes = kv_tile_bytes(D, G);
    __shared__ float qs[D];
    __shared__ float ps[kAttendThreads];
    __shared__ const unsigned char* tiles[kAttendThreads];
    __shared__ float red[4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x, head = blockIdx.y, kvh = head / (p.q_heads / p.v.heads);
    if (warp == 0 && head == 0) kv_check_starts(p.v, row, gridDim.x);
    const KvRow r = kv_find_row(p.v, row);
    if (r.seq < 0) return;
    if (tid < D) qs[tid] = __bfloat162float(p.q[row * p.ldq + (int64_t)head * D + tid]);
    float m = -INFINITY, l = 0.f, acc = 0.f;
    for (int t0 = 0; t0 <= r.token; t0 += kAttendThreads) {
        __syncthreads();
        const int t = t0 + tid;
        const unsigned char* tile = t <= r.token ? kv_tile_of(p.v, r.seq, t, kvh, kTileBytes) : nullptr;
        float a = -INFINITY;
        if (tile != nullptr) {
            float sum = 0.f;
            for (int d = 0; d < D; d += 2) {
                const int b = tile[kv_codes_at(D, 0) + (d / 32 * kKvTile + t % kKvTile) * 16 + d % 32 / 2];
                const float2 so = __half22float2(*reinterpret_cast<const __half2*>(
                    tile + kv_params_at(D, G, 0) + (d / G * kKvTile + t % kKvTile) * 4));
                sum += qs[d] * (so.x * ((b & 15) - 8) + so.y) + qs[d + 1] * (so.x * ((b >> 4) - 8) + so.y);
            }
            a = sum * p.scale;
        }
        float top = a;
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0) red[warp] = top;
        __syncthreads();
        const float mn = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
        const float f = mn > -INFINITY ? expf(m - mn) : 1.f;
        ps[tid] = a > -INFINITY ? expf(a - mn) : 0.f;
        tiles[tid] = tile;
        __syncthreads();
        acc *= f;
        l *= f;
        m = mn;
        for (int j = 0; j < kAttendThreads; ++j) {
            l += ps[j];
            if (tid < D && tiles[j] != nullptr) {
                const int b = tiles[j][kv_codes_at(D, 1) + (tid / 32 * kKvTile + j % kKvTile) * 16 + tid % 32 / 2];
                const float2 so = __half22float2(*reinterpret_cast<const __half2*>(
                    tiles[j] + kv_params_at(D, G, 1) + (tid / G * kKvTile + j % kKvTile) * 4));
                acc += ps[j] * (so.x * ((tid & 1 ? b >> 4 : b & 15) - 8) + so.y);
            }
        }
    }
    if (tid < D) p.out[row * p.ldo + (int64_t)head * D + tid] = __float2bfloat16_rn(l > 0.f ? acc / l : 0.f);
    if (tid == 0 && p.lse != nullptr) p.lse[(int64_t)row * p.q_heads + head] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace lora
