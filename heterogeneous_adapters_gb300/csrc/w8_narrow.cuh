// y = x W^T of 8-bit integers with a scale per row of x and per row of W, for few rows of x.
//
// sm_103a has no integer tensor core to speak of (mma.sync on s8 runs at a quarter of the rate
// of f16, 252 against 1,023 multiplications a clock and SM), so the integers go to the f16
// pipe, where they are exact: 1024 + 128 + c is the f16 with c + 128 in its last bits, and
// 1152 comes off exactly.  Products of two codes have 15 bits; 1,024 of them sum exactly in
// fp32 (2^24), after which the sums go on as integers: y is rounded from the exact sum.
#pragma once
#include "lora_w8.h"
#include "mma_legacy.cuh"
#include "step.cuh"

namespace lora {

constexpr int kW8Warps = 8;
constexpr int kW8Threads = kW8Warps * 32;
constexpr int kW8Rows = 16;        // rows of W of a tile
constexpr int kW8Chunk = 64;       // K of a warp's step: 16 bytes a lane and row

struct W8Prob {
    const unsigned char* x;
    const float* x_scales;
    __nv_bfloat16* y;
    const unsigned char* w;
    const float* w_scales;
    int64_t ldx, ldy;
    int32_t N, K;
    int32_t first;                 // tiles before the projection
};

// MAX: the most projections of a launch (a launch's parameters take the host time by their size).
template <int MAX>
struct W8Params {
    W8Prob prob[MAX];
    int32_t nprob;
    int32_t T;
    int32_t total;                 // tiles
};

// Four codes as two f16 pairs, in order.
__device__ __forceinline__ void codes8_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u;                        // c + 128
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(__byte_perm(u, 0x64646464u, 0x4140)), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(__byte_perm(u, 0x64646464u, 0x4342)), "r"(0x64806480u));
}

// By the column tiles: steps of a group, whose loads are on their way while the group before is
// multiplied, and CTAs that an SM should hold (8 rows of two 14336 x 4096: groups of two and three
// CTAs 23 us, four and two 27; 13 rows of q, k, v: one and four 9.2, two and two 9.8, four and one 10.9).
__host__ __device__ constexpr int w8_group(int nt) { return nt == 1 ? 2 : 1; }
__host__ __device__ constexpr int w8_ctas(int nt) { return nt == 1 ? 3 : nt == 2 ? 4 : 2; }

// Lane (g, t) = (lane / 4, lane % 4) takes the 16 bytes from k = 16 t of its row's 64: word j of
// them are the two pairs that an MMA of 16 of K wants of the lane, for W and for x alike, so
// that the order of K within the 64 is the same for both.
template <int NT, int MAX>
__global__ void __launch_bounds__(kW8Threads, w8_ctas(NT)) w8_narrow_kernel(const __grid_constant__ W8Params<MAX> p) {
    constexpr int G = w8_group(NT), kStride = kW8Warps * kW8Chunk;
    __shared__ int32_t red[kW8Warps][8 * NT][kW8Rows];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    int i = 0;
    while (i + 1 < p.nprob && (int)blockIdx.x >= p.prob[i + 1].first) ++i;
    const W8Prob& pr = p.prob[i];
    const int row0 = ((int)blockIdx.x - pr.first) * kW8Rows, K = pr.K, t0 = blockIdx.y * 8 * NT;
    const bool in1 = row0 + 8 + g < pr.N;                      // N is a multiple of 8
    const unsigned char* w0 = pr.w + (int64_t)(row0 + g) * K;
    const unsigned char* w1 = w0 + (in1 ? 8 * (int64_t)K : 0);
    const unsigned char* xr[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) xr[n] = pr.x + min(t0 + n * 8 + g, p.T - 1) * pr.ldx;   // rows past the last: the last again
    int32_t sum[NT][4];
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sum[n][j] = 0;
            acc[n][j] = 0.f;
        }
    auto flush = [&]() {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sum[n][j] += (int32_t)acc[n][j];
                acc[n][j] = 0.f;
            }
    };
    struct Group {
        uint4 a[G][2], b[G][NT];
    };
    // a group's words; what lies past K is zeros in W
    auto load = [&](Group& q, int k0) {
#pragma unroll
        for (int s = 0; s < G; ++s) {
            const int k = k0 + s * kStride;
            const bool in = k < K;
            q.a[s][0] = in ? ld_stream16(w0 + k) : make_uint4(0, 0, 0, 0);
            q.a[s][1] = in ? ld_stream16(w1 + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int n = 0; n < NT; ++n) q.b[s][n] = ld16(xr[n] + (in ? k : 0));
        }
    };
    auto multiply = [&](const Group& q) {
#pragma unroll
        for (int s = 0; s < G; ++s) {
            const uint32_t aw0[4] = {q.a[s][0].x, q.a[s][0].y, q.a[s][0].z, q.a[s][0].w};
            const uint32_t aw1[4] = {q.a[s][1].x, q.a[s][1].y, q.a[s][1].z, q.a[s][1].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t a[4];
                codes8_f16(aw0[j], a[0], a[2]);
                codes8_f16(aw1[j], a[1], a[3]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint32_t bw[4] = {q.b[s][n].x, q.b[s][n].y, q.b[s][n].z, q.b[s][n].w};
                    uint32_t b0, b1;
                    codes8_f16(bw[j], b0, b1);
                    mma16816_f16(acc[n], a[0], a[1], a[2], a[3], b0, b1);
                }
            }
        }
    };
    Group q[2];
    const int k0 = warp * kW8Chunk + 16 * t, end = K + 16 * t;  // a warp's lanes end together
    load(q[0], k0);
    int steps = 0;
    for (int k = k0; k < end;) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h == 1 && k >= end) break;
            if (k + G * kStride < end) load(q[1 - h], k + G * kStride);
            multiply(q[h]);
            k += G * kStride;
            if ((steps += G) == 1024 / kW8Chunk) {
                flush();
                steps = 0;
            }
        }
    }
    flush();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) red[warp][n * 8 + 2 * t + (j & 1)][(j >> 1) * 8 + g] = sum[n][j];
    __syncthreads();
    for (int e = tid; e < 8 * NT * kW8Rows; e += kW8Threads) {
        const int col = e / kW8Rows, r = e % kW8Rows;
        int32_t s = 0;
#pragma unroll
        for (int w = 0; w < kW8Warps; ++w) s += red[w][col][r];
        if (t0 + col < p.T && row0 + r < pr.N)
            pr.y[(t0 + col) * pr.ldy + row0 + r] = __float2bfloat16_rn((float)s * pr.x_scales[t0 + col] * pr.w_scales[row0 + r]);
    }
}

}  // namespace lora
