// y = x W^T of 8-bit integers with a scale per row of x and per row of W, for few rows of x.
//
// sm_103a has no integer tensor core to speak of (mma.sync on s8 runs at a quarter of the rate
// of f16, 252 against 1,023 multiplications a clock and SM), so the integers go to the f16
// pipe, where they are exact: 1024 + 128 + c is the f16 with c + 128 in its last bits, and
// 1152 comes off exactly.  Products of two codes have 15 bits; 1,024 of them sum exactly in
// fp32 (2^24), after which the sums go on as integers: y is rounded from the exact sum.
//
// A CTA takes 16 rows of W over all of K, its eight warps 128 of K each in turn; their sums meet in
// shared memory, and nothing waits for another CTA.  W and x come in pieces of 32 bytes a lane, a
// request a sector (W in L2: by 16 bytes 1 row of 4096 x 4096 takes 4.0 us and 13 rows of q, k, v 8.0, by 32
// bytes 3.9 and 7.1 to 7.5).  W from memory, as a layer finds it: 1 row of 4096 x 4096 6.1 to 6.3 us (2.7 TB/s), of
// q, k, v (25 MB) 7.5 (3.3), of 117 MB 23.5 (5.0); the launch and the first data bound the small ones, memory
// the large.  Up to 8 rows take as long as 1; beyond, the widening of x for each 16 rows of W counts (13 rows of
// q, k, v 10.5, 16 rows of 117 MB 31).
//
// The one-row kernel with loads of 32 bytes spills one register (4 bytes); none of the others does.
#pragma once
#include "lora_w8.h"
#include "mma_legacy.cuh"
#include "step.cuh"

namespace lora {

constexpr int kW8Warps = 8;
constexpr int kW8Threads = kW8Warps * 32;
constexpr int kW8Rows = 16;        // rows of W of a tile
constexpr int kW8Chunk = 128;      // K of a warp's step: 32 bytes a lane and row

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

// CTAs that an SM should hold, by the column tiles.
__host__ __device__ constexpr int w8_ctas(int nt) { return nt == 1 ? 3 : nt == 2 ? 2 : 1; }

// 32 bytes of a lane's row from k on, zeros past K (a multiple of 16); STREAM: 32 at a time past the first-level cache.
template <bool BY32, bool STREAM>
__device__ __forceinline__ void w8_load(uint32_t (&v)[8], const unsigned char* row, int k, int K) {
    if constexpr (BY32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0;
        if (k >= K) return;
        if constexpr (STREAM)
            asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                : "l"(row + k));
        else
            asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                         : "l"(row + k));
    } else {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const unsigned char* p = row + k + 4 * i;
            const uint4 x = k + 4 * i >= K ? make_uint4(0, 0, 0, 0) : ld16(p);
            v[i] = x.x;
            v[i + 1] = x.y;
            v[i + 2] = x.z;
            v[i + 3] = x.w;
        }
    }
}

// Lane (g, t) = (lane / 4, lane % 4) takes the 32 bytes from k = 32 t of its row's 128: word j of
// them are the two pairs that an MMA of 16 of K wants of the lane, for W and for x alike, so
// that the order of K within the 128 is the same for both.  The next step's loads are on their
// way while one is multiplied.  BY32: every row of x and W begins at a multiple of 32 bytes and is
// loaded by 32 at a time; else by 16.
template <int NT, int MAX, bool BY32>
__global__ void __launch_bounds__(kW8Threads, w8_ctas(NT)) w8_narrow_kernel(const __grid_constant__ W8Params<MAX> p) {
    constexpr int kStride = kW8Warps * kW8Chunk;
    __shared__ int32_t red[kW8Warps][8 * NT][kW8Rows];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    grid_wait();
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
    struct Step {
        uint32_t a[2][8], b[NT][8];
    };
    // a step's words; what lies past K is zeros
    auto load = [&](Step& q, int k) {
        w8_load<BY32, true>(q.a[0], w0, k, K);
        w8_load<BY32, true>(q.a[1], w1, k, K);
#pragma unroll
        for (int n = 0; n < NT; ++n) w8_load<BY32, false>(q.b[n], xr[n], k, K);
    };
    auto multiply = [&](const Step& q) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t a[4];
            codes8_f16(q.a[0][j], a[0], a[2]);
            codes8_f16(q.a[1][j], a[1], a[3]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                uint32_t b0, b1;
                codes8_f16(q.b[n][j], b0, b1);
                mma16816_f16(acc[n], a[0], a[1], a[2], a[3], b0, b1);
            }
        }
    };
    Step q[2];
    const int k0 = warp * kW8Chunk + 32 * t, end = K + 32 * t;      // a warp's lanes end together
    load(q[0], k0);
    int steps = 0;
    for (int k = k0; k < end;) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h == 1 && k >= end) break;
            if (k + kStride < end) load(q[1 - h], k + kStride);
            multiply(q[h]);
            k += kStride;
            if (++steps == 1024 / kW8Chunk) {
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
