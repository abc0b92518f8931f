// y = x W^T with 4-bit weights and group scales, up to 16 rows of x a launch.
//
// A group's part of an output is  scale * sum_k (c - zero) x: the differences of codes and
// zero point are whole numbers, exact in bf16, so the tensor core sums exact products and the
// scale enters once per group in fp32.  The weights are the long side: 16 rows of W are an
// MMA's rows and 8 rows of x its columns.  What bounds it is the stream of W (half a byte a
// weight), next the unpacking (11 / 8 instructions a weight and lane).
//
// Work.  A block of work is 32 rows of W by 256 of K (4 KB of codes); blocks of all
// projections lie in a row, K fastest, and the CTAs take equal contiguous ranges, a CTA's
// warps every eighth block.  Codes and scales come through a ring of cp.async stages per
// warp that runs on across row tiles.  Sums of a row tile are joined over the warps in
// shared memory, and where a tile is shared between CTAs, over partial sums in the workspace
// by the CTA that arrives last, in the order of K.
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"
#include "lora_w4.h"
#include "mma_legacy.cuh"
#include "ptx.cuh"

namespace lora {

constexpr int kW4Warps = 8;
constexpr int kW4Threads = kW4Warps * 32;
constexpr int kW4NarrowRows = 16;  // rows of x up to which this kernel serves
constexpr int kW4Rows = 32;        // rows of W of a block
constexpr int kW4K = 256;          // K of a block (128 bytes of codes a row)
constexpr int kW4Stages = 3;
constexpr int kW4MaxCtas = 512;
static_assert(kW4MaxCtas <= kStepTickets, "a counter per CTA");

struct W4Prob {
    const __nv_bfloat16* x;
    __nv_bfloat16* y;
    const unsigned char* codes;
    const unsigned char* scales;
    const unsigned char* zeros;
    int64_t ldx, ldy;
    int32_t N, K, group;
    int32_t kblocks;               // blocks of a row tile
    int32_t first;                 // blocks before the projection
};

struct W4Params {
    W4Prob prob[LORA_W4_MAX_PROBLEMS];
    int32_t nprob;
    int32_t T;
    int32_t total;                 // blocks
    int32_t per;                   // blocks of a CTA
    uint32_t* tickets;             // [kStepTickets], zero between calls
    float* part;                   // [kW4MaxCtas][2][32][8 NT]
};

// A stage: codes [32 rows][128 bytes] with the 16-byte columns of row r swapped by r % 8,
// then scales [256 / G][32] f16 and zeros [256 / G][16 bytes].
constexpr int kW4Codes = kW4Rows * 128;
__host__ __device__ constexpr int w4_stage_bytes(int group) { return kW4Codes + (kW4K / group) * (kW4Rows * 2 + 16); }
__host__ __device__ constexpr size_t w4_smem(int group, int nt) {
    return (size_t)kW4Warps * (kW4Stages * w4_stage_bytes(group) + kW4Rows * 8 * nt * 4);
}
__host__ __device__ constexpr size_t w4_workspace(int nt) {
    return kStepPartAt + (size_t)kW4MaxCtas * 2 * kW4Rows * 8 * nt * 4;
}

// Asynchronous copies global -> shared of which the first `n` bytes are read, the rest zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t n) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The projection that holds block u.
__device__ __forceinline__ int w4_prob_of(const W4Params& p, int u) {
    int i = 0;
    while (i + 1 < p.nprob && u >= p.prob[i + 1].first) ++i;
    return i;
}

template <int G, int NT>
__global__ void __launch_bounds__(kW4Threads, 2) w4_matvec_kernel(const __grid_constant__ W4Params p) {
    constexpr int kGroups = kW4K / G, kStage = w4_stage_bytes(G), kCols = 8 * NT;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint32_t last_in;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_addr(smem) + warp * kW4Stages * kStage;
    float* red = reinterpret_cast<float*>(smem + kW4Warps * kW4Stages * kStage);
    const int first = blockIdx.x * p.per, end = min(first + p.per, p.total);
    if (first >= end) return;

    // copies of block u into a stage
    auto put = [&](int u, uint32_t stage) {
        if (u < end) {
            const W4Prob& pr = p.prob[w4_prob_of(p, u)];
            const int b = u - pr.first, row0 = b / pr.kblocks * kW4Rows, kb = b % pr.kblocks;
            const uint32_t dst = ring + stage * kStage;
            const int half = pr.K / 2;                         // bytes of a row
            const int col = (lane & 7) * 16, at = kb * 128 + col;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = i * 4 + (lane >> 3), row = row0 + r;
                const bool in = row < pr.N && at < half;
                cp_async16(dst + r * 128 + (col ^ ((r & 7) << 4)), pr.codes + (in ? (int64_t)row * half + at : 0), in ? 16 : 0);
            }
#pragma unroll
            for (int j0 = 0; j0 < kGroups * 8; j0 += 32) {     // per group 4 pieces of scales, 4 of zeros
                const int j = j0 + lane, gr = j >> 3, piece = j & 3;
                const int grp = kb * kGroups + gr;
                if (kGroups * 8 >= 32 || j < kGroups * 8) {
                    const bool in = grp * G < pr.K;
                    if (!(j & 4)) {
                        const bool ok = in && row0 + piece * 8 < pr.N;
                        cp_async16(dst + kW4Codes + gr * 64 + piece * 16,
                                   pr.scales + (ok ? ((int64_t)grp * pr.N + row0 + piece * 8) * 2 : 0), ok ? 16 : 0);
                    } else if (pr.zeros) {
                        const bool ok = in && row0 + piece * 8 < pr.N;
                        cp_async4(dst + kW4Codes + kGroups * 64 + gr * 16 + piece * 4,
                                  pr.zeros + (ok ? (int64_t)grp * (pr.N / 2) + row0 / 2 + piece * 4 : 0), ok ? 4 : 0);
                    }
                }
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kW4Stages - 1; ++i) put(first + warp + i * kW4Warps, i);

    int u = first + warp;
    uint32_t it = 0;
    for (int at = first; at < end;) {
        const W4Prob& pr = p.prob[w4_prob_of(p, at)];
        const int tile = (at - pr.first) / pr.kblocks;
        const int tile_first = pr.first + tile * pr.kblocks, tile_end = tile_first + pr.kblocks;
        const int stop = min(tile_end, end);
        const int row0 = tile * kW4Rows;
        float acc[2][NT][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.f;
        for (; u < stop; u += kW4Warps, ++it) {
            const int k0 = (u - tile_first) * kW4K;
            put(u + (kW4Stages - 1) * kW4Warps, (it + kW4Stages - 1) % kW4Stages);
            // this lane's x: row 8 n + g, eight values of every 32
            uint4 xr[NT][8];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const int k = k0 + c * 32 + t * 8;
                    xr[n][c] = n * 8 + g < p.T && k < pr.K ? ld16(pr.x + (n * 8 + g) * pr.ldx + k) : make_uint4(0, 0, 0, 0);
                }
            cp_async_wait<kW4Stages - 1>();
            __syncwarp();
            const uint32_t st = ring + (it % kW4Stages) * kStage;
#pragma unroll
            for (int gr = 0; gr < kGroups; ++gr) {
                // scales and zero points of rows g, g + 8, g + 16, g + 24
                float sc[4];
                uint32_t minus[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    unsigned short h;
                    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(st + kW4Codes + gr * 64 + (r * 8 + g) * 2));
                    sc[r] = __half2float(__ushort_as_half(h));
                    minus[r] = kMinus8;
                    if (pr.zeros) {
                        uint32_t z;
                        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(z) : "r"(st + kW4Codes + kGroups * 64 + gr * 16 + r * 4));
                        minus[r] = 0x43004300u + ((z >> (4 * g)) & 15u) * 0x00010001u;
                    }
                }
                float s[2][NT][4];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n) s[m][n][0] = s[m][n][1] = s[m][n][2] = s[m][n][3] = 0.f;
#pragma unroll
                for (int c = gr * (G / 32); c < (gr + 1) * (G / 32); ++c) {
                    uint32_t w[4];
                    ldmatrix4(w, st + lane * 128 + ((c ^ (lane & 7)) << 4));
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const uint32_t w0 = w[2 * m], w1 = w[2 * m + 1], z0 = minus[2 * m], z1 = minus[2 * m + 1];
                        const uint32_t a0[4] = {code_pair<0>(w0, z0), code_pair<0>(w1, z1), code_pair<1>(w0, z0), code_pair<1>(w1, z1)};
                        const uint32_t a1[4] = {code_pair<2>(w0, z0), code_pair<2>(w1, z1), code_pair<3>(w0, z0), code_pair<3>(w1, z1)};
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint4 x = xr[n][c];
                            mma16816(s[m][n], a0, __byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632));
                            mma16816(s[m][n], a1, __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
                        }
                    }
                }
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[m][n][j] = fmaf(sc[2 * m + (j >> 1)], s[m][n][j], acc[m][n][j]);
            }
            __syncwarp();                                      // the stage may be filled again
        }
        // ---- the warps' sums: red[warp][x row][row of W]
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    red[(warp * kCols + n * 8 + 2 * t + (j & 1)) * kW4Rows + m * 16 + (j >> 1) * 8 + g] = acc[m][n][j];
        __syncthreads();
        const bool whole = at == tile_first && stop == tile_end;
        float* part = p.part + ((int64_t)blockIdx.x * 2 + (tile_first < first ? 0 : 1)) * kW4Rows * kCols;
        for (int e = tid; e < kCols * kW4Rows; e += kW4Threads) {
            const int col = e / kW4Rows, r = e % kW4Rows;
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kW4Warps; ++w) sum += red[w * kCols * kW4Rows + e];
            if (!whole) part[e] = sum;
            else if (col < p.T && row0 + r < pr.N) pr.y[col * pr.ldy + row0 + r] = __float2bfloat16_rn(sum);
        }
        if (!whole) {
            const int c0 = tile_first / p.per, c1 = (tile_end - 1) / p.per;
            __threadfence();
            __syncthreads();
            if (tid == 0) last_in = atomicAdd(&p.tickets[c0], 1u) == (uint32_t)(c1 - c0);
            __syncthreads();
            if (last_in) {
                __threadfence();
                if (tid == 0) p.tickets[c0] = 0;
                for (int e = tid; e < kCols * kW4Rows; e += kW4Threads) {
                    const int col = e / kW4Rows, r = e % kW4Rows;
                    float sum = 0.f;
#pragma unroll 4
                    for (int c = c0; c <= c1; ++c)
                        sum += __ldcg(p.part + ((int64_t)c * 2 + (tile_first < c * p.per ? 0 : 1)) * kW4Rows * kCols + e);
                    if (col < p.T && row0 + r < pr.N) pr.y[col * pr.ldy + row0 + r] = __float2bfloat16_rn(sum);
                }
            }
        }
        __syncthreads();
        at = stop;
    }
    cp_async_wait<0>();
}

}  // namespace lora
