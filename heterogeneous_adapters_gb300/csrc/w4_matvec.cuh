// y = x W^T with 4-bit weights and group scales, up to 16 rows of x a launch.
//
// A group's part of an output is  scale sum_k (c - zero) x: the differences of codes and zero
// point are whole numbers, exact in bf16 (128 + c is the bf16 whose last mantissa bits are the
// code, and 128 + zero comes off exactly), so that products are exact whatever x holds, and
// the scale enters once per group in fp32.  A code costs 11 / 8 instructions on its way to the
// tensor core.  (128 + c itself would be 7 / 8, less (128 + zero) sum x: two large sums whose
// difference is wrong near the zero point and for an infinite x, and not faster: 13 rows of
// q, k, v 11.6 us, and 10.5 as it is.)  The weights are the long side: 16 rows of W are an
// MMA's rows and 8 rows of x its columns.  What bounds it is the stream of W (half a byte a
// weight), next the unpacking: one row of 4096 x 4096 takes 7.7 us (two of launch, three to the
// first data), of two 14336 x 4096 21.7 us, 41% of the copy rate, where the copies alone
// take 12.6.
//
// Work.  A block of work is 32 rows of W by 256 of K (4 KB of codes); blocks of all
// projections lie in a row, K fastest, and the CTAs take equal contiguous ranges, a CTA's
// warps every eighth block.  Codes and scales come through a ring of cp.async stages per
// warp that runs on across row tiles.  Sums of a row tile are joined over the warps in
// shared memory, and where a tile is shared between CTAs, over partial sums in the workspace
// by the CTA that arrives last, in the order of K.
#pragma once
#include <cuda_fp16.h>

#include "lora_w4.h"
#include "mma_legacy.cuh"
#include "step.cuh"

namespace lora {

constexpr int kW4Warps = 8;
constexpr int kW4Threads = kW4Warps * 32;
// Rows of x up to which this kernel serves: always up to 8, and up to 16 where an SM has fewer
// than kW4WideBlocks blocks of w4_wide.cuh to itself, whose fixed part then weighs more (13
// rows: 3 blocks an SM 9.8 us here and 10.2 there, 5 blocks 10.5 and 12.5, 12 blocks 19.1 and
// 17.1, 24 blocks 28.1 and 23.7).
constexpr int kW4NarrowRows = 16;
constexpr int kW4WideBlocks = 8;
constexpr int kW4Rows = 32;        // rows of W of a block
constexpr int kW4K = 256;          // K of a block (128 bytes of codes a row)
constexpr int kW4Stages = 2;
// Blocks that joining a tile from several CTAs costs: one row of 4096 x 4096 9.9 us shared out
// evenly (7 blocks a CTA), 7.8 by whole tiles (16).
constexpr int kW4JoinCost = 16;
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

// Block u of the launch, and steps of kW4Warps blocks from it.
struct W4At {
    int prob, row0, kb;
};

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

    // the block that is copied next
    W4At nx = {0, 0, 0};
    if (first + warp < end) {
        nx.prob = w4_prob_of(p, first + warp);
        const int b = first + warp - p.prob[nx.prob].first;
        nx.row0 = b / p.prob[nx.prob].kblocks * kW4Rows;
        nx.kb = b - nx.row0 / kW4Rows * p.prob[nx.prob].kblocks;
    }
    // copies of block u (at nx) into a stage, and nx eight blocks on
    auto put = [&](int u, uint32_t stage) {
        if (u < end) {
            const W4Prob& pr = p.prob[nx.prob];
            const uint32_t dst = ring + stage * kStage;
            const int half = pr.K / 2;                         // bytes of a row
            const int col = (lane & 7) * 16, at = nx.kb * 128 + col;
            const unsigned char* src = pr.codes + (int64_t)(nx.row0 + (lane >> 3)) * half + at;
            const int rows = at < half ? pr.N - nx.row0 - (lane >> 3) : 0;
            const uint32_t to = dst + (lane >> 3) * 128;
            // rows i * 4 + lane / 8: the swizzle of row r is r % 8, which alternates with i
            const uint32_t c0 = col ^ ((lane >> 3) << 4), c1 = col ^ ((lane >> 3) + 4) << 4;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                cp_async16(to + i * 512 + (i & 1 ? c1 : c0), rows > i * 4 ? src : pr.codes, rows > i * 4 ? 16 : 0);
                src += 4 * (int64_t)half;
            }
#pragma unroll
            for (int j0 = 0; j0 < kGroups * 8; j0 += 32) {     // per group 4 pieces of scales, 4 of zeros
                const int j = j0 + lane, gr = j >> 3, piece = j & 3;
                const int grp = nx.kb * kGroups + gr;
                if (kGroups * 8 >= 32 || j < kGroups * 8) {
                    const bool ok = grp * G < pr.K && nx.row0 + piece * 8 < pr.N;
                    if (!(j & 4))
                        cp_async16(dst + kW4Codes + gr * 64 + piece * 16,
                                   pr.scales + (ok ? ((int64_t)grp * pr.N + nx.row0 + piece * 8) * 2 : 0), ok ? 16 : 0);
                    else if (pr.zeros)
                        cp_async4(dst + kW4Codes + kGroups * 64 + gr * 16 + piece * 4,
                                  pr.zeros + (ok ? (int64_t)grp * (pr.N / 2) + nx.row0 / 2 + piece * 4 : 0), ok ? 4 : 0);
                }
            }
            nx.kb += kW4Warps;
            while (nx.kb >= p.prob[nx.prob].kblocks && u + kW4Warps < end) {
                nx.kb -= p.prob[nx.prob].kblocks;
                nx.row0 += kW4Rows;
                if (nx.row0 >= p.prob[nx.prob].N) {
                    nx.row0 = 0;
                    ++nx.prob;
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
            // this lane's x of a group: row 8 n + g, eight values of every 32
            uint4 xr[NT][G / 32];
            auto load_x = [&](int gr) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < G / 32; ++c) {
                        const int k = k0 + gr * G + c * 32 + t * 8;
                        xr[n][c] = n * 8 + g < p.T && k < pr.K ? ld16(pr.x + (n * 8 + g) * pr.ldx + k) : make_uint4(0, 0, 0, 0);
                    }
            };
            load_x(0);
            cp_async_wait<kW4Stages - 1>();
            __syncwarp();
            const uint32_t st = ring + (it % kW4Stages) * kStage;
#pragma unroll
            for (int gr = 0; gr < kGroups; ++gr) {
                // scales, and 128 + zero twice, of rows g, g + 8, g + 16, g + 24
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
                        minus[r] = 0x43004300u + (z >> (4 * g) & 15u) * 0x00010001u;
                    }
                }
                float s[2][NT][4];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n) s[m][n][0] = s[m][n][1] = s[m][n][2] = s[m][n][3] = 0.f;
#pragma unroll
                for (int c = gr * (G / 32); c < (gr + 1) * (G / 32); ++c) {
                    uint32_t xb[NT][4];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint4 x = xr[n][c - gr * (G / 32)];
                        xb[n][0] = __byte_perm(x.x, x.z, 0x5410);
                        xb[n][1] = __byte_perm(x.x, x.z, 0x7632);
                        xb[n][2] = __byte_perm(x.y, x.w, 0x5410);
                        xb[n][3] = __byte_perm(x.y, x.w, 0x7632);
                    }
                    uint32_t w[4];
                    ldmatrix4(w, st + lane * 128 + ((c ^ (lane & 7)) << 4));
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const uint32_t w0 = w[2 * m], w1 = w[2 * m + 1], z0 = minus[2 * m], z1 = minus[2 * m + 1];
                        const uint32_t a0[4] = {code_pair<0>(w0, z0), code_pair<0>(w1, z1), code_pair<1>(w0, z0), code_pair<1>(w1, z1)};
                        const uint32_t a1[4] = {code_pair<2>(w0, z0), code_pair<2>(w1, z1), code_pair<3>(w0, z0), code_pair<3>(w1, z1)};
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma16816(s[m][n], a0, xb[n][0], xb[n][1]);
                            mma16816(s[m][n], a1, xb[n][2], xb[n][3]);
                        }
                    }
                }
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int r = 2 * m + (j >> 1);
                            acc[m][n][j] = fmaf(sc[r], s[m][n][j], acc[m][n][j]);
                        }
                if (gr + 1 < kGroups) load_x(gr + 1);
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
