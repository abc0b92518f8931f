// y = x W^T with 4-bit weights for 17 rows of x and more (up to 128 a launch).
//
// The same sums as w4_matvec.cuh (exact differences of codes and zero points, one scale per
// group in fp32), with the fifth-generation tensor cores: 128 rows of W are the M of a
// tcgen05.mma whose A operand lies in tensor memory, where the unpacking warps write it, and
// the rows of x are its N, in shared memory as TMA lays them (128-byte swizzle).  A group's
// product is complete in D before its scale is known to apply, so D is drained once per
// group: a thread per row of W reads its columns and adds scale * D to sums in registers.
// Half a byte a weight from memory is the floor; unpacking (13 / 8 instructions a weight, in
// the order of K) and draining (one FMA per group, row and column) fill most of the issue
// slots of that time at 64 rows.
//
// One CTA per SM: warp 0 streams codes (blocks of 128 rows x 256 of K) and x by TMA, warp 1
// issues the MMAs, warps 2-9 unpack, warps 10-17 drain.  CTAs take equal contiguous ranges of
// the blocks of all projections; a row tile shared by several CTAs is joined over partial
// sums in the workspace by the CTA that arrives last, in the order of K.
#pragma once
#include <cuda.h>

#include "w4_matvec.cuh"

namespace lora {

constexpr int kWideThreads = 18 * 32;
constexpr int kWideRows = 128;                 // rows of W of a block
constexpr int kWideK = 256;                    // K of a block
constexpr int kWideChunk = 128;                // K of an A buffer and of an x stage
constexpr int kWideCodeStages = 4;
constexpr int kWideA = 4;                      // A buffers in tensor memory
constexpr int kWideMaxCtas = 192;
constexpr int kWideCodeBytes = kWideRows * kWideK / 2;

__host__ __device__ constexpr int wide_x_stages(int n) { return n >= 128 ? 4 : 6; }
__host__ __device__ constexpr size_t wide_smem(int n) {
    return 1024 + (size_t)kWideCodeStages * kWideCodeBytes + (size_t)wide_x_stages(n) * n * kWideChunk * 2;
}
__host__ __device__ constexpr size_t wide_workspace(int n) {
    return kStepPartAt + (size_t)kWideMaxCtas * 2 * kWideRows * n * 4;
}

struct WideParams {
    CUtensorMap codes[LORA_W4_MAX_PROBLEMS];   // bytes {K / 2, N}, box {128, 128}, 128-byte swizzle
    CUtensorMap x[LORA_W4_MAX_PROBLEMS];       // bf16 {K, T}, box {64, N columns}, 128-byte swizzle
    W4Params p;                                // blocks of 128 x 256
    uint32_t* err;
};

// A block: projection, row tile and block of K.
struct WideAt {
    int prob, tile, kb;
};
__device__ __forceinline__ WideAt wide_at(const W4Params& p, int u) {
    WideAt a;
    a.prob = w4_prob_of(p, u);
    const int b = u - p.prob[a.prob].first;
    a.tile = b / p.prob[a.prob].kblocks;
    a.kb = b - a.tile * p.prob[a.prob].kblocks;
    return a;
}
__device__ __forceinline__ void wide_next(const W4Params& p, WideAt& a) {
    if (++a.kb < p.prob[a.prob].kblocks) return;
    a.kb = 0;
    if (++a.tile * kWideRows < p.prob[a.prob].N) return;
    a.tile = 0;
    ++a.prob;
}
// 128-wide pieces of K in a block.
__device__ __forceinline__ int wide_chunks(const W4Prob& pr, int kb) { return pr.K - kb * kWideK > kWideChunk ? 2 : 1; }

// The eight codes of a word minus the zero point, in order, as four bf16 pairs.
__device__ __forceinline__ void codes_in_order(uint32_t w, uint32_t minus, uint32_t* out) {
    const uint32_t h = w >> 4;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const uint32_t v = __byte_perm(w, h, b | (4 + b) << 8);   // bytes b of w and h, in the halves' low bytes
        uint32_t t;
        asm("lop3.b32 %0, %1, 0x000F000F, 0x43004300, 0xEA;" : "=r"(t) : "r"(v));
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(out[b]) : "r"(t), "r"(minus));
    }
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}

template <int G, int N>
__global__ void __launch_bounds__(kWideThreads, 1) w4_wide_kernel(const __grid_constant__ WideParams prm) {
    constexpr int kXStages = wide_x_stages(N), kXBytes = N * kWideChunk * 2, kGroups = kWideChunk / G;
    constexpr int kMine = N / 2;               // columns of a drain thread
    constexpr uint32_t kACol = 256;            // D buffers at columns 0 and N, A buffers from 256
    extern __shared__ unsigned char raw[];
    __shared__ __align__(8) uint64_t code_full[kWideCodeStages], code_empty[kWideCodeStages], x_full[kXStages], x_empty[kXStages],
        a_full[kWideA], a_empty[kWideA], d_full[2], d_empty[2], join, final_bar;
    __shared__ uint32_t tmem_slot, last_in;
    const W4Params& p = prm.p;
    unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const uint32_t codes0 = smem_addr(base), x0 = codes0 + kWideCodeStages * kWideCodeBytes;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int first = blockIdx.x * p.per, end = min(first + p.per, p.total);
    if (first >= end) return;
    auto bar = [](uint64_t& b) { return smem_addr(&b); };
    if (tid == 0) {
        for (int i = 0; i < kWideCodeStages; ++i) {
            mbar_init(bar(code_full[i]), 1);
            mbar_init(bar(code_empty[i]), 8);
        }
        for (int i = 0; i < kXStages; ++i) {
            mbar_init(bar(x_full[i]), 1);
            mbar_init(bar(x_empty[i]), 1);
        }
        for (int i = 0; i < kWideA; ++i) {
            mbar_init(bar(a_full[i]), 8);
            mbar_init(bar(a_empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(d_full[i]), 1);
            mbar_init(bar(d_empty[i]), 8);
        }
        mbar_init(bar(join), 8);
        mbar_init(bar(final_bar), 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(&tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&tmem_slot);
    bool ok = true;

    if (warp == 0) {
        // ------------------------------------------------------------------ codes and x
        if (lane == 0) {
            WideAt a = wide_at(p, first);
            uint32_t ic = 0, ix = 0;
            for (int u = first; u < end && ok; ++u, wide_next(p, a), ++ic) {
                const uint32_t s = ic % kWideCodeStages;
                if (!mbar_wait(bar(code_empty[s]), ((ic / kWideCodeStages) & 1) ^ 1, kWaitLimitNs)) { ok = false; break; }
                mbar_arrive_expect_tx(bar(code_full[s]), kWideCodeBytes);
                tma_load_2d(codes0 + s * kWideCodeBytes, &prm.codes[a.prob], a.kb * (kWideK / 2), a.tile * kWideRows, bar(code_full[s]));
                const int n = wide_chunks(p.prob[a.prob], a.kb);
                for (int c = 0; c < n; ++c, ++ix) {
                    const uint32_t t = ix % kXStages;
                    if (!mbar_wait(bar(x_empty[t]), ((ix / kXStages) & 1) ^ 1, kWaitLimitNs)) { ok = false; break; }
                    mbar_arrive_expect_tx(bar(x_full[t]), kXBytes);
                    for (int h = 0; h < 2; ++h)
                        tma_load_2d(x0 + t * kXBytes + h * (kXBytes / 2), &prm.x[a.prob], a.kb * kWideK + c * kWideChunk + h * 64, 0,
                                    bar(x_full[t]));
                }
            }
            if (!ok) set_error(prm.err, LORA_DERR_TIMEOUT);
            // every copy has landed before the CTA can end
            for (uint32_t k = ic > kWideCodeStages ? ic - kWideCodeStages : 0; k < ic; ++k)
                mbar_wait(bar(code_full[k % kWideCodeStages]), (k / kWideCodeStages) & 1, 100000000ull);
            for (uint32_t k = ix > kXStages ? ix - kXStages : 0; k < ix; ++k)
                mbar_wait(bar(x_full[k % kXStages]), (k / kXStages) & 1, 100000000ull);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------------ MMA issue
        constexpr uint32_t idesc = idesc_bf16(128, N, 0, 0);
        WideAt a = wide_at(p, first);
        uint32_t ix = 0, id = 0;               // chunks (A buffers, x stages) and groups (D buffers)
        for (int u = first; u < end && ok; ++u, wide_next(p, a)) {
            const int n = wide_chunks(p.prob[a.prob], a.kb);
            for (int c = 0; c < n && ok; ++c, ++ix) {
                const uint32_t t = ix % kXStages, b = ix % kWideA;
                if (!mbar_wait(bar(x_full[t]), (ix / kXStages) & 1, kWaitLimitNs) ||
                    !mbar_wait(bar(a_full[b]), (ix / kWideA) & 1, kWaitLimitNs)) { ok = false; break; }
                for (int g = 0; g < kGroups; ++g, ++id) {
                    if (!mbar_wait(bar(d_empty[id & 1]), ((id >> 1) & 1) ^ 1, kWaitLimitNs)) { ok = false; break; }
                    tc_fence_after();
                    if (lane == 0) {
#pragma unroll
                        for (int k = 0; k < G / 16; ++k) {
                            const int ks = g * (G / 16) + k;
                            const uint64_t db = smem_desc(x0 + t * kXBytes + (ks / 4) * (kXBytes / 2) + (ks % 4) * 32, 16, 1024, 2);
                            tc_mma_f16_ts(tmem + (id & 1) * N, tmem + kACol + b * 64 + ks * 8, db, idesc, k != 0);
                        }
                        tc_commit(bar(d_full[id & 1]));
                        if (g == kGroups - 1) {
                            tc_commit(bar(a_empty[b]));
                            tc_commit(bar(x_empty[t]));
                        }
                    }
                    __syncwarp();
                }
            }
        }
        if (!ok && lane == 0) set_error(prm.err, LORA_DERR_TIMEOUT);
        if (lane == 0) {                       // the MMAs are done before tensor memory is given back
            tc_commit(bar(final_bar));
            mbar_wait(bar(final_bar), 0, 100000000ull);
        }
        __syncwarp();
    } else if (warp < 10) {
        // ------------------------------------------------------------------ unpacking: a row, 64 of every 128 of K
        const int quad = warp & 3, half = (warp - 2) >> 2, r = quad * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        WideAt a = wide_at(p, first);
        uint32_t ic = 0, ia = 0;
        constexpr int kZ = G < 64 ? 2 : 1;     // zero points of 64 of K
        // the zero points of chunk c of block a, as 128 + zero twice
        auto zeros = [&](const WideAt& a, int c, uint32_t (&z)[kZ]) {
            const W4Prob& pr = p.prob[a.prob];
            const int row = a.tile * kWideRows + r;
#pragma unroll
            for (int i = 0; i < kZ; ++i) {
                const int g = (a.kb * kWideK + c * kWideChunk + half * 64 + i * 32) / G;
                uint32_t v = 8;
                if (pr.zeros && row < pr.N && g * G < pr.K)
                    v = __ldg(pr.zeros + (int64_t)g * (pr.N / 2) + row / 2) >> (row & 1) * 4 & 15;
                z[i] = 0x43004300u + v * 0x00010001u;
            }
        };
        uint32_t znext[kZ];
        zeros(a, 0, znext);
        for (int u = first; u < end && ok; ++u, ++ic) {
            const int n = wide_chunks(p.prob[a.prob], a.kb);
            WideAt an = a;
            wide_next(p, an);
            const uint32_t s = ic % kWideCodeStages;
            if (!mbar_wait(bar(code_full[s]), (ic / kWideCodeStages) & 1, kWaitLimitNs)) { ok = false; break; }
            for (int c = 0; c < n; ++c, ++ia) {
                uint32_t z[kZ];
#pragma unroll
                for (int i = 0; i < kZ; ++i) z[i] = znext[i];
                if (c + 1 < n) zeros(a, c + 1, znext);
                else if (u + 1 < end) zeros(an, 0, znext);
                uint32_t out[32];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int col = c * 4 + half * 2 + j;      // 16-byte column of the row
                    const uint4 w = lds128(codes0 + s * kWideCodeBytes + r * 128 + ((col ^ (r & 7)) << 4));
                    const uint32_t m = z[kZ > 1 ? j : 0];
                    codes_in_order(w.x, m, out + j * 16);
                    codes_in_order(w.y, m, out + j * 16 + 4);
                    codes_in_order(w.z, m, out + j * 16 + 8);
                    codes_in_order(w.w, m, out + j * 16 + 12);
                }
                const uint32_t b = ia % kWideA;
                if (!mbar_wait(bar(a_empty[b]), ((ia / kWideA) & 1) ^ 1, kWaitLimitNs)) { ok = false; break; }
                tc_fence_after();
                tmem_st32(tmem + lane_base + kACol + b * 64 + half * 32, out);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(a_full[b]));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(code_empty[s]));
            a = an;
        }
        if (!ok && lane == 0) set_error(prm.err, LORA_DERR_TIMEOUT);
    } else {
        // ------------------------------------------------------------------ draining: a row, half of the columns
        const int quad = warp & 3, half = (warp - 10) >> 2, r = quad * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        WideAt a = wide_at(p, first);
        uint32_t id = 0, ij = 0;
        // the eight draining warps meet (bounded, as every wait); false on a timeout
        auto meet = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(join));
            return mbar_wait(bar(join), ij++ & 1, kWaitLimitNs);
        };
        auto scales = [&](const WideAt& a, int c, float (&s)[kGroups]) {
            const W4Prob& pr = p.prob[a.prob];
            const int row = a.tile * kWideRows + r;
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                const int g = (a.kb * kWideK + c * kWideChunk) / G + i;
                s[i] = row < pr.N && g * G < pr.K
                           ? __half2float(__ldg(reinterpret_cast<const __half*>(pr.scales) + (int64_t)g * pr.N + row)) : 0.f;
            }
        };
        float snext[kGroups];
        scales(a, 0, snext);
        for (int at = first; at < end && ok;) {
            const W4Prob& pr = p.prob[a.prob];
            const int row0 = a.tile * kWideRows;
            const int tile_first = at - a.kb, tile_end = tile_first + pr.kblocks, stop = min(tile_end, end);
            float acc[kMine];
#pragma unroll
            for (int j = 0; j < kMine; ++j) acc[j] = 0.f;
            for (int u = at; u < stop && ok; ++u) {
                const int n = wide_chunks(pr, a.kb);
                WideAt an = a;
                wide_next(p, an);
                for (int c = 0; c < n && ok; ++c) {
                    float s[kGroups];
#pragma unroll
                    for (int i = 0; i < kGroups; ++i) s[i] = snext[i];
                    if (c + 1 < n) scales(a, c + 1, snext);
                    else if (u + 1 < end) scales(an, 0, snext);
#pragma unroll
                    for (int g = 0; g < kGroups; ++g, ++id) {
                        if (!mbar_wait(bar(d_full[id & 1]), (id >> 1) & 1, kWaitLimitNs)) { ok = false; break; }
                        tc_fence_after();
#pragma unroll
                        for (int j = 0; j < kMine; j += 16) {
                            float v[16];
                            tmem_ld16(tmem + lane_base + (id & 1) * N + half * kMine + j, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 16; ++i) acc[j + i] = fmaf(s[g], v[i], acc[j + i]);
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(d_empty[id & 1]));
                    }
                }
                a = an;
            }
            if (!ok) break;
            // ---- the row tile's sums: y, or a part of them
            const bool whole = at == tile_first && stop == tile_end;
            const bool in = row0 + r < pr.N;
            // y[half of the columns][row], the pointer moved on column by column
            auto store = [&]() {
                __nv_bfloat16* y = pr.y + half * kMine * pr.ldy + row0 + r;
#pragma unroll
                for (int j = 0; j < kMine; ++j, y += pr.ldy) {
                    if (j % 8 == 0) asm volatile("" : "+l"(y)::"memory");      // no 64 addresses at once
                    if (in && half * kMine + j < p.T) *y = __float2bfloat16_rn(acc[j]);
                }
            };
            if (whole) {
                store();
            } else {
                float* part = p.part + (((int64_t)blockIdx.x * 2 + (tile_first < first ? 0 : 1)) * N + half * kMine) * kWideRows + r;
#pragma unroll
                for (int j = 0; j < kMine; ++j) part[j * kWideRows] = acc[j];
            }
            if (!whole) {
                const int c0 = tile_first / p.per, c1 = (tile_end - 1) / p.per;
                __threadfence();
                if (!(ok = meet())) break;
                if (tid == 10 * 32) last_in = atomicAdd(&p.tickets[c0], 1u) == (uint32_t)(c1 - c0);
                if (!(ok = meet())) break;
                if (*reinterpret_cast<volatile uint32_t*>(&last_in)) {
                    __threadfence();
                    if (tid == 10 * 32) p.tickets[c0] = 0;
#pragma unroll
                    for (int j = 0; j < kMine; ++j) acc[j] = 0.f;
                    for (int c = c0; c <= c1; ++c) {
                        const float* from = p.part + (((int64_t)c * 2 + (tile_first < c * p.per ? 0 : 1)) * N + half * kMine) * kWideRows + r;
#pragma unroll
                        for (int j = 0; j < kMine; ++j) {
                            if (j % 8 == 0) asm volatile("" ::: "memory");     // eight loads at a time: registers
                            acc[j] += __ldcg(from + j * kWideRows);
                        }
                    }
                    store();
                }
                if (!(ok = meet())) break;
            }
            at = stop;
        }
        if (!ok && lane == 0) set_error(prm.err, LORA_DERR_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

}  // namespace lora
