// y = x W^T with 4-bit weights for more rows of x than w4_matvec.cuh takes (up to 128 a launch).
//
// The same sums as w4_matvec.cuh (exact differences of codes and zero points, one scale per
// group in fp32), with the fifth-generation tensor cores: 128 rows of W are the M of a
// tcgen05.mma whose A operand lies in tensor memory, where the unpacking warps write it, and
// the rows of x are its N, in shared memory as TMA lays them (128-byte swizzle).  A group's
// product is complete in D before its scale is known to apply, so D is drained once per
// group: a thread per row of W reads its columns and adds scale * D to sums in registers.
// Half a byte a weight from memory is the floor; unpacking (13 / 8 instructions a weight, in
// the order of K) and draining (one FMA per group, row and column) fill most of the issue
// slots of that time at 64 rows.  Measured on two 14336 x 4096 of groups of 128: 17 rows 24.2 us,
// 64 rows 26.5 us (36% of the copy rate), 128 rows 39.6 us (40% of the bf16 rate); groups of 64
// and 32 at 64 rows 30 and 41 us.  An MMA of 128 rows with A in tensor memory takes 64 clocks
// for any N up to 128, so a block is 1024 clocks of MMA at least; it takes about 1500, with some
// 3,900 instructions.
//
// One CTA per SM: warp 0 streams codes (blocks of 128 rows x 256 of K) by TMA and warp 11 x,
// warp 1 issues the MMAs, warps 2-9 unpack, warp 10 brings scales and zero points, the others
// drain.  CTAs take equal contiguous ranges of
// the blocks of all projections; a row tile shared by several CTAs is joined over partial
// sums in the workspace by the CTA that arrives last, in the order of K.
#pragma once
#include <cuda.h>

#include "w4_matvec.cuh"

namespace lora {

constexpr int kWideRows = 128;                 // rows of W of a block
constexpr int kWideK = 256;                    // K of a block
constexpr int kWideMaxCtas = 192;
constexpr int kWideCodeBytes = kWideRows * kWideK / 2;

// Shapes by the columns N (rows of x) and the group.  A span is what the roles hand over at
// once: a block's 256 of K, or 128 where the x stages of 256 would not fit.  Half of tensor
// memory holds the spans' A operands, half the D sums of `set` groups, twice.
__host__ __device__ constexpr int wide_span(int n) { return n > 64 ? 128 : 256; }
__host__ __device__ constexpr int wide_spans(int n) { return 512 / wide_span(n); }    // A buffers and x stages
__host__ __device__ constexpr int wide_set(int n, int group) {
    return 128 / n < wide_span(n) / group ? 128 / n : wide_span(n) / group;
}
__host__ __device__ constexpr int wide_code_stages(int n) { return n > 64 ? 3 : 4; }
// Warps that drain: a thread holds at most 64 columns' sums.
__host__ __device__ constexpr int wide_drain(int n) { return n > 64 ? 8 : 4; }
__host__ __device__ constexpr int wide_threads(int n) { return (12 + wide_drain(n)) * 32; }
// A stage's scales [groups][128] f16 and zeros [groups][64 bytes].
__host__ __device__ constexpr int wide_param_bytes(int group) { return (kWideK / group) * (kWideRows * 2 + kWideRows / 2); }
__host__ __device__ constexpr size_t wide_smem(int n, int group) {
    return 1024 + (size_t)wide_code_stages(n) * (kWideCodeBytes + wide_param_bytes(group)) + (size_t)n * 512 * 2 +
           (size_t)n * kWideRows * 2;
}
__host__ __device__ constexpr size_t wide_workspace(int n) {
    return kStepPartAt + (size_t)kWideMaxCtas * 2 * kWideRows * n * 4;
}

struct WideParams {
    CUtensorMap codes[LORA_W4_MAX_PROBLEMS];   // bytes {K / 2, N}, box {128, 128}, 128-byte swizzle
    CUtensorMap x[LORA_W4_MAX_PROBLEMS];       // bf16 {K, T}, box {64, N columns}, 128-byte swizzle
    CUtensorMap y[LORA_W4_MAX_PROBLEMS];       // bf16 {N, T}, box {128, N columns}
    W4Params p;                                // blocks of 128 x 256
    uint32_t* err;
    uint64_t limit_ns;                         // of every wait
    int32_t lost;                              // a block whose codes never come (a test of the waits), or -1
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

template <int G, int N>
__global__ void __launch_bounds__(wide_threads(N), 1) w4_wide_kernel(const __grid_constant__ WideParams prm) {
    constexpr int kSpan = wide_span(N), kSpans = wide_spans(N), kCodeStages = wide_code_stages(N);
    constexpr int kXBytes = N * kSpan * 2, kParams = wide_param_bytes(G), kBlockGroups = kWideK / G;
    constexpr int kSet = wide_set(N, G), kSets = kSpan / G / kSet;    // groups of a D set, sets of a span
    constexpr int kDrain = wide_drain(N), kMine = N / (kDrain / 4);   // columns of a drain thread
    // D sets at columns 0 and 128, A buffers from 256.  A set's MMAs end in one commit, to
    // d_full[set % kDone]; the commit of a span's last set also says that its A buffer and x
    // stage are free.
    constexpr uint32_t kDCols = 128, kACol = 256;
    constexpr int kDone = kSpans * kSets, kJoin = N > 64 ? 32 : 64;
    extern __shared__ unsigned char raw[];
    __shared__ __align__(8) uint64_t code_full[kCodeStages], code_empty[kCodeStages], a_full[kSpans], d_full[kDone], d_empty[2],
        final_bar;
    __shared__ uint32_t tmem_slot, last_in;
    const W4Params& p = prm.p;
    unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const uint32_t codes0 = smem_addr(base), x0 = codes0 + kCodeStages * kWideCodeBytes, y0 = x0 + kSpans * kXBytes;
    const uint32_t params0 = y0 + N * kWideRows * 2;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int first = blockIdx.x * p.per, end = min(first + p.per, p.total);
    if (first >= end) return;
    auto bar = [](uint64_t& b) { return smem_addr(&b); };
    if (tid == 0) {
        for (int i = 0; i < kCodeStages; ++i) {
            mbar_init(bar(code_full[i]), 1 + 32);      // the TMA's bytes, and each lane's copies
            mbar_init(bar(code_empty[i]), 8 + kDrain);
        }
        // x's bytes, and the unpacking warps of the span
        for (int i = 0; i < kSpans; ++i) mbar_init(bar(a_full[i]), 1 + (kSpan == kWideK ? 8 : 4));
        for (int i = 0; i < kDone; ++i) mbar_init(bar(d_full[i]), 1);
        for (int i = 0; i < 2; ++i) mbar_init(bar(d_empty[i]), kDrain);
        mbar_init(bar(final_bar), 1);
        fence_mbar_init();
    }
    if (tid == 0 || tid == 11 * 32) {          // the first tiles' descriptors
        const int i = w4_prob_of(p, first);
        if (tid == 0) prefetch_tmap(&prm.codes[i]);
        else prefetch_tmap(&prm.x[i]);
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

    const uint32_t spans = kWideK / kSpan * (uint32_t)(end - first);   // of this CTA's range
    // a wait by a warp together: its lanes go on, or give up, as one
    auto wait = [&](uint64_t& which, uint32_t parity) {
        return (bool)__all_sync(0xffffffffu, mbar_wait(bar(which), parity, prm.limit_ns));
    };
    if (warp == 0) {
        // ------------------------------------------------------------------ codes, one thread
        if (lane == 0) {
            WideAt a = wide_at(p, first);
            uint32_t ic = 0;
            for (int u = first; u < end && u != prm.lost; ++u, wide_next(p, a), ++ic) {
                const uint32_t s = ic % kCodeStages;
                if (!mbar_wait_quiet(bar(code_empty[s]), ((ic / kCodeStages) & 1) ^ 1, prm.limit_ns)) { ok = false; break; }
                mbar_arrive_expect_tx(bar(code_full[s]), kWideCodeBytes);
                tma_load_2d(codes0 + s * kWideCodeBytes, &prm.codes[a.prob], a.kb * (kWideK / 2), a.tile * kWideRows,
                            bar(code_full[s]));
            }
            if (!ok) set_error(prm.err, LORA_DERR_TIMEOUT);
            // every copy has landed before the CTA can end
            for (uint32_t k = ic > kCodeStages ? ic - kCodeStages : 0; k < ic; ++k)
                mbar_wait_quiet(bar(code_full[k % kCodeStages]), (k / kCodeStages) & 1, 100000000ull);
        }
        __syncwarp();
    } else if (warp == 11) {
        // ------------------------------------------------------------------ x, one thread
        if (lane == 0) {
            WideAt a = wide_at(p, first);
            uint32_t ix = 0;
            for (int u = first; u < end && ok; ++u, wide_next(p, a)) {
                for (int c = 0; c < kWideK / kSpan; ++c, ++ix) {
                    const uint32_t b = ix % kSpans;
                    if (!mbar_wait_quiet(bar(d_full[b * kSets + kSets - 1]), ((ix / kSpans) & 1) ^ 1, prm.limit_ns)) { ok = false; break; }
                    mbar_arrive_expect_tx(bar(a_full[b]), kXBytes);
#pragma unroll
                    for (int h = 0; h < kSpan / 64; ++h)
                        tma_load_2d(x0 + b * kXBytes + h * N * 128, &prm.x[a.prob], a.kb * kWideK + c * kSpan + h * 64, 0, bar(a_full[b]));
                }
            }
            if (!ok) set_error(prm.err, LORA_DERR_TIMEOUT);
            for (uint32_t k = ix > kSpans ? ix - kSpans : 0; k < ix; ++k)
                mbar_wait_quiet(bar(a_full[k % kSpans]), (k / kSpans) & 1, 100000000ull);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------------ MMA issue: the warp in step, one lane issues
        constexpr uint32_t idesc = idesc_bf16(128, N, 0, 0);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t x_desc = smem_desc(__shfl_sync(0xffffffffu, x0, 0), 16, 1024, 2);
        const uint32_t n_spans = __shfl_sync(0xffffffffu, spans, 0);
        auto wait_quiet = [&](uint64_t& which, uint32_t parity) {
            return (bool)__all_sync(0xffffffffu, mbar_wait_quiet(bar(which), parity, prm.limit_ns));
        };
        uint32_t id = 0;                       // D sets
        for (uint32_t i = 0; i < n_spans && ok; ++i) {
            const uint32_t b = i % kSpans;
            if (!wait_quiet(a_full[b], (i / kSpans) & 1)) { ok = false; break; }
            const uint64_t db = desc_at(x_desc, b * kXBytes);
#pragma unroll
            for (int s = 0; s < kSets; ++s, ++id) {
                if (!wait_quiet(d_empty[id & 1], ((id >> 1) & 1) ^ 1)) { ok = false; break; }
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kSet * G / 16; ++k) {
                        const int ks = s * (kSet * G / 16) + k;
                        tc_mma_f16_ts(tm + (id & 1) * kDCols + k / (G / 16) * N, tm + kACol + b * (kSpan / 2) + ks * 8,
                                      desc_at(db, (ks / 4) * (N * 128) + (ks % 4) * 32), idesc, k % (G / 16) != 0);
                    }
                    tc_commit(bar(d_full[b * kSets + s]));
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) set_error(prm.err, LORA_DERR_TIMEOUT);
        if (elect_one()) tc_commit(bar(final_bar));     // the MMAs are done before tensor memory is given back
        __syncwarp();
        mbar_wait_quiet(bar(final_bar), 0, 100000000ull);
        __syncwarp();
    } else if (warp == 10) {
        // ------------------------------------------------------------------ scales and zero points
        WideAt a = wide_at(p, first);
        uint32_t ic = 0;
        for (int u = first; u < end && ok; ++u, wide_next(p, a), ++ic) {
            const W4Prob& pr = p.prob[a.prob];
            const uint32_t s = ic % kCodeStages;
            if (!mbar_wait_quiet(bar(code_empty[s]), ((ic / kCodeStages) & 1) ^ 1, prm.limit_ns)) { ok = false; break; }
            const int row0 = a.tile * kWideRows, groups = pr.K / G;
            for (int i = lane; i < kBlockGroups * 16; i += 32) {       // 8 rows of a group's scales, and of its zeros
                const int g = i / 16, j = i % 16, grp = a.kb * kBlockGroups + g;
                const bool in = grp < groups && row0 + j * 8 < pr.N;
                const uint32_t dst = params0 + s * kParams;
                cp_async16(dst + g * kWideRows * 2 + j * 16, pr.scales + (in ? ((int64_t)grp * pr.N + row0 + j * 8) * 2 : 0), in ? 16 : 0);
                if (pr.zeros)
                    cp_async4(dst + kBlockGroups * kWideRows * 2 + g * (kWideRows / 2) + j * 4,
                              pr.zeros + (in ? (int64_t)grp * (pr.N / 2) + row0 / 2 + j * 4 : 0), in ? 4 : 0);
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar(code_full[s])) : "memory");
        }
        if (!ok && lane == 0) set_error(prm.err, LORA_DERR_TIMEOUT);
        cp_async_wait<0>();
    } else if (warp < 10) {
        // ------------------------------------------------------------------ unpacking: a row, every other 128 of K
        const int quad = warp & 3, turn = (warp - 2) >> 2, r = quad * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        WideAt a = wide_at(p, first);
        uint32_t ic = 0;
        for (int u = first; u < end && ok; ++u, ++ic, wide_next(p, a)) {
            const W4Prob& pr = p.prob[a.prob];
            const bool zeros = pr.zeros != nullptr;
            const uint32_t s = ic % kCodeStages;
            if (!wait(code_full[s], (ic / kCodeStages) & 1)) { ok = false; break; }
            {
                const int c = turn;
                const uint32_t i = kSpan == kWideK ? ic : 2 * ic + c, b = i % kSpans;   // span
                const uint32_t acol = tmem + lane_base + kACol + b * (kSpan / 2) + (kSpan == kWideK ? c * 64 : 0);
                uint32_t minus[128 / G];                           // 128 + zero twice, of the row's groups
#pragma unroll
                for (int g = 0; g < 128 / G; ++g) {
                    minus[g] = kMinus8;
                    if (zeros) {
                        uint32_t z;
                        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(z)
                                     : "r"(params0 + s * kParams + kBlockGroups * kWideRows * 2 + (c * (128 / G) + g) * (kWideRows / 2) + r / 2));
                        minus[g] = 0x43004300u + (z >> (r & 1) * 4 & 15u) * 0x00010001u;
                    }
                }
                uint32_t out[2][32];                               // 64 of K: 32 columns of tensor memory
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int col = c * 4 + h * 2 + j;         // 16-byte column of the row
                        const uint4 w = lds128(codes0 + s * kWideCodeBytes + r * 128 + ((col ^ (r & 7)) << 4));
                        const uint32_t m = minus[(h * 64 + j * 32) / G];
                        codes_in_order(w.x, m, out[h] + j * 16);
                        codes_in_order(w.y, m, out[h] + j * 16 + 4);
                        codes_in_order(w.z, m, out[h] + j * 16 + 8);
                        codes_in_order(w.w, m, out[h] + j * 16 + 12);
                    }
                if (!wait(d_full[b * kSets + kSets - 1], ((i / kSpans) & 1) ^ 1)) { ok = false; break; }
                tc_fence_after();
                tmem_st32(acol, out[0]);
                tmem_st32(acol + 32, out[1]);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(a_full[b]));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(code_empty[s]));
        }
        if (!ok && lane == 0) set_error(prm.err, LORA_DERR_TIMEOUT);
    } else {
        // ------------------------------------------------------------------ draining: a row, half of the columns
        const int quad = warp & 3, half = (warp - 12) >> 2, r = quad * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        WideAt a = wide_at(p, first);
        uint32_t id = 0, ic = 0;
        // The draining warps meet at a named barrier, so none of them leaves early: after a wait
        // that ran out they take no more part in the hand-overs, but still count their parts of
        // the range's tiles (with the error set), so that the counters end as they began.
        auto meet = [&]() { named_bar_sync(1, kDrain * 32); };
        for (int at = first; at < end;) {
            const W4Prob& pr = p.prob[a.prob];
            const int row0 = a.tile * kWideRows;
            const int tile_first = at - a.kb, tile_end = tile_first + pr.kblocks, stop = min(tile_end, end);
            float acc[kMine];
#pragma unroll
            for (int j = 0; j < kMine; ++j) acc[j] = 0.f;
            for (int u = at; u < stop && ok; ++u) {
                const uint32_t st = ic % kCodeStages;
                if (!wait(code_full[st], (ic / kCodeStages) & 1)) { ok = false; break; }
#pragma unroll
                for (int c = 0; c < kBlockGroups / kSet; ++c, ++id) {
                    float s[kSet];
#pragma unroll
                    for (int i = 0; i < kSet; ++i) {
                        unsigned short h;
                        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h)
                                     : "r"(params0 + st * kParams + ((c * kSet + i) * kWideRows + r) * 2));
                        s[i] = __half2float(__ushort_as_half(h));
                    }
                    if (!wait(d_full[id % kDone], (id / kDone) & 1)) { ok = false; break; }
                    tc_fence_after();
#pragma unroll
                    for (int g = 0; g < kSet; ++g)
#pragma unroll
                        for (int j = 0; j < kMine; j += 16) {
                            float v[16];
                            tmem_ld16(tmem + lane_base + (id & 1) * kDCols + g * N + half * kMine + j, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 16; i += 2) fma2_f32(acc[j + i], acc[j + i + 1], s[g], v[i], v[i + 1]);
                        }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(d_empty[id & 1]));
                }
                if (!ok) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(code_empty[st]));
                wide_next(p, a);
                ++ic;
            }
            if (!ok && stop < end) a = wide_at(p, stop);
            // ---- the row tile's sums: y, or a part of them
            const bool whole = at == tile_first && stop == tile_end;
            auto part_of = [&](int64_t slot) { return reinterpret_cast<float4*>(p.part + (slot * N + half * kMine) * kWideRows) + r; };
            // y's tile, [column][row of W], through shared memory and one bulk store (what lies
            // outside y is not written)
            auto store = [&]() {
                if (tid == 12 * 32) bulk_wait_read0();             // the last store has left the buffer
                meet();
#pragma unroll
                for (int j = 0; j < kMine; ++j)
                    asm volatile("st.shared.u16 [%0], %1;" ::"r"(y0 + ((half * kMine + j) * kWideRows + r) * 2),
                                 "h"(__bfloat16_as_ushort(__float2bfloat16_rn(acc[j]))) : "memory");
                fence_proxy_async_smem();
                meet();
                if (tid == 12 * 32) {
                    tma_store_2d(&prm.y[&pr - p.prob], row0, 0, y0);
                    bulk_commit();
                }
            };
            if (whole) {
                store();
            } else {
                // a part lies [column / 4][row][4]
                float4* part = part_of((int64_t)blockIdx.x * 2 + (tile_first < first ? 0 : 1));
#pragma unroll
                for (int j = 0; j < kMine; j += 4) part[j / 4 * kWideRows] = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
            }
            if (!whole) {
                const int c0 = tile_first / p.per, c1 = (tile_end - 1) / p.per;
                __threadfence();
                meet();
                if (tid == 12 * 32) last_in = atomicAdd(&p.tickets[c0], 1u) == (uint32_t)(c1 - c0);
                meet();
                if (*reinterpret_cast<volatile uint32_t*>(&last_in)) {
                    __threadfence();
                    if (tid == 12 * 32) p.tickets[c0] = 0;
#pragma unroll
                    for (int j = 0; j < kMine; ++j) acc[j] = 0.f;
                    for (int c = c0; c <= c1; ++c) {
                        const float4* from = part_of((int64_t)c * 2 + (tile_first < c * p.per ? 0 : 1));
#pragma unroll
                        for (int j = 0; j < kMine; j += 4) {
                            if (j % kJoin == 0) asm volatile("" ::: "memory"); // so many values in flight: registers
                            const float4 x = __ldcg(from + j / 4 * kWideRows);
                            acc[j] += x.x;
                            acc[j + 1] += x.y;
                            acc[j + 2] += x.z;
                            acc[j + 3] += x.w;
                        }
                    }
                    store();
                }
                meet();
            }
            at = stop;
        }
        if (tid == 12 * 32) bulk_wait0();
        if (!ok && lane == 0) set_error(prm.err, LORA_DERR_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

}  // namespace lora
