// y = x W^T of 8-bit integers with a scale per row of x and per row of W, for many rows of x.
//
// The sums of w8_narrow.cuh on the fifth-generation tensor cores: codes as f16, where they are
// exact, and their products summed in fp32, which holds whole numbers up to 2^24 exactly (sums
// past that are rounded as fp32 sums are).
//
// Two CTAs of a cluster make one tile of 256 rows of W by up to 256 rows of x: each holds its
// 128 rows of W, widened into its tensor memory as the A operand, and half of the rows of x in
// shared memory, where one TMA load serves both SMs' products.  x comes in f16 from the
// workspace, where w8_widen_kernel puts it once a call; W, the long side, is widened on the
// way, so that memory sees one byte a weight.
//
// Warp 0 streams W (128 rows x 128 of K a CTA and step) and warp 2 x by TMA, warps 4 to 11
// widen W into tensor memory, warp 1 of the even CTA issues the MMAs of both, warps 12 to 19
// take the sums out.  The pairs take equal contiguous ranges of the steps of all tiles, or whole
// tiles in turn, so that neighbours work on the same W at a time (300 rows of two 14336 x 4096:
// 49 us with a pair's tiles in a row, 46 in turn); a tile shared by several pairs is joined over
// partial sums in the workspace by the one that arrives last, in the order of K.
//
// 64 rows of 117 MB take 27 us (4.4 TB/s): TMA boxes of 128 bytes of 128 rows stream at 5.3 TB/s alone,
// and the start takes 4.9 us to the first W.  2,011 rows of two 14336 x 4096 take 232 us, 253 where the power
// limit holds the clock down (2.0 and 1.9 PFLOP/s, the tensor pipe busy 92% of the time), 700 rows of 4096 x 14336
// 55.8 (1.47 PFLOP/s: 64 tiles for 76 pairs, and 5 us of x's widening before them).  Small W is far from memory's
// rate: 64 rows of 17 MB take 15 to 16 us, of 25 MB 16 to 18, of 59 MB 22.5, the start and the join of few tiles.
#pragma once
#include <cuda.h>

#include "w8_narrow.cuh"

namespace lora {

constexpr int kW8WideRows = 256;               // rows of W of a tile: 128 a CTA
constexpr int kW8WideK = 128;                  // K of a step
constexpr int kW8WideThreads = 640;
constexpr int kW8MaxPairs = 96;
constexpr int kW8WBytes = 128 * kW8WideK;

constexpr int kW8Bufs = 4;                     // A buffers in tensor memory and stages of x
constexpr int kW8JoinBufs = 5;                 // pieces of parts under way in a join, 32 columns of 128 rows each
constexpr int kW8PieceBytes = 32 * 128 * 4;
// By the most columns (rows of x) of a tile: stages of W, an even number.  64 rows of two 14336 x 4096
// take 28 us with 6, 8 or 12 of them and 31 with 4.
__host__ __device__ constexpr int w8_w_stages(int n) { return n > 128 ? 6 : 8; }
__host__ __device__ constexpr size_t w8_wide_smem(int n) {
    return 1024 + (size_t)w8_w_stages(n) * kW8WBytes + (size_t)kW8Bufs * n * 128;
}
// Partial sums of a CTA: two tiles' of 128 rows.
__host__ __device__ constexpr size_t w8_part_floats(int n) { return (size_t)128 * n; }
__host__ __device__ constexpr size_t w8_part_bytes(int n) { return (size_t)kW8MaxPairs * 2 * 2 * w8_part_floats(n) * 4; }

struct W8WideProb {
    const float* x_scales;
    const float* w_scales;
    __nv_bfloat16* y;
    int64_t ldy;
    int32_t N;
    int32_t kblocks;
    int32_t first;                             // steps before the projection
    int32_t xi;                                // its map of x
};

struct W8WideParams {
    CUtensorMap w[LORA_W8_MAX_PROBLEMS];       // bytes {K, N}, box {128, 128}, 128-byte swizzle
    CUtensorMap x[LORA_W8_MAX_PROBLEMS];       // f16 {K, T}, box {64, cols / 2}, 128-byte swizzle
    W8WideProb prob[LORA_W8_MAX_PROBLEMS];
    int32_t nprob;
    int32_t T;
    int32_t cols;                              // rows of x of a tile, a multiple of 32 as an MMA over two CTAs takes them
    int32_t ttiles;                            // tiles along x
    int32_t total;                             // steps
    int32_t per;                               // shares: steps of a pair; whole tiles: its tiles, of the first `more` pairs one more
    int32_t more;
    int32_t over_rt, over_tt;                  // whole tiles: from a pair's tile to its next, along W and along x
    uint32_t* tickets;                         // [kStepTickets], zero between calls
    float* part;
    uint32_t* err;
    uint64_t limit_ns;                         // of every wait
    int32_t lost, lost_pair;                   // a step whose W never comes (a test of the waits), or -1; whole tiles: of that pair's
};

// ---------------------------------------------------------------------------- x in f16
struct W8Widen {
    const unsigned char* x[LORA_W8_MAX_PROBLEMS];
    uint32_t* out[LORA_W8_MAX_PROBLEMS];       // f16 [T][K]
    int64_t ldx[LORA_W8_MAX_PROBLEMS];
    int32_t K[LORA_W8_MAX_PROBLEMS];
    int32_t T;
};
constexpr int kWidenThreads = 256, kWidenAhead = 2;

// Sixteen codes a thread and time, two times in flight; blockIdx.y: the matrix.  At most one CTA of
// these for each that an SM holds: the next kernel begins when all have begun.
__global__ void __launch_bounds__(kWidenThreads, 8) w8_widen_kernel(const __grid_constant__ W8Widen p) {
    // The order matters: the next kernel fetches W without a wait of its own, and W may be what the kernel before this
    // one wrote.  It begins when all CTAs of this one have seen that kernel's end.
    grid_wait();
    grid_let_next();
    const int i = blockIdx.y;
    const uint32_t per_row = p.K[i] / 16, n = p.T * per_row, step = gridDim.x * kWidenThreads;   // n <= 2^28
    for (uint32_t e = blockIdx.x * kWidenThreads + threadIdx.x; e < n; e += kWidenAhead * step) {
        uint4 v[kWidenAhead];
#pragma unroll
        for (int k = 0; k < kWidenAhead; ++k) {
            const uint32_t at = min(e + k * step, n - 1), row = at / per_row;
            v[k] = ld16(p.x[i] + row * p.ldx[i] + (at - row * per_row) * 16);
        }
#pragma unroll
        for (int k = 0; k < kWidenAhead; ++k) {
            if (e + k * step >= n) break;
            uint4 a, b;
            codes8_f16(v[k].x, a.x, a.y);
            codes8_f16(v[k].y, a.z, a.w);
            codes8_f16(v[k].z, b.x, b.y);
            codes8_f16(v[k].w, b.z, b.w);
            // rows lie end to end, 32-byte aligned
            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p.out[i] + (int64_t)(e + k * step) * 8), "r"(a.x),
                         "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                         : "memory");
        }
    }
}

// ---------------------------------------------------------------------------- pairs of CTAs
__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// The address of `addr` (this CTA's shared memory) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Arrives on a barrier of either CTA.  What it announces is tensor memory, which tcgen05.wait and
// tcgen05.fence order, so the release is that of a CTA: one of cluster scope drains every memory
// access of the thread first (about 800 clocks a step, two thirds of the kernel's time).
__device__ __forceinline__ void mbar_arrive_at(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A 2-D TMA load into this CTA whose bytes count on the even CTA's barrier.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const void* tmap, int32_t c0, int32_t c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(tmap), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
// D[tmem of both] (+)= A[tmem of both] x B[half in each CTA's shared memory], f16.
__device__ __forceinline__ void tc_mma_pair(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive once on the barrier at `bar` of both CTAs when this thread's MMAs so far are done.
__device__ __forceinline__ void tc_commit_pair(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"((uint16_t)3)
                 : "memory");
}

// Waits for the loads of tensor memory into v.
__device__ __forceinline__ void tmem_ld_wait16(float (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]),
                   "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
                 :
                 : "memory");
}
template <int R>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// A step: projection, tiles along W and along x, block of K.
struct W8At {
    int prob, rt, tt, kb;
};
__device__ __forceinline__ W8At w8_at(const W8WideParams& p, int u) {
    W8At a;
    a.prob = 0;
    while (a.prob + 1 < p.nprob && u >= p.prob[a.prob + 1].first) ++a.prob;
    const int b = u - p.prob[a.prob].first, tile = b / p.prob[a.prob].kblocks;
    a.kb = b - tile * p.prob[a.prob].kblocks;
    a.rt = tile / p.ttiles;
    a.tt = tile - a.rt * p.ttiles;
    return a;
}
// A pair's next tile: the next one of all, or of whole tiles, which go to the pairs in turn, the one past the others'.
template <bool SPLIT>
__device__ __forceinline__ void w8_next_tile(const W8WideParams& p, W8At& a) {
    a.kb = 0;
    a.tt += SPLIT ? 1 : p.over_tt;
    if (!SPLIT) a.rt += p.over_rt;
    if (a.tt >= p.ttiles) {
        a.tt -= p.ttiles;
        ++a.rt;
    }
    while (a.prob < p.nprob && a.rt * kW8WideRows >= p.prob[a.prob].N) {
        a.rt -= (p.prob[a.prob].N + kW8WideRows - 1) / kW8WideRows;
        ++a.prob;
    }
}
template <bool SPLIT>
__device__ __forceinline__ void w8_next(const W8WideParams& p, W8At& a) {
    if (++a.kb == p.prob[a.prob].kblocks) w8_next_tile<SPLIT>(p, a);
}

// Sixteen columns' sums as bf16 pairs of y.
__device__ __forceinline__ void w8_scale(const float (&v)[16], const float* sx, float sw, uint32_t* to) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float4 f = reinterpret_cast<const float4*>(sx)[j];
        to[2 * j] = pack2(v[4 * j] * f.x * sw, v[4 * j + 1] * f.y * sw);
        to[2 * j + 1] = pack2(v[4 * j + 2] * f.z * sw, v[4 * j + 3] * f.w * sw);
    }
}
// Sixteen columns of y.  Neighbouring lanes swap halves, so that a lane stores two rows of W of one
// column: 64 bytes a column and warp.
__device__ __forceinline__ void w8_store(const uint32_t* from, __nv_bfloat16*& to, int64_t two, int& left) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t mine = from[j], other = __shfl_xor_sync(0xffffffffu, mine, 1);
        const uint32_t v = __byte_perm(mine, other, threadIdx.x & 1 ? 0x3276 : 0x5410);
        if (left > 0) *reinterpret_cast<uint32_t*>(to) = v;
        left -= 2;
        to += two;
    }
}

// Where part q of a tile's n lies, from the place of the pair that begins it: its own in the second of
// that pair's two slots, the next pairs' in their first.
__device__ __forceinline__ const float* w8_part(const float* first, int q, int64_t slot) { return first + (q ? 4 * q : 1) * slot; }
__device__ __forceinline__ void w8_add(float (&sum)[16], int i, const float4& x) {
    sum[4 * i] += x.x;
    sum[4 * i + 1] += x.y;
    sum[4 * i + 2] += x.z;
    sum[4 * i + 3] += x.w;
}

// NMAX: the most columns of a tile.  SPLIT: whether a pair's range may begin or end inside a tile
// (the code for that takes registers from the path of whole tiles).
template <int NMAX, bool SPLIT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kW8WideThreads, 1) w8_wide_kernel(const __grid_constant__ W8WideParams p) {
    constexpr int kWStages = w8_w_stages(NMAX), kXStage = NMAX * 128;
    // Registers move from the warps that issue and widen to those that hold a row's sums: the shares of
    // the five groups of four warps add up to the 480 of the launch.  (A few spilled registers in the
    // path of whole tiles cost as much as the path itself: those kernels spill none.  Of those for shares the one of
    // up to 128 columns spills seven, 28 bytes.)
    constexpr int kDs = NMAX > 128 ? 1 : 2;    // D buffers, 128 columns apart
    constexpr int kRegsOut = NMAX > 128 ? 160 : 136, kRegsWiden = NMAX > 128 ? 56 : 80, kRegsMisc = 48;
    static_assert(kRegsMisc + 2 * kRegsWiden + 2 * kRegsOut <= 480, "registers of the launch");
    // A wait for a barrier's phase must not fall two phases behind.  The two groups of widening warps take
    // the steps in turn, so each stage and buffer has to belong to one of them: with an odd number, a
    // group may come to a stage whose last step the other one has not even seen arrive.
    static_assert(kWStages % 2 == 0 && kW8Bufs % 2 == 0, "stages of one group each");
    constexpr uint32_t kACol = 256;            // D in columns 0 .. 255, four A buffers of 64 columns after it
    extern __shared__ unsigned char raw[];
    __shared__ __align__(8) uint64_t w_full[kWStages], w_empty[kWStages], ready[kW8Bufs], freed[kW8Bufs], d_full[kDs], d_empty[kDs], final_bar;
    __shared__ __align__(8) uint64_t piece[2][kW8JoinBufs];
    __shared__ __align__(16) float sx[2][128];
    __shared__ uint32_t tmem_slot, last_in[2], lost[2];
    unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const uint32_t w0 = smem_addr(base), x0 = w0 + kWStages * kW8WBytes;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cta_rank();
    const int pair = blockIdx.x >> 1;
    // The steps of this pair: of all tiles' steps, or counted within its own whole tiles
    const int blocks = p.prob[0].kblocks;
    const int first = SPLIT ? min(pair * p.per, p.total) : 0;
    const int end = SPLIT ? min(first + p.per, p.total) : (p.per + (pair < p.more)) * blocks;
    const int start = SPLIT ? first : pair * blocks;
    const int half_cols = p.cols / 2;
    auto bar = [](uint64_t& b) { return smem_addr(&b); };
    if (tid < kWStages) {
        mbar_init(bar(w_full[tid]), 1);
        mbar_init(bar(w_empty[tid]), 4);
        fence_mbar_init();
    } else if (tid >= 32 && tid < 32 + kW8Bufs) {
        mbar_init(bar(ready[tid - 32]), 1 + 8);        // of the even CTA: x's bytes in both, and both CTAs' four widening warps
        mbar_init(bar(freed[tid - 32]), 1);
        fence_mbar_init();
    } else if (tid == 64) {
        for (int i = 0; i < kDs; ++i) {
            mbar_init(bar(d_full[i]), 1);
            mbar_init(bar(d_empty[i]), 16);
        }
        mbar_init(bar(final_bar), 1);
        lost[0] = lost[1] = 0;
        fence_mbar_init();
    } else if (SPLIT && tid >= 128 && tid < 128 + 2 * kW8JoinBufs) {
        mbar_init(bar(piece[0][tid - 128]), 1);
        fence_mbar_init();
    }
    if (warp == 3) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&tmem_slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    if (tid == 352 || tid == 384) {                            // the first tile's maps, on their way meanwhile
        const W8At a = w8_at(p, start);
        prefetch_tmap(tid == 352 ? &p.w[a.prob] : &p.x[p.prob[a.prob].xi]);
    }
    tc_fence_before();
    cluster_sync();                                            // nothing is fetched before: W's loads delay all others
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&tmem_slot);
    bool ok = true;
    auto wait = [&](uint64_t& which, uint32_t parity) {
        return (bool)__all_sync(0xffffffffu, mbar_wait_quiet(bar(which), parity, p.limit_ns));
    };

    if (warp == 0) {
        // ------------------------------------------------------------------ W, one thread
        // No grid_wait: the widening, which this kernel's start overlaps, reads x and writes its copy, and let this kernel
        // begin only after the end of the kernel before it.  Everything else in global memory is touched after a grid_wait.
        regs_dec<kRegsMisc>();
        if (lane == 0) {
            W8At a = w8_at(p, start);
            const int lost = SPLIT || pair == p.lost_pair ? p.lost : -1;
            uint32_t i = 0;
            for (int u = first; u < end && u != lost; ++u, w8_next<SPLIT>(p, a), ++i) {
                const uint32_t s = i % kWStages;
                if (!mbar_wait_quiet(bar(w_empty[s]), ((i / kWStages) & 1) ^ 1, p.limit_ns)) { ok = false; break; }
                mbar_arrive_expect_tx(bar(w_full[s]), kW8WBytes);
                tma_load_2d(w0 + s * kW8WBytes, &p.w[a.prob], a.kb * kW8WideK, a.rt * kW8WideRows + (int)rank * 128, bar(w_full[s]));
            }
            if (!ok) set_error(p.err, LORA_DERR_TIMEOUT);
            // every copy has landed before the CTA can end
            for (uint32_t k = i > kWStages ? i - kWStages : 0; k < i; ++k)
                mbar_wait_quiet(bar(w_full[k % kWStages]), (k / kWStages) & 1, 100000000ull);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------------------------ x, one thread
        regs_dec<kRegsMisc>();
        if (lane == 0) {
            grid_wait();
            W8At a = w8_at(p, start);
            uint32_t i = 0;
            const uint32_t box = half_cols * 128;
            for (int u = first; u < end; ++u, w8_next<SPLIT>(p, a), ++i) {
                const uint32_t b = i % kW8Bufs;
                if (!mbar_wait_quiet(bar(freed[b]), ((i / kW8Bufs) & 1) ^ 1, p.limit_ns)) { ok = false; break; }
                const uint32_t at = mapa(bar(ready[b]), 0);
                if (rank == 0) mbar_arrive_expect_tx(bar(ready[b]), 4 * box);
                const CUtensorMap* map = &p.x[p.prob[a.prob].xi];
                const int row = a.tt * p.cols + (int)rank * half_cols;
                tma_load_2d_pair(x0 + b * kXStage, map, a.kb * kW8WideK, row, at);
                tma_load_2d_pair(x0 + b * kXStage + box, map, a.kb * kW8WideK + 64, row, at);
            }
            if (!ok) {
                // the copies count on the even CTA's barriers: those in flight land long before this
                set_error(p.err, LORA_DERR_TIMEOUT);
                for (const uint64_t t = global_timer_ns(); global_timer_ns() - t < 10000000ull;) {}
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------------ MMA issue, the even CTA's
        regs_dec<kRegsMisc>();
        if (rank == 0) {
            const uint32_t idesc = (1u << 4) | ((uint32_t)(p.cols >> 3) << 17) | ((256u >> 4) << 24);   // f16, fp32 sums
            const uint64_t x_desc = smem_desc(x0, 16, 1024, 2);
            const uint32_t box = half_cols * 128;
            W8At a = w8_at(p, start);
            uint32_t i = 0, tiles = 0;
            bool fresh = true;
            for (int u = first; u < end && ok; ++u, ++i) {
                const uint32_t b = i % kW8Bufs;
                const bool last = a.kb + 1 == p.prob[a.prob].kblocks || u + 1 == end;
                w8_next<SPLIT>(p, a);
                const uint32_t d = tiles % kDs;
                if (fresh && !wait(d_empty[d], ((tiles / kDs) & 1) ^ 1)) { ok = false; break; }
                if (!wait(ready[b], (i / kW8Bufs) & 1)) { ok = false; break; }
                tc_fence_after();
                const uint64_t db = desc_at(x_desc, b * kXStage);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kW8WideK / 16; ++k)
                        tc_mma_pair(tmem + d * 128, tmem + kACol + b * 64 + k * 8, desc_at(db, (k / 4) * box + (k % 4) * 32), idesc,
                                    !(fresh && k == 0));
                    tc_commit_pair(bar(freed[b]));
                    if (last) tc_commit_pair(bar(d_full[d]));
                }
                __syncwarp();
                fresh = last;
                tiles += last;
            }
            if (!ok && lane == 0) set_error(p.err, LORA_DERR_TIMEOUT);
            if (elect_one()) tc_commit_pair(bar(final_bar));
            __syncwarp();
        }
        mbar_wait_quiet(bar(final_bar), 0, 4 * p.limit_ns);   // the MMAs are done before tensor memory is given back
        __syncwarp();
    } else if (warp >= 4 && warp < 12) {
        // ------------------------------------------------------------------ widening: a row of W, every other step
        regs_dec<kRegsWiden>();
        const int quad = warp & 3, r = quad * 32 + lane;
        const uint32_t acol = tmem + ((uint32_t)(quad * 32) << 16) + kACol;
        uint32_t i = (warp - 4) >> 2;
        for (int u = first + (int)i; u < end; u += 2, i += 2) {
            const uint32_t s = i % kWStages, b = i % kW8Bufs;
            if (!wait(w_full[s], (i / kWStages) & 1)) { ok = false; break; }
#pragma unroll (NMAX > 128 ? 1 : 2)
            for (int h = 0; h < 2; ++h) {
                uint32_t out[32];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint4 v = lds128(w0 + s * kW8WBytes + r * 128 + (((h * 4 + c) ^ (r & 7)) << 4));
                    codes8_f16(v.x, out[c * 8], out[c * 8 + 1]);
                    codes8_f16(v.y, out[c * 8 + 2], out[c * 8 + 3]);
                    codes8_f16(v.z, out[c * 8 + 4], out[c * 8 + 5]);
                    codes8_f16(v.w, out[c * 8 + 6], out[c * 8 + 7]);
                }
                if (h == 0) {
                    if (!wait(freed[b], ((i / kW8Bufs) & 1) ^ 1)) { ok = false; break; }
                    tc_fence_after();
                }
                tmem_st32(acol + b * 64 + h * 32, out);
            }
            if (!ok) break;
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(w_empty[s]));
                mbar_arrive_at(mapa(bar(ready[b]), 0));
            }
        }
        if (!ok && lane == 0) set_error(p.err, LORA_DERR_TIMEOUT);
    } else if (warp >= 12) {
        // ------------------------------------------------------------------ sums out: a row of W, half of the columns
        regs_inc<kRegsOut>();
        grid_wait();                                           // the scales may be of the kernel before the widening
        const int quad = warp & 3, half = (warp - 12) >> 2, r = quad * 32 + lane, g = tid - (12 + 4 * half) * 32;
        constexpr int kChunks = NMAX / 32;
        const uint32_t dcol0 = tmem + ((uint32_t)(quad * 32) << 16) + half * half_cols;
        const int chunks = half_cols / 16;
        auto meet = [&]() { named_bar_sync(1 + half, 128); };
        W8At a = w8_at(p, start);
        uint32_t tiles = 0;
        for (int at = first; at < end; ++tiles) {
            const W8WideProb& pr = p.prob[a.prob];
            const uint32_t d = tiles % kDs, dcol = dcol0 + d * 128;
            const int tile_first = at - a.kb, tile_end = tile_first + pr.kblocks, stop = SPLIT ? min(tile_end, end) : tile_end;
            const int row0 = a.rt * kW8WideRows + (int)rank * 128, col0 = a.tt * p.cols + half * half_cols;
            const bool whole = !SPLIT || (at == tile_first && stop == tile_end);
            const float sw = row0 + r < pr.N ? pr.w_scales[row0 + r] : 0.f;
            meet();                                            // the last tile's scales have been read
            sx[half][g] = col0 + g < p.T && g < half_cols ? pr.x_scales[col0 + g] : 0.f;
            // after a wait that ran out the four warps take no more sums, as one, but still count
            // their parts of the range's tiles (with the error set), so that the tickets end as they began
            if (ok && !wait(d_full[d], (tiles / kDs) & 1)) lost[half] = 1;
            meet();
            ok = *reinterpret_cast<volatile uint32_t*>(&lost[half]) == 0;
            tc_fence_after();
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_at(mapa(bar(d_empty[d]), 0));
            };
            // a whole tile's sums become y in registers, a part goes out as it is: either way the
            // MMAs of the next tile wait for no store
            auto drain = [&](auto&& take) {
                float v[2][16];
                if (ok) {
                    tmem_ld16(dcol, v[0]);
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) {         // columns past the tile's are read for nothing
                        tmem_ld_wait16(v[c & 1]);
                        if (c + 1 < kChunks) tmem_ld16(dcol + (c + 1) * 16, v[(c + 1) & 1]);
                        take(c, v[c & 1]);
                    }
                }
                release();
            };
            if (whole) {
                uint32_t out[8 * kChunks];
                drain([&](int c, const float (&v)[16]) { w8_scale(v, &sx[half][c * 16], sw, out + c * 8); });
                if (ok) {
                    int left = row0 + r < pr.N ? p.T - col0 - (lane & 1) : 0;
                    int64_t two = 2 * pr.ldy;
                    __nv_bfloat16* to = pr.y + (int64_t)(col0 + (lane & 1)) * pr.ldy + row0 + (r & ~1);
                    asm volatile("" : "+l"(two), "+l"(to), "+r"(left));   // not before the sums are out: registers
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        if (c < chunks) w8_store(out + c * 8, to, two, left);
                }
            } else {
                // A part lies [column / 4][row][4].  This pair's, and the place of those of the pair that begins the tile:
                constexpr int64_t kSlot = w8_part_floats(NMAX);
                const int p0 = tile_first / p.per, p1 = (tile_end - 1) / p.per, n = p1 - p0 + 1;
                uint32_t* const ticket = p.tickets + (p0 * 2 + rank) * 2 + half;
                const float* const parts = p.part + (4 * (int64_t)p0 + 2 * rank) * kSlot + half * half_cols * 128;
                float4* const part = reinterpret_cast<float4*>(const_cast<float*>(w8_part(parts, pair - p0, kSlot))) + r;
                // The sum over all parts in the order of K; `mine`: the first one is in tensor memory.  At the end
                // of the pair's range its rings are free (the MMAs are done): the parts come through them
                // by bulk copies, since an answer takes 800 clocks, or 1,500 from the other die, and more
                // cannot be under way in registers.
                auto join = [&](int mine) {
                    const bool rings = stop == end && ok;
                    const uint32_t ring = w0 + half * kW8JoinBufs * kW8PieceBytes;
                    const int m = n - mine, all = (chunks + 1) / 2 * m;
                    int put = 0, got = 0;
                    auto fetch = [&]() {                       // pieces: 32 columns after 32, of one part after the other
                        for (; put < all && put < got + kW8JoinBufs; ++put) {
                            const int c = put / m, q = mine + put - c * m, b = put % kW8JoinBufs;
                            const uint32_t bytes = 2 * c + 1 < chunks ? kW8PieceBytes : kW8PieceBytes / 2;
                            mbar_arrive_expect_tx(bar(piece[half][b]), bytes);
                            bulk_g2s(ring + b * kW8PieceBytes, w8_part(parts, q, kSlot) + c * 4096, bytes, bar(piece[half][b]));
                        }
                    };
                    if (rings && g == 0) {
                        // parts were written by plain stores: they are seen by now, the copies have to see them too
                        asm volatile("fence.proxy.async;" ::: "memory");
                        fetch();
                    }
                    put = min(all, kW8JoinBufs);
                    int left = row0 + r < pr.N ? p.T - col0 - (lane & 1) : 0;
                    const int64_t two = 2 * pr.ldy;
                    __nv_bfloat16* to = pr.y + (int64_t)(col0 + (lane & 1)) * pr.ldy + row0 + (r & ~1);
                    for (int c = 0; c < chunks; c += 2) {      // past the last sixteen columns nothing is stored
                        float sum[2][16];
                        if (mine) {
                            tmem_ld16(dcol + c * 16, sum[0]);
                            tmem_ld16(dcol + (c + 1) * 16, sum[1]);
                            tmem_ld_wait16(sum[0]);
                            tmem_ld_wait16(sum[1]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i) sum[i / 16][i % 16] = 0.f;
                        }
                        for (int q = mine; q < n; ++q, ++got) {
                            if (rings && put < all && put - got <= kW8JoinBufs / 2) {
                                meet();                        // all have read the pieces before this one
                                if (g == 0) fetch();
                                put = min(all, got + kW8JoinBufs);
                            }
                            if (rings) {
                                const int b = got % kW8JoinBufs;
                                if (ok && !wait(piece[half][b], (got / kW8JoinBufs) & 1)) ok = false;
                                const uint32_t from = ring + b * kW8PieceBytes + r * 16;
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    const uint4 x = lds128(from + i * 2048);
                                    w8_add(sum[i / 4], i % 4, make_float4(__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w)));
                                }
                            } else {
                                const float4* from = reinterpret_cast<const float4*>(w8_part(parts, q, kSlot)) + c * 512 + r;
#pragma unroll
                                for (int i = 0; i < 8; ++i) w8_add(sum[i / 4], i % 4, __ldcg(from + (c + 1 < chunks ? i : i % 4) * 128));
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if (c + i == chunks) break;
                            uint32_t out[8];
                            w8_scale(sum[i], &sx[half][(c + i) * 16], sw, out);
                            w8_store(out, to, two, left);
                        }
                    }
                };
                // Where all other parts are there already (a pair comes to the tile that it begins last, when
                // the next pair has long done its rest), this one stays where it is.
                if (g == 0) {
                    uint32_t there = 0;
                    if (pair == p0) asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(there) : "l"(ticket) : "memory");
                    last_in[half] = there == (uint32_t)(n - 1);
                }
                meet();
                const bool early = *reinterpret_cast<volatile uint32_t*>(&last_in[half]) && ok;
                if (early) {
                    __threadfence();
                    join(1);
                    release();
                    if (g == 0) *ticket = 0;
                } else {
                    drain([&](int c, const float (&v)[16]) {
                        if (c >= chunks) return;
#pragma unroll
                        for (int j = 0; j < 4; ++j) part[(c * 4 + j) * 128] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                    });
                    __threadfence();
                    meet();
                    if (g == 0) last_in[half] = atomicAdd(ticket, 1u) == (uint32_t)(n - 1);
                    meet();
                    if (*reinterpret_cast<volatile uint32_t*>(&last_in[half])) {
                        __threadfence();
                        if (g == 0) *ticket = 0;
                        join(0);
                    }
                }
                meet();
            }
            at = stop;
            if (SPLIT && at < end) a = w8_at(p, at);
            if (!SPLIT) w8_next_tile<false>(p, a);
        }
        if (!ok && lane == 0) set_error(p.err, LORA_DERR_TIMEOUT);
    } else {
        regs_dec<kRegsMisc>();
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    if (warp == 3) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

}  // namespace lora
