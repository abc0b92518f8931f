// Causal attention of a batch's rows over the 4-bit cache, for few rows per request (decode
// and the check of a few drafted tokens).
//
// For one request and KV head the query rows that share the head (the request's rows times
// the query heads of the KV head) are the columns of a transposed product: with K and V as
// codes c in -8 .. 7 (exact in f16), a score is
//     q . k_t = sum over groups of  scale_t (q . c_t) + offset_t sum(q),
// so the MMA runs on the codes as they are, S^T = C_K q^T (tokens x rows, 16 tokens a tile),
// and the scale enters once per token in fp32.  q goes in as f16 times a power of two that
// puts a row's largest value at 2^13: its eight bits are kept for every value above 2^-27
// of the largest.  The output is likewise
//     O^T = C_V^T f16(x)  +  sum_t x_t (offset_t / scale_t),    x_t = scale_t p_t to 11 bits,
// where x_t is the one value that is rounded (2^-11 of itself) and both terms use it
// rounded: the sum is over whole values v_t with weights off by that much, however large
// scale and offset are against v_t.  The second sum takes x_t in fp32, at any size; only what
// f16 makes of an x_t below 2^-14, a multiple of 2^-24, is less exact, and it meets codes
// of 8 at most.  p_t = 2^(score log2 e - M) has the reference M where the largest scale_t p_t
// seen is 2^6 (x fits f16 whatever the scales), moved when an x exceeds f16's range: what is
// lost below it is 2^-31 of the largest x a token.
// ldmatrix hands each lane its words of codes in the operand's order (transposed for V,
// which pairs the tokens), so a code costs 9 / 8 instructions on its way to the tensor core.
// The tokens being the long side of both products, 8 rows fill an MMA; mma.sync serves
// because the kernel is bound by the bytes of the cache (136 a token and head) and next by
// the unpacking, not by the MMAs.
//
// Measured (grouped queries, 4 per KV head): 64 requests of 17 to 8191 tokens 64 us and two of
// 131k tokens 64 us, 62% of the copy rate on their 271 and 277 MB; one query head per KV head
// with groups of 32 (278 MB) 90 us.  (Weights rounded by the conversion to f16 alone, which loses
// those far below the largest: 63, 63 and 88.)  The tensor pipe is 22% busy, the issue slots 59%
// while warps are resident: about 650 instructions per 32 tokens of a head at 16 warps an SM.
//
// Work.  An item is (request, KV head, tile of 8 NT packed rows), of ceil(tokens / 32) steps
// and kAttItemCost more for its fixed part.  The units of all items in a row are dealt to
// the CTAs in equal contiguous ranges.  A short item that lies in one range is a warp's own
// (the CTA's warps take such items in turn, without meeting); of any other item the CTA's
// four warps take the steps in turn, each with its own bulk-copy ring and running maximum
// and sum, and merge at the end of the CTA's part.  An item that spans several CTAs is put
// together from partial results in the workspace by the CTA that arrives last, in the order
// of the parts, so the result does not depend on the order of arrival.
#pragma once
#include <type_traits>

#include "kv_layout.cuh"
#include "mma_legacy.cuh"

namespace lora {

constexpr int kAttWarps = 4;
constexpr int kAttThreads = kAttWarps * 32;
constexpr int kAttStep = 32;          // tokens of a step (two tiles)
constexpr int kAttStages = 2;
constexpr int kAttMaxCtas = kStepTickets;
constexpr int kAttJoin = 8;           // parts of an item whose loads are in flight together
// A scale below 2^-14 of its offset stands as that, so that offset / scale stays in range: a
// constant group's codes are 8, and otherwise the value is off by less than 2^-11 of itself.
constexpr float kScaleOfOffset = 6.1035156e-5f;
constexpr float kTinyScale = 9.0949470e-13f;   // 2^-40
// A new reference puts the largest weight at 2^kRefUp; weights above kMoveAbove, f16's largest
// value, make one.  A reference higher up leaves fewer bits to f16's end, and rows take a new
// one more often (2^10 in the chunk kernel: 149 us for 136).
constexpr float kRefUp = 6.f, kMoveAbove = 65504.f;
constexpr float kNoRef = -3e38f;               // M before the first token
// Units of an item beside its steps: what finding it, its first copies and its merge cost.
// 64 requests of 17 to 8191 tokens: 79 / 72 / 68 / 65 / 65 / 70 us at 3 / 6 / 8 / 14 / 18 / 32
// (two 131k contexts do not care: 67 / 68 / 66 / 65 / 65 / 65).
constexpr int kAttItemCost = 16;
constexpr int kAttMinUnits = 8;       // a CTA's range is at least this
// An item of at most this many steps is one warp's: 256 requests of 50 to 300 tokens 40 us at
// 8 and 36 at 12, 48 requests of 33 to 4095 tokens and up to 5 rows 26 at 8 and 29 at 12.
constexpr int kAttSolo = 10;

struct AttendParams {
    KvView v;
    const __nv_bfloat16* q;
    __nv_bfloat16* out;
    float* lse;
    int64_t ldq, ldo;
    int32_t q_heads, rep;
    float scale;
    uint32_t* tickets;      // [kStepTickets], zero between calls
    float* part;            // [kAttMaxCtas][2][8 NT][D + 4]
};

__host__ __device__ constexpr size_t attend_smem(int dim, int group) {
    return (size_t)kAttWarps * kAttStages * 2 * kv_tile_bytes(dim, group);
}
// CTAs of an SM that the registers are shared out for: four of 128 a thread, fewer where the
// step holds more (one query head per KV head with groups of 32: 96 us with four, 89.5 with
// three).
__host__ __device__ constexpr int attend_ctas(int dim, int group, int nt) {
    return nt == 1 ? (dim == 128 && group == 32 ? 3 : 4) : dim == 128 ? 2 : 3;
}
// Bytes of workspace: header, tickets and partial results.
__host__ __device__ constexpr size_t attend_part_floats(int nt, int dim) { return (size_t)2 * 8 * nt * (dim + 4); }
__host__ __device__ constexpr size_t attend_workspace(int nt, int dim) {
    return kStepPartAt + kAttMaxCtas * attend_part_floats(nt, dim) * 4;
}

// One request as the schedule sees it.
struct AttSeq {
    int32_t row0, rows;     // rows 0: no work
    int32_t len;            // cached tokens, limited to the block table
};

__device__ __forceinline__ AttSeq att_seq(const KvView& v, int s, bool report) {
    const int a = v.q_start[s], b = v.q_start[s + 1];
    const int len = kv_length(v, s);
    AttSeq q = {a, b - a, 0};
    uint32_t err = 0;
    if (b < a || a < 0 || b > v.T) err = LORA_DERR_SEGMENT;
    else if (b - a > v.max_q) err = LORA_DERR_KV;
    if (err) q.rows = 0;
    const int64_t cap = (int64_t)v.max_blocks * v.block_tokens;
    if (q.rows > 0 && len > cap) err = LORA_DERR_KV;
    if (q.rows < v.rows_lo || q.rows > v.rows_hi) q.rows = 0;
    q.len = len;
    if (report && err) set_error(v.err, err);
    return q;
}

// Steps (of Step tokens) of the tile of packed rows [r0, r0 + width) of a request: enough for
// the last row.
template <int Step>
__device__ __forceinline__ int att_steps(const KvView& v, const AttSeq& q, int rep, int r0, int width) {
    const int i = (min(r0 + width, q.rows * rep) - 1) / rep;
    const int64_t tokens = min((int64_t)q.len - q.rows + i + 1, (int64_t)v.max_blocks * v.block_tokens);
    return tokens <= 0 ? 1 : (int)((tokens + Step - 1) / Step);
}

// Units of one KV head of a request: its items' steps and fixed parts.
template <int Step, int Width, int Cost>
__device__ __forceinline__ int64_t att_head_units(const KvView& v, const AttSeq& q, int rep) {
    int64_t n = 0;
    for (int r0 = 0; r0 < q.rows * rep; r0 += Width) n += att_steps<Step>(v, q, rep, r0, Width) + Cost;
    return n;
}

// The deal, by all threads of a CTA: the units before each request by a scan over the
// requests, and of them this CTA's range [first, end) of `per` units; false if it is empty.
// found: request and KV head that hold the first unit, and the units before that head.
template <int Threads, int Step, int Width, int Cost, int MinUnits>
__device__ __forceinline__ bool att_deal(const KvView& v, int rep, int64_t* scan, int64_t* found, int64_t& per, int64_t& first,
                                         int64_t& end) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int chunk = (v.n_seq + Threads - 1) / Threads;
    const int s_lo = min(tid * chunk, v.n_seq), s_hi = min(s_lo + chunk, v.n_seq);
    int64_t mine = 0;
    for (int s = s_lo; s < s_hi; ++s) mine += v.heads * att_head_units<Step, Width, Cost>(v, att_seq(v, s, blockIdx.x == 0), rep);
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t n = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += n;
    }
    if (lane == 31) scan[warp + 1] = incl;
    __syncthreads();
    int64_t before = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < Threads / 32; ++w) {
        if (w < warp) before += scan[w + 1];
        total += scan[w + 1];
    }
    per = max((total + gridDim.x - 1) / gridDim.x, (int64_t)MinUnits);
    first = per * blockIdx.x;
    end = min(first + per, total);
    if (first >= end) return false;
    if (before <= first && first < before + mine) {   // this thread's requests hold the first unit
        int s = s_lo;
        int64_t n;
        for (;; ++s) {
            n = att_head_units<Step, Width, Cost>(v, att_seq(v, s, false), rep);
            if (first < before + v.heads * n) break;
            before += v.heads * n;
        }
        int head = 0;
        while (first >= before + n) {
            before += n;
            ++head;
        }
        found[0] = (int64_t)s << 32 | head;
        found[1] = before;
    }
    __syncthreads();
    return true;
}

// Two values of at most 2^100 rounded to 11 bits at any size: with t = (2^13 + 1) x,
// t - (t - x) is x without its last 13 bits (Veltkamp's splitting).
__device__ __forceinline__ void round11(float a, float b, float& ra, float& rb) {
    const uint64_t x = pack2f(a, b), less = pack2f(-1.f, -1.f), t = mul2(x, pack2f(8193.f, 8193.f));
    unpack2f(fma2(fma2(x, less, t), less, t), ra, rb);
}

__device__ __forceinline__ void att_store(const AttendParams& p, int row, int hq, int D, int d, float4 x, float sum) {
    const float f = sum != 0.f ? __fdividef(1.f, sum) : 0.f;     // no token: zeros
    uint2 w = make_uint2(pack2(x.x * f, x.y * f), pack2(x.z * f, x.w * f));
    *reinterpret_cast<uint2*>(p.out + row * p.ldo + (int64_t)hq * D + d) = w;
}
// A factor of scores, kept in the normal range.
__device__ __forceinline__ float att_normal(float x) { return fminf(fmaxf(x, 1.1754944e-38f), 3.4028235e38f); }

// (scale, offset) of tokens g and g + 8 of a tile and group, at shared address `at` of the first.
__device__ __forceinline__ void att_params(float2 (&k)[2], uint32_t at) {
    uint32_t a, b;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(a) : "r"(at));
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(b) : "r"(at + 32));
    k[0] = __half22float2(*reinterpret_cast<__half2*>(&a));
    k[1] = __half22float2(*reinterpret_cast<__half2*>(&b));
}

// ref: the reference M of the sum, in powers of two.
__device__ __forceinline__ void att_store_lse(const AttendParams& p, int row, int hq, float ref, float sum) {
    if (p.lse) p.lse[(int64_t)row * p.q_heads + hq] = sum == 0.f ? -INFINITY : ref * 0.693147181f + logf(sum);
}

template <int D, int G, int NT>
__global__ void __launch_bounds__(kAttThreads, attend_ctas(D, G, NT)) kv_attend_kernel(const __grid_constant__ AttendParams p) {
    constexpr int kRows = 8 * NT, kChunks = D / 32, kGroups = D / G, kPerG = G / 32;
    constexpr int kTile = kv_tile_bytes(D, G), kStage = 2 * kTile, kPitch = D + 4;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ __align__(8) uint64_t bars[kAttWarps][kAttStages];
    __shared__ int64_t scan[kAttWarps + 1];
    __shared__ int64_t found[2];
    __shared__ float stat[kAttWarps][kRows][2];
    __shared__ float2 vscale[kAttWarps][32 * kGroups];
    __shared__ uint32_t last_in;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const KvView& v = p.v;
    if (tid < kAttWarps * kAttStages) mbar_init(smem_addr(&bars[0][0]) + tid * 8, 1);
    fence_mbar_init();

    int64_t per, first, end;
    if (!att_deal<kAttThreads, kAttStep, kRows, kAttItemCost, kAttMinUnits>(v, p.rep, scan, found, per, first, end)) return;
    int seq = (int)(found[0] >> 32), head = (int)found[0], r0 = 0;
    int64_t item = found[1];                            // first unit of the item
    AttSeq q = att_seq(v, seq, false);
    const uint32_t wring = smem_addr(ring) + warp * kAttStages * kStage;
    const uint32_t wbar = smem_addr(&bars[warp][0]), vparams = smem_addr(&vscale[warp][0]);
    const int cap = (int)((int64_t)v.max_blocks * v.block_tokens);
    uint32_t it = 0;                                    // steps this warp has consumed
    uint32_t solos = 0;
    bool ok = true;

    while (item < end) {
        // ---- the item (seq, head, r0) and this CTA's steps of it
        const int steps = att_steps<kAttStep>(v, q, p.rep, r0, kRows);
        const int64_t body = item + kAttItemCost;
        const int cur_seq = seq, cur_head = head, cur_r0 = r0;
        const AttSeq cq = q;
        const int st0 = (int)max(first - body, (int64_t)0), st1 = (int)min(max(end - body, (int64_t)0), (int64_t)steps);
        const int width = min(kRows, cq.rows * p.rep - cur_r0);
        // the item after it
        item = body + steps;
        r0 += kRows;
        if (r0 >= q.rows * p.rep) {
            r0 = 0;
            if (++head == v.heads) {
                head = 0;
                do q = att_seq(v, min(++seq, v.n_seq - 1), false);
                while (seq < v.n_seq && q.rows == 0);
            }
        }
        if (st1 <= st0) continue;
        const bool whole = st0 == 0 && st1 == steps;
        const bool solo = whole && steps <= kAttSolo;
        if (solo && (int)(solos++ % kAttWarps) != warp) continue;
        const int way = solo ? 1 : kAttWarps, me = solo ? 0 : warp;
        const int lead = cq.len - cq.rows;              // row i's token is lead + i
        const int tokens = min(lead + (cur_r0 + width - 1) / p.rep + 1, cap);
        const int low = lead + cur_r0 / p.rep;          // the first row's token: steps before see no mask

        // ---- this warp's steps st0 + me + way i.  Lane j looks up the two tiles of the
        // warp's step i0 + j, for 32 steps at a time.
        const int mine_n = ok && st1 - st0 > me ? (st1 - st0 - me + way - 1) / way : 0;
        const unsigned char* tile_a = nullptr;
        const unsigned char* tile_b = nullptr;
        uint32_t now_a = 0, now_b = 0;                  // which of the 32 steps' tiles are there
        auto lookup = [&](int i) {
            const int tok = (st0 + me + way * (i + lane)) * kAttStep;
            tile_a = i + lane < mine_n && tok < tokens ? kv_tile_of(v, cur_seq, tok, cur_head, kTile) : nullptr;
            tile_b = i + lane < mine_n && tok + kKvTile < tokens ? kv_tile_of(v, cur_seq, tok + kKvTile, cur_head, kTile) : nullptr;
            now_a = __ballot_sync(0xffffffffu, tile_a != nullptr);
            now_b = __ballot_sync(0xffffffffu, tile_b != nullptr);
        };
        uint32_t have_a = 0, have_b = 0;                // tiles of the steps in the ring, bit step % 32
        auto put = [&](int i, uint32_t stage) {         // copies of step i into `stage`
            const int j = i & 31;
            if (j == 0) lookup(i);
            const uint32_t bit = 1u << j;
            have_a = (have_a & ~bit) | (now_a & bit);
            have_b = (have_b & ~bit) | (now_b & bit);
            if (lane == j) {
                mbar_arrive_expect_tx(wbar + stage * 8, (tile_a ? kTile : 0) + (tile_b ? kTile : 0));
                if (tile_a) bulk_g2s(wring + stage * kStage, tile_a, kTile, wbar + stage * 8);
                if (tile_b) bulk_g2s(wring + stage * kStage + kTile, tile_b, kTile, wbar + stage * 8);
            }
        };
        // q's loads are under way while the tiles are looked up
        uint4 qw[NT][kChunks];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = cur_r0 + n * 8 + g;
            const bool live = n * 8 + g < width;
            const __nv_bfloat16* src = p.q + (int64_t)(cq.row0 + (live ? r / p.rep : 0)) * p.ldq +
                                       (int64_t)(cur_head * p.rep + (live ? r % p.rep : 0)) * D;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) qw[n][c] = live ? ld16(src + c * 32 + t * 8) : make_uint4(0, 0, 0, 0);
        }
        for (int i = 0; i < min(kAttStages, mine_n); ++i) put(i, (it + i) % kAttStages);

        // ---- q as the right-hand operand, and its sums per group, both times 2^13 over the
        // power of two of the row's largest value; `sl` takes that out again
        uint32_t qb[NT][kChunks][4];
        float qsum[NT][kGroups][2], sl[NT][2];
        int32_t last[NT][2];                            // last token of this lane's columns
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            uint32_t big = 0;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const uint32_t x[4] = {qw[n][c].x, qw[n][c].y, qw[n][c].z, qw[n][c].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) big = max(big, max(x[j] << 16 & 0x7F800000u, x[j] & 0x7F800000u));
            }
            big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
            // 2^(13 - e) and its inverse, the exponent e kept where both are normal
            const int e = max(16, min((int)(big >> 23), 254)) - 127;
            const float up = __uint_as_float((uint32_t)(13 - e + 127) << 23);
            // (kept normal: -inf of a masked score times 0, or 0 times inf, would not be a number)
            const float back = att_normal(p.scale * 1.44269504f * __uint_as_float((uint32_t)(e - 13 + 127) << 23));
            sl[n][0] = __shfl_sync(0xffffffffu, back, t * 8);
            sl[n][1] = __shfl_sync(0xffffffffu, back, t * 8 + 4);
#pragma unroll
            for (int gr = 0; gr < kGroups; ++gr) {
                float sum = 0.f;
#pragma unroll
                for (int c = gr * kPerG; c < (gr + 1) * kPerG; ++c) {
                    float f[8];
                    unpack8(qw[n][c], f);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        f[j] *= up;
                        sum += f[j];
                    }
                    qb[n][c][0] = pack_f16(f[0], f[4]);
                    qb[n][c][1] = pack_f16(f[1], f[5]);
                    qb[n][c][2] = pack_f16(f[2], f[6]);
                    qb[n][c][3] = pack_f16(f[3], f[7]);
                }
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                qsum[n][gr][0] = __shfl_sync(0xffffffffu, sum, t * 8);
                qsum[n][gr][1] = __shfl_sync(0xffffffffu, sum, t * 8 + 4);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int col = n * 8 + 2 * t + j;
                last[n][j] = col < width ? min(lead + (cur_r0 + col) / p.rep, cap - 1) : -1;
            }
        }

        float o[NT][2 * kChunks][4];
        float m[NT][2], l[NT][2], off[NT][kGroups][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < 2 * kChunks; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                m[n][j] = kNoRef;
                l[n][j] = 0.f;
#pragma unroll
                for (int gr = 0; gr < kGroups; ++gr) off[n][gr][j] = 0.f;
            }
        }

        for (int i = 0; i < mine_n; ++i, ++it) {
            const uint32_t stage = it % kAttStages;
            if (!__all_sync(0xffffffffu, mbar_wait(wbar + stage * 8, (it / kAttStages) & 1, kWaitLimitNs))) {
                // (the warp as one) let the copies in flight land; the rest of the range does no work
                ok = false;
                for (int k = 1; k < kAttStages; ++k)
                    mbar_wait(wbar + ((it + k) % kAttStages) * 8, ((it + k) / kAttStages) & 1, 100000000ull);
                if (lane == 0) set_error(v.err, LORA_DERR_TIMEOUT);
                break;
            }
            const int tok0 = (st0 + me + way * i) * kAttStep;
            const bool has_a = have_a >> (i & 31) & 1, has_b = have_b >> (i & 31) & 1;
            const uint32_t base = wring + stage * kStage;
            auto step = [&](auto some_masked) {
            constexpr bool masked = decltype(some_masked)::value;
            // ---- S^T = K q^T, both tiles side by side
            float s[2][NT][4];
#pragma unroll
            for (int gr = 0; gr < kGroups; ++gr) {
                float acc[2][NT][4];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int n = 0; n < NT; ++n) acc[h][n][0] = acc[h][n][1] = acc[h][n][2] = acc[h][n][3] = 0.f;
#pragma unroll
                for (int c = gr * kPerG; c < (gr + 1) * kPerG; ++c) {
                    // the two tiles' words: lanes 0-15 address tile 0's rows, 16-31 tile 1's
                    uint32_t w[4];
                    ldmatrix4(w, base + (lane >> 4) * kTile + c * 256 + (lane & 15) * 16);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t a[4], b[4];
                        codes_f16(w[2 * h], a);
                        codes_f16(w[2 * h + 1], b);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma16816_f16(acc[h][n], a[0], b[0], a[1], b[1], qb[n][c][0], qb[n][c][1]);
                            mma16816_f16(acc[h][n], a[2], b[2], a[3], b[3], qb[n][c][2], qb[n][c][3]);
                        }
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float2 k[2];
                    att_params(k, base + h * kTile + kv_params_at(D, G, 0) + gr * 64 + g * 4);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float a = fmaf(k[j >> 1].x, acc[h][n][j], k[j >> 1].y * qsum[n][gr][j & 1]);
                            s[h][n][j] = gr ? s[h][n][j] + a : a;
                        }
                }
            }
            if (masked) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int tok = tok0 + h * kKvTile + g + (j >> 1) * 8;
                            if (tok > last[n][j & 1] || !(h ? has_b : has_a)) s[h][n][j] = -INFINITY;
                        }
            }
            // ---- V's scales, and offsets in units of them: worked out once per token and group,
            // (32 of them or 128 by the lanes), and read back by the lanes that need them
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                const int e = i * 32 + lane, h = e / (16 * kGroups), at = e % (16 * kGroups);
                uint32_t w;
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(base + h * kTile + kv_params_at(D, G, 1) + at * 4));
                float2 q = __half22float2(*reinterpret_cast<__half2*>(&w));
                q.x = fmaxf(fmaxf(q.x, fabsf(q.y) * kScaleOfOffset), kTinyScale);
                q.y *= rcp_approx(q.x);
                asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(vparams + e * 8), "f"(q.x), "f"(q.y) : "memory");
            }
            __syncwarp();
            float2 vp[2][kGroups][2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int gr = 0; gr < kGroups; ++gr)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                                     : "=f"(vp[h][gr][e].x), "=f"(vp[h][gr][e].y)
                                     : "r"(vparams + ((h * kGroups + gr) * 16 + e * 8 + g) * 8));
            // ---- probabilities, and with each group's scale the right-hand operand of V
            uint32_t pb[2][NT][kGroups][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float pr[2][4];
                auto weigh = [&]() {
                    float top = 0.f;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            pr[h][j] = exp2_approx(fmaf(s[h][n][j], sl[n][j & 1], -m[n][j & 1]));
#pragma unroll
                            for (int gr = 0; gr < kGroups; ++gr) {
                                float x = pr[h][j] * vp[h][gr][j >> 1].x;
                                if (masked && pr[h][j] == 0.f) x = 0.f;      // a masked token's parameters may be anything
                                top = fmaxf(top, x);
                            }
                        }
                    return top;
                };
                if (__any_sync(0xffffffffu, weigh() > kMoveAbove)) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float mn = m[n][j];
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float sc = vp[h][0][e].x;
#pragma unroll
                                for (int gr = 1; gr < kGroups; ++gr) sc = fmaxf(sc, vp[h][gr][e].x);
                                const float a = s[h][n][2 * e + j];
                                if (!masked || a != -INFINITY) mn = fmaxf(mn, fmaf(a, sl[n][j], log2_approx(sc) - kRefUp));
                            }
                        mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 4));
                        mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 8));
                        mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 16));
                        const float f = exp2_approx(m[n][j] - mn);
                        m[n][j] = mn;
                        l[n][j] *= f;
#pragma unroll
                        for (int gr = 0; gr < kGroups; ++gr) off[n][gr][j] *= f;
#pragma unroll
                        for (int k = 0; k < 2 * kChunks; ++k) {
                            o[n][k][j] *= f;
                            o[n][k][2 + j] *= f;
                        }
                    }
                    weigh();
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        l[n][0] += pr[h][2 * e];
                        l[n][1] += pr[h][2 * e + 1];
#pragma unroll
                        for (int gr = 0; gr < kGroups; ++gr) {
                            float x[2];
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                x[j] = pr[h][2 * e + j] * vp[h][gr][e].x;
                                if (masked && pr[h][2 * e + j] == 0.f) x[j] = 0.f;
                            }
                            float2 r;
                            round11(x[0], x[1], r.x, r.y);
                            const uint32_t w = pack_f16(r.x, r.y);
                            // (what a row does not see is left out; a weight of zero times a token
                            // that is not a number is not one either)
                            if (!masked || s[h][n][2 * e] != -INFINITY) off[n][gr][0] = fmaf(r.x, vp[h][gr][e].y, off[n][gr][0]);
                            if (!masked || s[h][n][2 * e + 1] != -INFINITY) off[n][gr][1] = fmaf(r.y, vp[h][gr][e].y, off[n][gr][1]);
                            pb[h][n][gr][e] = movmatrix_trans(w);
                        }
                    }
            }
            // ---- O^T += V^T P^T
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int c = 0; c < kChunks; c += 2) {
                    uint32_t w[4];
                    ldmatrix4_trans(w, base + h * kTile + kv_codes_at(D, 1) + c * 256 + lane * 16);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t a[4], b[4];
                        codes_f16(w[2 * e], a);
                        codes_f16(w[2 * e + 1], b);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const int gr = (c + e) / kPerG;
                            mma16816_f16(o[n][2 * (c + e)], a[0], a[1], b[0], b[1], pb[h][n][gr][0], pb[h][n][gr][1]);
                            mma16816_f16(o[n][2 * (c + e) + 1], a[2], a[3], b[2], b[3], pb[h][n][gr][0], pb[h][n][gr][1]);
                        }
                    }
                }
            };
            // most steps lie before the item's first row's token: nothing to mask
            if (tok0 + kAttStep - 1 > low || !has_a || !has_b) step(std::true_type{});
            else step(std::false_type{});
            __syncwarp();                               // every lane has read the stage
            if (i + kAttStages < mine_n) put(i + kAttStages, stage);
        }

        // ---- the lanes' sums, and the offsets' part of the output
        float* mine_o = reinterpret_cast<float*>(ring + warp * kAttStages * kStage);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float ls = l[n][j];
                ls += __shfl_xor_sync(0xffffffffu, ls, 4);
                ls += __shfl_xor_sync(0xffffffffu, ls, 8);
                ls += __shfl_xor_sync(0xffffffffu, ls, 16);
                const int col = n * 8 + 2 * t + j;
                float of[kGroups];
#pragma unroll
                for (int gr = 0; gr < kGroups; ++gr) {
                    of[gr] = off[n][gr][j];
                    of[gr] += __shfl_xor_sync(0xffffffffu, of[gr], 4);
                    of[gr] += __shfl_xor_sync(0xffffffffu, of[gr], 8);
                    of[gr] += __shfl_xor_sync(0xffffffffu, of[gr], 16);
                }
                const int row = cq.row0 + (cur_r0 + col) / p.rep, hq = cur_head * p.rep + (cur_r0 + col) % p.rep;
                if (g == 0) {
                    if (!solo) {
                        stat[warp][col][0] = m[n][j];
                        stat[warp][col][1] = ls;
                    } else if (col < width) {
                        att_store_lse(p, row, hq, m[n][j], ls);
                    }
                }
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    const float a = of[c / kPerG];
                    const float4 x = make_float4(o[n][2 * c][j] + a, o[n][2 * c][2 + j] + a, o[n][2 * c + 1][j] + a,
                                                 o[n][2 * c + 1][2 + j] + a);
                    if (!solo) *reinterpret_cast<float4*>(mine_o + col * D + c * 32 + 4 * g) = x;
                    else if (col < width) att_store(p, row, hq, D, c * 32 + 4 * g, x, ls);
                }
            }
        if (solo) {
            __syncwarp();
            continue;
        }

        // ---- the four warps' results, through the ring (idle now), four values a thread
        ok = !__syncthreads_or(!ok);
        float* part = p.part + ((int64_t)blockIdx.x * 2 + (body < first ? 0 : 1)) * kRows * kPitch;
        for (int e = tid; e < width * (D / 4); e += kAttThreads) {
            const int r = e / (D / 4), d = e % (D / 4) * 4;
            float top = kNoRef;
#pragma unroll
            for (int w = 0; w < kAttWarps; ++w) top = fmaxf(top, stat[w][r][0]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kAttWarps; ++w) {
                const float f = exp2_approx(stat[w][r][0] - top);
                const float4 x = *reinterpret_cast<const float4*>(ring + w * kAttStages * kStage + (r * D + d) * 4);
                acc.x += f * x.x;
                acc.y += f * x.y;
                acc.z += f * x.z;
                acc.w += f * x.w;
                sum += f * stat[w][r][1];
            }
            if (whole) {
                const int pr = cur_r0 + r, row = cq.row0 + pr / p.rep, hq = cur_head * p.rep + pr % p.rep;
                att_store(p, row, hq, D, d, acc, sum);
                if (d == 0) att_store_lse(p, row, hq, top, sum);
            } else {
                *reinterpret_cast<float4*>(part + r * kPitch + d) = acc;
                if (d == 0) *reinterpret_cast<float2*>(part + r * kPitch + D) = make_float2(top, sum);
            }
        }
        fence_proxy_async_smem();                       // the ring is written by copies next
        if (!whole) {
            const int64_t c0 = body / per, c1 = (body + steps - 1) / per;
            __threadfence();
            __syncthreads();
            if (tid == 0) last_in = atomicAdd(&p.tickets[c0], 1u) == (uint32_t)(c1 - c0);
            __syncthreads();
            if (last_in) {
                __threadfence();
                if (tid == 0) p.tickets[c0] = 0;
                const int n = (int)(c1 - c0) + 1;
                auto src = [&](int i) {                 // the item's part of CTA c0 + i
                    return p.part + ((c0 + i) * 2 + (body < (c0 + i) * per ? 0 : 1)) * (int64_t)(kRows * kPitch);
                };
                for (int e = tid; e < width * (D / 4); e += kAttThreads) {
                    const int r = e / (D / 4), d = e % (D / 4) * 4;
                    float top = kNoRef, sum = 0.f;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int i0 = 0; i0 < n; i0 += kAttJoin) {  // kAttJoin parts' loads in flight
                        float2 ms[kAttJoin];
                        float4 x[kAttJoin];
#pragma unroll
                        for (int i = 0; i < kAttJoin; ++i) {
                            ms[i] = make_float2(kNoRef, 0.f);
                            x[i] = acc;
                            if (i0 + i < n) {
                                const float* from = src(i0 + i) + r * kPitch;
                                ms[i] = __ldcg(reinterpret_cast<const float2*>(from + D));
                                x[i] = __ldcg(reinterpret_cast<const float4*>(from + d));
                            }
                        }
                        float mn = top;
#pragma unroll
                        for (int i = 0; i < kAttJoin; ++i) mn = fmaxf(mn, ms[i].x);
                        const float f0 = exp2_approx(top - mn);
                        acc = make_float4(acc.x * f0, acc.y * f0, acc.z * f0, acc.w * f0);
                        sum *= f0;
                        top = mn;
#pragma unroll
                        for (int i = 0; i < kAttJoin; ++i) {
                            if (i0 + i >= n) continue;
                            const float f = exp2_approx(ms[i].x - mn);
                            acc.x += f * x[i].x;
                            acc.y += f * x[i].y;
                            acc.z += f * x[i].z;
                            acc.w += f * x[i].w;
                            sum += f * ms[i].y;
                        }
                    }
                    const int pr = cur_r0 + r, row = cq.row0 + pr / p.rep, hq = cur_head * p.rep + pr % p.rep;
                    att_store(p, row, hq, D, d, acc, sum);
                    if (d == 0) att_store_lse(p, row, hq, top, sum);
                }
            }
        }
        __syncthreads();
    }
}

}  // namespace lora
