// Causal attention of a batch's rows over the 4-bit cache, for few rows per request (decode
// and the check of a few drafted tokens).
//
// For one request and KV head the query rows that share the head (the request's rows times
// the query heads of the KV head) are the columns of a transposed product: with K and V as
// codes c in -8 .. 7 (exact in bf16), a score is
//     q . k_t = sum over groups of  scale_t (q . c_t) + offset_t sum(q),
// so the MMA runs on the codes as they are, S^T = C_K q^T (tokens x rows, 16 tokens a tile),
// and the scale enters once per token in fp32.  The output is likewise
//     O^T = C_V^T (scale_t p_t)  +  sum_t offset_t p_t,
// scale_t p_t being the one value that is rounded to bf16 (2^-9 of a probability on average
// adds less than the output's own rounding does).  ldmatrix hands each lane its words of
// codes in the operand's order (transposed for V, which pairs the tokens), so a code costs
// 11 / 8 instructions on its way to the tensor core.  The tokens being the long side of both
// products, 8 rows fill an MMA; mma.sync serves because the kernel is bound by the bytes of
// the cache (136 a token and head) and next by the unpacking, not by the MMAs.
//
// Work.  An item is (request, KV head, tile of 8 NT packed rows), of ceil(tokens / 32) steps.
// The steps of all items in a row are dealt to the CTAs in equal contiguous ranges; a CTA's
// four warps take the steps of its part of an item in turn, each with its own bulk-copy ring
// and running maximum and sum, and merge at the part's end.  An item that spans several CTAs
// is put together from partial results in the workspace by the CTA that arrives last, in
// the order of the parts, so the result does not depend on the order of arrival.
#pragma once
#include "kv_layout.cuh"
#include "mma_legacy.cuh"
#include "ptx.cuh"

namespace lora {

constexpr int kAttWarps = 4;
constexpr int kAttThreads = kAttWarps * 32;
constexpr int kAttStep = 32;          // tokens of a step (two tiles)
constexpr int kAttStages = 3;
constexpr int kAttMaxCtas = 1024;
constexpr float kTinyScale = 9.0949470e-13f;   // 2^-40: stands for a scale of 0, below f16's smallest
constexpr int kAttMinSteps = kAttWarps;   // a CTA's range is at least a step per warp

struct AttendParams {
    KvView v;
    const __nv_bfloat16* q;
    __nv_bfloat16* out;
    float* lse;
    int64_t ldq, ldo;
    int32_t q_heads, rep;
    float scale;
    uint32_t* tickets;      // [kAttMaxCtas], zero between calls
    float* part;            // [kAttMaxCtas][2][8 NT][D + 2]
};

__host__ __device__ constexpr size_t attend_smem(int dim, int group) {
    return (size_t)kAttWarps * kAttStages * 2 * kv_tile_bytes(dim, group);
}
// Workspace after the header: tickets and partial results.
__host__ __device__ constexpr size_t attend_part_floats(int nt, int dim) { return (size_t)2 * 8 * nt * (dim + 2); }
__host__ __device__ constexpr size_t attend_workspace(int nt, int dim) {
    return kAttMaxCtas * 4 + kAttMaxCtas * attend_part_floats(nt, dim) * 4;
}

// One request as the schedule sees it.
struct AttSeq {
    int32_t row0, rows;     // rows 0: no work
    int32_t len;            // cached tokens, limited to the block table
};

__device__ __forceinline__ AttSeq att_seq(const KvView& v, int s, bool report) {
    const int a = v.q_start[s], b = v.q_start[s + 1];
    int len = v.kv_len[s];
    AttSeq q = {a, b - a, 0};
    uint32_t err = 0;
    if (b < a || a < 0 || b > v.T) err = LORA_DERR_SEGMENT;
    else if (b - a > v.max_q) err = LORA_DERR_KV;
    if (err) q.rows = 0;
    const int64_t cap = (int64_t)v.max_blocks * v.block_tokens;
    if (q.rows > 0 && len > cap) err = LORA_DERR_KV;
    q.len = len;
    if (report && err) set_error(v.err, err);
    return q;
}

// Steps of the tile of packed rows [r0, r0 + width) of a request: enough for the last row.
__device__ __forceinline__ int att_steps(const KvView& v, const AttSeq& q, int rep, int r0, int width) {
    const int i = (min(r0 + width, q.rows * rep) - 1) / rep;
    const int64_t tokens = min((int64_t)q.len - q.rows + i + 1, (int64_t)v.max_blocks * v.block_tokens);
    return tokens <= 0 ? 1 : (int)((tokens + kAttStep - 1) / kAttStep);
}

// Steps of one KV head of a request.
__device__ __forceinline__ int64_t att_head_steps(const KvView& v, const AttSeq& q, int rep, int width) {
    int64_t n = 0;
    for (int r0 = 0; r0 < q.rows * rep; r0 += width) n += att_steps(v, q, rep, r0, width);
    return n;
}

template <int D, int G, int NT>
__global__ void __launch_bounds__(kAttThreads, NT == 1 ? 4 : 2) kv_attend_kernel(const __grid_constant__ AttendParams p) {
    constexpr int kRows = 8 * NT, kChunks = D / 32, kGroups = D / G, kPerG = G / 32;
    constexpr int kTile = kv_tile_bytes(D, G), kStage = 2 * kTile, kPitch = D + 2;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ __align__(8) uint64_t bars[kAttWarps][kAttStages];
    __shared__ int64_t scan[kAttWarps + 1];
    __shared__ int64_t found[2];
    __shared__ float stat[kAttWarps][kRows][2];
    __shared__ uint32_t last_in;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const KvView& v = p.v;
    if (tid < kAttWarps * kAttStages) mbar_init(smem_addr(&bars[0][0]) + tid * 8, 1);
    fence_mbar_init();

    // ---- the schedule: the steps before each request, by a scan over the requests
    const int chunk = (v.n_seq + kAttThreads - 1) / kAttThreads;
    const int s_lo = min(tid * chunk, v.n_seq), s_hi = min(s_lo + chunk, v.n_seq);
    int64_t mine = 0;
    for (int s = s_lo; s < s_hi; ++s)
        mine += v.heads * att_head_steps(v, att_seq(v, s, blockIdx.x == 0), p.rep, kRows);
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t n = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += n;
    }
    if (lane == 31) scan[warp + 1] = incl;
    if (tid == 0) scan[0] = 0;
    __syncthreads();
    int64_t before = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kAttWarps; ++w) {
        if (w < warp) before += scan[w + 1];
        total += scan[w + 1];
    }
    const int64_t per = max((total + gridDim.x - 1) / gridDim.x, (int64_t)kAttMinSteps);
    const int64_t first = per * blockIdx.x, end = min(first + per, total);
    if (first >= end) return;
    if (before <= first && first < before + mine) {   // this thread's requests hold the first step
        int s = s_lo;
        for (;; ++s) {
            const int64_t n = v.heads * att_head_steps(v, att_seq(v, s, false), p.rep, kRows);
            if (first < before + n) break;
            before += n;
        }
        found[0] = s;
        found[1] = before;
    }
    __syncthreads();
    int seq = (int)found[0];
    int64_t at = found[1];                              // steps before request `seq`
    const float sl = p.scale * 1.44269504f;
    const uint32_t wring = smem_addr(ring) + warp * kAttStages * kStage;
    const uint32_t wbar = smem_addr(&bars[warp][0]);
    uint32_t it = 0;                                    // steps this warp has consumed
    bool ok = true;

    for (int64_t pos = first; pos < end && ok;) {
        // ---- the item at `pos`: request, KV head, row tile
        AttSeq q = att_seq(v, seq, false);
        int64_t per_head = att_head_steps(v, q, p.rep, kRows);
        while (pos >= at + v.heads * per_head) {
            at += v.heads * per_head;
            q = att_seq(v, ++seq, false);
            per_head = att_head_steps(v, q, p.rep, kRows);
        }
        const int head = (int)((pos - at) / per_head);
        int64_t item = at + head * per_head;            // first step of the item
        int r0 = 0, steps = att_steps(v, q, p.rep, 0, kRows);
        while (pos >= item + steps) {
            item += steps;
            r0 += kRows;
            steps = att_steps(v, q, p.rep, r0, kRows);
        }
        const int width = min(kRows, q.rows * p.rep - r0);
        const int st0 = (int)(pos - item), st1 = (int)min((int64_t)steps, end - item);
        const int lead = q.len - q.rows;                // row i's token is lead + i
        const int cap = v.max_blocks * v.block_tokens;
        const int tokens = min(lead + (r0 + width - 1) / p.rep + 1, cap);
        const int low = lead + r0 / p.rep;              // the first row's token: steps before see no mask

        // ---- q as the right-hand operand, and its sums per group
        uint32_t qb[NT][kChunks][4];
        float qsum[NT][kGroups][2];
        int32_t last[NT][2];                            // last token of this lane's columns
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = r0 + n * 8 + g;
            const bool live = n * 8 + g < width;
            const __nv_bfloat16* src = p.q + (int64_t)(q.row0 + (live ? r / p.rep : 0)) * p.ldq +
                                       (int64_t)(head * p.rep + (live ? r % p.rep : 0)) * D;
#pragma unroll
            for (int gr = 0; gr < kGroups; ++gr) {
                float sum = 0.f;
#pragma unroll
                for (int c = gr * kPerG; c < (gr + 1) * kPerG; ++c) {
                    const uint4 w = live ? ld16(src + c * 32 + t * 8) : make_uint4(0, 0, 0, 0);
                    qb[n][c][0] = __byte_perm(w.x, w.z, 0x5410);
                    qb[n][c][1] = __byte_perm(w.x, w.z, 0x7632);
                    qb[n][c][2] = __byte_perm(w.y, w.w, 0x5410);
                    qb[n][c][3] = __byte_perm(w.y, w.w, 0x7632);
                    float f[8];
                    unpack8(w, f);
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum += f[j];
                }
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                qsum[n][gr][0] = __shfl_sync(0xffffffffu, sum, t * 8);
                qsum[n][gr][1] = __shfl_sync(0xffffffffu, sum, t * 8 + 4);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int col = n * 8 + 2 * t + j;
                last[n][j] = col < width ? min(lead + (r0 + col) / p.rep, cap - 1) : -1;
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
                m[n][j] = -INFINITY;
                l[n][j] = 0.f;
#pragma unroll
                for (int gr = 0; gr < kGroups; ++gr) off[n][gr][j] = 0.f;
            }
        }

        // ---- this warp's steps st0 + warp + 4 i.  Lane j looks up the two tiles of the
        // warp's step i0 + j, for 32 steps at a time.
        const int mine_n = st1 - st0 > warp ? (st1 - st0 - warp + kAttWarps - 1) / kAttWarps : 0;
        const unsigned char* tile_a = nullptr;
        const unsigned char* tile_b = nullptr;
        auto lookup = [&](int i) {
            const int tok = (st0 + warp + kAttWarps * (i + lane)) * kAttStep;
            tile_a = i + lane < mine_n && tok < tokens ? kv_tile_of(v, seq, tok, head, kTile) : nullptr;
            tile_b = i + lane < mine_n && tok + kKvTile < tokens ? kv_tile_of(v, seq, tok + kKvTile, head, kTile) : nullptr;
        };
        int i_look = 0;
        uint32_t have_a = 0, have_b = 0;                // tiles present, one bit per looked-up step
        auto issue = [&](int i, uint32_t stage) {       // copies of step i into `stage`
            const int j = i - i_look;
            const unsigned char* a = reinterpret_cast<const unsigned char*>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(tile_a), j));
            const unsigned char* b = reinterpret_cast<const unsigned char*>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(tile_b), j));
            if (lane == 0) {
                mbar_arrive_expect_tx(wbar + stage * 8, (a ? kTile : 0) + (b ? kTile : 0));
                if (a) bulk_g2s(wring + stage * kStage, a, kTile, wbar + stage * 8);
                if (b) bulk_g2s(wring + stage * kStage + kTile, b, kTile, wbar + stage * 8);
            }
        };
        // presence bits follow the issue: bit (step % 32) is set when the step is issued
        auto put = [&](int i, uint32_t stage) {
            if (i - i_look >= 32) {
                i_look += 32;
                lookup(i_look);
            }
            const int j = i - i_look;
            const uint32_t ba = __ballot_sync(0xffffffffu, tile_a != nullptr), bb = __ballot_sync(0xffffffffu, tile_b != nullptr);
            const uint32_t bit = 1u << (i & 31);
            have_a = (ba >> j & 1) ? have_a | bit : have_a & ~bit;
            have_b = (bb >> j & 1) ? have_b | bit : have_b & ~bit;
            issue(i, stage);
        };
        lookup(0);
        for (int i = 0; i < min(kAttStages, mine_n); ++i) put(i, (it + i) % kAttStages);

        for (int i = 0; i < mine_n; ++i, ++it) {
            const uint32_t stage = it % kAttStages;
            if (!mbar_wait(wbar + stage * 8, (it / kAttStages) & 1, kWaitLimitNs)) {
                ok = false;
                break;
            }
            const int tok0 = (st0 + warp + kAttWarps * i) * kAttStep;
            const bool has_a = have_a >> (i & 31) & 1, has_b = have_b >> (i & 31) & 1;
            const bool masked = tok0 + kAttStep - 1 > low || !has_a || !has_b;
            const uint32_t base = wring + stage * kStage;
            // ---- S^T = K q^T
            float s[2][NT][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t tb = base + h * kTile;
#pragma unroll
                for (int gr = 0; gr < kGroups; ++gr) {
                    float acc[NT][4];
#pragma unroll
                    for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll
                    for (int c = gr * kPerG; c < (gr + 1) * kPerG; ++c) {
                        uint32_t w[2];
                        asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];"
                                     : "=r"(w[0]), "=r"(w[1])
                                     : "r"(tb + c * 256 + (lane & 15) * 16)
                                     : "memory");
                        const uint32_t a0[4] = {code_pair<0>(w[0], kMinus8), code_pair<0>(w[1], kMinus8),
                                                code_pair<1>(w[0], kMinus8), code_pair<1>(w[1], kMinus8)};
                        const uint32_t a1[4] = {code_pair<2>(w[0], kMinus8), code_pair<2>(w[1], kMinus8),
                                                code_pair<3>(w[0], kMinus8), code_pair<3>(w[1], kMinus8)};
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma16816(acc[n], a0, qb[n][c][0], qb[n][c][1]);
                            mma16816(acc[n], a1, qb[n][c][2], qb[n][c][3]);
                        }
                    }
                    const uint32_t pa = tb + kv_params_at(D, G, 0) + gr * 64 + g * 4;
                    uint32_t r0w, r1w;
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r0w) : "r"(pa));
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r1w) : "r"(pa + 32));
                    const float2 k0 = __half22float2(*reinterpret_cast<__half2*>(&r0w));
                    const float2 k1 = __half22float2(*reinterpret_cast<__half2*>(&r1w));
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float a = fmaf(k0.x, acc[n][j], k0.y * qsum[n][gr][j]);
                            const float b = fmaf(k1.x, acc[n][2 + j], k1.y * qsum[n][gr][j]);
                            s[h][n][j] = gr ? s[h][n][j] + a : a;
                            s[h][n][2 + j] = gr ? s[h][n][2 + j] + b : b;
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
            // ---- running maximum, probabilities, sums
            uint32_t pb[2][NT][kGroups][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float mn[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float x = fmaxf(fmaxf(s[0][n][j], s[0][n][2 + j]), fmaxf(s[1][n][j], s[1][n][2 + j]));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                    mn[j] = fmaxf(m[n][j], x);
                }
                if (__any_sync(0xffffffffu, mn[0] != m[n][0] || mn[1] != m[n][1])) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float f = mn[j] == -INFINITY ? 1.f : exp2_approx((m[n][j] - mn[j]) * sl);
                        m[n][j] = mn[j];
                        l[n][j] *= f;
#pragma unroll
                        for (int gr = 0; gr < kGroups; ++gr) off[n][gr][j] *= f;
#pragma unroll
                        for (int k = 0; k < 2 * kChunks; ++k) {
                            o[n][k][j] *= f;
                            o[n][k][2 + j] *= f;
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float ms = m[n][j & 1] == -INFINITY ? 0.f : m[n][j & 1] * sl;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        s[h][n][j] = exp2_approx(fmaf(s[h][n][j], sl, -ms));
                        l[n][j & 1] += s[h][n][j];
                    }
                }
            }
            // ---- V's scale and offset enter the probabilities of each group
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int gr = 0; gr < kGroups; ++gr) {
                    const uint32_t pa = base + h * kTile + kv_params_at(D, G, 1) + gr * 64 + g * 4;
                    uint32_t r0w, r1w;
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r0w) : "r"(pa));
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r1w) : "r"(pa + 32));
                    float2 vp[2] = {__half22float2(*reinterpret_cast<__half2*>(&r0w)),
                                    __half22float2(*reinterpret_cast<__half2*>(&r1w))};
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        vp[e].x = fmaxf(vp[e].x, kTinyScale);
                        vp[e].y = __fdividef(vp[e].y, vp[e].x);     // offset in units of the scale
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float x[2];
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                x[j] = s[h][n][2 * e + j] * vp[e].x;
                                if (masked && s[h][n][2 * e + j] == 0.f) x[j] = 0.f;   // its parameters may be anything
                            }
                            const uint32_t w = pack2(x[0], x[1]);
                            const float of[2] = {bf16lo(w), bf16hi(w)};
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                if (!masked || of[j] != 0.f) off[n][gr][j] = fmaf(of[j], vp[e].y, off[n][gr][j]);
                            pb[h][n][gr][e] = movmatrix_trans(w);
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
                        const uint32_t w0 = w[2 * e], w1 = w[2 * e + 1];
                        const uint32_t a0[4] = {code_pair<0>(w0, kMinus8), code_pair<1>(w0, kMinus8),
                                                code_pair<0>(w1, kMinus8), code_pair<1>(w1, kMinus8)};
                        const uint32_t a1[4] = {code_pair<2>(w0, kMinus8), code_pair<3>(w0, kMinus8),
                                                code_pair<2>(w1, kMinus8), code_pair<3>(w1, kMinus8)};
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const int gr = (c + e) / kPerG;
                            mma16816(o[n][2 * (c + e)], a0, pb[h][n][gr][0], pb[h][n][gr][1]);
                            mma16816(o[n][2 * (c + e) + 1], a1, pb[h][n][gr][0], pb[h][n][gr][1]);
                        }
                    }
                }
            __syncwarp();                               // every lane has read the stage
            if (i + kAttStages < mine_n) put(i + kAttStages, stage);
        }

        // ---- the four warps' results, through the ring (idle now)
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
                if (g == 0) {
                    stat[warp][col][0] = m[n][j];
                    stat[warp][col][1] = ls;
                }
                float of[kGroups];
#pragma unroll
                for (int gr = 0; gr < kGroups; ++gr) {
                    of[gr] = off[n][gr][j];
                    of[gr] += __shfl_xor_sync(0xffffffffu, of[gr], 4);
                    of[gr] += __shfl_xor_sync(0xffffffffu, of[gr], 8);
                    of[gr] += __shfl_xor_sync(0xffffffffu, of[gr], 16);
                }
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    const float a = of[c / kPerG];
                    *reinterpret_cast<float4*>(mine_o + col * D + c * 32 + 4 * g) =
                        make_float4(o[n][2 * c][j] + a, o[n][2 * c][2 + j] + a, o[n][2 * c + 1][j] + a,
                                    o[n][2 * c + 1][2 + j] + a);
                }
            }
        if (!ok) {                                      // let the copies in flight land
            for (int i = 1; i < kAttStages; ++i)
                mbar_wait(wbar + ((it + i) % kAttStages) * 8, ((it + i) / kAttStages) & 1, 100000000ull);
            if (lane == 0) set_error(v.err, LORA_DERR_TIMEOUT);
        }
        ok = !__syncthreads_or(!ok);
        const bool whole = st0 == 0 && st1 == steps;
        const int64_t c0 = item / per, c1 = (item + steps - 1) / per;
        const int slot = pos == first ? 0 : 1;
        float* part = p.part + ((int64_t)blockIdx.x * 2 + slot) * kRows * kPitch;
        for (int e = tid; e < width * D; e += kAttThreads) {
            const int r = e / D, d = e % D;
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kAttWarps; ++w) top = fmaxf(top, stat[w][r][0]);
            float acc = 0.f, sum = 0.f;
#pragma unroll
            for (int w = 0; w < kAttWarps; ++w) {
                const float f = top == -INFINITY ? 0.f : exp2_approx((stat[w][r][0] - top) * sl);
                acc += f * reinterpret_cast<const float*>(ring + w * kAttStages * kStage)[e];
                sum += f * stat[w][r][1];
            }
            if (whole) {
                const int pr = r0 + r, row = q.row0 + pr / p.rep, hq = head * p.rep + pr % p.rep;
                p.out[row * p.ldo + (int64_t)hq * D + d] = __float2bfloat16_rn(sum > 0.f || sum != sum ? acc / sum : 0.f);
                if (d == 0 && p.lse) p.lse[(int64_t)row * p.q_heads + hq] = top == -INFINITY ? -INFINITY : top * p.scale + logf(sum);
            } else {
                part[r * kPitch + d] = acc;
                if (d == 0) {
                    part[r * kPitch + D] = top;
                    part[r * kPitch + D + 1] = sum;
                }
            }
        }
        fence_proxy_async_smem();                       // the ring is written by copies next
        if (!whole) {
            __threadfence();
            __syncthreads();
            if (tid == 0) last_in = atomicAdd(&p.tickets[c0], 1u) == (uint32_t)(c1 - c0);
            __syncthreads();
            if (last_in) {
                __threadfence();
                if (tid == 0) p.tickets[c0] = 0;
                for (int e = tid; e < width * D; e += kAttThreads) {
                    const int r = e / D, d = e % D;
                    float top = -INFINITY, acc = 0.f, sum = 0.f;
                    for (int64_t c = c0; c <= c1; ++c) {
                        // a CTA's first part lies in its slot 0
                        const float* src = p.part + (c * 2 + (item > c * per ? 1 : 0)) * kRows * kPitch + r * kPitch;
                        const float mt = __ldcg(src + D), ls = __ldcg(src + D + 1), x = __ldcg(src + d);
                        const float mn = fmaxf(top, mt);
                        const float fa = mn == -INFINITY ? 1.f : exp2_approx((top - mn) * sl);
                        const float fb = mn == -INFINITY ? 0.f : exp2_approx((mt - mn) * sl);
                        acc = acc * fa + x * fb;
                        sum = sum * fa + ls * fb;
                        top = mn;
                    }
                    const int pr = r0 + r, row = q.row0 + pr / p.rep, hq = head * p.rep + pr % p.rep;
                    p.out[row * p.ldo + (int64_t)hq * D + d] = __float2bfloat16_rn(sum > 0.f || sum != sum ? acc / sum : 0.f);
                    if (d == 0 && p.lse) p.lse[(int64_t)row * p.q_heads + hq] = top == -INFINITY ? -INFINITY : top * p.scale + logf(sum);
                }
            }
        }
        __syncthreads();
        pos = item + st1;
    }
}

}  // namespace lora
