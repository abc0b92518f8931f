// Causal attention over the 4-bit cache for many rows per request (chunks of prompts), on the
// fifth-generation tensor cores; one scale per head vector (group = head_dim).
//
// A tile is 128 packed rows (rows times query heads of one KV head) of one request; a block is
// 128 tokens.  As in kv_attend.cuh the products run on the codes: with q in bf16 and c in
// -8 .. 7,
//     S = q C_K^T (128 x 128, tensor memory),   t = S k_t + kq_t sum(q) - M,   p = 2^t,
// where k_t and kq_t are the token's K scale and offset times softmax_scale log2 e; then
//     O += X W,   X = f16(p u_t),   W = f16((c - 8) V scale / u_t + V offset / u_t) = f16(v / u_t),
// with u_t a power of two near the token's largest |v|: X is as large as what the token brings,
// however its offset compares with its scale, and W, one FMA that rounds once (scale and offset
// over u_t are exact in f16 above 2^-14), is off by 2^-11 of itself.  X takes the place of S in
// tensor memory.  The output is O / sum p.  The reference M puts the largest p u_t at 2^6, so
// that f16 loses 2^-31 of it a token at most; it is moved, and O multiplied, only when a p u_t
// exceeds f16's range.
//
// Warps 0-7 hold half of a row a thread (64 of a block's tokens, half of the output): they
// bring q, turn S into X and write the output.  Warps 8-15 unpack a block's codes into the
// operands' swizzled rows (within eight values in the order 0 4 1 5 2 6 3 7, q alike, and the
// output put back).  Warp 16 issues the MMAs, S of the next block before X W of this one; warp
// 17 brings the codes.  Tiles are dealt, split and joined as kv_attend.cuh's items.
//
// A block costs 1024 clocks of MMA and as many of exponentials, but takes about 2900: a row
// warp is 2000 of them on its 64 tokens, with the unpacking warps (2,750 of the block's some
// 7,000 instructions, the rows 3,600) beside it on its scheduler.  Three requests of 300 to 512
// rows over 3111 to 6000 tokens (32 query and 8 KV heads of 128) take 137 us for 89 GFLOP, 34%
// of the measured bf16 rate.
#pragma once
#include "kv_attend.cuh"

namespace lora {

constexpr int kPreRows = 128, kPreStep = 128, kPreThreads = 18 * 32;
// Blocks' worth of a tile's fixed part: three requests' chunks 139.6 / 139.2 / 136.9 / 136.5 / 137.8
// us at 2 / 3 / 4 / 6 / 8, 16 requests of 12 rows 64.0 / 63.1 / 62.9 / 61.5 / 61.5, of 48 rows
// 108.2 / 106.3 / 106.5 / 107.3 / 108.1.
constexpr int kPreItemCost = 6;
constexpr int kPreMinUnits = 8;
constexpr int kPreMaxCtas = 192;
// A request's packed rows per KV head from which this kernel serves it: where the few-row kernel
// takes a third tile of 16 of them (heads of 128) or a fourth (64).  16 requests over 4000
// tokens, 8 KV heads, us there and here: heads of 128, 32 rows 57 and 61, 40 rows 77 and 61, 64
// rows 97 and 61; heads of 64, 48 rows 52 and 56, 64 rows 65 and 56.  Few requests reach the
// same point later (heads of 128, 4 requests: 32 rows 26 and 31, 40 rows 31 and 31; one: 40 rows
// 22 and 30, 128 rows 27 and 32, 192 rows 33 and 32), hence not before a fourth tile there.
__host__ __device__ constexpr int pre_min_packed(int dim, int64_t seq_heads) { return dim == 128 && seq_heads >= 32 ? 33 : 49; }

constexpr int kPreTable = 3 * kPreStep * 4 + 16;
__host__ __device__ constexpr int pre_code_bytes(int dim) { return kPreStep / kKvTile * kv_tile_bytes(dim, dim); }
struct PreSmem {
    int q, k, v, codes, table, mask, pair, total;
};
__host__ __device__ constexpr PreSmem pre_smem(int dim) {
    PreSmem L{};
    int o = 0;
    L.q = o;      o += kPreRows * dim * 2;
    L.k = o;      o += 2 * kPreStep * dim * 2;
    L.v = o;      o += 2 * kPreStep * dim * 2;
    L.codes = o;  o += 2 * pre_code_bytes(dim);
    L.table = o;  o += 4 * kPreTable;                // k, kq, u of a block's tokens, and its tiles that are there
    L.mask = o;   o += 16;
    L.pair = o;   o += 2 * kPreRows * 4 + 64;        // what a row's two threads exchange; flags [4 pairs][4]
    L.total = o + 1024;
    return L;
}
__host__ __device__ constexpr size_t pre_workspace(int dim) {
    return kStepPartAt + (size_t)kPreMaxCtas * 2 * kPreRows * (dim + 2) * 4;
}

// kind::f16 with f16 operands: idesc_bf16 without its two type bits.
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t m, uint32_t n, uint32_t a_mn, uint32_t b_mn) {
    return idesc_bf16(m, n, a_mn, b_mn) & ~((1u << 7) | (1u << 10));
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ float lds32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ ulonglong2 lds2x64(uint32_t addr) {
    ulonglong2 v;
    asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(v.x), "=l"(v.y) : "r"(addr));
    return v;
}

// Walks the parts of tiles in a CTA's range, the same for every role.
struct PrePart {
    AttSeq q;
    int seq, head, r0, width, st0, st1, steps;
    int64_t body;
    __device__ __forceinline__ bool whole() const { return st0 == 0 && st1 == steps; }
};
struct PreWalk {
    int64_t item, first, end;
    int seq, head, r0;
    AttSeq q;
    // the next part; false at the end of the range
    __device__ __forceinline__ bool next(const KvView& v, int rep, PrePart& c) {
        while (item < end) {
            c.q = q;
            c.seq = seq;
            c.head = head;
            c.r0 = r0;
            c.steps = att_steps<kPreStep>(v, q, rep, r0, kPreRows);
            c.width = min(kPreRows, q.rows * rep - r0);
            c.body = item + kPreItemCost;
            c.st0 = (int)max(first - c.body, (int64_t)0);
            c.st1 = (int)min(max(end - c.body, (int64_t)0), (int64_t)c.steps);
            item = c.body + c.steps;
            r0 += kPreRows;
            if (r0 >= q.rows * rep) {
                r0 = 0;
                if (++head == v.heads) {
                    head = 0;
                    do q = att_seq(v, min(++seq, v.n_seq - 1), false);
                    while (seq < v.n_seq && q.rows == 0);
                }
            }
            if (c.st1 > c.st0) return true;
        }
        return false;
    }
};

template <int D>
__global__ void __launch_bounds__(kPreThreads, 1) kv_prefill_kernel(const __grid_constant__ AttendParams p) {
    constexpr int kTile = kv_tile_bytes(D, D), kHalves = D / 64;
    constexpr PreSmem L = pre_smem(D);
    // tensor memory: S three times (X of tokens 0-63 in a buffer's columns 0-31, of 64-127 in
    // 64-95), so that S of the next block need not wait for X W of the block before; O
    constexpr uint32_t kSCol = 0, kOCol = 384;
    extern __shared__ unsigned char raw[];
    __shared__ __align__(8) uint64_t code_full[2], code_empty[2], k_full[2], v_full[2], v_empty[2], s_full[2],
        x_full[2], q_full, o_empty, final_bar;
    __shared__ int64_t scan[kPreThreads / 32 + 1], found[2];
    __shared__ uint32_t tmem_slot, last_in;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const KvView& v = p.v;
    unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sm = smem_addr(base);
    auto bar = [](uint64_t& b) { return smem_addr(&b); };

    PreWalk walk;
    int64_t per;
    if (!att_deal<kPreThreads, kPreStep, kPreRows, kPreItemCost, kPreMinUnits>(v, p.rep, scan, found, per, walk.first, walk.end)) return;
    walk.seq = (int)(found[0] >> 32);
    walk.head = (int)found[0];
    walk.r0 = 0;
    walk.item = found[1];
    walk.q = att_seq(v, walk.seq, false);

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(code_full[i]), 1);
            mbar_init(bar(code_empty[i]), 8);
            mbar_init(bar(k_full[i]), 8);
            mbar_init(bar(v_full[i]), 8);
            mbar_init(bar(v_empty[i]), 1);
            mbar_init(bar(s_full[i]), 1);
            mbar_init(bar(x_full[i]), 8);
        }
        mbar_init(bar(q_full), 8);
        mbar_init(bar(o_empty), 8);
        mbar_init(bar(final_bar), 1);
        fence_mbar_init();
    }
    if (tid < 4) sts128(sm + L.pair + 2 * kPreRows * 4 + tid * 16, 0, 0, 0, 0);
    if (warp == 16) {
        tmem_alloc(smem_addr(&tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&tmem_slot);
    bool ok = true;
    PrePart c;
    uint32_t n = 0;              // blocks so far: n % 2 is the buffer, n / 2 the phase

    // Registers: 576 threads start with 96; the unpacking warps give 40 each of theirs to the
    // rows' (256 x 136 + 256 x 56 + 64 x 96 = 576 x 96).
    if (warp < 8) {
        // ------------------------------------------------------------------ rows
        asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
        const int quad = warp & 3, half = warp >> 2, r = quad * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t flags = sm + L.pair + 2 * kPreRows * 4 + quad * 16;
        // These warps meet at named barriers, so none of them leaves early: after a wait that ran
        // out, `wait` returns at once and the rest of the range goes by (with the error set).
        auto wait = [&](uint64_t& which, uint32_t parity) {
            if (ok && !__all_sync(0xffffffffu, mbar_wait(bar(which), parity, kWaitLimitNs))) {
                ok = false;
                if (lane == 0) set_error(v.err, LORA_DERR_TIMEOUT);
            }
        };
        auto meet = [&]() { named_bar_sync(1, 256); };
        auto meet_pair = [&]() { named_bar_sync(2 + quad, 64); };    // the two warps of the same rows
        // the other thread's value for the row (the second meeting keeps the buffer whole)
        auto exchange = [&](float x) {
            float* buf = reinterpret_cast<float*>(base + L.pair);
            buf[half * kPreRows + r] = x;
            meet_pair();
            const float y = *reinterpret_cast<volatile float*>(&buf[(half ^ 1) * kPreRows + r]);
            meet_pair();
            return y;
        };
        const int cap = (int)((int64_t)v.max_blocks * v.block_tokens);
        while (walk.next(v, p.rep, c)) {
            // ---- q into its swizzled rows (every S of the part before is done), and its sum
            const int pr = c.r0 + r, row = c.q.row0 + pr / p.rep, hq = c.head * p.rep + pr % p.rep;
            const bool live = r < c.width;
            const int lead = c.q.len - c.q.rows, low = lead + c.r0 / p.rep;
            // (a row past the tile's end goes along with the last one)
            const int last = min(lead + min(pr, c.r0 + c.width - 1) / p.rep, cap - 1);
            float qs = 0.f;
            const __nv_bfloat16* src = p.q + (int64_t)row * p.ldq + (int64_t)hq * D;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const int i = half * (D / 16) + k;
                const uint4 w = live ? ld16(src + i * 8) : make_uint4(0, 0, 0, 0);
                float f[8];
                unpack8(w, f);
#pragma unroll
                for (int j = 0; j < 8; ++j) qs += f[j];
                sts128(sm + L.q + (i / 8) * (kPreRows * 128) + r * 128 + ((i % 8 ^ (r & 7)) << 4), __byte_perm(w.x, w.z, 0x5410),
                       __byte_perm(w.x, w.z, 0x7632), __byte_perm(w.y, w.w, 0x5410), __byte_perm(w.y, w.w, 0x7632));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(q_full));
            const float qo = exchange(qs);
            qs = half ? qo + qs : qs + qo;              // the same sum for both
            float m = kNoRef, l = 0.f;
            for (int st = c.st0; st < c.st1; ++st, ++n) {
                const uint32_t b = n & 1, sb = lanes + kSCol + n % 3 * 128 + half * 64;
                const uint32_t table = sm + L.table + (n & 3) * kPreTable + half * 256;
                const int tok0 = st * kPreStep + half * 64;
                wait(s_full[b], (n >> 1) & 1);
                tc_fence_after();
                uint32_t present;
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(present) : "r"(table - half * 256 + 3 * kPreStep * 4));
                const uint32_t here = present >> (half * 4);        // this half's four tiles
                // the reference 2^kRefUp below the row's largest p u_t of this block, if that is larger; with
                // 1 for the u of a token whose V is not a number, so that its p stays in range
                auto move = [&]() {
                    float mn = m;
#pragma unroll 1
                    for (int j0 = 0; j0 < 64; j0 += 16) {
                        float t[16];
                        tmem_ld16(sb + j0, t);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float k = lds32(table + (j0 + j) * 4), kq = lds32(table + (kPreStep + j0 + j) * 4);
                            const float u = lds32(table + (2 * kPreStep + j0 + j) * 4);
                            const float x = fmaf(k, t[j], kq * qs) + ((u == u ? log2_approx(u) : 0.f) - kRefUp);
                            if (tok0 + j0 + j <= last && (here >> (j0 / 16) & 1)) mn = fmaxf(mn, x);
                        }
                    }
                    mn = fmaxf(mn, exchange(mn));
                    const float f = exp2_approx(m - mn);
                    m = mn;
                    l *= f;
                    return f;
                };
                // X of the half, and the sum of its p; false where X does not fit the reference
                float sum = 0.f;
                uint32_t x[32];
                auto weigh = [&](auto some_masked) {
                    constexpr bool masked = decltype(some_masked)::value;
                    const uint64_t qs2 = pack2f(qs, qs), ref2 = pack2f(-m, -m);
                    float top = 0.f;
                    uint64_t sum2 = 0;
                    float t[2][16];
                    tmem_ld16(sb, t[0]);
#pragma unroll
                    for (int j0 = 0; j0 < 64; j0 += 16) {
                        tmem_ld_wait();
                        if (j0 < 48) tmem_ld16(sb + j0 + 16, t[j0 / 16 + 1 & 1]);
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            const ulonglong2 k = lds2x64(table + (j0 + j) * 4), kq = lds2x64(table + (kPreStep + j0 + j) * 4),
                                             sc = lds2x64(table + (2 * kPreStep + j0 + j) * 4);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const float* s = t[j0 / 16 & 1] + j + 2 * h;
                                const uint64_t e = fma2(h ? k.y : k.x, pack2f(s[0], s[1]), fma2(h ? kq.y : kq.x, qs2, ref2));
                                float e0, e1, x0, x1;
                                unpack2f(e, e0, e1);
                                const int tok = tok0 + j0 + j + 2 * h;
                                const bool in = here >> (j0 / 16) & 1;
                                const bool hide0 = masked && (tok > last || !in), hide1 = masked && (tok + 1 > last || !in);
                                if (hide0) e0 = -INFINITY;
                                if (hide1) e1 = -INFINITY;
                                e0 = exp2_approx(e0);
                                e1 = exp2_approx(e1);
                                const uint64_t pr = pack2f(e0, e1);
                                sum2 = add2(sum2, pr);
                                unpack2f(mul2(pr, h ? sc.y : sc.x), x0, x1);
                                if (hide0) x0 = 0.f;           // a hidden token's u may be anything
                                if (hide1) x1 = 0.f;
                                // (a weight that is not a number stays in the maximum)
                                asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(x0), "f"(x1));
                                x[(j0 + j + 2 * h) / 2] = pack_f16(x0, x1);
                            }
                        }
                    }
                    float s0, s1;
                    unpack2f(sum2, s0, s1);
                    sum = s0 + s1;
                    return (bool)__all_sync(0xffffffffu, top <= kMoveAbove);
                };
                // causal, or with tiles absent: the same for every row of the tile
                const bool masked = st * kPreStep + kPreStep - 1 > low || present != 0xFFu;
                const bool first = st == c.st0;
                if (first) move();
                // whether either warp of the rows has an X that does not fit (a flag a block, four in turn)
                const bool fits = masked ? weigh(std::true_type{}) : weigh(std::false_type{});
                if (!fits && lane == 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(flags + (n & 3) * 4), "r"(1u) : "memory");
                if (lane == 0 && half == 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(flags + ((n + 2) & 3) * 4), "r"(0u) : "memory");
                meet_pair();
                uint32_t again;
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(again) : "r"(flags + (n & 3) * 4));
                if (again) {
                    // a new reference: O (of the blocks before) follows, and X once more
                    const float f = move();
                    if (!first) wait(v_empty[b ^ 1], ((n - 1) >> 1) & 1);
                    tc_fence_after();
#pragma unroll 1
                    for (int j0 = half * (D / 2); j0 < (first ? 0 : (half + 1) * (D / 2)); j0 += 16) {
                        float o[16];
                        uint32_t w[16];
                        tmem_ld16(lanes + kOCol + j0, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(o[j] * f);
                        tmem_st16(lanes + kOCol + j0, w);
                    }
                    weigh(std::true_type{});
                }
                l += sum;
                tmem_st32(sb, x);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                // (two in turn: rows that need no new reference are a block ahead of others by then)
                if (lane == 0) mbar_arrive(bar(x_full[b]));
            }
            const float lo = exchange(l);
            l = half ? lo + l : l + lo;
            // ---- the part's sums
            wait(v_empty[(n - 1) & 1], ((n - 1) >> 1) & 1);
            tc_fence_after();
            const bool whole = c.whole();
            // 32 values of the row (eight by eight in the operands' order) to the output
            auto store = [&](int j0, const float (&o)[32], float f) {
                __nv_bfloat16* dst = p.out + (int64_t)row * p.ldo + (int64_t)hq * D + j0;
#pragma unroll
                for (int i = 0; i < 32; i += 8)
                    if (live)
                        st16(dst + i, make_uint4(pack2(o[i] * f, o[i + 2] * f), pack2(o[i + 4] * f, o[i + 6] * f),
                                                 pack2(o[i + 1] * f, o[i + 3] * f), pack2(o[i + 5] * f, o[i + 7] * f)));
            };
            const int slot = c.body < walk.first ? 0 : 1;
            float* part = p.part + ((int64_t)blockIdx.x * 2 + slot) * kPreRows * (D + 2) + r;
            const float inv = l != 0.f ? 1.f / l : 0.f;
            for (int j0 = half * (D / 2); j0 < (half + 1) * (D / 2); j0 += 32) {
                float o[32];
                tmem_ld32(lanes + kOCol + j0, o);
                tmem_ld_wait();
                if (whole) {
                    store(j0, o, inv);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) part[(j0 + j) * kPreRows] = o[j];
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(o_empty));
            if (whole) {
                if (live && half == 0) att_store_lse(p, row, hq, m, l);
                continue;
            }
            if (half == 0) {
                part[D * kPreRows] = m;
                part[(D + 1) * kPreRows] = l;
            }
            const int64_t c0 = c.body / per, c1 = (c.body + c.steps - 1) / per;
            __threadfence();
            meet();
            if (tid == 0) last_in = atomicAdd(&p.tickets[c0], 1u) == (uint32_t)(c1 - c0);
            meet();
            if (*reinterpret_cast<volatile uint32_t*>(&last_in)) {
                __threadfence();
                if (tid == 0) p.tickets[c0] = 0;
                auto from = [&](int64_t i) {
                    return p.part + (i * 2 + (c.body < i * per ? 0 : 1)) * kPreRows * (D + 2) + r;
                };
                m = kNoRef;
                for (int64_t i = c0; i <= c1; ++i) m = fmaxf(m, __ldcg(from(i) + D * kPreRows));
                l = 0.f;
                for (int64_t i = c0; i <= c1; ++i)
                    l += __ldcg(from(i) + (D + 1) * kPreRows) * exp2_approx(__ldcg(from(i) + D * kPreRows) - m);
                const float f = l != 0.f ? 1.f / l : 0.f;
                for (int j0 = half * (D / 2); j0 < (half + 1) * (D / 2); j0 += 32) {
                    float o[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = 0.f;
                    for (int64_t i = c0; i <= c1; ++i) {
                        const float* s = from(i) + j0 * kPreRows;
                        const float w = exp2_approx(__ldcg(from(i) + D * kPreRows) - m);
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = fmaf(w, __ldcg(s + j * kPreRows), o[j]);
                    }
                    store(j0, o, f);
                }
                if (live && half == 0) att_store_lse(p, row, hq, m, l);
            }
            meet();
        }
    } else if (warp < 16) {
        // ------------------------------------------------------------------ unpacking: a token, half of its values
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        const int tok = tid & 127, half = (tid - 256) >> 7;
        auto wait = [&](uint64_t& which, uint32_t parity) {
            return (bool)__all_sync(0xffffffffu, mbar_wait(bar(which), parity, kWaitLimitNs));
        };
        const float sl = att_normal(p.scale * 1.44269504f);
        while (ok && walk.next(v, p.rep, c)) {
            for (int st = c.st0; st < c.st1; ++st, ++n) {
                const uint32_t b = n & 1, ph = (n >> 1) & 1;
                if (!wait(code_full[b], ph)) { ok = false; break; }
                const uint32_t src = sm + L.codes + b * pre_code_bytes(D) + (tok / kKvTile) * kTile;
                const uint32_t at = src + (tok % kKvTile) * 16;
                // the buffer's last S is done (and with it the rows' use of the table four blocks ago)
                if (!wait(s_full[b], ph ^ 1)) { ok = false; break; }
                // K: 16-byte pieces of 32 values; a row of 64 values is 128 bytes, swizzled
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {
                    const int chunk = half * (D / 64) + i;
                    const uint4 w4 = lds128(at + chunk * 256);
                    const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
                    const uint32_t dst = sm + L.k + b * (kPreStep * D * 2) + (chunk / 2) * (kPreStep * 128) + tok * 128;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        sts128(dst + (((chunk % 2 * 4 + j) ^ (tok & 7)) << 4), code_pair<0>(w[j], kMinus8), code_pair<1>(w[j], kMinus8),
                               code_pair<2>(w[j], kMinus8), code_pair<3>(w[j], kMinus8));
                }
                uint32_t present;
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(present) : "r"(sm + L.mask + b * 4));
                const bool here = present >> (tok / kKvTile) & 1;
                uint32_t vw;
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(vw) : "r"(src + kv_params_at(D, D, 1) + tok % kKvTile * 4));
                const float2 vs = __half22float2(*reinterpret_cast<__half2*>(&vw));
                // u: the power of two at or below the larger of 8 scale and |offset|, and over it the two
                // (zeros for a token that is not there, and for one that is not a number, whose u says so)
                const bool number = fabsf(vs.x) + fabsf(vs.y) < 1e6f;
                const uint32_t ub = __float_as_uint(fmaxf(fmaxf(8.f * fabsf(vs.x), fabsf(vs.y)), kTinyScale)) & 0x7F800000u;
                const float over = here && number ? __uint_as_float(0x7F000000u - ub) : 0.f;
                const __half2 sc2 = __half2half2(__float2half_rn(over != 0.f ? vs.x * over : 0.f)),
                              of2 = __half2half2(__float2half_rn(over != 0.f ? vs.y * over : 0.f));
                if (half == 0) {
                    // the token's parameters; of a token that is not there nothing is used
                    uint32_t kw;
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(kw) : "r"(src + kv_params_at(D, D, 0) + tok % kKvTile * 4));
                    const float2 ks = __half22float2(*reinterpret_cast<__half2*>(&kw));
                    float* table = reinterpret_cast<float*>(base + L.table + (n & 3) * kPreTable);
                    // (kept finite, if a number: times a score of 0 it has to give 0)
                    auto finite = [](float x) { return fabsf(x) > 3.4028235e38f ? copysignf(3.4028235e38f, x) : x; };
                    table[tok] = here ? finite(ks.x * sl) : 0.f;
                    table[kPreStep + tok] = here ? finite(ks.y * sl) : 0.f;
                    table[2 * kPreStep + tok] = !here ? 0.f : number ? __uint_as_float(ub) : NAN;
                    if (tok == 0) reinterpret_cast<uint32_t*>(table)[3 * kPreStep] = present;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(k_full[b]));
                if (!wait(v_empty[b], ph ^ 1)) { ok = false; break; }
                // W: rows of tokens, [token / 8][64 values][token % 8]
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {
                    const int chunk = half * (D / 64) + i;
                    const uint4 w4 = lds128(at + kv_codes_at(D, 1) + chunk * 256);
                    const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
                    const uint32_t dst = sm + L.v + b * (kPreStep * D * 2) + (tok / 8) * (kHalves * 1024) + (chunk / 2) * 1024 + tok % 8 * 128;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t o[4];
                        codes_f16(w[j], o);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const __half2 x = __hfma2(*reinterpret_cast<__half2*>(&o[k]), sc2, of2);
                            o[k] = *reinterpret_cast<const uint32_t*>(&x);
                        }
                        sts128(dst + (((chunk % 2 * 4 + j) ^ (tok & 7)) << 4), o[0], o[1], o[2], o[3]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(v_full[b]));
                    mbar_arrive(bar(code_empty[b]));
                }
            }
        }
    } else if (warp == 16) {
        // ------------------------------------------------------------------ MMA issue: the warp in step, one lane issues
        constexpr uint32_t id_s = idesc_bf16(128, kPreStep, 0, 0), id_o = idesc_f16(128, D, 0, 1);
        uint32_t parts = 0;
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), sb = __shfl_sync(0xffffffffu, sm, 0);
        const uint64_t q_desc = smem_desc(sb + L.q, 16, 1024, 2), k_desc = smem_desc(sb + L.k, 16, 1024, 2),
                       w_desc = smem_desc(sb + L.v, 1024, kHalves * 1024, 2);
        auto wait = [&](uint64_t& which, uint32_t parity) {
            return (bool)__all_sync(0xffffffffu, mbar_wait_quiet(bar(which), parity, kWaitLimitNs));
        };
        // S of block i, in the place of X of block i - 3.  K of block i comes after V of i - 1,
        // and that after X W of i - 3: one wait stands for all of them.
        auto scores = [&](uint32_t i) {
            const uint32_t b = i & 1, d = tm + kSCol + i % 3 * 128;
            const uint64_t kb = desc_at(k_desc, b * (kPreStep * D * 2));
            if (!wait(k_full[b], (i >> 1) & 1)) return false;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    tc_mma_f16(d, desc_at(q_desc, (k / 4) * (kPreRows * 128) + (k % 4) * 32),
                               desc_at(kb, (k / 4) * (kPreStep * 128) + (k % 4) * 32), id_s, k != 0);
                tc_commit(bar(s_full[b]));
            }
            __syncwarp();
            return true;
        };
        while (ok && walk.next(v, p.rep, c)) {
            const int st0 = __shfl_sync(0xffffffffu, c.st0, 0), st1 = __shfl_sync(0xffffffffu, c.st1, 0);
            if (!wait(q_full, parts & 1) || !scores(n)) { ok = false; break; }
            for (int st = st0; st < st1; ++st, ++n) {
                const uint32_t b = n & 1, ph = (n >> 1) & 1, x = tm + kSCol + n % 3 * 128;
                const uint64_t wb = desc_at(w_desc, b * (kPreStep * D * 2));
                // (K of the next block came after V of this one)
                if (!(st + 1 < st1 ? scores(n + 1) : wait(v_full[b], ph))) { ok = false; break; }
                if (!wait(x_full[b], ph)) { ok = false; break; }
                // the part before has been read out of O
                if (st == st0 && !wait(o_empty, (parts & 1) ^ 1)) { ok = false; break; }
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kPreStep / 16; ++k)
                        tc_mma_f16_ts(tm + kOCol, x + (k / 4) * 64 + k % 4 * 8, desc_at(wb, k * (kHalves * 2048)), id_o,
                                      k != 0 || st != st0);
                    tc_commit(bar(v_empty[b]));
                }
                __syncwarp();
            }
            ++parts;
        }
        if (elect_one()) tc_commit(bar(final_bar));     // the MMAs are done before tensor memory is given back
        __syncwarp();
        mbar_wait_quiet(bar(final_bar), 0, 100000000ull);
        __syncwarp();
    } else {
        // ------------------------------------------------------------------ codes: eight tiles a block, a lane each
        while (ok && walk.next(v, p.rep, c)) {
            const int lead = c.q.len - c.q.rows;
            const int tokens = (int)min((int64_t)lead + (c.r0 + c.width - 1) / p.rep + 1, (int64_t)v.max_blocks * v.block_tokens);
            for (int st = c.st0; st < c.st1; ++st, ++n) {
                const uint32_t b = n & 1;
                const int t = st * kPreStep + lane * kKvTile;
                const unsigned char* tile = lane < 8 && t < tokens ? kv_tile_of(v, c.seq, t, c.head, kTile) : nullptr;
                const uint32_t present = __ballot_sync(0xffffffffu, tile != nullptr);
                if (!__all_sync(0xffffffffu, mbar_wait_quiet(bar(code_empty[b]), ((n >> 1) & 1) ^ 1, kWaitLimitNs))) { ok = false; break; }
                if (lane == 0) {
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(sm + L.mask + b * 4), "r"(present) : "memory");
                    mbar_arrive_expect_tx(bar(code_full[b]), __popc(present) * kTile);
                }
                __syncwarp();
                if (tile) bulk_g2s(sm + L.codes + b * pre_code_bytes(D) + lane * kTile, tile, kTile, bar(code_full[b]));
            }
        }
        for (uint32_t k = n > 2 ? n - 2 : 0; k < n; ++k) mbar_wait_quiet(bar(code_full[k & 1]), (k >> 1) & 1, 100000000ull);
    }
    if (!ok && lane == 0) set_error(v.err, LORA_DERR_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 16) tmem_dealloc(tmem, 512);
}

}  // namespace lora
