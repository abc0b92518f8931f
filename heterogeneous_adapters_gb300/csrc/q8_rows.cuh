// Rows into 8 bits: the residual's addition with the root-mean-square norm, and the gated
// activation (include/lora_w8.h).
//
// A row's codes need its largest magnitude, so a CTA holds one row in registers between its
// only read and its only write, with one exchange between the warps.  A CTA takes row after row,
// with the next row's loads on their way while it works on one.
//
// Memory bounds it: 8,191 rows of 4096 with the addition take 49.2 us (6.1 TB/s, 92% of a copy), 2,339
// gated rows of 14336 38.9 (6.0 TB/s), at 72 and 63% of the issue slots; wider norms, which have no registers for
// the next row, 72 to 86% of a copy.  One row takes 2.3: the launch
// and a chain of a load, two exchanges between warps and a store.
#pragma once
#include "lora_w8.h"
#include "mma_legacy.cuh"
#include "step.cuh"

namespace lora {

struct Q8Out {
    unsigned char* codes;
    float* scales;
    __nv_bfloat16* x;
    int64_t ldc, ldx;
    int32_t full;                  // LORA_Q8_X_FULL
};

struct Q8NormParams {
    const __nv_bfloat16* x;
    const __nv_bfloat16* residual;
    __nv_bfloat16* sum;
    const __nv_bfloat16* weight;
    int64_t ldx, ldr, lds;
    float eps, by_d;               // by_d = 1 / d
    int32_t d, T;
    Q8Out out;
};

struct Q8GateParams {
    const __nv_bfloat16* gate;
    const __nv_bfloat16* up;
    int64_t ldg, ldu;
    int32_t d, T;
    Q8Out out;
};

// Between these magnitudes of a row's largest value the quotients below are right; a row outside
// is multiplied by a power of two first.
constexpr float kQ8Small = 0x1p-96f, kQ8Large = 0x1p100f, kQ8Up = 0x1p64f, kQ8Down = 0x1p-80f;

// A word of two bf16 as a pair of fp32.
__device__ __forceinline__ uint64_t pair_of(uint32_t w) { return pack2f(bf16lo(w), bf16hi(w)); }
// The sum of two pairs, held in bf16: the norm is that of what is held.
__device__ __forceinline__ uint32_t add_pairs(uint32_t a, uint32_t b) {
    float lo, hi;
    unpack2f(add2(pair_of(a), pair_of(b)), lo, hi);
    return pack2(lo, hi);
}
// The larger of m and a pair's magnitudes (a NaN is passed over: the sums that go with the maxima show it).
__device__ __forceinline__ float max_pair(uint64_t v, float m) {
    float a, b;
    unpack2f(v, a, b);
    return fmaxf(m, fmaxf(fabsf(a), fabsf(b)));
}

// The block's largest `top` (not negative) and its sum of `ss`, for every thread.
__device__ __forceinline__ void q8_reduce(float& top, float& ss, uint32_t* red_top, float* red_ss) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (lane == 0) {
        red_top[warp] = bits;
        red_ss[warp] = ss;
    }
    __syncthreads();
    bits = lane < warps ? red_top[lane] : 0u;
    ss = lane < warps ? red_ss[lane] : 0.f;
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, bits));
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
}

// What a row's values p become: codes rint(127 p / top), and for the adapters bf16(scale code) or
// bf16(p over).
struct Q8Row {
    float top, inv, scale, over;
};

// Writes eight values from column `at` of a row.  1.5 * 2^23 + v rounds v to a whole number, ties to
// even, and shows it in the low byte.  v = p inv is within 2^-15 of the quotient, so where it lies
// further from a half the rounding is right; next to one, 127 p - c top (exact where p has 16
// bits, as a product of two bf16 does) decides.
__device__ __forceinline__ void q8_store(const Q8Out& o, int64_t row, int at, const uint64_t (&p)[4], const Q8Row& r) {
    constexpr float kMagic = 12582912.0f;
    const uint64_t inv = pack2f(r.inv, r.inv), magic = pack2f(kMagic, kMagic);
    const float by = o.full ? r.over : r.scale;
    uint32_t two[4], w[4];                                  // two codes' low bytes, two values of x
    auto put = [&](int i, uint64_t t) {                     // t: two codes + kMagic
        float lo, hi;
        unpack2f(t, lo, hi);
        two[i] = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x0040);
        unpack2f(mul2(o.full ? p[i] : add2(t, pack2f(-kMagic, -kMagic)), pack2f(by, by)), lo, hi);
        w[i] = pack2(lo, hi);
    };
    float far = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t t = fma2(p[i], inv, magic);
        far = max_pair(fma2(p[i], inv, add2(magic, mul2(t, pack2f(-1.f, -1.f)))), far);
        put(i, t);
    }
    if (far > 0.4999f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[2], t[2];
            unpack2f(p[i], v[0], v[1]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                t[j] = fmaf(v[j], r.inv, kMagic);
                const float e = fmaf(kMagic - t[j], r.top, 127.0f * v[j]), half = 0.5f * r.top;
                if (fabsf(e) > half || (fabsf(e) == half && (__float_as_uint(t[j]) & 1u))) t[j] += copysignf(1.0f, e);
            }
            put(i, pack2f(t[0], t[1]));
        }
    }
    *reinterpret_cast<uint2*>(o.codes + row * o.ldc + at) = make_uint2(__byte_perm(two[0], two[1], 0x5410), __byte_perm(two[2], two[3], 0x5410));
    if (o.x != nullptr) st16(o.x + row * o.ldx + at, make_uint4(w[0], w[1], w[2], w[3]));
}

// The row's constants from its largest magnitude `top`, where y = p over back.  A row that is not
// finite stands for NaN: codes of zero, which p of zero gives.
template <int V>
__device__ __forceinline__ Q8Row q8_row(uint64_t (&p)[V][4], float top, float over, float back, bool finite) {
    Q8Row r;
    r.top = top;
    r.scale = top * over * (1.f / 127.f) * back;
    r.inv = r.scale != 0.f ? 127.f * rcp_approx(top) : 0.f;
    r.over = over * back;
    if (!finite || !(r.scale < __uint_as_float(0x7F800000u))) {
        r.top = 1.f;
        r.inv = 0.f;
        r.scale = r.over = __uint_as_float(0x7FC00000u);
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) p[j][i] = 0;
    }
    return r;
}

// Rows blockIdx.x, blockIdx.x + gridDim.x, ...; thread i holds the eight values from columns
// 8 (i + j blockDim), j < V.  PRE: the next row is fetched ahead.
template <int V, bool PRE>
__global__ void __launch_bounds__(1024) q8_norm_kernel(const __grid_constant__ Q8NormParams q) {
    __shared__ uint32_t red_top[3][32];
    __shared__ float red_ss[3][32];
    const int tid = threadIdx.x;
    const bool add = q.residual != nullptr;
    uint4 xn[V], rn[V], gw = make_uint4(0, 0, 0, 0);
    auto fetch = [&](int64_t row, int j) {
        const int at = 8 * (tid + j * blockDim.x);
        xn[j] = rn[j] = make_uint4(0, 0, 0, 0);
        if (at < q.d && row < q.T) {
            xn[j] = ld16(q.x + row * q.ldx + at);
            if (add) rn[j] = ld16(q.residual + row * q.ldr + at);
        }
    };
    auto fetch_row = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < V; ++j) fetch(row, j);
    };
    grid_wait();
    if (PRE) fetch_row(blockIdx.x);
    float bad = 0.f;                                        // NaN where a weight is not finite
    // eight weights: kept where there are no more, else from the first-level cache
    auto weights = [&](int j) {
        const int at = 8 * (tid + j * blockDim.x);
        return V == 1 ? gw : at < q.d ? ld16(q.weight + at) : make_uint4(0, 0, 0, 0);
    };
    if (V == 1 && 8 * tid < q.d) gw = ld16(q.weight + 8 * tid);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float g[8];
        unpack8(weights(j), g);
#pragma unroll
        for (int i = 0; i < 8; ++i) bad = fmaf(g[i], 0.f, bad);
    }
    int turn = 0;
    for (int64_t row = blockIdx.x; row < q.T; row += gridDim.x, turn ^= 1) {
        uint64_t p[V][4], squares = pack2f(bad, 0.f);
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int at = 8 * (tid + j * blockDim.x);
            if (!PRE) fetch(row, j);
            const uint4 gj = weights(j);
            uint32_t w[4] = {xn[j].x, xn[j].y, xn[j].z, xn[j].w};
            const uint32_t r[4] = {rn[j].x, rn[j].y, rn[j].z, rn[j].w}, g[4] = {gj.x, gj.y, gj.z, gj.w};
            if (add) {
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = add_pairs(w[i], r[i]);
                if (q.sum && at < q.d) st16(q.sum + row * q.lds + at, make_uint4(w[0], w[1], w[2], w[3]));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint64_t h = pair_of(w[i]);
                p[j][i] = mul2(h, pair_of(g[i]));
                squares = fma2(h, h, squares);
                top = max_pair(p[j][i], top);
            }
        }
        if (PRE) fetch_row(row + gridDim.x);
        float ss, odd;
        unpack2f(squares, ss, odd);
        ss += odd;
        q8_reduce(top, ss, red_top[turn], red_ss[turn]);
        float over = rsqrtf(fmaf(ss, q.by_d, q.eps)), back = 1.f;
        bool large = !(ss < 0x1p125f);
        const bool huge = top > kQ8Large, tiny = top != 0.f && top < kQ8Small && !large;
        if (large || huge || tiny) {
            // squares or products near an end of fp32's range: once more by powers of two, the products' by one for the
            // larger factor and one for the smaller.  Squares that are not large say that h is below 2^63; large ones, that
            // eps is nothing and tiny products are too
            const float by_s = large ? kQ8Down : 1.f, larger = !huge ? 1.f : large ? kQ8Down : 0x1p-96f,
                        smaller = tiny ? kQ8Up : large && huge ? kQ8Down : 1.f;
            back = tiny ? 1.f / kQ8Up : !large ? 0x1p96f : huge ? 1.f / kQ8Down : kQ8Down;
            ss = bad;
            top = 0.f;
            // from h where that is held: x or the residual may have given it their place
            const __nv_bfloat16* from = q.sum ? q.sum + row * q.lds : q.x + row * q.ldx;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int at = 8 * (tid + j * blockDim.x);
                if (at >= q.d) continue;
                const uint4 x = ld16(from + at), gj = weights(j);
                uint32_t w[4] = {x.x, x.y, x.z, x.w};
                const uint32_t g[4] = {gj.x, gj.y, gj.z, gj.w};
                if (add && !q.sum) {
                    const uint4 y = ld16(q.residual + row * q.ldr + at);
                    const uint32_t r[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = add_pairs(w[i], r[i]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float h[2], m[2];
                    unpack2f(pair_of(w[i]), h[0], h[1]);
                    unpack2f(pair_of(g[i]), m[0], m[1]);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        ss = fmaf(h[k] * by_s, h[k] * by_s, ss);
                        const bool low = fabsf(h[k]) <= fabsf(m[k]);
                        h[k] *= low ? smaller : larger;
                        m[k] *= low ? larger : smaller;
                    }
                    p[j][i] = pack2f(h[0] * m[0], h[1] * m[1]);
                    top = max_pair(p[j][i], top);
                }
            }
            q8_reduce(top, ss, red_top[2], red_ss[2]);
            if (large) {
                over = rsqrtf(ss * q.by_d);
                large = !(ss < 0x1p125f);
            }
        }
        const Q8Row r = q8_row(p, top, over, back, !large && top <= kQ8Large);
        if (tid == 0) q.out.scales[row] = r.scale;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int at = 8 * (tid + j * blockDim.x);
            if (at < q.d) q8_store(q.out, row, at, p[j], r);
        }
    }
}

// Of the forms with a quotient, a / (1 + e^-z): -z log2(e), z = a or that of (1 + tanh(z / 2)) / 2.
template <int ACT>
__device__ __forceinline__ uint64_t q8_exponent(uint64_t v) {
    const uint64_t z = mul2(v, pack2f(-1.44269504f, -1.44269504f));
    if (ACT != LORA_ACT_GELU_TANH) return z;
    constexpr float k = 2.f * 0.79788456f;
    return mul2(z, fma2(mul2(v, v), pack2f(k * 0.044715f, k * 0.044715f), pack2f(k, k)));
}

// act of a pair; `most`: the largest e^-z so far.  Every value that is not finite gives one that is not.
template <int ACT>
__device__ __forceinline__ uint64_t q8_act(uint64_t v, float& most) {
    float a[2];
    unpack2f(v, a[0], a[1]);
    if (ACT == LORA_ACT_NONE) {
        return v;
    } else if (ACT == LORA_ACT_GELU) {
        // max(a, 0) - t F(t) e^(-t^2 / 2), t = |a|: with F(t) = e^(t^2 / 2) erfc(t / sqrt 2) / 2 neither side cancels, so
        // that far below zero y keeps its digits (1 + erf there has none).  F is s P(s), s = 1 / (1 + 0.34 t), P of degree
        // 8 fitted over t <= 14 for the least largest relative error, 2^-25; in fp32 it is within 7 * 2^-24.  t^2 is
        // exact.  2,339 gated rows of 14336 take 44.5 us, by erff 55
        const uint64_t t = v & 0x7FFFFFFF7FFFFFFFull;
        float d[2], e[2];
        unpack2f(fma2(t, pack2f(0.34f, 0.34f), pack2f(1.f, 1.f)), d[0], d[1]);
        const uint64_t s = pack2f(rcp_approx(d[0]), rcp_approx(d[1]));
        constexpr float kP[9] = {0.135620505f, 0.136112198f, 0.115197659f, 0.115359172f, -0.0447184853f,
                                 0.202182725f, -0.273132801f, 0.139499515f, -0.0261204802f};
        uint64_t f = pack2f(kP[8], kP[8]);
#pragma unroll
        for (int i = 7; i >= 0; --i) f = fma2(f, s, pack2f(kP[i], kP[i]));
        unpack2f(mul2(mul2(t, t), pack2f(-0.72134752f, -0.72134752f)), e[0], e[1]);
        const uint64_t below = mul2(mul2(mul2(f, s), t), pack2f(exp2_approx(e[0]), exp2_approx(e[1])));
        return fma2(below, pack2f(-1.f, -1.f), pack2f(fmaxf(a[0], 0.f), fmaxf(a[1], 0.f)));
    } else {
        // e^-z is right to 2^-24 (4 + 1.5 |z|) of itself
        float e[2];
        unpack2f(q8_exponent<ACT>(v), e[0], e[1]);
        e[0] = exp2_approx(e[0]);
        e[1] = exp2_approx(e[1]);
        most = fmaxf(most, fmaxf(e[0], e[1]));
        unpack2f(add2(pack2f(e[0], e[1]), pack2f(1.f, 1.f)), e[0], e[1]);
        return mul2(v, pack2f(rcp_approx(e[0]), rcp_approx(e[1])));
    }
}
// Above this e^-z the quotient leaves fp32's normal values before a e^z does (a of -87 and less: up to 2^-119.5): there
// a e^z goes by two halves of the exponent.  Nothing is left below a of -103.
constexpr float kQ8Tail = 0x1p125f;
template <int ACT>
__device__ __forceinline__ uint64_t q8_act_tail(uint64_t v) {
    float most = 0.f, z[2], a[2], y[2];
    unpack2f(q8_exponent<ACT>(v), z[0], z[1]);
    unpack2f(v, a[0], a[1]);
    unpack2f(q8_act<ACT>(v, most), y[0], y[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (z[i] > 125.f) {
            const float h = exp2_approx(-0.5f * z[i]);
            y[i] = a[i] * h * h;
        }
    return pack2f(y[0], y[1]);
}

template <int V, int ACT, bool PRE>
__global__ void __launch_bounds__(1024) q8_gate_kernel(const __grid_constant__ Q8GateParams q) {
    __shared__ uint32_t red_top[2][32];
    __shared__ float red_ss[2][32];
    constexpr bool kQuotient = ACT == LORA_ACT_SILU || ACT == LORA_ACT_GELU_TANH;
    const int tid = threadIdx.x;
    const bool gated = q.up != nullptr;
    uint4 an[V], un[V];
    auto fetch = [&](int64_t row, int j) {
        const int at = 8 * (tid + j * blockDim.x);
        an[j] = un[j] = make_uint4(0, 0, 0, 0);
        if (at < q.d && row < q.T) {
            an[j] = ld16(q.gate + row * q.ldg + at);
            if (gated) un[j] = ld16(q.up + row * q.ldu + at);
        }
    };
    auto fetch_row = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < V; ++j) fetch(row, j);
    };
    grid_wait();
    if (PRE) fetch_row(blockIdx.x);
    int turn = 0;
    for (int64_t row = blockIdx.x; row < q.T; row += gridDim.x, turn ^= 1) {
        uint64_t p[V][4], zeros = 0;                        // zeros: 0 y summed, NaN where a y is not finite
        float top = 0.f, most = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (!PRE) fetch(row, j);
            const uint32_t a[4] = {an[j].x, an[j].y, an[j].z, an[j].w}, u[4] = {un[j].x, un[j].y, un[j].z, un[j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[j][i] = q8_act<ACT>(pair_of(a[i]), most);
                if (gated) p[j][i] = mul2(p[j][i], pair_of(u[i]));
                zeros = fma2(p[j][i], 0, zeros);
                top = max_pair(p[j][i], top);
            }
        }
        if (kQuotient && most > kQ8Tail) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (!PRE) fetch(row, j);                    // nothing of the row is written yet
                const uint32_t a[4] = {an[j].x, an[j].y, an[j].z, an[j].w}, u[4] = {un[j].x, un[j].y, un[j].z, un[j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    p[j][i] = q8_act_tail<ACT>(pair_of(a[i]));
                    if (gated) p[j][i] = mul2(p[j][i], pair_of(u[i]));
                    zeros = fma2(p[j][i], 0, zeros);
                    top = max_pair(p[j][i], top);
                }
            }
        }
        if (PRE) fetch_row(row + gridDim.x);
        float none, odd;
        unpack2f(zeros, none, odd);
        none += odd;
        q8_reduce(top, none, red_top[turn], red_ss[turn]);
        const bool finite = none == 0.f;
        float back = 1.f;
        if (finite && top != 0.f && (top < kQ8Small || top > kQ8Large)) {   // near an end of fp32's range: by a power of two
            const float by = top < 1.f ? kQ8Up : kQ8Down;
            back = 1.f / by;
            top *= by;
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) p[j][i] = mul2(p[j][i], pack2f(by, by));
        }
        const Q8Row r = q8_row(p, top, 1.f, back, finite);
        if (tid == 0) q.out.scales[row] = r.scale;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int at = 8 * (tid + j * blockDim.x);
            if (at < q.d) q8_store(q.out, row, at, p[j], r);
        }
    }
}

}  // namespace lora
