// Rows into 8 bits: the residual's addition with the root-mean-square norm, and the gated
// activation (include/lora_w8.h).
//
// A row's codes need its largest magnitude, so a CTA holds one row in registers between its
// only read and its only write, with one exchange between the warps.  A CTA takes row after row,
// with the next row's loads on their way while it works on one.
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
    float eps;
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

constexpr uint32_t kInfBits = 0x7F800000u;
constexpr float kQ8Up = 18446744073709551616.0f, kQ8Small = 1.0f / kQ8Up;  // 2^64 and 2^-64

// The block's largest `top` (fp32 bits of magnitudes, in their order as integers, a NaN above
// all) and sum of `ss`, for every thread.  A second call needs a barrier in between.
__device__ __forceinline__ void q8_reduce(uint32_t& top, float& ss, uint32_t* red_top, float* red_ss) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    top = __reduce_max_sync(0xffffffffu, top);
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (lane == 0) {
        red_top[warp] = top;
        red_ss[warp] = ss;
    }
    __syncthreads();
    top = lane < warps ? red_top[lane] : 0u;
    ss = lane < warps ? red_ss[lane] : 0.f;
    top = __reduce_max_sync(0xffffffffu, top);
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
}

// Codes of eight values p of a row whose largest magnitude is `top` (> 0, and large enough for
// inv = 127 / top to be finite): rint(127 p / top), ties to even.  1.5 * 2^23 + v rounds v to a
// whole number and shows it in the low byte.  v is within 2^-15 of the quotient, so where it
// lies further from a half the rounding is right; next to one, 127 p - c top (exact where p has
// 16 bits, as a product of two bf16 does) decides.
__device__ __forceinline__ void q8_codes(const float (&p)[8], float top, float inv, float (&c)[8], uint2& packed) {
    constexpr float kMagic = 12582912.0f;
    uint32_t b[8];
    float far = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float t = fmaf(p[i], inv, kMagic);
        c[i] = t - kMagic;
        far = fmaxf(far, fabsf(fmaf(p[i], inv, -c[i])));
        b[i] = __float_as_uint(t);
    }
    if (far > 0.4999f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float e = fmaf(-c[i], top, 127.0f * p[i]), half = 0.5f * top;
            if (fabsf(e) > half || (fabsf(e) == half && (b[i] & 1u))) {
                c[i] += copysignf(1.0f, e);
                b[i] = __float_as_uint(c[i] + kMagic);
            }
        }
    }
    packed.x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    packed.y = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
}

// Writes eight values from column `at` of a row: y = p * over.
__device__ __forceinline__ void q8_store(const Q8Out& o, int64_t row, int at, const float (&p)[8], float top, float inv, float scale,
                                         float over) {
    float c[8];
    uint2 packed = make_uint2(0u, 0u);
    if (inv != 0.f) q8_codes(p, top, inv, c, packed);
    else
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = 0.f;
    *reinterpret_cast<uint2*>(o.codes + row * o.ldc + at) = packed;
    if (o.x == nullptr) return;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = o.full ? pack2(p[2 * i] * over, p[2 * i + 1] * over) : pack2(c[2 * i] * scale, c[2 * i + 1] * scale);
    st16(o.x + row * o.ldx + at, make_uint4(w[0], w[1], w[2], w[3]));
}

// Rows blockIdx.x, blockIdx.x + gridDim.x, ...; thread i holds the eight values from columns
// 8 (i + j blockDim), j < V.  PRE: the next row is fetched ahead.
template <int V, bool PRE>
__global__ void __launch_bounds__(1024) q8_norm_kernel(const __grid_constant__ Q8NormParams q) {
    __shared__ uint32_t red_top[3][32];
    __shared__ float red_ss[3][32];
    const int tid = threadIdx.x;
    const bool add = q.residual != nullptr;
    uint4 xn[V], rn[V];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int at = 8 * (tid + j * blockDim.x);
            xn[j] = rn[j] = make_uint4(0, 0, 0, 0);
            if (at < q.d && row < q.T) {
                xn[j] = ld16(q.x + row * q.ldx + at);
                if (add) rn[j] = ld16(q.residual + row * q.ldr + at);
            }
        }
    };
    uint4 gw[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int at = 8 * (tid + j * blockDim.x);
        gw[j] = at < q.d ? ld16(q.weight + at) : make_uint4(0, 0, 0, 0);
    }
    fetch(blockIdx.x);
    int turn = 0;
    for (int64_t row = blockIdx.x; row < q.T; row += gridDim.x, turn ^= 1) {
        float p[V][8];
        uint32_t top = 0;
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int at = 8 * (tid + j * blockDim.x);
            float h[8], g[8];
            unpack8(xn[j], h);
            if (add) {
                float r[8];
                unpack8(rn[j], r);
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // the sum is held in bf16, and the norm is that of what is held
                    w[i] = pack2(h[2 * i] + r[2 * i], h[2 * i + 1] + r[2 * i + 1]);
                    h[2 * i] = bf16lo(w[i]);
                    h[2 * i + 1] = bf16hi(w[i]);
                }
                if (q.sum && at < q.d) st16(q.sum + row * q.lds + at, make_uint4(w[0], w[1], w[2], w[3]));
            }
            unpack8(gw[j], g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[j][i] = h[i] * g[i];
                ss = fmaf(h[i], h[i], ss);
                top = max(top, __float_as_uint(fabsf(p[j][i])));
            }
        }
        if (PRE) fetch(row + gridDim.x);
        q8_reduce(top, ss, red_top[turn], red_ss[turn]);
        float over = 1.f / sqrtf(ss / (float)q.d + q.eps), back = 1.f;
        const bool large = __float_as_uint(ss) == kInfBits;
        if (large || (top != 0 && __uint_as_float(top) < kQ8Small)) {
            // squares past fp32's range, or products near its other end: once more by a power of two
            const float by_h = large ? 0x1p-80f : 0x1p32f, by_w = large ? 1.f : 0x1p32f;
            ss = 0.f;
            top = 0;
            // from h where that is held: x or the residual may have given it their place
            const __nv_bfloat16* from = q.sum ? q.sum + row * q.lds : q.x + row * q.ldx;
#pragma unroll 1
            for (int j = 0; j < V; ++j) {
                const int at = 8 * (tid + j * blockDim.x);
                if (at >= q.d) continue;
                float h[8], g[8];
                unpack8(ld16(from + at), h);
                if (add && !q.sum) {
                    float r[8];
                    unpack8(ld16(q.residual + row * q.ldr + at), r);
#pragma unroll
                    for (int i = 0; i < 8; ++i) h[i] = __bfloat162float(__float2bfloat16_rn(h[i] + r[i]));
                }
                unpack8(ld16(q.weight + at), g);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float v = h[i] * by_h, w = v * (g[i] * by_w);
#pragma unroll
                    for (int k = 0; k < V; ++k)
                        if (k == j) p[k][i] = w;
                    ss = fmaf(v, v, ss);
                    top = max(top, __float_as_uint(fabsf(w)));
                }
            }
            q8_reduce(top, ss, red_top[2], red_ss[2]);
            if (large) over = 1.f / sqrtf(ss / (float)q.d);     // of values so large that eps is nothing
            else back = kQ8Small;
        }
        float inv = 0.f, scale = 0.f;
        const float m = __uint_as_float(top);
        if (top >= kInfBits) scale = over = __uint_as_float(0x7FC00000u);
        else if (top != 0) {
            inv = 127.f / m;
            scale = m * over / 127.f * back;
            over *= back;
        }
        if (tid == 0) q.out.scales[row] = scale;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int at = 8 * (tid + j * blockDim.x);
            if (at < q.d) q8_store(q.out, row, at, p[j], m, inv, scale, over);
        }
        if (!PRE) fetch(row + gridDim.x);
    }
}

template <int ACT>
__device__ __forceinline__ float q8_act(float a) {
    // e^-a to 2^-24 (4 + |a|) of itself; where it passes fp32's range, a e^a is nothing
    if (ACT == LORA_ACT_SILU) return a * rcp_approx(1.f + exp2_approx(-1.44269504f * a));
    if (ACT == LORA_ACT_GELU) return 0.5f * a * (1.f + erff(a * 0.70710678f));
    if (ACT == LORA_ACT_GELU_TANH) return 0.5f * a * (1.f + tanhf(0.79788456f * (a + 0.044715f * a * a * a)));
    return a;
}

template <int V, int ACT, bool PRE>
__global__ void __launch_bounds__(1024) q8_gate_kernel(const __grid_constant__ Q8GateParams q) {
    __shared__ uint32_t red_top[2][32];
    __shared__ float red_ss[2][32];
    const int tid = threadIdx.x;
    const bool gated = q.up != nullptr;
    uint4 an[V], un[V];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int at = 8 * (tid + j * blockDim.x);
            an[j] = un[j] = make_uint4(0, 0, 0, 0);
            if (at < q.d && row < q.T) {
                an[j] = ld16(q.gate + row * q.ldg + at);
                if (gated) un[j] = ld16(q.up + row * q.ldu + at);
            }
        }
    };
    fetch(blockIdx.x);
    int turn = 0;
    for (int64_t row = blockIdx.x; row < q.T; row += gridDim.x, turn ^= 1) {
        float p[V][8];
        uint32_t top = 0;
        float none = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            unpack8(an[j], p[j]);
            float u[8];
            unpack8(un[j], u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool bad = max(__float_as_uint(fabsf(p[j][i])), __float_as_uint(fabsf(u[i]))) >= kInfBits;
                p[j][i] = q8_act<ACT>(p[j][i]);
                if (gated) p[j][i] *= u[i];
                top = max(top, bad ? 0x7FC00000u : __float_as_uint(fabsf(p[j][i])));
            }
        }
        if (PRE) fetch(row + gridDim.x);
        q8_reduce(top, none, red_top[turn], red_ss[turn]);
        float back = 1.f;
        if (top != 0 && __uint_as_float(top) < kQ8Small) {  // near fp32's smallest values: by a power of two
            back = kQ8Small;
            top = __float_as_uint(__uint_as_float(top) * kQ8Up);
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) p[j][i] *= kQ8Up;
        }
        float inv = 0.f, scale = 0.f, over = back;
        const float m = __uint_as_float(top);
        if (top >= kInfBits) scale = over = __uint_as_float(0x7FC00000u);
        else if (top != 0) {
            inv = 127.f / m;
            scale = m / 127.f * back;
        }
        if (tid == 0) q.out.scales[row] = scale;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int at = 8 * (tid + j * blockDim.x);
            if (at < q.d) q8_store(q.out, row, at, p[j], m, inv, scale, over);
        }
        if (!PRE) fetch(row + gridDim.x);
    }
}

}  // namespace lora
