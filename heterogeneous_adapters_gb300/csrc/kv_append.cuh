// Appending a batch's keys and values to the 4-bit cache, and reading them back.
#pragma once
#include "kv_layout.cuh"

namespace lora {

constexpr int kAppendWarps = 8;

struct AppendParams {
    KvView v;
    const __nv_bfloat16 *q, *k, *val;
    __nv_bfloat16* q_out;
    int64_t ldq, ldqo, ldk, ldv;
    const float *cos, *sin;
    const int32_t* positions;
    int32_t max_pos, rot_dim, style;
    int32_t q_heads;
    int32_t per_warp;        // steps of 32 / (D / 8) heads that a warp takes
};

// Eight values a lane, D / 8 lanes a head: a warp holds 256 / D heads at a time and all of
// them turn by the same angles, read once per row.  A lane's partner values of the halves
// style are D-wide exchanges between lanes (the rotation covers whole 8-value pieces).
template <int D, int G>
__global__ void __launch_bounds__(kAppendWarps * 32) kv_append_kernel(const __grid_constant__ AppendParams p) {
    constexpr int kLanes = D / 8, kHeads = 32 / kLanes;
    const int lane = threadIdx.x & 31;
    const int sub = lane / kLanes, piece = lane % kLanes, d0 = piece * 8;
    const int total = p.q_heads + 2 * p.v.heads;
    const int steps = (total + kHeads - 1) / kHeads;
    const int per_row = (steps + p.per_warp - 1) / p.per_warp;
    const int64_t w = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
    kv_check_starts(p.v, w, (int64_t)gridDim.x * kAppendWarps);
    const int row = (int)(w / per_row);
    if (row >= p.v.T) return;
    const KvRow r = kv_find_row(p.v, row);
    if (r.token < 0) return;
    const int pos = p.positions ? p.positions[row] : r.token;
    if (p.rot_dim > 0 && (pos < 0 || pos >= p.max_pos)) {
        if (lane == 0) set_error(p.v.err, LORA_DERR_KV);
        return;
    }
    // block and tile of the row's token, for head 0 (other heads follow at a fixed stride)
    constexpr int kTileBytes = kv_tile_bytes(D, G);
    unsigned char* tile0 = kv_tile_of(p.v, r.seq, r.token, 0, kTileBytes);
    if (tile0 == nullptr) return;
    const int64_t head_stride = (int64_t)(p.v.block_tokens / kKvTile) * kTileBytes;
    const int tok = r.token % kKvTile;
    // the angles of this lane's eight values: pair index i of value d
    const int half = p.rot_dim / 2;
    const bool turn = d0 < p.rot_dim;
    float c[8], s[8];
    if (turn) {
        const int64_t at = (int64_t)pos * half;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int d = d0 + j;
            const int i = p.style == LORA_ROPE_PAIRS ? d / 2 : d < half ? d : d - half;
            c[j] = p.cos[at + i];
            s[j] = p.sin[at + i];
        }
    }
    // halves style: value d pairs with d +- half, half / 8 lanes away
    const int partner = d0 < half ? lane + half / 8 : lane - half / 8;
    const int step0 = (int)(w % per_row) * p.per_warp;
    for (int st = step0; st < min(steps, step0 + p.per_warp); ++st) {
        const int head = st * kHeads + sub;
        const bool live = head < total;
        const bool is_q = head < p.q_heads, is_v = head >= p.q_heads + p.v.heads;
        const int kvh = is_q ? 0 : is_v ? head - p.q_heads - p.v.heads : head - p.q_heads;
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (live) {
            const __nv_bfloat16* src = is_q ? p.q + row * p.ldq + (int64_t)head * D
                                     : is_v ? p.val + row * p.ldv + (int64_t)kvh * D
                                            : p.k + row * p.ldk + (int64_t)kvh * D;
            raw = ld16(src + d0);
        }
        float x[8];
        unpack8(raw, x);
        if (p.rot_dim > 0) {
            uint4 other;
            const int from = turn ? partner : lane;
            other.x = __shfl_sync(0xffffffffu, raw.x, from);
            other.y = __shfl_sync(0xffffffffu, raw.y, from);
            other.z = __shfl_sync(0xffffffffu, raw.z, from);
            other.w = __shfl_sync(0xffffffffu, raw.w, from);
            if (turn && !is_v) {
                float o[8];
                unpack8(other, o);
                if (p.style == LORA_ROPE_PAIRS) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = x[j ^ 1];
                    const float t[8] = {x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]};
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        x[j] = j & 1 ? __fadd_rn(__fmul_rn(t[j], c[j]), __fmul_rn(o[j], s[j]))
                                     : __fsub_rn(__fmul_rn(t[j], c[j]), __fmul_rn(o[j], s[j]));
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        x[j] = d0 >= half ? __fadd_rn(__fmul_rn(x[j], c[j]), __fmul_rn(o[j], s[j]))
                                          : __fsub_rn(__fmul_rn(x[j], c[j]), __fmul_rn(o[j], s[j]));
                }
            }
        }
        if (live && is_q)
            st16(p.q_out + row * p.ldqo + (int64_t)head * D + d0,
                 make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7])));
        if (st * kHeads + kHeads <= p.q_heads) continue;    // a step of query heads only
        // minimum and maximum of the group, over its G / 8 lanes; a value that is not finite
        // makes the sum of zeros x - x not a number
        float lo = x[0], hi = x[0], bad = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            lo = fminf(lo, x[j]);
            hi = fmaxf(hi, x[j]);
            bad += x[j] - x[j];
        }
#pragma unroll
        for (int m = 1; m < G / 8; m <<= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
            bad += __shfl_xor_sync(0xffffffffu, bad, m);
        }
        if (!live || is_q) continue;
        __half scale = __float2half_rn(fminf(__fmul_rn(hi - lo, 1.0f / 15.0f), 65504.f));
        const float sf = __half2float(scale);
        __half offset = __float2half_rn(fminf(fmaxf(__fadd_rn(lo, __fmul_rn(8.f, sf)), -65504.f), 65504.f));
        const float of = __half2float(offset);
        const float inv = sf > 0.f ? __fdiv_rn(1.f, sf) : 0.f;
        if (bad != 0.f) scale = offset = __ushort_as_half(0x7fff);
        uint32_t word = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float f = fminf(fmaxf(rintf(__fmul_rn(__fsub_rn(x[j], of), inv)), -8.f), 7.f);
            word |= (uint32_t)((int)f + 8) << (4 * j);
        }
        unsigned char* tile = tile0 + kvh * head_stride;
        *reinterpret_cast<uint32_t*>(tile + kv_codes_at(D, is_v) + ((d0 / 32) * kKvTile + tok) * 16 + (d0 % 32) / 2) = word;
        if (d0 % G == 0)
            *reinterpret_cast<__half2*>(tile + kv_params_at(D, G, is_v) + ((d0 / G) * kKvTile + tok) * 4) =
                __halves2half2(scale, offset);
    }
}

struct ReadParams {
    KvView v;
    __nv_bfloat16 *k, *val;
    int64_t ldk, ldv;
    int32_t per_warp;
};

// The stored values of the batch's rows, laid out as the append reads them.
template <int D, int G>
__global__ void __launch_bounds__(kAppendWarps * 32) kv_read_kernel(const __grid_constant__ ReadParams p) {
    constexpr int kLanes = D / 8, kHeads = 32 / kLanes, kTileBytes = kv_tile_bytes(D, G);
    const int lane = threadIdx.x & 31;
    const int sub = lane / kLanes, d0 = lane % kLanes * 8;
    const int total = 2 * p.v.heads;
    const int steps = (total + kHeads - 1) / kHeads;
    const int per_row = (steps + p.per_warp - 1) / p.per_warp;
    const int64_t w = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
    kv_check_starts(p.v, w, (int64_t)gridDim.x * kAppendWarps);
    const int row = (int)(w / per_row);
    if (row >= p.v.T) return;
    const KvRow r = kv_find_row(p.v, row);
    if (r.seq < 0) return;
    const unsigned char* tile0 = r.token < 0 ? nullptr : kv_tile_of(p.v, r.seq, r.token, 0, kTileBytes);
    const int64_t head_stride = (int64_t)(p.v.block_tokens / kKvTile) * kTileBytes;
    const int tok = r.token % kKvTile;
    const int step0 = (int)(w % per_row) * p.per_warp;
    for (int st = step0; st < min(steps, step0 + p.per_warp); ++st) {
        const int head = st * kHeads + sub;
        if (head >= total) continue;
        const bool is_v = head >= p.v.heads;
        const int kvh = is_v ? head - p.v.heads : head;
        uint4 out = make_uint4(0, 0, 0, 0);
        if (tile0 != nullptr) {
            const unsigned char* tile = tile0 + kvh * head_stride;
            const uint32_t word = *reinterpret_cast<const uint32_t*>(
                tile + kv_codes_at(D, is_v) + ((d0 / 32) * kKvTile + tok) * 16 + (d0 % 32) / 2);
            const float2 so = __half22float2(*reinterpret_cast<const __half2*>(
                tile + kv_params_at(D, G, is_v) + ((d0 / G) * kKvTile + tok) * 4));
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = __fadd_rn(__fmul_rn(so.x, (float)(int)(word >> (4 * j) & 15) - 8.f), so.y);
            out = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
        }
        st16((is_v ? p.val + row * p.ldv : p.k + row * p.ldk) + (int64_t)kvh * D + d0, out);
    }
}

}  // namespace lora
