// Appending a batch's keys and values to the 4-bit cache, and reading them back.
#pragma once
#include "kv_layout.cuh"

namespace lora {

constexpr int kAppendWarps = 8;
constexpr int kAppendBatch = 4;

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

// Eight values a lane, D / 8 lanes a head: a warp holds 256 / D heads at a time (a step) and
// all of them turn by the same angles, read once per row.  A lane's partner values of the
// halves style are whole pieces of another lane.  What bounds it is the stream of q, k and v;
// a step is a few hundred clocks of work behind a load, so a warp has kAppendBatch steps'
// loads in flight.  Three CTAs an SM with four loads measured 51 us on 8.7k prompt rows (197
// MB, 58% of the copy rate), two CTAs 59, four (64 registers) 61, four with two loads 56.
template <int D, int G>
__global__ void __launch_bounds__(kAppendWarps * 32, 3) kv_append_kernel(const __grid_constant__ AppendParams p) {
    constexpr int kLanes = D / 8, kHeads = 32 / kLanes;
    const int lane = threadIdx.x & 31;
    const int sub = lane / kLanes, piece = lane % kLanes, d0 = piece * 8;
    const int kv0 = p.q_heads, v0 = p.q_heads + p.v.heads, total = p.q_heads + 2 * p.v.heads;
    const int steps = (total + kHeads - 1) / kHeads;
    const int per_row = (steps + p.per_warp - 1) / p.per_warp;
    const int64_t w = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
    kv_check_starts(p.v, w, (int64_t)gridDim.x * kAppendWarps);
    const int row = (int)(w / per_row);
    if (row >= p.v.T) return;
    const int step0 = (int)(w % per_row) * p.per_warp, step1 = min(steps, step0 + p.per_warp);
    const __nv_bfloat16 *qr = p.q + row * p.ldq + d0, *kr = p.k + row * p.ldk + d0, *vr = p.val + row * p.ldv + d0;
    // this lane's values of the steps st ..
    uint4 raw[kAppendBatch];
    auto load = [&](int st) {
#pragma unroll
        for (int i = 0; i < kAppendBatch; ++i) {
            const int head = (st + i) * kHeads + sub;
            raw[i] = make_uint4(0, 0, 0, 0);
            if (st + i < step1 && head < total)
                raw[i] = ld16(head < kv0 ? qr + (int64_t)head * D : head < v0 ? kr + (int64_t)(head - kv0) * D : vr + (int64_t)(head - v0) * D);
        }
    };
    load(step0);
    const KvRow r = kv_find_row(p.v, row);
    if (r.token < 0) return;
    const int pos = p.positions ? p.positions[row] : r.token;
    if (p.rot_dim > 0 && (pos < 0 || pos >= p.max_pos)) {
        if (lane == 0) set_error(p.v.err, LORA_DERR_KV);
        return;
    }
    // tile of the row's token, for head 0 (other heads follow at a fixed stride)
    constexpr int kTileBytes = kv_tile_bytes(D, G);
    unsigned char* tile0 = kv_tile_of(p.v, r.seq, r.token, 0, kTileBytes);
    if (tile0 == nullptr) return;
    const int64_t head_stride = (int64_t)(p.v.block_tokens / kKvTile) * kTileBytes;
    const int tok = r.token % kKvTile;
    // the angles of this lane's eight values (a rotation covers whole pieces of eight):
    // sines signed so that a turn is x c + other s
    const int half = p.rot_dim / 2;
    const bool turn = d0 < p.rot_dim, pairs = p.style == LORA_ROPE_PAIRS;
    float c[8], s[8];
    if (turn) {
        const int64_t at = (int64_t)pos * half;
        if (pairs) {
            const float4 cv = *reinterpret_cast<const float4*>(p.cos + at + d0 / 2), sv = *reinterpret_cast<const float4*>(p.sin + at + d0 / 2);
            c[0] = c[1] = cv.x, c[2] = c[3] = cv.y, c[4] = c[5] = cv.z, c[6] = c[7] = cv.w;
            s[1] = sv.x, s[3] = sv.y, s[5] = sv.z, s[7] = sv.w;
            s[0] = -sv.x, s[2] = -sv.y, s[4] = -sv.z, s[6] = -sv.w;
        } else {
            const int i0 = d0 < half ? d0 : d0 - half;
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
                const float4 cv = *reinterpret_cast<const float4*>(p.cos + at + i0 + j), sv = *reinterpret_cast<const float4*>(p.sin + at + i0 + j);
                c[j] = cv.x, c[j + 1] = cv.y, c[j + 2] = cv.z, c[j + 3] = cv.w;
                s[j] = sv.x, s[j + 1] = sv.y, s[j + 2] = sv.z, s[j + 3] = sv.w;
            }
            if (d0 < half)
#pragma unroll
                for (int j = 0; j < 8; ++j) s[j] = -s[j];
        }
    }
    const int from = turn ? (d0 < half ? lane + half / 8 : lane - half / 8) : lane;
    for (int st = step0; st < step1; st += kAppendBatch) {
        uint4 now[kAppendBatch];
#pragma unroll
        for (int i = 0; i < kAppendBatch; ++i) now[i] = raw[i];
        if (st + kAppendBatch < step1) load(st + kAppendBatch);
#pragma unroll
        for (int i = 0; i < kAppendBatch; ++i) {
            if (st + i >= step1) break;
            const int head = (st + i) * kHeads + sub;
            const bool live = head < total, is_q = head < kv0, is_v = head >= v0;
            float x[8];
            unpack8(now[i], x);
            if (p.rot_dim > 0 && (st + i) * kHeads < v0) {
                float o[8];
                if (pairs) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = x[j ^ 1];
                } else {
                    uint4 other;
                    other.x = __shfl_sync(0xffffffffu, now[i].x, from);
                    other.y = __shfl_sync(0xffffffffu, now[i].y, from);
                    other.z = __shfl_sync(0xffffffffu, now[i].z, from);
                    other.w = __shfl_sync(0xffffffffu, now[i].w, from);
                    unpack8(other, o);
                }
                if (turn && !is_v) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = __fadd_rn(__fmul_rn(x[j], c[j]), __fmul_rn(o[j], s[j]));
                }
            }
            if (live && is_q)
                st16(p.q_out + row * p.ldqo + (int64_t)head * D + d0,
                     make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7])));
            if ((st + i + 1) * kHeads <= kv0) continue;         // a step of query heads only
            // minimum and maximum of the group, over its G / 8 lanes; zero times a value that is
            // not finite is not a number
            float lo = x[0], hi = x[0], zero = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                lo = fminf(lo, x[j]);
                hi = fmaxf(hi, x[j]);
                zero = fmaf(x[j], 0.f, zero);
            }
#pragma unroll
            for (int m = 1; m < G / 8; m <<= 1) {
                lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
                hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
            }
            const uint32_t bad = __ballot_sync(0xffffffffu, zero != 0.f) >> (lane & ~(G / 8 - 1)) & ((1u << (G / 8)) - 1);
            if (!live || is_q) continue;
            __half scale = __float2half_rn(fminf(__fmul_rn(hi - lo, 1.0f / 15.0f), 65504.f));
            const float sf = __half2float(scale);
            __half offset = __float2half_rn(fminf(fmaxf(__fadd_rn(lo, __fmul_rn(8.f, sf)), -65504.f), 65504.f));
            const float of = __half2float(offset);
            const float inv = sf > 0.f ? __frcp_rn(sf) : 0.f;
            if (bad) scale = offset = __ushort_as_half(0x7fff);
            // adding 1.5 2^23 + 8 rounds to a whole number, to even at ties, whose last four bits
            // are the code
            uint32_t word = 0;
#pragma unroll
            for (int j = 7; j >= 0; --j) {
                const float f = fminf(fmaxf(__fmul_rn(__fsub_rn(x[j], of), inv), -8.f), 7.f);
                word = word * 16u + (__float_as_uint(__fadd_rn(f, 12582920.f)) - 0x4B400000u);
            }
            unsigned char* tile = tile0 + (is_v ? head - v0 : head - kv0) * head_stride;
            *reinterpret_cast<uint32_t*>(tile + kv_codes_at(D, is_v) + ((d0 / 32) * kKvTile + tok) * 16 + (d0 % 32) / 2) = word;
            if (d0 % G == 0)
                *reinterpret_cast<__half2*>(tile + kv_params_at(D, G, is_v) + ((d0 / G) * kKvTile + tok) * 4) =
                    __halves2half2(scale, offset);
        }
    }
}

struct ReadParams {
    KvView v;
    __nv_bfloat16 *k, *val;
    int64_t ldk, ldv;
    int32_t per_warp;
};

// The stored values of the batch's rows, laid out as the append reads them: 15 us for 8.7k rows
// of 8 heads (55 MB, from L2 after the append; 55% of the copy rate, instructions at 66% of the
// issue slots).
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
    const int step0 = (int)(w % per_row) * p.per_warp, step1 = min(steps, step0 + p.per_warp);
    for (int st = step0; st < step1; st += kAppendBatch) {
        uint32_t word[kAppendBatch], so[kAppendBatch];
#pragma unroll
        for (int i = 0; i < kAppendBatch; ++i) {
            const int head = (st + i) * kHeads + sub;
            const bool is_v = head >= p.v.heads;
            word[i] = so[i] = 0;
            if (st + i < step1 && head < total && tile0 != nullptr) {
                const unsigned char* tile = tile0 + (is_v ? head - p.v.heads : head) * head_stride;
                word[i] = *reinterpret_cast<const uint32_t*>(tile + kv_codes_at(D, is_v) + ((d0 / 32) * kKvTile + tok) * 16 + (d0 % 32) / 2);
                so[i] = *reinterpret_cast<const uint32_t*>(tile + kv_params_at(D, G, is_v) + ((d0 / G) * kKvTile + tok) * 4);
            }
        }
#pragma unroll
        for (int i = 0; i < kAppendBatch; ++i) {
            const int head = (st + i) * kHeads + sub;
            if (st + i >= step1 || head >= total) continue;
            const bool is_v = head >= p.v.heads;
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&so[i]));   // zeros: a row that is not there
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = __fadd_rn(__fmul_rn(f.x, (float)(int)(word[i] >> (4 * j) & 15) - 8.f), f.y);
            st16((is_v ? p.val + row * p.ldv + (int64_t)(head - p.v.heads) * D : p.k + row * p.ldk + (int64_t)head * D) + d0,
                 make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7])));
        }
    }
}

}  // namespace lora
