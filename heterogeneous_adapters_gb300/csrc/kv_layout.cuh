// The 4-bit KV cache (include/lora_kv.h) as the kernels see it: addresses of tiles, the
// batch's rows, and the errors found in the batch's arrays.
#pragma once
#include <cuda_fp16.h>

#include "step.cuh"
#include "lora_kv.h"

namespace lora {

constexpr int kKvTile = 16;   // tokens of a tile

// Bytes of a tile of 16 tokens of one head: K and V codes, K and V parameters.
__host__ __device__ constexpr int kv_tile_bytes(int dim, int group) { return kKvTile * (dim + 8 * (dim / group)); }
// Offsets inside a tile.
__host__ __device__ constexpr int kv_codes_at(int dim, int which) { return which * kKvTile * dim / 2; }
__host__ __device__ constexpr int kv_params_at(int dim, int group, int which) {
    return kKvTile * dim + which * kKvTile * 4 * (dim / group);
}

struct KvView {
    unsigned char* blocks;
    int64_t num_blocks;
    int64_t block_stride;
    int32_t block_tokens;
    int32_t heads;          // KV heads
    const int32_t* q_start;
    const int32_t* kv_len;
    const int32_t* table;
    int32_t n_seq;
    int32_t T;
    int32_t max_blocks;
    int32_t max_q;
    int32_t rows_lo, rows_hi;   // requests with rows_lo .. rows_hi rows are this launch's (attention)
    uint32_t* err;
};

// A row's request (-1: of none, or of one whose rows are in error; the row is left alone)
// and its token (< 0: before the request's first token).
struct KvRow {
    int32_t seq;
    int32_t token;
};

// Cached tokens of a request; any negative number is none of them (and stays far from the
// type's end, so that rows can be counted from it).
__device__ __forceinline__ int kv_length(const KvView& v, int s) { return max(v.kv_len[s], -(1 << 25)); }

// The request that owns `row` and the row's token, by all 32 lanes of a warp together: most
// decode batches have one row a request, so request `row` is looked at first; else 32
// places of q_start are read at a time (log32 n_seq dependent reads).
__device__ __forceinline__ KvRow kv_find_row(const KvView& v, int row) {
    const int lane = threadIdx.x & 31;
    const int guess = min(row, v.n_seq - 1);
    int s = guess;
    int a = v.q_start[s], b = v.q_start[s + 1];
    if (!(a <= row && row < b)) {
        // the last request that starts at or before the row, in [lo, lo + n)
        int lo = 0, n = v.n_seq;
        while (n > 1) {
            const int step = (n + 31) / 32;
            const int at = lo + lane * step;
            const bool le = lane * step < n && v.q_start[at] <= row;
            const unsigned m = __ballot_sync(0xffffffffu, le);
            const int k = m ? 31 - __clz(m) : 0;
            n = min(step, n - k * step);
            lo += k * step;
        }
        s = lo;
        a = v.q_start[s];
        b = v.q_start[s + 1];
    }
    KvRow r;
    r.seq = s;
    r.token = -1;
    if (a <= row && row < b) {
        const bool bad = a < 0 || b > v.T, big = b - a > v.max_q;
        if (!bad && !big) r.token = kv_length(v, s) - (b - row);
        else {
            r.seq = -1;
            if (lane == 0) set_error(v.err, bad ? LORA_DERR_SEGMENT : LORA_DERR_KV);
        }
    } else {
        r.seq = -1;
    }
    return r;
}

// Looks for requests whose rows decrease or leave [0, T], 32 places of q_start a warp of the launch.
__device__ __forceinline__ void kv_check_starts(const KvView& v, int64_t warp, int64_t warps) {
    for (int64_t i = warp * 32 + (threadIdx.x & 31); i < v.n_seq; i += warps * 32) {
        const int a = v.q_start[i], b = v.q_start[i + 1];
        if (a > b || a < 0 || b > v.T) set_error(v.err, LORA_DERR_SEGMENT);
    }
}

// Address of the tile that holds `token` (>= 0) of request `seq` and head; nullptr (and the
// error bit) if the batch's arrays do not give one.
__device__ __forceinline__ unsigned char* kv_tile_of(const KvView& v, int seq, int token, int head, int tile_bytes) {
    const int j = token / v.block_tokens;
    if (j < v.max_blocks) {
        const int b = v.table[(int64_t)seq * v.max_blocks + j];
        if (b >= 0 && b < v.num_blocks)
            return v.blocks + (int64_t)b * v.block_stride +
                   (int64_t)(head * (v.block_tokens / kKvTile) + token % v.block_tokens / kKvTile) * tile_bytes;
    }
    set_error(v.err, LORA_DERR_KV);
    return nullptr;
}

}  // namespace lora
