// C ABI of the 4-bit KV cache (include/lora_kv.h): argument checks and launches.
#include <string.h>

#include <algorithm>

#include "host.h"
#include "kv_append.cuh"
#include "kv_attend.cuh"
#include "kv_prefill.cuh"

using namespace lora;
using namespace lora::host;

namespace {

lora_status check_shape(int32_t block_tokens, int32_t heads, int32_t dim, int32_t group) {
    if (block_tokens <= 0 || block_tokens % kKvTile != 0 || heads <= 0) return LORA_EINVAL;
    if (dim != 64 && dim != 128) return LORA_EINVAL;
    if (group != 32 && group != dim) return LORA_EINVAL;
    if (block_tokens > 1024 || heads > LORA_KV_MAX_HEADS) return LORA_ETOOBIG;
    return LORA_OK;
}

int64_t block_bytes(const lora_kv_cache_desc* c) {
    return (int64_t)c->num_kv_heads * (c->block_tokens / kKvTile) * kv_tile_bytes(c->head_dim, c->group);
}

// Sizes only (the arrays are not looked at).
lora_status check_sizes(const lora_kv_cache_desc* c, const lora_kv_batch* b) {
    if (c == nullptr || b == nullptr) return LORA_EINVAL;
    lora_status st = check_shape(c->block_tokens, c->num_kv_heads, c->head_dim, c->group);
    if (st != LORA_OK) return st;
    if (b->n_seq < 0 || b->T < 0 || b->max_q < 0 || b->max_blocks < 0) return LORA_EINVAL;
    if (b->n_seq > LORA_KV_MAX_SEQS || b->T > (1 << 24) || (int64_t)b->max_blocks * c->block_tokens > (1 << 30))
        return LORA_ETOOBIG;
    return LORA_OK;
}

size_t workspace_bytes() { return align256(std::max(attend_workspace(2, 128), pre_workspace(128))); }

// Arrays of 32-bit values (an odd address would fault the kernels).
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

lora_status check_call(const lora_kv_cache_desc* c, const lora_kv_batch* b, const void* ws, size_t ws_bytes, size_t need) {
    lora_status st = check_sizes(c, b);
    if (st != LORA_OK) return st;
    if (c->blocks == nullptr || c->num_blocks <= 0) return LORA_EINVAL;
    if (!aligned16(c->blocks) || c->block_stride % 16 != 0) return LORA_EALIGN;
    if (c->block_stride < block_bytes(c) || c->num_blocks > INT32_MAX || c->num_blocks > INT64_MAX / c->block_stride)
        return LORA_EINVAL;
    if (b->n_seq > 0 && (b->q_start == nullptr || b->kv_len == nullptr || (b->max_blocks > 0 && b->block_table == nullptr)))
        return LORA_EINVAL;
    if (!aligned4(b->q_start) || !aligned4(b->kv_len) || !aligned4(b->block_table)) return LORA_EALIGN;
    if (ws == nullptr || ((uintptr_t)ws & 255u) != 0 || ws_bytes < need) return LORA_EWORKSPACE;
    return LORA_OK;
}

// A bf16 matrix argument of `cols` columns.
lora_status check_rows(const void* p, int64_t ld, int64_t cols) {
    if (p == nullptr || ld < cols) return LORA_EINVAL;
    if (!aligned16(p) || ld % 8 != 0) return LORA_EALIGN;
    return LORA_OK;
}

KvView view_of(const lora_kv_cache_desc* c, const lora_kv_batch* b, void* ws) {
    KvView v;
    v.blocks = reinterpret_cast<unsigned char*>(c->blocks);
    v.num_blocks = c->num_blocks;
    v.block_stride = c->block_stride;
    v.block_tokens = c->block_tokens;
    v.heads = c->num_kv_heads;
    v.q_start = b->q_start;
    v.kv_len = b->kv_len;
    v.table = b->block_table;
    v.n_seq = b->n_seq;
    v.T = b->T;
    v.max_blocks = b->max_blocks;
    v.max_q = b->max_q;
    v.rows_lo = 0;
    v.rows_hi = INT32_MAX;
    v.err = &reinterpret_cast<WsHeader*>(ws)->err;
    return v;
}

// Heads a warp of the row kernels (append, read) takes, in steps of 256 values: as few as
// give every SM 32 warps, so that a single token still uses many warps, and
// a prompt's rows read their angles and look their request up once for several heads.
int steps_per_warp(const DeviceInfo* di, int T, int steps) {
    const int64_t slots = (int64_t)di->sm_count * 32;
    return (int)std::min<int64_t>(std::max<int64_t>((int64_t)T * steps / slots, 1), steps);
}

template <template <int, int> class Launch, class P>
lora_status by_shape(const lora_kv_cache_desc* c, const P& p, dim3 grid, cudaStream_t s) {
    if (c->head_dim == 128) {
        if (c->group == 32) Launch<128, 32>::run(p, grid, s);
        else Launch<128, 128>::run(p, grid, s);
    } else {
        if (c->group == 32) Launch<64, 32>::run(p, grid, s);
        else Launch<64, 64>::run(p, grid, s);
    }
    return cuda_status(cudaGetLastError());
}

template <int D, int G>
struct Append {
    static void run(const AppendParams& p, dim3 grid, cudaStream_t s) { kv_append_kernel<D, G><<<grid, kAppendWarps * 32, 0, s>>>(p); }
};
template <int D, int G>
struct Read {
    static void run(const ReadParams& p, dim3 grid, cudaStream_t s) { kv_read_kernel<D, G><<<grid, kAppendWarps * 32, 0, s>>>(p); }
};
template <int D, int G, int NT>
lora_status attend(const AttendParams& p, cudaStream_t s) {
    DeviceInfo* di = nullptr;
    lora_status st = device_info(&di);
    if (st != LORA_OK) return st;
    constexpr size_t smem = attend_smem(D, G);
    auto kern = kv_attend_kernel<D, G, NT>;
    static thread_local const DeviceInfo* ready = nullptr;
    static thread_local int per_sm = 0;
    if (ready != di) {
        st = cuda_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
        if (st != LORA_OK) return st;
        st = cuda_status(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kAttThreads, smem));
        if (st != LORA_OK) return st;
        ready = di;
    }
    const int grid = std::min(di->sm_count * std::max(per_sm, 1), kAttMaxCtas);
    kern<<<grid, kAttThreads, smem, s>>>(p);
    return cuda_status(cudaGetLastError());
}

template <int D>
lora_status prefill(const AttendParams& p, cudaStream_t s) {
    DeviceInfo* di = nullptr;
    lora_status st = device_info(&di);
    if (st != LORA_OK) return st;
    constexpr size_t smem = pre_smem(D).total;
    auto kern = kv_prefill_kernel<D>;
    static thread_local const DeviceInfo* ready = nullptr;
    if (ready != di) {
        st = cuda_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
        if (st != LORA_OK) return st;
        ready = di;
    }
    kern<<<std::min(di->sm_count, kPreMaxCtas), kPreThreads, smem, s>>>(p);
    return cuda_status(cudaGetLastError());
}

template <int NT>
lora_status attend_by_shape(const lora_kv_cache_desc* c, const AttendParams& p, cudaStream_t s) {
    if (c->head_dim == 128) return c->group == 32 ? attend<128, 32, NT>(p, s) : attend<128, 128, NT>(p, s);
    return c->group == 32 ? attend<64, 32, NT>(p, s) : attend<64, 64, NT>(p, s);
}

}  // namespace

extern "C" {

lora_status lora_kv_block_bytes(int32_t block_tokens, int32_t num_kv_heads, int32_t head_dim, int32_t group,
                                size_t* bytes) {
    if (bytes == nullptr) return LORA_EINVAL;
    lora_status st = check_shape(block_tokens, num_kv_heads, head_dim, group);
    if (st != LORA_OK) return st;
    *bytes = (size_t)num_kv_heads * (block_tokens / kKvTile) * kv_tile_bytes(head_dim, group);
    return LORA_OK;
}

lora_status lora_kv_workspace_size(const lora_kv_cache_desc* cache, const lora_kv_batch* batch, int32_t num_q_heads,
                                   size_t* bytes) {
    if (bytes == nullptr) return LORA_EINVAL;
    lora_status st = check_sizes(cache, batch);
    if (st != LORA_OK) return st;
    if (num_q_heads < 0 || num_q_heads % cache->num_kv_heads != 0) return LORA_EINVAL;
    if (num_q_heads > 65536) return LORA_ETOOBIG;
    *bytes = workspace_bytes();
    return LORA_OK;
}

lora_status lora_kv_workspace_init(void* ws, size_t ws_bytes, void* stream) {
    if (ws == nullptr || ((uintptr_t)ws & 255u) != 0 || ws_bytes < sizeof(WsHeader)) return LORA_EWORKSPACE;
    return cuda_status(cudaMemsetAsync(ws, 0, ws_bytes, (cudaStream_t)stream));
}

lora_status lora_kv_append(const lora_kv_cache_desc* cache, const lora_kv_batch* batch, const void* q, int64_t ldq,
                           void* q_out, int64_t ldqo, int32_t num_q_heads, const void* k, int64_t ldk, const void* v,
                           int64_t ldv, const lora_rope* rope, void* ws, size_t ws_bytes, void* stream) {
    lora_status st = check_call(cache, batch, ws, ws_bytes, sizeof(WsHeader));
    if (st != LORA_OK) return st;
    const int64_t dim = cache->head_dim, cols = cache->num_kv_heads * dim;
    if (num_q_heads < 0 || rope == nullptr || rope->reserved != 0) return LORA_EINVAL;
    if (num_q_heads > 65536) return LORA_ETOOBIG;
    if (rope->rot_dim < 0 || rope->rot_dim > dim || rope->rot_dim % 16 != 0 ||
        (rope->style != LORA_ROPE_HALVES && rope->style != LORA_ROPE_PAIRS))
        return LORA_EINVAL;
    if (rope->rot_dim > 0) {
        if (rope->cos == nullptr || rope->sin == nullptr || rope->max_pos <= 0) return LORA_EINVAL;
        if (!aligned16(rope->cos) || !aligned16(rope->sin)) return LORA_EALIGN;
    }
    if (!aligned4(rope->positions)) return LORA_EALIGN;
    if (batch->T == 0 || batch->n_seq == 0) return LORA_OK;
    if (num_q_heads > 0) {
        if ((st = check_rows(q, ldq, num_q_heads * dim)) != LORA_OK) return st;
        if ((st = check_rows(q_out, ldqo, num_q_heads * dim)) != LORA_OK) return st;
        if (q == q_out && ldq != ldqo) return LORA_EINVAL;
    }
    if ((st = check_rows(k, ldk, cols)) != LORA_OK) return st;
    if ((st = check_rows(v, ldv, cols)) != LORA_OK) return st;
    DeviceInfo* di = nullptr;
    if ((st = device_info(&di)) != LORA_OK) return st;
    AppendParams p;
    p.v = view_of(cache, batch, ws);
    p.q = reinterpret_cast<const __nv_bfloat16*>(q);
    p.q_out = reinterpret_cast<__nv_bfloat16*>(q_out);
    p.k = reinterpret_cast<const __nv_bfloat16*>(k);
    p.val = reinterpret_cast<const __nv_bfloat16*>(v);
    p.ldq = ldq;
    p.ldqo = ldqo;
    p.ldk = ldk;
    p.ldv = ldv;
    p.cos = rope->cos;
    p.sin = rope->sin;
    p.positions = rope->positions;
    p.max_pos = rope->max_pos;
    p.rot_dim = rope->rot_dim;
    p.style = rope->style;
    p.q_heads = num_q_heads;
    const int per_step = 256 / cache->head_dim;
    const int steps = (num_q_heads + 2 * cache->num_kv_heads + per_step - 1) / per_step;
    p.per_warp = steps_per_warp(di, batch->T, steps);
    const int64_t warps = (int64_t)batch->T * ((steps + p.per_warp - 1) / p.per_warp);
    return by_shape<Append>(cache, p, dim3((unsigned)((warps + kAppendWarps - 1) / kAppendWarps)), (cudaStream_t)stream);
}

lora_status lora_kv_read(const lora_kv_cache_desc* cache, const lora_kv_batch* batch, void* k_out, int64_t ldk,
                         void* v_out, int64_t ldv, void* ws, size_t ws_bytes, void* stream) {
    lora_status st = check_call(cache, batch, ws, ws_bytes, sizeof(WsHeader));
    if (st != LORA_OK) return st;
    if (batch->T == 0 || batch->n_seq == 0) return LORA_OK;
    const int64_t cols = (int64_t)cache->num_kv_heads * cache->head_dim;
    if ((st = check_rows(k_out, ldk, cols)) != LORA_OK) return st;
    if ((st = check_rows(v_out, ldv, cols)) != LORA_OK) return st;
    DeviceInfo* di = nullptr;
    if ((st = device_info(&di)) != LORA_OK) return st;
    ReadParams p;
    p.v = view_of(cache, batch, ws);
    p.k = reinterpret_cast<__nv_bfloat16*>(k_out);
    p.val = reinterpret_cast<__nv_bfloat16*>(v_out);
    p.ldk = ldk;
    p.ldv = ldv;
    const int per_step = 256 / cache->head_dim;
    const int steps = (2 * cache->num_kv_heads + per_step - 1) / per_step;
    p.per_warp = steps_per_warp(di, batch->T, steps);
    const int64_t warps = (int64_t)batch->T * ((steps + p.per_warp - 1) / p.per_warp);
    return by_shape<Read>(cache, p, dim3((unsigned)((warps + kAppendWarps - 1) / kAppendWarps)), (cudaStream_t)stream);
}

lora_status lora_kv_attend(const lora_kv_cache_desc* cache, const lora_kv_batch* batch, const void* q, int64_t ldq,
                           int32_t num_q_heads, float softmax_scale, void* out, int64_t ldo, float* lse, void* ws,
                           size_t ws_bytes, void* stream) {
    lora_status st = check_sizes(cache, batch);
    if (st != LORA_OK) return st;
    if (num_q_heads <= 0 || num_q_heads % cache->num_kv_heads != 0 || !(softmax_scale > 0.f && softmax_scale <= 3.4e38f))
        return LORA_EINVAL;
    if (num_q_heads > 65536) return LORA_ETOOBIG;
    if ((st = check_call(cache, batch, ws, ws_bytes, workspace_bytes())) != LORA_OK) return st;
    if (batch->T == 0 || batch->n_seq == 0) return LORA_OK;
    const int64_t cols = (int64_t)num_q_heads * cache->head_dim;
    if ((st = check_rows(q, ldq, cols)) != LORA_OK) return st;
    if ((st = check_rows(out, ldo, cols)) != LORA_OK) return st;
    if (!aligned4(lse)) return LORA_EALIGN;
    AttendParams p;
    p.v = view_of(cache, batch, ws);
    p.q = reinterpret_cast<const __nv_bfloat16*>(q);
    p.out = reinterpret_cast<__nv_bfloat16*>(out);
    p.lse = lse;
    p.ldq = ldq;
    p.ldo = ldo;
    p.q_heads = num_q_heads;
    p.rep = num_q_heads / cache->num_kv_heads;
    p.scale = softmax_scale;
    p.tickets = reinterpret_cast<uint32_t*>(reinterpret_cast<char*>(ws) + sizeof(WsHeader));
    p.part = reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + kStepPartAt);
    cudaStream_t cs = (cudaStream_t)stream;
    // requests with many packed rows take the tensor-core tiles, the others the decode kernel:
    // a launch each (how many rows a request has only the device knows)
    const int32_t many = (pre_min_packed(cache->head_dim, (int64_t)batch->n_seq * cache->num_kv_heads) + p.rep - 1) / p.rep;
    if (cache->group == cache->head_dim && batch->max_q >= many) {
        p.v.rows_lo = many;
        if ((st = cache->head_dim == 128 ? prefill<128>(p, cs) : prefill<64>(p, cs)) != LORA_OK) return st;
        p.v.rows_lo = 0;
        p.v.rows_hi = many - 1;
    }
    const bool narrow = std::min<int64_t>(batch->max_q, p.v.rows_hi) * p.rep <= 8;
    return narrow ? attend_by_shape<1>(cache, p, cs) : attend_by_shape<2>(cache, p, cs);
}

}  // extern "C"
