// C ABI of the products with 4-bit weights (include/lora_w4.h): argument checks and launch.
#include <string.h>

#include <algorithm>

#include "host.h"
#include "w4_matvec.cuh"
#include "w4_wide.cuh"

using namespace lora;
using namespace lora::host;

namespace {

lora_status check_sizes(const lora_w4_problem* probs, int32_t nprob, int32_t T) {
    if (nprob < 0 || T < 0 || (nprob > 0 && probs == nullptr)) return LORA_EINVAL;
    if (nprob > LORA_W4_MAX_PROBLEMS || T > LORA_W4_MAX_ROWS) return LORA_ETOOBIG;
    for (int32_t i = 0; i < nprob; ++i) {
        const lora_w4_problem& p = probs[i];
        if (p.N <= 0 || p.K <= 0 || p.N % 8 != 0 || p.reserved != 0) return LORA_EINVAL;
        if ((p.group != 32 && p.group != 64 && p.group != 128) || p.K % p.group != 0) return LORA_EINVAL;
        if (p.N > (1 << 24) || p.K > (1 << 20)) return LORA_ETOOBIG;
    }
    return LORA_OK;
}

size_t workspace_bytes() { return align256(std::max(w4_workspace(2), wide_workspace(128))); }

// Blocks of a CTA: an equal share of all, or whole row tiles where the largest share of them
// is at most `join` blocks more (what joining a tile from parts costs a CTA).  Whole tiles
// need one K for all projections.
int32_t w4_per(const W4Params& p, int grid, int join) {
    const int32_t share = (p.total + grid - 1) / grid;
    const int32_t kb = p.prob[0].kblocks;
    for (int32_t i = 1; i < p.nprob; ++i)
        if (p.prob[i].kblocks != kb) return share;
    const int32_t whole = (p.total / kb + grid - 1) / grid * kb;
    return whole <= share + join ? whole : share;
}

template <int G, int NT>
lora_status launch(W4Params& p, cudaStream_t s) {
    DeviceInfo* di = nullptr;
    lora_status st = device_info(&di);
    if (st != LORA_OK) return st;
    constexpr size_t smem = w4_smem(G, NT);
    auto kern = w4_matvec_kernel<G, NT>;
    static thread_local const DeviceInfo* ready = nullptr;
    static thread_local int per_sm = 0;
    if (ready != di) {
        st = cuda_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
        if (st != LORA_OK) return st;
        st = cuda_status(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kW4Threads, smem));
        if (st != LORA_OK) return st;
        ready = di;
    }
    const int grid = std::min(di->sm_count * std::max(per_sm, 1), kW4MaxCtas);
    p.per = w4_per(p, grid, kW4JoinCost);
    kern<<<grid, kW4Threads, smem, s>>>(p);
    return cuda_status(cudaGetLastError());
}

// 2-D map of `rows` rows of `inner` elements, box {box0, box1}, zeros outside.
lora_status map2d(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* map, CUtensorMapDataType type, const void* base,
                  uint64_t inner, uint64_t rows, uint64_t pitch, uint32_t box0, uint32_t box1, CUtensorMapSwizzle swizzle) {
    const cuuint64_t dims[2] = {inner, rows};
    const cuuint64_t strides[1] = {pitch};
    const cuuint32_t box[2] = {box0, box1}, one[2] = {1, 1};
    const CUresult r = enc(map, type, 2, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r == CUDA_SUCCESS) return LORA_OK;
    g_last_cuda_error = 10000 + (int)r;
    return LORA_ECUDA;
}

template <int G, int N>
lora_status launch_wide(WideParams& w, cudaStream_t s) {
    DeviceInfo* di = nullptr;
    lora_status st = device_info(&di);
    if (st != LORA_OK) return st;
    PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    if ((st = encode_fn(&enc)) != LORA_OK) return st;
    for (int i = 0; i < w.p.nprob; ++i) {
        const W4Prob& pr = w.p.prob[i];
        st = map2d(enc, &w.codes[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, pr.codes, pr.K / 2, pr.N, pr.K / 2, kWideK / 2, kWideRows,
                   CU_TENSOR_MAP_SWIZZLE_128B);
        if (st != LORA_OK) return st;
        st = map2d(enc, &w.x[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, pr.x, pr.K, w.p.T, pr.ldx * 2, 64, N,
                   CU_TENSOR_MAP_SWIZZLE_128B);
        if (st != LORA_OK) return st;
        st = map2d(enc, &w.y[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, pr.y, pr.N, w.p.T, pr.ldy * 2, kWideRows, N,
                   CU_TENSOR_MAP_SWIZZLE_NONE);
        if (st != LORA_OK) return st;
    }
    constexpr size_t smem = wide_smem(N, G);
    auto kern = w4_wide_kernel<G, N>;
    static thread_local const DeviceInfo* ready = nullptr;
    if (ready != di) {
        st = cuda_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
        if (st != LORA_OK) return st;
        ready = di;
    }
    const int grid = std::min(di->sm_count, kWideMaxCtas);
    w.p.per = (w.p.total + grid - 1) / grid;
    kern<<<grid, wide_threads(N), smem, s>>>(w);
    return cuda_status(cudaGetLastError());
}

template <int G>
lora_status launch_group(WideParams& w, bool narrow, cudaStream_t s) {
    const int T = w.p.T;
    if (narrow) return T <= 8 ? launch<G, 1>(w.p, s) : launch<G, 2>(w.p, s);
    if (T <= 32) return launch_wide<G, 32>(w, s);
    return T <= 64 ? launch_wide<G, 64>(w, s) : launch_wide<G, 128>(w, s);
}

// All launches of a call.  `lost` and `limit_ns`: see WideParams.
lora_status run(const lora_w4_problem* probs, int32_t nprob, int32_t T, void* ws, size_t ws_bytes, void* stream, int32_t lost,
                uint64_t limit_ns) {
    lora_status st = check_sizes(probs, nprob, T);
    if (st != LORA_OK) return st;
    for (int32_t i = 0; i < nprob; ++i) {
        const lora_w4_problem& pr = probs[i];
        if (pr.x == nullptr || pr.y == nullptr || pr.codes == nullptr || pr.scales == nullptr) return LORA_EINVAL;
        if (!aligned16(pr.x) || !aligned16(pr.y) || !aligned16(pr.codes) || !aligned16(pr.scales) ||
            ((uintptr_t)pr.zeros & 3u) != 0 || pr.ldx % 8 != 0 || pr.ldy % 8 != 0)
            return LORA_EALIGN;
        if (pr.ldx < pr.K || pr.ldy < pr.N) return LORA_EINVAL;
    }
    if (nprob == 0 || T == 0) return LORA_OK;
    if (ws == nullptr || ((uintptr_t)ws & 255u) != 0 || ws_bytes < workspace_bytes()) return LORA_EWORKSPACE;
    // one launch per group size of the call and 128 rows
    static_assert(kW4K == kWideK, "both kernels' blocks are 256 of K");
    static thread_local WideParams w;
    DeviceInfo* di = nullptr;
    if ((st = device_info(&di)) != LORA_OK) return st;
    for (const int32_t group : {32, 64, 128}) {
        for (int32_t t0 = 0; t0 < T; t0 += 128) {
            memset(&w, 0, sizeof w);
            W4Params& p = w.p;
            p.T = std::min(T - t0, 128);
            int64_t wide_blocks = 0;
            for (int32_t i = 0; i < nprob; ++i)
                if (probs[i].group == group)
                    wide_blocks += (int64_t)((probs[i].N + kWideRows - 1) / kWideRows) * ((probs[i].K + kWideK - 1) / kWideK);
            const bool narrow = p.T <= 8 || (p.T <= kW4NarrowRows && wide_blocks < (int64_t)kW4WideBlocks * di->sm_count);
            const int32_t block_rows = narrow ? kW4Rows : kWideRows;
            int64_t total = 0;
            for (int32_t i = 0; i < nprob; ++i) {
                const lora_w4_problem& pr = probs[i];
                if (pr.group != group) continue;
                W4Prob& o = p.prob[p.nprob++];
                o.x = reinterpret_cast<const __nv_bfloat16*>(pr.x) + t0 * pr.ldx;
                o.y = reinterpret_cast<__nv_bfloat16*>(pr.y) + t0 * pr.ldy;
                o.codes = reinterpret_cast<const unsigned char*>(pr.codes);
                o.scales = reinterpret_cast<const unsigned char*>(pr.scales);
                o.zeros = reinterpret_cast<const unsigned char*>(pr.zeros);
                o.ldx = pr.ldx;
                o.ldy = pr.ldy;
                o.N = pr.N;
                o.K = pr.K;
                o.group = pr.group;
                o.kblocks = (pr.K + kW4K - 1) / kW4K;
                o.first = (int32_t)total;
                total += (int64_t)((pr.N + block_rows - 1) / block_rows) * o.kblocks;
                if (total > INT32_MAX) return LORA_ETOOBIG;
            }
            if (p.nprob == 0) break;
            p.total = (int32_t)total;
            p.tickets = reinterpret_cast<uint32_t*>(reinterpret_cast<char*>(ws) + sizeof(WsHeader));
            p.part = reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + kStepPartAt);
            w.err = &reinterpret_cast<WsHeader*>(ws)->err;
            w.limit_ns = limit_ns;
            w.lost = lost;
            cudaStream_t s = (cudaStream_t)stream;
            st = group == 32 ? launch_group<32>(w, narrow, s) : group == 64 ? launch_group<64>(w, narrow, s) : launch_group<128>(w, narrow, s);
            if (st != LORA_OK) return st;
        }
    }
    return LORA_OK;
}

}  // namespace

extern "C" {

lora_status lora_w4_workspace_size(const lora_w4_problem* probs, int32_t nprob, int32_t T, size_t* bytes) {
    if (bytes == nullptr) return LORA_EINVAL;
    lora_status st = check_sizes(probs, nprob, T);
    if (st != LORA_OK) return st;
    *bytes = workspace_bytes();
    return LORA_OK;
}

lora_status lora_w4_matvec(const lora_w4_problem* probs, int32_t nprob, int32_t T, void* ws, size_t ws_bytes,
                           void* stream) {
    return run(probs, nprob, T, ws, ws_bytes, stream, -1, kWaitLimitNs);
}

lora_status lora_debug_w4_lost_block(const lora_w4_problem* probs, int32_t nprob, int32_t T, int32_t block, uint64_t limit_ns,
                                     void* ws, size_t ws_bytes, void* stream) {
    if (T <= kW4NarrowRows || block < 0 || limit_ns < 1000000ull) return LORA_EINVAL;
    if (limit_ns > kWaitLimitNs) return LORA_ETOOBIG;
    return run(probs, nprob, T, ws, ws_bytes, stream, block, limit_ns);
}

}  // extern "C"
