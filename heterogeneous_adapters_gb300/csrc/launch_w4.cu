// C ABI of the products with 4-bit weights (include/lora_w4.h): argument checks and launch.
#include <string.h>

#include "host.h"
#include "w4_matvec.cuh"

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

}  // namespace

extern "C" {

lora_status lora_w4_workspace_size(const lora_w4_problem* probs, int32_t nprob, int32_t T, size_t* bytes) {
    if (bytes == nullptr) return LORA_EINVAL;
    lora_status st = check_sizes(probs, nprob, T);
    if (st != LORA_OK) return st;
    *bytes = sizeof(WsHeader);
    return LORA_OK;
}

lora_status lora_w4_matvec(const lora_w4_problem* probs, int32_t nprob, int32_t T, void* ws, size_t ws_bytes,
                           void* stream) {
    lora_status st = check_sizes(probs, nprob, T);
    if (st != LORA_OK) return st;
    if (ws == nullptr || ((uintptr_t)ws & 255u) != 0 || ws_bytes < sizeof(WsHeader)) return LORA_EWORKSPACE;
    if (nprob == 0 || T == 0) return LORA_OK;
    W4Params p;
    memset(&p, 0, sizeof p);
    for (int32_t i = 0; i < nprob; ++i) {
        const lora_w4_problem& pr = probs[i];
        if (pr.x == nullptr || pr.y == nullptr || pr.codes == nullptr || pr.scales == nullptr) return LORA_EINVAL;
        if (!aligned16(pr.x) || !aligned16(pr.y) || !aligned16(pr.codes) || !aligned16(pr.scales) ||
            ((uintptr_t)pr.zeros & 3u) != 0 || pr.ldx % 8 != 0 || pr.ldy % 8 != 0)
            return LORA_EALIGN;
        if (pr.ldx < pr.K || pr.ldy < pr.N) return LORA_EINVAL;
        p.prob[i] = pr;
        p.first[i + 1] = p.first[i] + (pr.N + kW4Warps - 1) / kW4Warps;
    }
    p.nprob = nprob;
    p.T = T;
    p.err = &reinterpret_cast<WsHeader*>(ws)->err;
    w4_matvec_kernel<<<dim3(p.first[nprob], (T + kW4Rows - 1) / kW4Rows), kW4Warps * 32, 0, (cudaStream_t)stream>>>(p);
    return cuda_status(cudaGetLastError());
}

}  // extern "C"
