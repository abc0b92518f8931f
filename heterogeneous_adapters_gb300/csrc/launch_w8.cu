// C ABI of an 8-bit base model's operators (include/lora_w8.h): argument checks and launch.
#include <string.h>

#include <algorithm>

#include "host.h"
#include "q8_rows.cuh"
#include "w8_narrow.cuh"

using namespace lora;
using namespace lora::host;

namespace {

// ---------------------------------------------------------------------------- rows in 8 bits
// A 16-bit matrix of rows of width d.
lora_status check_rows(const void* p, int64_t ld, int32_t d) {
    if (p == nullptr) return LORA_EINVAL;
    if (!aligned16(p) || ld % 8 != 0) return LORA_EALIGN;
    return ld >= d ? LORA_OK : LORA_EINVAL;
}

lora_status check_out(const lora_q8_rows& o, int32_t d) {
    if (o.codes == nullptr || o.scales == nullptr || o.reserved != 0) return LORA_EINVAL;
    if (o.x_kind != LORA_Q8_X_HELD && o.x_kind != LORA_Q8_X_FULL) return LORA_EINVAL;
    if (!aligned16(o.codes) || o.ldc % 16 != 0 || ((uintptr_t)o.scales & 3u) != 0) return LORA_EALIGN;
    if (o.ldc < d) return LORA_EINVAL;
    return o.x != nullptr ? check_rows(o.x, o.ldx, d) : LORA_OK;
}

lora_status check_shape(int32_t T, int32_t d) {
    if (T < 0 || d <= 0 || d % 16 != 0) return LORA_EINVAL;
    return T > LORA_Q8_MAX_ROWS || d > LORA_Q8_MAX_WIDTH ? LORA_ETOOBIG : LORA_OK;
}

// In place is fine where both sides have one pitch.
bool pitch_differs(const void* a, int64_t lda, const void* b, int64_t ldb) { return a != nullptr && a == b && lda != ldb; }

Q8Out out_of(const lora_q8_rows& o) {
    return {reinterpret_cast<unsigned char*>(o.codes), o.scales, reinterpret_cast<__nv_bfloat16*>(o.x), o.ldc, o.ldx,
            o.x_kind == LORA_Q8_X_FULL};
}

// Eights of a row a thread, and threads of a row.
struct RowShape {
    int v, threads;
};
RowShape row_shape(int32_t d) {
    const int eights = d / 8, v = eights <= 512 ? 1 : eights <= 1024 ? 2 : 4;
    return {v, ((eights + v - 1) / v + 31) / 32 * 32};
}

template <int ACT>
void launch_gate(const Q8GateParams& q, RowShape sh, int32_t T, cudaStream_t s) {
    if (sh.v == 1) q8_gate_kernel<1, ACT><<<T, sh.threads, 0, s>>>(q);
    else if (sh.v == 2) q8_gate_kernel<2, ACT><<<T, sh.threads, 0, s>>>(q);
    else q8_gate_kernel<4, ACT><<<T, sh.threads, 0, s>>>(q);
}

// ---------------------------------------------------------------------------- products
lora_status check_sizes(const lora_w8_problem* probs, int32_t nprob, int32_t T) {
    if (nprob < 0 || T < 0 || (nprob > 0 && probs == nullptr)) return LORA_EINVAL;
    if (nprob > LORA_W8_MAX_PROBLEMS || T > LORA_W8_MAX_ROWS) return LORA_ETOOBIG;
    for (int32_t i = 0; i < nprob; ++i) {
        const lora_w8_problem& p = probs[i];
        if (p.N <= 0 || p.K <= 0 || p.N % 8 != 0 || p.K % 16 != 0) return LORA_EINVAL;
        if (p.N > (1 << 24) || p.K > LORA_W8_MAX_K) return LORA_ETOOBIG;
    }
    return LORA_OK;
}

size_t workspace_bytes(const lora_w8_problem* probs, int32_t nprob, int32_t T) {
    (void)probs; (void)nprob; (void)T;
    return align256(kStepPartAt);
}

}  // namespace

extern "C" {

lora_status lora_q8_norm(const lora_q8_norm_desc* n, int32_t T, void* stream) {
    if (n == nullptr) return LORA_EINVAL;
    lora_status st = check_shape(T, n->d);
    if (st != LORA_OK) return st;
    if (!(n->eps >= 1e-30f) || !(n->eps <= 3.4e38f)) return LORA_EINVAL;
    if ((st = check_rows(n->x, n->ldx, n->d)) != LORA_OK) return st;
    if (n->residual != nullptr && (st = check_rows(n->residual, n->ldr, n->d)) != LORA_OK) return st;
    if (n->sum != nullptr && n->residual == nullptr) return LORA_EINVAL;
    if (n->sum != nullptr && (st = check_rows(n->sum, n->lds, n->d)) != LORA_OK) return st;
    if ((st = check_rows(n->weight, n->d, n->d)) != LORA_OK) return st;
    if (pitch_differs(n->sum, n->lds, n->x, n->ldx) || pitch_differs(n->sum, n->lds, n->residual, n->ldr)) return LORA_EINVAL;
    if ((st = check_out(n->out, n->d)) != LORA_OK) return st;
    if (T == 0) return LORA_OK;
    const Q8NormParams q = {reinterpret_cast<const __nv_bfloat16*>(n->x), reinterpret_cast<const __nv_bfloat16*>(n->residual),
                            reinterpret_cast<__nv_bfloat16*>(n->sum), reinterpret_cast<const __nv_bfloat16*>(n->weight),
                            n->ldx, n->ldr, n->lds, n->eps, n->d, out_of(n->out)};
    const RowShape sh = row_shape(n->d);
    cudaStream_t s = (cudaStream_t)stream;
    if (sh.v == 1) q8_norm_kernel<1><<<T, sh.threads, 0, s>>>(q);
    else if (sh.v == 2) q8_norm_kernel<2><<<T, sh.threads, 0, s>>>(q);
    else q8_norm_kernel<4><<<T, sh.threads, 0, s>>>(q);
    return cuda_status(cudaGetLastError());
}

lora_status lora_q8_gate(const lora_q8_gate_desc* n, int32_t T, void* stream) {
    if (n == nullptr) return LORA_EINVAL;
    lora_status st = check_shape(T, n->d);
    if (st != LORA_OK) return st;
    if (n->act < LORA_ACT_NONE || n->act > LORA_ACT_GELU_TANH) return LORA_EINVAL;
    if ((st = check_rows(n->gate, n->ldg, n->d)) != LORA_OK) return st;
    if (n->up != nullptr && (st = check_rows(n->up, n->ldu, n->d)) != LORA_OK) return st;
    if ((st = check_out(n->out, n->d)) != LORA_OK) return st;
    if (pitch_differs(n->out.x, n->out.ldx, n->gate, n->ldg) || pitch_differs(n->out.x, n->out.ldx, n->up, n->ldu)) return LORA_EINVAL;
    if (T == 0) return LORA_OK;
    const Q8GateParams q = {reinterpret_cast<const __nv_bfloat16*>(n->gate), reinterpret_cast<const __nv_bfloat16*>(n->up),
                            n->ldg, n->ldu, n->d, out_of(n->out)};
    const RowShape sh = row_shape(n->d);
    cudaStream_t s = (cudaStream_t)stream;
    switch (n->act) {
        case LORA_ACT_NONE: launch_gate<LORA_ACT_NONE>(q, sh, T, s); break;
        case LORA_ACT_SILU: launch_gate<LORA_ACT_SILU>(q, sh, T, s); break;
        case LORA_ACT_GELU: launch_gate<LORA_ACT_GELU>(q, sh, T, s); break;
        default: launch_gate<LORA_ACT_GELU_TANH>(q, sh, T, s);
    }
    return cuda_status(cudaGetLastError());
}

lora_status lora_w8_workspace_size(const lora_w8_problem* probs, int32_t nprob, int32_t T, size_t* bytes) {
    if (bytes == nullptr) return LORA_EINVAL;
    lora_status st = check_sizes(probs, nprob, T);
    if (st != LORA_OK) return st;
    *bytes = workspace_bytes(probs, nprob, T);
    return LORA_OK;
}

lora_status lora_w8_matmul(const lora_w8_problem* probs, int32_t nprob, int32_t T, void* ws, size_t ws_bytes, void* stream) {
    lora_status st = check_sizes(probs, nprob, T);
    if (st != LORA_OK) return st;
    for (int32_t i = 0; i < nprob; ++i) {
        const lora_w8_problem& pr = probs[i];
        if (pr.x == nullptr || pr.x_scales == nullptr || pr.y == nullptr || pr.w == nullptr || pr.w_scales == nullptr) return LORA_EINVAL;
        if (!aligned16(pr.x) || !aligned16(pr.y) || !aligned16(pr.w) || ((uintptr_t)pr.x_scales & 3u) != 0 ||
            ((uintptr_t)pr.w_scales & 3u) != 0 || pr.ldx % 16 != 0 || pr.ldy % 8 != 0)
            return LORA_EALIGN;
        if (pr.ldx < pr.K || pr.ldy < pr.N) return LORA_EINVAL;
    }
    if (nprob == 0 || T == 0) return LORA_OK;
    if (ws == nullptr || ((uintptr_t)ws & 255u) != 0 || ws_bytes < workspace_bytes(probs, nprob, T)) return LORA_EWORKSPACE;
    static thread_local W8Params p;
    memset(&p, 0, sizeof p);
    p.T = T;
    p.nprob = nprob;
    int64_t total = 0;
    for (int32_t i = 0; i < nprob; ++i) {
        const lora_w8_problem& pr = probs[i];
        p.prob[i] = {reinterpret_cast<const unsigned char*>(pr.x), pr.x_scales, reinterpret_cast<__nv_bfloat16*>(pr.y),
                     reinterpret_cast<const unsigned char*>(pr.w), pr.w_scales, pr.ldx, pr.ldy, pr.N, pr.K, (int32_t)total};
        total += (pr.N + kW8Rows - 1) / kW8Rows;
    }
    p.total = (int32_t)total;
    cudaStream_t s = (cudaStream_t)stream;
    const int nt = T <= 8 ? 1 : T <= 16 ? 2 : 4;
    const dim3 grid((unsigned)total, (unsigned)((T + 8 * nt - 1) / (8 * nt)));
    if (nt == 1) w8_narrow_kernel<1><<<grid, kW8Threads, 0, s>>>(p);
    else if (nt == 2) w8_narrow_kernel<2><<<grid, kW8Threads, 0, s>>>(p);
    else w8_narrow_kernel<4><<<grid, kW8Threads, 0, s>>>(p);
    return cuda_status(cudaGetLastError());
}

}  // extern "C"
