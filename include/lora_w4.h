/* lora_w4.h - products with 4-bit weights for decode batches (liblora.so).
 *
 * The projection that the delta of lora.h is added to: y = x W^T with the base weights in
 * 4 bits beside 16-bit adapters ("Multi-LoRA serving: S-LoRA, Punica and adapter batching"
 * (pofe.ai), the paragraph on quantised bases with 16-bit adapters).  Conventions are those
 * of lora.h. */
#ifndef LORA_W4_GB300_H
#define LORA_W4_GB300_H

#include "lora.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LORA_W4_MAX_ROWS 256
#define LORA_W4_MAX_PROBLEMS 16

/* One projection, y[t, n] = sum_k x[t, k] W[n, k], W[n, k] = scale[k / group, n] * (c[n, k] - zero[k / group, n]):
 *   x       bf16 [T][ldx]; y bf16 [T][ldy], overwritten (16-byte aligned, ld % 8 == 0)
 *   codes   uint8 [N][K / 2], 16-byte aligned; byte j: weight 2j in its low half, 2j + 1 high
 *   scales  f16 [K / group][N], 16-byte aligned
 *   zeros   uint8 [K / group][N / 2], low half first, 4-byte aligned; NULL: every zero is 8
 * N a multiple of 8, K a multiple of group, group 32, 64 or 128.  Products are exact and
 * summed in fp32; y is rounded to bf16 once. */
typedef struct {
    const void* x;
    void* y;
    int64_t ldx;
    int64_t ldy;
    const void* codes;
    const void* scales;
    const void* zeros;
    int32_t N;
    int32_t K;
    int32_t group;
    int32_t reserved;      /* 0                                                        */
} lora_w4_problem;

/* Bytes of device workspace for the call (the device error word and partial sums); the
 * pointers of the problems are not read.  Prepare it once with lora_kv_workspace_init
 * (lora_kv.h); one workspace, large enough for both, may serve those calls and this one. */
lora_status lora_w4_workspace_size(const lora_w4_problem* probs, int32_t nprob, int32_t T, size_t* bytes);

/* All projections of the call, at most LORA_W4_MAX_PROBLEMS, over the same T <=
 * LORA_W4_MAX_ROWS rows (their x may differ), in one launch per group size and 128 rows. */
lora_status lora_w4_matvec(const lora_w4_problem* probs, int32_t nprob, int32_t T, void* ws, size_t ws_bytes,
                           void* stream);

/* Self-test of the bounded waits: lora_w4_matvec (17 rows and more) for which the codes of
 * `block` of each launch (128 rows of a W by 256 of K, counted K fastest through the
 * projections of a group size) never come and every wait gives up after limit_ns nanoseconds
 * (1 ms .. 2 s, else LORA_EINVAL / LORA_ETOOBIG).  LORA_DERR_TIMEOUT is set, y is incomplete,
 * and the workspace serves later calls as before. */
lora_status lora_debug_w4_lost_block(const lora_w4_problem* probs, int32_t nprob, int32_t T, int32_t block, uint64_t limit_ns,
                                     void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* LORA_W4_GB300_H */
