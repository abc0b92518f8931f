/* lora_w8.h - an 8-bit base model's layers beside 16-bit adapters (liblora.so).
 *
 * Products y = x W^T of 8-bit integers, for decode batches and whole prompts, and the two
 * operators that leave rows in the 8 bits that these products read: the residual's addition
 * with the root-mean-square norm (before q/k/v and before the MLP), and the gated activation
 * (before the MLP's last projection; without an activation it puts any rows into 8 bits, such
 * as the attention's output).  The delta of lora.h is added to the products' y, and reads the
 * same rows in 16 bits ("Multi-LoRA serving: S-LoRA, Punica and adapter batching" (pofe.ai),
 * the paragraph on quantised bases with 16-bit adapters).  Because the deltas are added to the
 * two projections of the MLP before their activation, that is not part of the product.
 * Conventions (streams, status codes, no allocation, no host synchronisation, bounded waits,
 * threading) are those of lora.h.
 *
 * A row y of width d in 8 bits:
 *     scale = max |y| / 127,   code_i = rint(y_i / scale)  (ties to even; 0 if scale = 0),
 * and a code c stands for scale * c.  y and scale are fp32.  A row that holds a value that is
 * not finite (or whose values leave fp32's range on the way) has the scale NaN and codes 0, and
 * so stands for NaN in every product. */
#ifndef LORA_W8_GB300_H
#define LORA_W8_GB300_H

#include "lora.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LORA_Q8_MAX_WIDTH 32768
#define LORA_Q8_MAX_ROWS (1 << 24)
#define LORA_W8_MAX_ROWS 65536
#define LORA_W8_MAX_PROBLEMS 16
#define LORA_W8_MAX_K 65536

/* Rows in 8 bits, and the same rows in bf16 for the adapters of the layer. */
enum { LORA_Q8_X_HELD = 0,       /* x = bf16(scale * code): what the base product sees, so that
                                    base and delta are the product with W + s B A           */
       LORA_Q8_X_FULL = 1 };     /* x = bf16(y)                                             */
typedef struct {
    void* codes;                 /* int8 [T][ldc], 16-byte aligned, ldc % 16 == 0           */
    float* scales;               /* [T], 4-byte aligned                                     */
    void* x;                     /* bf16 [T][ldx], 16-byte aligned, ldx % 8 == 0; or NULL   */
    int64_t ldc;
    int64_t ldx;
    int32_t x_kind;
    int32_t reserved;            /* 0                                                       */
} lora_q8_rows;

/* The norm: with h = bf16(x + residual) (x itself without a residual),
 *     y = h weight / sqrt(mean h^2 + eps),
 * left in 8 bits.  The sum of squares is fp32.  The codes are those of the exact quotients
 * (they depend on h weight alone, which is fp32: 0 below 2^-150); scales are within a few 2^-24 of theirs.
 * In the full x a value below 2^-64 of its row's largest may be 0. */
typedef struct {
    const void* x;               /* bf16 [T][ldx]                                           */
    const void* residual;        /* bf16 [T][ldr], or NULL                                  */
    void* sum;                   /* bf16 [T][lds]: h; NULL without a residual, or if unused.
                                    May be x or residual with its pitch                     */
    const void* weight;          /* bf16 [d]                                                */
    int64_t ldx;
    int64_t ldr;
    int64_t lds;
    float eps;                   /* 1e-30 .. 1                                              */
    int32_t d;                   /* a multiple of 16, at most LORA_Q8_MAX_WIDTH             */
    lora_q8_rows out;
} lora_q8_norm_desc;

/* The gated activation: y = act(gate) up (act(gate) without up), in fp32, left in 8 bits.  act(gate) is right to a
 * share of its own size (up to 4e-5 where it is smallest); one below 2^-126 may be 0. */
enum { LORA_ACT_NONE = 0, LORA_ACT_SILU = 1, LORA_ACT_GELU = 2, LORA_ACT_GELU_TANH = 3 };
typedef struct {
    const void* gate;            /* bf16 [T][ldg]                                           */
    const void* up;              /* bf16 [T][ldu], or NULL                                  */
    int64_t ldg;
    int64_t ldu;
    int32_t act;
    int32_t d;                   /* a multiple of 16, at most LORA_Q8_MAX_WIDTH             */
    lora_q8_rows out;            /* out.x may be gate or up with its pitch                  */
} lora_q8_gate_desc;

/* Rows 0 .. T - 1; T <= LORA_Q8_MAX_ROWS.  Arrays are 16-byte aligned with pitches that are
 * multiples of 8 and at least d (LORA_EALIGN, LORA_EINVAL); apart from the cases named above,
 * what is written overlaps nothing else. */
lora_status lora_q8_norm(const lora_q8_norm_desc* norm, int32_t T, void* stream);
lora_status lora_q8_gate(const lora_q8_gate_desc* gate, int32_t T, void* stream);

/* One projection, y[t, n] = bf16(x_scales[t] w_scales[n] sum_k x[t, k] w[n, k]). */
typedef struct {
    const void* x;               /* int8 [T][ldx], 16-byte aligned, ldx % 16 == 0           */
    const float* x_scales;       /* [T], 4-byte aligned                                     */
    void* y;                     /* bf16 [T][ldy], overwritten, 16-byte aligned, ldy % 8 == 0 */
    const void* w;               /* int8 [N][K], 16-byte aligned                            */
    const float* w_scales;       /* [N], 4-byte aligned                                     */
    int64_t ldx;
    int64_t ldy;
    int32_t N;                   /* a multiple of 8, at most 2^24                           */
    int32_t K;                   /* a multiple of 16, at most LORA_W8_MAX_K                 */
} lora_w8_problem;

/* Bytes of device workspace for the call: the device error word, partial sums and, for many
 * rows, x in the type that the tensor cores read; problems with the same x, ldx and K share
 * that.  (Other pointers are not read.)  A workspace serves calls of fewer rows too.  Prepare
 * it once with lora_kv_workspace_init (lora_kv.h); one workspace, large enough for all, may
 * serve the calls of lora_kv.h, lora_w4.h and this one. */
lora_status lora_w8_workspace_size(const lora_w8_problem* probs, int32_t nprob, int32_t T, size_t* bytes);

/* All projections of the call, at most LORA_W8_MAX_PROBLEMS, over the same T <=
 * LORA_W8_MAX_ROWS rows (their x may differ); at most 2^30 steps, as counted below (LORA_ETOOBIG).
 * What is written overlaps nothing else of the call.  Sums that stay below 2^24 on the way are
 * whole numbers, and y is theirs times the scales in fp32, rounded once, the same for any T;
 * larger sums are fp32 sums (whole numbers up to 8 rows, rounded to fp32 once). */
lora_status lora_w8_matmul(const lora_w8_problem* probs, int32_t nprob, int32_t T, void* ws, size_t ws_bytes,
                           void* stream);

/* Self-test of the bounded waits: lora_w8_matmul in which W of `step` (256 rows of a W by 128 of K,
 * counted K fastest, then the tiles along x, then those along W) never comes and every wait gives up
 * after limit_ns nanoseconds (1 ms .. 2 s, else LORA_EINVAL / LORA_ETOOBIG).  LORA_EINVAL for calls
 * whose kernel does not wait (up to 8 rows, and more where rows times W are few) and for a step past the call's last.
 * LORA_DERR_TIMEOUT is set, y is incomplete, and the workspace serves later calls as before. */
lora_status lora_debug_w8_lost_step(const lora_w8_problem* probs, int32_t nprob, int32_t T, int32_t step, uint64_t limit_ns,
                                    void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* LORA_W8_GB300_H */
