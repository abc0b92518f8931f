/* lora_kv.h - the 4-bit KV cache beside the adapters (liblora.so).
 *
 * The unified pool holds two kinds of tenants, adapter rows and KV blocks ("S-LoRA: Serving
 * Thousands of Concurrent LoRA Adapters" (fdeinterviews), "Unified paging").  lora.h serves
 * the first kind; these calls fill and read the second: a paged cache of keys and values in
 * 4 bits, appended to with the rotary positions applied on the way, and the attention that
 * reads it.  Conventions (streams, status codes, the device error word, no allocation, no
 * host synchronisation, bounded waits, threading) are those of lora.h.
 *
 * Format.  For each token, KV head and K or V, every `group` neighbouring values share a
 * scale and an offset (f16); a 4-bit code c in 0..15 stands for
 *
 *     value = scale * (c - 8) + offset,    scale >= 0.
 *
 * A block holds block_tokens tokens of every KV head of one layer as tiles of 16 tokens of
 * one head, [num_kv_heads][block_tokens / 16] tiles, each
 *     K codes   [head_dim / 32][16 tokens][16 bytes]   (byte j: dims 2j low half, 2j + 1 high)
 *     V codes   likewise
 *     K params  [head_dim / group][16 tokens] of (f16 scale, f16 offset)
 *     V params  likewise
 * i.e. 16 * (head_dim + 8 * head_dim / group) bytes.  Block b starts block_stride * b bytes
 * after `blocks`.  To keep the blocks in a lora_pool's pages, pass the pool's pages and a
 * block_stride of m pages (m * 2 * h bytes) of at least lora_kv_block_bytes: block b then
 * is the run of pool pages [b m, (b + 1) m).  Bytes of a block that hold no token yet are
 * never used, whatever they contain. */
#ifndef LORA_KV_GB300_H
#define LORA_KV_GB300_H

#include "lora.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The cache of one layer (plain values, read during the call only). */
typedef struct {
    void* blocks;          /* device, 16-byte aligned                                  */
    int64_t num_blocks;
    int64_t block_stride;  /* bytes, a multiple of 16, >= lora_kv_block_bytes          */
    int32_t block_tokens;  /* a multiple of 16, at most 1024                           */
    int32_t num_kv_heads;  /* at most LORA_KV_MAX_HEADS                                */
    int32_t head_dim;      /* 64 or 128                                                */
    int32_t group;         /* 32 or head_dim                                           */
} lora_kv_cache_desc;

#define LORA_KV_MAX_HEADS 256
#define LORA_KV_MAX_SEQS 16384

/* The batch: request s owns rows [q_start[s], q_start[s + 1]) of q, k, v and the outputs
 * (q_start[0] >= 0, non-decreasing, q_start[n_seq] <= T; a request may have no rows) and
 * the tokens 0 .. kv_len[s] - 1 of the cache, of which its rows are the last ones: the
 * request's row i (of m) is token kv_len[s] - m + i.  Token t lies in block
 * block_table[s][t / block_tokens].  All arrays are device memory, 4-byte aligned (as are
 * positions and lse below, else LORA_EALIGN).  Entries of the table beyond a request's
 * tokens are not read. */
typedef struct {
    const int32_t* q_start;      /* [n_seq + 1]                                        */
    const int32_t* kv_len;       /* [n_seq]                                            */
    const int32_t* block_table;  /* [n_seq][max_blocks]                                */
    int32_t n_seq;
    int32_t T;                   /* rows of the batch's tensors                        */
    int32_t max_blocks;
    int32_t max_q;               /* the most rows a request has (host knowledge)       */
} lora_kv_batch;

/* Rotary positions.  Row r at position p (its cache token, or positions[r] if given) has
 * the first rot_dim values of each head turned: (a, b) -> (a c - b s, b c + a s) with
 * c = cos[p][i], s = sin[p][i] for pair i, in fp32, each product and sum rounded. */
enum { LORA_ROPE_HALVES = 0,    /* pair i = values (i, i + rot_dim / 2)               */
       LORA_ROPE_PAIRS = 1 };   /* pair i = values (2 i, 2 i + 1)                     */
typedef struct {
    const float* cos;            /* device [max_pos][rot_dim / 2], 16-byte aligned     */
    const float* sin;
    const int32_t* positions;    /* device [T], or NULL: the cache token               */
    int32_t max_pos;
    int32_t rot_dim;             /* 0 (no rotation) .. head_dim, a multiple of 16      */
    int32_t style;
    int32_t reserved;            /* 0                                                  */
} lora_rope;

/* Device error bit beside those of lora.h: a request's tokens outside its block table, a
 * block id outside the cache, a position outside the rotation tables, or a request with
 * more than max_q rows.  A request with too many rows, or whose q_start entries decrease or
 * leave [0, T] (LORA_DERR_SEGMENT), has its rows left alone by every call.  Otherwise a row
 * whose block or position is missing is not appended (nor its q_out row written) and reads
 * back as zeros, and attention treats the tokens of a missing block as absent. */
#define LORA_DERR_KV 0x40u

/* Bytes of one block of this shape.  LORA_EINVAL / LORA_ETOOBIG for a shape not supported. */
lora_status lora_kv_block_bytes(int32_t block_tokens, int32_t num_kv_heads, int32_t head_dim, int32_t group,
                                size_t* bytes);

/* Bytes of device workspace that the calls below need for batches of at most this batch's
 * n_seq, T and max_q with num_q_heads query heads (the arrays of the batch are not read).  It holds the device
 * error word (lora_get_device_error) and the partial results of long rows.  The workspace
 * of lora_segment holds the batch's grouping: give these calls one of their own. */
lora_status lora_kv_workspace_size(const lora_kv_cache_desc* cache, const lora_kv_batch* batch, int32_t num_q_heads,
                                   size_t* bytes);
/* Prepares a fresh workspace: once, before its first use, on the stream that will use it. */
lora_status lora_kv_workspace_init(void* ws, size_t ws_bytes, void* stream);

/* Appends the batch's rows to the cache: turns q (into q_out) and k by their positions and
 * stores k and v in 4 bits.  For the `group` fp32 values x of one group
 *     scale  = f16((max x - min x) * (1/15)),   offset = f16(min x + 8 scale),
 *     c      = clamp(rint((x - offset) * (1 / scale)), -8, 7) + 8        (c = 8 if scale = 0),
 * scale and offset limited to f16's finite range; a group that holds a value that is not
 * finite is stored with NaN for both, and so reads back as NaN.
 *   q      bf16 [T][ldq], num_q_heads * head_dim columns; num_q_heads 0: no q (q, q_out NULL)
 *   q_out  bf16 [T][ldqo]; may be q itself with ldqo = ldq
 *   k, v   bf16 [T][ldk], [T][ldv], num_kv_heads * head_dim columns
 * (16-byte aligned, ld % 8 == 0; slices of one fused projection's output will do.)  A block
 * that requests share must not be appended to by more than one of them in a call. */
lora_status lora_kv_append(const lora_kv_cache_desc* cache, const lora_kv_batch* batch, const void* q, int64_t ldq,
                           void* q_out, int64_t ldqo, int32_t num_q_heads, const void* k, int64_t ldk, const void* v,
                           int64_t ldv, const lora_rope* rope, void* ws, size_t ws_bytes, void* stream);

/* Reads the batch's rows back from the cache as bf16: what attention sees of them (the
 * keys as stored, after their rotation).  A batch whose rows are all tokens of a request
 * exports the request. */
lora_status lora_kv_read(const lora_kv_cache_desc* cache, const lora_kv_batch* batch, void* k_out, int64_t ldk,
                         void* v_out, int64_t ldv, void* ws, size_t ws_bytes, void* stream);

/* Causal attention of the batch's rows over the cache (query head j reads KV head
 * j / (num_q_heads / num_kv_heads)): with t running over the tokens 0 .. the row's own,
 *     a_t = softmax_scale * (q . k_t),   out = sum_t exp(a_t - lse) v_t,   lse = log sum_t exp(a_t).
 *   q, out  bf16 [T][ldq], [T][ldo]; lse: f32 [T][num_q_heads], or NULL
 * A row with no token (kv_len smaller than the request's rows) gets zeros and lse = -inf.
 * Scores, softmax statistics and sums are fp32.  A token's weight in the output is rounded to 11
 * bits once (2^-11 of itself), and v by as much (where a request has many rows, v over a power
 * of two to f16; where it has few, a V scale below 2^-14 of its offset counts as that).  Codes
 * meet the weights in f16, whose steps end at 2^-28 of a row's largest p |v|: a token may be
 * off by that much beside.  The result does not depend on how the device schedules the work.
 * A token whose V is not a number makes the outputs of its group so, for the rows that see it.
 * num_q_heads is a multiple of num_kv_heads.  Requests with many rows (chunks of prompts) are
 * served fast where group = head_dim; with groups of 32 the cache is read and unpacked once per
 * 16 rows times query heads of a KV head (three chunks of 300 to 512 rows over 3,111 to 6,000
 * tokens, 32 query and 8 KV heads of 128: 137 us and 741 us). */
lora_status lora_kv_attend(const lora_kv_cache_desc* cache, const lora_kv_batch* batch, const void* q, int64_t ldq,
                           int32_t num_q_heads, float softmax_scale, void* out, int64_t ldo, float* lse, void* ws,
                           size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* LORA_KV_GB300_H */
