"""GB300-native multi-LoRA delta: BGMV (decode) and SGMV (prefill) over a unified
paged adapter pool, as hand-written sm_103a CUDA kernels behind a C ABI
(include/lora.h, liblora.so), and the host runtime around them: the adapter cache over
the pool's pages and the batch scheduler (include/lora_runtime.h).  This package holds
the sources (csrc/), the in-tree build, the ctypes binding and the byte/flop model used
to report throughput against the HBM roofline.  Around the delta: a paged KV cache in 4
bits with its attention (include/lora_kv.h) and products with 4-bit weights
(include/lora_w4.h)."""
from . import costmodel
from ._binding import (DERR, LORA_ENOSPACE, LORA_MAX_PROBLEMS_PER_LAUNCH, LORA_MAX_RANK,
                       LORA_MAX_SEGMENTS, LORA_NOALLOC_MAX_TOKENS, LORA_STAGE_MAX_RUNS, LORA_UNIT_ABSENT,
                       LORA_UNIT_LOADING,
                       LORA_UNIT_READY, AdapterCache, LoraError, Pool, Scheduler, apply_mixed, bgmv,
                       bgmv_noalloc, debug_delta_with_t, debug_page_list, debug_wait_limit, delta_grouped,
                       expand, get_device_error, shrink,
                       lib, segment, sgmv, stage_pages, stage_pages_ce, workspace_init, workspace_size,
                       workspace_view)
from ._binding import (LORA_KV_MAX_HEADS, LORA_KV_MAX_SEQS, LORA_ROPE_HALVES, LORA_ROPE_PAIRS,
                       LORA_W4_MAX_PROBLEMS, LORA_W4_MAX_ROWS, KvBatch, KvCache, Rope, debug_w4_lost_block, kv_append,
                       kv_attend, kv_block_bytes, kv_read, kv_workspace_init, kv_workspace_size, w4_matvec, w4_problems,
                       w4_workspace_size)

__all__ = ["costmodel", "DERR", "LORA_ENOSPACE", "LORA_MAX_PROBLEMS_PER_LAUNCH", "LORA_MAX_RANK",
           "LORA_MAX_SEGMENTS", "LORA_NOALLOC_MAX_TOKENS", "LORA_STAGE_MAX_RUNS", "LORA_UNIT_ABSENT",
           "LORA_UNIT_LOADING",
           "LORA_UNIT_READY", "AdapterCache", "LoraError", "Pool", "Scheduler", "apply_mixed",
           "bgmv", "bgmv_noalloc", "debug_delta_with_t", "debug_page_list", "debug_wait_limit",
           "delta_grouped", "expand", "shrink",
           "get_device_error", "lib", "segment", "sgmv", "stage_pages", "stage_pages_ce", "workspace_init",
           "workspace_size", "workspace_view",
           "LORA_KV_MAX_HEADS", "LORA_KV_MAX_SEQS", "LORA_ROPE_HALVES", "LORA_ROPE_PAIRS",
           "LORA_W4_MAX_PROBLEMS", "LORA_W4_MAX_ROWS", "KvBatch", "KvCache", "Rope", "debug_w4_lost_block",
           "kv_append", "kv_attend", "kv_block_bytes", "kv_read", "kv_workspace_init", "kv_workspace_size", "w4_matvec", "w4_problems",
           "w4_workspace_size"]
