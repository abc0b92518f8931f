"""ctypes binding of liblora.so: the same names as include/*.h, argument
marshalling only.  Every step of the path runs in the library's CUDA kernels;
there is no Python or CPU fallback: if the library is missing, loading fails.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
SO = os.path.join(_PKG, "liblora.so")

(LORA_OK, LORA_EINVAL, LORA_EALIGN, LORA_EWORKSPACE, LORA_ETOOBIG, LORA_ECUDA, LORA_EDEVICE,
 LORA_ENOSPACE) = range(8)
LORA_UNIT_ABSENT, LORA_UNIT_LOADING, LORA_UNIT_READY = range(3)
DERR = {0x1: "adapter", 0x2: "rank", 0x4: "page-table block", 0x8: "page", 0x10: "segment",
        0x20: "timeout", 0x40: "KV cache arrays"}
LORA_MAX_PROBLEMS_PER_LAUNCH = 256
LORA_MAX_SEGMENTS = 16384
LORA_MAX_RANK = 256
LORA_NOALLOC_MAX_TOKENS = 4096
LORA_STAGE_MAX_RUNS = 64
LORA_KV_MAX_HEADS = 256
LORA_KV_MAX_SEQS = 16384
LORA_ROPE_HALVES, LORA_ROPE_PAIRS = range(2)
LORA_W4_MAX_ROWS = 256
LORA_W4_MAX_PROBLEMS = 16
LORA_Q8_MAX_WIDTH = 32768
LORA_Q8_MAX_ROWS = 1 << 24
LORA_W8_MAX_ROWS = 65536
LORA_W8_MAX_PROBLEMS = 16
LORA_W8_MAX_K = 65536
LORA_Q8_X_HELD, LORA_Q8_X_FULL = range(2)
LORA_ACT_NONE, LORA_ACT_SILU, LORA_ACT_GELU, LORA_ACT_GELU_TANH = range(4)

EXPORTED = ["lora_pool_create", "lora_pool_destroy", "lora_pool_set_tuning", "lora_pool_get_tuning",
            "lora_workspace_size", "lora_workspace_init",
            "lora_segment", "lora_workspace_view", "lora_bgmv", "lora_sgmv", "lora_apply_mixed",
            "lora_delta_grouped", "lora_debug_page_list", "lora_debug_delta_with_t", "lora_debug_wait_limit",
            "lora_stage_pages", "lora_bgmv_noalloc", "lora_get_device_error", "lora_shrink",
            "lora_expand", "lora_stage_pages_ce",
            "lora_last_cuda_error", "lora_status_string",
            # host runtime (include/lora_runtime.h)
            "lora_cache_create", "lora_cache_destroy", "lora_cache_acquire", "lora_cache_loaded",
            "lora_cache_release", "lora_cache_query", "lora_cache_stats", "lora_sched_create",
            "lora_sched_destroy", "lora_sched_enqueue", "lora_sched_pick", "lora_sched_pending",
            # the 4-bit KV cache (include/lora_kv.h) and 4-bit weights (include/lora_w4.h)
            "lora_kv_block_bytes", "lora_kv_workspace_size", "lora_kv_workspace_init", "lora_kv_append",
            "lora_kv_read", "lora_kv_attend", "lora_w4_workspace_size", "lora_w4_matvec", "lora_debug_w4_lost_block",
            # an 8-bit base model (include/lora_w8.h)
            "lora_q8_norm", "lora_q8_gate", "lora_w8_workspace_size", "lora_w8_matmul", "lora_debug_w8_lost_step"]


class lora_pool_desc(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("h", ctypes.c_int32),
                ("num_adapters", ctypes.c_int32), ("num_layers", ctypes.c_int32),
                ("num_proj", ctypes.c_int32), ("r_max", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("page_table", ctypes.c_void_p),
                ("page_table_len", ctypes.c_int64), ("adapter_pt_off", ctypes.c_void_p),
                ("ranks", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("proj_dims", ctypes.c_void_p)]


class lora_tuning(ctypes.Structure):
    _fields_ = [("ring_rows_per_stage", ctypes.c_int32), ("split_max_problems", ctypes.c_int32),
                ("mma_min_rows", ctypes.c_int32), ("mma_y_stages", ctypes.c_int32),
                ("fused_ring_speed", ctypes.c_float), ("reserved", ctypes.c_int32 * 3)]


# lora_tuning fields and the value that keeps a field's default
TUNING_KEEP = {"ring_rows_per_stage": 0, "split_max_problems": -1, "mma_min_rows": -1,
               "mma_y_stages": 0, "fused_ring_speed": 0.0}


class lora_problem(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("ldx", ctypes.c_int64),
                ("ldy", ctypes.c_int64), ("layer", ctypes.c_int32), ("proj", ctypes.c_int32)]


class lora_ws_view(ctypes.Structure):
    _fields_ = [("error_word", ctypes.c_void_p), ("counts", ctypes.c_void_p),
                ("perm", ctypes.c_void_p), ("grp_start", ctypes.c_void_p),
                ("grp_adapter", ctypes.c_void_p)]


class lora_kv_cache_desc(ctypes.Structure):
    _fields_ = [("blocks", ctypes.c_void_p), ("num_blocks", ctypes.c_int64), ("block_stride", ctypes.c_int64),
                ("block_tokens", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("group", ctypes.c_int32)]


class lora_kv_batch(ctypes.Structure):
    _fields_ = [("q_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("n_seq", ctypes.c_int32), ("T", ctypes.c_int32), ("max_blocks", ctypes.c_int32),
                ("max_q", ctypes.c_int32)]


class lora_rope(ctypes.Structure):
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("max_pos", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("style", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class lora_w4_problem(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("ldy", ctypes.c_int64),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p),
                ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("group", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class lora_q8_rows(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("x", ctypes.c_void_p), ("ldc", ctypes.c_int64),
                ("ldx", ctypes.c_int64), ("x_kind", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class lora_q8_norm_desc(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("sum", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("ldx", ctypes.c_int64), ("ldr", ctypes.c_int64), ("lds", ctypes.c_int64), ("eps", ctypes.c_float),
                ("d", ctypes.c_int32), ("out", lora_q8_rows)]


class lora_q8_gate_desc(ctypes.Structure):
    _fields_ = [("gate", ctypes.c_void_p), ("up", ctypes.c_void_p), ("ldg", ctypes.c_int64), ("ldu", ctypes.c_int64),
                ("act", ctypes.c_int32), ("d", ctypes.c_int32), ("out", lora_q8_rows)]


class lora_w8_problem(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("x_scales", ctypes.c_void_p), ("y", ctypes.c_void_p), ("w", ctypes.c_void_p),
                ("w_scales", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("ldy", ctypes.c_int64), ("N", ctypes.c_int32),
                ("K", ctypes.c_int32)]


class LoraError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        msg = f"{where}: {status_string(status)}"
        if status == LORA_ECUDA:
            msg += f" (cudaError {lib().lora_last_cuda_error()})"
        super().__init__(msg + (f" {detail}" if detail else ""))


_lib = None


def lib():
    """Load liblora.so (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(SO):
            raise RuntimeError(f"{SO} is missing: build it with __graft_entry__.build()")
        L = ctypes.CDLL(SO)
        p, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        sig = {
            "lora_pool_create": [ctypes.POINTER(p), ctypes.POINTER(lora_pool_desc)],
            "lora_pool_destroy": [p],
            "lora_pool_set_tuning": [p, ctypes.POINTER(lora_tuning)],
            "lora_pool_get_tuning": [p, ctypes.POINTER(lora_tuning)],
            "lora_workspace_size": [p, i32, i32, ctypes.POINTER(sz)],
            "lora_workspace_init": [p, sz, p],
            "lora_segment": [p, p, p, i32, p, i32, i32, p, sz, p],
            "lora_workspace_view": [p, p, sz, i32, i32, ctypes.POINTER(lora_ws_view)],
            "lora_bgmv": [p, p, i32, p, i32, p, sz, p],
            "lora_sgmv": [p, p, i32, p, p, i32, i32, p, sz, p],
            "lora_apply_mixed": [p, p, i32, p, p, i32, p, i32, i32, p, sz, p],
            "lora_delta_grouped": [p, p, i32, i32, i32, p, sz, p],
            "lora_debug_page_list": [p, p, sz, i32, i32, p, i64, p, p],
            "lora_debug_delta_with_t": [p, ctypes.POINTER(lora_problem), p, sz, p, p],
            "lora_debug_wait_limit": [p, sz, ctypes.c_uint64, p, p],
            "lora_stage_pages": [p, p, p, i32, p, p, p, i64, p],
            "lora_stage_pages_ce": [p, p, p, sz, p, i32, p, p, p, i64, p, p],
            "lora_bgmv_noalloc": [p, p, i32, p, i32, p, p],
            "lora_shrink": [p, p, i32, p, i32, p, sz, p, p],
            "lora_expand": [p, p, i32, i32, p, sz, p, p],
            "lora_get_device_error": [p, p, ctypes.POINTER(ctypes.c_uint32)],
            "lora_last_cuda_error": [],
            "lora_status_string": [ctypes.c_int],
            "lora_cache_create": [ctypes.POINTER(p), p, i64, p, i32],
            "lora_cache_destroy": [p],
            "lora_cache_acquire": [p, i32, ctypes.POINTER(i32), p, i64, p, i32, ctypes.POINTER(i32)],
            "lora_cache_loaded": [p, i32],
            "lora_cache_release": [p, i32],
            "lora_cache_query": [p, i32, ctypes.POINTER(i32), ctypes.POINTER(i32), p, i64],
            "lora_cache_stats": [p] + [ctypes.POINTER(i64)] * 4,
            "lora_sched_create": [ctypes.POINTER(p), p],
            "lora_sched_destroy": [p],
            "lora_sched_enqueue": [p, i64, i32, i32],
            "lora_sched_pick": [p, i32, i32, p, p, p, i32, ctypes.POINTER(i32), ctypes.POINTER(i32),
                                ctypes.POINTER(i32)],
            "lora_sched_pending": [p, ctypes.POINTER(i64)],
            "lora_kv_block_bytes": [i32, i32, i32, i32, ctypes.POINTER(sz)],
            "lora_kv_workspace_size": [p, p, i32, ctypes.POINTER(sz)],
            "lora_kv_workspace_init": [p, sz, p],
            "lora_kv_append": [p, p, p, i64, p, i64, i32, p, i64, p, i64, p, p, sz, p],
            "lora_kv_read": [p, p, p, i64, p, i64, p, sz, p],
            "lora_kv_attend": [p, p, p, i64, i32, ctypes.c_float, p, i64, p, p, sz, p],
            "lora_w4_workspace_size": [p, i32, i32, ctypes.POINTER(sz)],
            "lora_w4_matvec": [p, i32, i32, p, sz, p],
            "lora_debug_w4_lost_block": [p, i32, i32, i32, ctypes.c_uint64, p, sz, p],
            "lora_q8_norm": [p, i32, p],
            "lora_q8_gate": [p, i32, p],
            "lora_w8_workspace_size": [p, i32, i32, ctypes.POINTER(sz)],
            "lora_w8_matmul": [p, i32, i32, p, sz, p],
            "lora_debug_w8_lost_step": [p, i32, i32, i32, ctypes.c_uint64, p, sz, p],
        }
        for name, args in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        L.lora_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def status_string(st: int) -> str:
    return lib().lora_status_string(st).decode()


def _check(st: int, where: str):
    if st != LORA_OK:
        raise LoraError(st, where)


def _ptr(t) -> int | None:
    """Device or host address of a tensor / integer (None stays NULL)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def problems_array(problems):
    """problems: iterable of (x, y, ldx, ldy, layer, proj) with x/y tensors or addresses."""
    problems = list(problems)
    arr = (lora_problem * max(1, len(problems)))()
    for i, (x, y, ldx, ldy, layer, proj) in enumerate(problems):
        arr[i] = lora_problem(_ptr(x), _ptr(y), ldx, ldy, layer, proj)
    return arr, len(problems)


class Pool:
    """Handle of a lora_pool (host metadata only; device arrays stay the caller's)."""

    def __init__(self, pages, num_pages, h, page_table, page_table_len, pt_off, ranks, scales,
                 num_adapters, num_layers, num_proj, r_max, proj_dims=None):
        """proj_dims: (d_in, d_out) of every projection (copied by the library), or None
        for h x h projections."""
        import numpy as np
        dims = None if proj_dims is None else np.ascontiguousarray(proj_dims, np.int32).reshape(-1)
        d = lora_pool_desc(_ptr(pages), num_pages, h, num_adapters, num_layers, num_proj, r_max, 0,
                           _ptr(page_table), page_table_len, _ptr(pt_off), _ptr(ranks), _ptr(scales),
                           dims.ctypes.data if dims is not None else None)
        self._h = ctypes.c_void_p()
        _check(lib().lora_pool_create(ctypes.byref(self._h), ctypes.byref(d)), "lora_pool_create")
        self.h = h
        self.r_max = r_max

    @property
    def handle(self):
        return self._h

    def set_tuning(self, **fields):
        """Launch tuning (lora_pool_set_tuning): the named fields, every other one at its
        default; no fields restores all the defaults."""
        unknown = set(fields) - set(TUNING_KEEP)
        if unknown:
            raise ValueError(f"unknown tuning fields {sorted(unknown)}")
        t = lora_tuning(**{k: fields.get(k, v) for k, v in TUNING_KEEP.items()})
        _check(lib().lora_pool_set_tuning(self._h, ctypes.byref(t)), "lora_pool_set_tuning")

    def get_tuning(self) -> dict:
        t = lora_tuning()
        _check(lib().lora_pool_get_tuning(self._h, ctypes.byref(t)), "lora_pool_get_tuning")
        return {k: getattr(t, k) for k in TUNING_KEEP}

    def close(self):
        if self._h:
            lib().lora_pool_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def workspace_size(pool: Pool, max_tokens: int, max_segments: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().lora_workspace_size(pool.handle, max_tokens, max_segments, ctypes.byref(n)),
           "lora_workspace_size")
    return n.value


def workspace_init(ws, ws_bytes: int, stream: int):
    _check(lib().lora_workspace_init(_ptr(ws), ws_bytes, stream), "lora_workspace_init")


def segment(pool, seg_start, seg_adapter, S, dec_adapter, Td, T, ws, ws_bytes, stream):
    _check(lib().lora_segment(pool.handle, _ptr(seg_start), _ptr(seg_adapter), S,
                              _ptr(dec_adapter), Td, T, _ptr(ws), ws_bytes, stream), "lora_segment")


def workspace_view(pool, ws, ws_bytes, max_tokens, max_segments) -> lora_ws_view:
    v = lora_ws_view()
    _check(lib().lora_workspace_view(pool.handle, _ptr(ws), ws_bytes, max_tokens, max_segments,
                                     ctypes.byref(v)), "lora_workspace_view")
    return v


def bgmv(pool, problems, token_adapter, T, ws, ws_bytes, stream):
    arr, n = problems_array(problems)
    _check(lib().lora_bgmv(pool.handle, arr, n, _ptr(token_adapter), T, _ptr(ws), ws_bytes, stream),
           "lora_bgmv")


def sgmv(pool, problems, seg_start, seg_adapter, S, T, ws, ws_bytes, stream):
    arr, n = problems_array(problems)
    _check(lib().lora_sgmv(pool.handle, arr, n, _ptr(seg_start), _ptr(seg_adapter), S, T, _ptr(ws),
                           ws_bytes, stream), "lora_sgmv")


def apply_mixed(pool, problems, seg_start, seg_adapter, S, dec_adapter, Td, T, ws, ws_bytes, stream):
    arr, n = problems_array(problems)
    _check(lib().lora_apply_mixed(pool.handle, arr, n, _ptr(seg_start), _ptr(seg_adapter), S,
                                  _ptr(dec_adapter), Td, T, _ptr(ws), ws_bytes, stream),
           "lora_apply_mixed")


def delta_grouped(pool, problems, T, S, ws, ws_bytes, stream):
    arr, n = problems_array(problems)
    _check(lib().lora_delta_grouped(pool.handle, arr, n, T, S, _ptr(ws), ws_bytes, stream),
           "lora_delta_grouped")


def debug_page_list(pool, ws, ws_bytes, layer, proj, out_pages, cap, count_dev, stream):
    _check(lib().lora_debug_page_list(pool.handle, _ptr(ws), ws_bytes, layer, proj, _ptr(out_pages),
                                      cap, _ptr(count_dev), stream), "lora_debug_page_list")


def debug_delta_with_t(pool, problem, ws, ws_bytes, t_out, stream):
    arr, _ = problems_array([problem])
    _check(lib().lora_debug_delta_with_t(pool.handle, arr, _ptr(ws), ws_bytes, _ptr(t_out), stream),
           "lora_debug_delta_with_t")


def debug_wait_limit(ws, ws_bytes, limit_ns, elapsed_ns, stream):
    """elapsed_ns: device uint64 (int64 tensor of one element) or None."""
    _check(lib().lora_debug_wait_limit(_ptr(ws), ws_bytes, limit_ns, _ptr(elapsed_ns), stream),
           "lora_debug_wait_limit")


def stage_pages(pool, host_rows, dst_pages, npages, page_table, upd_index, upd_page, nupd, stream):
    """host_rows, dst_pages, upd_index, upd_page: pinned host tensors (or addresses)."""
    _check(lib().lora_stage_pages(pool.handle, _ptr(host_rows), _ptr(dst_pages), npages,
                                  _ptr(page_table), _ptr(upd_index), _ptr(upd_page), nupd, stream),
           "lora_stage_pages")


def stage_pages_ce(pool, host_rows, staging, staging_bytes, dst_pages, npages, page_table, upd_index, upd_page,
                   nupd, stream, copied_event=None):
    """Staging through the copy engines: each run of consecutive destination pages copied
    straight into the pool (at most LORA_STAGE_MAX_RUNS runs), else host rows -> device
    staging buffer (one copy) -> pool pages (one kernel); then the page-table rewrite.
    host_rows, dst_pages, upd_index, upd_page: pinned host tensors; staging: a device buffer of
    npages * 2h bytes, or None when the pages form at most LORA_STAGE_MAX_RUNS runs;
    copied_event: a torch.cuda.Event (or raw handle) recorded right after the copies."""
    ev = None
    if copied_event is not None:
        ev = copied_event.cuda_event if hasattr(copied_event, "cuda_event") else copied_event
    _check(lib().lora_stage_pages_ce(pool.handle, _ptr(host_rows), _ptr(staging), staging_bytes,
                                     _ptr(dst_pages), npages, _ptr(page_table), _ptr(upd_index),
                                     _ptr(upd_page), nupd, ev, stream), "lora_stage_pages_ce")


def bgmv_noalloc(pool, problems, token_adapter, T, error_bits, stream):
    """BGMV with the library's own fixed scratch (no caller workspace, no allocation)."""
    arr, n = problems_array(problems)
    _check(lib().lora_bgmv_noalloc(pool.handle, arr, n, _ptr(token_adapter), T, _ptr(error_bits),
                                   stream), "lora_bgmv_noalloc")


def shrink(pool, problems, token_adapter, T, ws, ws_bytes, t, stream):
    """t[p][row][j] = s * x_p[row] . A_j (fp32 [nprob][T][r_max]); groups the batch into ws."""
    arr, n = problems_array(problems)
    _check(lib().lora_shrink(pool.handle, arr, n, _ptr(token_adapter), T, _ptr(ws), ws_bytes, _ptr(t),
                             stream), "lora_shrink")


def expand(pool, problems, T, ws, ws_bytes, t, stream):
    """y_p[row] += t[p][row] . B^T with the grouping lora_shrink left in ws."""
    arr, n = problems_array(problems)
    _check(lib().lora_expand(pool.handle, arr, n, T, _ptr(ws), ws_bytes, _ptr(t), stream), "lora_expand")


def get_device_error(ws, stream) -> int:
    """Synchronises the stream; returns and clears the device error bits (no raise)."""
    bits = ctypes.c_uint32()
    st = lib().lora_get_device_error(_ptr(ws), stream, ctypes.byref(bits))
    if st not in (LORA_OK, LORA_EDEVICE):
        raise LoraError(st, "lora_get_device_error")
    return bits.value


# ----------------------------------------------------------------------------- 4-bit KV cache

class _Desc:
    """A description passed by pointer on every call; keeps the tensors it names alive."""

    def __init__(self, struct, *owners):
        self.struct, self._owners = struct, owners
        self.ref = ctypes.addressof(struct)


class KvCache(_Desc):
    """One layer's 4-bit paged cache (lora_kv_cache_desc): block b starts block_stride * b
    bytes after `blocks`."""

    def __init__(self, blocks, num_blocks, block_stride, block_tokens, num_kv_heads, head_dim, group):
        super().__init__(lora_kv_cache_desc(_ptr(blocks), num_blocks, block_stride, block_tokens, num_kv_heads,
                                            head_dim, group), blocks)


class KvBatch(_Desc):
    """A batch of requests over a cache (lora_kv_batch): device arrays q_start [n_seq + 1],
    kv_len [n_seq], block_table [n_seq][max_blocks]; T rows, at most max_q of one request."""

    def __init__(self, q_start, kv_len, block_table, n_seq, T, max_blocks, max_q):
        super().__init__(lora_kv_batch(_ptr(q_start), _ptr(kv_len), _ptr(block_table), n_seq, T, max_blocks, max_q),
                         q_start, kv_len, block_table)


class Rope(_Desc):
    """Rotation tables (lora_rope): cos, sin f32 [max_pos][rot_dim / 2], style LORA_ROPE_*;
    positions int32 [T], or None: each row's cache token."""

    def __init__(self, cos, sin, max_pos, rot_dim, style=LORA_ROPE_HALVES, positions=None):
        super().__init__(lora_rope(_ptr(cos), _ptr(sin), _ptr(positions), max_pos, rot_dim, style, 0),
                         cos, sin, positions)


def kv_block_bytes(block_tokens, num_kv_heads, head_dim, group) -> int:
    n = ctypes.c_size_t()
    _check(lib().lora_kv_block_bytes(block_tokens, num_kv_heads, head_dim, group, ctypes.byref(n)),
           "lora_kv_block_bytes")
    return n.value


def kv_workspace_size(cache: KvCache, batch: KvBatch, num_q_heads: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().lora_kv_workspace_size(cache.ref, batch.ref, num_q_heads, ctypes.byref(n)),
           "lora_kv_workspace_size")
    return n.value


def kv_workspace_init(ws, ws_bytes: int, stream: int):
    _check(lib().lora_kv_workspace_init(_ptr(ws), ws_bytes, stream), "lora_kv_workspace_init")


def kv_append(cache, batch, q, ldq, q_out, ldqo, num_q_heads, k, ldk, v, ldv, rope, ws, ws_bytes, stream):
    """q_out = q turned by its positions; k (turned) and v stored in the cache."""
    _check(lib().lora_kv_append(cache.ref, batch.ref, _ptr(q), ldq, _ptr(q_out), ldqo, num_q_heads, _ptr(k), ldk,
                                _ptr(v), ldv, rope.ref, _ptr(ws), ws_bytes, stream), "lora_kv_append")


def kv_read(cache, batch, k_out, ldk, v_out, ldv, ws, ws_bytes, stream):
    """The batch's rows as the cache holds them, bf16."""
    _check(lib().lora_kv_read(cache.ref, batch.ref, _ptr(k_out), ldk, _ptr(v_out), ldv, _ptr(ws), ws_bytes,
                              stream), "lora_kv_read")


def kv_attend(cache, batch, q, ldq, num_q_heads, softmax_scale, out, ldo, lse, ws, ws_bytes, stream):
    """Causal attention of the batch's rows over the cache; lse: f32 [T][num_q_heads] or None."""
    _check(lib().lora_kv_attend(cache.ref, batch.ref, _ptr(q), ldq, num_q_heads, softmax_scale, _ptr(out), ldo,
                                _ptr(lse), _ptr(ws), ws_bytes, stream), "lora_kv_attend")


# ----------------------------------------------------------------------------- 4-bit weights

def w4_problems(problems):
    """The projections of a call, kept by the caller for as long as the tensors stay where
    they are: (x, y, ldx, ldy, codes, scales, zeros or None, N, K, group) each."""
    problems = list(problems)
    arr = (lora_w4_problem * max(1, len(problems)))()
    for i, (x, y, ldx, ldy, codes, scales, zeros, n, k, group) in enumerate(problems):
        arr[i] = lora_w4_problem(_ptr(x), _ptr(y), ldx, ldy, _ptr(codes), _ptr(scales), _ptr(zeros), n, k, group, 0)
    return _Problems(arr, problems)


class _Problems(_Desc):
    def __init__(self, arr, problems):
        super().__init__(arr, problems)
        self.n = len(problems)


def w4_workspace_size(problems, T: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().lora_w4_workspace_size(problems.ref, problems.n, T, ctypes.byref(n)), "lora_w4_workspace_size")
    return n.value


def w4_matvec(problems, T, ws, ws_bytes, stream):
    """y = x W^T for every projection of w4_problems(...)."""
    _check(lib().lora_w4_matvec(problems.ref, problems.n, T, _ptr(ws), ws_bytes, stream), "lora_w4_matvec")


def debug_w4_lost_block(problems, T, block, limit_ns, ws, ws_bytes, stream):
    """w4_matvec with one block's codes missing: its waits run out after limit_ns."""
    _check(lib().lora_debug_w4_lost_block(problems.ref, problems.n, T, block, limit_ns, _ptr(ws), ws_bytes, stream),
           "lora_debug_w4_lost_block")


# ----------------------------------------------------------------------------- an 8-bit base model

class Q8Rows(_Desc):
    """Where rows go in 8 bits (lora_q8_rows): int8 codes [T][ldc], f32 scales [T], and in bf16 x
    [T][ldx] (or None) what the codes stand for (LORA_Q8_X_HELD) or the rows themselves (LORA_Q8_X_FULL)."""

    def __init__(self, codes, ldc, scales, x=None, ldx=0, x_kind=LORA_Q8_X_HELD):
        super().__init__(lora_q8_rows(_ptr(codes), _ptr(scales), _ptr(x), ldc, ldx, x_kind, 0), codes, scales, x)


class Q8Norm(_Desc):
    """A norm's buffers (lora_q8_norm_desc), kept by the caller for as long as the tensors stay where
    they are: bf16 x and residual (or None) in, their sum out (or None), bf16 weight [d], rows a Q8Rows."""

    def __init__(self, x, ldx, residual, ldr, total, lds, weight, eps, d, rows):
        super().__init__(lora_q8_norm_desc(_ptr(x), _ptr(residual), _ptr(total), _ptr(weight), ldx, ldr, lds, eps, d, rows.struct),
                         x, residual, total, weight, rows)


class Q8Gate(_Desc):
    """A gated activation's buffers (lora_q8_gate_desc): bf16 gate and up (or None), act one of
    LORA_ACT_*, rows a Q8Rows."""

    def __init__(self, gate, ldg, up, ldu, act, d, rows):
        super().__init__(lora_q8_gate_desc(_ptr(gate), _ptr(up), ldg, ldu, act, d, rows.struct), gate, up, rows)


def q8_norm(norm, T, stream):
    """The residual's addition and root-mean-square norm of T rows, left in 8 bits."""
    _check(lib().lora_q8_norm(norm.ref, T, stream), "lora_q8_norm")


def q8_gate(gate, T, stream):
    """act(gate) * up of T rows, left in 8 bits."""
    _check(lib().lora_q8_gate(gate.ref, T, stream), "lora_q8_gate")


def w8_problems(problems):
    """The projections of a call, kept by the caller for as long as the tensors stay where
    they are: (x, x_scales, y, ldx, ldy, w, w_scales, N, K) each."""
    problems = list(problems)
    arr = (lora_w8_problem * max(1, len(problems)))()
    for i, (x, x_scales, y, ldx, ldy, w, w_scales, n, k) in enumerate(problems):
        arr[i] = lora_w8_problem(_ptr(x), _ptr(x_scales), _ptr(y), _ptr(w), _ptr(w_scales), ldx, ldy, n, k)
    return _Problems(arr, problems)


def w8_workspace_size(problems, T: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().lora_w8_workspace_size(problems.ref, problems.n, T, ctypes.byref(n)), "lora_w8_workspace_size")
    return n.value


def w8_matmul(problems, T, ws, ws_bytes, stream):
    """y = x W^T of 8-bit integers for every projection of w8_problems(...)."""
    _check(lib().lora_w8_matmul(problems.ref, problems.n, T, _ptr(ws), ws_bytes, stream), "lora_w8_matmul")


def debug_w8_lost_step(problems, T, step, limit_ns, ws, ws_bytes, stream):
    """w8_matmul with one step's W missing: its waits run out after limit_ns."""
    _check(lib().lora_debug_w8_lost_step(problems.ref, problems.n, T, step, limit_ns, _ptr(ws), ws_bytes, stream),
           "lora_debug_w8_lost_step")


# ----------------------------------------------------------------------------- host runtime

def _np_ptr(a):
    return a.ctypes.data if a is not None and a.size else None


class AdapterCache:
    """lora_cache_*: LRU residency of units (adapters or adapter slices) in pool pages."""

    def __init__(self, managed_pages, unit_pages):
        import numpy as np
        self._np = np
        self.managed = np.ascontiguousarray(managed_pages, np.int32)
        self.unit_pages = np.ascontiguousarray(unit_pages, np.int32)
        h = ctypes.c_void_p()
        _check(lib().lora_cache_create(ctypes.byref(h), _np_ptr(self.managed), self.managed.size,
                                       _np_ptr(self.unit_pages), self.unit_pages.size), "lora_cache_create")
        self.handle = h

    def _unit_pages(self, u: int) -> int:
        # out-of-range units go to the library, which rejects them
        return int(self.unit_pages[u]) if 0 <= u < self.unit_pages.size else 1

    def acquire(self, u: int, evicted_cap: int = 64):
        """(loaded, pages or None, evicted units); raises LoraError (LORA_ENOSPACE) when full."""
        np = self._np
        pages = np.empty(self._unit_pages(u), np.int32)
        ev = np.empty(evicted_cap, np.int32)
        loaded, n_ev = ctypes.c_int32(), ctypes.c_int32()
        _check(lib().lora_cache_acquire(self.handle, u, ctypes.byref(loaded), pages.ctypes.data, pages.size,
                                        ev.ctypes.data, evicted_cap, ctypes.byref(n_ev)), "lora_cache_acquire")
        return bool(loaded.value), (pages if loaded.value else None), ev[:min(n_ev.value, evicted_cap)].copy()

    def try_acquire(self, u: int):
        """acquire, or None when no pages can be freed."""
        try:
            return self.acquire(u)
        except LoraError as e:
            if e.status == LORA_ENOSPACE:
                return None
            raise

    def loaded(self, u: int):
        _check(lib().lora_cache_loaded(self.handle, u), "lora_cache_loaded")

    def release(self, u: int):
        _check(lib().lora_cache_release(self.handle, u), "lora_cache_release")

    def query(self, u: int):
        """(state, users, pages of a resident unit)."""
        np = self._np
        st, us = ctypes.c_int32(), ctypes.c_int32()
        pages = np.empty(self._unit_pages(u), np.int32)
        _check(lib().lora_cache_query(self.handle, u, ctypes.byref(st), ctypes.byref(us), pages.ctypes.data,
                                      pages.size), "lora_cache_query")
        return st.value, us.value, (pages if st.value != LORA_UNIT_ABSENT else None)

    def stats(self):
        """dict of hits, misses, evictions, free_pages."""
        v = [ctypes.c_int64() for _ in range(4)]
        _check(lib().lora_cache_stats(self.handle, *[ctypes.byref(x) for x in v]), "lora_cache_stats")
        return dict(zip(("hits", "misses", "evictions", "free_pages"), (x.value for x in v)))

    def close(self):
        if self.handle:
            lib().lora_cache_destroy(self.handle)
            self.handle = None


class Scheduler:
    """lora_sched_*: arrival-ordered request queue and the per-step batch pick."""

    def __init__(self, cache: AdapterCache | None = None):
        h = ctypes.c_void_p()
        _check(lib().lora_sched_create(ctypes.byref(h), cache.handle if cache is not None else None),
               "lora_sched_create")
        self.handle = h
        self.cache = cache

    def enqueue(self, req_id: int, adapter: int, tokens: int = 1):
        _check(lib().lora_sched_enqueue(self.handle, req_id, adapter, tokens), "lora_sched_enqueue")

    def pick(self, max_tokens: int, max_distinct: int, cap: int = 4096):
        """(ids, adapters, tokens) of the batch, numpy arrays in queue order."""
        import numpy as np
        ids = np.empty(cap, np.int64)
        ad = np.empty(cap, np.int32)
        tk = np.empty(cap, np.int32)
        n, nt, nd = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
        _check(lib().lora_sched_pick(self.handle, max_tokens, max_distinct, ids.ctypes.data, ad.ctypes.data,
                                     tk.ctypes.data, cap, ctypes.byref(n), ctypes.byref(nt), ctypes.byref(nd)),
               "lora_sched_pick")
        k = n.value
        return ids[:k].copy(), ad[:k].copy(), tk[:k].copy()

    def pending(self) -> int:
        v = ctypes.c_int64()
        _check(lib().lora_sched_pending(self.handle, ctypes.byref(v)), "lora_sched_pending")
        return v.value

    def close(self):
        if self.handle:
            lib().lora_sched_destroy(self.handle)
            self.handle = None
