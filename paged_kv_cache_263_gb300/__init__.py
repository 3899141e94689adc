"""GB300-native paged KV-cache attention: Python binding of libpagedkv.so.

The binding only marshals arguments: every step runs in the library (host
block manager in C++, kernels in CUDA for sm_103a).  Functions carry the
C-ABI names of ``include/pagedkv.h``; torch tensors supply device memory and
the current CUDA stream.  There is no fallback: if the library is missing or
a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import importlib
import os

import torch

__all__ = [
    "KVError", "lib", "KVPool", "kv_status_string", "reshape_and_cache",
    "paged_attention_workspace_size", "paged_attention_decode",
    "paged_attention_chunked_prefill_workspace_size", "paged_attention_chunked_prefill",
    "paged_attention_launch_count",
    "kv_last_device_status", "kv_last_device_status_flags", "KV_BF16", "KV_FP8_E4M3",
    "HEAD_DIM", "BLOCK_SIZE", "library_path", "PrefixCache", "kv_swap_out", "kv_swap_in", "kv_waste_stats",
    "kv_trace_prefill", "kv_trace_prefill_kernel_ms", "kv_selftest_bounded_wait",
    "kv_build_step_tables", "reshape_and_cache_latent", "paged_latent_attention",
    "paged_latent_attention_workspace_size", "latent_prefill_attention",
    "latent_prefill_attention_workspace_size", "LATENT_DIM", "LATENT_ROPE_DIM", "LATENT_MAX_HEADS",
    "paged_attention_shared_prefix", "paged_attention_shared_prefix_workspace_size",
    "paged_attention_shared_prefix_way", "kv_copy_blocks", "kv_fork_tables", "kv_remap_tables",
]

HEAD_DIM = 128
BLOCK_SIZE = 16
LATENT_DIM, LATENT_ROPE_DIM, LATENT_MAX_HEADS = 512, 64, 128
_LATENT_ROW, _EXPANDED_QK = LATENT_DIM + LATENT_ROPE_DIM, HEAD_DIM + LATENT_ROPE_DIM
KV_BF16, KV_FP8_E4M3 = 0, 1
_STATUS = {0: "ok", 1: "invalid argument", 2: "out of blocks", 3: "unsupported",
           4: "CUDA error", 5: "device data out of range"}

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libpagedkv.so")
_lib = None


class KVError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {_STATUS.get(status, status)} (status {status})")
        self.status = status


class _Stats(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int32), ("free_blocks", ctypes.c_int32),
                ("live_blocks", ctypes.c_int32), ("shared_blocks", ctypes.c_int32),
                ("cow_copies", ctypes.c_int64), ("alloc_failures", ctypes.c_int64)]


class _PrefixStats(ctypes.Structure):
    _fields_ = [("lookups", ctypes.c_int64), ("query_blocks", ctypes.c_int64),
                ("hit_blocks", ctypes.c_int64), ("inserted_blocks", ctypes.c_int64),
                ("evicted_blocks", ctypes.c_int64), ("cached_blocks", ctypes.c_int32),
                ("evictable_blocks", ctypes.c_int32)]


class _WasteStats(ctypes.Structure):
    _fields_ = [("used_tokens", ctypes.c_int64), ("contiguous_reserved_slots", ctypes.c_int64),
                ("contiguous_untouched_slots", ctypes.c_int64), ("paged_blocks", ctypes.c_int64),
                ("paged_slots", ctypes.c_int64), ("paged_waste_slots", ctypes.c_int64),
                ("contiguous_untouched_percent", ctypes.c_double), ("paged_waste_percent", ctypes.c_double)]


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(library_path):
            raise RuntimeError(f"{library_path} is not built (run __graft_entry__.build())")
        L = ctypes.CDLL(library_path)
        c = ctypes
        P, I, I64, F, SZ = c.c_void_p, c.c_int32, c.c_int64, c.c_float, c.c_size_t
        sig = {
            "kv_status_string": (c.c_char_p, [c.c_int]),
            "kv_pool_create": (c.c_int, [I, P, c.POINTER(P)]),
            "kv_pool_destroy": (None, [P]),
            "kv_block_alloc": (c.c_int, [P, I, P]),
            "kv_block_free": (c.c_int, [P, P, I]),
            "kv_block_share": (c.c_int, [P, P, I]),
            "kv_copy_on_write": (c.c_int, [P, I, c.POINTER(I), P, P, I, c.c_int, P]),
            "kv_block_refcount": (c.c_int, [P, I, c.POINTER(I)]),
            "kv_pool_stats": (c.c_int, [P, c.POINTER(_Stats)]),
            "kv_pool_fail_alloc_after": (c.c_int, [P, I]),
            "kv_waste_stats": (c.c_int, [P, I, I, c.POINTER(_WasteStats)]),
            "kv_prefix_cache_create": (c.c_int, [P, c.POINTER(P)]),
            "kv_prefix_cache_destroy": (None, [P]),
            "kv_prefix_match": (c.c_int, [P, P, I, c.c_uint64, I, P, c.POINTER(I)]),
            "kv_prefix_insert": (c.c_int, [P, P, I, c.c_uint64, P, I, c.POINTER(I)]),
            "kv_prefix_evict": (c.c_int, [P, I, P, c.POINTER(I)]),
            "kv_prefix_alloc": (c.c_int, [P, I, P]),
            "kv_prefix_stats": (c.c_int, [P, c.POINTER(_PrefixStats)]),
            "reshape_and_cache": (c.c_int, [P, P, P, P, P, I, I, I, c.c_int, P, P, P]),
            "paged_attention_workspace_size": (SZ, [I, I, I, I]),
            "paged_attention_decode": (c.c_int, [P, P, P, P, P, I, P, I, I, I, I, F, c.c_int, P, P,
                                                 I, P, SZ, P]),
            "paged_attention_chunked_prefill_workspace_size": (SZ, [I, I, I, I, I, I, I]),
            "paged_attention_launch_count": (I, [I, I, I, I, I, I, I]),
            "paged_attention_chunked_prefill": (c.c_int, [P, P, P, P, I, I, I, P, P, P, I, I, I, I,
                                                          F, c.c_int, P, P, I, P, SZ, P]),
            "paged_attention_decode_static_scratch_bytes": (SZ, []),
            "paged_attention_decode_static_scratch": (c.c_int, [P, P, P, P, P, I, P, I, I, I, I, F, c.c_int, P,
                                                                P, I, P]),
            "kv_build_step_tables": (c.c_int, [P, I, P, P, I, P, I, I, P, P, P, P, I, P, P]),
            "reshape_and_cache_latent": (c.c_int, [P, I64, P, I64, P, P, I, I, P]),
            "paged_latent_attention_workspace_size": (SZ, [I, I, I, I]),
            "paged_latent_attention": (c.c_int, [P, P, P, P, I, I, P, P, I, I, I, F, P, SZ, P]),
            "latent_prefill_attention_workspace_size": (SZ, [I, I, I]),
            "latent_prefill_attention": (c.c_int, [P, P, P, P, I64, P, P, I, I, I, I, F, P, SZ, P]),
            "kv_pool_compact": (c.c_int, [P, I, P, P, c.POINTER(I)]),
            "kv_prefix_remap": (c.c_int, [P, P, P, I]),
            "paged_attention_shared_prefix_workspace_size": (SZ, [I, I, I, I, I, I, I, I]),
            "paged_attention_shared_prefix_way": (I, [I, I, I, I, I, I, I, I, c.c_int]),
            "paged_attention_shared_prefix": (c.c_int, [P, P, P, P, I, I, I, P, P, I, I, I, P, P, P, I, I, I, I, F,
                                                        c.c_int, P, P, P, SZ, P]),
            "kv_copy_blocks": (c.c_int, [P, I, I64, I, P, P, I, P]),
            "kv_fork_tables": (c.c_int, [P, I, P, I, P, I, I, P, I, P, P, P, P, P, P]),
            "kv_remap_tables": (c.c_int, [P, I, P, I, P, P, I, P]),
            "kv_swap_out": (c.c_int, [P, P, I, I, c.c_int, P, I, P, P, P]),
            "kv_swap_in": (c.c_int, [P, P, I, I, c.c_int, P, I, P, P, P]),
            "kv_trace_prefill": (c.c_int, [I]),
            "kv_trace_prefill_kernel_ms": (c.c_double, []),
            "kv_last_device_status": (c.c_int, [P]),
            "kv_last_device_status_flags": (c.c_uint32, []),
            "kv_selftest_bounded_wait": (c.c_int, [c.c_uint32, P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


_fast_module = None


class _ByCtypes:
    """The entries of the module _fastcall through ctypes, where it was not built (no
    Python headers) or not for this interpreter."""

    def __init__(self, L):
        for name in ("paged_attention_shared_prefix", "paged_attention_shared_prefix_workspace_size", "kv_fork_tables",
                     "kv_remap_tables"):
            setattr(self, name, getattr(L, name))
        self._copy = L.kv_copy_blocks

    def kv_copy_blocks(self, caches, *args):
        return self._copy((ctypes.c_void_p * len(caches))(*caches), len(caches), *args)


def _fast():
    """The library's shortest calls without ctypes, which takes 0.15 us an argument."""
    global _fast_module
    if _fast_module is None:
        L = lib()
        try:
            _fast_module = importlib.import_module("._fastcall", __name__)
        except ModuleNotFoundError:
            _fast_module = _ByCtypes(L)
    return _fast_module


def _check(st: int, where: str):
    if st != 0:
        raise KVError(st, where)


def kv_status_string(st: int) -> str:
    return lib().kv_status_string(st).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dt(kv_dtype) -> int:
    if kv_dtype in (KV_BF16, "bf16", torch.bfloat16):
        return KV_BF16
    if kv_dtype in (KV_FP8_E4M3, "fp8", "fp8_e4m3", torch.float8_e4m3fn, torch.uint8):
        return KV_FP8_E4M3
    raise ValueError(f"unsupported kv dtype {kv_dtype}")


def _need(t, name, dtype=None, dev=True, contig=True):
    if t is None:
        raise ValueError(f"{name} is required")
    if dev and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if contig and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _cache_dtype(k_cache):
    return KV_BF16 if k_cache.dtype == torch.bfloat16 else KV_FP8_E4M3


# ------------------------------------------------------------------- pool
class KVPool:
    """Host block manager (free list, refcounts, copy-on-write)."""

    def __init__(self, num_blocks: int, initial_free_order=None):
        L = lib()
        self._p = ctypes.c_void_p()
        order = None
        if initial_free_order is not None:
            import numpy as np
            order = np.ascontiguousarray(initial_free_order, dtype=np.int32)
            if order.shape != (num_blocks,):
                raise ValueError("initial_free_order must have num_blocks entries")
        _check(L.kv_pool_create(int(num_blocks), None if order is None else order.ctypes.data_as(ctypes.c_void_p),
                                ctypes.byref(self._p)), "kv_pool_create")
        self.num_blocks = int(num_blocks)

    def close(self):
        if self._p:
            lib().kv_pool_destroy(self._p)
            self._p = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def alloc(self, n: int):
        import numpy as np
        out = np.empty(max(int(n), 0), dtype=np.int32)
        _check(lib().kv_block_alloc(self._p, int(n), out.ctypes.data_as(ctypes.c_void_p)), "kv_block_alloc")
        return out

    def free(self, ids):
        import numpy as np
        a = np.ascontiguousarray(ids, dtype=np.int32)
        _check(lib().kv_block_free(self._p, a.ctypes.data_as(ctypes.c_void_p), a.size), "kv_block_free")

    def share(self, ids):
        import numpy as np
        a = np.ascontiguousarray(ids, dtype=np.int32)
        _check(lib().kv_block_share(self._p, a.ctypes.data_as(ctypes.c_void_p), a.size), "kv_block_share")

    def copy_on_write(self, block_id: int, k_cache=None, v_cache=None, stream=None) -> int:
        """Returns the block to write into; copies K/V on the device if caches are given."""
        out = ctypes.c_int32()
        if k_cache is None:
            st = lib().kv_copy_on_write(self._p, int(block_id), ctypes.byref(out), None, None, 0, 0, None)
        else:
            _need(k_cache, "k_cache")
            _need(v_cache, "v_cache")
            st = lib().kv_copy_on_write(self._p, int(block_id), ctypes.byref(out), _ptr(k_cache),
                                        _ptr(v_cache), int(k_cache.shape[1]), _cache_dtype(k_cache),
                                        _stream(stream))
        _check(st, "kv_copy_on_write")
        return int(out.value)

    def refcount(self, block_id: int) -> int:
        out = ctypes.c_int32()
        _check(lib().kv_block_refcount(self._p, int(block_id), ctypes.byref(out)), "kv_block_refcount")
        return int(out.value)

    def stats(self) -> dict:
        s = _Stats()
        _check(lib().kv_pool_stats(self._p, ctypes.byref(s)), "kv_pool_stats")
        return {"num_blocks": s.num_blocks, "free": s.free_blocks, "live": s.live_blocks,
                "shared": s.shared_blocks, "cow_copies": s.cow_copies, "alloc_failures": s.alloc_failures}

    def compact(self, max_moves=None):
        """Moves live blocks from the pool's upper end into free ones at its lower end:
        (src, dst), both ascending.  The caller copies the blocks (kv_copy_blocks) and
        rewrites what holds ids (kv_remap_tables, PrefixCache.remap) before it allocates
        again."""
        import numpy as np
        n = self.num_blocks if max_moves is None else int(max_moves)
        src, dst = np.empty(max(n, 0), dtype=np.int32), np.empty(max(n, 0), dtype=np.int32)
        k = ctypes.c_int32()
        _check(lib().kv_pool_compact(self._p, n, src.ctypes.data_as(ctypes.c_void_p),
                                     dst.ctypes.data_as(ctypes.c_void_p), ctypes.byref(k)), "kv_pool_compact")
        return src[:k.value].copy(), dst[:k.value].copy()

    def fail_alloc_after(self, k: int):
        _check(lib().kv_pool_fail_alloc_after(self._p, int(k)), "kv_pool_fail_alloc_after")


def kv_waste_stats(lens, reservation_tokens: int) -> dict:
    """Contiguous-vs-paged memory waste of requests of the given lengths."""
    import numpy as np
    a = np.ascontiguousarray(lens, dtype=np.int32)
    w = _WasteStats()
    _check(lib().kv_waste_stats(a.ctypes.data_as(ctypes.c_void_p), a.size, int(reservation_tokens),
                                ctypes.byref(w)), "kv_waste_stats")
    return {f: getattr(w, f) for f, _ in _WasteStats._fields_}


class PrefixCache:
    """Block-hash prefix cache over a KVPool (kept alive by this object): exact,
    block-aligned matching from the first token under a tenant key, LRU
    eviction of leaves that only the cache holds."""

    def __init__(self, pool: KVPool):
        self.pool = pool
        self._c = ctypes.c_void_p()
        _check(lib().kv_prefix_cache_create(pool._p, ctypes.byref(self._c)), "kv_prefix_cache_create")

    def close(self):
        if self._c:
            lib().kv_prefix_cache_destroy(self._c)
            self._c = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @staticmethod
    def _tokens(tokens):
        import numpy as np
        return np.ascontiguousarray(tokens, dtype=np.int32)

    def match(self, tokens, salt: int = 0, max_blocks=None):
        """Ids of the longest cached prefix (one reference each for the caller)."""
        import numpy as np
        t = self._tokens(tokens)
        cap = t.size // BLOCK_SIZE if max_blocks is None else int(max_blocks)
        out = np.empty(max(cap, 0), dtype=np.int32)
        n = ctypes.c_int32()
        _check(lib().kv_prefix_match(self._c, t.ctypes.data_as(ctypes.c_void_p), t.size, int(salt) & (2**64 - 1),
                                     cap, out.ctypes.data_as(ctypes.c_void_p), ctypes.byref(n)), "kv_prefix_match")
        return out[:n.value]

    def insert(self, tokens, block_ids, salt: int = 0) -> int:
        import numpy as np
        t = self._tokens(tokens)
        b = np.ascontiguousarray(block_ids, dtype=np.int32)
        n = ctypes.c_int32()
        _check(lib().kv_prefix_insert(self._c, t.ctypes.data_as(ctypes.c_void_p), t.size, int(salt) & (2**64 - 1),
                                      b.ctypes.data_as(ctypes.c_void_p), b.size, ctypes.byref(n)),
               "kv_prefix_insert")
        return int(n.value)

    def evict(self, n: int):
        import numpy as np
        out = np.empty(max(int(n), 0), dtype=np.int32)
        k = ctypes.c_int32()
        _check(lib().kv_prefix_evict(self._c, int(n), out.ctypes.data_as(ctypes.c_void_p), ctypes.byref(k)),
               "kv_prefix_evict")
        return out[:k.value]

    def alloc(self, n: int):
        import numpy as np
        out = np.empty(max(int(n), 0), dtype=np.int32)
        _check(lib().kv_prefix_alloc(self._c, int(n), out.ctypes.data_as(ctypes.c_void_p)), "kv_prefix_alloc")
        return out

    def remap(self, src, dst):
        """The cached blocks src[i] (strictly ascending) are blocks dst[i] from now on (see KVPool.compact)."""
        import numpy as np
        a, b = np.ascontiguousarray(src, dtype=np.int32), np.ascontiguousarray(dst, dtype=np.int32)
        if a.shape != b.shape:
            raise ValueError("src and dst must have the same length")
        _check(lib().kv_prefix_remap(self._c, a.ctypes.data_as(ctypes.c_void_p), b.ctypes.data_as(ctypes.c_void_p),
                                     a.size), "kv_prefix_remap")

    def stats(self) -> dict:
        s = _PrefixStats()
        _check(lib().kv_prefix_stats(self._c, ctypes.byref(s)), "kv_prefix_stats")
        return {f: int(getattr(s, f)) for f, _ in _PrefixStats._fields_}


# ------------------------------------------------------------------ kernels
def reshape_and_cache(k, v, k_cache, v_cache, slot_mapping, k_scale=None, v_scale=None, stream=None):
    """Scatter K/V rows [T][Hkv][128] (bf16) into the paged caches at slot_mapping."""
    _need(k, "k", torch.bfloat16)
    _need(v, "v", torch.bfloat16)
    _need(k_cache, "k_cache", (torch.bfloat16, torch.uint8, torch.float8_e4m3fn))
    _need(v_cache, "v_cache", (torch.bfloat16, torch.uint8, torch.float8_e4m3fn))
    _need(slot_mapping, "slot_mapping", torch.int64)
    T, hkv, d = k.shape
    if d != HEAD_DIM or tuple(v.shape) != (T, hkv, d) or k_cache.shape[1:] != (hkv, BLOCK_SIZE, HEAD_DIM):
        raise ValueError("shape mismatch")
    dt = _cache_dtype(k_cache)
    _check(lib().reshape_and_cache(_ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(slot_mapping),
                                   T, hkv, k_cache.shape[0], dt, _ptr(k_scale), _ptr(v_scale),
                                   _stream(stream)), "reshape_and_cache")


def paged_attention_workspace_size(num_seqs, num_q_heads, max_blocks_per_seq, num_splits=0) -> int:
    return int(lib().paged_attention_workspace_size(num_seqs, num_q_heads, max_blocks_per_seq, num_splits))


def paged_attention_chunked_prefill_workspace_size(num_seqs, total_q_tokens, max_q_len, num_q_heads,
                                                   num_kv_heads, max_blocks_per_seq, num_splits=0) -> int:
    return int(lib().paged_attention_chunked_prefill_workspace_size(
        num_seqs, total_q_tokens, max_q_len, num_q_heads, num_kv_heads, max_blocks_per_seq, num_splits))


def paged_attention_launch_count(num_seqs, total_q_tokens, max_q_len, num_q_heads, num_kv_heads,
                                 max_blocks_per_seq, num_splits=0) -> int:
    return int(lib().paged_attention_launch_count(
        num_seqs, total_q_tokens, max_q_len, num_q_heads, num_kv_heads, max_blocks_per_seq, num_splits))


def _workspace(nbytes, device):
    if nbytes == 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def paged_attention_decode(out, q, k_cache, v_cache, block_tables, context_lens, scale=None,
                           k_scale=None, v_scale=None, num_splits=0, workspace=None, stream=None):
    """Decode attention: out[B][Hq][128] fp32 from q[B][Hq][128] bf16 over the paged cache."""
    _need(out, "out", torch.float32)
    _need(q, "q", torch.bfloat16)
    _need(k_cache, "k_cache")
    _need(v_cache, "v_cache")
    _need(block_tables, "block_tables", torch.int32)
    _need(context_lens, "context_lens", torch.int32)
    B, hq, d = q.shape
    nb, hkv = k_cache.shape[0], k_cache.shape[1]
    mb = block_tables.shape[1]
    if scale is None:
        scale = HEAD_DIM ** -0.5
    need = paged_attention_workspace_size(B, hq, mb, num_splits)
    if workspace is None:
        workspace = _workspace(need, q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().paged_attention_decode(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                        mb, _ptr(context_lens), B, hq, hkv, nb, float(scale),
                                        _cache_dtype(k_cache), _ptr(k_scale), _ptr(v_scale), int(num_splits),
                                        _ptr(workspace), ws_bytes, _stream(stream)), "paged_attention_decode")
    return out


def paged_attention_decode_static_scratch(out, q, k_cache, v_cache, block_tables, context_lens, scale=None,
                                          k_scale=None, v_scale=None, num_splits=0, stream=None):
    """Decode for callers that cannot allocate device memory: same as
    paged_attention_decode, but the split partials live in the library's own
    fixed-size device array (see paged_attention_decode_static_scratch_bytes).
    Calls that overlap on the GPU share that array and must be serialised."""
    _need(out, "out", torch.float32)
    _need(q, "q", torch.bfloat16)
    _need(k_cache, "k_cache")
    _need(v_cache, "v_cache")
    _need(block_tables, "block_tables", torch.int32)
    _need(context_lens, "context_lens", torch.int32)
    B, hq, d = q.shape
    nb, hkv = k_cache.shape[0], k_cache.shape[1]
    if scale is None:
        scale = HEAD_DIM ** -0.5
    _check(lib().paged_attention_decode_static_scratch(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), block_tables.shape[1],
        _ptr(context_lens), B, hq, hkv, nb, float(scale), _cache_dtype(k_cache), _ptr(k_scale), _ptr(v_scale),
        int(num_splits), _stream(stream)), "paged_attention_decode_static_scratch")
    return out


def paged_attention_decode_static_scratch_bytes() -> int:
    return int(lib().paged_attention_decode_static_scratch_bytes())


def paged_attention_chunked_prefill(out, q, cu_q_lens, context_lens, max_q_len, k_cache, v_cache,
                                    block_tables, scale=None, k_scale=None, v_scale=None, num_splits=0,
                                    workspace=None, stream=None):
    """Mixed chunked-prefill / decode attention over the paged cache."""
    _need(out, "out", torch.float32)
    _need(q, "q", torch.bfloat16)
    _need(cu_q_lens, "cu_q_lens", torch.int32)
    _need(context_lens, "context_lens", torch.int32)
    _need(block_tables, "block_tables", torch.int32)
    R, hq, d = q.shape
    B = context_lens.shape[0]
    nb, hkv = k_cache.shape[0], k_cache.shape[1]
    mb = block_tables.shape[1]
    if scale is None:
        scale = HEAD_DIM ** -0.5
    need = paged_attention_chunked_prefill_workspace_size(B, R, int(max_q_len), hq, hkv, mb, num_splits)
    if workspace is None:
        workspace = _workspace(need, q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().paged_attention_chunked_prefill(
        _ptr(out), _ptr(q), _ptr(cu_q_lens), _ptr(context_lens), B, R, int(max_q_len), _ptr(k_cache),
        _ptr(v_cache), _ptr(block_tables), mb, hq, hkv, nb, float(scale), _cache_dtype(k_cache),
        _ptr(k_scale), _ptr(v_scale), int(num_splits), _ptr(workspace), ws_bytes, _stream(stream)),
        "paged_attention_chunked_prefill")
    return out


# ----------------------------------------------------------- latent attention
# These calls are microseconds long on the GPU, so their checks are kept to a few
# cheap attribute reads a tensor (device as a number, dtypes by identity); what is
# wrong is worked out only after something is.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_BF, _I32, _I64 = torch.bfloat16, torch.int32, torch.int64


def _wrong(name, t, dev, dtype, shape):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda or t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on the other tensors' device")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if len(t.shape) != len(shape) or any(b is not None and a != b for a, b in zip(t.shape, shape)):
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _device(name, t):
    """Index of the CUDA device that t is on."""
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _at(name, t, dev, dtype, shape):
    """Address of t, a contiguous CUDA tensor on device `dev` of this dtype and (whole) shape."""
    if t is None or t.get_device() != dev or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _wrong(name, t, dev, dtype, shape)
    return t.data_ptr()


def _at_nd(name, t, dev, dtype, free, ends=()):
    """As _at, for a tensor whose first `free` extents may be anything, the others `ends`."""
    if t is None or t.get_device() != dev or t.dtype is not dtype or t.dim() != free + len(ends) or \
            (ends and t.shape[free:] != ends) or not t.is_contiguous():
        _wrong(name, t, dev, dtype, (None,) * free + ends)
    return t.data_ptr()


def _rows_at(name, t, dev, rows, width):
    """Rows of `width` bf16 values whose first dimension may be strided: (address, row stride)."""
    if t is None or t.get_device() != dev or t.dtype is not _BF or t.shape != (rows, width):
        _wrong(name, t, dev, _BF, (rows, width))
    # (without rows no stride means anything, and with one row its distance to the next does not)
    row, one = t.stride()
    if one != 1 and rows > 0:
        raise ValueError(f"{name}'s rows must be contiguous")
    return t.data_ptr(), row if rows > 1 else width


def _call_on(dev, stream, fn, *args):
    """fn(*args, stream) with device `dev` current: its current stream unless one is given."""
    if stream is None:
        raw = _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream
    elif stream.device_index != dev:
        raise ValueError("stream must belong to the tensors' device")
    else:
        raw = stream.cuda_stream
    if _get_device() == dev:
        return fn(*args, raw)
    with torch.cuda.device(dev):
        return fn(*args, raw)


def _scratch(workspace, dev, stream, size, *sizes):
    """(address, bytes, tensor) of the given workspace, or of a new one of size(*sizes) bytes.
    The new one belongs to the stream that the call runs on: it is given back as the call
    returns, and what that stream does next with the memory comes after the call's kernels."""
    if workspace is None:
        need = size(*sizes)
        if not need:
            return None, 0, None
        if stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=torch.device("cuda", dev))
        else:
            with torch.cuda.stream(stream):
                workspace = torch.empty(need, dtype=torch.uint8, device=torch.device("cuda", dev))
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the other tensors' device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def kv_build_step_tables(block_tables, context_lens, new_lens, free_blocks, num_blocks, cu_q_lens, total_lens,
                         slot_mapping, positions, totals, stream=None):
    """Block tables and slot numbers of one step from request lengths, on the device.

    Sequence s holds context_lens[s] tokens and gains new_lens[s]; the blocks it
    newly needs come from free_blocks in sequence order and go into its row of
    block_tables.  Outputs (int32; slot_mapping int64): cu_q_lens [B+1],
    total_lens [B], slot_mapping and positions [max_tokens], totals [2] (rows,
    free blocks taken).  Lengths that do not fit refuse the sequence and set the
    device status (see kv_last_device_status)."""
    dev = _device("block_tables", block_tables)
    tables = _at_nd("block_tables", block_tables, dev, _I32, 2)
    B, mb = block_tables.shape
    free = _at_nd("free_blocks", free_blocks, dev, _I32, 1)
    slots = _at_nd("slot_mapping", slot_mapping, dev, _I64, 1)
    n, each = slot_mapping.shape[0], (B,)
    _check(_call_on(dev, stream, lib().kv_build_step_tables, tables, mb,
                    _at("context_lens", context_lens, dev, _I32, each), _at("new_lens", new_lens, dev, _I32, each), B,
                    free, free_blocks.shape[0], int(num_blocks), _at("cu_q_lens", cu_q_lens, dev, _I32, (B + 1,)),
                    _at("total_lens", total_lens, dev, _I32, each), slots,
                    _at("positions", positions, dev, _I32, (n,)), n, _at("totals", totals, dev, _I32, (2,))),
           "kv_build_step_tables")


def reshape_and_cache_latent(latent, rope, cache, slot_mapping, stream=None):
    """Write latent rows [T][512] and rotary keys [T][64] (bf16; rows may be views
    of a wider tensor) into the paged latent cache [num_blocks][16][576]."""
    dev = _device("cache", cache)
    nb, T = cache.shape[0], 0 if slot_mapping is None else slot_mapping.shape[0]
    c = _at("cache", cache, dev, _BF, (nb, BLOCK_SIZE, _LATENT_ROW))
    slots = _at("slot_mapping", slot_mapping, dev, _I64, (T,))
    lat, ls = _rows_at("latent", latent, dev, T, LATENT_DIM)
    rp, rs = _rows_at("rope", rope, dev, T, LATENT_ROPE_DIM)
    _check(_call_on(dev, stream, lib().reshape_and_cache_latent, lat, ls, rp, rs, c, slots, T, nb),
           "reshape_and_cache_latent")


def paged_latent_attention_workspace_size(num_seqs, total_q_tokens, num_heads, max_blocks_per_seq) -> int:
    return int(lib().paged_latent_attention_workspace_size(num_seqs, total_q_tokens, num_heads, max_blocks_per_seq))


def paged_latent_attention(out, q, cache, block_tables, context_lens, cu_q_lens=None, scale=None, workspace=None,
                           stream=None):
    """Attention over the paged latent cache, absorbed form: out[R][H][512] from
    q[R][H][576] (bf16), one row a sequence, or cu_q_lens [B+1] rows.  scale
    defaults to (128 + 64) ** -0.5, the expanded form's."""
    dev = _device("q", q)
    qp = _at_nd("q", q, dev, _BF, 2, (_LATENT_ROW,))
    R, h, _ = q.shape
    tables = _at_nd("block_tables", block_tables, dev, _I32, 2)
    B, mb = block_tables.shape
    if cu_q_lens is None and R != B:
        raise ValueError("without cu_q_lens, q must have one row a sequence")
    c = _at_nd("cache", cache, dev, _BF, 1, (BLOCK_SIZE, _LATENT_ROW))
    L = lib()
    ws, nbytes, _keep = _scratch(workspace, dev, stream, L.paged_latent_attention_workspace_size, B, R, h, mb)
    _check(_call_on(dev, stream, L.paged_latent_attention, _at("out", out, dev, _BF, (R, h, LATENT_DIM)), qp,
                    None if cu_q_lens is None else _at("cu_q_lens", cu_q_lens, dev, _I32, (B + 1,)),
                    _at("context_lens", context_lens, dev, _I32, (B,)), B, R, c, tables, mb, h, cache.shape[0],
                    _EXPANDED_QK ** -0.5 if scale is None else float(scale), ws, nbytes), "paged_latent_attention")
    return out


def latent_prefill_attention_workspace_size(num_seqs, total_q_tokens, num_heads) -> int:
    return int(lib().latent_prefill_attention_workspace_size(num_seqs, total_q_tokens, num_heads))


def latent_prefill_attention(out, q, kv, k_rope, cu_q_lens, cu_k_lens, scale=None, workspace=None, stream=None):
    """Prompt attention over expanded latents: out[Rq][H][128] from q[Rq][H][192],
    kv[Rk][H][256] (key part, value) and the shared rotary keys k_rope[Rk][64]
    (bf16; k_rope's rows may be views of a wider tensor), ragged by cu_q_lens and
    cu_k_lens [B+1], causal from the end.  scale defaults to 192 ** -0.5."""
    dev = _device("q", q)
    qp = _at_nd("q", q, dev, _BF, 2, (_EXPANDED_QK,))
    R, h, _ = q.shape
    kvp = _at_nd("kv", kv, dev, _BF, 1, (h, 2 * HEAD_DIM))
    K = kv.shape[0]
    rp, rs = _rows_at("k_rope", k_rope, dev, K, LATENT_ROPE_DIM)
    cu_q = _at_nd("cu_q_lens", cu_q_lens, dev, _I32, 1)
    B = cu_q_lens.shape[0] - 1
    if B < 0:
        raise ValueError("cu_q_lens must have at least one entry")
    L = lib()
    ws, nbytes, _keep = _scratch(workspace, dev, stream, L.latent_prefill_attention_workspace_size, B, R, h)
    _check(_call_on(dev, stream, L.latent_prefill_attention, _at("out", out, dev, _BF, (R, h, HEAD_DIM)), qp, kvp, rp,
                    rs, cu_q, _at("cu_k_lens", cu_k_lens, dev, _I32, (B + 1,)), B, R, K, h,
                    _EXPANDED_QK ** -0.5 if scale is None else float(scale), ws, nbytes), "latent_prefill_attention")
    return out


# ------------------------------------------------- shared prefixes, forks, moves
_CACHE_TYPES = (torch.bfloat16, torch.uint8, torch.float8_e4m3fn)


def _cache_at(name, t, dev, shape=None):
    """Address of a K or V cache [num_blocks][Hkv][16][128], bf16 or e4m3."""
    if t is None or t.get_device() != dev or t.dtype not in _CACHE_TYPES or t.dim() != 4 or \
            t.shape[2:] != (BLOCK_SIZE, HEAD_DIM) or (shape is not None and t.shape != shape) or not t.is_contiguous():
        if t is not None and t.is_cuda and t.dtype not in _CACHE_TYPES:
            raise ValueError(f"{name} must be bf16 or e4m3 (uint8 or float8_e4m3fn), got {t.dtype}")
        _wrong(name, t, dev, None if t is None else t.dtype, (None, None, BLOCK_SIZE, HEAD_DIM) if shape is None else shape)
    return t.data_ptr()


def paged_attention_shared_prefix_workspace_size(num_seqs, total_q_tokens, max_q_len, num_groups, num_q_heads,
                                                 num_kv_heads, max_prefix_len, max_tail_len) -> int:
    return _fast().paged_attention_shared_prefix_workspace_size(
        num_seqs, total_q_tokens, max_q_len, num_groups, num_q_heads, num_kv_heads, max_prefix_len, max_tail_len)


def paged_attention_shared_prefix_way(num_seqs, total_q_tokens, max_q_len, num_groups, num_q_heads, num_kv_heads,
                                      max_prefix_len, max_tail_len, fp8=False) -> int:
    """How a call of these sizes and bounds is done: 0 whole contexts, 1 prefixes apart, 2 joined."""
    return lib().paged_attention_shared_prefix_way(num_seqs, total_q_tokens, max_q_len, num_groups, num_q_heads,
                                                   num_kv_heads, max_prefix_len, max_tail_len, 1 if fp8 else 0)


def paged_attention_shared_prefix(out, q, k_cache, v_cache, block_tables, context_lens, cu_groups, prefix_lens,
                                  cu_q_lens=None, max_q_len=None, max_prefix_len=None, max_tail_len=None, scale=None,
                                  k_scale=None, v_scale=None, workspace=None, stream=None):
    """Decode attention that attends a prefix once for all sequences that share it:
    out[R][Hq][128] from q[R][Hq][128] (bf16), one row a sequence, or cu_q_lens [B+1]
    rows (at most max_q_len each).

    Sequences cu_groups[g] .. cu_groups[g+1]-1 (int32 [G+1]) have their first
    prefix_lens[g] tokens in common (int32 [G]; rounded down to whole blocks, and read
    through the first of these sequences' row of block_tables).  max_prefix_len and
    max_tail_len bound the prefixes and what follows them; without them the width of
    block_tables does, which sizes grids and workspace for far more than most batches
    hold."""
    dev = _device("q", q)
    qp = _at_nd("q", q, dev, _BF, 2, (HEAD_DIM,))
    R, hq, _ = q.shape
    tables = _at_nd("block_tables", block_tables, dev, _I32, 2)
    B, mb = block_tables.shape
    if cu_q_lens is None:
        if R != B:
            raise ValueError("without cu_q_lens, q must have one row a sequence")
        n = 1
    else:
        n = max(R, 1) if max_q_len is None else int(max_q_len)
    kc = _cache_at("k_cache", k_cache, dev)
    vc = _cache_at("v_cache", v_cache, dev, k_cache.shape)
    nb, hkv = k_cache.shape[0], k_cache.shape[1]
    if v_cache.dtype is not k_cache.dtype:
        raise ValueError("k_cache and v_cache must have one dtype")
    groups = _at_nd("cu_groups", cu_groups, dev, _I32, 1)
    G = cu_groups.shape[0] - 1
    if G < 0:
        raise ValueError("cu_groups must have at least one entry")
    longest = mb * BLOCK_SIZE
    mp = longest if max_prefix_len is None else int(max_prefix_len)
    mt = longest if max_tail_len is None else int(max_tail_len)
    L = _fast()
    ws, nbytes, _keep = _scratch(workspace, dev, stream, L.paged_attention_shared_prefix_workspace_size, B, R, n, G, hq,
                                 hkv, mp, mt)
    each = (hkv,)
    _check(_call_on(dev, stream, L.paged_attention_shared_prefix, _at("out", out, dev, _BF, (R, hq, HEAD_DIM)), qp,
                    None if cu_q_lens is None else _at("cu_q_lens", cu_q_lens, dev, _I32, (B + 1,)),
                    _at("context_lens", context_lens, dev, _I32, (B,)), B, R, n, groups,
                    _at("prefix_lens", prefix_lens, dev, _I32, (G,)), G, mp, mt, kc, vc, tables, mb, hq, hkv, nb,
                    HEAD_DIM ** -0.5 if scale is None else float(scale), _cache_dtype(k_cache),
                    None if k_scale is None else _at("k_scale", k_scale, dev, torch.float32, each),
                    None if v_scale is None else _at("v_scale", v_scale, dev, torch.float32, each), ws, nbytes),
           "paged_attention_shared_prefix")
    return out


def kv_copy_blocks(caches, src, dst, stream=None):
    """Copy block src[i] to block dst[i] (int32) in every cache of the list: tensors of
    one shape and dtype whose first dimension counts blocks (the K and V caches of all
    layers, or latent caches).  A pair of negative ids is skipped."""
    dev = _device("src", src)
    s = _at_nd("src", src, dev, _I32, 1)
    n = src.shape[0]
    d = _at("dst", dst, dev, _I32, (n,))
    if not caches:
        return
    shape, dtype = caches[0].shape, caches[0].dtype
    if len(shape) < 2 or shape[0] < 1:
        raise ValueError("caches must be [num_blocks][...]")
    _check(_call_on(dev, stream, _fast().kv_copy_blocks, [_at("caches", t, dev, dtype, shape) for t in caches],
                    caches[0].nbytes // shape[0], shape[0], s, d, n), "kv_copy_blocks")


def kv_fork_tables(block_tables, context_lens, parents, free_blocks, child_tables, child_lens, copy_src, copy_dst, taken,
                   first_keeps=False, stream=None):
    """Fork sequences on the device: child c shares the full blocks of sequence
    parents[c]; a partly filled last block stays with the parent's first child if
    first_keeps, and every other child gets a block of free_blocks, to be filled by
    kv_copy_blocks(caches, copy_src, copy_dst).  Outputs (int32): child_tables [C][mb],
    child_lens, copy_src, copy_dst [C], taken [1] (free blocks used)."""
    dev = _device("block_tables", block_tables)
    tables = _at_nd("block_tables", block_tables, dev, _I32, 2)
    P, mb = block_tables.shape
    par = _at_nd("parents", parents, dev, _I32, 1)
    C = parents.shape[0]
    free, each = _at_nd("free_blocks", free_blocks, dev, _I32, 1), (C,)
    _check(_call_on(dev, stream, _fast().kv_fork_tables, tables, mb, _at("context_lens", context_lens, dev, _I32, (P,)), P,
                    par, C, 1 if first_keeps else 0, free, free_blocks.shape[0],
                    _at("child_tables", child_tables, dev, _I32, (C, mb)), _at("child_lens", child_lens, dev, _I32, each),
                    _at("copy_src", copy_src, dev, _I32, each), _at("copy_dst", copy_dst, dev, _I32, each),
                    _at("taken", taken, dev, _I32, (1,))), "kv_fork_tables")


def kv_remap_tables(block_tables, context_lens, src, dst, stream=None):
    """Rewrite block tables after blocks have moved: of each row's used entries, those
    equal to src[i] become dst[i] (int32, src strictly ascending)."""
    dev = _device("block_tables", block_tables)
    tables = _at_nd("block_tables", block_tables, dev, _I32, 2)
    B, mb = block_tables.shape
    s = _at_nd("src", src, dev, _I32, 1)
    n = src.shape[0]
    _check(_call_on(dev, stream, _fast().kv_remap_tables, tables, mb, _at("context_lens", context_lens, dev, _I32, (B,)), B,
                    s, _at("dst", dst, dev, _I32, (n,)), n), "kv_remap_tables")


def _swap_args(k_cache, v_cache, block_ids, host_k, host_v):
    _need(k_cache, "k_cache", (torch.bfloat16, torch.uint8, torch.float8_e4m3fn))
    _need(v_cache, "v_cache", (torch.bfloat16, torch.uint8, torch.float8_e4m3fn))
    _need(block_ids, "block_ids", torch.int32)
    n = block_ids.numel()
    for name, h in (("host_k", host_k), ("host_v", host_v)):
        _need(h, name, k_cache.dtype, dev=False)
        if h.is_cuda or not h.is_pinned():
            raise ValueError(f"{name} must be pinned host memory")
        if tuple(h.shape) != (n,) + tuple(k_cache.shape[1:]):
            raise ValueError(f"{name} must be [n][Hkv][16][128]")
    return n


def kv_swap_out(k_cache, v_cache, block_ids, host_k, host_v, stream=None):
    """Copy the listed blocks' K/V tiles to pinned host tensors [n][Hkv][16][128]."""
    n = _swap_args(k_cache, v_cache, block_ids, host_k, host_v)
    _check(lib().kv_swap_out(_ptr(k_cache), _ptr(v_cache), k_cache.shape[0], k_cache.shape[1],
                             _cache_dtype(k_cache), _ptr(block_ids), n, _ptr(host_k), _ptr(host_v),
                             _stream(stream)), "kv_swap_out")


def kv_swap_in(k_cache, v_cache, block_ids, host_k, host_v, stream=None):
    """Copy pinned host tensors [n][Hkv][16][128] into the listed (distinct) blocks."""
    n = _swap_args(k_cache, v_cache, block_ids, host_k, host_v)
    _check(lib().kv_swap_in(_ptr(k_cache), _ptr(v_cache), k_cache.shape[0], k_cache.shape[1],
                            _cache_dtype(k_cache), _ptr(block_ids), n, _ptr(host_k), _ptr(host_v),
                            _stream(stream)), "kv_swap_in")


def kv_trace_prefill(enable: bool):
    """Record CUDA events around the chunk kernel of each mixed call (tracing aid)."""
    _check(lib().kv_trace_prefill(1 if enable else 0), "kv_trace_prefill")


def kv_trace_prefill_kernel_ms() -> float:
    """Duration of the last traced chunk kernel in ms (waits for it); < 0 if none."""
    return float(lib().kv_trace_prefill_kernel_ms())


def kv_last_device_status(stream=None) -> int:
    """Synchronises the stream; returns 0 or 5 (device data out of range), clearing it."""
    st = lib().kv_last_device_status(_stream(stream))
    if st not in (0, 5):
        raise KVError(st, "kv_last_device_status")
    return st


def kv_last_device_status_flags() -> int:
    return int(lib().kv_last_device_status_flags())


def kv_selftest_bounded_wait(limit_us: int = 10000, stream=None) -> None:
    """Launches the failure-path self-test: a device wait that nothing ends gives
    up after limit_us and sets the timeout flag (8) in the status word."""
    _check(lib().kv_selftest_bounded_wait(int(limit_us), _stream(stream)), "kv_selftest_bounded_wait")
