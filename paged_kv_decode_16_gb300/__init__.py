"""GB300-native paged GQA decode attention: thin Python binding of libpagedkv.so.

Every function here has the name of the C-ABI entry point it calls
(``include/pagedkv.h``) and only marshals arguments: torch tensors are
checked for device, dtype and contiguity and passed as raw device pointers
(through ctypes, or for the calls with selected pages by a small native module);
the current torch CUDA stream is passed as the stream.  All computation runs
in the library's CUDA kernels.  There is no fallback: if the library was not
built, or a call fails, an exception is raised.

PyTorch is used only to own device memory and streams.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import numpy as np
import torch

from . import build as _build

__all__ = [
    "PagedKVError", "load_library", "library_path", "pkv_status_string", "pkv_version",
    "Pool", "kv_pool_create", "PrefixCache", "kv_append", "kv_append_rope", "kv_gather",
    "paged_decode_workspace_size", "paged_decode_step_rope", "paged_decode_attention_prefix",
    "paged_decode_prefix_workspace_size", "alloc_prefix_workspace", "DEV_BAD_PREFIX",
    "paged_decode_attention_multi", "paged_decode_multi_workspace_size", "alloc_multi_workspace",
    "check_bounded_wait",
    "paged_decode_plan", "paged_decode_run", "paged_decode_combine", "paged_decode_attention",
    "paged_decode_step", "paged_decode_attention_no_alloc", "NO_ALLOC_SCRATCH_BYTES",
    "paged_decode_step_host", "paged_decode_step_host_workspace_size", "alloc_step_host_workspace",
    "kv8_pool_create", "kv8_append", "kv8_append_rope", "paged_decode_kv8_workspace_size",
    "alloc_kv8_workspace", "paged_decode_attention_kv8", "paged_decode_attention_multi_kv8",
    "paged_decode_step_kv8", "DEV_BAD_SEQ",
    "paged_tables_build", "Rope", "kv_append_tokens", "kv_page_bounds",
    "paged_select_workspace_size", "alloc_select_workspace", "paged_select_pages",
    "paged_decode_attention_selected", "DEV_NO_PAGES",
    "pkv_read_device_status", "pkv_read_no_alloc_status", "alloc_workspace", "DEV_BAD_PAGE", "DEV_BAD_LEN", "DEV_TIMEOUT",
    "VARIANT_AUTO", "VARIANT_CUDA_CORES", "VARIANT_TENSOR_CORES", "VARIANT_TCGEN05",
]

PKV_OK = 0
STATUS_NAMES = {0: "PKV_OK", 1: "PKV_ERR_INVALID_ARG", 2: "PKV_ERR_UNSUPPORTED",
                3: "PKV_ERR_ALIAS", 4: "PKV_ERR_OUT_OF_PAGES", 5: "PKV_ERR_WORKSPACE",
                6: "PKV_ERR_CUDA", 7: "PKV_ERR_DEVICE_CHECK", 8: "PKV_ERR_REFCOUNT"}
DEV_BAD_PAGE, DEV_BAD_LEN, DEV_TIMEOUT, DEV_BAD_PREFIX = 0x1, 0x2, 0x4, 0x8
DEV_BAD_SEQ, DEV_NO_PAGES = 0x10, 0x20
# decode kernels (pkv_decode_variant)
VARIANT_AUTO, VARIANT_CUDA_CORES, VARIANT_TENSOR_CORES, VARIANT_TCGEN05 = 0, 1, 2, 3
# size of the library's fixed device scratch (PKV_NO_ALLOC_SCRATCH_BYTES)
NO_ALLOC_SCRATCH_BYTES = 32 << 20
_DT = {torch.float16: 0, torch.bfloat16: 1}

# fields of pkv_prefix_cache_stats, in order (all uint64)
PREFIX_STATS_FIELDS = ("lookups", "hits", "misses", "pages_hit", "pages_missed",
                       "pages_inserted", "pages_evicted")

_lib = None


class PagedKVError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        self.name = STATUS_NAMES.get(code, str(code))
        super().__init__(f"{where}: {self.name} ({pkv_status_string(code)})")


def library_path() -> str:
    return _build.LIB


def load_library(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libpagedkv.so (building it first when missing and nvcc is present)."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB
    if not os.path.exists(path):
        if not build_if_missing:
            raise RuntimeError(f"CUDA library not built: {path}")
        _build.build_library()
    lib = ctypes.CDLL(path)
    V, I, Z, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    D, L = ctypes.c_double, ctypes.c_int64
    sig = {
        "pkv_status_string": ([I], ctypes.c_char_p),
        "pkv_version": ([], I),
        "kv_pool_create": ([I, I, I, I, I, V, V, ctypes.POINTER(V)], I),
        "kv_pool_destroy": ([V], I),
        "kv_pool_k": ([V], V),
        "kv_pool_v": ([V], V),
        "kv_pool_alloc_pages": ([V, I, V], I),
        "kv_pool_retain_pages": ([V, V, I], I),
        "kv_pool_release_pages": ([V, V, I], I),
        "kv_pool_free_count": ([V], I),
        "kv_pool_refcount": ([V, ctypes.c_int32], I),
        "kv_pool_info": ([V, V, V, V, V, V], I),
        "kv_append": ([V, V, V, V, I, V, I, V, V], I),
        "pkv_prefix_cache_create": ([V, ctypes.POINTER(V)], I),
        "pkv_prefix_cache_destroy": ([V], I),
        "pkv_prefix_cache_insert": ([V, V, I, V, ctypes.POINTER(I)], I),
        "pkv_prefix_cache_match": ([V, V, I, V, I, ctypes.POINTER(I)], I),
        "pkv_prefix_cache_evict": ([V, I, ctypes.POINTER(I)], I),
        "pkv_prefix_cache_pages": ([V], I),
        "pkv_prefix_cache_get_stats": ([V, I, V], I),
        "kv_append_rope": ([V, V, V, V, V, I, V, I, I, ctypes.c_double, V, V, F, V, V, V], I),
        "paged_decode_prefix_workspace_size": ([I, I, I, I, I, I, ctypes.POINTER(Z)], I),
        "paged_decode_multi_workspace_size": ([I, I, I, I, I, I, I, ctypes.POINTER(Z)], I),
        "pkv_check_bounded_wait": ([ctypes.c_uint32, V, V, V], I),
        "paged_decode_attention_multi": ([V, V, V, V, I, V, I, I, I, I, I, I, I, I, F, V, V, Z, I,
                                          I, V], I),
        "paged_decode_attention_prefix": ([V, V, V, V, I, V, I, I, I, I, I, I, I, F, I, V, V, Z,
                                           I, I, V], I),
        "paged_decode_step_rope": ([V, V, V, V, V, V, V, I, V, I, I, I, I, I, I, I, F,
                                    ctypes.c_double, V, V, F, V, V, Z, I, I, V], I),
        "kv_gather": ([V, V, I, V, I, I, V, V, V, V], I),
        "paged_decode_workspace_size": ([I, I, I, I, I, I, ctypes.POINTER(Z)], I),
        "paged_decode_plan": ([V, I, I, I, I, I, I, I, I, V, Z, V], I),
        "paged_decode_run": ([V, V, V, V, I, I, I, I, I, I, I, I, F, V, V, Z, I, I, I, V], I),
        "paged_decode_combine": ([I, I, I, I, I, V, V, Z, I, I, V], I),
        "paged_decode_attention": ([V, V, V, V, I, V, I, I, I, I, I, I, I, F, V, V, Z, I, I, V],
                                   I),
        "paged_decode_step": ([V, V, V, V, V, V, V, I, V, I, I, I, I, I, I, I, F, V, V, Z, I, I,
                               V], I),
        "paged_decode_attention_no_alloc": ([V, V, V, V, I, V, I, I, I, I, I, I, I, F, V, I, I,
                                             V], I),
        "paged_decode_step_host": ([V, V, V, V, V, V, V, I, V, I, I, I, I, I, I, I, F, V, V, Z, I,
                                    I, V], I),
        "paged_decode_step_host_workspace_size": ([I, I, I, I, I, I, I, ctypes.POINTER(Z)], I),
        "kv8_pool_create": ([I, I, I, I, V, V, V, ctypes.POINTER(V)], I),
        "kv8_pool_scales": ([V], V),
        "kv8_append": ([V, V, V, I, V, I, I, V, V, I, V, V], I),
        "kv8_append_rope": ([V, V, V, V, I, V, I, I, V, V, I, I, ctypes.c_double, V, V, F, V, V,
                             V], I),
        "paged_decode_kv8_workspace_size": ([I, I, I, I, I, I, ctypes.POINTER(Z)], I),
        "paged_decode_attention_kv8": ([V, V, V, V, V, I, V, I, I, I, I, I, I, I, F, V, V, Z, I,
                                        V], I),
        "paged_decode_attention_multi_kv8": ([V, V, V, V, V, I, V, I, I, I, I, I, I, I, I, F, V,
                                              V, Z, I, V], I),
        "paged_decode_step_kv8": ([V, V, V, V, V, V, V, V, I, V, I, I, I, I, I, I, I, F,
                                   ctypes.c_double, V, V, F, V, V, Z, I, V], I),
        "paged_tables_build": ([V, V, I, V, I, V, V, I, I, V, I, V, V, I, V, V, V, V, V], I),
        "pkv_rope_init": ([V, I, D, I, D, I, D, D, D, D], I),
        "kv_append_tokens": ([V, V, L, V, L, V, I, V, L, I, V, V, V, V, F, V, L, V, V], I),
        "kv_page_bounds": ([V, V, I, V, V, V], I),
        "paged_select_workspace_size": ([I, I, I, ctypes.POINTER(Z)], I),
        "paged_select_pages": ([V, V, V, I, V, I, I, I, I, I, I, I, I, I, I, V, V, Z, V, V], I),
        "paged_decode_attention_selected": ([V, V, V, V, I, V, V, I, I, I, I, I, I, I, I, F, V, V,
                                             V], I),
        "pkv_read_device_status": ([V, ctypes.POINTER(ctypes.c_uint32)], I),
        "pkv_read_no_alloc_status": ([ctypes.POINTER(ctypes.c_uint32)], I),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def pkv_status_string(code: int) -> str:
    return load_library().pkv_status_string(int(code)).decode()


def pkv_version() -> int:
    return load_library().pkv_version()


def _check(code: int, where: str):
    if code != PKV_OK:
        raise PagedKVError(code, where)


def _ptr(t: torch.Tensor | None):
    # ctypes converts a plain int for a c_void_p argument
    return None if t is None else t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _on_current_device(t) -> bool:
    # the library launches on the current device's stream and, for the
    # allocation-free call, uses that device's scratch: operands elsewhere
    # would be read by the wrong GPU
    idx = t.device.index
    return idx is None or idx == torch.cuda.current_device()


def _dev(t: torch.Tensor, name: str, dtype=None, ndim=None):
    """A contiguous CUDA tensor on the current device (of dtype / ndim when
    given), else raise."""
    try:
        ok = (t.is_cuda and t.is_contiguous() and (dtype is None or t.dtype == dtype)
              and (ndim is None or t.dim() == ndim) and _on_current_device(t))
    except AttributeError:
        raise TypeError(f"{name} must be a torch tensor") from None
    if ok:
        return t
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if not _on_current_device(t):
        raise ValueError(f"{name} is on {t.device} but the current device is "
                         f"cuda:{torch.cuda.current_device()}: call inside "
                         f"torch.cuda.device({t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise ValueError(f"dtype {t.dtype} not supported (float16 or bfloat16)")
    return _DT[t.dtype]


# ---------------------------------------------------------------------------
class Pool:
    """Handle of a page pool (kv_pool_create).  Borrowed torch tensors are kept
    alive by the handle."""

    def __init__(self, handle: int, k: torch.Tensor | None, v: torch.Tensor | None,
                 num_pages: int, page_size: int, n_kv_heads: int, head_dim: int, dtype):
        self._h = ctypes.c_void_p(handle)
        self._address = handle  # of the pool (None once destroyed)
        self.device = None
        self._keep = (k, v)
        self.num_pages, self.page_size = num_pages, page_size
        self.n_kv_heads, self.head_dim, self.dtype = n_kv_heads, head_dim, dtype

    @property
    def handle(self):
        if not self._h:
            raise ValueError("pool destroyed")
        return self._h

    def k_ptr(self) -> int:
        return load_library().kv_pool_k(self.handle) or 0

    def v_ptr(self) -> int:
        return load_library().kv_pool_v(self.handle) or 0

    def scales_ptr(self) -> int:
        """The block scales of an 8-bit pool (0: a 16-bit pool)."""
        return load_library().kv8_pool_scales(self.handle) or 0

    def alloc_pages(self, n: int) -> list[int]:
        ids = (ctypes.c_int32 * max(n, 1))()
        _check(load_library().kv_pool_alloc_pages(self.handle, n, ids), "kv_pool_alloc_pages")
        return list(ids[:n])

    def retain_pages(self, ids) -> None:
        arr = (ctypes.c_int32 * max(len(ids), 1))(*ids)
        _check(load_library().kv_pool_retain_pages(self.handle, arr, len(ids)),
               "kv_pool_retain_pages")

    def release_pages(self, ids) -> None:
        arr = (ctypes.c_int32 * max(len(ids), 1))(*ids)
        _check(load_library().kv_pool_release_pages(self.handle, arr, len(ids)),
               "kv_pool_release_pages")

    def free_count(self) -> int:
        return load_library().kv_pool_free_count(self.handle)

    def refcount(self, page_id: int) -> int:
        return load_library().kv_pool_refcount(self.handle, int(page_id))

    def destroy(self) -> None:
        if self._h:
            code = load_library().kv_pool_destroy(self._h)
            self._h = ctypes.c_void_p(None)
            self._address = None
            self._keep = (None, None)
            _check(code, "kv_pool_destroy")

    def __del__(self):
        try:
            if self._h:
                load_library().kv_pool_destroy(self._h)
        except Exception:
            pass


def kv_pool_create(num_pages: int, page_size: int, n_kv_heads: int, head_dim: int,
                   dtype=torch.bfloat16, k_pool: torch.Tensor | None = None,
                   v_pool: torch.Tensor | None = None) -> Pool:
    """Create a pool; with k_pool/v_pool given ([NP, Hkv, P, D] device tensors)
    the pool borrows them, otherwise it allocates device memory itself."""
    if (k_pool is None) != (v_pool is None):
        raise ValueError("give both k_pool and v_pool or neither")
    code_dt = _DT.get(dtype)
    if code_dt is None:
        raise ValueError(f"dtype {dtype} not supported")
    if k_pool is not None:
        shape = (num_pages, n_kv_heads, page_size, head_dim)
        for name, t in (("k_pool", k_pool), ("v_pool", v_pool)):
            _dev(t, name, dtype, 4)
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} shape {tuple(t.shape)} != {shape}")
    h = ctypes.c_void_p()
    _check(load_library().kv_pool_create(num_pages, page_size, n_kv_heads, head_dim, code_dt,
                                         _ptr(k_pool), _ptr(v_pool), ctypes.byref(h)),
           "kv_pool_create")
    pool = Pool(h.value, k_pool, v_pool, num_pages, page_size, n_kv_heads, head_dim, dtype)
    # the device of the pool's memory (None: borrowed addresses without a GPU)
    pool.device = _get_device() if k_pool is not None or torch.cuda.is_available() else None
    return pool


class PrefixCache:
    """Host radix tree of cached prompt prefixes over a pool (whole pages of
    token ids -> pool pages).  `pool` is a Pool or a raw pool handle; it must
    outlive the cache.  match() hands the caller one reference per returned
    page (release them through the pool when the sequence ends)."""

    def __init__(self, pool):
        self._pool = pool
        h = pool.handle if isinstance(pool, Pool) else pool
        self._h = ctypes.c_void_p()
        _check(load_library().pkv_prefix_cache_create(h, ctypes.byref(self._h)),
               "pkv_prefix_cache_create")
        ps = ctypes.c_int()
        _check(load_library().kv_pool_info(h, None, ctypes.byref(ps), None, None, None),
               "kv_pool_info")
        self._page_size = ps.value

    @staticmethod
    def _i32(xs):
        # contiguous int32 numpy arrays are passed without a copy
        if isinstance(xs, np.ndarray) and xs.dtype == np.int32 and xs.flags.c_contiguous:
            return xs.ctypes.data if xs.size else None
        return (ctypes.c_int32 * max(len(xs), 1))(*[int(x) for x in xs])

    def insert(self, tokens, pages) -> int:
        """Cache the full pages of `tokens` stored in `pages`; returns how many
        pages were new to the cache."""
        n = ctypes.c_int()
        _check(load_library().pkv_prefix_cache_insert(self._h, self._i32(tokens), len(tokens),
                                                      self._i32(pages), ctypes.byref(n)),
               "pkv_prefix_cache_insert")
        return n.value

    def match(self, tokens, max_pages: int | None = None) -> list[int]:
        """Pages of the longest cached whole-page prefix of `tokens` (retained
        for the caller)."""
        cap = len(tokens) // self._page_size if max_pages is None else int(max_pages)
        out = (ctypes.c_int32 * max(cap, 1))()
        n = ctypes.c_int()
        _check(load_library().pkv_prefix_cache_match(self._h, self._i32(tokens), len(tokens), out,
                                                     cap, ctypes.byref(n)),
               "pkv_prefix_cache_match")
        return out[:n.value]

    def evict(self, n_pages: int) -> int:
        n = ctypes.c_int()
        _check(load_library().pkv_prefix_cache_evict(self._h, int(n_pages), ctypes.byref(n)),
               "pkv_prefix_cache_evict")
        return n.value

    def pages(self) -> int:
        return load_library().pkv_prefix_cache_pages(self._h)

    def stats(self, reset: bool = False) -> dict:
        """Lookup, hit and miss counters and pages inserted / evicted
        (pkv_prefix_cache_get_stats); reset zeroes them after reading."""
        buf = (ctypes.c_uint64 * len(PREFIX_STATS_FIELDS))()
        _check(load_library().pkv_prefix_cache_get_stats(self._h, int(bool(reset)), buf),
               "pkv_prefix_cache_get_stats")
        return dict(zip(PREFIX_STATS_FIELDS, (int(x) for x in buf)))

    def destroy(self) -> None:
        if self._h:
            h, self._h = self._h, ctypes.c_void_p(None)
            _check(load_library().pkv_prefix_cache_destroy(h), "pkv_prefix_cache_destroy")

    def __del__(self):
        try:
            if self._h:
                load_library().pkv_prefix_cache_destroy(self._h)
        except Exception:
            pass


def kv_append(pool: Pool, k_new: torch.Tensor, v_new: torch.Tensor, page_table: torch.Tensor,
              positions: torch.Tensor, dev_status: torch.Tensor | None = None,
              stream=None) -> None:
    """Write k_new/v_new [B, Hkv, D] into slot positions[b] of each sequence."""
    _dev(k_new, "k_new", pool.dtype, 3)
    _dev(v_new, "v_new", pool.dtype, 3)
    _dev(page_table, "page_table", torch.int32, 2)
    _dev(positions, "positions", torch.int32, 1)
    B = positions.shape[0]
    if k_new.shape != v_new.shape or k_new.shape != (B, pool.n_kv_heads, pool.head_dim):
        raise ValueError("k_new/v_new must be [B, Hkv, D] matching the pool")
    if page_table.shape[0] != B:
        raise ValueError("page_table rows != batch")
    if dev_status is not None:
        _dev(dev_status, "dev_status", torch.int32)
    _check(load_library().kv_append(pool.handle, _ptr(k_new), _ptr(v_new), _ptr(page_table),
                                    page_table.shape[1], _ptr(positions), B, _ptr(dev_status),
                                    _stream(stream)), "kv_append")


def _norm_weights(q_norm_weight, k_norm_weight, dtype, head_dim: int):
    for name, w in (("q_norm_weight", q_norm_weight), ("k_norm_weight", k_norm_weight)):
        if w is not None:
            _dev(w, name, dtype, 1)
            if w.shape[0] != head_dim:
                raise ValueError(f"{name} must hold head_dim values")


def kv_append_rope(pool: Pool, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                   page_table: torch.Tensor, positions: torch.Tensor, rope_theta: float,
                   q_out: torch.Tensor, dev_status: torch.Tensor | None = None,
                   stream=None, q_norm_weight: torch.Tensor | None = None,
                   k_norm_weight: torch.Tensor | None = None,
                   norm_eps: float = 1e-6) -> torch.Tensor:
    """Rotary embedding of q [B, Hq, D] (into q_out) and k_new at positions[b],
    then the append of the rotated k_new and v_new into the pool; with a norm
    weight [D], the per-head RMS norm of that side comes first."""
    _dev(q, "q", pool.dtype, 3)
    _dev(q_out, "q_out", pool.dtype, 3)
    _dev(k_new, "k_new", pool.dtype, 3)
    _dev(v_new, "v_new", pool.dtype, 3)
    _dev(page_table, "page_table", torch.int32, 2)
    _dev(positions, "positions", torch.int32, 1)
    B = positions.shape[0]
    if k_new.shape != v_new.shape or k_new.shape != (B, pool.n_kv_heads, pool.head_dim):
        raise ValueError("k_new/v_new must be [B, Hkv, D] matching the pool")
    if q.shape[0] != B or q.shape[2] != pool.head_dim or q_out.shape != q.shape:
        raise ValueError("q/q_out must be [B, Hq, D] matching the pool")
    if page_table.shape[0] != B:
        raise ValueError("page_table rows != batch")
    if dev_status is not None:
        _dev(dev_status, "dev_status", torch.int32)
    _norm_weights(q_norm_weight, k_norm_weight, pool.dtype, pool.head_dim)
    _check(load_library().kv_append_rope(
        pool.handle, _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(page_table), page_table.shape[1],
        _ptr(positions), B, q.shape[1], float(rope_theta), _ptr(q_norm_weight),
        _ptr(k_norm_weight), float(norm_eps), _ptr(q_out), _ptr(dev_status), _stream(stream)),
        "kv_append_rope")
    return q_out


def kv_gather(pool: Pool, page_table: torch.Tensor, context_lens: torch.Tensor, max_len: int,
              k_out: torch.Tensor, v_out: torch.Tensor, dev_status: torch.Tensor | None = None,
              stream=None) -> None:
    """Dense [B, Hkv, max_len, D] copy of each sequence's cached rows."""
    _dev(page_table, "page_table", torch.int32, 2)
    _dev(context_lens, "context_lens", torch.int32, 1)
    B = context_lens.shape[0]
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        _dev(t, name, pool.dtype, 4)
        if tuple(t.shape) != (B, pool.n_kv_heads, max_len, pool.head_dim):
            raise ValueError(f"{name} must be [B, Hkv, max_len, D]")
    if dev_status is not None:
        _dev(dev_status, "dev_status", torch.int32)
    _check(load_library().kv_gather(pool.handle, _ptr(page_table), page_table.shape[1],
                                    _ptr(context_lens), B, max_len, _ptr(k_out), _ptr(v_out),
                                    _ptr(dev_status), _stream(stream)), "kv_gather")


def paged_decode_workspace_size(batch: int, n_q_heads: int, n_kv_heads: int, head_dim: int,
                                num_workers: int = 0, variant: int = VARIANT_AUTO) -> int:
    n = ctypes.c_size_t()
    _check(load_library().paged_decode_workspace_size(batch, n_q_heads, n_kv_heads, head_dim,
                                                      num_workers, variant, ctypes.byref(n)),
           "paged_decode_workspace_size")
    return n.value


def alloc_workspace(batch: int, n_q_heads: int, n_kv_heads: int, head_dim: int,
                    num_workers: int = 0, device=None, variant: int = VARIANT_AUTO) -> torch.Tensor:
    """A torch uint8 buffer of the size paged_decode_attention needs (256-B aligned)."""
    n = paged_decode_workspace_size(batch, n_q_heads, n_kv_heads, head_dim, num_workers, variant)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def _decode_shapes(q, k_pool, v_pool, page_table, out):
    _dev(q, "q", None, 3)
    dt = _dtype_code(q)
    _dev(k_pool, "k_pool", q.dtype, 4)
    _dev(v_pool, "v_pool", q.dtype, 4)
    _dev(out, "out", q.dtype, 3)
    _dev(page_table, "page_table", torch.int32, 2)
    B, Hq, D = q.shape
    NP, Hkv, P, D2 = k_pool.shape
    if D2 != D or v_pool.shape != k_pool.shape or out.shape != q.shape:
        raise ValueError("q/out [B, Hq, D] and pools [NP, Hkv, P, D] disagree")
    if page_table.shape[0] != B:
        raise ValueError("page_table rows != batch")
    return B, Hq, Hkv, D, P, NP, dt


def paged_decode_attention(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                           page_table: torch.Tensor, context_lens: torch.Tensor, scale: float,
                           out: torch.Tensor, workspace: torch.Tensor, num_workers: int = 0,
                           stream=None, variant: int = VARIANT_AUTO) -> torch.Tensor:
    """out[b, hq] = softmax(scale * q[b, hq] . K_b^T) V_b over context_lens[b]
    tokens read through page_table[b] (plan + decode + combine kernels)."""
    B, Hq, Hkv, D, P, NP, dt = _decode_shapes(q, k_pool, v_pool, page_table, out)
    _dev(context_lens, "context_lens", torch.int32, 1)
    _dev(workspace, "workspace", torch.uint8)
    _check(load_library().paged_decode_attention(
        _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(page_table), page_table.shape[1],
        _ptr(context_lens), B, Hq, Hkv, D, P, NP, dt, float(scale), _ptr(out), _ptr(workspace),
        workspace.numel(), int(num_workers), int(variant), _stream(stream)),
        "paged_decode_attention")
    return out


def paged_decode_attention_no_alloc(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                                    page_table: torch.Tensor, context_lens: torch.Tensor,
                                    scale: float, out: torch.Tensor, num_workers: int = 0,
                                    stream=None, variant: int = VARIANT_AUTO) -> torch.Tensor:
    """paged_decode_attention without a workspace argument: the library uses its
    own fixed device scratch of NO_ALLOC_SCRATCH_BYTES bytes and allocates
    nothing.  For callers that must not allocate device memory at decode time.
    Calls share that scratch, so calls that overlap on the GPU race; make the
    first call on a device before any stream capture (it looks the scratch up)."""
    B, Hq, Hkv, D, P, NP, dt = _decode_shapes(q, k_pool, v_pool, page_table, out)
    _dev(context_lens, "context_lens", torch.int32, 1)
    _check(load_library().paged_decode_attention_no_alloc(
        _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(page_table), page_table.shape[1],
        _ptr(context_lens), B, Hq, Hkv, D, P, NP, dt, float(scale), _ptr(out), int(num_workers),
        int(variant), _stream(stream)),
        "paged_decode_attention_no_alloc")
    return out


def check_bounded_wait(tries: int, stream=None) -> tuple[int, int]:
    """One bounded wait that never succeeds (pkv_check_bounded_wait): returns
    (device status bits, wait duration in ns) once it has given up."""
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ns = torch.zeros(1, dtype=torch.int64, device="cuda")
    _check(load_library().pkv_check_bounded_wait(int(tries), _ptr(st), _ptr(ns), _stream(stream)),
           "pkv_check_bounded_wait")
    torch.cuda.synchronize()
    return int(st.item()) & 0xFFFFFFFF, int(ns.item())


def paged_decode_multi_workspace_size(batch: int, n_queries: int, n_q_heads: int,
                                      n_kv_heads: int, head_dim: int, num_workers: int = 0,
                                      variant: int = VARIANT_AUTO) -> int:
    n = ctypes.c_size_t()
    _check(load_library().paged_decode_multi_workspace_size(
        batch, n_queries, n_q_heads, n_kv_heads, head_dim, int(num_workers), int(variant),
        ctypes.byref(n)), "paged_decode_multi_workspace_size")
    return n.value


def alloc_multi_workspace(batch: int, n_queries: int, n_q_heads: int, n_kv_heads: int,
                          head_dim: int, num_workers: int = 0, device=None,
                          variant: int = VARIANT_AUTO) -> torch.Tensor:
    n = paged_decode_multi_workspace_size(batch, n_queries, n_q_heads, n_kv_heads, head_dim,
                                          num_workers, variant)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def paged_decode_attention_multi(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                                 page_table: torch.Tensor, context_lens: torch.Tensor,
                                 scale: float, out: torch.Tensor, workspace: torch.Tensor,
                                 num_workers: int = 0, stream=None,
                                 variant: int = VARIANT_AUTO) -> torch.Tensor:
    """q, out [B, Qn, Hq, D]: query j of sequence b attends causally to tokens
    0 .. context_lens[b] - Qn + j."""
    _dev(q, "q", None, 4)
    dt = _dtype_code(q)
    _dev(out, "out", q.dtype, 4)
    _dev(k_pool, "k_pool", q.dtype, 4)
    _dev(v_pool, "v_pool", q.dtype, 4)
    _dev(page_table, "page_table", torch.int32, 2)
    _dev(context_lens, "context_lens", torch.int32, 1)
    _dev(workspace, "workspace", torch.uint8)
    B, Qn, Hq, D = q.shape
    NP, Hkv, P, D2 = k_pool.shape
    if D2 != D or v_pool.shape != k_pool.shape or out.shape != q.shape or page_table.shape[0] != B:
        raise ValueError("q/out [B, Qn, Hq, D], pools [NP, Hkv, P, D] and table disagree")
    _check(load_library().paged_decode_attention_multi(
        _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(page_table), page_table.shape[1],
        _ptr(context_lens), B, Qn, Hq, Hkv, D, P, NP, dt, float(scale), _ptr(out),
        _ptr(workspace), workspace.numel(), int(num_workers), int(variant), _stream(stream)),
        "paged_decode_attention_multi")
    return out


def paged_decode_prefix_workspace_size(batch: int, n_q_heads: int, n_kv_heads: int,
                                       head_dim: int, num_workers: int = 0,
                                       variant: int = VARIANT_AUTO) -> int:
    n = ctypes.c_size_t()
    _check(load_library().paged_decode_prefix_workspace_size(
        batch, n_q_heads, n_kv_heads, head_dim, int(num_workers), int(variant), ctypes.byref(n)),
        "paged_decode_prefix_workspace_size")
    return n.value


def alloc_prefix_workspace(batch: int, n_q_heads: int, n_kv_heads: int, head_dim: int,
                           num_workers: int = 0, device=None,
                           variant: int = VARIANT_AUTO) -> torch.Tensor:
    """A torch uint8 buffer of the size paged_decode_attention_prefix needs."""
    n = paged_decode_prefix_workspace_size(batch, n_q_heads, n_kv_heads, head_dim, num_workers,
                                           variant)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def paged_decode_attention_prefix(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                                  page_table: torch.Tensor, context_lens: torch.Tensor,
                                  scale: float, prefix_tokens: int, out: torch.Tensor,
                                  workspace: torch.Tensor, num_workers: int = 0, stream=None,
                                  variant: int = VARIANT_AUTO) -> torch.Tensor:
    """Decode attention for a batch whose rows share their first prefix_tokens
    tokens (the same pages): the prefix is attended once for all queries."""
    B, Hq, Hkv, D, P, NP, dt = _decode_shapes(q, k_pool, v_pool, page_table, out)
    _dev(context_lens, "context_lens", torch.int32, 1)
    _dev(workspace, "workspace", torch.uint8)
    _check(load_library().paged_decode_attention_prefix(
        _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(page_table), page_table.shape[1],
        _ptr(context_lens), B, Hq, Hkv, D, P, NP, dt, float(scale), int(prefix_tokens), _ptr(out),
        _ptr(workspace), workspace.numel(), int(num_workers), int(variant), _stream(stream)),
        "paged_decode_attention_prefix")
    return out


def paged_decode_step(k_new: torch.Tensor, v_new: torch.Tensor, positions: torch.Tensor,
                      q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                      page_table: torch.Tensor, context_lens: torch.Tensor, scale: float,
                      out: torch.Tensor, workspace: torch.Tensor, num_workers: int = 0,
                      stream=None, variant: int = VARIANT_AUTO) -> torch.Tensor:
    """One decode step: append k_new/v_new [B, Hkv, D] at positions[b] (fused
    into the plan launch), then decode attention into out."""
    B, Hq, Hkv, D, P, NP, dt = _decode_shapes(q, k_pool, v_pool, page_table, out)
    _dev(context_lens, "context_lens", torch.int32, 1)
    _dev(workspace, "workspace", torch.uint8)
    _dev(k_new, "k_new", q.dtype, 3)
    _dev(v_new, "v_new", q.dtype, 3)
    _dev(positions, "positions", torch.int32, 1)
    if k_new.shape != (B, Hkv, D) or v_new.shape != (B, Hkv, D):
        raise ValueError("k_new/v_new must be [B, Hkv, D]")
    _check(load_library().paged_decode_step(
        _ptr(k_new), _ptr(v_new), _ptr(positions), _ptr(q), _ptr(k_pool), _ptr(v_pool),
        _ptr(page_table), page_table.shape[1], _ptr(context_lens), B, Hq, Hkv, D, P, NP, dt,
        float(scale), _ptr(out), _ptr(workspace), workspace.numel(), int(num_workers),
        int(variant), _stream(stream)), "paged_decode_step")
    return out


def _host(t: torch.Tensor, name: str, dtype=None, ndim=None):
    """A contiguous pinned (page-locked) CPU tensor (of dtype / ndim when
    given), else raise.  The library checks the pages themselves again."""
    try:
        ok = (not t.is_cuda and t.is_contiguous() and t.is_pinned()
              and (dtype is None or t.dtype == dtype) and (ndim is None or t.dim() == ndim))
    except AttributeError:
        raise TypeError(f"{name} must be a torch tensor") from None
    if ok:
        return t
    if t.is_cuda or not t.is_pinned():
        raise ValueError(f"{name} must be a pinned host tensor (tensor.pin_memory())")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")


def paged_decode_step_host_workspace_size(batch: int, n_q_heads: int, n_kv_heads: int,
                                          head_dim: int, table_stride: int, num_workers: int = 0,
                                          variant: int = VARIANT_AUTO) -> int:
    n = ctypes.c_size_t()
    _check(load_library().paged_decode_step_host_workspace_size(
        batch, n_q_heads, n_kv_heads, head_dim, table_stride, num_workers, variant,
        ctypes.byref(n)), "paged_decode_step_host_workspace_size")
    return n.value


def alloc_step_host_workspace(batch: int, n_q_heads: int, n_kv_heads: int, head_dim: int,
                              table_stride: int, num_workers: int = 0, device=None,
                              variant: int = VARIANT_AUTO) -> torch.Tensor:
    """A torch uint8 device buffer of the size paged_decode_step_host needs."""
    n = paged_decode_step_host_workspace_size(batch, n_q_heads, n_kv_heads, head_dim,
                                              table_stride, num_workers, variant)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def paged_decode_step_host(k_new: torch.Tensor, v_new: torch.Tensor, positions: torch.Tensor,
                           q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                           page_table: torch.Tensor, context_lens: torch.Tensor, scale: float,
                           out: torch.Tensor, workspace: torch.Tensor, num_workers: int = 0,
                           stream=None, variant: int = VARIANT_AUTO) -> torch.Tensor:
    """paged_decode_step with k_new, v_new, positions, q, page_table,
    context_lens and out in pinned host memory (the pools and the workspace on
    the device): the kernels read the inputs and write out across the
    host-device link themselves.  out holds the result once the stream has
    finished the step."""
    _host(q, "q", None, 3)
    dt = _dtype_code(q)
    _dev(k_pool, "k_pool", q.dtype, 4)
    _dev(v_pool, "v_pool", q.dtype, 4)
    _dev(workspace, "workspace", torch.uint8)
    _host(out, "out", q.dtype, 3)
    _host(page_table, "page_table", torch.int32, 2)
    _host(context_lens, "context_lens", torch.int32, 1)
    _host(k_new, "k_new", q.dtype, 3)
    _host(v_new, "v_new", q.dtype, 3)
    _host(positions, "positions", torch.int32, 1)
    B, Hq, D = q.shape
    NP, Hkv, P, D2 = k_pool.shape
    if D2 != D or v_pool.shape != k_pool.shape or out.shape != q.shape:
        raise ValueError("q/out [B, Hq, D] and pools [NP, Hkv, P, D] disagree")
    if page_table.shape[0] != B:
        raise ValueError("page_table rows != batch")
    if k_new.shape != (B, Hkv, D) or v_new.shape != (B, Hkv, D):
        raise ValueError("k_new/v_new must be [B, Hkv, D]")
    _check(load_library().paged_decode_step_host(
        _ptr(k_new), _ptr(v_new), _ptr(positions), _ptr(q), _ptr(k_pool), _ptr(v_pool),
        _ptr(page_table), page_table.shape[1], _ptr(context_lens), B, Hq, Hkv, D, P, NP, dt,
        float(scale), _ptr(out), _ptr(workspace), workspace.numel(), int(num_workers),
        int(variant), _stream(stream)), "paged_decode_step_host")
    return out


def paged_decode_step_rope(k_new: torch.Tensor, v_new: torch.Tensor, positions: torch.Tensor,
                           q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                           page_table: torch.Tensor, context_lens: torch.Tensor, scale: float,
                           rope_theta: float, out: torch.Tensor, workspace: torch.Tensor,
                           num_workers: int = 0, stream=None,
                           variant: int = VARIANT_AUTO,
                           q_norm_weight: torch.Tensor | None = None,
                           k_norm_weight: torch.Tensor | None = None,
                           norm_eps: float = 1e-6) -> torch.Tensor:
    """paged_decode_step with the rotary embedding of q and k_new at positions[b]
    (angle base rope_theta) fused into the append, after the optional per-head
    RMS norm of either side; q stays as given, the rotated queries pass through
    out before the result overwrites them."""
    B, Hq, Hkv, D, P, NP, dt = _decode_shapes(q, k_pool, v_pool, page_table, out)
    _dev(context_lens, "context_lens", torch.int32, 1)
    _dev(workspace, "workspace", torch.uint8)
    _dev(k_new, "k_new", q.dtype, 3)
    _dev(v_new, "v_new", q.dtype, 3)
    _dev(positions, "positions", torch.int32, 1)
    if k_new.shape != (B, Hkv, D) or v_new.shape != (B, Hkv, D):
        raise ValueError("k_new/v_new must be [B, Hkv, D]")
    _norm_weights(q_norm_weight, k_norm_weight, q.dtype, D)
    _check(load_library().paged_decode_step_rope(
        _ptr(k_new), _ptr(v_new), _ptr(positions), _ptr(q), _ptr(k_pool), _ptr(v_pool),
        _ptr(page_table), page_table.shape[1], _ptr(context_lens), B, Hq, Hkv, D, P, NP, dt,
        float(scale), float(rope_theta), _ptr(q_norm_weight), _ptr(k_norm_weight),
        float(norm_eps), _ptr(out), _ptr(workspace), workspace.numel(), int(num_workers),
        int(variant), _stream(stream)), "paged_decode_step_rope")
    return out


def paged_decode_plan(context_lens: torch.Tensor, n_q_heads: int, n_kv_heads: int,
                      head_dim: int, page_size: int, table_stride: int, workspace: torch.Tensor,
                      num_workers: int = 0, stream=None, variant: int = VARIANT_AUTO) -> None:
    _dev(context_lens, "context_lens", torch.int32, 1)
    _dev(workspace, "workspace", torch.uint8)
    _check(load_library().paged_decode_plan(
        _ptr(context_lens), context_lens.shape[0], n_q_heads, n_kv_heads, head_dim, page_size,
        table_stride, int(num_workers), int(variant), _ptr(workspace), workspace.numel(),
        _stream(stream)), "paged_decode_plan")


def paged_decode_run(q, k_pool, v_pool, page_table, scale: float, out, workspace,
                     num_workers: int = 0, stream=None, variant: int = VARIANT_AUTO,
                     merge: bool = False) -> None:
    """The decode kernel; merge=True also merges split units (no combine needed)."""
    B, Hq, Hkv, D, P, NP, dt = _decode_shapes(q, k_pool, v_pool, page_table, out)
    _dev(workspace, "workspace", torch.uint8)
    _check(load_library().paged_decode_run(
        _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(page_table), page_table.shape[1], B, Hq, Hkv,
        D, P, NP, dt, float(scale), _ptr(out), _ptr(workspace), workspace.numel(),
        int(num_workers), int(variant), int(bool(merge)), _stream(stream)), "paged_decode_run")


def paged_decode_combine(out: torch.Tensor, n_kv_heads: int, workspace: torch.Tensor,
                         num_workers: int = 0, stream=None, variant: int = VARIANT_AUTO) -> None:
    _dev(out, "out", None, 3)
    _dev(workspace, "workspace", torch.uint8)
    B, Hq, D = out.shape
    _check(load_library().paged_decode_combine(
        B, Hq, n_kv_heads, D, _dtype_code(out), _ptr(out), _ptr(workspace), workspace.numel(),
        int(num_workers), int(variant), _stream(stream)), "paged_decode_combine")


# ---------------------------------------------------------------------------
# 8-bit cache: e4m3 pools with a power-of-two scale (E8M0) for each block of 16
# tokens, KV head and side
# ---------------------------------------------------------------------------
# These calls are short beside a decode of a few sequences, so their checks are one
# expression of cheap tensor queries; only when it is false does _kv8_explain look
# for what is wrong (and raises the usual error).
_SCALE_DTYPES = (torch.float8_e8m0fnu, torch.uint8)
_E4M3, _E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
_I32 = torch.int32
_get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _current(stream, dev):
    """The raw stream of a call on the current device `dev`."""
    if stream is not None or _raw_stream is None:
        return _stream(stream)
    return _raw_stream(dev)


def _kv8_explain(*checks):
    """Raise for the first (tensor, name, dtype, ndim) that _dev refuses."""
    for c in checks:
        _dev(*c)
    raise ValueError("arguments disagree")


def _kv8_scales(scales):
    if scales.dtype not in _SCALE_DTYPES:
        raise ValueError(f"scales must be float8_e8m0fnu (or its bytes), got {scales.dtype}")


def _kv8_pools(k_pool, v_pool, scales):
    _dev(k_pool, "k_pool", _E4M3, 4)
    _dev(v_pool, "v_pool", _E4M3, 4)
    _dev(scales, "scales", None, 4)
    _kv8_scales(scales)
    NP, Hkv, P, D = k_pool.shape
    if v_pool.shape != k_pool.shape or scales.shape != (NP, Hkv, P // 16, 2):
        raise ValueError("k_pool/v_pool must be [NP, Hkv, P, D] and scales [NP, Hkv, P / 16, 2]")
    return NP, Hkv, P, D


def kv8_pool_create(num_pages: int, page_size: int, n_kv_heads: int, head_dim: int,
                    k_pool: torch.Tensor | None = None, v_pool: torch.Tensor | None = None,
                    scales: torch.Tensor | None = None) -> Pool:
    """Create an 8-bit pool; with k_pool / v_pool (float8_e4m3fn [NP, Hkv, P, D])
    and scales (float8_e8m0fnu [NP, Hkv, P / 16, 2], K then V) the pool borrows
    them, otherwise it allocates device memory itself."""
    given = [t is not None for t in (k_pool, v_pool, scales)]
    if any(given) and not all(given):
        raise ValueError("give k_pool, v_pool and scales, or none of them")
    if all(given):
        if _kv8_pools(k_pool, v_pool, scales) != (num_pages, n_kv_heads, page_size, head_dim):
            raise ValueError(f"k_pool shape {tuple(k_pool.shape)} != "
                             f"{(num_pages, n_kv_heads, page_size, head_dim)}")
    h = ctypes.c_void_p()
    _check(load_library().kv8_pool_create(num_pages, page_size, n_kv_heads, head_dim,
                                          _ptr(k_pool), _ptr(v_pool), _ptr(scales),
                                          ctypes.byref(h)), "kv8_pool_create")
    pool = Pool(h.value, k_pool, v_pool, num_pages, page_size, n_kv_heads, head_dim,
                torch.float8_e4m3fn)
    pool._keep = (k_pool, v_pool, scales)
    pool.device = _get_device()
    return pool


def _kv8_new_rows(pool, k_new, v_new, page_table, positions, seq_ids, dev_status):
    """(current device, tokens, dtype code) of an append's checked arguments."""
    if pool.dtype is not _E4M3:
        raise ValueError("pool must be an 8-bit pool (kv8_pool_create)")
    dev = -1
    try:
        dev = k_new.get_device()
        ok = (dev >= 0 and v_new.get_device() == dev
              and page_table.get_device() == dev and positions.get_device() == dev
              and v_new.dtype is k_new.dtype and page_table.dtype is _I32
              and positions.dtype is _I32 and page_table.dim() == 2
              and positions.dim() == 1 and k_new.dtype in _DT and k_new.is_contiguous() and v_new.is_contiguous()
              and page_table.is_contiguous() and positions.is_contiguous()
              and dev == _get_device())
    except AttributeError:
        ok = False
    if not ok:
        _dev(k_new, "k_new", None, 3)
        _dtype_code(k_new)
        _kv8_explain((v_new, "v_new", k_new.dtype, 3), (page_table, "page_table", _I32, 2),
                     (positions, "positions", _I32, 1))
    if pool.device != dev:
        raise ValueError(f"pool is on cuda:{pool.device} but k_new is on cuda:{dev}")
    dt = _DT[k_new.dtype]
    N = positions.shape[0]
    if k_new.shape != (N, pool.n_kv_heads, pool.head_dim) or v_new.shape != k_new.shape:
        raise ValueError("k_new/v_new must be [tokens, Hkv, D] matching the pool and positions")
    if seq_ids is not None:
        _dev(seq_ids, "seq_ids", _I32, 1)
        if seq_ids.shape[0] != N:
            raise ValueError("seq_ids must have one entry per token")
    elif page_table.shape[0] < N:
        raise ValueError("page_table has fewer rows than tokens (give seq_ids)")
    if dev_status is not None:
        _dev(dev_status, "dev_status", _I32)
    return dev, N, dt


def kv8_append(pool: Pool, k_new: torch.Tensor, v_new: torch.Tensor, page_table: torch.Tensor,
               positions: torch.Tensor, seq_ids: torch.Tensor | None = None,
               dev_status: torch.Tensor | None = None, stream=None) -> None:
    """Append k_new/v_new [tokens, Hkv, D] (float16 or bfloat16) at positions[i]
    of sequence seq_ids[i] (default: token i's is row i of page_table): single
    tokens of a step, or prompts laid end to end."""
    dev, N, dt = _kv8_new_rows(pool, k_new, v_new, page_table, positions, seq_ids, dev_status)
    rows, cols = page_table.shape
    _check(load_library().kv8_append(pool.handle, k_new.data_ptr(), v_new.data_ptr(), dt,
                                     page_table.data_ptr(), cols, rows, positions.data_ptr(),
                                     _ptr(seq_ids), N, _ptr(dev_status), _current(stream, dev)),
           "kv8_append")


def kv8_append_rope(pool: Pool, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                    page_table: torch.Tensor, positions: torch.Tensor, rope_theta: float,
                    q_out: torch.Tensor, seq_ids: torch.Tensor | None = None,
                    dev_status: torch.Tensor | None = None, stream=None,
                    q_norm_weight: torch.Tensor | None = None,
                    k_norm_weight: torch.Tensor | None = None,
                    norm_eps: float = 1e-6) -> torch.Tensor:
    """kv8_append with the rotary embedding of q [tokens, Hq, D] (into q_out) and
    of k_new; with a norm weight [D], the per-head RMS norm of that side first."""
    dev, N, dt = _kv8_new_rows(pool, k_new, v_new, page_table, positions, seq_ids, dev_status)
    try:
        ok = (q.get_device() == dev and q_out.get_device() == dev and q.dtype is k_new.dtype
              and q_out.dtype is k_new.dtype and q.dim() == 3 and q.is_contiguous()
              and q_out.is_contiguous() and q_out.dim() == 3)
    except AttributeError:
        ok = False
    if not ok:
        _kv8_explain((q, "q", k_new.dtype, 3), (q_out, "q_out", k_new.dtype, 3))
    nq, Hq, D = q.shape
    if nq != N or D != pool.head_dim or q_out.shape != q.shape:
        raise ValueError("q/q_out must be [tokens, Hq, D] matching the pool and positions")
    if q_norm_weight is not None or k_norm_weight is not None:
        _norm_weights(q_norm_weight, k_norm_weight, q.dtype, D)
    rows, cols = page_table.shape
    _check(load_library().kv8_append_rope(
        pool.handle, q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), dt, page_table.data_ptr(),
        cols, rows, positions.data_ptr(), _ptr(seq_ids), N, Hq, float(rope_theta), _ptr(q_norm_weight),
        _ptr(k_norm_weight), float(norm_eps), q_out.data_ptr(), _ptr(dev_status),
        _current(stream, dev)), "kv8_append_rope")
    return q_out


def paged_decode_kv8_workspace_size(batch: int, n_q_heads: int, n_kv_heads: int, head_dim: int,
                                    n_queries: int = 1, num_workers: int = 0) -> int:
    n = ctypes.c_size_t()
    _check(load_library().paged_decode_kv8_workspace_size(
        batch, n_queries, n_q_heads, n_kv_heads, head_dim, int(num_workers), ctypes.byref(n)),
        "paged_decode_kv8_workspace_size")
    return n.value


def alloc_kv8_workspace(batch: int, n_q_heads: int, n_kv_heads: int, head_dim: int,
                        n_queries: int = 1, num_workers: int = 0, device=None) -> torch.Tensor:
    """A torch uint8 buffer of the size the 8-bit attention calls need."""
    n = paged_decode_kv8_workspace_size(batch, n_q_heads, n_kv_heads, head_dim, n_queries,
                                        num_workers)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def _kv8_call(q, k_pool, v_pool, scales, page_table, context_lens, out, workspace, ndim):
    """(current device, table columns, pages, Hkv, P, D, dtype code) of an attention
    call's checked arguments.  (The numbers of dims are checked with the shapes.)"""
    dev = -1
    try:
        dev = q.get_device()
        dtype = q.dtype
        sdt = scales.dtype
        ok = (dev >= 0 and out.get_device() == dev and k_pool.get_device() == dev
              and v_pool.get_device() == dev and scales.get_device() == dev
              and page_table.get_device() == dev and context_lens.get_device() == dev
              and workspace.get_device() == dev and out.dtype is dtype
              and k_pool.dtype is _E4M3 and v_pool.dtype is _E4M3 and page_table.dtype is _I32
              and context_lens.dtype is _I32 and workspace.dtype is torch.uint8
              and (sdt is _E8M0 or sdt is torch.uint8) and q.is_contiguous()
              and out.is_contiguous() and k_pool.is_contiguous() and v_pool.is_contiguous()
              and scales.is_contiguous() and page_table.is_contiguous()
              and context_lens.is_contiguous() and workspace.is_contiguous()
              and dev == _get_device())
        if ok:
            qs, ks, ts = q.shape, k_pool.shape, page_table.shape
            ok = len(qs) == ndim and len(ks) == 4 and len(ts) == 2 and dtype in _DT
    except AttributeError:
        ok = False
    if not ok:
        _dev(q, "q", None, ndim)
        _dtype_code(q)
        _dev(scales, "scales", None, 4)
        _kv8_scales(scales)
        _kv8_explain((out, "out", q.dtype, ndim), (k_pool, "k_pool", _E4M3, 4),
                     (v_pool, "v_pool", _E4M3, 4), (page_table, "page_table", _I32, 2),
                     (context_lens, "context_lens", _I32, 1),
                     (workspace, "workspace", torch.uint8))
    NP, Hkv, P, D = ks
    B, cols = ts
    if v_pool.shape != ks or scales.shape != (NP, Hkv, P // 16, 2):
        raise ValueError("k_pool/v_pool must be [NP, Hkv, P, D] and scales [NP, Hkv, P / 16, 2]")
    if qs[-1] != D or out.shape != qs:
        raise ValueError("q/out [..., Hq, D] and pools [NP, Hkv, P, D] disagree")
    if qs[0] != B or context_lens.shape != (B,):
        raise ValueError("page_table rows or context_lens != batch")
    return dev, cols, NP, Hkv, P, D, _DT[dtype]


def paged_decode_attention_kv8(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                               scales: torch.Tensor, page_table: torch.Tensor,
                               context_lens: torch.Tensor, scale: float, out: torch.Tensor,
                               workspace: torch.Tensor, num_workers: int = 0,
                               stream=None) -> torch.Tensor:
    """paged_decode_attention over an 8-bit cache: q, out [B, Hq, D] in float16
    or bfloat16, pools float8_e4m3fn, scales float8_e8m0fnu."""
    dev, cols, NP, Hkv, P, D, dt = _kv8_call(q, k_pool, v_pool, scales, page_table, context_lens,
                                             out, workspace, 3)
    B, Hq, _ = q.shape
    _check(load_library().paged_decode_attention_kv8(
        q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), scales.data_ptr(),
        page_table.data_ptr(), cols, context_lens.data_ptr(), B, Hq, Hkv, D, P, NP,
        dt, float(scale), out.data_ptr(), workspace.data_ptr(), workspace.numel(),
        int(num_workers), _current(stream, dev)), "paged_decode_attention_kv8")
    return out


def paged_decode_attention_multi_kv8(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                                     scales: torch.Tensor, page_table: torch.Tensor,
                                     context_lens: torch.Tensor, scale: float, out: torch.Tensor,
                                     workspace: torch.Tensor, num_workers: int = 0,
                                     stream=None) -> torch.Tensor:
    """paged_decode_attention_multi over an 8-bit cache: q, out [B, Qn, Hq, D],
    query j of sequence b attends causally to tokens 0 .. context_lens[b] - Qn + j."""
    dev, cols, NP, Hkv, P, D, dt = _kv8_call(q, k_pool, v_pool, scales, page_table, context_lens,
                                             out, workspace, 4)
    B, Qn, Hq, _ = q.shape
    _check(load_library().paged_decode_attention_multi_kv8(
        q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), scales.data_ptr(),
        page_table.data_ptr(), cols, context_lens.data_ptr(), B, Qn, Hq, Hkv, D, P,
        NP, dt, float(scale), out.data_ptr(), workspace.data_ptr(), workspace.numel(),
        int(num_workers), _current(stream, dev)), "paged_decode_attention_multi_kv8")
    return out


def paged_decode_step_kv8(k_new: torch.Tensor, v_new: torch.Tensor, positions: torch.Tensor,
                          q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                          scales: torch.Tensor, page_table: torch.Tensor,
                          context_lens: torch.Tensor, scale: float, out: torch.Tensor,
                          workspace: torch.Tensor, rope_theta: float = 0.0, num_workers: int = 0,
                          stream=None, q_norm_weight: torch.Tensor | None = None,
                          k_norm_weight: torch.Tensor | None = None,
                          norm_eps: float = 1e-6) -> torch.Tensor:
    """One decode step over an 8-bit cache: append k_new/v_new [B, Hkv, D] at
    positions[b], then decode attention into out; with rope_theta > 0 the rotary
    embedding of q and k_new (after the optional per-head RMS norm) comes first."""
    dev, cols, NP, Hkv, P, D, dt = _kv8_call(q, k_pool, v_pool, scales, page_table, context_lens,
                                             out, workspace, 3)
    B, Hq, _ = q.shape
    try:
        ok = (k_new.get_device() == dev and v_new.get_device() == dev
              and positions.get_device() == dev and k_new.dtype is q.dtype
              and v_new.dtype is q.dtype and positions.dtype is _I32 and k_new.is_contiguous()
              and v_new.is_contiguous() and positions.is_contiguous())
    except AttributeError:
        ok = False
    if not ok:
        _kv8_explain((k_new, "k_new", q.dtype, 3), (v_new, "v_new", q.dtype, 3),
                     (positions, "positions", _I32, 1))
    if k_new.shape != (B, Hkv, D) or v_new.shape != k_new.shape or positions.shape != (B,):
        raise ValueError("k_new/v_new must be [B, Hkv, D] and positions [B]")
    if q_norm_weight is not None or k_norm_weight is not None:
        _norm_weights(q_norm_weight, k_norm_weight, q.dtype, D)
    _check(load_library().paged_decode_step_kv8(
        k_new.data_ptr(), v_new.data_ptr(), positions.data_ptr(), q.data_ptr(),
        k_pool.data_ptr(), v_pool.data_ptr(), scales.data_ptr(), page_table.data_ptr(),
        cols, context_lens.data_ptr(), B, Hq, Hkv, D, P, NP, dt, float(scale), float(rope_theta),
        _ptr(q_norm_weight), _ptr(k_norm_weight), float(norm_eps), out.data_ptr(),
        workspace.data_ptr(), workspace.numel(), int(num_workers), _current(stream, dev)),
        "paged_decode_step_kv8")
    return out


# ---------------------------------------------------------------------------
# Serving with selected pages: tables, appends of any tokens, page bounds, the
# selection and the attention over it.  Their arguments are checked by the
# binding's native part (binding/calls.cpp), which raises ValueError or TypeError
# for what it refuses and calls the entry point of the same name.
# ---------------------------------------------------------------------------
_calls = None


def load_binding():
    """The binding's native part (built first when missing)."""
    global _calls
    if _calls is None:
        load_library()
        path = _build.binding_path()
        if not os.path.exists(path):
            _build.build()
        spec = importlib.util.spec_from_file_location("_pagedkv_calls", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _calls = module
    return _calls


def paged_tables_build(cached_lens: torch.Tensor, new_lens: torch.Tensor,
                       free_pages: torch.Tensor, free_begin: torch.Tensor | None,
                       free_end: torch.Tensor, page_table: torch.Tensor, page_size: int,
                       num_pages: int, context_lens: torch.Tensor, query_starts: torch.Tensor,
                       positions: torch.Tensor, seq_ids: torch.Tensor, slots: torch.Tensor,
                       dev_status: torch.Tensor | None = None, stream=None) -> None:
    """From the requests' cached and new lengths [B], on the GPU: the entries of
    their new pages in page_table [B, cols] (taken in order from free_pages,
    from entry free_begin[0] on; free_end[0] is where the next call goes on),
    context_lens [B], query_starts [B + 1], and each token row's positions,
    seq_ids and slots [tokens] (-1 behind the last request's).  Everything is
    int32 but slots (int64)."""
    code = (_calls or load_binding()).paged_tables_build(
        cached_lens, new_lens, free_pages, free_begin, free_end, page_table, page_size, num_pages,
        context_lens, query_starts, positions, seq_ids, slots, dev_status,
        None if stream is None else stream.cuda_stream)
    if code:
        raise PagedKVError(code, "paged_tables_build")


class _RopeStruct(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("magnitude", ctypes.c_float), ("reserved", ctypes.c_uint32),
                ("turns", ctypes.c_uint64 * 64)]


ROPE_SCALINGS = {"none": 0, "linear": 1, "turns": 2, "index": 3}


class Rope:
    """A rotary embedding (pkv_rope_init): the leading rotary_dim elements of a
    head turn, in halves or (interleaved) neighbouring pairs, by position *
    theta^(-2i / rotary_dim), scaled for long contexts by `scaling` ("none",
    "linear", "turns" or "index") and `factor`; magnitude multiplies what turns."""

    def __init__(self, rotary_dim: int, theta: float = 10000.0, interleaved: bool = False,
                 scaling: str = "none", factor: float = 1.0, low_turns: float = 1.0,
                 high_turns: float = 4.0, original_context: float = 8192.0,
                 magnitude: float = 1.0):
        if scaling not in ROPE_SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}, got {scaling!r}")
        self._s = _RopeStruct()
        self._p = ctypes.addressof(self._s)
        _check(load_library().pkv_rope_init(
            self._p, int(rotary_dim), float(theta), int(bool(interleaved)), float(magnitude),
            ROPE_SCALINGS[scaling], float(factor), float(low_turns), float(high_turns),
            float(original_context)), "pkv_rope_init")

    @property
    def rotary_dim(self) -> int:
        return self._s.rotary_dim

    def turns(self) -> list[float]:
        """Turns a position of each pair, as fractions of a turn."""
        return [self._s.turns[i] / 2.0 ** 64 for i in range(self._s.rotary_dim // 2)]


def kv_append_tokens(pool: Pool, k_new: torch.Tensor, v_new: torch.Tensor, slots: torch.Tensor,
                     q: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                     rope: Rope | None = None, q_out: torch.Tensor | None = None,
                     q_norm_weight: torch.Tensor | None = None,
                     k_norm_weight: torch.Tensor | None = None, norm_eps: float = 1e-6,
                     dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """Write k_new / v_new [tokens, Hkv, D] at slots [tokens] (int64, < 0: not
    written); with a rope, turn q [tokens, Hq, D] at positions [tokens] into
    q_out and k_new on its way, after the optional per-head RMS norms.  Rows may
    be slices of a wider tensor; q_out may be q."""
    code = (_calls or load_binding()).kv_append_tokens(
        pool._address, pool.device, k_new, v_new, slots, q, positions,
        None if rope is None else rope._p, q_out, q_norm_weight, k_norm_weight, norm_eps,
        dev_status, None if stream is None else stream.cuda_stream)
    if code:
        raise PagedKVError(code, "kv_append_tokens")
    return q_out


def kv_page_bounds(pool: Pool, slots: torch.Tensor, bounds: torch.Tensor,
                   dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The smallest and largest key, element by element, of every page that holds
    one of slots [tokens], into bounds [num_pages, Hkv, 2, D]."""
    code = (_calls or load_binding()).kv_page_bounds(
        pool._address, pool.device, slots, bounds, dev_status,
        None if stream is None else stream.cuda_stream)
    if code:
        raise PagedKVError(code, "kv_page_bounds")
    return bounds


def paged_select_workspace_size(batch: int, n_kv_heads: int, table_cols: int) -> int:
    n = ctypes.c_size_t()
    _check(load_library().paged_select_workspace_size(batch, n_kv_heads, table_cols,
                                                      ctypes.byref(n)),
           "paged_select_workspace_size")
    return n.value


def alloc_select_workspace(batch: int, n_kv_heads: int, table_cols: int,
                           device=None) -> torch.Tensor:
    """A torch uint8 buffer of the size paged_select_pages needs."""
    n = paged_select_workspace_size(batch, n_kv_heads, table_cols)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def paged_select_pages(q: torch.Tensor, bounds: torch.Tensor, page_table: torch.Tensor,
                       context_lens: torch.Tensor, page_size: int, selected: torch.Tensor,
                       workspace: torch.Tensor, keep_first: int = 1, keep_last: int = 1,
                       dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The pages that q [B, Hq, D] attends to, for each KV head: the first
    keep_first, the last keep_last and those of the highest score by bounds
    [num_pages, Hkv, 2, D], into selected [B, Hkv, max_pages] (indexes into the
    rows of page_table, ascending, -1 behind them)."""
    code = (_calls or load_binding()).paged_select_pages(
        q, bounds, page_table, context_lens, page_size, selected, workspace, keep_first, keep_last,
        dev_status, None if stream is None else stream.cuda_stream)
    if code:
        raise PagedKVError(code, "paged_select_pages")
    return selected


def paged_decode_attention_selected(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                                    page_table: torch.Tensor, context_lens: torch.Tensor,
                                    selected: torch.Tensor, scale: float, out: torch.Tensor,
                                    dev_status: torch.Tensor | None = None,
                                    stream=None) -> torch.Tensor:
    """Decode attention of q [B, Hq, D] over the pages selected[b][h] (indexes into
    the rows of page_table; negative entries are skipped) into out."""
    code = (_calls or load_binding()).paged_decode_attention_selected(
        q, k_pool, v_pool, page_table, context_lens, selected, scale, out, dev_status,
        None if stream is None else stream.cuda_stream)
    if code:
        raise PagedKVError(code, "paged_decode_attention_selected")
    return out


def pkv_read_device_status(workspace: torch.Tensor) -> int:
    """The status word of the last decode on this workspace (synchronises)."""
    _dev(workspace, "workspace", torch.uint8)
    v = ctypes.c_uint32()
    code = load_library().pkv_read_device_status(_ptr(workspace), ctypes.byref(v))
    if code not in (0, 7):
        _check(code, "pkv_read_device_status")
    return v.value


def pkv_read_no_alloc_status() -> int:
    """The status word of the last paged_decode_attention_no_alloc call on the
    current device (synchronises)."""
    v = ctypes.c_uint32()
    code = load_library().pkv_read_no_alloc_status(ctypes.byref(v))
    if code not in (0, 7):
        _check(code, "pkv_read_no_alloc_status")
    return v.value
