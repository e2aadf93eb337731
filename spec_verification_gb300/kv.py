"""ctypes binding of the KV-cache entry points of libss.so (include/ss_kv.h):
argument marshalling only, as in native.py.  torch tensors go in as device
pointers and strides; nothing is copied, cast or allocated here.
"""
from __future__ import annotations

import ctypes as C

import numpy as np

from . import native

SS_F16, SS_E4M3 = 2, 3
DTYPES = {"bf16": native.SS_BF16, "f16": SS_F16, "e4m3": SS_E4M3}
# row status bits (beside those of native.py)
ST_KV_POOL, ST_KV_TABLE, ST_KV_PAGE = 1 << 11, 1 << 12, 1 << 13

_p, _i32, _i64, _f32 = C.c_void_p, C.c_int32, C.c_int64, C.c_float


class Config(C.Structure):
    _fields_ = [(n, _i32) for n in ("max_rows", "max_tokens", "max_new", "q_heads", "kv_heads", "head_dim", "page_size",
                                    "num_pages", "max_blocks", "dtype", "cache_dtype", "device")]


class Cache(C.Structure):
    _fields_ = [("k", _p), ("v", _p), ("page_stride", _i64), ("token_stride", _i64), ("head_stride", _i64),
                ("k_scale", _p), ("v_scale", _p)]


class Pool(C.Structure):
    _fields_ = [("B", _i32), ("block_table", _p), ("kv_len", _p), ("free_pages", _p), ("free_count", _p),
                ("stream", _p), ("plan", _p)]


class RopeBatch(C.Structure):
    _fields_ = [("T", _i32), ("q", _p), ("k", _p), ("v", _p), ("q_stride", _i64), ("k_stride", _i64),
                ("v_stride", _i64), ("q_weight", _p), ("k_weight", _p), ("eps", _f32), ("inv_freq", _p),
                ("rot_dim", _i32), ("interleaved", _i32), ("rope_scale", _f32), ("positions", _p), ("slots", _p),
                ("q_out", _p), ("q_out_stride", _i64), ("stream", _p), ("plan", _p)]


class AttendBatch(C.Structure):
    _fields_ = [("B", _i32), ("q", _p), ("q_stride", _i64), ("cu_new", _p), ("seq_len", _p), ("block_table", _p),
                ("scale", _f32), ("window", _i32), ("sinks", _i32), ("out", _p), ("out_stride", _i64), ("lse", _p),
                ("row_status", _p), ("workspace", _p), ("workspace_bytes", C.c_size_t), ("stream", _p), ("plan", _p)]


EXPORTS = ["ss_kv_plan_create", "ss_kv_plan_destroy", "ss_kv_workspace_bytes", "ss_kv_append", "ss_kv_commit",
           "ss_rope_store", "ss_rope_frequencies", "ss_attend"]

_lib = None


def library() -> C.CDLL:
    """libss.so with the KV-cache entry points' signatures set."""
    global _lib
    if _lib is not None:
        return _lib
    L = native.library()
    L.ss_kv_plan_create.argtypes = [C.POINTER(_p), C.POINTER(Config)]
    L.ss_kv_plan_destroy.argtypes = [_p]
    L.ss_kv_plan_destroy.restype = None
    L.ss_kv_workspace_bytes.argtypes = [_p]
    L.ss_kv_workspace_bytes.restype = C.c_size_t
    L.ss_kv_append.argtypes = [C.POINTER(Pool), _p, _p, _p, _p, _p]
    L.ss_kv_commit.argtypes = [C.POINTER(Pool), _p, _p, _i32, _p]
    L.ss_rope_store.argtypes = [C.POINTER(RopeBatch), C.POINTER(Cache)]
    L.ss_rope_frequencies.argtypes = [C.POINTER(C.c_double), _i32, C.c_double, C.c_double, _i32, C.c_double, C.c_double]
    L.ss_attend.argtypes = [C.POINTER(AttendBatch), C.POINTER(Cache)]
    for name in ("ss_kv_plan_create", "ss_kv_append", "ss_kv_commit", "ss_rope_store", "ss_rope_frequencies", "ss_attend"):
        getattr(L, name).restype = C.c_int
    _lib = L
    return L


class Plan:
    """ss_kv_plan_create / ss_kv_plan_destroy."""

    def __init__(self, *, max_rows: int, max_tokens: int, q_heads: int, kv_heads: int, head_dim: int, page_size: int,
                 num_pages: int, max_blocks: int, max_new: int = 1, dtype: str = "bf16", cache_dtype: str | None = None,
                 device: int = 0):
        L = library()
        self._p = _p()
        cfg = Config(max_rows, max_tokens, max_new, q_heads, kv_heads, head_dim, page_size, num_pages, max_blocks,
                     DTYPES[dtype], DTYPES[cache_dtype or dtype], device)
        native._check(L.ss_kv_plan_create(C.byref(self._p), C.byref(cfg)))
        self.handle = self._p.value
        self.page_size, self.num_pages, self.max_blocks = page_size, num_pages, max_blocks
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.dtype, self.cache_dtype = dtype, cache_dtype or dtype
        self.workspace_bytes = L.ss_kv_workspace_bytes(self._p)

    def __del__(self):
        try:
            if self._p:
                library().ss_kv_plan_destroy(self._p)
                self._p = _p()
        except Exception:
            pass


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check_type(name, t, dtype):
    """Tensors whose element type the library could not see for itself."""
    got = str(t.dtype)
    want = {"bf16": "torch.bfloat16", "f16": "torch.float16", "e4m3": "torch.float8_e4m3fn", "i32": "torch.int32",
            "f32": "torch.float32", "f64": "torch.float64"}[dtype]
    if got != want:
        raise native.SSError(-1, f"{name} must be {want}, got {got}")


def _cache(plan, k_cache, v_cache, k_scale, v_scale):
    """k_cache and v_cache seen as [pages, page_size, kv_heads, head_dim], in any memory order of the first three."""
    want = (plan.num_pages, plan.page_size, plan.kv_heads, plan.head_dim)
    if k_cache.shape != want or v_cache.shape != want:
        raise native.SSError(-1, f"caches must be seen as [pages, page_size, kv_heads, head_dim] = {list(want)}, got "
                                 f"{list(k_cache.shape)} and {list(v_cache.shape)}")
    st = k_cache.stride()
    if st != v_cache.stride() or st[3] != 1:
        raise native.SSError(-1, "both caches must have the same strides, and a head's values must be contiguous")
    _check_type("k_cache", k_cache, plan.cache_dtype)
    _check_type("v_cache", v_cache, plan.cache_dtype)
    return Cache(k_cache.data_ptr(), v_cache.data_ptr(), st[0], st[1], st[2], _ptr(k_scale), _ptr(v_scale))


def _tokens(name, t, heads, plan):
    """[tokens, heads, head_dim] with contiguous heads -> stride between tokens."""
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != plan.head_dim or t.stride(2) != 1 or \
            (heads > 1 and t.stride(1) != plan.head_dim):
        raise native.SSError(-1, f"{name} must be [tokens, {heads}, {plan.head_dim}] with contiguous heads, got "
                                 f"{list(t.shape)} with strides {list(t.stride())}")
    _check_type(name, t, plan.dtype)
    return t.stride(0) if t.shape[0] > 1 else heads * plan.head_dim


def _ints(**tensors):
    for name, t in tensors.items():
        if t is not None:
            _check_type(name, t, "i32")
            if not t.is_contiguous():
                raise native.SSError(-1, f"{name} must be contiguous")


def _pool(plan, block_table, kv_len, free_pages, free_count, B, stream):
    _ints(block_table=block_table, kv_len=kv_len, free_pages=free_pages, free_count=free_count)
    B = kv_len.shape[0] if B is None else B
    if block_table.dim() != 2 or block_table.shape[0] < B or block_table.shape[1] != plan.max_blocks:
        raise native.SSError(-1, f"block_table must be [rows, {plan.max_blocks}], got {list(block_table.shape)}")
    if free_pages.numel() < plan.num_pages:
        raise native.SSError(-1, "free_pages must have num_pages entries")
    return Pool(B, block_table.data_ptr(), kv_len.data_ptr(), free_pages.data_ptr(), free_count.data_ptr(),
                native._stream_ptr(stream), plan.handle)


def ss_kv_append(plan: Plan, block_table, kv_len, free_pages, free_count, cu_new, *, slots, positions, seq_len,
                 row_status, B=None, stream=None):
    """ss_kv_append on int32 tensors: pages, slots and positions of each row's new tokens."""
    _ints(cu_new=cu_new, slots=slots, positions=positions, seq_len=seq_len, row_status=row_status)
    pool = _pool(plan, block_table, kv_len, free_pages, free_count, B, stream)
    native._check(library().ss_kv_append(C.byref(pool), cu_new.data_ptr(), slots.data_ptr(), positions.data_ptr(),
                                         seq_len.data_ptr(), row_status.data_ptr()))


def ss_kv_commit(plan: Plan, block_table, kv_len, free_pages, free_count, seq_len, *, counts=None, plus=0, finished=None,
                 B=None, stream=None):
    """ss_kv_commit on int32 tensors: lengths move past what is kept, other pages go back to the pool."""
    _ints(seq_len=seq_len, counts=counts, finished=finished)
    pool = _pool(plan, block_table, kv_len, free_pages, free_count, B, stream)
    native._check(library().ss_kv_commit(C.byref(pool), seq_len.data_ptr(), _ptr(counts), plus, _ptr(finished)))


def ss_rope_store(plan: Plan, q, k, v, k_cache, v_cache, inv_freq, positions, slots, *, q_out, q_weight=None,
                  k_weight=None, eps=1e-6, interleaved=False, rope_scale=1.0, k_scale=None, v_scale=None, stream=None):
    """ss_rope_store: q, k, v, q_out [tokens, heads, head_dim]; caches seen as [pages, page_size, kv_heads, head_dim];
    inv_freq [rot_dim / 2] float64 on the device (None: no rotation)."""
    T = q.shape[0]
    cache = _cache(plan, k_cache, v_cache, k_scale, v_scale)
    qs, ks = _tokens("q", q, plan.q_heads, plan), _tokens("k", k, plan.kv_heads, plan)
    vs, os = _tokens("v", v, plan.kv_heads, plan), _tokens("q_out", q_out, plan.q_heads, plan)
    if not (k.shape[0] == v.shape[0] == q_out.shape[0] == positions.shape[0] == slots.shape[0] == T):
        raise native.SSError(-1, "q, k, v, q_out, positions and slots must have the same number of tokens")
    _ints(positions=positions, slots=slots)
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _check_type(name, w, plan.dtype)
    rot = 0
    if inv_freq is not None:
        _check_type("inv_freq", inv_freq, "f64")
        rot = 2 * inv_freq.shape[0]
    b = RopeBatch(T, q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs, _ptr(q_weight), _ptr(k_weight), eps, _ptr(inv_freq),
                  rot, 1 if interleaved else 0, rope_scale, positions.data_ptr(), slots.data_ptr(), q_out.data_ptr(), os,
                  native._stream_ptr(stream), plan.handle)
    native._check(library().ss_rope_store(C.byref(b), C.byref(cache)))


def rope_frequencies(rot_dim: int, base: float = 10000.0, *, factor: float = 1.0, original_len: int = 0,
                     low_turns: float = 1.0, high_turns: float = 32.0) -> np.ndarray:
    """ss_rope_frequencies: float64 [rot_dim / 2] on the host."""
    out = np.empty(max(rot_dim // 2, 1), np.float64)
    native._check(library().ss_rope_frequencies(out.ctypes.data_as(C.POINTER(C.c_double)), rot_dim, base, factor,
                                                original_len, low_turns, high_turns))
    return out


def ss_attend(plan: Plan, q, k_cache, v_cache, block_table, seq_len, cu_new, *, out, row_status, workspace, scale,
              window=0, sinks=0, lse=None, k_scale=None, v_scale=None, B=None, stream=None):
    """ss_attend: q, out [tokens, q_heads, head_dim]; caches seen as [pages, page_size, kv_heads, head_dim]."""
    cache = _cache(plan, k_cache, v_cache, k_scale, v_scale)
    qs, os = _tokens("q", q, plan.q_heads, plan), _tokens("out", out, plan.q_heads, plan)
    _ints(block_table=block_table, seq_len=seq_len, cu_new=cu_new, row_status=row_status)
    B = seq_len.shape[0] if B is None else B
    if block_table.dim() != 2 or block_table.shape[0] < B or block_table.shape[1] != plan.max_blocks:
        raise native.SSError(-1, f"block_table must be [rows, {plan.max_blocks}], got {list(block_table.shape)}")
    b = AttendBatch(B, q.data_ptr(), qs, cu_new.data_ptr(), seq_len.data_ptr(), block_table.data_ptr(), scale, window, sinks,
                    out.data_ptr(), os, _ptr(lse), row_status.data_ptr(), workspace.data_ptr(),
                    workspace.numel() * workspace.element_size(), native._stream_ptr(stream), plan.handle)
    native._check(library().ss_attend(C.byref(b), C.byref(cache)))
