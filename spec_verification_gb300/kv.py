"""ctypes binding of the KV-cache entry points of libss.so (include/ss_kv.h):
argument marshalling only, as in native.py.  torch tensors go in as device
pointers and strides; nothing is copied, cast or allocated here.
"""
from __future__ import annotations

import ctypes as C
import struct

import numpy as np
import torch

from . import native

SS_F16, SS_E4M3 = 2, 3
DTYPES = {"bf16": native.SS_BF16, "f16": SS_F16, "e4m3": SS_E4M3}
# row status bits (beside those of native.py)
ST_KV_POOL, ST_KV_TABLE, ST_KV_PAGE = 1 << 11, 1 << 12, 1 << 13

_TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}

_I32 = torch.int32
_p, _i32, _i64, _f32 = C.c_void_p, C.c_int32, C.c_int64, C.c_float


class Config(C.Structure):
    _fields_ = [(n, _i32) for n in ("max_rows", "max_tokens", "max_new", "q_heads", "kv_heads", "head_dim", "page_size",
                                    "num_pages", "max_blocks", "dtype", "cache_dtype", "device")]


class Cache(C.Structure):
    _fields_ = [("k", _p), ("v", _p), ("page_stride", _i64), ("token_stride", _i64), ("head_stride", _i64),
                ("k_scale", _p), ("v_scale", _p)]


class Pool(C.Structure):
    _fields_ = [("B", _i32), ("tokens", _i32), ("block_table", _p), ("kv_len", _p), ("free_pages", _p), ("free_count", _p),
                ("stream", _p), ("plan", _p)]


class RopeBatch(C.Structure):
    _fields_ = [("T", _i32), ("q", _p), ("k", _p), ("v", _p), ("q_stride", _i64), ("k_stride", _i64),
                ("v_stride", _i64), ("q_weight", _p), ("k_weight", _p), ("eps", _f32), ("inv_freq", _p),
                ("rot_dim", _i32), ("interleaved", _i32), ("rope_scale", _f32), ("positions", _p), ("slots", _p),
                ("q_out", _p), ("q_out_stride", _i64), ("stream", _p), ("plan", _p)]


class AttendBatch(C.Structure):
    _fields_ = [("B", _i32), ("tokens", _i32), ("q", _p), ("q_stride", _i64), ("cu_new", _p), ("seq_len", _p), ("block_table", _p),
                ("scale", _f32), ("window", _i32), ("sinks", _i32), ("out", _p), ("out_stride", _i64), ("lse", _p),
                ("row_status", _p), ("workspace", _p), ("workspace_bytes", C.c_size_t), ("stream", _p), ("plan", _p)]


class BlockCache(C.Structure):
    _fields_ = [("k", _p), ("v", _p), ("page_stride", _i64), ("token_stride", _i64), ("head_stride", _i64),
                ("k_scale", _p), ("v_scale", _p), ("block_tokens", _i32)]


class StoreBatch(C.Structure):
    _fields_ = [("B", _i32), ("tokens", _i32), ("k", _p), ("v", _p), ("k_stride", _i64), ("v_stride", _i64), ("cu_new", _p), ("kv_len", _p),
                ("seq_len", _p), ("block_table", _p), ("row_status", _p), ("stream", _p), ("plan", _p)]


class LoadBatch(C.Structure):
    _fields_ = [("T", _i32), ("slots", _p), ("k", _p), ("v", _p), ("k_stride", _i64), ("v_stride", _i64), ("stream", _p), ("plan", _p)]


class PromptBatch(C.Structure):
    _fields_ = [("B", _i32), ("tokens", _i32), ("q", _p), ("k", _p), ("v", _p), ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64),
                ("cu_seq", _p), ("scale", _f32), ("window", _i32), ("sinks", _i32), ("out", _p), ("out_stride", _i64), ("lse", _p),
                ("row_status", _p), ("workspace", _p), ("workspace_bytes", C.c_size_t), ("stream", _p), ("plan", _p)]


# The same layouts as native struct formats: packing one takes a fifth of the time that filling a ctypes structure does.
_CACHE = struct.Struct("@PPqqqPP")
_POOL = struct.Struct("@iiPPPPPP")
_ROPE = struct.Struct("@iPPPqqqPPfPiifPPPqPP")
_ATTEND = struct.Struct("@iiPqPPPfiiPqPPPNPP")
_BLOCKS = struct.Struct("@PPqqqPPi0q")
_STORE = struct.Struct("@iiPPqqPPPPPPP")
_LOAD = struct.Struct("@iPPPqqPP")
_PROMPT = struct.Struct("@iiPPPqqqPfiiPqPPPNPP")
assert [_CACHE.size, _POOL.size, _ROPE.size, _ATTEND.size] == [C.sizeof(c) for c in (Cache, Pool, RopeBatch, AttendBatch)]
assert [_BLOCKS.size, _STORE.size, _LOAD.size, _PROMPT.size] == [C.sizeof(c) for c in (BlockCache, StoreBatch, LoadBatch, PromptBatch)]

EXPORTS = ["ss_kv_plan_create", "ss_kv_plan_destroy", "ss_kv_workspace_bytes", "ss_kv_append", "ss_kv_commit",
           "ss_rope_store", "ss_rope_frequencies", "ss_attend", "ss_kv_store_blocks", "ss_kv_load_blocks", "ss_attend_blocks",
           "ss_attend_prompt"]

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
    # structs go in by address: a reference to one, or its packed bytes
    L.ss_kv_append.argtypes = [_p, _p, _p, _p, _p, _p]
    L.ss_kv_commit.argtypes = [_p, _p, _p, _i32, _p]
    L.ss_rope_store.argtypes = [_p, _p]
    L.ss_rope_frequencies.argtypes = [C.POINTER(C.c_double), _i32, C.c_double, C.c_double, _i32, C.c_double, C.c_double]
    for name in ("ss_attend", "ss_kv_store_blocks", "ss_kv_load_blocks", "ss_attend_blocks"):
        getattr(L, name).argtypes = [_p, _p]
    L.ss_attend_prompt.argtypes = [_p]
    for name in ("ss_kv_plan_create", "ss_kv_append", "ss_kv_commit", "ss_rope_store", "ss_rope_frequencies", "ss_attend",
                 "ss_kv_store_blocks", "ss_kv_load_blocks", "ss_attend_blocks", "ss_attend_prompt"):
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
        self.dtype, self.cache_dtype, self.device = dtype, cache_dtype or dtype, device
        self.type, self.cache_type = _TORCH[self.dtype], _TORCH[self.cache_dtype]
        self.cache_shape = torch.Size((num_pages, page_size, kv_heads, head_dim))
        self.workspace_bytes = L.ss_kv_workspace_bytes(self._p)

    def __del__(self):
        try:
            if self._p:
                library().ss_kv_plan_destroy(self._p)
                self._p = _p()
        except Exception:
            pass


# The calls below are made once per layer and step, so their host time counts: element types are compared as objects,
# structs are packed, and the current stream is asked for by its raw handle.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, plan):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(plan.device)
    return torch.cuda.current_stream(plan.device).cuda_stream


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _bad(msg):
    return native.SSError(-1, msg)


def _elsewhere(name, t, plan):
    """The refusal of a tensor that is not on the plan's device."""
    if t.is_cuda:
        return _bad(f"{name} is on {t.device}, its plan on cuda:{plan.device}")
    return _bad(f"{name} is on the host: a device tensor is needed")


def _strides(plan, k_cache, v_cache):
    """Strides of k_cache and v_cache seen as [pages, page_size, kv_heads, head_dim], in any memory order of the first three."""
    if k_cache.shape != plan.cache_shape or v_cache.shape != plan.cache_shape:
        raise _bad(f"caches must be seen as [pages, page_size, kv_heads, head_dim] = {list(plan.cache_shape)}, got "
                   f"{list(k_cache.shape)} and {list(v_cache.shape)}")
    for t in (k_cache, v_cache):
        if t.get_device() != plan.device:
            raise _elsewhere("the cache", t, plan)
    if k_cache.dtype is not plan.cache_type or v_cache.dtype is not plan.cache_type:
        raise _bad(f"caches must be {plan.cache_type}, got {k_cache.dtype} and {v_cache.dtype}")
    st = k_cache.stride()
    if st != v_cache.stride() or st[3] != 1:
        raise _bad("both caches must have the same strides, and a head's values must be contiguous")
    return st


def _cache(plan, k_cache, v_cache, k_scale, v_scale):
    st = _strides(plan, k_cache, v_cache)
    if k_scale is not None or v_scale is not None:
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t is not None and (t.dtype is not torch.float32 or t.numel() != plan.kv_heads or not t.is_contiguous()):
                raise _bad(f"{name} must be {plan.kv_heads} contiguous float32 values")
            if t is not None and t.get_device() != plan.device:
                raise _elsewhere(name, t, plan)
    return _CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), st[0], st[1], st[2], _ptr(k_scale), _ptr(v_scale))


def _blocks(plan, k_cache, v_cache, k_scale, v_scale):
    """A cache with factors [pages, kv_heads, blocks of a page]."""
    if plan.cache_dtype != "e4m3":
        raise _bad(f"factors of blocks belong to a plan with cache_dtype e4m3, not {plan.cache_dtype}")
    st = _strides(plan, k_cache, v_cache)
    shape, f32, device = k_scale.shape, torch.float32, plan.device
    if len(shape) != 3 or shape[0] != plan.num_pages or shape[1] != plan.kv_heads or shape[2] < 1 or plan.page_size % shape[2]:
        raise _bad(f"k_scale must be [{plan.num_pages}, {plan.kv_heads}, blocks of a page], got {list(shape)}")
    if k_scale.dtype is not f32 or not k_scale.is_contiguous():
        raise _bad(f"k_scale must be contiguous float32, got {k_scale.dtype}")
    if v_scale.dtype is not f32 or v_scale.shape != shape or not v_scale.is_contiguous():
        raise _bad(f"v_scale must be contiguous float32 {list(shape)}, got {v_scale.dtype}, {list(v_scale.shape)}")
    if k_scale.get_device() != device:
        raise _elsewhere("k_scale", k_scale, plan)
    if v_scale.get_device() != device:
        raise _elsewhere("v_scale", v_scale, plan)
    return _BLOCKS.pack(k_cache.data_ptr(), v_cache.data_ptr(), st[0], st[1], st[2], k_scale.data_ptr(), v_scale.data_ptr(),
                        plan.page_size // shape[2])


def _tokens(name, t, heads, plan):
    """[tokens, heads, head_dim] with contiguous heads -> stride between tokens."""
    shape, st, d = t.shape, t.stride(), plan.head_dim
    if len(shape) != 3 or shape[1] != heads or shape[2] != d or st[2] != 1 or (heads > 1 and st[1] != d):
        raise _bad(f"{name} must be [tokens, {heads}, {d}] with contiguous heads, got {list(shape)} with strides {list(st)}")
    if t.dtype is not plan.type:
        raise _bad(f"{name} must be {plan.type}, got {t.dtype}")
    if t.get_device() != plan.device:
        raise _elsewhere(name, t, plan)
    if shape[0] <= 1:
        return heads * d  # the stride of one token is of no matter
    if st[0] % 8:
        raise native.SSError(-2, f"{name}: token strides must be multiples of 8 elements, got {st[0]}")
    return st[0]


def _int(plan, name, t, least):
    """Address of an int32 tensor of at least `least` entries."""
    if t.dtype is not _I32 or not t.is_contiguous() or t.numel() < least:
        raise _bad(f"{name} must be contiguous int32 with at least {least} entries, got {t.dtype}, {list(t.shape)}")
    if t.get_device() != plan.device:
        raise _elsewhere(name, t, plan)
    return t.data_ptr()


def _pool(plan, block_table, kv_len, free_pages, free_count, B, tokens, stream):
    return _POOL.pack(B, tokens, _int(plan, "block_table", block_table, B * plan.max_blocks), _int(plan, "kv_len", kv_len, B),
                      _int(plan, "free_pages", free_pages, plan.num_pages), _int(plan, "free_count", free_count, 1), _stream(stream, plan),
                      plan.handle)


def ss_kv_append(plan: Plan, block_table, kv_len, free_pages, free_count, cu_new, *, slots, positions, seq_len,
                 row_status, B=None, stream=None):
    """ss_kv_append on int32 tensors: pages, slots and positions of each row's new tokens.  A row with a token past the
    entries of slots or positions is not served."""
    B = kv_len.shape[0] if B is None else B
    pool = _pool(plan, block_table, kv_len, free_pages, free_count, B, min(slots.numel(), positions.numel()), stream)
    code = _lib.ss_kv_append(pool, _int(plan, "cu_new", cu_new, B + 1), _int(plan, "slots", slots, 0), _int(plan, "positions", positions, 0),
                             _int(plan, "seq_len", seq_len, B), _int(plan, "row_status", row_status, B))
    if code:
        native._check(code)


def ss_kv_commit(plan: Plan, block_table, kv_len, free_pages, free_count, seq_len, *, counts=None, plus=0, finished=None,
                 B=None, stream=None):
    """ss_kv_commit on int32 tensors: lengths move past what is kept, other pages go back to the pool."""
    B = kv_len.shape[0] if B is None else B
    pool = _pool(plan, block_table, kv_len, free_pages, free_count, B, 0, stream)
    code = _lib.ss_kv_commit(pool, _int(plan, "seq_len", seq_len, B), None if counts is None else _int(plan, "counts", counts, B), plus,
                             None if finished is None else _int(plan, "finished", finished, B))
    if code:
        native._check(code)


def ss_kv_store_blocks(plan: Plan, k, v, k_cache, v_cache, k_scale, v_scale, block_table, kv_len, seq_len, cu_new, *, row_status, B=None,
                       stream=None):
    """ss_kv_store_blocks: k, v [tokens, kv_heads, head_dim]; caches seen as [pages, page_size, kv_heads, head_dim]; k_scale, v_scale
    float32 [pages, kv_heads, page_size / block_tokens]; the lengths before and after the step as ss_kv_append has them."""
    B = kv_len.shape[0] if B is None else B
    cache = _blocks(plan, k_cache, v_cache, k_scale, v_scale)
    ks, vs = _tokens("k", k, plan.kv_heads, plan), _tokens("v", v, plan.kv_heads, plan)
    if k.shape[0] != v.shape[0]:
        raise _bad("k and v must have the same number of tokens")
    b = _STORE.pack(B, k.shape[0], k.data_ptr(), v.data_ptr(), ks, vs, _int(plan, "cu_new", cu_new, B + 1), _int(plan, "kv_len", kv_len, B),
                    _int(plan, "seq_len", seq_len, B), _int(plan, "block_table", block_table, B * plan.max_blocks),
                    _int(plan, "row_status", row_status, B), _stream(stream, plan), plan.handle)
    code = _lib.ss_kv_store_blocks(b, cache)
    if code:
        native._check(code)


def ss_kv_load_blocks(plan: Plan, k_cache, v_cache, k_scale, v_scale, slots, *, k_out, v_out, stream=None):
    """ss_kv_load_blocks: the tokens held at slots into k_out, v_out [tokens, kv_heads, head_dim]."""
    cache = _blocks(plan, k_cache, v_cache, k_scale, v_scale)
    ks, vs = _tokens("k_out", k_out, plan.kv_heads, plan), _tokens("v_out", v_out, plan.kv_heads, plan)
    T = slots.shape[0]
    if k_out.shape[0] != T or v_out.shape[0] != T:
        raise _bad("slots, k_out and v_out must have the same number of tokens")
    code = _lib.ss_kv_load_blocks(_LOAD.pack(T, _int(plan, "slots", slots, T), k_out.data_ptr(), v_out.data_ptr(), ks, vs, _stream(stream, plan),
                                             plan.handle), cache)
    if code:
        native._check(code)


def ss_rope_store(plan: Plan, q, k, v, k_cache, v_cache, inv_freq, positions, slots, *, q_out, q_weight=None,
                  k_weight=None, eps=1e-6, interleaved=False, rope_scale=1.0, k_scale=None, v_scale=None, stream=None):
    """ss_rope_store: q, k, v, q_out [tokens, heads, head_dim]; caches seen as [pages, page_size, kv_heads, head_dim];
    inv_freq [rot_dim / 2] float64 on the device (None: no rotation)."""
    T = q.shape[0]
    cache = _cache(plan, k_cache, v_cache, k_scale, v_scale)
    qs, ks = _tokens("q", q, plan.q_heads, plan), _tokens("k", k, plan.kv_heads, plan)
    vs, os = _tokens("v", v, plan.kv_heads, plan), _tokens("q_out", q_out, plan.q_heads, plan)
    if not (k.shape[0] == v.shape[0] == q_out.shape[0] == positions.shape[0] == slots.shape[0] == T):
        raise _bad("q, k, v, q_out, positions and slots must have the same number of tokens")
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None and (w.dtype is not plan.type or w.numel() != plan.head_dim or not w.is_contiguous()):
            raise _bad(f"{name} must be {plan.head_dim} contiguous {plan.type} values")
        if w is not None and w.get_device() != plan.device:
            raise _elsewhere(name, w, plan)
    rot = 0
    if inv_freq is not None:
        if inv_freq.dtype is not torch.float64 or not inv_freq.is_contiguous():
            raise _bad("inv_freq must be contiguous float64")
        if inv_freq.get_device() != plan.device:
            raise _elsewhere("inv_freq", inv_freq, plan)
        rot = 2 * inv_freq.shape[0]
    b = _ROPE.pack(T, q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs, _ptr(q_weight), _ptr(k_weight), eps, _ptr(inv_freq),
                  rot, 1 if interleaved else 0, rope_scale, _int(plan, "positions", positions, T), _int(plan, "slots", slots, T),
                  q_out.data_ptr(), os, _stream(stream, plan), plan.handle)
    code = _lib.ss_rope_store(b, cache)
    if code:
        native._check(code)


def rope_frequencies(rot_dim: int, base: float = 10000.0, *, factor: float = 1.0, original_len: int = 0,
                     low_turns: float = 1.0, high_turns: float = 32.0) -> np.ndarray:
    """ss_rope_frequencies: float64 [rot_dim / 2] on the host."""
    out = np.empty(max(rot_dim // 2, 1), np.float64)
    native._check(library().ss_rope_frequencies(out.ctypes.data_as(C.POINTER(C.c_double)), rot_dim, base, factor,
                                                original_len, low_turns, high_turns))
    return out


def _outputs(plan, q, out, lse, workspace):
    """Checks of an attention call's outputs and workspace."""
    if out.shape[0] < q.shape[0]:
        raise _bad("out must have as many tokens as q")
    if lse is not None and (lse.dtype is not torch.float32 or not lse.is_contiguous() or lse.numel() < q.shape[0] * plan.q_heads):
        raise _bad("lse must be contiguous float32 [tokens, q_heads]")
    if not workspace.is_contiguous():
        raise _bad(f"workspace must be contiguous, got strides {list(workspace.stride())}")
    for name, t in (("workspace", workspace), ("lse", lse)):
        if t is not None and t.get_device() != plan.device:
            raise _elsewhere(name, t, plan)


def _attend(plan, q, block_table, seq_len, cu_new, out, row_status, workspace, scale, window, sinks, lse, B, stream):
    """The batch of an attention call."""
    B = seq_len.shape[0] if B is None else B
    qs, os = _tokens("q", q, plan.q_heads, plan), _tokens("out", out, plan.q_heads, plan)
    _outputs(plan, q, out, lse, workspace)
    return _ATTEND.pack(B, q.shape[0], q.data_ptr(), qs, _int(plan, "cu_new", cu_new, B + 1), _int(plan, "seq_len", seq_len, B),
                        _int(plan, "block_table", block_table, B * plan.max_blocks), scale, window, sinks, out.data_ptr(), os, _ptr(lse),
                        _int(plan, "row_status", row_status, B), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                        _stream(stream, plan), plan.handle)


def ss_attend(plan: Plan, q, k_cache, v_cache, block_table, seq_len, cu_new, *, out, row_status, workspace, scale,
              window=0, sinks=0, lse=None, k_scale=None, v_scale=None, B=None, stream=None):
    """ss_attend: q, out [tokens, q_heads, head_dim]; caches seen as [pages, page_size, kv_heads, head_dim]; lse float32
    [tokens, q_heads] or None.  A row with a token past those of q is left out."""
    b = _attend(plan, q, block_table, seq_len, cu_new, out, row_status, workspace, scale, window, sinks, lse, B, stream)
    code = _lib.ss_attend(b, _cache(plan, k_cache, v_cache, k_scale, v_scale))
    if code:
        native._check(code)


def ss_attend_blocks(plan: Plan, q, k_cache, v_cache, k_scale, v_scale, block_table, seq_len, cu_new, *, out, row_status, workspace, scale,
                     window=0, sinks=0, lse=None, B=None, stream=None):
    """ss_attend_blocks: as ss_attend, over a cache with factors k_scale, v_scale float32 [pages, kv_heads, page_size / block_tokens]."""
    b = _attend(plan, q, block_table, seq_len, cu_new, out, row_status, workspace, scale, window, sinks, lse, B, stream)
    code = _lib.ss_attend_blocks(b, _blocks(plan, k_cache, v_cache, k_scale, v_scale))
    if code:
        native._check(code)


def ss_attend_prompt(plan: Plan, q, k, v, cu_seq, *, out, row_status, workspace, scale, window=0, sinks=0, lse=None, B=None, stream=None):
    """ss_attend_prompt: q, out [tokens, q_heads, head_dim], k, v [tokens, kv_heads, head_dim], prompts one after the other; lse float32
    [tokens, q_heads] or None.  A prompt with a token past those of q is left out."""
    B = cu_seq.shape[0] - 1 if B is None else B
    qs, os = _tokens("q", q, plan.q_heads, plan), _tokens("out", out, plan.q_heads, plan)
    ks, vs = _tokens("k", k, plan.kv_heads, plan), _tokens("v", v, plan.kv_heads, plan)
    if k.shape[0] != q.shape[0] or v.shape[0] != q.shape[0]:
        raise _bad("q, k and v must have the same number of tokens")
    _outputs(plan, q, out, lse, workspace)
    b = _PROMPT.pack(B, q.shape[0], q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs, _int(plan, "cu_seq", cu_seq, B + 1), scale, window, sinks,
                     out.data_ptr(), os, _ptr(lse), _int(plan, "row_status", row_status, B), workspace.data_ptr(),
                     workspace.numel() * workspace.element_size(), _stream(stream, plan), plan.handle)
    code = _lib.ss_attend_prompt(b)
    if code:
        native._check(code)
