"""Attention and the 8-bit key/value cache (``include/entro_attn.h``).

The part of a layer between the fused products: ``attn_prompt`` (causal
attention of packed prompts), ``kv_store`` and ``kv_load`` (keys and values
into the paged 8-bit cache and back), ``attn_cache`` (one new token per
sequence over the cache).  Operands are torch tensors on the HIP device; the
functions check shapes and types, pass pointers and strides on, and return
without waiting.  Work goes to ``stream`` (a torch stream or a raw handle;
default: the current stream).  The caller orders it after the work that made
its tensors; their memory is kept until a torch stream has used them (on a raw
handle that, too, is the caller's).  ``status`` is an int32 tensor with one entry per sequence,
zeroed by the caller, in which faults found in the data are OR-ed
(``FLAGS["length"]``, ``FLAGS["page"]``).  There is no backward pass: operands that
require a gradient are refused outside ``torch.no_grad()``.
"""
from __future__ import annotations

import ctypes
import operator

__all__ = ["KVCache", "attn_prompt", "kv_store", "kv_load", "attn_cache", "attn_prompt_work_bytes", "attn_cache_work_bytes"]

_P, _U32, _I64 = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_int64


# The structures of the C ABI, for callers of it through ctypes.  (The functions
# below fill them in C++, csrc/entro_attn_py.cpp.)

class Rows(ctypes.Structure):
    _fields_ = [("d", _P), ("stride_t", _I64), ("stride_h", _I64)]


class Cache(ctypes.Structure):
    _fields_ = [("d_k_codes", _P), ("d_v_codes", _P), ("d_k_scales", _P), ("d_v_scales", _P), ("n_pages", _U32),
                ("page_tokens", _U32), ("n_kv_heads", _U32), ("head_dim", _U32)]


class Table(ctypes.Structure):
    _fields_ = [("d_table", _P), ("table_stride", _U32), ("table_pages", _U32), ("n_seq", _U32)]


class PromptArgs(ctypes.Structure):
    _fields_ = [("q", Rows), ("k", Rows), ("v", Rows), ("out", Rows), ("d_cu_q", _P), ("d_cu_k", _P), ("n_seq", _U32),
                ("total_q", _U32), ("total_k", _U32), ("n_heads", _U32), ("n_kv_heads", _U32), ("head_dim", _U32),
                ("dtype", ctypes.c_int), ("scale", ctypes.c_float), ("d_work", _P), ("work_bytes", ctypes.c_uint64)]


class StoreArgs(ctypes.Structure):
    _fields_ = [("k", Rows), ("v", Rows), ("d_pos", _P), ("d_cu", _P), ("total", _U32), ("dtype", ctypes.c_int)]


class CacheArgs(ctypes.Structure):
    _fields_ = [("q", Rows), ("out", Rows), ("d_lens", _P), ("n_heads", _U32), ("dtype", ctypes.c_int),
                ("scale", ctypes.c_float), ("d_work", _P), ("work_bytes", ctypes.c_uint64)]


def _bind(lib):
    for name in ("entro_kv_store", "entro_kv_load", "entro_attn_cache"):
        getattr(lib, name).argtypes = [_P, _P, _P, _P, _P]
        getattr(lib, name).restype = ctypes.c_int
    lib.entro_attn_prompt.argtypes = [_P, _P, _P]
    lib.entro_attn_prompt.restype = ctypes.c_int
    lib.entro_attn_prompt_work_bytes.argtypes = [_U32] * 6
    lib.entro_attn_prompt_work_bytes.restype = ctypes.c_uint64
    lib.entro_attn_cache_work_bytes.argtypes = [_U32] * 4
    lib.entro_attn_cache_work_bytes.restype = ctypes.c_uint64
    lib.entro_attn_set_max_workgroups.argtypes = [_U32]
    lib.entro_attn_set_max_workgroups.restype = _U32


# torch and the binding in C++, from the first call on (the package's host side
# works without)
torch = None
_ext = None


def _load_ext():
    """The binding in C++ (``_attn.so`` next to this file)."""
    global torch, _ext
    if _ext is None:
        import torch as t

        from . import LibraryNotBuilt, _check, load

        lib = load()
        try:
            from . import _attn as e
        except ImportError as x:
            raise LibraryNotBuilt(
                f"_attn.so: {x}; build it with `python -m entropy_coded_weight_canonical_amd.build`") from x
        e.bind(*(ctypes.cast(getattr(lib, f), _P).value for f in (
            "entro_attn_prompt", "entro_attn_prompt_work_bytes", "entro_kv_store", "entro_kv_load", "entro_attn_cache",
            "entro_attn_cache_work_bytes")), t._C._cuda_getCurrentRawStream, _check)
        torch, _ext = t, e
    return _ext


def _kept(slot):
    """A KVCache's attribute, held in `slot`: it can only be set to what it is
    (as an operation in place does)."""

    def keep(self, value):
        if value is not getattr(self, slot):
            raise AttributeError("a KVCache keeps the tensors that it was made of: make another of the new ones")

    return property(operator.attrgetter(slot), keep)


class KVCache:
    """Pages of 8-bit keys and values: ``k_codes`` int8 [pages][kv heads][page
    tokens][dim], ``v_codes`` int8 [pages][kv heads][dim][page tokens],
    ``k_scales`` / ``v_scales`` float32 [pages][kv heads].  Holds the tensors,
    so that the device memory outlives the calls; they cannot be replaced."""

    __slots__ = ("_k_codes", "_v_codes", "_k_scales", "_v_scales", "_desc")
    k_codes, v_codes, k_scales, v_scales, desc = (_kept(s) for s in __slots__)

    def __init__(self, k_codes, v_codes, k_scales, v_scales):
        self._desc = (_ext or _load_ext()).cache_desc(k_codes, v_codes, k_scales, v_scales)
        self._k_codes, self._v_codes, self._k_scales, self._v_scales = k_codes, v_codes, k_scales, v_scales

    @property
    def tensors(self):
        return self.k_codes, self.v_codes, self.k_scales, self.v_scales

    @classmethod
    def empty(cls, n_pages: int, n_kv_heads: int, head_dim: int, page_tokens: int = 64, device="cuda"):
        """A cache of ``n_pages`` unused pages (16, 32, 64 or 128 tokens each)."""
        _load_ext()
        codes = lambda *s: torch.zeros(n_pages, n_kv_heads, *s, dtype=torch.int8, device=device)  # noqa: E731
        scales = lambda: torch.zeros(n_pages, n_kv_heads, dtype=torch.float32, device=device)  # noqa: E731
        return cls(codes(page_tokens, head_dim), codes(head_dim, page_tokens), scales(), scales())


def _on(stream, call, *args):
    """``call`` on a given stream.  Tensors that a torch stream other than their
    own uses are noted with torch, which then keeps their memory until that
    stream is through with them, however early the caller drops them; memory of
    results is that stream's.  On a raw handle all that is the caller's."""
    if not hasattr(stream, "cuda_stream"):
        return call(*args, False, int(stream))
    cache = [x for x in args if isinstance(x, KVCache)]
    with torch.cuda.stream(stream):
        r = call(*args, True, stream.cuda_stream)
    for x in (*args, *(y for c in cache for y in c.tensors), *(r if isinstance(r, tuple) else (r,))):
        if isinstance(x, torch.Tensor):
            x.record_stream(stream)
    return r


def attn_prompt_work_bytes(n_seq: int, rows_q: int, rows_k: int, n_heads: int, n_kv_heads: int, head_dim: int) -> int:
    """``entro_attn_prompt_work_bytes``: the workspace of ``attn_prompt`` (0:
    none)."""
    from . import load

    return int(load().entro_attn_prompt_work_bytes(n_seq, rows_q, rows_k, n_heads, n_kv_heads, head_dim))


def attn_prompt(q, k, v, cu_q, cu_k, status, scale=None, out=None, stream=None, work=None):
    """Causal attention of packed sequences (``entro_attn_prompt``): ``q``
    [rows][heads][dim], ``k`` and ``v`` [rows][kv heads][dim] with any row and
    head strides that are multiples of 8, ``cu_q`` and ``cu_k`` int32 running
    sums (n + 1).  A sequence's last keys are its queries' own; more keys than
    queries are tokens in front of them.  ``work``: a contiguous tensor of at
    least ``attn_prompt_work_bytes`` bytes that no call on another stream uses
    meanwhile (made for the call by default, but on a raw stream handle: there
    the keys of few queries are then not split over more workgroups).  Returns
    ``out`` [rows][heads][dim] (rows of no sequence are left as they are)."""
    e = _ext or _load_ext()
    if stream is not None:
        return _on(stream, e.attn_prompt, q, k, v, cu_q, cu_k, status, scale, out, work)
    return e.attn_prompt(q, k, v, cu_q, cu_k, status, scale, out, work, True, None)


def kv_store(cache: KVCache, k, v, table, held, cu_new, status, stream=None) -> None:
    """Write packed new keys and values behind the ``held`` tokens of each
    sequence (``entro_kv_store``)."""
    e = _ext or _load_ext()
    if stream is not None:
        _on(stream, e.kv_store, cache, k, v, table, held, cu_new, status)
    else:
        e.kv_store(cache, k, v, table, held, cu_new, status, True, None)


def kv_load(cache: KVCache, table, first, cu_out, total: int, status, dtype=None, out=None, stream=None):
    """Read tokens back as 16-bit values (``entro_kv_load``): for sequence b
    the ``cu_out[b + 1] - cu_out[b]`` tokens from position ``first[b]`` on.
    Returns ``(k, v)``, each [total][kv heads][dim], of ``dtype`` (default
    bfloat16) or the pair ``out``, whose type it then is."""
    e = _ext or _load_ext()
    k, v = (None, None) if out is None else out
    if dtype is not None:
        if dtype is not torch.bfloat16 and dtype is not torch.float16:
            raise ValueError(f"element type {dtype}: bfloat16 or float16 expected")
        for x in out or ():
            if isinstance(x, torch.Tensor) and x.dtype is not dtype:
                raise ValueError(f"element type {dtype} with outputs of type {x.dtype}")
    f16 = dtype is torch.float16
    if stream is not None:
        return _on(stream, e.kv_load, cache, table, first, cu_out, total, status, f16, k, v)
    return e.kv_load(cache, table, first, cu_out, total, status, f16, k, v, True, None)


def attn_cache_work_bytes(n_seq: int, n_heads: int, n_kv_heads: int, head_dim: int) -> int:
    """``entro_attn_cache_work_bytes``: the workspace of ``attn_cache``."""
    from . import load

    return int(load().entro_attn_cache_work_bytes(n_seq, n_heads, n_kv_heads, head_dim))


def attn_cache(q, cache: KVCache, table, lens, status, scale=None, out=None, work=None, stream=None):
    """Attention of one new token per sequence over the cache
    (``entro_attn_cache``): ``q`` [n][heads][dim], ``lens`` the tokens of each
    sequence in the cache, the new one among them.  ``work``: a contiguous
    tensor of at least ``attn_cache_work_bytes`` bytes that no call on another
    stream uses meanwhile (made for the call by default).  Returns ``out``
    [n][heads][dim]."""
    e = _ext or _load_ext()
    if stream is not None:
        return _on(stream, e.attn_cache, q, cache, table, lens, status, scale, out, work)
    return e.attn_cache(q, cache, table, lens, status, scale, out, work, True, None)
