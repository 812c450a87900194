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
(``FLAGS["length"]``, ``FLAGS["page"]``).
"""
from __future__ import annotations

import ctypes
import math
import struct

__all__ = ["KVCache", "attn_prompt", "kv_store", "kv_load", "attn_cache", "attn_prompt_work_bytes", "attn_cache_work_bytes"]

_P, _U32, _I64 = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_int64


# The structures of the C ABI.  The functions below pack the same bytes
# themselves (a tenth of the time of filling a structure by its fields: a
# call's work in Python is of the order of a small call's time on the GPU).

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


_PROMPT = struct.Struct("@PqqPqqPqqPqqPPIIIIIIifPQ")
_STORE = struct.Struct("@PqqPqqPPIi")
_CACHE = struct.Struct("@PqqPqqPIifPQ")
_TABLE = struct.Struct("@PIIIi")
_PAGES = struct.Struct("@PPPPIIII")

# torch and what of it the calls use, from the first call on (the package's
# host side works without)
torch = None
_DTYPES: dict = {}
_raw_stream = None


def _torch_once() -> None:
    global torch, _raw_stream
    if torch is None:
        import torch as t

        _DTYPES.update({t.bfloat16: 0, t.float16: 1})
        _raw_stream = t._C._cuda_getCurrentRawStream
        torch = t


def _dtype_id(dtype) -> int:
    i = _DTYPES.get(dtype)
    if i is None:
        raise ValueError(f"element type {dtype}: bfloat16 or float16 expected")
    return i


def _rows(x, what: str, dtype, heads: int, dim: int):
    """(pointer, row stride, head stride) of a 16-bit operand."""
    shape = x.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{what}: shape {tuple(shape)}, expected [rows, {heads}, {dim}]")
    if x.dtype is not dtype or not x.is_cuda:
        raise ValueError(f"{what}: a {dtype} tensor on the GPU expected, got {x.dtype} on {x.device}")
    st, sh, sd = x.stride()
    if sd != 1:
        raise ValueError(f"{what}: the head dimension has to be contiguous")
    return x.data_ptr(), st if shape[0] > 1 else heads * dim, sh if heads > 1 else dim


def _ints(x, what: str, n: int) -> int:
    if x.dtype is not torch.int32 or x.shape != (n,) or not x.is_cuda or (n > 1 and not x.is_contiguous()):
        raise ValueError(f"{what}: {n} contiguous int32 values on the GPU expected, got {x.dtype} {tuple(x.shape)} on {x.device}")
    return x.data_ptr()


class KVCache:
    """Pages of 8-bit keys and values: ``k_codes`` int8 [pages][kv heads][page
    tokens][dim], ``v_codes`` int8 [pages][kv heads][dim][page tokens],
    ``k_scales`` / ``v_scales`` float32 [pages][kv heads].  Holds the tensors,
    so that the device memory outlives the calls."""

    __slots__ = ("k_codes", "v_codes", "k_scales", "v_scales", "tensors", "kv_heads", "dim", "desc")

    def __init__(self, k_codes, v_codes, k_scales, v_scales):
        _torch_once()
        if k_codes.dim() != 4 or v_codes.dim() != 4:
            raise ValueError("k_codes and v_codes have four dimensions")
        pages, kv, page, dim = k_codes.shape
        if v_codes.shape != (pages, kv, dim, page) or k_scales.shape != (pages, kv) or v_scales.shape != (pages, kv):
            raise ValueError("the shapes of codes and scales do not belong together")
        for x, dtype in ((k_codes, torch.int8), (v_codes, torch.int8), (k_scales, torch.float32), (v_scales, torch.float32)):
            if x.dtype is not dtype or not x.is_cuda or not x.is_contiguous():
                raise ValueError("int8 codes and float32 scales, contiguous and on the GPU, expected")
        self.tensors = self.k_codes, self.v_codes, self.k_scales, self.v_scales = k_codes, v_codes, k_scales, v_scales
        self.kv_heads, self.dim = kv, dim
        self.desc = _PAGES.pack(k_codes.data_ptr(), v_codes.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), pages, page,
                                kv, dim)

    @classmethod
    def empty(cls, n_pages: int, n_kv_heads: int, head_dim: int, page_tokens: int = 64, device="cuda"):
        """A cache of ``n_pages`` unused pages (16, 32, 64 or 128 tokens each)."""
        _torch_once()
        codes = lambda *s: torch.zeros(n_pages, n_kv_heads, *s, dtype=torch.int8, device=device)  # noqa: E731
        scales = lambda: torch.zeros(n_pages, n_kv_heads, dtype=torch.float32, device=device)  # noqa: E731
        return cls(codes(page_tokens, head_dim), codes(head_dim, page_tokens), scales(), scales())


def _table(table, n: int) -> bytes:
    if table.dtype is not torch.int32 or table.dim() != 2 or table.shape[0] != n or not table.is_cuda:
        raise ValueError(f"table: int32 [{n}][pages] on the GPU expected, got {table.dtype} {tuple(table.shape)} on {table.device}")
    pages = table.shape[1]
    sn, sp = table.stride()
    if pages > 1 and sp != 1:
        raise ValueError("table: the pages of a sequence have to lie side by side")
    return _TABLE.pack(table.data_ptr(), sn if n > 1 else pages, pages, n, 0)


def _on(stream, *used) -> int:
    """The stream's handle.  Tensors that a torch stream other than their own
    uses are noted with torch, which then keeps their memory until that stream
    is through with them, however early the caller drops them."""
    if stream is None:
        return _raw_stream(used[0].get_device())
    if hasattr(stream, "cuda_stream"):
        for x in used:
            x.record_stream(stream)
        return stream.cuda_stream
    return int(stream)


_fns: dict = {}


def _call(name: str, *args) -> None:
    fn = _fns.get(name)
    if fn is None:
        from . import load

        fn = _fns[name] = getattr(load(), name)
    status = fn(*args)
    if status:
        from . import _check

        _check(status, name)


def _empty(shape, dtype, like, stream):
    """Memory of a result: from the stream that writes it, so that torch does
    not hand it out again before."""
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device=like.device)
    if not hasattr(stream, "cuda_stream"):
        raise ValueError("on a raw stream handle the caller gives the memory of results and workspace")
    with torch.cuda.stream(stream):
        return torch.empty(*shape, dtype=dtype, device=like.device)


def _workspace(work):
    """(pointer, bytes) of a workspace."""
    if not work.is_cuda or not work.is_contiguous():
        raise ValueError("work: a contiguous tensor on the GPU expected")
    return work.data_ptr(), work.numel() * work.element_size()


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
    _torch_once()
    n = cu_q.shape[0] - 1
    if n < 0 or q.dim() != 3 or k.dim() != 3:
        raise ValueError("q, k, v are [rows][heads][dim], cu_q and cu_k hold n + 1 sums")
    rows, heads, dim = q.shape
    kv = k.shape[1]
    if v.shape[0] != k.shape[0]:
        raise ValueError("k and v have the same rows")
    t = q.dtype
    if out is None:
        out = _empty((rows, heads, dim), t, q, stream)
        ro = out.data_ptr(), heads * dim, dim
    else:
        ro = _rows(out, "out", t, heads, dim)
        if out.shape[0] != rows:
            raise ValueError("out has the rows of q")
    w = size = 0
    if work is not None:
        w, size = _workspace(work)
    elif n and k.shape[0] >= 1024 * n and (stream is None or hasattr(stream, "cuda_stream")):   # (none below)
        size = attn_prompt_work_bytes(n, rows, k.shape[0], heads, kv, dim)
        if size:
            work = _empty((size,), torch.uint8, q, stream)
            w = work.data_ptr()
    a = _PROMPT.pack(*_rows(q, "q", t, heads, dim), *_rows(k, "k", t, kv, dim), *_rows(v, "v", t, kv, dim), *ro,
                     _ints(cu_q, "cu_q", n + 1), _ints(cu_k, "cu_k", n + 1), n, rows,
                     k.shape[0], heads, kv, dim, _dtype_id(t), 1.0 / math.sqrt(dim) if scale is None else scale, w, size)
    used = (q, k, v, cu_q, cu_k, status, out) if work is None else (q, k, v, cu_q, cu_k, status, out, work)
    _call("entro_attn_prompt", a, _ints(status, "status", n), _on(stream, *used))
    return out


def kv_store(cache: KVCache, k, v, table, held, cu_new, status, stream=None) -> None:
    """Write packed new keys and values behind the ``held`` tokens of each
    sequence (``entro_kv_store``)."""
    _torch_once()
    n = table.shape[0]
    kv, dim = cache.kv_heads, cache.dim
    if k.shape[0] != v.shape[0]:
        raise ValueError("k and v have the same rows")
    t = k.dtype
    a = _STORE.pack(*_rows(k, "k", t, kv, dim), *_rows(v, "v", t, kv, dim), _ints(held, "held", n),
                    _ints(cu_new, "cu_new", n + 1), k.shape[0], _dtype_id(t))
    _call("entro_kv_store", cache.desc, _table(table, n), a, _ints(status, "status", n),
          _on(stream, k, v, *cache.tensors, table, held, cu_new, status))


def kv_load(cache: KVCache, table, first, cu_out, total: int, status, dtype=None, out=None, stream=None):
    """Read tokens back as 16-bit values (``entro_kv_load``): for sequence b
    the ``cu_out[b + 1] - cu_out[b]`` tokens from position ``first[b]`` on.
    Returns ``(k, v)``, each [total][kv heads][dim], of ``dtype`` (default
    bfloat16) or the pair ``out``."""
    _torch_once()
    n = table.shape[0]
    kv, dim = cache.kv_heads, cache.dim
    if out is None:
        dtype = torch.bfloat16 if dtype is None else dtype
        out = (_empty((total, kv, dim), dtype, cache.k_codes, stream), _empty((total, kv, dim), dtype, cache.k_codes, stream))
    k, v = out
    if k.shape[0] != total or v.shape[0] != total:
        raise ValueError("the outputs have `total` rows")
    t = k.dtype
    a = _STORE.pack(*_rows(k, "k", t, kv, dim), *_rows(v, "v", t, kv, dim), _ints(first, "first", n),
                    _ints(cu_out, "cu_out", n + 1), total, _dtype_id(t))
    _call("entro_kv_load", cache.desc, _table(table, n), a, _ints(status, "status", n),
          _on(stream, k, v, *cache.tensors, table, first, cu_out, status))
    return k, v


def attn_cache_work_bytes(n_seq: int, n_heads: int, n_kv_heads: int, head_dim: int) -> int:
    """``entro_attn_cache_work_bytes``: the workspace of ``attn_cache``."""
    from . import load

    return int(load().entro_attn_cache_work_bytes(n_seq, n_heads, n_kv_heads, head_dim))


_work_sizes: dict = {}   # workspace by the call's sizes


def attn_cache(q, cache: KVCache, table, lens, status, scale=None, out=None, work=None, stream=None):
    """Attention of one new token per sequence over the cache
    (``entro_attn_cache``): ``q`` [n][heads][dim], ``lens`` the tokens of each
    sequence in the cache, the new one among them.  ``work``: a contiguous
    tensor of at least ``attn_cache_work_bytes`` bytes that no call on another
    stream uses meanwhile (made for the call by default).  Returns ``out``
    [n][heads][dim]."""
    _torch_once()
    if q.dim() != 3:
        raise ValueError("q is [sequences][heads][dim]")
    n, heads, dim = q.shape
    kv = cache.kv_heads
    if dim != cache.dim:
        raise ValueError(f"q has head dimension {dim}, the cache {cache.dim}")
    t = q.dtype
    if out is None:
        out = _empty((n, heads, dim), t, q, stream)
        ro = out.data_ptr(), heads * dim, dim
    else:
        ro = _rows(out, "out", t, heads, dim)
        if out.shape[0] != n:
            raise ValueError("out has the rows of q")
    if work is None:
        need = _work_sizes.get((n, heads, kv, dim))
        if need is None:
            if len(_work_sizes) >= 4096:
                _work_sizes.clear()
            need = _work_sizes[n, heads, kv, dim] = attn_cache_work_bytes(n, heads, kv, dim)
        work = _empty((max(need, 16),), torch.uint8, q, stream)
    w, size = _workspace(work)
    a = _CACHE.pack(*_rows(q, "q", t, heads, dim), *ro, _ints(lens, "lens", n), heads, _dtype_id(t),
                    1.0 / math.sqrt(dim) if scale is None else scale, w, size)
    _call("entro_attn_cache", cache.desc, _table(table, n), a, _ints(status, "status", n),
          _on(stream, q, *cache.tensors, table, lens, status, out, work))
    return out
