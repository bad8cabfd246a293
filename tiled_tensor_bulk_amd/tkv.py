"""Python binding of libtkv: a paged key/value cache in 4 bits and the
operators on it (include/tkv.h).  Argument checks and marshalling only; raises
if libtkv.so or _tkv.so has not been built -- there is no fallback.  The calls
that a step of decoding makes go through _tkv.so (csrc/tkv_torch.cpp), the
others through ctypes, whose structures are those of the header.

Names match the C ABI.  Tensors lie on the current GPU; work goes to `stream`
(an int, a torch stream, or None: torch's current one).  Outputs and the
workspace are allocated with torch where they are not given, from the memory
of that stream; outputs are kept for torch's current stream too.  A caller who
names a stream orders it after the work that makes the inputs, and keeps these
until it is done with them, as everywhere in torch.  There is no backward pass:
a tensor that requires a gradient is refused outside torch.no_grad().

    pool  = torch.empty(n_pages * tkv_page_bytes_of(heads, dim, page, group), dtype=torch.uint8, device="cuda")
    cache = tkv_encode(pool, heads, dim, page, group)
    tkv_append(cache, k, v, table, lens)               # new tokens at lens[b] ..
    out, lse = tkv_attend(cache, q, table, lens + 1)   # one new token each
    kept, lens, scores = tkv_evict(cache, table, lens, scores, budget, recent, new_table)
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import torch

from .tmap import SUCCESS, TmapError

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtkv.so")

TILE = 32  # positions of a record
_DTYPES = {torch.float16: 3, torch.bfloat16: 4, torch.float32: 7}


class tkv_cache(ctypes.Structure):
    """The encoded descriptor; keeps its pool alive and remembers its shape."""
    _fields_ = [("opaque", ctypes.c_uint64 * 16)]


class tkv_tokens(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int32)]


class tkv_batch(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("lens", ctypes.c_void_p),
                ("starts", ctypes.c_void_p), ("n_tokens", ctypes.c_int64), ("n_seq", ctypes.c_int32),
                ("table_width", ctypes.c_int32), ("max_new", ctypes.c_int32)]


class tkv_attend_args(ctypes.Structure):
    _fields_ = [("q", tkv_tokens), ("out", tkv_tokens), ("lse", ctypes.c_void_p), ("scores_in", ctypes.c_void_p),
                ("scores_out", ctypes.c_void_p), ("score_stride", ctypes.c_int64), ("q_heads", ctypes.c_int32),
                ("max_len", ctypes.c_int32), ("scale", ctypes.c_float), ("causal", ctypes.c_int32),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_uint64)]


class tkv_evict_args(ctypes.Structure):
    _fields_ = [("scores", ctypes.c_void_p), ("scores_out", ctypes.c_void_p), ("score_stride", ctypes.c_int64),
                ("kept", ctypes.c_void_p), ("lens_out", ctypes.c_void_p), ("dst_table", ctypes.c_void_p),
                ("dst_stride", ctypes.c_int64), ("dst_width", ctypes.c_int32), ("budget", ctypes.c_int32),
                ("recent", ctypes.c_int32), ("max_len", ctypes.c_int32)]


_lib = None


def lib():
    """Load libtkv.so (raises if it is missing)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run: python -m tiled_tensor_bulk_amd.build")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER
        vp, u32 = ctypes.c_void_p, ctypes.c_uint32
        L.tkv_encode.argtypes = [P(tkv_cache), vp, ctypes.c_int64, u32, u32, u32, u32]
        L.tkv_encode.restype = ctypes.c_int
        L.tkv_page_bytes.argtypes = [P(tkv_cache)]
        L.tkv_page_bytes.restype = ctypes.c_uint64
        for name in ("tkv_append", "tkv_read"):
            f = getattr(L, name)
            f.argtypes = [P(tkv_cache), P(tkv_tokens), P(tkv_tokens), P(tkv_batch), vp]
            f.restype = ctypes.c_int
        L.tkv_attend.argtypes = [P(tkv_cache), P(tkv_attend_args), P(tkv_batch), vp]
        L.tkv_attend.restype = ctypes.c_int
        for name in ("tkv_attend_workspace", "tkv_attend_workspace_bound"):
            f = getattr(L, name)
            f.argtypes = [P(tkv_cache), P(tkv_attend_args), P(tkv_batch), P(ctypes.c_uint64)]
            f.restype = ctypes.c_int
        L.tkv_evict.argtypes = [P(tkv_cache), P(tkv_evict_args), P(tkv_batch), vp]
        L.tkv_evict.restype = ctypes.c_int
        L.tkv_last_error_detail.argtypes = []
        L.tkv_last_error_detail.restype = ctypes.c_char_p
        _lib = L
    return _lib


_torch = None


def _calls():
    """Load _tkv.so (raises if it is missing)."""
    global _torch
    if _torch is None:
        lib()
        try:
            from . import _tkv
        except ImportError as err:
            raise ImportError(f"{_HERE}/_tkv.so is not built; run: python -m tiled_tensor_bulk_amd.build ({err})") from None
        _torch = _tkv
    return _torch


def tkv_last_error_detail() -> str:
    return lib().tkv_last_error_detail().decode()


def _check(st: int, where: str) -> None:
    if st != SUCCESS:
        raise TmapError(st, where, tkv_last_error_detail())


def _stream(s):
    """None for torch's current stream, else the stream's handle."""
    if s is None or isinstance(s, int):
        return s
    return s.cuda_stream


def _keep(s, device, *made):
    """Tensors made from the memory of stream s are kept for torch's current one, where the caller goes on with them."""
    here = torch.cuda.current_stream(device)
    if here.cuda_stream != _stream(s):
        for t in made:
            if t is not None:
                t.record_stream(here)


def tkv_page_bytes_of(n_heads: int, head_dim: int, page_tokens: int, group: int) -> int:
    """Bytes of one page, before there is a pool."""
    return n_heads * (page_tokens // TILE) * (32 * head_dim + 256 * (head_dim // group))


def tkv_encode(pool, n_heads: int, head_dim: int, page_tokens: int, group: int = 64) -> tkv_cache:
    """Describe a pool: a contiguous uint8 GPU tensor of whole pages."""
    if not isinstance(pool, torch.Tensor) or pool.dtype != torch.uint8:
        raise ValueError("pool must be a uint8 tensor")
    if not pool.is_cuda:
        raise ValueError("pool must be a GPU tensor")
    if not pool.is_contiguous():
        raise ValueError("pool must be contiguous")
    c = tkv_cache()
    each = tkv_page_bytes_of(n_heads, head_dim, page_tokens, group) if group > 0 else 0
    n_pages = pool.numel() // each if each > 0 else 1
    _check(lib().tkv_encode(ctypes.byref(c), pool.data_ptr(), n_pages, n_heads, head_dim, page_tokens, group),
           "tkv_encode")
    if pool.numel() % each:
        raise ValueError(f"pool holds {pool.numel()} bytes, not a multiple of a page's {each}")
    c.pool, c.n_heads, c.head_dim, c.page_tokens, c.group, c.n_pages = (pool, n_heads, head_dim, page_tokens, group,
                                                                        n_pages)
    c.calls = _calls().Cache(ctypes.addressof(c), pool, n_heads, head_dim, page_tokens)
    return c


def tkv_page_bytes(cache: tkv_cache) -> int:
    return int(lib().tkv_page_bytes(ctypes.byref(cache)))


def tkv_append(cache: tkv_cache, k, v, table, lens, starts=None, max_new: Optional[int] = None, stream=None) -> None:
    """Quantise k and v [tokens, heads, head_dim] (fp16 or bf16) and put them at positions lens[b] .. of each
    sequence's pages.  starts: int32 [sequences + 1] row offsets, None for equally many tokens each; max_new: a
    bound on a sequence's new tokens (default: what the shapes allow)."""
    st = _torch.append(cache.calls, k, v, table, lens, starts, max_new, _stream(stream))
    _check(st, "tkv_append")


def tkv_read(cache: tkv_cache, table, lens, starts=None, max_new: Optional[int] = None, n_tokens: Optional[int] = None,
             dtype=torch.float16, k=None, v=None, stream=None):
    """Keys and values at positions lens[b] .. of each sequence as numbers, [n_tokens, heads, head_dim] in dtype
    (fp16, bf16, fp32); arguments as for tkv_append.  Rows that no sequence's range names are left as they were
    (in tensors made here: undefined)."""
    given = k
    st, k, v = _torch.read(cache.calls, table, lens, starts, max_new, n_tokens, dtype, k, v,
                           _stream(stream))
    if stream is not None and given is None:
        _keep(stream, cache.pool.device, k, v)
    _check(st, "tkv_read")
    return k, v


def tkv_attend(cache: tkv_cache, q, table, lens, starts=None, max_new: Optional[int] = None,
               max_len: Optional[int] = None, scale: Optional[float] = None, causal: bool = True, scores=None,
               scores_out=None, out=None, lse=None, workspace=None, stream=None):
    """Attention of q [tokens, query heads, head_dim] over each sequence's lens[b] cached positions (the new tokens'
    own among them).  Returns out, like q, and lse, fp32 [tokens, query heads].

    max_len: a bound on lens (default: what the table holds); the split of the work goes by it, and positions past
    it are not seen.  scale: default 1 / sqrt(head_dim).  scores_out (fp32 [sequences, heads, positions]): written
    with scores (None: 0) plus each position's attention weight summed over the new tokens and the head's query
    heads; may be scores itself.  workspace: a uint8 tensor of at least tkv_attend_workspace bytes."""
    st, o, ls = _torch.attend(cache.calls, q, table, lens, starts, max_new, max_len, scale, causal, scores, scores_out,
                              out, lse, workspace, _stream(stream))
    if stream is not None:
        _keep(stream, cache.pool.device, o if out is None else None, ls if lse is None else None)
    _check(st, "tkv_attend")
    return o, ls


def tkv_attend_workspace(cache: tkv_cache, n_seq: int, q_heads: int, max_new: int, max_len: int,
                         scores: bool = False) -> int:
    """Bytes of workspace that are enough for every tkv_attend call with at most n_seq sequences, max_new new tokens
    of each and max_len positions (as given, or as what the table holds), with scores if asked for.  With scores of few
    rows, 4 bytes for each sequence, head, row and position of max_len are the most of it."""
    width = -(-max_len // cache.page_tokens)
    t = tkv_tokens(None, 0, 0, _DTYPES[torch.bfloat16])
    a = tkv_attend_args(t, t, None, None, 4 if scores else None, max_len, q_heads, max_len, 1.0, 0, None, 0)
    b = tkv_batch(4, width, 4, None, n_seq * max_new, n_seq, width, max_new)  # pointers are not read
    need = ctypes.c_uint64()
    _check(lib().tkv_attend_workspace_bound(ctypes.byref(cache), ctypes.byref(a), ctypes.byref(b), ctypes.byref(need)),
           "tkv_attend_workspace_bound")
    return need.value


def tkv_evict(cache: tkv_cache, table, lens, scores, budget: int, recent: int, dst_table, max_len: Optional[int] = None,
              kept=None, lens_out=None, scores_out=None, stream=None):
    """Shrink each sequence to `budget` positions a head: the last `recent` and, of the others, those of the largest
    scores (fp32 [sequences, heads, positions]), in their order, moved to the pages of dst_table, which the source
    table must not name.  Returns kept (int32 [sequences, heads, budget], -1 past the end), the new lens (lens_out,
    which may be lens) and the kept positions' scores (0 past the end)."""
    st, ke, le, sc = _torch.evict(cache.calls, table, lens, scores, budget, recent, dst_table, max_len, kept, lens_out,
                                  scores_out, _stream(stream))
    if stream is not None:
        _keep(stream, cache.pool.device, ke if kept is None else None, le if lens_out is None else None,
              sc if scores_out is None else None)
    _check(st, "tkv_evict")
    return ke, le, sc
