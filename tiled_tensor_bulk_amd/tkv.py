"""Python binding of libtkv (ctypes): a paged key/value cache in 4 bits and
the operators on it (include/tkv.h).  Argument checks and marshalling only;
raises if libtkv.so has not been built -- there is no fallback.

Names match the C ABI.  Tensors lie on the current GPU; work goes to `stream`
(an int, a torch stream, or None: torch's current one).  Outputs and the
workspace are allocated with torch where they are not given.

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
        L.tkv_attend_workspace.argtypes = [P(tkv_cache), P(tkv_attend_args), P(tkv_batch), P(ctypes.c_uint64)]
        L.tkv_attend_workspace.restype = ctypes.c_int
        L.tkv_evict.argtypes = [P(tkv_cache), P(tkv_evict_args), P(tkv_batch), vp]
        L.tkv_evict.restype = ctypes.c_int
        L.tkv_last_error_detail.argtypes = []
        L.tkv_last_error_detail.restype = ctypes.c_char_p
        _lib = L
    return _lib


def tkv_last_error_detail() -> str:
    return lib().tkv_last_error_detail().decode()


def _check(st: int, where: str) -> None:
    if st != SUCCESS:
        raise TmapError(st, where, tkv_last_error_detail())


def _stream(s, device, made=()):
    """The stream's handle; tensors made here are kept for it."""
    if s is None:
        return torch.cuda.current_stream(device).cuda_stream
    if isinstance(s, int):
        on = torch.cuda.ExternalStream(s, device=device) if s else torch.cuda.default_stream(device)
    else:
        on = s
    if on != torch.cuda.current_stream(device):
        for t in made:
            t.record_stream(on)
    return on.cuda_stream


def _gpu(t, what: str, dtype, device=None):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{what} must be a tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} must be {str(dtype).replace('torch.', '')}, not {str(t.dtype).replace('torch.', '')}")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{what} is on {t.device}, the cache on {device}")
    return t


def _tokens(t, what: str, heads: Optional[int], dim: int, n_tokens: Optional[int], device, dtypes):
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{what} must be a tensor [tokens, heads, head_dim]")
    if t.dtype not in dtypes:
        raise ValueError(f"{what} must be one of {', '.join(str(d).replace('torch.', '') for d in dtypes)}")
    _gpu(t, what, None, device)
    if t.shape[2] != dim or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{what} is {tuple(t.shape)}, the cache has {heads or 'n'} heads of {dim}")
    if n_tokens is not None and t.shape[0] != n_tokens:
        raise ValueError(f"{what} has {t.shape[0]} tokens, not {n_tokens}")
    if t.numel() and t.stride(2) != 1:
        raise ValueError(f"{what}'s last dimension must be contiguous")
    return tkv_tokens(t.data_ptr(), t.stride(0), t.stride(1), _DTYPES[t.dtype])


def _table(t, what: str, n_seq: Optional[int], device):
    _gpu(t, what, torch.int32, device)
    if t.dim() != 2 or (n_seq is not None and t.shape[0] != n_seq):
        raise ValueError(f"{what} must be [{'sequences' if n_seq is None else n_seq}, pages]")
    if t.numel() and t.stride(1) != 1:
        raise ValueError(f"{what}'s rows must be contiguous")
    return t.data_ptr(), max(t.stride(0), t.shape[1]) if t.shape[0] > 1 else t.shape[1], t.shape[1]


def _batch(cache, table, lens, starts, n_tokens: int, max_new: Optional[int]):
    device = cache.pool.device
    if torch.cuda.current_device() != device.index:
        raise ValueError(f"the cache is on {device}, the current device is {torch.cuda.current_device()}")
    _gpu(lens, "lens", torch.int32, device)
    if lens.dim() != 1 or (lens.numel() > 1 and lens.stride(0) != 1):
        raise ValueError("lens must be a contiguous vector")
    n_seq = lens.shape[0]
    if isinstance(table, torch.Tensor) and table.dim() == 2 and table.shape[0] > 1 and table.stride(0) < table.shape[1]:
        raise ValueError("table's rows must not overlap")
    ptr, stride, width = _table(table, "table", n_seq, device)
    if starts is not None:
        _gpu(starts, "starts", torch.int32, device)
        if starts.dim() != 1 or starts.shape[0] != n_seq + 1 or starts.stride(0) != 1:
            raise ValueError("starts must be a contiguous vector of sequences + 1")
        if max_new is None:
            max_new = n_tokens
    else:
        if n_seq and n_tokens % n_seq:
            raise ValueError(f"without starts, {n_tokens} tokens must be a multiple of {n_seq} sequences")
        if max_new is None:
            max_new = n_tokens // n_seq if n_seq else 0
    return tkv_batch(ptr, stride, lens.data_ptr(), None if starts is None else starts.data_ptr(), n_tokens, n_seq,
                     width, int(max_new))


def tkv_page_bytes_of(n_heads: int, head_dim: int, page_tokens: int, group: int) -> int:
    """Bytes of one page, before there is a pool."""
    return n_heads * (page_tokens // TILE) * (32 * head_dim + 256 * (head_dim // group))


def tkv_encode(pool, n_heads: int, head_dim: int, page_tokens: int, group: int = 64) -> tkv_cache:
    """Describe a pool: a contiguous uint8 GPU tensor of whole pages."""
    _gpu(pool, "pool", torch.uint8)
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
    return c


def tkv_page_bytes(cache: tkv_cache) -> int:
    return int(lib().tkv_page_bytes(ctypes.byref(cache)))


def tkv_append(cache: tkv_cache, k, v, table, lens, starts=None, max_new: Optional[int] = None, stream=None) -> None:
    """Quantise k and v [tokens, heads, head_dim] (fp16 or bf16) and put them at positions lens[b] .. of each
    sequence's pages.  starts: int32 [sequences + 1] row offsets, None for equally many tokens each; max_new: a
    bound on a sequence's new tokens (default: what the shapes allow)."""
    device, n = cache.pool.device, k.shape[0]
    two = (torch.float16, torch.bfloat16)
    kt = _tokens(k, "k", cache.n_heads, cache.head_dim, None, device, two)
    vt = _tokens(v, "v", cache.n_heads, cache.head_dim, n, device, two)
    b = _batch(cache, table, lens, starts, n, max_new)
    _check(lib().tkv_append(ctypes.byref(cache), ctypes.byref(kt), ctypes.byref(vt), ctypes.byref(b),
                            _stream(stream, device)), "tkv_append")


def tkv_read(cache: tkv_cache, table, lens, starts=None, max_new: Optional[int] = None, n_tokens: Optional[int] = None,
             dtype=torch.float16, k=None, v=None, stream=None):
    """Keys and values at positions lens[b] .. of each sequence as numbers, [n_tokens, heads, head_dim] in dtype
    (fp16, bf16, fp32); arguments as for tkv_append.  Rows that no sequence's range names are left as they were
    (in tensors made here: undefined)."""
    device = cache.pool.device
    made = []
    if (k is None) != (v is None):
        raise ValueError("give both k and v, or neither")
    if k is None:
        if n_tokens is None:
            raise ValueError("n_tokens is needed where k and v are not given")
        shape = (n_tokens, cache.n_heads, cache.head_dim)
        k, v = (torch.empty(shape, dtype=dtype, device=device) for _ in range(2))
        made = [k, v]
    n = k.shape[0]
    three = (torch.float16, torch.bfloat16, torch.float32)
    kt = _tokens(k, "k", cache.n_heads, cache.head_dim, n_tokens, device, three)
    vt = _tokens(v, "v", cache.n_heads, cache.head_dim, n, device, three)
    b = _batch(cache, table, lens, starts, n, max_new)
    _check(lib().tkv_read(ctypes.byref(cache), ctypes.byref(kt), ctypes.byref(vt), ctypes.byref(b),
                          _stream(stream, device, made)), "tkv_read")
    return k, v


def _scores(t, what: str, cache, n_seq: int, max_len: int):
    _gpu(t, what, torch.float32, cache.pool.device)
    if t.dim() != 3 or t.shape[:2] != (n_seq, cache.n_heads) or t.shape[2] < max_len or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous [{n_seq}, {cache.n_heads}, at least {max_len}], "
                         f"not {tuple(t.shape)}")


def tkv_attend(cache: tkv_cache, q, table, lens, starts=None, max_new: Optional[int] = None,
               max_len: Optional[int] = None, scale: Optional[float] = None, causal: bool = True, scores=None,
               scores_out=None, out=None, lse=None, workspace=None, stream=None):
    """Attention of q [tokens, query heads, head_dim] over each sequence's lens[b] cached positions (the new tokens'
    own among them).  Returns out, like q, and lse, fp32 [tokens, query heads].

    max_len: a bound on lens (default: what the table holds); the split of the work goes by it, and positions past
    it are not seen.  scale: default 1 / sqrt(head_dim).  scores_out (fp32 [sequences, heads, positions]): written
    with scores (None: 0) plus each position's attention weight summed over the new tokens and the head's query
    heads; may be scores itself.  workspace: a uint8 tensor of at least tkv_attend_workspace bytes."""
    device = cache.pool.device
    two = (torch.float16, torch.bfloat16)
    qt = _tokens(q, "q", None, cache.head_dim, None, device, two)
    n, heads = q.shape[:2]
    made = []
    if out is None:
        out = torch.empty((n, heads, cache.head_dim), dtype=q.dtype, device=device)
        made.append(out)
    if lse is None:
        lse = torch.empty((n, heads), dtype=torch.float32, device=device)
        made.append(lse)
    ot = _tokens(out, "out", heads, cache.head_dim, n, device, (q.dtype,))
    _gpu(lse, "lse", torch.float32, device)
    if lse.shape != (n, heads) or not lse.is_contiguous():
        raise ValueError(f"lse must be contiguous [{n}, {heads}]")
    b = _batch(cache, table, lens, starts, n, max_new)
    held = b.table_width * cache.page_tokens
    max_len = held if max_len is None else min(int(max_len), held)
    if scores is not None and scores_out is None:
        raise ValueError("scores are only read where scores_out is given")
    stride = 0
    if scores_out is not None:
        _scores(scores_out, "scores_out", cache, b.n_seq, max_len)
        stride = scores_out.shape[2]
        if scores is not None:
            _scores(scores, "scores", cache, b.n_seq, max_len)
            if scores.shape != scores_out.shape:
                raise ValueError("scores and scores_out must have one shape")
    a = tkv_attend_args(qt, ot, lse.data_ptr(), None if scores is None else scores.data_ptr(),
                        None if scores_out is None else scores_out.data_ptr(), stride, heads, max_len,
                        1.0 / math.sqrt(cache.head_dim) if scale is None else scale, 1 if causal else 0, None, 0)
    need = _workspace(cache, a, b)
    if need:
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
            made.append(workspace)
        else:
            _gpu(workspace, "workspace", torch.uint8, device)
            if not workspace.is_contiguous():
                raise ValueError("workspace must be contiguous")
        a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
    _check(lib().tkv_attend(ctypes.byref(cache), ctypes.byref(a), ctypes.byref(b), _stream(stream, device, made)),
           "tkv_attend")
    return out, lse


def _workspace(cache, a, b) -> int:
    need = ctypes.c_uint64()
    _check(lib().tkv_attend_workspace(ctypes.byref(cache), ctypes.byref(a), ctypes.byref(b), ctypes.byref(need)),
           "tkv_attend_workspace")
    return need.value


def tkv_attend_workspace(cache: tkv_cache, n_seq: int, q_heads: int, max_new: int, max_len: int,
                         scores: bool = False) -> int:
    """Bytes of workspace for tkv_attend with at most max_new tokens a sequence and positions below max_len."""
    width = -(-max_len // cache.page_tokens)
    t = tkv_tokens(None, 0, 0, _DTYPES[torch.bfloat16])
    a = tkv_attend_args(t, t, None, None, 4 if scores else None, max_len, q_heads, max_len, 1.0, 0, None, 0)
    b = tkv_batch(4, width, 4, None, n_seq * max_new, n_seq, width, max_new)  # pointers are not read
    return _workspace(cache, a, b)


def tkv_evict(cache: tkv_cache, table, lens, scores, budget: int, recent: int, dst_table, max_len: Optional[int] = None,
              kept=None, lens_out=None, scores_out=None, stream=None):
    """Shrink each sequence to `budget` positions a head: the last `recent` and, of the others, those of the largest
    scores (fp32 [sequences, heads, positions]), in their order, moved to the pages of dst_table, which the source
    table must not name.  Returns kept (int32 [sequences, heads, budget], -1 past the end), the new lens and the
    kept positions' scores (0 past the end)."""
    device = cache.pool.device
    b = _batch(cache, table, lens, None, 0, 0)
    held = b.table_width * cache.page_tokens
    _gpu(scores, "scores", torch.float32, device)
    max_len = held if max_len is None else min(int(max_len), held)
    _scores(scores, "scores", cache, b.n_seq, max_len)
    if budget < 0 or recent < 0:
        raise ValueError("budget and recent must not be negative")
    shape = (b.n_seq, cache.n_heads, budget)
    made = []

    def output(t, what, shape, dtype):
        if t is None:
            t = torch.empty(shape, dtype=dtype, device=device)
            made.append(t)
        else:
            _gpu(t, what, dtype, device)
            if t.shape != shape or not t.is_contiguous():
                raise ValueError(f"{what} must be contiguous {list(shape)}")
        return t

    kept = output(kept, "kept", shape, torch.int32)
    lens_out = output(lens_out, "lens_out", (b.n_seq,), torch.int32)
    scores_out = output(scores_out, "scores_out", shape, torch.float32)
    ptr, stride, width = _table(dst_table, "dst_table", b.n_seq, device)
    a = tkv_evict_args(scores.data_ptr(), scores_out.data_ptr(), scores.shape[2], kept.data_ptr(), lens_out.data_ptr(),
                       ptr, stride, width, budget, recent, max_len)
    _check(lib().tkv_evict(ctypes.byref(cache), ctypes.byref(a), ctypes.byref(b), _stream(stream, device, made)),
           "tkv_evict")
    return kept, lens_out, scores_out
