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
import struct
from typing import Optional

import torch

from .tmap import SUCCESS, TmapError

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtkv.so")

TILE = 32  # positions of a record
_DTYPES = {torch.float16: 3, torch.bfloat16: 4, torch.float32: 7}
_TWO = (torch.float16, torch.bfloat16)
_THREE = (torch.float16, torch.bfloat16, torch.float32)


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


# The same structures as bytes, which take a small call a few microseconds less to fill.
_TOKENS = struct.Struct("@Pqqi4x")
_BATCH = struct.Struct("@PqPPqiii4x")
_ATTEND = struct.Struct("@PPPqiifi")  # from lse on, before the workspace
_WORKSPACE = struct.Struct("@PQ")
_EVICT = struct.Struct("@PPqPPPqiiii")
assert (_TOKENS.size, _BATCH.size, _EVICT.size) == tuple(map(ctypes.sizeof, (tkv_tokens, tkv_batch, tkv_evict_args)))
assert 2 * _TOKENS.size + _ATTEND.size + _WORKSPACE.size == ctypes.sizeof(tkv_attend_args)


def _pack(form, what: str, *values) -> bytes:
    try:
        return form.pack(*values)
    except (struct.error, OverflowError) as err:
        raise ValueError(f"{what}: a number is out of range ({err})") from None


_lib = None


def lib():
    """Load libtkv.so (raises if it is missing)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run: python -m tiled_tensor_bulk_amd.build")
        L = ctypes.CDLL(LIB_PATH)
        # structures are given by reference, as an address or as bytes
        vp, u32 = ctypes.c_void_p, ctypes.c_uint32
        L.tkv_encode.argtypes = [vp, vp, ctypes.c_int64, u32, u32, u32, u32]
        L.tkv_encode.restype = ctypes.c_int
        L.tkv_page_bytes.argtypes = [vp]
        L.tkv_page_bytes.restype = ctypes.c_uint64
        for name in ("tkv_append", "tkv_read"):
            f = getattr(L, name)
            f.argtypes = [vp] * 5
            f.restype = ctypes.c_int
        L.tkv_attend.argtypes = [vp] * 4
        L.tkv_attend.restype = ctypes.c_int
        L.tkv_attend_workspace.argtypes = [vp] * 4
        L.tkv_attend_workspace.restype = ctypes.c_int
        L.tkv_evict.argtypes = [vp] * 4
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
        return torch._C._cuda_getCurrentRawStream(device.index)
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
    if device is None:
        if not t.is_cuda:
            raise ValueError(f"{what} must be a GPU tensor")
    elif t.device != device:
        if not t.is_cuda:
            raise ValueError(f"{what} must be a GPU tensor")
        raise ValueError(f"{what} is on {t.device}, the cache on {device}")
    return t


def _tokens(t, what: str, heads: Optional[int], dim: int, n_tokens: Optional[int], device, dtypes) -> bytes:
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{what} must be a tensor [tokens, heads, head_dim]")
    dtype = t.dtype
    if dtype not in dtypes:
        raise ValueError(f"{what} must be one of {', '.join(str(d).replace('torch.', '') for d in dtypes)}")
    _gpu(t, what, None, device)
    shape, stride = t.shape, t.stride()
    if shape[2] != dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{what} is {tuple(shape)}, the cache has {heads or 'n'} heads of {dim}")
    if n_tokens is not None and shape[0] != n_tokens:
        raise ValueError(f"{what} has {shape[0]} tokens, not {n_tokens}")
    if stride[2] != 1 and t.numel():
        raise ValueError(f"{what}'s last dimension must be contiguous")
    return _TOKENS.pack(t.data_ptr(), stride[0], stride[1], _DTYPES[dtype])


def _table(t, what: str, n_seq: int, device):
    """Address, stride and width of a table whose rows are contiguous."""
    _gpu(t, what, torch.int32, device)
    shape = t.shape
    if len(shape) != 2 or shape[0] != n_seq:
        raise ValueError(f"{what} must be [{n_seq}, pages]")
    stride, width = t.stride(), shape[1]
    if stride[1] != 1 and t.numel():
        raise ValueError(f"{what}'s rows must be contiguous")
    if n_seq < 2:
        return t.data_ptr(), width, width
    if stride[0] < width:
        raise ValueError(f"{what}'s rows must not overlap")
    return t.data_ptr(), stride[0], width


def _batch(cache, table, lens, starts, n_tokens: int, max_new: Optional[int]):
    """The structure, the number of sequences and the positions that a row of the table holds."""
    device = cache.pool.device
    if torch.cuda.current_device() != device.index:
        raise ValueError(f"the cache is on {device}, the current device is {torch.cuda.current_device()}")
    _gpu(lens, "lens", torch.int32, device)
    shape = lens.shape
    if len(shape) != 1 or (shape[0] > 1 and lens.stride(0) != 1):
        raise ValueError("lens must be a contiguous vector")
    n_seq = shape[0]
    ptr, stride, width = _table(table, "table", n_seq, device)
    if starts is not None:
        _gpu(starts, "starts", torch.int32, device)
        if starts.dim() != 1 or starts.shape[0] != n_seq + 1 or starts.stride(0) != 1:
            raise ValueError("starts must be a contiguous vector of sequences + 1")
        if max_new is None:
            max_new = n_tokens
        starts = starts.data_ptr()
    else:
        if n_seq and n_tokens % n_seq:
            raise ValueError(f"without starts, {n_tokens} tokens must be a multiple of {n_seq} sequences")
        if max_new is None:
            max_new = n_tokens // n_seq if n_seq else 0
        starts = 0
    b = _pack(_BATCH, "max_new", ptr, stride, lens.data_ptr(), starts, n_tokens, n_seq, width, int(max_new))
    return b, n_seq, width * cache.page_tokens


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
    c.at = ctypes.addressof(c)
    return c


def tkv_page_bytes(cache: tkv_cache) -> int:
    return int(lib().tkv_page_bytes(ctypes.byref(cache)))


def tkv_append(cache: tkv_cache, k, v, table, lens, starts=None, max_new: Optional[int] = None, stream=None) -> None:
    """Quantise k and v [tokens, heads, head_dim] (fp16 or bf16) and put them at positions lens[b] .. of each
    sequence's pages.  starts: int32 [sequences + 1] row offsets, None for equally many tokens each; max_new: a
    bound on a sequence's new tokens (default: what the shapes allow)."""
    device = cache.pool.device
    kt = _tokens(k, "k", cache.n_heads, cache.head_dim, None, device, _TWO)
    n = k.shape[0]
    vt = _tokens(v, "v", cache.n_heads, cache.head_dim, n, device, _TWO)
    b = _batch(cache, table, lens, starts, n, max_new)[0]
    _check(lib().tkv_append(cache.at, kt, vt, b, _stream(stream, device)), "tkv_append")


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
    kt = _tokens(k, "k", cache.n_heads, cache.head_dim, n_tokens, device, _THREE)
    n = k.shape[0]
    vt = _tokens(v, "v", cache.n_heads, cache.head_dim, n, device, _THREE)
    b = _batch(cache, table, lens, starts, n, max_new)[0]
    _check(lib().tkv_read(cache.at, kt, vt, b, _stream(stream, device, made)), "tkv_read")
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
    qt = _tokens(q, "q", None, cache.head_dim, None, device, _TWO)
    n, heads = q.shape[:2]
    made = []
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        made.append(out)
    if lse is None:
        lse = torch.empty((n, heads), dtype=torch.float32, device=device)
        made.append(lse)
    else:
        _gpu(lse, "lse", torch.float32, device)
        if lse.shape != (n, heads) or not lse.is_contiguous():
            raise ValueError(f"lse must be contiguous [{n}, {heads}]")
    ot = _tokens(out, "out", heads, cache.head_dim, n, device, (q.dtype,))
    b, n_seq, held = _batch(cache, table, lens, starts, n, max_new)
    max_len = held if max_len is None else min(int(max_len), held)
    stride = from_ = to = 0
    if scores_out is not None:
        _scores(scores_out, "scores_out", cache, n_seq, max_len)
        stride, to = scores_out.shape[2], scores_out.data_ptr()
        if scores is not None:
            _scores(scores, "scores", cache, n_seq, max_len)
            if scores.shape != scores_out.shape:
                raise ValueError("scores and scores_out must have one shape")
            from_ = scores.data_ptr()
    elif scores is not None:
        raise ValueError("scores are only read where scores_out is given")
    scale = 1.0 / math.sqrt(cache.head_dim) if scale is None else scale
    a = qt + ot + _pack(_ATTEND, "max_len or scale", lse.data_ptr(), from_, to, stride, heads, max_len, scale,
                        1 if causal else 0)
    need = _workspace(cache, a + bytes(16), b)
    where = size = 0
    if need:
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
            made.append(workspace)
        else:
            _gpu(workspace, "workspace", torch.uint8, device)
            if not workspace.is_contiguous():
                raise ValueError("workspace must be contiguous")
        where, size = workspace.data_ptr(), workspace.numel()
    _check(lib().tkv_attend(cache.at, a + _WORKSPACE.pack(where, size), b, _stream(stream, device, made)), "tkv_attend")
    return out, lse


def _workspace(cache, a: bytes, b: bytes) -> int:
    need = ctypes.c_uint64()
    _check(lib().tkv_attend_workspace(cache.at, a, b, ctypes.byref(need)), "tkv_attend_workspace")
    return need.value


def tkv_attend_workspace(cache: tkv_cache, n_seq: int, q_heads: int, max_new: int, max_len: int,
                         scores: bool = False) -> int:
    """Bytes of workspace for tkv_attend with at most max_new tokens a sequence and positions below max_len."""
    width = -(-max_len // cache.page_tokens)
    t = _TOKENS.pack(0, 0, 0, _DTYPES[torch.bfloat16])
    a = t + t + _pack(_ATTEND, "max_len", 0, 0, 4 if scores else 0, max_len, q_heads, max_len, 1.0, 0) + bytes(16)
    # pointers are not read
    b = _pack(_BATCH, "a size", 4, width, 4, 0, n_seq * max_new, n_seq, width, max_new)
    return _workspace(cache, a, b)


def tkv_evict(cache: tkv_cache, table, lens, scores, budget: int, recent: int, dst_table, max_len: Optional[int] = None,
              kept=None, lens_out=None, scores_out=None, stream=None):
    """Shrink each sequence to `budget` positions a head: the last `recent` and, of the others, those of the largest
    scores (fp32 [sequences, heads, positions]), in their order, moved to the pages of dst_table, which the source
    table must not name.  Returns kept (int32 [sequences, heads, budget], -1 past the end), the new lens and the
    kept positions' scores (0 past the end)."""
    device = cache.pool.device
    b, n_seq, held = _batch(cache, table, lens, None, 0, 0)
    max_len = held if max_len is None else min(int(max_len), held)
    _scores(scores, "scores", cache, n_seq, max_len)
    if budget < 0 or recent < 0:
        raise ValueError("budget and recent must not be negative")
    shape = (n_seq, cache.n_heads, budget)
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
    lens_out = output(lens_out, "lens_out", (n_seq,), torch.int32)
    scores_out = output(scores_out, "scores_out", shape, torch.float32)
    ptr, stride, width = _table(dst_table, "dst_table", n_seq, device)
    a = _pack(_EVICT, "budget or recent", scores.data_ptr(), scores_out.data_ptr(), scores.shape[2], kept.data_ptr(),
              lens_out.data_ptr(), ptr, stride, width, budget, recent, max_len)
    _check(lib().tkv_evict(cache.at, a, b, _stream(stream, device, made)), "tkv_evict")
    return kept, lens_out, scores_out
