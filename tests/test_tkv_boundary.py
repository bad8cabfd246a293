"""libtkv's C ABI without a GPU: the descriptor, sizes, and every refusal, made with pointers that nothing reads."""
import ctypes
import itertools

import pytest

torch = pytest.importorskip("torch")

from tiled_tensor_bulk_amd import tkv as T  # noqa: E402
from tiled_tensor_bulk_amd.tmap import INVALID_VALUE, SUCCESS, UNSUPPORTED_DEVICE, TmapError  # noqa: E402

AT = 1 << 20  # an address that is never read
F16, BF16, F32 = 3, 4, 7


def encode(pool=AT, n_pages=10, heads=4, dim=128, page=64, group=64):
    c = T.tkv_cache()
    return T.lib().tkv_encode(ctypes.byref(c), pool, n_pages, heads, dim, page, group), c


def tokens(data=AT, ts=512, hs=128, dtype=BF16):
    return T.tkv_tokens(data, ts, hs, dtype)


def batch(**kw):
    d = dict(table=AT, table_stride=8, lens=AT, starts=None, n_tokens=6, n_seq=3, table_width=8, max_new=2)
    d.update(kw)
    return T.tkv_batch(*(d[f] for f, _ in T.tkv_batch._fields_))


def attend_args(**kw):
    d = dict(q=tokens(), out=tokens(), lse=AT, scores_in=None, scores_out=None, score_stride=0, q_heads=8, max_len=300,
             scale=0.1, causal=1, workspace=AT, workspace_bytes=1 << 40)
    d.update(kw)
    return T.tkv_attend_args(*(d[f] for f, _ in T.tkv_attend_args._fields_))


def evict_args(**kw):
    d = dict(scores=AT, scores_out=AT, score_stride=512, kept=AT, lens_out=AT, dst_table=AT, dst_stride=4, dst_width=4,
             budget=100, recent=10, max_len=512)
    d.update(kw)
    return T.tkv_evict_args(*(d[f] for f, _ in T.tkv_evict_args._fields_))


def refused(st, word):
    assert st == INVALID_VALUE, st
    assert word in T.tkv_last_error_detail(), T.tkv_last_error_detail()


def test_encode_and_page_bytes():
    for dim, group, page, heads in itertools.product((64, 96, 128, 256), (32, 64, 128), (32, 64, 1024), (1, 5)):
        st, c = encode(heads=heads, dim=dim, page=page, group=group)
        if dim % group:
            refused(st, "group")
            continue
        assert st == SUCCESS and T.tkv_last_error_detail() == ""
        want = heads * page // 32 * (2 * 16 * dim + 2 * 32 * (dim // group) * 4)
        assert T.tkv_page_bytes(c) == want == T.tkv_page_bytes_of(heads, dim, page, group)
    assert T.lib().tkv_page_bytes(ctypes.byref(T.tkv_cache())) == 0
    assert T.lib().tkv_page_bytes(None) == 0


@pytest.mark.parametrize("kw,word", [
    (dict(pool=None), "pool"), (dict(pool=AT + 8), "pool"), (dict(n_pages=0), "n_pages"),
    (dict(n_pages=1 << 31), "n_pages"), (dict(heads=0), "n_heads"), (dict(heads=65536), "n_heads"),
    (dict(dim=80), "head_dim"), (dict(dim=0), "head_dim"), (dict(page=16), "page_tokens"), (dict(page=48), "page_tokens"),
    (dict(page=2048), "page_tokens"), (dict(group=16), "group"), (dict(group=0), "group"), (dict(dim=96, group=64), "group"),
])
def test_encode_refuses(kw, word):
    refused(encode(**kw)[0], word)
    refused(T.lib().tkv_encode(None, AT, 1, 1, 128, 64, 64), "cache")


BATCH_REFUSALS = [
    (dict(n_seq=-1), "n_seq"), (dict(table_width=9), "table_width"), (dict(table_width=-1), "table_width"),
    (dict(lens=None), "lens"), (dict(lens=AT + 2), "lens"), (dict(table=None), "table"), (dict(table=AT + 1), "table"),
]
TOKEN_REFUSALS = [
    (dict(n_tokens=-1), "n_tokens"), (dict(n_tokens=1 << 31), "n_tokens"), (dict(max_new=-1), "max_new"),
    (dict(starts=AT + 2), "starts"), (dict(n_tokens=7), "multiple"),
]


@pytest.mark.parametrize("name", ["tkv_append", "tkv_read"])
def test_moves_refuse(name):
    f, (_, c) = getattr(T.lib(), name), encode()
    k, v = tokens(), tokens()

    def call(cache=c, k=k, v=v, b=batch()):
        ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
        return f(ref(cache), ref(k), ref(v), ref(b), None)

    for kw, word in BATCH_REFUSALS + TOKEN_REFUSALS:
        refused(call(b=batch(**kw)), word)
    refused(call(cache=T.tkv_cache()), "cache")
    refused(call(cache=None), "cache")
    refused(call(k=None), "k or v")
    refused(call(b=None), "batch")
    refused(call(k=tokens(data=None)), "k is")
    refused(call(v=tokens(data=AT + 1)), "v is")
    refused(call(k=tokens(dtype=5)), "k must")
    refused(call(v=tokens(dtype=F16)), "one type")
    refused(call(k=tokens(ts=-1)), "stride")
    both = dict(k=tokens(dtype=F32), v=tokens(dtype=F32))
    if name == "tkv_append":
        refused(call(**both), "fp16 or bf16")
    elif not torch.cuda.is_available():
        assert call(**both) == UNSUPPORTED_DEVICE
    refused(call(b=batch(n_seq=1 << 30, n_tokens=1 << 30, max_new=1)), "too many")


def test_attend_refuses():
    _, c = encode()

    def call(a=attend_args(), b=batch(), cache=c):
        return T.lib().tkv_attend(ctypes.byref(cache), ctypes.byref(a), ctypes.byref(b), None)

    for kw, word in BATCH_REFUSALS + TOKEN_REFUSALS:
        refused(call(b=batch(**kw)), word)
    for kw, word in [
        (dict(q=tokens(dtype=F32)), "q must"), (dict(out=tokens(dtype=F16)), "one type"), (dict(q=tokens(data=None)), "q is"),
        (dict(lse=None), "lse"), (dict(lse=AT + 2), "lse"), (dict(q_heads=6), "q_heads"), (dict(q_heads=0), "q_heads"),
        (dict(q_heads=-4), "q_heads"), (dict(max_len=-1), "max_len"), (dict(scale=float("nan")), "scale"),
        (dict(scale=float("inf")), "scale"), (dict(causal=2), "causal"), (dict(scores_in=AT), "scores_out"),
        (dict(scores_out=AT, score_stride=299), "score_stride"), (dict(scores_out=AT + 2, score_stride=300), "scores"),
    ]:
        refused(call(a=attend_args(**kw)), word)
    refused(call(cache=T.tkv_cache()), "cache")
    refused(T.lib().tkv_attend(ctypes.byref(c), None, ctypes.byref(batch()), None), "args")
    refused(T.lib().tkv_attend_workspace(ctypes.byref(c), ctypes.byref(attend_args()), ctypes.byref(batch()), None), "bytes")
    refused(call(a=attend_args(q_heads=1 << 30), b=batch(n_tokens=6, max_new=6)), "too many")


def test_evict_refuses():
    _, c = encode()

    def call(a=evict_args(), b=batch(), cache=c):
        return T.lib().tkv_evict(ctypes.byref(cache), ctypes.byref(a), ctypes.byref(b), None)

    for kw, word in BATCH_REFUSALS:
        refused(call(b=batch(**kw)), word)
    for kw, word in [
        (dict(budget=-1), "budget"), (dict(recent=-1), "recent"), (dict(max_len=513), "score_stride"),
        (dict(max_len=-1), "score_stride"), (dict(dst_width=5), "dst_width"), (dict(dst_width=-1), "dst_width"),
        (dict(lens_out=None), "lens_out"), (dict(kept=None), "kept"), (dict(scores_out=None), "scores_out"),
        (dict(scores=None), "scores"), (dict(scores=AT + 2), "scores"), (dict(dst_table=None), "dst_table"),
    ]:
        refused(call(a=evict_args(**kw)), word)
    refused(call(cache=T.tkv_cache()), "cache")
    refused(call(a=evict_args(budget=1 << 30), b=batch(n_seq=1000)), "too many")


@pytest.mark.skipif(torch.cuda.is_available(), reason="with a GPU these would run")
def test_without_a_gpu_every_call_says_so():
    _, c = encode()
    k = tokens()
    r = ctypes.byref
    assert T.lib().tkv_append(r(c), r(k), r(k), r(batch()), None) == UNSUPPORTED_DEVICE
    assert T.lib().tkv_read(r(c), r(k), r(k), r(batch()), None) == UNSUPPORTED_DEVICE
    assert T.lib().tkv_attend(r(c), r(attend_args()), r(batch()), None) == UNSUPPORTED_DEVICE
    assert T.lib().tkv_evict(r(c), r(evict_args()), r(batch()), None) == UNSUPPORTED_DEVICE


def test_the_wrapper_refuses_what_is_not_on_the_gpu():
    with pytest.raises(ValueError, match="GPU"):
        T.tkv_encode(torch.zeros(4608, dtype=torch.uint8), 1, 128, 32, 64)
    with pytest.raises(ValueError, match="uint8"):
        T.tkv_encode(torch.zeros(4608), 1, 128, 32, 64)
    err = None
    try:
        T._check(encode(dim=80)[0], "tkv_encode")
    except TmapError as e:
        err = e
    assert err is not None and err.status == INVALID_VALUE and "head_dim" in str(err)
