"""What libtkv refuses of the 8-bit cache, of rotations and of windows.  Without a GPU, with pointers that nothing reads;
what is not refused stops at the device."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from tests.test_tkv_boundary import AT, F16, attend_args, batch, encode, evict_args, refused, tokens  # noqa: E402
from tiled_tensor_bulk_amd import tkv as T  # noqa: E402
from tiled_tensor_bulk_amd.tmap import INVALID_VALUE, SUCCESS, UNSUPPORTED_DEVICE  # noqa: E402

r = ctypes.byref
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="with a GPU what is accepted would run")


def encode8(pool=AT, pages=4, heads=4, dim=128, page=64):
    c = T.tkv_cache()
    return T.lib().tkv_encode8(r(c), pool, pages, heads, dim, page), c


def test_encode8():
    assert encode8()[0] == SUCCESS
    for kw in (dict(dim=32), dict(dim=160), dict(page=16), dict(page=2048), dict(page=48), dict(heads=0), dict(heads=65536),
               dict(pages=0), dict(pages=1 << 31), dict(pool=None), dict(pool=AT + 4)):
        st, c = encode8(**kw)
        assert st != SUCCESS, kw
        assert T.lib().tkv_append(r(c), r(tokens()), r(tokens()), r(batch()), None) != SUCCESS, kw  # never encoded
    assert T.lib().tkv_encode8(None, AT, 4, 4, 128, 64) != SUCCESS


def test_bytes_of_a_page():
    assert T.tkv_page_bytes_of(3, 128, 64, bits=8) == 3 * 2 * (64 * 128 + 128)
    for bits in (0, 2, 16):
        with pytest.raises(Exception):
            T.tkv_page_bytes_of(3, 128, 64, bits=bits)


def rotation(table=AT, stride=128, positions=None, n=100, dim=128, neighbours=0, q=None, q_out=None, heads=0):
    x = T.tkv_rotation()
    x.cos_sin, x.stride, x.positions, x.n_positions, x.rot_dim, x.neighbours = table, stride, positions, n, dim, neighbours
    if q is not None:
        x.q, x.q_out, x.q_heads = q, q if q_out is None else q_out, heads
    return x


def rotated(rot, c=None, **kw):
    c = encode8()[1] if c is None else c
    return T.lib().tkv_append_rotated(r(c), r(tokens()), r(tokens()), r(rot) if rot is not None else None, r(batch(**kw)), None)


@pytest.mark.parametrize("kw", [
    dict(dim=8), dict(dim=24), dict(dim=144), dict(dim=0), dict(dim=-16), dict(n=-1), dict(n=1 << 31), dict(stride=127),
    dict(stride=-128), dict(table=None), dict(table=AT + 2), dict(positions=AT + 2), dict(neighbours=2)])
def test_rotations_that_are_refused(kw):
    word = {"dim": "rot_dim", "n": "n_positions", "stride": "stride", "table": "cos_sin"}.get(*kw, *kw)
    refused(rotated(rotation(**kw)), word)


def test_no_rotation_is_refused():
    refused(rotated(None), "rotation is NULL")


def test_queries_that_are_refused():
    big = tokens(data=AT + (1 << 24))
    for q, out, heads, word in ((tokens(), big, -1, "q_heads"), (tokens(data=None), big, 8, "q's"), (tokens(), tokens(data=None), 8, "q_out"),
                                (tokens(), tokens(data=AT + (1 << 24), hs=64), 8, "q_out's rows overlap"),
                                (tokens(), tokens(data=AT + (1 << 24), dtype=F16), 8, "one type"),
                                (tokens(), tokens(ts=4096, hs=256), 8, "other strides")):
        assert rotated(rotation(q=q, q_out=out, heads=heads)) == INVALID_VALUE, word
        assert word.split("'")[0] in T.tkv_last_error_detail(), (word, T.tkv_last_error_detail())


@no_gpu
def test_rotations_that_are_taken():
    for kw in (dict(), dict(dim=16), dict(neighbours=1, dim=64), dict(n=0, table=None), dict(positions=AT), dict(table=AT + 4)):
        assert rotated(rotation(**kw)) == UNSUPPORTED_DEVICE, (kw, T.lib().tkv_last_error_detail())
    assert rotated(rotation(q=tokens(), heads=4)) == UNSUPPORTED_DEVICE
    assert rotated(rotation(dim=64), c=encode()[1]) == UNSUPPORTED_DEVICE  # 4 bits


def window(w, s=0):
    x = T.tkv_window()
    x.window, x.sinks = w, s
    return x


def attend(c=None, w=None, size=False, **kw):
    c = encode8()[1] if c is None else c
    b = {k: kw.pop(k) for k in list(kw) if k in dict(T.tkv_batch._fields_)}
    a, bt = attend_args(**kw), batch(**b)
    wp = r(w) if w is not None else None
    if size:
        n = ctypes.c_uint64()
        return T.lib().tkv_attend_window_workspace(r(c), r(a), wp, r(bt), r(n)), n.value
    return T.lib().tkv_attend_window(r(c), r(a), wp, r(bt), None)


@pytest.mark.parametrize("w,s", [(0, 0), (-1, 0), (5, -1), (0, 4)])
def test_windows_that_are_refused(w, s):
    for c in (encode8()[1], encode()[1]):
        word = "window" if w < 1 else "sinks"
        refused(attend(c, window(w, s)), word)
        refused(attend(c, window(w, s), size=True)[0], word)


def test_scores_and_eviction_are_of_the_4_bit_cache():
    scored = dict(scores_out=AT, score_stride=4096, max_len=128)
    refused(attend(**scored), "in 4 bits")
    refused(attend(encode()[1], window(100, 4), **scored), "not kept with a window")
    _, c = encode8()
    refused(T.lib().tkv_evict(r(c), r(evict_args()), r(batch()), None), "4 bits")


@no_gpu
def test_windows_that_are_taken():
    top = (1 << 31) - 1
    for c in (encode8()[1], encode()[1]):
        for w in (window(1), window(top, top), window(4096, 4), None):
            assert attend(c, w) == UNSUPPORTED_DEVICE, T.lib().tkv_last_error_detail()


# ------------------------------------------------------------------ sizes

def append8(**kw):
    _, c = encode8(heads=kw.pop("heads", 4))
    return [f(r(c), r(tokens()), r(tokens()), r(batch(**kw)), None) for f in (T.lib().tkv_append, T.lib().tkv_read)]


def test_more_threads_than_a_launch_has_are_refused():
    """one new token: two waves for each of 2^26 records, with 4 bits one in append"""
    for st in append8(n_tokens=1 << 24, max_new=1, n_seq=1 << 23, starts=AT):
        refused(st, "too many")


@no_gpu
def test_what_a_launch_has_is_taken():
    assert append8(n_tokens=1 << 24, max_new=1, n_seq=(1 << 22) - 1, starts=AT) == [UNSUPPORTED_DEVICE] * 2
