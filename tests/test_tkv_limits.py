"""What libtkv refuses beyond tests/test_tkv_boundary.py: overlaps, sizes that no
launch has, gradients.  Without a GPU, with pointers that nothing reads;
what is not refused stops at the device."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from tests.test_tkv_boundary import AT, attend_args, batch, encode, evict_args, refused, tokens  # noqa: E402
from tiled_tensor_bulk_amd import tkv as T  # noqa: E402
from tiled_tensor_bulk_amd.tmap import INVALID_VALUE, UNSUPPORTED_DEVICE  # noqa: E402

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="with a GPU what is accepted would run")


def evict(**kw):
    _, c = encode()
    b = {k: kw.pop(k) for k in list(kw) if k in dict(T.tkv_batch._fields_)}
    return T.lib().tkv_evict(ctypes.byref(c), ctypes.byref(evict_args(**kw)), ctypes.byref(batch(**b)), None)


@pytest.mark.parametrize("off", [-8, -4, 4, 8])
def test_evict_refuses_lengths_that_overlap(off):
    refused(evict(lens_out=AT + off, n_seq=3), "overlaps")


@no_gpu
@pytest.mark.parametrize("off", [-12, 0, 12])
def test_evict_takes_lengths_in_place_and_apart(off):
    assert evict(lens_out=AT + off, n_seq=3) == UNSUPPORTED_DEVICE


# ------------------------------------------------------------------ sizes

def moves(**kw):
    _, c = encode(heads=kw.pop("heads", 4), page=kw.pop("page", 64))
    k, b = tokens(), batch(**kw)
    return [f(ctypes.byref(c), ctypes.byref(k), ctypes.byref(k), ctypes.byref(b), None)
            for f in (T.lib().tkv_append, T.lib().tkv_read)]


def attend(heads=4, page=64, scored=False, **kw):
    _, c = encode(heads=heads, page=page)
    b = {k: kw.pop(k) for k in list(kw) if k in dict(T.tkv_batch._fields_)}
    if scored:
        kw.update(scores_out=AT, score_stride=kw["max_len"])
    return T.lib().tkv_attend(ctypes.byref(c), ctypes.byref(attend_args(**kw)), ctypes.byref(batch(**b)), None)


MANY = (1 << 31) - 1


@pytest.mark.parametrize("kw", [
    dict(n_tokens=MANY, max_new=MANY, n_seq=1, starts=AT, heads=32),            # the number of records passes 31 bits
    dict(n_tokens=MANY, max_new=MANY, n_seq=MANY, starts=AT, heads=65535),      # and their product 64
    dict(n_tokens=1 << 30, max_new=1 << 30, n_seq=1 << 25, starts=AT, heads=1 << 13),  # which comes out as 0 there
])
def test_moves_refuse_sizes_past_what_integers_hold(kw):
    for st in moves(**kw):
        refused(st, "too many")


def test_attend_and_evict_refuse_sizes_past_what_integers_hold():
    wide = dict(table_width=1 << 20, table_stride=1 << 20, page=1024)
    refused(attend(n_seq=1 << 26, n_tokens=0, heads=1 << 15, q_heads=1 << 15,
                   max_len=1 << 30, **wide), "too many")  # 2^64 steps
    refused(attend(n_seq=1 << 24, n_tokens=MANY, starts=AT, max_new=1 << 16, heads=1 << 13, q_heads=1 << 24, max_len=5),
            "too many")
    refused(evict(n_seq=1 << 27, budget=(1 << 31) - 32, score_stride=512), "too many")  # 2^55 records
    _, c = encode(heads=1 << 14)
    assert T.lib().tkv_evict(ctypes.byref(c), ctypes.byref(evict_args(budget=(1 << 31) - 32)),
                             ctypes.byref(batch(n_seq=1 << 30)), None) == INVALID_VALUE  # 2^70


def test_tables_that_hold_2_to_the_31_positions_are_refused():
    wide = dict(table_width=1 << 21, table_stride=1 << 21)
    for st in moves(page=1024, **wide) + [attend(page=1024, **wide)]:
        refused(st, "2^31")
    _, c = encode(page=1024)
    refused(T.lib().tkv_evict(ctypes.byref(c), ctypes.byref(evict_args()), ctypes.byref(batch(**wide)), None), "2^31")


@pytest.mark.parametrize("kw", [
    dict(n_tokens=1 << 29, max_new=1 << 29, n_seq=1, starts=AT),                 # two waves for each of 2^26 records
    dict(n_tokens=1 << 25, max_new=1, n_seq=1 << 24, starts=AT),                 # one for each of 2^26
])
def test_moves_refuse_more_threads_than_a_launch_has(kw):
    refused(moves(**kw)[1], "too many")
    if kw["max_new"] > 4:
        refused(moves(**kw)[0], "too many")


def test_evict_refuses_more_threads_than_a_launch_has():
    refused(evict(n_seq=1 << 20, budget=0), "too many")                  # 2^22 workgroups of 1024
    wide = dict(table_width=16, table_stride=16, max_len=1024, score_stride=1024)
    refused(evict(n_seq=1 << 19, budget=2000, **wide), "too many")       # four waves each for 2^26 records


@no_gpu
def test_what_a_launch_has_is_taken():
    st = moves(n_tokens=1 << 25, max_new=1, n_seq=(1 << 23) - 1, starts=AT)  # 2^25 records less 4
    assert st == [UNSUPPORTED_DEVICE] * 2
    assert evict(n_seq=(1 << 20) - 1, budget=0) == UNSUPPORTED_DEVICE


# ------------------------------------------------------------------ rows that are written over one another

@pytest.mark.parametrize("kw", [dict(ts=0), dict(hs=0), dict(ts=127), dict(hs=64)])
def test_written_rows_that_overlap_are_refused(kw):
    _, c = encode()
    r = ctypes.byref
    refused(T.lib().tkv_read(r(c), r(tokens(**kw)), r(tokens()), r(batch()), None), "k's rows overlap")
    refused(T.lib().tkv_read(r(c), r(tokens()), r(tokens(**kw)), r(batch()), None), "v's rows overlap")
    refused(attend(out=tokens(**kw)), "out's rows overlap")


@no_gpu
def test_rows_that_are_read_may_be_one():
    _, c = encode()
    one, r = tokens(ts=0, hs=0), ctypes.byref
    assert T.lib().tkv_append(r(c), r(one), r(one), r(batch()), None) == UNSUPPORTED_DEVICE
    assert attend(q=one) == UNSUPPORTED_DEVICE
    alone = batch(n_seq=1, n_tokens=1, max_new=1)  # the stride of a single row is not looked at
    assert T.lib().tkv_read(r(c), r(tokens(ts=0)), r(tokens(ts=0)), r(alone), None) == UNSUPPORTED_DEVICE


# ------------------------------------------------------------------ gradients

def test_a_gradient_that_would_be_lost_is_refused():
    st, c = encode()
    calls = T._calls()
    cache = calls.Cache(ctypes.addressof(c), torch.zeros(16, dtype=torch.uint8), 4, 128, 64)
    ints = torch.zeros((1, 1), dtype=torch.int32)
    k = torch.zeros((1, 4, 128), dtype=torch.bfloat16)
    asks = k.clone().requires_grad_()
    for x, word in ((k, "GPU"), (asks, "requires a gradient"), (asks * 2, "requires a gradient")):
        with pytest.raises(ValueError, match=word):
            calls.append(cache, x, x, ints, ints[0], None, None, None)
        with pytest.raises(ValueError, match=word):
            calls.attend(cache, x, ints, ints[0], None, None, None, None, True, None, None, None, None, None, None)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):  # on to the next check
        calls.append(cache, asks, asks, ints, ints[0], None, None, None)
