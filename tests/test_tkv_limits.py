"""What libtkv refuses beyond tests/test_tkv_boundary.py: overlaps.  Without a GPU, with pointers that nothing reads;
what is not refused stops at the device."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from tests.test_tkv_boundary import AT, batch, encode, evict_args, refused  # noqa: E402
from tiled_tensor_bulk_amd import tkv as T  # noqa: E402
from tiled_tensor_bulk_amd.tmap import UNSUPPORTED_DEVICE  # noqa: E402

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
