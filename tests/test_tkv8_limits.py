"""Sizes that a rotation's queries may have (CPU only, with pointers that nothing reads)."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_tkv8_boundary import refused, rotated, rotation  # noqa: E402
from tests.test_tkv_boundary import encode, tokens  # noqa: E402
from tiled_tensor_bulk_amd.tmap import UNSUPPORTED_DEVICE  # noqa: E402

TOP = 1 << 30


@pytest.mark.parametrize("heads", [TOP + 1, (1 << 31) - 1024, (1 << 31) - 64, (1 << 31) - 1])
def test_heads_whose_count_would_pass_31_bits_are_refused(heads):
    """a wave goes on by up to 64 * 16 heads from one that is there"""
    refused(rotated(rotation(q=tokens(), heads=heads)), "q_heads")
    refused(rotated(rotation(q=tokens(), heads=heads), c=encode()[1]), "q_heads")


@pytest.mark.skipif(torch.cuda.is_available(), reason="with a GPU what is accepted would run")
def test_heads_that_are_taken():
    for heads in (1, 300, TOP):
        assert rotated(rotation(q=tokens(), heads=heads)) == UNSUPPORTED_DEVICE, heads
