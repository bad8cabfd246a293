"""The operators of the 8-bit cache run together, as examples/decode_window.py does: chunks of prompts, turned; a captured
step; a window whose pages are used again."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("args", [
    ["--batch", "2", "--heads", "2", "--prompt", "300", "--steps", "40", "--window", "100", "--chunk", "90"],
    ["--batch", "3", "--heads", "1", "--group-heads", "2", "--dim", "64", "--prompt", "70", "--steps", "9", "--window", "500",
     "--sinks", "0"]])
def test_the_windowed_decoding_example(args):
    path = os.path.join(ROOT, "examples", "decode_window.py")
    spec = importlib.util.spec_from_file_location("decode_window", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    first, worst = example.main(args)
    # Relative to a vector: a code is off by at most 2^-4 of its number and in the root mean square by some 2^-5.3, the
    # values' errors average as the values do, and the keys' make a logarithm of a few units uncertain by as much: 0.03 and
    # 0.03 of the output's norm. A page that is not there, or of another sequence, costs all of a position.
    assert first < 0.15 and worst < 0.2
