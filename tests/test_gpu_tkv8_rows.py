"""Attention over the 8-bit cache with 17 to 64 rows of a head, which go in tiles of 16 or 32: in chunks, and in tables so
wide that the work is dealt out by the lengths.  Against tests/tkv8_ref.py, with the tolerances of tests/test_gpu_tkv.py."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from tests import tkv8_ref  # noqa: E402
from tests.test_gpu_tkv import T, ints, say, tables, typed  # noqa: E402
from tests.test_gpu_tkv8 import a_cache8, a_ref8, check_attend  # noqa: E402


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dim,group,new", [(128, 4, 16), (128, 3, 11), (128, 1, 17), (64, 5, 12), (64, 2, 32), (96, 4, 9),
                                           (256, 2, 32), (256, 7, 7), (256, 3, 17)])
def test_some_rows(dim, group, new, wide):
    say(f"some rows {dim} {group} {new} {wide}")
    rng = np.random.default_rng(dim + 10 * group + new)
    heads, page = (8, 1024) if wide else (2, 32)
    lens, news = [700, 60, 0], [new, new - 3, 0]
    width = 40 if wide else 23  # 48 workgroups a chunk over 40960 positions
    table, _ = tables(rng, 3, width)
    if wide:
        table = np.full((3, width), -1, np.int32)
        table[:2, 0] = [1, 0]
    ref = a_ref8(rng, 2 if wide else table.size, heads, dim, page, table, lens)
    cache, _ = a_cache8(ref)
    starts = np.concatenate(([0], np.cumsum(news)))
    qt, q = typed(rng.standard_normal((starts[-1], group * heads, dim)), "bf16" if new % 2 else "f16")
    for window, sinks, causal in ((None, 0, True), (None, 0, False), (100, 5, True), (3, 70, True)):
        out, lse, mags = tkv8_ref.attend(ref, table, lens, starts, q, dim ** -0.5, causal, window, sinks)
        got = T.tkv_attend(cache, qt, ints(table), ints(lens), starts=ints(starts), max_new=new, causal=causal,
                           window=window, sinks=sinks)
        torch.cuda.synchronize()
        check_attend(got, (out, lse), mags, "bf16" if new % 2 else "f16", dim)
