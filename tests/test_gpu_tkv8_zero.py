"""Records of the 8-bit cache whose power is E = 0, which stands for 0 whatever their codes are, before, between and after
others.  Against tests/tkv8_ref.py, which has the rule; tolerances as in tests/test_gpu_tkv8.py: what such a record brings
is 0 exactly."""
import numpy as np
import pytest

from tests import tkv8_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from tests.test_gpu_tkv import T, ints, say, tables, typed  # noqa: E402
from tests.test_gpu_tkv8 import a_cache8, a_ref8, check_attend  # noqa: E402

# Which of a sequence's records have E = 0.  Of few rows a wave takes every fourth record, of many rows every one.
PATTERNS = {
    "first": lambda i, n: i < min(6, n - 1),
    "between": lambda i, n: 4 <= i < n - 4,
    "last": lambda i, n: i >= n - 5,
    "every other": lambda i, n: i % 2 == 0,
    "all": lambda i, n: True,
}


def cleared(ref, table, lens, pattern, which):
    """E of the keys (0), of the values (1) or of both is 0 in the pattern's records; their codes stay"""
    for b, length in enumerate(lens):
        n = -(-length // 32)
        for i in range(n):
            if pattern(i, n):
                rec = ref.raw[ref.page_of(table[b], 32 * i), :, 32 * i % ref.page // 32]
                for w in which:
                    rec[:, 64 * ref.dim + w] = 0


@pytest.mark.parametrize("which", [(0,), (1,), (0, 1)], ids=["keys", "values", "both"])
@pytest.mark.parametrize("pattern", PATTERNS)
# 1, 6 and 24 rows, in tiles of 16 and 32, and 70, of a workgroup's 128
@pytest.mark.parametrize("dim,heads,group,new", [(128, 2, 2, 1), (64, 1, 3, 2), (96, 1, 4, 6), (128, 1, 4, 6), (256, 1, 4, 6),
                                                 (64, 1, 2, 35), (96, 1, 1, 70), (128, 1, 1, 70), (256, 1, 2, 35)])
def test_records_that_stand_for_0(dim, heads, group, new, pattern, which):
    say(f"E = 0: {dim} {heads} {group} {new} {pattern} {which}")
    rng = np.random.default_rng(dim + new)
    page, lens = 64, [700, 289, 90]  # two chunks and one
    table, _ = tables(rng, 3, 11)
    ref = a_ref8(rng, table.size, heads, dim, page, table, lens)
    # a record's codes are of all sizes, and its values have a mean, so that a wrong sum is far from 0
    for b, n in enumerate(lens):
        for p0 in range(0, n, 32):
            x = rng.standard_normal((2, min(32, n - p0), heads, dim))
            x[1] += 2.0
            ref.append(table[b], p0, x[0], x[1] * 2.0 ** rng.integers(-2, 3))
    cleared(ref, table, lens, PATTERNS[pattern], which)
    cache, _ = a_cache8(ref)
    qt, q = typed(rng.standard_normal((3 * new, group * heads, dim)), "f16")
    starts = np.arange(4) * new
    for window, sinks, causal in ((None, 0, True), (None, 0, False), (200, 40, True)):
        out, lse, mags = tkv8_ref.attend(ref, table, lens, starts, q, dim ** -0.5, causal, window, sinks)
        got = T.tkv_attend(cache, qt, ints(table), ints(lens), causal=causal, window=window, sinks=sinks)
        torch.cuda.synchronize()
        check_attend(got, (out, lse), mags, "f16", dim)
    rk, rv = T.tkv_read(cache, ints(table), ints([0, 0, 0]), n_tokens=3 * 64, dtype=torch.float32)
    for b in range(3):
        for h in range(heads):
            (k, _, _), (v, _, _), _ = ref.parts(table[b], h, np.arange(64))
            for got, want in ((rk, k), (rv, v)):
                assert np.array_equal(got[64 * b:64 * b + 64, h].cpu().numpy(), want.astype(np.float32))
