"""Attention over the 4-bit cache in every way of splitting it, with comparisons that a NaN fails, where what no row may
see is full of infinities and NaNs: bytes at random past the ends of sequences, pages that do not exist after a kernel
that has left NaNs in LDS.  Also batches past those that are dealt evenly, and pages that tile copies have moved."""
import numpy as np
import pytest

from tests import tkv_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import tests.test_gpu_tkv as operators  # noqa: E402
import tests.test_gpu_tkv_paths as paths  # noqa: E402
from tests.test_gpu_tkv import DEV, T, a_cache, a_ref, ints, say, tables, typed  # noqa: E402
from tests.test_gpu_tkv_limits import check_numbers  # noqa: E402
from tiled_tensor_bulk_amd import tmap  # noqa: E402


@pytest.fixture
def strict(monkeypatch):
    monkeypatch.setattr(operators, "check_attend", check_numbers)
    monkeypatch.setattr(paths, "check_attend", check_numbers)


@pytest.mark.parametrize("case", operators.ATTENDS, ids=lambda c: "-".join(map(str, c[:6])) + f"-{c[7][0]}")
def test_attend(strict, case):
    operators.test_attend(case)


@pytest.mark.parametrize("case", paths.ROWS, ids=lambda c: f"{c[0]}-{c[1]}-{c[3] * max(c[6])}")
def test_attend_rows(strict, case):
    paths.test_attend_rows(case)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", paths.EVEN, ids=lambda c: f"{c[0]}-{c[1]}-{c[3] * max(c[6])}")
def test_attend_positions_dealt_evenly(strict, case, causal):
    paths.test_attend_positions_dealt_evenly(case, causal)


@pytest.mark.parametrize("n,longest", [(256, 40), (200, 500), (37, 1500)])
def test_attend_even_shares_over_many_sequences(strict, n, longest):
    paths.test_attend_even_shares_over_many_sequences(n, longest)


@pytest.mark.parametrize("gh,new", [(2, 5), (3, 40)])
def test_rows_that_see_nothing(strict, gh, new):
    paths.test_rows_that_see_nothing(gh, new)


def test_attend_without_pages_and_past_the_table(strict):
    operators.test_attend_skips_pages_that_do_not_exist()
    operators.test_attend_clamps_lengths_and_refuses_wild_starts()
    operators.test_attend_without_starts_strided_and_on_another_stream()
    operators.test_attend_numbers_that_fp16_cannot_hold()


@pytest.mark.parametrize("dim,group", [(64, 32), (96, 32), (128, 64), (128, 128), (256, 32), (256, 128)])
@pytest.mark.parametrize("gh,new", [(3, 1), (1, 16), (7, 4), (3, 40)])
def test_missing_pages_after_nans(dim, group, gh, new):
    """A kernel over a pool of NaNs leaves NaNs in LDS and in registers; then pages are missing everywhere, and at every
    other place."""
    say(f"nans {dim} {group} {gh} {new}")
    rng = np.random.default_rng(dim + gh)
    heads, page, n, held = 2, 32, 16, 20
    nans = torch.full((n * held * T.tkv_page_bytes_of(heads, dim, page, group),), 0xFF, dtype=torch.uint8, device=DEV)
    bad = T.tkv_encode(nans, heads, dim, page, group)
    q, values = typed(rng.standard_normal((n * new, heads * gh, dim)), "bf16")
    full = ints(rng.permutation(n * held).reshape(n, held))
    lens = ints([held * page] * n)
    so = torch.zeros((n, heads, held * page), device=DEV)
    assert torch.isnan(T.tkv_attend(bad, q, full, lens, scores_out=so)[0]).all()
    so.zero_()
    out, lse = T.tkv_attend(bad, q, torch.full_like(full, -1), lens, scores_out=so)
    assert (out == 0).all() and torch.isneginf(lse).all() and (so == 0).all()
    # every other page missing, and an end inside a page
    table = rng.permutation(2 * held).astype(np.int32).reshape(2, held)
    table[:, 1::2] = -1
    some = [held * page - 45, 300]
    ref = a_ref(rng, 2 * held, heads, dim, page, group, table, some)
    cache, _ = a_cache(ref)
    want = tkv_ref.attend(ref, table, some, [0, new, 2 * new], values[:2 * new], dim ** -0.5, True)
    T.tkv_attend(bad, q, full, lens)
    check_numbers(T.tkv_attend(cache, q[:2 * new], ints(table), ints(some)), want[:2], want[3], "bf16", dim)


@pytest.mark.parametrize("n", [256, 257, 300])
def test_more_sequences_than_are_dealt_evenly(strict, n):
    """Tables that are far wider than the lengths, with as many sequences as an even split has, and more."""
    say(f"sequences {n}")
    rng = np.random.default_rng(n)
    lens = [int(x) for x in rng.integers(1, 130, n)]
    lens[n // 3], lens[-1] = 700, 0
    new = [1] * n
    paths.even_batch(rng, 64, 64, 2, 2, "bf16", lens, new, True, True, 1200)


def test_pages_that_tile_copies_have_moved():
    """A page is a run of bytes that the tile copies move: pages gathered out of one pool into packed boxes and scattered
    into another one read, and are attended over, as they were."""
    rng = np.random.default_rng(8)
    heads, gh, dim, page, group, held = 2, 3, 128, 32, 64, 7
    table, _ = tables(rng, 1, held, 3)
    ref = a_ref(rng, held + 3, heads, dim, page, group, table, [200])
    cache, pool = a_cache(ref)
    rows = T.tkv_page_bytes(cache) // 128  # of a page, 128 bytes each: one box
    other = torch.zeros(12 * rows * 128, dtype=torch.uint8, device=DEV)
    to = rng.permutation(12)[:held].astype(np.int32)
    maps = [tmap.tmap_encode("u8", 2, x.data_ptr(), [128, x.numel() // 128], [128], [128, rows]) for x in (pool, other)]
    corners = [ints([[0, int(p) * rows] for p in pages]) for pages in (table[0], to)]
    packed = torch.empty(held * rows * 128, dtype=torch.uint8, device=DEV)
    tmap.tmap_load_tiles(maps[0], corners[0], held, packed)
    tmap.tmap_store_tiles(maps[1], corners[1], held, packed)
    assert tmap.tmap_sync_status() == tmap.SUCCESS
    moved = T.tkv_encode(other, heads, dim, page, group)
    q, _ = typed(rng.standard_normal((1, heads * gh, dim)), "f16")
    for f in (lambda c, t: T.tkv_attend(c, q, t, ints([200])),
              lambda c, t: T.tkv_read(c, t, ints([0]), n_tokens=200, dtype=torch.float32)):
        for x, y in zip(f(cache, ints(table)), f(moved, ints(to[None]))):
            assert torch.equal(x, y)
