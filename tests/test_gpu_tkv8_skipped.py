"""New tokens that a rotation's table does not turn are left alone.  A record none of whose positions has been cached has
no power yet: what its bytes were before may not become one, or count for the tokens that come later."""
import numpy as np
import pytest

from tests import tkv8_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from tests.test_gpu_tkv import DEV, T, ints, say, tables, typed  # noqa: E402
from tests.test_gpu_tkv8 import a_cache8, a_ref8, cos_sin  # noqa: E402


@pytest.mark.parametrize("was", [255, 254, 134, 20])
@pytest.mark.parametrize("skipped,new", [(2, 1), (2, 9), (9, 1), (9, 20), (40, 3), (40, 30)])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_a_record_whose_first_tokens_are_left_alone(dim, skipped, new, was):
    say(f"left alone {dim} {skipped} {new} {was}")
    rng = np.random.default_rng(dim + skipped + new)
    heads, page, lens = 2, 32, [0, 37, 64]
    table, _ = tables(rng, 3, 5)
    ref = a_ref8(rng, table.size, heads, dim, page, table, lens)
    live = np.zeros(ref.raw.shape, bool)
    for b in range(3):
        live |= ref.live(table[b], lens[b])
    # memory as it comes: numbers for codes, and a power that nobody has put there
    wild = rng.integers(0, 127, ref.raw.shape, dtype=np.uint8)
    wild[..., 64 * dim:64 * dim + 2] = was
    ref.raw[~live] = wild[~live]
    cache, pool = a_cache8(ref)
    before = ref.raw.copy()
    cs = cos_sin(160, dim)
    cst = torch.from_numpy(cs).to(DEV)
    kt, k = typed(rng.standard_normal((3 * skipped, heads, dim)), "f16")
    T.tkv_append(cache, kt, kt, ints(table), ints(lens), cos_sin=cst, positions=ints([-1] * (3 * skipped)))
    torch.cuda.synchronize()
    have = pool.cpu().numpy().reshape(ref.raw.shape)
    power = np.zeros(ref.raw.shape, bool)
    power[..., 64 * dim:64 * dim + 2] = True
    assert np.array_equal(have[live], before[live]) and np.array_equal(have[~power], before[~power])
    at = [n + skipped for n in lens]
    for b in range(3):
        for p0 in range(-(-lens[b] // 32) * 32, at[b], 32):  # records that had no positions and got none
            ref.raw[ref.page_of(table[b], p0), :, 0, 64 * dim:64 * dim + 2] = 0
    others = ref.raw == before
    assert np.array_equal(have[others], before[others])  # and no other record's power has changed
    kt, k = typed(rng.standard_normal((3 * new, heads, dim)), "f16")
    T.tkv_append(cache, kt, kt, ints(table), ints(at), cos_sin=cst)
    rk, rv = T.tkv_read(cache, ints(table), ints(at), n_tokens=3 * new, dtype=torch.float32)
    torch.cuda.synchronize()
    for b in range(3):
        rows = range(b * new, (b + 1) * new)
        turned = np.array([tkv8_ref.turned(k[i], cs, at[b] + i - b * new, False) for i in rows])
        ref.append(table[b], at[b], turned, k[rows])
        for h in range(heads):
            (wk, _, _), (wv, _, _), _ = ref.parts(table[b], h, at[b] + np.arange(new))
            for got, want in ((rk, wk), (rv, wv)):
                assert np.array_equal(got[rows, h].cpu().numpy(), want.astype(np.float32)), (b, h)
