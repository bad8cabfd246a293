"""A dimension of one element has no stride that counts: tables of one page a sequence, and the starts of no sequences, are
taken with any."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from tests.test_gpu_tkv import DEV, T, ints  # noqa: E402


@pytest.mark.parametrize("bits", [4, 8])
def test_tables_of_one_page(bits):
    heads, dim, n = 2, 64, 3
    size = n * T.tkv_page_bytes_of(heads, dim, 32, 64, bits)
    k = torch.randn((n, heads, dim), device=DEV).half()
    plain = ints([[2], [0], [1]])
    odd = ints([2, 0, 1]).as_strided((n, 1), (1, 0))
    wide = ints([2, 7, 0, 7, 1, 7]).as_strided((n, 1), (2, 5))
    results = []
    for table in (plain, odd, wide):
        pool = torch.zeros(size, dtype=torch.uint8, device=DEV)
        cache = T.tkv_encode(pool, heads, dim, 32, 64, bits=bits)
        T.tkv_append(cache, k, k, table, ints([0, 0, 0]))
        out, lse = T.tkv_attend(cache, k, table, ints([1, 1, 1]))
        results.append((pool, out, lse))
    for other in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))
    with pytest.raises(ValueError, match="contiguous"):
        T.tkv_append(cache, k, k, ints([[2, 0], [1, 2], [0, 1]])[:, ::2].expand(n, 2), ints([0, 0, 0]))


def test_starts_of_no_sequences():
    pool = torch.zeros(T.tkv_page_bytes_of(2, 64, 32), dtype=torch.uint8, device=DEV)
    cache = T.tkv_encode(pool, 2, 64, 32)
    none = torch.zeros((0, 2, 64), dtype=torch.float16, device=DEV)
    T.tkv_append(cache, none, none, torch.zeros((0, 1), dtype=torch.int32, device=DEV), ints([]), starts=ints([0]).as_strided((1,), (3,)))
