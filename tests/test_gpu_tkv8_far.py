"""The 8-bit cache in a pool of more than 4 GiB: what lies in its last pages gives, bit for bit, what it gives in a small
pool.  Calls on two streams, each with its own workspace, give what they give one after the other.  And a pool's description
takes no account of groups."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from tests.test_gpu_tkv import DEV, T, ints, say  # noqa: E402


def turns(n, dim):
    angle = torch.arange(n, device=DEV)[:, None] * 0.9 ** torch.arange(dim // 2, device=DEV)
    return torch.cat((angle.cos(), angle.sin()), -1)


def rows(n, heads, dim, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn((n, heads, dim), device=DEV, generator=g).to(torch.float16)


def test_pages_past_4_gib():
    say("pages past 4 GiB")
    heads, dim, page, n = 8, 256, 1024, 1500
    size = T.tkv_page_bytes_of(heads, dim, page, bits=8)
    many = (9 << 29) // size
    assert many * size > 1 << 32
    cs, got = turns(2 * page, dim), []
    k, v, q = (rows(n + 1, heads * g, dim, 5 + g) for g in (1, 1, 2))
    for pages, table in ((many, [[many - 1, many - 2]]), (2, [[1, 0]])):
        pool = torch.empty(pages * size, dtype=torch.uint8, device=DEV)
        cache = T.tkv_encode(pool, heads, dim, page, bits=8)
        table, res = ints(table), []
        res.append(T.tkv_append(cache, k[:n], v[:n], table, ints([0]), cos_sin=cs, q=q[:n]))
        res.append(T.tkv_append(cache, k[n:], v[n:], table, ints([n]), cos_sin=cs, q=q[n:]))
        res += T.tkv_read(cache, table, ints([0]), n_tokens=n + 1)
        for window, sinks in ((None, 0), (300, 4)):
            res += T.tkv_attend(cache, res[1], table, ints([n + 1]), window=window, sinks=sinks)
            res += T.tkv_attend(cache, res[0][:200], table, ints([n]), max_new=200, window=window, sinks=sinks)
        torch.cuda.synchronize()
        got.append(res)
        del pool, cache
    for a, b in zip(*got):
        assert torch.equal(a, b) and not a.isnan().any()


def test_calls_on_two_streams():
    say("two streams")
    heads, dim, page, n = 4, 128, 64, 700
    cs, sides = turns(n, dim), [torch.cuda.Stream(), torch.cuda.Stream()]
    want, got = [], []
    for out, streams in ((want, [None, None]), (got, sides)):
        for s in range(2):
            pool = torch.zeros(12 * T.tkv_page_bytes_of(heads, dim, page, bits=8), dtype=torch.uint8, device=DEV)
            cache = T.tkv_encode(pool, heads, dim, page, bits=8)
            k, v, q = (rows(n, heads * g, dim, s + 10 * g) for g in (1, 1, 2))
            table = torch.arange(12, dtype=torch.int32, device=DEV).flip(0)[None].contiguous()
            zero, length = ints([0]), ints([n])
            torch.cuda.synchronize()
            qt = T.tkv_append(cache, k, v, table, zero, cos_sin=cs, q=q, stream=streams[s])
            o, lse = T.tkv_attend(cache, qt, table, length, window=200 + s, sinks=3, stream=streams[s])
            one, _ = T.tkv_attend(cache, qt[-1:], table, length, stream=streams[s])
            out.append((pool, qt, o, lse, one, cache, k, v, q, table, zero, length))
        torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a[:5], b[:5]))


def test_groups_mean_nothing_in_8_bits():
    say("groups")
    size = T.tkv_page_bytes_of(2, 96, 32, bits=8)
    pool = torch.zeros(3 * size, dtype=torch.uint8, device=DEV)
    for group in (0, 64, 128):
        cache = T.tkv_encode(pool, 2, 96, 32, group, bits=8)
        assert (cache.n_pages, cache.group, cache.bits, T.tkv_page_bytes(cache)) == (3, 0, 8, size)
    with pytest.raises(ValueError, match="multiple"):
        T.tkv_encode(pool[:-16], 2, 96, 32, 0, bits=8)
    for group in (0, 64):
        with pytest.raises(ValueError, match="4 or 8"):
            T.tkv_encode(pool, 2, 64, 32, group, bits=2)
