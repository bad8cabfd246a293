"""The rotation and the window at the sizes that tests/test_gpu_tkv8.py leaves out: queries of so many heads that a token's go
to several waves, or to a wave several times; 4-bit caches with other groups, and heads of 96 channels."""
import numpy as np
import pytest

from tests import tkv8_ref, tkv_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from tests.test_gpu_tkv import DEV, DT, T, a_cache, a_ref, ints, say, tables, typed  # noqa: E402
from tests.test_gpu_tkv8 import ATTENDS, check_attend, cos_sin, specials  # noqa: E402


def turned(x, cs, at, neighbours):
    """x [tokens, heads, dim] of 16 bits on the host, turned by rows `at` of cs: each product and sum rounded to fp32"""
    half = cs.shape[1] // 2
    c, s = (torch.from_numpy(cs[at][:, None, i * half:(i + 1) * half]) for i in (0, 1))
    y = x.float()
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if neighbours else (slice(0, half), slice(half, 2 * half))
    a, b = y[..., first], y[..., second]
    out = y.clone()
    out[..., first], out[..., second] = a * c - b * s, b * c + a * s
    return out.to(x.dtype)


# A wave has 16, 10, 8 or 4 heads of 64, 96, 128 or 256 channels at once: one wave and more of them, the most there are, and
# more heads than those have at once
QUERIES = [(64, 32), (64, 17), (64, 1100), (96, 32), (96, 11), (96, 700), (128, 32), (128, 9), (128, 600), (256, 16), (256, 5),
           (256, 300)]


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("new", [1, 3, 9, 40])
@pytest.mark.parametrize("dim,q_heads", QUERIES)
def test_queries_of_many_heads(dim, q_heads, new, bits):
    say(f"queries {dim} {q_heads} {new} {bits}")
    rng = np.random.default_rng(dim + q_heads + new)
    page, lens = 32, [0, 70, 31]
    table = ints(tables(rng, 3, 4)[0])
    pool = torch.zeros(12 * T.tkv_page_bytes_of(1, dim, page, 32, bits), dtype=torch.uint8, device=DEV)
    cache = T.tkv_encode(pool, 1, dim, page, 32, bits=bits)
    gen = torch.Generator().manual_seed(q_heads)
    at = np.concatenate([n + np.arange(new) for n in lens])
    k = torch.randn((3 * new, 1, dim), generator=gen).half().to(DEV)
    for rot, neighbours, dtype in ((dim, False, "f16"), (dim // 2, True, "bf16")):
        cs = cos_sin(128, rot)
        q = torch.randn((3 * new, q_heads, dim), generator=gen).to(DT[dtype])
        want = turned(q, cs, at, neighbours)
        kw = dict(cos_sin=torch.from_numpy(cs).to(DEV), neighbours=neighbours)
        qt = q.to(DEV)
        out = T.tkv_append(cache, k, k, table, ints(lens), q=qt, **kw)
        assert torch.equal(out.cpu(), want)
        room = torch.full((3 * new, q_heads + 1, dim), 7.0, dtype=DT[dtype], device=DEV)
        T.tkv_append(cache, k, k, table, ints(lens), q=qt, q_out=room[:, :-1], **kw)
        assert torch.equal(room[:, :-1].cpu(), want) and (room[:, -1] == 7.0).all()
        T.tkv_append(cache, k, k, table, ints(lens), q=qt, q_out=qt, **kw)
        assert torch.equal(qt.cpu(), want)


@pytest.mark.parametrize("new", [1, 2])
def test_queries_of_many_tokens_a_few_each(new):
    """More tokens than have several waves each."""
    rng = np.random.default_rng(new)
    dim, q_heads, n_seq = 128, 20, 1100
    pool = torch.zeros(n_seq * T.tkv_page_bytes_of(1, dim, 32, bits=8), dtype=torch.uint8, device=DEV)
    cache = T.tkv_encode(pool, 1, dim, 32, bits=8)
    lens = rng.integers(0, 30, n_seq)
    at = (lens[:, None] + np.arange(new)).reshape(-1)
    q = torch.randn((n_seq * new, q_heads, dim), generator=torch.Generator().manual_seed(1)).half()
    cs = cos_sin(32, dim)
    k = torch.ones((n_seq * new, 1, dim), dtype=torch.float16, device=DEV)
    out = T.tkv_append(cache, k, k, ints(np.arange(n_seq)[:, None]), ints(lens), cos_sin=torch.from_numpy(cs).to(DEV), q=q.to(DEV))
    assert torch.equal(out.cpu(), turned(q, cs, at, False))


@pytest.mark.parametrize("turn", [("all", False), ("half", True)], ids=str)
@pytest.mark.parametrize("new", [[1, 4, 2], [9, 40, 33]], ids=str)
@pytest.mark.parametrize("dim,group", [(64, 64), (96, 32), (128, 64), (128, 128), (256, 64), (256, 128)])
def test_rotated_append_in_groups(dim, group, new, turn):
    say(f"append in groups {dim} {group} {new} {turn}")
    rng = np.random.default_rng(dim + group)
    heads, page, lens = 2, 64, [31, 0, 62]
    table, _ = tables(rng, 3, 2, 1)
    starts = np.concatenate(([0], np.cumsum(new)))
    ref = tkv_ref.Ref(table.size + 1, heads, dim, page, group, rng)
    cache, pool = a_cache(ref)
    kt, k = typed(specials(rng, starts[-1], heads, dim), "bf16")
    vt, v = typed(specials(rng, starts[-1], heads, dim)[::-1], "bf16")
    cs = cos_sin(128, dim if turn[0] == "all" else dim // 2)
    T.tkv_append(cache, kt, vt, ints(table), ints(lens), starts=ints(starts), max_new=max(new),
                 cos_sin=torch.from_numpy(cs).to(DEV), neighbours=turn[1])
    torch.cuda.synchronize()
    for b in range(3):
        for i in range(new[b]):
            k[starts[b] + i] = tkv8_ref.turned(k[starts[b] + i], cs, lens[b] + i, turn[1])
    kc, ks, kz = tkv_ref.quantise(k, group)
    vc, vs, vz = tkv_ref.quantise(v, group)
    for b in range(3):
        for i in range(new[b]):
            pos, row = lens[b] + i, starts[b] + i
            for h in range(heads):
                ref.put(ref.page_of(table[b], pos), h, pos, kc[row, h], ks[row, h], kz[row, h], vc[row, h], vs[row, h], vz[row, h])
    assert np.array_equal(pool.cpu().numpy().reshape(ref.raw.shape), ref.raw)


@pytest.mark.parametrize("case,group", [(c, g) for c in ATTENDS for g in (32, 128) if (c[0], g) in ((96, 32), (128, 128), (256, 128))],
                         ids=lambda c: "-".join(map(str, c[:5])) + f"-{c[6][0]}" if isinstance(c, tuple) else str(c))
def test_window_in_4_bits_in_groups(case, group):
    dim, page, heads, q_heads, dtype, lens, new, causal = case
    rng = np.random.default_rng(sum(lens) + dim)
    width = max(-(-n // page) for n in lens) + 1
    table, _ = tables(rng, len(lens), width, 2)
    ref = a_ref(rng, table.size + 2, heads, dim, page, group, table, lens)
    cache, _ = a_cache(ref)
    starts = np.concatenate(([0], np.cumsum(new)))
    qt, q = typed(1.5 * rng.standard_normal((starts[-1], q_heads, dim)), dtype)
    for window, sinks in ((7, 3), (40, 0), (64, 33), (100000, 5)):
        say(f"window in 4 bits {case} {group} {window} {sinks}")
        out, lse, mags = tkv8_ref.attend(ref, table, lens, starts, q, dim ** -0.5, causal, window, sinks)
        got = T.tkv_attend(cache, qt, ints(table), ints(lens), starts=ints(starts), max_new=max(new), causal=causal,
                           window=window, sinks=sinks)
        torch.cuda.synchronize()
        check_attend(got, (out, lse), mags, dtype, dim)
