"""The 8-bit cache, the rotation on the way into a cache and attention through a window, against the plain implementation
of tests/tkv8_ref.py.

Codes, powers and turned queries have to be equal.  Attention's tolerances are those of tests/test_gpu_tkv.py, which count
roundings: in 8 bits a value enters the matrix unit as it is, so that its part of them is not used up."""
import itertools

import numpy as np
import pytest

from tests import tkv8_ref, tkv_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from tests.test_gpu_tkv import DEV, DT, T, a_cache, a_ref, bounds, ints, say, tables, to64, typed  # noqa: E402


def a_cache8(ref):
    pool = torch.from_numpy(ref.raw.reshape(-1).copy()).to(DEV)
    return T.tkv_encode(pool, ref.heads, ref.dim, ref.page, bits=8), pool


def a_ref8(rng, pages, heads, dim, page, table, lens, spread=3):
    """a pool with ordinary keys and values at positions below lens and random bytes elsewhere; records' powers differ"""
    ref = tkv8_ref.Ref8(pages, heads, dim, page, rng)
    for b, n in enumerate(lens):
        for p0 in range(0, n, 32):
            m = min(32, n - p0)
            x = rng.standard_normal((2, m, heads, dim)) * 2.0 ** rng.integers(-spread, 1, (2, 1, heads, 1))
            ref.append(table[b], p0, x[0], x[1])
    return ref


def check_attend(got, want, mags, dtype, dim):
    out, lse = to64(got[0]), to64(got[1])
    tol, tol_lse = bounds(want, mags, dtype, dim)
    empty = ~np.isfinite(want[1])
    assert np.array_equal(lse[empty], want[1][empty])
    assert not out[empty].any()
    good = np.abs(out - want[0]) <= tol
    assert good.all(), (np.argwhere(~good)[:5], out[~good][:5], want[0][~good][:5], tol[~good][:5])
    assert (np.abs(lse[~empty] - want[1][~empty]) <= tol_lse[~empty]).all()


def cos_sin(n, dim):
    angle = np.arange(n)[:, None] * 10000.0 ** (-np.arange(dim // 2) / (dim // 2))
    return np.concatenate((np.cos(angle), np.sin(angle)), 1).astype(np.float32)


def specials(rng, n, heads, dim):
    """rows of ordinary numbers, and of those that quantising has to look at"""
    x = rng.standard_normal((n, heads, dim)) * np.exp(rng.standard_normal((n, heads, 1)))
    for i, v in enumerate([0.0, 1.75, np.nan, np.inf, -np.inf, 1e-7, 60000.0]):
        if i < n:
            x[i, 0, :8] = v                # a run alike
            x[n - 1 - i, -1, dim - 3] = v  # one element among others
    if n > 40:
        x[33:40, 0] = 2.0 ** -12 * rng.integers(-15, 16, (7, dim))  # what is subnormal, and on borders
    return x


# ------------------------------------------------------------------ append and read

APPENDS = [
    # dim, page, heads, dtype, lens before, new tokens
    (128, 64, 2, "bf16", [0, 5, 31, 63], [1, 1, 1, 1]),
    (128, 32, 1, "f16", [0, 7, 30], [32, 29, 70]),
    (128, 128, 3, "bf16", [100, 0, 96], [3, 200, 0]),
    (64, 32, 2, "f16", [1, 40], [0, 33]),
    (64, 256, 1, "bf16", [250], [9]),
    (96, 64, 2, "bf16", [15, 16, 17], [2, 1, 47]),
    (96, 32, 1, "f16", [31], [4]),
    (256, 32, 1, "f16", [3], [60]),
    (256, 64, 2, "bf16", [0, 64, 62], [64, 1, 4]),
    (256, 32, 2, "f16", [31], [2]),
]
TURNS = [None, ("all", False), ("all", True), ("half", False), ("half", True)]


def append_both(case, turn, bits, q_heads=3):
    dim, page, heads, dtype, lens, new = case
    rng = np.random.default_rng(dim + page + len(new))
    width = max(-(-(a + b) // page) for a, b in zip(lens, new)) + 1
    table, _ = tables(rng, len(lens), width, 1)
    starts = np.concatenate(([0], np.cumsum(new)))
    n = int(starts[-1])
    kt, k = typed(specials(rng, n, heads, dim), dtype)
    vt, v = typed(specials(rng, n, heads, dim)[::-1], dtype)
    qt, q = typed(rng.standard_normal((n, q_heads, dim)), dtype)
    if bits == 8:
        ref = a_ref8(rng, table.size + 1, heads, dim, page, table, lens)
        cache, pool = a_cache8(ref)
    else:
        ref = tkv_ref.Ref(table.size + 1, heads, dim, page, 32, rng)
        cache, pool = a_cache(ref)
    kw, cs = {}, None
    if turn:
        cs = cos_sin(max(a + b for a, b in zip(lens, new)), dim if turn[0] == "all" else dim // 2)
        kw = dict(cos_sin=torch.from_numpy(cs).to(DEV), neighbours=turn[1], q=qt)
    q_out = T.tkv_append(cache, kt, vt, ints(table), ints(lens), starts=ints(starts), max_new=max(new), **kw)
    torch.cuda.synchronize()
    if turn:
        for b in range(len(lens)):
            for i in range(new[b]):
                row = starts[b] + i
                k[row] = tkv8_ref.turned(k[row], cs, lens[b] + i, turn[1])
                q[row] = tkv8_ref.turned(q[row], cs, lens[b] + i, turn[1])
        assert torch.equal(q_out, torch.from_numpy(q).to(DT[dtype]).to(DEV))
    else:
        assert q_out is None
    return ref, cache, pool, table, starts, k, v


@pytest.mark.parametrize("turn", TURNS, ids=str)
@pytest.mark.parametrize("case", APPENDS, ids=lambda c: "-".join(map(str, c[:5])))
def test_append_and_read(case, turn):
    dim, page, heads, dtype, lens, new = case
    say(f"append in 8 bits {case} {turn}")
    ref, cache, pool, table, starts, k, v = append_both(case, turn, 8)
    before = ref.raw.copy()
    keep = np.zeros(ref.raw.shape, bool)
    for b in range(len(lens)):
        ref.append(table[b], lens[b], k[starts[b]:starts[b + 1]], v[starts[b]:starts[b + 1]])
        keep |= ref.live(table[b], lens[b] + new[b])
    have = pool.cpu().numpy().reshape(ref.raw.shape)
    assert np.array_equal(have[keep], ref.raw[keep])
    touched = (have != before).any(-1)  # records that no new position lies in are as they were
    assert not (touched & ~(ref.raw != before).any(-1)).any()
    # back, from the first position on
    full = [a + b for a, b in zip(lens, new)]
    at = np.concatenate(([0], np.cumsum(full)))
    for out in (torch.float32, DT[dtype]):
        rk, rv = T.tkv_read(cache, ints(table), ints([0] * len(lens)), starts=ints(at), n_tokens=int(at[-1]), dtype=out)
        for b in range(len(lens)):
            for h in range(heads):
                (want_k, _, _), (want_v, _, _), _ = ref.parts(table[b], h, np.arange(full[b]))
                for got, want in ((rk, want_k), (rv, want_v)):
                    want = torch.from_numpy(want.astype(np.float32)).to(out)
                    assert torch.equal(got[at[b]:at[b + 1], h].cpu(), want)


@pytest.mark.parametrize("turn", TURNS[1:], ids=str)
@pytest.mark.parametrize("case", APPENDS, ids=lambda c: "-".join(map(str, c[:5])))
def test_rotated_append_in_4_bits(case, turn):
    dim, page, heads, dtype, lens, new = case
    say(f"append in 4 bits {case} {turn}")
    ref, cache, pool, table, starts, k, v = append_both(case, turn, 4)
    kc, ks, kz = tkv_ref.quantise(k, 32)
    vc, vs, vz = tkv_ref.quantise(v, 32)
    for b in range(len(lens)):
        for i in range(new[b]):
            pos, row = lens[b] + i, starts[b] + i
            page_at = ref.page_of(table[b], pos)
            for h in range(heads):
                ref.put(page_at, h, pos, kc[row, h], ks[row, h], kz[row, h], vc[row, h], vs[row, h], vz[row, h])
    assert np.array_equal(pool.cpu().numpy().reshape(ref.raw.shape), ref.raw)


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_append_few_tokens_as_many(dim):
    """Tokens of falling size put in one by one, four at a time and all at once have one power, so the same bytes; and of
    rising size, one by one, those of the plain implementation."""
    say(f"few tokens in 8 bits {dim}")
    rng = np.random.default_rng(dim)
    n, heads, page = 41, 2, 32
    table, _ = tables(rng, 1, 3)
    size = np.exp2(-np.arange(n) / 8)[:, None, None]
    for x in (size, size[::-1]):
        kt, k = typed(rng.uniform(0.5, 1, (n, heads, dim)) * x * rng.choice([-1, 1], (n, heads, dim)), "bf16")
        vt, v = typed(3 * x * rng.uniform(0.5, 1, (n, heads, dim)), "bf16")
        steps = (1, 4, n) if x is size else (1, 3, 5)
        for step in steps:
            ref = tkv8_ref.Ref8(3, heads, dim, page, np.random.default_rng(1))
            cache, pool = a_cache8(ref)
            for at in range(0, n, step):
                m = min(step, n - at)
                T.tkv_append(cache, kt[at:at + m], vt[at:at + m], ints(table), ints([at]))
                ref.append(table[0], at, k[at:at + m], v[at:at + m])
            torch.cuda.synchronize()
            keep = ref.live(table[0], n)
            assert np.array_equal(pool.cpu().numpy().reshape(ref.raw.shape)[keep], ref.raw[keep]), step


@pytest.mark.parametrize("bits,new", [(8, 2), (8, 9), (4, 2), (4, 9)])
def test_tokens_that_the_table_does_not_turn(bits, new):
    """Given positions, some outside the table: such a token changes nothing, also not its query."""
    rng = np.random.default_rng(bits + new)
    dim, heads, page, lens = 64, 2, 32, [30, 5]
    table, _ = tables(rng, 2, 2)
    cs = cos_sin(50, 32)
    positions = rng.integers(0, 50, 2 * new)
    positions[[0, new + 1]] = [-1, 50]
    kt, k = typed(rng.standard_normal((2 * new, heads, dim)), "f16")
    qt, q = typed(rng.standard_normal((2 * new, 5, dim)), "f16")
    if bits == 8:
        ref = a_ref8(rng, 4, heads, dim, page, table, lens)
        cache, pool = a_cache8(ref)
    else:
        ref = tkv_ref.Ref(4, heads, dim, page, 32, rng)
        cache, pool = a_cache(ref)
    out = torch.full_like(qt, 7.0)
    same = qt.clone()
    for to in (out, same):
        T.tkv_append(cache, kt, kt, ints(table), ints(lens), cos_sin=torch.from_numpy(cs).to(DEV), positions=ints(positions),
                     q=same if to is same else qt, q_out=to)
    turned = [tkv8_ref.turned(k[i], cs, positions[i], False) for i in range(2 * new)]
    live = np.array([t is not None for t in turned])
    assert live.sum() == 2 * new - 2
    for i in range(2 * new):
        want = tkv8_ref.turned(q[i], cs, positions[i], False)
        assert torch.equal(out[i].cpu(), torch.full((5, dim), 7.0).half() if want is None else torch.from_numpy(want).half())
        assert torch.equal(same[i].cpu(), torch.from_numpy(q[i] if want is None else want).half())
    tk = np.array([k[i] if t is None else t for i, t in enumerate(turned)])
    have = pool.cpu().numpy().reshape(ref.raw.shape)
    if bits == 8:
        keep = np.zeros(ref.raw.shape, bool)
        for b in range(2):
            ref.append(table[b], lens[b], tk[b * new:(b + 1) * new], k[b * new:(b + 1) * new], live[b * new:(b + 1) * new])
            keep |= ref.live(table[b], lens[b] + new)
        # a skipped position's bytes are as they were, but in a record whose power has grown nothing says so
        assert np.array_equal(have[keep], ref.raw[keep])
    else:
        kc, ks, kz = tkv_ref.quantise(tk, 32)
        vc, vs, vz = tkv_ref.quantise(k, 32)
        for i in np.flatnonzero(live):
            b, pos = i // new, lens[i // new] + i % new
            for h in range(heads):
                ref.put(ref.page_of(table[b], pos), h, pos, kc[i, h], ks[i, h], kz[i, h], vc[i, h], vs[i, h], vz[i, h])
        assert np.array_equal(have, ref.raw)


@pytest.mark.parametrize("bits", [4, 8])
def test_append_unaligned_strided_and_missing_pages(bits):
    rng = np.random.default_rng(5)
    heads, dim, n = 2, 128, 9
    big, vals = typed(rng.standard_normal((2 * n, 3 * heads * dim + 3)), "f16")
    cs = np.zeros((40, dim + 1), np.float32)
    cs[:, 1:] = cos_sin(40, dim)
    cst = torch.from_numpy(cs).to(DEV)
    table = np.array([[1, -1], [7, 0]], np.int32)  # a page missing in each
    for off in (0, 1):
        k = big.as_strided((2 * n, heads, dim), (big.stride(0), dim, 1), off)
        v = big.as_strided((2 * n, heads, dim), (big.stride(0), dim, 1), off + heads * dim)
        q = big.as_strided((2 * n, heads, dim), (big.stride(0), dim, 1), off + 2 * heads * dim)
        room = torch.zeros((2 * n, heads + 1, dim + 8), dtype=torch.float16, device=DEV)
        if bits == 8:
            ref = tkv8_ref.Ref8(2, heads, dim, 32, rng)
            cache, pool = a_cache8(ref)
        else:
            ref = tkv_ref.Ref(2, heads, dim, 32, 64, rng)
            cache, pool = a_cache(ref)
        lens = [27, 30]
        ref.raw[0] = ref.raw[1] = 0
        pool.zero_()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        T.tkv_append(cache, k, v, ints(table), ints(lens), cos_sin=cst[:, 1:] if off else cst[:, 1:].contiguous(), q=q,
                     q_out=room[:, 1:, off:dim + off], stream=side)
        side.synchronize()
        for b in range(2):
            at = b * n
            x = vals[at:at + n, off:off + 3 * heads * dim].reshape(n, 3, heads, dim)
            tk = np.array([tkv8_ref.turned(x[i, 0], cs[:, 1:], lens[b] + i, False) if lens[b] + i < 40 else x[i, 0] for i in range(n)])
            tq = np.array([tkv8_ref.turned(x[i, 2], cs[:, 1:], lens[b] + i, False) if lens[b] + i < 40 else 0 * x[i, 2] for i in range(n)])
            assert np.array_equal(to64(room[at:at + n, 1:, off:dim + off]), tq.astype(np.float16).astype(np.float64))
            for i in range(n) if bits == 4 else ():
                pg = ref.page_of(table[b], lens[b] + i)
                if pg >= 0:
                    kc, ks, kz = tkv_ref.quantise(tk[i], 64)
                    vc, vs, vz = tkv_ref.quantise(x[i, 1], 64)
                    for h in range(heads):
                        ref.put(pg, h, lens[b] + i, kc[h], ks[h], kz[h], vc[h], vs[h], vz[h])
            if bits == 8:
                ref.append(table[b], lens[b], tk, x[:, 1])
        assert not room[:, 0].any()
        have = pool.cpu().numpy().reshape(ref.raw.shape)
        assert np.array_equal(have, ref.raw)
        rk, _ = T.tkv_read(cache, ints(table), ints([0, 0]), n_tokens=128, dtype=torch.float32)
        assert not rk[32:64].any() and not rk[64:96].any()  # pages that do not exist read as 0


# ------------------------------------------------------------------ attention

ATTENDS = [
    # dim, page, heads, q heads, dtype, lens (new tokens included), new tokens, causal
    (128, 64, 2, 8, "bf16", [1, 31, 32, 33, 100, 0], [1, 1, 1, 1, 1, 1], True),
    (128, 64, 1, 1, "f16", [2000], [1], True),               # many chunks
    (128, 32, 1, 5, "bf16", [700, 64, 3], [1, 1, 1], True),
    (128, 128, 2, 6, "f16", [129, 300], [5, 3], True),       # 16 rows and fewer
    (128, 32, 1, 3, "bf16", [90, 50], [9, 7], True),         # 32 rows and fewer
    (128, 64, 1, 4, "f16", [333, 40, 65], [37, 40, 1], True),  # blocks of many rows, ragged
    (128, 64, 1, 7, "bf16", [300], [50], False),
    (128, 64, 1, 3, "bf16", [40], [40], True),
    (64, 32, 5, 15, "f16", [500, 5], [5, 5], True),
    (64, 256, 1, 16, "bf16", [600], [1], True),
    (64, 64, 1, 17, "bf16", [100], [3], False),              # rows past one tile of 16
    (64, 32, 2, 2, "f16", [257], [100], True),
    (96, 64, 2, 4, "bf16", [200, 33], [1, 1], True),
    (96, 32, 1, 3, "f16", [150], [8], True),
    (96, 128, 1, 1, "f16", [400], [90], False),
    (256, 32, 1, 2, "bf16", [77, 130], [1, 1], True),
    (256, 64, 1, 4, "f16", [200], [20], True),
    (256, 32, 1, 8, "bf16", [140], [3], False),
    (256, 64, 1, 1, "bf16", [150], [70], True),
]
WINDOWS = [(None, 0), (1, 0), (7, 3), (40, 0), (64, 33), (100000, 5)]


@pytest.mark.parametrize("case", ATTENDS, ids=lambda c: "-".join(map(str, c[:5])) + f"-{c[6][0]}")
def test_attend(case):
    dim, page, heads, q_heads, dtype, lens, new, causal = case
    rng = np.random.default_rng(sum(lens) + dim)
    width = max(-(-n // page) for n in lens) + 1
    table, _ = tables(rng, len(lens), width, 2)
    ref = a_ref8(rng, table.size + 2, heads, dim, page, table, lens)
    cache, _ = a_cache8(ref)
    starts = np.concatenate(([0], np.cumsum(new)))
    qt, q = typed(1.5 * rng.standard_normal((starts[-1], q_heads, dim)), dtype)
    for window, sinks in WINDOWS:
        say(f"attend in 8 bits {case} {window} {sinks}")
        out, lse, mags = tkv8_ref.attend(ref, table, lens, starts, q, dim ** -0.5, causal, window, sinks)
        for max_len in (None, max(lens)):
            got = T.tkv_attend(cache, qt, ints(table), ints(lens), starts=ints(starts), max_new=max(new), max_len=max_len,
                               causal=causal, window=window, sinks=sinks)
            torch.cuda.synchronize()
            check_attend(got, (out, lse), mags, dtype, dim)


@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("case", [c for c in ATTENDS if c[0] != 96], ids=lambda c: "-".join(map(str, c[:5])) + f"-{c[6][0]}")
def test_window_in_4_bits(case, group):
    dim, page, heads, q_heads, dtype, lens, new, causal = case
    rng = np.random.default_rng(sum(lens) + dim)
    width = max(-(-n // page) for n in lens) + 1
    table, _ = tables(rng, len(lens), width, 2)
    ref = a_ref(rng, table.size + 2, heads, dim, page, group, table, lens)
    cache, _ = a_cache(ref)
    starts = np.concatenate(([0], np.cumsum(new)))
    qt, q = typed(1.5 * rng.standard_normal((starts[-1], q_heads, dim)), dtype)
    for window, sinks in WINDOWS[1:]:
        say(f"window in 4 bits {case} {window} {sinks}")
        out, lse, mags = tkv8_ref.attend(ref, table, lens, starts, q, dim ** -0.5, causal, window, sinks)
        got = T.tkv_attend(cache, qt, ints(table), ints(lens), starts=ints(starts), max_new=max(new), causal=causal,
                           window=window, sinks=sinks)
        torch.cuda.synchronize()
        check_attend(got, (out, lse), mags, dtype, dim)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("new,window,sinks", [(1, 300, 4), (1, 1000, 200), (6, 129, 0), (9, 700, 40), (60, 250, 65)])
def test_windows_far_from_the_sinks(bits, new, window, sinks):
    """Long sequences whose pages between the sinks and the window are gone from the table, and hold NaNs."""
    say(f"far window {bits} {new} {window} {sinks}")
    rng = np.random.default_rng(new + window)
    dim, heads, page, lens = 64, 2, 32, [5000, 2100, window + sinks + 3]
    width = 160
    table, _ = tables(rng, 3, width)
    if bits == 8:
        ref = tkv8_ref.Ref8(3 * width, heads, dim, page, rng)
    else:
        ref = tkv_ref.Ref(3 * width, heads, dim, page, 32, rng)
    for b, n in enumerate(lens):  # what is not seen stays at random bytes
        first = max(0, n - new + 1 - window) // 32 * 32
        for p0 in itertools.chain(range(0, min(n, sinks), 32), range(first, n, 32)):
            x = rng.standard_normal((2, min(32, n - p0), heads, dim))
            if bits == 8:
                ref.append(table[b], p0, x[0], x[1])
            else:
                (kc, ks, kz), (vc, vs, vz) = (tkv_ref.quantise(y, 32) for y in x)
                for i, h in itertools.product(range(x.shape[1]), range(heads)):
                    ref.put(ref.page_of(table[b], p0), h, p0 + i, kc[i, h], ks[i, h], kz[i, h], vc[i, h], vs[i, h], vz[i, h])
        if b == 0:
            table[b, -(-sinks // 32):first // 32] = -1
    cache, _ = a_cache8(ref) if bits == 8 else a_cache(ref)
    qt, q = typed(rng.standard_normal((3 * new, 2 * heads, dim)), "f16")
    starts = [0, new, 2 * new, 3 * new]
    out, lse, mags = tkv8_ref.attend(ref, table, lens, starts, q, 0.125, True, window, sinks)
    got = T.tkv_attend(cache, qt, ints(table), ints(lens), window=window, sinks=sinks)
    check_attend(got, (out, lse), mags, "f16", dim)


def test_attend_edges_of_lengths_and_tables():
    """Lengths past the table (the border goes by the length), negative ones, missing pages, wild starts."""
    rng = np.random.default_rng(13)
    table = np.array([[0, 1], [2, -1], [3, 4]], np.int32)
    ref = a_ref8(rng, 5, 1, 64, 32, table, [64, 32, 64])
    cache, _ = a_cache8(ref)
    qt, q = typed(rng.standard_normal((6, 2, 64)), "bf16")
    for causal, window in itertools.product((True, False), (None, 5, 50)):
        for lens in ([66, 64, -3], [10 ** 9, 40, 64], [64, 33, 2]):
            want = tkv8_ref.attend(ref, table, lens, [0, 2, 4, 6], q, 0.125, causal, window, 3 if window else 0)
            got = T.tkv_attend(cache, qt, ints(table), ints(lens), scale=0.125, causal=causal, window=window,
                               sinks=3 if window else 0)
            check_attend(got, want[:2], want[2], "bf16", 64)
    out, lse = torch.zeros_like(qt), torch.zeros((6, 2), device=DEV)
    for starts in ([0, 9, 4, 4], [-3, 0, 0, 0], [0, -1, 0, 0]):  # rows outside q belong to nobody
        T.tkv_attend(cache, qt, ints(table), ints([64, 32, 64]), starts=ints(starts), out=out, lse=lse)
        assert not out.any() and not lse.any()


def test_powers_far_apart():
    """Values of 2^-40 and of 10^4 in neighbouring records, the weight on either; queries of all sizes."""
    rng = np.random.default_rng(3)
    table = np.array([[2, 0, 1, 3]], np.int32)
    for sizes in ([1e4, 2.0 ** -40, 1e4, 1], [2.0 ** -40, 1e-3, 2.0 ** -30, 1e-6], [1e-6, 1, 1e4, 1e4]):
        for wanted in range(4):
            ref = tkv8_ref.Ref8(4, 1, 64, 32, rng)
            for i, size in enumerate(sizes):
                k = np.zeros((32, 1, 64))
                k[:, 0, i] = 1.0
                k += 0.01 * rng.standard_normal(k.shape)
                ref.append(table[0], 32 * i, k, size * rng.standard_normal((32, 1, 64)))
            cache, _ = a_cache8(ref)
            for dtype, new in (("bf16", 1), ("f16", 70)):
                x = 0.1 * rng.standard_normal((new, 1, 64))
                x[:, 0, wanted] += 300.0
                qt, q = typed(x, dtype)
                want = tkv8_ref.attend(ref, table, [128], [0, new], q, 1.0, False)
                got = T.tkv_attend(cache, qt, ints(table), ints([128]), scale=1.0, causal=False)
                lost = 2.0 ** -31 * 2.0 ** (int(ref.raw[:, 0, 0, 64 * 64 + 1].max()) - 127)
                out, tol = to64(got[0]), bounds(want[:2], want[2], dtype, 64)[0]
                good = np.abs(out - want[0]) <= tol + 448 * lost
                assert good.all(), (sizes, wanted, dtype)


def test_a_wide_range_of_numbers():
    """Keys, values and queries from 2^-90 to 3 * 10^4 in bf16; a NaN or an infinity in one query's row only."""
    rng = np.random.default_rng(14)
    table = np.array([[1, 0]], np.int32)
    for size in (2.0 ** -90, 1e-3, 100.0):
        ref = tkv8_ref.Ref8(2, 1, 128, 32, rng)
        x = size * rng.standard_normal((2, 50, 1, 128))
        kt, k = typed(x[0], "bf16")
        vt, v = typed(x[1], "bf16")
        cache, _ = a_cache8(ref)
        T.tkv_append(cache, kt, vt, ints(table), ints([0]))
        ref.append(table[0], 0, k, v)
        qt, q = typed(rng.standard_normal((40, 1, 128)) / size, "bf16")
        want = tkv8_ref.attend(ref, table, [50], [0, 40], q, 0.05, True)
        check_attend(T.tkv_attend(cache, qt, ints(table), ints([50]), scale=0.05), want[:2], want[2], "bf16", 128)
        one = T.tkv_attend(cache, qt[-1:], ints(table), ints([50]), scale=0.05)
        check_attend(one, [w[-1:] for w in want[:2]], [m[-1:] for m in want[2]], "bf16", 128)
    for bad in (float("nan"), float("inf")):
        spoiled = qt.clone()
        spoiled[3, 0, 5] = bad
        out, lse = T.tkv_attend(cache, spoiled, ints(table), ints([50]), scale=0.05)
        clean, clean_lse = T.tkv_attend(cache, qt, ints(table), ints([50]), scale=0.05)
        rest = [i for i in range(40) if i != 3]
        assert torch.equal(out[rest], clean[rest]) and torch.equal(lse[rest], clean_lse[rest])
        assert not torch.isfinite(out[3]).all()


# ------------------------------------------------------------------ the paths that the operators choose between

@pytest.mark.parametrize("dim,new", [(128, 1), (64, 5), (256, 1)])
@pytest.mark.parametrize("window,sinks", [(None, 0), (2500, 40)])
@pytest.mark.parametrize("bits", [8, 4])
def test_even_shares(dim, new, window, sinks, bits):
    """Enough sequences and positions that few rows are dealt evenly."""
    say(f"even shares {dim} {new} {window} {bits}")
    rng = np.random.default_rng(dim)
    heads, page, n_seq = 8, 128, 24
    lens = [int(n) for n in rng.integers(1, 9000, n_seq)]
    lens[:3] = [9000, 0, new]
    lens = [max(n, new) if n else 0 for n in lens]
    width = 80
    table, _ = tables(rng, n_seq, width)
    gen = torch.Generator(device=DEV).manual_seed(dim)
    pool = torch.zeros(n_seq * width * T.tkv_page_bytes_of(heads, dim, page, 64, bits), dtype=torch.uint8, device=DEV)
    cache = T.tkv_encode(pool, heads, dim, page, 64, bits=bits)
    starts = np.concatenate(([0], np.cumsum(lens)))
    k, v = (torch.randn((int(starts[-1]), heads, dim), device=DEV, generator=gen).half() for _ in range(2))
    T.tkv_append(cache, k, v, ints(table), ints([0] * n_seq), starts=ints(starts), max_new=9000)
    q = torch.randn((n_seq * new, heads, dim), device=DEV, generator=gen).half()
    out, lse = T.tkv_attend(cache, q, ints(table), ints(lens), window=window, sinks=sinks, max_len=9000)
    rk, rv = T.tkv_read(cache, ints(table), ints([0] * n_seq), starts=ints(starts), n_tokens=int(starts[-1]),
                        max_new=9000, dtype=torch.float32)
    for b, n in enumerate(lens):
        for i in range(new):
            border = n - new + 1 + i
            pos = torch.arange(n, device=DEV)
            seen = pos < border
            if window:
                seen &= (pos >= border - window) | (pos < sinks)
            row = b * new + i
            if not seen.any():
                assert not out[row].any() and torch.isinf(lse[row]).all()
                continue
            kk, vv = (x[starts[b]:starts[b + 1]][seen].double() for x in (rk, rv))
            x = (kk * q[row].double()).sum(-1) * dim ** -0.5  # positions, heads
            p = torch.softmax(x, 0)
            want = (p[..., None] * vv).sum(0)
            # weights and the output, half a step of fp16 each, and in 4 bits scale * (code - 8): its size is at most
            # 8 / 15 of the distance between a group's largest and smallest value, so 16 / 15 of the largest magnitude
            size = (p[..., None] * vv.abs()).sum(0)
            tol = 2.0 ** -9 * size + 1e-6 + (2.0 ** -11 * 16 / 15 * vv.abs().amax((0, 2))[:, None] if bits == 4 else 0)
            assert ((out[row].double() - want).abs() <= tol).all(), (b, i)
            assert torch.allclose(lse[row].double(), torch.logsumexp(x, 0), atol=1e-4)


@pytest.mark.parametrize("bits", [8, 4])
def test_a_step_captured_and_replayed(bits):
    """Append with a rotation, attend through a window, in a graph; lengths grow between the replays, eager work in between."""
    rng = np.random.default_rng(8)
    dim, heads, page, n_seq, steps = 64, 2, 32, 3, 40
    table, _ = tables(rng, n_seq, 8)
    tb = ints(table)
    size = n_seq * 8 * T.tkv_page_bytes_of(heads, dim, page, 64, bits)
    cs = torch.from_numpy(cos_sin(256, dim)).to(DEV)
    gen = torch.Generator(device=DEV).manual_seed(1)
    x = (torch.randn((steps, 3, n_seq, heads, dim), device=DEV, generator=gen) * torch.linspace(0.2, 3, steps, device=DEV).view(-1, 1, 1, 1, 1)).half()
    results = []
    for graphed in (False, True):
        pool = torch.zeros(size, dtype=torch.uint8, device=DEV)
        cache = T.tkv_encode(pool, heads, dim, page, 64, bits=bits)
        lens = ints([0, 31, 64])
        k, v, q = (torch.empty_like(x[0, 0]) for _ in range(3))

        def step():
            q_out = T.tkv_append(cache, k, v, tb, lens, cos_sin=cs, q=q)
            lens.add_(1)
            return T.tkv_attend(cache, q_out, tb, lens, window=20, sinks=2, max_len=256)

        def load(i):
            for to, j in ((k, 0), (v, 1), (q, 2)):
                to.copy_(x[i, j])

        if graphed:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                load(0)
                step()
            torch.cuda.current_stream().wait_stream(side)
            pool.zero_()
            lens.copy_(ints([0, 31, 64]))
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out, lse = step()
        got = []
        for i in range(steps):
            load(i)
            if graphed:
                graph.replay()
                torch.cuda.synchronize()
                T.tkv_read(cache, tb, lens, n_tokens=3)  # eager work between
            else:
                out, lse = step()
            got.append((out.clone(), lse.clone()))
        results.append((got, pool.clone()))
    for (a, la), (b, lb) in zip(results[0][0], results[1][0]):
        assert torch.equal(a, b) and torch.equal(la, lb)
    assert torch.equal(results[0][1], results[1][1])


def test_workspace_that_is_enough_for_any_window():
    rng = np.random.default_rng(4)
    dim, heads, page = 128, 4, 64
    pool = torch.zeros(64 * T.tkv_page_bytes_of(heads, dim, page, bits=8), dtype=torch.uint8, device=DEV)
    cache = T.tkv_encode(pool, heads, dim, page, bits=8)
    table = ints(rng.integers(0, 64, (4, 200)))
    for new, q_heads in ((1, 8), (9, 8), (70, 12)):
        room = torch.empty(T.tkv_attend_workspace(cache, 4, q_heads, new, 12000), dtype=torch.uint8, device=DEV)
        q = torch.randn((4 * new, q_heads, dim), device=DEV).half()
        for window, sinks in ((1, 0), (300, 3), (5000, 100), (20000, 1)):
            a = T.tkv_attend(cache, q, table, ints([12000, 7000, 100, 4000]), window=window, sinks=sinks, workspace=room)
            b = T.tkv_attend(cache, q, table, ints([12000, 7000, 100, 4000]), window=window, sinks=sinks)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_refusals_on_the_gpu():
    pool = torch.zeros(4 * T.tkv_page_bytes_of(2, 64, 32, bits=8), dtype=torch.uint8, device=DEV)
    cache = T.tkv_encode(pool, 2, 64, 32, bits=8)
    table, lens = ints([[0, 1], [2, 3]]), ints([5, 6])
    k = torch.zeros((2, 2, 64), dtype=torch.float16, device=DEV)
    cs = torch.zeros((64, 64), device=DEV)
    scores = torch.zeros((2, 2, 64), device=DEV)
    calls = [
        (lambda: T.tkv_encode(pool, 2, 64, 32, bits=6), "bits"),
        (lambda: T.tkv_encode(pool[:-1], 2, 64, 32, bits=8), "multiple"),
        (lambda: T.tkv_attend(cache, k, table, lens, sinks=3), "window"),
        (lambda: T.tkv_attend(cache, k, table, lens, window=0), "window"),
        (lambda: T.tkv_attend(cache, k, table, lens, window=4, sinks=-1), "sinks"),
        (lambda: T.tkv_attend(cache, k, table, lens, scores_out=scores), "4 bits"),
        (lambda: T.tkv_evict(cache, table, lens, scores, 4, 2, table), "4 bits"),
        (lambda: T.tkv_append(cache, k, k, table, lens, q=k), "cos_sin"),
        (lambda: T.tkv_append(cache, k, k, table, lens, positions=lens), "cos_sin"),
        (lambda: T.tkv_append(cache, k, k, table, lens, cos_sin=cs.half()), "cos_sin"),
        (lambda: T.tkv_append(cache, k, k, table, lens, cos_sin=cs.cpu()), "GPU"),
        (lambda: T.tkv_append(cache, k, k, table, lens, cos_sin=cs[0]), "cos_sin"),
        (lambda: T.tkv_append(cache, k, k, table, lens, cos_sin=cs[:, ::2]), "contiguous"),
        (lambda: T.tkv_append(cache, k, k, table, lens, cos_sin=cs[:, :24]), "rot_dim"),
        (lambda: T.tkv_append(cache, k, k, table, lens, cos_sin=torch.zeros((3, 80), device=DEV)), "channels"),
        (lambda: T.tkv_append(cache, k, k, table, lens, cos_sin=cs, positions=ints([1, 2, 3])), "positions"),
        (lambda: T.tkv_append(cache, k, k, table, lens, cos_sin=cs, q_out=k), "q_out"),
        (lambda: T.tkv_append(cache, k, k, table, lens, cos_sin=cs, q=k.float()), "q must"),
        (lambda: T.tkv_append(cache, k, k, table, lens, cos_sin=cs, q=k[:1]), "tokens"),
        (lambda: T.tkv_append(cache, k, k, table, lens, cos_sin=cs, q=k, q_out=k.bfloat16()), "q_out"),
        (lambda: T.tkv_append(cache, k, k, table, lens, cos_sin=cs, q=k, q_out=k[:1].expand(2, 2, 64)), "overlap"),
        (lambda: T.tkv_append(cache, k, k, table, lens, cos_sin=cs.clone().requires_grad_()), "no_grad"),
    ]
    before = pool.clone()
    for call, word in calls:
        with pytest.raises((ValueError, T.TmapError), match=word):
            call()
    assert torch.equal(pool, before)
    four = T.tkv_encode(torch.zeros(T.tkv_page_bytes_of(2, 64, 32, 64), dtype=torch.uint8, device=DEV), 2, 64, 32, 64)
    with pytest.raises(T.TmapError, match="window"):
        T.tkv_attend(four, k, table, lens, window=4, scores_out=scores)


def test_nothing_to_do():
    pool = torch.zeros(4 * T.tkv_page_bytes_of(2, 64, 32, bits=8), dtype=torch.uint8, device=DEV)
    cache = T.tkv_encode(pool, 2, 64, 32, bits=8)
    none = torch.zeros((0, 2, 64), dtype=torch.float16, device=DEV)
    cs = torch.zeros((64, 64), device=DEV)
    for n_seq in (0, 2):
        table, lens = ints(np.zeros((n_seq, 2))), ints([3] * n_seq)
        q = T.tkv_append(cache, none, none, table, lens, cos_sin=cs, q=none)
        assert q.shape == none.shape
        out, lse = T.tkv_attend(cache, none, table, lens, window=3)
        assert out.shape == none.shape and lse.shape == (0, 2)
    assert not pool.any()
    # an empty rotation table turns nothing, and so nothing is cached
    k = torch.ones((2, 2, 64), dtype=torch.float16, device=DEV)
    T.tkv_append(cache, k, k, ints([[0], [1]]), ints([0, 0]), cos_sin=torch.zeros((0, 64), device=DEV))
    assert not pool.any()
