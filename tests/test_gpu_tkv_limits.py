"""The operators on the 4-bit cache at the edges of their calls: lengths past what a table holds, lengths shrunk and outputs
written in place, streams other than the current one, batches with nothing new, a workspace made once, errors of others,
gradients, offsets past 32 bits.  The plain implementation is tests/tkv_ref.py, asked for one new token at a time;
tolerances are those of tests/test_gpu_tkv.py, and what is not a number fails."""
import numpy as np
import pytest

from tests import tkv_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from tests.test_gpu_tkv import DEV, T, a_cache, a_ref, bounds, ints, say, tables, to64, typed  # noqa: E402


def attend_by_token(ref, table, lens, starts, q, scale, causal=True):
    """out, lse, the weights [sequences, heads, positions] and the magnitudes of tkv_ref.attend, where the i-th of n new
    tokens sees positions below lens[b] - n + 1 + i (all of lens[b] if not causal) as far as the table goes."""
    n, hq, dim = q.shape
    held = table.shape[1] * ref.page
    out, lse = np.zeros((n, hq, dim)), np.full((n, hq), -np.inf)
    mags = [np.zeros((n, hq, dim)), np.zeros((n, hq, dim)), np.zeros((n, hq))]
    weights = np.zeros((len(lens), ref.heads, held))
    none = np.zeros((1, ref.heads, held))
    for b, length in enumerate(lens):
        new = starts[b + 1] - starts[b]
        for i in range(new):
            row = starts[b] + i
            sees = max(0, min(length - new + 1 + i if causal else length, held))
            o, ls, w, m = tkv_ref.attend(ref, table[b:b + 1], [sees], [0, 1], q[row:row + 1], scale, False, none)
            out[row], lse[row] = o[0], ls[0]
            weights[b] += w[0]
            for all_, one in zip(mags, m):
                all_[row] = one[0]
    return out, lse, weights, mags


def check_numbers(got, want, mags, dtype, dim):
    """As check_attend of tests/test_gpu_tkv.py, with comparisons that a NaN fails."""
    out, lse = to64(got[0]), to64(got[1])
    tol, tol_lse = bounds(want, mags, dtype, dim)
    assert np.isfinite(tol).all()
    empty = ~np.isfinite(want[1])
    assert np.array_equal(lse[empty], want[1][empty]) and (out[empty] == 0).all()
    assert np.isfinite(out).all()
    good = np.abs(out - want[0]) <= tol
    assert good.all(), (np.argwhere(~good)[:5], out[~good][:5], want[0][~good][:5], tol[~good][:5])
    assert (np.abs(lse - want[1])[~empty] <= tol_lse[~empty]).all()


def check_weights(have, weights, mags, rows, dim):
    """scores_out that began at 0"""
    worst = 2 * ((dim + 16) * 2.0 ** -24 * mags[2].max() + 2.0 ** -19)
    tol = (worst + 2.0 ** -23 + 2.0 ** -24 * rows) * weights + 1e-30
    assert (np.abs(have - weights) <= tol).all()


# ------------------------------------------------------------------ lengths past the table

PAST = [
    # dim, group, heads, group heads, dtype, lens, new tokens: 64 positions are held
    (128, 64, 2, 1, "bf16", [70, 64, 65], [8, 8, 3]),     # 8 rows: the logarithms are kept for the scores
    (128, 64, 1, 3, "f16", [70, 500, 66], [8, 8, 1]),     # 24 rows
    (64, 32, 1, 2, "bf16", [80, 40], [40, 40]),           # waves with rows of their own
    (96, 32, 1, 1, "f16", [100, 63], [60, 63]),
    (256, 64, 1, 4, "bf16", [67, 2000], [9, 12]),
    (128, 128, 1, 2, "f16", [150], [75]),                 # two blocks of rows
]


@pytest.mark.parametrize("bounded", [False, True])
@pytest.mark.parametrize("case", PAST, ids=lambda c: f"{c[0]}-{c[1]}-{c[3] * max(c[6])}")
def test_causal_lengths_past_the_table(case, bounded):
    """A sequence that has outgrown its table: its last positions do not exist, and which ones a new token sees goes by
    the length all the same.  Bounded: the table holds them, max_len does not reach them."""
    dim, group, heads, gh, dtype, lens, new = case
    say(f"past {case} {bounded}")
    rng = np.random.default_rng(sum(lens) + dim)
    page, held = 32, 64
    table, _ = tables(rng, len(lens), held // page + (2 if bounded else 0), 1)
    ref = a_ref(rng, table.size + 1, heads, dim, page, group, table, [min(n, held) for n in lens])
    cache, _ = a_cache(ref)
    starts = np.concatenate(([0], np.cumsum(new)))
    qt, q = typed(1.5 * rng.standard_normal((starts[-1], heads * gh, dim)), dtype)
    out, lse, weights, mags = attend_by_token(ref, table[:, :held // page], lens, starts, q, dim ** -0.5)
    so = torch.zeros((len(lens), heads, table.shape[1] * page), device=DEV)
    got = T.tkv_attend(cache, qt, ints(table), ints(lens), starts=ints(starts), max_new=max(new),
                       max_len=held if bounded else None, scores_out=so)
    check_numbers(got, (out, lse), mags, dtype, dim)
    have = to64(so)
    assert (have[..., held:] == 0).all()
    check_weights(have[..., :held], weights, mags, max(new) * gh, dim)


# ------------------------------------------------------------------ eviction: lengths in place

@pytest.mark.parametrize("heads,page,lens,budget,recent", [
    (64, 32, [300, 20, 301, 0, 299, 128, 129, 300], 128, 30),  # many heads: one's workgroups long after another's
    (3, 1024, [40000, 9000, 8999], 9000, 100),                 # scores read anew in each pass
    (2, 64, [70, 5], 0, 3),                                    # nothing stays
])
def test_evict_shrinks_lens_in_place(heads, page, lens, budget, recent):
    say(f"in place {heads} {lens} {budget}")
    rng = np.random.default_rng(budget)
    dim, group, n = 64, 64, len(lens)
    width, dst_width = -(-max(lens) // page), max(1, -(-budget // page))
    table, rest = tables(rng, n, width, n * dst_width)
    pool = torch.from_numpy(rng.integers(0, 256, (table.size + rest.size) * T.tkv_page_bytes_of(heads, dim, page, group),
                                         dtype=np.uint8)).to(DEV)
    scores = torch.from_numpy(rng.random((n, heads, width * page)).astype(np.float32)).to(DEV)
    results = []
    for in_place in (False, True):
        held = pool.clone()
        cache = T.tkv_encode(held, heads, dim, page, group)
        now = ints(lens)
        kept, out, sc = T.tkv_evict(cache, ints(table), now, scores, budget, recent, ints(rest.reshape(n, dst_width)),
                                    lens_out=now if in_place else None)
        assert out.tolist() == [min(x, budget) for x in lens] and (out is now) == in_place
        assert in_place or now.tolist() == lens
        results.append((kept, sc, held))
    for a, b in zip(*results):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    for b, length in enumerate(lens):
        for h in range(heads):
            want = tkv_ref.evict(length, scores[b, h].cpu().numpy(), budget, recent)
            assert results[1][0][b, h, :len(want)].tolist() == want.tolist()


# ------------------------------------------------------------------ streams

def stream_calls():
    """A cache and calls on it that make their outputs: {name: f(stream) -> outputs}, and shapes as large as those and
    the workspace."""
    rng = np.random.default_rng(31)
    heads, gh, dim, page, n = 2, 4, 64, 64, 700
    width = -(-n // page)
    table, rest = tables(rng, 2, width, 2 * 4)
    ref = a_ref(rng, table.size + rest.size, heads, dim, page, 64, table, [n, n])
    cache, pool = a_cache(ref)
    tab, lens, dst, zero = ints(table), ints([n, n - 1]), ints(rest.reshape(2, 4)), ints([0, 0])
    q, _ = typed(rng.standard_normal((2, heads * gh, dim)), "bf16")
    scores = torch.from_numpy(rng.random((2, heads, width * page)).astype(np.float32)).to(DEV)
    so = torch.zeros_like(scores)
    calls = {
        "attend": lambda s: T.tkv_attend(cache, q, tab, lens, max_len=n, scores=scores, scores_out=so, stream=s) + (so,),
        "read": lambda s: T.tkv_read(cache, tab, zero, n_tokens=2 * n, stream=s),
        "evict": lambda s: T.tkv_evict(cache, tab, lens, scores, 200, 20, dst, max_len=n, stream=s),
    }
    room = T.tkv_attend_workspace(cache, 2, heads * gh, 1, n, scores=True)
    sizes = {
        "attend": [2 * heads * gh * dim * 2, 2 * heads * gh * 4, room],
        "read": [2 * n * heads * dim * 2] * 2,
        "evict": [2 * heads * 200 * 4, 8, 2 * heads * 200 * 4],
    }
    return calls, sizes, pool


@pytest.mark.parametrize("name", ["attend", "read", "evict"])
@pytest.mark.parametrize("how", ["stream", "handle"])
def test_outputs_made_on_another_stream(name, how):
    """Memory that was given back on the current stream, with work on it still queued there, is not what a call on
    another stream writes to: neither disturbs the other."""
    say(f"stream {name} {how}")
    calls, sizes, pool = stream_calls()
    f = calls[name]
    want = [x.clone() for x in f(None)]
    side = torch.cuda.Stream()
    big = torch.randn((8192, 8192), device=DEV).bfloat16()
    other = torch.empty_like(big)
    f(side)  # whatever a first call sets up
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    blocks = [torch.zeros(n, dtype=torch.uint8, device=DEV) for n in sizes[name] for _ in range(3)]
    at = {b.data_ptr() for b in blocks}
    torch.cuda.synchronize()
    for _ in range(30):  # some 25 ms
        torch.mm(big, big, out=other)
    for b in blocks:
        b.fill_(0x55)
    del blocks, b
    got = f(side.cuda_stream if how == "handle" else side)
    side.synchronize()
    made = got[:2] if name == "attend" else got
    assert not at & {x.data_ptr() for x in made}
    with torch.cuda.stream(side):
        early = [x.cpu() for x in got]
    torch.cuda.synchronize()
    for w, e, g in zip(want, early, got):
        assert torch.equal(w.cpu(), e) and torch.equal(w, g)


def test_the_default_stream_by_its_handle():
    calls, _, _ = stream_calls()
    want = [x.clone() for x in calls["attend"](None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = calls["attend"](0)
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert torch.equal(w, g)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()


# ------------------------------------------------------------------ scores of sequences without new tokens

@pytest.mark.parametrize("from_scores", [False, True])
@pytest.mark.parametrize("gh,new", [(1, [0, 0, 0]), (2, [0, 3, 0]), (5, [0, 3, 0]), (9, [0, 9, 0])])
def test_scores_where_nothing_is_new(gh, new, from_scores):
    """scores_out is scores, or 0, for a sequence with no new token: in a batch that has none at all, and beside one
    that has some, of few rows and of many."""
    say(f"scores {gh} {new} {from_scores}")
    rng = np.random.default_rng(gh)
    heads, dim, page, lens = 2, 64, 32, [60, 1030, 0]
    table, _ = tables(rng, 3, 33)
    ref = a_ref(rng, table.size, heads, dim, page, 32, table, lens)
    cache, _ = a_cache(ref)
    starts = np.concatenate(([0], np.cumsum(new)))
    qt, q = typed(rng.standard_normal((starts[-1], heads * gh, dim)), "f16")
    base = torch.from_numpy(rng.random((3, heads, 33 * page)).astype(np.float32)).to(DEV)
    so = torch.full_like(base, 5.0)
    T.tkv_attend(cache, qt, ints(table), ints(lens), starts=ints(starts), max_new=max(new),
                 scores=base if from_scores else None, scores_out=so)
    for b, n in enumerate(lens):
        if new[b] == 0:
            assert torch.equal(so[b, :, :n], base[b, :, :n] if from_scores else torch.zeros_like(so[b, :, :n]))
        assert (so[b, :, n:] == 5.0).all()
    if starts[-1]:
        _, _, weights, mags = attend_by_token(ref, table, lens, starts, q, dim ** -0.5)
        have = to64(so[1, :, :lens[1]]) - (to64(base[1, :, :lens[1]]) if from_scores else 0.0)
        assert np.abs(have - weights[1, :, :lens[1]]).max() < 1e-5  # the sum's rounding is 2^-24 of at most 1 + 9 * 9
    else:
        st = base.clone()
        T.tkv_attend(cache, qt, ints(table), ints(lens), starts=ints(starts), max_new=0, scores=st, scores_out=st)
        assert torch.equal(st, base)


# ------------------------------------------------------------------ errors of others

def test_an_earlier_error_of_the_runtime_is_not_the_calls():
    """A HIP call of somebody else that was refused on this thread, here one that names no device, is not reported as a
    launch that failed, and stops none of a call's launches."""
    import ctypes

    hip = ctypes.CDLL("libamdhip64.so")
    calls, _, _ = stream_calls()
    want = {name: [x.clone() for x in f(None)] for name, f in calls.items()}
    torch.cuda.synchronize()
    for name, f in calls.items():
        got = None
        assert hip.hipSetDevice(4711) != 0  # stays this thread's last error
        got = f(None)
        torch.cuda.synchronize()
        for w, g in zip(want[name], got):
            assert torch.equal(w, g), name
    q = torch.ones((2, 2, 64), dtype=torch.float16, device=DEV)
    pool = torch.zeros(2 * T.tkv_page_bytes_of(2, 64, 32, 32), dtype=torch.uint8, device=DEV)
    cache, table, lens = T.tkv_encode(pool, 2, 64, 32, 32), ints([[0], [1]]), ints([0, 0])
    torch.cuda.synchronize()
    assert hip.hipSetDevice(4711) != 0
    T.tkv_append(cache, q, q, table, lens)
    torch.cuda.synchronize()
    assert pool.any()


# ------------------------------------------------------------------ a workspace made once

def test_a_workspace_serves_smaller_calls():
    """Room for the largest call of a loop is room for every other one: fewer new tokens, sequences and positions are
    split in other ways, which may take more of it than the largest call does."""
    say("workspace")
    gen = torch.Generator(device=DEV).manual_seed(5)
    heads, gh, dim, page, n, longest, most = 2, 6, 64, 1024, 3, 60000, 8
    width = -(-longest // page)
    pool = torch.empty(n * width * T.tkv_page_bytes_of(heads, dim, page, 64), dtype=torch.uint8, device=DEV)
    cache = T.tkv_encode(pool, heads, dim, page, 64)
    table = torch.randperm(n * width, device=DEV, generator=gen).to(torch.int32).view(n, width)
    k, v = (torch.randn((n * longest, heads, dim), device=DEV, generator=gen).half() for _ in range(2))
    T.tkv_append(cache, k, v, table, ints([0] * n))
    q = torch.randn((n * most, heads * gh, dim), device=DEV, generator=gen).half()
    for scored in (False, True):
        room = torch.empty(T.tkv_attend_workspace(cache, n, heads * gh, most, longest, scores=scored), dtype=torch.uint8,
                           device=DEV)
        for new, max_new, max_len in (([8, 8, 8], 8, 60000), ([8], 8, 60000), ([5], 8, 60000), ([5], 5, 60000), ([1], 1, 60000),
                                      ([1, 1, 0], 8, 60000), ([1, 1, 1], 1, 30000), ([3], 3, 2000), ([8, 1], 8, 511),
                                      ([2, 2, 1], 2, 16385)):
            b, t = len(new), sum(new)
            lens, starts = ints([max_len - i for i in range(b)]), ints(np.concatenate(([0], np.cumsum(new))))
            results = []
            for ws in (None, room):
                so = torch.zeros((b, heads, width * page), device=DEV) if scored else None
                got = T.tkv_attend(cache, q[:t], table[:b], lens, starts=starts, max_new=max_new, max_len=max_len,
                                   scores_out=so, workspace=ws)
                results.append(got + ((so,) if scored else ()))
            for x, y in zip(*results):
                assert torch.equal(x, y), (new, max_new, max_len)


# ------------------------------------------------------------------ outputs over one another, and over the queries

def test_outputs_whose_rows_overlap_are_refused():
    rng = np.random.default_rng(1)
    table, _ = tables(rng, 1, 2)
    ref = a_ref(rng, 2, 2, 64, 32, 32, table, [40])
    cache, _ = a_cache(ref)
    q = torch.ones((3, 4, 64), dtype=torch.float16, device=DEV)
    flat = torch.zeros(4096, dtype=torch.float16, device=DEV)
    for out in (q[:1].expand(3, 4, 64), q[:, :1].expand(3, 4, 64), flat.as_strided((3, 4, 64), (128, 64, 1)),
                flat.as_strided((3, 4, 64), (64, 128, 1))):
        with pytest.raises(ValueError, match="out's rows overlap"):
            T.tkv_attend(cache, q, ints(table), ints([40]), out=out)
    k = flat[:2 * 64].view(1, 2, 64).expand(3, 2, 64)
    with pytest.raises(ValueError, match="k's rows overlap"):
        T.tkv_read(cache, ints(table), ints([0]), k=k, v=k)
    # rows by heads first, and queries that are one row
    out = torch.zeros((4, 3, 64), dtype=torch.float16, device=DEV).transpose(0, 1)
    one = q[:1, :1].expand(3, 4, 64)
    T.tkv_attend(cache, one, ints(table), ints([40]), out=out)
    want, _ = T.tkv_attend(cache, q, ints(table), ints([40]))
    assert torch.equal(out, want)


@pytest.mark.parametrize("gh,new,wide,length", [(4, 1, 1, 30), (4, 1, 1, 3000), (8, 1, 600, 900), (7, 3, 1, 700), (5, 13, 1, 600),
                                                (3, 50, 1, 3000)])
def test_the_output_in_place_of_the_queries(gh, new, wide, length):
    """Every way of splitting the work reads a row of q before it, or a later kernel, writes that row."""
    say(f"in place {gh} {new} {length}")
    rng = np.random.default_rng(gh + new)
    heads, dim, page, n = 2, 128, 32, 3
    held = -(-length // page)
    table = np.full((n, held * wide), -1, np.int32)
    table[:, :held] = rng.permutation(n * held).reshape(n, held)
    ref = a_ref(rng, n * held, heads, dim, page, 64, table, [length] * n)
    cache, _ = a_cache(ref)
    q, _ = typed(rng.standard_normal((n * new, heads * gh, dim)), "bf16")
    for scored in (False, True):
        got = []
        for out in (None, q.clone()):
            so = torch.zeros((n, heads, held * wide * page), device=DEV) if scored else None
            o, lse = T.tkv_attend(cache, q if out is None else out, ints(table), ints([length, length - 5, 1]), scores_out=so,
                                  out=out)
            got.append((o, lse) + ((so,) if scored else ()))
        for x, y in zip(*got):
            assert torch.equal(x, y)


# ------------------------------------------------------------------ gradients

def test_gradients_are_refused_and_not_needed_under_no_grad():
    pool = torch.zeros(T.tkv_page_bytes_of(2, 64, 32, 32), dtype=torch.uint8, device=DEV)
    cache, table, lens = T.tkv_encode(pool, 2, 64, 32, 32), ints([[0]]), ints([0])
    x = torch.ones((1, 2, 64), dtype=torch.float16, device=DEV, requires_grad=True)
    scores = torch.zeros((1, 2, 32), device=DEV, requires_grad=True)
    for call in (lambda: T.tkv_append(cache, x, x, table, lens), lambda: T.tkv_attend(cache, x, table, lens + 1),
                 lambda: T.tkv_attend(cache, x.detach(), table, lens + 1, scores=scores, scores_out=scores.detach()),
                 lambda: T.tkv_read(cache, table, lens, k=x, v=x),
                 lambda: T.tkv_evict(cache, table, lens, scores, 5, 1, table)):
        with pytest.raises(ValueError, match="gradient"):
            call()
    with torch.no_grad():
        T.tkv_append(cache, x, x, table, lens)
        out, _ = T.tkv_attend(cache, x, table, lens + 1)
    assert torch.equal(out, torch.ones_like(out))


# ------------------------------------------------------------------ offsets past 32 bits

def test_offsets_past_32_bits():
    """Pages, token rows and scores that lie past 2^32 bytes, and 2^31 elements, of their tensors: the same answers as
    near their beginnings."""
    say("offsets")
    heads, gh, dim, page, group = 2, 2, 128, 1024, 32
    each = T.tkv_page_bytes_of(heads, dim, page, group)
    many = (9 << 30) // each
    n, new = 2, 40  # tokens before and now, of two sequences
    gen = torch.Generator(device=DEV).manual_seed(9)
    rows = torch.randn((3, n * new, heads * gh, dim), device=DEV, generator=gen).half()
    far = torch.empty((n * new, 1 << 26), dtype=torch.float16, device=DEV)  # 2^26 elements between tokens
    wide = 1 << 30
    results = []
    for high in (False, True):
        pool = torch.empty((many if high else 4) * each, dtype=torch.uint8, device=DEV)
        cache = T.tkv_encode(pool, heads, dim, page, group)
        last = cache.n_pages - 1
        table, dst = ints([[last], [last - 2]]), ints([[last - 1], [last - 3]])
        for p in (last, last - 1, last - 2, last - 3):
            pool[p * each:(p + 1) * each].zero_()

        def place(x, column=0):
            if not high:
                return x
            y = far[:, column:column + x.shape[1] * dim].unflatten(1, (x.shape[1], dim))
            y.copy_(x)
            return y

        lens = ints([0, 3])
        T.tkv_append(cache, place(rows[0][:, :heads]), rows[1][:, :heads], table, lens)
        T.tkv_append(cache, rows[0][:2, :heads], place(rows[1][:, :heads])[-2:], table, lens + new)
        lens += new + 1
        got = []
        cap = wide if high else page
        so = torch.empty((n, heads, cap), device=DEV)
        si = so.new_zeros((n, heads, 50)) + torch.arange(50, device=DEV) / 8
        so[:, :, :50] = si
        for q in (rows[2][:n], rows[2]):  # kept logarithms, and computed again
            q = place(torch.cat((q, rows[2]))[:n * new])[-q.shape[0]:]
            got += T.tkv_attend(cache, q, table, lens, max_len=50, scores=so, scores_out=so)
            out = place(torch.zeros_like(rows[2]), 4096)[-q.shape[0]:]  # beside q
            T.tkv_attend(cache, q, table, lens, max_len=50, out=out)
            got.append(out.clone())
        got.append(so[:, :, :41].clone())
        kept, left, ks = T.tkv_evict(cache, table, lens, so, 20, 4, dst, max_len=50)
        k, v = place(torch.zeros_like(rows[0][:, :heads])), torch.zeros_like(rows[0][:, :heads])
        T.tkv_read(cache, dst, ints([0, 0]), starts=ints([40, 60, 80]), max_new=20, k=k, v=v)
        got += [kept, left, ks, k[40:].clone(), v[40:].clone()]
        results.append(got)
        del pool, cache, so
    for i, (x, y) in enumerate(zip(*results)):
        assert torch.equal(x, y), i
    assert results[1][-1].any() and (results[1][-5] >= 0).all()
