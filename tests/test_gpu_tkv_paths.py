"""The paths that the operators on the 4-bit cache choose between, on both sides of each choice; wrong arguments on a
GPU; the decoding example.  Tolerances are those of tests/test_gpu_tkv.py."""
import importlib.util
import os

import numpy as np
import pytest

from tests import tkv_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from tests.test_gpu_tkv import DEV, DT, T, a_cache, a_ref, check_attend, ints, say, tables, to64, typed  # noqa: E402


# ------------------------------------------------------------------ append: few tokens and many

@pytest.mark.parametrize("dim,group", [(64, 32), (64, 64), (96, 32), (128, 32), (128, 64), (128, 128), (256, 32),
                                       (256, 64), (256, 128)])
def test_append_few_tokens_as_many(dim, group):
    """Tokens put in one by one, four at a time and all at once leave the same bytes."""
    say(f"few tokens {dim} {group}")
    rng = np.random.default_rng(dim + group)
    n, heads, page = 41, 2, 32
    table, _ = tables(rng, 1, 3)
    kt, k = typed(rng.standard_normal((n, heads, dim)), "bf16")
    vt, v = typed(3 * rng.standard_normal((n, heads, dim)) + 1, "bf16")
    pools = []
    for step in (1, 4, n):
        ref = tkv_ref.Ref(3, heads, dim, page, group, np.random.default_rng(1))
        cache, pool = a_cache(ref)
        for at in range(0, n, step):
            m = min(step, n - at)
            T.tkv_append(cache, kt[at:at + m], vt[at:at + m], ints(table), ints([7 + at]))
        torch.cuda.synchronize()
        pools.append(pool)
    assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[2])
    kc, ks, kz = tkv_ref.quantise(k, group)
    rk, _ = T.tkv_read(cache, ints(table), ints([7]), n_tokens=n, dtype=torch.float32)
    want = kc * ks.astype(np.float64).repeat(group, -1) + kz.astype(np.float64).repeat(group, -1)
    assert np.array_equal(to64(rk), want.astype(np.float32))


def test_append_few_tokens_unaligned():
    rng = np.random.default_rng(2)
    heads, dim = 2, 128
    big, vals = typed(rng.standard_normal((3, 2 * heads * dim + 3)), "f16")
    table, _ = tables(rng, 3, 1)
    ref = tkv_ref.Ref(3, heads, dim, 64, 32)
    cache, _ = a_cache(ref)
    k = big.as_strided((3, heads, dim), (big.stride(0), dim, 1), 1)
    v = big.as_strided((3, heads, dim), (big.stride(0), dim, 1), 3 + heads * dim)
    T.tkv_append(cache, k, v, ints(table), ints([0, 17, 63]))
    rk, rv = T.tkv_read(cache, ints(table), ints([0, 17, 63]), n_tokens=3, dtype=torch.float32)
    for got, at in ((rk, 1), (rv, 3 + heads * dim)):
        c, s, z = tkv_ref.quantise(vals[:, at:at + heads * dim].reshape(3, heads, dim), 32)
        want = c * s.astype(np.float64).repeat(32, -1) + z.astype(np.float64).repeat(32, -1)
        assert np.array_equal(to64(got), want.astype(np.float32))


# ------------------------------------------------------------------ attention: rows of every kernel

ROWS = [
    # dim, group, heads, group heads, dtype, lens, new tokens, causal: rows = group heads * new tokens
    (128, 64, 1, 8, "bf16", [700, 33], [1, 1], True),       # 8: the logarithms are kept for the scores
    (128, 64, 1, 9, "f16", [700, 33], [1, 1], True),        # 9: they are computed again
    (128, 32, 1, 16, "bf16", [300], [1], True),
    (128, 128, 2, 1, "f16", [300, 64], [33, 20], True),     # 33: waves with rows of their own
    (128, 64, 1, 1, "bf16", [200], [64], False),
    (128, 64, 1, 5, "bf16", [300, 129], [13, 1], True),     # 65: eight waves' worth
    (128, 64, 1, 2, "f16", [600, 5], [65, 5], True),        # 130: two blocks
    (64, 64, 1, 3, "bf16", [100, 700], [60, 50], True),
    (64, 32, 2, 1, "f16", [64, 65], [64, 65], True),
    (96, 32, 1, 7, "bf16", [333], [21], True),
    (96, 32, 1, 5, "f16", [90, 40], [5, 5], False),
    (256, 64, 1, 1, "f16", [150], [17], True),              # 256 channels: tiles of 16 rows up to 48
    (256, 32, 1, 3, "bf16", [150, 70], [16, 2], True),
    (256, 128, 1, 7, "bf16", [210], [7], True),             # 49: waves with rows of their own
    (256, 32, 1, 4, "f16", [130, 64], [25, 3], True),
]


@pytest.mark.parametrize("case", ROWS, ids=lambda c: f"{c[0]}-{c[1]}-{c[3] * max(c[6])}")
def test_attend_rows(case):
    dim, group, heads, gh, dtype, lens, new, causal = case
    say(f"rows {case}")
    rng = np.random.default_rng(sum(lens) + dim)
    page = 32
    width = max(-(-n // page) for n in lens)
    table, _ = tables(rng, len(lens), width, 2)
    table[0, min(1, width - 1)] = -1 if width > 2 else table[0, min(1, width - 1)]  # a page that does not exist
    ref = a_ref(rng, table.size + 2, heads, dim, page, group, table, lens)
    cache, _ = a_cache(ref)
    starts = np.concatenate(([0], np.cumsum(new)))
    qt, q = typed(1.5 * rng.standard_normal((starts[-1], heads * gh, dim)), dtype)
    scores = rng.random((len(lens), heads, width * page)).astype(np.float32)
    st = torch.from_numpy(scores).to(DEV)
    out, lse, after, mags = tkv_ref.attend(ref, table, lens, starts, q, dim ** -0.5, causal, scores)
    so = torch.full_like(st, -7.0)
    got = T.tkv_attend(cache, qt, ints(table), ints(lens), starts=ints(starts), max_new=max(new), causal=causal,
                       scores=st, scores_out=so)
    check_attend(got, (out, lse), mags, dtype, dim)
    have = to64(so)
    worst = 2 * ((dim + 16) * 2.0 ** -24 * mags[2].max() + 2.0 ** -19)
    for b, n in enumerate(lens):
        w = after[b, :, :n] - scores[b, :, :n]
        tol = worst * w + 2.0 ** -23 * after[b, :, :n] + 2.0 ** -24 * max(new) * heads * gh * w
        assert (np.abs(have[b, :, :n] - after[b, :, :n]) <= tol + 1e-30).all(), b
        assert (have[b, :, n:] == -7.0).all()


EVEN = [
    # dim, group, heads, group heads, dtype, lens, new tokens, scores: the table is so wide that positions are dealt evenly
    (128, 64, 1, 4, "bf16", [2500, 33, 0, 700], [1, 1, 1, 1], True),
    (128, 64, 2, 3, "f16", [5000], [5], True),                # parts in more than one run of the joining kernel
    (128, 32, 1, 9, "bf16", [640, 1300], [2, 3], True),       # 27 rows: two tiles, weights computed again
    (128, 128, 1, 1, "f16", [513, 129, 128], [7, 0, 9], False),
    (64, 32, 1, 8, "bf16", [1000, 300], [4, 2], False),
    (64, 64, 2, 2, "f16", [90, 1100], [1, 6], True),
    (96, 32, 1, 7, "bf16", [777], [2], False),
    (256, 64, 1, 4, "f16", [300, 600], [10, 3], True),        # 40 rows: three blocks of 16, then one
    (256, 32, 1, 2, "bf16", [700], [1], False),
]


def even_batch(rng, dim, group, heads, gh, dtype, lens, new, causal, scored, width):
    page = 32
    ends = np.cumsum([0] + [-(-n // page) for n in lens])
    table = np.full((len(lens), width), -1, np.int32)
    order = rng.permutation(max(1, ends[-1])).astype(np.int32)
    for b in range(len(lens)):
        table[b, :ends[b + 1] - ends[b]] = order[ends[b]:ends[b + 1]]
    ref = a_ref(rng, order.size, heads, dim, page, group, table, lens)
    cache, pool = a_cache(ref)
    starts = np.concatenate(([0], np.cumsum(new)))
    qt, q = typed(1.5 * rng.standard_normal((starts[-1], heads * gh, dim)), dtype)
    longest = max(lens)
    scores = rng.random((len(lens), heads, longest)).astype(np.float32) if scored else None
    out, lse, after, mags = tkv_ref.attend(ref, table, lens, starts, q, dim ** -0.5, causal, scores)
    extra = {}
    if scored:
        wide = torch.zeros((len(lens), heads, width * page), device=DEV)
        wide[:, :, :longest] = torch.from_numpy(scores).to(DEV)
        extra = dict(scores=wide, scores_out=wide)
    got = T.tkv_attend(cache, qt, ints(table), ints(lens), starts=ints(starts), max_new=max(new), causal=causal, **extra)
    check_attend(got, (out, lse), mags, dtype, dim)
    if scored:
        have = to64(wide)
        worst = 2 * ((dim + 16) * 2.0 ** -24 * mags[2].max() + 2.0 ** -19)
        for b, n in enumerate(lens):
            w = after[b, :, :n] - scores[b, :, :n]
            tol = worst * w + 2.0 ** -23 * after[b, :, :n] + 2.0 ** -24 * max(new) * heads * gh * w
            assert (np.abs(have[b, :, :n] - after[b, :, :n]) <= tol + 1e-30).all(), b
            assert np.array_equal(have[b, :, n:longest], scores[b, :, n:]) and not have[b, :, longest:].any()
    return cache, qt, table, starts, got


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", EVEN, ids=lambda c: f"{c[0]}-{c[1]}-{c[3] * max(c[6])}")
def test_attend_positions_dealt_evenly(case, causal):
    dim, group, heads, gh, dtype, lens, new, scored = case
    say(f"even {case} {causal}")
    blocks = -(-gh * max(new) // 16)
    # past 8 workgroups of 512 positions for a compute unit
    width = 8 * 512 * torch.cuda.get_device_properties(0).multi_processor_count // (heads * blocks * 32 * len(lens)) * 2 + 32
    even_batch(np.random.default_rng(sum(lens) + dim), dim, group, heads, gh, dtype, lens, new, causal, scored, width)


@pytest.mark.parametrize("n,longest", [(256, 40), (200, 500), (37, 1500)])
def test_attend_even_shares_over_many_sequences(n, longest):
    """More row blocks than workgroups, empty sequences among them; the same batch with its sequences in another order
    has the same rows up to the order of sums."""
    say(f"even sequences {n} {longest}")
    rng = np.random.default_rng(n)
    lens = [int(x) for x in rng.integers(0, longest + 1, n)]
    lens[0], lens[n // 2], lens[-1] = 0, longest, 0
    new = [int(rng.integers(0, min(3, m) + 1)) for m in lens]
    new[n // 2] = 2
    even_batch(rng, 64, 64, 8, 2, "bf16", lens, new, True, False, 600)


def test_even_shares_in_a_graph():
    """The shares go by the lengths in device memory: a captured call follows them from replay to replay, and gives the
    same bits as an eager one."""
    say("even graph")
    rng = np.random.default_rng(3)
    n, heads, gh, dim, page, width = 3, 2, 4, 128, 32, 24000
    held = 1300 // page + 1
    table = np.full((n, width), -1, np.int32)
    table[:, :held] = rng.permutation(n * held).reshape(n, held)
    ref = a_ref(rng, n * held, heads, dim, page, 64, table, [1300] * n)
    cache, pool = a_cache(ref)
    tab, lens = ints(table), ints([700, 1, 64])
    qt, q = typed(rng.standard_normal((n, heads * gh, dim)), "bf16")
    out, lse = torch.empty_like(qt), torch.empty((n, heads * gh), device=DEV)
    ws = torch.empty(T.tkv_attend_workspace(cache, n, heads * gh, 1, width * page), dtype=torch.uint8, device=DEV)
    T.tkv_attend(cache, qt, tab, lens, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        T.tkv_attend(cache, qt, tab, lens, out=out, lse=lse, workspace=ws)
    for now in ([700, 1, 64], [1300, 1299, 1], [0, 1300, 0], [0, 0, 0], [129, 128, 127]):
        lens.copy_(ints(now))
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        eager = T.tkv_attend(cache, qt, tab, lens)
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])
        o, ls, _, mags = tkv_ref.attend(ref, table, now, np.arange(n + 1), q, dim ** -0.5, True)
        check_attend((out, lse), (o, ls), mags, "bf16", dim)


@pytest.mark.parametrize("n,length", [(1, 512), (1, 513), (2, 900), (9, 2100)])
def test_attend_chunks_by_how_many_there_are(n, length):
    """One chunk, chunks of 256 and of 512."""
    say(f"chunks {n} {length}")
    rng = np.random.default_rng(length)
    heads, gh, dim, page = 8, 2, 64, 64
    lens = [length - 5 * i for i in range(n)]
    table, _ = tables(rng, n, -(-length // page))
    ref = a_ref(rng, table.size, heads, dim, page, 64, table, lens)
    cache, _ = a_cache(ref)
    qt, q = typed(rng.standard_normal((n, heads * gh, dim)), "f16")
    out, lse, _, mags = tkv_ref.attend(ref, table, lens, np.arange(n + 1), q, dim ** -0.5, True)
    check_attend(T.tkv_attend(cache, qt, ints(table), ints(lens), max_len=length), (out, lse), mags, "f16", dim)


@pytest.mark.parametrize("gh,new", [(2, 5), (3, 40)])
def test_rows_that_see_nothing(gh, new):
    """More new tokens than cached positions: the first of them see none."""
    rng = np.random.default_rng(gh)
    lens = [3, new - 1]
    table, _ = tables(rng, 2, 2)
    ref = a_ref(rng, 4, 1, 128, 32, 64, table, lens)
    cache, _ = a_cache(ref)
    qt, q = typed(rng.standard_normal((2 * new, gh, 128)), "bf16")
    scores = np.zeros((2, 1, 64), np.float32)
    want = tkv_ref.attend(ref, table, lens, [0, new, 2 * new], q, 128 ** -0.5, True, scores)
    so = torch.zeros((2, 1, 64), device=DEV)
    got = T.tkv_attend(cache, qt, ints(table), ints(lens), scores_out=so)
    assert np.isneginf(want[1]).any()
    check_attend(got, want[:2], want[3], "bf16", 128)
    assert np.abs(to64(so) - want[2]).max() < 1e-5


@pytest.mark.parametrize("scale", [-0.11, 0.0, 1e-30])
@pytest.mark.parametrize("new", [1, 30])
def test_scales_of_any_sign(scale, new):
    rng = np.random.default_rng(new)
    lens = [new + 70]
    table, _ = tables(rng, 1, 4)
    ref = a_ref(rng, 4, 1, 64, 32, 32, table, lens)
    cache, _ = a_cache(ref)
    qt, q = typed(rng.standard_normal((new, 3, 64)), "f16")
    scores = np.zeros((1, 1, 128), np.float32)
    want = tkv_ref.attend(ref, table, lens, [0, new], q, scale, True, scores)
    so = torch.zeros((1, 1, 128), device=DEV)
    got = T.tkv_attend(cache, qt, ints(table), ints(lens), scale=scale, scores_out=so)
    check_attend(got, want[:2], want[3], "f16", 64)
    assert np.abs(to64(so) - want[2]).max() < 1e-4


def exact(cache, table, lens, q, group_heads, heads, causal):
    """out and lse in 64 bits on the GPU for some heads of a cache that was filled with tkv_append: what tkv_read
    gives is a fp32 rounding of each element."""
    n, dim = q.shape[0] // len(lens), q.shape[2]
    outs, lses = [], []
    for b, length in enumerate(lens):
        k, v = T.tkv_read(cache, table[b:b + 1], torch.zeros(1, dtype=torch.int32, device=DEV), n_tokens=length,
                          dtype=torch.float32)
        for h in heads:
            x = q[b * n:(b + 1) * n, h * group_heads:(h + 1) * group_heads].double() @ k[:, h].double().T.contiguous()
            x = x * dim ** -0.5
            if causal:
                ahead = torch.arange(length, device=DEV) > torch.arange(length - n, length, device=DEV)[:, None]
                x = x.masked_fill(ahead[:, None], -torch.inf)
            lse = torch.logsumexp(x, -1)
            outs.append(torch.exp(x - lse[..., None]) @ v[:, h].double())
            lses.append(lse)
    return torch.stack(outs), torch.stack(lses)


@pytest.mark.parametrize("heads,gh,length,new,page", [
    (700, 1, 5000, 1, 32),    # more pages in a chunk than a wave holds at once
    (1, 4, 60001, 1, 1024),   # many chunks of a row
    (1, 2, 20011, 40, 32),    # the same where waves have rows of their own
    (3, 1, 9000, 300, 64),
])
def test_long_contexts(heads, gh, length, new, page):
    say(f"long {heads} {gh} {length} {new} {page}")
    dim = 64
    gen = torch.Generator(device=DEV).manual_seed(length)
    pages = -(-length // page)
    pool = torch.empty(pages * T.tkv_page_bytes_of(heads, dim, page, 64), dtype=torch.uint8, device=DEV)
    cache = T.tkv_encode(pool, heads, dim, page, 64)
    table = torch.randperm(pages, device=DEV, generator=gen).to(torch.int32)[None]
    k, v = (torch.randn((length, heads, dim), device=DEV, generator=gen).half() for _ in range(2))
    T.tkv_append(cache, k, v, table, ints([0]))
    q = torch.randn((new, heads * gh, dim), device=DEV, generator=gen).bfloat16()
    scores = torch.zeros((1, heads, pages * page), device=DEV)
    out, lse = T.tkv_attend(cache, q, table, ints([length]), max_len=length, scores_out=scores)
    some = sorted({0, heads // 2, heads - 1})
    want, want_lse = exact(cache, table, [length], q, gh, some, True)
    for i, h in enumerate(some):
        got = out[:, h * gh:(h + 1) * gh].double()
        # half a step of bf16, and what fp16 weights and values leave of sums of thousands of them
        assert ((got - want[i]).abs() <= 2.0 ** -8 * want[i].abs() + 2.0 ** -10).all()
        assert ((lse[:, h * gh:(h + 1) * gh].double() - want_lse[i]).abs() <= 2.0 ** -17 * want_lse[i].abs()).all()
        # each row's weights add up to 1
        assert abs(float(scores[0, h].double().sum()) / (new * gh) - 1) < 1e-5
    assert not scores[..., length:].any()


# ------------------------------------------------------------------ eviction: rows of every length

@pytest.mark.parametrize("length,budget,recent,cap", [(3000, 1000, 100, 3001), (4200, 64, 0, 4200), (33001, 9000, 33, 33024),
                                                      (40007, 40006, 5, 40035)])
def test_evict_lengths(length, budget, recent, cap):
    """Scores in registers of every size and read anew, at rows that are aligned and not."""
    say(f"evict {length} {budget}")
    heads, dim, page = 3, 64, 1024
    width, out_width = -(-max(length, cap) // page), -(-budget // page)
    rng = np.random.default_rng(length)
    pool = torch.zeros((width + out_width) * T.tkv_page_bytes_of(heads, dim, page, 64), dtype=torch.uint8, device=DEV)
    cache = T.tkv_encode(pool, heads, dim, page, 64)
    scores = np.exp(rng.standard_normal((1, heads, cap))).astype(np.float32)
    scores = np.where(rng.random(scores.shape) < 0.7, np.round(scores, 1), scores).astype(np.float32)
    kept, lens, out = T.tkv_evict(cache, ints(np.arange(width)[None]), ints([length]), torch.from_numpy(scores).to(DEV),
                                  budget, recent, ints(np.arange(width, width + out_width)[None]), max_len=length)
    for h in range(heads):
        want = tkv_ref.evict(length, scores[0, h], budget, recent)
        assert np.array_equal(kept[0, h].cpu().numpy(), want)
        assert np.array_equal(out[0, h].cpu().numpy(), scores[0, h, want])
    assert lens.tolist() == [budget]


# ------------------------------------------------------------------ nothing to do, and what is refused

def test_nothing_to_do():
    pool = torch.zeros(T.tkv_page_bytes_of(2, 64, 32, 32), dtype=torch.uint8, device=DEV)
    cache = T.tkv_encode(pool, 2, 64, 32, 32)
    none = torch.zeros((0, 2, 64), dtype=torch.float16, device=DEV)
    table, lens = ints([[0]]), ints([0])
    T.tkv_append(cache, none, none, table, lens)
    k, v = T.tkv_read(cache, table, lens, n_tokens=0)
    assert k.shape == (0, 2, 64) == v.shape
    out, lse = T.tkv_attend(cache, none, table, lens)
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    empty = torch.zeros((0, 1), dtype=torch.int32, device=DEV)
    T.tkv_append(cache, none, none, empty, ints([]))
    q = torch.ones((1, 2, 64), dtype=torch.float16, device=DEV)
    out, lse = T.tkv_attend(cache, q, table, lens)
    assert not out.any() and torch.isneginf(lse).all()
    kept, lens, scores = T.tkv_evict(cache, table, lens, torch.zeros((1, 2, 32), device=DEV), 0, 4, table)
    assert kept.shape == (1, 2, 0) and lens.tolist() == [0] and scores.shape == (1, 2, 0)


def test_wrong_arguments_are_value_errors():
    pool = torch.zeros(4 * T.tkv_page_bytes_of(2, 64, 32, 32), dtype=torch.uint8, device=DEV)
    cache = T.tkv_encode(pool, 2, 64, 32, 32)
    k = torch.zeros((2, 2, 64), dtype=torch.float16, device=DEV)
    table, lens = ints([[0, 1], [2, 3]]), ints([0, 0])
    good = dict(table=table, lens=lens)

    def refuses(match, f, *args, **kw):
        with pytest.raises(ValueError, match=match):
            f(cache, *args, **kw)

    for f, args in ((T.tkv_append, (k, k)), (T.tkv_attend, (k,))):
        refuses("int32", f, *args, table=table.long(), lens=lens)
        refuses("int32", f, *args, table=table, lens=lens.float())
        refuses("GPU", f, *args, table=table.cpu(), lens=lens)
        refuses("sequences", f, *([torch.cat((k, k[:1]))] * len(args)), **good)
        refuses("pages", f, *args, table=table[:1], lens=lens)
        refuses("overlap", f, *args, table=table[:1].expand(2, 2), lens=lens)
        refuses("starts", f, *args, starts=ints([0, 2]), **good)
        refuses("range", f, *args, max_new=1 << 40, **good)
        refuses("float16", f, *[x.float() for x in args], **good)
        refuses("heads", f, *[x[..., :32] for x in args], **good)
        refuses("contiguous", f, *[x.transpose(1, 2).contiguous().transpose(1, 2) for x in args], **good)
        refuses("GPU", f, *[x.cpu() for x in args], **good)
    refuses("tokens", T.tkv_append, k, k[:1], **good)
    refuses("both", T.tkv_read, k=k, **good)
    refuses("n_tokens", T.tkv_read, **good)
    refuses("must be one of", T.tkv_read, n_tokens=2, dtype=torch.int32, **good)
    refuses("lse", T.tkv_attend, k, lse=torch.zeros((2, 3), device=DEV), **good)
    refuses("out", T.tkv_attend, k, out=k.bfloat16(), **good)
    refuses("scores", T.tkv_attend, k, scores=torch.zeros((2, 2, 64), device=DEV), **good)
    refuses("contiguous", T.tkv_attend, k, scores_out=torch.zeros((2, 2, 63), device=DEV), **good)
    refuses("workspace", T.tkv_attend, k, scores_out=torch.zeros((2, 2, 64), device=DEV),
            workspace=torch.zeros(4, device=DEV), **good)
    refuses("negative", T.tkv_evict, table, lens, torch.zeros((2, 2, 64), device=DEV), -1, 0, table)
    refuses("kept", T.tkv_evict, table, lens, torch.zeros((2, 2, 64), device=DEV), 2, 0, table,
            kept=torch.zeros((2, 2, 3), dtype=torch.int32, device=DEV))
    with pytest.raises(T.TmapError, match="workspace"):
        T.tkv_attend(cache, k, table, lens, scores_out=torch.zeros((2, 2, 64), device=DEV),
                     workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(T.TmapError, match="q_heads"):
        T.tkv_attend(cache, torch.zeros((2, 3, 64), dtype=torch.float16, device=DEV), table, lens)
    with pytest.raises(ValueError, match="multiple"):
        T.tkv_encode(pool[:-1], 2, 64, 32, 32)


def test_the_decoding_example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_4bit.py")
    spec = importlib.util.spec_from_file_location("decode_4bit", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    err, worst = example.main(["--batch", "2", "--heads", "2", "--prompt", "300", "--steps", "9", "--budget", "200",
                               "--recent", "50"])
    # 4 bits round to half a step of a range of 64 normal numbers, about 5 / 15: an error near 0.1 of each element
    assert err < 0.2 and worst < 0.3
