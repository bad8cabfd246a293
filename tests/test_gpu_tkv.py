"""The operators on the 4-bit cache against the plain 64-bit implementation of tests/tkv_ref.py.

Codes, scales, zeros, kept positions, lengths and moved scores have to be equal.  Attention's tolerances count its
roundings: half a step of the output's type; of fp16 once for each weight and once for each V element's scale * code
(2^-11 each, relative); and for the logits fp32 sums of dim + 16 terms (2^-24 of the sum of the magnitudes each)."""
import sys

import numpy as np
import pytest

from tests import tkv_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from tiled_tensor_bulk_amd import tkv as T  # noqa: E402

DEV = "cuda:0"
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


def to64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def typed(x, dtype):
    """float64 array rounded to dtype, on the GPU, and the values that it then has"""
    t = torch.from_numpy(np.ascontiguousarray(x)).to(DT[dtype])
    return t.to(DEV), t.to(torch.float64).numpy()


def a_ref(rng, pages, heads, dim, page, group, table, lens):
    """a pool with ordinary keys and values at positions below lens and random bytes elsewhere"""
    ref = tkv_ref.Ref(pages, heads, dim, page, group, rng)
    f = ref.raw.view(np.float16)
    for b, n in enumerate(lens):
        for p0 in range(0, n, 32):
            pg = ref.page_of(table[b], p0)
            if pg < 0:
                continue
            t = np.arange(min(32, n - p0))
            r = f[pg, :, p0 % page // 32]
            for at, d in ((ref.kp, 1), (ref.vp, 32)):
                shape = (heads,) + at[t].shape
                s = (0.1 + 0.5 * rng.random(shape)).astype(np.float16)
                r[:, at[t]] = s
                r[:, at[t] + d] = (-7.5 * s + 0.3 * rng.standard_normal(shape)).astype(np.float16)
    return ref


def a_cache(ref):
    pool = torch.from_numpy(ref.raw.reshape(-1).copy()).to(DEV)
    return T.tkv_encode(pool, ref.heads, ref.dim, ref.page, ref.group), pool


def tables(rng, n_seq, width, extra=0):
    order = rng.permutation(n_seq * width + extra).astype(np.int32)
    return order[:n_seq * width].reshape(n_seq, width), order[n_seq * width:]


# ------------------------------------------------------------------ append and read

APPENDS = [
    # dim, group, page, heads, dtype, lens before, new tokens
    (128, 64, 64, 2, "bf16", [0, 5, 31, 63], [1, 1, 1, 1]),
    (128, 32, 32, 1, "f16", [0, 7, 30], [32, 29, 70]),
    (128, 128, 128, 3, "bf16", [100, 0], [3, 200]),
    (64, 32, 32, 2, "f16", [1, 40], [0, 33]),
    (64, 64, 256, 1, "bf16", [250], [9]),
    (96, 32, 64, 2, "bf16", [15, 16, 17], [2, 1, 47]),
    (256, 32, 32, 1, "f16", [3], [40]),
    (256, 64, 64, 1, "bf16", [0, 64], [64, 1]),
    (256, 128, 32, 2, "f16", [31], [2]),
]


def specials(rng, n, heads, dim, group):
    """rows of ordinary numbers, and of those that quantising has to look at"""
    x = rng.standard_normal((n, heads, dim)) * np.exp(rng.standard_normal((n, heads, dim // group)).repeat(group, -1))
    for i, v in enumerate([0.0, 1.5, np.nan, np.inf, -np.inf, 1e-7, 60000.0]):
        if i < n:
            x[i, 0, :group] = v           # a whole group alike
            x[n - 1 - i, -1, dim - 3] = v  # one element among others
    if n > 8:
        x[7, 0, :group] = np.arange(group) % 16 * 0.5 + 0.25 * (np.arange(group) % 3 == 0)  # on the borders
        x[7, 0, 0], x[7, 0, 1] = 0.0, 7.5
    return x


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: "-".join(map(str, c[:5])))
def test_append_and_read(case):
    dim, group, page, heads, dtype, lens, new = case
    say(f"append {case}")
    rng = np.random.default_rng(dim + group + page)
    width = max(-(-(a + b) // page) for a, b in zip(lens, new)) + 1
    table, _ = tables(rng, len(lens), width, 1)
    ref = tkv_ref.Ref(table.size + 1, heads, dim, page, group, rng)
    cache, pool = a_cache(ref)
    starts = np.concatenate(([0], np.cumsum(new)))
    n = int(starts[-1])
    kt, k = typed(specials(rng, n, heads, dim, group), dtype)
    vt, v = typed(specials(rng, n, heads, dim, group)[::-1], dtype)
    T.tkv_append(cache, kt, vt, ints(table), ints(lens), starts=ints(starts), max_new=max(new))
    kc, ks, kz = tkv_ref.quantise(k, group)
    vc, vs, vz = tkv_ref.quantise(v, group)
    for b in range(len(lens)):
        for i in range(new[b]):
            pos, row = lens[b] + i, starts[b] + i
            for h in range(heads):
                ref.put(ref.page_of(table[b], pos), h, pos, kc[row, h], ks[row, h], kz[row, h], vc[row, h], vs[row, h],
                        vz[row, h])
    torch.cuda.synchronize()
    assert np.array_equal(pool.cpu().numpy().reshape(ref.raw.shape), ref.raw)  # what was not named is as it was
    def values(c, s, z):
        return c * s.astype(np.float64).repeat(group, -1) + z.astype(np.float64).repeat(group, -1)
    for out in ("f32", "f16", "bf16"):
        rk, rv = T.tkv_read(cache, ints(table), ints(lens), starts=ints(starts), max_new=max(new), n_tokens=n,
                            dtype=DT[out])
        for got, want in ((rk, values(kc, ks, kz)), (rv, values(vc, vs, vz))):
            # fp32 is one rounding of the exact value, 16 bits one more: through fp32
            want = torch.from_numpy(want).to(torch.float32).to(DT[out])
            assert torch.equal(got.cpu(), want)


def test_append_strided_and_unaligned():
    rng = np.random.default_rng(5)
    n, heads, dim, page, group = 37, 2, 128, 64, 64
    table, _ = tables(rng, 1, 2)
    x = rng.standard_normal((n, 3 * heads * dim + 3))
    big, vals = typed(x, "bf16")
    results = []
    for off in (0, 3):  # keys and values inside a wider row; from element 3 on no row is 16-byte aligned
        ref = tkv_ref.Ref(2, heads, dim, page, group)
        cache, pool = a_cache(ref)
        k = big[:, off:off + heads * dim].unflatten(1, (heads, dim))
        v = big.as_strided((n, heads, dim), (big.stride(0), dim, 1), 2 * heads * dim)
        T.tkv_append(cache, k, v, ints(table), ints([0]))
        rk, rv = T.tkv_read(cache, ints(table), ints([0]), n_tokens=n, dtype=torch.float32)
        for got, at in ((rk, off), (rv, 2 * heads * dim)):
            c, s, z = tkv_ref.quantise(vals[:, at:at + heads * dim].reshape(n, heads, dim), group)
            want = c * s.astype(np.float64).repeat(group, -1) + z.astype(np.float64).repeat(group, -1)
            assert np.array_equal(to64(got), want.astype(np.float32))
        results.append(rk)
    # reading into rows of a wider tensor that are not 16-byte aligned
    wide = torch.zeros((n, heads, dim + 5), dtype=torch.float32, device=DEV)
    other = torch.zeros_like(wide)
    T.tkv_read(cache, ints(table), ints([0]), k=wide[..., 1:dim + 1], v=other[..., 2:dim + 2])
    assert torch.equal(wide[..., 1:dim + 1], results[1]) and not wide[..., 0].any() and not wide[..., dim + 1:].any()


def test_pages_outside_the_pool_do_not_exist():
    rng = np.random.default_rng(6)
    ref = tkv_ref.Ref(3, 1, 64, 32, 32, rng)
    cache, pool = a_cache(ref)
    table = np.array([[2, -1, 0], [3, 1, 2 ** 30]], np.int32)
    n = 2 * 110  # past the table's width too
    kt, k = typed(rng.standard_normal((n, 1, 64)), "f16")
    T.tkv_append(cache, kt, kt, ints(table), ints([0, 0]))
    c, s, z = tkv_ref.quantise(k, 32)
    want = np.zeros((n, 1, 64))
    for b in range(2):
        for i in range(110):
            p = ref.page_of(table[b], i)
            if p >= 0:
                row = 110 * b + i
                ref.put(p, 0, i, c[row, 0], s[row, 0], z[row, 0], c[row, 0], s[row, 0], z[row, 0])
                want[row] = c[row] * s[row].astype(np.float64).repeat(32, -1) + z[row].astype(np.float64).repeat(32, -1)
    torch.cuda.synchronize()
    assert np.array_equal(pool.cpu().numpy().reshape(ref.raw.shape), ref.raw)
    rk, rv = T.tkv_read(cache, ints(table), ints([0, 0]), n_tokens=n, dtype=torch.float32)
    assert np.array_equal(to64(rk), want.astype(np.float32)) and torch.equal(rk, rv)


# ------------------------------------------------------------------ attention

ATTENDS = [
    # dim, group, page, heads, q heads, dtype, lens (new tokens included), new tokens, causal, scores
    (128, 64, 64, 2, 8, "bf16", [1, 31, 32, 33, 100, 0], [1, 1, 1, 1, 1, 1], True, False),
    (128, 64, 64, 1, 1, "f16", [2000], [1], True, True),            # many chunks
    (128, 32, 32, 1, 5, "bf16", [700, 64, 3], [1, 1, 1], True, True),
    (128, 128, 128, 2, 6, "f16", [129, 300], [5, 3], True, True),   # 16 rows and fewer
    (128, 64, 32, 1, 3, "bf16", [90, 50], [9, 7], True, True),      # 32 rows and fewer
    (128, 64, 64, 1, 4, "f16", [333, 40, 65], [37, 40, 1], True, True),  # blocks of 64, ragged
    (128, 32, 64, 1, 7, "bf16", [300], [50], False, True),
    (64, 32, 32, 5, 15, "f16", [500, 5], [5, 5], True, False),
    (64, 64, 256, 1, 16, "bf16", [600], [1], True, True),
    (64, 64, 64, 1, 17, "bf16", [100], [3], False, True),           # rows past one tile of 16
    (64, 32, 32, 2, 2, "f16", [257], [100], True, False),
    (96, 32, 64, 2, 4, "bf16", [200, 33], [1, 1], True, True),
    (96, 32, 32, 1, 3, "f16", [150], [8], True, False),
    (96, 32, 128, 1, 1, "f16", [400], [90], False, True),
    (256, 32, 32, 1, 2, "bf16", [77, 130], [1, 1], True, True),
    (256, 64, 64, 1, 4, "f16", [200], [20], True, True),
    (256, 128, 32, 1, 8, "bf16", [140], [3], False, False),
]


def bounds(want, mags, dtype, dim):
    """tolerances of out and lse"""
    out, lse = want
    mag_c, mag_v, mag_x = mags
    logit = (dim + 16) * 2.0 ** -24 * mag_x  # fp32 sums
    weight = 2 * logit + 2.0 ** -20          # of a weight and of the denominator, exp2 and the other fp32 steps
    half = torch.finfo(DT[dtype]).eps / 2
    tol = 2 * 2.0 ** -11 * mag_c + weight[..., None] * mag_v + half * np.abs(out) * (1 + 2.0 ** -8)
    tiny = 2.0 ** -25 if dtype == "f16" else 2.0 ** -130  # half of the smallest step
    return tol * (1 + 2.0 ** -8) + tiny, logit + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0))


def check_attend(got, want, mags, dtype, dim):
    out, lse = to64(got[0]), to64(got[1])
    tol, tol_lse = bounds(want, mags, dtype, dim)
    empty = ~np.isfinite(want[1])
    assert np.array_equal(lse[empty], want[1][empty])
    assert not out[empty].any()
    bad = np.abs(out - want[0]) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], out[bad][:5], want[0][bad][:5], tol[bad][:5])
    assert (np.abs(lse - want[1])[~empty] <= tol_lse[~empty]).all()


@pytest.mark.parametrize("case", ATTENDS, ids=lambda c: "-".join(map(str, c[:6])) + f"-{c[7][0]}")
def test_attend(case):
    dim, group, page, heads, q_heads, dtype, lens, new, causal, scored = case
    say(f"attend {case}")
    rng = np.random.default_rng(sum(lens) + dim)
    width = max(-(-n // page) for n in lens) + 1
    table, _ = tables(rng, len(lens), width, 2)
    ref = a_ref(rng, table.size + 2, heads, dim, page, group, table, lens)
    cache, _ = a_cache(ref)
    starts = np.concatenate(([0], np.cumsum(new)))
    qt, q = typed(1.5 * rng.standard_normal((starts[-1], q_heads, dim)), dtype)
    scores = rng.random((len(lens), heads, width * page)).astype(np.float32) if scored else None
    out, lse, after, mags = tkv_ref.attend(ref, table, lens, starts, q, dim ** -0.5, causal, scores)
    kw = {}
    if scored:
        st = torch.from_numpy(scores).to(DEV)
        kw = dict(scores=st, scores_out=torch.full_like(st, -7.0))
    for max_len in (None, max(lens)):
        got = T.tkv_attend(cache, qt, ints(table), ints(lens), starts=ints(starts), max_new=max(new), max_len=max_len,
                           causal=causal, **kw)
        torch.cuda.synchronize()
        check_attend(got, (out, lse), mags, dtype, dim)
        if scored:
            have = to64(kw["scores_out"])
            worst = 2 * ((dim + 16) * 2.0 ** -24 * mags[2].max() + 2.0 ** -19)
            for b, n in enumerate(lens):
                w = after[b, :, :n] - scores[b, :, :n]
                tol = worst * w + 2.0 ** -23 * after[b, :, :n] + 2.0 ** -24 * max(new) * q_heads * w
                assert (np.abs(have[b, :, :n] - after[b, :, :n]) <= tol + 1e-30).all(), b
                assert (have[b, :, n:] == -7.0).all()  # other places are left alone
    if scored:  # in place, and from nothing
        T.tkv_attend(cache, qt, ints(table), ints(lens), starts=ints(starts), max_new=max(new), causal=causal,
                     scores=st, scores_out=st)
        zero = torch.full_like(st, 5.0)
        T.tkv_attend(cache, qt, ints(table), ints(lens), starts=ints(starts), max_new=max(new), causal=causal,
                     scores_out=zero)
        for b, n in enumerate(lens):
            assert torch.equal(st[b, :, :n].cpu(), kw["scores_out"][b, :, :n].cpu())
            base = torch.from_numpy(scores[b, :, :n]).to(DEV)
            assert torch.allclose(zero[b, :, :n] + base, st[b, :, :n], rtol=2.0 ** -22, atol=0)


def test_attend_without_starts_strided_and_on_another_stream():
    rng = np.random.default_rng(11)
    dim, heads, q_heads, lens = 128, 2, 4, [70, 41]
    table, _ = tables(rng, 2, 2)
    ref = a_ref(rng, 4, heads, dim, 64, 64, table, lens)
    cache, _ = a_cache(ref)
    new = 3
    big, vals = typed(rng.standard_normal((2 * new, q_heads * dim + 7)), "bf16")
    side = torch.cuda.Stream()
    for off in (0, 5):  # aligned to 16 bytes only where the row is
        q = big.as_strided((2 * new, q_heads, dim), (big.stride(0), dim, 1), off)
        want = tkv_ref.attend(ref, table, lens, [0, new, 2 * new],
                              vals[:, off:off + q_heads * dim].reshape(2 * new, q_heads, dim), 0.2, True)
        room = torch.zeros((2 * new, q_heads + 1, dim + 8), dtype=torch.bfloat16, device=DEV)
        torch.cuda.synchronize()
        got = T.tkv_attend(cache, q, ints(table), ints(lens), scale=0.2, out=room[:, 1:, 3:dim + 3], stream=side)
        side.synchronize()
        check_attend(got, want[:2], want[3], "bf16", dim)
        assert not room[:, 0].any() and not room[..., :3].any() and not room[..., dim + 3:].any()


def test_attend_skips_pages_that_do_not_exist():
    rng = np.random.default_rng(12)
    lens, new = [128, 64, 100], [2, 1, 1]
    table = np.array([[0, -1, 2, 3], [-5, 99, 0, 0], [4, 5, 6, 7]], np.int32)
    ref = a_ref(rng, 8, 1, 64, 32, 32, table, lens)
    cache, _ = a_cache(ref)
    starts = [0, 2, 3, 4]
    qt, q = typed(rng.standard_normal((4, 2, 64)), "f16")
    scores = np.zeros((3, 1, 128), np.float32)
    out, lse, after, mags = tkv_ref.attend(ref, table, lens, starts, q, 0.125, True, scores)
    so = torch.zeros((3, 1, 128), device=DEV)
    got = T.tkv_attend(cache, qt, ints(table), ints(lens), starts=ints(starts), scores_out=so)
    check_attend(got, (out, lse), mags, "f16", 64)
    assert not got[0][2].any() and torch.isinf(got[1][2]).all()  # every page is missing
    assert np.abs(to64(so) - after).max() < 1e-5


def test_attend_clamps_lengths_and_refuses_wild_starts():
    rng = np.random.default_rng(13)
    table, _ = tables(rng, 2, 2)
    ref = a_ref(rng, 4, 1, 64, 32, 64, table, [64, 64])
    cache, _ = a_cache(ref)
    qt, q = typed(rng.standard_normal((2, 1, 64)), "bf16")
    want = tkv_ref.attend(ref, table, [64, 64], [0, 1, 2], q, 0.125, False)
    got = T.tkv_attend(cache, qt, ints(table), ints([10 ** 9, 64]), causal=False)  # past the table: nothing is there
    check_attend(got, want[:2], want[3], "bf16", 64)
    out, lse = torch.zeros_like(qt), torch.zeros((2, 1), device=DEV)
    for starts in ([0, 5, 2], [-3, 0, 0], [0, -1, 0]):  # rows outside q belong to nobody
        T.tkv_attend(cache, qt, ints(table), ints([64, 64]), starts=ints(starts), out=out, lse=lse)
        assert not out.any() and not lse.any()


def test_attend_numbers_that_fp16_cannot_hold():
    """large and tiny queries in bf16, one dominant position, and a NaN or infinity in one row only"""
    rng = np.random.default_rng(14)
    dim, lens = 128, [200]
    table, _ = tables(rng, 1, 4)
    ref = a_ref(rng, 4, 1, dim, 64, 64, table, lens)
    cache, _ = a_cache(ref)
    base = rng.standard_normal((1, 6, dim))
    base[0, 0] *= 1e6   # one position takes all
    base[0, 1] *= 1e-9  # all positions alike
    base[0, 2, 0] = 3e4
    base[0, 3] = 0.0
    base[0, 4, 7] = np.nan
    base[0, 5, 9] = np.inf
    qt, q = typed(base, "bf16")
    want = tkv_ref.attend(ref, table, lens, [0, 1], q[:, :4], dim ** -0.5, True)
    out, lse = T.tkv_attend(cache, qt, ints(table), ints(lens))
    assert torch.isnan(out[0, 4:]).all() and torch.isnan(lse[0, 4:]).all()
    # row 0's logits are so large that their fp32 rounding alone may move weight: its position of the maximum decides
    check_attend((out[:, 1:4], lse[:, 1:4]), (want[0][:, 1:], want[1][:, 1:]), [m[:, 1:] for m in want[3]], "bf16", dim)
    assert abs(float(lse[0, 0]) / want[1][0, 0] - 1) < 1e-5


def test_long_context_keeps_small_weights():
    """one position outweighs each other one by 2^20, and there are 2^16 of those: fp16 weights may not lose them"""
    dim, n = 64, 1 << 16
    ref = tkv_ref.Ref(n // 1024, 1, dim, 1024, 64)
    f = ref.raw.view(np.float16)
    table = np.arange(n // 1024, dtype=np.int32)[None]
    rec = f.reshape(n // 32, -1)
    rec[:, ref.kp[:, 0]], rec[:, ref.kp[:, 0] + 1] = 0.0, 0.0
    rec[:, ref.vp[:, 0]], rec[:, ref.vp[:, 0] + 32] = 1.0, 0.0
    raw = ref.raw.reshape(n // 32, -1)
    raw[:, 16 * dim:32 * dim] = 0x11   # every V element is 1
    rec[0, ref.kp[0, 0] + 1] = 1.0     # the first position's key is all ones
    raw[0, ref.vb[0]] &= (0xF0 >> ref.vs[0]).astype(np.uint8)  # and its V is 0
    cache, _ = a_cache(ref)
    q = torch.full((1, 1, dim), 20 * np.log(2) / dim, dtype=torch.float16, device=DEV)
    out, lse = T.tkv_attend(cache, q, ints(table), ints([n]), scale=1.0)
    x = float(q[0, 0, 0]) * dim
    want = (n - 1) / (n - 1 + np.exp(x))
    # a weight is 2^-20 of the largest: 2^-13 in the kernel's scale, a normal fp16 number
    assert abs(float(out[0, 0, 5]) / want - 1) < 3 * 2.0 ** -11
    assert abs(float(lse[0, 0]) - np.log(n - 1 + np.exp(x))) < 1e-4


# ------------------------------------------------------------------ eviction

EVICTS = [
    # dim, group, page, heads, lens, budget, recent
    (128, 64, 64, 2, [100, 50, 0, 1], 50, 10),
    (128, 32, 32, 1, [2000], 777, 0),
    (128, 128, 128, 1, [300, 299], 299, 299),
    (64, 32, 32, 3, [70, 33], 32, 40),      # recent is more than the budget
    (64, 64, 256, 1, [5000], 33, 1),
    (96, 32, 64, 2, [200, 10], 65, 64),
    (256, 32, 32, 1, [90], 64, 5),
    (256, 64, 64, 1, [130], 1, 0),
    (256, 128, 32, 1, [99], 98, 3),
    (64, 64, 32, 1, [40], 0, 3),
]


def some_scores(rng, shape):
    s = np.exp(2 * rng.standard_normal(shape)).astype(np.float32)
    s = np.where(rng.random(shape) < 0.5, np.round(s), s)           # many equal
    flat = s.reshape(-1)
    pick = rng.permutation(flat.size)[:max(7, flat.size // 20)]
    flat[pick] = np.resize([np.nan, np.inf, -np.inf, -0.0, 0.0, 1e-42, -3.0], pick.size)
    return flat.reshape(shape).astype(np.float32)


@pytest.mark.parametrize("case", EVICTS, ids=lambda c: "-".join(map(str, c[:4])) + f"-{c[5]}-{c[6]}")
def test_evict(case):
    dim, group, page, heads, lens, budget, recent = case
    say(f"evict {case}")
    rng = np.random.default_rng(budget + dim)
    width, dst_width = max(-(-n // page) for n in lens) + 1, max(1, -(-budget // page))
    table, rest = tables(rng, len(lens), width, len(lens) * dst_width)
    dst = rest.reshape(len(lens), dst_width)
    ref = a_ref(rng, table.size + dst.size, heads, dim, page, group, table, lens)
    cache, pool = a_cache(ref)
    scores = some_scores(rng, (len(lens), heads, width * page))
    kept, new_lens, out = T.tkv_evict(cache, ints(table), ints(lens), torch.from_numpy(scores).to(DEV), budget, recent,
                                      ints(dst))
    torch.cuda.synchronize()
    after = tkv_ref.Ref(ref.pages, heads, dim, page, group)
    after.raw = pool.cpu().numpy().reshape(ref.raw.shape)
    assert new_lens.tolist() == [min(n, budget) for n in lens]
    for b, n in enumerate(lens):
        m = min(n, budget)
        for h in range(heads):
            want = tkv_ref.evict(n, scores[b, h], budget, recent)
            assert kept[b, h].tolist() == want.tolist() + [-1] * (budget - m)
            assert np.array_equal(out[b, h].cpu().numpy(), np.concatenate((scores[b, h, want], np.zeros(budget - m, np.float32))),
                                  equal_nan=True)
            if m:
                have, had = after.parts(dst[b], h, np.arange(m)), ref.parts(table[b], h, want)
                for x, y in zip(have[:2], had[:2]):
                    for i in range(3):
                        assert np.array_equal(x[i], y[i])
    for p in table.reshape(-1):  # the source is as it was
        assert np.array_equal(after.raw[p], ref.raw[p])


def test_evict_long_rows_of_equal_scores():
    """every score alike, and a row longer than a pass of the workgroup: the lowest positions stay"""
    heads, dim, page, n, budget = 1, 64, 256, 20000, 9001
    rng = np.random.default_rng(3)
    table, rest = tables(rng, 1, 79, 36)
    ref = tkv_ref.Ref(79 + 36, heads, dim, page, 64)
    cache, _ = a_cache(ref)
    scores = torch.ones((1, heads, 79 * page), device=DEV)
    kept, lens, out = T.tkv_evict(cache, ints(table), ints([n]), scores, budget, 1001, ints(rest[None]))
    assert torch.equal(kept[0, 0].cpu(), torch.cat((torch.arange(8000), torch.arange(n - 1001, n))).to(torch.int32))
    assert lens.tolist() == [budget] and (out == 1).all()


def test_evict_from_and_to_pages_that_do_not_exist():
    rng = np.random.default_rng(4)
    table, dst = np.array([[0, 7, 1]], np.int32), np.array([[2, -1]], np.int32)
    ref = a_ref(rng, 4, 1, 64, 32, 64, table, [96])
    cache, pool = a_cache(ref)
    scores = np.arange(96, dtype=np.float32)[None, None] * np.array([1, -1])[np.arange(96) % 2]
    kept, lens, _ = T.tkv_evict(cache, ints(table), ints([96]), torch.from_numpy(scores.astype(np.float32)).to(DEV), 40,
                                3, ints(dst))
    torch.cuda.synchronize()
    after = tkv_ref.Ref(4, 1, 64, 32, 64)
    after.raw = pool.cpu().numpy().reshape(ref.raw.shape)
    want = tkv_ref.evict(96, scores[0, 0].astype(np.float32), 40, 3)
    assert kept[0, 0].tolist() == want.tolist()
    k0, _, there = ref.parts(table[0], 0, want[:32])
    k1 = after.parts(dst[0], 0, np.arange(32))[0]
    for x, y in zip(k1, k0):
        assert np.array_equal(x[there], y[there]) and not x[~there].any()
    assert np.array_equal(after.raw[[0, 1, 3]], ref.raw[[0, 1, 3]])


# ------------------------------------------------------------------ graphs

def test_a_decoding_step_in_a_graph():
    """append, attend with scores, captured once and replayed as the lengths on the device move on"""
    rng = np.random.default_rng(21)
    heads, q_heads, dim, page, group, n_seq = 2, 6, 128, 64, 64, 3
    table, _ = tables(rng, n_seq, 3)
    lens0 = [60, 5, 127]
    ref = a_ref(rng, 9, heads, dim, page, group, table, lens0)
    cache, pool = a_cache(ref)
    steps = [rng.standard_normal((n_seq, 2 * heads + q_heads, dim)) for _ in range(4)]
    x = torch.zeros((n_seq, 2 * heads + q_heads, dim), dtype=torch.bfloat16, device=DEV)
    tab, before, after = ints(table), ints(lens0), ints([n + 1 for n in lens0])
    scores = torch.zeros((n_seq, heads, 3 * page), device=DEV)
    out, lse = torch.zeros((n_seq, q_heads, dim), dtype=torch.bfloat16, device=DEV), torch.zeros((n_seq, q_heads), device=DEV)
    ws = torch.empty(T.tkv_attend_workspace(cache, n_seq, q_heads, 1, 3 * page, scores=True), dtype=torch.uint8, device=DEV)

    def step(stream=None):
        T.tkv_append(cache, x[:, :heads], x[:, heads:2 * heads], tab, before, stream=stream)
        T.tkv_attend(cache, x[:, 2 * heads:], tab, after, scores=scores, scores_out=scores, out=out, lse=lse,
                     workspace=ws, stream=stream)

    results = []
    for graphed in (False, True):
        pool.copy_(torch.from_numpy(ref.raw.reshape(-1)).to(DEV))
        scores.zero_()
        before.copy_(ints(lens0)), after.copy_(ints([n + 1 for n in lens0]))
        if graphed:
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                step()
        got = []
        for s in steps:
            x.copy_(torch.from_numpy(s).to(torch.bfloat16).to(DEV))
            graph.replay() if graphed else step()
            torch.cuda.synchronize()
            got.append((out.clone(), lse.clone(), scores.clone(), pool.clone()))
            before += 1
            after += 1
        results.append(got)
    for a, b in zip(*results):
        for s, t in zip(a, b):
            assert torch.equal(s, t)


def test_the_same_call_gives_the_same_bits():
    rng = np.random.default_rng(22)
    lens = [900, 300]
    table, _ = tables(rng, 2, 15)
    ref = a_ref(rng, 30, 1, 128, 64, 64, table, lens)
    cache, _ = a_cache(ref)
    qt, _ = typed(rng.standard_normal((2, 4, 128)), "bf16")
    runs = []
    for _ in range(3):
        so = torch.zeros((2, 1, 960), device=DEV)
        runs.append((*T.tkv_attend(cache, qt, ints(table), ints(lens), scores_out=so), so))
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], r))
