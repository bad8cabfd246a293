"""Attention whose rows' positions go to several workgroups and are joined: windows that are dealt out evenly by the lengths,
and many rows in chunks, which with a window are another number for each block of rows, in 8 and 4 bits.  The sizes are
those of tests/tkv8_plan.py, whose paths tests/test_tkv8_plan.py asks the host for.

Against attention in 64 bits over the positions read back, whose numbers are what the cache holds (one rounding to fp32).
Tolerances count roundings: of fp16 half a step, 2^-11, of a weight, of the sum of weights that the output is divided by and
of the output, and in 4 bits of scale * (code - 8), which is at most 8 / 15 of the distance between a group's largest and
smallest value, so 16 / 15 of the largest magnitude; for a logit fp32 sums of dim + 16 terms, 2^-24 of the sum of their
magnitudes each, in 4 bits of |scale * code| + |zero|, at most |value| and twice the largest; they count for a weight and
for the denominator."""
import numpy as np
import pytest

from tests import tkv8_plan

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from tests.test_gpu_tkv import DEV, T, ints, say, tables  # noqa: E402


def filled(c, lens, gen, rng):
    """a cache with keys and values at positions below lens, bytes at random elsewhere, and what it holds"""
    table, _ = tables(rng, c.n_seq, tkv8_plan.width(c))
    size = table.size * T.tkv_page_bytes_of(c.heads, c.dim, tkv8_plan.PAGE, c.group, c.bits)
    pool = torch.randint(0, 256, (size,), dtype=torch.uint8, device=DEV, generator=gen)
    cache = T.tkv_encode(pool, c.heads, c.dim, tkv8_plan.PAGE, c.group, bits=c.bits)
    starts = np.concatenate(([0], np.cumsum(lens)))
    n = int(starts[-1])
    k, v = (torch.randn((n, c.heads, c.dim), device=DEV, generator=gen) for _ in range(2))
    # records' powers differ, and values have a mean
    step = torch.randint(-2, 2, (n // 50 + 1, c.heads, 1), device=DEV, generator=gen).repeat_interleave(50, 0)[:n]
    v = (v + 0.5) * torch.exp2(step.float())
    tb, zero = ints(table), ints([0] * c.n_seq)
    T.tkv_append(cache, k.half(), v.half(), tb, zero, starts=ints(starts), max_new=max(lens))
    rk, rv = T.tkv_read(cache, tb, zero, starts=ints(starts), n_tokens=n, max_new=max(lens), dtype=torch.float32)
    return cache, tb, [(rk[a:b], rv[a:b]) for a, b in zip(starts, starts[1:])]


def reference(c, k, v, q, n, causal):
    """q [new, heads, group_heads, dim] of a sequence of n positions; out, lse and their tolerances"""
    new, heads, dim = len(q), c.heads, c.dim
    rows = q.double().permute(1, 0, 2, 3).reshape(heads, -1, dim)
    keys, values = (x.double().permute(1, 0, 2).contiguous() for x in (k, v))
    turned = keys.transpose(1, 2).contiguous()
    scale = dim ** -0.5
    border = torch.arange(n - new + 1, n + 1, device=DEV) if causal else torch.full((new,), n, device=DEV)
    pos = torch.arange(n, device=DEV)
    seen = pos[None] < border[:, None]
    if c.window:
        seen &= (pos[None] >= border[:, None] - c.window) | (pos[None] < c.sinks)
    seen = seen.repeat_interleave(c.group_heads, 0)[None]
    x = torch.where(seen, (rows @ turned) * scale, -torch.inf)
    p = torch.softmax(x, -1)
    lse = torch.logsumexp(x, -1)
    out, size = p @ values, p @ values.abs()
    magnitude = keys.abs()
    if c.bits == 4:
        top = magnitude.unflatten(-1, (-1, c.group)).amax(-1, keepdim=True)
        magnitude = (magnitude.unflatten(-1, (-1, c.group)) + 2 * top).flatten(-2)
    sums = torch.where(seen, (rows.abs() @ magnitude.transpose(1, 2).contiguous()) * scale, 0.0).amax(-1)
    logit = (dim + 16) * 2.0 ** -24 * sums
    tol = 3 * 2.0 ** -11 * size + (2 * logit[..., None] + 2.0 ** -20) * size
    if c.bits == 4:
        tol += 2.0 ** -11 * 16 / 15 * values.abs().amax((1, 2), keepdim=True)
    tol = tol * (1 + 2.0 ** -8) + 2.0 ** -25
    tol_lse = logit + 2.0 ** -20 + 2.0 ** -22 * lse.abs()
    return [y.unflatten(1, (new, c.group_heads)).transpose(0, 1) for y in (out, lse, tol, tol_lse)]


def compare(c, lens, new, causal=(True,)):
    rng = np.random.default_rng(c.dim + c.new + c.window)
    gen = torch.Generator(device=DEV).manual_seed(c.dim + c.window)
    cache, table, held = filled(c, lens, gen, rng)
    starts = np.concatenate(([0], np.cumsum(new)))
    q = 2.0 * torch.randn((int(starts[-1]), c.heads * c.group_heads, c.dim), device=DEV, generator=gen)
    q = q.half()
    args = dict(starts=ints(starts), max_new=c.new, max_len=c.longest, window=c.window or None, sinks=c.sinks)
    room = torch.full((T.tkv_attend_workspace(cache, c.n_seq, c.heads * c.group_heads, c.new, c.longest),), 255,
                      dtype=torch.uint8, device=DEV)  # NaNs
    for way in causal:
        say(f"joined {c} causal {way}")
        out, lse = T.tkv_attend(cache, q, table, ints(lens), causal=way, workspace=room, **args)
        again, again_lse = T.tkv_attend(cache, q, table, ints(lens), causal=way, **args)
        torch.cuda.synchronize()
        assert torch.equal(out, again) and torch.equal(lse, again_lse)
        for b, n in enumerate(lens):
            rows = slice(int(starts[b]), int(starts[b + 1]))
            if new[b] == 0:
                continue
            if n == 0:
                assert not out[rows].any() and (lse[rows] == -torch.inf).all()
                continue
            want, want_lse, tol, tol_lse = reference(c, *held[b], q[rows].unflatten(1, (c.heads, c.group_heads)), n, way)
            off = (out[rows].double().unflatten(1, (c.heads, c.group_heads)) - want).abs()
            assert (off <= tol).all(), (b, n, float((off / tol).max()))
            off = (lse[rows].double().unflatten(1, (c.heads, c.group_heads)) - want_lse).abs()
            assert (off <= tol_lse).all(), (b, n, float((off / tol_lse).max()))


def name(c):
    return f"{c.bits}b-{c.dim}-{c.heads}x{c.group_heads}-{c.new}new-{c.window}+{c.sinks}"


@pytest.mark.parametrize("c", tkv8_plan.EVEN_WINDOWS, ids=name)
def test_windows_dealt_evenly(c):
    """Long, short and empty sequences, some with fewer new tokens."""
    rng = np.random.default_rng(c.dim)
    lens = [int(n) for n in rng.integers(c.new, c.longest, c.n_seq)]
    new = [c.new] * c.n_seq
    lens[:5] = [c.longest, 0, c.new, c.window + c.sinks + 1, c.longest - 31]
    new[5] = 0
    new[6] = (c.new + 1) // 2
    lens[-1] = 90
    compare(c, lens, new)


@pytest.mark.parametrize("c", tkv8_plan.MANY_ROWS + tkv8_plan.MANY_CHUNKS, ids=name)
def test_many_rows_in_chunks(c):
    lens = [c.longest, 1700, c.new + 9][:c.n_seq]
    compare(c, lens, [c.new, c.new - 3, c.new][:c.n_seq], causal=(True, False))
