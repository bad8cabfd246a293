"""Plain numpy implementation of the 8-bit cache's format, of the rotation on the way into a cache and of attention
through a window (include/tkv.h), written from the header's formulas; shares no code with the library."""
import numpy as np

TILE = 32
LIMIT = 32000.0
TOP = 448.0


def _table():
    """the number of every e4m3 byte"""
    out = np.zeros(256)
    for b in range(256):
        power, fraction = b >> 3 & 15, b & 7
        x = fraction * 2.0 ** -9 if power == 0 else (8 + fraction) * 2.0 ** (power - 10)
        out[b] = np.nan if b & 127 == 127 else -x if b & 128 else x
    return out


NUMBER = _table()


def code_of(x):
    """the nearest e4m3 numbers' bytes, ties to the even one; |x| at most 448"""
    x = np.asarray(x, np.float64)
    size = np.abs(x)
    step = 2.0 ** (np.maximum(np.frexp(size)[1], -5) - 4)
    size = np.rint(size / step) * step
    byte = np.searchsorted(NUMBER[:127], size)
    assert (NUMBER[byte] == size).all()
    return (byte + 128 * np.signbit(x)).astype(np.uint8)


def power_for(top):
    """the smallest E of at least 27 with top <= 448 * 2^(E - 127)"""
    e = 27
    while top > TOP * 2.0 ** (e - 127):
        e += 1
    return e


def limited(x):
    return np.where(np.isnan(x), 0.0, np.clip(x, -LIMIT, LIMIT))


def turned(x, table, p, neighbours):
    """rows x float64 [heads, dim] (fp16 or bf16 numbers) of a token at position p, in fp32 steps; None: not in the table"""
    if not 0 <= p < len(table):
        return None
    half = table.shape[1] // 2
    c, s = table[p, :half].astype(np.float32), table[p, half:].astype(np.float32)
    y = x.astype(np.float32)
    a, b = (y[:, 0:2 * half:2], y[:, 1:2 * half:2]) if neighbours else (y[:, :half], y[:, half:2 * half])
    with np.errstate(invalid="ignore", over="ignore"):
        first, second = a * c - b * s, b * c + a * s
    out = y.copy()
    if neighbours:
        out[:, 0:2 * half:2], out[:, 1:2 * half:2] = first, second
    else:
        out[:, :half], out[:, half:2 * half] = first, second
    return out.astype(np.float64)


class Ref8:
    """A pool on the host: uint8 [pages, heads, tiles, record]."""

    def __init__(self, pages, heads, dim, page, rng=None):
        self.pages, self.heads, self.dim, self.page = pages, heads, dim, page
        self.record = 64 * dim + 128
        shape = (pages, heads, page // TILE, self.record)
        # bytes at random: where nothing was written there are NaNs and wild powers
        self.raw = np.zeros(shape, np.uint8) if rng is None else rng.integers(0, 256, shape, dtype=np.uint8)
        t, ch = np.meshgrid(np.arange(TILE), np.arange(dim), indexing="ij")
        self.kb = (((t // 16) * (dim // 32) + ch // 32) * 64 + 16 * (ch % 32 // 8) + t % 16) * 8 + ch % 8
        self.vb = 32 * dim + ((ch // 16) * 64 + 16 * (t % 16 // 4) + ch % 16) * 8 + t % 4 + 4 * (t // 16)

    def page_of(self, table_row, pos):
        i = pos // self.page
        p = int(table_row[i]) if 0 <= i < len(table_row) else -1
        return p if 0 <= p < self.pages else -1

    def parts(self, table_row, head, pos):
        """values at positions `pos` as tkv_ref.Ref gives them (code, scale 1, zero 0), and which positions exist"""
        pos = np.asarray(pos, np.int64)
        page = np.array([self.page_of(table_row, int(p)) for p in pos], np.int64)
        there = page >= 0
        r = self.raw[np.where(there, page, 0), head, pos % self.page // TILE]
        t, row = pos % TILE, np.arange(len(pos))[:, None]
        out = []
        for i, at in enumerate((self.kb, self.vb)):
            e = r[:, 64 * self.dim + i].astype(np.float64)[:, None]
            out.append((NUMBER[r[row, at[t]]] * np.where(e > 0, 2.0 ** (e - 127), 0.0), 1.0, 0.0))
        return out[0], out[1], there

    def append(self, table_row, first, k, v, live=None):
        """new positions first .. of one sequence: k, v float64 [n, heads, dim], already turned; live: of each token"""
        live = np.ones(len(k), bool) if live is None else live
        for p0 in range(first // TILE * TILE, first + len(k), TILE):
            page = self.page_of(table_row, p0)
            pos = np.array([p for p in range(max(first, p0), min(first + len(k), p0 + TILE)) if live[p - first]], int)
            if page < 0 or not len(pos):
                continue
            for h in range(self.heads):
                rec = self.raw[page, h, p0 % self.page // TILE]
                for i, (x, at) in enumerate(((k, self.kb), (v, self.vb))):
                    y = limited(x[pos - first, h])
                    e = power_for(np.abs(y).max())
                    if first > p0:
                        had = int(rec[64 * self.dim + i])
                        e = max(e, had)
                        old = at[:first - p0]
                        if e > had:
                            rec[old] = code_of(NUMBER[rec[old]] * 2.0 ** (had - e))
                    rec[64 * self.dim + i] = e
                    rec[at[pos - p0]] = code_of(y / 2.0 ** (e - 127))

    def live(self, table_row, n):
        """the bytes that the first n positions' values depend on, as a mask like raw"""
        mask = np.zeros(self.raw.shape, bool)
        for p in range(n):
            page = self.page_of(table_row, p)
            if page >= 0:
                m = mask[page, :, p % self.page // TILE]
                m[:, self.kb[p % TILE]] = m[:, self.vb[p % TILE]] = True
                m[:, 64 * self.dim:64 * self.dim + 2] = True
        return mask


def attend(ref, table, lens, starts, q, scale, causal, window=None, sinks=0):
    """q float64 [tokens, q_heads, dim]; ref: a Ref8 or tkv_ref.Ref.  out, lse, and the magnitudes that error bounds go by:
    for each row, the sum of p * |scale * code|, the sum of p * |v|, and the largest sum of |products| in a logit"""
    heads = ref.heads
    n, hq, dim = q.shape
    g = hq // heads
    out, lse = np.zeros((n, hq, dim)), np.full((n, hq), -np.inf)
    mag_c, mag_v, mag_x = np.zeros((n, hq, dim)), np.zeros((n, hq, dim)), np.zeros((n, hq))
    for b in range(len(lens)):
        given, new = int(lens[b]), int(starts[b + 1] - starts[b])
        length = min(given, table.shape[1] * ref.page)
        if length <= 0:
            continue
        pos = np.arange(length)
        for h in range(heads):
            (kc, ks, kz), (vc, vs, vz), there = ref.parts(table[b], h, pos)
            with np.errstate(invalid="ignore"):
                k, sc = kc * ks + kz, vc * vs
            v = sc + vz
            for i in range(new):
                border = given - new + 1 + i if causal else given
                seen = there & (pos < border)
                if window is not None:
                    seen &= (pos >= border - window) | (pos < sinks)
                if not seen.any():
                    continue
                for a in range(h * g, (h + 1) * g):
                    row = starts[b] + i, a
                    x = scale * (k[seen] @ q[row])
                    top = x.max()
                    e = np.exp(x - top)
                    p = e / e.sum()
                    lse[row] = top + np.log(e.sum())
                    out[row] = p @ v[seen]
                    mag_c[row] = p @ np.abs(sc[seen])
                    mag_v[row] = p @ (np.abs(sc[seen]) + np.abs(vz * np.ones_like(sc))[seen])
                    mag_x[row] = (abs(scale) * ((np.abs(ks * kc) + np.abs(kz))[seen] @ np.abs(q[row]))).max()
    return out, lse, (mag_c, mag_v, mag_x)
