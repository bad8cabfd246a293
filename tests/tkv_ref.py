"""Plain numpy implementation, in 64 bits, of the 4-bit cache's format and operators (include/tkv.h), written from the
header's formulas position by position; shares no code with the library."""
import numpy as np

TILE = 32
LIMIT = 32000.0


class Ref:
    """A pool on the host: uint8 [pages, heads, tiles, record]."""

    def __init__(self, pages, heads, dim, page, group, rng=None):
        self.pages, self.heads, self.dim, self.page, self.group = pages, heads, dim, page, group
        self.groups = dim // group
        self.record = 32 * dim + 256 * self.groups
        shape = (pages, heads, page // TILE, self.record)
        # bytes at random: where nothing was written scales are often huge, infinite or NaN
        self.raw = np.zeros(shape, np.uint8) if rng is None else rng.integers(0, 256, shape, dtype=np.uint8)
        t, ch = np.meshgrid(np.arange(TILE), np.arange(dim), indexing="ij")
        words = dim // 32
        w = words if words <= 4 else words // 2

        def place(half, word, g, m, j):
            nib = (j >> 1) + 4 * (j & 1)
            at = ((half * (words // w) + word // w) * 64 + 16 * g + m) * w + word % w
            return 4 * at + nib // 2, 4 * (nib % 2)

        self.kb, self.ks = place(t // 16, ch // 32, ch % 32 // 8, t % 16, ch % 8)
        chunk = ch // 16
        vb, self.vs = place(chunk // words, chunk % words, t % 16 // 4, ch % 16, t % 4 + 4 * (t // 16))
        self.vb = vb + 16 * dim
        tt, gg = np.meshgrid(np.arange(TILE), np.arange(self.groups), indexing="ij")
        slot = 8 * (tt % 16 // 4) + 4 * (tt // 16) + tt % 4
        half = 16 * dim  # in fp16 units
        self.kp = half + (gg * TILE + tt) * 2
        self.vp = half + 64 * self.groups + gg * 64 + slot

    def rec(self, page, head, pos):
        return self.raw[page, head, pos % self.page // TILE]

    def get(self, page, head, pos):
        """codes and pairs of one position: (k codes, k scale, k zero, v codes, v scale, v zero)"""
        r, t = self.rec(page, head, pos), pos % TILE
        f = r.view(np.float16)
        return ((r[self.kb[t]] >> self.ks[t]) & 15, f[self.kp[t]], f[self.kp[t] + 1],
                (r[self.vb[t]] >> self.vs[t]) & 15, f[self.vp[t]], f[self.vp[t] + 32])

    def put(self, page, head, pos, kc, ksc, kz, vc, vsc, vz):
        r, t = self.rec(page, head, pos), pos % TILE
        f = r.view(np.float16)
        for b, s, c in ((self.kb, self.ks, kc), (self.vb, self.vs, vc)):
            for ch in range(self.dim):
                r[b[t, ch]] = (int(r[b[t, ch]]) & (0xF0 >> s[t, ch])) | (int(c[ch]) << s[t, ch])
        f[self.kp[t]], f[self.kp[t] + 1], f[self.vp[t]], f[self.vp[t] + 32] = ksc, kz, vsc, vz

    def page_of(self, table_row, pos):
        i = pos // self.page
        p = int(table_row[i]) if i < len(table_row) else -1
        return p if 0 <= p < self.pages else -1

    def parts(self, table_row, head, pos):
        """codes, scales and zeros at positions `pos`, by whole records: two of (code [n, dim], scale, zero [n, dim]),
        and which positions exist"""
        pos = np.asarray(pos, np.int64)
        page = np.array([self.page_of(table_row, int(p)) for p in pos], np.int64)
        there = page >= 0
        r = self.raw[np.where(there, page, 0), head, pos % self.page // TILE]  # [n, record]
        f = np.ascontiguousarray(r).view(np.float16)
        t = pos % TILE
        row = np.arange(len(pos))[:, None]
        out = []
        for b, s, p, d in ((self.kb, self.ks, self.kp, 1), (self.vb, self.vs, self.vp, 32)):
            code = ((r[row, b[t]] >> s[t].astype(np.uint8)) & 15).astype(np.float64)
            scale = np.repeat(f[row, p[t]].astype(np.float64), self.group, 1)
            zero = np.repeat(f[row, p[t] + d].astype(np.float64), self.group, 1)
            out.append((code, scale, zero))
        return out[0], out[1], there


def quantise(x, group):
    """x float64 [..., dim] (values of fp16 or bf16 numbers): codes, scales, zeros"""
    x = np.where(np.isnan(x), 0.0, np.clip(x, -LIMIT, LIMIT)).reshape(*x.shape[:-1], -1, group)
    lo, hi = x.min(-1), x.max(-1)
    scale = ((hi - lo).astype(np.float32) / np.float32(15)).astype(np.float16)
    zero = lo.astype(np.float32).astype(np.float16)
    s, z = scale.astype(np.float64)[..., None], zero.astype(np.float64)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        code = np.clip(np.rint((x - z) / s), 0, 15)
    code = np.where(s == 0, 0, code).astype(np.int64)
    return code.reshape(*code.shape[:-2], -1), scale, zero


def attend(ref, table, lens, starts, q, scale, causal, scores=None):
    """q float64 [tokens, q_heads, dim].  out, lse, scores after, and the magnitudes that error bounds go by: for each
    row, the sum of p * |scale * code|, the sum of p * |v|, and the largest sum of |products| in a logit"""
    heads = ref.heads
    n, hq, dim = q.shape
    g = hq // heads
    out, lse = np.zeros((n, hq, dim)), np.full((n, hq), -np.inf)
    mag_c, mag_v, mag_x = np.zeros((n, hq, dim)), np.zeros((n, hq, dim)), np.zeros((n, hq))
    after = None if scores is None else scores.astype(np.float64).copy()
    for b in range(len(lens)):
        length, new = int(lens[b]), int(starts[b + 1] - starts[b])
        length = min(length, table.shape[1] * ref.page)
        if length <= 0:
            continue
        for h in range(heads):
            (kc, ks, kz), (vc, vs, vz), there = ref.parts(table[b], h, np.arange(length))
            with np.errstate(invalid="ignore"):
                k, sc = kc * ks + kz, vc * vs
            v = sc + vz
            for i in range(new):
                seen = there & (np.arange(length) < (length - new + 1 + i if causal else length))
                if not seen.any():
                    continue
                for a in range(h * g, (h + 1) * g):
                    x = scale * (k[seen] @ q[starts[b] + i, a])
                    top = x.max()
                    e = np.exp(x - top)
                    p = e / e.sum()
                    row = starts[b] + i, a
                    lse[row] = top + np.log(e.sum())
                    out[row] = p @ v[seen]
                    mag_c[row] = p @ np.abs(sc[seen])
                    mag_v[row] = p @ (np.abs(sc[seen]) + np.abs(vz[seen]))
                    mag_x[row] = (abs(scale) * ((np.abs(ks * kc) + np.abs(kz))[seen] @ np.abs(q[row]))).max()
                    if after is not None:
                        after[b, h, :length][seen] += p
    return out, lse, after, (mag_c, mag_v, mag_x)


def evict(length, scores, budget, recent):
    """kept positions of one (sequence, head)"""
    if length <= budget:
        return np.arange(length)
    recent = min(recent, budget)
    old = scores[:length - recent].astype(np.float64)
    old = np.where(np.isnan(old), -np.inf, old)
    nan = np.isnan(scores[:length - recent])
    order = np.lexsort((np.arange(old.size), nan, -old))  # NaN after everything, -inf included
    return np.concatenate((np.sort(order[:budget - recent]), np.arange(length - recent, length)))
