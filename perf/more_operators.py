"""Cases of more operators on a paged key/value cache, and their plain forms.

A pool is pages x heads x tiles x record bytes; a record holds 32 positions of one head.  In 8 bits: K codes, V codes
(e4m3, in the order in which the matrix unit takes them), then a byte E for the keys and one for the values; an element's
value is 2^(E - 127) * code.  In 4 bits: K codes, V codes, K scales and zeros, V scales and zeros (fp16, one pair for each
position and group of channels); an element's value is scale * code + zero.

  rotate   appends new tokens' keys and values to the pages that the table names, the keys rotated by a table's cosines
           and sines of their positions, and the queries with them; reads the records that were touched back, in the
           model's type.  In 8 bits a record's E grows where new tokens need it, and the codes of its earlier positions
           are rounded again
  attend   attention of new queries over the cached positions held in 8 bits
  window   the same where a query sees only the last positions before its border and a few first ones, in 8 or 4 bits
"""
import math

import numpy as np
import torch

own = False

LIMIT = 32000.0  # largest magnitude that is cached
TILE = 32
TOP = 448.0      # largest e4m3 number
LEAST = 27       # smallest E
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _case(op, name, batch, kv_heads, group_heads, dim, page, dtype, length, new=1, bits=8, group=0, ragged=True,
          causal=True, window=0, sinks=0, turned=0, neighbours=False):
    c = dict(op=op, batch=batch, kv_heads=kv_heads, group_heads=group_heads, dim=dim, page=page, dtype=dtype,
             length=length, new=new, bits=bits, group=group, ragged=ragged, causal=causal, window=window, sinks=sinks,
             turned=turned, neighbours=neighbours)
    return dict(c, name=name) if name else c


def listed():
    return [
        # every decoding step of a served batch: one token of each sequence, its query among them
        _case("rotate", "rotate_one", 32, 8, 4, 128, 64, "bf16", 4096, turned=128),
        # prompts of many lengths enter the cache at once
        _case("rotate", "rotate_prompts", 8, 8, 4, 128, 64, "f16", 0, new=4001, turned=128),
        # a few drafted tokens, half of the channels turned as neighbouring pairs, into 4 bits
        _case("rotate", "rotate_draft_4bit", 12, 5, 3, 64, 32, "f16", 8191, new=5, bits=4, group=32, turned=32,
              neighbours=True),
        # a chat's first tokens: latency is all there is
        _case("attend", "one_token_short", 1, 8, 4, 128, 64, "bf16", 57),
        # one decoding step of an ordinary batch, lengths from a few hundred up
        _case("attend", "one_token_batch", 16, 8, 4, 128, 64, "bf16", 4099),
        # a full server: the cache is far larger than the last-level cache
        _case("attend", "one_token_full", 64, 8, 4, 128, 64, "bf16", 32768),
        # a decoder's queries over an encoder's states: no causal order, wide heads
        _case("attend", "cross_states", 8, 4, 2, 256, 32, "bf16", 1500, new=17, causal=False),
        # a chunk of a long prompt over what came before it
        _case("attend", "prompt_chunk", 2, 8, 4, 128, 64, "f16", 8192, new=512),
        # a full server that sees the last 4096 positions
        _case("window", "window_full", 64, 8, 4, 128, 64, "bf16", 32768, window=4096, sinks=4),
        # a whole prompt at once, each token over the last 1024
        _case("window", "window_prompt", 1, 8, 4, 128, 64, "bf16", 6000, new=6000, window=1024, sinks=16),
        # one user far into a stream, odd window, eight query heads to a key head
        _case("window", "window_stream", 1, 4, 8, 96, 128, "f16", 131071, ragged=False, window=1000, sinks=7),
        # a decoding step over the cache held in 4 bits
        _case("window", "window_4bit", 16, 8, 4, 128, 64, "bf16", 16384, bits=4, group=64, window=2048, sinks=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "attend", "attend", "window", "window"])
    dim = rng.choice([64, 96, 128, 128, 256])
    bits = 8 if op == "attend" else rng.choice([8, 8, 4])
    group = rng.choice([g for g in (32, 64, 128) if dim % g == 0]) if bits == 4 else 0
    page = rng.choice([32, 64, 128, 256])
    kv_heads, group_heads = _log(rng, 1, 16), _log(rng, 1, 16)
    dtype = rng.choice(["bf16", "f16"])
    batch = _log(rng, 1, 64)
    small = batch * kv_heads * dim
    if op == "rotate":
        most = max(2, min(8192, (1 << 25) // small, (1 << 27) // (small * group_heads)))
        return _case(op, None, batch, kv_heads, group_heads, dim, page, dtype, rng.choice([0, _log(rng, 1, 20000)]),
                     new=1 if rng.random() < 0.5 else _log(rng, 1, most), bits=bits, group=group,
                     turned=rng.choice([dim, dim, dim // 2]), neighbours=rng.random() < 0.3)
    products = 4 * small * group_heads  # for each position that one new token sees
    length = _log(rng, 1, max(2, min(131072, int(9e10) // products, (1 << 30) // small)))
    # the plain form multiplies with all positions, seen through the window or not
    most = max(1, min(length, int(9e10) // (products * length)))
    new = 1 if rng.random() < 0.5 else rng.randint(1, min(most, rng.choice([8, 64, 700])))
    window = _log(rng, 1, max(2, length)) if op == "window" else 0
    return _case(op, None, batch, kv_heads, group_heads, dim, page, dtype, length, new=new, bits=bits, group=group,
                 ragged=rng.random() < 0.7, causal=rng.random() < 0.8, window=window,
                 sinks=rng.choice([0, 4, _log(rng, 1, 200)]) if op == "window" else 0)


# ------------------------------------------------------------------ lengths, from the case alone

def _news(c):
    """New tokens of each sequence: ragged from c['new'] down to half of it."""
    n, b = c["new"], c["batch"]
    if not c["ragged"] or n == 1:
        return [n] * b
    return [max(1, n - (n * i) // (2 * b)) for i in range(b)]


def _lens(c):
    """Cached positions of each sequence (of attention: the new ones among them), shuffled from c['length'] to an eighth."""
    b, n = c["batch"], c["length"]
    if not c["ragged"] or b == 1:
        return [n] * b
    lens = [max(1 if n else 0, n - (7 * n * ((i * 5) % b)) // (8 * b)) for i in range(b)]
    return lens if c["op"] == "rotate" else [max(v, w) for v, w in zip(lens, _news(c))]


def _record(c):
    return 2 * TILE * c["dim"] + 128 if c["bits"] == 8 else TILE * c["dim"] + 256 * (c["dim"] // c["group"])


def _width(c):
    """Pages of the longest sequence."""
    new = _news(c) if c["op"] == "rotate" else [0] * c["batch"]
    return max(1, -(-max(a + b for a, b in zip(_lens(c), new)) // c["page"]))


def work(c):
    lens, news = _lens(c), _news(c)
    h, d, g = c["kv_heads"], c["dim"], c["group_heads"]
    # a position's codes and what goes with them: of 8 bits two bytes for 32 positions
    per = 2 * d + 2 / TILE if c["bits"] == 8 else _record(c) / TILE
    if c["op"] == "rotate":
        t = sum(news)
        back = t + (sum(v % TILE for v in lens) if c["bits"] == 8 else 0)
        return {"bytes": t * h * (4 * d + per) + t * (4 * h * g * d + 4 * c["turned"]) + back * h * (per + 4 * d),
                "flops": t * (h * d * 2 * 4 + 3 * h * (g + 1) * c["turned"])}
    read = seen = 0
    for v, w in zip(lens, news):
        first = np.arange(v - w + 1, v + 1) if c["causal"] else np.full(w, v)  # each new token's border
        low = np.maximum(first - c["window"], 0) if c["window"] else np.zeros_like(first)
        seen += int((first - low + np.minimum(low, c["sinks"])).sum())
        read += int(v - low[0] + min(low[0], c["sinks"]))
    return {"bytes": h * per * read + h * g * sum(news) * (4 * d + 4), "flops": h * g * seen * (4 * d + 4)}


# ------------------------------------------------------------------ inputs

def _pool(c, pages, gen):
    """Pages as filled from keys and values near a normal distribution."""
    d, h, record = c["dim"], c["kv_heads"], _record(c)
    n = pages * h * (c["page"] // TILE)
    pool = torch.empty((n, record), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 28) // (64 * d))
    for i in range(0, n, step):
        m = min(step, n - i)
        if c["bits"] == 8:
            x = torch.empty((m, 64 * d), dtype=torch.float16, device="cuda").normal_(0, 64, generator=gen)
            pool[i:i + m, :64 * d] = x.clamp_(-TOP, TOP).to(torch.float8_e4m3fn).view(torch.uint8)
            pool[i:i + m, 64 * d:] = torch.randint(120, 123, (m, 128), dtype=torch.uint8, device="cuda", generator=gen)
            continue
        groups = d // c["group"]
        codes = torch.empty((2, m, 32 * d), dtype=torch.float16, device="cuda").normal_(7.5, 2.6, generator=gen)
        codes = codes.round_().clamp_(0, 15).to(torch.uint8)
        pool[i:i + m, :32 * d] = codes[0] | (codes[1] << 4)
        scale = 0.2 + 0.4 * torch.rand((m, groups, 2, TILE), device="cuda", generator=gen)
        zero = -7.5 * scale + 0.1 * torch.randn((m, groups, 2, TILE), device="cuda", generator=gen)
        kp = torch.stack((scale[:, :, 0], zero[:, :, 0]), -1).half()
        vp = torch.stack((scale[:, :, 1], zero[:, :, 1]), -2).half()
        pool[i:i + m, 32 * d:] = torch.cat((kp.reshape(m, -1), vp.reshape(m, -1)), 1).view(torch.uint8)
    return pool.view(pages, h, c["page"] // TILE, record)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    b, h, d, width = c["batch"], c["kv_heads"], c["dim"], _width(c)
    dt = DTYPES[c["dtype"]]
    lens, news = _lens(c), _news(c)
    pages = b * width
    order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    s = dict(case=c, table=order.view(b, width).contiguous(), lens=_ints(lens), pool=_pool(c, pages, gen),
             starts=_ints([0] + list(np.cumsum(news))), max_new=max(news), max_len=max(lens))
    s["q"] = (2 * torch.randn((sum(news), h * c["group_heads"], d), device="cuda", generator=gen)).to(dt)
    if c["op"] != "rotate":
        return s
    spread = torch.exp(0.5 * torch.randn((2, h, d), device="cuda", generator=gen))
    centre = 0.7 * torch.randn((2, h, d), device="cuda", generator=gen)
    for i, name in enumerate("kv"):
        x = torch.randn((sum(news), h, d), device="cuda", generator=gen)
        s[name] = (x * spread[i] + centre[i]).to(dt)
    # cosines and sines of every position that there may be, made once in a program
    half = c["turned"] // 2
    angle = torch.arange(width * c["page"], dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (
        -torch.arange(half, dtype=torch.float64, device="cuda") / half)
    s["cos_sin"] = torch.cat((angle.cos(), angle.sin()), -1).float()
    # what is read back: in 8 bits from the beginning of the first record that new tokens touch
    first = [v // TILE * TILE if c["bits"] == 8 else v for v in lens]
    back = [v + n - f for v, n, f in zip(lens, news, first)]
    s.update(back_lens=_ints(first), back_starts=_ints([0] + list(np.cumsum(back))), total_back=sum(back),
             max_back=max(back))
    return s


# ------------------------------------------------------------------ plain forms

def _unpack(codes):
    """Bytes [..., 4] of words into their 8 values, in three axes: [..., low bit, high bit, middle bit] of the index."""
    return torch.stack((codes & 15, codes >> 4), -1).unflatten(-2, (2, 2)).flatten(-3).unflatten(-1, (2, 2, 2))


def _scale(e):
    """2^(E - 127), from a number's bits."""
    return (e.to(torch.int32) << 23).view(torch.float32)


def _values(raw, c):
    """Keys and values [.., heads, positions, dim] in 32 bits of records [.., heads, tiles, record]."""
    d = c["dim"]
    lead, t = raw.shape[:-2], raw.shape[-2]
    if c["bits"] == 8:
        x = raw[..., :64 * d].view(torch.float8_e4m3fn).float()
        scale = _scale(raw[..., 64 * d:64 * d + 2])[..., None, None]
        k = x[..., :32 * d].reshape(-1, 2, d // 32, 4, 16, 8).permute(0, 1, 4, 2, 3, 5).reshape(*lead, t, TILE, d)
        v = x[..., 32 * d:].reshape(-1, d // 16, 4, 16, 2, 4).permute(0, 4, 2, 5, 1, 3).reshape(*lead, t, TILE, d)
        return (k * scale[..., 0, :, :]).flatten(-3, -2), (v * scale[..., 1, :, :]).flatten(-3, -2)
    groups, words = d // c["group"], d // 32
    sub = 2 if words > 4 else 1
    w = words // sub
    k = _unpack(raw[..., :16 * d].reshape(-1, 2, sub, 4, 16, w, 4))  # half sub g m w | low high middle
    k = k.permute(0, 1, 4, 2, 5, 3, 7, 8, 6).reshape(*lead, t, TILE, groups, c["group"])
    kp = raw[..., 32 * d:32 * d + 128 * groups].contiguous().view(torch.float16).view(*lead, t, groups, TILE, 2)
    kp = kp.transpose(-3, -2).float()
    k = k * kp[..., 0, None] + kp[..., 1, None]
    v = _unpack(raw[..., 16 * d:32 * d].reshape(-1, 2, sub, 4, 16, w, 4))
    v = v.permute(0, 7, 3, 8, 6, 1, 2, 5, 4).reshape(*lead, t, TILE, groups, c["group"])
    vp = raw[..., 32 * d + 128 * groups:].contiguous().view(torch.float16).view(-1, groups, 2, 4, 2, 4)
    vp = vp.permute(0, 4, 3, 5, 1, 2).reshape(*lead, t, TILE, groups, 2).float()
    v = v * vp[..., 0, None] + vp[..., 1, None]
    return k.reshape(*lead, t * TILE, d), v.reshape(*lead, t * TILE, d)


def _turn(x, cos_sin, c):
    """x [tokens, heads, dim] in 32 bits, its first channels turned by the tokens' rows of cosines and sines."""
    half = c["turned"] // 2
    cos, sin = cos_sin[:, None, :half], cos_sin[:, None, half:]
    if c["neighbours"]:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., 2 * half:]), -1)


def _limited(x):
    return torch.nan_to_num(x, 0.0, LIMIT, -LIMIT).clamp(-LIMIT, LIMIT)


def _quantise4(x, group):
    """The values that keys or values [tokens, heads, dim] have once they are held in 4 bits."""
    shape = x.shape
    x = x.view(*shape[:2], -1, group)
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    # a tensor, as a division by a number may become a product with its reciprocal
    scale, zero = ((hi - lo) / torch.full_like(lo, 15)).half(), lo.half()
    # which code is nearest is decided in 64 bits: 32 lose what lies next to a border
    code = torch.round((x.double() - zero.double()) / scale.double()).clamp(0, 15)
    code = torch.where(scale == 0, 0.0, code)
    return (scale.float() * code.float() + zero.float()).view(shape)


def _exponent(top):
    """The smallest E with top <= 448 * 2^(E - 127)."""
    fraction, power = torch.frexp(top)
    return torch.where(top > 0, power - 9 + 127 + (fraction > 0.875).to(torch.int32), 0).clamp(min=LEAST)


def _held(x, e):
    """The values that x has once it is held as e4m3 numbers times 2^(E - 127)."""
    scale = _scale(e)
    # times the power of two's reciprocal: a quotient in 32 bits may be a step off, and many values lie on a border
    return (x * _scale(254 - e)).to(torch.float8_e4m3fn).float() * scale


def _rotate(s):
    c = s["case"]
    starts, lens = s["starts"].long(), s["lens"].long()
    row = torch.arange(s["k"].shape[0], device="cuda")
    seq = torch.searchsorted(starts, row, right=True) - 1
    pos = lens[seq] + row - starts[seq]
    cos_sin = s["cos_sin"][pos]
    k, v = _limited(_turn(s["k"].float(), cos_sin, c)), _limited(s["v"].float())
    q = _turn(s["q"].float(), cos_sin, c).to(s["q"].dtype)
    if c["bits"] == 4:
        return {"k": _quantise4(k, c["group"]).to(q.dtype), "v": _quantise4(v, c["group"]).to(q.dtype), "q": q}
    # rows of what is read back: earlier positions of the first records, then the new ones
    back = s["back_starts"].long()
    out = torch.arange(s["total_back"], device="cuda")
    at = torch.searchsorted(back, out, right=True) - 1
    where = s["back_lens"].long()[at] + out - back[at]
    new = where >= lens[at]
    token = (starts[at] + where - lens[at]).clamp(min=0)
    # the earlier positions, by the records that hold them
    page = s["table"].long()[torch.arange(lens.shape[0], device="cuda"), lens // c["page"]]
    first = s["pool"][page, :, lens % c["page"] // TILE]  # sequences, heads, record
    old = torch.stack(_values(first[:, :, None], c))      # 2, sequences, heads, 32, dim
    old = old[:, at, :, where % TILE].transpose(0, 1)     # 2, rows, heads, dim
    x = torch.where(new[None, :, None, None], torch.stack((k, v))[:, token], old)
    # E of every record: by its new positions, and at least what its earlier ones have
    per = (back[1:] - back[:-1] + TILE - 1) // TILE
    record = (per.cumsum(0) - per)[at] + (where - s["back_lens"].long()[at]) // TILE
    top = torch.zeros((2, s["total_back"], c["kv_heads"]), device="cuda")
    top.scatter_reduce_(1, record[None, :, None].expand_as(top), torch.where(new[None, :, None], x.abs().amax(-1), 0.0),
                        "amax")
    had = first[..., 64 * c["dim"]:64 * c["dim"] + 2].permute(2, 0, 1).to(torch.int32)
    had = torch.where((lens % TILE > 0)[None, :, None], had, 0)
    e = _exponent(top)[:, record]
    e = torch.where((where < (lens + TILE - 1)[at] // TILE * TILE)[None, :, None], torch.maximum(e, had[:, at]), e)
    x = _held(x, e[..., None]).to(q.dtype)
    return {"k": x[0], "v": x[1], "q": q}


def _attend(s):
    c = s["case"]
    b, h, g, d = c["batch"], c["kv_heads"], c["group_heads"], c["dim"]
    k, v = _values(s["pool"][s["table"].long()].transpose(1, 2).flatten(2, 3), c)
    n, cap = s["max_new"], k.shape[2]
    starts = s["starts"].long()
    news = starts[1:] - starts[:-1]
    i = torch.arange(n, device="cuda")
    at = (starts[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    there = i < news[:, None]
    q = s["q"].float()[at].view(b, n, h, g, d).permute(0, 2, 1, 3, 4).reshape(b, h, n * g, d)
    x = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    border = (s["lens"].long()[:, None] - (news[:, None] - 1 - i if c["causal"] else torch.zeros_like(at)))[..., None]
    p = torch.arange(cap, device="cuda")
    seen = (p < border) & there[..., None]
    if c["window"]:
        seen = seen & ((p >= border - c["window"]) | (p < c["sinks"]))
    x = x.view(b, h, n, g, cap).masked_fill_(~seen[:, None, :, None], -math.inf).view(b, h, n * g, cap)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    x = x.div_(torch.where(total == 0, 1.0, total))
    o = torch.matmul(x, v).view(b, h, n, g, d).permute(0, 2, 1, 3, 4).reshape(b, n, h * g, d)
    lse = (torch.log(total) + top).view(b, h, n, g).permute(0, 2, 1, 3).reshape(b, n, h * g)
    return {"out": o[there].to(s["q"].dtype), "lse": lse[there]}


def run(s):
    if own:
        return _own(s)
    return _rotate(s) if s["case"]["op"] == "rotate" else _attend(s)


def _own(s):
    from tiled_tensor_bulk_amd import tkv as T

    c = s["case"]
    if c["bits"] == 8:
        cache = T.tkv_encode(s["pool"], c["kv_heads"], c["dim"], c["page"], bits=8)
    else:
        cache = T.tkv_encode(s["pool"], c["kv_heads"], c["dim"], c["page"], c["group"])
    if c["op"] == "rotate":
        q = T.tkv_append(cache, s["k"], s["v"], s["table"], s["lens"], starts=s["starts"], max_new=s["max_new"],
                         cos_sin=s["cos_sin"], neighbours=c["neighbours"], q=s["q"])
        k, v = T.tkv_read(cache, s["table"], s["back_lens"], starts=s["back_starts"], max_new=s["max_back"],
                          n_tokens=s["total_back"], dtype=s["q"].dtype)
        return {"k": k, "v": v, "q": q}
    out, lse = T.tkv_attend(cache, s["q"], s["table"], s["lens"], starts=s["starts"], max_new=s["max_new"],
                            max_len=s["max_len"], causal=c["causal"], window=c["window"] or None, sinks=c["sinks"])
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ the definition in 64 bits

def _places(c):
    """For each position of a record and each channel: the byte and shift of its K code and of its V code; in 4 bits also
    the fp16 places of the scale and zero of each."""
    d = c["dim"]
    words = d // 32
    t, ch = np.meshgrid(np.arange(TILE), np.arange(d), indexing="ij")
    if c["bits"] == 8:
        kb = ((t // 16 * words + ch // 32) * 64 + ch % 32 // 8 * 16 + t % 16) * 8 + ch % 8
        vb = 32 * d + (ch // 16 * 64 + t % 16 // 4 * 16 + ch % 16) * 8 + t % 4 + t // 16 * 4
        places = [kb, vb]
    else:
        groups = d // c["group"]
        w = words if words <= 4 else words // 2

        def place(half, word, g, m, j):
            nibble = (j >> 1) + 4 * (j & 1)
            index = ((half * (words // w) + word // w) * 64 + 16 * g + m) * w + word % w
            return 4 * index + nibble // 2, 4 * (nibble % 2)

        kb, ks = place(t // 16, ch // 32, (ch % 32) // 8, t % 16, ch % 8)
        chunk = ch // 16
        vb, vs = place(chunk // words, chunk % words, (t % 16) // 4, ch % 16, (t % 4) + 4 * (t // 16))
        grp = ch // c["group"]
        kp = 16 * d + (grp * TILE + t) * 2
        vp = 16 * d + 64 * groups + grp * 64 + 8 * ((t % 16) // 4) + 4 * (t // 16) + t % 4
        places = [kb, ks, kp, kp + 1, vb + 16 * d, vs, vp, vp + TILE]
    return [torch.from_numpy(x.reshape(-1).copy()).cuda() for x in places]


def _two_to(power):
    """2^power from the number's bits, as a power function may be a step off."""
    return (power.long() + 1023 << 52).view(torch.float64)


def _double(rec, c, places):
    """Keys and values [heads, positions, dim] of records [heads, tiles, record]."""
    h, t, _ = rec.shape
    out = []
    if c["bits"] == 8:
        # a byte's number: sign, four bits of exponent, three of fraction
        byte = torch.arange(256, dtype=torch.float64, device="cuda")
        power, fraction = (byte % 128 / 8).floor(), byte % 8
        number = torch.where(power == 0, fraction * 2.0 ** -9, (8 + fraction) * _two_to(power - 10))
        number = torch.where(byte >= 128, -number, number)
        for i, at in enumerate(places):
            scale = _two_to(rec[..., 64 * c["dim"] + i].long() - 127)
            out.append((number[rec[..., at].long()] * scale[..., None]).reshape(h, t * TILE, c["dim"]))
        return out
    half = rec.view(torch.float16)
    for code, shift, scale, zero in (places[:4], places[4:]):
        x = (rec[..., code] >> shift.to(torch.uint8)) & 15
        out.append((x.double() * half[..., scale].double() + half[..., zero].double()).reshape(h, t * TILE, c["dim"]))
    return out


def _nearest(x, e):
    """x as the nearest e4m3 number times 2^(E - 127), ties to the even one."""
    scale = _two_to(e - 127)
    # a step is three bits below the first one, and 2^-9 at least
    step = _two_to(torch.frexp((x / scale).abs())[1].clamp(min=-5) - 4) * scale
    return torch.round(x / step) * step


def _exact_rotate(s, c):
    places, lens, news, half = _places(c), _lens(c), _news(c), c["turned"] // 2
    outs = {"k": [], "v": [], "q": []}
    at = 0
    for b, (n, m) in enumerate(zip(lens, news)):
        t = s["cos_sin"][n:n + m].double()[:, None]
        one = {}
        for name in "kvq":
            x = s[name][at:at + m].double()
            if name != "v":
                y = x[..., :2 * half]
                y = y.unflatten(-1, (half, 2)).mT.flatten(-2) if c["neighbours"] else y
                turn = torch.cat((-y[..., half:], y[..., :half]), -1)
                y = y * t[..., :half].repeat(1, 1, 2) + turn * t[..., half:].repeat(1, 1, 2)
                y = y.unflatten(-1, (2, half)).mT.flatten(-2) if c["neighbours"] else y
                x = torch.cat((y, x[..., 2 * half:]), -1)
            one[name] = x if name == "q" else torch.where(x.isnan(), 0.0, x).clamp(-LIMIT, LIMIT)
        at += m
        outs["q"].append(one["q"])
        if c["bits"] == 4:
            for name in "kv":
                x = one[name].unflatten(-1, (-1, c["group"]))
                lo = x.min(-1, keepdim=True).values
                step = ((x.max(-1, keepdim=True).values - lo) / 15).half().double()
                lo = lo.half().double()
                code = torch.clamp(torch.round((x - lo) / torch.where(step == 0, 1.0, step)), 0, 15) * (step != 0)
                outs[name].append((lo + step * code).flatten(-2))
            continue
        r = n % TILE
        if r:
            rec = s["pool"][s["table"][b, n // c["page"]].long(), :, n % c["page"] // TILE][:, None].contiguous()
            old = _double(rec, c, places)
        for i, name in enumerate("kv"):
            x = one[name]
            if r:
                x = torch.cat((old[i][:, :r].transpose(0, 1), x))
            x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, -x.shape[0] % TILE)).unflatten(0, (-1, TILE))
            new = x.abs().amax(-1)
            new[0, :r] = 0
            new = new.amax(1)
            fraction, power = torch.frexp(new / TOP)  # a power of two is its own ceiling
            e = torch.where(new > 0, power + 127 - (fraction == 0.5).int(), 0).clamp(min=LEAST)
            if r:
                e[0] = torch.maximum(e[0], rec[:, 0, 64 * c["dim"] + i].int())
            outs[name].append(_nearest(x, e[:, None, :, None]).flatten(0, 1)[:r + m])
    return {name: torch.cat(x) for name, x in outs.items()}


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rotate":
        return _exact_rotate(s, c)
    places, lens, news = _places(c), _lens(c), _news(c)
    g, d = c["group_heads"], c["dim"]
    outs, lses, at = [], [], 0
    for b, (n, m) in enumerate(zip(lens, news)):
        rec = s["pool"][s["table"][b].long()].transpose(0, 1).flatten(1, 2).contiguous()
        q = s["q"][at:at + m].double().unflatten(1, (-1, g)).permute(1, 2, 0, 3)  # heads, group, tokens, dim
        at += m
        border = torch.arange(n - m + 1, n + 1, device="cuda") if c["causal"] else torch.full((m,), n, device="cuda")
        p = torch.arange(n, device="cuda")
        hidden = p >= border[:, None]
        if c["window"]:
            hidden |= (p < border[:, None] - c["window"]) & (p >= c["sinks"])
        out, lse = [], []
        for h in range(c["kv_heads"]):  # one by one, as a prompt's products take much room in 64 bits
            k, v = (x[0, :n] for x in _double(rec[h:h + 1], c, places))
            for a in range(g):
                x = (q[h, a] @ k.T.contiguous() / math.sqrt(d)).masked_fill_(hidden, -math.inf)
                lse.append(torch.logsumexp(x, -1))
                out.append(x.sub_(lse[-1][:, None]).exp_() @ v)
        outs.append(torch.stack(out, 1))
        lses.append(torch.stack(lse, 1))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
