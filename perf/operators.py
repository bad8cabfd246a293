"""Cases of the operators on a paged key/value cache held in 4 bits, and their plain forms.

A pool is pages x heads x tiles x record bytes.  A record holds 32 positions of one head: K codes, V codes
(4 bits each, in the order in which the matrix unit takes them), K scales and zeros, V scales and zeros (fp16,
one pair for each position and group of channels).  An element's value is scale * code + zero.

  append   quantises new tokens' keys and values into the pages that the table names, and reads them back
  attend   attention of new queries over the cached positions; with weights, also the sum of each cached
           position's attention weights added to its running score
  evict    keeps the last positions and those of the largest scores, moves them into other pages, and reads
           what these then hold
"""
import math

import numpy as np
import torch

own = False

LIMIT = 32000.0  # largest magnitude that is quantised: 15 * scale stays inside fp16
TILE = 32
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _case(op, name, batch, kv_heads, group_heads, dim, page, group, dtype, length, new=1, ragged=True, causal=True,
          weights=False, budget=0, recent=0):
    c = dict(op=op, batch=batch, kv_heads=kv_heads, group_heads=group_heads, dim=dim, page=page, group=group,
             dtype=dtype, length=length, new=new, ragged=ragged, causal=causal, weights=weights, budget=budget,
             recent=recent)
    return dict(c, name=name) if name else c


def listed():
    return [
        # every decoding step of a served batch adds one token to each sequence
        _case("append", "append_one", 32, 8, 4, 128, 64, 64, "bf16", 4096),
        # prompts of many lengths enter the cache at once
        _case("append", "append_prompts", 8, 8, 4, 128, 64, 64, "f16", 0, new=4001),
        # a chat's first tokens: latency is all there is
        _case("attend", "one_token_short", 1, 8, 4, 128, 64, 64, "bf16", 57),
        # one decoding step of an ordinary batch, lengths from a few hundred up
        _case("attend", "one_token_batch", 16, 8, 4, 128, 64, 64, "bf16", 4099),
        # one user with a very long context, eight query heads to a key head
        _case("attend", "one_token_long", 1, 4, 8, 128, 128, 64, "f16", 131071, ragged=False),
        # a full server: the cache is far larger than the last-level cache
        _case("attend", "one_token_full", 64, 8, 4, 128, 64, 64, "bf16", 32768),
        # the same step where the scores that eviction goes by are kept up to date
        _case("attend", "one_token_scored", 16, 8, 4, 128, 64, 64, "bf16", 16384, weights=True),
        # a few drafted tokens checked at once, odd head count, small heads
        _case("attend", "draft_check", 12, 5, 3, 64, 32, 32, "f16", 8191, new=5),
        # a decoder's queries over an encoder's states: no causal order, wide heads
        _case("attend", "cross_states", 8, 4, 2, 256, 32, 128, "bf16", 1500, new=17, causal=False),
        # a chunk of a long prompt over what came before it, scored for eviction
        _case("attend", "prompt_chunk", 2, 8, 4, 128, 64, 64, "bf16", 8192, new=512, weights=True),
        # one small sequence is halved
        _case("evict", "evict_one", 1, 8, 4, 128, 64, 64, "bf16", 1000, budget=500, recent=64, ragged=False),
        # a batch of long sequences shrinks to a quarter
        _case("evict", "evict_batch", 8, 8, 4, 128, 64, 64, "bf16", 32768, budget=8192, recent=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "evict"])
    dim = rng.choice([64, 96, 128, 128, 256])
    group = rng.choice([g for g in (32, 64, 128) if dim % g == 0])
    page = rng.choice([32, 64, 128, 256])
    kv_heads, group_heads = _log(rng, 1, 16), _log(rng, 1, 16)
    dtype = rng.choice(["bf16", "f16"])
    batch = _log(rng, 1, 64)
    small = batch * kv_heads * dim
    if op == "append":
        new = 1 if rng.random() < 0.5 else _log(rng, 1, max(2, min(8192, (1 << 25) // small)))
        return _case(op, None, batch, kv_heads, group_heads, dim, page, group, dtype,
                     rng.choice([0, _log(rng, 1, 20000)]), new=new)
    products = 4 * small * group_heads  # of attend, for each position that one new token sees
    length = _log(rng, 1, max(2, min(131072, int(9e10) // products if op == "attend" else 131072,
                                     (1 << (30 if op == "attend" else 28)) // small)))
    if op == "evict":
        budget = max(1, int(length * rng.uniform(0.05, 1.1)))
        return _case(op, None, batch, kv_heads, group_heads, dim, page, group, dtype, length, budget=budget,
                     recent=int(budget * rng.uniform(0, 1)), ragged=rng.random() < 0.7)
    most = max(1, min(length, int(9e10) // (products * length)))
    new = 1 if rng.random() < 0.5 else rng.randint(1, min(most, rng.choice([8, 64, 700])))
    return _case(op, None, batch, kv_heads, group_heads, dim, page, group, dtype, length, new=new,
                 ragged=rng.random() < 0.7, causal=rng.random() < 0.8, weights=rng.random() < 0.4)


# ------------------------------------------------------------------ lengths, from the case alone

def _news(c):
    """New tokens of each sequence: ragged from c['new'] down to half of it."""
    n, b = c["new"], c["batch"]
    if not c["ragged"] or n == 1:
        return [n] * b
    return [max(1, n - (n * i) // (2 * b)) for i in range(b)]


def _lens(c):
    """Cached positions of each sequence (of attend: the new ones among them), shuffled from c['length'] to an eighth."""
    b, n = c["batch"], c["length"]
    if not c["ragged"] or b == 1:
        return [n] * b
    lens = [max(1 if n else 0, n - (7 * n * ((i * 5) % b)) // (8 * b)) for i in range(b)]
    return [max(v, w) for v, w in zip(lens, _news(c))] if c["op"] == "attend" else lens


def _shape(c):
    groups = c["dim"] // c["group"]
    record = TILE * c["dim"] + 256 * groups
    if c["op"] == "append":
        top = max(a + b for a, b in zip(_lens(c), _news(c)))
    else:
        top = max(_lens(c))
    return groups, record, max(1, -(-top // c["page"]))


def work(c):
    groups, record, _ = _shape(c)
    lens, news = _lens(c), _news(c)
    h, d, per = c["kv_heads"], c["dim"], record / TILE
    if c["op"] == "append":
        t = sum(news)
        return {"bytes": t * h * (2 * d * 2 + 2 * per + 2 * d * 4), "flops": t * h * d * 2 * 6}
    if c["op"] == "evict":
        n = sum(min(v, c["budget"]) for v in lens)
        return {"bytes": h * (4 * sum(lens) + n * (3 * per + 4 + 2 * d * 2)) + 4 * c["batch"] * h * 2 * c["budget"],
                "flops": h * sum(lens) * 8}
    rows = c["group_heads"]
    seen = sum(w * v - (w * (w - 1) // 2 if c["causal"] else 0) for v, w in zip(lens, news))
    products = 6 if c["weights"] else 4  # the weights need each row's last sum first
    b = h * per * sum(lens) + h * rows * sum(news) * (4 * d + 4) + (8 * h * sum(lens) if c["weights"] else 0)
    return {"bytes": b, "flops": h * rows * seen * (4 * d + products)}


# ------------------------------------------------------------------ inputs

def _pool(c, pages, gen):
    """Pages as filled from keys and values near a normal distribution."""
    groups, record, _ = _shape(c)
    d = c["dim"]
    n = pages * c["kv_heads"] * (c["page"] // TILE)
    pool = torch.empty((n, record), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 28) // (32 * d))
    for i in range(0, n, step):
        m = min(step, n - i)
        codes = torch.empty((2, m, 32 * d), dtype=torch.float16, device="cuda").normal_(7.5, 2.6, generator=gen)
        codes = codes.round_().clamp_(0, 15).to(torch.uint8)
        pool[i:i + m, :32 * d] = codes[0] | (codes[1] << 4)
        scale = 0.2 + 0.4 * torch.rand((m, groups, 2, TILE), device="cuda", generator=gen)
        zero = -7.5 * scale + 0.1 * torch.randn((m, groups, 2, TILE), device="cuda", generator=gen)
        kp = torch.stack((scale[:, :, 0], zero[:, :, 0]), -1).half()
        vp = torch.stack((scale[:, :, 1], zero[:, :, 1]), -2).half()
        both = torch.cat((kp.reshape(m, -1), vp.reshape(m, -1)), 1)
        pool[i:i + m, 32 * d:] = both.view(torch.uint8)
    return pool.view(pages, c["kv_heads"], c["page"] // TILE, record)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    _, _, width = _shape(c)
    b, h, d = c["batch"], c["kv_heads"], c["dim"]
    dt = DTYPES[c["dtype"]]
    lens, news = _lens(c), _news(c)
    cut = min(width, -(-c["budget"] // c["page"])) if c["op"] == "evict" else 0
    pages = b * (width + cut)
    order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    s = dict(case=c, table=order[:b * width].view(b, width).contiguous(), lens=_ints(lens),
             pool=_pool(c, pages, gen), max_new=max(news), max_len=max(lens))
    if c["op"] != "evict":
        s["starts"] = _ints([0] + list(np.cumsum(news)))
    if c["op"] == "append":
        spread = torch.exp(0.5 * torch.randn((2, h, d), device="cuda", generator=gen))
        centre = 0.7 * torch.randn((2, h, d), device="cuda", generator=gen)
        for i, name in enumerate("kv"):
            x = torch.randn((sum(news), h, d), device="cuda", generator=gen)
            s[name] = (x * spread[i] + centre[i]).to(dt)
        return s
    if c["op"] == "evict" or c["weights"]:
        cap = width * c["page"]
        x = torch.exp(2 * torch.randn((b, h, cap), device="cuda", generator=gen))
        x = torch.where(torch.rand((b, h, cap), device="cuda", generator=gen) < 0.5, x, (x * 4).round() / 4)
        s["scores"] = x * (torch.arange(cap, device="cuda") < s["lens"][:, None, None])
    if c["op"] == "evict":
        s["dst_table"] = order[b * width:].view(b, cut).contiguous()
        kept = [min(v, c["budget"]) for v in lens]
        s["kept_starts"], s["total_kept"], s["none"] = _ints([0] + list(np.cumsum(kept))), sum(kept), _ints([0] * b)
        return s
    s["q"] = (2 * torch.randn((sum(news), h * c["group_heads"], d), device="cuda", generator=gen)).to(dt)
    if c["weights"]:
        s["scores_out"] = torch.zeros_like(s["scores"])
    return s


# ------------------------------------------------------------------ plain forms

def _quantise(x, group):
    """The values that keys or values [tokens, heads, dim] have once they are held in 4 bits."""
    shape = x.shape
    x = torch.nan_to_num(x.float(), 0.0, LIMIT, -LIMIT).clamp(-LIMIT, LIMIT).view(*shape[:2], -1, group)
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    # a tensor, as a division by a number may become a product with its reciprocal
    scale, zero = ((hi - lo) / torch.full_like(lo, 15)).half(), lo.half()
    # which code is nearest is decided in 64 bits: 32 lose what lies next to a border
    code = torch.round((x.double() - zero.double()) / scale.double()).clamp(0, 15)
    code = torch.where(scale == 0, 0.0, code)
    return (scale.float() * code.float() + zero.float()).view(shape)


def _unpack(codes):
    """Bytes [..., 4] of words into their 8 values, in three axes: [..., low bit, high bit, middle bit] of the index."""
    return torch.stack((codes & 15, codes >> 4), -1).unflatten(-2, (2, 2)).flatten(-3).unflatten(-1, (2, 2, 2))


def _values(pool, table, c):
    """Keys and values [batch, heads, positions, dim] in 32 bits of the pages that the table names."""
    groups, record, _ = _shape(c)
    d, h = c["dim"], c["kv_heads"]
    words = d // 32
    sub = 2 if words > 4 else 1
    w = words // sub
    raw = pool[table.long()].transpose(1, 2).flatten(2, 3)  # batch, heads, tiles, record
    b, _, t, _ = raw.shape
    k = _unpack(raw[..., :16 * d].reshape(b, h, t, 2, sub, 4, 16, w, 4))  # half sub g m w | low high middle
    k = k.permute(0, 1, 2, 3, 6, 4, 7, 5, 9, 10, 8).reshape(b, h, t, TILE, groups, c["group"])
    kp = raw[..., 32 * d:32 * d + 128 * groups].contiguous().view(torch.float16).view(b, h, t, groups, TILE, 2)
    kp = kp.transpose(3, 4).float()
    k = k * kp[..., 0, None] + kp[..., 1, None]
    v = _unpack(raw[..., 16 * d:32 * d].reshape(b, h, t, 2, sub, 4, 16, w, 4))
    v = v.permute(0, 1, 2, 9, 5, 10, 8, 3, 4, 7, 6).reshape(b, h, t, TILE, groups, c["group"])
    vp = raw[..., 32 * d + 128 * groups:].contiguous().view(torch.float16).view(b, h, t, groups, 2, 4, 2, 4)
    vp = vp.permute(0, 1, 2, 6, 5, 7, 3, 4).reshape(b, h, t, TILE, groups, 2).float()
    v = v * vp[..., 0, None] + vp[..., 1, None]
    return k.view(b, h, t * TILE, d), v.view(b, h, t * TILE, d)


def _attend(s):
    c = s["case"]
    b, h, g, d = c["batch"], c["kv_heads"], c["group_heads"], c["dim"]
    k, v = _values(s["pool"], s["table"], c)
    n, cap = s["max_new"], k.shape[2]
    starts = s["starts"].long()
    news = starts[1:] - starts[:-1]
    i = torch.arange(n, device="cuda")
    at = (starts[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    there = i < news[:, None]
    q = s["q"].float()[at].view(b, n, h, g, d).permute(0, 2, 1, 3, 4).reshape(b, h, n * g, d)
    x = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    last = s["lens"].long()[:, None] - (news[:, None] - 1 - i if c["causal"] else torch.zeros_like(at))
    seen = (torch.arange(cap, device="cuda") < last[..., None]) & there[..., None]
    seen = seen[:, None].repeat_interleave(g, 2)  # batch, 1, rows, positions
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    o = torch.matmul(p, v).view(b, h, n, g, d).permute(0, 2, 1, 3, 4).reshape(b, n, h * g, d)
    lse = (torch.log(total) + top).view(b, h, n, g).permute(0, 2, 1, 3).reshape(b, n, h * g)
    out = {"out": o[there].to(s["q"].dtype), "lse": lse[there]}
    if c["weights"]:
        out["scores"] = s["scores"] + p.sum(2)
    return out


def _evict(s):
    c = s["case"]
    scores, lens, budget = s["scores"], s["lens"].long()[:, None, None], c["budget"]
    cap = scores.shape[2]
    at = torch.arange(cap, device="cuda")
    n = lens.clamp(max=budget)
    first = lens - min(c["recent"], budget)  # from here on all are kept
    rank = torch.where(at < lens, torch.where(at >= first, math.inf, scores), -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :budget]
    if budget > cap:
        order = torch.nn.functional.pad(order, (0, budget - cap), value=cap)
    column = torch.arange(budget, device="cuda")
    kept = torch.sort(torch.where(column < n, order, cap), dim=-1).values
    live = column < n
    kept = torch.where(live, kept, -1)
    safe = kept.clamp(min=0)
    k, v = _values(s["pool"], s["table"], c)
    cols = torch.zeros((), dtype=torch.int64, device="cuda")
    k = torch.gather(k, 2, (safe + cols)[..., None].expand(-1, -1, -1, c["dim"]))
    v = torch.gather(v, 2, (safe + cols)[..., None].expand(-1, -1, -1, c["dim"]))
    one = live[:, 0].expand(-1, budget)
    return {"kept": kept.to(torch.int32), "lens": n[:, 0, 0].to(torch.int32),
            "scores": torch.where(live, torch.gather(scores, 2, safe), 0.0),
            "k": k.transpose(1, 2)[one].half(), "v": v.transpose(1, 2)[one].half()}


def run(s):
    c = s["case"]
    if own:
        return _own(s)
    if c["op"] == "append":
        return {"k": _quantise(s["k"], c["group"]), "v": _quantise(s["v"], c["group"])}
    return _attend(s) if c["op"] == "attend" else _evict(s)


def _own(s):
    from tiled_tensor_bulk_amd import tkv as T

    c = s["case"]
    cache = T.tkv_encode(s["pool"], c["kv_heads"], c["dim"], c["page"], c["group"])
    if c["op"] == "append":
        T.tkv_append(cache, s["k"], s["v"], s["table"], s["lens"], starts=s["starts"], max_new=s["max_new"])
        k, v = T.tkv_read(cache, s["table"], s["lens"], starts=s["starts"], max_new=s["max_new"],
                          n_tokens=s["k"].shape[0], dtype=torch.float32)
        return {"k": k, "v": v}
    if c["op"] == "attend":
        out, lse = T.tkv_attend(cache, s["q"], s["table"], s["lens"], starts=s["starts"], max_new=s["max_new"],
                                max_len=s["max_len"], causal=c["causal"], scores=s.get("scores"),
                                scores_out=s.get("scores_out"))
        r = {"out": out, "lse": lse}
        return dict(r, scores=s["scores_out"]) if c["weights"] else r
    kept, lens, scores = T.tkv_evict(cache, s["table"], s["lens"], s["scores"], c["budget"], c["recent"],
                                     s["dst_table"], max_len=s["max_len"])
    k, v = T.tkv_read(cache, s["dst_table"], s["none"], starts=s["kept_starts"],
                      max_new=min(c["budget"], s["max_len"]), n_tokens=s["total_kept"], dtype=torch.float16)
    return {"kept": kept, "lens": lens, "scores": scores, "k": k, "v": v}


# ------------------------------------------------------------------ the definition in 64 bits

def _places(c):
    """For each position of a record and each channel: the byte and shift of its K code and of its V code, and the
    fp16 places of the scale and zero of each."""
    d, groups = c["dim"], c["dim"] // c["group"]
    words = d // 32
    w = words if words <= 4 else words // 2
    t, ch = np.meshgrid(np.arange(TILE), np.arange(d), indexing="ij")

    def place(half, word, g, m, j):
        lane = 16 * g + m
        nibble = (j >> 1) + 4 * (j & 1)
        index = ((half * (words // w) + word // w) * 64 + lane) * w + word % w
        return 4 * index + nibble // 2, 4 * (nibble % 2)

    kb, ks = place(t // 16, ch // 32, (ch % 32) // 8, t % 16, ch % 8)
    chunk = ch // 16
    vb, vs = place(chunk // words, chunk % words, (t % 16) // 4, ch % 16, (t % 4) + 4 * (t // 16))
    grp = ch // c["group"]
    kp = 16 * d + (grp * TILE + t) * 2
    slot = 8 * ((t % 16) // 4) + 4 * (t // 16) + t % 4
    vp = 16 * d + 64 * groups + grp * 64 + slot
    places = [kb, ks, kp, kp + 1, vb + 16 * d, vs, vp, vp + TILE]
    return [torch.from_numpy(x.reshape(-1).copy()).cuda() for x in places]


def _double(pool, pages, c, places):
    """Keys and values [heads, positions, dim] of one sequence's pages."""
    rec = pool[pages.long()].transpose(0, 1).flatten(1, 2).contiguous()
    h, t, _ = rec.shape
    half = rec.view(torch.float16)
    out = []
    for code, shift, scale, zero in (places[:4], places[4:]):
        x = (rec[..., code] >> shift.to(torch.uint8)) & 15
        out.append((x.double() * half[..., scale].double() + half[..., zero].double()).reshape(h, t * TILE, c["dim"]))
    return out


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "append":
        out = {}
        for name in "kv":
            x = s[name].double()
            x = torch.where(x.isnan(), 0.0, x).clamp(-LIMIT, LIMIT).unflatten(-1, (-1, c["group"]))
            lo = x.min(-1, keepdim=True).values
            step = ((x.max(-1, keepdim=True).values - lo) / 15).half().double()
            lo = lo.half().double()
            code = torch.clamp(torch.round((x - lo) / torch.where(step == 0, 1.0, step)), 0, 15) * (step != 0)
            out[name] = (lo + step * code).flatten(-2)
        return out
    places, lens, news = _places(c), _lens(c), _news(c)
    if c["op"] == "evict":
        scores, outs = s["scores"].cpu().numpy().astype(np.float64), {"k": [], "v": [], "scores": []}
        out = np.zeros((c["batch"], c["kv_heads"], c["budget"]))
        for b, n in enumerate(lens):
            k, v = _double(s["pool"], s["table"][b], c, places)
            m = min(n, c["budget"])
            recent = min(c["recent"], c["budget"])
            pick = []
            for h in range(c["kv_heads"]):
                if n <= c["budget"]:
                    keep = np.arange(n)
                else:
                    old = scores[b, h, :n - recent]
                    best = np.lexsort((np.arange(old.size), -old))[:m - recent]
                    keep = np.concatenate((np.sort(best), np.arange(n - recent, n)))
                out[b, h, :m] = scores[b, h, keep]
                pick.append(torch.from_numpy(keep).cuda())
            pick = torch.stack(pick)[..., None].expand(-1, -1, c["dim"])
            outs["k"].append(k.gather(1, pick).transpose(0, 1).half())
            outs["v"].append(v.gather(1, pick).transpose(0, 1).half())
        return {"kept": None, "lens": None, "scores": torch.from_numpy(out), "k": torch.cat(outs["k"]).double(),
                "v": torch.cat(outs["v"]).double()}
    g, d = c["group_heads"], c["dim"]
    outs, lses, at = [], [], 0
    scores = s["scores"].double() if c["weights"] else None
    for b, (n, m) in enumerate(zip(lens, news)):
        k, v = _double(s["pool"], s["table"][b], c, places)
        k, v = k[:, :n], v[:, :n]
        q = s["q"][at:at + m].double().unflatten(1, (-1, g)).permute(1, 2, 0, 3).flatten(1, 2)  # heads, rows, dim
        at += m
        x = q @ k.mT.contiguous() / math.sqrt(d)
        if c["causal"]:
            ahead = torch.arange(n, device="cuda") > torch.arange(n - m, n, device="cuda")[:, None]
            x = x.masked_fill(ahead.repeat(g, 1), -math.inf)
        lse = torch.logsumexp(x, -1, keepdim=True)
        p = torch.exp(x - lse)
        outs.append((p @ v).unflatten(1, (g, m)).permute(2, 0, 1, 3).flatten(1, 2))
        lses.append(lse[..., 0].unflatten(1, (g, m)).permute(2, 0, 1).flatten(1, 2))
        if c["weights"]:
            scores[b, :, :n] += p.sum(1)
    r = {"out": torch.cat(outs), "lse": torch.cat(lses)}
    return dict(r, scores=scores) if c["weights"] else r
