"""A decoding loop on the 8-bit cache whose tokens see a window: prompts enter in chunks, keys and queries turned by their
positions on the way; tokens are decoded in a captured graph; pages that lie between the first positions and the window go
to the sequence's next ones, so that the pool stays as large as what is seen.

    python examples/decode_window.py [--batch 4 --heads 8 --group-heads 4 --dim 128 --prompt 900 --steps 200 --window 512]

One attention layer on synthetic keys, values and queries; outputs are compared with attention over the same keys and values
before they were rounded, so what is printed is what 8 bits cost.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from tiled_tensor_bulk_amd import tkv as T  # noqa: E402


def turned(x, cos_sin):
    """x [tokens, heads, dim], pairs (i, i + dim / 2) turned by each token's row of cosines and sines."""
    c, s = cos_sin[:, None].float().chunk(2, -1)
    a, b = x.float().chunk(2, -1)
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def plain(q, k, v, window, sinks):
    """Attention of a last token's q [heads * group, dim] over k, v [positions, heads, dim], in fp32."""
    n, heads, dim = k.shape
    at = torch.arange(n, device=k.device)
    seen = (at >= n - window) | (at < sinks)
    x = torch.matmul(q.view(heads, -1, dim), k[seen].permute(1, 2, 0).contiguous()) * dim ** -0.5
    return torch.matmul(torch.softmax(x, -1), v[seen].float().transpose(0, 1).contiguous()).reshape(-1, dim)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("batch", 4), ("heads", 8), ("group-heads", 4), ("dim", 128), ("prompt", 900), ("chunk", 256),
                        ("steps", 200), ("window", 512), ("sinks", 4), ("page", 32)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(0)
    b, h, d, n = a.batch, a.heads, a.dim, a.prompt + a.steps
    heads = h * a.group_heads

    # pages that a sequence holds at a time: its first ones, the window's and a chunk's
    first = -(-a.sinks // a.page)
    held = first + -(-(a.window + max(a.chunk, 1)) // a.page) + 2
    width = -(-n // a.page)
    pool = torch.zeros(b * held * T.tkv_page_bytes_of(h, d, a.page, bits=8), dtype=torch.uint8, device=dev)
    cache = T.tkv_encode(pool, h, d, a.page, bits=8)
    free = [list(range(i * held, (i + 1) * held)) for i in range(b)]
    pages = torch.full((b, width), -1, dtype=torch.int32)  # as the host plans them
    table = pages.to(dev)

    def make_room(at, new):
        """Pages for positions at .. at + new - 1; those that no token from `at` on sees any more are free again."""
        gone = max(0, at + 1 - a.window) // a.page
        for i in range(b):
            for p in range(first, min(gone, width)):
                if pages[i, p] >= 0:
                    free[i].append(int(pages[i, p]))
                    pages[i, p] = -1
            for p in range(at // a.page, (at + new - 1) // a.page + 1):
                if pages[i, p] < 0:
                    pages[i, p] = free[i].pop()
        table.copy_(pages)

    angle = torch.arange(n, device=dev)[:, None] * 10000.0 ** -(torch.arange(d // 2, device=dev) / (d // 2))
    cos_sin = torch.cat((angle.cos(), angle.sin()), -1).float()

    def normal(*shape):
        return torch.randn(shape, device=dev, generator=gen).to(torch.bfloat16)

    k, v, q = normal(b, n, h, d), normal(b, n, h, d), normal(b, n, heads, d)
    wanted = [turned(k[i], cos_sin) for i in range(b)]

    def error(out, at):
        worst = 0.0
        for i in range(b):
            want = plain(turned(q[i, at:at + 1], cos_sin[at:at + 1])[0], wanted[i][:at + 1], v[i, :at + 1], a.window, a.sinks)
            worst = max(worst, float((out[i].float() - want).norm() / want.norm()))
        return worst

    # the prompts, in chunks
    before = torch.zeros(b, dtype=torch.int32, device=dev)
    for at in range(0, a.prompt, a.chunk):
        m = min(a.chunk, a.prompt - at)
        make_room(at, m)
        part = [x[:, at:at + m].reshape(b * m, -1, d) for x in (k, v, q)]
        qt = T.tkv_append(cache, part[0], part[1], table, before, cos_sin=cos_sin, q=part[2])
        before += m
        out, _ = T.tkv_attend(cache, qt, table, before, max_len=at + m, window=a.window, sinks=a.sinks)
    first_error = error(out.view(b, -1, heads, d)[:, -1], a.prompt - 1)
    print(f"prompt of {a.prompt}: error of 8 bits {first_error:.4f} (relative, last token)", flush=True)

    # decoding: one graph, whose tensors are refilled for each step
    after = before + 1
    kt, vt, qt = k[:, 0].clone(), v[:, 0].clone(), q[:, 0].clone()
    out = torch.empty_like(qt)
    lse = torch.empty((b, heads), device=dev)
    room = torch.empty(max(16, T.tkv_attend_workspace(cache, b, heads, 1, n)), dtype=torch.uint8, device=dev)

    def step():
        T.tkv_append(cache, kt, vt, table, before, cos_sin=cos_sin, q=qt, q_out=qt)
        T.tkv_attend(cache, qt, table, after, max_len=n, window=a.window, sinks=a.sinks, out=out, lse=lse, workspace=room)
        before.add_(1)
        after.add_(1)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    worst, spent = 0.0, 0.0
    for s in range(a.steps):
        at = a.prompt + s
        make_room(at, 1)
        kt.copy_(k[:, at]), vt.copy_(v[:, at]), qt.copy_(q[:, at])
        torch.cuda.synchronize()
        t = time.perf_counter()
        graph.replay()
        torch.cuda.synchronize()
        spent += time.perf_counter() - t
        worst = max(worst, error(out, at))
    print(f"{a.steps} steps in {held} pages a sequence, {spent / max(1, a.steps) * 1e6:.0f} us each; error of 8 bits at most "
          f"{worst:.4f}", flush=True)
    return first_error, worst


if __name__ == "__main__":
    main()
