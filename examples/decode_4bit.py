"""A decoding loop on the 4-bit cache: prompts enter in chunks, tokens are decoded in a captured graph, and sequences
that have grown past a budget are shrunk by their accumulated attention weights.

    python examples/decode_4bit.py [--batch 4 --heads 8 --group-heads 4 --dim 128 --prompt 700 --steps 64 --budget 512]

One attention layer on synthetic keys, values and queries; every step's output is compared with attention over the
same keys and values before they were quantised, so what is printed is what 4 bits cost.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from tiled_tensor_bulk_amd import tkv as T  # noqa: E402


def plain(q, k, v, positions):
    """Attention of q [heads * group, dim] over k, v [positions, heads, dim], in fp32; positions: bool [heads, n]."""
    heads, dim = k.shape[1:]
    q = q.float().view(heads, -1, dim)
    x = torch.matmul(q, k.float().permute(1, 2, 0).contiguous()) * dim ** -0.5
    x = x.masked_fill(~positions[:, None], float("-inf"))
    return torch.matmul(torch.softmax(x, -1), v.float().transpose(0, 1).contiguous()).reshape(-1, dim)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("batch", 4), ("heads", 8), ("group-heads", 4), ("dim", 128), ("prompt", 700), ("chunk", 256),
                        ("steps", 64), ("budget", 512), ("recent", 128), ("page", 64), ("group", 64)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(0)
    b, h, d = a.batch, a.heads, a.dim
    longest = max(a.prompt, a.budget) + a.steps
    width = -(-longest // a.page)

    # two sets of pages for each sequence: eviction moves a sequence from one to the other
    pages = 2 * b * width
    pool = torch.empty(pages * T.tkv_page_bytes_of(h, d, a.page, a.group), dtype=torch.uint8, device=dev)
    cache = T.tkv_encode(pool, h, d, a.page, a.group)
    order = torch.randperm(pages, device=dev, generator=gen).to(torch.int32).view(2, b, width)
    table = order[0].clone()

    def normal(*shape):
        return torch.randn(shape, device=dev, generator=gen).to(torch.bfloat16)

    n = a.prompt + a.steps
    k, v, q = normal(b, n, h, d), normal(b, n, h, d), normal(b, n, h * a.group_heads, d)
    before = torch.zeros(b, dtype=torch.int32, device=dev)  # positions before a step's tokens
    after = torch.zeros_like(before)
    scores = torch.zeros((b, h, width * a.page), device=dev)

    # the prompts, in chunks
    for at in range(0, a.prompt, a.chunk):
        m = min(a.chunk, a.prompt - at)
        part = [x[:, at:at + m].reshape(b * m, -1, d) for x in (k, v, q)]
        after = before + m
        T.tkv_append(cache, part[0], part[1], table, before)
        out, _ = T.tkv_attend(cache, part[2], table, after, max_len=at + m, scores=scores, scores_out=scores)
        before = after
    for i in range(b):
        want = plain(q[i, a.prompt - 1], k[i, :a.prompt], v[i, :a.prompt],
                     torch.ones((h, a.prompt), dtype=torch.bool, device=dev))
        got = out.view(b, -1, h * a.group_heads, d)[i, -1].float()
        err = float((got - want).norm() / want.norm())
    print(f"prompt of {a.prompt}: error of 4 bits {err:.3f} (relative, last token)", flush=True)

    # shrink the prompts; what every head keeps is followed for the comparison
    where = torch.full((b, h, longest), -1, dtype=torch.int64, device=dev)
    where[:, :, :a.prompt] = torch.arange(a.prompt, device=dev)
    length = a.prompt
    if a.prompt > a.budget:
        kept, lens, kept_scores = T.tkv_evict(cache, table, before, scores, a.budget, a.recent, order[1],
                                              max_len=a.prompt)
        table.copy_(order[1])
        before.copy_(lens)
        scores.zero_()[:, :, :a.budget] = kept_scores
        length = a.budget
        where.fill_(-1)[:, :, :length] = kept
        print(f"shrunk to {a.budget} positions a head", flush=True)

    # decoding: one graph, whose tensors are refilled for each step
    after = before + 1
    kt, vt, qt = k[:, 0].clone(), v[:, 0].clone(), q[:, 0].clone()
    out = torch.empty_like(qt)
    lse = torch.empty((b, h * a.group_heads), device=dev)
    room = torch.empty(max(16, T.tkv_attend_workspace(cache, b, h * a.group_heads, 1, longest, scores=True)),
                       dtype=torch.uint8, device=dev)

    def step():
        T.tkv_append(cache, kt, vt, table, before)
        T.tkv_attend(cache, qt, table, after, max_len=longest, scores=scores, scores_out=scores, out=out, lse=lse,
                     workspace=room)
        before.add_(1)
        after.add_(1)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    worst, spent = 0.0, 0.0
    for s in range(a.steps):
        at = a.prompt + s
        kt.copy_(k[:, at]), vt.copy_(v[:, at]), qt.copy_(q[:, at])
        where[:, :, length + s] = at
        torch.cuda.synchronize()
        t = time.perf_counter()
        graph.replay()
        torch.cuda.synchronize()
        spent += time.perf_counter() - t
        for i in range(b):
            held = torch.zeros((h, n), dtype=torch.bool, device=dev)
            held.scatter_(1, where[i, :, :length + s + 1], True)
            want = plain(q[i, at], k[i], v[i], held)
            worst = max(worst, float((out[i].float() - want).norm() / want.norm()))
    print(f"{a.steps} steps, {spent / max(1, a.steps) * 1e6:.0f} us each; error of 4 bits at most {worst:.3f}", flush=True)
    return err, worst


if __name__ == "__main__":
    main()
