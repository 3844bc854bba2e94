"""A round of agents that draft trees: room, rotation, verification, acceptance, over one paged pool.

The round's prefix is list 0 of the page books, each agent's own tokens a list of their own.  A step
drafts a tree of tokens for every agent: `pages_extend` makes room behind the lists, `rotary`
turns the nodes' queries and keys to their places (the context's length plus the node's depth),
`pool_write` stores them, and `tree_attend` gives every node's attention over prefix, own tokens
and its line of descent.  The accepted path then moves up and the rest of the tree is dropped by
`pages_cut`.  Both halves of a step are captured into graphs and replayed: lists, lengths and trees
are read on the device.  After the first step the last agent ends and begins again as a fork of the first;
at the end `pages_compact` moves what is in use to the front of the pool.  The last step is
checked by a plain attention over the rows read back, and the moves by reading rows before and after.

    python examples/draft_round.py --format e4m3 --agents 5 --steps 4
"""
from __future__ import annotations

import argparse
import pathlib
import random
import sys

import torch

sys.path.insert(0, str(pathlib.Path(__file__).resolve().parents[1]))

from cross_context_kv_gb300 import kvfix  # noqa: E402


def plain_attention(q, k, v, sees, scale):
    """q [nodes][heads][dim], k and v [keys][kv_heads][dim] float, sees [nodes][keys]."""
    k, v = (t.repeat_interleave(q.shape[1] // k.shape[1], 1) for t in (k, v))
    z = torch.einsum("thd,khd->thk", q, k) * scale
    return torch.einsum("thk,khd->thd", torch.softmax(z.masked_fill(~sees[:, None], -torch.inf), -1), v)


def run(format="e4m3", agents=5, steps=4, nodes=12, layers=2, prefix=300, heads=2, group=4, dim=128, page=16, seed=0):
    """Drafts and accepts `steps` times; returns the largest error of the last step's outputs, the
    largest output, and whether every row is where the books say."""
    dev, T = torch.device("cuda"), nodes
    gen, rng = torch.Generator(device=dev).manual_seed(seed), random.Random(seed)
    i32 = lambda *shape, fill=0: torch.full(shape, fill, dtype=torch.int32, device=dev)  # noqa: E731
    rope = kvfix.Rope(5e5, scaling="bands", factor=8.0, low=1.0, high=4.0, original=8192)

    # the books: list 0 is the prefix, list 1 + a agent a's own tokens
    lists, wide = 1 + agents, -(-max(prefix, (steps + 1) * T) // page) + 1
    total = -(-prefix // page) + 2 * agents * wide
    refs, pages, lens = i32(total), i32(lists, wide, fill=-1), i32(lists)
    pool = kvfix.pool_empty(format, layers, total * page, heads, dim)
    at = torch.arange(max(prefix, wide * page), device=dev)

    def slots_of(table, first, n):
        """Pool rows of n tokens from `first` on (one per list) of page lists `table`."""
        t = first.long()[:, None] + torch.arange(n, device=dev)
        return (table.long().gather(1, t // page) * page + t % page).int()

    # the prefix, turned to its places
    extra = i32(lists)
    extra[0] = prefix
    kvfix.pages_extend(pool, page, refs, pages, lens, extra)
    rows = lambda *shape, h=heads: torch.randn(*shape, h, dim, device=dev, generator=gen).bfloat16()  # noqa: E731
    k = rows(1, layers, prefix)
    kvfix.rotary(None, k, at[:prefix].int().view(1, -1), rope, k_out=k)
    kvfix.pool_write(pool, k, rows(1, layers, prefix), slots_of(pages[:1], lens[:1] * 0, prefix))

    # a step's tensors: trees, places, rows
    mask, depth, count = i32(agents, T, (T + 31) // 32), i32(agents, T), i32(agents)
    before, path, kept = i32(lists), i32(lists, T), i32(lists)
    parent = torch.arange(lists, dtype=torch.int32, device=dev)
    q, k, v = rows(agents, layers, T, h=heads * group), rows(agents, layers, T), rows(agents, layers, T)
    out = torch.empty(layers, agents, T, heads * group, dim, dtype=torch.bfloat16, device=dev)
    prefix_len, group_begin = lens[:1], torch.tensor([0, agents], dtype=torch.int32, device=dev)
    workspace = torch.empty(kvfix.shared_attend_workspace_bytes(out[0], pool, 1), dtype=torch.uint8, device=dev)
    extra.fill_(T)
    extra[0] = 0

    def draft():
        kvfix.pages_extend(pool, page, refs, pages, lens, extra, parent)
        before.copy_(lens - extra)
        kvfix.rotary(q, k, before[1:, None] + prefix + depth, rope, q_out=q, k_out=k)
        kvfix.pool_write(pool, k, v, slots_of(pages[1:], before[1:], T))
        for i in range(layers):
            kvfix.tree_attend(q[:, i], pool.layer(i), page, pages[1:], lens[1:], mask, count, pages[:1], prefix_len,
                              group_begin, out=out[i], workspace=workspace)

    def accept():
        kvfix.pages_cut(pool, page, refs, pages, lens, before, path, kept)

    def new_step():
        """Trees, a path through each, and the nodes' rows (nodes of smaller trees come last and are nobody's)."""
        trees = [[-1] + [rng.randrange(-1, t) for t in range(1, T)] for _ in range(agents)]
        for x, y in zip((mask, depth, count), kvfix.tree_masks(trees, device=dev)):
            x.copy_(y)
        paths = []
        for tree in trees:
            line, t = [], rng.randrange(T)
            while t >= 0:
                line.insert(0, t)
                t = tree[t]
            paths.append(line)
        path[1:] = torch.tensor([p + [0] * (T - len(p)) for p in paths], device=dev)
        kept[1:] = torch.tensor([len(p) for p in paths], device=dev)
        for x in (q, k, v):
            x.normal_(generator=gen)
        return trees

    def read(list_, n):
        """A list's first n rows, keys and values [layers][n][heads][dim] as they are stored."""
        if n == 0:
            return [torch.zeros(layers, 0, heads, dim, dtype=torch.bfloat16, device=dev)] * 2
        return [x[0] for x in kvfix.pool_read(pool, slots_of(pages[list_:list_ + 1], lens[:1] * 0, n))]

    # the first step as it is, then from graphs
    trees = new_step()
    draft()
    accept()
    kvfix.check_status()

    # the last agent ends, and begins again as a fork of the first, which drafts beside it
    if agents > 1:
        end = i32(lists, fill=-1)
        end[-1] = 0
        kvfix.pages_cut(pool, page, refs, pages, lens, end)
        fork, none = i32(lists, fill=-1), i32(lists)
        fork[-1] = 1
        kvfix.pages_extend(pool, page, refs, pages, lens, none, fork)

    stream, drafts, accepts = torch.cuda.Stream(), torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    worst, top, placed = 0.0, 0.0, True
    with torch.cuda.stream(stream):
        for graph, half in ((drafts, draft), (accepts, accept)):
            graph.capture_begin()
            half()
            graph.capture_end()
        for n in range(1, steps):
            trees = new_step()
            drafts.replay()
            ends = lens.tolist()                                    # (the whole trees are in the lists)
            drafted = [read(x, ends[x]) for x in range(lists)]
            accepts.replay()
            # accepted rows moved up, bit for bit
            kept_rows = [drafted[0]]
            for a in range(agents):
                first, line = ends[1 + a] - T, path[1 + a, :int(kept[1 + a])].long()
                keep = torch.cat((at[:first], first + line))
                kept_rows.append([x[:, keep] for x in drafted[1 + a]])
            now = lens.tolist()
            for x in range(lists):
                placed &= all(torch.equal(y, z) for y, z in zip(read(x, now[x]), kept_rows[x]))
        if steps > 1:
            # the last step plainly, over the rows as they were stored
            for a in range(agents):
                first = ends[1 + a] - T
                line = [set() for _ in range(T)]
                for t, up in enumerate(trees[a]):
                    line[t] = (line[up] if up >= 0 else set()) | {t}
                sees = torch.ones(T, prefix + ends[1 + a], dtype=torch.bool)
                for t in range(T):
                    sees[t, prefix + first:] = torch.tensor([j in line[t] for j in range(T)])
                for i in range(layers):
                    ks, vs = (torch.cat((drafted[0][p][i], drafted[1 + a][p][i])).float() for p in (0, 1))
                    want = plain_attention(q[a, i].float(), ks, vs, sees.to(dev), dim ** -0.5)
                    worst = max(worst, (want - out[i, a].float()).abs().max().item())
            top = out.float().abs().max().item()
            # what is in use moves to the front, and every list reads as before
            live = kvfix.pages_compact(pool, page, refs, pages, lens).item()
            placed &= not refs[live:].any().item() and bool((refs[:live] > 0).all())
            for x in range(lists):
                placed &= all(torch.equal(y, z) for y, z in zip(read(x, now[x]), kept_rows[x]))
    torch.cuda.current_stream().wait_stream(stream)
    kvfix.check_status()
    return worst, top, bool(placed)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--format", choices=sorted(kvfix.POOL_FORMATS), default="e4m3")
    p.add_argument("--agents", type=int, default=5)
    p.add_argument("--steps", type=int, default=4)
    p.add_argument("--nodes", type=int, default=12)
    p.add_argument("--prefix", type=int, default=300)
    a = p.parse_args(argv)
    worst, top, placed = run(a.format, a.agents, a.steps, a.nodes, prefix=a.prefix)
    print(f"{a.agents} agents, {a.steps} trees of {a.nodes} over {a.prefix} shared tokens in {a.format}: largest error "
          f"{worst:.4f} of outputs up to {top:.2f}, rows {'in' if placed else 'OUT OF'} place")


if __name__ == "__main__":
    main()
