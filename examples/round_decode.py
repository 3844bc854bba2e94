"""One round of agents over a shared paged pool: reuse, decode, answer.

A chunk cached at other positions becomes the round's shared prefix: `pool_write` rotates its
keys to their new places and stores them once, in the pool's format.  Then every agent decodes:
each step's new rows go to the agent's own pages (`pool_write` again), and `shared_attend` gives
every layer's attention over prefix and own tokens, the prefix read once for all agents.  The
step is captured into a CUDA graph and replayed: lengths, pages and slots are read on the
device, so the same graph serves every step.  At the end `pool_read` brings the rows back and a
plain attention over them checks the last step.

    python examples/round_decode.py --format e4m3 --agents 6 --steps 4
"""
from __future__ import annotations

import argparse
import pathlib
import sys

import torch

sys.path.insert(0, str(pathlib.Path(__file__).resolve().parents[1]))

from cross_context_kv_gb300 import kvfix  # noqa: E402


def plain_attention(q, k, v, scale):
    """q [heads][dim], k and v [keys][kv_heads][dim], float."""
    group = q.shape[0] // k.shape[1]
    k, v = (t.repeat_interleave(group, 1) for t in (k, v))
    return torch.einsum("hk,khd->hd", torch.softmax(torch.einsum("hd,khd->hk", q, k) * scale, -1), v)


def run(format="e4m3", agents=6, steps=4, layers=3, prefix=700, heads=4, group=4, dim=128, page=16, shift=1234,
        rope_base=10000.0, seed=0):
    """Decodes `steps` tokens per agent; returns the largest error of the last step's outputs and
    the largest output."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    rows = lambda *shape: torch.randn(*shape, heads, dim, device=dev, generator=gen).bfloat16()  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731

    # pages: the prefix's, then each agent's own (shuffled, as a serving pool would have them)
    shared_pages, own_pages = -(-prefix // page), -(-steps // page)
    order = torch.randperm(shared_pages + agents * own_pages, generator=gen, device=dev).int()
    prefix_pages = order[:shared_pages].view(1, -1).contiguous()
    suffix_pages = order[shared_pages:].view(agents, own_pages).contiguous()
    pool = kvfix.pool_empty(format, layers, order.numel() * page, heads, dim)

    # the cached chunk, rotated to its new positions, is stored once for the round
    at = torch.arange(prefix, device=dev)
    slots = (prefix_pages[0, at // page] * page + at % page).view(1, -1).int()
    kvfix.pool_write(pool, rows(1, layers, prefix), rows(1, layers, prefix), slots, delta=i32([shift]),
                     rope_base=rope_base)

    prefix_len, group_begin = i32([prefix]), i32([0, agents])
    own_len = torch.zeros(agents, dtype=torch.int32, device=dev)
    step_slots = torch.zeros(agents, 1, dtype=torch.int32, device=dev)
    new_k, new_v = rows(agents, layers, 1), rows(agents, layers, 1)
    q = torch.randn(layers, agents, 1, heads * group, dim, device=dev, generator=gen).bfloat16()
    out = torch.empty_like(q)
    workspace = torch.empty(kvfix.shared_attend_workspace_bytes(q[0], pool, 1), dtype=torch.uint8, device=dev)

    def step():
        kvfix.pool_write(pool, new_k, new_v, step_slots)
        own_len.add_(1)
        for i in range(layers):
            kvfix.shared_attend(q[i], pool.layer(i), page, suffix_pages, own_len, prefix_pages, prefix_len, group_begin,
                                out=out[i], workspace=workspace)

    def place(n):
        step_slots.copy_((suffix_pages[:, n // page] * page + n % page).view(-1, 1))

    # the first step as it is, the others from the graph of one
    place(0)
    step()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph.capture_begin()
        step()
        graph.capture_end()
        for n in range(1, steps):
            place(n)
            new_k.normal_(generator=gen)
            new_v.normal_(generator=gen)
            q.normal_(generator=gen)
            graph.replay()
    torch.cuda.current_stream().wait_stream(stream)

    # the rows as they are stored, and the last step done plainly over them
    k0, v0 = kvfix.pool_read(pool, slots)
    at = torch.arange(steps, device=dev)
    own = (suffix_pages[:, at // page] * page + at % page).int().contiguous()
    k1, v1 = kvfix.pool_read(pool, own)
    kvfix.check_status()
    worst = 0.0
    for i in range(layers):
        for a in range(agents):
            k, v = (torch.cat((x[0, i], y[a, i])).float() for x, y in ((k0, k1), (v0, v1)))
            worst = max(worst, (plain_attention(q[i, a, 0].float(), k, v, dim ** -0.5) - out[i, a, 0].float()).abs().max().item())
    return worst, out.float().abs().max().item()


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--format", choices=sorted(kvfix.POOL_FORMATS), default="e4m3")
    p.add_argument("--agents", type=int, default=6)
    p.add_argument("--steps", type=int, default=4)
    p.add_argument("--prefix", type=int, default=700)
    a = p.parse_args(argv)
    worst, top = run(a.format, a.agents, a.steps, prefix=a.prefix)
    print(f"{a.agents} agents, {a.steps} steps over {a.prefix} shared tokens in {a.format}: "
          f"largest error {worst:.4f} of outputs up to {top:.2f}")


if __name__ == "__main__":
    main()
