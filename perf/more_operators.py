"""Workloads of a drafting step over a paged pool: rotary positions of its queries and keys, the
attention of a tree of drafted tokens, and the pages that sequences take, share, give back and
leave behind.

`run` computes them in plain torch (`own` false) or through the library's entry points (`own`
true) on what `prepare` makes; `work` counts the bytes and operations a pass cannot do without;
`exact` restates the definitions in 64 bits.

  rotary   y = m R(p theta) x for the first `rot` values of every head of token t at position
           p = positions[t]; pairs (i, i + rot/2) ("half") or (2i, 2i + 1) ("interleaved"); the
           other values as they are.  theta_i = base^(-2i/rot), scaled for long contexts:
             linear  theta / factor
             bands   by the turns r = original theta / 2 pi over the original context: s = (r - low) /
                     (high - low) within [0, 1], theta (s + (1 - s) / factor)
             yarn    s by the pair's number instead: 1 up to the pair with `high` turns, 0 from the
                     one with `low`; m = `attention`
  tree     attention of the last nodes[a] own tokens of each agent, a tree of drafts: node t sees
           the prefix, the agent's own tokens before the tree, and the nodes j <= t of its mask.
  extend   room for `extra` tokens behind each list of pages; a fork first takes over its parent's
           pages.  A last page that is partly full and that others hold is copied.  New pages: the
           lowest free ones, in the order of lists.
  cut      each list keeps its first base tokens, then the tokens base + path[j]; pages behind its
           new end are given back.
  compact  pages in use move to the front of the pool, the j-th lowest of those behind to the j-th
           lowest hole, and the lists follow.
"""
import math

import torch

own = False

GROUP = 32
PLANES = ("k", "v")
ROPES = {
    "none": dict(base=1e4, factor=1.0, low=0.0, high=0.0, original=0, attention=1.0),
    "linear": dict(base=1e4, factor=4.0, low=0.0, high=0.0, original=0, attention=1.0),
    "bands": dict(base=5e5, factor=8.0, low=1.0, high=4.0, original=8192, attention=1.0),
    "yarn": dict(base=1e6, factor=16.0, low=1.0, high=32.0, original=32768, attention=0.1 * math.log(16.0) + 1.0),
}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # queries and keys of eight drafted tokens of 16 agents, one layer: launch latency
        dict(name="rotary_draft_bands", op="rotary", chunks=16, layers=1, tokens=8, q_heads=32, k_heads=8, dim=128,
             rot=128, layout="half", scaling="bands"),
        # a 4096-token chunk of a 32-layer cache re-aligned, half of each head rotated
        dict(name="rotary_cache_partial", op="rotary", chunks=1, layers=32, tokens=4096, q_heads=0, k_heads=8, dim=128,
             rot=64, layout="interleaved", scaling="linear"),
        # one agent's eight drafts on a short block: the smallest verification
        dict(name="tree_tiny_bf16", op="tree", fmt="bf16", agents=1, groups=1, nodes=8, ragged=False, heads=4, group=2,
             dim=64, page=16, prefix=256, own_lo=9, own_hi=9),
        # a round of 8 agents, 32 drafts each over 8 shared blocks of 512 and ragged histories
        dict(name="tree_round_bf16", op="tree", fmt="bf16", agents=8, groups=1, nodes=32, ragged=False, heads=8, group=4,
             dim=128, page=16, prefix=4096, own_lo=200, own_hi=3000),
        # 16 agents over a long shared context in 8 bits
        dict(name="tree_long_e4m3", op="tree", fmt="e4m3", agents=16, groups=1, nodes=16, ragged=True, heads=8, group=4,
             dim=128, page=32, prefix=32768, own_lo=16, own_hi=1024),
        # three groups, odd lengths, trees of different sizes, 4 bits
        dict(name="tree_ragged_int4", op="tree", fmt="int4", agents=13, groups=3, nodes=61, ragged=True, heads=5, group=5,
             dim=64, page=64, prefix=3001, own_lo=0, own_hi=1500),
        # 64 agents make room for eight drafts each: a few new pages, launch latency
        dict(name="extend_step_e4m3", op="extend", fmt="e4m3", layers=32, heads=8, dim=128, page=16, pages=2048,
             roots=64, clones=0, forks=0, context=400, extra=8),
        # 4 agents fork into 32 more, every one with a page to copy in all layers
        dict(name="extend_fork_bf16", op="extend", fmt="bf16", layers=32, heads=8, dim=128, page=32, pages=640,
             roots=4, clones=4, forks=32, context=4120, extra=48),
        # 32 agents keep the accepted nodes of 32-node trees in all layers
        dict(name="cut_accept_bf16", op="cut", fmt="bf16", layers=32, heads=8, dim=128, page=16, lists=32, context=600,
             nodes=32, keep=6, gone=0),
        # 48 lists of 9 layers, some given back whole, odd heads, 4 bits
        dict(name="cut_free_int4", op="cut", fmt="int4", layers=9, heads=5, dim=64, page=64, lists=48, context=2000,
             nodes=61, keep=9, gone=16),
        # what is left of a 32-layer pool of 32768 tokens, two fifths free, moved to its front
        dict(name="compact_large_e4m3", op="compact", fmt="e4m3", layers=32, heads=8, dim=128, page=32, pages=1024,
             lists=64, shared=8, use=0.6),
        # a small pool with odd numbers
        dict(name="compact_small_int4", op="compact", fmt="int4", layers=9, heads=5, dim=64, page=16, pages=333,
             lists=7, shared=3, use=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotary", "rotary", "tree", "tree", "tree", "extend", "cut", "compact"))
    if op == "rotary":
        dim = rng.choice((64, 96, 128, 256))
        k_heads, q_heads = rng.choice((1, 2, 5, 8)), rng.choice((0, 8, 32, 40))
        chunks, layers = _log(rng, 1, 16), _log(rng, 1, 32)
        most = max(1, (32 * 4096 * 8 * 128) // (chunks * layers * (k_heads + q_heads) * dim))
        return dict(op=op, chunks=chunks, layers=layers, tokens=_log(rng, 1, min(8192, most)), q_heads=q_heads,
                    k_heads=k_heads, dim=dim, rot=rng.choice((dim, dim, dim // 2, dim // 4, 20)),
                    layout=rng.choice(("half", "interleaved")), scaling=rng.choice(sorted(ROPES)))
    fmt = rng.choice(("bf16", "e4m3", "int4"))
    heads, dim, page = rng.choice((1, 2, 4, 5, 8)), rng.choice((64, 128)), rng.choice((16, 32, 64, 128))
    if op == "tree":
        agents, group = _log(rng, 1, 32), rng.choice((1, 2, 4, 5, 8))
        nodes = rng.choice((1, 2, 7, _log(rng, 4, 128)))
        cap = max(64, min(65536, int(1.5e8 / (agents * nodes * heads * group))))
        prefix = rng.choice((0, _log(rng, 1, cap), _log(rng, 64, cap)))
        return dict(op=op, fmt=fmt, agents=agents, groups=min(agents, rng.choice((1, 1, 2, 3))), nodes=nodes,
                    ragged=rng.random() < 0.5, heads=heads, group=group, dim=dim, page=page, prefix=prefix,
                    own_lo=0, own_hi=_log(rng, 1, max(2, min(4000, cap))))
    layers, layer_page = _log(rng, 1, 32), heads * dim * 4 * page
    few = lambda pages: min(layers, max(1, int(1.5e9 / (layer_page * pages))))  # noqa: E731  (1.5 GB as bf16)
    if op == "extend":
        roots, clones, forks = _log(rng, 1, 24), rng.choice((0, 3)), rng.choice((0, 1, _log(rng, 1, 40)))
        context, extra = _log(rng, 1, 2000), _log(rng, 1, 200)
        need = roots * (context // page + 2) + (roots + clones + forks) * (extra // page + 3)
        return dict(op=op, fmt=fmt, layers=few(need), heads=heads, dim=dim, page=page,
                    pages=need + rng.randrange(1, 50), roots=roots, clones=min(clones, roots),
                    forks=forks, context=context, extra=extra)
    if op == "cut":
        lists, nodes, context = _log(rng, 1, 32), _log(rng, 2, 100), _log(rng, 1, 1500)
        return dict(op=op, fmt=fmt, layers=few(lists * ((context + nodes) // page + 1)), heads=heads, dim=dim, page=page,
                    lists=lists, context=context, nodes=nodes, keep=rng.randrange(0, min(nodes, 12) + 1),
                    gone=rng.randrange(0, lists // 2 + 1))
    pages = _log(rng, 8, 3000)
    return dict(op=op, fmt=fmt, layers=few(pages), heads=heads, dim=dim, page=page, pages=pages,
                lists=_log(rng, 1, 40), shared=rng.randrange(0, 4), use=round(rng.uniform(0.1, 0.95), 2))


# ------------------------------------------------------------------ what a program holds before the call

def _spread(lo, hi, n):
    """n whole numbers over [lo, hi], the last one hi."""
    mine = [lo + int(round((hi - lo) * ((i * 0.6180339887498949) % 1.0))) for i in range(n)]
    if n:
        mine[-1] = hi
    return mine


def _tree_lengths(c):
    """By group its prefix, by agent its own tokens before the tree and its nodes, the groups' first agents."""
    g, a = c["groups"], c["agents"]
    prefix = [c["prefix"] if i == 0 else max(0, c["prefix"] * (g - i) // g - i) for i in range(g)]
    before = _spread(c["own_lo"], c["own_hi"], a)
    nodes = [max(0, c["nodes"] - (7 * i) % c["nodes"]) if c["ragged"] else c["nodes"] for i in range(a)]
    return prefix, before, nodes, [i * a // g for i in range(g)] + [a]


def _lengths(c):
    """Tokens of a case's lists on entry, by list."""
    if c["op"] == "extend":
        roots = _spread((c["context"] + 1) // 2, c["context"], c["roots"])
        return roots + roots[:c["clones"]] + [0] * c["forks"]
    before = _spread((c["context"] + 1) // 2, c["context"], c["lists"])
    return [n + c["nodes"] for n in before]


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _rows(gen, lead, heads, dim):
    """Rows as caches and projections hold them: some channels run several times the others' size."""
    gain = torch.ones(heads, dim, device="cuda")
    gain[torch.rand(heads, dim, generator=gen, device="cuda") < 0.04] = 4.0
    return (_normal(gen, *lead, heads, dim) * gain).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    if case["op"] == "rotary":
        return _prepare_rotary(case, gen)
    return _prepare_tree(case, gen) if case["op"] == "tree" else _prepare_pages(case, gen)


def _prepare_rotary(c, gen):
    C, L, T = c["chunks"], c["layers"], c["tokens"]
    if L == 1:
        # a context of some length for each agent, its tokens (a tree's depths) behind it
        at = torch.randint(0, 100000, (C, 1), generator=gen, device="cuda")
        positions = at + torch.randint(0, 64, (C, T), generator=gen, device="cuda")
    else:
        # a cache moved by one shift per chunk, backwards too
        positions = torch.randint(-8000, 8000, (C, 1), generator=gen, device="cuda").expand(C, T)
    s = dict(case=c, positions=positions.to(torch.int32).contiguous(), rope=ROPES[c["scaling"]])
    for name in "qk":
        heads = c[name + "_heads"]
        s[name] = _rows(gen, (C, L, T), heads, c["dim"]) if heads else None
        s[name + "_out"] = torch.empty_like(s[name]) if heads else None
    return s


def _trees(gen, nodes, T):
    """Parents [agents][T] of random trees (-1: the root is the context), each node's line of
    descent as bits [agents][T][T] and as 32-bit words."""
    A = len(nodes)
    t = torch.arange(T, device="cuda")
    parent = (torch.rand(A, T, generator=gen, device="cuda") * (t + 1)).long() - 1       # -1 .. t - 1
    # most nodes hang on a recent one
    near = torch.rand(A, T, generator=gen, device="cuda") < 0.6
    parent = torch.where(near, torch.maximum(parent, (t - 3).clamp(min=-1)), parent)
    up = torch.zeros(A, T, T + 1, device="cuda").scatter_(2, (parent + 1).unsqueeze(2), 1.0)[:, :, 1:]
    line = torch.eye(T, device="cuda") + up
    for _ in range(max(1, math.ceil(math.log2(T + 1)))):
        line = (line @ line > 0).float()
    live = t < torch.tensor(nodes, device="cuda")[:, None]
    bits = (line > 0) & live[:, :, None]
    W = (T + 31) // 32
    padded = torch.zeros(A, T, W * 32, dtype=torch.int64, device="cuda")
    padded[:, :, :T] = bits
    words = (padded.view(A, T, W, 32) << torch.arange(32, device="cuda")).sum(-1)
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)
    return bits, words.contiguous()


def _prepare_tree(c, gen):
    prefix, before, nodes, begin = _tree_lengths(c)
    mine = [b + n for b, n in zip(before, nodes)]
    P, H, D = c["page"], c["heads"], c["dim"]
    pages = lambda n: (n + P - 1) // P  # noqa: E731
    total = sum(map(pages, prefix)) + sum(map(pages, mine)) + 2
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)

    def tables(lens, at):
        wide = max(1, max(map(pages, lens)))
        out = torch.full((len(lens), wide), -1, dtype=torch.int32, device="cuda")
        for i, n in enumerate(lens):
            out[i, :pages(n)] = order[at:at + pages(n)]
            at += pages(n)
        return out, at

    prefix_pages, at = tables(prefix, 0)
    own_pages, _ = tables(mine, at)
    pool = _pool(c["fmt"], 1, total * P, H, D, gen)
    q = (1.5 * _normal(gen, c["agents"], c["nodes"], H * c["group"], D)).to(torch.bfloat16)
    bits, words = _trees(gen, nodes, c["nodes"])
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(case=c, q=q, pool=pool, page=P, prefix_pages=prefix_pages, suffix_pages=own_pages, bits=bits, words=words,
                prefix_len=torch.tensor(prefix, **i32), suffix_len=torch.tensor(mine, **i32),
                nodes=torch.tensor(nodes, **i32), group_begin=torch.tensor(begin, **i32), host=(prefix, before, nodes, begin))


def _pool(fmt, layers, slots, heads, dim, gen):
    """A pool full of stored rows: bf16 values, or codes and scales as writing leaves them."""
    pool = dict(fmt=fmt, slots=slots, heads=heads, dim=dim, layers=layers)
    dev = dict(generator=gen, device="cuda")
    for p in PLANES:
        if fmt == "bf16":
            pool[p], pool[p + "_scales"] = torch.randn(layers, slots, heads, dim, dtype=torch.bfloat16, **dev), None
        elif fmt == "e4m3":
            # (the bit that NaN codes have cleared)
            code = torch.randint(0, 256, (layers, slots, heads, dim), dtype=torch.uint8, **dev)
            pool[p] = code & 0xF7
            pool[p + "_scales"] = torch.randint(118, 121, (layers, heads, slots), dtype=torch.uint8, **dev)
        else:
            pool[p] = torch.randint(0, 256, (layers, slots, heads, dim // 2), dtype=torch.uint8, **dev)
            lo = -2.0 - torch.rand(layers, heads, slots, dim // GROUP, **dev)
            pool[p + "_scales"] = torch.stack((-lo / 8, lo), -1).to(torch.bfloat16)
    return pool


def _prepare_pages(c, gen):
    P, op = c["page"], c["op"]
    host = torch.Generator().manual_seed(torch.randint(0, 2 ** 31, (1,), generator=gen, device="cuda").item())
    take = lambda n: (n + P - 1) // P  # noqa: E731
    s = dict(case=c, page=P)
    if op == "compact":
        # lists on the pages in use, their first pages shared
        total, L = c["pages"], c["lists"]
        order = torch.randperm(total, generator=host)[:max(1, int(total * c["use"]))]
        first, rest = order[:c["shared"]], order[c["shared"]:]
        each = [rest[i * len(rest) // L:(i + 1) * len(rest) // L] for i in range(L)]
        rows = [torch.cat((first, x)) if len(x) else x for x in each]
        wide = max(1, max(map(len, rows)))
        lens = [max(0, len(x) * P - (i * 5) % P) for i, x in enumerate(rows)]
    else:
        lens = _lengths(c)
        L = len(lens)
        fresh = [0 if op == "extend" and i >= c["roots"] else take(n) for i, n in enumerate(lens)]
        total = c["pages"] if op == "extend" else sum(fresh) + 17
        order, at, rows = torch.randperm(total, generator=host), 0, []
        for n in fresh:
            rows.append(order[at:at + n])
            at += n
        if op == "extend":
            for i in range(c["clones"]):
                rows[c["roots"] + i] = rows[i]
        most = max(lens) + (c["extra"] if op == "extend" else 0)
        wide = take(most) + 2
    pages = torch.full((L, wide), -1, dtype=torch.int32)
    for i, x in enumerate(rows):
        pages[i, :len(x)] = x.to(torch.int32)
    refs = torch.bincount(torch.cat(rows).long(), minlength=total).to(torch.int32)
    # how many lists hold each page, the lists' pages, their lengths: one buffer, so that a pass begins
    # from the same state with one copy
    s["book0"] = torch.cat((refs, pages.flatten(), torch.tensor(lens, dtype=torch.int32))).cuda()
    s["book"] = s["book0"].clone()
    s["refs"] = s["book"][:total]
    s["pages"] = s["book"][total:total + L * wide].view(L, wide)
    s["lens"] = s["book"][total + L * wide:]
    s["pool"] = _pool(c["fmt"], c["layers"], total * P, c["heads"], c["dim"], gen)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    if op == "extend":
        mine = c["roots"] + c["clones"]
        s["parent"] = i32([i if i < mine else (i - mine) % c["roots"] for i in range(L)])
        s["extra"] = i32(_spread((c["extra"] + 1) // 2, c["extra"], L))
    elif op == "cut":
        before = [n - c["nodes"] for n in lens]
        kept = [max(0, c["keep"] - i % 4) for i in range(L)]
        base = list(before)
        for i in range(c["gone"]):                     # every third list or so is given back whole
            j = (3 * i) % L
            base[j], kept[j] = 0, 0
        pick = torch.stack([torch.randperm(c["nodes"], generator=host)[:max(1, c["keep"])].sort().values for _ in range(L)])
        s["base"], s["kept"], s["path"] = i32(base), i32(kept), pick.to(torch.int32).cuda()
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if op in ("extend", "cut", "compact"):
        # every pass begins from the same lists, as a program's next step would not
        state["book"].copy_(state["book0"])
    if own:
        return {"rotary": _own_rotary, "tree": _own_tree, "extend": _own_extend, "cut": _own_cut,
                "compact": _own_compact}[op](state)
    return {"rotary": _plain_rotary, "tree": _plain_tree, "extend": _plain_extend, "cut": _plain_cut,
            "compact": _plain_compact}[op](state)


def _outputs(s):
    """The lists and the pool's planes; 8-bit codes and scales as the values they stand for."""
    pool = s["pool"]
    out = dict(refs=s["refs"], pages=s["pages"], lens=s["lens"])
    for p in PLANES:
        e4m3 = pool["fmt"] == "e4m3"
        out[p] = pool[p].view(torch.float8_e4m3fn) if e4m3 else pool[p]
        if pool[p + "_scales"] is not None:
            x = pool[p + "_scales"]
            out[p + "_scales"] = x.view(torch.float8_e8m0fnu) if e4m3 else x
    return out


def _own_pool(pool):
    from cross_context_kv_gb300 import kvfix
    return kvfix.Pool(pool["fmt"], pool["k"], pool["v"], pool["k_scales"], pool["v_scales"])


def _own_rotary(s):
    from cross_context_kv_gb300 import kvfix
    c, r = s["case"], s["rope"]
    rope = kvfix.Rope(base=r["base"], rotary_dim=c["rot"], layout=c["layout"], scaling=c["scaling"], factor=r["factor"],
                      low=r["low"], high=r["high"], original=r["original"], attention=r["attention"])
    q, k = kvfix.rotary(s["q"], s["k"], s["positions"], rope, q_out=s["q_out"], k_out=s["k_out"])
    return [x for x in (q, k) if x is not None]


def _own_tree(s):
    from cross_context_kv_gb300 import kvfix
    out, lse = kvfix.tree_attend(s["q"], _own_pool(s["pool"]), s["page"], s["suffix_pages"], s["suffix_len"], s["words"],
                                 s["nodes"], s["prefix_pages"], s["prefix_len"], s["group_begin"], return_lse=True)
    return {"out": out, "lse": lse}


def _own_extend(s):
    from cross_context_kv_gb300 import kvfix
    kvfix.pages_extend(_own_pool(s["pool"]), s["page"], s["refs"], s["pages"], s["lens"], s["extra"], s["parent"])
    return _outputs(s)


def _own_cut(s):
    from cross_context_kv_gb300 import kvfix
    kvfix.pages_cut(_own_pool(s["pool"]), s["page"], s["refs"], s["pages"], s["lens"], s["base"], s["path"], s["kept"])
    return _outputs(s)


def _own_compact(s):
    from cross_context_kv_gb300 import kvfix
    live = kvfix.pages_compact(_own_pool(s["pool"]), s["page"], s["refs"], s["pages"], s["lens"])
    return {**_outputs(s), "live": live}


# ---- rotary

def _theta(c, r, device):
    rot, base = c["rot"], r["base"]
    i = torch.arange(rot // 2, dtype=torch.float64, device=device)
    theta = base ** (-2.0 * i / rot)
    if c["scaling"] == "none":
        return theta
    if c["scaling"] == "linear":
        return theta / r["factor"]
    if c["scaling"] == "bands":
        s = ((r["original"] * theta / (2 * math.pi) - r["low"]) / (r["high"] - r["low"])).clamp(0, 1)
    else:
        pair = lambda turns: rot * math.log(r["original"] / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
        a, b = max(math.floor(pair(r["high"])), 0), min(math.ceil(pair(r["low"])), rot - 1)
        s = 1 - ((i - a) / max(b - a, 1e-3)).clamp(0, 1)
    return theta * (s + (1 - s) / r["factor"])


def _plain_rotary(s):
    c, r, rot = s["case"], s["rope"], s["case"]["rot"]
    angle = s["positions"].double()[:, None, :, None, None] * _theta(c, r, s["positions"].device)
    cos, sin = (r["attention"] * angle.cos()).float(), (r["attention"] * angle.sin()).float()
    out = []
    for name in "qk":
        if s[name] is None:
            continue
        x = s[name][..., :rot].float()
        a, b = (x[..., :rot // 2], x[..., rot // 2:]) if c["layout"] == "half" else (x[..., 0::2], x[..., 1::2])
        y = (a * cos - b * sin, b * cos + a * sin)
        y = torch.cat(y, -1) if c["layout"] == "half" else torch.stack(y, -1).flatten(-2)
        o = s[name + "_out"]
        o[..., :rot] = y.to(torch.bfloat16)
        o[..., rot:] = s[name][..., rot:]
        out.append(o)
    return out


# ---- the tree

def _decode(fmt, codes, scales):
    """The values that stored rows stand for, in float32."""
    if fmt == "bf16":
        return codes.float()
    if fmt == "e4m3":
        return torch.ldexp(codes.view(torch.float8_e4m3fn).float(), (scales.int() - 127).unsqueeze(-1))
    w = codes.int().unflatten(-1, (-1, 4))
    even, odd = w[..., 0] | (w[..., 1] << 8), w[..., 2] | (w[..., 3] << 8)
    at = torch.arange(4, device=codes.device, dtype=torch.int32) * 4
    c = torch.stack(((even.unsqueeze(-1) >> at) & 15, (odd.unsqueeze(-1) >> at) & 15), -1)
    g = c.flatten(-3).unflatten(-1, (-1, GROUP)).float()
    return (g * scales[..., 0:1].float() + scales[..., 1:2].float()).bfloat16().flatten(-2).float()


def _load(pool, p, at):
    scales = pool[p + "_scales"]
    return _decode(pool["fmt"], pool[p][0, at], None if scales is None else scales[0][:, at].transpose(0, 1))


def _slots_of(pages, page, n):
    """Pool rows of the first n keys of each page list [lists][pages] (unused pages read row 0)."""
    at = torch.arange(n, device=pages.device)
    return pages.clamp(min=0).long()[:, at // page] * page + at % page


def _plain_tree(s):
    c, q, pool, page = s["case"], s["q"].float(), s["pool"], s["page"]
    prefix, before, nodes, begin = s["host"]
    A, T, D = c["agents"], c["nodes"], c["dim"]
    q = q.view(A, T, c["heads"], c["group"], D)
    out = torch.zeros(A, T, c["heads"], c["group"], D, device="cuda")
    lse = torch.full((A, T, c["heads"], c["group"]), -math.inf, device="cuda")
    live = torch.arange(T, device="cuda") < s["nodes"][:, None]                            # [agents][T]
    for g in range(c["groups"]):
        a = slice(begin[g], begin[g + 1])
        most = max(b + n for b, n in zip(before[a], nodes[a]))
        # the group's shared keys once, its agents' own keys padded to the longest
        kp, vp = (_load(pool, p, _slots_of(s["prefix_pages"][g:g + 1], page, prefix[g])[0]) for p in PLANES)
        ks, vs = (_load(pool, p, _slots_of(s["suffix_pages"][a], page, most).flatten()).view(-1, most, c["heads"], D)
                  for p in PLANES)
        z = torch.cat((torch.einsum("athgd,khd->athgk", q[a], kp), torch.einsum("athgd,akhd->athgk", q[a], ks)), -1)
        z *= D ** -0.5
        # own key i is node i - first: seen where the mask's bit says so; before the tree by all
        first = (s["suffix_len"][a] - s["nodes"][a]).long()[:, None]
        node = torch.arange(most, device="cuda") - first                                   # [agents][most]
        bit = torch.gather(s["bits"][a], 2, node.clamp(0, T - 1)[:, None].expand(-1, T, -1))
        sees = (node < 0)[:, None] | ((node < s["nodes"][a][:, None])[:, None] & bit)      # [agents][T][most]
        sees = torch.cat((torch.ones(sees.shape[0], T, prefix[g], dtype=torch.bool, device="cuda"), sees), -1)
        z.masked_fill_(~(sees & live[a][:, :, None])[:, :, None, None], -math.inf)
        top = z.amax(-1, keepdim=True)
        p = (z - torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
        total = p.sum(-1, keepdim=True)
        o = torch.einsum("athgk,khd->athgd", p[..., :prefix[g]], vp) + \
            torch.einsum("athgk,akhd->athgd", p[..., prefix[g]:], vs)
        out[a] = torch.where(total > 0, o / total, torch.zeros_like(o))
        lse[a] = (top + total.log())[..., 0]
    return {"out": out.view(A, T, -1, D).to(torch.bfloat16), "lse": lse.view(A, T, -1)}


# ---- pages

def _copy_rows(pool, src, dst):
    """Rows src of every layer to rows dst, codes and scales."""
    for p in PLANES:
        pool[p][:, dst] = pool[p][:, src]
        if pool[p + "_scales"] is not None:
            pool[p + "_scales"][:, :, dst] = pool[p + "_scales"][:, :, src]


def _plain_extend(s):
    P, refs, pages, lens = s["page"], s["refs"], s["pages"], s["lens"]
    L, wide = pages.shape
    i = torch.arange(L, device="cuda")
    src, extra = s["parent"].long(), s["extra"].long()
    have_tokens = lens.long()[src]
    fork = src != i
    have, want = (have_tokens + P - 1) // P, (have_tokens + extra + P - 1) // P
    held = pages[src]                                                        # the pages each list begins with
    last = held.gather(1, (have - 1).clamp(min=0)[:, None])[:, 0].long().clamp(min=0)
    copy = (extra > 0) & (have_tokens % P != 0) & (fork | (refs[last] > 1))
    need = want - have + copy
    upto = need.cumsum(0)
    ok = (need == 0) | (upto <= (refs == 0).sum())
    free = torch.argsort((refs != 0).to(torch.int8), stable=True)            # free pages first, lowest first
    begin = upto - need
    # entry by entry: shared, a copy, or new
    col = torch.arange(wide, device="cuda")[None]
    copied = copy[:, None] & (col == have[:, None] - 1)
    new = copied | ((col >= have[:, None]) & (col < want[:, None]))
    rank = begin[:, None] + torch.where(copied, 0, copy[:, None] + col - have[:, None])
    table = torch.where(new, free[rank.clamp(0, refs.numel() - 1)].to(torch.int32),
                        torch.where(fork[:, None] & (col < have[:, None]), held, pages))
    shared = fork[:, None] & (col < have[:, None]) & ~copied & ok[:, None]
    new &= ok[:, None]
    rows = (torch.arange(P, device="cuda")[None] < (have_tokens % P)[:, None]) & (copy & ok)[:, None]
    lists, row = rows.nonzero(as_tuple=True)
    to = table.gather(1, (have - 1).clamp(min=0)[:, None])[:, 0].long()
    refs.index_add_(0, held[shared].long(), torch.ones_like(held[shared]))
    own_copy = copy & ok & ~fork
    refs.index_add_(0, last[own_copy], -torch.ones_like(last[own_copy], dtype=torch.int32))
    refs[table[new].long()] = 1
    pages.copy_(torch.where(ok[:, None], table, pages))
    lens.copy_(torch.where(ok, have_tokens + extra, lens.long()).to(torch.int32))
    _copy_rows(s["pool"], last[lists] * P + row, to[lists] * P + row)
    return _outputs(s)


def _plain_cut(s):
    P, refs, pages, lens = s["page"], s["refs"], s["pages"], s["lens"]
    base, kept, path = s["base"].long(), s["kept"].long(), s["path"].long()
    j = torch.arange(path.shape[1], device="cuda")
    lists, j = (j[None] < kept[:, None]).nonzero(as_tuple=True)
    src, dst = base[lists] + path[lists, j], base[lists] + j
    slot = lambda at: pages[lists, at // P].long() * P + at % P  # noqa: E731
    _copy_rows(s["pool"], slot(src), slot(dst))
    col = torch.arange(pages.shape[1], device="cuda")[None]
    end = base + kept
    gone = (col >= ((end + P - 1) // P)[:, None]) & (col < ((lens.long() + P - 1) // P)[:, None])
    given = pages[gone].long()
    refs.index_add_(0, given, -torch.ones_like(given, dtype=torch.int32))
    pages.masked_fill_(gone, -1)
    lens.copy_(end)
    return _outputs(s)


def _plain_compact(s):
    P, refs, pages, lens = s["page"], s["refs"], s["pages"], s["lens"]
    n = refs.numel()
    used = refs > 0
    live = used.sum()
    at = torch.arange(n, device="cuda")
    src = (used & (at >= live)).nonzero()[:, 0]
    dst = (~used & (at < live)).nonzero()[:, 0]
    to = at.to(torch.int32)
    to[src] = dst.to(torch.int32)
    row = torch.arange(P, device="cuda")
    _copy_rows(s["pool"], (src[:, None] * P + row).flatten(), (dst[:, None] * P + row).flatten())
    refs[dst] = refs[src]
    refs[src] = 0
    mine = torch.arange(pages.shape[1], device="cuda")[None] < ((lens + P - 1) // P)[:, None]
    pages.copy_(torch.where(mine, to[pages.long().clamp(min=0)], pages))
    return {**_outputs(s), "live": live.to(torch.int32).view(1)}


# ------------------------------------------------------------------ what a pass cannot do without

def _row_bytes(fmt, dim):
    return {"bf16": 2 * dim, "e4m3": dim + 1, "int4": dim // 2 + 4 * (dim // GROUP)}[fmt]


def work(case):
    c = case
    if c["op"] == "rotary":
        rows = c["chunks"] * c["layers"] * c["tokens"] * (c["q_heads"] + c["k_heads"])
        return {"bytes": 4 * rows * c["dim"] + 4 * c["chunks"] * c["tokens"], "flops": 3 * rows * c["rot"]}
    if c["op"] == "tree":
        prefix, before, nodes, begin = _tree_lengths(c)
        keys = sum(prefix) + sum(before) + sum(nodes)
        pairs = 0
        for g in range(c["groups"]):
            for a in range(begin[g], begin[g + 1]):
                # (a node's line of descent: about the logarithm of the tree)
                pairs += nodes[a] * (prefix[g] + before[a] + max(1, nodes[a]).bit_length())
        rows = c["agents"] * c["nodes"] * c["heads"] * c["group"]
        return {"bytes": 2 * keys * c["heads"] * _row_bytes(c["fmt"], c["dim"]) + rows * (4 * c["dim"] + 4)
                + 4 * (keys // c["page"]), "flops": 4 * pairs * c["heads"] * c["group"] * c["dim"]}
    P = c["page"]
    row = 2 * 2 * c["layers"] * c["heads"] * _row_bytes(c["fmt"], c["dim"])      # read and written, both planes
    if c["op"] == "extend":
        lens = _lengths(c)
        roots = lens[:c["roots"]]
        moved = sum(n % P for n in roots[:c["clones"]]) + sum(n % P for n in lens[c["roots"]:c["roots"] + c["clones"]])
        begins = [roots[i % c["roots"]] for i in range(c["forks"])]
        moved += sum(n % P for n in begins)
        table = sum(2 * (n + P - 1) // P for n in begins) + len(lens) * (2 + c["extra"] // P)
        return {"bytes": row * moved + 4 * (c["pages"] + table), "flops": 0}
    if c["op"] == "cut":
        moved = sum(max(0, c["keep"] - i % 4) for i in range(c["lists"]))
        given = sum((n + P - 1) // P for n in _lengths(c)[:c["gone"]]) + c["lists"] * (c["nodes"] // P)
        return {"bytes": row * moved * (1 - c["gone"] / c["lists"]) + 12 * (given + c["lists"]), "flops": 0}
    live = max(1, int(c["pages"] * c["use"]))
    moved = live * (c["pages"] - live) // c["pages"]                              # of a random set, on average
    return {"bytes": row * P * moved + 8 * (c["pages"] + live), "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(s)
    return _exact_tree(s) if case["op"] == "tree" else _exact_pages(s)


def _exact_rotary(s):
    """Pairs as complex numbers times m e^(i p theta), the frequencies one by one."""
    c, r, rot = s["case"], s["rope"], s["case"]["rot"]
    theta = []
    for i in range(rot // 2):
        t, k = r["base"] ** (-2.0 * i / rot), 1.0 / r["factor"]
        if c["scaling"] == "linear":
            t *= k
        elif c["scaling"] == "bands":
            turns = r["original"] * t / (2 * math.pi)
            if turns < r["low"]:
                t *= k
            elif turns <= r["high"]:
                x = (turns - r["low"]) / (r["high"] - r["low"])
                t = (1 - x) * t * k + x * t
        elif c["scaling"] == "yarn":
            # the pair whose frequency makes so many turns over the original context
            where = [math.log(r["original"] / (2 * math.pi * n)) / math.log(r["base"]) * rot / 2 for n in (r["high"], r["low"])]
            lo, hi = max(0, math.floor(where[0])), min(rot - 1, math.ceil(where[1]))
            x = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            t = x * t * k + (1 - x) * t
        theta.append(t)
    turn = torch.polar(torch.tensor(float(r["attention"]), dtype=torch.float64, device="cuda"),
                       s["positions"].double()[:, None, :, None, None] * torch.tensor(theta, dtype=torch.float64, device="cuda"))
    out = []
    for name in "qk":
        if s[name] is None:
            continue
        y = s[name].double()
        if c["layout"] == "half":
            z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * turn
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        else:
            z = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) * turn
            y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
        out.append(y)
    return out


def _half_even(x, digits, least):
    """x rounded to `digits` binary digits, ties to even, with no step below 2^least."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - digits).clamp(min=least).double())
    return (x / step).round() * step


def _stood_for(pool, p, rows):
    """Rows [rows][H][D] of a one-layer pool in 64 bits, from the bits."""
    codes = pool[p][0, rows]
    if pool["fmt"] == "bf16":
        return codes.double()
    scales = pool[p + "_scales"][0][:, rows].transpose(0, 1)
    if pool["fmt"] == "e4m3":
        b = codes.int()
        e, m = (b >> 3) & 15, (b & 7).double()
        size = torch.where(e > 0, (8 + m) * torch.exp2(e.double() - 10), m * 2.0 ** -9)
        return torch.where(b > 127, -size, size) * torch.exp2(scales.double() - 127)[..., None]
    D = pool["dim"]
    d = torch.arange(D, device="cuda")
    nibble = (d % 8) // 2 + 4 * (d % 2)
    byte = d // 8 * 4 + nibble // 2
    c = ((codes[..., byte].int() >> (4 * (nibble % 2)).int()) & 15).double()
    sz = scales.double().repeat_interleave(GROUP, dim=-2)
    return _half_even(c * sz[..., 0] + sz[..., 1], 8, -133)


def _exact_tree(s):
    c, page = s["case"], s["page"]
    prefix, before, nodes, begin = s["host"]
    A, T, H, G, D = c["agents"], c["nodes"], c["heads"], c["group"], c["dim"]
    if work(c)["flops"] > 2e12:
        return None
    out = torch.zeros(A, T, H * G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((A, T, H * G), -math.inf, dtype=torch.float64, device="cuda")
    words = s["words"].cpu().tolist()
    for g in range(c["groups"]):
        shared = (s["prefix_pages"][g].long()[:, None] * page + torch.arange(page, device="cuda")).flatten()
        shared = [_stood_for(s["pool"], p, shared[:prefix[g]]) for p in PLANES]
        for a in range(begin[g], begin[g + 1]):
            N = nodes[a]
            if N == 0:
                continue
            at = (s["suffix_pages"][a].long()[:, None] * page + torch.arange(page, device="cuda")).flatten()[:before[a] + N]
            k, v = (torch.cat((x, _stood_for(s["pool"], p, at))) for x, p in zip(shared, PLANES))
            hidden = torch.zeros(N, k.shape[0], dtype=torch.bool)
            for t in range(N):
                for j in range(N):
                    hidden[t, k.shape[0] - N + j] = not (j <= t and words[a][t][j // 32] >> (j % 32) & 1)
            hidden = hidden.cuda()
            for h in range(H):
                z = s["q"][a, :N, h * G:(h + 1) * G].double() @ k[:, h].T / math.sqrt(D)      # [N][G][n]
                z = torch.where(hidden[:, None], -math.inf, z)
                w = torch.logsumexp(z, -1)
                lse[a, :N, h * G:(h + 1) * G] = w
                seen = w > -math.inf
                w = torch.where(seen, w, torch.zeros_like(w))
                out[a, :N, h * G:(h + 1) * G] = torch.exp(z - w[..., None]) @ v[:, h] * seen[..., None]
    return {"out": out, "lse": lse}


def _exact_pages(s):
    """List after list on the host; then the rows that moved."""
    c, P = s["case"], s["page"]
    refs, pages, lens = (s[x].cpu().tolist() for x in ("refs", "pages", "lens"))
    moves = []                                                               # (from slot, to slot)
    take = lambda n: -(-n // P)  # noqa: E731
    if c["op"] == "extend":
        was = ([list(p) for p in pages], list(lens), list(refs))
        free = [p for p, r in enumerate(was[2]) if r == 0]
        for i, (src, extra) in enumerate(zip(s["parent"].tolist(), s["extra"].tolist())):
            n, mine = was[1][src], list(was[0][src][:take(was[1][src])])
            cow = extra > 0 and n % P and (src != i or was[2][mine[-1]] > 1)
            need = take(n + extra) - take(n) + bool(cow)
            if need > len(free):
                free = [] if need else free
                continue
            new, free = free[:need], free[need:]
            if src != i:
                for p in mine[:-1] if cow else mine:
                    refs[p] += 1
            elif cow:
                refs[mine[-1]] -= 1
            if cow:
                moves += [(mine[-1] * P + r, new[0] * P + r) for r in range(n % P)]
                mine[-1] = new.pop(0)
                refs[mine[-1]] = 1
            for p in new:
                refs[p] = 1
            mine += new
            pages[i][:len(mine)] = mine
            lens[i] = n + extra
    elif c["op"] == "cut":
        for i, (base, kept, path) in enumerate(zip(s["base"].tolist(), s["kept"].tolist(), s["path"].tolist())):
            slot = lambda at: pages[i][at // P] * P + at % P  # noqa: E731,B023
            moves += [(slot(base + path[j]), slot(base + j)) for j in range(kept)]
            for k in range(take(base + kept), take(lens[i])):
                refs[pages[i][k]] -= 1
                pages[i][k] = -1
            lens[i] = base + kept
    else:
        live = sum(r > 0 for r in refs)
        to = {}
        holes = [p for p in range(live) if refs[p] == 0]
        for p in range(live, len(refs)):
            if refs[p]:
                to[p] = holes.pop(0)
                refs[to[p]], refs[p] = refs[p], 0
                moves += [(p * P + r, to[p] * P + r) for r in range(P)]
        for i, n in enumerate(lens):
            for k in range(take(n)):
                pages[i][k] = to.get(pages[i][k], pages[i][k])
    src, dst = (torch.tensor([m[k] for m in moves], dtype=torch.long, device="cuda") for k in (0, 1))
    pool, out = s["pool"], dict(refs=torch.tensor(refs), pages=torch.tensor(pages), lens=torch.tensor(lens))
    for p in PLANES:
        if pool["fmt"] == "int4":
            out[p] = None                                                    # whole numbers
        else:
            x = pool[p].view(torch.float8_e4m3fn) if pool["fmt"] == "e4m3" else pool[p]
            out[p] = x.to(torch.float64)
            out[p].index_copy_(1, dst, out[p].index_select(1, src))
        if pool["fmt"] == "e4m3":
            x = torch.exp2(pool[p + "_scales"].double() - 127)
        elif pool["fmt"] == "int4":
            x = pool[p + "_scales"].double()
        else:
            continue
        out[p + "_scales"] = x.index_copy(2, dst, x.index_select(2, src))
    if c["op"] == "compact":
        out["live"] = torch.tensor([live])
    return out
