"""Workloads of the paged-pool operators: writing a cache into a pool (bf16, e4m3 or int4),
reading it back, and the attention of a round's agents over a shared prefix and their own
tokens.

`run` computes them in plain torch (`own` false) or through the library's entry points
(`own` true) on what `prepare` makes; `work` counts the bytes and operations a pass cannot do
without; `exact` restates the definitions in 64 bits.

Formats of a stored row (one token, one KV head, D values):
  bf16  the values.
  e4m3  one byte per value and one byte b per row: value = e4m3(code) * 2^(b - 127).  With A
        the row's largest finite magnitude, 2^(b-127) is the smallest power of two with
        A <= 448 * 2^(b-127), kept within [2^-110, 2^119]; codes round to nearest even and
        infinities saturate.
  int4  groups of 32 values share a bf16 scale and a bf16 zero: value = bf16(scale*code + zero),
        zero = min, scale = bf16((max - min) / 15), code = rint((x - zero) * (1 / scale)) in
        [0, 15].  Each 32-bit word holds 8 codes: value 2i in nibble i, value 2i+1 in nibble
        i + 4.
"""
import math

import torch

own = False

FORMATS = ("bf16", "e4m3", "int4")
GROUP = 32
PLANES = ("k", "v")


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step's new rows of a 16-agent round, one layer: launch latency
        dict(name="write_step_e4m3", op="write", fmt="e4m3", chunks=16, layers=1, tokens=1, heads=8, dim=128,
             rotate=False, skip=0.0),
        # a 4096-token chunk of a 32-layer cache moved to its place in the shared prefix
        dict(name="write_chunk_e4m3", op="write", fmt="e4m3", chunks=1, layers=32, tokens=4096, heads=8, dim=128,
             rotate=True, skip=0.0),
        # ragged blocks with rows that are not kept, at canonical positions
        dict(name="write_ragged_int4", op="write", fmt="int4", chunks=3, layers=9, tokens=1237, heads=5, dim=64,
             rotate=False, skip=0.1),
        # eight 512-token blocks of a 48-layer cache read back at new positions
        dict(name="read_blocks_e4m3", op="read", fmt="e4m3", chunks=8, layers=48, tokens=512, heads=8, dim=128,
             rotate=True, skip=0.0),
        # odd blocks, odd heads, some rows absent
        dict(name="read_ragged_int4", op="read", fmt="int4", chunks=2, layers=7, tokens=333, heads=5, dim=128,
             rotate=True, skip=0.2),
        # one agent on a 256-token block: the smallest decode call
        dict(name="attend_tiny_bf16", op="attend", fmt="bf16", agents=1, groups=1, new=1, heads=4, group=2, dim=64,
             page=16, prefix=256, own_lo=9, own_hi=9),
        # a round's decode step: 8 agents, 8 shared blocks of 512, ragged histories
        dict(name="attend_round_bf16", op="attend", fmt="bf16", agents=8, groups=1, new=1, heads=8, group=5, dim=128,
             page=16, prefix=4096, own_lo=200, own_hi=3000),
        # 16 agents over a long shared context, short histories
        dict(name="attend_long_bf16", op="attend", fmt="bf16", agents=16, groups=1, new=1, heads=8, group=8, dim=128,
             page=16, prefix=131072, own_lo=16, own_hi=1024),
        # the same cache in 8 bits
        dict(name="attend_long_e4m3", op="attend", fmt="e4m3", agents=16, groups=1, new=1, heads=8, group=8, dim=128,
             page=16, prefix=131072, own_lo=16, own_hi=1024),
        # two draft tokens of five agents, odd lengths, 4 bits
        dict(name="attend_draft_int4", op="attend", fmt="int4", agents=5, groups=1, new=2, heads=8, group=5, dim=128,
             page=16, prefix=16383, own_lo=2, own_hi=700),
        # three groups with prefixes of their own, agents whose histories dominate
        dict(name="attend_own_e4m3", op="attend", fmt="e4m3", agents=48, groups=3, new=1, heads=8, group=4, dim=128,
             page=32, prefix=2048, own_lo=0, own_hi=4000),
        # 256 new tokens of each of 8 agents at once (a message that every agent answers)
        dict(name="attend_message_bf16", op="attend", fmt="bf16", agents=8, groups=1, new=256, heads=8, group=4,
             dim=128, page=16, prefix=8192, own_lo=256, own_hi=768),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("write", "read", "attend", "attend"))
    if op != "attend":
        fmt = rng.choice(FORMATS)
        heads, dim = rng.choice((1, 2, 4, 5, 8)), rng.choice((64, 128))
        chunks, layers = _log(rng, 1, 16), _log(rng, 1, 32)
        most = max(1, min(8192, (32 * 4096 * 8 * 128) // (chunks * layers * heads * dim)))
        tokens = _log(rng, 1, most)
        # int4 rows are written as cached (rotation comes with reading), so that codes compare exactly
        rotate = rng.random() < 0.5 and not (op == "write" and fmt == "int4")
        return dict(op=op, fmt=fmt, chunks=chunks, layers=layers, tokens=tokens, heads=heads, dim=dim, rotate=rotate,
                    skip=rng.choice((0.0, 0.0, 0.15)))
    fmt = rng.choice(FORMATS)
    heads, dim = rng.choice((1, 2, 4, 8)), rng.choice((64, 128))
    group = rng.choice((1, 2, 4, 5, 8))
    agents = _log(rng, 1, 48)
    new = rng.choice((1, 1, 1, 2, 3, 17, _log(rng, 4, 200)))
    rows = agents * new * heads * group
    cap = max(64, min(131072, int(1.2e9 / rows)))    # query rows x keys: at most about the longest listed case's
    prefix = rng.choice((0, _log(rng, 1, cap), _log(rng, 64, cap)))
    own_hi = max(new, _log(rng, 1, max(2, min(4000, cap))))
    return dict(op=op, fmt=fmt, agents=agents, groups=min(agents, rng.choice((1, 1, 2, 3))), new=new, heads=heads,
                group=group, dim=dim, page=rng.choice((16, 32, 64, 128)), prefix=prefix,
                own_lo=rng.choice((0, new)), own_hi=own_hi)


# ------------------------------------------------------------------ what a program holds before the call

def _lengths(c):
    """Prefix lengths of the groups, own lengths of the agents, first agent of each group
    (from the case alone: a program knows them on the host)."""
    g, a = c["groups"], c["agents"]
    prefix = [c["prefix"] if i == 0 else c["prefix"] * (g - i) // g - (i if c["prefix"] else 0) for i in range(g)]
    prefix = [max(0, p) for p in prefix]
    lo, hi = c["own_lo"], c["own_hi"]
    # a low-discrepancy spread over [lo, hi], both ends among them
    mine = [lo + int(round((hi - lo) * ((i * 0.6180339887498949) % 1.0))) for i in range(a)]
    mine[-1] = hi
    begin = [i * a // g for i in range(g)] + [a]
    return prefix, mine, begin


def _positions(c):
    """Slots of [chunks][tokens] rows before they are shuffled: -1 where the row is not kept."""
    n = c["chunks"] * c["tokens"]
    slots = (n + 15) // 16 * 16 + 16
    return n, slots


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _cache_rows(gen, lead, heads, dim):
    """Keys and values as caches hold them: some channels of the keys run several times the
    others' size (they differ by head), values have small means."""
    gain = torch.ones(heads, dim, device="cuda")
    gain[torch.rand(heads, dim, generator=gen, device="cuda") < 0.04] = 4.0
    k = (_normal(gen, *lead, heads, dim) * gain).to(torch.bfloat16)
    v = (_normal(gen, *lead, heads, dim) + 0.25 * _normal(gen, heads, dim)).to(torch.bfloat16)
    return k, v


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    if c["op"] == "attend":
        return _prepare_attend(c, gen)
    n, slots = _positions(c)
    C, L, T, H, D = c["chunks"], c["layers"], c["tokens"], c["heads"], c["dim"]
    order = torch.randperm(slots, generator=gen, device="cuda")[:n].to(torch.int32)
    keep = torch.rand(n, generator=gen, device="cuda") >= c["skip"]
    if c["skip"] == 0.0:
        keep[:] = True
    slot_mapping = torch.where(keep, order, torch.full_like(order, -1)).view(C, T)
    delta = torch.randint(500, 8000, (C,), generator=gen, device="cuda", dtype=torch.int32) if c["rotate"] else None
    s = dict(case=c, slot_mapping=slot_mapping, delta=delta, rope_base=5e5,
             rows=keep.nonzero()[:, 0], slots=order[keep].long())
    if c["op"] == "write":
        s["k"], s["v"] = _cache_rows(gen, (C, L, T), H, D)
        s["pool"] = _pool_zeros(c["fmt"], L, slots, H, D)
    else:
        s["pool"] = _pool_zeros(c["fmt"], L, slots, H, D)
        for layer in range(L):
            for p, x in zip(PLANES, _cache_rows(gen, (slots,), H, D)):
                _store(s["pool"], p, layer, slice(None), _encode(c["fmt"], x))
        # rows that are not read keep what the caller's buffers hold
        s["k_out"] = torch.zeros(C, L, T, H, D, dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.zeros(C, L, T, H, D, dtype=torch.bfloat16, device="cuda")
    return s


def _prepare_attend(c, gen):
    prefix, mine, begin = _lengths(c)
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
    pool = _pool_zeros(c["fmt"], 1, total * P, H, D)
    for p, x in zip(PLANES, _cache_rows(gen, (total * P,), H, D)):
        _store(pool, p, 0, slice(None), _encode(c["fmt"], x))
    q = (1.5 * _normal(gen, c["agents"], c["new"], H * c["group"], D)).to(torch.bfloat16)
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(case=c, q=q, pool=pool, page=P, prefix_pages=prefix_pages, suffix_pages=own_pages,
                prefix_len=torch.tensor(prefix, **i32), suffix_len=torch.tensor(mine, **i32),
                group_begin=torch.tensor(begin, **i32), host=(prefix, mine, begin))


def _pool_zeros(fmt, layers, slots, heads, dim):
    z = lambda *shape, dtype: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
    pool = dict(fmt=fmt, slots=slots, heads=heads, dim=dim, layers=layers)
    for p in PLANES:
        if fmt == "bf16":
            pool[p], pool[p + "_scales"] = z(layers, slots, heads, dim, dtype=torch.bfloat16), None
        elif fmt == "e4m3":
            pool[p] = z(layers, slots, heads, dim, dtype=torch.uint8)
            pool[p + "_scales"] = z(layers, heads, slots, dtype=torch.uint8)
        else:
            pool[p] = z(layers, slots, heads, dim // 2, dtype=torch.uint8)
            pool[p + "_scales"] = z(layers, heads, slots, dim // GROUP, 2, dtype=torch.bfloat16)
    return pool


# ------------------------------------------------------------------ the formats in plain torch

def _encode(fmt, x):
    """bf16 rows [..., heads, dim] -> (codes, scales) with scales [..., heads(, groups, 2)]."""
    if fmt == "bf16":
        return x, None
    f = x.float()
    fine = torch.isfinite(f)
    if fmt == "e4m3":
        big = torch.where(fine, f.abs(), torch.zeros_like(f)).amax(-1)
        m, e = torch.frexp(big)
        k = torch.where(m <= 0.875, e - 9, e - 8)                       # big <= 448 * 2^k
        k = torch.where(big > 0, k, torch.full_like(k, -110)).clamp(-110, 119)
        y = torch.ldexp(f, -k.unsqueeze(-1)).clamp(-448.0, 448.0)
        return y.to(torch.float8_e4m3fn).view(torch.uint8), (k + 127).to(torch.uint8)
    g = f.unflatten(-1, (-1, GROUP))
    fine = fine.unflatten(-1, (-1, GROUP))
    some = fine.any(-1)
    lo = torch.where(fine, g, torch.full_like(g, math.inf)).amin(-1)
    hi = torch.where(fine, g, torch.full_like(g, -math.inf)).amax(-1)
    lo, hi = torch.where(some, lo, 0.0), torch.where(some, hi, 0.0)
    scale = ((hi - lo).clamp(max=torch.finfo(torch.float32).max) / 15.0).bfloat16().float()
    scale = torch.where(scale < 2.0 ** -120, torch.zeros_like(scale), scale)
    inv = torch.where(scale > 0, 1.0 / scale, torch.zeros_like(scale))
    code = torch.nan_to_num(((g - lo.unsqueeze(-1)) * inv.unsqueeze(-1)).round(), nan=0.0).clamp(0, 15)
    c = code.flatten(-2).to(torch.int32).unflatten(-1, (-1, 4, 2))      # word, i, (2i, 2i + 1)
    at = torch.arange(4, device=x.device, dtype=torch.int32) * 4
    # nibbles 0..3 hold the even values, 4..7 the odd ones: bytes 0, 1 and 2, 3 of a word
    even, odd = (c[..., 0] << at).sum(-1), (c[..., 1] << at).sum(-1)
    b = torch.stack((even & 255, even >> 8, odd & 255, odd >> 8), -1).flatten(-2)
    return b.to(torch.uint8), torch.stack((scale, lo), -1).bfloat16()


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


def _store(pool, p, layer, at, coded):
    codes, scales = coded
    pool[p][layer, at] = codes
    if scales is not None:
        pool[p + "_scales"][layer][:, at] = scales.transpose(0, 1)


def _load(pool, p, layer, at):
    scales = pool[p + "_scales"]
    return _decode(pool["fmt"], pool[p][layer, at],
                   None if scales is None else scales[layer][:, at].transpose(0, 1))


def _rotate(x, delta, base):
    """Rotate-half RoPE by delta[c] of rows [c][...][heads][dim], in 64 bits (far angles)."""
    D = x.shape[-1]
    theta = base ** (-2.0 * torch.arange(D // 2, dtype=torch.float64, device=x.device) / D)
    a = delta.double()[:, None] * theta
    a = a.view(x.shape[0], *([1] * (x.dim() - 2)), D // 2)
    lo, hi = x[..., :D // 2].double(), x[..., D // 2:].double()
    return torch.cat((lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()), -1).to(torch.bfloat16)


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"write": _own_write, "read": _own_read, "attend": _own_attend}[op](state)
    return {"write": _plain_write, "read": _plain_read, "attend": _plain_attend}[op](state)


def _outputs(pool):
    """The pool's planes; 8-bit codes and scales as the values they stand for."""
    out = {}
    for p in PLANES:
        e4m3 = pool["fmt"] == "e4m3"
        out[p] = pool[p].view(torch.float8_e4m3fn) if e4m3 else pool[p]
        if pool[p + "_scales"] is not None:
            s = pool[p + "_scales"]
            out[p + "_scales"] = s.view(torch.float8_e8m0fnu) if e4m3 else s
    return out


def _own_pool(pool):
    from cross_context_kv_gb300 import kvfix
    return kvfix.Pool(pool["fmt"], pool["k"], pool["v"], pool["k_scales"], pool["v_scales"])


def _own_write(s):
    from cross_context_kv_gb300 import kvfix
    kvfix.pool_write(_own_pool(s["pool"]), s["k"], s["v"], s["slot_mapping"], delta=s["delta"],
                     rope_base=s["rope_base"])
    return _outputs(s["pool"])


def _own_read(s):
    from cross_context_kv_gb300 import kvfix
    k, v = kvfix.pool_read(_own_pool(s["pool"]), s["slot_mapping"], delta=s["delta"], rope_base=s["rope_base"],
                           k_out=s["k_out"], v_out=s["v_out"])
    return {"k": k, "v": v}


def _own_attend(s):
    from cross_context_kv_gb300 import kvfix
    out, lse = kvfix.shared_attend(s["q"], _own_pool(s["pool"]), s["page"], s["suffix_pages"], s["suffix_len"],
                                   s["prefix_pages"], s["prefix_len"], s["group_begin"], return_lse=True)
    return {"out": out, "lse": lse}


def _plain_write(s):
    pool = s["pool"]
    for p, x in (("k", s["k"]), ("v", s["v"])):
        if p == "k" and s["delta"] is not None:
            x = _rotate(x, s["delta"], s["rope_base"])
        codes, scales = _encode(pool["fmt"], x)
        # [C][L][T] rows -> [L][C*T], the kept ones to their slots
        pool[p][:, s["slots"]] = codes.transpose(0, 1).flatten(1, 2)[:, s["rows"]]
        if scales is not None:
            pool[p + "_scales"][:, :, s["slots"]] = \
                scales.transpose(0, 1).flatten(1, 2)[:, s["rows"]].transpose(1, 2)
    return _outputs(pool)


def _plain_read(s):
    pool, c = s["pool"], s["case"]
    out = {}
    for p in PLANES:
        scales = pool[p + "_scales"]
        x = _decode(pool["fmt"], pool[p][:, s["slots"]],
                    None if scales is None else scales[:, :, s["slots"]].transpose(1, 2))   # [L][kept][H][D]
        if p == "k" and s["delta"] is not None:
            x = _rotate(x.transpose(0, 1), s["delta"][s["rows"] // c["tokens"]], s["rope_base"]).transpose(0, 1)
        o = s[p + "_out"]
        rows = o.transpose(0, 1).reshape(c["layers"], -1, c["heads"], c["dim"])
        rows[:, s["rows"]] = x.to(torch.bfloat16)
        o.copy_(rows.view(c["layers"], c["chunks"], c["tokens"], c["heads"], c["dim"]).transpose(0, 1))
        out[p] = o
    return out


def _slots_of(pages, page, n):
    """Pool rows of the first n keys of each page list [lists][pages] (unused pages read row 0)."""
    at = torch.arange(n, device=pages.device)
    return pages.clamp(min=0).long()[:, at // page] * page + at % page


def _plain_attend(s):
    c, q, pool, page = s["case"], s["q"].float(), s["pool"], s["page"]
    prefix, mine, begin = s["host"]
    A, T, D = c["agents"], c["new"], c["dim"]
    q = q.view(A, T, c["heads"], c["group"], D)
    out = torch.zeros(A, T, c["heads"], c["group"], D, device="cuda")
    lse = torch.full((A, T, c["heads"], c["group"]), -math.inf, device="cuda")
    step = torch.arange(T, device="cuda")
    for g in range(c["groups"]):
        a = slice(begin[g], begin[g + 1])
        most = max(mine[a])
        # the group's shared keys once, its agents' own keys padded to the longest
        kp, vp = (_load(pool, p, 0, _slots_of(s["prefix_pages"][g:g + 1], page, prefix[g])[0]) for p in PLANES)
        ks, vs = (_load(pool, p, 0, _slots_of(s["suffix_pages"][a], page, most).flatten())
                  .view(-1, most, c["heads"], D) for p in PLANES)
        z = torch.cat((torch.einsum("athgd,khd->athgk", q[a], kp), torch.einsum("athgd,akhd->athgk", q[a], ks)), -1)
        z *= D ** -0.5
        # query t of an agent sees its prefix and own keys up to its own place
        sees = prefix[g] + s["suffix_len"][a].long()[:, None] - T + 1 + step           # [agents][T]
        key = torch.arange(prefix[g] + most, device="cuda")
        z.masked_fill_((key >= sees[..., None])[:, :, None, None], -math.inf)
        if z.shape[-1]:
            top = z.amax(-1, keepdim=True)
            p = (z - torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
            total = p.sum(-1, keepdim=True)
            o = torch.einsum("athgk,khd->athgd", p[..., :prefix[g]], vp) + \
                torch.einsum("athgk,akhd->athgd", p[..., prefix[g]:], vs)
            out[a] = torch.where(total > 0, o / total, torch.zeros_like(o))
            lse[a] = (top + total.log())[..., 0]
    return {"out": out.view(A, T, -1, D).to(torch.bfloat16), "lse": lse.view(A, T, -1)}


# ------------------------------------------------------------------ what a pass cannot do without

def _row_bytes(fmt, dim):
    return {"bf16": 2 * dim, "e4m3": dim + 1, "int4": dim // 2 + 4 * (dim // GROUP)}[fmt]


def work(case):
    c = case
    if c["op"] != "attend":
        n = c["chunks"] * c["tokens"]
        kept = n * (1.0 - c["skip"])
        rows = 2 * kept * c["layers"] * c["heads"]
        return {"bytes": rows * (2 * c["dim"] + _row_bytes(c["fmt"], c["dim"])) + 4 * n, "flops": 0}
    prefix, mine, begin = _lengths(c)
    T = c["new"]
    keys = sum(prefix) + sum(mine)
    pairs = 0
    for g in range(c["groups"]):
        for a in range(begin[g], begin[g + 1]):
            sees = [max(0, prefix[g] + mine[a] - T + 1 + t) for t in range(T)]
            pairs += sum(sees)
    rows = c["agents"] * T * c["heads"] * c["group"]
    return {"bytes": 2 * keys * c["heads"] * _row_bytes(c["fmt"], c["dim"]) + rows * (4 * c["dim"] + 4)
            + 4 * (keys // c["page"]),
            "flops": 4 * pairs * c["heads"] * c["group"] * c["dim"]}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"write": _exact_write, "read": _exact_read, "attend": _exact_attend}[case["op"]](s)


def _turned(x, delta, base):
    """Rows [c][l][t][h][d] in 64 bits, turned pair by pair as complex numbers."""
    D = x.shape[-1]
    angle = torch.tensor([base ** (-2.0 * i / D) for i in range(D // 2)], dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       delta.double()[:, None, None, None, None] * angle)
    z = torch.complex(x[..., :D // 2], x[..., D // 2:]) * turn
    return torch.cat((z.real, z.imag), -1)


def _half_even(x, digits, least):
    """x rounded to `digits` binary digits, ties to even, with no step below 2^least."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - digits).clamp(min=least).double())
    return (x / step).round() * step


def _exact_write(s):
    pool, c = s["pool"], s["case"]
    out = {}
    for p in PLANES:
        x = s[p].double()
        if p == "k" and s["delta"] is not None:
            x = _half_even(_turned(x, s["delta"], s["rope_base"]), 8, -133)   # the rotated bf16 key
        rows = x.transpose(0, 1).flatten(1, 2)[:, s["rows"]]
        if c["fmt"] == "bf16":
            out[p] = torch.zeros(pool[p].shape, dtype=torch.float64, device="cuda")
            out[p][:, s["slots"]] = rows
        elif c["fmt"] == "e4m3":
            A = rows.abs().amax(-1)
            m, e = torch.frexp((A / 448).clamp(min=2.0 ** -140))
            k = (e - (m == 0.5).int()).clamp(-110, 119).double()            # ceil(log2(A / 448))
            out[p] = torch.zeros(pool[p].shape, dtype=torch.float64, device="cuda")
            out[p][:, s["slots"]] = _half_even(rows / torch.exp2(k)[..., None], 4, -9)
            scales = torch.full(pool[p + "_scales"].shape, 2.0 ** -127, dtype=torch.float64, device="cuda")
            scales[:, :, s["slots"]] = torch.exp2(k).transpose(1, 2)
            out[p + "_scales"] = scales
        else:
            g = rows.unflatten(-1, (-1, GROUP))
            lo, hi = g.amin(-1), g.amax(-1)
            out[p] = None                                                   # whole numbers
            scales = torch.zeros(pool[p + "_scales"].shape, dtype=torch.float64, device="cuda")
            scales[:, :, s["slots"]] = torch.stack((_half_even((hi - lo) / 15, 8, -133), lo), -1).transpose(1, 2)
            out[p + "_scales"] = scales
    return out


def _stood_for(pool, p, rows):
    """Layer-major rows [L][rows][H][D] of a pool in 64 bits, from the bits."""
    codes = pool[p][:, rows]
    if pool["fmt"] == "bf16":
        return codes.double()
    scales = pool[p + "_scales"][:, :, rows].transpose(1, 2)
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


def _exact_read(s):
    c, out = s["case"], {}
    for p in PLANES:
        full = torch.zeros(c["layers"], c["chunks"] * c["tokens"], c["heads"], c["dim"], dtype=torch.float64,
                           device="cuda")
        full[:, s["rows"]] = _stood_for(s["pool"], p, s["slots"])
        full = full.view(c["layers"], c["chunks"], c["tokens"], c["heads"], c["dim"]).transpose(0, 1)
        out[p] = _turned(full, s["delta"], s["rope_base"]) if p == "k" and s["delta"] is not None else full
    return out


def _exact_attend(s):
    c, page = s["case"], s["page"]
    prefix, mine, begin = s["host"]
    A, T, H, G, D = c["agents"], c["new"], c["heads"], c["group"], c["dim"]
    if work(c)["flops"] > 2e12:
        return None
    out = torch.zeros(A, T, H * G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((A, T, H * G), -math.inf, dtype=torch.float64, device="cuda")
    for g in range(c["groups"]):
        shared = (s["prefix_pages"][g].long()[:, None] * page + torch.arange(page, device="cuda")).flatten()
        shared = [_stood_for(s["pool"], p, shared[:prefix[g]])[0] for p in PLANES]
        for a in range(begin[g], begin[g + 1]):
            at = (s["suffix_pages"][a].long()[:, None] * page + torch.arange(page, device="cuda")).flatten()[:mine[a]]
            k, v = (torch.cat((x, _stood_for(s["pool"], p, at)[0])) for x, p in zip(shared, PLANES))
            n = k.shape[0]
            place = n - T + torch.arange(T, device="cuda")
            hidden = torch.arange(n, device="cuda") > place[:, None]
            for h in range(H):
                z = s["q"][a, :, h * G:(h + 1) * G].double() @ k[:, h].T / math.sqrt(D)      # [T][G][n]
                z = torch.where(hidden[:, None], -math.inf, z)
                w = torch.logsumexp(z, -1) if n else torch.full((T, G), -math.inf, dtype=torch.float64, device="cuda")
                lse[a, :, h * G:(h + 1) * G] = w
                seen = w > -math.inf
                w = torch.where(seen, w, torch.zeros_like(w))
                out[a, :, h * G:(h + 1) * G] = torch.exp(z - w[..., None]) @ v[:, h] * seen[..., None]
    return {"out": out, "lse": lse}
