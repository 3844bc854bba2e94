"""kvfix_shared_attend against its definition in 64 bits, on the values the pool stands for.

Tolerance of an output, from the arithmetic the call states: one rounding to bf16 (2^-8 of the
value), the softmax weights rounded to bf16 before the product with the values (2^-8 of the
weighted mean V of |v|), float sums over D products in a logit (at most D 2^-24 of the sum of
their magnitudes, entering each weight by its exponential, in numerator and denominator) and
over the keys (n 2^-24 of V), and 2^-22 for each exponential.
"""
import ctypes

import numpy as np
import pytest
import torch

import pool_ref as ref

FORMATS = ("bf16", "e4m3", "int4")
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvfix():
    from cross_context_kv_gb300 import build
    build.build()
    from cross_context_kv_gb300 import kvfix
    return kvfix


def words_of(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


class Round:
    """A pool with a prefix per group and own keys per agent on shuffled pages; every row that
    belongs to no key holds NaN (bf16), NaN codes (e4m3) or wild scales (int4)."""

    def __init__(self, kvfix, fmt, heads, group, dim, page, new, prefix, begin, own, seed=0, spare=3):
        self.kvfix, self.fmt, self.page, self.new, self.group = kvfix, fmt, page, new, group
        self.prefix, self.begin, self.own = list(prefix), list(begin), list(own)
        A, r = len(own), np.random.default_rng(seed)
        pages = lambda n: -(-n // page)  # noqa: E731
        total = sum(map(pages, self.prefix)) + sum(map(pages, self.own)) + spare
        order, at = r.permutation(total).astype(np.int32), 0
        self.tables = []
        for lens in (self.prefix, self.own):
            wide = max([1] + [pages(n) for n in lens]) + 1
            t = np.full((len(lens), wide), 1 << 30, np.int32)      # entries past a length are not read
            for i, n in enumerate(lens):
                t[i, :pages(n)] = order[at:at + pages(n)]
                at += pages(n)
            self.tables.append(t)
        slots = total * page
        self.pool = kvfix.pool_empty(fmt, 1, slots, heads, dim)
        used = np.zeros(slots, bool)
        for t, lens in zip(self.tables, (self.prefix, self.own)):
            for i, n in enumerate(lens):
                used[self.rows(t[i], n)] = True
        k = ref.bf16_of(r.standard_normal((1, 1, slots, heads, dim)) * np.where(r.random(dim) < 0.05, 4.0, 1.0))
        v = ref.bf16_of(r.standard_normal((1, 1, slots, heads, dim)) + 0.25)
        put = lambda w: torch.from_numpy(w.view(np.int16)).cuda().view(torch.bfloat16)  # noqa: E731
        kvfix.pool_write(self.pool, put(k), put(v), torch.arange(slots, dtype=torch.int32, device="cuda").view(1, -1))
        free = torch.from_numpy(~used).cuda()
        if fmt == "bf16":
            for t in self.pool[1:3]:
                t[:, free] = float("nan")
        elif fmt == "e4m3":
            for t in self.pool[1:3]:
                t[:, free] = 0x7F
            for t in self.pool[3:]:
                t[:, :, free] = 0xFF
        else:
            for t in self.pool[3:]:
                t[:, :, free] = float("nan")
        self.q_words = ref.bf16_of(1.5 * r.standard_normal((A, new, heads * group, dim)))
        self.q = put(self.q_words)
        i32 = lambda x: torch.tensor(np.asarray(x, np.int32), device="cuda")  # noqa: E731
        self.args = dict(suffix_pages=i32(self.tables[1]), suffix_len=i32(self.own))
        if self.prefix:
            self.args.update(prefix_pages=i32(self.tables[0]), prefix_len=i32(self.prefix),
                             group_begin=i32(self.begin))
        self.scale = dim ** -0.5

    def rows(self, table, n):
        i = np.arange(n)
        return table[i // self.page].astype(np.int64) * self.page + i % self.page

    def call(self, **kw):
        return self.kvfix.shared_attend(self.q, self.pool, self.page, **{**self.args, "return_lse": True, **kw})

    def values(self, p):
        codes = getattr(self.pool, p)
        codes = words_of(codes) if codes.dtype == torch.bfloat16 else codes.cpu().numpy()
        s = getattr(self.pool, p + "_scales")
        if s is not None:
            s = np.moveaxis(words_of(s) if s.dtype == torch.bfloat16 else s.cpu().numpy(), 1, 2)[0]
        return lambda at: ref.decode(self.fmt, codes[0, at], None if s is None else s[at])

    def check(self, out, lse, absent=()):
        """`absent`: (agent, key place) pairs that count as not there."""
        K, V, q = self.values("k"), self.values("v"), ref.of_bf16(self.q_words)
        got, got_lse = ref.of_bf16(words_of(out)), lse.cpu().numpy().astype(np.float64)
        T = self.new
        for a in range(len(self.own)):
            g = next((g for g in range(len(self.prefix)) if self.begin[g] <= a < self.begin[g + 1]), None)
            n0 = 0 if g is None else self.prefix[g]
            at = np.concatenate((self.rows(self.tables[0][g], n0) if n0 else np.zeros(0, np.int64),
                                 self.rows(self.tables[1][a], self.own[a])))
            gone = {p for b, p in absent if b == a}
            keep = np.array([i for i in range(len(at)) if i not in gone], np.int64)
            k, v = K(at[keep]), V(at[keep])
            n = len(at)
            sees = np.array([np.searchsorted(keep, n - T + 1 + t) for t in range(T)])
            want, want_lse = ref.attend(q[a], k, v, sees, self.scale)
            mean, _ = ref.attend(q[a], k, np.abs(v), sees, self.scale)
            mags, D = np.zeros(want_lse.shape), q.shape[-1]
            for h in range(q.shape[2]):
                if len(keep):
                    mags[:, h] = (np.abs(q[a, :, h]) @ np.abs(k[:, h // self.group]).T).max(-1)
            z = D * 2.0 ** -24 * mags * self.scale + 2.0 ** -22
            tol = 2.0 ** -8 * (np.abs(want) + mean) + (2 * z + (n + 8) * 2.0 ** -23)[..., None] * mean
            err = np.abs(got[a] - want)
            assert (err <= tol).all(), f"agent {a}: {np.nanmax(err - tol)} over, at {np.argwhere(~(err <= tol))[:4]}"
            empty = want_lse == -np.inf
            assert (got_lse[a][empty] == -np.inf).all() and (got[a][empty] == 0).all()
            err = np.abs(got_lse[a][~empty] - want_lse[~empty])
            tol = (z + n * 2.0 ** -24 + np.where(empty, 0, np.abs(want_lse)) * 2.0 ** -22 + 2.0 ** -21)[~empty]
            assert (err <= tol).all(), f"agent {a}: lse {np.max(err - tol)} over"


CASES = {
    # heads, group, dim, page, new, prefix lengths, group_begin, own lengths
    "one_key": (1, 1, 64, 16, 1, [], [], [1]),
    "one_agent": (2, 4, 128, 16, 1, [256], [0, 1], [9]),
    "ragged": (2, 5, 128, 16, 1, [300], [0, 5], [0, 1, 17, 128, 333]),
    "pages_of_128": (1, 8, 64, 128, 1, [129], [0, 3], [127, 128, 130]),
    "groups": (4, 1, 64, 32, 1, [64, 0, 1, 200], [0, 2, 3, 3, 6], [5, 0, 70, 0, 31, 90]),
    "some_outside": (2, 2, 64, 16, 1, [40], [1, 3], [3, 0, 8, 20, 0]),
    "empty_rows": (2, 2, 64, 16, 3, [1], [0, 2], [0, 1, 0, 2]),
    "drafts": (2, 5, 128, 16, 2, [511], [0, 3], [2, 40, 129]),
    "many_new": (1, 4, 64, 16, 70, [100], [0, 2], [70, 200]),
    "many_rows": (1, 8, 128, 16, 1, [700], [0, 40], [3 * i for i in range(40)]),
    "message": (1, 2, 128, 64, 150, [130], [0, 2], [150, 400]),
    "long": (1, 3, 64, 16, 1, [3001], [0, 2], [2, 900]),
    # more tiles than the work in flight on an SM, halves of an SM that end far apart
    "uneven": (8, 1, 64, 16, 1, [40000], [0, 8], [0, 3000, 5, 1, 2000, 0, 64, 1300]),
    "uneven_pairs": (4, 40, 64, 64, 4, [9000], [0, 2], [4, 2500]),
    "seven_heads": (3, 7, 64, 16, 4, [31], [0, 3], [4, 5, 77]),
}


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", list(CASES))
def test_attention(kvfix, fmt, name):
    r = Round(kvfix, fmt, *CASES[name], seed=len(name))
    out, lse = r.call()
    kvfix.check_status()
    r.check(out, lse)


# blocks of 8, 16 and more rows, own and shared: each size goes its own way through the kernels
FEW = {
    "eight_rows": (2, 4, 128, 16, 1, [90], [0, 2], [33, 70]),
    "sixteen_rows": (2, 8, 128, 16, 1, [100], [0, 2], [33, 70]),
    "sixteen_of_one": (2, 4, 64, 16, 4, [50], [0, 1], [20]),
    "nine_then_eighteen": (1, 3, 64, 32, 3, [77], [0, 2], [3, 50]),
    "sixteen_then_many": (1, 4, 128, 64, 4, [200], [0, 20], [4 + 9 * i for i in range(20)]),
    "seventeen_rows": (1, 17, 64, 16, 1, [40], [0, 1], [30]),
    "own_alone": (2, 4, 128, 32, 1, [], [], [37 * i % 500 for i in range(24)]),
    "own_long": (1, 8, 64, 128, 1, [], [], [20000, 1, 15]),
    "fewer_own_than_new": (2, 2, 64, 16, 3, [40], [0, 1], [0]),
    "fewer_own_than_new_of_two": (1, 2, 128, 16, 4, [21, 2], [0, 1, 2], [1, 3]),
    "a_last_block_of_few": (1, 8, 64, 16, 1, [300], [0, 33], [5] * 33),
}


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", list(FEW))
def test_few_rows(kvfix, fmt, name):
    r = Round(kvfix, fmt, *FEW[name], seed=len(name))
    out, lse = r.call()
    kvfix.check_status()
    r.check(out, lse)


@gpu
@pytest.mark.parametrize("heads,group", ((2, 4), (1, 24)))
def test_scales_far_apart(kvfix, heads, group):
    """e4m3 rows whose scales differ by many powers of two, queries that undo the keys'."""
    r = Round(kvfix, "e4m3", heads, group, 128, 16, 1, [200], [0, 3], [30, 77, 5])
    rng = np.random.default_rng(3)
    used = (r.pool.k_scales[0] != 0xFF).cpu().numpy()            # [heads][slots]
    shift = np.where(used, rng.integers(-50, 51, used.shape), 0)
    v = r.pool.v_scales[0].cpu().numpy().astype(np.int64) + shift
    r.pool.v_scales[0] = torch.from_numpy(v.astype(np.uint8)).cuda()
    k = r.pool.k_scales[0].cpu().numpy().astype(np.int64) - np.where(used, 40, 0)
    r.pool.k_scales[0] = torch.from_numpy(k.astype(np.uint8)).cuda()
    r.q.mul_(2.0 ** 40)
    r.q_words = words_of(r.q)
    out, lse = r.call()
    kvfix.check_status()
    r.check(out, lse)


@gpu
@pytest.mark.parametrize("fmt", ("bf16", "e4m3"))
@pytest.mark.parametrize("group", (3, 24))
def test_a_row_of_nan_reaches_its_own_queries_alone(kvfix, fmt, group):
    r = Round(kvfix, fmt, 2, group, 64, 16, 1, [40], [0, 2], [30, 21])
    want, want_lse = r.call()
    at = int(r.rows(r.tables[1][1], 21)[7])
    for plane, scales in (("k", "k_scales"), ("v", "v_scales")):
        t = getattr(r.pool, plane if fmt == "bf16" else scales)
        where = (0, at, 1) if fmt == "bf16" else (0, 1, at)
        was = t[where].clone()
        t[where] = float("nan") if fmt == "bf16" else 0xFF       # key 7 of agent 1, KV head 1
        out, lse = r.call()
        kvfix.check_status()
        t[where] = was
        assert torch.isnan(out[1, :, group:].float()).all()
        assert torch.isnan(lse[1, :, group:]).all() if plane == "k" else torch.equal(lse, want_lse)
        out[1, :, group:], lse[1, :, group:] = want[1, :, group:], want_lse[1, :, group:]
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("group,new", ((4, 1), (5, 2), (6, 4)))
def test_same_bits_every_time(kvfix, fmt, group, new):
    """Many short units on every SM, again and again: nothing depends on who comes first."""
    own = [new + 53 * i % 700 for i in range(24)]
    r = Round(kvfix, fmt, 8, group, 128, 16, new, [900, 300], [0, 16, 24], own)
    first = None
    for _ in range(60):
        out, lse = r.call()
        kvfix.check_status()
        if first is None:
            first = out, lse
        assert torch.equal(out.view(torch.int16), first[0].view(torch.int16))
        assert torch.equal(lse.view(torch.int32), first[1].view(torch.int32))


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_same_bits_whatever_the_workspace_holds(kvfix, fmt):
    r = Round(kvfix, fmt, 2, 5, 128, 16, 2, [511, 90], [0, 2, 4], [2, 40, 129, 300])
    n = kvfix.shared_attend_workspace_bytes(r.q, r.pool, 2)
    first = None
    for fill in (0, 0xFF, 0x7F, 0x3C):
        w = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        out, lse = r.call(workspace=w)
        if first is None:
            first = out, lse
        assert torch.equal(out.view(torch.int16), first[0].view(torch.int16))
        assert torch.equal(lse.view(torch.int32), first[1].view(torch.int32))
    kvfix.check_status()


@gpu
def test_strided_queries_and_outputs(kvfix):
    r = Round(kvfix, "bf16", 2, 3, 64, 16, 3, [50], [0, 2], [3, 60])
    want, lse = r.call()
    A, T, H, D = r.q.shape
    wide = torch.full((2 * A, T + 2, H + 5, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = wide[::2, 1:1 + T, 2:2 + H]
    q.copy_(r.q)
    # heads of one token are contiguous; agents and tokens lie apart
    out_wide = torch.full((A, T + 1, 2, H, D), 5.0, dtype=torch.bfloat16, device="cuda")
    out = out_wide[:, :T, 1]
    got, got_lse = kvfix.shared_attend(q, r.pool, r.page, **r.args, out=out, return_lse=True)
    kvfix.check_status()
    assert got.data_ptr() == out.data_ptr()
    assert torch.equal(got, want) and torch.equal(got_lse, lse)
    assert (out_wide[:, :, 0] == 5).all() and (out_wide[:, T:] == 5).all()


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_pages_out_of_range_count_as_absent(kvfix, fmt):
    r = Round(kvfix, fmt, 2, 2, 64, 16, 1, [100], [0, 2], [40, 200])
    pages = r.pool.k.shape[1] // 16
    r.args["prefix_pages"][0, 2] = -1
    r.args["suffix_pages"][1, 5] = pages
    out, lse = r.call()
    with pytest.raises(kvfix.KvfixError) as e:
        kvfix.check_status()
    assert e.value.status == kvfix.EDEVICE
    absent = [(a, 32 + i) for a in (0, 1) for i in range(16)] + [(1, 100 + 80 + i) for i in range(16)]
    r.check(out, lse, absent)
    kvfix.check_status()


@gpu
def test_lengths_and_groups_out_of_range_are_clamped(kvfix):
    r = Round(kvfix, "bf16", 1, 2, 64, 16, 1, [48, 30], [0, 2, 3], [20, 5, 16])
    r.args["suffix_len"][1] = -4
    r.own[1] = 0
    r.args["group_begin"][2] = 9                                 # clamped to the agents' count
    out, lse = r.call()
    with pytest.raises(kvfix.KvfixError):
        kvfix.check_status()
    r.check(out, lse)
    wide = r.args["suffix_pages"].shape[1]
    r.args["group_begin"][2] = 3
    r.args["suffix_len"][1] = 16 * wide + 1                      # clamped to the page list: its spare page is absent
    out, lse = r.call()
    with pytest.raises(kvfix.KvfixError):
        kvfix.check_status()
    assert torch.isfinite(lse[[0, 2]]).all()
    r.args["suffix_len"][1] = 0
    out, lse = r.call()
    kvfix.check_status()
    r.check(out, lse)


@gpu
@pytest.mark.parametrize("fmt", ("bf16", "int4"))
def test_on_a_stream_and_in_a_graph(kvfix, fmt):
    """A captured call follows lengths and pages that change between replays."""
    r = Round(kvfix, fmt, 2, 4, 128, 16, 1, [260], [0, 3], [30, 140, 7])
    out = torch.zeros_like(r.q)
    ws = torch.empty(kvfix.shared_attend_workspace_bytes(r.q, r.pool, 1), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        g.capture_begin()
        _, lse = r.call(out=out, workspace=ws)
        g.capture_end()
        g.replay()
        s.synchronize()
        r.check(out, lse)
        r.prefix[0], r.own[1] = 70, 9
        r.args["prefix_len"].fill_(70)
        r.args["suffix_len"][1] = 9
        g.replay()
        s.synchronize()
        r.check(out, lse)
    kvfix.check_status()


@gpu
def test_a_pool_beyond_32_bit_offsets(kvfix):
    """Pages past 4 GB of a plane (and past 2^31 elements) are reached."""
    H, D, page = 8, 128, 128
    slots = (5 << 30) // (H * D * 2) // page * page
    k = torch.zeros(1, slots, H, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(1, slots, H, D, dtype=torch.bfloat16, device="cuda")
    pages = np.array([[slots // page - 1, 3]], np.int32)
    small = Round(kvfix, "bf16", H, 1, D, page, 1, [], [], [200], seed=6)
    src = small.rows(small.tables[1][0], 256)
    dst = (pages[0][:, None].astype(np.int64) * page + np.arange(page)).reshape(-1)
    for a, b in ((k, small.pool.k), (v, small.pool.v)):
        a[0, torch.from_numpy(dst).cuda()] = b[0, torch.from_numpy(src).cuda()]
    want, lse = small.call()
    got, got_lse = kvfix.shared_attend(small.q, kvfix.Pool("bf16", k, v), page,
                                       torch.from_numpy(pages).cuda(), small.args["suffix_len"], return_lse=True)
    kvfix.check_status()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, got_lse)


@gpu
def test_large_logits_do_not_overflow(kvfix):
    """Logits in the thousands, one key far above the others."""
    r = Round(kvfix, "bf16", 1, 4, 64, 16, 1, [300], [0, 1], [20])
    r.pool.k.mul_(40)
    r.q.mul_(16)
    r.q_words = words_of(r.q)
    out, lse = r.call()
    kvfix.check_status()
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    r.check(out, lse)


def test_refusals(kvfix):
    """Bad arguments return KVFIX_EINVAL before anything is launched (no GPU involved)."""
    L = kvfix.lib
    at = lambda i: ctypes.c_void_p(i << 32)  # noqa: E731

    def desc(A=2, n=1, H=4, D=64, layers=1):
        return kvfix.KvDesc(A, layers, n, H, D, n * H * D, n * H * D, H * D)

    def pool(fmt=0, layers=1, slots=64, H=2, D=64, ks=9 << 32, vs=10 << 32):
        w = H * (2 * D, D, D // 2)[fmt]
        return kvfix.PoolDesc(fmt, layers, slots, H, D, slots * w, w, 7 << 32, 8 << 32, ks, vs)

    def call(q=at(1), qd=None, p=None, page=16, pp=at(2), mp=4, pl=at(2), gb=at(2), groups=1, sp=at(2), ms=4, sl=at(2),
             scale=0.125, out=at(3), od=None, lse=at(4), ws=at(5), wb=1 << 31):
        return L.kvfix_shared_attend(q, qd or desc(), p or pool(), page, pp, mp, pl, gb, groups, sp, ms, sl, scale, out,
                                     od or desc(), lse, ws, wb, None)

    odd = ctypes.c_void_p((1 << 32) + 2)
    bad = [
        (dict(q=None), b"null"), (dict(q=odd), b"aligned"), (dict(out=None), b"null"),
        (dict(od=desc(A=3)), b"shapes"), (dict(od=desc(H=2)), b"shapes"),
        (dict(qd=desc(layers=2), od=desc(layers=2)), b"one layer"), (dict(p=pool(layers=2)), b"one layer"),
        (dict(p=pool(H=3)), b"multiple"), (dict(p=pool(D=128)), b"head_dim"),
        (dict(page=8), b"page_tokens"), (dict(page=48), b"page_tokens"), (dict(page=256), b"page_tokens"),
        (dict(page=128), b"multiple of page_tokens"), (dict(p=pool(fmt=1, ks=(9 << 32) + 4)), b"16-byte"),
        (dict(p=pool(fmt=2, vs=(9 << 32) + 8)), b"16-byte"), (dict(p=pool(fmt=1, ks=None)), b"scales"),
        (dict(groups=-1), b"groups"), (dict(mp=-1), b"2^30"), (dict(mp=1 << 26), b"2^30"), (dict(ms=1 << 26), b"2^30"),
        (dict(pl=None), b"required"), (dict(gb=None), b"required"), (dict(pp=None), b"required"),
        (dict(sl=None), b"required"), (dict(sp=None), b"required"),
        (dict(scale=0.0), b"scale"), (dict(scale=float("nan")), b"scale"), (dict(scale=float("inf")), b"scale"),
        (dict(ws=None), b"workspace"), (dict(ws=odd), b"workspace"), (dict(wb=15), b"workspace"),
        (dict(out=at(1)), b"overlap"), (dict(out=at(7)), b"overlap"), (dict(lse=at(3)), b"overlap"),
        (dict(lse=at(1)), b"overlap"), (dict(ws=at(3)), b"overlap"), (dict(ws=at(4)), b"overlap"),
        (dict(ws=at(8)), b"overlap"),
        (dict(qd=desc(A=1 << 20, n=64), od=desc(A=1 << 20, n=64)), b"2^27"),
    ]
    for kw, said in bad:
        assert call(**kw) == kvfix.EINVAL, kw
        msg = L.kvfix_last_error()
        assert msg.startswith(b"kvfix_shared_attend") and said in msg, (kw, msg)
    empty = desc(A=0)                                             # no agents: nothing to do, no GPU needed
    assert call(qd=empty, od=empty, sl=None, sp=None, groups=0) == kvfix.OK, L.kvfix_last_error()
    size = L.kvfix_shared_attend_workspace_bytes
    assert size(2, 1, 4, 2, 64, 1) > 0
    assert size(2, 1, 4, 3, 64, 1) == 0 and size(2, 1, 4, 2, 96, 1) == 0 and size(-1, 1, 4, 2, 64, 1) == 0


def test_the_definition_itself():
    """The restatement on a case done by hand: two keys of weights 1:3."""
    q = np.zeros((1, 1, 64))
    q[0, 0, 0] = np.log(3.0) * 8
    k = np.zeros((2, 1, 64))
    k[1, 0, 0] = 1.0
    v = np.stack((np.full((1, 64), 4.0), np.full((1, 64), 8.0)))
    out, lse = ref.attend(q, k, v, [2], 0.125)
    assert np.allclose(out, 7.0) and np.allclose(lse, np.log(4.0))
    out, lse = ref.attend(q, k, v, [0], 0.125)
    assert not out.any() and lse[0, 0] == -np.inf
