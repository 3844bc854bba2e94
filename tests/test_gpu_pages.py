"""kvfix_pages_extend, _cut and _compact against the books kept one list after another, and the pool's
rows bit for bit."""
import numpy as np
import pytest
import torch

import draft_ref as ref

FORMATS = ("bf16", "e4m3", "int4")
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvfix():
    from cross_context_kv_gb300 import build
    build.build()
    from cross_context_kv_gb300 import kvfix
    return kvfix


def i32(x, *shape):
    t = torch.tensor(np.asarray(x, np.int32), device="cuda")
    return t.view(*shape) if shape else t


def noisy(t, gen):
    """Random bits in a tensor."""
    raw = t.view(torch.uint8)
    raw.copy_(torch.randint(0, 256, raw.shape, generator=gen, device="cuda", dtype=torch.uint8))


class Paged:
    """A pool of random bits and lists on shuffled pages.  lens: the lists' lengths; like: {i: j}, list i
    holds the pages of list j (of the same length); spare: free pages; room: entries behind each list's."""

    def __init__(self, kvfix, fmt="bf16", page=16, lens=(), like=None, spare=10, room=4, layers=2, heads=2, dim=64, seed=0,
                 interleave=False):
        self.kvfix, self.page = kvfix, page
        r, like = np.random.default_rng(seed), like or {}
        take = lambda n: -(-n // page)  # noqa: E731
        total = sum(take(n) for i, n in enumerate(lens) if i not in like) + spare
        order, at = r.permutation(total).astype(np.int32), 0
        wide = max([0] + [take(n) for n in lens]) + room
        pages = np.full((len(lens), wide), 1 << 30, np.int32)    # entries behind a list mean nothing
        for i, n in enumerate(lens):
            if i in like:
                pages[i, :take(n)] = pages[like[i], :take(n)]
            else:
                pages[i, :take(n)] = order[at:at + take(n)]
                at += take(n)
        refs = np.zeros(total, np.int32)
        for i, n in enumerate(lens):
            refs[pages[i, :take(n)]] += 1
        slots = total * page
        pool = kvfix.pool_empty(fmt, layers, slots, heads, dim)
        if interleave:                                           # a slot's values behind its keys
            w = pool.k.shape[-1]
            both = torch.zeros(layers, slots, 2, heads, w, dtype=pool.k.dtype, device="cuda")
            pool = pool._replace(k=both[:, :, 0], v=both[:, :, 1])
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.planes = [t for t in pool[1:] if t is not None]
        for t in self.planes:
            if t.is_contiguous():
                noisy(t, gen)
            else:
                x = torch.empty(t.shape, dtype=t.dtype, device="cuda")
                noisy(x, gen)
                t.view(torch.uint8).copy_(x.view(torch.uint8))
        self.pool, self.refs, self.pages, self.lens = pool, i32(refs), i32(pages, len(lens), wide), i32(lens)
        self.snap()

    def snap(self):
        """The state as it is now: what the next call is compared with."""
        self.books = ref.Books(self.page, self.refs.tolist(), self.pages.tolist(), self.lens.tolist())
        self.was = [self.raw(t).clone() for t in self.planes]

    @staticmethod
    def raw(t):
        """A plane's or scales' rows as bytes [layers][slots][...] (scales lie heads first)."""
        return t.contiguous().view(torch.uint8)

    def check(self, moves, flags=()):
        """The state against the books, after `moves` of rows."""
        kvfix = self.kvfix
        assert self.books.flags == set(flags)
        if flags:
            with pytest.raises(kvfix.KvfixError) as e:
                kvfix.check_status()
            assert e.value.status == (kvfix.ENOSPACE if "space" in flags else kvfix.EDEVICE)
        kvfix.check_status()
        assert self.refs.tolist() == self.books.refs
        assert self.lens.tolist() == self.books.lens
        assert self.pages.tolist() == self.books.pages
        # a row of the pool after the moves is some row before them
        src = np.arange(self.pool.k.shape[1])
        for a, b in moves:
            src[b] = src[a]
        src = torch.from_numpy(src).cuda()
        for t, was in zip(self.planes, self.was):
            axis = 1 if t.shape[1] == len(src) and t.dim() == 4 else 2
            assert torch.equal(self.raw(t), was.index_select(axis, src)), (t.shape, axis)
        self.snap()

    def extend(self, extra, parent=None, flags=(), **kw):
        moves = self.books.extend(extra, parent)
        self.kvfix.pages_extend(self.pool, self.page, self.refs, self.pages, self.lens, i32(extra),
                                None if parent is None else i32(parent), **kw)
        self.check(moves, flags)

    def cut(self, base, path=None, kept=None, flags=()):
        moves = self.books.cut(base, path, kept)
        self.kvfix.pages_cut(self.pool, self.page, self.refs, self.pages, self.lens, i32(base),
                             None if path is None else i32(path, len(base), -1), None if kept is None else i32(kept))
        self.check(moves, flags)

    def compact(self, **kw):
        moves, live = self.books.compact()
        got = self.kvfix.pages_compact(self.pool, self.page, self.refs, self.pages, self.lens, **kw)
        assert got.item() == live
        self.check(moves)


# ------------------------------------------------------------------ extend

@gpu
@pytest.mark.parametrize("page", (16, 32, 64, 128))
@pytest.mark.parametrize("fmt", FORMATS)
def test_lists_grow(kvfix, fmt, page):
    p = Paged(kvfix, fmt, page, lens=[0, 1, page - 1, page, page + 1, 5 * page + 7, 0], spare=30)
    p.extend([1, 0, 1, 1, page, 3 * page + 9, 0])
    p.extend([0] * 7)
    p.extend([page] * 7)


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_lists_fork(kvfix, fmt):
    """Forks with and without room, of full and of partly full last pages, of empty lists; parents that
    grow, or do nothing, in the same call."""
    lens = [40, 32, 0, 17, 0, 0, 0, 0, 0, 0]
    p = Paged(kvfix, fmt, 16, lens=lens, spare=30)
    p.extend([5, 0, 3, 0, 1, 0, 20, 0, 16, 0], [0, 1, 2, -1, 0, 0, 1, 1, 2, 3])
    # pages that several hold now: whoever writes behind his tokens gets a copy
    p.extend([1] * 10)
    p.extend([1] * 10)


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_shared_last_pages_are_copied(kvfix, fmt):
    """Two holders of a page that both grow both get a copy, and the page comes free."""
    p = Paged(kvfix, fmt, 32, lens=[45, 45, 64, 64, 45], like={1: 0, 3: 2, 4: 0}, spare=12, layers=3, heads=3, dim=128)
    p.extend([1, 1, 1, 1, 0])
    p.extend([0, 0, 0, 0, 1])
    p.extend([30, 30, 30, 30, 30])


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_planes_that_interleave(kvfix, fmt):
    for heads, dim in ((3, 64), (40, 128)):        # rows below and above a CTA's copies at a time
        p = Paged(kvfix, fmt, 16, lens=[30, 30, 7, 0], like={1: 0}, heads=heads, dim=dim, interleave=True)
        p.extend([1, 9, 20, 2], [0, 1, 2, 2])
        p.cut([30, 30, 7, 0], [[0], [5], [11], [0]], [1, 1, 1, 0])
        p.compact()


@gpu
def test_a_pool_that_is_full(kvfix):
    """Lists in order take what is there; whoever does not fit stays as he was."""
    lens = [16, 16, 5, 0, 30, 16]
    p = Paged(kvfix, "bf16", 16, lens=lens, spare=3)
    p.extend([1, 40, 1, 0, 1, 1], flags=("space",))            # one page, three: refused, and so is a later one
    p.extend([0, 16, 1, 17, 0, 0], flags=("space",))
    p.extend([0, 0, 1, 0, 1, 0])
    full = Paged(kvfix, "int4", 16, lens=[16, 9, 9], like={2: 1}, spare=0)
    full.extend([1, 0, 1], flags=("space",))
    full.extend([0, 0, 0])


@gpu
def test_refused_entries_are_left_alone(kvfix):
    p = Paged(kvfix, "bf16", 16, lens=[20, 0, 9, 0, 0, 33, 0, 0], room=2)
    most = p.pages.shape[1] * 16
    # too long, extra below 0, no such parent, a fork onto tokens, a fork too long, a good one
    p.extend([most, 1, -1, 1, 1, 1, most, 3], [0, 8, 2, 99, -5, 0, 0, 5], flags=("bounds",))
    p.lens[2], p.lens[5] = -1, most + 1
    p.snap()
    p.extend([1, 0, 1, 0, 1, 0, 1, 1], [0, 1, 2, 2, 4, 5, 5, 7], flags=("bounds",))
    p.lens[2], p.lens[5] = 9, 33
    p.pages[0, 1], p.pages[5, 2] = -1, p.refs.numel()          # last pages out of range
    p.snap()
    p.extend([1, 1, 0, 0, 1, 1, 0, 0], [0, 0, 2, 5, 2, 5, 6, 7], flags=("bounds",))


@gpu
def test_many_lists_and_pages(kvfix):
    """More lists than a CTA's threads, more pages than a warp's loads, tables beyond a CTA's part."""
    r = np.random.default_rng(4)
    n = 2500
    lens = [int(x) for x in r.integers(0, 60, n // 2)] + [0] * (n - n // 2)
    lens[7] = 40000
    p = Paged(kvfix, "int4", 16, lens=lens, spare=20000, layers=1, heads=1)
    parent = list(range(n // 2)) + [int(x) for x in r.integers(0, n // 2, n - n // 2)]
    parent[-1] = parent[-2] = 7
    p.extend([int(x) for x in r.integers(0, 40, n)], parent)
    base = [int(x) for x in r.integers(0, 2, n) * np.array(p.lens.tolist())]
    p.cut(base)
    p.compact()


@gpu
@pytest.mark.parametrize("free", ("behind", "before", "between"))
def test_free_pages_in_runs(kvfix, free):
    """Whole spans of pages without a free one, or with nothing else; the pool moved together after."""
    n, each, gap = 8, 600, 700
    p = Paged(kvfix, "int4", 16, lens=[16 * each - 5] * n, spare=gap, layers=1, heads=1)
    first = {"behind": 0, "before": gap, "between": 0}[free]
    rows = np.arange(n * each).reshape(n, each) + first
    if free == "between":
        rows[3:] += gap
    p.pages[:, :each] = i32(rows)
    p.refs.zero_()
    p.refs[torch.from_numpy(rows.reshape(-1)).cuda()] = 1
    p.snap()
    p.extend([3, 40, 0, 6, 5, 64, 1, 20])
    p.cut([-1, 0, -1, 16, -1, -1, -1, -1])
    p.extend([64] * n, flags=("bounds",))                       # (list 5 has 64 already, and a table of 604 pages)
    p.compact()
    p.cut([-1] * 7 + [0])
    p.compact()


# ------------------------------------------------------------------ cut

@gpu
@pytest.mark.parametrize("page", (16, 128))
@pytest.mark.parametrize("fmt", FORMATS)
def test_accepted_nodes_move_up(kvfix, fmt, page):
    lens = [page + 9 + 8, 8, 3 * page + 8, 2 * page + 8, 50, 300, 20]
    p = Paged(kvfix, fmt, page, lens=lens, layers=3, heads=3)
    T = 8
    path = [[0, 1, 2, 3, 4, 5, 6, 7], [7, 0, 0, 0, 0, 0, 0, 0], [1, 3, 4, 0, 0, 0, 0, 0], [0, 2, 7, 0, 0, 0, 0, 0],
            [0] * 8, [2, 5, 6, 7, 0, 0, 0, 0], [0] * 8]
    kept = [8, 1, 3, 3, 0, 4, 5]
    base = [n - T for n in lens]
    base[5], base[6] = 100, -1
    p.cut(base, path, kept)


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_long_paths(kvfix, fmt):
    """More rows than a CTA keeps places for, over many pages, every row from one of the next."""
    lens = [700, 500]
    p = Paged(kvfix, fmt, 16, lens=lens, dim=128)
    r = np.random.default_rng(1)
    path = np.zeros((2, 300), np.int64)
    path[0, :250] = np.sort(r.choice(600, 250, replace=False))
    path[1] = np.sort(r.choice(500, 300, replace=False))
    p.cut([100, 0], path.tolist(), [250, 300])


@gpu
def test_lists_roll_back_and_come_free(kvfix):
    p = Paged(kvfix, "e4m3", 16, lens=[100, 100, 48, 33, 0, 16], like={1: 0}, spare=4)
    p.cut([65, 100, 48, 0, 0, -1])
    p.cut([64, 0, 17, 0, 0, 0])
    p.extend([200 - 64, 40, 0, 0, 10, 0], flags=("bounds",))      # (a table has room for 176 tokens)
    p.cut([0] * 6)
    assert not p.refs.any() and not p.lens.any()


@gpu
def test_bad_cuts_are_left_alone(kvfix):
    lens = [40] * 9
    p = Paged(kvfix, "bf16", 16, lens=lens)
    path = [[3, 1], [-1, 0], [0, 8], [2, 2], [1, 2], [0, 1], [0, 1], [0, 1], [5, 7]]
    base = [32, 32, 32, 32, 41, 32, 32, 32, 32]
    p.cut(base, path, [2, 2, 2, 2, 0, 3, -1, 2, 2], flags=("bounds",))
    p.lens[3] = -2
    p.pages[5, 2], p.pages[7, 1] = p.refs.numel(), -7             # entries that the cut gives back, or moves through
    p.snap()
    p.cut([0] * 9, flags=("bounds",))
    twice = Paged(kvfix, "bf16", 16, lens=[20, 20], like={1: 0})
    twice.refs[twice.pages[0, 1].item()] = 1                      # a page that two lists hold and one counts
    twice.snap()
    twice.cut([0, 0], flags=("bounds",))


# ------------------------------------------------------------------ compact

@gpu
@pytest.mark.parametrize("page", (16, 64))
@pytest.mark.parametrize("fmt", FORMATS)
def test_pages_in_use_move_to_the_front(kvfix, fmt, page):
    p = Paged(kvfix, fmt, page, lens=[5 * page + 3, 0, 2 * page, 2 * page, page - 1, 7 * page], like={3: 2}, spare=40, heads=3,
              layers=3, dim=128)
    p.compact()
    p.compact()                                                   # nothing left to move
    p.cut([page, 0, -1, 0, -1, 3])
    p.compact()
    p.extend([9 * page] * 6, flags=("space",))


@gpu
def test_full_and_empty_pools(kvfix):
    full = Paged(kvfix, "bf16", 16, lens=[16, 40, 3], spare=0)
    full.compact()
    empty = Paged(kvfix, "e4m3", 16, lens=[0, 0], spare=7)
    empty.compact()
    one = Paged(kvfix, "int4", 16, lens=[1], spare=0)
    one.compact()


@gpu
@pytest.mark.parametrize("seed", range(4))
def test_a_history_of_rounds(kvfix, seed):
    """Rounds of forks, drafts, accepted paths, ends and moves, one after another on the same pool."""
    r = np.random.default_rng(seed)
    fmt, page, T = FORMATS[seed % 3], (16, 32)[seed % 2], 9
    p = Paged(kvfix, fmt, page, lens=[70, 33, 0, 0, 0, 0, 0, 0], spare=90, room=30, seed=seed)
    n = 8
    for step in range(12):
        lens = p.lens.tolist()
        parent = [i if lens[i] else int(r.integers(-1, n)) for i in range(n)]
        parent = [j if j < 0 or lens[j] else -1 for j in parent]
        p.extend([T] * n, parent)
        grown = [b if x >= 0 else 0 for b, x in zip(p.lens.tolist(), parent)]
        kept = [int(r.integers(0, 4)) if g >= T else 0 for g in grown]
        path = [sorted(r.choice(T, 4, replace=False).tolist()) for _ in range(n)]
        base = [g - T if g else -1 for g in grown]
        for i in range(n):
            if r.random() < 0.15:
                base[i], kept[i] = 0, 0
        p.cut(base, path, kept)
        if step % 3 == 2:
            p.compact()


@gpu
def test_on_a_stream_and_in_a_graph(kvfix):
    """A captured step (room, then an accepted path) follows the books from replay to replay."""
    p = Paged(kvfix, "e4m3", 16, lens=[30, 30, 5], like={1: 0}, spare=20, room=10)
    extra, kept = [8] * 3, [2, 3, 1]
    path = [[1, 4, 0], [0, 2, 7], [6, 0, 0]]
    te, tp, tk, tb = i32(extra), i32(path), i32(kept), torch.empty(3, dtype=torch.int32, device="cuda")
    ws = torch.empty(kvfix.lib.kvfix_pages_extend_workspace_bytes(p.refs.numel(), 3), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        g.capture_begin()
        tb.copy_(p.lens)
        kvfix.pages_extend(p.pool, 16, p.refs, p.pages, p.lens, te, workspace=ws)
        kvfix.pages_cut(p.pool, 16, p.refs, p.pages, p.lens, tb, tp, tk)
        g.capture_end()
        for _ in range(9):
            base = list(p.books.lens)
            moves = p.books.extend(extra) + p.books.cut(base, path, kept)
            g.replay()
            s.synchronize()
            p.check(moves)


@gpu
def test_two_pools_at_once(kvfix):
    """Steps of two pools on two streams, in flight together, leave what they leave one by one."""
    both = [Paged(kvfix, fmt, 16, lens=[30, 30, 5, 70], like={1: 0}, spare=40, room=20, seed=i) for i, fmt in enumerate(("e4m3", "int4"))]
    extra, base, path, kept = [8] * 4, [30, 30, 5, 70], [[1, 4], [0, 2], [6, 0], [3, 7]], [2, 2, 1, 2]
    args = [i32(x) for x in (extra, base, path, kept)]
    moves = [p.books.extend(extra) + p.books.cut(base, path, kept) for p in both]
    for p, m in zip(both, moves):
        m += p.books.compact()[0]
    torch.cuda.synchronize()
    streams, lives = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for p, s in zip(both, streams):
        with torch.cuda.stream(s):
            kvfix.pages_extend(p.pool, 16, p.refs, p.pages, p.lens, args[0])
            kvfix.pages_cut(p.pool, 16, p.refs, p.pages, p.lens, *args[1:])
            lives.append(kvfix.pages_compact(p.pool, 16, p.refs, p.pages, p.lens))
    torch.cuda.synchronize()
    for p, m, n in zip(both, moves, lives):
        assert n.item() == sum(x > 0 for x in p.books.refs)
        p.check(m)


@gpu
def test_a_pool_beyond_32_bit_offsets(kvfix):
    """Pages past 4 GB of a plane are copied, moved up and moved to the front."""
    H, D, page = 8, 128, 128
    total = (5 << 30) // (H * D * 2) // page
    k, v = (torch.zeros(1, total * page, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pool = kvfix.Pool("bf16", k, v)
    at = slice((total - 1) * page, total * page)
    for t in (k, v):
        t[0, at].normal_()
    want = [t[0, at].clone() for t in (k, v)]
    refs, pages, lens = torch.zeros(total, dtype=torch.int32, device="cuda"), i32([[total - 1, 0], [total - 1, 0]]), i32([100, 100])
    refs[total - 1] = 2
    kvfix.pages_extend(pool, page, refs, pages, lens, i32([0, 1]))
    assert pages[:, 0].tolist() == [total - 1, 0] and refs[0] == 1 and refs[total - 1] == 1
    for t, w in zip((k, v), want):
        assert torch.equal(t[0, :100], w[:100]) and not t[0, 100:128].any()
    kvfix.pages_cut(pool, page, refs, pages, lens, i32([50, 0]), i32([[7, 49]] * 2), i32([2, 0]))
    for t, w in zip((k, v), want):
        assert torch.equal(t[0, at.start + 50], w[57]) and torch.equal(t[0, at.start + 51], w[99])
    assert refs[0] == 0
    assert kvfix.pages_compact(pool, page, refs, pages, lens).item() == 1
    assert pages[0, 0] == 0 and refs[0] == 1 and refs[total - 1] == 0
    for t, w in zip((k, v), want):
        assert torch.equal(t[0, :50], w[:50]) and torch.equal(t[0, 50], w[57]) and torch.equal(t[0, 51], w[99])
    kvfix.check_status()
