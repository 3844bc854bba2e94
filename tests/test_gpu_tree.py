"""kvfix_tree_attend against its definition in 64 bits, on the values the pool stands for.

Tolerances are kvfix_shared_attend's (test_gpu_attend.py derives them): a tree changes which keys a
row sees, not how it is computed.
"""
import numpy as np
import pytest
import torch

import draft_ref as ref
import pool_ref
from test_gpu_attend import Round, words_of

FORMATS = ("bf16", "e4m3", "int4")
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvfix():
    from cross_context_kv_gb300 import build
    build.build()
    from cross_context_kv_gb300 import kvfix
    return kvfix


def i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


class Trees(Round):
    """A Round whose agents' last nodes[a] own keys are trees.  `kind`: "tree" (lines of descent of random
    trees), "any" (random bits, the node's own among them or not) or "chain"; rows of queries past an
    agent's nodes and bits past a query's own hold anything."""

    def __init__(self, kvfix, fmt, heads, group, dim, page, T, prefix, begin, before, nodes, kind="tree", seed=0):
        own = [b + n for b, n in zip(before, nodes)]
        super().__init__(kvfix, fmt, heads, group, dim, page, T, prefix, begin, own, seed=seed)
        r = np.random.default_rng(seed + 1)
        self.nodes, A = list(nodes), len(nodes)
        bits = np.zeros((A, T, T), bool)
        for a in range(A):
            for t in range(T):
                if kind == "chain":
                    bits[a, t, :t + 1] = True
                elif kind == "any":
                    bits[a, t, :t + 1] = r.random(t + 1) < 0.4
                else:
                    up = int(r.integers(-1, t)) if t else -1
                    if up >= 0:
                        bits[a, t] = bits[a, up]
                    bits[a, t, t] = True
        self.bits = bits
        noise = r.random((A, T, T)) < 0.5
        t = np.arange(T)
        given = np.where((t[None, :] > t[:, None]) | (t[None, :, None] >= np.array(nodes)[:, None, None]), noise, bits)
        self.words = i32(ref.words_of(given))
        self.nodes_t = i32(nodes)

    def call(self, **kw):
        return self.kvfix.tree_attend(self.q, self.pool, self.page, tree_mask=self.words,
                                      **{**self.args, "nodes": self.nodes_t, "return_lse": True, **kw})

    def check(self, out, lse, absent=()):
        """`absent`: (agent, place in its sequence) pairs of keys that count as not there."""
        K, V, q = self.values("k"), self.values("v"), pool_ref.of_bf16(self.q_words)
        got, got_lse = pool_ref.of_bf16(words_of(out)), lse.cpu().numpy().astype(np.float64)
        T, D = self.new, q.shape[-1]
        for a in range(len(self.own)):
            g = next((g for g in range(len(self.prefix)) if self.begin[g] <= a < self.begin[g + 1]), None)
            n0 = 0 if g is None else self.prefix[g]
            at = np.concatenate((self.rows(self.tables[0][g], n0) if n0 else np.zeros(0, np.int64),
                                 self.rows(self.tables[1][a], self.own[a])))
            gone = [p for b, p in absent if b == a]
            at[gone] = 0
            k, v, n, N = K(at), V(at), len(at), self.nodes[a]
            sees = np.zeros((T, n), bool)
            sees[:N, :n - N] = True
            sees[:N, n - N:] = self.bits[a, :N, :N]
            sees[:, gone] = False
            want, want_lse = ref.attend(q[a], k, v, sees, self.scale)
            mean, _ = ref.attend(q[a], k, np.abs(v), sees, self.scale)
            mags = np.zeros(want_lse.shape)
            for h in range(q.shape[2]):
                if n:
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
    # heads, group, dim, page, T, prefix lengths, group_begin, own lengths before the trees, nodes
    "one_node": (1, 1, 64, 16, 1, [], [], [0], [1]),
    "one_of_one": (2, 4, 128, 16, 1, [40], [0, 2], [9, 0], [1, 1]),
    "eight_rows": (2, 2, 128, 16, 4, [90], [0, 2], [33, 70], [4, 3]),
    "sixteen_rows": (2, 2, 64, 32, 8, [100], [0, 1], [7], [8]),
    "own_few_shared_many": (1, 1, 128, 16, 16, [300], [0, 4], [5, 16, 0, 130], [16, 15, 1, 0]),
    "many": (2, 4, 128, 16, 16, [200], [0, 3], [30, 0, 129], [16, 9, 0]),
    "no_prefix": (2, 4, 64, 16, 33, [], [], [0, 100, 1], [33, 32, 7]),
    "two_words": (1, 4, 128, 64, 61, [129], [0, 2], [127, 3], [61, 33]),
    "over_a_tile": (1, 2, 64, 16, 130, [31], [0, 2], [60, 200], [130, 129]),
    "several_tiles": (1, 1, 128, 128, 300, [77], [0, 2], [5, 250], [300, 299]),
    "blocks": (1, 8, 64, 16, 70, [500], [0, 3], [10, 64, 0], [70, 33, 64]),
    "groups": (4, 3, 64, 32, 10, [64, 0, 1, 200], [0, 2, 3, 3, 6], [5, 0, 70, 0, 31, 90], [10, 4, 0, 10, 1, 9]),
    "some_outside": (2, 5, 128, 16, 7, [40], [1, 3], [3, 0, 8, 20, 0], [7, 0, 7, 2, 7]),
    "many_agents": (1, 2, 64, 16, 3, [20, 7], [0, 150, 290], [5 * i % 37 for i in range(300)], [i % 4 for i in range(300)]),
    "many_groups": (1, 1, 64, 16, 17, [3 * g % 50 for g in range(270)], list(range(271)), [i % 5 for i in range(280)],
                    [17 - i % 3 for i in range(280)]),
    "nobody": (2, 2, 64, 16, 5, [40], [0, 2], [0, 20], [0, 0]),
}


@gpu
@pytest.mark.parametrize("kind", ("tree", "any", "chain"))
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", list(CASES))
def test_trees(kvfix, fmt, name, kind):
    r = Trees(kvfix, fmt, *CASES[name], kind=kind, seed=len(name))
    out, lse = r.call()
    kvfix.check_status()
    r.check(out, lse)


# rows enough for the join that takes many at a time: borders of blocks inside its runs of rows, last runs
# that are short, parts of long prefixes and of several pieces
LARGE = {
    "borders": (4, 5, 128, 16, 33, [700], [0, 6], [10, 64, 0, 200, 33, 5], [33, 30, 33, 0, 1, 33]),
    "ragged_64": (5, 3, 64, 64, 61, [3001, 0], [0, 2, 4], [900, 3, 0, 77], [61, 54, 47, 33]),
    "no_prefix": (8, 4, 64, 32, 17, [], [], [300, 0, 5, 90, 1200, 7], [17] * 6),
    "short_trees": (4, 3, 128, 16, 3, [700, 0], [0, 50, 90], [53 * i % 400 for i in range(100)], [i % 4 for i in range(100)]),
    "a_run_and_one": (8, 3, 64, 16, 3, [90], [2, 30], [7 * i % 50 for i in range(40)], [3 - i % 2 for i in range(40)]),
}


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", list(LARGE))
def test_many_rows(kvfix, fmt, name):
    r = Trees(kvfix, fmt, *LARGE[name], kind="any", seed=len(name))
    out, lse = r.call()
    kvfix.check_status()
    assert lse.numel() > 16 * torch.cuda.get_device_properties(0).multi_processor_count
    r.check(out, lse)


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("case", ((2, 2, 64, 16, 3, [40], [0, 2], [2, 50], [3, 3]), (2, 4, 128, 16, 40, [300], [0, 3], [3, 140, 0], [40] * 3),
                                  (1, 1, 128, 32, 11, [], [], [0, 33], [11, 11])))
def test_a_chain_is_new_tokens_in_a_row(kvfix, fmt, case):
    r = Trees(kvfix, fmt, *case, kind="chain", seed=3)
    want, want_lse = Round.call(r)
    for nodes in (r.nodes_t, None):
        out, lse = r.call(nodes=nodes)
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
        assert torch.equal(lse.view(torch.int32), want_lse.view(torch.int32))
    kvfix.check_status()


@gpu
@pytest.mark.parametrize("T,group", ((3, 2), (40, 4)))
def test_numbers_of_nodes_out_of_range_are_clamped(kvfix, T, group):
    r = Trees(kvfix, "bf16", 1, group, 64, 16, T, [50], [0, 3], [0, 20, 4], [2, T, 1], kind="tree")
    r.nodes_t.copy_(i32([T, T + 5, -3]))           # more than its own keys, more than T, fewer than none
    r.nodes = [2, T, 0]
    out, lse = r.call()
    with pytest.raises(kvfix.KvfixError) as e:
        kvfix.check_status()
    assert e.value.status == kvfix.EDEVICE
    r.check(out, lse)
    out, lse = r.call(nodes=None)                   # T each, of which agents 0 and 2 have 2 and 5 own keys
    with pytest.raises(kvfix.KvfixError):
        kvfix.check_status()
    kvfix.check_status()


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,group", ((4, 2), (40, 2)))
def test_pages_out_of_range_count_as_absent(kvfix, fmt, T, group):
    """Before the trees, in them, and in the prefix."""
    r = Trees(kvfix, fmt, 2, group, 64, 16, T, [100], [0, 2], [40, 20], [T, T], kind="any")
    # (row 0 of the pool, which stands for the keys that are not there, must be some key's)
    zero = [i for t in r.tables for i in np.argwhere(t == 0)]
    if not zero:
        r.pool.k[:, 0], r.pool.v[:, 0] = r.pool.k[:, int(r.tables[1][0, 0]) * 16], r.pool.v[:, int(r.tables[1][0, 0]) * 16]
        for s in r.pool[3:]:
            if s is not None:
                s[:, :, 0] = s[:, :, int(r.tables[1][0, 0]) * 16]
    r.args["prefix_pages"][0, 2] = -1
    r.args["suffix_pages"][0, 1] = -5
    last = (20 + T - 1) // 16
    r.args["suffix_pages"][1, last] = r.pool.k.shape[1] // 16
    out, lse = r.call()
    with pytest.raises(kvfix.KvfixError) as e:
        kvfix.check_status()
    assert e.value.status == kvfix.EDEVICE
    absent = [(a, 32 + i) for a in (0, 1) for i in range(16)] + [(0, 100 + 16 + i) for i in range(16)]
    absent += [(1, 100 + i) for i in range(16 * last, 20 + T)]
    r.check(out, lse, absent)
    kvfix.check_status()


@gpu
@pytest.mark.parametrize("fmt", ("bf16", "e4m3"))
@pytest.mark.parametrize("group,T", ((2, 4), (8, 6)))
def test_a_key_of_nan_reaches_those_that_see_it(kvfix, fmt, group, T):
    r = Trees(kvfix, fmt, 1, group, 64, 16, T, [40], [0, 2], [30, 5], [T, T], kind="any", seed=9)
    r.bits[1, :, 1] = False
    r.bits[1, 2, 1] = r.bits[1, 1, 1] = True       # node 1 is seen by itself and by node 2 alone
    r.words.copy_(i32(ref.words_of(r.bits)))
    want, want_lse = r.call()
    at = int(r.rows(r.tables[1][1], r.own[1])[5 + 1])
    if fmt == "bf16":
        r.pool.k[0, at] = float("nan")
    else:
        r.pool.k_scales[0, :, at] = 0xFF
    out, lse = r.call()
    kvfix.check_status()
    assert torch.isnan(lse[1, 1:3]).all() and torch.isnan(out[1, 1:3].float()).all()
    out[1, 1:3], lse[1, 1:3] = want[1, 1:3], want_lse[1, 1:3]
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("group,T", ((2, 4), (4, 30)))
def test_same_bits_every_time(kvfix, fmt, group, T):
    before = [53 * i % 700 for i in range(12)]
    r = Trees(kvfix, fmt, 8, group, 128, 16, T, [900, 300], [0, 8, 12], before, [T - i % 3 for i in range(12)])
    first = r.call()
    n = kvfix.shared_attend_workspace_bytes(r.q, r.pool, 2)
    for i in range(30):
        w = torch.full((n,), (0, 0xFF, 0x7F)[i % 3], dtype=torch.uint8, device="cuda")
        out, lse = r.call(workspace=w)
        assert torch.equal(out.view(torch.int16), first[0].view(torch.int16))
        assert torch.equal(lse.view(torch.int32), first[1].view(torch.int32))
    kvfix.check_status()


@gpu
@pytest.mark.parametrize("T,group", ((4, 2), (24, 4)))
def test_on_a_stream_and_in_a_graph(kvfix, T, group):
    """A captured call follows trees, numbers of nodes and lengths that change between replays."""
    r = Trees(kvfix, "bf16", 2, group, 128, 16, T, [260], [0, 3], [30, 140, 7], [T, T, T])
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
        r.nodes[1], r.own[1] = 2, 12
        r.nodes_t[1] = 2
        r.args["suffix_len"][1] = 12
        r.bits[0] = np.eye(T, dtype=bool)
        r.words[0] = i32(ref.words_of(r.bits[0]))
        g.replay()
        s.synchronize()
        r.check(out, lse)
    kvfix.check_status()


@gpu
@pytest.mark.parametrize("heads,T,group", ((2, 4, 2), (8, 30, 4)))
def test_two_calls_at_once(kvfix, heads, T, group):
    """Rounds on two streams, each with a workspace of its own, give what they give one by one."""
    rounds, want = [], []
    for i in range(2):
        r = Trees(kvfix, ("bf16", "e4m3")[i], heads, group, 128, 16, T, [900 - 500 * i], [0, 12], [53 * j % 300 for j in range(12)],
                  [T - j % 3 for j in range(12)], seed=i)
        rounds.append(r)
        want.append(r.call())
        r.check(*want[i])
    ws = [torch.empty(kvfix.shared_attend_workspace_bytes(r.q, r.pool, 1), dtype=torch.uint8, device="cuda") for r in rounds]
    outs = [[torch.zeros_like(r.q) for _ in range(10)] for r in rounds]
    lses = [[], []]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for j in range(10):
        for i, r in enumerate(rounds):
            with torch.cuda.stream(streams[i]):
                lses[i].append(r.call(out=outs[i][j], workspace=ws[i])[1])
    torch.cuda.synchronize()
    kvfix.check_status()
    for i in range(2):
        for j in range(10):
            assert torch.equal(outs[i][j].view(torch.int16), want[i][0].view(torch.int16))
            assert torch.equal(lses[i][j].view(torch.int32), want[i][1].view(torch.int32))


def test_masks_of_parents(kvfix):
    """tree_masks: lines of descent as bits, depths, ragged trees, more than one word."""
    parents = [[-1, 0, 0, 1, -1], [], [-1] + list(range(69))]
    mask, depth, nodes = kvfix.tree_masks(parents)
    assert mask.shape == (3, 70, 3) and mask.dtype == depth.dtype == nodes.dtype == torch.int32
    bits = ref.bits_of(mask.numpy(), 70)
    assert [list(np.flatnonzero(b)) for b in bits[0, :5]] == [[0], [0, 1], [0, 2], [0, 1, 3], [4]]
    assert not bits[0, 5:].any() and not bits[1].any()
    assert (bits[2] == np.tri(70, dtype=bool)).all()
    assert depth[0, :5].tolist() == [0, 1, 1, 2, 0] and depth[2].tolist() == list(range(70))
    assert nodes.tolist() == [5, 0, 70]
    for bad in ([[0]], [[-1, 1]], [[-2]]):
        with pytest.raises(ValueError, match="parent"):
            kvfix.tree_masks(bad)
