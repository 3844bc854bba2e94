"""The ways through kvfix_shared_attend that only larger calls take, and keys lost or counted
twice at the cuts of long segments."""
import math

import numpy as np
import pytest
import torch

import pool_ref as ref
from test_gpu_attend import CASES, FEW, FORMATS, Round, gpu, kvfix, words_of  # noqa: F401

CUTS = {**CASES, **FEW,
        "rows_97": (2, 97, 64, 32, 1, [5000], [0, 1], [3000]),
        "rows_40_long": (8, 5, 128, 16, 1, [20000], [0, 8], [17, 0, 1, 900, 4000, 5, 16, 33])}


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", list(CUTS))
def test_every_key_counts_once(kvfix, fmt, name):  # noqa: F811
    """Queries of zero weigh every key the same: lse is the logarithm of their number, sums of
    weights are whole numbers that float holds, and with values of one per tile of 16 keys, in a
    channel that comes round and one that moves on, an output is the share of that channel's keys.
    (A lost tile of 16 among 43000 keys moves lse by 67 times its tolerance.)"""
    r = Round(kvfix, fmt, *CUTS[name], seed=len(name))
    H, D = r.pool.k.shape[2], r.q.shape[-1]
    slots = r.pool.k.shape[1]
    v = np.zeros((slots, D))
    mine = np.full(slots, -1, np.int32)
    for table, lens in zip(r.tables, (r.prefix, r.own)):
        for i, n in enumerate(lens):
            at, tile = r.rows(table[i], n), np.arange(n) // 16
            v[at, tile % (D // 2)] = 1
            v[at, D // 2 + tile * (D // 2) // max(1, -(-n // 16))] = 1
            mine[at] = at
    words = ref.bf16_of(np.repeat(v[:, None], H, 1))[None, None]
    rows = torch.from_numpy(words.view(np.int16)).cuda().view(torch.bfloat16)
    kvfix.pool_write(r.pool, rows, rows.clone(), torch.from_numpy(mine).cuda().view(1, -1))
    r.q.zero_()
    out, lse = r.call()
    kvfix.check_status()
    V = r.values("v")
    got, got_lse = ref.of_bf16(words_of(out)), lse.cpu().numpy().astype(np.float64)
    for a, own in enumerate(r.own):
        g = next((g for g in range(len(r.prefix)) if r.begin[g] <= a < r.begin[g + 1]), None)
        n0 = 0 if g is None else r.prefix[g]
        at = np.concatenate((r.rows(r.tables[0][g], n0) if n0 else np.zeros(0, np.int64), r.rows(r.tables[1][a], own)))
        sums = np.concatenate((np.zeros((1, D)), np.cumsum(V(at)[:, 0], 0)))
        for t in range(r.new):
            n = max(0, len(at) - r.new + 1 + t)
            if n == 0:
                assert not got[a, t].any() and (got_lse[a, t] == -np.inf).all()
                continue
            want = sums[n] / n
            # lse: an exponential of 0 (2^-22), the logarithm and its factor (2^-22 of the result each)
            assert np.abs(got_lse[a, t] - math.log(n)).max() <= 2.0 ** -21 * (1 + math.log(n)), (a, t)
            # out: its rounding, the exponential, and sums of n values of one size
            assert (np.abs(got[a, t] - want) <= (2.0 ** -8 + 2.0 ** -20 + n * 2.0 ** -24) * want).all(), (a, t)


def wide_round(kvfix, fmt, dim):  # noqa: F811
    """Rows beyond 128 an SM (the join takes four at a time there), an odd number of them per agent:
    a row's four straddle tokens and blocks of 256.  Own keys fewer than the new tokens, and none."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    group = 23
    new = 128 * sms // (4 * group) // 2 * 2 + 31
    assert 4 * new * group > 128 * sms and new * group % 4
    return Round(kvfix, fmt, 1, group, dim, 16, new, [40], [0, 3], [new, 100, 0, new + 90], seed=3)


@gpu
@pytest.mark.parametrize("fmt,dim", (("bf16", 64), ("bf16", 128), ("e4m3", 64), ("int4", 128)))
def test_many_rows_of_few_keys(kvfix, fmt, dim):  # noqa: F811
    r = wide_round(kvfix, fmt, dim)
    out, lse = r.call()
    kvfix.check_status()
    r.check(out, lse)


@gpu
def test_a_nan_key_among_many_rows(kvfix):  # noqa: F811
    """It reaches the queries that see it, and no bit of another."""
    r = wide_round(kvfix, "bf16", 64)
    want, want_lse = r.call()
    own, place = r.own[3], r.own[3] - 50
    r.pool.k[0, int(r.rows(r.tables[1][3], own)[place])] = float("nan")
    out, lse = r.call()
    kvfix.check_status()
    seen = r.new - 50                                        # the first of agent 3's tokens that sees it
    assert torch.isnan(out[3, seen:].float()).all() and torch.isnan(lse[3, seen:]).all()
    out[3, seen:], lse[3, seen:] = want[3, seen:], want_lse[3, seen:]
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    assert torch.equal(lse.view(torch.int32), want_lse.view(torch.int32))


MANY = {
    # more segments than the plan has threads, more blocks of a kind than it keeps in shared memory
    "agents_300": (2, 4, 64, 16, 1, [33, 0, 90, 7], [0, 7, 7, 150, 290], [29 * i % 67 for i in range(300)]),
    "agents_300_of_18_rows": (1, 9, 64, 16, 2, [33, 90], [0, 150, 290], [29 * i % 67 for i in range(300)]),
    "agents_260_of_270_rows": (1, 90, 64, 16, 3, [20, 5, 30], [0, 30, 31, 255], [11 * i % 24 for i in range(260)]),
    "groups_300": (1, 2, 128, 32, 1, [13 * i % 80 for i in range(300)], [min(i, 260) for i in range(301)], [5] * 260),
}


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", list(MANY))
def test_many_segments(kvfix, fmt, name):  # noqa: F811
    r = Round(kvfix, fmt, *MANY[name], seed=len(name))
    out, lse = r.call()
    kvfix.check_status()
    r.check(out, lse)


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_calls_on_two_streams(kvfix, fmt):  # noqa: F811
    """Two rounds, each with buffers of its own, at the same time."""
    rounds = [Round(kvfix, fmt, 8, 5, 128, 16, 1, [5000], [0, 6], [300 + 70 * i for i in range(6)], seed=1),
              Round(kvfix, fmt, 2, 4, 64, 32, 2, [900, 300], [0, 16, 24], [2 + 53 * i % 700 for i in range(24)], seed=2)]
    want = [r.call() for r in rounds]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in rounds], [[], []]
    for _ in range(20):
        for r, s, g in zip(rounds, streams, got):
            with torch.cuda.stream(s):
                g.append(r.call())
    torch.cuda.synchronize()
    kvfix.check_status()
    for (out, lse), g in zip(want, got):
        for o, l in g:
            assert torch.equal(o.view(torch.int16), out.view(torch.int16))
            assert torch.equal(l.view(torch.int32), lse.view(torch.int32))


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_no_rows(kvfix, fmt):  # noqa: F811
    """No agents, no new tokens, no rows to write or read: empty results, and the pool as it was."""
    r = Round(kvfix, fmt, 2, 4, 64, 16, 1, [20], [0, 2], [3, 9])
    i32 = dict(dtype=torch.int32, device="cuda")
    for A, T in ((0, 1), (2, 0), (0, 0)):
        q = torch.empty(A, T, 8, 64, dtype=torch.bfloat16, device="cuda")
        out, lse = kvfix.shared_attend(q, r.pool, 16, torch.zeros(A, 3, **i32), torch.zeros(A, **i32), return_lse=True)
        assert out.shape == q.shape and lse.shape == (A, T, 8)
    before = [None if t is None else t.clone() for t in r.pool[1:]]
    none = torch.empty(2, 1, 0, 2, 64, dtype=torch.bfloat16, device="cuda")
    kvfix.pool_write(r.pool, none, none, torch.empty(2, 0, **i32))
    k, v = kvfix.pool_read(r.pool, torch.empty(2, 0, **i32))
    kvfix.check_status()
    assert k.shape == v.shape == none.shape
    for a, b in zip(before, r.pool[1:]):
        assert a is b is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
