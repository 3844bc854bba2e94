"""Index arrays of a drafting step's calls that lie where the calls write are refused: on the host, without
a GPU."""
import random

from test_draft_calls import Rotary, at, desc, kvfix, pool, refused  # noqa: F401  (the fixture)


def test_positions_where_rows_go(kvfix):  # noqa: F811
    call, fn = Rotary(kvfix), b"kvfix_rotary"
    # rows of 5 x 64 values, 2 chunks of 3 tokens: 3840 bytes a plane; positions: 24 bytes
    d, none = desc(kvfix, H=5), kvfix.KvDesc()
    both = dict(qd=d, kd=d)
    for kw in (dict(p=at(4), **both), dict(p=at(4, 3836), **both), dict(p=(4 << 32) - 4, **both), dict(p=at(5, 512), **both),
               dict(p=at(4), qd=d, kd=none), dict(p=at(1, 4), qo=at(1), **both), dict(p=at(2, 3816), ko=at(2), **both)):
        refused(kvfix, fn, call(**kw), b"overlaps positions")
    # just before, just behind, and between rows that leave room (800 bytes from one to the next): these
    # come to the next check, the rotation's
    wide = desc(kvfix, H=5, st=400)
    apart = dict(qd=wide, kd=wide)
    bad = call.rope(rot=66)
    for kw in (dict(p=(4 << 32) - 24, **both), dict(p=at(4, 3840), **both), dict(p=at(4, 640), **apart), dict(p=at(4, 776), **apart)):
        refused(kvfix, fn, call(rope=bad, **kw), b"rotary_dim")
    for kw in (dict(p=at(4, 636), **apart), dict(p=at(4, 780), **apart)):
        refused(kvfix, fn, call(rope=bad, **kw), b"overlaps positions")


def test_positions_between_rows_of_any_layout(kvfix):  # noqa: F811
    """Random layouts against the rows' addresses one by one."""
    call, fn = Rotary(kvfix), b"kvfix_rotary"
    r, base, seen = random.Random(5), 4 << 32, [0, 0]
    none, bad = kvfix.KvDesc(), call.rope(rot=18)
    for _ in range(6000):
        C, n, L, H = r.choice((1, 2, 3)), r.choice((1, 2, 4)), r.choice((1, 2, 3)), r.choice((1, 2, 3))
        row = 16 * H
        dims = [("st", n), ("sl", L), ("sc", C)]
        r.shuffle(dims)
        strides, covered = {}, row
        for name, count in dims:                               # one dimension inside the next, in any order
            strides[name] = covered + 8 * r.choice((0, 0, 1, 3, 9))
            covered = strides[name] * count
        if n > 1 and strides["st"] < row:
            continue
        d = desc(kvfix, C=C, n=n, H=H, D=16, layers=L, **strides)
        rows = [2 * (c * strides["sc"] + l * strides["sl"] + t * strides["st"]) for c in range(C) for l in range(L) for t in range(n)]
        p, size = 4 * r.randint(-4 * C * n, covered // 2 + 4), 4 * C * n
        meets = any(x < p + size and p < x + 2 * row for x in rows)
        refused(kvfix, fn, call(q=1 << 32, qd=d, kd=none, p=base + p, rope=bad), b"overlaps positions" if meets else b"rotary_dim")
        seen[meets] += 1
    assert min(seen) > 500


def test_numbers_of_nodes_where_results_go(kvfix):  # noqa: F811
    def call(nodes):
        qd = desc(kvfix)
        return kvfix.lib.kvfix_tree_attend(at(1), qd, pool(kvfix, layers=1), 16, at(2), 4, at(2), at(2), 1, at(2), 4, at(2), nodes,
                                           at(12), 0.125, at(3), qd, at(4), at(5), 1 << 31, None)

    fn = b"kvfix_tree_attend"
    need = kvfix.lib.kvfix_shared_attend_workspace_bytes(2, 3, 4, 2, 64, 1)
    # out: 6 rows of 4 x 64 values; lse: 6 of 4
    for nodes in (at(3), at(3, 6 * 512 - 4), (3 << 32) - 4, at(4), at(4, 92), at(5), at(5, need - 4), (5 << 32) - 4):
        refused(kvfix, fn, call(nodes), b"nodes")
