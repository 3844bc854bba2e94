"""Index arrays of a drafting step's calls that lie where the calls write are refused: on the host, without
a GPU."""
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
