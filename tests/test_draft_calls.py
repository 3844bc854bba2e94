"""Calls of a drafting step's entry points and of their binding that are refused, or that have nothing
to do: all on the host, without a GPU."""
import ctypes
import random

import pytest
import torch

import draft_ref as ref
from test_pool_calls import NoLaunch, OnGpu, attend_args


@pytest.fixture(scope="module")
def kvfix():
    from cross_context_kv_gb300 import build
    build.build()
    from cross_context_kv_gb300 import kvfix
    return kvfix


def at(i, byte=0):
    return ctypes.c_void_p((i << 32) + byte)


def desc(kvfix, C=2, n=3, H=4, D=64, layers=1, st=None, sl=None, sc=None):
    st = H * D if st is None else st
    sl = n * st if sl is None else sl
    return kvfix.KvDesc(C, layers, n, H, D, layers * sl if sc is None else sc, sl, st)


def pool(kvfix, fmt=0, layers=2, slots=64, H=2, D=64, ss=None, k=7 << 32, v=8 << 32, ks=9 << 32, vs=10 << 32):
    ss = H * (2 * D, D, D // 2)[fmt] if ss is None else ss
    return kvfix.PoolDesc(fmt, layers, slots, H, D, slots * ss, ss, k, v, ks, vs)


def refused(kvfix, fn, status, said):
    msg = kvfix.lib.kvfix_last_error()
    assert status == kvfix.EINVAL and said in msg and msg.startswith(fn), (status, msg)


# ------------------------------------------------------------------ rotary

class Rotary:
    def __init__(self, kvfix):
        self.kvfix = kvfix

    def rope(self, layout=0, rot=64, scaling=0, original=0, base=1e4, factor=1.0, low=0.0, high=0.0, attention=1.0):
        return self.kvfix.RopeDesc(layout, rot, scaling, original, base, factor, low, high, attention)

    def __call__(self, q=at(1), qd=None, k=at(2), kd=None, p=at(3), rope=None, qo=at(4), qod=None, ko=at(5), kod=None):
        d = desc(self.kvfix)
        qd, kd = qd or d, kd or d
        return self.kvfix.lib.kvfix_rotary(q, qd, k, kd, p, rope or self.rope(), qo, qod or qd, ko, kod or kd, None)


def test_rotary_refusals(kvfix):
    call, fn = Rotary(kvfix), b"kvfix_rotary"
    d = lambda **kw: desc(kvfix, **kw)  # noqa: E731
    none = kvfix.KvDesc()
    yarn = dict(scaling=3, original=4096, factor=4.0, low=1.0, high=32.0)
    r = call.rope
    nan, inf = float("nan"), float("inf")
    for kw, said in (
            (dict(q=None), b"null"), (dict(qo=None), b"null"), (dict(k=None), b"null"), (dict(ko=None), b"null"),
            (dict(q=at(1, 8)), b"aligned"), (dict(ko=at(5, 2)), b"aligned"), (dict(p=None), b"positions"),
            (dict(p=at(3, 2)), b"4-byte"), (dict(qd=none, kd=none), b"neither"),
            (dict(qod=d(n=4)), b"shape"), (dict(kod=d(C=3)), b"shape"), (dict(kd=d(n=4)), b"same chunks"),
            (dict(kd=d(D=128)), b"same chunks"), (dict(qd=d(D=24)), b"head_dim"), (dict(qd=d(H=-1)), b"kv_heads"),
            (dict(qd=d(st=12)), b"multiples of 8"),
            (dict(qo=at(1, 16)), b"overlaps its input"), (dict(qo=at(2)), b"other plane"), (dict(ko=at(1)), b"other plane"),
            (dict(qo=at(5)), b"other plane"),
            (dict(qd=d(C=1 << 20, n=1 << 12, sc=0), qod=d(C=1 << 20, n=1 << 12, H=4), qo=at(900), kd=none), b"2^31"),
            (dict(qod=d(sc=0)), b"overlap each other"), (dict(kod=d(sc=256)), b"overlap each other"),
            (dict(rope=r(layout=2)), b"layout"), (dict(rope=r(scaling=4)), b"scaling"), (dict(rope=r(scaling=-1)), b"scaling"),
            (dict(rope=r(rot=0)), b"rotary_dim"), (dict(rope=r(rot=7)), b"rotary_dim"), (dict(rope=r(rot=66)), b"rotary_dim"),
            (dict(rope=r(base=1.0)), b"base"), (dict(rope=r(base=nan)), b"base"), (dict(rope=r(base=inf)), b"base"),
            (dict(rope=r(attention=0.0)), b"attention"), (dict(rope=r(attention=nan)), b"attention"),
            (dict(rope=r(attention=1e39)), b"attention"), (dict(rope=r(attention=1e-39)), b"attention"),
            (dict(rope=r(scaling=1, factor=0.5)), b"factor"), (dict(rope=r(scaling=1, factor=inf)), b"factor"),
            (dict(rope=r(**{**yarn, "original": 0})), b"original"), (dict(rope=r(**{**yarn, "low": 0.0})), b"low"),
            (dict(rope=r(**{**yarn, "high": 1.0})), b"low"), (dict(rope=r(**{**yarn, "high": inf})), b"low"),
            (dict(rope=r(**{**yarn, "low": nan})), b"low")):
        refused(kvfix, fn, call(**kw), said)


def test_no_rows_to_turn(kvfix):
    call = Rotary(kvfix)
    for none in (desc(kvfix, C=0), desc(kvfix, n=0), desc(kvfix, layers=0)):
        nothing = dict(qd=none, kd=none, q=None, k=None, qo=None, ko=None)
        assert call(**nothing, p=None) == kvfix.OK, kvfix.lib.kvfix_last_error()
        refused(kvfix, b"kvfix_rotary", call(**nothing, rope=call.rope(rot=3)), b"rotary_dim")


def test_rows_behind_each_other_may_share_a_buffer(kvfix):
    """Queries, keys and values of a token side by side, turned in place; random layouts against the
    rows' addresses one by one."""
    call = Rotary(kvfix)
    base = 1 << 32
    r, taken = random.Random(3), 0
    for _ in range(6000):
        C, n, L = r.choice((1, 2, 3)), r.choice((1, 2, 4)), r.choice((1, 1, 2))
        Hq, Hk = r.choice((1, 2, 3)), r.choice((1, 2))
        st = 16 * r.randint(4, 14)                             # elements; heads of 16
        st = max(st, 16 * max(Hq, Hk))
        sl, sc = 16 * r.randint(0, 60), 16 * r.randint(0, 120)
        qd, kd = (desc(kvfix, C=C, n=n, H=h, D=16, layers=L, st=st, sl=sl, sc=sc) for h in (Hq, Hk))
        q, k = (base + 32 * r.randint(0, 40) for _ in range(2))
        # no rows, so nothing is launched: the checks look at pairs of planes
        rows = [{b + 2 * (c * sc + l * sl + t * st) + 16 * i for c in range(C) for l in range(L) for t in range(n)
                 for i in range(2 * h)} for b, h in ((q, Hq), (k, Hk))]
        apart = [len(x) == C * L * n * 2 * h for x, h in zip(rows, (Hq, Hk))]
        st_ = kvfix.lib.kvfix_rotary(q, qd, k, kd, None, call.rope(rot=16), q, qd, k, kd, None)
        msg = kvfix.lib.kvfix_last_error()
        assert st_ == kvfix.EINVAL                              # (positions is null: nothing is launched)
        if b"positions" in msg:
            taken += 1
            assert not rows[0] & rows[1], (C, n, L, Hq, Hk, st, sl, sc, q, k)
            assert all(apart), (C, n, L, Hq, Hk, st, sl, sc)
        else:
            assert b"other plane" in msg or b"each other" in msg
    assert taken > 300
    qkv = (4 + 2 * 2) * 64
    qd, kd = desc(kvfix, C=3, n=5, H=4, st=qkv), desc(kvfix, C=3, n=5, H=2, st=qkv)
    k = base + 2 * 4 * 64
    call(q=base, qd=qd, k=k, kd=kd, qo=base, ko=k, p=None)
    assert b"positions is null" in kvfix.lib.kvfix_last_error()


# ------------------------------------------------------------------ the tree

def test_tree_refusals(kvfix):
    def call(q=at(1), qd=None, p=None, nodes=at(11), tree=at(12), out=at(3), lse=at(4), ws=at(5), wb=1 << 31, page=16):
        qd = qd or desc(kvfix)
        return kvfix.lib.kvfix_tree_attend(q, qd, p or pool(kvfix, layers=1), page, at(2), 4, at(2), at(2), 1, at(2), 4, at(2),
                                           nodes, tree, 0.125, out, qd, lse, ws, wb, None)

    fn = b"kvfix_tree_attend"
    for kw, said in ((dict(tree=None), b"tree_mask"), (dict(tree=at(12, 2)), b"4-byte"), (dict(nodes=at(11, 1)), b"4-byte"),
                     (dict(tree=at(3)), b"tree_mask"), (dict(tree=at(4)), b"tree_mask"), (dict(tree=at(5)), b"tree_mask"),
                     (dict(q=None), b"null"), (dict(out=None), b"null"), (dict(page=8), b"page_tokens"),
                     (dict(p=pool(kvfix, layers=2)), b"one layer"), (dict(wb=99), b"workspace"), (dict(lse=at(3)), b"overlap")):
        refused(kvfix, fn, call(**kw), said)
    none = desc(kvfix, n=0)
    assert call(qd=none, q=None, out=None, lse=None, tree=None, nodes=None) == kvfix.OK, kvfix.lib.kvfix_last_error()


# ------------------------------------------------------------------ page books

class Books:
    def __init__(self, kvfix):
        self.kvfix, self.lib = kvfix, kvfix.lib

    def first(self, p=None, page=16, refs=at(21), pages=at(22), wide=8, lens=at(23), lists=3):
        return (p or pool(self.kvfix), page, refs, pages, wide, lens, lists)

    def extend(self, parent=at(24), extra=at(25), ws=at(26), wb=1 << 30, **kw):
        return self.lib.kvfix_pages_extend(*self.first(**kw), parent, extra, ws, wb, None)

    def cut(self, base=at(24), path=at(25), most=4, kept=at(26), **kw):
        return self.lib.kvfix_pages_cut(*self.first(**kw), base, path, most, kept, None)

    def compact(self, live=at(24), ws=at(26), wb=1 << 30, **kw):
        return self.lib.kvfix_pages_compact(*self.first(**kw), live, ws, wb, None)


def test_page_book_refusals(kvfix):
    b = Books(kvfix)
    p = lambda **kw: pool(kvfix, **kw)  # noqa: E731
    for name in ("extend", "cut", "compact"):
        call, fn = getattr(b, name), b"kvfix_pages_" + name.encode()
        for kw, said in (
                (dict(p=p(fmt=3, ss=256)), b"format"), (dict(p=p(D=96)), b"head_dim"), (dict(p=p(k=None)), b"16-byte"),
                (dict(p=p(fmt=1, ks=None)), b"scales"), (dict(p=p(fmt=2, ks=(9 << 32) + 2)), b"4-byte"),
                (dict(p=p(v=7 << 32)), b"each other"), (dict(p=p(fmt=1, vs=9 << 32)), b"each other"),
                (dict(p=p(layers=1 << 16, ss=0)), b"stride_slot"), (dict(p=p(layers=70000)), b"65535"),
                (dict(page=8), b"page_tokens"), (dict(page=48), b"page_tokens"), (dict(page=128), b"multiple of page_tokens"),
                (dict(p=p(slots=0)), b"slots"), (dict(p=p(slots=72)), b"slots"),
                (dict(lists=-1), b"lists"), (dict(wide=-1), b"lists"), (dict(lists=1 << 25), b"lists"),
                (dict(lists=1 << 20, wide=1 << 10), b"lists"), (dict(wide=1 << 26), b"lists"),
                (dict(refs=None), b"required"), (dict(pages=None), b"required"), (dict(lens=None), b"required"),
                (dict(refs=at(21, 2)), b"4-byte"), (dict(pages=at(22, 1)), b"4-byte"), (dict(lens=at(23, 3)), b"4-byte"),
                (dict(refs=at(22)), b"overlap"), (dict(lens=at(21)), b"overlap"), (dict(pages=at(7)), b"overlap"),
                (dict(lens=at(8)), b"overlap"), (dict(refs=at(9), p=p(fmt=1)), b"overlap")):
            refused(kvfix, fn, call(**kw), said)
    need = kvfix.lib.kvfix_pages_extend_workspace_bytes(4, 3)
    for kw, said in ((dict(extra=None), b"extra"), (dict(extra=at(25, 2)), b"4-byte"), (dict(parent=at(24, 1)), b"4-byte"),
                     (dict(ws=None), b"workspace"), (dict(ws=at(26, 8)), b"workspace"), (dict(wb=need - 1), b"workspace"),
                     (dict(ws=at(24)), b"overlap"), (dict(ws=at(25)), b"overlap"), (dict(ws=at(21)), b"overlap"),
                     (dict(extra=at(23)), b"overlap"), (dict(parent=at(22)), b"overlap"), (dict(ws=at(8)), b"overlap")):
        refused(kvfix, b"kvfix_pages_extend", b.extend(**kw), said)
    for kw, said in ((dict(base=None), b"base"), (dict(path=None), b"required"), (dict(kept=None), b"required"),
                     (dict(most=0), b"max_path"), (dict(most=0, path=None), b"max_path"), (dict(most=-1), b"max_path"),
                     (dict(most=1 << 29), b"max_path"), (dict(base=at(24, 2)), b"4-byte"), (dict(path=at(25, 1)), b"4-byte"),
                     (dict(kept=at(26, 2)), b"4-byte"), (dict(base=at(23)), b"overlap"), (dict(path=at(22)), b"overlap"),
                     (dict(kept=at(21)), b"overlap"), (dict(path=at(7)), b"overlap")):
        refused(kvfix, b"kvfix_pages_cut", b.cut(**kw), said)
    need = kvfix.lib.kvfix_pages_compact_workspace_bytes(4)
    for kw, said in ((dict(live=None), b"live"), (dict(live=at(24, 2)), b"live"), (dict(ws=None), b"workspace"),
                     (dict(wb=need - 1), b"workspace"), (dict(live=at(21)), b"overlap"), (dict(ws=at(24)), b"overlap"),
                     (dict(ws=at(22)), b"overlap"), (dict(live=at(8)), b"overlap")):
        refused(kvfix, b"kvfix_pages_compact", b.compact(**kw), said)


def test_no_lists(kvfix):
    b = Books(kvfix)
    none = dict(lists=0, pages=None, lens=None)
    assert b.extend(**none, parent=None, extra=None) == kvfix.OK, kvfix.lib.kvfix_last_error()
    assert b.cut(**none, base=None, path=None, kept=None, most=0) == kvfix.OK, kvfix.lib.kvfix_last_error()
    assert kvfix.lib.kvfix_pages_extend_workspace_bytes(0, 3) == 0
    assert kvfix.lib.kvfix_pages_extend_workspace_bytes(4, -1) == 0
    assert kvfix.lib.kvfix_pages_compact_workspace_bytes(0) == 0


# ------------------------------------------------------------------ the binding, on stand-ins

@pytest.fixture
def lib(kvfix, monkeypatch):
    lib = NoLaunch(kvfix.lib)
    monkeypatch.setattr(kvfix, "lib", lib)
    monkeypatch.setattr(kvfix, "_raw_stream", lambda t: 0)
    monkeypatch.setattr(kvfix, "_empty", lambda shape, stride, dtype: OnGpu(*shape, dtype=dtype))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return lib


BF16 = dict(dtype=torch.bfloat16)


def books(kvfix, device=0, **kw):
    plane = OnGpu(2, 64, 2, 64, device=device, **BF16)
    return {**dict(pool=kvfix.Pool("bf16", plane, plane), page_tokens=16, refs=OnGpu(4, device=device),
                   pages=OnGpu(3, 8, device=device), lens=OnGpu(3, device=device)), **kw}


def test_the_binding_checks_what_it_is_given(kvfix, lib):
    x, p = OnGpu(2, 3, 4, 64, **BF16), OnGpu(2, 3)
    rope = kvfix.Rope(1e4)
    kvfix.rotary(x, None, p, rope, q_out=x)
    kvfix.rotary(None, x, p, rope, k_out=x)
    for args, kw, error in (((None, None, p), {}, "neither"), ((x, None, OnGpu(2, 2)), dict(q_out=x), "positions"),
                            ((x, None, p), dict(q_out=OnGpu(2, 3, 2, 64, **BF16)), "shape"),
                            ((x, None, p), dict(q_out=x, k_out=x), "without")):
        with pytest.raises(ValueError, match=error):
            kvfix.rotary(*args, rope, **kw)
    for bad in (kvfix.Rope(1e4, layout="thirds"), kvfix.Rope(1e4, scaling="more")):
        with pytest.raises(ValueError, match="unknown rope"):
            kvfix.rotary(x, None, p, bad, q_out=x)
    with pytest.raises(TypeError, match="positions"):
        kvfix.rotary(x, None, OnGpu(2, 3, dtype=torch.int64), rope, q_out=x)
    mask = OnGpu(2, 1, 1)
    kvfix.tree_attend(**attend_args(tree_mask=mask))
    kvfix.tree_attend(**attend_args(tree_mask=mask, nodes=OnGpu(2)))
    for kw, error in ((dict(tree_mask=OnGpu(2, 1, 2)), "tree_mask"), (dict(tree_mask=mask, nodes=OnGpu(3)), "nodes"),
                      (dict(tree_mask=mask, workspace=OnGpu(1 << 28, dtype=torch.uint8)[::2]), "contiguous")):
        with pytest.raises(ValueError, match=error):
            kvfix.tree_attend(**attend_args(**kw))
    kvfix.pages_extend(**books(kvfix), extra=OnGpu(3), parent=OnGpu(3))
    kvfix.pages_cut(**books(kvfix), base=OnGpu(3))
    kvfix.pages_cut(**books(kvfix), base=OnGpu(3), path=OnGpu(3, 5), kept=OnGpu(3))
    kvfix.pages_cut(**books(kvfix), base=OnGpu(3), path=OnGpu(3, 0), kept=OnGpu(3))
    kvfix.pages_compact(**books(kvfix))
    for call, kw, error in (
            (kvfix.pages_extend, dict(extra=OnGpu(2)), "extra"), (kvfix.pages_extend, dict(extra=OnGpu(3, 2)), "extra"),
            (kvfix.pages_cut, dict(base=OnGpu(3), path=OnGpu(3, 2), kept=OnGpu(2)), "kept"),
            (kvfix.pages_cut, dict(base=OnGpu(3), path=OnGpu(3, 2, device=1), kept=OnGpu(3)), "one device"), (kvfix.pages_extend, dict(extra=OnGpu(3), parent=OnGpu(4)), "parent"),
            (kvfix.pages_extend, dict(extra=OnGpu(3), refs=OnGpu(5)), "refs"), (kvfix.pages_extend, dict(extra=OnGpu(3), lens=OnGpu(2)), "pages"),
            (kvfix.pages_extend, dict(extra=OnGpu(3), workspace=OnGpu(1 << 20, dtype=torch.uint8)[::2]), "contiguous"),
            (kvfix.pages_compact, dict(workspace=OnGpu(1 << 20, dtype=torch.uint8)[::2]), "contiguous"),
            (kvfix.pages_cut, dict(base=OnGpu(2)), "base"), (kvfix.pages_cut, dict(base=OnGpu(3), kept=OnGpu(3)), "together"),
            (kvfix.pages_cut, dict(base=OnGpu(3), path=OnGpu(3, 2, 2), kept=OnGpu(3)), "path"),
            (kvfix.pages_cut, dict(base=OnGpu(3), path=OnGpu(2, 2), kept=OnGpu(3)), "path")):
        with pytest.raises(ValueError, match=error):
            call(**books(kvfix, **kw))
    assert lib.called == ["kvfix_rotary"] * 2 + ["kvfix_tree_attend"] * 2 + \
        ["kvfix_pages_extend"] + ["kvfix_pages_cut"] * 3 + ["kvfix_pages_compact"]


def test_tensors_of_another_device_are_refused(kvfix, lib, monkeypatch):
    current = [1]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(kvfix, "_empty", lambda shape, stride, dtype: OnGpu(*shape, dtype=dtype, device=current[0]))
    rows = OnGpu(2, 3, 4, 64, device=1, **BF16)
    on = lambda *shape, device=1: OnGpu(*shape, device=device)  # noqa: E731
    calls = [lambda: kvfix.rotary(rows, None, on(2, 3), kvfix.Rope(1e4), q_out=rows),
             lambda: kvfix.tree_attend(**attend_args(1, tree_mask=on(2, 1, 1))),
             lambda: kvfix.pages_extend(**books(kvfix, 1), extra=on(3)),
             lambda: kvfix.pages_cut(**books(kvfix, 1), base=on(3)),
             lambda: kvfix.pages_compact(**books(kvfix, 1))]
    for call in calls:
        call()
    assert len(lib.called) == 5
    current[0] = 0
    for call in calls:
        with pytest.raises(ValueError, match="current device"):
            call()
    current[0] = 1
    for call in (lambda: kvfix.rotary(rows, None, on(2, 3, device=0), kvfix.Rope(1e4), q_out=rows),
                 lambda: kvfix.rotary(rows, OnGpu(2, 3, 4, 64, **BF16), on(2, 3), kvfix.Rope(1e4), q_out=rows, k_out=rows),
                 lambda: kvfix.tree_attend(**attend_args(1, tree_mask=on(2, 1, 1, device=0))),
                 lambda: kvfix.pages_extend(**books(kvfix, 1), extra=on(3, device=0)),
                 lambda: kvfix.pages_cut(**books(kvfix, 1, refs=on(4, device=0)), base=on(3))):
        with pytest.raises(ValueError, match="device"):
            call()
    assert len(lib.called) == 5


# ------------------------------------------------------------------ the restatements themselves

def test_the_books_by_hand():
    """Two holders of a page, one grows; a fork; an accepted path; a hole is filled."""
    b = ref.Books(16, [2, 1, 0, 1, 0, 0], [[0, 1, -1], [0, -1, -1], [3, -1, -1], [-1, -1, -1]], [20, 10, 16, 0])
    assert b.extend([0, 1, 1, 3], [0, 1, 2, 0]) == [(r, 32 + r) for r in range(10)] + [(16 + r, 80 + r) for r in range(4)]
    assert b.pages == [[0, 1, -1], [2, -1, -1], [3, 4, -1], [0, 5, -1]] and b.lens == [20, 11, 17, 23]
    assert b.refs == [2, 1, 1, 1, 1, 1]
    assert b.cut([0, -1, 0, 20], [[0], [0], [2], [2]], [0, 0, 0, 1]) == [(86, 84)]
    assert b.refs == [1, 0, 1, 0, 0, 1] and b.pages[0] == [-1, -1, -1] and b.lens == [0, 11, 0, 21]
    moves, live = b.compact()
    assert live == 3 and moves == [(80 + r, 16 + r) for r in range(16)]
    assert b.refs == [1, 1, 1, 0, 0, 0] and b.pages[3][:2] == [0, 1] and not b.flags
