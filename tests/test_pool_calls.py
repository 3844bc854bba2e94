"""Calls of the paged-pool entry points and of their binding that are refused, or that have
nothing to do: all on the host, without a GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def kvfix():
    from cross_context_kv_gb300 import build
    build.build()
    from cross_context_kv_gb300 import kvfix
    return kvfix


def at(i, byte=0):
    return ctypes.c_void_p((i << 32) + byte)


class Calls:
    """The three entry points on made-up addresses; whatever passes all checks has no rows, so
    nothing is launched."""

    def __init__(self, kvfix):
        self.kvfix, self.lib = kvfix, kvfix.lib

    def desc(self, C=2, n=1, H=4, D=64, layers=1):
        return self.kvfix.KvDesc(C, layers, n, H, D, layers * n * H * D, n * H * D, H * D)

    def pool(self, fmt=0, layers=1, slots=64, H=2, D=64, ss=None, sl=None, k=7 << 32, v=8 << 32, ks=9 << 32, vs=10 << 32):
        ss = H * (2 * D, D, D // 2)[fmt] if ss is None else ss
        return self.kvfix.PoolDesc(fmt, layers, slots, H, D, slots * ss if sl is None else sl, ss, k, v, ks, vs)

    def attend(self, q=at(1), qd=None, p=None, page=16, pp=at(2), mp=4, pl=at(2), gb=at(2), groups=1, sp=at(2), ms=4,
               sl=at(2), scale=0.125, out=at(3), lse=at(4), ws=at(5), wb=1 << 31):
        qd = qd or self.desc()
        return self.lib.kvfix_shared_attend(q, qd, p or self.pool(), page, pp, mp, pl, gb, groups, sp, ms, sl, scale, out,
                                            qd, lse, ws, wb, None)

    def write(self, d=None, p=None, k=at(11), v=at(12), slots=at(13), delta=None, base=1e4):
        return self.lib.kvfix_pool_write(k, v, d or self.desc(H=2), delta, base, slots, p or self.pool(), None)

    def read(self, d=None, p=None, k=at(11), v=at(12), slots=at(13), delta=None, base=1e4):
        return self.lib.kvfix_pool_read(p or self.pool(), slots, delta, base, k, v, d or self.desc(H=2), None)


@pytest.fixture
def calls(kvfix):
    return Calls(kvfix)


def refused(kvfix, status, said):
    msg = kvfix.lib.kvfix_last_error()
    assert status == kvfix.EINVAL and said in msg, (status, msg)


@pytest.mark.parametrize("byte", (1, 2, 3))
def test_arrays_of_words_are_aligned(kvfix, calls, byte):
    """int32 arrays and lse are read and written as words."""
    for name in ("pp", "pl", "gb", "sp", "sl", "lse"):
        refused(kvfix, calls.attend(**{name: at(6, byte)}), b"4-byte aligned")
    for call in (calls.write, calls.read):
        refused(kvfix, call(slots=at(6, byte)), b"4-byte aligned")
        refused(kvfix, call(delta=at(6, byte)), b"4-byte aligned")
