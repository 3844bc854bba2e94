"""Calls of the paged-pool entry points and of their binding that are refused, or that have
nothing to do: all on the host, without a GPU."""
import ctypes

import pytest
import torch


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


# ------------------------------------------------------------------ the binding, on stand-ins

class OnGpu:
    """What the binding asks of a CUDA tensor, without one: the shape and strides of a meta
    tensor, a device of its own and a made-up address."""
    is_cuda = True

    def __init__(self, *shape, dtype=torch.int32, device=0, like=None):
        self.meta = torch.empty(shape, dtype=dtype, device="meta") if like is None else like
        self.device = torch.device("cuda", device)

    def __getattr__(self, name):
        return getattr(self.meta, name)

    def __getitem__(self, i):
        return OnGpu(like=self.meta[i], device=self.device.index)

    def get_device(self):
        return self.device.index

    def data_ptr(self):
        return 1 << 32


class NoLaunch:
    """The library with its launching entry points in place of a GPU: they note that they were
    called."""

    def __init__(self, lib):
        self.lib, self.called = lib, []

    def __getattr__(self, name):
        if name.endswith("_bytes") or name == "kvfix_last_error":
            return getattr(self.lib, name)
        return lambda *a: self.called.append(name) or 0


@pytest.fixture
def lib(kvfix, monkeypatch):
    lib = NoLaunch(kvfix.lib)
    monkeypatch.setattr(kvfix, "lib", lib)
    monkeypatch.setattr(kvfix, "_raw_stream", lambda t: 0)
    monkeypatch.setattr(kvfix, "_empty", lambda shape, stride, dtype: OnGpu(*shape, dtype=dtype))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return lib


def attend_args(device=0, **kw):
    bf16 = dict(dtype=torch.bfloat16, device=device)
    pool = OnGpu(1, 64, 2, 64, **bf16)
    from cross_context_kv_gb300 import kvfix
    args = dict(q=OnGpu(2, 1, 4, 64, **bf16), pool=kvfix.Pool("bf16", pool, pool), page_tokens=16,
                suffix_pages=OnGpu(2, 3, device=device), suffix_len=OnGpu(2, device=device),
                prefix_pages=OnGpu(1, 4, device=device), prefix_len=OnGpu(1, device=device),
                group_begin=OnGpu(2, device=device))
    return {**args, **kw}


def test_workspace_is_contiguous(kvfix, lib):
    """A view with gaps has fewer bytes behind its address than its elements count."""
    n = kvfix.lib.kvfix_shared_attend_workspace_bytes(2, 1, 4, 2, 64, 1)
    kvfix.shared_attend(**attend_args(workspace=OnGpu(n, dtype=torch.uint8)))
    assert lib.called == ["kvfix_shared_attend"]
    for w in (OnGpu(2 * n, dtype=torch.uint8)[::2], OnGpu(n // 4, 4, dtype=torch.uint8)[:, :3],
              OnGpu(like=torch.empty(1, dtype=torch.uint8, device="meta").expand(n))):
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            kvfix.shared_attend(**attend_args(workspace=w))
    assert lib.called == ["kvfix_shared_attend"]


def test_tensors_of_another_device_are_refused(kvfix, lib, monkeypatch):
    """The library launches on the current device: tensors of another one never reach it."""
    current = [0]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(kvfix, "_empty", lambda shape, stride, dtype: OnGpu(*shape, dtype=dtype, device=current[0]))
    rows = lambda device: OnGpu(2, 1, 3, 2, 64, dtype=torch.bfloat16, device=device)  # noqa: E731

    def calls(device):
        pool = attend_args(device)["pool"]
        slots = OnGpu(2, 3, device=device)
        return [lambda: kvfix.shared_attend(**attend_args(device)),
                lambda: kvfix.pool_write(pool, rows(device), rows(device), slots),
                lambda: kvfix.pool_read(pool, slots, k_out=rows(device), v_out=rows(device))]

    for device in (0, 1):
        current[0] = device
        for call in calls(device):
            call()
    assert len(lib.called) == 6
    for current[0] in (0, 2):
        for call in calls(1) + [lambda: kvfix.rerope(rows(1), OnGpu(2, device=1), 1e4, out=rows(1))]:
            with pytest.raises(ValueError, match="current device"):
                call()
    assert len(lib.called) == 6


def attend_scale(calls, scale):
    none = calls.desc(C=0)
    return calls.attend(qd=none, groups=0, sp=None, sl=None, lse=None, scale=scale)


@pytest.mark.parametrize("scale", (1e-300, 1e-46, 5e-39, 2.4e38, 1e39, 1e300, -0.125, 0.0))
def test_a_scale_beyond_float_is_refused(kvfix, calls, scale):
    """The kernels multiply by the float scale * log2 e: 0 would make a masked logit NaN."""
    refused(kvfix, attend_scale(calls, scale), b"scale")


@pytest.mark.parametrize("scale", (1e-38, 1e-6, 0.125, 1.0, 3.0, 2.3e38))
def test_a_scale_within_float_is_taken(kvfix, calls, scale):
    assert attend_scale(calls, scale) == kvfix.OK, kvfix.lib.kvfix_last_error()


@pytest.mark.parametrize("given", (("prefix_pages",), ("group_begin",), ("prefix_pages", "group_begin")))
def test_a_prefix_without_lengths_is_refused(kvfix, lib, given):
    """Half a prefix is not taken for none."""
    kw = {name: None for name in ("prefix_pages", "prefix_len", "group_begin") if name not in given}
    with pytest.raises(ValueError, match="prefix_len"):
        kvfix.shared_attend(**attend_args(**kw))
    assert not lib.called
    kvfix.shared_attend(**attend_args(prefix_pages=None, prefix_len=None, group_begin=None))
    # no group at all: lists without an entry
    kvfix.shared_attend(**attend_args(prefix_pages=OnGpu(0, 4), prefix_len=OnGpu(0), group_begin=OnGpu(1)))
    assert len(lib.called) == 2


def test_the_binding_needs_no_private_part_of_torch(kvfix, monkeypatch):
    """A torch without the private allocator and stream look-up has every entry point all the same."""
    import importlib.util
    import sys

    monkeypatch.setitem(sys.modules, "torch._C._dynamo.guards", None)      # (importing it raises)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    spec = importlib.util.spec_from_file_location("kvfix_on_another_torch", kvfix.__file__)
    other = importlib.util.module_from_spec(spec)
    monkeypatch.setitem(sys.modules, spec.name, other)
    spec.loader.exec_module(other)
    assert all(hasattr(other, name) for name in dir(kvfix) if not name.startswith("_"))
    asked = []
    monkeypatch.setattr(torch, "empty_strided", lambda *a, **kw: asked.append((a, kw)) or "tensor")
    assert other._empty((2, 3), (3, 1), torch.uint8) == "tensor"
    assert asked == [(((2, 3), (3, 1)), dict(dtype=torch.uint8, device="cuda"))]

    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: Stream)
    assert other._raw_stream(OnGpu(1)) == 77


def test_interleaved_planes_are_written(kvfix, calls):
    """K and V side by side in a slot, in a layer or in a slot's layers share no byte."""
    none = calls.desc(C=1, n=0, H=2, layers=3)
    base, row = 7 << 32, 2 * 64 * 2
    for ss, sl, apart in ((2 * row, 64 * 2 * row, row),            # [layer][slot][2]
                          (row, 2 * 64 * row, 64 * row),           # [layer][2][slot]
                          (3 * 2 * row, 2 * row, row),             # [slot][layer][2]
                          (3 * 2 * row, row, 3 * row),             # [slot][2][layer]
                          (2 * row + 32, 64 * (2 * row + 32), row + 16)):
        for k, v in ((base, base + apart), (base + apart, base)):
            p = calls.pool(layers=3, ss=ss, sl=sl, k=k, v=v)
            assert calls.write(d=none, p=p) == kvfix.OK, kvfix.lib.kvfix_last_error()
            p = calls.pool(layers=3, ss=ss, sl=sl, k=k, v=v + 16 if v > k else v - 16)
            if ss != 2 * row + 32:                                 # (this one has room for the 16 bytes)
                refused(kvfix, calls.write(d=none, p=p), b"each other")
    one = calls.desc(C=1, n=0, H=2)
    assert calls.write(d=one, p=calls.pool(slots=1, k=base, v=base + row)) == kvfix.OK
    refused(kvfix, calls.write(d=one, p=calls.pool(slots=1, k=base, v=base + row - 16)), b"each other")
    refused(kvfix, calls.write(d=one, p=calls.pool(k=base, v=base)), b"each other")


def test_no_two_rows_of_planes_that_are_written_meet(kvfix, calls):
    """Random small layouts against the rows' addresses one by one."""
    import random

    r, taken = random.Random(5), 0
    none = {L: calls.desc(C=1, n=0, H=1, layers=L) for L in (1, 2, 3)}
    for _ in range(4000):
        L, n, row = r.choice((1, 2, 3)), r.choice((1, 2, 3, 5)), 64
        ss, sl = 16 * r.randint(4, 30), 16 * r.randint(0, 90)
        k, v = ((1 << 32) + 16 * r.randint(0, 120) for _ in range(2))
        st = calls.write(d=none[L], p=calls.pool(fmt=1, layers=L, slots=n, H=1, ss=ss, sl=sl, k=k, v=v))
        at = [{b + l * sl + s * ss + i for l in range(L) for s in range(n) for i in range(0, row, 16)} for b in (k, v)]
        if st == kvfix.OK:
            taken += 1
            assert not at[0] & at[1], (L, n, ss, sl, k, v)
    assert taken > 400


def test_calls_without_rows_do_nothing(kvfix, calls):
    """Tensors without elements have no address: no rows, no agents or no new tokens are no error."""
    for none in (calls.desc(C=0, H=2), calls.desc(n=0, H=2)):
        for call in (calls.write, calls.read):
            for kw in (dict(), dict(slots=None), dict(k=None, v=None, slots=None)):
                assert call(d=none, **kw) == kvfix.OK, kvfix.lib.kvfix_last_error()
            refused(kvfix, call(d=calls.desc(H=2), k=None), b"null")
    for none, lists in ((calls.desc(C=0), dict(sp=None, sl=None)), (calls.desc(n=0), {})):
        assert calls.attend(qd=none, q=None, out=None, lse=None, **lists) == kvfix.OK, kvfix.lib.kvfix_last_error()
    for name in ("q", "out"):
        refused(kvfix, calls.attend(**{name: None}), b"null")


def test_the_rankings_workspaces_are_contiguous(kvfix, lib):
    bf16 = dict(dtype=torch.bfloat16)
    k, q = OnGpu(1, 2, 128, 2, 64, **bf16), OnGpu(1, 2, 4, 4, 64, **bf16)
    A, B = OnGpu(1, 2, 2, 128, 16, **bf16), OnGpu(1, 2, 2, 16, 64, **bf16)
    for call in (lambda w: kvfix.draft_rank(k, q, 1, 8, workspace=w),
                 lambda w: kvfix.lowrank_draft(k, A, B, q, 1, 8, out=k, workspace=w)):
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            call(OnGpu(1 << 24, dtype=torch.uint8)[::2])
    assert not lib.called
