"""kvfix_pool_write and kvfix_pool_read against the 64-bit restatement of the stored forms.

Without rotation every code, scale and value is a matter of exact rules, so all comparisons
are bit for bit; rotated keys are those of kvfix_rerope, bit for bit too.
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


def tensor_of(words, device="cuda"):
    return torch.from_numpy(np.ascontiguousarray(words).view(np.int16)).to(device).view(torch.bfloat16)


def rows(seed, *shape):
    """bf16 words of normal rows with some larger channels and some constant rows."""
    r = np.random.default_rng(seed)
    x = r.standard_normal(shape) * np.where(r.random(shape[-1]) < 0.05, 6.0, 1.0)
    x[..., 0, :] *= 1e-3
    return ref.bf16_of(x)


def canonical(words):
    """Words with every NaN the same (payloads and signs of NaN are not defined)."""
    return np.where((words & 0x7FFF) > 0x7F80, np.uint16(0x7FFF), words)


def stored(pool, p):
    """(codes, scales as [L][slots][H]...) of one plane in numpy."""
    codes = getattr(pool, p)
    codes = words_of(codes) if codes.dtype == torch.bfloat16 else codes.cpu().numpy()
    s = getattr(pool, p + "_scales")
    if s is None:
        return codes, None
    s = words_of(s) if s.dtype == torch.bfloat16 else s.cpu().numpy()
    return codes, np.moveaxis(s, 1, 2)


def assert_same_rows(fmt, got, want):
    (gc, gs), (wc, ws) = got, want
    if fmt == "bf16":
        assert np.array_equal(gc, wc)
        return
    if fmt == "e4m3":
        assert np.array_equal(gs, ws)
        gc, wc = (np.where((s == ref.NAN_ROW)[..., None], c & 127, c) for c, s in ((gc, gs), (wc, ws)))
    else:
        assert np.array_equal(ref.of_bf16(gs), ref.of_bf16(ws))  # -0 and +0 zeros are the same zero
    assert np.array_equal(gc, wc)


SHAPES = [  # chunks, layers, tokens, heads, dim
    (1, 1, 1, 1, 64), (16, 1, 1, 8, 128), (2, 3, 37, 5, 64), (1, 2, 129, 8, 128), (3, 1, 65, 3, 128),
    (1, 5, 300, 1, 64),
]


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", SHAPES)
def test_write_stores_the_rows(kvfix, fmt, shape):
    C, L, n, H, D = shape
    k, v = rows(1, C, L, n, H, D), rows(2, C, L, n, H, D)
    slots = C * n + 11
    at = np.random.default_rng(3).permutation(slots)[:C * n].astype(np.int32)
    at[::7] = -1 if C * n > 3 else at[::7]
    pool = kvfix.pool_empty(fmt, L, slots, H, D)
    kvfix.pool_write(pool, tensor_of(k), tensor_of(v), torch.from_numpy(at.reshape(C, n)).cuda())
    kvfix.check_status()
    kept = at >= 0
    for p, x in (("k", k), ("v", v)):
        codes, scales = stored(pool, p)
        flat = np.moveaxis(x, 1, 0).reshape(L, C * n, H, D)
        wc, ws = ref.encode(fmt, flat)
        assert_same_rows(fmt, (codes[:, at[kept]], None if scales is None else scales[:, at[kept]]),
                         (wc[:, kept], None if ws is None else ws[:, kept]))
        rest = np.setdiff1d(np.arange(slots), at[kept])
        assert not codes[:, rest].any()                       # rows that no slot names stay as they were
        assert scales is None or not scales[:, rest].any()


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", SHAPES)
def test_read_gives_what_is_stored(kvfix, fmt, shape):
    C, L, n, H, D = shape
    slots = C * n + 5
    k, v = rows(4, 1, L, slots, H, D), rows(5, 1, L, slots, H, D)
    pool = kvfix.pool_empty(fmt, L, slots, H, D)
    ident = torch.arange(slots, dtype=torch.int32, device="cuda").view(1, -1)
    kvfix.pool_write(pool, tensor_of(k), tensor_of(v), ident)
    at = np.random.default_rng(6).integers(0, slots, C * n).astype(np.int32)  # rows may repeat
    if C * n > 3:
        at[1::5] = -1
    ko = torch.full((C, L, n, H, D), 3.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    kvfix.pool_read(pool, torch.from_numpy(at.reshape(C, n)).cuda(), k_out=ko, v_out=vo)
    kvfix.check_status()
    for p, got in (("k", ko), ("v", vo)):
        codes, scales = stored(pool, p)
        want = ref.decode(fmt, codes[:, at], None if scales is None else scales[:, at])
        want[:, at < 0] = 3.0
        want = np.moveaxis(want.reshape(L, C, n, H, D), 0, 1)
        assert np.array_equal(ref.of_bf16(words_of(got)), want)


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", (64, 128))
def test_rotation_is_rerope(kvfix, fmt, dim):
    """Writing with a shift stores what writing the re-roped keys stores; reading with a shift
    returns kvfix_rerope of the rows read without one."""
    C, L, n, H = 3, 2, 41, 4
    k, v = tensor_of(rows(7, C, L, n, H, dim)), tensor_of(rows(8, C, L, n, H, dim))
    delta = torch.tensor([137, 0, -6000], dtype=torch.int32, device="cuda")
    at = torch.arange(C * n, dtype=torch.int32, device="cuda").view(C, n)
    a, b = (kvfix.pool_empty(fmt, L, C * n, H, dim) for _ in range(2))
    kvfix.pool_write(a, k, v, at, delta=delta, rope_base=5e5)
    kvfix.pool_write(b, kvfix.rerope(k, delta, 5e5), v, at)
    for x, y in zip(a[1:], b[1:]):
        assert x is y is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    turned, same_v = kvfix.pool_read(b, at, delta=delta, rope_base=1e4)
    plain, plain_v = kvfix.pool_read(b, at)
    kvfix.check_status()
    assert torch.equal(turned.view(torch.int16), kvfix.rerope(plain, delta, 1e4).view(torch.int16))
    assert torch.equal(same_v.view(torch.int16), plain_v.view(torch.int16))


def odd_rows(dim):
    """Rows where the forms can go wrong: zeros, one value, the scale's borders, subnormals,
    the largest values, infinities, NaN, nothing finite."""
    big, inf, nan = 0x7F7F, 0x7F80, 0x7FC0
    base = rows(9, 24, 2, dim)[:, 1]
    base[0] = 0
    base[1] = 0x8000
    base[2] = 0x3F80
    base[3, :] = 0
    base[3, 5] = 0x43E0                # 448 alone: scale 1
    base[4, :] = 0
    base[4, dim - 1] = 0x43E1          # the next bf16 above: scale 2
    base[5] = np.arange(1, dim + 1)    # subnormal words
    base[6, 0] = big
    base[7, 0], base[7, 1] = big, big | 0x8000
    base[8, 3] = inf
    base[9, 3], base[9, dim // 2] = inf | 0x8000, nan
    base[10] = nan
    base[11] = inf
    base[12] = inf | 0x8000
    base[13, 1::2] = nan
    base[14] = 0x0080                  # the smallest normal number
    base[15] = np.where(np.arange(dim) % 2, 0x0080, 0x0081)
    base[16] = 0xBF80
    base[17, :] = np.where(np.arange(dim) % 2, 0x4680, 0x4681)  # large values, one step apart
    base[18, 0] = 0x7F60               # 1.75 * 2^127
    base[19, 0] = 0x7F61
    return base


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", (64, 128))
def test_odd_values(kvfix, fmt, dim):
    x = odd_rows(dim)
    n = len(x)
    words = x.reshape(1, 1, n, 1, dim)
    pool = kvfix.pool_empty(fmt, 1, n, 1, dim)
    at = torch.arange(n, dtype=torch.int32, device="cuda").view(1, n)
    kvfix.pool_write(pool, tensor_of(words), tensor_of(words[:, :, ::-1]), at)
    k, v = kvfix.pool_read(pool, at)
    kvfix.check_status()
    for p, w, back in (("k", x, k), ("v", x[::-1], v)):
        codes, scales = stored(pool, p)
        want = ref.encode(fmt, np.ascontiguousarray(w).reshape(1, n, 1, dim))
        assert_same_rows(fmt, (codes, scales), want)
        value = ref.decode(fmt, *want).reshape(n, dim)
        got = ref.of_bf16(words_of(back)).reshape(n, dim)
        assert np.array_equal(np.isnan(got), np.isnan(value))
        assert np.array_equal(got[~np.isnan(value)], value[~np.isnan(value)])


@gpu
def test_every_e4m3_code_at_every_scale_reads_exactly(kvfix):
    """All 254 codes that are written at the 230 scales the format allows, and the NaN scale."""
    dim, n = 128, 2 * 230
    pool = kvfix.pool_empty("e4m3", 1, n, 1, dim)
    codes = np.arange(256, dtype=np.uint8).reshape(2, 128)
    codes[codes & 127 == 127] = 0
    pool.k.copy_(torch.from_numpy(np.tile(codes, (230, 1)).reshape(1, n, 1, dim)))
    scale = np.repeat(np.arange(-110, 120) + 127, 2).astype(np.uint8)
    scale[100] = ref.NAN_ROW
    pool.k_scales.copy_(torch.from_numpy(scale.reshape(1, 1, n)))
    k, _ = kvfix.pool_read(pool, torch.arange(n, dtype=torch.int32, device="cuda").view(1, n))
    got = ref.of_bf16(words_of(k)).reshape(n, dim)
    want = ref.e4m3_decode(np.tile(codes, (230, 1)), scale)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_views_with_strides(kvfix, fmt):
    """Source and destination rows inside larger tensors; a pool whose slots lie apart and
    whose layers are a slice of a larger pool."""
    L, n, H, D = 2, 19, 2, 64
    wide = tensor_of(rows(10, 3, 2 * L, 2 * n, H, D))
    k, v = wide[:1, ::2, ::2], wide[1:2, 1::2, :n]
    v = torch.empty_strided(k.shape, k.stride(), dtype=k.dtype, device="cuda").copy_(v)
    full = kvfix.pool_empty(fmt, 5, 2 * n, H, D)
    every = lambda t: t[1:3]  # noqa: E731  layers 1 and 2
    planes = [torch.zeros(2, n, 2, *t.shape[2:], dtype=t.dtype, device="cuda")[:, :, 0] for t in (full.k, full.v)]
    scales = [None if t is None else torch.zeros(L, H, n, *t.shape[3:], dtype=t.dtype, device="cuda")
              for t in (full.k_scales, full.v_scales)]
    apart = kvfix.Pool(fmt, *planes, *scales)
    at = torch.arange(n, dtype=torch.int32, device="cuda").flip(0).view(1, n)
    kvfix.pool_write(apart, k, v, at)
    sliced = kvfix.Pool(fmt, every(full.k), every(full.v), *(None if t is None else every(t)
                                                             for t in (full.k_scales, full.v_scales)))
    kvfix.pool_write(sliced, k.contiguous(), v.contiguous(), at)
    out = torch.zeros(1, L, 3 * n, H, D, dtype=torch.bfloat16, device="cuda")
    a = kvfix.pool_read(apart, at, k_out=out[:, :, ::3], v_out=torch.zeros_like(out)[:, :, ::3])
    b = kvfix.pool_read(sliced, at)
    kvfix.check_status()
    for x, y, src in zip(a, b, (k, v)):
        assert torch.equal(x.contiguous().view(torch.int16), y.view(torch.int16))
        c, s = ref.encode(fmt, words_of(src))
        assert np.array_equal(ref.of_bf16(words_of(y)), ref.decode(fmt, c, s))
    assert not out[:, :, 1::3].any() and not full.k[0].any() and not full.k[3:].any()


@gpu
def test_a_slot_beyond_the_pool_is_skipped_and_flagged(kvfix):
    k = tensor_of(rows(11, 1, 1, 3, 2, 64))
    pool = kvfix.pool_empty("e4m3", 1, 4, 2, 64)
    at = torch.tensor([[4, -1, 1]], dtype=torch.int32, device="cuda")
    kvfix.pool_write(pool, k, k.clone(), at)
    with pytest.raises(kvfix.KvfixError) as e:
        kvfix.check_status()
    assert e.value.status == kvfix.EDEVICE
    assert pool.k[0, 1].any() and not pool.k[0, [0, 2, 3]].any()
    out = torch.full((1, 1, 3, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    kvfix.pool_read(pool, at, k_out=out, v_out=out.clone())
    with pytest.raises(kvfix.KvfixError):
        kvfix.check_status()
    assert (out[0, 0, :2] == 7).all() and not (out[0, 0, 2] == 7).all()
    kvfix.check_status()


@gpu
def test_on_a_stream_and_in_a_graph(kvfix):
    k, v = tensor_of(rows(12, 2, 1, 33, 4, 128)), tensor_of(rows(13, 2, 1, 33, 4, 128))
    at = torch.randperm(66, device="cuda").to(torch.int32).view(2, 33)
    want = kvfix.pool_empty("int4", 1, 66, 4, 128)
    kvfix.pool_write(want, k, v, at)
    torch.cuda.synchronize()
    got = kvfix.pool_empty("int4", 1, 66, 4, 128)
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        g.capture_begin()
        kvfix.pool_write(got, k, v, at)
        kvfix.pool_read(got, at, k_out=ko, v_out=vo)
        g.capture_end()
        for _ in range(2):
            g.replay()
    s.synchronize()
    for x, y in zip(got[1:], want[1:]):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    a, b = kvfix.pool_read(want, at)
    assert torch.equal(a, ko) and torch.equal(b, vo)


def test_refusals(kvfix):
    """Bad arguments return KVFIX_EINVAL before anything is launched (no GPU involved)."""
    L = kvfix.lib
    fake, far, odd = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 30), ctypes.c_void_p((1 << 20) + 2)
    fk, fv = 1 << 32, 1 << 33

    def desc(C=1, Ln=1, n=16, H=2, D=64, st=None):
        row = H * D
        return kvfix.KvDesc(C, Ln, n, H, D, Ln * n * row, n * row, row if st is None else st)

    def pool(fmt=1, layers=1, slots=64, H=2, D=64, ss=None, k=fk, v=fv, ks=1 << 34, vs=1 << 35):
        w = H * (2 * D, D, D // 2)[fmt if 0 <= fmt <= 2 else 0]
        return kvfix.PoolDesc(fmt, layers, slots, H, D, slots * w, w if ss is None else ss, k, v, ks, vs)

    def write(d=None, p=None, k=fake, v=far, slots=fake, delta=None, base=1e4):
        return L.kvfix_pool_write(k, v, d or desc(), delta, base, slots, p or pool(), None)

    def read(d=None, p=None, k=fake, v=far, slots=fake, delta=None, base=1e4):
        return L.kvfix_pool_read(p or pool(), slots, delta, base, k, v, d or desc(), None)

    for call, name in ((write, b"kvfix_pool_write"), (read, b"kvfix_pool_read")):
        bad = [
            (dict(p=pool(fmt=3)), b"format"), (dict(p=pool(fmt=-1)), b"format"),
            (dict(p=pool(layers=2)), b"layers"), (dict(p=pool(H=4)), b"heads"),
            (dict(d=desc(D=32), p=pool(D=32)), b"head_dim"), (dict(d=desc(D=256), p=pool(D=256)), b"head_dim"),
            (dict(p=pool(ss=112)), b"smaller"), (dict(p=pool(ss=136)), b"multiples of 16"),
            (dict(p=pool(k=(1 << 32) + 8)), b"aligned"), (dict(p=pool(v=None)), b"aligned"),
            (dict(p=pool(ks=None)), b"scales"), (dict(p=pool(fmt=2, vs=(1 << 35) + 2)), b"4-byte"),
            (dict(p=pool(slots=-1)), b"negative"), (dict(k=None), b"null"), (dict(v=odd), b"aligned"),
            (dict(slots=None), b"slot_mapping"), (dict(delta=fake, base=1.0), b"rope_base"),
            (dict(delta=fake, base=float("nan")), b"rope_base"), (dict(p=pool(k=1 << 20)), b"overlaps"),
            (dict(p=pool(vs=1 << 30)), b"overlaps"), (dict(d=desc(n=1 << 30), k=1 << 45, v=1 << 46), b"kv_heads must be"),
        ]
        for kw, said in bad:
            assert call(**kw) == kvfix.EINVAL, (name, kw)
            msg = L.kvfix_last_error()
            assert msg.startswith(name) and said in msg, (kw, msg)
    assert write(p=pool(v=fk + 64)) == kvfix.EINVAL and b"each other" in L.kvfix_last_error()
    assert read(v=fake) == kvfix.EINVAL and b"overlap" in L.kvfix_last_error()
    # nothing to do is no error, and needs no GPU
    empty = desc(n=0)
    assert write(d=empty, slots=None) == kvfix.OK and read(d=empty, slots=None) == kvfix.OK


def test_binding_refusals(kvfix):
    """The binding's own checks, on tensors that are not on a GPU."""
    pool = kvfix.pool_empty("int4", 1, 8, 2, 64, device="cpu")
    with pytest.raises(TypeError):
        kvfix.pool_desc(pool)
    with pytest.raises(ValueError):
        kvfix.pool_empty("fp8", 1, 8, 2, 64, device="cpu")
    with pytest.raises(ValueError):
        kvfix.pool_desc(pool._replace(format="e5m2"))
    with pytest.raises(TypeError):
        kvfix.pool_write(pool, torch.zeros(1, 1, 4, 2, 64), torch.zeros(1, 1, 4, 2, 64), torch.zeros(1, 4))


def test_the_restatement_itself():
    """pool_ref's forms: every code round-trips, and the error of a stored value is at most
    half a step of its form."""
    v = ref.e4m3_values()
    codes = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    assert v[126] == 448 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[0x38] == 1.0
    row = np.concatenate((v[codes], [448.0, 0.0]))           # the largest code fixes the scale at 1
    got, k = ref.e4m3_encode(row)
    assert k == 127 and np.array_equal(v[got], row)
    x = ref.of_bf16(rows(14, 50, 2, 64))
    c, k = ref.e4m3_encode(x)
    err = np.abs(ref.e4m3_decode(c, k) - x)
    step = 2.0 ** (k.astype(float) - 127)[..., None]
    assert (err <= np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -10 * step)).all()
    b, sz = ref.int4_encode(x)
    err = np.abs(ref.int4_decode(b, sz) - x).reshape(50, 2, 2, 32)
    s = ref.of_bf16(sz[..., 0])[..., None]
    # half a step; up to 15 steps of the scale's own rounding (2^-9 each) at the top; the value's rounding
    assert (err <= s * (0.5 + 15 * 2.0 ** -8) + np.abs(x).reshape(err.shape) * 2.0 ** -8 + 1e-30).all()
