"""kvfix_rotary against its definition in 64 bits.

Tolerance of an output y of a pair (a, b), m the attention factor: one rounding to bf16, 2^-8 |y|; cos
and sin in float: their argument, at most one half turn, is off by 2^-25 of it (pi 2^-25 < 2^-23 in
the angle), sincospi by 2^-23 of its value and the product with m by 2^-24: below 2^-21 m (|a| + |b|)
together with the two roundings of the pair's sum; and the frequencies, doubles on either side that
may differ in their last places (2^-50 of them), times the position: |p| 2^-50 m (|a| + |b|).
"""
import numpy as np
import pytest
import torch

import draft_ref as ref
import pool_ref

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvfix():
    from cross_context_kv_gb300 import build
    build.build()
    from cross_context_kv_gb300 import kvfix
    return kvfix


def words(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def floats(t):
    return pool_ref.of_bf16(words(t))


def rows(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * 3).bfloat16()


def theta_of(rope, dim):
    return ref.frequencies(rope.base, rope.rotary_dim or dim, rope.scaling, rope.factor, rope.low, rope.high, rope.original)


def check(got, x, positions, rope):
    """x (a tensor before the call) and got, [C][L][T][H][D]."""
    want, size = ref.rotate(floats(x), positions.cpu().numpy(), theta_of(rope, x.shape[-1]), rope.layout, rope.attention)
    far = np.abs(positions.cpu().numpy().astype(np.float64))[:, None, :, None, None]
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -21 + far * 2.0 ** -50) * rope.attention * size
    rot = rope.rotary_dim or x.shape[-1]
    err = np.abs(floats(got) - want)
    assert (err[..., :rot] <= tol[..., :rot]).all(), np.argwhere(~(err <= tol))[:4]
    assert torch.equal(got[..., rot:].contiguous().view(torch.int16), x[..., rot:].contiguous().view(torch.int16))


SHAPES = {
    # chunks, layers, tokens, query heads, key heads, dim, rotary_dim
    "one": (1, 1, 1, 1, 0, 64, 64),
    "draft": (16, 1, 8, 32, 8, 128, 128),
    "keys": (2, 3, 37, 0, 5, 128, 64),
    "odd_heads": (3, 1, 5, 7, 3, 96, 48),
    "part_of_20": (2, 2, 9, 5, 1, 80, 20),
    "part_of_24": (2, 1, 19, 4, 2, 96, 24),
    "all_but_eight": (1, 3, 21, 3, 2, 64, 56),
    "part_of_6": (3, 1, 7, 2, 3, 32, 6),
    "two_values": (1, 2, 3, 2, 2, 16, 2),
    "all_but_two": (2, 1, 4, 3, 1, 16, 14),
    "wide": (1, 1, 70, 3, 2, 256, 256),
    "wide_part": (1, 1, 33, 1, 1, 256, 250),
    "many_tokens": (1, 2, 3000, 4, 1, 64, 32),
    "many_layers": (1, 40, 300, 0, 8, 128, 128),
    "many_chunks": (700, 1, 1, 2, 1, 64, 64),
    "many_heads": (1, 1, 2, 129, 3, 112, 96),
}
ROPES = {
    "none": dict(base=1e4),
    "linear": dict(base=1e4, scaling="linear", factor=4.0),
    "bands": dict(base=5e5, scaling="bands", factor=8.0, low=1.0, high=4.0, original=8192),
    "yarn": dict(base=1e6, scaling="yarn", factor=16.0, low=1.0, high=32.0, original=32768, attention=1.2772588722239781),
    "yarn_short": dict(base=1e4, scaling="yarn", factor=3.0, low=0.5, high=600.0, original=100, attention=0.5),
}


@gpu
@pytest.mark.parametrize("layout", ("half", "interleaved"))
@pytest.mark.parametrize("scaling", list(ROPES))
@pytest.mark.parametrize("shape", list(SHAPES))
def test_rotary(kvfix, shape, scaling, layout):
    C, L, T, Hq, Hk, D, rot = SHAPES[shape]
    rope = kvfix.Rope(rotary_dim=rot, layout=layout, **ROPES[scaling])
    q = rows(C, L, T, Hq, D, seed=1) if Hq else None
    k = rows(C, L, T, Hk, D, seed=2) if Hk else None
    positions = torch.randint(-200000, 200000, (C, T), device="cuda", dtype=torch.int32)
    positions[0, 0] = 0
    got = kvfix.rotary(q, k, positions, rope)
    # in place gives the same bits
    q2, k2 = (None if x is None else x.clone() for x in (q, k))
    kvfix.rotary(q2, k2, positions, rope, q_out=q2, k_out=k2)
    for x, y, z in zip((q, k), got, (q2, k2)):
        assert (x is None) == (y is None)
        if x is not None:
            check(y, x, positions, rope)
            assert torch.equal(y.view(torch.int16), z.view(torch.int16))


@gpu
@pytest.mark.parametrize("rot", (128, 20))
@pytest.mark.parametrize("layout", ("half", "interleaved"))
def test_far_positions(kvfix, layout, rot):
    """Positions to the ends of 32 bits: the angle keeps its place within a turn."""
    x = rows(1, 1, 8, 2, 128)
    positions = torch.tensor([[2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, -12345677, 2 ** 24 + 1, 1, -1, 2 ** 31 - 2]],
                             dtype=torch.int32, device="cuda")
    for name in ("none", "bands"):
        rope = kvfix.Rope(rotary_dim=rot, layout=layout, **ROPES[name])
        check(kvfix.rotary(x, None, positions, rope)[0], x, positions, rope)


@gpu
@pytest.mark.parametrize("rot", (64, 20))
@pytest.mark.parametrize("layout", ("half", "interleaved"))
def test_position_zero_is_the_identity(kvfix, layout, rot):
    x = rows(1, 1, 2, 3, 64)
    odd = torch.tensor([float("inf"), -float("inf"), float("nan"), -0.0, 0.0, 1e-40, 3e38, -1.0], device="cuda").bfloat16()
    x.view(-1)[:] = odd.repeat(x.numel() // 8)
    zero = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    got = kvfix.rotary(x, None, zero, kvfix.Rope(1e4, rot, layout))[0]
    assert torch.equal(got.view(torch.int16), x.view(torch.int16))


@gpu
@pytest.mark.parametrize("layout", ("half", "interleaved"))
def test_views_of_a_projection(kvfix, layout):
    """Queries, keys and values of a token behind each other in one buffer, turned in place."""
    C, T, Hq, Hk, D = 3, 11, 6, 2, 64
    buf = rows(C, T, Hq + 2 * Hk, D)
    was = buf.clone()
    q, k = buf[:, :, :Hq], buf[:, :, Hq:Hq + Hk]
    positions = torch.randint(0, 9999, (C, T), device="cuda", dtype=torch.int32)
    rope = kvfix.Rope(1e4, 32, layout)
    kvfix.rotary(q, k, positions, rope, q_out=q, k_out=k)
    check(q.unsqueeze(1), was[:, None, :, :Hq], positions, rope)
    check(k.unsqueeze(1), was[:, None, :, Hq:Hq + Hk], positions, rope)
    assert torch.equal(buf[:, :, Hq + Hk:], was[:, :, Hq + Hk:])
    # from one buffer to another, with gaps between rows
    wide = torch.full((C, T + 1, Hq + Hk + 3, D), 7.0, dtype=torch.bfloat16, device="cuda")
    kvfix.rotary(was[:, :, :Hq], was[:, :, Hq:Hq + Hk], positions, rope, q_out=wide[:, :T, 3:3 + Hq], k_out=wide[:, :T, 3 + Hq:])
    assert torch.equal(wide[:, :T, 3:3 + Hq], q) and torch.equal(wide[:, :T, 3 + Hq:], k)
    assert (wide[:, T:] == 7).all() and (wide[:, :, :3] == 7).all()


@gpu
def test_one_of_two_in_place(kvfix):
    q, k = rows(2, 3, 4, 64), rows(2, 3, 2, 64, seed=3)
    positions = torch.randint(0, 999, (2, 3), device="cuda", dtype=torch.int32)
    rope = kvfix.Rope(1e4, 32)
    want = kvfix.rotary(q, k, positions, rope)
    out = torch.zeros_like(q)
    kvfix.rotary(q, k, positions, rope, q_out=out, k_out=k)
    assert torch.equal(out, want[0]) and torch.equal(k, want[1])


@gpu
@pytest.mark.parametrize("layout", ("half", "interleaved"))
def test_a_gradient_is_the_rotation_back(kvfix, layout):
    """<g, dy> = <turned back g, dx>: against the transposed formula, and against differences."""
    C, T, H, D, rot = 2, 5, 3, 64, 48
    rope = kvfix.Rope(rotary_dim=rot, layout=layout, **ROPES["yarn"])
    g = rows(C, T, H, D, seed=4)
    positions = torch.randint(0, 99999, (C, T), device="cuda", dtype=torch.int32)
    back = kvfix.rotary(g, None, -positions, rope)[0]
    check(back.unsqueeze(1), g.unsqueeze(1), -positions, rope)
    theta, p = theta_of(rope, D), positions.cpu().numpy()
    r = np.random.default_rng(0)
    x, dx = r.standard_normal((2, C, 1, T, H, D))
    turn = lambda v: ref.rotate(v, p, theta, layout, rope.attention)[0]  # noqa: E731
    h = 1e-6
    slope = (floats(g)[:, None] * (turn(x + h * dx) - turn(x - h * dx)) / (2 * h)).sum()
    size = (np.abs(floats(back)[:, None]) * np.abs(dx)).sum()
    # each component of the turned gradient is off by 2^-8 of it (and 2^-21 of its pair)
    assert abs(slope - (floats(back)[:, None] * dx).sum()) <= (2.0 ** -8 + 2.0 ** -10) * size


@gpu
def test_rotations_add_up(kvfix):
    """Cached keys moved by a shift are keys at the shifted positions, to the two roundings."""
    x = rows(1, 4, 50, 2, 128)
    p = torch.arange(50, dtype=torch.int32, device="cuda").view(1, -1)
    rope = kvfix.Rope(layout="interleaved", **ROPES["bands"])
    at = kvfix.rotary(None, x, p, rope)[1]
    moved = kvfix.rotary(None, at, torch.full_like(p, 777), rope)[1]
    want, size = ref.rotate(floats(x), (p + 777).cpu().numpy(), theta_of(rope, 128), "interleaved")
    assert (np.abs(floats(moved) - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -8 * 1.5 + 2.0 ** -20) * size).all()


@gpu
def test_on_a_stream_and_in_a_graph(kvfix):
    q, k = rows(4, 2, 8, 64), rows(4, 2, 2, 64, seed=5)
    q_out, k_out = torch.empty_like(q), torch.empty_like(k)
    positions = torch.full((4, 2), 5, dtype=torch.int32, device="cuda")
    rope = kvfix.Rope(1e4)
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        g.capture_begin()
        kvfix.rotary(q, k, positions, rope, q_out=q_out, k_out=k_out)
        g.capture_end()
        for p in (5, 60000):
            positions.fill_(p)
            g.replay()
            s.synchronize()
            check(q_out.unsqueeze(1), q.unsqueeze(1), positions, rope)
            check(k_out.unsqueeze(1), k.unsqueeze(1), positions, rope)


@gpu
def test_nothing_to_turn(kvfix):
    none = torch.empty(0, 3, 2, 64, dtype=torch.bfloat16, device="cuda")
    p = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    q, k = kvfix.rotary(none, none, p, kvfix.Rope(1e4))
    assert q.shape == none.shape and k.shape == none.shape
