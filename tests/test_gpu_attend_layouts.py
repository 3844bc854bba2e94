"""Pools whose slots lie apart: written, read back and attended over as contiguous ones are."""
import pytest
import torch

from test_gpu_attend import FORMATS, Round, gpu, kvfix  # noqa: F401


def interleaved(kvfix, pool, order):
    """A zeroed pool of the same form whose K and V rows share one buffer."""
    L, n, H, W = pool.k.shape
    if order == "slot":                # [layer][slot][2 and a gap]
        k, v = torch.zeros(L, n, 3, H, W, dtype=pool.k.dtype, device="cuda")[:, :, :2].unbind(2)
    elif order == "layer":             # [layer][2][slot]
        k, v = torch.zeros(L, 2, n, H, W, dtype=pool.k.dtype, device="cuda").unbind(1)
    else:                              # [slot][layer][2]
        k, v = (t.transpose(0, 1) for t in torch.zeros(n, L, 2, H, W, dtype=pool.k.dtype, device="cuda").unbind(2))
    zeros = lambda t: None if t is None else torch.zeros_like(t)  # noqa: E731
    return kvfix.Pool(pool.format, k, v, zeros(pool.k_scales), zeros(pool.v_scales))


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("order", ("slot", "layer", "slot_major"))
def test_planes_that_interleave(kvfix, fmt, order):  # noqa: F811
    L, n, H, D = 3, 50, 2, 64
    gen = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(2, L, n // 2, H, D, generator=gen, device="cuda").bfloat16() for _ in range(2))
    at = torch.randperm(n, generator=gen, device="cuda").int().view(2, -1)
    plain = kvfix.pool_empty(fmt, L, n, H, D)
    mixed = interleaved(kvfix, plain, order)
    kvfix.pool_write(plain, k, v, at)
    kvfix.pool_write(mixed, k, v, at)
    for a, b in zip(plain[1:], mixed[1:]):
        assert a is b is None or torch.equal(a.view(torch.uint8), b.contiguous().view(torch.uint8))
    for a, b in zip(kvfix.pool_read(plain, at), kvfix.pool_read(mixed, at)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    kvfix.check_status()


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", (64, 128))
@pytest.mark.parametrize("order", ("slot", "layer", "slot_major"))
@pytest.mark.parametrize("group,new", ((1, 1), (4, 2), (24, 1)))       # blocks of 8, of 16, of more rows
def test_attention_over_slots_that_lie_apart(kvfix, fmt, dim, order, group, new):  # noqa: F811
    r = Round(kvfix, fmt, 2, group, dim, 32, new, [200], [0, 2], [3, 70], seed=group)
    want, want_lse = r.call()
    # the pool of three layers that this one is the middle of
    three = kvfix.Pool(fmt, *(None if t is None else torch.cat((t, t, t)) for t in r.pool[1:]))
    mixed = interleaved(kvfix, three, order)
    for a, b in zip(mixed[1:], three[1:]):
        if a is not None:
            a[1].copy_(b[1])
    r.pool = mixed.layer(1)
    out, lse = r.call()
    kvfix.check_status()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    assert torch.equal(lse.view(torch.int32), want_lse.view(torch.int32))
    assert not mixed.k[0].any() and not mixed.v[2].any()
