"""Softmax scales other than the default, and e4m3 scale bytes at and beyond the format's ends."""
import numpy as np
import pytest
import torch

import pool_ref as ref
from test_gpu_attend import FORMATS, Round, gpu, kvfix, words_of  # noqa: F401

GROUPS = ((1, 1), (4, 2), (24, 1))       # (query heads of a KV head, new tokens): blocks of 8, of 16, of more rows


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("group,new", GROUPS)
@pytest.mark.parametrize("scale", (1e-30, 0.01, 1.0, 2.5))
def test_other_scales(kvfix, fmt, group, new, scale):  # noqa: F811
    r = Round(kvfix, fmt, 2, group, 64, 16, new, [40], [0, 2], [3, 70], seed=5)
    r.scale = scale
    out, lse = r.call(scale=scale)
    kvfix.check_status()
    r.check(out, lse)


@gpu
@pytest.mark.parametrize("group,new", GROUPS)
@pytest.mark.parametrize("plane,low,high", (("k", 0, 16), ("k", 247, 254), ("v", 0, 16), ("v", 247, 254)))
def test_scale_bytes_beyond_the_ends_are_the_ends(kvfix, group, new, plane, low, high):  # noqa: F811
    """A byte below 17 counts as 17 (2^-110), one of 247 to 254 as 246 (2^119), for every block size
    as for pool_read."""
    r = Round(kvfix, "e4m3", 2, group, 64, 16, new, [40], [0, 2], [3, 70], seed=9)
    scales = getattr(r.pool, plane + "_scales")
    used = scales != 0xFF
    rng = np.random.default_rng(2)
    odd = torch.from_numpy(rng.integers(low, high + 1, scales.shape).astype(np.uint8)).cuda()
    end = 17 if high < 17 else 246
    if plane == "k":
        # queries that undo the keys' size
        r.q.mul_(2.0 ** (127 - end) if end == 246 else 2.0 ** 100)
    elif end == 246:
        # the smallest codes, at most 7 * 2^-9: sums of what they stand for stay within float
        r.pool.v.bitwise_and_(0x87)
    scales.copy_(torch.where(used, torch.full_like(scales, end), scales))
    want, want_lse = r.call()
    slots = torch.arange(scales.shape[-1], dtype=torch.int32, device="cuda").view(1, -1)
    want_rows = kvfix.pool_read(r.pool, slots)
    scales.copy_(torch.where(used, odd, scales))
    out, lse = r.call()
    rows = kvfix.pool_read(r.pool, slots)
    kvfix.check_status()
    assert torch.isfinite(want.float()).all() and torch.isfinite(want_lse).all()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    assert torch.equal(lse.view(torch.int32), want_lse.view(torch.int32))
    for a, b in zip(rows, want_rows):
        a, b = ref.of_bf16(words_of(a)), ref.of_bf16(words_of(b))
        assert np.array_equal(a, b, equal_nan=True)
