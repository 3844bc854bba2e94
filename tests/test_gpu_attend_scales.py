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


@gpu
@pytest.mark.parametrize("group,new", GROUPS)
@pytest.mark.parametrize("gap", (8, 20, 30, 40))
def test_small_value_rows_beside_large_ones(kvfix, group, new, gap):  # noqa: F811
    """Rows with values in the even dims alone are 2^gap times those in the odd ones: what an output
    keeps of the small rows is what the call states.  A block of up to 16 rows rounds exp(z) times a
    row's scale to f16: by 2^-11 of it, or, below 2^-21 of the row's largest such product, by 2^-32
    of that.  A larger one rounds exp(z) to bf16, by 2^-8 of it whatever the scales are."""
    D = 64
    r = Round(kvfix, "e4m3", 2, group, D, 16, new, [40], [0, 2], [3, 70], seed=11)
    slots = r.pool.k.shape[1]
    odd_row = torch.arange(slots, device="cuda") % 2 == 1
    odd_dim = torch.arange(D, device="cuda") % 2 == 1
    r.pool.v[0][(odd_row[:, None] != odd_dim)[:, None].expand(-1, 2, -1)] = 0
    s = r.pool.v_scales[0]
    s.copy_(torch.where((s != 0xFF) & ~odd_row, s + gap, s))
    out, lse = r.call()
    kvfix.check_status()
    K, V, q = r.values("k"), r.values("v"), ref.of_bf16(r.q_words)
    bytes_of = s.cpu().numpy().astype(np.float64)                       # [heads][slots]
    got, T = ref.of_bf16(words_of(out)), new
    few = group * new <= 8 and 2 * group * new <= 16
    for a in range(2):
        at = np.concatenate((r.rows(r.tables[0][0], 40), r.rows(r.tables[1][a], r.own[a])))
        k, v, n = K(at), V(at), len(at)
        for t in range(T):
            m = n - T + 1 + t
            for h in range(2 * group):
                z = k[:m, h // group] @ q[a, t, h] * r.scale
                p = np.exp(z - z.max())
                x = v[:m, h // group]
                want, mean = p @ x / p.sum(), p @ np.abs(x) / p.sum()
                unit = 2.0 ** (bytes_of[h // group, at[:m]] - 127)
                codes = np.abs(x) / unit[:, None]
                # logits: D products in float, entering weight and sum; sums over the keys
                zerr = D * 2.0 ** -24 * (np.abs(k[:m, h // group]) @ np.abs(q[a, t, h])).max() * r.scale + 2.0 ** -22
                tol = 2.0 ** -8 * np.abs(want) + (2 * zerr + (n + 8) * 2.0 ** -23) * mean
                if few:
                    tol += 2.0 ** -11 * mean + 2.0 ** -32 * (p * unit).max() * codes.sum(0) / p.sum()
                else:
                    tol += 2.0 ** -8 * mean
                err = np.abs(got[a, t, h] - want)
                assert (err <= tol).all(), (a, t, h, np.max(err / tol))
