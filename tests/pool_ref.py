"""The paged pool's stored forms and its attention, restated in numpy with 64-bit floats.

bf16 values are handled as their 16-bit words (uint16) and as the floats those stand for.
"""
import numpy as np

GROUP = 32


def bf16_of(x):
    """float64 -> bf16 words, round to nearest even (through float32 where that is exact or
    the rounding below it cannot tie differently: callers pass float32-exact values)."""
    f = np.asarray(x, np.float64).astype(np.float32)
    u = f.view(np.uint32)
    nan = np.isnan(f)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(nan, np.uint16(0x7FFF), r)


def of_bf16(w):
    return (np.asarray(w, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def e4m3_values():
    """The value of every e4m3 code."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(e > 0, (8 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9)
    return np.where(c > 127, -v, v)


NAN_ROW = 255  # the scale byte of a row that holds a NaN


def e4m3_encode(x):
    """Rows [..., D] of floats -> (codes uint8 [..., D], scale bytes uint8 [...])."""
    fine = np.isfinite(x)
    a = np.where(fine, np.abs(x), 0.0).max(-1)
    k = np.full(a.shape, -110)
    some = a > 0
    with np.errstate(divide="ignore"):
        m, e = np.frexp(np.where(some, a, 1.0) / 448.0)       # a / 448 = m 2^e, m in [0.5, 1)
    k[some] = np.clip(np.where(m == 0.5, e - 1, e), -110, 119)[some]
    y = np.abs(x) / 2.0 ** k[..., None].astype(np.float64)
    grid = e4m3_values()[:127]                                # 0 .. 448, ascending
    y = np.where(np.isnan(y), 0.0, np.minimum(y, 448.0))
    up = np.clip(np.searchsorted(grid, y), 1, 126)
    lo, hi = grid[up - 1], grid[up]
    pick = np.where((y - lo < hi - y) | ((y - lo == hi - y) & ((up - 1) % 2 == 0)), up - 1, up)
    code = pick | np.where(np.signbit(x), 128, 0)
    bad = np.isnan(x).any(-1)
    code[bad] &= 128  # (the sign of a zero code means nothing)
    return code.astype(np.uint8), np.where(bad, NAN_ROW, k + 127).astype(np.uint8)


def e4m3_decode(codes, scale):
    v = e4m3_values()[codes] * 2.0 ** (scale.astype(np.float64) - 127)[..., None]
    return np.where((scale == NAN_ROW)[..., None], np.nan, v)


def int4_encode(x):
    """Rows [..., D] -> (bytes uint8 [..., D/2], scale and zero as bf16 words [..., D/32, 2]).
    Scale and codes follow the float32 operations of the definition."""
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    fine = np.isfinite(g)
    some = fine.any(-1)
    lo = np.where(some, np.where(fine, g, np.inf).min(-1), 0.0).astype(np.float32)
    hi = np.where(some, np.where(fine, g, -np.inf).max(-1), 0.0).astype(np.float32)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        span = np.minimum(hi - lo, np.finfo(np.float32).max)
        scale = bf16_of((span / np.float32(15)).astype(np.float64))
        s = of_bf16(scale).astype(np.float32)
        s = np.where(s < np.float32(2.0 ** -120), np.float32(0), s)
        inv = np.where(s > 0, np.float32(1) / s, np.float32(0))
        c = np.rint((g.astype(np.float32) - lo[..., None]) * inv[..., None])
    c = np.clip(np.where(np.isnan(c), 0, c), 0, 15).astype(np.uint32).reshape(*x.shape[:-1], -1, 8)
    at = np.array([0, 16, 4, 20, 8, 24, 12, 28], np.uint32)
    words = (c << at).sum(-1).astype("<u4")
    sz = np.stack((bf16_of(s.astype(np.float64)), bf16_of(lo.astype(np.float64))), -1)
    return words.view(np.uint8).reshape(*x.shape[:-1], -1), sz


def int4_decode(codes, sz):
    w = np.ascontiguousarray(codes).view("<u4")
    at = np.array([0, 16, 4, 20, 8, 24, 12, 28], np.uint32)
    c = ((w[..., None] >> at) & 15).astype(np.float64).reshape(*codes.shape[:-1], sz.shape[-2], GROUP)
    s, z = of_bf16(sz[..., 0])[..., None], of_bf16(sz[..., 1])[..., None]
    v = c * s + z                                             # exact in float32 (see the range note)
    return of_bf16(bf16_of(v)).reshape(*codes.shape[:-1], 2 * codes.shape[-1])


def encode(fmt, words):
    """bf16 words [..., D] -> (codes, scales or None)."""
    if fmt == "bf16":
        return words, None
    return (e4m3_encode if fmt == "e4m3" else int4_encode)(of_bf16(words))


def decode(fmt, codes, scales):
    """Stored rows -> the floats they stand for."""
    if fmt == "bf16":
        return of_bf16(codes)
    return (e4m3_decode if fmt == "e4m3" else int4_decode)(codes, scales)


def attend(q, k, v, visible, scale):
    """One sequence: q [T][Hq][D], k and v [n][H][D] floats, query t sees the first visible[t]
    keys.  Returns (out [T][Hq][D], lse [T][Hq]); a row that sees nothing: zeros and -inf."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    for t in range(T):
        n = int(min(max(visible[t], 0), k.shape[0]))
        if n == 0:
            continue
        for h in range(Hq):
            z = k[:n, h // G] @ q[t, h] * scale
            top = z.max()
            p = np.exp(z - top)
            out[t, h] = p @ v[:n, h // G] / p.sum()
            lse[t, h] = top + np.log(p.sum())
    return out, lse
