"""A drafting step's operators restated plainly: rotary positions and masked attention in 64-bit
floats, page books one list after another."""
import math

import numpy as np


# ------------------------------------------------------------------ rotary

def frequencies(base, rot, scaling="none", factor=1.0, low=0.0, high=0.0, original=0):
    """theta_i of the pairs i < rot / 2."""
    out = []
    for i in range(rot // 2):
        t = base ** (-2.0 * i / rot)
        keep = 1.0
        if scaling == "linear":
            keep = 0.0
        elif scaling == "bands":
            keep = (original * t / (2 * math.pi) - low) / (high - low)
        elif scaling == "yarn":
            z = lambda r: rot * math.log(original / (2 * math.pi * r)) / (2 * math.log(base))  # noqa: E731
            lo, hi = max(math.floor(z(high)), 0), min(math.ceil(z(low)), rot - 1)
            keep = 1 - (i - lo) / max(hi - lo, 1e-3)
        keep = min(max(keep, 0.0), 1.0)
        out.append(t * (keep + (1 - keep) / factor))
    return np.array(out)


def rotate(x, positions, theta, layout, attention=1.0):
    """x [C][L][T][H][D] floats at positions [C][T]; the first 2 len(theta) values turn.  Also returns
    what each output's error is measured by: the sum of its pair's magnitudes."""
    n = 2 * len(theta)
    a = positions.astype(np.float64)[:, None, :, None, None] * theta
    c, s = attention * np.cos(a), attention * np.sin(a)
    y, size = x.astype(np.float64).copy(), np.zeros(x.shape)
    i, j = (slice(0, n // 2), slice(n // 2, n)) if layout == "half" else (slice(0, n, 2), slice(1, n, 2))
    y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., j] * c + x[..., i] * s
    size[..., i] = size[..., j] = np.abs(x[..., i]) + np.abs(x[..., j])
    return y, size


# ------------------------------------------------------------------ attention

def attend(q, k, v, sees, scale):
    """One sequence: q [T][Hq][D], k and v [n][H][D], sees [T][n] truth values.  Returns (out, lse); a
    row that sees nothing: zeros and -inf."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    for t in range(T):
        at = np.flatnonzero(sees[t])
        if not len(at):
            continue
        for h in range(Hq):
            z = k[at, h // G] @ q[t, h] * scale
            p = np.exp(z - z.max())
            out[t, h] = p @ v[at, h // G] / p.sum()
            lse[t, h] = z.max() + np.log(p.sum())
    return out, lse


def bits_of(words, T):
    """Mask words int32 [..., W] -> truth values [..., T]."""
    j = np.arange(T)
    return (words[..., j // 32].astype(np.int64) >> (j % 32) & 1).astype(bool)


def words_of(bits):
    """Truth values [..., T] -> int32 words [..., ceil(T / 32)]."""
    T = bits.shape[-1]
    W = (T + 31) // 32
    wide = np.zeros((*bits.shape[:-1], W * 32), np.uint32)
    wide[..., :T] = bits
    return (wide.reshape(*bits.shape[:-1], W, 32) << np.arange(32, dtype=np.uint32)).sum(-1, dtype=np.uint32).view(np.int32)


# ------------------------------------------------------------------ page books

class Books:
    """refs, the lists' pages and lengths, and the moves of rows that the calls ask for (from slot, to
    slot), in the order in which they would be done one by one."""

    def __init__(self, page, refs, pages, lens):
        self.page = page
        self.refs, self.pages, self.lens = list(map(int, refs)), [list(map(int, p)) for p in pages], list(map(int, lens))
        self.flags = set()

    def take(self, n):
        return -(-n // self.page)

    def extend(self, extra, parent=None):
        P, most = self.page, len(self.pages[0]) * self.page if self.pages else 0
        refs, pages, lens = list(self.refs), [list(p) for p in self.pages], list(self.lens)
        free, moves, spent = [p for p, r in enumerate(refs) if r <= 0], [], False
        for i, add in enumerate(extra):
            src = i if parent is None else parent[i]
            if src < 0:
                continue
            n = lens[src] if src < len(lens) else -1
            if n < 0 or add < 0 or n > most or n + add > most or (src != i and lens[i] != 0):
                self.flags.add("bounds")
                continue
            mine = pages[src][:self.take(n)]
            if mine and not 0 <= mine[-1] < len(refs):
                self.flags.add("bounds")
                continue
            copy = add > 0 and n % P != 0 and (src != i or refs[mine[-1]] > 1)
            need = self.take(n + add) - len(mine) + copy
            if need and (spent or need > len(free)):
                self.flags.add("space")
                spent = True
                continue
            new, free = free[:need], free[need:]
            if src != i:
                for p in mine[:-1] if copy else mine:
                    self.refs[p] += 1
            elif copy:
                self.refs[mine[-1]] -= 1
            for p in new:
                self.refs[p] = 1
            if copy:
                moves += [(mine[-1] * P + r, new[0] * P + r) for r in range(n % P)]
                mine = mine[:-1]
            mine = mine + new
            self.pages[i][:len(mine)] = mine
            self.lens[i] = n + add
        return moves

    def cut(self, base, path=None, kept=None):
        P, moves, given = self.page, [], []
        for i, b in enumerate(base):
            if b < 0:
                continue
            n = kept[i] if kept is not None else 0
            way = list(path[i][:n]) if path is not None else []
            fine = 0 <= self.lens[i] <= len(self.pages[i]) * P and b <= self.lens[i] and 0 <= n <= (len(path[i]) if path is not None else 0)
            fine = fine and all(y > x for x, y in zip([-1] + way, way)) and all(b + x < self.lens[i] for x in way)
            if not fine:
                self.flags.add("bounds")
                continue
            slot = lambda t: self.pages[i][t // P] * P + t % P  # noqa: E731,B023
            moves += [(slot(b + x), slot(b + j)) for j, x in enumerate(way)]
            given.append((i, self.take(b + n), self.take(self.lens[i])))
            self.lens[i] = b + n
        for i, lo, hi in given:
            for c in range(lo, hi):
                p = self.pages[i][c]
                if 0 <= p < len(self.refs) and self.refs[p] > 0:
                    self.refs[p] -= 1
                else:
                    self.flags.add("bounds")
                self.pages[i][c] = -1
        return moves

    def compact(self):
        P, live = self.page, sum(r > 0 for r in self.refs)
        holes = [p for p in range(live) if self.refs[p] <= 0]
        to = {}
        for p in range(live, len(self.refs)):
            if self.refs[p] > 0:
                to[p] = holes[len(to)]
        moves = [(p * P + r, q * P + r) for p, q in to.items() for r in range(P)]
        for p, q in to.items():
            self.refs[q], self.refs[p] = self.refs[p], 0
        for i, n in enumerate(self.lens):
            for c in range(self.take(n)):
                self.pages[i][c] = to.get(self.pages[i][c], self.pages[i][c])
        return moves, live
