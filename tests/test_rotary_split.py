"""How kvfix_rotary's work falls to threads, on the CPU: every token, layer, column and run of heads once, up to
the documented sizes (chunks * layers * tokens < 2^31), where sums of 32 bits with a sign would wrap."""
import ctypes
import itertools
import pathlib
import subprocess

import pytest

HEADER = pathlib.Path(__file__).resolve().parents[1] / "cross_context_kv_gb300" / "csrc" / "rotary_split.h"
SOURCE = '''
#include "%s"
extern "C" void split(const int* x, int* w) {
    const kvfix::RotarySplit s = kvfix::rotary_split(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]);
    const int got[] = {s.columns, s.runs, s.tile, s.tiles, s.layer_block, s.layer_blocks};
    for (int i = 0; i < 6; ++i) w[i] = got[i];
}
extern "C" int place(const int* w, int layers, int tokens, unsigned block, int thread, long long* p) {
    const kvfix::RotarySplit s = {w[0], w[1], w[2], w[3], w[4], w[5]};
    kvfix::RotaryPlace at;
    const bool there = kvfix::rotary_place(s, tokens, block, thread, at);
    p[0] = at.column; p[1] = at.run; p[2] = at.chunk; p[3] = at.layer0; p[5] = at.token;
    p[4] = (long long)at.layer0 + kvfix::rotary_layers(s, layers, at.layer0);
    return there;
}
'''


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("rotary_split")
    (d / "split.cpp").write_text(SOURCE % HEADER)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-shared", "-fPIC", "-o", str(d / "split.so"), str(d / "split.cpp")],
                   check=True)
    return ctypes.CDLL(str(d / "split.so"))


def split(lib, chunks, layers, tokens, heads, dim, rot, half, in_place):
    w = (ctypes.c_int * 6)()
    lib.split((ctypes.c_int * 8)(chunks, layers, tokens, heads, dim, rot, half, in_place), w)
    return w


def place(lib, w, layers, tokens, block, thread):
    """(column, run, chunk, first layer, the one behind the last, token, whether there is work)."""
    p = (ctypes.c_longlong * 6)()
    there = bool(lib.place(w, layers, tokens, ctypes.c_uint(block), thread, p))
    return (*p, there)


FORMS = [(64, 64, 1, 1), (64, 20, 1, 0), (128, 24, 1, 1), (96, 96, 0, 0), (16, 2, 1, 1), (256, 250, 1, 0), (16, 16, 0, 1)]


def test_small_sizes_whole(lib):
    for (dim, rot, half, here), C, L, T, H in itertools.product(FORMS, (1, 3), (1, 2, 9), (1, 5, 40), (1, 7)):
        w = split(lib, C, L, T, H, dim, rot, half, here)
        seen = set()
        for block in range(C * w[3] * w[5]):
            for thread in range(256):
                column, run, chunk, l0, l1, t, there = place(lib, w, L, T, block, thread)
                if there:
                    assert 0 <= t < T
                    for layer in range(l0, l1):
                        key = (column, run, chunk, layer, t)
                        assert key not in seen
                        seen.add(key)
        assert len(seen) == w[0] * w[1] * C * L * T


BIG = 2 ** 31 - 1


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("C,L,T", ((1, 1, BIG), (1, BIG, 1), (BIG, 1, 1), (1, 1, BIG - 127), (1, BIG - 3, 1), (1, 2, 2 ** 30 - 1),
                                   (3, 7, BIG // 21), (1, 65535, 32767)))
def test_the_largest_sizes_at_their_ends(lib, form, C, L, T):
    w = split(lib, C, L, T, 3, *form)
    columns, runs, tile, tiles, layer_block, layer_blocks = w
    assert columns > 0 and runs > 0 and tile > 0 and columns * runs * tile <= 256
    assert (tiles - 1) * tile < T <= tiles * tile and (layer_blocks - 1) * layer_block < L <= layer_blocks * layer_block
    assert C * tiles * layer_blocks <= BIG
    for chunk, at, lb in itertools.product({0, C - 1}, {0, tiles - 1}, {0, layer_blocks - 1}):
        block = (chunk * tiles + at) * layer_blocks + lb
        tokens = []
        for thread in range(256):
            column, run, c, l0, l1, t, there = place(lib, w, L, T, block, thread)
            assert c == chunk and l0 == lb * layer_block and l1 == min(L, l0 + layer_block)
            if there:
                assert t // tile == at
                tokens.append((t, run, column))
        here = range(at * tile, min(T, (at + 1) * tile))
        assert sorted(tokens) == [(t, r, c) for t in here for r in range(runs) for c in range(columns)]
