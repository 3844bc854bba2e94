"""Page books at the edges of what their calls allow: paths without columns, compactions that move nothing."""
import pytest
import torch

from test_gpu_pages import Paged, i32, kvfix  # noqa: F401  (the fixture)

gpu = pytest.mark.gpu


@gpu
def test_kept_of_a_path_without_columns(kvfix):  # noqa: F811
    """Nothing can be kept of it: lists that ask for some are left alone and flagged, the others are cut."""
    p = Paged(kvfix, "bf16", 16, lens=[40, 40, 40, 0, 33])
    base, kept = [20, 20, 20, 0, 16], [0, 1, -1, 0, 3]
    none = torch.empty(5, 0, dtype=torch.int32, device="cuda")
    moves = p.books.cut(base, [[]] * 5, kept)
    assert p.books.lens == [20, 40, 40, 0, 33]
    kvfix.pages_cut(p.pool, 16, p.refs, p.pages, p.lens, i32(base), none, i32(kept))
    p.check(moves, flags=("bounds",))
    kvfix.pages_cut(p.pool, 16, p.refs, p.pages, p.lens, i32(base), none, i32([0] * 5))
    p.check(p.books.cut(base))


@gpu
@pytest.mark.parametrize("what", ("a length below 0", "a length past the table", "an entry below 0", "an entry past the pool"))
@pytest.mark.parametrize("moves", (False, True))
def test_compactions_flag_what_is_out_of_range(kvfix, what, moves):  # noqa: F811
    """Whether some page moves or none, and whatever is in range follows its pages."""
    p = Paged(kvfix, "e4m3", 16, lens=[40, 17, 70, 20], spare=9)
    p.compact()                                                   # in place now
    if moves:
        p.cut([-1, 0, -1, -1])                                    # (two pages come free)
    if "length" in what:
        p.lens[3] = -1 if "below" in what else p.pages.shape[1] * 16 + 1
    else:
        p.pages[3, 1] = -1 if "below" in what else p.refs.numel()
    p.snap()
    books, length = p.books, p.books.lens[3]
    if "length" in what:
        books.lens[3] = 0                                         # such a list is left as it is
    rows, live = books.compact()
    books.lens[3] = length
    books.flags.add("bounds")
    assert bool(rows) == moves
    assert kvfix.pages_compact(p.pool, 16, p.refs, p.pages, p.lens).item() == live
    p.check(rows, flags=("bounds",))
