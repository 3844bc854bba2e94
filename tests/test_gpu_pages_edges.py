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
