"""kvfix_tree_attend where rows are many or numbers of nodes are left out: keys of NaN through the join that
takes many rows at a time, and trees of all new tokens with fewer own keys than those."""
import numpy as np
import pytest
import torch

import draft_ref as ref
from test_gpu_tree import FORMATS, Trees, i32, kvfix  # noqa: F401  (the fixture)

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_keys_of_nan_among_many_rows(kvfix, fmt):  # noqa: F811
    """Rows that see nothing but a key of NaN, rows that see it beside others, rows that never do."""
    T = 33
    # (agent 5 has no prefix and nothing before its tree)
    r = Trees(kvfix, fmt, 4, 5, 128, 16, T, [700], [0, 5], [10, 64, 0, 200, 33, 0], [T, 30, T, 5, T, T], kind="any", seed=21)
    hit = {0: 7, 3: 0, 5: 0}                                      # by agent: the node whose key is NaN
    for a, j in hit.items():
        r.bits[a, :, j] = False
        r.bits[a, j + 1, j] = r.bits[a, j + 3, j] = True
    r.bits[5, 1] = r.bits[5, 4] = False
    r.bits[5, 1, 0] = r.bits[5, 4, 0] = True                      # nothing else is left to these two
    r.words.copy_(i32(ref.words_of(r.bits)))
    want, want_lse = r.call()
    kvfix.check_status()
    assert want_lse.numel() > 16 * torch.cuda.get_device_properties(0).multi_processor_count
    r.check(want, want_lse)
    for a, j in hit.items():
        at = int(r.rows(r.tables[1][a], r.own[a])[r.own[a] - r.nodes[a] + j])
        if fmt == "bf16":
            r.pool.k[0, at] = float("nan")
        elif fmt == "e4m3":
            r.pool.k_scales[0, :, at] = 0xFF
        else:
            r.pool.k_scales[0, :, at] = float("nan")
    out, lse = r.call()
    kvfix.check_status()
    for a in hit:
        rows = [t for t in range(r.nodes[a]) if r.bits[a, t, hit[a]]]
        assert len(rows) >= 2
        assert torch.isnan(lse[a, rows]).all() and torch.isnan(out[a, rows].float()).all()
        out[a, rows], lse[a, rows] = want[a, rows], want_lse[a, rows]
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    assert torch.equal(lse.view(torch.int32), want_lse.view(torch.int32))


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("heads,group,T", ((1, 2, 3), (1, 4, 40), (4, 5, 61)))
def test_every_new_token_is_a_node_where_no_number_is_given(kvfix, fmt, heads, group, T):  # noqa: F811
    """nodes None: T each, and as many as there are own keys where these are fewer (flagged)."""
    own = [2, T + 20, 0, T, 1, T - 1, T + 1, 300]
    r = Trees(kvfix, fmt, heads, group, 64, 16, T, [50, 7], [0, 3, 6], own, [0] * len(own), kind="any", seed=T)
    assert r.own == own
    r.words.copy_(i32(ref.words_of(r.bits)))
    r.nodes = [min(T, n) for n in own]
    out, lse = r.call(nodes=None)
    with pytest.raises(kvfix.KvfixError) as e:
        kvfix.check_status()
    assert e.value.status == kvfix.EDEVICE
    r.check(out, lse)
    empty = np.array([[t >= n for t in range(T)] for n in r.nodes])
    assert (out[torch.from_numpy(empty).cuda()] == 0).all()
    kvfix.check_status()
