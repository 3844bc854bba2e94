"""The example that uses a drafting step's operators together, run as a user would."""
import importlib.util
import pathlib

import pytest

gpu = pytest.mark.gpu
EXAMPLE = pathlib.Path(__file__).resolve().parents[1] / "examples" / "draft_round.py"


def load():
    spec = importlib.util.spec_from_file_location("draft_round", EXAMPLE)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@gpu
@pytest.mark.parametrize("format", ("bf16", "e4m3", "int4"))
@pytest.mark.parametrize("agents,steps,nodes,prefix", ((5, 4, 12, 300), (1, 2, 1, 5), (3, 6, 3, 17), (20, 3, 40, 130)))
def test_a_round_drafts(format, agents, steps, nodes, prefix):
    worst, top, placed = load().run(format, agents, steps, nodes, prefix=prefix)
    # outputs are means of values: a rounding of the output and one of the weights, 2^-8 of the
    # largest value each (values are normal: below 6)
    assert worst <= 2 * 6 * 2.0 ** -8 and top > 0
    assert placed
