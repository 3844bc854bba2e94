"""The example that uses the paged-pool operators together, run as a user would."""
import importlib.util
import pathlib

import pytest

gpu = pytest.mark.gpu
EXAMPLE = pathlib.Path(__file__).resolve().parents[1] / "examples" / "round_decode.py"


def load():
    spec = importlib.util.spec_from_file_location("round_decode", EXAMPLE)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@gpu
@pytest.mark.parametrize("format", ("bf16", "e4m3", "int4"))
@pytest.mark.parametrize("agents,steps,prefix", ((6, 4, 700), (1, 1, 5), (40, 19, 130)))
def test_a_round_decodes(format, agents, steps, prefix):
    worst, top = load().run(format, agents, steps, prefix=prefix)
    # outputs are means of values: a rounding of the output and one of the weights, 2^-8 of the
    # largest value each (values are normal: below 6)
    assert worst <= 2 * 6 * 2.0 ** -8 and top > 0
