"""The example runs chunk attention, the recurrent chunks, their steps and the
paged calls together (GPU)."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# Attention: averages of N(0, 1) values, below 6; probabilities and outputs are off by
# 2^-8 each at most (pages are compared with what they hold).  Recurrent outputs and states
# stay below 8 times a value's size and a state's share of it: outputs off by 2^-8 for
# operands of one part and 2^-8 for their rounding, states by 2^-14, of at most 8.
@pytest.mark.parametrize("args", [[], ["--window", "96", "--sinks", "4"], ["--e4m3"]])
def test_example(cuda_lib, args):
    spec = importlib.util.spec_from_file_location("hybrid_serving", os.path.join(ROOT, "examples", "hybrid_serving.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    worst = example.main(args)
    assert worst["attention"] <= 6 * 2 * 2.0 ** -8
    assert worst["outputs"] <= 8 * 2 * 2.0 ** -8
    assert worst["states"] <= 8 * 2.0 ** -14
