"""The example runs the four paged-cache calls together (GPU)."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# Outputs are averages of N(0, 1) values, below 6: bf16 queries, keys, P and
# outputs, each off by 2^-8 at most, against unrounded ones; e4m3 values by 2^-4.
@pytest.mark.parametrize("args,tol", [([], 6 * 6 * 2.0 ** -8), (["--window", "96", "--sinks", "4"], 6 * 6 * 2.0 ** -8),
                                      (["--e4m3"], 6 * 2.0 ** -4 * 2)])
def test_example(cuda_lib, args, tol):
    spec = importlib.util.spec_from_file_location("paged_serving", os.path.join(ROOT, "examples", "paged_serving.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.main(args) <= tol
