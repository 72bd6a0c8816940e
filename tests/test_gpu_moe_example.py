"""The example that runs router, dispatch, experts, combine, the one-GPU layer and a 4-bit projection together.

Both ways add the same fp32 contributions; the group rounds each rank's sum to
bf16 (2^-8 of it at most) and then the total, the one-GPU layer only the total:
|z - y| <= 2^-8 (sum_r |z_r| + |z| + |y|) per element. With four ranks whose
sums are alike and independent, sum_r |z_r| has about 2 times the norm of the
total, so the relative difference of the norms is at most 4 * 2^-8.
"""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

_spec = importlib.util.spec_from_file_location(
    "moe_decode", os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "moe_decode.py"))


@pytest.mark.parametrize("int4", [False, True])
def test_example(int4):
    example = importlib.util.module_from_spec(_spec)
    _spec.loader.exec_module(example)
    off, same = example.main(int4=int4)
    assert same, "the graph's replay differs from the eager step"
    assert off <= 4 * 2.0 ** -8
