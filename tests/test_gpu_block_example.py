"""The block operators together with the all-reduce, as the example runs them:
join, int8 products, 4-bit all-reduce, join, and the join's gradients."""
import importlib.util
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu
FILE = Path(__file__).resolve().parents[1] / "examples" / "tensor_parallel_block.py"


@pytest.mark.parametrize("tokens,ranks", [(1, 2), (16, 4), (96, 8), (512, 4)])
def test_a_block_step_stays_near_fp32(tokens, ranks):
    """bf16 results are within its rounding (2^-8 of an element); int8 rows and
    weights add about 1/127 of their maximum an element, three to four standard
    deviations: 1% a product; 4-bit codes of the ranks' partial sums, and of
    their sum, add half a step of a fifteenth of a group's range each, 15% of
    the standard deviation of 128 values between +-3."""
    spec = importlib.util.spec_from_file_location("tensor_parallel_block", FILE)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    off = example.run(tokens=tokens, ranks=ranks, seed=tokens)
    assert off.pop("status") == 0
    limits = {"residual": 2 ** -8, "block": 0.25, "out": 0.25, "h": 0.25,
              "dx": 2 ** -7, "dy": 2 ** -7, "dw_post": 2 ** -7, "dw_pre": 2 ** -7}
    assert {k: v for k, v in off.items() if not v <= limits[k]} == {}
