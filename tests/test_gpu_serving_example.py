"""The serving operators together with the join and the all-reduce, as the
example runs them: a prompt, then tokens one at a time."""
import importlib.util
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu
FILE = Path(__file__).resolve().parents[1] / "examples" / "tensor_parallel_decode.py"


@pytest.mark.parametrize("sequences,prompt,steps,ranks,bits", [(1, 1, 3, 2, 8), (8, 200, 4, 4, 4), (3, 77, 2, 8, 4)])
def test_steps_stay_near_64_bits(sequences, prompt, steps, ranks, bits):
    """bf16 results are within its rounding, 2^-8 of an element (the attention
    adds 2^-11 a weight, the sum of P ranks' partial results one rounding each);
    a 4-bit group of 128 normal values has a step of a fifteenth of its range of
    5.5 standard deviations, so a rounding error of 0.11 of them; the 4-bit
    all-reduce quantises partial sums and their sum, as in the other example."""
    spec = importlib.util.spec_from_file_location("tensor_parallel_decode", FILE)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    off = example.run(sequences=sequences, prompt=prompt, steps=steps, ranks=ranks, bits=bits, seed=prompt)
    assert off.pop("status") == 0
    limits = {"query": 2 ** -8, "attention": 2 ** -8 + 2 ** -11, "partial": 2 ** -7, "block": 0.25, "weights": 0.2}
    assert {k: v for k, v in off.items() if not v <= limits[k]} == {}
