"""Starts that give more rows than there are."""
import pytest
import torch

from test_gpu_serving import full_cache, gen, tensors, values

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_status():
    from bit_error_compensated_gb300 import echo
    echo.echo_serving_status()


@pytest.mark.parametrize("sequences,tokens", [(6, 8), (46, 8), (6, 800), (46, 800), (4097, 65536)])
def test_starts_that_give_more_rows_than_there_are_give_none(sequences, tokens):
    """Starts that fall and rise again give several sequences the same rows, in
    sum more than there are: the attention writes nothing, and reports."""
    from bit_error_compensated_gb300 import echo
    g = gen(sequences)
    starts = [tokens * (i % 2) for i in range(sequences + 1)]
    table = torch.zeros(sequences, 2, dtype=torch.int32, device="cuda")
    cache = full_cache(g, 1, 16, 1, 64, 4)
    q = values(g, tokens, 2, 64, dtype=torch.bfloat16)
    out, lse = torch.full_like(q, 7), torch.full((tokens, 2), 7.0, device="cuda")
    echo.echo_attention(cache, tensors(starts, [20] * sequences, table), q, out, lse=lse)
    assert echo.echo_serving_status() == echo.ECHO_ERR_SHAPE
    assert torch.all(out == 7) and torch.all(lse == 7)
