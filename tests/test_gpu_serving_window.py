"""Sliding windows over tables whose pages behind the window are gone."""
import pytest
import torch

import _serve_ref as ref
from test_gpu_serving import check, full_cache, gen, make_batch, spoil_behind, tensors, values

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_status():
    from bit_error_compensated_gb300 import echo
    echo.echo_serving_status()


@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("gone", [-1, 1 << 30, "spare"])
@pytest.mark.parametrize("counts,lengths,group,dim,bits", [
    ([1], [1000], 4, 128, 4), ([1, 1, 1], [900, 333, 4000], 4, 64, 8), ([1, 1], [777, 1500], 2, 256, 8),
    ([200], [1111], 1, 128, 4), ([200, 90], [901, 1700], 4, 64, 8), ([130], [1300], 2, 256, 4)])
@pytest.mark.parametrize("window", [1, 17, 64, 100, 200])
def test_pages_wholly_behind_the_window_are_nobody_s_business(page, gone, counts, lengths, group, dim, bits, window):
    """A page that no token's window reaches may be anything in the table (a mark,
    or a page of others that holds no numbers): no report, and the same result as
    with the page in place."""
    from bit_error_compensated_gb300 import echo
    g = gen(window + page)
    starts, table, pages = make_batch(counts, lengths, page, g)
    cache = full_cache(g, pages, page, 2, dim, bits)
    spoil_behind(cache, lengths, table)
    q = values(g, starts[-1], 2 * group, dim, dtype=torch.bfloat16)
    whole = check(cache, tensors(starts, lengths, table), q, starts, lengths, table, window=window)
    if gone == "spare":
        gone = next(p for p in range(pages) if not any((table[b, :(n + page - 1) // page] == p).any() for b, n in enumerate(lengths)))
        cache.meta[gone], cache.codes[gone] = 0x7E007E00, 255
    for b, (n, length) in enumerate(zip(counts, lengths)):
        first = max(0, length - n - window + 1)              # the first key that any of them sees
        table[b, :first // page] = gone
    out = torch.full_like(q, 7)
    echo.echo_attention(cache, tensors(starts, lengths, table), q, out, window=window)
    assert echo.echo_serving_status() == 0
    assert torch.equal(out, whole)


@pytest.mark.parametrize("counts,lengths,dim", [([1], [500], 128), ([150], [500], 64), ([80], [500], 256)])
def test_a_page_that_a_window_reaches_is_reported(counts, lengths, dim):
    from bit_error_compensated_gb300 import echo
    g = gen(dim)
    starts, table, pages = make_batch(counts, lengths, 16, g)
    cache = full_cache(g, pages, 16, 1, dim, 8)
    q = values(g, starts[-1], 2, dim, dtype=torch.bfloat16)
    window = 40
    first = lengths[0] - counts[0] - window + 1
    table[0, :first // 16 + 1] = -1                          # the page that holds it, too
    out = torch.full_like(q, 7)
    echo.echo_attention(cache, tensors(starts, lengths, table), q, out, window=window)
    assert echo.echo_serving_status() == echo.ECHO_ERR_ARG
    exact, _, tol = ref.attention(cache, q, starts, lengths, table, dim ** -0.5, window=window)
    assert ((out.double() - exact).abs() <= tol + ref.half_step(q.dtype) * (exact.abs() + tol)).all()
