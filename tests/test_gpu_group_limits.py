"""Groups whose step is the largest that fp16 holds."""
import pytest
import torch

import _serve_ref as ref
from test_gpu_serving import DTYPES, tensors

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_status():
    from bit_error_compensated_gb300 import echo
    echo.echo_serving_status()


def ranges(bits, dtype):
    """Rows of 64 whose range is the largest step's, and what lies beside it."""
    top = 65504.0 * (2 ** bits - 1)
    dt, rows = DTYPES[dtype], []
    if dtype == "f32":
        for d in (top, torch.tensor(top).nextafter(torch.tensor(0.0)).item(), top * (1 - 2.0 ** -14),
                  torch.tensor(top).nextafter(torch.tensor(2 * top)).item(), top * (1 + 2.0 ** -14)):
            for part in (0.0, 0.25, 1.0):
                rows.append([d * (1 - part), -d * part])
        rows.append([top, -1e-3])                            # beyond, by less than an fp32 step
    else:
        assert bits == 4                                     # 982560 = 978944 + 3616, both of 8 bits
        rows = [[978944.0, -3616.0], [978944.0, -3600.0], [978944.0, -3632.0], [3616.0, -978944.0], [978944.0, 0.0]]
    v = torch.zeros(len(rows), 64)
    for i, (hi, lo) in enumerate(rows):
        v[i, 3], v[i, 40] = hi, lo
        v[i, 7], v[i, 8] = hi * 0.37, lo * 0.61
    return v.to(dt).cuda()


def same(meta, codes, v, bits):
    code, s, z = ref.groups(v, bits)
    want, held = ref.words(s, z), ~torch.isnan(s.squeeze(-1))
    assert held.any() and bool((~held).any()) == bool((meta & 0x7FFF == 0x7E00).any())
    assert torch.equal(meta[held], want[held]) and torch.equal(codes, ref.pack(code, bits))
    assert torch.all(meta[~held] & 0x7FFF == 0x7E00)
    return bool((~held).any())


@pytest.mark.parametrize("bits,dtype", [(4, "f32"), (8, "f32"), (4, "bf16")])
def test_rows_of_the_largest_step(bits, dtype):
    from bit_error_compensated_gb300 import echo
    v = ranges(bits, dtype)
    n = len(v)
    cache = echo.Cache(2, 16, 1, 64, bits)
    table = torch.arange(2, dtype=torch.int32, device="cuda")[None]
    echo.echo_cache_append(cache, tensors([0, n], [n], table), v[:, None], v[:, None])
    rows = lambda t: t.permute(1, 0, 3, 2, *range(4, t.dim())).flatten(1, 3)[:, :n]      # noqa: E731
    for i in range(2):
        over = same(rows(cache.meta)[i], rows(cache.codes)[i], v, bits)
    assert echo.echo_serving_status() == (echo.ECHO_ERR_OVERFLOW if over else 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_weights_of_the_largest_step(dtype):
    from bit_error_compensated_gb300 import echo
    v = ranges(4, dtype)
    codes = torch.empty(len(v), 32, dtype=torch.uint8, device="cuda")
    meta = torch.empty(len(v), 1, dtype=torch.int32, device="cuda")
    echo.echo_quantize_weights(v, codes, meta, group=64)
    over = same(meta[:, 0], codes, v, 4)
    assert echo.echo_serving_status() == (echo.ECHO_ERR_OVERFLOW if over else 0)
