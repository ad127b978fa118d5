"""fp32 numbers at the ends of what a token's three parts hold."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 8, 16, 40])
@pytest.mark.parametrize("bits32", [0x7F800001, 0x7F80FFFF, -0x7FFFFF, 0x7FC00000])
def test_every_nan_is_one_in_a_product(tokens, bits32):
    """All fp32 NaN, those among them whose payload lies in the bits that the first
    of a token's three parts does not have; the other tokens stay as they are."""
    from bit_error_compensated_gb300 import echo
    g = torch.Generator().manual_seed(tokens)
    w = (1 + torch.rand(48, 256, generator=g)).cuda()        # positive: an infinity would stay one
    x = torch.randn(tokens, 256, generator=g).cuda()
    codes = torch.empty(48, 128, dtype=torch.uint8, device="cuda")
    meta = torch.empty(48, 2, dtype=torch.int32, device="cuda")
    echo.echo_quantize_weights(w, codes, meta)
    clean, out = torch.empty(tokens, 48, device="cuda"), torch.empty(tokens, 48, device="cuda")
    echo.echo_linear_int4(x, codes, meta, clean)
    x.view(torch.int32)[tokens // 2, 77] = bits32
    assert torch.isnan(x).sum() == 1
    echo.echo_linear_int4(x, codes, meta, out)
    assert torch.isnan(out[tokens // 2]).all()
    keep = torch.arange(tokens, device="cuda") != tokens // 2
    assert torch.equal(out[keep], clean[keep])
