"""Products of 9 to 16 tokens by both ways, and fp32 numbers at the ends of what a
token's three parts hold."""
import math

import pytest
import torch

import _serve_ref as ref
from test_gpu_int4 import DTYPES, buffers, gen, quantised

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ranks,tokens,channels,depth", [(1, 9, 1024, 1024), (2, 16, 2048, 2048), (1, 16, 2049, 4095),
                                                         (1, 12, 4096, 4096), (1, 16, 8193, 4096)])
def test_products_on_both_sides_of_the_rule(dtype, ranks, tokens, channels, depth):
    """Products are exact.  fp32 sums: 16 terms in a matrix instruction, at most
    24 instructions in a window of 128, the windows of a row, and eight warps or
    blocks; then one rounding."""
    from bit_error_compensated_gb300 import echo
    g = gen(tokens + channels)
    dt = DTYPES[dtype]
    x = torch.randn(ranks, tokens, depth, generator=g, device="cuda").to(dt)
    w = torch.randn(ranks, channels, depth, generator=g, device="cuda") / math.sqrt(depth)
    codes, meta = buffers(ranks, channels, depth, 128)
    echo.echo_quantize_weights(w, codes, meta)
    out = torch.full((ranks, tokens, channels), 7, dtype=dt, device="cuda")
    echo.echo_linear_int4(x, codes, meta, out)
    code, s, z = quantised(w, 128)
    adds = 16 + 24 + math.ceil(depth / 128) + 8
    for p in range(ranks):
        want, size = ref.linear4(x[p], code[p], s[p], z[p], 128)
        tol = adds * 2.0 ** -23 * size
        tol = tol + ref.half_step(dt) * (want.abs() + tol) + torch.finfo(dt).smallest_normal * ref.half_step(dt)
        assert ((out[p].double() - want).abs() <= tol).all()


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
