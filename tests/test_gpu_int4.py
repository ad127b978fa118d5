"""4-bit weights: their quantizer, bit by bit, and products of few tokens with
them, against 64 bits."""
import math

import pytest
import torch

import _serve_ref as ref

pytestmark = pytest.mark.gpu
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def quantised(w, group):
    """Codes [..., depth], and steps and zero points a group, in 64 bits."""
    depth = w.shape[-1]
    padded = torch.nn.functional.pad(w.double(), (0, -depth % group)).unflatten(-1, (-1, group))
    code, s, z = ref.groups(padded, 4)
    return code.flatten(-2)[..., :depth], s.squeeze(-1), z.squeeze(-1)


def buffers(ranks, channels, depth, group):
    return (torch.full((ranks, channels, (depth + 1) // 2), 255, dtype=torch.uint8, device="cuda"),
            torch.full((ranks, channels, (depth + group - 1) // group), -1, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("group", [64, 128, 256])
@pytest.mark.parametrize("ranks,channels,depth", [(1, 1, 1), (2, 33, 255), (1, 17, 2051), (3, 8, 1024), (1, 5, 130)])
def test_weights_are_quantised_exactly(dtype, group, ranks, channels, depth):
    from bit_error_compensated_gb300 import echo
    w = torch.randn(ranks, channels, depth, generator=gen(depth), device="cuda").to(DTYPES[dtype])
    codes, meta = buffers(ranks, channels, depth, group)
    echo.echo_quantize_weights(w, codes, meta, group=group)
    code, s, z = quantised(w, group)
    assert torch.equal(codes, ref.pack(code, 4))
    assert torch.equal(meta, ref.words(s[..., None], z[..., None]))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("group", [64, 128, 256])
@pytest.mark.parametrize("ranks,channels,depth", [(1, 10000, 72), (2, 2500, 1027), (1, 1250, 4096), (1, 1100, 4616)])
def test_many_weights_are_quantised_exactly(dtype, group, ranks, channels, depth):
    """As above, with so many that a warp has several steps of a row's, the last of
    them in part or not at all, and groups that cannot be held among them."""
    from bit_error_compensated_gb300 import echo
    echo.echo_serving_status()
    w = torch.randn(ranks, channels, depth, generator=gen(depth), device="cuda").to(DTYPES[dtype])
    code, s, z = quantised(w, group)
    bad = [(0, 5, 3, float("nan")), (ranks - 1, channels - 1, depth - 1, float("inf")), (0, channels // 2, depth // 2, float("-inf"))]
    for p, c, k, x in bad:
        w[p, c, k] = x
    codes, meta = buffers(ranks, channels, depth, group)
    echo.echo_quantize_weights(w, codes, meta, group=group)
    assert echo.echo_serving_status() == echo.ECHO_ERR_OVERFLOW
    want_codes, want_meta = ref.pack(code, 4), ref.words(s[..., None], z[..., None])
    for p, c, k, _ in bad:
        at = k // group
        assert int(meta[p, c, at]) & 0x7FFF == 0x7E00
        want_meta[p, c, at] = meta[p, c, at]
        of = slice(at * group // 2, (at + 1) * group // 2)
        assert not codes[p, c, of].any()                     # a group without a step has codes of 0
        want_codes[p, c, of] = 0
    assert torch.equal(codes, want_codes) and torch.equal(meta, want_meta)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("group", [64, 128, 256])
@pytest.mark.parametrize("ranks,tokens,channels,depth", [
    (1, 1, 1, 1), (1, 1, 16, 128), (2, 3, 33, 257), (1, 8, 100, 1000), (1, 9, 64, 512), (4, 16, 48, 384),
    (1, 17, 40, 2051), (1, 32, 96, 4096), (2, 33, 31, 640), (1, 70, 65, 320), (1, 5, 130, 8192)])
def test_product(dtype, group, ranks, tokens, channels, depth):
    """Products are exact.  fp32 sums: 16 terms in a matrix instruction, at most
    8 instructions for each of at most three parts of x in a window, the windows
    of one of eight warps, and the eight warps; then one rounding."""
    from bit_error_compensated_gb300 import echo
    g = gen(tokens * depth + group)
    dt = DTYPES[dtype]
    x = torch.randn(ranks, tokens, depth, generator=g, device="cuda").to(dt)
    w = torch.randn(ranks, channels, depth, generator=g, device="cuda") / math.sqrt(depth)
    codes, meta = buffers(ranks, channels, depth, group)
    echo.echo_quantize_weights(w, codes, meta, group=group)
    out = torch.full((ranks, tokens, channels), 7, dtype=dt, device="cuda")
    echo.echo_linear_int4(x, codes, meta, out, group=group)
    code, s, z = quantised(w, group)
    adds = 16 + 24 + math.ceil(depth / 64 / 8) + 9
    for p in range(ranks):
        want, size = ref.linear4(x[p], code[p], s[p], z[p], group)
        tol = adds * 2.0 ** -23 * size
        tol = tol + ref.half_step(dt) * (want.abs() + tol) + torch.finfo(dt).smallest_normal * ref.half_step(dt)
        assert ((out[p].double() - want).abs() <= tol).all()


def test_tokens_do_not_depend_on_the_batch():
    """A token's sums take the same order for the same form of the kernel."""
    from bit_error_compensated_gb300 import echo
    g = gen(3)
    x = torch.randn(8, 1000, generator=g, device="cuda").bfloat16()
    w = torch.randn(77, 1000, generator=g, device="cuda")
    codes, meta = (t[0] for t in buffers(1, 77, 1000, 128))
    echo.echo_quantize_weights(w, codes, meta)
    all8, one = torch.empty(8, 77, dtype=torch.bfloat16, device="cuda"), torch.empty(1, 77, dtype=torch.bfloat16, device="cuda")
    echo.echo_linear_int4(x, codes, meta, all8)
    for t in range(8):
        echo.echo_linear_int4(x[t:t + 1], codes, meta, one)
        assert torch.equal(one[0], all8[t])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tokens", [2, 12, 20])
def test_strides_shared_operands_and_unaligned_rows(dtype, tokens):
    from bit_error_compensated_gb300 import echo
    g = gen(tokens)
    dt = DTYPES[dtype]
    ranks, channels, depth = 3, 37, 389
    rows = torch.randn(tokens, ranks * depth, generator=g, device="cuda").to(dt)
    x = rows.view(tokens, ranks, depth).transpose(0, 1)      # slices of one row a token, side by side
    w = torch.randn(ranks, channels, depth, generator=g, device="cuda")
    codes, meta = buffers(ranks, channels, depth, 64)
    echo.echo_quantize_weights(w, codes, meta, group=64)
    want = torch.empty(ranks, tokens, channels, dtype=dt, device="cuda")
    echo.echo_linear_int4(x.contiguous(), codes, meta, want, group=64)
    out = torch.zeros(ranks, tokens, channels + 3, dtype=dt, device="cuda")
    echo.echo_linear_int4(x, codes, meta, out[..., 1:1 + channels], group=64)
    assert torch.equal(out[..., 1:1 + channels], want)
    assert torch.all(out[..., 0] == 0) and torch.all(out[..., 1 + channels:] == 0)
    odd = torch.zeros(ranks * channels * 199 + 1, dtype=torch.uint8, device="cuda")[1:].view(ranks, channels, 199)[..., :195]
    words = torch.zeros(ranks, channels, 9, dtype=torch.int32, device="cuda")[..., 2:]
    echo.echo_quantize_weights(w, odd, words, group=64)
    assert torch.equal(odd, codes) and torch.equal(words, meta)
    got = torch.empty_like(want)
    echo.echo_linear_int4(x, odd, words, got, group=64)
    assert torch.equal(got, want)
    # all ranks share the tokens, or the weights
    echo.echo_linear_int4(x[0].contiguous(), codes, meta, got, group=64)
    for p in range(ranks):
        echo.echo_linear_int4(x[0].contiguous(), codes[p], meta[p], want[p], group=64)
    assert torch.equal(got, want)
    echo.echo_linear_int4(x, codes[1], meta[1], got, group=64)
    for p in range(ranks):
        echo.echo_linear_int4(x[p], codes[1], meta[1], want[p], group=64)
    assert torch.equal(got, want)


def test_groups_that_cannot_be_held_and_non_finite_tokens():
    from bit_error_compensated_gb300 import echo
    w = torch.randn(4, 300, device="cuda")
    w[1, 200], w[2, 299], w[3, 0] = math.nan, math.inf, 1e10
    codes, meta = (t[0] for t in buffers(1, 4, 300, 128))
    echo.echo_serving_status()
    echo.echo_quantize_weights(w, codes, meta)
    assert echo.echo_serving_status() == echo.ECHO_ERR_OVERFLOW
    for dt in DTYPES.values():
        x = torch.randn(2, 300, device="cuda").to(dt)
        out = torch.empty(2, 4, dtype=dt, device="cuda")
        echo.echo_linear_int4(x, codes, meta, out)
        assert torch.equal(torch.isnan(out), torch.tensor([[False, True, True, True]] * 2, device="cuda"))
        x[1, 5] = math.inf
        echo.echo_linear_int4(x, codes, meta, out)
        assert torch.isfinite(out[0, 0]) and not torch.isfinite(out[1, 0])


def test_no_depth_and_no_tokens():
    from bit_error_compensated_gb300 import echo
    codes, meta = (t[0] for t in buffers(1, 6, 0, 128))
    echo.echo_quantize_weights(torch.empty(6, 0, device="cuda"), codes, meta)
    out = torch.full((3, 6), 7.0, device="cuda")
    echo.echo_linear_int4(torch.empty(3, 0, device="cuda"), codes, meta, out)
    assert torch.all(out == 0)
    codes, meta = (t[0] for t in buffers(1, 6, 64, 64))
    codes.zero_(), meta.zero_()
    echo.echo_linear_int4(torch.empty(0, 64, device="cuda"), codes, meta, torch.empty(0, 6, device="cuda"), group=64)


def test_more_tokens_than_one_launch_takes():
    from bit_error_compensated_gb300 import echo
    g = gen(9)
    tokens = 65535 * 8 + 5
    x = torch.randn(tokens, 64, generator=g, device="cuda")
    w = torch.randn(3, 64, generator=g, device="cuda")
    codes, meta = (t[0] for t in buffers(1, 3, 64, 64))
    echo.echo_quantize_weights(w, codes, meta, group=64)
    out = torch.full((tokens, 3), 7.0, device="cuda")
    echo.echo_linear_int4(x, codes, meta, out, group=64)
    code, s, z = quantised(w, 64)
    want, size = ref.linear4(x, code, s, z, 64)
    assert ((out.double() - want).abs() <= 64 * 2.0 ** -23 * size).all()
