"""echo_quantize_tokens, echo_matmul_int8 and echo_linear_int8 against their
definitions: the quantizer's every step is one fp32 rounding and the product's
sum is exact, so all comparisons are bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def gen_of(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def want_quantized(x):
    """Codes and scales of [..., depth] by the definition, in fp32."""
    v = x.float()
    amax = torch.full_like(v[..., :1], 2.0 ** -110)
    if v.shape[-1]:
        amax = torch.maximum(v.abs().amax(-1, keepdim=True), amax)        # NaN stays NaN
    top = torch.full_like(amax, 127.0)       # a tensor: a scalar divisor becomes its reciprocal
    codes = torch.round(v * (top / amax))
    return torch.nan_to_num(codes, nan=0.0).to(torch.int8), (amax / top).squeeze(-1)


def want_product(a, sa, w, sw, dtype):
    """[ranks][tokens][channels]: an exact sum (64-bit floats hold it), then two
    fp32 products and the output's rounding."""
    total = torch.matmul(a.double(), w.double().transpose(-1, -2))
    return (total.float() * sa.unsqueeze(-1) * sw.unsqueeze(-2)).to(dtype)


def same_bits(got, want):
    kind = {2: torch.int16, 4: torch.int32, 1: torch.int8}[got.element_size()]
    nan = want.isnan() if want.is_floating_point() else torch.zeros_like(want, dtype=torch.bool)
    assert torch.equal(got.isnan() if got.is_floating_point() else nan, nan)
    assert torch.equal(got.contiguous().view(kind)[~nan], want.contiguous().view(kind)[~nan])


def codes_of(gen, *shape, low=-128, high=128):
    return torch.randint(low, high, shape, generator=gen, device="cuda", dtype=torch.int32).to(torch.int8)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 5, 7), (3, 17, 256), (1, 4, 4096), (2, 3, 9999),
                                   (1, 2, 40000), (4, 33, 1024)])
def test_quantize(dtype, shape):
    from bit_error_compensated_gb300 import echo
    x = (torch.randn(shape, generator=gen_of(sum(shape)), device="cuda") * 3).to(dtype)
    codes, scales = torch.empty(shape, dtype=torch.int8, device="cuda"), torch.empty(shape[:-1], device="cuda")
    echo.echo_quantize_tokens(x, codes, scales)
    want, want_scales = want_quantized(x)
    same_bits(codes, want)
    same_bits(scales, want_scales)


def test_quantize_strided_slices_and_odd_rows():
    """The ranks' slices of one row; zero rows, infinities, NaN, the smallest values."""
    from bit_error_compensated_gb300 import echo
    P, M, K = 4, 37, 200
    for offset, dtype in ((0, F32), (1, BF16), (8, F16)):
        base = torch.randn(M * P * K + offset, generator=gen_of(offset), device="cuda").to(dtype)
        x = base[offset:].view(M, P, K).transpose(0, 1)
        x[0, 3] = 0
        x[1, 4, 7], x[2, 5, 0], x[3, 6, K - 1] = float("inf"), float("nan"), -float("inf")
        x[0, 7] = 1e-7
        if dtype == F32:
            x[0, 8], x[0, 9, 1:], x[0, 9, 0] = 1e-44, 0, 2.0 ** -111
        codes = torch.empty(M, P, K, dtype=torch.int8, device="cuda").transpose(0, 1)
        scales = torch.empty(P, M, device="cuda")
        echo.echo_quantize_tokens(x, codes, scales)
        want, want_scales = want_quantized(x)
        same_bits(codes, want)
        same_bits(scales, want_scales)
        assert (codes[0, 3] == 0).all() and (codes[1, 4] == 0).all() and scales[1, 4].isinf()
        assert (codes[2, 5] == 0).all() and scales[2, 5].isnan()


SHAPES = [
    # ranks, tokens, channels, depth
    (1, 1, 1, 1), (1, 1, 4096, 4096), (1, 2, 130, 64), (1, 3, 1000, 4096), (1, 4, 257, 515),
    (1, 7, 512, 1024), (1, 8, 4096, 2048), (1, 13, 333, 4097), (1, 16, 6144, 512), (1, 17, 64, 16),
    (1, 31, 999, 1111), (1, 32, 1024, 1024), (1, 33, 300, 2064), (1, 64, 512, 4096), (1, 65, 129, 96),
    (1, 100, 1111, 2051), (1, 128, 256, 1024), (1, 129, 257, 1025), (1, 200, 4096, 1040), (1, 256, 512, 8192),
    (1, 300, 1000, 48), (1, 513, 770, 2050), (1, 1000, 2000, 1500), (1, 1024, 4096, 1024),
    (2, 1, 512, 512), (4, 5, 264, 384), (8, 16, 128, 1024), (4, 129, 500, 1024), (16, 40, 72, 80),
    (3, 700, 515, 333), (1, 5, 70000, 64), (1, 3000, 40, 64),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_product(shape, dtype):
    from bit_error_compensated_gb300 import echo
    P, M, N, K = shape
    gen = gen_of(M * 7 + N + K)
    a, w = codes_of(gen, P, M, K), codes_of(gen, P, N, K)
    sa, sw = torch.rand(P, M, generator=gen, device="cuda"), torch.rand(P, N, generator=gen, device="cuda") * 1e-3
    out = torch.full((P, M, N), float("nan"), dtype=dtype, device="cuda")
    echo.echo_matmul_int8(a, sa, w, sw, out)
    same_bits(out, want_product(a, sa, w, sw, dtype))


@pytest.mark.parametrize("tokens", [1, 9, 40, 300])
@pytest.mark.parametrize("depth", [1023, 1024, 1025, 8192, 131071])
@pytest.mark.parametrize("a_value,w_value", [(-128, -128), (127, -128), (127, 127)])
def test_sums_are_exact_at_the_largest_magnitudes(tokens, depth, a_value, w_value):
    """All codes at an end of their range: the sum reaches 2^31 - 2^14, far past
    the 24 bits of an fp32 significand; some are turned, so that sums differ."""
    from bit_error_compensated_gb300 import echo
    N = 96
    gen = gen_of(depth)
    a = torch.full((1, tokens, depth), a_value, dtype=torch.int8, device="cuda")
    w = torch.full((1, N, depth), w_value, dtype=torch.int8, device="cuda")
    flip = torch.rand(w.shape, generator=gen, device="cuda") < 0.001
    w[flip] = 1
    one, ones = torch.ones(1, tokens, device="cuda"), torch.ones(1, N, device="cuda")
    out = torch.empty(1, tokens, N, device="cuda")
    echo.echo_matmul_int8(a, one, w, ones, out)
    same_bits(out, want_product(a, one, w, ones, F32))
    # 24 low bits of the sum: exact differences of two exact sums
    total = torch.matmul(a.double(), w.double().transpose(-1, -2))
    assert total.abs().max() <= 2 ** 31


def test_a_token_does_not_depend_on_the_others():
    """The same token in calls of every size gives the same bits."""
    from bit_error_compensated_gb300 import echo
    N, K = 520, 2176
    gen = gen_of(5)
    a, w = codes_of(gen, 700, K), codes_of(gen, N, K)
    sa, sw = torch.rand(700, generator=gen, device="cuda"), torch.rand(N, generator=gen, device="cuda")
    whole = torch.empty(700, N, dtype=F32, device="cuda")
    echo.echo_matmul_int8(a, sa, w, sw, whole)
    for m in (1, 2, 5, 8, 9, 16, 24, 33, 64, 100, 128, 130, 257, 512):
        out = torch.empty(m, N, dtype=F32, device="cuda")
        echo.echo_matmul_int8(a[:m], sa[:m].contiguous(), w, sw, out)
        assert torch.equal(out, whole[:m]), m


@pytest.mark.parametrize("tokens", [1, 6, 20, 150, 600])
@pytest.mark.parametrize("pad,offset", [(0, 0), (16, 0), (3, 0), (0, 5), (16, 16), (5, 3)])
def test_strides_and_alignment(tokens, pad, offset):
    """Rows of wider tensors, off 16-byte boundaries, and an output in a wider one."""
    from bit_error_compensated_gb300 import echo
    P, N, K = 2, 136, 272
    gen = gen_of(tokens + pad)

    def padded(rows, cols, make):
        ld = cols + pad
        flat = make(P * rows * ld + offset)
        return flat[offset:].view(P, rows, ld)[:, :, :cols]

    a = padded(tokens, K, lambda n: codes_of(gen, n))
    w = padded(N, K, lambda n: codes_of(gen, n))
    sa, sw = torch.rand(P, tokens, generator=gen, device="cuda"), torch.rand(P, N, generator=gen, device="cuda")
    flat = torch.full((P * tokens * (N + pad) + offset,), 7.0, dtype=BF16, device="cuda")
    out = flat[offset:].view(P, tokens, N + pad)[:, :, :N]
    echo.echo_matmul_int8(a, sa, w, sw, out)
    same_bits(out, want_product(a, sa, w, sw, BF16))
    rest = flat[offset:].view(P, tokens, N + pad)[:, :, N:]
    assert (flat[:offset] == 7).all() and (rest == 7).all()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("tokens,channels,depth", [(33, 513, 1024), (257, 259, 17), (300, 516, 640), (511, 1022, 96),
                                                   (290, 130, 1025), (700, 65, 2000)])
@pytest.mark.parametrize("pad,offset", [(0, 0), (1, 1), (2, 2), (5, 4), (8, 0)])
def test_results_in_rows_of_any_place(dtype, tokens, channels, depth, pad, offset):
    """Rows of results that start on any element, and nothing written beside them."""
    from bit_error_compensated_gb300 import echo
    gen, ld = gen_of(tokens + channels), channels + pad
    a, w = codes_of(gen, 2, tokens, depth), codes_of(gen, 2, channels, depth)
    sa = torch.rand(2, tokens, generator=gen, device="cuda") * 0.01
    sw = torch.rand(2, channels, generator=gen, device="cuda") * 0.01
    base = torch.full((offset + 2 * tokens * ld + 64,), 7.0, dtype=dtype, device="cuda")
    rows = base[offset:offset + 2 * tokens * ld].view(2, tokens, ld)
    echo.echo_matmul_int8(a, sa, w, sw, rows[..., :channels])
    same_bits(rows[..., :channels].clone(), want_product(a, sa, w, sw, dtype))
    rows[..., :channels] = 7.0
    assert bool((base == 7.0).all())


@pytest.mark.parametrize("tokens", [3, 50, 300])
def test_operands_shared_by_the_ranks(tokens):
    from bit_error_compensated_gb300 import echo
    P, N, K = 4, 160, 256
    gen = gen_of(tokens)
    a, w = codes_of(gen, tokens, K), codes_of(gen, P, N, K)
    sa, sw = torch.rand(tokens, generator=gen, device="cuda"), torch.rand(N, generator=gen, device="cuda")
    out = torch.empty(P, tokens, N, dtype=F16, device="cuda")
    echo.echo_matmul_int8(a, sa, w, sw, out)
    same_bits(out, want_product(a.expand(P, tokens, K), sa.expand(P, tokens), w, sw.expand(P, N), F16))
    echo.echo_matmul_int8(a.expand(P, tokens, K), sa.repeat(P, 1), w[0], sw, out)
    same_bits(out, want_product(a.expand(P, tokens, K), sa.expand(P, tokens), w[0].expand(P, N, K), sw.expand(P, N), F16))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("shape", [(1, 1, 4096, 4096), (4, 3, 136, 1024), (1, 8, 999, 2051), (2, 40, 512, 640),
                                   (1, 203, 1111, 2051), (4, 260, 512, 1024)])
def test_linear_is_the_two_calls(shape, dtype):
    from bit_error_compensated_gb300 import echo
    P, M, N, K = shape
    gen = gen_of(N)
    x = torch.randn(M, P, K, generator=gen, device="cuda").to(dtype).transpose(0, 1)
    x[0, M // 2, 3] = float("nan")
    w, sw = codes_of(gen, P, N, K), torch.rand(P, N, generator=gen, device="cuda") * 1e-2
    codes, scales = torch.empty(P, M, K, dtype=torch.int8, device="cuda"), torch.empty(P, M, device="cuda")
    out = torch.empty(P, M, N, dtype=dtype, device="cuda")
    echo.echo_linear_int8(x, w, sw, out, codes, scales)
    want_codes, want_scales = want_quantized(x)
    same_bits(codes, want_codes)
    same_bits(scales, want_scales)
    same_bits(out, want_product(want_codes, want_scales, w, sw, dtype))
    assert out[0, M // 2].isnan().all() and int(out.isnan().sum()) == N


def test_empty_sizes():
    from bit_error_compensated_gb300 import echo
    i8 = dict(dtype=torch.int8, device="cuda")
    for M, N, K in ((0, 64, 64), (5, 0, 64), (5, 64, 0)):
        out = torch.full((M, N), 3.0, device="cuda")
        echo.echo_matmul_int8(torch.ones(M, K, **i8), torch.ones(M, device="cuda"), torch.ones(N, K, **i8),
                              torch.ones(N, device="cuda"), out)
        assert (out == 0).all()                                         # a sum over nothing
        x = torch.ones(M, K, device="cuda")
        codes, scales = torch.empty(M, K, **i8), torch.empty(M, device="cuda")
        echo.echo_linear_int8(x, torch.ones(N, K, **i8), torch.ones(N, device="cuda"), out, codes, scales)
        assert (out == 0).all() if K == 0 else True


def test_offsets_past_32_bits():
    """Token, channel and output rows that start beyond 2^31 bytes and elements."""
    from bit_error_compensated_gb300 import echo
    for M, N, K in ((6, 40, 128), (70, 200, 128), (300, 300, 1040)):
        gen = gen_of(M)
        a, w = codes_of(gen, M, K), codes_of(gen, N, K)
        sa, sw = torch.rand(M, generator=gen, device="cuda"), torch.rand(N, generator=gen, device="cuda")
        far = lambda rows, cols, dt: torch.empty(                                  # noqa: E731
            ((1 << 31) // (rows - 1) // 16 + 8) * 16 * rows, dtype=dt, device="cuda").view(rows, -1)[:, :cols]
        a2, w2, out = far(M, K, torch.int8), far(N, K, torch.int8), far(M, N, BF16)
        a2.copy_(a)
        w2.copy_(w)
        echo.echo_matmul_int8(a2, sa, w2, sw, out)
        same_bits(out, want_product(a, sa, w, sw, BF16))


def test_another_stream_and_a_graph():
    from bit_error_compensated_gb300 import echo
    for M in (1, 20, 300):
        gen = gen_of(M)
        x = torch.randn(M, 1024, generator=gen, device="cuda").to(BF16)
        w, sw = codes_of(gen, 512, 1024), torch.rand(512, generator=gen, device="cuda")
        bufs = [torch.empty(M, 512, dtype=BF16, device="cuda"), torch.empty(M, 1024, dtype=torch.int8, device="cuda"),
                torch.empty(M, device="cuda")]
        echo.echo_linear_int8(x, w, sw, *bufs)
        want = bufs[0].clone()
        bufs[0].zero_()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        echo.echo_linear_int8(x, w, sw, *bufs, stream=side)
        side.synchronize()
        assert torch.equal(bufs[0], want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            echo.echo_linear_int8(x, w, sw, *bufs)
        bufs[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bufs[0], want)


def test_refusals():
    from bit_error_compensated_gb300 import echo
    M, N, K = 8, 64, 128
    i8 = dict(dtype=torch.int8, device="cuda")
    a, w, sa, sw = torch.zeros(M, K, **i8), torch.zeros(N, K, **i8), torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    out = torch.zeros(M, N, device="cuda")
    x = torch.zeros(M, K, device="cuda")

    def status(want, call, *args):
        with pytest.raises(echo.EchoError) as e:
            call(*args)
        assert e.value.status == want

    bytes_ = torch.zeros(M * N * 4 + 64, **i8)
    over = bytes_[:M * N * 4].view(torch.float32).view(M, N)
    status(echo.ECHO_ERR_ARG, echo.echo_matmul_int8, bytes_[:M * K].view(M, K), sa, w, sw, over)
    status(echo.ECHO_ERR_ARG, echo.echo_matmul_int8, a, out[0, :M], w, sw, out)
    status(echo.ECHO_ERR_SHAPE, echo.echo_matmul_int8, a.as_strided((M, K), (K - 1, 1)), sa, w, sw, out)
    ranks = torch.zeros(17, M, K, **i8)
    status(echo.ECHO_ERR_ARG, echo.echo_matmul_int8, ranks, torch.ones(17, M, device="cuda"), w, sw,
           torch.zeros(17, M, N, device="cuda"))
    status(echo.ECHO_ERR_SHAPE, echo.echo_matmul_int8, a, sa, w, sw, out.expand(3, M, N))
    deep = 131072
    status(echo.ECHO_ERR_UNSUPPORTED, echo.echo_matmul_int8, torch.zeros(1, deep, **i8), sa[:1], torch.zeros(2, deep, **i8),
           sw[:2].contiguous(), torch.zeros(1, 2, device="cuda"))
    odd = torch.zeros(M * K * 4 + 4, **i8)[1:1 + M * K * 4].view(M, 4 * K)
    assert odd.data_ptr() % 4
    status(echo.ECHO_ERR_ARG, echo.echo_quantize_tokens, x, x.view(torch.int8)[:, :K], sa)     # codes over x
    for word, call, args in (
            ("dtype", echo.echo_matmul_int8, (a.float(), sa, w, sw, out)),
            ("dtype", echo.echo_matmul_int8, (a, sa.double(), w, sw, out)),
            ("dtype", echo.echo_matmul_int8, (a, sa, w, sw, out.double())),
            ("shape", echo.echo_matmul_int8, (a[:, :64], sa, w, sw, out)),
            ("shape", echo.echo_matmul_int8, (a, sa[:4], w, sw, out)),
            ("shape", echo.echo_matmul_int8, (a, sa, w, sw[:4], out)),
            ("contiguous", echo.echo_matmul_int8, (a, sa, w, sw, torch.zeros(M, 2 * N, device="cuda")[:, ::2])),
            ("CUDA device", echo.echo_matmul_int8, (a.cpu(), sa, w, sw, out)),
            ("dtype", echo.echo_linear_int8, (x.bfloat16(), w, sw, out, a, sa)),
            ("shape", echo.echo_linear_int8, (x, w, sw, out, a[:4], sa))):
        with pytest.raises(ValueError, match=word):
            call(*args)


@pytest.mark.parametrize("shape", [(300, 5000, 1024), (300, 5000, 2048), (256, 512, 2048)])
def test_a_wait_that_runs_out_ends_the_call(shape):
    """One block never reports its work (the hold hook): every wait on it gives
    up after its second, the call ends, the status says so, and the next call
    is exact again.  Shapes of each form: one chunk, several, a shared tile."""
    from bit_error_compensated_gb300 import echo
    M, N, K = shape
    gen = gen_of(M)
    a, w = codes_of(gen, M, K), codes_of(gen, N, K)
    sa, sw = torch.rand(M, generator=gen, device="cuda"), torch.rand(N, generator=gen, device="cuda")
    out = torch.empty(M, N, device="cuda")
    assert echo.echo_matmul_status() == echo.ECHO_OK
    echo.echo_debug_hold_product(True)
    try:
        echo.echo_matmul_int8(a, sa, w, sw, out)
        assert echo.echo_matmul_status() == echo.ECHO_ERR_TIMEOUT
    finally:
        echo.echo_debug_hold_product(False)
    assert echo.echo_matmul_status() == echo.ECHO_OK
    echo.echo_matmul_int8(a, sa, w, sw, out)
    same_bits(out, want_product(a, sa, w, sw, F32))
    assert echo.echo_matmul_status() == echo.ECHO_OK


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("shape", [(600, 20000, 1024), (600, 20000, 1100), (129, 1024, 2048)])
def test_a_call_that_gave_up_ends_cleanly(shape, dtype):
    """The same with several tiles a pair (or a tile shared by pairs), each type
    of results: every issuing warp waits for what it has in flight, and the call
    after it is exact in every tile."""
    from bit_error_compensated_gb300 import echo
    M, N, K = shape
    gen = gen_of(N)
    a, w = codes_of(gen, M, K), codes_of(gen, N, K)
    sa, sw = torch.rand(M, generator=gen, device="cuda"), torch.rand(N, generator=gen, device="cuda")
    out = torch.empty(M, N, dtype=dtype, device="cuda")
    echo.echo_matmul_status()
    echo.echo_debug_hold_product(True)
    try:
        echo.echo_matmul_int8(a, sa, w, sw, out)
        assert echo.echo_matmul_status() == echo.ECHO_ERR_TIMEOUT
    finally:
        echo.echo_debug_hold_product(False)
    echo.echo_matmul_int8(a, sa, w, sw, out)
    same_bits(out, want_product(a, sa, w, sw, dtype))
    assert echo.echo_matmul_status() == echo.ECHO_OK


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("shape", [(1, 1500, 7000, 1024), (1, 1500, 7000, 2048), (1, 1500, 7001, 1100), (2, 1030, 5136, 640),
                                   (1, 2600, 5000, 3000), (1, 9000, 600, 512), (3, 700, 5003, 1300), (1, 1025, 6144, 4096)],
                         ids=lambda s: "x".join(map(str, s)))
def test_product_of_several_tiles_a_pair(shape, dtype):
    """More tiles than pairs of SMs: a pair goes on to a second and third one,
    in one chunk and in several."""
    from bit_error_compensated_gb300 import echo
    P, M, N, K = shape
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    assert P * ((M + 255) // 256) * ((N + 255) // 256) > pairs
    gen = gen_of(M + N + K)
    a, w = codes_of(gen, P, M, K), codes_of(gen, P, N, K)
    sa, sw = torch.rand(P, M, generator=gen, device="cuda"), torch.rand(P, N, generator=gen, device="cuda") * 1e-3
    out = torch.full((P, M, N), float("nan"), dtype=dtype, device="cuda")
    want = want_product(a, sa, w, sw, dtype)
    for _ in range(3):
        echo.echo_matmul_int8(a, sa, w, sw, out)
        same_bits(out, want)
        out.fill_(float("nan"))
    assert echo.echo_matmul_status() == echo.ECHO_OK


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("shape", [(1, 8, 6144, 4096), (1, 5, 7000, 2051), (4, 3, 2000, 1024), (1, 1, 9000, 515),
                                   (1, 8, 14336, 1040), (1, 1, 4096, 8192)], ids=lambda s: "x".join(map(str, s)))
def test_product_of_few_tokens_and_many_channels(shape, dtype):
    """Up to 8 tokens with more blocks of 16 channels than two an SM, and depths
    of several turns of a block's warps."""
    from bit_error_compensated_gb300 import echo
    P, M, N, K = shape
    gen = gen_of(M + N + K)
    a, w = codes_of(gen, P, M, K), codes_of(gen, P, N, K)
    sa, sw = torch.rand(P, M, generator=gen, device="cuda"), torch.rand(P, N, generator=gen, device="cuda") * 1e-3
    out = torch.full((P, M, N), float("nan"), dtype=dtype, device="cuda")
    echo.echo_matmul_int8(a, sa, w, sw, out)
    same_bits(out, want_product(a, sa, w, sw, dtype))


@pytest.mark.parametrize("tokens", [1, 12, 30, 100, 700])
@pytest.mark.parametrize("P,N,K", [(4, 520, 1024), (2, 300, 1040), (4, 260, 1000), (3, 4100, 512), (2, 300, 333)])
def test_weights_that_are_slices_of_one_matrix(tokens, P, N, K):
    """A row-parallel layer's weights as the ranks' columns of one matrix: rows
    lie farther apart than ranks, on 16 bytes or on any."""
    from bit_error_compensated_gb300 import echo
    gen = gen_of(tokens + N)
    w = codes_of(gen, N, P * K).view(N, P, K).transpose(0, 1)
    a = codes_of(gen, tokens, P * K).view(tokens, P, K).transpose(0, 1)
    sa, sw = torch.rand(P, tokens, generator=gen, device="cuda"), torch.rand(P, N, generator=gen, device="cuda")
    out = torch.full((tokens, P, N), float("nan"), dtype=BF16, device="cuda").transpose(0, 1)
    echo.echo_matmul_int8(a, sa, w, sw, out)
    same_bits(out, want_product(a, sa, w, sw, BF16))
