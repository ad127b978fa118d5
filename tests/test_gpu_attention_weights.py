"""What the attention's weights keep where one key's weight or step is far above
the others', against 64 bits and relative to the result itself."""
import math

import pytest
import torch

import _serve_ref as ref
from test_gpu_serving import DTYPES, gen, tensors

pytestmark = pytest.mark.gpu


def one_loud_key(bits, dim, keys, place, loud, lead, mean, seed):
    """A sequence whose keys are rows of zeros (scores of 0) but for the one at
    `place`, and a q row whose score with that one is `lead` powers of two.  Its
    value is a row of zeros, with a step of 1 by definition, or 0 but for one
    channel of 1000.  Other values are normal around `mean`."""
    from bit_error_compensated_gb300 import echo
    g = gen(seed)
    page = 64
    cache = echo.Cache(keys // page, page, 1, dim, bits)
    k, v = torch.zeros(keys, dim, device="cuda"), mean + torch.randn(keys, dim, generator=g, device="cuda")
    k[place, 0] = 1
    v[place] = 0
    if loud == "step":
        v[place, 5] = 1000
    for i, t in enumerate((k, v)):
        code, s, z = ref.groups(t, bits)
        cache.codes[:, i, 0] = ref.pack(code, bits).view(keys // page, page, -1)
        cache.meta[:, i, 0] = ref.words(s, z).view(keys // page, page)
    table = torch.arange(keys // page, dtype=torch.int32, device="cuda")[None]
    q = torch.zeros(dim, device="cuda")
    q[0] = lead * math.log(2)                                # (the scale is 1, the key's element 1 within a step)
    q[1:] = torch.randn(dim - 1, generator=g, device="cuda")
    return cache, table, q


def below(new):
    """The step of weights far below the largest, as a power of two of it."""
    return 34 if new <= 64 else 30


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("loud", ["zeros", "step"])
@pytest.mark.parametrize("lead", [18, 20, 22])
@pytest.mark.parametrize("place", [0, 20000])
@pytest.mark.parametrize("bits,dim,new", [(8, 128, 1), (4, 128, 1), (8, 64, 9), (8, 128, 90), (4, 64, 130), (8, 256, 70),
                                          (8, 256, 1)])
def test_one_loud_key_takes_no_bits_from_the_others(dtype, loud, lead, place, bits, dim, new):
    """32768 keys, one of them with a weight 2^lead above the others'.  Weights
    without their steps' powers of two are rounded to 11 bits, 2^-12 of each, or
    where they are 2^-24 of the largest or less by 2^-35 of it (2^-20 and 2^-31 where
    a sequence has more than 64 rows): 2^(lead - 35) of a quiet one's, its steps' part
    of 1 to 2 twice.  Values have a mean of 3 normal
    deviations and a row's weights are alike, so the mean of |v| is |out| within
    one part in 100 (in the loud key's own channel, a sum of two numbers of one
    sign, it is out).  Scores are a product each of one element, 8 2^-23 of them
    and 2^-20 (the exponential), on both sides of the quotient; sums of 32768
    add 2^-23 each, of one sign, 2^-8 at the very worst and 2^-12 for errors of
    either sign.  out is rounded by half a step."""
    keys = 32768
    cache, table, q0 = one_loud_key(bits, dim, keys, place, loud, lead, 3.0, lead + bits + dim)
    from bit_error_compensated_gb300 import echo
    starts, lengths = [0, new], [keys]
    q = q0.to(DTYPES[dtype]).expand(new, 1, dim).contiguous()
    out = torch.full_like(q, 7)
    echo.echo_attention(cache, tensors(starts, lengths, table), q, out, scale=1.0)
    exact, _, _ = ref.attention(cache, q, starts, lengths, table, 1.0)
    score = lead * math.log(2)
    limit = (2.0 ** -12 + 2.0 ** (lead - below(new)) + 2 * (8 * 2.0 ** -23 * score + 2.0 ** -20) + 2.0 ** -12) * 1.01 \
        + ref.half_step(q.dtype)
    off = (out.double() - exact).abs()
    assert (exact.abs() > 0).all()
    subnormal = torch.finfo(q.dtype).smallest_normal * ref.half_step(q.dtype)
    assert (off <= limit * exact.abs() + subnormal).all(), (off / exact.abs()).max().item()


@pytest.mark.parametrize("bits,dim,new", [(8, 128, 1), (4, 128, 5), (8, 64, 100), (8, 256, 100)])
@pytest.mark.parametrize("lead", [16, 20])
def test_a_row_of_zeros_under_a_dominant_key_leaves_the_row(bits, dim, new, lead):
    """The same with values around 0, whose weighted sum is far less than the mean
    of |v|: independent errors of 2^-12 and 2^(lead - 34) (or - 30) of each value's part are,
    together, that much of the row's length; four times that, and out's rounding."""
    keys = 32768
    cache, table, q0 = one_loud_key(bits, dim, keys, 0, "zeros", lead, 0.0, lead + dim)
    from bit_error_compensated_gb300 import echo
    starts, lengths = [0, new], [keys]
    q = q0.bfloat16().expand(new, 1, dim).contiguous()
    out = torch.full_like(q, 7)
    echo.echo_attention(cache, tensors(starts, lengths, table), q, out, scale=1.0)
    exact, _, _ = ref.attention(cache, q, starts, lengths, table, 1.0)
    off = (out.double() - exact).norm(dim=-1) / exact.norm(dim=-1)
    assert off.max().item() <= 4 * (2.0 ** -12 + 2.0 ** (lead - below(new))) + 2.0 ** -9


@pytest.mark.parametrize("lead", [17.1, 17.37, 17.6, 17.9])
@pytest.mark.parametrize("bits,dim,new", [(8, 128, 1), (4, 64, 5), (8, 128, 90), (4, 256, 90)])
def test_the_weight_of_a_dominant_key_is_exact(bits, dim, new, lead):
    """One key of 2048, the first, has all but 2^(11 - lead) of the row: its weight is
    a power of two, so that out is off by its own rounding, 2^-12 of what the others
    add, and fp32's errors (an error of its own weight is in both sums; scores of 12
    and the exponential are off by 2^-18, of the others' part; the sums' 2048
    additions of parts of 2^-17 by 2^-23 each)."""
    from bit_error_compensated_gb300 import echo
    keys, page = 2048, 64
    g = gen(int(10 * lead) + dim)
    cache, table, q = one_loud_key(bits, dim, keys, 0, "zeros", lead, 0.0, int(10 * lead) + dim)
    v = torch.randn(keys, dim, generator=g, device="cuda")
    code, s, z = ref.groups(v, bits)
    cache.codes[:, 1, 0] = ref.pack(code, bits).view(keys // page, page, -1)
    cache.meta[:, 1, 0] = ref.words(s, z).view(keys // page, page)
    q = q.half().expand(new, 1, dim).contiguous()
    out = torch.full_like(q, 7)
    echo.echo_attention(cache, tensors([0, new], [keys], table), q, out, scale=1.0, causal=False)
    exact, _, _ = ref.attention(cache, q, [0, new], [keys], table, 1.0, causal=False)
    size = (s * (code.double() - z)).abs().amax()
    limit = ref.half_step(q.dtype) * exact.abs() * (1 + 2.0 ** -9) + 2.0 ** -12 * 2.0 ** (11 - lead) * size + 2.0 ** -20 * size
    assert ((out.double() - exact).abs() <= limit).all()
