"""The quantised cache and attention over its pages, against 64 bits."""
import math

import pytest
import torch

import _serve_ref as ref

pytestmark = pytest.mark.gpu
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def clean_status():
    from bit_error_compensated_gb300 import echo
    echo.echo_serving_status()
    yield
    torch.cuda.synchronize()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def make_batch(counts, lengths, page, g, spare=2, extra_cols=1):
    """starts, lengths, and a table of pages in random order; the pool has `spare` more."""
    each = [(n + page - 1) // page for n in lengths]
    pages = sum(each) + spare
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.zeros(len(lengths), max(each + [0]) + extra_cols, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(each):
        table[b, :n] = order[at:at + n]
        at += n
    starts = [0]
    for c in counts:
        starts.append(starts[-1] + c)
    return starts, table, pages


def tensors(starts, lengths, table):
    from bit_error_compensated_gb300 import echo
    to = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")             # noqa: E731
    return echo.CacheBatch(to(starts), to(lengths), table)


def values(g, *shape, dtype=torch.float32):
    v = torch.randn(*shape, generator=g, device="cuda")
    loud = torch.rand(shape[-1], generator=g, device="cuda") < 0.03
    return (v * torch.where(loud, 8.0, 1.0)).to(dtype)


def full_cache(g, pages, page, heads, dim, bits, spoil=True):
    """A cache whose every place holds quantised values, or (where `spoil`) for
    places that no test looks at, garbage: pages are filled before they are used."""
    from bit_error_compensated_gb300 import echo
    cache = echo.Cache(pages, page, heads, dim, bits)
    code, s, z = ref.groups(values(g, pages, 2, heads, page, dim), bits)
    cache.codes.copy_(ref.pack(code, bits))
    cache.meta.copy_(ref.words(s, z))
    return cache


def spoil_behind(cache, lengths, table):
    """NaN steps and zero points behind each sequence's last token, in its last page."""
    for b, n in enumerate(lengths):
        if n % cache.page_size:
            page = int(table[b, n // cache.page_size])
            cache.meta[page, :, :, n % cache.page_size:] = 0x7E007E00
            cache.codes[page, :, :, n % cache.page_size:] = 255


# ------------------------------------------------------------------- cache
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dim,heads,page", [(64, 5, 16), (128, 1, 64), (128, 8, 256), (256, 3, 32)])
def test_rows_are_quantised_exactly_and_read_back(dtype, bits, dim, heads, page):
    """Codes, steps and zero points are whole numbers and fp16 numbers of an
    exact definition, so all bits are equal; a value read back is one exact
    product, rounded once."""
    from bit_error_compensated_gb300 import echo
    g = gen(dim + bits)
    dt = DTYPES[dtype]
    counts, lengths = [3, 1, 0, 40], [3, 18, 7, 100]
    starts, table, pages = make_batch(counts, lengths, page, g)
    cache = echo.Cache(pages, page, heads, dim, bits)
    before = torch.randint(0, 256, cache.codes.shape, generator=g, device="cuda", dtype=torch.uint8)
    cache.codes.copy_(before)
    batch = tensors(starts, lengths, table)
    k, v = (values(g, starts[-1], heads, dim).mul(10.0 ** torch.randint(-4, 4, (starts[-1], heads, 1), generator=g,
                                                                        device="cuda")).to(dt) for _ in range(2))
    k[0], v[1], k[2] = 0, v[1].abs(), -k[2].abs()            # rows of zeros, and of one sign
    echo.echo_cache_append(cache, batch, k, v)
    want_codes, want_meta = before.clone(), torch.zeros_like(cache.meta)
    back = {}
    for i, t in enumerate((k, v)):
        code, s, z = ref.groups(t, bits)
        back[i] = (s * (code.double() - z)).to(dt)
        for b, row, place in ref.sequences(starts, lengths, starts[-1]):
            at = int(table[b, place // page]), i, slice(None), place % page
            want_codes[at] = ref.pack(code[row], bits)
            want_meta[at] = ref.words(s[row], z[row])
    assert torch.equal(cache.meta, want_meta)
    assert torch.equal(cache.codes, want_codes)
    got = [torch.full_like(k, 7), torch.full_like(v, 7)]
    echo.echo_cache_read(cache, batch, *got)
    assert torch.equal(got[0], back[0]) and torch.equal(got[1], back[1])
    only = torch.full_like(v, 7)
    echo.echo_cache_read(cache, batch, None, only)
    assert torch.equal(only, back[1])
    assert echo.echo_serving_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("tokens,dim,heads", [(9800, 64, 1), (3300, 64, 9), (5000, 128, 3), (3300, 128, 5), (3300, 256, 3)])
def test_many_rows_are_quantised_exactly(dtype, bits, tokens, dim, heads):
    """As above, with so many rows that a warp has several steps of a token's, the
    last of them in part or not at all, and groups that cannot be held among them."""
    from bit_error_compensated_gb300 import echo
    g = gen(dim + bits + heads)
    page, pages = 64, (tokens + 63) // 64
    cache = echo.Cache(pages, page, heads, dim, bits)
    batch = tensors([0, tokens], [tokens], torch.arange(pages, dtype=torch.int32, device="cuda")[None])
    k, v = (values(g, tokens, heads, dim).mul(10.0 ** torch.randint(-4, 4, (tokens, heads, 1), generator=g, device="cuda"))
            .to(DTYPES[dtype]) for _ in range(2))
    bad = [(0, 17, 0, float("nan")), (0, 500, heads - 1, float("inf")), (1, tokens - 1, heads // 2, float("-inf"))]
    both = torch.stack((k, v))                               # as they are without those
    code, s, z = ref.groups(both, bits)
    for i, token, head, x in bad:
        (k, v)[i][token, head, (7 * token) % dim] = x
    echo.echo_cache_append(cache, batch, k, v)
    assert echo.echo_serving_status() == echo.ECHO_ERR_OVERFLOW
    rows = lambda t: t.permute(1, 0, 3, 2, *range(4, t.dim())).flatten(1, 2)[:, :tokens]     # noqa: E731  (pages' places in a row)
    got_codes, got_meta = rows(cache.codes), rows(cache.meta)
    want_codes, want_meta = ref.pack(code, bits), ref.words(s, z)
    assert want_meta.shape == got_meta.shape and want_codes.shape == got_codes.shape
    for i, token, head, _ in bad:
        assert int(got_meta[i, token, head]) & 0x7FFF == 0x7E00
        want_meta[i, token, head] = got_meta[i, token, head]
        want_codes[i, token, head] = got_codes[i, token, head]
    assert torch.equal(got_meta, want_meta) and torch.equal(got_codes, want_codes)


@pytest.mark.parametrize("bits", [4, 8])
def test_values_next_to_a_border_are_rounded_exactly(bits):
    """fp32 values a step of their own beside k + 1/2 steps of the group, and
    ranges beside a multiple of an fp16 step: where a rounded quotient would
    fall on the other side."""
    from bit_error_compensated_gb300 import echo
    g = gen(bits)
    top, rows = 2 ** bits - 1, 512
    s = (0.5 + torch.rand(rows, 1, generator=g, device="cuda")).half().float()
    v = s * (torch.randint(0, top, (rows, 128), generator=g, device="cuda") + 0.5)
    v = torch.nextafter(v, v + torch.randint(-1, 2, v.shape, generator=g, device="cuda"))
    v[:, 0] = 0
    v[:, 1] = (s * top).squeeze(1)                           # the range, exactly s * top or a step beside
    v[:, 1] = torch.nextafter(v[:, 1], v[:, 1] + torch.randint(-1, 2, (rows,), generator=g, device="cuda"))
    table = torch.arange(rows // 16, dtype=torch.int32, device="cuda")[None]
    cache = echo.Cache(rows // 16, 16, 1, 128, bits)
    batch = tensors([0, rows], [rows], table)
    k = v[:, None].contiguous()
    echo.echo_cache_append(cache, batch, k, -k)
    for i, t in enumerate((k, -k)):
        code, step, z = ref.groups(t, bits)
        assert torch.equal(cache.meta[:, i, 0].flatten(), ref.words(step, z).flatten())
        assert torch.equal(cache.codes[:, i, 0].flatten(0, 1), ref.pack(code[:, 0], bits))


def test_groups_that_cannot_be_held_read_as_nan_and_are_reported():
    from bit_error_compensated_gb300 import echo
    k = torch.randn(6, 2, 64, device="cuda")
    v = torch.randn(6, 2, 64, device="cuda")
    k[1, 0, 5], k[2, 1, 63], v[3, 0, 0], v[4, 1, 7] = math.nan, math.inf, -math.inf, 1e9
    v[5, 0, 0], v[5, 0, 1] = 3e38, -3e38
    cache = echo.Cache(1, 16, 2, 64, 4)
    batch = tensors([0, 6], [6], torch.zeros(1, 1, dtype=torch.int32, device="cuda"))
    echo.echo_cache_append(cache, batch, k, v)
    assert echo.echo_serving_status() == echo.ECHO_ERR_OVERFLOW
    assert echo.echo_serving_status() == 0
    got = [torch.empty_like(k), torch.empty_like(v)]
    echo.echo_cache_read(cache, batch, *got)
    for t, want in ((got[0], [(1, 0), (2, 1)]), (got[1], [(3, 0), (4, 1), (5, 0)])):
        nan = torch.isnan(t).all(-1)
        assert nan.nonzero().tolist() == [list(w) for w in want]
        assert torch.equal(torch.isnan(t).any(-1), nan)


def test_rows_behind_the_batch_and_before_a_sequence_are_left():
    """Rows outside starts[0]..starts[-1] are not touched; tokens before their
    sequence's begin are not written and read as zeros."""
    from bit_error_compensated_gb300 import echo
    g = gen(5)
    table = torch.tensor([[2], [0]], dtype=torch.int32, device="cuda")
    cache = echo.Cache(3, 16, 2, 64, 8)
    batch = tensors([2, 7, 9], [3, 2], table)               # five rows for three tokens: two before the begin
    k, v = (values(g, 12, 2, 64) for _ in range(2))
    echo.echo_cache_append(cache, batch, k, v)
    got = [torch.full_like(k, 7), torch.full_like(v, 7)]
    echo.echo_cache_read(cache, batch, *got)
    for t, x in zip(got, (k, v)):
        code, s, z = ref.groups(x, 8)
        want = (s * (code.double() - z)).float()
        want[2:4] = 0
        want[:2], want[9:] = 7, 7
        assert torch.equal(t, want)
    assert torch.count_nonzero(cache.meta[1]) == 0 and torch.count_nonzero(cache.meta[2, :, :, 3:]) == 0
    q = values(g, 12, 4, 64, dtype=torch.bfloat16)
    out = torch.full_like(q, 7)
    lse = torch.full((12, 4), 7.0, device="cuda")
    echo.echo_attention(cache, batch, q, out, lse=lse)
    assert torch.all(out[:2] == 7) and torch.all(out[9:] == 7) and torch.all(out[2:4] == 0)
    assert torch.all(lse[:2] == 7) and torch.all(lse[9:] == 7) and torch.all(lse[2:4] == -math.inf)
    assert torch.isfinite(lse[4:9]).all()
    assert echo.echo_serving_status() == 0


@pytest.mark.parametrize("what", ["page", "table", "rows", "falling"])
def test_arrays_that_make_no_sense_are_reported_and_left_out(what):
    """The kernels check what the arrays hold: nothing outside the tensors is
    touched, the rest is computed, and the status says so."""
    from bit_error_compensated_gb300 import echo
    g = gen(6)
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    starts, lengths = [0, 4, 8], [30, 20]
    if what == "page":
        table[0, 0], table[1, 1] = 99, -5
    if what == "table":
        lengths[1] = 100                                     # its last places lie past the table
    if what == "rows":
        starts[2] = 11
    if what == "falling":
        starts[1] = 9
    cache = full_cache(g, 4, 16, 2, 64, 8)
    batch = tensors(starts, lengths, table)
    k, v, q = (values(g, 8, 2, 64, dtype=torch.float16) for _ in range(3))
    want = {"page": echo.ECHO_ERR_ARG, "table": echo.ECHO_ERR_ARG}.get(what, echo.ECHO_ERR_SHAPE)
    out, back = torch.zeros_like(q), [torch.full_like(k, 7) for _ in range(2)]
    echo.echo_attention(cache, batch, q, out)
    assert echo.echo_serving_status() == want
    if what in ("page", "table"):
        exact, _, tol = ref.attention(cache, q, starts, lengths, table, 64 ** -0.5)
        assert ((out.double() - exact).abs() <= tol + ref.half_step(torch.float16) * exact.abs()).all()
    echo.echo_cache_append(cache, batch, k, v)
    assert echo.echo_serving_status() == want
    echo.echo_cache_read(cache, batch, *back)
    assert echo.echo_serving_status() == want
    if what == "table":
        assert torch.all(back[0][4:] == 0) and torch.all(back[0][:4] != 7)
    if what == "page":
        assert torch.all(back[0][4:] == 0)                  # of the second sequence all four lie in its missing page


# --------------------------------------------------------------- attention
def check(cache, batch, q, starts, lengths, table, scale=None, causal=True, window=0, lse=True, out=None):
    from bit_error_compensated_gb300 import echo
    out = torch.full_like(q, 7) if out is None else out
    logs = torch.full(q.shape[:2], 7.0, device="cuda") if lse else None
    echo.echo_attention(cache, batch, q, out, scale=scale, causal=causal, window=window, lse=logs)
    scale = cache.head_dim ** -0.5 if scale is None else scale
    exact, exact_lse, tol = ref.attention(cache, q, starts, lengths, table, scale, causal, window)
    rows = torch.tensor([r for _, r, _ in ref.sequences(starts, lengths, q.shape[0])], device="cuda", dtype=torch.long)
    got, want = out[rows].double(), exact[rows]
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    # one rounding to out's type, of its subnormal step at the least
    limit = tol[rows] + ref.half_step(q.dtype) * (want.abs() + tol[rows]) + torch.finfo(q.dtype).smallest_normal * ref.half_step(q.dtype)
    off = torch.nan_to_num((got - want).abs() - limit, nan=-1.0)
    assert off.max().item() <= 0, (off.max().item(), off.argmax().item())
    if lse:
        finite = torch.isfinite(exact_lse[rows])
        assert torch.equal(torch.isfinite(logs[rows]), finite)
        # scores' errors as in the tolerance of out (at most 2^-10 for these inputs), and fp32's own
        near = (logs[rows].double() - exact_lse[rows]).abs() <= 2.0 ** -10 + 2.0 ** -21 * exact_lse[rows].abs()
        assert near[finite].all()
    assert echo.echo_serving_status() == 0
    return out


SHAPES = [
    # counts, lengths, heads, group, dim, page
    ([1], [1], 1, 1, 64, 16),
    ([1], [15], 2, 1, 128, 16),
    ([1], [64], 1, 8, 128, 64),
    ([1], [65], 3, 3, 256, 32),
    ([1], [2000], 8, 4, 128, 64),
    ([1] * 9, [1, 2, 16, 17, 63, 64, 65, 129, 700], 2, 4, 128, 64),
    ([1, 0, 1, 1], [300, 50, 0, 33], 2, 7, 64, 128),
    ([5] * 4, [5, 70, 131, 1000], 2, 7, 64, 16),
    ([3, 1, 2], [3, 200, 90], 2, 16, 256, 256),
    ([2, 3], [400, 17], 1, 33, 64, 64),
    ([33], [33], 2, 4, 128, 16),
    ([70, 1, 200], [70, 500, 333], 2, 5, 128, 64),
    ([130, 257], [1000, 257], 1, 8, 64, 32),
    ([100, 3], [612, 40], 2, 2, 256, 128),
    ([300], [1300], 1, 1, 128, 256),
]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("counts,lengths,heads,group,dim", [
    ([600], [5000], 1, 4, 256), ([700], [4000], 3, 5, 128), ([90] * 40, [130 + 7 * i for i in range(40)], 2, 4, 64),
    ([1] * 33, [2000 + i for i in range(33)], 4, 8, 128), ([1, 500, 2], [9000, 500, 4000], 2, 6, 128)])
def test_blocks_that_walk_several_units(bits, counts, lengths, heads, group, dim):
    """Enough rows and keys that a block has whole units and parts of others one
    after the other, and more sequences than a warp has lanes."""
    g = gen(bits + group)
    starts, table, pages = make_batch(counts, lengths, 64, g)
    cache = full_cache(g, pages, 64, heads, dim, bits)
    spoil_behind(cache, lengths, table)
    q = values(g, starts[-1], heads * group, dim, dtype=torch.bfloat16)
    check(cache, tensors(starts, lengths, table), q, starts, lengths, table)


@pytest.mark.parametrize("new", [3, 200])
def test_without_causal_order_tokens_before_the_begin_see_nothing(new):
    from bit_error_compensated_gb300 import echo
    g = gen(19)
    starts, table, pages = make_batch([new], [new - 2], 16, g)
    cache = full_cache(g, pages, 16, 1, 64, 4)
    q = values(g, new, 2, 64, dtype=torch.float16)
    out = torch.full_like(q, 7)
    echo.echo_attention(cache, tensors(starts, [new - 2], table), q, out, causal=False)
    assert torch.all(out[:2] == 0) and torch.all(out[2:].abs().amax(-1) > 0) and torch.all(out[2:] != 7)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, (len(s[0]), max(s[0]), max(s[1]), *s[2:]))))
def test_attention(dtype, bits, shape):
    counts, lengths, heads, group, dim, page = shape
    g = gen(sum(lengths) + bits)
    starts, table, pages = make_batch(counts, lengths, page, g)
    cache = full_cache(g, pages, page, heads, dim, bits)
    spoil_behind(cache, lengths, table)
    q = (1.5 * values(g, starts[-1], heads * group, dim)).to(DTYPES[dtype])
    check(cache, tensors(starts, lengths, table), q, starts, lengths, table)


@pytest.mark.parametrize("counts,lengths,group,dim", [([1, 1, 1], [5, 300, 1000], 4, 128), ([9, 40], [700, 40], 3, 64),
                                                      ([200], [900], 4, 128)])
@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 200, 5000])
def test_window(counts, lengths, group, dim, window):
    g = gen(window)
    starts, table, pages = make_batch(counts, lengths, 32, g)
    cache = full_cache(g, pages, 32, 2, dim, 4)
    spoil_behind(cache, lengths, table)
    q = values(g, starts[-1], 2 * group, dim, dtype=torch.bfloat16)
    check(cache, tensors(starts, lengths, table), q, starts, lengths, table, window=window)


@pytest.mark.parametrize("counts,lengths", [([1, 4], [100, 333]), ([150], [260]), ([40], [7])])
def test_without_causal_order_every_token_sees_all(counts, lengths):
    g = gen(7)
    starts, table, pages = make_batch(counts, lengths, 16, g)
    cache = full_cache(g, pages, 16, 2, 128, 8)
    spoil_behind(cache, lengths, table)
    q = values(g, starts[-1], 8, 128, dtype=torch.float16)
    check(cache, tensors(starts, lengths, table), q, starts, lengths, table, causal=False, scale=-0.05)


@pytest.mark.parametrize("new,length", [(1, 3000), (130, 3000), (300, 100)])
def test_no_key_and_fewer_keys_than_tokens(new, length):
    """Tokens before their sequence's begin, and a sequence of no length."""
    g = gen(new)
    counts, lengths = [new, 2], [length, 0]
    starts, table, pages = make_batch(counts, lengths, 64, g)
    cache = full_cache(g, pages, 64, 1, 128, 4)
    spoil_behind(cache, lengths, table)
    q = values(g, starts[-1], 4, 128, dtype=torch.bfloat16)
    out = check(cache, tensors(starts, lengths, table), q, starts, lengths, table)
    assert torch.all(out[-2:] == 0)
    if new > length:
        assert torch.all(out[:new - length] == 0) and torch.any(out[new - length] != 0)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("new", [1, 80])
def test_places_that_were_never_written_are_zeros(new, bits):
    """A new cache holds words of 0, whose values are 0: their weights count, alone
    and among written places."""
    from bit_error_compensated_gb300 import echo
    g = gen(new + bits)
    counts, lengths = [new, new], [700, 333]
    starts, table, pages = make_batch(counts, lengths, 64, g)
    cache = full_cache(g, pages, 64, 2, 128, bits)
    gone = torch.rand(pages, 1, 1, 64, generator=g, device="cuda") < 0.5
    gone[table[1].long()] = True                             # all of the second sequence
    gone = gone.expand(cache.meta.shape)
    cache.meta[gone] = 0
    cache.codes[gone] = 0
    q = values(g, 2 * new, 8, 128, dtype=torch.bfloat16)
    out = check(cache, tensors(starts, lengths, table), q, starts, lengths, table)
    assert torch.all(out[new:] == 0) and torch.any(out[:new] != 0)
    fresh = echo.Cache(pages, 64, 2, 128, bits)
    assert torch.all(check(fresh, tensors(starts, lengths, table), q, starts, lengths, table) == 0)


@pytest.mark.parametrize("new", [1, 70])
def test_extreme_scales_of_queries_keys_and_values(new):
    """Rows of q from 2^-60 to 2^60 of each other, values' steps over six orders
    of magnitude, scores large enough that one key takes all."""
    g = gen(11)
    starts, table, pages = make_batch([new], [500], 64, g)
    from bit_error_compensated_gb300 import echo
    cache = echo.Cache(pages, 64, 2, 128, 8)
    v = values(g, pages, 2, 2, 64, 128)
    v[:, 1] *= 10.0 ** torch.randint(-3, 4, (pages, 2, 64, 1), generator=g, device="cuda")
    code, s, z = ref.groups(v, 8)
    cache.codes.copy_(code)
    cache.meta.copy_(ref.words(s, z))
    q = values(g, new, 8, 128)
    q[:, 1] *= 2.0 ** -60
    q[:, 2] = 0
    q[:, 3] *= 30
    q[:, 5] *= 2.0 ** -20
    batch = tensors(starts, [500], table)
    check(cache, batch, q.bfloat16(), starts, [500], table, lse=False)
    check(cache, batch, q.bfloat16(), starts, [500], table, scale=0.0, lse=False)


@pytest.mark.parametrize("new", [3, 100])
def test_nan_and_infinity_reach_only_the_rows_that_see_them(new):
    g = gen(12)
    counts, lengths = [new, new], [400, 400]
    starts, table, pages = make_batch(counts, lengths, 32, g)
    cache = full_cache(g, pages, 32, 2, 128, 4)
    q = values(g, starts[-1], 8, 128, dtype=torch.bfloat16)
    q[0, 1, 3], q[1, 2, 5] = math.nan, math.inf
    place = 400 - 2                                          # the second sequence's last two tokens see it
    page = int(table[1, place // 32])
    cache.meta[page, 0, 1, place % 32] = 0x7E00              # a key of NaN
    cache.codes[page, 0, 1, place % 32] = 0
    page = int(table[1, 399 // 32])
    cache.meta[page, 1, 0, 399 % 32] = 0x7E00                # a value of NaN
    cache.codes[page, 1, 0, 399 % 32] = 0
    out = torch.empty_like(q)
    from bit_error_compensated_gb300 import echo
    echo.echo_attention(cache, tensors(starts, lengths, table), q, out)
    nan = torch.isnan(out)
    assert torch.equal(nan.any(-1), nan.all(-1))
    want = torch.zeros_like(nan[..., 0])
    want[0, 1] = want[1, 2] = True
    want[-2:, 4:] = True
    want[-1:, :4] = True
    assert torch.equal(nan.any(-1), want)


@pytest.mark.parametrize("new", [1, 90])
def test_strided_and_unaligned_tensors(new):
    """q as a part of a projection's rows, out in [heads][tokens] order, and both
    off every boundary but their element's: the same bits as contiguous ones."""
    from bit_error_compensated_gb300 import echo
    g = gen(13)
    starts, table, pages = make_batch([new], [257], 16, g)
    cache = full_cache(g, pages, 16, 2, 64, 8)
    batch = tensors(starts, [257], table)
    q = values(g, new, 6, 64, dtype=torch.float16)
    want = check(cache, batch, q, starts, [257], table)
    rows = torch.zeros(new, 6 * 64 + 1 + 37, dtype=torch.float16, device="cuda")
    part = rows[:, 1:1 + 6 * 64].unflatten(1, (6, 64))
    part.copy_(q)
    turned = torch.zeros(6, new + 1, 65, dtype=torch.float16, device="cuda")[:, 1:, 1:].transpose(0, 1)
    echo.echo_attention(cache, batch, part, turned)
    assert torch.equal(turned, want)
    k = values(g, new, 2, 64)
    flat = torch.zeros(new * 2 * 65 + 1, device="cuda")[1:].view(new, 2, 65)[..., :64]
    flat.copy_(k)
    wide = torch.zeros(1, table.shape[1] + 3, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    echo.echo_cache_append(cache, batch, k, k)
    codes, meta = cache.codes.clone(), cache.meta.clone()
    cache.codes.zero_()
    echo.echo_cache_append(cache, echo.CacheBatch(batch.starts, batch.lengths, wide[:, :table.shape[1]]), flat, flat)
    assert torch.equal(cache.meta, meta)
    got = torch.zeros(new * 2 * 65 + 1, device="cuda")[1:].view(new, 2, 65)[..., :64]
    echo.echo_cache_read(cache, batch, got, None)
    code, s, z = ref.groups(k, 8)
    assert torch.equal(got, (s * (code.double() - z)).float())


@pytest.mark.parametrize("new", [1, 80])
def test_a_repeated_call_gives_the_same_bits(new):
    from bit_error_compensated_gb300 import echo
    g = gen(14)
    starts, table, pages = make_batch([new, new], [3000, 1234], 64, g)
    cache = full_cache(g, pages, 64, 4, 128, 4)
    batch = tensors(starts, [3000, 1234], table)
    q = values(g, 2 * new, 16, 128, dtype=torch.bfloat16)
    first, again = torch.empty_like(q), torch.empty_like(q)
    echo.echo_attention(cache, batch, q, first)
    for _ in range(5):
        echo.echo_attention(cache, batch, q, again)
        assert torch.equal(first, again)


def test_a_cache_past_32_bits_of_bytes():
    """Codes beyond 4 GiB and groups beyond 2^31 bits of index arithmetic: the
    last pages of a cache of 4.6 GB hold a sequence."""
    from bit_error_compensated_gb300 import echo
    g = gen(15)
    pages = 8800                                             # 512 KiB of codes each
    cache = echo.Cache(pages, 256, 4, 256, 8)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    starts, lengths = [0, 300], [300]
    batch = tensors(starts, lengths, table)
    k, v = (values(g, 300, 4, 256) for _ in range(2))
    echo.echo_cache_append(cache, batch, k, v)
    got = [torch.empty_like(k), torch.empty_like(v)]
    echo.echo_cache_read(cache, batch, *got)
    for t, x in zip(got, (k, v)):
        code, s, z = ref.groups(x, 8)
        assert torch.equal(t, (s * (code.double() - z)).float())
    assert torch.count_nonzero(cache.meta[:pages - 2]) == 0
    q = values(g, 300, 4, 256, dtype=torch.bfloat16)
    check(cache, batch, q, starts, lengths, table)
    one = tensors([0, 1], lengths, table)
    check(cache, one, q[:1].contiguous(), [0, 1], lengths, table)


def test_captured_calls_follow_the_arrays():
    """Append and attention captured once and replayed while lengths grow: a
    decode loop in a graph; two graphs have workspaces of their own."""
    from bit_error_compensated_gb300 import echo
    g = gen(16)
    cache, other = (full_cache(g, 40, 16, 2, 64, 4) for _ in range(2))
    table = torch.randperm(40, generator=g, device="cuda").int().view(2, 20)
    starts = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([17, 200], dtype=torch.int32, device="cuda")
    batch = echo.CacheBatch(starts, lengths, table)
    k, v = torch.empty(2, 2, 64, device="cuda"), torch.empty(2, 2, 64, device="cuda")
    q = torch.empty(2, 8, 64, dtype=torch.bfloat16, device="cuda")
    outs, graphs = [torch.empty_like(q) for _ in range(2)], []
    for c, out in ((cache, outs[0]), (other, outs[1])):
        echo.echo_cache_append(c, batch, k.normal_(generator=g), v.normal_(generator=g))
        echo.echo_attention(c, batch, q.normal_(generator=g), out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            echo.echo_cache_append(c, batch, k, v)
            echo.echo_attention(c, batch, q, out)
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(40):
        lengths += 1
        for t in (k, v, q):
            t.normal_(generator=g)
        for st, graph in zip(streams, graphs):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                graph.replay()
        for st in streams:
            torch.cuda.current_stream().wait_stream(st)
        now = lengths.tolist()
        for c, out in ((cache, outs[0]), (other, outs[1])):
            exact, _, tol = ref.attention(c, q, [0, 1, 2], now, table, 64 ** -0.5)
            assert ((out.double() - exact).abs() <= tol + ref.half_step(q.dtype) * (exact.abs() + tol)).all()
    assert echo.echo_serving_status() == 0


def test_another_stream_than_the_current_one():
    from bit_error_compensated_gb300 import echo
    g = gen(17)
    starts, table, pages = make_batch([2, 60], [900, 800], 64, g)
    cache = full_cache(g, pages, 64, 2, 128, 8)
    batch = tensors(starts, [900, 800], table)
    q = values(g, 62, 8, 128, dtype=torch.float16)
    want = check(cache, batch, q, starts, [900, 800], table)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for raw in (stream, stream.cuda_stream):
        out = torch.zeros_like(q)
        stream.wait_stream(torch.cuda.current_stream())
        echo.echo_attention(cache, batch, q, out, stream=raw)
        stream.synchronize()
        assert torch.equal(out, want)


def test_many_sequences():
    """More sequences than a block has threads, some without tokens or keys."""
    g = gen(18)
    n = 1500
    lengths = torch.randint(0, 60, (n,), generator=torch.Generator().manual_seed(3)).tolist()
    counts = [(i * 7) % 3 for i in range(n)]
    starts, table, pages = make_batch(counts, lengths, 16, g)
    cache = full_cache(g, pages, 16, 1, 64, 4)
    spoil_behind(cache, lengths, table)
    from bit_error_compensated_gb300 import echo
    batch = tensors(starts, lengths, table)
    q = values(g, starts[-1], 3, 64, dtype=torch.bfloat16)
    k, v = values(g, starts[-1], 1, 64), values(g, starts[-1], 1, 64)
    echo.echo_cache_append(cache, batch, k, v)
    got = torch.full_like(k, 7)
    echo.echo_cache_read(cache, batch, got, None)
    code, s, z = ref.groups(k, 4)
    want = (s * (code.double() - z)).float()
    for _, row, place in ref.sequences(starts, lengths, starts[-1]):
        if place < 0:
            want[row] = 0
    assert torch.equal(got, want)
    check(cache, batch, q, starts, lengths, table)
