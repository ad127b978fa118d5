"""Host side of the serving operators without a GPU: the C calls' refusals
(reported before any CUDA call), the packed structures, the binding's checks,
and rules of their kernels that no run shows."""
import ctypes
import re
from pathlib import Path

import pytest
import torch

from test_block_sources import body_after, source

ROOT = Path(__file__).resolve().parents[1]
CSRC = ROOT / "bit_error_compensated_gb300" / "csrc"
MB = 1 << 20
FILES = ["serve_common.h", "attn_common.h", "cache_rows.cu", "attn_few.cu", "attn_many.cu", "int4_few.cu", "int4_quantize.cu"]


@pytest.fixture(scope="module")
def echo():
    from bit_error_compensated_gb300.build import build_library
    build_library()
    from bit_error_compensated_gb300 import echo
    return echo


def test_packed_structures_follow_the_header(echo):
    text = re.sub(r"/\*.*?\*/", "", (ROOT / "include" / "echo.h").read_text(), flags=re.S)
    for name, packed, fields in (
            ("echo_cache", echo._CACHE, ["codes", "meta", "pages", "page_size", "heads", "head_dim", "bits"]),
            ("echo_batch", echo._BATCH, ["sequences", "tokens", "starts", "lengths", "table", "table_pages", "ld_table"]),
            ("echo_heads", echo._HEADS, ["data", "ld", "head_stride"])):
        body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", text).group(1)
        declared = []
        for line in filter(None, (x.strip() for x in body.split(";"))):
            assert line.startswith("int64_t ") or "*" in line, line          # 8 bytes each
            declared += [re.search(r"(\w+)\s*$", part).group(1) for part in line.split(",")]
        assert declared == fields and packed.size == 8 * len(fields)
    for name in ("ECHO_CACHE_MAX_HEADS", "ECHO_BATCH_MAX_TOKENS"):
        assert int(re.search(rf"#define {name}\s+(\d+)", text).group(1)) == getattr(echo, name)


def cache(echo, codes=MB, meta=2 * MB, pages=4, page_size=16, heads=2, head_dim=64, bits=4):
    return echo._CACHE.pack(codes, meta, pages, page_size, heads, head_dim, bits)


def batch(echo, sequences=2, tokens=8, starts=3 * MB, lengths=3 * MB + 64, table=3 * MB + 128, pages=2, ld=2):
    return echo._BATCH.pack(sequences, tokens, starts, lengths, table, pages, ld)


def heads(echo, data=4 * MB, ld=128, stride=64):
    return echo._HEADS.pack(data, ld, stride)


BAD_CACHE = [(dict(head_dim=96), "UNSUPPORTED"), (dict(bits=3), "UNSUPPORTED"), (dict(page_size=48), "UNSUPPORTED"),
             (dict(page_size=8), "UNSUPPORTED"), (dict(heads=1025), "UNSUPPORTED"), (dict(pages=2 ** 31), "UNSUPPORTED"),
             (dict(heads=0), "SHAPE"), (dict(pages=-1), "SHAPE"), (dict(codes=0), "ARG"), (dict(meta=0), "ARG"),
             (dict(codes=MB + 8), "ALIGN"), (dict(meta=2 * MB + 4), "ALIGN")]
BAD_BATCH = [(dict(sequences=-1), "SHAPE"), (dict(tokens=-1), "SHAPE"), (dict(pages=-1), "SHAPE"), (dict(ld=1), "SHAPE"),
             (dict(sequences=2 ** 20 + 1), "UNSUPPORTED"), (dict(tokens=2 ** 20 + 1), "UNSUPPORTED"),
             (dict(pages=2 ** 26 + 1, ld=2 ** 27), "UNSUPPORTED"), (dict(starts=0), "ARG"), (dict(lengths=0), "ARG"),
             (dict(table=0), "ARG"), (dict(starts=3 * MB + 2), "ALIGN"), (dict(table=3 * MB + 129), "ALIGN")]


def test_calls_over_a_cache_are_checked_before_any_cuda_call(echo):
    lib = echo._lib
    calls = {
        "append": lambda c, b, k=heads(echo), v=heads(echo, 5 * MB), dtype=1: lib.echo_cache_append(c, b, dtype, k, v, None),
        "read": lambda c, b, k=heads(echo), v=heads(echo, 5 * MB), dtype=1: lib.echo_cache_read(c, b, dtype, k, v, None),
        "attention": lambda c, b, k=heads(echo), v=heads(echo, 5 * MB), dtype=1: lib.echo_attention(
            c, b, 2, dtype, k, v, 0.1, 1, 0, None, 16 * MB, 2 ** 30, None),
    }
    for name, call in calls.items():
        assert call(None, batch(echo)) == call(cache(echo), None) == echo.ECHO_ERR_ARG, name
        for bad, status in BAD_CACHE:
            assert call(cache(echo, **bad), batch(echo)) == getattr(echo, "ECHO_ERR_" + status), (name, bad)
        for bad, status in BAD_BATCH:
            assert call(cache(echo), batch(echo, **bad)) == getattr(echo, "ECHO_ERR_" + status), (name, bad)
        assert call(cache(echo), batch(echo), dtype=7) == echo.ECHO_ERR_UNSUPPORTED
        assert call(cache(echo), batch(echo), k=heads(echo, 4 * MB + 1)) == echo.ECHO_ERR_ALIGN
        assert call(cache(echo), batch(echo), v=heads(echo, 5 * MB, ld=-1)) == echo.ECHO_ERR_SHAPE
        # nothing to do: no tokens, no sequences
        for none in (dict(tokens=0), dict(sequences=0)):
            assert call(cache(echo), batch(echo, starts=0, **none)) == echo.ECHO_OK
        # in the place of the cache, or of the batch's arrays where they are written
        assert call(cache(echo), batch(echo), v=heads(echo, MB)) == echo.ECHO_ERR_ARG, name
        if name != "append":
            assert call(cache(echo), batch(echo), v=heads(echo, 3 * MB)) == echo.ECHO_ERR_ARG, name
            assert call(cache(echo), batch(echo), v=heads(echo, 4 * MB + 64)) == echo.ECHO_ERR_ARG, name
            # rows that share elements
            assert call(cache(echo), batch(echo), v=heads(echo, 5 * MB, ld=64)) == echo.ECHO_ERR_SHAPE, name
            assert call(cache(echo), batch(echo), v=heads(echo, 5 * MB, stride=32)) == echo.ECHO_ERR_SHAPE, name
    assert calls["append"](cache(echo), batch(echo), k=None) == echo.ECHO_ERR_ARG
    assert calls["append"](cache(echo, codes=3 * MB), batch(echo)) == echo.ECHO_ERR_ARG        # the cache over the batch
    assert calls["append"](cache(echo, meta=MB + 4096), batch(echo)) == echo.ECHO_ERR_ARG      # meta in the codes


def test_attention_arguments_are_checked_before_any_cuda_call(echo):
    c, b = cache(echo), batch(echo)

    def status(heads_=2, dtype=1, scale=0.1, causal=1, window=0, tokens=8):
        return echo._lib.echo_attention(c, batch(echo, tokens=tokens), heads_, dtype, heads(echo), heads(echo, 5 * MB), scale,
                                        causal, window, None, 16 * MB, 2 ** 30, None)

    assert status(heads_=3) == status(heads_=0) == status(heads_=-2) == echo.ECHO_ERR_SHAPE
    assert status(dtype=0) == echo.ECHO_ERR_UNSUPPORTED                 # fp32
    assert status(heads_=2 ** 12, tokens=2 ** 20) == echo.ECHO_ERR_UNSUPPORTED
    assert status(scale=float("nan")) == status(scale=float("inf")) == echo.ECHO_ERR_ARG
    assert status(causal=2) == status(window=-1) == status(causal=0, window=4) == echo.ECHO_ERR_ARG
    assert echo._lib.echo_attention_workspace_bytes(c, b, 3) == 0
    assert echo._lib.echo_attention_workspace_bytes(cache(echo, bits=5), b, 2) == 0
    assert echo._lib.echo_serving_status(None, None) == echo.ECHO_ERR_ARG


def test_weights_are_checked_before_any_cuda_call(echo):
    m = lambda at, ld, stride=0: echo._MATRIX.pack(at, ld, stride)               # noqa: E731

    def quantize(ranks=1, channels=8, depth=130, dtype=1, group=128, w=m(MB, 130), codes=m(2 * MB, 65), meta=m(3 * MB, 2)):
        return echo._lib.echo_quantize_weights(ranks, channels, depth, dtype, group, w, codes, meta, None)

    def linear(ranks=1, tokens=4, channels=8, depth=130, dtype=1, group=128, x=m(MB, 130), codes=m(2 * MB, 65),
               meta=m(3 * MB, 2), out=m(4 * MB, 8)):
        return echo._lib.echo_linear_int4(ranks, tokens, channels, depth, dtype, group, x, codes, meta, out, None)

    for call in (quantize, linear):
        assert call(ranks=0) == call(ranks=17) == echo.ECHO_ERR_ARG
        assert call(channels=-1) == call(depth=-1) == echo.ECHO_ERR_SHAPE
        assert call(group=96) == call(group=32) == call(dtype=5) == call(depth=131072) == echo.ECHO_ERR_UNSUPPORTED
        assert call(channels=2 ** 20 + 1) == echo.ECHO_ERR_UNSUPPORTED
        assert call(codes=None) == call(meta=m(0, 2)) == echo.ECHO_ERR_ARG
        assert call(codes=m(2 * MB, 64)) == call(meta=m(3 * MB, 1)) == echo.ECHO_ERR_SHAPE
        assert call(meta=m(3 * MB + 2, 2)) == echo.ECHO_ERR_ALIGN
    assert quantize(codes=m(MB + 100, 65)) == quantize(meta=m(MB, 2)) == quantize(meta=m(2 * MB, 2)) == echo.ECHO_ERR_ARG
    assert linear(out=m(MB, 8)) == linear(out=m(2 * MB, 8)) == linear(out=m(3 * MB, 8)) == echo.ECHO_ERR_ARG
    assert linear(ranks=2, x=m(MB, 130), out=m(4 * MB, 8, 8)) == echo.ECHO_ERR_ARG      # one rank's rows over another's
    assert linear(tokens=0) == linear(channels=0) == quantize(channels=0) == quantize(depth=0) == echo.ECHO_OK


def test_the_binding_refuses_what_is_not_on_a_gpu_or_does_not_fit(echo):
    for kw in (dict(page_size=24), dict(head_dim=80), dict(bits=2), dict(heads=0), dict(pages=-1)):
        with pytest.raises(ValueError):
            echo.Cache(**{**dict(pages=2, page_size=16, heads=2, head_dim=64, bits=4), **kw})
    codes, meta = torch.zeros(2, 2, 2, 16, 32, dtype=torch.uint8), torch.zeros(2, 2, 2, 16, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        echo.Cache(2, 16, 2, 64, 4, codes=codes, meta=meta)
    with pytest.raises(ValueError, match="belong together"):
        echo.Cache(2, 16, 2, 64, 4, codes=codes)
    ints = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        echo.CacheBatch(ints, ints[:2], torch.zeros(2, 4, dtype=torch.int32))
    with pytest.raises(ValueError, match="group"):
        echo._weight_shapes(None, 4, 128, 100)
    assert echo._weight_shapes(2, 4, 129, 64) == ((2, 4, 65), (2, 4, 3))
    with pytest.raises(ValueError, match="CUDA"):
        echo.echo_quantize_weights(torch.zeros(4, 128), None, None)
    with pytest.raises(ValueError, match="CUDA"):
        echo.echo_linear_int4(torch.zeros(1, 128), None, None, torch.zeros(1, 4))


# -------------------------------------------------------------- the kernels
def test_kernels_wait_for_the_one_before_and_read_by_ordinary_loads():
    """Blocks are in place while the kernel before still runs: each kernel but
    the status words' waits, and reads nothing as read-only data."""
    for name in FILES:
        text = source(name)
        assert "__ldg" not in text and "global.nc" not in text, name
        for kernel in re.finditer(r"__global__ (?!void clear_status)", text):
            assert "pdl_wait();" in body_after(text[kernel.start():], r"__global__"), name


def test_warps_are_together_at_aligned_instructions():
    """Loads and stores of tensor memory begin with a __syncwarp, and one stands
    between the selects of hidden keys and the matrix instructions on weights."""
    text = source("attn_many.cu")
    for m in re.finditer(r"void (tmem_load|tmem_store|tmem_store_pairs)\(", text):
        body = body_after(text[m.start():], r"void ")
        first = min(body.index("tcgen05."), len(body))
        assert 0 <= body.find("__syncwarp();") < first
    few = body_after(source("attn_few.cu"), r"attention_few_kernel\(")
    assert few.index("kNone") < few.index("__syncwarp();", few.index("kNone")) < few.index("transposed(")


def test_waits_of_the_attention_are_bounded_and_end_together():
    """Every wait goes through the bounded one, a block's flag is cleared only
    where it begins, and the issuing warp waits for what it issued however its
    loop ended."""
    text = source("attn_many.cu")
    assert "mbarrier.try_wait" not in text and "mbarrier.test_wait" not in text
    kernel = body_after(text, r"attention_many_kernel\(")
    assert re.findall(r"\bgive_up\s*=[^=]\s*[^;]*;", kernel) == ["give_up = 0;"]
    issuing = body_after(kernel, r"if \(warp >= kIssuer\)")
    last = issuing.index("mbar_wait_bounded(bar + B::kLast")
    assert "ok" not in issuing[issuing.rindex("if (one)", 0, last):last]
    assert kernel.index("tcgen05.dealloc") > kernel.rindex("__syncthreads();")


def test_register_split_is_within_the_launch():
    text = source("attn_many.cu")
    regs = {n: int(v) for n, v in re.findall(r"(k\w+Regs) = (\d+)", text)}
    assert 4 * regs["kWeightRegs"] + 2 * regs["kTurnRegs"] + regs["kIssueRegs"] <= 7 * 72
    assert 7 * 128 * 72 <= 65536


def test_a_report_that_was_not_read_is_not_cleared():
    body = body_after(source("serve_api.cu"), r"int echo_serving_status\(")
    assert re.search(r"if \(word\[i\]\) ECHO_OPS_CUDA\(words\[i\]\.clear\(word\[i\], s\)\);", body)
    assert "atomicAnd(&g_status, ~bits)" in source("serve_common.h")


# --------------------------------- the protocol of the tensor-core kernel's barriers
class Barrier:
    def __init__(self, count):
        self.count, self.arrived, self.phase = count, 0, 0

    def arrive(self):
        self.arrived += 1
        if self.arrived == self.count:
            self.arrived, self.phase = 0, self.phase + 1

    def done(self, parity):
        return self.phase & 1 != parity


def simulate(tiles_of_rows, units, seed):
    """The kernel's roles (issuing warp, keys, values, weights), as generators
    that yield what they wait for, and the tensor cores' queue, stepped in random
    order; True if all end.  units: tiles of each."""
    import random
    rng, NT = random.Random(seed), tiles_of_rows
    bars = {"query": Barrier(NT)}
    for i in range(2):
        bars.update({(n, i): Barrier(1) for n in ("keys", "keys_free", "values", "values_free", "scores", "weights", "sums")})
    bars.update({("steps", i): Barrier(2) for i in range(4)})
    queue, made = [], [0] * NT

    def issue():
        i = 0
        for u, n in enumerate(units):
            yield "query", u & 1
            yield ("keys", i & 1), i >> 1 & 1
            if NT == 2:
                queue.extend([("scores", 0), ("scores", 1), ("keys_free", i & 1)])
            else:
                queue.extend([("scores", i & 1), ("keys_free", i & 1)])
            for k in range(n):
                more = k + 1 < n
                if NT == 2:
                    for t in range(2):
                        yield ("weights", t), i & 1
                        if t == 0:
                            yield ("values", i & 1), i >> 1 & 1
                        if more:
                            if t == 0:
                                yield ("keys", i + 1 & 1), i + 1 >> 1 & 1
                            queue.append(("scores", t))
                        else:
                            queue.append(("sums", t))
                    queue.append(("values_free", i & 1))
                    if more:
                        queue.append(("keys_free", i + 1 & 1))
                else:
                    if more:
                        yield ("keys", i + 1 & 1), i + 1 >> 1 & 1
                        queue.extend([("scores", i + 1 & 1), ("keys_free", i + 1 & 1)])
                    yield ("weights", i & 1), i >> 1 & 1
                    yield ("values", i & 1), i >> 1 & 1
                    queue.append(("values_free", i & 1))
                    if not more:
                        queue.append(("sums", 0))
                i += 1

    def turn(what):
        for i in range(sum(units)):
            yield (what + "_free", i & 1), (i >> 1 & 1) ^ 1
            assert min(made) >= i - 3                        # the slot's steps have been used
            bars["steps", i & 3].arrive()
            yield None
            bars[what, i & 1].arrive()

    def weights(t):
        i = 0
        bars["query"].arrive()
        for u, n in enumerate(units):
            for k in range(n):
                yield ("steps", i & 3), i >> 2 & 1
                yield (("scores", t), i & 1) if NT == 2 else (("scores", i & 1), i >> 1 & 1)
                if NT == 1 and k > 0 and rng.random() < 0.3:
                    yield ("values_free", i - 1 & 1), i - 1 >> 1 & 1
                yield None
                made[t] = i + 1
                bars["weights", t if NT == 2 else i & 1].arrive()
                i += 1
            if u + 1 < len(units):
                bars["query"].arrive()
            yield ("sums", t), u & 1

    roles = [issue(), turn("keys"), turn("values")] + [weights(t) for t in range(NT)]
    waiting = {r: None for r in range(len(roles))}
    while waiting:
        ready = [r for r, w in waiting.items() if w is None or bars[w[0]].done(w[1])]
        if queue:
            ready.append(-1)
        if not ready:
            return False
        r = rng.choice(ready)
        if r < 0:
            bars[queue.pop(0)].arrive()
            continue
        try:
            waiting[r] = next(roles[r])
        except StopIteration:
            del waiting[r]
    return True


@pytest.mark.parametrize("tiles_of_rows", [1, 2])
def test_barriers_of_the_attention_end_in_any_order(tiles_of_rows):
    """Whatever role runs when, no wait misses its phase: with one barrier for
    the weights of one tile of rows, whose scores are two tiles ahead, one could."""
    import random
    for seed in range(300):
        rng = random.Random(seed)
        units = [rng.randrange(1, 9) for _ in range(rng.randrange(1, 7))]
        assert simulate(tiles_of_rows, units, seed), (units, seed)
