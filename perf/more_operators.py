"""Cases of the operators of a serving step: what is measured and in which sizes.

Between two all-reduces of a tensor-parallel block that serves a model, the ranks' heads attend over a cache that is kept in
the library's 4- or 8-bit groups, and few tokens are multiplied with weights in the same 4-bit groups.

  cache        keys and values of new tokens are quantised into a paged cache, a head's row one group (fp16 step s and
               zero point z: lo = min(0, min v), hi = max(0, max v), s = (hi - lo) / (2^b - 1) rounded up to fp16,
               z = rint(-lo / s), code = clamp(rint(v / s) + z, 0, 2^b - 1)), and read back as s * (code - z).
               The quotients are rounded as exact numbers: the plain form takes them in 64 bits.
  attention    new tokens, which are the last of their sequences, attend over those sequences' pages:
                   out = softmax(scale * q k^T) v    over the keys up to each token's own place (or the last `window`)
               with `group` query heads to a head of the cache.
  linear4      out = x w^T for weights in 4-bit groups along their depth.
  load4        weights in 16 or 32 bits are quantised to such groups, and a first product is made with them.

Plain form: elementary torch operations in 32 bits, rounded once at the end.  With `own` set, run() calls the library.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one decode step of 64 sequences: a token each is written to the cache (and read back); latency only
        dict(name="cache_decode_64", op="cache", dtype="bf16", bits=8, heads=8, dim=128, page=64, sequences=64, new=1,
             context=1000, pattern=1),
        # the prompt of one sequence, 4 bits
        dict(name="cache_prefill_8192", op="cache", dtype="bf16", bits=4, heads=8, dim=128, page=64, sequences=1, new=8192,
             context=0, pattern=2),
        # one token of one sequence over a short cache: latency
        dict(name="attention_decode_1", op="attention", dtype="bf16", bits=4, heads=8, group=4, dim=128, page=64,
             sequences=1, new=1, context=1999, ragged=False, window=0, pattern=3),
        # a decode step of 64 sequences of unequal length, 4 bits
        dict(name="attention_decode_64", op="attention", dtype="bf16", bits=4, heads=8, group=4, dim=128, page=64,
             sequences=64, new=1, context=16384, ragged=True, window=0, pattern=4),
        # four very long sequences, 8 bits
        dict(name="attention_decode_long", op="attention", dtype="f16", bits=8, heads=8, group=5, dim=128, page=256,
             sequences=4, new=1, context=131071, ragged=False, window=0, pattern=5),
        # verification of five drafted tokens a sequence, seven query heads to a small head of the cache
        dict(name="attention_draft_16", op="attention", dtype="bf16", bits=8, heads=4, group=7, dim=64, page=16,
             sequences=16, new=5, context=6000, ragged=True, window=0, pattern=6),
        # chunks of long prompts, 4 bits
        dict(name="attention_chunk_512", op="attention", dtype="bf16", bits=4, heads=8, group=4, dim=128, page=64,
             sequences=4, new=512, context=16000, ragged=True, window=0, pattern=7),
        # a whole prompt over its own cache, 8 bits
        dict(name="attention_prefill_8192", op="attention", dtype="bf16", bits=8, heads=8, group=4, dim=128, page=64,
             sequences=1, new=8192, context=0, ragged=False, window=0, pattern=8),
        # one token against a square weight: the decode loop's product
        dict(name="linear4_decode_1", op="linear4", dtype="bf16", ranks=1, tokens=1, channels=4096, depth=4096, group=128),
        # sixteen sequences, the row-parallel product that fills four ranks' partial sums
        dict(name="linear4_rows_p4_16", op="linear4", dtype="bf16", ranks=4, tokens=16, channels=4096, depth=1024, group=128),
        # a wide layer is loaded, then 32 sequences' next tokens
        dict(name="load4_wide_32", op="load4", dtype="bf16", ranks=1, tokens=32, channels=14336, depth=4096, group=128),
        # odd sizes in 32 bits, small groups
        dict(name="load4_ragged", op="load4", dtype="f32", ranks=1, tokens=7, channels=1111, depth=2051, group=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size in [lo, hi]: half of them multiples of 256, the others odd."""
    if rng.random() < 0.5:
        pool = [v for v in (256, 512, 768, 1024, 1536, 2048, 2560, 3584, 4096, 5120, 6144, 7168, 8192, 11008, 14336)
                if lo <= v <= hi]
        return rng.choice(pool)
    return min(_log(rng, lo, hi) | 1, hi - 1 | 1)


def draw(rng):
    op = rng.choice(["cache", "attention", "attention", "attention", "linear4", "load4"])
    if op in ("linear4", "load4"):
        case = dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]), ranks=rng.choice([1, 1, 2, 4]), tokens=_log(rng, 1, 64),
                    channels=_size(rng, 256, 14336), depth=_size(rng, 256, 8192), group=rng.choice([64, 128, 128, 256]))
        while case["ranks"] * case["channels"] * case["depth"] * case["tokens"] > 14336 * 4096 * 32:
            case.update(ranks=1, channels=_size(rng, 256, 8192), depth=_size(rng, 256, 4096), tokens=_log(rng, 1, 48))
        return case
    dim = rng.choice([64, 128, 128, 256])
    case = dict(op=op, dtype=rng.choice(["bf16", "f16"]), bits=rng.choice([4, 8]), heads=rng.choice([1, 2, 4, 5, 8]),
                dim=dim, page=rng.choice([16, 32, 64, 128, 256]), sequences=_log(rng, 1, 64), pattern=rng.randrange(1 << 20))
    if op == "cache":
        case["dtype"] = rng.choice(["bf16", "f16", "f32"])
        most = 8192 * 8 * 128 // (case["sequences"] * case["heads"] * dim)
        case.update(new=_log(rng, 1, max(1, most)), context=_log(rng, 1, 4000) - 1)
        return case
    case["group"] = rng.choice([1, 3, 4, 5, 7, 8, 16])
    kind = rng.choice(["decode", "draft", "chunk", "prompt"])
    keys = 4 * 131071 * 8 * 128 // (case["heads"] * dim)         # that a case's caches hold at the most
    if kind in ("decode", "draft"):
        new = 1 if kind == "decode" else rng.randrange(2, 9)
        context = _log(rng, 1, min(131071, keys // case["sequences"]))
    else:
        case["sequences"] = _log(rng, 1, 8)
        new = _log(rng, 16, 8192)
        context = 0 if kind == "prompt" else _log(rng, 256, 32768)
        pairs = 8192 * 8192 // 2 * 32 * 128 // (case["heads"] * case["group"] * dim * case["sequences"])
        while new * (context + new // 2) > pairs or (context + new) * case["sequences"] > keys:
            new, context = max(1, new // 2), context * 3 // 4
    case.update(new=new, context=context, ragged=rng.random() < 0.6, window=rng.choice([0, 0, 0, _log(rng, 1, 8192)]))
    return case


def _lengths(case):
    """(new tokens, tokens in the cache with them) of each sequence, by the case alone."""
    rng = random.Random(case["pattern"])
    out = []
    for _ in range(case["sequences"]):
        new, context = case["new"], case["context"]
        if case.get("ragged"):
            context = rng.randint(context // 4, context)
            new = new if new <= 8 else rng.randint((new + 1) // 2, new)
        out.append((new, context + new))
    return out


def _pairs(case):
    """Pairs of a new token and a key that it sees."""
    total = 0
    for new, length in _lengths(case):
        window = case["window"] or length
        first = length - new + 1                                 # keys that the first new token could see
        full = max(0, length - max(first, window + 1) + 1)       # tokens that see a whole window and could see more
        rest = new - full
        total += full * window + rest * first + rest * (rest - 1) // 2
    return total


def _keys(case):
    """Keys that any new token sees, over the sequences."""
    return sum(min(length, (case["window"] or length) + new - 1) for new, length in _lengths(case))


def work(case):
    e = BYTES[case["dtype"]]
    if case["op"] in ("linear4", "load4"):
        p, m, n, k = case["ranks"], case["tokens"], case["channels"], case["depth"]
        packed = n * ((k + 1) // 2 + 4 * ((k + case["group"] - 1) // case["group"]))
        weights = packed + (e * n * k if case["op"] == "load4" else 0)
        return {"bytes": p * (e * m * (k + n) + weights), "flops": 2 * p * m * n * k}
    row = case["dim"] * case["bits"] // 8 + 4                    # a head's keys or values of a token in the cache
    tokens = sum(new for new, _ in _lengths(case))
    if case["op"] == "cache":
        values = 2 * tokens * case["heads"] * case["dim"]
        return {"bytes": 2 * e * values + 2 * tokens * case["heads"] * row, "flops": 10 * values}
    heads = case["heads"] * case["group"]
    return {"bytes": 2 * e * tokens * heads * case["dim"] + 2 * _keys(case) * case["heads"] * row,
            "flops": 4 * _pairs(case) * heads * case["dim"]}


# ------------------------------------------------------------------ inputs
def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _loud(gen, width):
    """Channels of unequal scale, 2% of them 8 times larger."""
    scale = torch.exp(0.3 * _normal(gen, width))
    return torch.where(torch.rand(width, generator=gen, device="cuda") < 0.02, 8 * scale, scale)


def _quantise(v, bits):
    """Codes, steps and zero points of groups along the last dimension; quotients in 64 bits, for values next to a border."""
    v, top = v.double(), 2 ** bits - 1
    low, high = v.amin(-1, keepdim=True).clamp_max(0), v.amax(-1, keepdim=True).clamp_min(0)
    wide = (high - low) / torch.full_like(low, top)              # a tensor: true divisions
    step = wide.half()
    step = (step.view(torch.int16) + (step.double() < wide).to(torch.int16)).view(torch.float16).double()
    step = torch.where(step == 0, torch.ones_like(step), step)
    zero = torch.round(-low / step).clamp(0, top)
    return (torch.round(v / step) + zero).clamp(0, top), step, zero


def _pack(codes, bits):
    codes = codes.to(torch.uint8)
    return codes if bits == 8 else codes[..., 0::2] | codes[..., 1::2] << 4


def _meta(step, zero):
    """One word a group: the step in the low half, the zero point in the high one."""
    return torch.cat([step, zero], -1).half().view(torch.int32).squeeze(-1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] in ("linear4", "load4"):
        _prepare_linear(case, gen, dt, s)
        return s
    lengths = _lengths(case)
    tokens, heads, dim = sum(new for new, _ in lengths), case["heads"], case["dim"]
    each = [(length + case["page"] - 1) // case["page"] for _, length in lengths]
    pages = sum(each) + 3                                        # the pool holds a few that no sequence has
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    s["table"] = torch.zeros(len(lengths), max(each), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(each):
        s["table"][b, :n] = order[at:at + n]
        at += n
    starts = [0]
    for new, _ in lengths:
        starts.append(starts[-1] + new)
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["lengths"] = torch.tensor([length for _, length in lengths], dtype=torch.int32, device="cuda")
    s["codes"] = torch.zeros(pages, 2, heads, case["page"], dim * case["bits"] // 8, dtype=torch.uint8, device="cuda")
    s["meta"] = torch.zeros(pages, 2, heads, case["page"], dtype=torch.int32, device="cuda")
    loud = torch.stack([_loud(gen, heads * dim).view(heads, 1, dim), torch.ones(heads, 1, dim, device="cuda")])
    if case["op"] == "cache":
        # keys and values as a projection leaves them: parts of one row a token
        rows = _normal(gen, tokens, 2, heads, dim) * loud.view(2, heads, dim)
        s["k"], s["v"] = rows.to(dt).unbind(1)
        if own:
            s["k_back"], s["v_back"] = (torch.empty(tokens, heads, dim, dtype=dt, device="cuda") for _ in range(2))
    else:
        some = max(1, (1 << 25) // (2 * heads * case["page"] * dim))
        for p in range(0, pages, some):
            n = min(some, pages - p)
            codes, step, zero = _quantise(_normal(gen, n, 2, heads, case["page"], dim) * loud, case["bits"])
            s["codes"][p:p + n], s["meta"][p:p + n] = _pack(codes, case["bits"]), _meta(step, zero)
        s["q"] = (1.5 * _normal(gen, tokens, heads * case["group"], dim)).to(dt)
        if own:
            s["out"] = torch.empty_like(s["q"])
    if own:                                                      # the cache and the batch that a program keeps
        from bit_error_compensated_gb300 import echo
        s["cache"] = echo.Cache(pages, case["page"], heads, dim, case["bits"], codes=s["codes"], meta=s["meta"])
        s["batch"] = echo.CacheBatch(s["starts"], s["lengths"], s["table"])
    return s


def _prepare_linear(case, gen, dt, s):
    p, m, n, k, group = case["ranks"], case["tokens"], case["channels"], case["depth"], case["group"]
    # one row holds the ranks' slices side by side, as the layer before leaves it
    s["x"] = (_normal(gen, m, p * k) * _loud(gen, p * k)).to(dt).view(m, p, k).transpose(0, 1)
    w = _normal(gen, p, n, k) * (_loud(gen, n)[:, None] / math.sqrt(k))
    if case["op"] == "load4":
        s["w"] = w.to(dt)
    if case["op"] == "linear4":
        s["codes"], s["meta"] = _pack_weights(w, group)
    elif own:
        s["codes"] = torch.empty(p, n, (k + 1) // 2, dtype=torch.uint8, device="cuda")
        s["meta"] = torch.empty(p, n, (k + group - 1) // group, dtype=torch.int32, device="cuda")
    if own:
        s["out"] = torch.empty(p, m, n, dtype=dt, device="cuda")


def _pack_weights(w, group):
    """Codes [ranks][channels][depth / 2, rounded up] and a word for each group along the depth (the last may be shorter)."""
    p, n, k = w.shape
    padded = torch.nn.functional.pad(w, (0, -k % group))         # zeros, which every range holds anyway
    codes, step, zero = _quantise(padded.view(p, n, -1, group), 4)
    codes = codes.view(p, n, -1)[..., :k]
    return _pack(torch.nn.functional.pad(codes, (0, k % 2)), 4), _meta(step, zero)


# --------------------------------------------------------------- the passes
def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(s, op)
    if op == "cache":
        return _plain_cache(s)
    if op == "attention":
        return _plain_attention(s)
    if op == "load4":
        return _plain_product(s, *_pack_weights(s["w"], s["case"]["group"]))
    return _plain_product(s, s["codes"], s["meta"])


def _run_own(s, op):
    from bit_error_compensated_gb300 import echo
    if op == "cache":
        echo.echo_cache_append(s["cache"], s["batch"], s["k"], s["v"])
        echo.echo_cache_read(s["cache"], s["batch"], s["k_back"], s["v_back"])
        return {"k": s["k_back"], "v": s["v_back"]}
    if op == "attention":
        echo.echo_attention(s["cache"], s["batch"], s["q"], s["out"], window=s["case"]["window"])
        return s["out"]
    if op == "load4":
        echo.echo_quantize_weights(s["w"], s["codes"], s["meta"], group=s["case"]["group"])
    echo.echo_linear_int4(s["x"], s["codes"], s["meta"], s["out"], group=s["case"]["group"])
    return s["out"]


def _values(codes, meta, bits):
    """s * (code - z) in 32 bits of packed codes [..., bytes] and words [...]."""
    if bits == 4:
        codes = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    both = meta.contiguous().view(torch.float16).view(*meta.shape, 2).float()
    return both[..., :1] * (codes.float() - both[..., 1:])


def _places(s):
    """Page and place in it of each new token."""
    case, page, place = s["case"], [], []
    for b, (new, length) in enumerate(_lengths(case)):
        at = torch.arange(length - new, length, device="cuda")
        page.append(s["table"][b][at // case["page"]].long())
        place.append(at % case["page"])
    return torch.cat(page), torch.cat(place)


def _plain_cache(s):
    bits, dt = s["case"]["bits"], DTYPES[s["case"]["dtype"]]
    page, place = _places(s)
    back = {}
    for i, name in enumerate(("k", "v")):
        codes, step, zero = _quantise(s[name].float(), bits)
        s["codes"][page, i, :, place] = _pack(codes, bits)
        s["meta"][page, i, :, place] = _meta(step, zero)
    for i, name in enumerate(("k", "v")):
        back[name] = _values(s["codes"][page, i, :, place], s["meta"][page, i, :, place], bits).to(dt)
    return back


def _plain_attention(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    heads, group, dim = case["heads"], case["group"], case["dim"]
    out, at = torch.empty_like(s["q"]), 0
    for b, (new, length) in enumerate(_lengths(case)):
        pages = s["table"][b, :(length + case["page"] - 1) // case["page"]].long()
        for h in range(heads):
            k, v = (_values(s["codes"][pages, i, h], s["meta"][pages, i, h], case["bits"]).view(-1, dim)[:length]
                    for i in (0, 1))
            some = max(1, (1 << 27) // (group * length))
            for t in range(0, new, some):
                n = min(some, new - t)
                q = s["q"][at + t:at + t + n, h * group:(h + 1) * group].float().reshape(n * group, dim)
                score = (q @ k.T) * (1 / math.sqrt(dim))
                own_place = torch.arange(length - new + t, length - new + t + n, device="cuda").repeat_interleave(group)[:, None]
                key = torch.arange(length, device="cuda")
                hidden = key > own_place
                if case["window"]:
                    hidden |= key <= own_place - case["window"]
                score.masked_fill_(hidden, -math.inf)
                weight = torch.exp(score - score.amax(1, keepdim=True))
                got = (weight @ v) / weight.sum(1, keepdim=True)
                out[at + t:at + t + n, h * group:(h + 1) * group] = got.view(n, group, dim).to(dt)
        at += new
    return out


def _plain_product(s, codes, meta):
    k, group = s["case"]["depth"], s["case"]["group"]
    padded = torch.nn.functional.pad(codes, (0, (meta.shape[-1] * group) // 2 - codes.shape[-1]))
    w = _values(padded.view(*meta.shape, group // 2), meta, 4).flatten(-2)[..., :k]
    return (s["x"].float() @ w.transpose(-1, -2)).to(DTYPES[s["case"]["dtype"]])


# ------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "cache":
        return {name: _exact_groups(s[name].double(), case["bits"]) for name in ("k", "v")}
    if case["op"] == "attention":
        return _exact_attention(case, s)
    n, k, group = case["channels"], case["depth"], case["group"]
    out = []
    for p in range(case["ranks"]):
        w = torch.zeros(n, k, dtype=torch.float64, device="cuda")
        for g, first in enumerate(range(0, k, group)):
            last = min(k, first + group)
            if case["op"] == "load4":
                w[:, first:last] = _exact_groups(s["w"][p, :, first:last].double(), 4)
            else:
                word = s["meta"][p, :, g].long() & 0xFFFFFFFF
                step, zero = _half_bits(word & 0xFFFF), _half_bits(word >> 16)
                for i in range(first, last):
                    code = (s["codes"][p, :, i // 2].long() >> (4 * (i % 2))) & 15
                    w[:, i] = step * (code.double() - zero)
        out.append(torch.einsum("mk,nk->mn", s["x"][p].double(), w))
    return torch.stack(out)


def _power(exponent):
    """2 to whole numbers, exactly."""
    return (exponent.long() + 1023 << 52).view(torch.float64)


def _half_bits(word):
    """The values of fp16 numbers given as whole numbers: sign, exponent, fraction."""
    sign, exponent, fraction = 1 - 2 * (word >> 15), word >> 10 & 31, word & 1023
    normal = _power(exponent - 25) * (1024 + fraction)
    return sign * torch.where(exponent == 0, fraction * 2.0 ** -24, normal)


def _exact_groups(v, bits):
    """What groups along the last dimension are read back as."""
    most = 2 ** bits - 1
    low, high = -torch.relu(-v.amin(-1)), torch.relu(v.amax(-1))
    step = (high - low) / torch.full_like(high, most)         # a true division
    unit = _power(torch.frexp(step.clamp_min(2.0 ** -14)).exponent - 11)                # spacing of fp16 there
    step = torch.where(step > 0, torch.ceil(step / unit) * unit, 1.0).unsqueeze(-1)
    zero = torch.round(-low.unsqueeze(-1) / step).clamp(0, most)
    return step * (torch.clamp(torch.round(v / step), -zero, most - zero))


def _exact_attention(case, s):
    heads, group, dim, size = case["heads"], case["group"], case["dim"], case["page"]
    q = s["q"].double().unflatten(1, (heads, group))
    out, row = torch.zeros_like(q), 0
    for b, (new, length) in enumerate(_lengths(case)):
        place = torch.arange(length, device="cuda")
        page = s["table"][b].long()[place // size]
        for h in range(heads):
            kv = []
            for i in range(2):
                code = s["codes"][page, i, h, place % size].long()
                if case["bits"] == 4:
                    code = torch.stack([code % 16, code // 16], 2).reshape(length, dim)
                word = s["meta"][page, i, h, place % size].long() & 0xFFFFFFFF
                kv.append((code - _half_bits(word >> 16)[:, None]) * _half_bits(word & 0xFFFF)[:, None])
            for t in range(0, new, 512):
                n = min(512, new - t)
                mine = length - new + t + torch.arange(n, device="cuda")
                seen = place[None] <= mine[:, None]
                if case["window"]:
                    seen &= place[None] > mine[:, None] - case["window"]
                score = torch.einsum("tgd,sd->tgs", q[row + t:row + t + n, h], kv[0]) / math.sqrt(dim)
                weight = torch.softmax(score.masked_fill(~seen[:, None], -math.inf), -1)
                out[row + t:row + t + n, h] = torch.einsum("tgs,sd->tgd", weight, kv[1])
        row += new
    return out.flatten(1, 2)
