"""Cases of the block operators around the all-reduce: what is measured and in which sizes.

A tensor-parallel transformer block ends in an all-reduce; these are the operators on either side of it.

  join         the all-reduced block output y joins the residual stream x, and the next block's input is normalised:
                   n = norm(y) * w_post + b_post        (or n = y without the norm after the block)
                   r = x + scale * gate * n
                   h = norm(r) * w_pre + b_pre
               norm is v / rms(v) ("rms") or (v - mean(v)) / std(v) ("layer"), eps under the root.
  join_bwd     its gradients, from those of r and h: of x, y, the weights, the biases and the gate.
  linear8      x in 16 or 32 bits is quantised to int8, one scale a token (amax / 127), and multiplied with int8 weights
               that have one scale a channel; `ranks` products of one slice of x each, as in a row-parallel layer,
               whose results the all-reduce then adds.
  join_linear8 join whose h goes straight to int8 codes, and the product that reads them: one serving step between two blocks.

Plain form: elementary torch operations in 32 bits, rounded once at the end.  With `own` set, run() calls the library.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
TINY = 2.0 ** -110          # the smallest amax a token is scaled by


def listed():
    return [
        # one token of a decode loop between two blocks: latency only
        dict(name="join_decode_1", op="join", dtype="bf16", params="bf16", kind="rms", post=True, gate="none",
             tokens=1, width=4096, sequences=1, scale=1.0),
        # the forward pass of a training or prefill batch (the all-reduce workload of 8192 x 4096 per rank), with a layer scale
        dict(name="join_prefill_8192", op="join", dtype="bf16", params="bf16", kind="rms", post=True, gate="channel",
             tokens=8192, width=4096, sequences=1, scale=1.0),
        # an odd width, layer norms with biases, a gate row for each of 7 sequences, 32-bit training
        dict(name="join_ragged_f32", op="join", dtype="f32", params="f32", kind="layer", post=True, gate="channel",
             tokens=1001, width=1537, sequences=7, scale=0.25),
        # the backward pass of one such training batch
        dict(name="join_bwd_8192", op="join_bwd", dtype="bf16", params="bf16", kind="rms", post=True, gate="channel",
             tokens=8192, width=4096, sequences=1, scale=1.0),
        # small model, short odd sequences, fp16 with 32-bit parameters, modulated by a gate row per sequence
        dict(name="join_bwd_sequences", op="join_bwd", dtype="f16", params="f32", kind="layer", post=False, gate="channel",
             tokens=4 * 513, width=1024, sequences=4, scale=1.0),
        # the largest batch of the all-reduce workloads by tokens, a learned scalar gate a token
        dict(name="join_bwd_32768", op="join_bwd", dtype="bf16", params="f32", kind="rms", post=True, gate="scalar",
             tokens=32768, width=4096, sequences=32768, scale=0.5),
        # one token against a square weight: the decode loop's product
        dict(name="linear8_decode_1", op="linear8", dtype="bf16", ranks=1, tokens=1, channels=4096, depth=4096),
        # a small odd batch with sizes that are multiples of nothing, fp16
        dict(name="linear8_ragged", op="linear8", dtype="f16", ranks=1, tokens=203, channels=1111, depth=2051),
        # the row-parallel product that fills the four ranks' partial sums of the 2048 x 4096 all-reduce workload
        dict(name="linear8_rows_p4_2048", op="linear8", dtype="bf16", ranks=4, tokens=2048, channels=4096, depth=1024),
        # a prefill batch through a wide layer
        dict(name="linear8_prefill_8192", op="linear8", dtype="bf16", ranks=1, tokens=8192, channels=14336, depth=4096),
        # eight sequences in a decode loop, from one block's output to the next one's projections
        dict(name="step_decode_8", op="join_linear8", dtype="bf16", params="bf16", kind="rms", post=False, gate="none",
             tokens=8, width=4096, sequences=1, scale=1.0, channels=6144),
        # the same for a prefill chunk, sandwich norms
        dict(name="step_chunk_512", op="join_linear8", dtype="bf16", params="bf16", kind="rms", post=True, gate="none",
             tokens=512, width=4096, sequences=1, scale=1.0, channels=6144),
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
    op = rng.choice(["join", "join_bwd", "linear8", "join_linear8"])
    if op == "linear8":
        ranks = rng.choice([1, 1, 2, 4, 8])
        channels, depth = _size(rng, 256, 14336), _size(rng, 256, 8192)
        most = min(8192, 8192 * 14336 * 4096 // (ranks * channels * depth))
        return dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]), ranks=ranks, tokens=_log(rng, 1, most),
                    channels=channels, depth=depth)
    width = _size(rng, 256, 8192)
    most = 32768 * 4096 // width // (1 if op != "join_linear8" else 16)
    gate = "none" if op == "join_linear8" else rng.choice(["none", "channel", "channel", "scalar"])
    sequences = 1 if gate == "none" else rng.choice([1, 3, 16])
    if gate == "scalar" and rng.random() < 0.5:
        tokens = sequences = _log(rng, 1, min(most, 32768))
    else:
        tokens = sequences * _log(rng, 1, max(1, min(most, 32768) // sequences))
    dtype = rng.choice(["bf16", "f16"] if op == "join_linear8" else ["bf16", "f16", "f32"])
    case = dict(op=op, dtype=dtype, params=rng.choice([dtype, "f32"]), kind=rng.choice(["rms", "layer"]),
                post=rng.random() < 0.6, gate=gate, tokens=tokens, width=width, sequences=sequences,
                scale=rng.choice([1.0, 0.25]))
    if op == "join_linear8":
        case["channels"] = _size(rng, 256, 8192)
    return case


def work(case):
    e = {"bf16": 2, "f16": 2, "f32": 4}[case["dtype"]]
    if case["op"] == "linear8":
        m, n, k = case["tokens"], case["channels"], case["depth"]
        return {"bytes": case["ranks"] * (e * m * k + n * k + 4 * n + e * m * n), "flops": 2 * case["ranks"] * m * n * k}
    t, w = case["tokens"], case["width"]
    p = {"bf16": 2, "f16": 2, "f32": 4}[case["params"]]
    vectors = (1 + int(case["post"])) * (1 + int(case["kind"] == "layer"))
    gate = {"none": 0, "channel": case["sequences"] * w, "scalar": case["sequences"]}[case["gate"]]
    small = p * (vectors * w + gate)
    if case["op"] == "join":                       # x, y read; r, h written
        return {"bytes": 4 * e * t * w + small, "flops": 12 * t * w}
    if case["op"] == "join_bwd":                   # x, y and the gradients of r, h read; those of x, y and the parameters written
        return {"bytes": 6 * e * t * w + 16 * t + 2 * small, "flops": 30 * t * w}
    n = case["channels"]                           # x, y, the weights read; r and the product written
    return {"bytes": 3 * e * t * w + small + n * w + 4 * n + e * t * n, "flops": 2 * t * n * w}


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _activations(gen, tokens, width):
    """Normal values on channels of unequal scale, 1% of the channels 20 times larger."""
    scale = torch.exp(0.5 * _normal(gen, width))
    loud = torch.rand(width, generator=gen, device="cuda") < 0.01
    return _normal(gen, tokens, width) * torch.where(loud, 20 * scale, scale)


def _weights8(gen, ranks, channels, depth):
    """int8 codes of normal weights with one scale a channel, and the scales."""
    codes = torch.empty(ranks, channels, depth, dtype=torch.int8, device="cuda")
    scales = torch.empty(ranks, channels, device="cuda")
    for p in range(ranks):
        w = _normal(gen, channels, depth) * (0.5 / math.sqrt(depth))
        scales[p] = w.abs().amax(1) / 127
        codes[p] = torch.round(w / scales[p][:, None]).to(torch.int8)
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "linear8":
        ranks, m, n, k = case["ranks"], case["tokens"], case["channels"], case["depth"]
        # one row holds the ranks' slices side by side, as the layer before leaves it
        s["x"] = _activations(gen, m, ranks * k).to(dt).view(m, ranks, k).transpose(0, 1)
        s["w"], s["w_scales"] = _weights8(gen, ranks, n, k)
        if own:                                    # the buffers that a program keeps for its layer
            s["codes"] = torch.empty(ranks, m, k, dtype=torch.int8, device="cuda")
            s["scales"] = torch.empty(ranks, m, device="cuda")
            s["out"] = torch.empty(ranks, m, n, dtype=dt, device="cuda")
        return s
    t, w, pt = case["tokens"], case["width"], DTYPES[case["params"]]
    s["x"] = (3 * _activations(gen, t, w)).to(dt)
    s["y"] = _activations(gen, t, w).to(dt)
    one = lambda: (1 + 0.1 * _normal(gen, w)).to(pt)                              # noqa: E731
    small = lambda: (0.1 * _normal(gen, w)).to(pt)                                # noqa: E731
    layer = case["kind"] == "layer"
    s["w_pre"], s["b_pre"] = one(), small() if layer else None
    s["w_post"] = one() if case["post"] else None
    s["b_post"] = small() if case["post"] and layer else None
    g = {"none": None, "channel": (case["sequences"], w), "scalar": (case["sequences"], 1)}[case["gate"]]
    s["gate"] = None if g is None else (0.5 + 0.2 * _normal(gen, *g)).to(pt)
    if case["op"] == "join_linear8":
        codes, scales = _weights8(gen, 1, case["channels"], w)
        s["w"], s["w_scales"] = codes[0], scales[0]
    if case["op"] == "join_bwd":
        s["dr"] = (0.01 * _normal(gen, t, w)).to(dt)
        s["dh"] = (0.01 * _normal(gen, t, w)).to(dt)
        s["stats"] = _plain_join(s)[2]             # kept from the forward pass: mean and 1/deviation of each norm
    if own:
        _keep(s)
    return s


def _keep(s):
    """The plan, the parameters' handle and the output buffers that a program makes once."""
    from bit_error_compensated_gb300 import echo
    case = s["case"]
    kind = {"rms": echo.ECHO_NORM_RMS, "layer": echo.ECHO_NORM_LAYER}[case["kind"]]
    s["plan"] = echo.echo_norm_plan(case["width"], DTYPES[case["dtype"]], DTYPES[case["params"]], kind=kind,
                                    post=case["post"], eps=EPS, scale=case["scale"])
    names = [n for n in ("w_post", "b_post", "w_pre", "b_pre") if s[n] is not None]
    s["params"] = echo.NormParams(s["plan"], **{n: s[n] for n in names})
    if case["op"] == "join_bwd":
        s["dx"], s["dy"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
        s["d"] = {n: torch.empty_like(s[n]) for n in names}
        s["dparams"] = echo.NormParams(s["plan"], **s["d"])
        s["dgate"] = None if s["gate"] is None else torch.empty_like(s["gate"])
    else:
        s["r"] = torch.empty_like(s["x"])
    if case["op"] == "join":
        s["h"] = torch.empty_like(s["x"])
    if case["op"] == "join_linear8":
        s["codes"] = torch.empty(s["x"].shape, dtype=torch.int8, device="cuda")
        s["scales"] = torch.empty(case["tokens"], device="cuda")
        s["out"] = torch.empty(case["tokens"], case["channels"], dtype=DTYPES[case["dtype"]], device="cuda")


def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(s, op)
    dt = DTYPES[s["case"]["dtype"]]
    if op == "linear8":
        return _plain_product(s["x"].float(), s["w"], s["w_scales"]).to(dt)
    if op == "join_bwd":
        return _plain_backward(s)
    r, h, _ = _plain_join(s)
    if op == "join":
        return r.to(dt), h.to(dt)
    return r.to(dt), _plain_product(h, s["w"], s["w_scales"]).to(dt)


def _run_own(s, op):
    from bit_error_compensated_gb300 import echo
    if op == "linear8":
        echo.echo_linear_int8(s["x"], s["w"], s["w_scales"], s["out"], s["codes"], s["scales"])
        return s["out"]
    if op == "join":
        echo.echo_norm(s["plan"], s["params"], s["x"], s["y"], s["r"], s["h"], gate=s["gate"])
        return s["r"], s["h"]
    if op == "join_bwd":
        echo.echo_norm_backward(s["plan"], s["params"], s["x"], s["y"], s["stats"], s["dr"], s["dh"],
                                s["dx"], s["dy"], s["dparams"], gate=s["gate"], dgate=s["dgate"])
        return dict(s["d"], x=s["dx"], y=s["dy"], **({} if s["dgate"] is None else {"gate": s["dgate"]}))
    echo.echo_norm(s["plan"], s["params"], s["x"], s["y"], s["r"], None, codes=s["codes"], scales=s["scales"])
    echo.echo_matmul_int8(s["codes"], s["scales"], s["w"], s["w_scales"], s["out"])
    return s["r"], s["out"]


def _plain_norm(v, kind, weight, bias):
    mean = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    c = v - mean
    rstd = torch.rsqrt((c * c).mean(1, keepdim=True) + EPS)
    n = c * rstd * weight.float()
    return (n if bias is None else n + bias.float()), mean, rstd


def _plain_gate(s):
    """The gate as one row a token (or one row for all of them)."""
    if s["gate"] is None:
        return 1.0
    g = s["gate"].float()
    return g if g.shape[0] == 1 else g.repeat_interleave(s["case"]["tokens"] // g.shape[0], 0)


def _plain_join(s):
    case, x, n = s["case"], s["x"].float(), s["y"].float()
    mean1, rstd1 = torch.zeros_like(x[:, :1]), torch.ones_like(x[:, :1])
    if case["post"]:
        n, mean1, rstd1 = _plain_norm(n, case["kind"], s["w_post"], s["b_post"])
    r = x + case["scale"] * _plain_gate(s) * n
    h, mean2, rstd2 = _plain_norm(r, case["kind"], s["w_pre"], s["b_pre"])
    return r, h, torch.cat([mean1, rstd1, mean2, rstd2], 1)


def _plain_norm_backward(d, hat, rstd, kind):
    out = d - hat * (d * hat).mean(1, keepdim=True)
    return rstd * (out - d.mean(1, keepdim=True) if kind == "layer" else out)


def _plain_backward(s):
    case, got = s["case"], {}
    dt, pt, kind = DTYPES[case["dtype"]], DTYPES[case["params"]], case["kind"]
    mean1, rstd1, mean2, rstd2 = s["stats"].split(1, 1)
    x, y, dh, gate = s["x"].float(), s["y"].float(), s["dh"].float(), _plain_gate(s)
    hat1 = n = y
    if case["post"]:
        hat1 = (y - mean1) * rstd1
        n = hat1 * s["w_post"].float() + (0.0 if s["b_post"] is None else s["b_post"].float())
    hat2 = (x + case["scale"] * gate * n - mean2) * rstd2
    got["w_pre"] = (dh * hat2).sum(0).to(pt)
    if s["b_pre"] is not None:
        got["b_pre"] = dh.sum(0).to(pt)
    d = s["dr"].float() + _plain_norm_backward(dh * s["w_pre"].float(), hat2, rstd2, kind)
    got["x"] = d.to(dt)
    if s["gate"] is not None:
        dg = (case["scale"] * d * n).view(case["sequences"], -1, case["width"]).sum(1)
        got["gate"] = (dg.sum(1, keepdim=True) if s["gate"].shape[1] == 1 else dg).to(pt)
    dn = case["scale"] * gate * d
    if case["post"]:
        got["w_post"] = (dn * hat1).sum(0).to(pt)
        if s["b_post"] is not None:
            got["b_post"] = dn.sum(0).to(pt)
        dn = _plain_norm_backward(dn * s["w_post"].float(), hat1, rstd1, kind)
    got["y"] = dn.to(dt)
    return got


def _plain_product(x, w, w_scales):
    amax = x.abs().amax(-1, keepdim=True).clamp_min(TINY)
    top = torch.full_like(amax, 127.0)       # a tensor: true divisions, no reciprocal of a constant
    q = torch.round(x * (top / amax))
    return torch.matmul(q, w.float().transpose(-1, -2)) * (amax / top) * w_scales.unsqueeze(-2)


def exact(case, seed):
    """The definition in 64 bits; the gradients by automatic differentiation of it."""
    s = prepare(case, seed)
    to = lambda v: None if v is None else v.double()                              # noqa: E731
    if case["op"] == "linear8":
        return _exact_product(to(s["x"]), s)
    training = case["op"] == "join_bwd"
    leaf = {n: to(s[n]) for n in ("x", "y", "w_post", "b_post", "w_pre", "b_pre", "gate")}
    leaf = {n: v.requires_grad_(training) for n, v in leaf.items() if v is not None}
    norm = torch.nn.functional.layer_norm if case["kind"] == "layer" else None

    def normed(v, at):
        if norm is not None:
            return norm(v, (case["width"],), leaf["w_" + at], leaf["b_" + at], EPS)
        return v / torch.sqrt(v.square().sum(1, keepdim=True) / case["width"] + EPS) * leaf["w_" + at]

    n = normed(leaf["y"], "post") if case["post"] else leaf["y"]
    if "gate" in leaf:
        shape = (case["sequences"], case["tokens"] // case["sequences"], case["width"])
        n = (n.view(shape) * leaf["gate"].unsqueeze(1)).view(case["tokens"], case["width"])
    r = leaf["x"] + n * case["scale"]
    h = normed(r, "pre")
    if training:
        grads = torch.autograd.grad([r, h], list(leaf.values()), [to(s["dr"]), to(s["dh"])])
        return dict(zip(leaf, grads))
    return (r, h) if case["op"] == "join" else (r, _exact_product(h, s))


def _exact_product(x, s):
    step = x.abs().amax(-1, keepdim=True).clamp_min(TINY) / 127
    codes = torch.round(x / step)
    return torch.einsum("...mk,...nk->...mn", codes, s["w"].double()) * step * s["w_scales"].double().unsqueeze(-2)
