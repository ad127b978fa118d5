"""echo_norm and echo_norm_backward against the formulas in 64 bits
(_block_ref.py: values and error bounds), element by element."""
import itertools

import pytest
import torch

import _block_ref as ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
RMS, LAYER = 0, 1
EPS = 1e-5


def make(rows, width, dtype, pdtype, kind, post, gate, seed, ld=None, offset=0, biases=True):
    """Inputs of one call; ld/offset: row distance and start of every row tensor."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    ld = width if ld is None else ld
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")               # noqa: E731

    def rows_of(scale):
        t = torch.zeros(rows * ld + offset, dtype=dtype, device="cuda")
        view = t[offset:].view(rows, ld)[:, :width] if rows else t[offset:].view(0, ld)[:, :width]
        view.copy_(rand(rows, width) * scale * torch.exp(0.5 * rand(width)))
        return view

    v = {"x": rows_of(3.0), "y": rows_of(1.0), "dr": rows_of(0.1), "dh": rows_of(0.1)}
    p = {"w_pre": (1 + 0.1 * rand(width)).to(pdtype)}
    if post:
        p["w_post"] = (1 + 0.1 * rand(width)).to(pdtype)
    if kind == LAYER and biases:
        p["b_pre"] = (0.1 * rand(width)).to(pdtype)
        if post:
            p["b_post"] = (0.1 * rand(width)).to(pdtype)
    v["gate"] = None if gate is None else (0.5 + 0.3 * rand(*gate)).to(pdtype)
    return v, p


def dbl(t):
    return None if t is None else t.double()


def like(t):
    """An empty tensor with the row distance and start of t."""
    base = torch.empty(t.storage_offset() + t.shape[0] * t.stride(0) if t.shape[0] else 1,
                       dtype=t.dtype, device=t.device)
    base.fill_(float("nan"))
    return base.as_strided(t.shape, t.stride(), t.storage_offset() if t.shape[0] else 0)


def call_forward(v, p, width, dtype, pdtype, kind, post, scale, codes=False):
    from bit_error_compensated_gb300 import echo
    plan = echo.echo_norm_plan(width, dtype, pdtype, kind=kind, post=post, eps=EPS, scale=scale)
    params = echo.NormParams(plan, **p)
    rows = v["x"].shape[0]
    r, h = like(v["x"]), like(v["x"])
    stats = torch.empty(rows, 4, device="cuda")
    c = torch.empty(rows, width, dtype=torch.int8, device="cuda") if codes else None
    s = torch.empty(rows, device="cuda") if codes else None
    echo.echo_norm(plan, params, v["x"], v["y"], r, h, gate=v["gate"], codes=c, scales=s, stats=stats)
    return plan, params, r, h, stats, c, s


def check_forward(v, p, width, dtype, pdtype, kind, post, scale):
    plan, params, r, h, stats, c, s = call_forward(v, p, width, dtype, pdtype, kind, post, scale, codes=True)
    torch.cuda.synchronize()
    want_r, want_h, want_stats, err_r, err_h = ref.forward(
        kind, post, EPS, scale, dbl(v["x"]), dbl(v["y"]), dbl(v["gate"]), {k: t.double() for k, t in p.items()})
    ref.within(r, want_r, err_r, "r")
    ref.within(h, want_h, err_h, "h")
    # codes: the value each stands for is within half a step (and the error of h) of h
    if r.shape[0]:
        top = want_h.abs().amax(1)
        assert ((s.double() * 127 - top).abs() <= err_h.amax(1) + 2e-7 * top).all()
        off = (c.double() * s.double()[:, None] - want_h).abs()
        assert (off <= s.double()[:, None] * 0.500001 + err_h + 2e-7 * want_h.abs()).all()
    return plan, params, stats


def check_backward(v, p, plan, params, stats, width, pdtype, kind, post, scale, dr=True, dh=True):
    from bit_error_compensated_gb300 import echo
    dx, dy = like(v["x"]), like(v["x"])
    d = {k: torch.full_like(t, float("nan")) for k, t in p.items()}
    dgate = None if v["gate"] is None else torch.full_like(v["gate"], float("nan"))
    grads = echo.NormParams(plan, **d)
    for _ in range(2):
        echo.echo_norm_backward(plan, params, v["x"], v["y"], stats, v["dr"] if dr else None,
                                v["dh"] if dh else None, dx, dy, grads, gate=v["gate"], dgate=dgate)
        first = [t.clone() for t in (dx, dy, *d.values())] if _ == 0 else first     # noqa: F821
    torch.cuda.synchronize()
    for a, b in zip(first, (dx, dy, *d.values())):
        assert torch.equal(a, b), "a repeated call gives other bits"
    want = ref.backward(kind, post, EPS, scale, dbl(v["x"]), dbl(v["y"]), dbl(v["gate"]),
                        {k: t.double() for k, t in p.items()}, dbl(v["dr"]) if dr else None,
                        dbl(v["dh"]) if dh else None)
    for name, got in [("x", dx), ("y", dy), ("gate", dgate), *d.items()]:
        if got is not None:
            ref.within(got, *want[name], f"d{name}")


CASES = [
    # rows, width, dtype, pdtype, kind, post, gate, ld, offset
    (1, 4096, BF16, BF16, RMS, True, None, None, 0),
    (3, 4096, BF16, F32, RMS, False, (1, 4096), None, 0),
    (700, 1024, BF16, BF16, RMS, True, (7, 1024), None, 0),
    (37, 1, F32, F32, RMS, True, (37, 1), None, 0),
    (37, 1, F16, F16, LAYER, True, (1, 1), None, 0),
    (65, 7, F16, F32, LAYER, True, (5, 1), None, 0),
    (129, 33, BF16, BF16, LAYER, False, (129, 33), None, 0),
    (1001, 257, F32, F32, LAYER, True, (7, 257), None, 0),
    (330, 1537, F32, F32, LAYER, True, (3, 1537), None, 0),
    (330, 1537, BF16, BF16, RMS, True, (330, 1), None, 0),
    (640, 2048, F16, F16, LAYER, True, (640, 2048), None, 0),
    (61, 2056, F16, F16, RMS, True, (1, 1), None, 0),
    (33, 5120, F32, F32, RMS, True, (11, 5120), None, 0),
    (40, 8192, BF16, F32, LAYER, True, (2, 8192), None, 0),
    (17, 12288, F16, F16, LAYER, True, (1, 12288), None, 0),
    (9, 16384, F32, F32, LAYER, True, (3, 16384), None, 0),
    (9, 16384, BF16, BF16, RMS, True, (9, 1), None, 0),
    (5, 16383, BF16, BF16, LAYER, True, (5, 16383), None, 0),
    (301, 512, BF16, BF16, RMS, True, (43, 512), 640, 0),       # rows of a wider tensor
    (301, 512, BF16, BF16, RMS, True, (43, 512), 641, 0),       # at any element distance
    (50, 768, F32, F32, LAYER, True, None, 768, 1),             # a start off the 16-byte boundary
    (1500, 256, BF16, F32, LAYER, True, (4, 1), None, 0),       # narrow rows: several workers a block
    (2000, 96, F32, F32, RMS, True, (8, 96), None, 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}x{c[1]}")
def test_forward_and_backward(case):
    rows, width, dtype, pdtype, kind, post, gate, ld, offset = case
    v, p = make(rows, width, dtype, pdtype, kind, post, gate, 11 * rows + width, ld, offset)
    scale = 0.75
    plan, params, stats = check_forward(v, p, width, dtype, pdtype, kind, post, scale)
    check_backward(v, p, plan, params, stats, width, pdtype, kind, post, scale)


@pytest.mark.parametrize("span", [1, 2, 5, 63, 126, 315, 630])
@pytest.mark.parametrize("cols", ["width", 1])
def test_gate_rows_that_workers_share(span, cols):
    """Gate rows that end inside, at and beyond a worker's range of rows."""
    rows, width = 630, 640
    v, p = make(rows, width, BF16, F32, RMS, True, (rows // span, width if cols == "width" else 1), span)
    plan, params, stats = check_forward(v, p, width, BF16, F32, RMS, True, 1.0)
    check_backward(v, p, plan, params, stats, width, F32, RMS, True, 1.0)


@pytest.mark.parametrize("dr,dh", [(True, False), (False, True)])
@pytest.mark.parametrize("kind", [RMS, LAYER])
def test_one_gradient_missing(dr, dh, kind):
    v, p = make(70, 384, F32, F32, kind, True, (7, 384), 5)
    plan, params, stats = check_forward(v, p, 384, F32, F32, kind, True, 0.5)
    check_backward(v, p, plan, params, stats, 384, F32, kind, True, 0.5, dr=dr, dh=dh)


@pytest.mark.parametrize("gate", [(1, 384), (7, 384), (70, 384), (7, 1), (70, 1)])
def test_gate_without_its_gradient(gate):
    """dx and dy are the same bits whether or not dgate is asked for."""
    from bit_error_compensated_gb300 import echo
    rows, width = 1400, 384
    gate = (gate[0] * (rows // 70) if gate[0] > 1 else 1, gate[1])
    v, p = make(rows, width, BF16, BF16, RMS, True, gate, 6)
    plan, params, stats = check_forward(v, p, width, BF16, BF16, RMS, True, 1.0)
    got = []
    for dgate in (torch.empty_like(v["gate"]), None):
        dx, dy = torch.empty_like(v["x"]), torch.empty_like(v["x"])
        echo.echo_norm_backward(plan, params, v["x"], v["y"], stats, v["dr"], v["dh"], dx, dy,
                                gate=v["gate"], dgate=dgate)
        got.append((dx, dy))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("rows", [40000, 65000])
def test_gradient_of_a_gate_that_all_rows_share(rows):
    """One scalar gate for every row.  A row's term is exact (16 values of 20
    bits), so what is left is the sum over rows: compensated twice, within a
    worker and over the workers, at most two unit roundoffs of 2^-24 each.  A
    plain running sum is up to 3e-6 to 8e-6 off on these terms."""
    from bit_error_compensated_gb300 import echo
    width, value = 16, 1 + 2 ** -17 + 2 ** -19
    x = torch.zeros(rows, width, device="cuda")
    y, dr = torch.full_like(x, value), torch.ones_like(x)
    gate, dgate = torch.ones(1, 1, device="cuda"), torch.empty(1, 1, device="cuda")
    v = {"x": x, "y": y, "gate": gate}
    p = {"w_pre": torch.ones(width, device="cuda")}
    plan, params, _, _, stats, _, _ = call_forward(v, p, width, F32, F32, RMS, False, 1.0)
    echo.echo_norm_backward(plan, params, x, y, stats, dr, None, torch.empty_like(x),
                            torch.empty_like(x), gate=gate, dgate=dgate)
    exact = rows * width * value
    assert abs(dgate.double().item() - exact) <= 2 ** -22 * exact


@pytest.mark.parametrize("kind,post", list(itertools.product([RMS, LAYER], [True, False])))
def test_gradient_against_differences(kind, post):
    """The derivative along a random direction of every input at once, by
    central differences of the 64-bit forward, against the kernel's gradients."""
    from bit_error_compensated_gb300 import echo
    rows, width, scale = 24, 320, 0.5
    v, p = make(rows, width, F32, F32, kind, post, (6, width), 77)
    plan, params, r, h, stats, _, _ = call_forward(v, p, width, F32, F32, kind, post, scale)
    dx, dy, dgate = torch.empty_like(v["x"]), torch.empty_like(v["x"]), torch.empty_like(v["gate"])
    d = {k: torch.empty_like(t) for k, t in p.items()}
    echo.echo_norm_backward(plan, params, v["x"], v["y"], stats, v["dr"], v["dh"], dx, dy,
                            echo.NormParams(plan, **d), gate=v["gate"], dgate=dgate)
    at = {"x": v["x"], "y": v["y"], "gate": v["gate"], **p}
    got = {"x": dx, "y": dy, "gate": dgate, **d}
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    way = {k: torch.randn(t.shape, generator=gen, device="cuda", dtype=torch.float64) for k, t in at.items()}

    def loss(step):
        q = {k: t.double() + step * way[k] for k, t in at.items()}
        r64, h64, *_ = ref.forward(kind, post, EPS, scale, q["x"], q["y"], q["gate"], q)
        return float((r64 * v["dr"].double()).sum() + (h64 * v["dh"].double()).sum())

    step = 1e-4
    wanted = (loss(step) - loss(-step)) / (2 * step)
    along = sum(float((got[k].double() * way[k]).sum()) for k in at)
    bounds = ref.backward(kind, post, EPS, scale, v["x"].double(), v["y"].double(), v["gate"].double(),
                          {k: t.double() for k, t in p.items()}, v["dr"].double(), v["dh"].double())
    limit = sum(float(((bounds[k][1] + 2.0 ** -24 * bounds[k][0].abs()) * way[k].abs()).sum()) for k in at)
    # the difference errs by step^2 / 6 of the third derivative, here of the
    # size of the terms themselves (unit directions, unit-sized rows)
    terms = sum(float((got[k].double() * way[k]).abs().sum()) for k in at)
    assert abs(along - wanted) <= limit + step * step * terms


def test_no_block_output_and_single_outputs():
    """y None: the model's first norm.  Each output alone gives the same bits."""
    from bit_error_compensated_gb300 import echo
    v, p = make(50, 1024, BF16, BF16, RMS, False, None, 3)
    plan = echo.echo_norm_plan(1024, BF16, eps=EPS, post=True)
    params = echo.NormParams(plan, w_pre=p["w_pre"])
    h, r = torch.empty_like(v["x"]), torch.empty_like(v["x"])
    stats = torch.empty(50, 4, device="cuda")
    echo.echo_norm(plan, params, v["x"], None, r, h, stats=stats)
    want_r, want_h, _, err_r, err_h = ref.forward(RMS, False, EPS, 1.0, dbl(v["x"]), None, None,
                                                  {"w_pre": dbl(p["w_pre"])})
    assert torch.equal(r, v["x"])
    ref.within(h, want_h, err_h, "h")
    dx, dw = torch.empty_like(h), torch.empty_like(p["w_pre"])
    echo.echo_norm_backward(plan, params, v["x"], None, stats, None, v["dh"], dx, None,
                            echo.NormParams(plan, w_pre=dw))
    want = ref.backward(RMS, False, EPS, 1.0, dbl(v["x"]), None, None, {"w_pre": dbl(p["w_pre"])}, None, dbl(v["dh"]))
    ref.within(dx, *want["x"], "dx")
    ref.within(dw, *want["w_pre"], "dw_pre")
    r2, h2 = torch.empty_like(r), torch.empty_like(h)
    echo.echo_norm(plan, params, v["x"], v["y"], r, h)
    echo.echo_norm(plan, params, v["x"], v["y"], r2, None)
    echo.echo_norm(plan, params, v["x"], v["y"], None, h2)
    assert torch.equal(r, r2) and torch.equal(h, h2)


def test_in_place_gives_the_same_bits():
    from bit_error_compensated_gb300 import echo
    v, p = make(211, 2048, BF16, BF16, RMS, True, (1, 2048), 9)
    plan, params, r, h, stats, _, _ = call_forward(v, p, 2048, BF16, BF16, RMS, True, 1.0)
    x2, y2 = v["x"].clone(), v["y"].clone()
    echo.echo_norm(plan, params, x2, y2, x2, y2, gate=v["gate"])
    assert torch.equal(x2, r) and torch.equal(y2, h)
    dx, dy = torch.empty_like(r), torch.empty_like(r)
    echo.echo_norm_backward(plan, params, v["x"], v["y"], stats, v["dr"], v["dh"], dx, dy, gate=v["gate"])
    dr, dh = v["dr"].clone(), v["dh"].clone()
    echo.echo_norm_backward(plan, params, v["x"], v["y"], stats, dr, dh, dr, dh, gate=v["gate"])
    assert torch.equal(dr, dx) and torch.equal(dh, dy)


def test_rows_of_zeros_infinities_and_nans():
    """A zero row gives zeros (1/sqrt(eps) is finite); a row with an infinity or
    a NaN gives what the formula gives and touches no other row."""
    from bit_error_compensated_gb300 import echo
    v, p = make(40, 1024, F32, F32, RMS, True, None, 4)
    clean = call_forward(v, p, 1024, F32, F32, RMS, True, 1.0, codes=True)
    for row, value in ((3, float("inf")), (7, float("nan")), (11, -float("inf"))):
        v["y"][row, 5] = value
        v["x"][row + 1, 900] = value
    v["x"][20], v["y"][20] = 0, 0
    plan, params, r, h, stats, c, s = call_forward(v, p, 1024, F32, F32, RMS, True, 1.0, codes=True)
    odd = torch.zeros(40, dtype=torch.bool, device="cuda")
    odd[[3, 4, 7, 8, 11, 12, 20]] = True
    for a, b in zip(clean[2:], (r, h, stats, c, s)):
        assert torch.equal(a[~odd], b[~odd])
    assert (r[20] == 0).all() and (h[20] == 0).all() and (c[20] == 0).all() and s[20] > 0
    assert r[7].isnan().all() and h[7].isnan().all() and h[8].isnan().all()
    assert r[3, 5].isnan() and (r[3, :5] == v["x"][3, :5]).all()      # inf * 0, and 0 elsewhere
    assert h[4, 900].isnan() and (h[4, :900] == 0).all()
    for row in (3, 4, 7, 8, 11, 12):
        assert (c[row] == 0).all() and not s[row].isfinite()
    dx, dy = torch.empty_like(r), torch.empty_like(r)
    echo.echo_norm_backward(plan, params, v["x"], v["y"], stats, v["dr"], v["dh"], dx, dy)
    assert dx[~odd].isfinite().all() and dy[~odd].isfinite().all()
    assert dx[20].isfinite().all() and dy[20].isfinite().all() and dx[7].isnan().all()


def test_no_rows():
    from bit_error_compensated_gb300 import echo
    plan = echo.echo_norm_plan(256, BF16, F32)
    e = torch.empty(0, 256, dtype=BF16, device="cuda")
    g = torch.ones(1, 256, device="cuda")
    dw, dg = torch.ones(256, device="cuda"), torch.ones(1, 256, device="cuda")
    echo.echo_norm(plan, None, e, e.clone(), e.clone(), e.clone(), gate=g)
    echo.echo_norm_backward(plan, None, e, e.clone(), torch.empty(0, 4, device="cuda"), None, e.clone(),
                            e.clone(), e.clone(), echo.NormParams(plan, w_pre=dw), gate=g, dgate=dg)
    assert (dw == 0).all() and (dg == 0).all()


def test_offsets_past_32_bits():
    """Rows 2^25 elements apart: the last ones start beyond 2^31 elements."""
    rows, width, ld = 70, 512, 1 << 25
    v, p = make(rows, width, BF16, BF16, RMS, True, None, 8)
    plan, params, r, h, stats, _, _ = call_forward(v, p, width, BF16, BF16, RMS, True, 1.0)
    from bit_error_compensated_gb300 import echo
    far = {}
    for k in ("x", "y", "dr", "dh"):
        far[k] = torch.empty(rows * ld, dtype=BF16, device="cuda").view(rows, ld)[:, :width]
        far[k].copy_(v[k])
    r2 = torch.empty(rows * ld, dtype=BF16, device="cuda").view(rows, ld)[:, :width]
    h2, dx2 = r2[:, :], torch.empty_like(r)
    echo.echo_norm(plan, params, far["x"], far["y"], r2, None)
    assert torch.equal(r, r2)
    echo.echo_norm(plan, params, far["x"], far["y"], None, h2)
    assert torch.equal(h, h2)
    dx = torch.empty_like(r)
    echo.echo_norm_backward(plan, params, v["x"], v["y"], stats, v["dr"], v["dh"], dx, None)
    echo.echo_norm_backward(plan, params, far["x"], far["y"], stats, far["dr"], far["dh"], dx2, r2)
    assert torch.equal(dx, dx2)


def test_another_stream_and_a_graph():
    from bit_error_compensated_gb300 import echo
    v, p = make(300, 4096, BF16, BF16, RMS, True, None, 21)
    plan, params, r, h, stats, _, _ = call_forward(v, p, 4096, BF16, BF16, RMS, True, 1.0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    r2, h2 = torch.zeros_like(r), torch.zeros_like(h)
    echo.echo_norm(plan, params, v["x"], v["y"], r2, h2, stream=side)
    side.synchronize()
    assert torch.equal(r, r2) and torch.equal(h, h2)
    dx, dy, dw = torch.empty_like(r), torch.empty_like(r), torch.empty_like(p["w_pre"])
    args = (plan, params, v["x"], v["y"], stats, v["dr"], v["dh"], dx, dy, echo.NormParams(plan, w_pre=dw))
    echo.echo_norm_backward(*args)
    want = [t.clone() for t in (dx, dy, dw)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        echo.echo_norm_backward(*args)
    for t in (dx, dy, dw):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, (dx, dy, dw)):
        assert torch.equal(a, b)


def test_refusals():
    from bit_error_compensated_gb300 import echo
    plan = echo.echo_norm_plan(256, BF16)
    t = lambda: torch.zeros(8, 256, dtype=BF16, device="cuda")                   # noqa: E731
    x, y, r, h = t(), t(), t(), t()

    def status(want, *a, **k):
        with pytest.raises(echo.EchoError) as e:
            echo.echo_norm(plan, None, *a, **k)
        assert e.value.status == want

    both = torch.zeros(9, 256, dtype=BF16, device="cuda")
    status(echo.ECHO_ERR_ARG, both[:8], y, both[1:], h)                  # r one row behind x
    status(echo.ECHO_ERR_ARG, x, y, r, r)
    status(echo.ECHO_ERR_ARG, x, y, y, h)                                # r over y
    status(echo.ECHO_ERR_ARG, x, None, r, h, gate=torch.ones(1, 256, dtype=BF16, device="cuda"))
    status(echo.ECHO_ERR_SHAPE, x.as_strided((8, 256), (128, 1)), y, r, h)
    wide = torch.zeros(8, 512, dtype=BF16, device="cuda")
    echo.echo_norm(plan, None, x, y, wide[:, :256], wide[:, 256:])       # halves of one tensor: fine
    for bad in (dict(kind=2), dict(eps=float("nan")), dict(eps=-1.0), dict(scale=float("inf"))):
        with pytest.raises(echo.EchoError) as e:
            echo.echo_norm_plan(256, BF16, **bad)
        assert e.value.status == echo.ECHO_ERR_ARG
    for width, want in ((0, echo.ECHO_ERR_SHAPE), (16385, echo.ECHO_ERR_UNSUPPORTED)):
        with pytest.raises(echo.EchoError) as e:
            echo.echo_norm_plan(width, BF16)
        assert e.value.status == want
    with pytest.raises(echo.EchoError) as e:
        echo.echo_norm_plan(256, BF16, F16)
    assert e.value.status == echo.ECHO_ERR_UNSUPPORTED
    for word, args, kw in (
            ("dtype", (x.float(), y, r, h), {}), ("shape", (x, y[:7], r, h), {}),
            ("shape", (x[:, :128], y, r, h), {}), ("contiguous", (torch.zeros(8, 512, dtype=BF16, device="cuda")[:, ::2], y, r, h), {}),
            ("gate", (x, y, r, h), dict(gate=torch.ones(3, 256, dtype=BF16, device="cuda"))),
            ("gate", (x, y, r, h), dict(gate=torch.ones(2, 2, dtype=BF16, device="cuda"))),
            ("together", (x, y, r, h), dict(scales=torch.zeros(8, device="cuda"))),
            ("CUDA device", (x.cpu(), y, r, h), {})):
        with pytest.raises(ValueError, match=word):
            echo.echo_norm(plan, None, *args, **kw)
    w = torch.ones(256, dtype=BF16, device="cuda")
    no_post = echo.echo_norm_plan(256, BF16, post=False)
    for pl, names in ((no_post, ("w_post",)), (plan, ("b_pre",)), (plan, ("b_post",))):
        with pytest.raises(echo.EchoError) as e:
            echo.echo_norm(pl, echo.NormParams(pl, **{n: w for n in names}), x, y, r, h)
        assert e.value.status == echo.ECHO_ERR_ARG
    with pytest.raises(ValueError, match="shape"):
        echo.NormParams(plan, w_pre=w[:128])
    stats = torch.zeros(8, 4, device="cuda")
    for kw in (dict(dx=x, dy=None), dict(dx=r, dy=r), dict(dx=None, dy=x)):
        with pytest.raises(echo.EchoError) as e:
            echo.echo_norm_backward(plan, None, x, y, stats, h, h.clone(), **kw)
        assert e.value.status == echo.ECHO_ERR_ARG
    with pytest.raises(echo.EchoError) as e:
        echo.echo_norm_backward(plan, None, x, y, None, h, h.clone(), r, None)
    assert e.value.status == echo.ECHO_ERR_ARG
    with pytest.raises(ValueError, match="dgate"):
        echo.echo_norm_backward(plan, None, x, y, stats, h, h.clone(), r, dgate=torch.ones(1, 256, dtype=BF16, device="cuda"))


@pytest.mark.parametrize("width", [256, 4096, 8192, 8200, 12288, 12289, 16384])
def test_a_variance_that_overflows(width):
    """Finite rows whose variance passes fp32's range have 1/deviation 0: the
    normalised row is 0 and the bias is left, at every width."""
    v, p = make(5, width, F32, F32, LAYER, True, (5, 1), width)
    v["y"].mul_(1e25)
    assert v["y"].isfinite().all()
    plan, params, r, h, stats, _, _ = call_forward(v, p, width, F32, F32, LAYER, True, 0.5)
    assert (stats[:, 1] == 0).all()
    want = v["x"].double() + 0.5 * v["gate"].double() * p["b_post"].double()
    # two products and a sum
    assert ((r.double() - want).abs() <= 3 * 2.0 ** -24 * (v["x"].double().abs() + want.abs())).all()
    assert h.isfinite().all()


def test_parameters_that_were_assigned_anew():
    """A call uses what its parameters hold then, not what they held when they
    were first checked; on another device or of another type they are refused."""
    from bit_error_compensated_gb300 import echo
    v, p = make(20, 512, BF16, F32, RMS, True, None, 12)
    plan, params, r, h, *_ = call_forward(v, p, 512, BF16, F32, RMS, True, 1.0)
    old = p["w_pre"].detach()
    p["w_pre"].data = 2 * old
    h2 = torch.empty_like(h)
    echo.echo_norm(plan, params, v["x"], v["y"], None, h2)
    assert torch.equal(h2, 2 * h)                       # twice the weight: an exact factor
    for other, word in ((old.cpu(), "CUDA device"), (old.bfloat16(), "dtype")):
        p["w_pre"].data = other
        with pytest.raises(ValueError, match=word):
            echo.echo_norm(plan, params, v["x"], v["y"], None, h2)
    p["w_pre"].data = old
    echo.echo_norm(plan, params, v["x"], v["y"], None, h2)
    assert torch.equal(h2, h)


@pytest.mark.parametrize("width", [1, 96, 1024, 4096, 4097, 8192, 12288, 16384])
def test_a_plan_allocates_what_its_calls_can_use(width):
    """Six fp32 sums for each of the columns that the device's threads hold at
    once: 512 threads an SM, 16 columns each (and the allocator's 2 MB)."""
    from bit_error_compensated_gb300 import echo
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    plans = [echo.echo_norm_plan(width, BF16) for _ in range(4)]
    used = (before - torch.cuda.mem_get_info()[0]) / len(plans)
    assert used <= 6 * 4 * sms * 512 * 16 + (1 << 21)


@pytest.mark.parametrize("width", [4104, 5120, 8000, 8192])
@pytest.mark.parametrize("dtype,kind,post,gate", [
    (F32, LAYER, True, None), (F32, LAYER, True, "token"), (F32, LAYER, False, None), (F32, RMS, True, "sequence"),
    (BF16, LAYER, True, "sequence"), (F16, LAYER, False, "sequence"), (BF16, RMS, False, "sequence"),
    (F32, RMS, False, "sequence"), (BF16, LAYER, True, None), (F16, RMS, True, "sequence")])
def test_rows_of_two_blocks(width, dtype, kind, post, gate):
    """Aligned rows past 4096 columns, which one block or a cluster of two takes."""
    rows = 333
    gate = {None: None, "token": (rows, 1), "sequence": (9, width)}[gate]
    v, p = make(rows, width, dtype, F32, kind, post, gate, width)
    plan, params, stats = check_forward(v, p, width, dtype, F32, kind, post, 0.5)
    check_backward(v, p, plan, params, stats, width, F32, kind, post, 0.5)


# Rows enough that every block (and every worker of the backward call) goes
# several times round its ring of rows, with a ragged last turn.  On 152 SMs a
# forward block of 4096 columns takes 9 or 10 rows (16 elements a thread) or 18
# to 19, and its ring holds 4 at most; a worker 10 or 19.
MANY = 2744


def check_many_rows(rows):
    """That there are as many: an SM holds two rows of 4096 columns at most."""
    assert rows >= 9 * 2 * torch.cuda.get_device_properties(0).multi_processor_count


def gate_of(name, rows, width):
    return {"none": None, "all": (1, width), "sequence": (rows // 49, width), "scalar": (1, 1), "token": (rows, 1)}[name]


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("gate", ["none", "all", "sequence", "token"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("kind", [RMS, LAYER])
@pytest.mark.parametrize("dtype,width", [(BF16, 4096), (F16, 4096), (F32, 4096), (BF16, 4095), (F32, 4095), (BF16, 8192)])
def test_forward_many_rows_a_block(dtype, width, kind, post, gate, codes):
    """Distinct rows through every slot of the ring, many times; without codes
    this is the form that training and prefill take."""
    check_many_rows(MANY)
    v, p = make(MANY, width, dtype, F32, kind, post, gate_of(gate, MANY, width), width + post)
    if codes:
        check_forward(v, p, width, dtype, F32, kind, post, 0.5)
        return
    _, _, r, h, stats, _, _ = call_forward(v, p, width, dtype, F32, kind, post, 0.5)
    want_r, want_h, want_stats, err_r, err_h = ref.forward(
        kind, post, EPS, 0.5, dbl(v["x"]), dbl(v["y"]), dbl(v["gate"]), {k: t.double() for k, t in p.items()})
    ref.within(r, want_r, err_r, "r")
    ref.within(h, want_h, err_h, "h")


@pytest.mark.parametrize("rows,width,dtype,kind", [(700, 12288, BF16, RMS), (700, 9001, F32, LAYER),
                                                   (700, 16384, F16, LAYER), (460, 10000, F32, RMS)])
def test_forward_many_wide_rows_a_block(rows, width, dtype, kind):
    v, p = make(rows, width, dtype, F32, kind, True, (rows // 20, width), width)
    check_forward(v, p, width, dtype, F32, kind, True, 0.5)


@pytest.mark.parametrize("width", [4096, 4095, 1001])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", [RMS, LAYER])
def test_in_place_many_rows(dtype, width, kind):
    """Every tensor that may be written in place, the rows ahead of it in flight."""
    from bit_error_compensated_gb300 import echo
    check_many_rows(MANY)
    v, p = make(MANY, width, dtype, F32, kind, True, (56, width), 3 + width)
    plan, params, r, h, stats, _, _ = call_forward(v, p, width, dtype, F32, kind, True, 1.0)
    x2, y2 = v["x"].clone(), v["y"].clone()
    echo.echo_norm(plan, params, x2, y2, x2, y2, gate=v["gate"])
    assert torch.equal(x2, r) and torch.equal(y2, h)
    dx, dy = torch.empty_like(r), torch.empty_like(r)
    echo.echo_norm_backward(plan, params, v["x"], v["y"], stats, v["dr"], v["dh"], dx, dy, gate=v["gate"])
    for to_dx, to_dy in (("dr", "dh"), ("dh", "dr"), ("dr", "y"), ("dh", "y"), (None, "dr"), ("dr", None)):
        t = {k: v[k].clone() for k in ("dr", "dh", "y")}
        dx2 = t[to_dx] if to_dx else torch.empty_like(r)
        dy2 = t[to_dy] if to_dy else torch.empty_like(r)
        echo.echo_norm_backward(plan, params, v["x"], t["y"], stats, t["dr"], t["dh"], dx2, dy2, gate=v["gate"])
        assert torch.equal(dx2, dx) and torch.equal(dy2, dy), (to_dx, to_dy)


def check_gradients(v, p, plan, params, stats, width, kind, post, scale, full=True):
    """All gradients, the gate's too, twice the same bits and within their
    bounds; not `full`: without that of x."""
    from bit_error_compensated_gb300 import echo
    got = {"x": like(v["x"]) if full else None, "y": like(v["x"])}
    d = {k: torch.full_like(t, float("nan")) for k, t in p.items()}
    got["gate"] = None if v["gate"] is None else torch.full_like(v["gate"], float("nan"))
    grads, first = echo.NormParams(plan, **d), None
    got.update(d)
    got = {k: t for k, t in got.items() if t is not None}
    for _ in range(2):
        echo.echo_norm_backward(plan, params, v["x"], v["y"], stats, v["dr"], v["dh"], got.get("x"), got["y"], grads,
                                gate=v["gate"], dgate=got.get("gate"))
        if first is None:
            first = {k: t.clone() for k, t in got.items()}
            for t in d.values():
                t.fill_(float("nan"))
            if "gate" in got:
                got["gate"].fill_(float("nan"))
    for k, t in got.items():
        assert torch.equal(first[k], t), f"d{k}: a repeated call gives other bits"
    want = ref.backward(kind, post, EPS, scale, dbl(v["x"]), dbl(v["y"]), dbl(v["gate"]),
                        {k: t.double() for k, t in p.items()}, dbl(v["dr"]), dbl(v["dh"]))
    for k, t in got.items():
        ref.within(t, *want[k], f"d{k}")


@pytest.mark.parametrize("full", [True, False])
@pytest.mark.parametrize("gate", ["none", "all", "sequence", "scalar", "token"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("kind", [RMS, LAYER])
@pytest.mark.parametrize("dtype,width", [(BF16, 4096), (F32, 4096), (F16, 4095), (F32, 4095)])
def test_backward_many_rows_a_worker(dtype, width, kind, post, gate, full):
    """Distinct rows many times round a worker's ring."""
    check_many_rows(MANY)
    v, p = make(MANY, width, dtype, F32, kind, post, gate_of(gate, MANY, width), width + 7)
    plan, params, _, _, stats, _, _ = call_forward(v, p, width, dtype, F32, kind, post, 0.5)
    check_gradients(v, p, plan, params, stats, width, kind, post, 0.5, full)


@pytest.mark.parametrize("rows,span", [(2744, 1), (2744, 7), (2744, 8), (2744, 14), (2744, 49), (2744, 343), (2744, 1372),
                                       (2740, 5), (2740, 10), (2740, 20), (2755, 19), (2755, 95), (2744, 2744)])
@pytest.mark.parametrize("cols", ["width", 1])
@pytest.mark.parametrize("kind", [RMS, LAYER])
@pytest.mark.parametrize("dtype,width", [(BF16, 4096), (F32, 4096), (F32, 4095)])
def test_gate_rows_across_workers_of_many_rows(dtype, width, kind, cols, rows, span):
    """Gate rows that begin and end inside a worker's rows (10 with 16 elements a
    thread, 19 with 8), at their ends, and that many workers share."""
    check_many_rows(rows)
    v, p = make(rows, width, dtype, F32, kind, True, (rows // span, width if cols == "width" else 1), span)
    plan, params, _, _, stats, _, _ = call_forward(v, p, width, dtype, F32, kind, True, 1.0)
    check_gradients(v, p, plan, params, stats, width, kind, True, 1.0)
